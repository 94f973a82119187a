// Attention over the int8 K/V cache for few query rows (single tokens), and
// the merge of partial rows over key splits.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j - max),
//   k_j = kq_j ks_j, v_j = vq_j vs_j  (8-bit codes, one scale per key)
//
// One pass over the keys with the running maximum and sum of a softmax.  The
// codes enter the products as bf16 integers, which is exact; the key's scale
// multiplies its score afterwards, the value's scale its probability (rounded
// once to bf16, as an attention with bf16 values rounds its probabilities).
//
// Bound: bytes of the cache (2 (d + 4) per key and KV head).  The G query
// heads of a KV head share every byte, 8 rows at a time as the N side of
// mma.sync m16n8k16 (keys, then value channels, on the M side): a warp turns
// the 16 bytes that a lane loads straight into A fragments in registers, with
// no trip through shared memory (a 128-row tensor-core tile would be 94 %
// padding here and its operands would have to be staged).  The contraction
// index may be permuted freely, so fragments are cut from contiguous 16-byte
// loads:
//   K: lane (g, t) = (lane / 4, lane % 4) loads 16 channels [64 j + 16 t, +16)
//      of keys g and g + 8; step s of block j takes bytes 4 s .. 4 s + 3
//   V: lane (g, t) loads 16 channels [128 h + 16 g, +16) of keys 2t, 2t + 1,
//      2t + 8, 2t + 9; product m of block h takes channels 2 m (row g) and
//      2 m + 1 (row g + 8)
// Each warp of the block takes every W-th group of 16 keys with statistics of
// its own; the warps meet once at the end.  Long caches and small batches
// split the keys over blocks (partials in fp32, merged by k_kv8_merge).
#include <algorithm>
#include <cmath>

#include "int8.h"
#include "launch.cuh"

namespace pae {

namespace {

constexpr int kWarps = 4;
constexpr int kTileKeys = 16;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit elements across the warp
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two signed bytes in bits 0-7 and 16-23 of w (the other bits are ignored) ->
// bf16x2, exactly: with v the low 7 bits and s the sign bit, 0x4300 | v is
// 128 + v and 0x4300 | s << 7 is 128 (1 + s); their difference is v - 128 s.
__device__ __forceinline__ uint32_t bytes_bf16x2(uint32_t w) {
  const uint32_t a = (w & 0x007F007Fu) | 0x43004300u;
  const uint32_t b = (w & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)__bfloat16_as_ushort(f2bf(lo)) | ((uint32_t)__bfloat16_as_ushort(f2bf(hi)) << 16);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, D == 256 ? 2 : 4) k_kv8_attn_few(const Kv8AttnArgs a) {
  constexpr int KBLK = D / 64;               // 64-channel blocks of a K row
  constexpr int VB = D >= 128 ? 16 : 8;      // bytes of a V row per lane and block
  constexpr int VBLK = D / (8 * VB);         // blocks of a V row
  constexpr int VM = VB / 2;                 // products per block
  extern __shared__ float s_o[];             // [kWarps][8][D + 4]
  __shared__ float s_m[kWarps][8], s_l[kWarps][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, splits = gridDim.x, rg = blockIdx.y, bg = blockIdx.z;
  const int b = bg / a.c.heads, h = bg - b * a.c.heads;
  const int rows = a.group * a.n_q;
  pdl_launch_dependents();
  pdl_wait();

  const int len = max(0, min(a.lens[b], a.c.cap));
  // this block's keys: an equal share of those any of its rows can see, in
  // whole groups of kWarps tiles
  constexpr int STEP = kWarps * kTileKeys;
  const int share = (int)((((long long)len + splits - 1) / splits + STEP - 1) / STEP) * STEP;
  const long long k_lo = (long long)split * share;
  const int key0 = (int)min((long long)len, k_lo), key1 = (int)min((long long)len, k_lo + share);

  // Q: row r = query * group + head-in-group; lane (g, t) holds channels
  // [64 j + 16 t, +16) of row 8 rg + g
  uint32_t qf[KBLK][8];
  {
    const int r = rg * 8 + g;
    const bool live = r < rows;
    const int qi = live ? r / a.group : 0, hl = live ? r - qi * a.group : 0;
    const bf16* qp = a.q + b * a.q_seq + qi * a.q_tok + (long long)(h * a.group + hl) * a.q_head;
#pragma unroll
    for (int j = 0; j < KBLK; ++j) {
      uint4 x = make_uint4(0, 0, 0, 0), y = x;
      if (live) {
        x = *reinterpret_cast<const uint4*>(qp + 64 * j + 16 * t);
        y = *reinterpret_cast<const uint4*>(qp + 64 * j + 16 * t + 8);
      }
      qf[j][0] = x.x; qf[j][1] = x.y; qf[j][2] = x.z; qf[j][3] = x.w;
      qf[j][4] = y.x; qf[j][5] = y.y; qf[j][6] = y.z; qf[j][7] = y.w;
    }
  }
  // first key that rows 2t and 2t + 1 of the group cannot see
  int lim[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = rg * 8 + 2 * t + i;
    lim[i] = a.causal && r < rows ? min(len, len - a.n_q + 1 + r / a.group) : len;
  }

  const size_t base = ((size_t)b * a.c.heads + h) * a.c.cap;
  const int8_t* kb = a.c.k + base * D;
  const int8_t* vb = a.c.v + base * D;
  const float* ksb = a.c.k_scale + base;
  const float* vsb = a.c.v_scale + base;

  float o[VBLK][VM][4];
#pragma unroll
  for (int i = 0; i < VBLK; ++i)
#pragma unroll
    for (int m = 0; m < VM; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][m][j] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};

  uint4 kr[2][KBLK];          // keys g, g + 8
  uint32_t vr[4][VBLK][VB / 4];  // keys 2t, 2t + 1, 2t + 8, 2t + 9
  float ks[2], vs[2];
  auto load_k = [&](int at) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = min(at + g + 8 * i, key1 - 1);  // past the range: a key of it, masked below
      ks[i] = __ldg(ksb + key);
      vs[i] = __ldg(vsb + key);
#pragma unroll
      for (int j = 0; j < KBLK; ++j)
        kr[i][j] = __ldg(reinterpret_cast<const uint4*>(kb + (size_t)key * D + 64 * j + 16 * t));
    }
  };
  auto load_v = [&](int at) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = min(at + 2 * t + (i & 1) + (i >> 1) * 8, key1 - 1);
#pragma unroll
      for (int j = 0; j < VBLK; ++j) {
        const int8_t* p = vb + (size_t)key * D + (8 * VB) * j + VB * g;
        if constexpr (VB == 16) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
          vr[i][j][0] = x.x; vr[i][j][1] = x.y; vr[i][j][2] = x.z; vr[i][j][3] = x.w;
        } else {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
          vr[i][j][0] = x.x; vr[i][j][1] = x.y;
        }
      }
    }
  };

  int at = key0 + warp * kTileKeys;
  if (at < key1) {
    load_k(at);
    load_v(at);
  }
  for (; at < key1; at += STEP) {
    // scores of 16 keys x 8 rows: lane holds keys g, g + 8, rows 2t, 2t + 1
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < KBLK; ++j) {
      const uint32_t w0[4] = {kr[0][j].x, kr[0][j].y, kr[0][j].z, kr[0][j].w};
      const uint32_t w1[4] = {kr[1][j].x, kr[1][j].y, kr[1][j].z, kr[1][j].w};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t f[4] = {bytes_bf16x2(__byte_perm(w0[s], 0, 0x4140)), bytes_bf16x2(__byte_perm(w1[s], 0, 0x4140)),
                               bytes_bf16x2(__byte_perm(w0[s], 0, 0x4342)), bytes_bf16x2(__byte_perm(w1[s], 0, 0x4342))};
        mma_bf16(c, f, qf[j][2 * s], qf[j][2 * s + 1]);
      }
    }
    const float k0 = ks[0] * a.scale_log2, k1 = ks[1] * a.scale_log2;
    const float v0 = vs[0], v1 = vs[1];
    if (at + STEP < key1) load_k(at + STEP);  // the next tile's keys under this one's softmax
    const int ka = at + g, kc = ka + 8;
    float x[4];
    x[0] = ka < min(lim[0], key1) ? c[0] * k0 : -INFINITY;
    x[1] = ka < min(lim[1], key1) ? c[1] * k0 : -INFINITY;
    x[2] = kc < min(lim[0], key1) ? c[2] * k1 : -INFINITY;
    x[3] = kc < min(lim[1], key1) ? c[3] * k1 : -INFINITY;
    float al[2];
    bool grow = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = fmaxf(x[i], x[i + 2]);
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
      // the reference moves only when the maximum grows by more than 8 (a
      // factor 256): probabilities stay below 256 and O is rescaled rarely
      const bool up = mx > m_run[i] + 8.f || m_run[i] == -INFINITY;
      const float nm = up ? fmaxf(mx, m_run[i]) : m_run[i];
      al[i] = nm == -INFINITY ? 1.f : ex2(m_run[i] - nm);
      grow |= al[i] != 1.f;
      m_run[i] = nm;
    }
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = x[i] == -INFINITY ? 0.f : ex2(x[i] - m_run[i & 1]);
    l_run[0] = l_run[0] * al[0] + (p[0] + p[2]);
    l_run[1] = l_run[1] * al[1] + (p[1] + p[3]);
    if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
      for (int i = 0; i < VBLK; ++i)
#pragma unroll
        for (int m = 0; m < VM; ++m) {
          o[i][m][0] *= al[0];
          o[i][m][1] *= al[1];
          o[i][m][2] *= al[0];
          o[i][m][3] *= al[1];
        }
    }
    // P times the value scales; masked places stay 0 whatever their scale is
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = x[i] == -INFINITY ? 0.f : p[i] * (i < 2 ? v0 : v1);
    const uint32_t b0 = movmatrix(pack_bf16(p[0], p[1])), b1 = movmatrix(pack_bf16(p[2], p[3]));
#pragma unroll
    for (int j = 0; j < VBLK; ++j)
#pragma unroll
      for (int m = 0; m < VM; ++m) {
        const int w = m >> 1;
        const uint32_t lo = (m & 1) ? 0x0602u : 0x0400u, hi = (m & 1) ? 0x0703u : 0x0501u;
        const uint32_t f[4] = {bytes_bf16x2(__byte_perm(vr[0][j][w], vr[1][j][w], lo)),
                               bytes_bf16x2(__byte_perm(vr[0][j][w], vr[1][j][w], hi)),
                               bytes_bf16x2(__byte_perm(vr[2][j][w], vr[3][j][w], lo)),
                               bytes_bf16x2(__byte_perm(vr[2][j][w], vr[3][j][w], hi))};
        mma_bf16(o[j][m], f, b0, b1);
      }
    if (at + STEP < key1) load_v(at + STEP);
  }

  // row sums over the 8 lanes that share t
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float l = l_run[i];
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
    // NaN scores alone leave the maximum at -inf: the row is not empty
    if (m_run[i] == -INFINITY && l != 0.f) m_run[i] = 0.f;
    if (g == 0) {
      s_m[warp][2 * t + i] = m_run[i];
      s_l[warp][2 * t + i] = l;
    }
  }
  __syncthreads();
  // the warps' rows in units of the block's maximum
  constexpr int LD = D + 4;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 2 * t + i;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
    const float f = m_run[i] == -INFINITY ? 0.f : ex2(m_run[i] - M);
    float* dst = s_o + (warp * 8 + r) * LD;
#pragma unroll
    for (int j = 0; j < VBLK; ++j)
#pragma unroll
      for (int m = 0; m < VM; m += 2)
        *reinterpret_cast<float4*>(dst + (8 * VB) * j + VB * g + 2 * m) =
            make_float4(o[j][m][i] * f, o[j][m][2 + i] * f, o[j][m + 1][i] * f, o[j][m + 1][2 + i] * f);
  }
  __syncthreads();
  const int rowsp = gridDim.y * 8;
  for (int e = threadIdx.x; e < 8 * (D / 4); e += kWarps * 32) {
    const int r = e / (D / 4), c4 = e - r * (D / 4);
    float M = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) l += s_m[w][r] == -INFINITY ? 0.f : s_l[w][r] * ex2(s_m[w][r] - M);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(s_o + (w * 8 + r) * LD + 4 * c4);
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
    const int row = rg * 8 + r;
    if (splits == 1) {
      if (row < rows) {
        const int qi = row / a.group, hl = row - qi * a.group;
        const float inv = l == 0.f ? 0.f : 1.f / l;  // no visible key: zeros
        bf16* op = a.o + b * a.o_seq + qi * a.o_tok + (long long)(h * a.group + hl) * a.o_head + 4 * c4;
        *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      }
    } else {
      const size_t pr = ((size_t)bg * splits + split) * rowsp + row;
      if (M != -INFINITY) *reinterpret_cast<float4*>(a.part_o + pr * D + 4 * c4) = acc;
      if (c4 == 0) a.part_ml[pr] = make_float2(M, l);
    }
  }
}

// o = sum_s w_s O_s / sum_s w_s l_s with w_s = 2^(m_s - max m): one block per
// (sequence, KV head, row).  Splits without a visible key (m = -inf) wrote no
// row and are passed over.
template <int D>
__global__ void __launch_bounds__(256) k_kv8_merge(const Kv8AttnArgs a, int splits, int rowsp) {
  constexpr int C4 = D / 4, NS = 256 / C4;
  __shared__ float s_w[kMaxKv8Splits];
  __shared__ float s_red[8];
  __shared__ float4 s_acc[256];
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x, bg = blockIdx.y;
  const int b = bg / a.c.heads, h = bg - b * a.c.heads;
  const size_t p0 = (size_t)bg * splits * rowsp + row;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float2 ml = make_float2(-INFINITY, 0.f);
  if (tid < splits) ml = __ldcg(a.part_ml + p0 + (size_t)tid * rowsp);
  float M = warp_max(ml.x);
  if (lane == 0) s_red[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) M = fmaxf(M, s_red[w]);
  const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
  if (tid < splits) s_w[tid] = w;
  const float l = block_sum(ml.x == -INFINITY ? 0.f : w * ml.y, s_red);  // (its barriers also order s_w)
  const int c4 = tid % C4, part = tid / C4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = part; s < splits; s += NS) {
    const float ws = s_w[s];
    if (ws == 0.f) continue;
    const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part_o + (p0 + (size_t)s * rowsp) * D + 4 * c4));
    acc.x = fmaf(ws, x.x, acc.x);
    acc.y = fmaf(ws, x.y, acc.y);
    acc.z = fmaf(ws, x.z, acc.z);
    acc.w = fmaf(ws, x.w, acc.w);
  }
  s_acc[tid] = acc;
  __syncthreads();
  if (part == 0) {
#pragma unroll
    for (int s = 1; s < NS; ++s) {
      const float4 x = s_acc[s * C4 + c4];
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
    const int qi = row / a.group, hl = row - qi * a.group;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    bf16* op = a.o + b * a.o_seq + qi * a.o_tok + (long long)(h * a.group + hl) * a.o_head + 4 * c4;
    *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  }
}

size_t few_smem(int d) { return (size_t)kWarps * 8 * (d + 4) * 4; }

template <int D>
cudaError_t few_launch(const Kv8AttnPlan& p, const Kv8AttnArgs& a, bool pdl, cudaStream_t st) {
  return launch_ex(k_kv8_attn_few<D>, dim3(p.splits, p.qtiles, a.n_seq * a.c.heads), dim3(kWarps * 32), few_smem(D), st,
                   1, pdl, a);
}
template <int D>
cudaError_t merge_launch(const Kv8AttnPlan& p, const Kv8AttnArgs& a, cudaStream_t st) {  // (PDL behind its own attention)
  return launch_ex(k_kv8_merge<D>, dim3(a.group * a.n_q, a.n_seq * a.c.heads), dim3(256), 0, st, 1, true, a, p.splits,
                   p.qtiles * (p.tc ? 128 : 8));
}

}  // namespace

// Rows of a KV head (query heads in its group x queries): up to 16 take groups
// of 8 rows on mma.sync, more (or any fresh keys) tiles of 128 rows on the
// tcgen05 tensor cores.  Keys are split until the blocks fill the SMs, each
// split keeping at least 128 keys of the largest cache.
Kv8AttnPlan plan_kv8_attn(int n_seq, int heads_kv, int group, int n_q, int n_new, int max_keys, int d) {
  Kv8AttnPlan p{};
  const long long rows = (long long)group * n_q;
  p.tc = rows > 16 || n_new > 0;
  const int tile = p.tc ? 128 : 8;
  p.qtiles = (int)((rows + tile - 1) / tile);
  const long long blocks = (long long)n_seq * heads_kv * p.qtiles;
  const int keys = std::max(1, max_keys + n_new);
  int splits = 1;
  if (p.tc) {
    while (splits < 8 && blocks * splits * 2 <= 148 && keys / (splits * 2) >= 64) splits *= 2;
  } else {
    // several waves of blocks even out sequences of different length
    const long long want = (4 * 148 + blocks - 1) / blocks;
    splits = (int)std::max<long long>(1, std::min<long long>({want, (long long)kMaxKv8Splits, keys / 128}));
    if (blocks * splits < 148) splits = (int)std::max<long long>(1, std::min<long long>(keys / 128, 148 / blocks));
    splits = std::min(splits, kMaxKv8Splits);
  }
  p.splits = splits;
  p.ws_bytes = splits > 1 ? (size_t)blocks * splits * tile * ((size_t)d * 4 + 8) : 0;
  return p;
}

cudaError_t kv8_attn_init() {
  cudaError_t e = cudaFuncSetAttribute(k_kv8_attn_few<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)few_smem(256));
  return e == cudaSuccess ? kv8_attn_tc_init() : e;
}

cudaError_t launch_kv8_attn(const Kv8AttnPlan& p, const Kv8AttnArgs& a, bool pdl, cudaStream_t st) {
  cudaError_t e;
  if (p.tc)
    e = launch_kv8_attn_tc(p, a, pdl, st);
  else if (a.c.d == 64)
    e = few_launch<64>(p, a, pdl, st);
  else if (a.c.d == 128)
    e = few_launch<128>(p, a, pdl, st);
  else
    e = few_launch<256>(p, a, pdl, st);
  if (e != cudaSuccess || p.splits == 1) return e;
  if (a.c.d == 64) return merge_launch<64>(p, a, st);
  if (a.c.d == 128) return merge_launch<128>(p, a, st);
  return merge_launch<256>(p, a, st);
}

}  // namespace pae
