// Attention over the int8 K/V cache, and fresh bf16 keys behind it, for many
// query rows: the denoise loop's chunk of action tokens, or a causal prompt.
//
// Mathematics as in k_i8_attn.cu.  The query heads that share a KV head times
// the queries (row = query * group + head-in-group, so that a tile spans few
// queries and a causal tile skips the keys behind its last one) are cut into
// tiles of 128 rows, the M dimension of tcgen05.mma.  Per chunk of 64 keys:
//   converters (8 warps)  read the codes (16-byte loads, the next chunk's in
//                         flight while this one is written), turn them into
//                         bf16 integers (exact) in the 128-byte swizzled tiles
//                         the MMA reads, and put the keys' scales beside them;
//                         fresh keys and values are copied as they are, scale 1
//   MMA thread            S = Q K^T (128 x 64, double-buffered in TMEM), then
//                         O += P V (P read from TMEM, V read MN-major)
//   softmax (8 warps)     two threads per row: scores x key scale, online
//                         softmax in the log2 domain (O is rescaled only when
//                         the maximum grows by more than 2^8), P x value scale
//                         as bf16 over S's own columns
// Bound: the softmax and conversion work per tile, between the tensor cores'
// and the cache's floors (K and V of a sequence are converted once per tile).
// Key splits (small batches) write unnormalised fp32 rows with their maximum
// and sum to the workspace; k_kv8_merge joins them.
#include "int8.h"
#include "launch.cuh"

namespace pae {

namespace {

constexpr int QROWS = 128, CK = 64;
constexpr int kSmx = 256;                  // softmax threads (warps 0-7)
constexpr int kConv = 128;                 // converter threads per operand
constexpr int kThreads = kSmx + 32 + 2 * kConv;
constexpr long long kDrainNs = 4000000000LL;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)__bfloat16_as_ushort(f2bf(lo)) | ((uint32_t)__bfloat16_as_ushort(f2bf(hi)) << 16);
}
// Two signed bytes in bits 0-7 and 16-23 -> bf16x2, exactly (see k_i8_attn.cu).
__device__ __forceinline__ uint32_t bytes_bf16x2(uint32_t w) {
  const uint32_t a = (w & 0x007F007Fu) | 0x43004300u;
  const uint32_t b = (w & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// AND over the 64 threads of the two warps that share 32 rows.
__device__ __forceinline__ bool pair_and(int id, bool v) {
  __syncwarp();
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

template <int D>
struct Smem {
  static constexpr uint32_t kTile = CK * D * 2;  // one chunk of K (or V) in bf16
  static constexpr uint32_t q = 0, k = QROWS * D * 2, v = k + 2 * kTile, sc = v + 2 * kTile;
  static constexpr uint32_t pm = sc + 2 * 2 * CK * 4;    // scales: 2 chunks of [ks 64 | vs 64]
  static constexpr uint32_t l = pm + 2 * 2 * QROWS * 4;  // partial maxima [2][2][128]
  static constexpr uint32_t bar = l + 2 * QROWS * 4;     // partial sums [2][128]
  static constexpr uint32_t total = bar + 256 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_kv8_attn_tc(const Kv8AttnArgs a) {
  constexpr int NBOX = D / 64;
  using L = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::bar);
  uint64_t* q_full = bars;          // Q tile written
  uint64_t* k_full = bars + 1;      // [2] K tile written
  uint64_t* v_full = bars + 3;      // [2]
  uint64_t* k_empty = bars + 5;     // [2] S of the slot's chunk done
  uint64_t* v_empty = bars + 7;     // [2] PV of the slot's chunk done
  uint64_t* s_full = bars + 9;      // [2] S computed
  uint64_t* p_full = bars + 11;     // [2] P written over S
  uint64_t* o_done = bars + 13;     // [2] PV of the buffer's chunk done
  uint64_t* drain = bars + 15;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 16);
  volatile int* s_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* s_sc = reinterpret_cast<float*>(smem + L::sc);
  float* s_pm = reinterpret_cast<float*>(smem + L::pm);
  float* s_l = reinterpret_cast<float*>(smem + L::l);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qt = blockIdx.x, split = blockIdx.y, splits = gridDim.y, bg = blockIdx.z;
  const int b = bg / a.c.heads, h = bg - b * a.c.heads;
  const int rows = a.group * a.n_q;
  constexpr uint32_t ncols = 2 * CK + D <= 256 ? 256 : 512;

  if (threadIdx.x == 0) {
    mbar_init(q_full, kSmx);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], kConv);
      mbar_init(&v_full[i], kConv);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kSmx);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(drain, 1);
    s_flag[0] = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, ncols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t t_o = tmem + 2 * CK;

  // chunks of this CTA: an equal share of the cached chunks its rows can see
  // followed by the fresh ones
  const int len = max(0, min(a.lens[b], a.c.cap));
  const int r_last = min(rows, qt * QROWS + QROWS) - 1;
  const int seen = a.causal ? max(0, min(len, len - a.n_q + 1 + r_last / a.group)) : len;
  const int nc = (seen + CK - 1) / CK, nf = (a.n_new + CK - 1) / CK;
  const int c0 = (int)((long long)(nc + nf) * split / splits), c1 = (int)((long long)(nc + nf) * (split + 1) / splits);
  const int nch = c1 - c0;

  if (warp >= 9) {
    // ------------------------------------------------------------ converters
    // A warp's 16-byte pieces cover 8 rows x 64 channels: lane = 4 row + piece.
    // Rows of different parity land in different halves of the swizzled 128-byte
    // rows, so the two 16-byte stores of 8 lanes touch all banks once.
    const bool is_v = warp >= 13;
    const int cw = (warp - 9) & 3;                       // warp within the operand's four
    const int cp = lane & 3, rl = lane >> 2;
    constexpr int UNITS = NBOX * 8 / 4;                  // (box, 8 rows) units per warp
    const size_t base = ((size_t)b * a.c.heads + h) * a.c.cap;
    const int8_t* src = (is_v ? a.c.v : a.c.k) + base * D;
    const float* ksc = a.c.k_scale + base;
    const float* vsc = a.c.v_scale + base;
    const bf16* fresh = is_v ? a.v_new : a.k_new;
    const long long f_tok = is_v ? a.vn_tok : a.kn_tok;
    if (fresh) fresh += b * (is_v ? a.vn_seq : a.kn_seq) + (long long)h * (is_v ? a.vn_head : a.kn_head);
    uint64_t* full = is_v ? v_full : k_full;
    uint64_t* empty = is_v ? v_empty : k_empty;
    const uint32_t tile0 = smem_u32(smem + (is_v ? L::v : L::k));
    const int ct = cw * 32 + lane;
    uint4 raw[UNITS];
    float sc = 0.f;  // V converters: thread j < 64 carries key j's K scale, 64 + j its V scale
    auto load = [&](int c) {  // a cached chunk's codes and scales
      const int key0 = c * CK;
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int unit = cw * UNITS + u, box = unit >> 3, row = (unit & 7) * 8 + rl;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (key0 + row < seen) raw[u] = __ldg(reinterpret_cast<const uint4*>(src + (size_t)(key0 + row) * D + box * 64 + cp * 16));
      }
      if (is_v) {
        const int key = key0 + (ct & (CK - 1));
        sc = key < seen ? (ct < CK ? __ldg(ksc + key) * a.scale_log2 : __ldg(vsc + key)) : 0.f;
      }
    };
    if (nch > 0 && c0 < nc) load(c0);
    for (int i = 0; i < nch; ++i) {
      const int c = c0 + i, slot = i & 1;
      if (i >= 2 && !mbar_wait(&empty[slot], ((i >> 1) & 1) ^ 1, a.err.wait_ns)) {
        s_flag[0] = 1;
        set_error(a.err, DEV_TIMEOUT);
        break;
      }
      const uint32_t tile = tile0 + (uint32_t)slot * L::kTile;
      if (c < nc) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const int unit = cw * UNITS + u, box = unit >> 3, row = (unit & 7) * 8 + rl;
          const uint32_t at = tile + (uint32_t)(box * CK * 128 + row * 128);
          const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
          uint32_t o[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            o[2 * q] = bytes_bf16x2(__byte_perm(w[q], 0, 0x4140));
            o[2 * q + 1] = bytes_bf16x2(__byte_perm(w[q], 0, 0x4342));
          }
          sts128(at + (uint32_t)(((2 * cp) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
          sts128(at + (uint32_t)(((2 * cp + 1) ^ (row & 7)) << 4), o[4], o[5], o[6], o[7]);
        }
      } else {
        const int t0 = (c - nc) * CK;
#pragma unroll 4
        for (int u = 0; u < UNITS; ++u) {
          const int unit = cw * UNITS + u, box = unit >> 3, row = (unit & 7) * 8 + rl;
          const uint32_t at = tile + (uint32_t)(box * CK * 128 + row * 128);
          uint4 x = make_uint4(0, 0, 0, 0), y = x;
          if (t0 + row < a.n_new) {
            const bf16* p = fresh + (long long)(t0 + row) * f_tok + box * 64 + cp * 16;
            x = *reinterpret_cast<const uint4*>(p);
            y = *reinterpret_cast<const uint4*>(p + 8);
          }
          sts128(at + (uint32_t)(((2 * cp) ^ (row & 7)) << 4), x.x, x.y, x.z, x.w);
          sts128(at + (uint32_t)(((2 * cp + 1) ^ (row & 7)) << 4), y.x, y.y, y.z, y.w);
        }
        sc = t0 + (ct & (CK - 1)) >= a.n_new ? 0.f : ct < CK ? a.scale_log2 : 1.f;
      }
      // The V converters bring both scales: a chunk's softmax waits for v_full,
      // and its scales are overwritten only after its PV.
      if (is_v) s_sc[slot * 2 * CK + ct] = sc;
      fence_proxy_async_smem();
      mbar_arrive(&full[slot]);
      if (i + 1 < nch && c + 1 < nc) load(c + 1);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------------- MMA
    if (lane == 0 && nch > 0) {
      constexpr uint32_t idesc_s = idesc_bf16(QROWS, CK), idesc_o = idesc_bf16(QROWS, D, 0, 1);
      bool good = mbar_wait(q_full, 0, a.err.wait_ns);
      const uint64_t q_desc = sw128_desc(smem_u32(smem + L::q), 16, 1024);
      const uint64_t k_desc = sw128_desc(smem_u32(smem + L::k), 16, 1024);
      const uint64_t v_desc = sw128_desc(smem_u32(smem + L::v), CK * 128, 1024);
      // S of chunk i goes over P of chunk i - 2: that chunk's PV must be done
      auto issue_s = [&](int i) -> bool {
        const int st = i & 1;
        if (!mbar_wait(&k_full[st], (i >> 1) & 1, a.err.wait_ns)) return false;
        if (i >= 2 && !mbar_wait(&o_done[st], ((i >> 1) & 1) ^ 1, a.err.wait_ns)) return false;
        tc_fence_after();
#pragma unroll
        for (int k16 = 0; k16 < D / 16; ++k16) {
          const uint32_t x = (uint32_t)k16 >> 2, w = ((uint32_t)k16 & 3u) * 32u;
          umma_bf16(tmem + (uint32_t)(st * CK), desc_add(q_desc, x * QROWS * 128u + w),
                    desc_add(k_desc, st * L::kTile + x * CK * 128u + w), idesc_s, k16 > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[st]);
        umma_commit(&k_empty[st]);
        return true;
      };
      if (good) good = issue_s(0);
      for (int i = 0; good && i < nch; ++i) {
        const int st = i & 1;
        if (i + 1 < nch && !(good = issue_s(i + 1))) break;
        if (!mbar_wait(&p_full[st], (i >> 1) & 1, a.err.wait_ns) || !mbar_wait(&v_full[st], (i >> 1) & 1, a.err.wait_ns)) {
          good = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int k16 = 0; k16 < CK / 16; ++k16)
          umma_bf16_tmem_a(t_o, tmem + (uint32_t)(st * CK) + k16 * 8u, desc_add(v_desc, st * L::kTile + k16 * 16u * 128u),
                           idesc_o, (i > 0 || k16 > 0) ? 1u : 0u);
        umma_commit(&o_done[st]);
        umma_commit(&v_empty[st]);
      }
      if (!good) {
        s_flag[0] = 1;
        set_error(a.err, DEV_TIMEOUT);
      }
      // every MMA this thread issued must finish before TMEM is freed
      umma_commit(drain);
      if (!mbar_wait(drain, 0, kDrainNs)) set_error(a.err, DEV_DRAIN);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- softmax
    {
      // Q tile: 16-byte chunks, rows past the last are zeros
      const uint32_t q0 = smem_u32(smem + L::q);
#pragma unroll 8
      for (int e = threadIdx.x; e < QROWS * D / 8; e += kSmx) {
        const int row = e / (D / 8), ch = e - row * (D / 8), rq = qt * QROWS + row;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (rq < rows) {
          const int qi = rq / a.group, hl = rq - qi * a.group;
          x = *reinterpret_cast<const uint4*>(a.q + b * a.q_seq + qi * a.q_tok + (long long)(h * a.group + hl) * a.q_head + ch * 8);
        }
        sts128(q0 + (uint32_t)((ch >> 3) * QROWS * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4)), x.x, x.y, x.z, x.w);
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full);
    }
    const int part = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int rq = qt * QROWS + r;
    const int oc0 = part * (D / 2);
    const int lim = a.causal ? min(len, len - a.n_q + 1 + min(rq, rows - 1) / a.group) : len;
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int i = 0; i < nch; ++i) {
      const int st = i & 1, c = c0 + i;
      const bool got = mbar_wait(&s_full[st], (i >> 1) & 1, a.err.wait_ns) &&
                       mbar_wait(&v_full[st], (i >> 1) & 1, a.err.wait_ns);
      __syncwarp();
      tc_fence_after();
      float sv[32];
      tmem_ld16(tmem + (uint32_t)(st * CK) + lane_off + part * 32, sv);
      tmem_ld16(tmem + (uint32_t)(st * CK) + lane_off + part * 32 + 16, sv + 16);
      tmem_ld_wait();
      reg_fence16(sv);
      reg_fence16(sv + 16);
      const float* sc = s_sc + st * 2 * CK + part * 32;
      // visible keys of this part's 32
      const int vis = (c < nc ? lim - c * CK : a.n_new - (c - nc) * CK) - part * 32;
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(sc + j);
        sv[j] *= k4.x;
        sv[j + 1] *= k4.y;
        sv[j + 2] *= k4.z;
        sv[j + 3] *= k4.w;
      }
      if (vis < 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) sv[j] = j < vis ? sv[j] : -INFINITY;
      }
      float mt[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) mt[j] = fmaxf(sv[j], sv[j + 16]);
#pragma unroll
      for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
        for (int j = 0; j < w; ++j) mt[j] = fmaxf(mt[j], mt[j + w]);
      s_pm[(st * 2 + part) * QROWS + r] = mt[0];
      // both parts of the row have their scores in registers (P overwrites S)
      // and their maxima in place, and go on or stop together
      if (!pair_and(1 + (warp & 3), got && s_flag[0] == 0)) {
        ok = false;
        break;
      }
      const float cmax = fmaxf(s_pm[st * 2 * QROWS + r], s_pm[(st * 2 + 1) * QROWS + r]);
      const float mx = cmax > m_run + 8.f ? cmax : m_run;
      const float ref = mx == -INFINITY ? 0.f : mx;  // no visible key so far
      const float alpha = ex2(m_run - ref);          // 1 when unchanged, 0 at first
#pragma unroll
      for (int j = 0; j < 32; ++j) sv[j] = ex2(sv[j] - ref);
#pragma unroll
      for (int j = 0; j < 16; ++j) mt[j] = sv[j] + sv[j + 16];
#pragma unroll
      for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
        for (int j = 0; j < w; ++j) mt[j] += mt[j + w];
      l_run = l_run * (m_run == -INFINITY ? 1.f : alpha) + mt[0];
      const bool scale_o = i > 0 && alpha != 1.f && m_run != -INFINITY;
      m_run = mx;
      if (__any_sync(0xffffffffu, scale_o)) {
        // O may be rescaled only once PV of the previous chunk has landed in it
        const bool good = __all_sync(0xffffffffu, mbar_wait(&o_done[st ^ 1], ((i - 1) >> 1) & 1, a.err.wait_ns));
        if (good) {
          const float f = scale_o ? alpha : 1.f;
          tc_fence_after();
          for (int jj = oc0; jj < oc0 + D / 2; jj += 16) {
            float ov[16];
            tmem_ld16(t_o + lane_off + jj, ov);
            tmem_ld_wait();
            reg_fence16(ov);
#pragma unroll
            for (int t = 0; t < 16; ++t) ov[t] *= f;
            tmem_st16(t_o + lane_off + jj, ov);
          }
          tmem_st_wait();
        } else {
          s_flag[0] = 1;
        }
      }
      uint32_t pk[16];
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 v4 = *reinterpret_cast<const float4*>(sc + CK + j);
        sv[j] *= v4.x;
        sv[j + 1] *= v4.y;
        sv[j + 2] *= v4.z;
        sv[j + 3] *= v4.w;
      }
      if (vis < 32) {  // masked places stay 0 whatever their scale is
#pragma unroll
        for (int j = 0; j < 32; ++j) sv[j] = j < vis ? sv[j] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) pk[j] = pack_bf16(sv[2 * j], sv[2 * j + 1]);
      tmem_st16u(tmem + (uint32_t)(st * CK) + lane_off + part * 16, pk);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[st]);
    }
    if (!ok) set_error(a.err, DEV_TIMEOUT);
    // PVs complete in issue order: the last chunk's commit covers them all
    if (nch > 0 && ok) ok = mbar_wait(&o_done[(nch - 1) & 1], ((nch - 1) >> 1) & 1, kDrainNs);
    s_l[part * QROWS + r] = l_run;
    ok = pair_and(1 + (warp & 3), ok && s_flag[0] == 0);
    tc_fence_after();
    const float l = s_l[r] + s_l[QROWS + r];
    // NaN scores alone leave the maximum at -inf: the row is not empty
    if (m_run == -INFINITY && l != 0.f) m_run = 0.f;
    const int qi = rq / a.group, hl = rq - qi * a.group;
    const bool live = rq < rows;
    if (splits == 1) {
      const float inv = l == 0.f ? 0.f : 1.f / l;  // no visible key: zeros
      bf16* op = a.o + b * a.o_seq + qi * a.o_tok + (long long)(h * a.group + hl) * a.o_head;
      for (int jj = oc0; jj < oc0 + D / 2; jj += 16) {
        float ov[16];
        if (ok && nch > 0) {
          tmem_ld16(t_o + lane_off + jj, ov);
          tmem_ld_wait();
          reg_fence16(ov);
        } else {
#pragma unroll
          for (int t = 0; t < 16; ++t) ov[t] = 0.f;
        }
        if (live && ok) {
          uint32_t w[8];
#pragma unroll
          for (int t = 0; t < 8; ++t) w[t] = pack_bf16(ov[2 * t] * inv, ov[2 * t + 1] * inv);
          uint4* dst = reinterpret_cast<uint4*>(op + jj);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
    } else {
      const size_t pr = ((size_t)bg * splits + split) * ((size_t)gridDim.x * QROWS) + rq;
      const bool some = ok && nch > 0 && m_run != -INFINITY;
      if (part == 0) a.part_ml[pr] = some ? make_float2(m_run, l) : make_float2(-INFINITY, 0.f);
      if (ok && nch > 0) {
        for (int jj = oc0; jj < oc0 + D / 2; jj += 16) {
          float ov[16];
          tmem_ld16(t_o + lane_off + jj, ov);
          tmem_ld_wait();
          reg_fence16(ov);
          if (some) {
            float4* dst = reinterpret_cast<float4*>(a.part_o + pr * D + jj);
#pragma unroll
            for (int t = 0; t < 4; ++t) dst[t] = make_float4(ov[4 * t], ov[4 * t + 1], ov[4 * t + 2], ov[4 * t + 3]);
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, ncols);
}

template <int D>
cudaError_t tc_init() {
  return cudaFuncSetAttribute(k_kv8_attn_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<D>::total);
}
template <int D>
cudaError_t tc_launch(const Kv8AttnPlan& p, const Kv8AttnArgs& a, bool pdl, cudaStream_t st) {
  return launch_ex(k_kv8_attn_tc<D>, dim3(p.qtiles, p.splits, a.n_seq * a.c.heads), dim3(kThreads), Smem<D>::total, st,
                   1, pdl, a);
}

}  // namespace

cudaError_t kv8_attn_tc_init() {
  cudaError_t e = tc_init<64>();
  if (e == cudaSuccess) e = tc_init<128>();
  if (e == cudaSuccess) e = tc_init<256>();
  return e;
}

cudaError_t launch_kv8_attn_tc(const Kv8AttnPlan& p, const Kv8AttnArgs& a, bool pdl, cudaStream_t st) {
  if (a.c.d == 64) return tc_launch<64>(p, a, pdl, st);
  if (a.c.d == 128) return tc_launch<128>(p, a, pdl, st);
  return tc_launch<256>(p, a, pdl, st);
}

}  // namespace pae
