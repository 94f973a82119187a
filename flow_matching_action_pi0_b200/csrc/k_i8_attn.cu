// Attention over the int8 K/V cache for few query rows (single tokens), and
// the merge of partial rows over key splits.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j - max),
//   k_j = kq_j ks_j, v_j = vq_j vs_j  (8-bit codes, one scale per key)
//
// One pass over the keys with the running maximum and sum of a softmax.
// Scores: a query row becomes integers of a power of two qs, q = (2^16 hi + 2^8
// mid + lo) qs with three signed 8-bit digits and 2^21 <= max|q| / qs < 2^22, so the
// key codes go into integer products as they lie in memory, three per 32
// channels, and the sums are exact.  (As bf16 operands every pair of codes
// costs four instructions, half of the loop.)  An element is exact unless it is
// below 2^-14 of the row's largest, and off by 2^-22 of that at most: no more than
// an fp32 sum of the products may be.  (Two digits, 2^-16, took 32.1
// instead of 33.0 us for 48 sequences of up to 8192 keys, but lost the small
// channels of rows with a large one.)  Values: the codes become fp16
// integers, exactly, and the value's scale joins the exponent:
//   c_j = exp2(s_j + log2 vs_j - ref) = p_j vs_j 2^(m - ref),
// so that c in fp16 (rounded once, to 11 bits) is in units of the row's largest
// contribution whatever the scales are: max c lies in [2^7, 2^15], so the steps of
// 2^-24 at fp16's bottom put each contribution off by at most 2^-32 of the
// largest, and the n keys of a warp's share by n 2^-32 at worst (all of them below
// the step: the row sum counts what they lose).  The row sums have a reference m
// of their own, since a key may weigh much and carry little: sum p_j in fp32, lane
// by lane.  The two meet in the exponent of the row's last factor, 2^(ref - m) /
// sum, and partial rows are parked as averages with the logarithm of their weight,
// so no size of V overflows or is lost.
//
// Bound: bytes of the cache (2 (d + 4) per key and KV head).  The G query
// heads of a KV head share every byte, 8 rows at a time as the N side of
// mma.sync (m16n8k32 for keys, m16n8k16 for value channels, on the M side): a lane turns
// the 16 bytes that it copied itself straight into A fragments, with no
// exchange between lanes (a 128-row tensor-core tile would be 94 %
// padding here and its operands would have to be staged).  The contraction
// index may be permuted freely, so fragments are cut from contiguous 16-byte
// loads:
//   K: lane (g, t) = (lane / 4, lane % 4) loads 16 channels [64 j + 16 t, +16)
//      of keys g and g + 8: two products of 32 channels
//   V: lane (g, t) loads 16 channels [128 h + 16 g, +16) of keys 2t, 2t + 1,
//      2t + 8, 2t + 9; product m of block h takes channels 2 m (row g) and
//      2 m + 1 (row g + 8)
// Work is cut into units of 64 keys (16 per warp) of one (sequence, KV head, row
// group); every sequence has one at least.  Units in that order are dealt out
// evenly: block i of G takes units [T i / G, T (i + 1) / G), whatever the lengths,
// so a batch of ragged sequences finishes together (an equal number of splits per
// sequence left the SMs to the longest ones: 36.8 us for 48 sequences of up to
// 8192 keys, 33 now, 3.1 TB/s).  Inside a block each warp has statistics of its
// own and the warps meet once per sequence.  A sequence that lies in one block is
// written out by it; of the others each block parks its fp32 rows in one of its
// two workspace slots (0: the part continues an earlier block's, 1: it begins
// here), and k_kv8_merge_few joins them.
#include <algorithm>
#include <cmath>

#include <cuda_fp16.h>

#include "int8.h"
#include "launch.cuh"

namespace pae {

namespace {

constexpr int kWarps = 4;
constexpr int kTileKeys = 16;
constexpr float kLift = 7.f, kTop = 15.f;  // log2 of the largest c where the reference is set, and where it moves

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// int8 x int8 -> int32, 32 channels
__device__ __forceinline__ void mma_s8(int* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit elements across the warp
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two signed bytes in bits 0-7 and 16-23 of w (the other bits are ignored) ->
// fp16x2, exactly: 0x6400 | (byte ^ 0x80) is 1024 + 128 + code.
__device__ __forceinline__ uint32_t bytes_f16x2(uint32_t w) {
  const uint32_t u = (w & 0x00FF00FFu) ^ 0x64806480u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&u), __floats2half2_rn(1152.f, 1152.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Units of 64 keys of a sequence: at least one, so that an empty sequence is
// written (as zeros) by some block.
constexpr int kUnit = kWarps * kTileKeys;
__device__ __forceinline__ int seq_len(const Kv8AttnArgs& a, int b) { return max(0, min(__ldg(a.lens + b), a.c.cap)); }
__device__ __forceinline__ int seq_units(int len) { return len < 1 ? 1 : (len - 1) / kUnit + 1; }

// a / b for a >= 0, b > 0: in 32 bits where they suffice
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Exclusive prefix sums of the sequences' units over the block: thread i holds
// a slice [b0, b1) and gets the units before it; returns the total.  `sh` has
// NT / 32 entries.
template <int NT>
__device__ __forceinline__ long long scan_units(const Kv8AttnArgs& a, long long* sh, int& b0, int& b1, long long& before) {
  const int per = (a.n_seq + NT - 1) / NT, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  b0 = min(a.n_seq, (int)threadIdx.x * per);
  b1 = min(a.n_seq, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += seq_units(seq_len(a, b));
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  long long total = 0, pre = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) pre += sh[w];
    total += sh[w];
  }
  before = pre + inc - mine;
  return total;
}

constexpr int kStages = 2;  // tiles of 16 keys per warp, the one at work included
constexpr long long kDrainNs = 4000000000LL;
// K codes | V codes of a tile: [16 keys][d] each, as they lie in the cache
__host__ __device__ constexpr int few_stage(int d) { return 2 * kTileKeys * d; }

// Untiled bulk copy global -> shared, completion on `bar` (16-byte units).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, D == 256 ? 2 : 4) k_kv8_attn_few(const Kv8AttnArgs a, int rgs) {
  constexpr int KBLK = D / 64;               // 64-channel blocks of a K row
  constexpr int VB = D >= 128 ? 16 : 8;      // bytes of a V row per lane and block
  constexpr int VBLK = D / (8 * VB);         // blocks of a V row
  constexpr int VM = VB / 2;                 // products per block
  constexpr int STEP = kUnit;
  extern __shared__ __align__(16) float s_o[];  // the warps' rings; at the end of a sequence [kWarps][8][D + 4]
  __shared__ float s_m[kWarps][8], s_x[kWarps][8], s_l[kWarps][8];
  __shared__ float2 s_row[8];
  __shared__ uint64_t s_bar[kWarps][kStages];
  __shared__ long long s_scan[kWarps];
  __shared__ int s_b;
  __shared__ long long s_before;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rows = a.group * a.n_q;
  const int hr = a.c.heads * rgs;  // items (KV head, row group) of a sequence
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&s_bar[warp][i], 1);
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();  // after the wait: the merge may read the lengths before its own

  // this block's units, and the sequence the first of them lies in
  long long unit, unit_end;
  int b;
  long long b_unit;  // first unit of sequence b
  {
    int b0, b1;
    long long before;
    const long long total = scan_units<kWarps * 32>(a, s_scan, b0, b1, before) * hr;
    const long long G = min((long long)gridDim.x, total);  // blocks with units
    if (blockIdx.x >= G) return;
    unit = div_ll(total * blockIdx.x, G);
    unit_end = div_ll(total * (blockIdx.x + 1), G);
    before *= hr;
    for (int i = b0; i < b1; ++i) {
      const long long n = (long long)seq_units(seq_len(a, i)) * hr;
      if (before <= unit && unit < before + n) {
        s_b = i;
        s_before = before;
      }
      before += n;
    }
    __syncthreads();
    b = s_b;
    b_unit = s_before;
  }

  int tiles = 0;  // tiles this warp has asked for: tile i goes through stage i % kStages
  while (unit < unit_end) {
  const int len = seq_len(a, b), units = seq_units(len);
  const int item = (int)div_ll(unit - b_unit, units), u0 = (int)((unit - b_unit) - (long long)item * units);
  const int u1 = (int)min((long long)units, u0 + (unit_end - unit));
  const int h = item / rgs, rg = item - h * rgs;
  const int key0 = min(len, u0 * STEP), key1 = (int)min((long long)len, (long long)u1 * STEP);

  // Q: row r = query * group + head-in-group; lane (g, t) holds channels
  // [64 j + 16 t, +16) of row 8 rg + g (asked for before the key tiles, which
  // would keep it waiting)
  uint4 x[KBLK][2];
  {
    const int r = rg * 8 + g;
    const bool live = r < rows;
    const int qi = live ? r / a.group : 0, hl = live ? r - qi * a.group : 0;
    const bf16* qp = a.q + b * a.q_seq + qi * a.q_tok + (long long)(h * a.group + hl) * a.q_head + 16 * t;
#pragma unroll
    for (int j = 0; j < KBLK; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        x[j][i] = live ? __ldg(reinterpret_cast<const uint4*>(qp + 64 * j + 8 * i)) : make_uint4(0, 0, 0, 0);
  }

  const size_t base = ((size_t)b * a.c.heads + h) * a.c.cap;
  // Each warp streams its own tiles through a ring of its own: one bulk copy
  // for the K codes of 16 keys and one for their V codes (copied by the lanes
  // 16 bytes at a time, the same bytes kept the load/store unit busy for as
  // long as the memory).  Rows past the range are not copied: what the stage
  // holds there is masked.  The scales ride in a register, one per lane.
  int8_t* ring = reinterpret_cast<int8_t*>(s_o) + warp * (kStages * few_stage(D));
  auto fill = [&](int at) {
    if (lane == 0) {
      const uint32_t bytes = (uint32_t)min(kTileKeys, key1 - at) * D;
      const int st = tiles % kStages;
      const uint32_t dst = smem_u32(ring + st * few_stage(D));
      mbar_arrive_expect_tx(&s_bar[warp][st], 2 * bytes);
      bulk_load(dst, a.c.k + (base + at) * D, bytes, &s_bar[warp][st]);
      bulk_load(dst + kTileKeys * D, a.c.v + (base + at) * D, bytes, &s_bar[warp][st]);
    }
    ++tiles;
  };
  auto scales = [&](int at) {  // lanes 0-15: K scales of keys at.., 16-31: V scales
    const int key = min(at + (lane & 15), key1 - 1);
    return __ldg((lane < 16 ? a.c.k_scale : a.c.v_scale) + base + key);
  };
  int at = key0 + warp * kTileKeys;
  float sc_next[kStages];
  int cur = tiles;  // the tile at work
#pragma unroll
  for (int i = 0; i < kStages; ++i)
    if (at + i * STEP < key1) {
      fill(at + i * STEP);
      sc_next[i] = scales(at + i * STEP);
    }

  uint32_t qh[KBLK][4], qm[KBLK][4], ql[KBLK][4];  // digits of 4 channels per word
  float qs[2];                                     // scales of rows 2t, 2t + 1
  {
    uint32_t am = 0;
#pragma unroll
    for (int j = 0; j < KBLK; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        am = __vmaxu2(am, __vmaxu2(__vmaxu2(x[j][i].x & 0x7FFF7FFFu, x[j][i].y & 0x7FFF7FFFu),
                                   __vmaxu2(x[j][i].z & 0x7FFF7FFFu, x[j][i].w & 0x7FFF7FFFu)));
      }
    am = max(am << 16, am & 0xFFFF0000u);
    am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
    am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
    // rows below 2^-105 count as zeros; a NaN or an infinity makes every score NaN
    const uint32_t e = am >> 23;
    const bool some = e >= 22 && e < 255;
    const float inv = some ? __uint_as_float((275 - e) << 23) : 0.f;  // 2^21 / 2^(e - 127)
    const float sc = e == 255 ? __int_as_float(0x7FC00000) : some ? __uint_as_float((e - 21) << 23) : 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) qs[i] = __shfl_sync(0xFFFFFFFFu, sc, (2 * t + i) * 4) * a.scale_log2;
    // q inv + 1.5 2^23 rounds to a whole number in the low bits of the sum; that
    // number + 0x8080 has hi in byte 2, mid + 128 in byte 1 and lo + 128 in byte 0
#pragma unroll
    for (int j = 0; j < KBLK; ++j)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t s0 = (w & 1) ? x[j][w >> 1].z : x[j][w >> 1].x, s1 = (w & 1) ? x[j][w >> 1].w : x[j][w >> 1].y;
        const float f[4] = {__uint_as_float(s0 << 16), __uint_as_float(s0 & 0xFFFF0000u), __uint_as_float(s1 << 16),
                            __uint_as_float(s1 & 0xFFFF0000u)};
        uint32_t m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = some ? __float_as_uint(fmaf(f[i], inv, 12582912.f)) + (0x8080u - 0x4B400000u) : 0x8080u;
        qh[j][w] = __byte_perm(__byte_perm(m[0], m[1], 0x0062), __byte_perm(m[2], m[3], 0x0062), 0x5410);
        qm[j][w] = __byte_perm(__byte_perm(m[0], m[1], 0x0051), __byte_perm(m[2], m[3], 0x0051), 0x5410) ^ 0x80808080u;
        ql[j][w] = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410) ^ 0x80808080u;
      }
  }
  // first key that rows 2t and 2t + 1 of the group cannot see
  int lim[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = rg * 8 + 2 * t + i;
    lim[i] = a.causal && r < rows ? min(len, len - a.n_q + 1 + r / a.group) : len;
  }

  float o[VBLK][VM][4];
#pragma unroll
  for (int i = 0; i < VBLK; ++i)
#pragma unroll
    for (int m = 0; m < VM; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][m][j] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY};                      // reference of c, the warp's
  float x_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};  // of the sum, this lane's

  for (; at < key1; at += STEP) {
    const float sc = sc_next[0];
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) sc_next[i] = sc_next[i + 1];
    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&s_bar[warp][cur % kStages], (cur / kStages) & 1, a.err.wait_ns))) {
      set_error(a.err, DEV_TIMEOUT);
      for (int i = cur; i < tiles; ++i)  // copies still in flight must land before their stage is used again
        if (!mbar_wait(&s_bar[warp][i % kStages], (i / kStages) & 1, kDrainNs)) set_error(a.err, DEV_DRAIN);
      break;
    }
    const int8_t* tile = ring + (cur % kStages) * few_stage(D);
    // scores of 16 keys x 8 rows: lane holds keys g, g + 8, rows 2t, 2t + 1
    int ch[4] = {0, 0, 0, 0}, cm[4] = {0, 0, 0, 0}, cl[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < KBLK; ++j) {
      const uint4 x0 = *reinterpret_cast<const uint4*>(tile + g * D + 64 * j + 16 * t);
      const uint4 x1 = *reinterpret_cast<const uint4*>(tile + (g + 8) * D + 64 * j + 16 * t);
      mma_s8(ch, x0.x, x1.x, x0.y, x1.y, qh[j][0], qh[j][1]);
      mma_s8(cm, x0.x, x1.x, x0.y, x1.y, qm[j][0], qm[j][1]);
      mma_s8(cl, x0.x, x1.x, x0.y, x1.y, ql[j][0], ql[j][1]);
      mma_s8(ch, x0.z, x1.z, x0.w, x1.w, qh[j][2], qh[j][3]);
      mma_s8(cm, x0.z, x1.z, x0.w, x1.w, qm[j][2], qm[j][3]);
      mma_s8(cl, x0.z, x1.z, x0.w, x1.w, ql[j][2], ql[j][3]);
    }
    const float lv_l = __log2f(sc);  // (of the V scales, lanes 16-31; 0, with codes 0, gives -inf)
    float ks[2], lv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ks[i] = __shfl_sync(0xFFFFFFFFu, sc, g + 8 * i);
      lv[i] = __shfl_sync(0xFFFFFFFFu, lv_l, 16 + g + 8 * i);
    }
    float c[4];  // (|hi| <= 64: |256 hi + mid| sums stay below 2^30)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = fmaf((float)(ch[i] * 256 + cm[i]), 256.f, (float)cl[i]) * qs[i & 1];
    const int ka = at + g, kc = ka + 8;
    const bool in[4] = {ka < min(lim[0], key1), ka < min(lim[1], key1), kc < min(lim[0], key1), kc < min(lim[1], key1)};
    float x[4];  // masked places: -inf, whatever their scale is
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = in[i] ? c[i] * ks[i >> 1] : -INFINITY;
    // The sum's reference moves when a score exceeds it by 64: fp32 holds both
    // sides, and what is under 2^-126 of it is nothing beside the maximum.
    bool far[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) far[i] = fmaxf(x[i], x[i + 2]) > x_run[i] + 64.f;
    if (__any_sync(0xFFFFFFFFu, far[0] || far[1])) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!far[i]) continue;
        const float nx = fmaxf(x[i], x[i + 2]);
        l_run[i] *= ex2(x_run[i] - nx);
        x_run[i] = nx;
      }
    }
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = x[i] == -INFINITY ? 0.f : ex2(x[i] - x_run[i & 1]);
    l_run[0] += p[0] + p[2];
    l_run[1] += p[1] + p[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = in[i] ? x[i] + lv[i >> 1] : -INFINITY;
    float al[2];
    bool grow = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = fmaxf(x[i], x[i + 2]);
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
      // the reference moves only when the maximum grows by a factor 256 above
      // where it was set: c stays within 2^15 and O is rescaled rarely
      const bool up = mx > m_run[i] + kTop || m_run[i] == -INFINITY;
      const float nm = up ? fmaxf(mx - kLift, m_run[i]) : m_run[i];
      al[i] = nm == -INFINITY ? 1.f : ex2(m_run[i] - nm);
      grow |= al[i] != 1.f;
      m_run[i] = nm;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = x[i] == -INFINITY ? 0.f : ex2(x[i] - m_run[i & 1]);
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
    const uint32_t b0 = movmatrix(pack_f16(p[0], p[1])), b1 = movmatrix(pack_f16(p[2], p[3]));
#pragma unroll
    for (int j = 0; j < VBLK; ++j) {
      uint32_t vr[4][VB / 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int8_t* p8 = tile + (kTileKeys + 2 * t + (i & 1) + (i >> 1) * 8) * D + (8 * VB) * j + VB * g;
        if constexpr (VB == 16) {
          const uint4 x4 = *reinterpret_cast<const uint4*>(p8);
          vr[i][0] = x4.x; vr[i][1] = x4.y; vr[i][2] = x4.z; vr[i][3] = x4.w;
        } else {
          const uint2 x2 = *reinterpret_cast<const uint2*>(p8);
          vr[i][0] = x2.x; vr[i][1] = x2.y;
        }
      }
#pragma unroll
      for (int m = 0; m < VM; ++m) {
        const int w = m >> 1;
        const uint32_t lo = (m & 1) ? 0x0602u : 0x0400u, hi = (m & 1) ? 0x0703u : 0x0501u;
        const uint32_t f[4] = {bytes_f16x2(__byte_perm(vr[0][w], vr[1][w], lo)),
                               bytes_f16x2(__byte_perm(vr[0][w], vr[1][w], hi)),
                               bytes_f16x2(__byte_perm(vr[2][w], vr[3][w], lo)),
                               bytes_f16x2(__byte_perm(vr[2][w], vr[3][w], hi))};
        mma_f16(o[j][m], f, b0, b1);
      }
    }
    __syncwarp();  // every lane has read the stage: the next copy may overwrite it
    if (at + kStages * STEP < key1) {
      fill(at + kStages * STEP);
      sc_next[kStages - 1] = scales(at + kStages * STEP);
    }
    ++cur;
  }

  // row sums over the 8 lanes that share t, in units of their largest reference
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float mx = x_run[i];
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
    float l = x_run[i] == -INFINITY ? l_run[i] : l_run[i] * ex2(x_run[i] - mx);  // (0, or NaN of NaN scores alone)
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
    if (g == 0) {
      s_m[warp][2 * t + i] = m_run[i];
      s_x[warp][2 * t + i] = mx;
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
  const bool whole = u0 == 0 && u1 == units;
  // the root of a row's last factor (2^(M - lw) may be below fp32 where the average
  // is not) and the logarithm of its weight, by one warp's first lanes
  if (threadIdx.x < 8) {
    const int r = threadIdx.x;
    float M = -INFINITY, X = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      M = fmaxf(M, s_m[w][r]);
      X = fmaxf(X, s_x[w][r]);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) l += s_x[w][r] == -INFINITY ? s_l[w][r] : s_l[w][r] * ex2(s_x[w][r] - X);
    const float lw = X == -INFINITY ? l : X + __log2f(l);  // (without a maximum l is 0 or NaN)
    s_row[r] = l == 0.f ? make_float2(0.f, -INFINITY) : make_float2(ex2(0.5f * (M - lw - (whole ? 0.f : kPartShift))), lw);  // no visible key: zeros
  }
  __syncthreads();
#pragma unroll
  for (int e = threadIdx.x; e < 8 * (D / 4); e += kWarps * 32) {
    const int r = e / (D / 4), c4 = e - r * (D / 4);
    const float f = s_row[r].x, lw = s_row[r].y;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(s_o + (w * 8 + r) * LD + 4 * c4);
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
    acc = make_float4(acc.x * f * f, acc.y * f * f, acc.z * f * f, acc.w * f * f);
    const int row = rg * 8 + r;
    if (whole) {
      if (row < rows) {
        const int qi = row / a.group, hl = row - qi * a.group;
        bf16* op = a.o + b * a.o_seq + qi * a.o_tok + (long long)(h * a.group + hl) * a.o_head + 4 * c4;
        *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
      }
    } else {
      const size_t pr = ((size_t)blockIdx.x * 2 + (u0 == 0 ? 1 : 0)) * 8 + r;
      *reinterpret_cast<float4*>(a.part_o + pr * D + 4 * c4) = acc;
      if (c4 == 0) a.part_ml[pr] = part_weight(lw);
    }
  }
  unit += u1 - u0;
  if (unit - b_unit == (long long)units * hr) {  // on to the next sequence
    b_unit = unit;
    ++b;
  }
  fence_proxy_async_smem();  // s_o was written by threads, the rings are written by copies
  __syncthreads();           // s_o and the statistics are free again
  }
}

constexpr float kUnshift = 16384.f;  // 2^kPartShift

// (m, l, acc) joined with the row x of maximum and sum ml; no maximum: nothing
// was visible there, and x is passed over.
__device__ __forceinline__ void merge_part(float2 ml, float4 x, float& m, float& l, float4& acc) {
  if (ml.x == -INFINITY) return;
  const float nm = fmaxf(m, ml.x), f = m == -INFINITY ? 0.f : ex2(m - nm), w = ex2(ml.x - nm);
  m = nm;
  l = fmaf(l, f, w * ml.y);
  acc.x = fmaf(acc.x, f, w * x.x);
  acc.y = fmaf(acc.y, f, w * x.y);
  acc.z = fmaf(acc.z, f, w * x.z);
  acc.w = fmaf(acc.w, f, w * x.w);
}

// Joins the parts of the (sequence, KV head, row group) items that
// k_kv8_attn_few left to several blocks: one block per (row, item).
template <int D, int NT>
__global__ void __launch_bounds__(NT) k_kv8_merge_few(const Kv8AttnArgs a, int rgs, int blocks) {
  constexpr int C4 = D / 4, NS = NT / C4;
  __shared__ long long s_scan[NT / 32];
  __shared__ long long s_before;
  __shared__ float2 s_ml[NS];
  __shared__ float4 s_acc[NT];
  const int item_all = blockIdx.x, r = blockIdx.y;  // ((sequence, KV head), row group); row of the group
  const int hr = a.c.heads * rgs, b = item_all / hr, item = item_all - b * hr;
  const int h = item / rgs, rg = item - h * rgs;
  const int row = rg * 8 + r;
  pdl_launch_dependents();
  if (row >= a.group * a.n_q) return;
  // which blocks hold the item: only the lengths are needed, which no kernel
  // in flight writes (the attention let this one start after its own wait)
  const int units = seq_units(seq_len(a, b));
  long long total;
  {
    int b0, b1;
    long long before;
    total = scan_units<NT>(a, s_scan, b0, b1, before) * hr;
    for (int i = b0; i < b1; ++i) {
      if (i == b) s_before = before;
      before += seq_units(seq_len(a, i));
    }
    __syncthreads();
  }
  const long long first = s_before * hr + (long long)item * units, last = first + units - 1;
  // block i of G holds units [total i / G, total (i + 1) / G)
  const long long G = min((long long)blocks, total);
  const int c0 = (int)div_ll((first + 1) * G - 1, total), c1 = (int)div_ll((last + 1) * G - 1, total);
  pdl_wait();
  if (c0 == c1) return;  // written by its one block
  const int tid = threadIdx.x;
  const int c4 = tid % C4, part = tid / C4;
  // every NS-th part, its running maximum and sums as in the attention
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int cb = c0 + part; cb <= c1; cb += 4 * NS) {
    float2 ml[4];
    float4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // four parts in flight
      const int c = cb + i * NS;
      const size_t pr = ((size_t)c * 2 + (c == c0 ? 1 : 0)) * 8 + r;  // the item begins in c0 only
      ml[i] = c <= c1 ? __ldcg(a.part_ml + pr) : make_float2(-INFINITY, 0.f);
      x[i] = c <= c1 ? __ldcg(reinterpret_cast<const float4*>(a.part_o + pr * D + 4 * c4)) : acc;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) merge_part(ml[i], x[i], m, l, acc);
  }
  s_acc[tid] = acc;
  if (c4 == 0) s_ml[part] = make_float2(m, l);
  __syncthreads();
  if (part == 0) {
#pragma unroll
    for (int s = 1; s < NS; ++s) merge_part(s_ml[s], s_acc[s * C4 + c4], m, l, acc);
    const int qi = row / a.group, hl = row - qi * a.group;
    const float inv = l == 0.f ? 0.f : kUnshift / l;
    bf16* op = a.o + b * a.o_seq + qi * a.o_tok + (long long)(h * a.group + hl) * a.o_head + 4 * c4;
    *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  }
}

// The parts of k_kv8_attn_tc, averages over their keys and the logarithms lw_s of
// their weights: o = sum_s 2^lw_s O_s / sum_s 2^lw_s.  rowsp: rows of a part.
template <int D>
__global__ void __launch_bounds__(256) k_kv8_merge(const Kv8AttnArgs a, int splits, int rowsp) {
  constexpr int C4 = D / 4, NR = 256 / C4;  // rows per block
  const int row = blockIdx.x * NR + threadIdx.x / C4, c4 = threadIdx.x % C4, bg = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  if (row >= a.group * a.n_q) return;
  const int b = bg / a.c.heads, h = bg - b * a.c.heads;
  const size_t p0 = (size_t)bg * splits * rowsp + row;
  constexpr int NP = 8;  // parts in flight
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto join = [&](int s0) {
    float2 ml[NP];
    float4 x[NP];
#pragma unroll
    for (int s = 0; s < NP; ++s)
      if (s0 + s < splits) {
        const size_t at = p0 + (size_t)(s0 + s) * rowsp;
        ml[s] = __ldcg(a.part_ml + at);
        x[s] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D + 4 * c4));
      }
#pragma unroll
    for (int s = 0; s < NP; ++s)
      if (s0 + s < splits) merge_part(ml[s], x[s], m, l, acc);
  };
  join(0);
  for (int s0 = NP; s0 < splits; s0 += NP) join(s0);
  const int qi = row / a.group, hl = row - qi * a.group;
  const float inv = l == 0.f ? 0.f : kUnshift / l;
  bf16* op = a.o + b * a.o_seq + qi * a.o_tok + (long long)(h * a.group + hl) * a.o_head + 4 * c4;
  *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

size_t few_smem(int d) { return (size_t)kWarps * kStages * few_stage(d); }  // (covers [kWarps][8][d + 4] floats)

template <int D>
cudaError_t few_launch(const Kv8AttnPlan& p, const Kv8AttnArgs& a, bool pdl, cudaStream_t st) {
  cudaError_t e = launch_ex(k_kv8_attn_few<D>, dim3(p.splits), dim3(kWarps * 32), few_smem(D), st, 1, pdl, a, p.qtiles);
  if (e != cudaSuccess || p.ws_bytes == 0) return e;
  // twice the threads where an item may have more than 32 parts (one sequence of
  // 65536 keys: 27.0 us with 256, 19.8 with 512; 32 of 968 and two row groups: 16.6
  // and 19.9)
  const dim3 items(a.n_seq * a.c.heads * p.qtiles, 8);
  if (p.splits > 32LL * items.x) return launch_ex(k_kv8_merge_few<D, 512>, items, dim3(512), 0, st, 1, true, a, p.qtiles, p.splits);
  return launch_ex(k_kv8_merge_few<D, 256>, items, dim3(256), 0, st, 1, true, a, p.qtiles, p.splits);
}
template <int D>
cudaError_t merge_launch(const Kv8AttnPlan& p, const Kv8AttnArgs& a, cudaStream_t st) {  // (PDL behind its own attention)
  const int nr = 1024 / D;  // rows per block
  return launch_ex(k_kv8_merge<D>, dim3((a.group * a.n_q + nr - 1) / nr, a.n_seq * a.c.heads), dim3(256), 0, st, 1, true, a, p.splits, p.qtiles * 128);
}

}  // namespace

// Two forms: groups of 8 rows (query heads of a KV head x queries) on mma.sync,
// which read the cache once per group, and tiles of 128 rows on the tcgen05
// tensor cores (fresh keys always, the groups have no place for them: one query and
// one fresh key over 968 keys 11.7 us; 11.2 when the key is written to the cache
// first, 48 sequences 21.7 and 18.9), whose keys are split until the CTAs fill
// the SMs, each split keeping at least 64 keys of a full cache (one sequence of
// 968 keys and 400 rows: 12.6 us; 14.8 with at least 128, 20.2 with 256).
// Measured over 1 to 32 sequences of 256 to 16384 keys, 8 to 256 rows, head_dim d:
//   groups  5.4 + d / 100 us, and 3.2 + d / 80 ns per unit (64 keys of 8 rows)
//   tiles   4.7 + d / 100 us, and 1.0 + d / 570 us per chunk of 64 keys that a CTA
//           walks
// e.g. (d 256) 32 rows over 968 keys: 8.0 and 10.9 us for 1 sequence, 13.5 and 11.3
// for 8; 8 rows, 32 sequences: 13.5 and 14.9; 64 rows over 4096 keys: 11.9 and 19.6
// for 1, 53.5 and 22.2 for 16.
Kv8AttnPlan plan_kv8_attn(int n_seq, int heads_kv, int group, int n_q, int n_new, int max_keys, int d) {
  const long long rows = (long long)group * n_q, seqs = (long long)n_seq * heads_kv;
  Kv8AttnPlan t{};  // tiles
  t.tc = 1;
  t.qtiles = (int)((rows + 127) / 128);
  const long long blocks = seqs * t.qtiles;
  const long long keys = std::max(1LL, (long long)max_keys + n_new);
  t.splits = 1;
  while (t.splits < 8 && blocks * t.splits * 2 <= 148 && keys / (t.splits * 2) >= 64) t.splits *= 2;
  while (keys > kTileRefKeys * t.splits) t.splits *= 2;
  t.ws_bytes = t.splits > 1 ? (size_t)blocks * t.splits * 128 * ((size_t)d * 4 + 8) : 0;
  const long long chunks = ((keys - 1) / 64 + t.splits) / t.splits * ((blocks * t.splits + 147) / 148);

  Kv8AttnPlan g{};  // groups
  g.qtiles = (int)((rows + 7) / 8);
  // blocks that deal out the units: two (four for head_dim < 256) resident per
  // SM, more where a warp's share of a full cache would be too long for one
  // reference, and no more than there are units in it
  const long long units = seqs * g.qtiles * ((std::max(max_keys, 1) - 1) / kUnit + 1);
  const long long shares = (units * kTileKeys - 1) / kGroupRefKeys + 1;
  g.splits = (int)std::min<long long>(units, std::max(148LL * (d == 256 ? 2 : 4), shares));
  // (with one unit per item no item is shared)
  g.ws_bytes = g.splits > 1 && max_keys > kUnit ? (size_t)g.splits * 2 * 8 * ((size_t)d * 4 + 8) : 0;
  return n_new == 0 && 700 + (3.2 + d / 80.0) * (double)units < (1010 + 1.75 * d) * (double)chunks ? g : t;
}

cudaError_t kv8_attn_init() {
  cudaError_t e = cudaFuncSetAttribute(k_kv8_attn_few<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)few_smem(256));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_kv8_attn_few<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)few_smem(128));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_kv8_attn_few<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)few_smem(64));
  return e == cudaSuccess ? kv8_attn_tc_init() : e;
}

cudaError_t launch_kv8_attn(const Kv8AttnPlan& p, const Kv8AttnArgs& a, bool pdl, cudaStream_t st) {
  cudaError_t e;
  if (!p.tc) return a.c.d == 64 ? few_launch<64>(p, a, pdl, st) : a.c.d == 128 ? few_launch<128>(p, a, pdl, st) : few_launch<256>(p, a, pdl, st);
  e = launch_kv8_attn_tc(p, a, pdl, st);
  if (e != cudaSuccess || p.splits == 1) return e;
  if (a.c.d == 64) return merge_launch<64>(p, a, st);
  if (a.c.d == 128) return merge_launch<128>(p, a, st);
  return merge_launch<256>(p, a, st);
}

}  // namespace pae
