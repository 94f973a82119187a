// Attention over the int8 K/V cache, and fresh bf16 keys behind it, for many
// query rows: the denoise loop's chunk of action tokens, or a causal prompt.
//
// Mathematics as in k_i8_attn.cu: scores are products with the codes (bf16
// integers here), and c = p vs, in units of the largest contribution, is
// rounded to fp16 against V codes as fp16 integers.  Fresh tiles take c and V in
// bf16, whose range fresh values may need.  The query heads that share a KV
// head times the queries (row = query * group + head-in-group, so that a tile
// spans few queries and a causal tile skips the keys behind its last one) are
// cut into tiles of 128 rows, the M dimension of tcgen05.mma.  Per chunk of 64
// keys:
//   converters (8 warps)  read the codes (16-byte loads, the next chunk's in
//                         flight while this one is written), turn them into
//                         integers (exact; K bf16, V fp16) in the 128-byte
//                         swizzled tiles the MMA reads; fresh keys and values
//                         are copied as they are
//   two MMA warps         S = Q K^T (128 x 64, double-buffered in TMEM) and
//                         O += P V (P read from TMEM, V read MN-major): an
//                         issuing warp gets one instruction in thirty cycles
//                         or so beside the others, and one warp for both was
//                         part of the chunk-to-chunk chain
//   scale warp            the chunk's key and value scales, see there
//   softmax (16 warps)    four threads per row: online softmax in the log2
//                         domain (O is rescaled only when the maximum grows by
//                         more than 2^8), c over S's own columns.  The
//                         chunk-to-chunk chain runs through it, so its latency
//                         counts: with two threads per row a chunk took 2900
//                         cycles.
// Bound: the latency of that chain, 2600 cycles per chunk (the tensor cores are
// busy for 1050 of them, the issue slots for about half): 50 queries x 8 heads of
// 32 sequences over 968 + 50 keys, 128 CTAs of 17 chunks, 32 us; K and V of a
// sequence are converted once per tile.
// Key splits (small batches) write fp32 averages with the logarithm of their
// weight to the workspace; k_kv8_merge joins them.
#include <climits>

#include <cuda_fp16.h>

#include "int8.h"
#include "launch.cuh"

namespace pae {

namespace {

constexpr int QROWS = 128, CK = 64;
constexpr int kSmxWarps = 16;              // softmax warps (0-15): four threads per row
constexpr int kSmx = kSmxWarps * 32;
constexpr int kMmaWarp = kSmxWarps, kPvWarp = kMmaWarp + 1, kScaleWarp = kMmaWarp + 2, kConvWarp = kMmaWarp + 3;
constexpr int kConv = 128;                 // converter threads per operand
constexpr int kThreads = kConvWarp * 32 + 2 * kConv;
constexpr int KP = CK / 4;                 // keys per softmax part
constexpr int kSc = 2 * CK + 4;            // a chunk's scales: ks [64], vs' or log2 vs [64], (narrow, E)
// The reference of a row's contributions is set kLift below the largest one and
// moves once one exceeds it by kTop.  fp16 holds c in steps of 2^-24 at the bottom,
// an error of 2^-25 at most, so in units of the largest contribution each is off by
// at most 2^-(25 + kLift): n of them, all of the same sign, by n times that (the row
// sum counts what they lose).  kTileRefKeys (int8.h) bounds n.  At the top c stays below
// 2^(kTop + 1 + kSpread), in fp16.
constexpr float kLift = 3.f, kTop = 11.f;
constexpr int kSpread = 3;                 // of a narrow chunk's value scales, see the scale warp
constexpr long long kDrainNs = 4000000000LL;

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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

// Bytes 0, 1 (sel 0x4140) or 2, 3 (0x4342) of codes ^ 0x80 -> fp16x2, exactly:
// 0x6400 | u is 1024 + u, u = code + 128.
__device__ __forceinline__ uint32_t biased_f16x2(uint32_t u, uint32_t sel) {
  const uint32_t w = __byte_perm(u, 0x64646464u, sel);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&w), __floats2half2_rn(1152.f, 1152.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// OR over the 128 threads of the four warps that share 32 rows.
__device__ __forceinline__ bool rows_or(int id, bool v) {
  __syncwarp();
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}
// AND over them.
__device__ __forceinline__ bool rows_and(int id, bool v) {
  __syncwarp();
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}

// D[tmem] (+)= A B^T, bf16, descriptors as (low word, common high word).  The
// accumulate flag is a compile-time constant, so an MMA costs little more than
// its own issue.
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Offsets of the rows r, r + step, ... (row = query * group + head) of a
// [token][head] layout: two divisions and products for all of them (per 16-byte
// chunk they made the first and last phases of a tile 5000 cycles longer).
struct RowWalk {
  long long at, step, wrap;
  int hl, dh, group;
  __device__ __forceinline__ RowWalk(int r, int rows_apart, int g, long long tok, long long head) : group(g) {
    const int qi = (int)((unsigned)r / (unsigned)g), dq = (int)((unsigned)rows_apart / (unsigned)g);
    hl = r - qi * g;
    dh = rows_apart - dq * g;
    at = qi * tok + hl * head;
    step = dq * tok + dh * head;
    wrap = tok - g * head;
  }
  __device__ __forceinline__ void next() {
    at += step;
    hl += dh;
    if (hl >= group) {
      hl -= group;
      at += wrap;
    }
  }
};

template <int D>
struct Smem {
  static constexpr uint32_t kTile = CK * D * 2;  // one chunk of K (or V) in bf16
  static constexpr uint32_t q = 0, k = QROWS * D * 2, v = k + 2 * kTile, sc = v + 2 * kTile;
  static constexpr uint32_t pm = sc + 2 * kSc * 4;
  static constexpr uint32_t l = pm + 4 * QROWS * 4;      // partial maxima [4][128]
  static constexpr uint32_t bar = l + 4 * QROWS * 4;     // partial sums [4][128]
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
  uint64_t* sc_full = bars + 15;    // [2] the chunk's scales in place
  uint64_t* drain = bars + 17;      // [2] one per MMA warp
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 19);
  volatile int* s_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* s_sc = reinterpret_cast<float*>(smem + L::sc);
  float* s_pm = reinterpret_cast<float*>(smem + L::pm);
  float* s_l = reinterpret_cast<float*>(smem + L::l);

  // (a shuffle tells the compiler that the warp index is the same in all lanes)
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
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
      mbar_init(&sc_full[i], 32);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    s_flag[0] = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
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
  // (a power of two splits; as 64-bit divisions by all threads the two took 1000
  // cycles)
  const int sh = 31 - __clz(splits);
  const int c0 = (int)(((unsigned long long)(nc + nf) * split) >> sh), c1 = (int)(((unsigned long long)(nc + nf) * (split + 1)) >> sh);
  const int nch = c1 - c0;

  if (warp >= kConvWarp) {
    // ------------------------------------------------------------ converters
    // A warp's 16-byte pieces cover 8 rows x 64 channels: lane = 4 row + piece.
    // Rows of different parity land in different halves of the swizzled 128-byte
    // rows, so the two 16-byte stores of 8 lanes touch all banks once.
    const bool is_v = warp >= kConvWarp + 4;
    const int cw = (warp - kConvWarp) & 3;               // warp within the operand's four
    const int cp = lane & 3, rl = lane >> 2;
    constexpr int UNITS = NBOX * 8 / 4;                  // (box, 8 rows) units per warp
    const size_t base = ((size_t)b * a.c.heads + h) * a.c.cap;
    const int8_t* src = (is_v ? a.c.v : a.c.k) + base * D;
    const bf16* fresh = is_v ? a.v_new : a.k_new;
    const long long f_tok = is_v ? a.vn_tok : a.kn_tok;
    if (fresh) fresh += b * (is_v ? a.vn_seq : a.kn_seq) + (long long)h * (is_v ? a.vn_head : a.kn_head);
    uint64_t* full = is_v ? v_full : k_full;
    uint64_t* empty = is_v ? v_empty : k_empty;
    const uint32_t tile0 = smem_u32(smem + (is_v ? L::v : L::k));
    // unit u of this warp: box box0, rows row0 + 8 u
    const int box0 = cw * UNITS >> 3, row0 = (cw * UNITS & 7) * 8 + rl;
    const int8_t* src0 = src + (size_t)row0 * D + box0 * 64 + cp * 16;
    const uint32_t dst0 = tile0 + (uint32_t)(box0 * CK * 128 + row0 * 128);
    const uint32_t sw0 = (uint32_t)((2 * cp) ^ rl) << 4, sw1 = (uint32_t)((2 * cp + 1) ^ rl) << 4;
    uint4 raw[UNITS];
    auto load = [&](int c) {  // a cached chunk's codes
      const int key0 = c * CK;
      const int8_t* p = src0 + (size_t)key0 * D;
      if (key0 + CK <= seen) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) raw[u] = __ldg(reinterpret_cast<const uint4*>(p + u * 8 * D));
      } else {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          raw[u] = make_uint4(0, 0, 0, 0);
          if (key0 + row0 + 8 * u < seen) raw[u] = __ldg(reinterpret_cast<const uint4*>(p + u * 8 * D));
        }
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
      const uint32_t dst = dst0 + (uint32_t)slot * L::kTile;
      if (c < nc && is_v) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const uint32_t at = dst + u * 8 * 128;
          const uint32_t w[4] = {raw[u].x ^ 0x80808080u, raw[u].y ^ 0x80808080u, raw[u].z ^ 0x80808080u, raw[u].w ^ 0x80808080u};
          uint32_t o[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            o[2 * q] = biased_f16x2(w[q], 0x4140);
            o[2 * q + 1] = biased_f16x2(w[q], 0x4342);
          }
          sts128(at + sw0, o[0], o[1], o[2], o[3]);
          sts128(at + sw1, o[4], o[5], o[6], o[7]);
        }
      } else if (c < nc) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const uint32_t at = dst + u * 8 * 128;
          const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
          uint32_t o[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            o[2 * q] = bytes_bf16x2(__byte_perm(w[q], 0, 0x4140));
            o[2 * q + 1] = bytes_bf16x2(__byte_perm(w[q], 0, 0x4342));
          }
          sts128(at + sw0, o[0], o[1], o[2], o[3]);
          sts128(at + sw1, o[4], o[5], o[6], o[7]);
        }
      } else {
        const int t0 = (c - nc) * CK;
#pragma unroll 4
        for (int u = 0; u < UNITS; ++u) {
          const int row = row0 + 8 * u;
          const uint32_t at = dst + u * 8 * 128;
          uint4 x = make_uint4(0, 0, 0, 0), y = x;
          if (t0 + row < a.n_new) {
            const bf16* p = fresh + (long long)(t0 + row) * f_tok + box0 * 64 + cp * 16;
            x = *reinterpret_cast<const uint4*>(p);
            y = *reinterpret_cast<const uint4*>(p + 8);
          }
          sts128(at + sw0, x.x, x.y, x.z, x.w);
          sts128(at + sw1, y.x, y.y, y.z, y.w);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&full[slot]);
      if (i + 1 < nch && c + 1 < nc) load(c + 1);
    }
  } else if (warp == kScaleWarp) {
    // ---------------------------------------------------------------- scales
    // lane l: key and value scales of keys l and l + 32, the next chunk's in
    // flight; a slot is written again only after its chunk's PV
    const size_t base = ((size_t)b * a.c.heads + h) * a.c.cap;
    //
    // A chunk whose value scales lie within a factor 8 of one another takes the
    // smallest one's exponent E for all: c = exp2(s ks + E - ref) vs', vs' =
    // vs / 2^E in [1, 16) (c stays below 2^15), and the exponentials serve the
    // row sums too.  Others take log2 vs
    // key by key, so that a large row that a query does not see or weigh, or a
    // zero one that it weighs most, costs the others nothing.  So do chunks that
    // some of the tile's queries see in part: no bit of a result may depend on a
    // key behind the query.
    const int all_see = a.causal ? (len - a.n_q + 1 + qt * QROWS / a.group) & ~(CK - 1) : INT_MAX;
    float k[2], v[2];
    auto load = [&](int c) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int at = lane + 32 * j;
        const bool in = c < nc ? c * CK + at < seen : (c - nc) * CK + at < a.n_new;
        k[j] = !in ? 0.f : c < nc ? __ldg(a.c.k_scale + base + c * CK + at) * a.scale_log2 : a.scale_log2;
        v[j] = !in ? -0.f : c < nc ? __ldg(a.c.v_scale + base + c * CK + at) : 1.f;
      }
    };
    if (nch > 0) load(c0);
    for (int i = 0; i < nch; ++i) {
      const int slot = i & 1;
      if (!__all_sync(0xffffffffu, i < 2 || mbar_wait(&o_done[slot], ((i >> 1) & 1) ^ 1, a.err.wait_ns))) {
        s_flag[0] = 1;
        set_error(a.err, DEV_TIMEOUT);
        break;
      }
      // exponents of the largest and the smallest scale (bits of non-negative
      // floats sort as integers; NaN above all, -0 marks a place without a key)
      const uint32_t b0 = __float_as_uint(v[0]), b1 = __float_as_uint(v[1]);
      const int hi = (int)(__reduce_max_sync(0xffffffffu, max(b0 & 0x7FFFFFFFu, b1 & 0x7FFFFFFFu)) >> 23);
      const int lo = (int)(__reduce_min_sync(0xffffffffu, min(b0, b1)) >> 23);
      const bool narrow = hi < 254 && lo > 0 && hi - lo <= kSpread && (c0 + i) * CK < all_see;
      const int e = narrow ? lo - 127 : 0;
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-E (-126 <= E <= 126)
      float* sl = s_sc + slot * kSc;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int at = lane + 32 * j;
        sl[at] = k[j];
        sl[CK + at] = narrow ? v[j] * down : __log2f(v[j]);  // (0, with codes 0: -inf)
      }
      if (lane == 0) *reinterpret_cast<float2*>(sl + 2 * CK) = make_float2(narrow ? 1.f : 0.f, (float)e);
      mbar_arrive(&sc_full[slot]);
      if (i + 1 < nch) load(c0 + i + 1);
    }
  } else if (warp == kMmaWarp || warp == kPvWarp) {
    // ------------------------------------------------------------------- MMA
    // A whole warp walks the loop and one lane issues (the same one each time):
    // addresses then live in uniform registers.  Issued from a one-lane branch,
    // the 20 MMAs of a chunk took 1900 cycles.
    if (nch > 0) {
      bool good = true;
      if (warp == kMmaWarp) {
        constexpr uint32_t idesc_s = idesc_bf16(QROWS, CK);
        const uint64_t q_desc = sw128_desc(smem_u32(smem + L::q), 16, 1024);
        const uint64_t k_desc = sw128_desc(smem_u32(smem + L::k), 16, 1024);
        const uint32_t q_lo = (uint32_t)q_desc, k_lo = (uint32_t)k_desc, hi = (uint32_t)(q_desc >> 32);
        good = __all_sync(0xffffffffu, mbar_wait(q_full, 0, a.err.wait_ns));
        for (int i = 0; good && i < nch; ++i) {
          const int st = i & 1;
          // S of chunk i goes over P of chunk i - 2: that chunk's PV must be done
          good = mbar_wait(&k_full[st], (i >> 1) & 1, a.err.wait_ns) &&
                 (i < 2 || mbar_wait(&o_done[st], ((i >> 1) & 1) ^ 1, a.err.wait_ns));
          if (!(good = __all_sync(0xffffffffu, good))) break;
          tc_fence_after();
          const uint32_t d = tmem + (uint32_t)(st * CK), kl = k_lo + (uint32_t)st * (L::kTile >> 4);
          if (elect_one()) {
            mma_ss<false>(d, q_lo, kl, hi, idesc_s);
#pragma unroll
            for (uint32_t k16 = 1; k16 < D / 16; ++k16) {
              const uint32_t x = k16 >> 2, w = (k16 & 3u) * 32u;
              mma_ss<true>(d, q_lo + ((x * QROWS * 128u + w) >> 4), kl + ((x * CK * 128u + w) >> 4), hi, idesc_s);
            }
            umma_commit(&s_full[st]);
            umma_commit(&k_empty[st]);
          }
          __syncwarp();
        }
      } else {
        constexpr uint32_t idesc_new = idesc_bf16(QROWS, D, 0, 1);
        constexpr uint32_t idesc_old = idesc_new & ~((7u << 7) | (7u << 10));  // A and B fp16 (format 0)
        const uint64_t v_desc = sw128_desc(smem_u32(smem + L::v), CK * 128, 1024);
        const uint32_t v_lo = (uint32_t)v_desc, hi = (uint32_t)(v_desc >> 32);
        for (int i = 0; good && i < nch; ++i) {
          const int st = i & 1;
          good = mbar_wait(&v_full[st], (i >> 1) & 1, a.err.wait_ns) && mbar_wait(&p_full[st], (i >> 1) & 1, a.err.wait_ns);
          if (!(good = __all_sync(0xffffffffu, good))) break;
          tc_fence_after();
          const uint32_t idesc_o = c0 + i < nc ? idesc_old : idesc_new;
          const uint32_t p = tmem + (uint32_t)(st * CK), vl = v_lo + (uint32_t)st * (L::kTile >> 4);
          if (elect_one()) {
            mma_ts(t_o, p, vl, hi, idesc_o, i > 0 ? 1u : 0u);
#pragma unroll
            for (uint32_t k16 = 1; k16 < CK / 16; ++k16) mma_ts(t_o, p + k16 * 8u, vl + ((k16 * 16u * 128u) >> 4), hi, idesc_o, 1u);
            umma_commit(&o_done[st]);
            umma_commit(&v_empty[st]);
          }
          __syncwarp();
        }
      }
      if (!good) {
        s_flag[0] = 1;
        set_error(a.err, DEV_TIMEOUT);
      }
      // every MMA issued must finish before TMEM is freed
      if (elect_one()) {
        umma_commit(&drain[warp - kMmaWarp]);
        if (!mbar_wait(&drain[warp - kMmaWarp], 0, kDrainNs)) set_error(a.err, DEV_DRAIN);
      }
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- softmax
    if (nch > 0) {
      // Q tile: 16-byte chunks, all of a thread's in flight at once; rows past
      // the last are zeros
      constexpr int NQ = QROWS * D / 8 / kSmx, STEP = kSmx / (D / 8);  // rows from one of a thread's chunks to the next
      const uint32_t q0 = smem_u32(smem + L::q);
      uint4 x[NQ];
      RowWalk walk(qt * QROWS + (int)threadIdx.x / (D / 8), STEP, a.group, a.q_tok, a.q_head);
      const bf16* qp = a.q + b * a.q_seq + h * a.group * a.q_head + (threadIdx.x % (D / 8)) * 8;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);
        if (qt * QROWS + (int)threadIdx.x / (D / 8) + i * STEP < rows) x[i] = __ldg(reinterpret_cast<const uint4*>(qp + walk.at));
        walk.next();
      }
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int e = threadIdx.x + i * kSmx, row = e / (D / 8), ch = e % (D / 8);
        sts128(q0 + (uint32_t)((ch >> 3) * QROWS * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4)), x[i].x, x[i].y, x[i].z, x[i].w);
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full);
    }
    const int part = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int rq = qt * QROWS + r;
    const int oc0 = part * (D / 4);
    const int lim = a.causal ? min(len, len - a.n_q + 1 + min(rq, rows - 1) / a.group) : len;
    float ref = 0.f;               // reference of c, the row's, in the log2 domain; has: some key was visible
    float xref = 0.f, l_run = 0.f; // the sum's, this part's of the row (k_i8_attn.cu says why they differ)
    bool ok = true, has = false, xhas = false;
    for (int i = 0; i < nch; ++i) {
      const int st = i & 1, c = c0 + i;
      const bool got = mbar_wait(&sc_full[st], (i >> 1) & 1, a.err.wait_ns) &&
                       mbar_wait(&s_full[st], (i >> 1) & 1, a.err.wait_ns);
      __syncwarp();
      tc_fence_after();
      float sv[KP];
      tmem_ld16(tmem + (uint32_t)(st * CK) + lane_off + part * KP, sv);
      tmem_ld_wait();
      reg_fence16(sv);
      const float* sc = s_sc + st * kSc + part * KP;
      const float2 ch = *reinterpret_cast<const float2*>(s_sc + st * kSc + 2 * CK);
      const bool narrow = ch.x != 0.f;
      // visible keys of this part's
      const int vis = (c < nc ? lim - c * CK : a.n_new - (c - nc) * CK) - part * KP;
      // Exponents in units of the row's reference: y = s ks + E - ref.  The reference
      // moves only when an exponent of c exceeds it by more than kTop, a factor 256
      // above where it was set, so that O is rescaled rarely; until then no part
      // needs another part's maximum, only everyone's word that it stays.
      float2* s2 = reinterpret_cast<float2*>(sv);
      const float2 nref = make_float2(ch.y - ref, ch.y - ref);
#pragma unroll
      for (int j = 0; j < KP / 2; j += 2) {
        const float4 k4 = *reinterpret_cast<const float4*>(sc + 2 * j);
        s2[j] = fma2(s2[j], make_float2(k4.x, k4.y), nref);
        s2[j + 1] = fma2(s2[j + 1], make_float2(k4.z, k4.w), nref);
      }
      if (vis < KP) {
#pragma unroll
        for (int j = 0; j < KP; ++j) sv[j] = j < vis ? sv[j] : -INFINITY;
      }
      float mt[KP / 4];
#pragma unroll
      for (int j = 0; j < KP / 4; ++j) mt[j] = fmaxf(max3(sv[4 * j], sv[4 * j + 1], sv[4 * j + 2]), sv[4 * j + 3]);
      float xmax = fmaxf(max3(mt[0], mt[1], mt[2]), mt[3]), pmax = xmax;
      if (!narrow) {
        pmax = -INFINITY;
#pragma unroll
        for (int j = 0; j < KP; ++j) pmax = fmaxf(pmax, j < vis ? sv[j] + sc[CK + j] : -INFINITY);
      }
      // Every part of the rows has its scores in registers (P overwrites S).
      // A part that must stop asks for a move too, so all meet below.
      const bool mine = got && s_flag[0] == 0;
      float alpha = 1.f;
      if (rows_or(1 + (warp & 3), !mine || (has ? pmax > kTop : pmax != -INFINITY))) {
        float* pm = s_pm + r;
        pm[part * QROWS] = pmax;
        if (!rows_and(1 + (warp & 3), mine)) {
          ok = false;
          break;
        }
        const float cmax = fmaxf(max3(pm[0], pm[QROWS], pm[2 * QROWS]), pm[3 * QROWS]);
        const bool move = has ? cmax > kTop : cmax != -INFINITY;  // (NaN alone: the reference stays)
        const float up = move && cmax == cmax ? cmax - kLift : 0.f;
        ref += up;
        xmax -= up;
        alpha = has ? ex2(-up) : 1.f;
        has = has || move;
        const float2 nup = make_float2(-up, -up);
#pragma unroll
        for (int j = 0; j < KP / 2; ++j) s2[j] = add2(s2[j], nup);
        rows_and(1 + (warp & 3), true);  // the maxima are read: the next move may write them
      }
      // The sum: 2^(y + f) in units of its own reference, which moves when a
      // score exceeds it by 64 (fp32 holds both sides).
      float f = ref - ch.y - xref;
      const bool far = xmax > -INFINITY && (!xhas || xmax + f > 64.f);
      if (__any_sync(0xffffffffu, far)) {
        if (far) {
          if (xhas) l_run *= ex2(-(xmax + f));
          xref += xmax + f;
          f = -xmax;
          xhas = true;
        }
      }
      // A narrow chunk's exponentials serve both sums, but for rows to which the
      // chunk's largest contribution is next to nothing, though its weight may not be.
      const bool shared = narrow && !__any_sync(0xffffffffu, xmax < -60.f && xmax > -INFINITY);
      if (!shared) {
#pragma unroll
        for (int j = 0; j < KP; ++j) l_run += ex2(sv[j] + f);
      }
      if (narrow) {
#pragma unroll
        for (int j = 0; j < KP / 2; ++j) {
          s2[j].x = ex2(s2[j].x);
          s2[j].y = ex2(s2[j].y);
        }
        if (shared) {
          float2 sum[2] = {s2[0], s2[1]};
#pragma unroll
          for (int j = 2; j < KP / 2; ++j) sum[j & 1] = add2(sum[j & 1], s2[j]);
          sum[0] = add2(sum[0], sum[1]);
          l_run += (sum[0].x + sum[0].y) * ex2(fminf(f, 126.f));  // (f <= 124 unless the part sees no key)
        }
#pragma unroll
        for (int j = 0; j < KP / 2; j += 2) {
          const float4 v4 = *reinterpret_cast<const float4*>(sc + CK + 2 * j);
          s2[j] = mul2(s2[j], make_float2(v4.x, v4.y));
          s2[j + 1] = mul2(s2[j + 1], make_float2(v4.z, v4.w));
        }
      } else {  // masked places stay 0 whatever their scale is
#pragma unroll
        for (int j = 0; j < KP; ++j) sv[j] = j < vis ? ex2(sv[j] + sc[CK + j]) : 0.f;
      }
      const bool scale_o = i > 0 && alpha != 1.f;
      uint32_t pk[KP / 2];
      if (c < nc) {
#pragma unroll
        for (int j = 0; j < KP / 2; ++j) pk[j] = pack_f16(sv[2 * j], sv[2 * j + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < KP / 2; ++j) pk[j] = pack_bf16(sv[2 * j], sv[2 * j + 1]);
      }
      tmem_st8u(tmem + (uint32_t)(st * CK) + lane_off + part * (KP / 2), pk);
      if (__any_sync(0xffffffffu, scale_o)) {
        // O may be rescaled only once PV of the previous chunk has landed in it
        const bool good = __all_sync(0xffffffffu, mbar_wait(&o_done[st ^ 1], ((i - 1) >> 1) & 1, a.err.wait_ns));
        if (good) {
          const float f = scale_o ? alpha : 1.f;
          tc_fence_after();
          for (int jj = oc0; jj < oc0 + D / 4; jj += 16) {
            float ov[16];
            tmem_ld16(t_o + lane_off + jj, ov);
            tmem_ld_wait();
            reg_fence16(ov);
#pragma unroll
            for (int t = 0; t < 16; ++t) ov[t] *= f;
            tmem_st16(t_o + lane_off + jj, ov);
          }
        } else {
          s_flag[0] = 1;
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[st]);
    }
    if (!ok) set_error(a.err, DEV_TIMEOUT);
    // PVs complete in issue order: the last chunk's commit covers them all
    if (nch > 0 && ok) ok = mbar_wait(&o_done[(nch - 1) & 1], ((nch - 1) >> 1) & 1, kDrainNs);
    s_l[part * QROWS + r] = l_run;
    s_pm[part * QROWS + r] = xhas ? xref : -INFINITY;
    ok = rows_and(1 + (warp & 3), ok && s_flag[0] == 0);
    tc_fence_after();
    // the parts' sums in units of their largest reference X; a part without one
    // has 0, or NaN of NaN scores alone
    const float X = fmaxf(fmaxf(s_pm[r], s_pm[QROWS + r]), fmaxf(s_pm[2 * QROWS + r], s_pm[3 * QROWS + r]));
    float l = 0.f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float x = s_pm[p * QROWS + r];
      l += x == -INFINITY ? s_l[p * QROWS + r] : s_l[p * QROWS + r] * ex2(x - X);
    }
    const float lw = X == -INFINITY ? l : X + __log2f(l);
    // O in units of 2^ref -> the average over the keys; no visible key, or none
    // with a value (ref is then not set, O is 0, or NaN of a NaN value scale): zeros
    // 2^(ref - lw) may be below fp32 where the average is not: its root, twice
    const float root = l == 0.f || (!has && l == l) ? 0.f : ex2(0.5f * (ref - lw - (splits > 1 ? kPartShift : 0.f)));
    // Output rows go through shared memory (every MMA is done: the tiles are
    // free), so that a row leaves as one run of 16-byte stores; straight from
    // the registers, a warp's store touches 32 rows and the 128 rows of a tile
    // took 7000 cycles.  Chunks of 16 bytes are swizzled by the row.
    const size_t pr0 = ((size_t)bg * splits + split) * ((size_t)gridDim.x * QROWS) + qt * QROWS;
    if (splits > 1 && part == 0) a.part_ml[pr0 + r] = part_weight(ok && l != 0.f ? lw : -INFINITY);
    const uint32_t stage = smem_u32(smem);
    const int esz = splits == 1 ? 2 : 4;
    const uint32_t rowb = (uint32_t)(D * esz), srow = stage + (uint32_t)r * rowb;
#pragma unroll
    for (int j = 0; j < D / 4; j += 16) {
      float ov[16];
      if (ok && nch > 0) {
        tmem_ld16(t_o + lane_off + oc0 + j, ov);
        tmem_ld_wait();
        reg_fence16(ov);
      } else {
#pragma unroll
        for (int t = 0; t < 16; ++t) ov[t] = 0.f;
      }
#pragma unroll
      for (int t = 0; t < 16; ++t) ov[t] = ov[t] * root * root;
      if (splits == 1) {
        const uint32_t ch = (uint32_t)(oc0 + j) / 8;
#pragma unroll
        for (int t = 0; t < 2; ++t)
          sts128(srow + (((ch + t) ^ (r & 7)) << 4), pack_bf16(ov[8 * t], ov[8 * t + 1]),
                 pack_bf16(ov[8 * t + 2], ov[8 * t + 3]), pack_bf16(ov[8 * t + 4], ov[8 * t + 5]),
                 pack_bf16(ov[8 * t + 6], ov[8 * t + 7]));
      } else {
        const uint32_t ch = (uint32_t)(oc0 + j) / 4;
#pragma unroll
        for (int t = 0; t < 4; ++t)
          sts128(srow + (((ch + t) ^ (r & 7)) << 4), __float_as_uint(ov[4 * t]), __float_as_uint(ov[4 * t + 1]),
                 __float_as_uint(ov[4 * t + 2]), __float_as_uint(ov[4 * t + 3]));
      }
    }
    ok = rows_and(1 + (warp & 3), ok);
    if (ok) {
      // the four warps of these 32 rows take 8 rows each
      const int base = (warp & 3) * 32 + part * 8;
      if (splits == 1) {
        constexpr int CPR = D / 8, STEP = 32 / CPR;  // 16-byte chunks per row, rows per warp-wide store
        RowWalk walk(qt * QROWS + base + lane / CPR, STEP, a.group, a.o_tok, a.o_head);
        bf16* op = a.o + b * a.o_seq + h * a.group * a.o_head + (lane % CPR) * 8;
#pragma unroll
        for (int i = 0; i < 8 / STEP; ++i) {
          const int row = base + lane / CPR + i * STEP, ch = lane % CPR;
          const uint4 x = lds128(stage + (uint32_t)row * rowb + (uint32_t)((ch ^ (row & 7)) << 4));
          if (qt * QROWS + row < rows) *reinterpret_cast<uint4*>(op + walk.at) = x;
          walk.next();
        }
      } else {
        constexpr int CPR = D / 4;
#pragma unroll
        for (int e = 0; e < 8 * CPR; e += 32) {
          const int row = base + (e + lane) / CPR, ch = (e + lane) % CPR;
          const uint4 x = lds128(stage + (uint32_t)row * rowb + (uint32_t)((ch ^ (row & 7)) << 4));
          if (qt * QROWS + row < rows) *reinterpret_cast<uint4*>(a.part_o + (pr0 + row) * D + ch * 4) = x;
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, ncols);
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
