// Product of 8-bit integer matrices with one scale per token and per output
// channel:
//   y[t][f] = (sum_k x[t][k] w[f][k]) sx[t] sw[f]
// on the tcgen05 tensor cores (kind::i8: signed 8-bit operands, 32-bit sums in
// TMEM).  The sums are exact for k <= 131071 (|code| <= 128), so any order
// and any split of k gives the same bits; the two scales are applied in fp32
// and the result is rounded once to the output type.
//
// Two forms of one tile product D[128 rows][tn columns], chosen by the number
// of tokens:
//   tokens on the rows   (many tokens) a persistent grid walks the tiles; the
//                        accumulator is double-buffered in TMEM, so the
//                        epilogue of a tile runs under the next one's MMAs.
//                        Where filling shared memory bounds the loop (8-bit
//                        MMAs eat 96 bytes per cycle of a 128 x 256 tile, an
//                        SM gets about 64 from L2), two CTAs share a tile of
//                        256 rows (cta_group::2): each brings 128 token rows
//                        and half of the weight rows, 64 bytes per cycle
//   weights on the rows  (few tokens: streaming the weights is what bounds
//                        it) tokens pad only to a multiple of 16; tiles of 32
//                        to 128 weight rows spread the weights over the SMs,
//                        and where those are too few the k range of a tile is
//                        split over a cluster of CTAs so that all
//                        SMs stream weights, and the int32 partials are summed
//                        through distributed shared memory
// Warp 0 streams both operands by TMA in 128-byte k blocks (128-byte swizzle)
// through a ring of stages, warp 1 issues the MMAs (K = 32 codes each), the
// warps from 4 on read the accumulator (thread = TMEM lane = row).
#include <algorithm>

#include "int8.h"
#include "launch.cuh"

namespace pae {

namespace {

constexpr long long kDrainNs = 4000000000LL;
constexpr int KB = 128;  // k block: one 128-byte swizzled row

// D[tmem] (+)= A[smem] B[smem]^T, signed 8-bit inputs, int32 accumulate.
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::i8: D format [4,6) = 2 (s32), A [7,10) = B
// [10,13) = 1 (signed), both K-major, N>>3 at [17,23), M>>4 at [24,29).
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld16i(uint32_t taddr, int* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void reg_fence16i(int* v) {
  asm volatile(""
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]));
}

__host__ __device__ inline uint32_t stage_bytes(int tn) { return 128u * KB + (uint32_t)tn * KB; }

__host__ __device__ inline uint32_t tmem_cols(int n) {
  uint32_t c = 32;
  while ((int)c < n) c <<= 1;
  return c;
}

// Shared memory: ring | output boxes | barriers | per-tile column scales | int32 partials.
struct I8Smem {
  uint32_t out_off, bar_off, sw_off, part_off, total;
};
__host__ __device__ inline I8Smem i8_layout(const I8GemmPlan& p) {
  I8Smem L;
  L.out_off = stage_bytes(p.swap ? p.tn : p.tn / p.cg) * (uint32_t)p.stages;  // output boxes: 8 warps x 4 KB
  L.bar_off = L.out_off + (p.swap ? 0u : 32768u);
  L.sw_off = L.bar_off + 512;
  L.part_off = L.sw_off + 2 * 256 * 4;
  L.total = L.part_off + (p.swap && p.splits > 1 ? 128u * (uint32_t)p.tn * 4u : 0u) + 1024;
  return L;
}

// Results are (sum sx) sw: in this order a product of the scales alone, which may
// be subnormal, does not occur.  A sum times a token scale above 2^64 could overflow
// where the result does not: such a scale is split into x y, y = 2^64, and the
// result is (sum x) sw y.  Both steps with y are exact.
__device__ __forceinline__ float2 token_scale(float sx) {
  return fabsf(sx) > 0x1p64f ? make_float2(sx * 0x1p-64f, 0x1p64f) : make_float2(sx, 1.f);
}

template <typename TO>
__device__ __forceinline__ void st_out(TO* p, float v);
template <>
__device__ __forceinline__ void st_out<float>(float* p, float v) { *p = v; }
template <>
__device__ __forceinline__ void st_out<bf16>(bf16* p, float v) { *p = f2bf(v); }

// 16 consecutive outputs of one row; `n` of them exist.
__device__ __forceinline__ void store16(float* p, const float* v, int n, bool vec) {
  if (vec && n >= 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store16(bf16* p, const float* v, int n, bool vec) {
  if (vec && n >= 16) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = (uint32_t)__bfloat16_as_ushort(f2bf(v[2 * i])) | ((uint32_t)__bfloat16_as_ushort(f2bf(v[2 * i + 1])) << 16);
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = f2bf(v[i]);
  }
}

// ------------------------------------------------------- tokens on the rows
// cta_group::2 forms: the MMA and its commit are issued by rank 0 of the pair;
// the loads of both CTAs complete on rank 0's barrier.
__device__ __forceinline__ void umma_i8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs once the MMAs so far finish.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Wait on an own barrier that the peer CTA arrives at.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, long long limit_ns) {
  const unsigned long long t0 = globaltimer_ns();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((long long)(globaltimer_ns() - t0) > limit_ns) return false;
  }
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* tm, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tm)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}
constexpr int kEpiWarps = 8;  // epilogue warps: two per TMEM lane quarter, taking turns by box of columns
constexpr int kThreads = 128 + kEpiWarps * 32;
__device__ __forceinline__ bool bar_and_epi(int id, bool v) {
  __syncwarp();
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}

// Stage and phase of a ring position, stepped without divisions (the ring
// length is a run-time number, and both threads of the pipeline take a step
// every few hundred cycles).
struct RingPos {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++st == stages) {
      st = 0;
      ph ^= 1;
    }
  }
};

// CG CTAs per tile of 128 CG token rows x tn weight rows, neighbours along x (a
// cluster of 2 for pairs).  tmY: the output, boxes of 32 rows x 128
// bytes (only used with a.tma_out).
template <typename TO, int CG>
__global__ void __launch_bounds__(kThreads, 1)
    k_i8_gemm(const __grid_constant__ CUtensorMap tmR, const __grid_constant__ CUtensorMap tmC,
              const __grid_constant__ CUtensorMap tmY, const I8GemmPlan p, const I8GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const I8Smem L = i8_layout(p);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L.bar_off);
  uint64_t* empty = full + p.stages;
  uint64_t* acc_full = empty + p.stages;  // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2]
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* s_sw = reinterpret_cast<float*>(smem + L.sw_off);  // [2][256]
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0, first = blockIdx.x / CG, step = gridDim.x / CG;
  const int nkb = (a.k + KB - 1) / KB;
  const int tiles = p.tiles_m * p.tiles_n;
  const uint32_t ncols = tmem_cols(2 * p.tn);
  const int brows = p.tn / CG;                                   // weight rows this CTA brings
  const uint32_t sbytes = (uint32_t)(128 + brows) * KB;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], CG);
    }
    mbar_init(drain, 1);
    s_flag[0] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmR);
    tma_prefetch_desc(&tmC);
    if (a.tma_out) tma_prefetch_desc(&tmY);
  }
  if (warp == 2) {
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(ncols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(tmem_slot, ncols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // both CTAs' barriers are initialised
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();  // the token codes and scales come from the quantiser

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    RingPos r;
    int it = 0;
    bool good = true;
    for (int tile = first; tile < tiles && good; tile += step) {
      const int tm = tile % p.tiles_m, tn = tile / p.tiles_m;
      const int y_r = (tm * CG + rank) * 128, y_c = tn * p.tn + rank * brows;
      for (int kb = 0; kb < nkb; ++kb, ++it, r.next(p.stages)) {
        good = __all_sync(0xffffffffu, it < p.stages || mbar_wait(&empty[r.st], r.ph ^ 1, a.err.wait_ns));
        if (!good) {
          s_flag[0] = 1;
          set_error(a.err, DEV_TIMEOUT);
          break;
        }
        uint8_t* s = smem + (uint32_t)r.st * sbytes;
        if (elect_one()) {
          if constexpr (CG == 2) {
            const uint32_t bar = map_cluster(smem_u32(&full[r.st]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[r.st], 2 * sbytes);  // both CTAs' bytes
            tma_load_2d_pair(s, &tmR, kb * KB, y_r, bar);
            tma_load_2d_pair(s + 128 * KB, &tmC, kb * KB, y_c, bar);
          } else {
            mbar_arrive_expect_tx(&full[r.st], sbytes);
            tma_load_2d(s, &tmR, kb * KB, y_r, &full[r.st]);
            tma_load_2d(s + 128 * KB, &tmC, kb * KB, y_c, &full[r.st]);
          }
        }
        __syncwarp();
      }
    }
    // loads still in flight must land before this CTA may exit (the peer's land
    // on rank 0's barriers, and no CTA leaves before rank 0 has seen them)
    if (rank == 0 && lane == 0)
      for (int i = it > p.stages ? it - p.stages : 0; i < it; ++i)
        if (!mbar_wait(&full[i % p.stages], (i / p.stages) & 1, kDrainNs)) set_error(a.err, DEV_DRAIN);
  } else if (warp == 1 && rank == 0) {
    // ----------------------------------------------------------------- MMA
    const uint32_t idesc = idesc_i8(128 * CG, p.tn);
    const uint64_t a0 = sw128_desc(smem_u32(smem), 16, 1024), b0 = sw128_desc(smem_u32(smem) + 128 * KB, 16, 1024);
    RingPos r;
    int n = 0;
    bool good = true;
    for (int tile = first; tile < tiles && good; tile += step, ++n) {
      const int buf = n & 1;
      if (n >= 2) {
        const uint32_t par = ((n >> 1) & 1) ^ 1;
        good = CG == 2 ? mbar_wait_cluster(&acc_empty[buf], par, a.err.wait_ns) : mbar_wait(&acc_empty[buf], par, a.err.wait_ns);
        good = __all_sync(0xffffffffu, good);
      }
      const uint32_t d = tmem + buf * p.tn;
      for (int kb = 0; kb < nkb && good; ++kb, r.next(p.stages)) {
        good = __all_sync(0xffffffffu, mbar_wait(&full[r.st], r.ph, a.err.wait_ns));
        if (!good) break;
        tc_fence_after();
        const uint64_t ad = desc_add(a0, (uint32_t)r.st * sbytes), bd = desc_add(b0, (uint32_t)r.st * sbytes);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < KB / 32; ++kk) {
            const uint32_t acc = (kb | kk) != 0 ? 1u : 0u;
            if constexpr (CG == 2)
              umma_i8_pair(d, desc_add(ad, kk * 32u), desc_add(bd, kk * 32u), idesc, acc);
            else
              umma_i8(d, desc_add(ad, kk * 32u), desc_add(bd, kk * 32u), idesc, acc);
          }
          if constexpr (CG == 2) {
            umma_commit_pair(&empty[r.st]);
            if (kb == nkb - 1) umma_commit_pair(&acc_full[buf]);
          } else {
            umma_commit(&empty[r.st]);
            if (kb == nkb - 1) umma_commit(&acc_full[buf]);
          }
        }
        __syncwarp();
      }
    }
    if (!good) {
      s_flag[0] = 1;
      set_error(a.err, DEV_TIMEOUT);
    }
    // every MMA issued must finish before TMEM is freed (the elected lane is the
    // same one each time)
    if (elect_one()) {
      if constexpr (CG == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(drain)) : "memory");
      else
        umma_commit(drain);
      if (!mbar_wait(drain, 0, kDrainNs)) set_error(a.err, DEV_DRAIN);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    // Thread = row; the two warps of a lane quarter take the 128-byte boxes of
    // columns in turn.  A box goes through the warp's 4 KB buffer (32 rows,
    // swizzled) and leaves as one bulk tensor store, which clips at the matrix's
    // edges.  Outputs that a tensor map cannot describe leave from the registers in
    // 16-byte stores, or, where their rows start off 16 bytes, element by element
    // along the rows of the buffer (a lane's own row in single elements is 32 rows
    // per store: 3997 x 9999 x 1024: fp32 275 us so, 81 now; bf16 375 and 56).
    constexpr int CPB = 128 / (int)sizeof(TO), NB = CPB / 16;  // columns and 16-column chunks per box
    const int et = threadIdx.x - 128, half = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t box = smem_u32(smem + L.out_off) + (uint32_t)(warp - 4) * 4096u;
    TO* y = static_cast<TO*>(a.y);
    const bool vec = (reinterpret_cast<uintptr_t>(y) & 15) == 0 && (a.ldy * (long long)sizeof(TO)) % 16 == 0;
    const bool staged = a.tma_out || !vec;
    const int nc = p.tn / 16;
    int n = 0;
    for (int tile = first; tile < tiles; tile += step, ++n) {
      const int buf = n & 1;
      const int tm = tile % p.tiles_m, tn = tile / p.tiles_m;
      const int row0 = (tm * CG + rank) * 128, t = row0 + row, f0 = tn * p.tn;
      float* sw = s_sw + buf * 256;
      for (int i = et; i < p.tn; i += kEpiWarps * 32) sw[i] = f0 + i < a.n ? __ldg(a.sw + f0 + i) : 0.f;
      const float2 sx = token_scale(t < a.tokens ? a.sx[t] : 0.f);
      // the column scales are in place for all warps, and all go on or stop
      const bool got = mbar_wait(&acc_full[buf], (n >> 1) & 1, a.err.wait_ns);
      if (!bar_and_epi(1, got && s_flag[0] == 0)) {
        set_error(a.err, DEV_TIMEOUT);
        break;
      }
      tc_fence_after();
      const uint32_t acc0 = tmem + buf * p.tn + lane_off;
      for (int b0 = half * NB; b0 < nc; b0 += 2 * NB) {  // this warp's boxes
        int acc[NB][16];
#pragma unroll
        for (int i = 0; i < NB; ++i)
          if (b0 + i < nc) tmem_ld16i(acc0 + (b0 + i) * 16, acc[i]);
        if (a.tma_out) {
          // the store that last read the buffer is done reading
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        __syncwarp();
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < NB; ++i) reg_fence16i(acc[i]);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int c = b0 + i;
          if (c >= nc) break;
          float o[16];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 w = *reinterpret_cast<const float4*>(sw + c * 16 + 4 * q);
            o[4 * q] = (float)acc[i][4 * q] * sx.x * w.x * sx.y;
            o[4 * q + 1] = (float)acc[i][4 * q + 1] * sx.x * w.y * sx.y;
            o[4 * q + 2] = (float)acc[i][4 * q + 2] * sx.x * w.z * sx.y;
            o[4 * q + 3] = (float)acc[i][4 * q + 3] * sx.x * w.w * sx.y;
          }
          if (!staged) {
            if (t < a.tokens && f0 + c * 16 < a.n) store16(y + (size_t)t * a.ldy + f0 + c * 16, o, a.n - (f0 + c * 16), vec);
            continue;
          }
          const uint32_t rowp = box + (uint32_t)lane * 128u;
          if constexpr (sizeof(TO) == 2) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(o[8 * q + 2 * k], o[8 * q + 2 * k + 1]);
                w[k] = *reinterpret_cast<const uint32_t*>(&h);
              }
              sts128(rowp + (uint32_t)(((i * 2 + q) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              sts128(rowp + (uint32_t)(((i * 4 + q) ^ (lane & 7)) << 4), __float_as_uint(o[4 * q]),
                     __float_as_uint(o[4 * q + 1]), __float_as_uint(o[4 * q + 2]), __float_as_uint(o[4 * q + 3]));
          }
        }
        if (a.tma_out) {  // (tn is then a whole number of boxes)
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int x = f0 + b0 * 16, yr = row0 + (warp & 3) * 32;
            if (x < a.n && yr < a.tokens) tma_store_2d(&tmY, box, x, yr);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else if (staged) {  // row by row, element by element
          __syncwarp();
          const int rows = min(32, a.tokens - row0 - (warp & 3) * 32), cols = min(min(CPB, (nc - b0) * 16), a.n - f0 - b0 * 16);
          TO* yr = y + (size_t)(row0 + (warp & 3) * 32) * a.ldy + f0 + b0 * 16;
          for (int r = 0; r < rows; ++r, yr += a.ldy)
#pragma unroll
            for (int c = lane; c < CPB; c += 32) {
              const int at = c * (int)sizeof(TO);
              const TO v = *reinterpret_cast<const TO*>(smem + L.out_off + (warp - 4) * 4096 + r * 128 + ((((at >> 4) ^ (r & 7)) << 4) | (at & 15)));
              if (c < cols) yr[c] = v;
            }
          __syncwarp();
        }
      }
      // this CTA's epilogue warps are done with the accumulator
      tc_fence_before();
      bar_and_epi(2, true);
      if (et == 0) {
        if constexpr (CG == 2)
          mbar_arrive_cluster(map_cluster(smem_u32(&acc_empty[buf]), 0));
        else
          mbar_arrive(&acc_empty[buf]);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // every store has left shared memory
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // no CTA frees or leaves what the pair still uses
  if (warp == 2) {
    if constexpr (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(ncols) : "memory");
    else
      tmem_dealloc(tmem, ncols);
  }
}

// ------------------------------------------------------ weights on the rows
template <typename TO>
__global__ void __launch_bounds__(256, 1)
    k_i8_gemm_few(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const I8GemmPlan p,
                  const I8GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const I8Smem L = i8_layout(p);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L.bar_off);
  uint64_t* empty = full + p.stages;
  uint64_t* acc_full = empty + p.stages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* s_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float2* s_sx = reinterpret_cast<float2*>(smem + L.sw_off);  // [tn <= 64]
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int f0 = blockIdx.x * p.th, split = blockIdx.y, t0 = blockIdx.z * p.tn;
  const int nkb_all = (a.k + KB - 1) / KB;
  const int kb0 = (int)((long long)nkb_all * split / p.splits), kb1 = (int)((long long)nkb_all * (split + 1) / p.splits);
  const int nkb = kb1 - kb0;  // >= 1: the plan has splits <= k blocks
  const uint32_t ncols = tmem_cols(p.tn);
  const uint32_t sbytes = stage_bytes(p.tn);

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(acc_full, 1);
    s_flag[0] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, ncols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();

  if (warp == 0) {
    // Tiles of th < 128 weight rows fill the front of the A tile; the MMA's
    // remaining rows multiply whatever lies behind and are never read.
    const uint32_t tx = (uint32_t)(p.th + p.tn) * KB;
    if (!a.w_ready) pdl_wait();
    const int npre = min(nkb, p.stages);
    if (elect_one())
      for (int i = 0; i < npre; ++i) {
        mbar_arrive_expect_tx(&full[i], tx);
        tma_load_2d(smem + (uint32_t)i * sbytes, &tmW, (kb0 + i) * KB, f0, &full[i]);
      }
    __syncwarp();
    pdl_wait();
    if (elect_one())
      for (int i = 0; i < npre; ++i) tma_load_2d(smem + (uint32_t)i * sbytes + 128 * KB, &tmX, (kb0 + i) * KB, t0, &full[i]);
    __syncwarp();
    RingPos r;  // the stage of load npre + j is that of load j
    int it = npre;
    if (npre == p.stages)
      for (; it < nkb; ++it, r.next(p.stages)) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[r.st], r.ph, a.err.wait_ns))) {
          s_flag[0] = 1;
          set_error(a.err, DEV_TIMEOUT);
          break;
        }
        uint8_t* s = smem + (uint32_t)r.st * sbytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[r.st], tx);
          tma_load_2d(s, &tmW, (kb0 + it) * KB, f0, &full[r.st]);
          tma_load_2d(s + 128 * KB, &tmX, (kb0 + it) * KB, t0, &full[r.st]);
        }
        __syncwarp();
      }
    if (lane == 0)
      for (int i = it > p.stages ? it - p.stages : 0; i < it; ++i)
        if (!mbar_wait(&full[i % p.stages], (i / p.stages) & 1, kDrainNs)) set_error(a.err, DEV_DRAIN);
  } else if (warp == 1) {
    const uint32_t idesc = idesc_i8(128, p.tn);
    const uint64_t a0 = sw128_desc(smem_u32(smem), 16, 1024), b0 = sw128_desc(smem_u32(smem) + 128 * KB, 16, 1024);
    RingPos r;
    for (int it = 0; it < nkb; ++it, r.next(p.stages)) {
      if (!__all_sync(0xffffffffu, mbar_wait(&full[r.st], r.ph, a.err.wait_ns))) {
        s_flag[0] = 1;
        set_error(a.err, DEV_TIMEOUT);
        break;
      }
      tc_fence_after();
      const uint64_t ad = desc_add(a0, (uint32_t)r.st * sbytes), bd = desc_add(b0, (uint32_t)r.st * sbytes);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < KB / 32; ++kk)
          umma_i8(tmem, desc_add(ad, kk * 32u), desc_add(bd, kk * 32u), idesc, (it | kk) != 0 ? 1u : 0u);
        umma_commit(&empty[r.st]);
      }
      __syncwarp();
    }
    if (elect_one()) umma_commit(acc_full);  // always issued, so the epilogue's wait ends
  }
  __syncwarp();
  pdl_wait();
  const bool acc_ok = mbar_wait(acc_full, 0, kDrainNs);
  if (!acc_ok) set_error(a.err, DEV_DRAIN);
  tc_fence_after();
  for (int i = threadIdx.x; i < p.tn; i += 256) s_sx[i] = token_scale(t0 + i < a.tokens ? a.sx[t0 + i] : 0.f);
  const bool ok = __syncthreads_and(acc_ok ? 1 : 0) != 0 && s_flag[0] == 0;

  // warp w: TMEM lanes 32 (w % 4).. (features), 16-token chunks c with c % 2 == w / 4
  const int row = (warp & 3) * 32 + lane;
  const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  TO* y = static_cast<TO*>(a.y);
  const int nc = p.tn / 16;
  const int ntok = min(p.tn, a.tokens - t0);
  const bool mine = (warp & 3) * 32 < p.th;  // this warp's rows exist
  if (p.splits == 1) {
    const int f = f0 + row;
    const float sw = mine && f < a.n ? a.sw[f] : 0.f;
    if (ok && mine)
      for (int c = warp >> 2; c < nc; c += 2) {
        int v[16];
        tmem_ld16i(trow + c * 16, v);
        tmem_ld_wait();
        reg_fence16i(v);
        if (f < a.n) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c * 16 + j < ntok) {
              const float2 sx = s_sx[c * 16 + j];
              st_out(y + (size_t)(t0 + c * 16 + j) * a.ldy + f, (float)v[j] * sx.x * sw * sx.y);
            }
        }
      }
  } else {
    // partials [token][128 features] in this CTA's shared memory; rank r of the
    // cluster sums and writes features [r R, r R + R) of every token
    int* part = reinterpret_cast<int*>(smem + L.part_off);
    if (ok && mine)
      for (int c = warp >> 2; c < nc; c += 2) {
        int v[16];
        tmem_ld16i(trow + c * 16, v);
        tmem_ld_wait();
        reg_fence16i(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c * 16 + j) * 128 + row] = v[j];
      }
    cluster_sync();
    const int S = p.splits, R4 = p.th / S / 4;  // R / 4: groups of 4 features
    const int rank = (int)cluster_rank();
    if (ok) {
      for (int e = threadIdx.x; e < R4 * ntok; e += 256) {
        const int tok = e / R4, r = (rank * R4 + e % R4) * 4;
        const uint32_t at = smem_u32(part + tok * 128 + r);
        uint4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < S) v[q] = ld_cluster_u32x4(map_cluster(at, (uint32_t)q));
        uint4 sum = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < S) {
            sum.x += v[q].x;
            sum.y += v[q].y;
            sum.z += v[q].z;
            sum.w += v[q].w;
          }
        const int f = f0 + r;
        const int s4[4] = {(int)sum.x, (int)sum.y, (int)sum.z, (int)sum.w};
        const float2 sx = s_sx[tok];
        TO* yp = y + (size_t)(t0 + tok) * a.ldy + f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (f + i < a.n) st_out(yp + i, (float)s4[i] * sx.x * a.sw[f + i] * sx.y);
      }
    }
    cluster_sync();  // no rank leaves while another still reads its partials
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, ncols);
}

}  // namespace

// Tokens go to the N side while they fit one tile of at most 64: the weights
// are then read once and padding stays under 16 tokens.  With more, tokens on
// the rows; one or two CTAs per tile and the N tile are those whose waves over
// the 148 SMs cost least.
I8GemmPlan plan_i8_gemm(int tokens, int n, int k, int out_bytes) {
  I8GemmPlan p{};
  const int nkb = (k + KB - 1) / KB;
  p.splits = 1;
  p.cg = 1;
  if (tokens <= 64) {
    p.swap = 1;
    p.tn = std::max(16, (tokens + 15) / 16 * 16);
    // narrower tiles until they occupy most SMs, then split k
    p.th = 128;
    while (p.th > 32 && (n + p.th - 1) / p.th < 100) p.th /= 2;
    p.tiles_m = (n + p.th - 1) / p.th;
    p.tiles_n = 1;
    while (p.splits < 8 && p.splits * 2 <= nkb && p.tiles_m * p.splits * 2 <= 148) p.splits *= 2;
    const uint32_t part = p.splits > 1 ? 128u * (uint32_t)p.tn * 4u : 0u;
    p.stages = std::min({8, (nkb + p.splits - 1) / p.splits, (int)((196u * 1024u - part) / stage_bytes(p.tn))});
  } else {
    // Measured cycles (fit over tiles of 32 to 256 columns at 300 to 7743 tokens):
    // a k block costs its fill at about 60 bytes per cycle, or, for pairs, its
    // MMAs; a tile 1100 more; pairs 2000 once.  Tiles are whole 128-byte boxes of
    // the output wide (or 32), so that it can leave as bulk tensor stores.
    const int box = 128 / out_bytes;
    double best = 0;
    for (int cg = 1; cg <= 2; ++cg) {
      const int tm = (tokens + 128 * cg - 1) / (128 * cg), units = 148 / cg;
      for (int tn = 32; tn <= 256; tn += tn < box ? box - tn : box) {
        if (tn > 32 && tn - 32 >= n) break;
        const long long tiles = (long long)tm * ((n + tn - 1) / tn);
        const double kblock = cg == 1 ? 2.1 * (128 + tn) : std::max(2.2 * (128 + tn / 2), 2.85 * tn);
        const double cost = (double)((tiles + units - 1) / units) * (nkb * kblock + 1100.0) + (cg == 2 ? 2000.0 : 0.0);
        if (p.tn == 0 || cost < best * 0.999) {
          best = cost;
          p.tn = tn;
          p.cg = cg;
          p.tiles_m = tm;
        }
      }
    }
    p.tiles_n = (n + p.tn - 1) / p.tn;
    p.ctas = std::min(148 / p.cg, p.tiles_m * p.tiles_n);
    p.stages = std::min(8, (int)(160u * 1024u / stage_bytes(p.tn / p.cg)));
  }
  p.stages = std::max(2, p.stages);
  return p;
}

cudaError_t i8_gemm_init() {
  cudaError_t e = cudaSuccess;
  const int smem = 227 * 1024;
  auto set = [&](auto kern) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  };
  set(k_i8_gemm<float, 1>);
  set(k_i8_gemm<bf16, 1>);
  set(k_i8_gemm<float, 2>);
  set(k_i8_gemm<bf16, 2>);
  set(k_i8_gemm_few<float>);
  set(k_i8_gemm_few<bf16>);
  return e;
}

template <typename TO>
static cudaError_t i8_launch(const CUtensorMap& r, const CUtensorMap& c, const CUtensorMap& y, const I8GemmPlan& p,
                             const I8GemmArgs& a, cudaStream_t st) {
  const size_t smem = i8_layout(p).total;
  if (p.swap)
    return launch_ex(k_i8_gemm_few<TO>, dim3(p.tiles_m, p.splits, p.tiles_n), dim3(256), smem, st, p.splits, true, r,
                     c, p, a);
  if (p.cg == 1) return launch_ex(k_i8_gemm<TO, 1>, dim3(p.ctas), dim3(kThreads), smem, st, 1, true, r, c, y, p, a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;  // pairs lie along x
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_i8_gemm<TO, 2>, r, c, y, p, a);
}

cudaError_t launch_i8_gemm(bool out_bf16, const CUtensorMap* tm_rows, const CUtensorMap* tm_cols,
                           const CUtensorMap* tm_out, const I8GemmPlan& p, const I8GemmArgs& a, cudaStream_t st) {
  I8GemmArgs b = a;
  b.tma_out = tm_out != nullptr;
  const CUtensorMap& y = tm_out ? *tm_out : *tm_rows;  // (not read without tma_out)
  return out_bf16 ? i8_launch<bf16>(*tm_rows, *tm_cols, y, p, b, st) : i8_launch<float>(*tm_rows, *tm_cols, y, p, b, st);
}

}  // namespace pae
