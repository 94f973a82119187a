// Row quantisation to 8 bits, and the int8 K/V cache's write and read-back.
//
// A row x becomes codes q_i = rint(x_i / s) in [-127, 127] with s = max|x| /
// 127 (rounded once to fp32), so x_i is read back as q_i s, off by at most
// s / 2.  The code is that of the exact quotient, ties to even: x_i (1/s) in
// fp32 can land on the wrong side of a half, so near one the sign of
// x_i - (n + 1/2) s decides, which one fused multiply-add gives exactly.
// s below 2^-120 is taken as 0 (codes 0): above it 1/s, the products and that
// sign are free of overflow and underflow.  A row with a NaN or an infinity
// gets scale NaN and codes 0: it reads back as NaN and says so.
//
// Bound: bytes.  Each row is read once into registers (16-byte loads), its
// maximum found by a shuffle tree over the lanes that share it, and its codes
// written from the same registers.  Every kernel here is launched with
// programmatic dependent launch and waits for its predecessor before it reads
// anything, so only its start overlaps the predecessor's end.
#include <algorithm>

#include "int8.h"
#include "launch.cuh"

namespace pae {

namespace {

constexpr float kTinyScale = 7.52316384526264e-37f;  // 2^-120

// Scale of a row from the bits of its largest |x| (as an integer maximum: NaN
// and infinity sort above every finite value).
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return __int_as_float(0x7FC00000);
  const float s = __fdiv_rn(__uint_as_float(amax_bits), 127.f);
  return s < kTinyScale ? 0.f : s;
}

// rint(x / s) for |x| <= 127 s (1 + 2^-23), inv = 1 / s (0 when s is 0 or NaN)
__device__ __forceinline__ int quant1(float x, float s, float inv) {
  const float t = x * inv;
  float q = rintf(t);
  if (fabsf(t - q) > 0.4999f) {
    // within 1e-4 of a half: t is off by at most 127 * 2^-22, so floor(t) is
    // the lower neighbour, and the fused product has the difference's sign
    const float lo = floorf(t);
    const float e = __fmaf_rn(-(lo + 0.5f), s, x);
    q = e > 0.f ? lo + 1.f : e < 0.f ? lo : rintf(lo + 0.5f);
  }
  return (int)q;
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return (uint32_t)(a & 0xFF) | ((uint32_t)(b & 0xFF) << 8) | ((uint32_t)(c & 0xFF) << 16) | ((uint32_t)d << 24);
}

// 8 consecutive elements of a row in registers.
template <typename T>
struct Vec8;
template <>
struct Vec8<bf16> {
  uint4 w;
  __device__ __forceinline__ void load(const bf16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Vec8<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const uint4*>(p)[0];
    b = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void put(const float* f) {
    a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  }
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t k = 0x7FFFFFFFu;
    return max(max(max(a.x & k, a.y & k), max(a.z & k, a.w & k)), max(max(b.x & k, b.y & k), max(b.z & k, b.w & k)));
  }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
  }
};

__device__ __forceinline__ uint2 quant8(const float* f, float s, float inv) {
  int q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = quant1(f[i], s, inv);
  return make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
}

__device__ __forceinline__ float inv_scale(float s) { return s > 0.f ? __fdiv_rn(1.f, s) : 0.f; }

// s / sqrt(mean x^2 + eps).  Squares of rows with s >= 1 are taken in units of
// s (they cannot overflow), others as they are (eps / s^2 cannot).
__device__ __forceinline__ float rms_unit(float s, float inv) { return s >= 1.f ? inv : 1.f; }
__device__ __forceinline__ float rms_scale(float s, float inv, float mean_sq, float eps) {
  return s >= 1.f ? rsqrtf(mean_sq + eps * inv * inv) : s * rsqrtf(mean_sq + eps);
}

// ------------------------------------------------------------ row quantiser
// TPR threads per row (32: a warp, 256: the block), NV groups of 8 elements
// per thread in registers; width % 8 == 0, rows 16-byte aligned.
template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(256) k_quantize_rows(const T* __restrict__ x, long long ldx, int rows, int width,
                                                       float rms_eps, int8_t* __restrict__ codes,
                                                       float* __restrict__ scale) {
  __shared__ uint32_t s_max[8];
  __shared__ float s_sum[8];
  pdl_launch_dependents();
  pdl_wait();
  constexpr int RPB = 256 / TPR;
  const int lane = threadIdx.x % TPR;
  const int row = blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = row < rows;  // uniform over the threads of a row
  const int nv = width / 8;
  const T* xr = x + (size_t)(live ? row : 0) * ldx;
  Vec8<T> v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + i * TPR;
    if (live && c < nv)
      v[i].load(xr + (size_t)c * 8);
    else
      v[i].zero();
  }
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) am = max(am, v[i].amax());
  am = __reduce_max_sync(0xFFFFFFFFu, am);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = am;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) am = max(am, s_max[w]);
  }
  const float s = row_scale(am);
  const float inv = inv_scale(s);
  const float unit = rms_unit(s, inv);
  uint2* cr = reinterpret_cast<uint2*>(codes + (size_t)row * width);
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + i * TPR;
    if (live && c < nv) {
      float f[8];
      v[i].get(f);
      cr[c] = inv > 0.f ? quant8(f, s, inv) : make_uint2(0, 0);
      if (rms_eps > 0.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float t = f[j] * unit;
          ss = fmaf(t, t, ss);
        }
      }
    }
  }
  if (rms_eps > 0.f) {
    ss = warp_sum(ss);
    if constexpr (TPR > 32) {
      if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = ss;
      __syncthreads();
      ss = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) ss += s_sum[w];
    }
  }
  if (live && lane == 0) scale[row] = rms_eps > 0.f ? rms_scale(s, inv, ss / (float)width, rms_eps) : s;
}

// Any width, alignment and stride: one block per row, the row read twice.
template <typename T>
__global__ void __launch_bounds__(256) k_quantize_rows_any(const T* __restrict__ x, long long ldx, int rows, int width,
                                                           float rms_eps, int8_t* __restrict__ codes,
                                                           float* __restrict__ scale) {
  __shared__ uint32_t s_max[8];
  __shared__ float s_sum[8];
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x;
  const T* xr = x + (size_t)row * ldx;
  uint32_t am = 0;
  for (int i = threadIdx.x; i < width; i += 256) am = max(am, __float_as_uint(ld_act<T>(xr + i)) & 0x7FFFFFFFu);
  am = __reduce_max_sync(0xFFFFFFFFu, am);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = am;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) am = max(am, s_max[w]);
  const float s = row_scale(am);
  const float inv = inv_scale(s);
  const float unit = rms_unit(s, inv);
  int8_t* cr = codes + (size_t)row * width;
  float ss = 0.f;
  for (int i = threadIdx.x; i < width; i += 256) {
    const float f = ld_act<T>(xr + i);
    cr[i] = inv > 0.f ? (int8_t)quant1(f, s, inv) : (int8_t)0;
    ss = fmaf(f * unit, f * unit, ss);
  }
  ss = warp_sum(ss);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = ss;
  __syncthreads();
  ss = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) ss += s_sum[w];
  if (threadIdx.x == 0) scale[row] = rms_eps > 0.f ? rms_scale(s, inv, ss / (float)width, rms_eps) : s;
}

template <typename T, int TPR, int NV>
cudaError_t quant_launch(const void* x, long long ldx, int rows, int width, float eps, int8_t* codes, float* scale,
                         cudaStream_t st) {
  constexpr int RPB = 256 / TPR;
  return launch_ex(k_quantize_rows<T, TPR, NV>, dim3((rows + RPB - 1) / RPB), dim3(256), 0, st, 1, true,
                   static_cast<const T*>(x), ldx, rows, width, eps, codes, scale);
}

template <typename T>
cudaError_t quant_sel(const void* x, long long ldx, int rows, int width, float eps, int8_t* codes, float* scale,
                      cudaStream_t st) {
  const bool vec = width % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0 &&
                   (ldx * (long long)sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(codes) & 7) == 0;
  const int nv = width / 8;
  if (!vec || nv > 256 * 8)
    return launch_ex(k_quantize_rows_any<T>, dim3(rows), dim3(256), 0, st, 1, true, static_cast<const T*>(x), ldx, rows,
                     width, eps, codes, scale);
  // A warp per row while its registers hold the row; a block per row when the
  // row is longer, or when so few rows would leave most SMs idle.
  constexpr int kWarpNv = sizeof(T) == 2 ? 8 : 4;
  if (nv <= 32 * kWarpNv && rows >= 148 * 8) {
    if (nv <= 64) return quant_launch<T, 32, 2>(x, ldx, rows, width, eps, codes, scale, st);
    if (nv <= 128) return quant_launch<T, 32, 4>(x, ldx, rows, width, eps, codes, scale, st);
    return quant_launch<T, 32, kWarpNv>(x, ldx, rows, width, eps, codes, scale, st);
  }
  if (nv <= 256) return quant_launch<T, 256, 1>(x, ldx, rows, width, eps, codes, scale, st);
  if (nv <= 512) return quant_launch<T, 256, 2>(x, ldx, rows, width, eps, codes, scale, st);
  return quant_launch<T, 256, 8>(x, ldx, rows, width, eps, codes, scale, st);
}

// ---------------------------------------------------------------- K/V cache
// Slot and position of packed row t: sequence b = the last with cu[b] <= t
// (binary search; empty sequences have cu[b] == cu[b + 1] and are passed
// over).  Rows outside every sequence, and rows that would fall outside the
// slot, have no place.
__device__ __forceinline__ bool kv8_place(const Kv8Rows& r, int cap, int t, int& slot, int& pos) {
  int b = 0;
  long long at = t;
  if (r.cu) {
    if (r.n_seq < 1 || t < __ldg(r.cu) || t >= __ldg(r.cu + r.n_seq)) return false;
    int lo = 0, hi = r.n_seq;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(r.cu + mid) <= t)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;
    at = (long long)t - __ldg(r.cu + b);
  }
  if (r.start) at += __ldg(r.start + b);
  slot = r.slot0 + b;
  pos = (int)at;
  return at >= 0 && at < cap;
}

// d / 8 lanes per row; a thread takes UNR (token, head) pairs, K and V of each
// loaded before any is quantised.
template <typename T, int D, bool ROPE>
__global__ void __launch_bounds__(256)
    k_kv8_write(const Kv8 c, const Kv8Rows r, const Kv8Io io, const float2* __restrict__ rope_cs, long long items) {
  constexpr int LPR = D / 8, UNR = 2;
  pdl_launch_dependents();
  pdl_wait();
  const int sub = threadIdx.x % LPR;
  const long long gstep = (long long)gridDim.x * (256 / LPR);
  const long long g0 = (long long)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  // whole warps stay in the loop together: the shuffles below need all lanes
  const long long rounds = (items + gstep * UNR - 1) / (gstep * UNR);
  for (long long rd = 0; rd < rounds; ++rd) {
    Vec8<T> kv[UNR][2];
    long long it[UNR];
    int tok[UNR], head[UNR];
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      it[u] = g0 + (rd * UNR + u) * gstep;
      if (it[u] < items) {
        tok[u] = (int)(it[u] / c.heads);
        head[u] = (int)(it[u] - (long long)tok[u] * c.heads);
        kv[u][0].load(static_cast<const T*>(io.k) + tok[u] * io.k_tok + head[u] * io.k_head + sub * 8);
        kv[u][1].load(static_cast<const T*>(io.v) + tok[u] * io.v_tok + head[u] * io.v_head + sub * 8);
      } else {
        kv[u][0].zero();
        kv[u][1].zero();
      }
    }
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      int slot = 0, pos = 0;
      const bool ok = it[u] < items && kv8_place(r, c.cap, tok[u], slot, pos);
      const size_t row = ((size_t)slot * c.heads + (ok ? head[u] : 0)) * c.cap + pos;
      if constexpr (ROPE) {
        // Rotate-half: channel i < d/2 pairs with i + d/2, which the lane LPR/2
        // away holds: a' = a cos - b sin, b' = b cos + a sin.
        float f[8], g[8];
        kv[u][0].get(f);
        const bool hi = sub >= LPR / 2;
        const float2* cs = rope_cs + (size_t)(ok ? pos : 0) * (D / 2) + (sub % (LPR / 2)) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl_xor_sync(0xFFFFFFFFu, f[i], LPR / 2);
          const float2 t = cs[i];
          g[i] = hi ? f[i] * t.x + o * t.y : f[i] * t.x - o * t.y;
        }
        kv[u][0].put(g);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t am = kv[u][w].amax();
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
        const float s = row_scale(am);
        const float inv = inv_scale(s);
        if (ok) {
          float f[8];
          kv[u][w].get(f);
          const uint2 q = inv > 0.f ? quant8(f, s, inv) : make_uint2(0, 0);
          *reinterpret_cast<uint2*>((w ? c.v : c.k) + row * D + sub * 8) = q;
          if (sub == 0) (w ? c.v_scale : c.k_scale)[row] = s;
        }
      }
    }
  }
}

__device__ __forceinline__ float code_at(uint32_t w, int i) { return (float)(int)(int8_t)(w >> (8 * i)); }

template <typename T>
__device__ __forceinline__ void put8(T* p, const uint2 q, float s);
template <>
__device__ __forceinline__ void put8<float>(float* p, const uint2 q, float s) {
  float4* d = reinterpret_cast<float4*>(p);
  d[0] = make_float4(code_at(q.x, 0) * s, code_at(q.x, 1) * s, code_at(q.x, 2) * s, code_at(q.x, 3) * s);
  d[1] = make_float4(code_at(q.y, 0) * s, code_at(q.y, 1) * s, code_at(q.y, 2) * s, code_at(q.y, 3) * s);
}
template <>
__device__ __forceinline__ void put8<bf16>(bf16* p, const uint2 q, float s) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t src = i < 2 ? q.x : q.y;
    const int b = (2 * i) & 3;
    w[i] = (uint32_t)__bfloat16_as_ushort(f2bf(code_at(src, b) * s)) |
           ((uint32_t)__bfloat16_as_ushort(f2bf(code_at(src, b + 1) * s)) << 16);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The inverse of k_kv8_write: rows without a place read as zeros.
template <typename T, int D>
__global__ void __launch_bounds__(256) k_kv8_read(const Kv8 c, const Kv8Rows r, const Kv8Io io, long long items) {
  constexpr int LPR = D / 8;
  pdl_launch_dependents();
  pdl_wait();
  const int sub = threadIdx.x % LPR;
  const long long gstep = (long long)gridDim.x * (256 / LPR);
  for (long long it = (long long)blockIdx.x * (256 / LPR) + threadIdx.x / LPR; it < items; it += gstep) {
    const int tok = (int)(it / c.heads), head = (int)(it - (long long)tok * c.heads);
    int slot = 0, pos = 0;
    const bool ok = kv8_place(r, c.cap, tok, slot, pos);
    uint2 qk = make_uint2(0, 0), qv = make_uint2(0, 0);
    float sk = 0.f, sv = 0.f;
    if (ok) {
      const size_t row = ((size_t)slot * c.heads + head) * c.cap + pos;
      qk = *reinterpret_cast<const uint2*>(c.k + row * D + sub * 8);
      qv = *reinterpret_cast<const uint2*>(c.v + row * D + sub * 8);
      sk = c.k_scale[row];
      sv = c.v_scale[row];
    }
    put8<T>(static_cast<T*>(io.k) + tok * io.k_tok + head * io.k_head + sub * 8, qk, sk);
    put8<T>(static_cast<T*>(io.v) + tok * io.v_tok + head * io.v_head + sub * 8, qv, sv);
  }
}

int kv8_grid(long long items, int d, int unr) {
  const long long per = 256 / (d / 8) * unr;
  return (int)std::min<long long>((items + per - 1) / per, 148 * 8);
}

template <typename T, bool ROPE>
cudaError_t kv8_write_sel(const Kv8& c, const Kv8Rows& r, const Kv8Io& io, const float2* cs, cudaStream_t st) {
  const long long items = (long long)r.n_rows * c.heads;
  const int grid = kv8_grid(items, c.d, 2);
  auto kern = c.d == 64 ? k_kv8_write<T, 64, ROPE> : c.d == 128 ? k_kv8_write<T, 128, ROPE> : k_kv8_write<T, 256, ROPE>;
  return launch_ex(kern, dim3(grid), dim3(256), 0, st, 1, true, c, r, io, cs, items);
}

template <typename T>
cudaError_t kv8_read_sel(const Kv8& c, const Kv8Rows& r, const Kv8Io& io, cudaStream_t st) {
  const long long items = (long long)r.n_rows * c.heads;
  const int grid = kv8_grid(items, c.d, 1);
  auto kern = c.d == 64 ? k_kv8_read<T, 64> : c.d == 128 ? k_kv8_read<T, 128> : k_kv8_read<T, 256>;
  return launch_ex(kern, dim3(grid), dim3(256), 0, st, 1, true, c, r, io, items);
}

}  // namespace

cudaError_t launch_quantize_rows(bool in_bf16, const void* x, long long ldx, int rows, int width, float rms_eps,
                                 int8_t* codes, float* scale, cudaStream_t st) {
  return in_bf16 ? quant_sel<bf16>(x, ldx, rows, width, rms_eps, codes, scale, st)
                 : quant_sel<float>(x, ldx, rows, width, rms_eps, codes, scale, st);
}

cudaError_t launch_kv8_write(bool bf16_rows, const Kv8& c, const Kv8Rows& r, const Kv8Io& io, const float2* rope_cs,
                             cudaStream_t st) {
  if (bf16_rows) return rope_cs ? cudaErrorInvalidValue : kv8_write_sel<bf16, false>(c, r, io, nullptr, st);
  return rope_cs ? kv8_write_sel<float, true>(c, r, io, rope_cs, st) : kv8_write_sel<float, false>(c, r, io, nullptr, st);
}

cudaError_t launch_kv8_read(bool bf16_rows, const Kv8& c, const Kv8Rows& r, const Kv8Io& io, cudaStream_t st) {
  return bf16_rows ? kv8_read_sel<bf16>(c, r, io, st) : kv8_read_sel<float>(c, r, io, st);
}

}  // namespace pae
