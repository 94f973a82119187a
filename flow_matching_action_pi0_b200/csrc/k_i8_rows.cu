// Row quantisation to 8 bits, and the int8 K/V cache's write and read-back.
//
// A row x becomes codes q_i = rint(x_i / s) in [-127, 127] with s = max|x| /
// 127 (rounded once to fp32), so x_i is read back as q_i s, off by at most
// s / 2.  The code is that of the exact quotient, ties to even: x_i (1/s) in
// fp32 can land on the wrong side of a half, so near one the sign of
// x_i - (n + 1/2) s decides, which one fused multiply-add gives exactly.  Few
// values are that near; the others cost five instructions each.
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

// Scale of a row from the bits of its largest |x| (NaN and infinity sort above
// every finite value).
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return __int_as_float(0x7FC00000);
  const float s = __fdiv_rn(__uint_as_float(amax_bits), 127.f);
  return s < kTinyScale ? 0.f : s;
}
__device__ __forceinline__ float inv_scale(float s) { return s > 0.f ? __fdiv_rn(1.f, s) : 0.f; }

// rint(x / s) for |x| <= 127 s (1 + 2^-23), inv = 1 / s > 0.  t = x inv is off
// by at most 127 * 2^-22: within 1e-4 of a half, floor(t) is the lower
// neighbour of the exact quotient, and the fused product has the sign of the
// quotient's difference from the half.
__device__ __forceinline__ int quant1(float x, float s, float inv) {
  const float t = x * inv;
  float q = rintf(t);
  if (fabsf(t - q) > 0.4999f) {
    const float lo = floorf(t);
    const float e = __fmaf_rn(-(lo + 0.5f), s, x);
    q = e > 0.f ? lo + 1.f : e < 0.f ? lo : rintf(lo + 0.5f);
  }
  return (int)q;
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return (uint32_t)(a & 0xFF) | ((uint32_t)(b & 0xFF) << 8) | ((uint32_t)(c & 0xFF) << 16) | ((uint32_t)d << 24);
}

// Largest magnitude of three; NaN if one of them is.
__device__ __forceinline__ float amax3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 8 elements of a row in registers, lane i of a row: bf16 elements [8 i, +8);
// fp32 elements [4 i, +4) and [half + 4 i, +4), so that every 16-byte access of
// neighbouring lanes is one contiguous run.
template <typename T>
struct Vec8;
template <>
struct Vec8<bf16> {
  uint4 w;
  __device__ __forceinline__ void load(const bf16* row, int lane, int) { w = reinterpret_cast<const uint4*>(row)[lane]; }
  static __device__ __forceinline__ void put_codes(int8_t* row, int lane, int, uint2 q) { reinterpret_cast<uint2*>(row)[lane] = q; }
  static __device__ __forceinline__ uint2 get_codes(const int8_t* row, int lane, int) { return reinterpret_cast<const uint2*>(row)[lane]; }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  // the bits of the largest |x|, as fp32
  __device__ __forceinline__ uint32_t amax() const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
    return max(u << 16, u & 0xFFFF0000u);
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
  float4 a, b;
  __device__ __forceinline__ void load(const float* row, int lane, int half) {
    a = reinterpret_cast<const float4*>(row)[lane];
    b = reinterpret_cast<const float4*>(row + half)[lane];
  }
  static __device__ __forceinline__ void put_codes(int8_t* row, int lane, int half, uint2 q) {
    reinterpret_cast<uint32_t*>(row)[lane] = q.x;
    reinterpret_cast<uint32_t*>(row + half)[lane] = q.y;
  }
  static __device__ __forceinline__ uint2 get_codes(const int8_t* row, int lane, int half) {
    return make_uint2(reinterpret_cast<const uint32_t*>(row)[lane], reinterpret_cast<const uint32_t*>(row + half)[lane]);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void put(const float* f) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ uint32_t amax() const {
    return __float_as_uint(amax3(amax3(amax3(a.x, a.y, a.z), a.w, b.x), amax3(b.y, b.z, b.w), 0.f));
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

// 8 codes.  x inv + 1.5 2^23 rounds to a whole number in the low bits of the
// sum (the codes are its low bytes); the residual x - q s tells whether the
// rounding can be wrong, which only values within 1e-6 of a half are, and
// those go through quant1.
__device__ __forceinline__ uint2 quant8(const float* f, float s, float inv) {
  constexpr float kMagic = 12582912.f;
  uint32_t m[8];
  float worst = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {  // two at a time
    const float2 x = make_float2(f[i], f[i + 1]);
    const float2 r = fma2(x, make_float2(inv, inv), make_float2(kMagic, kMagic));
    m[i] = __float_as_uint(r.x);
    m[i + 1] = __float_as_uint(r.y);
    const float2 e = fma2(add2(r, make_float2(-kMagic, -kMagic)), make_float2(-s, -s), x);
    worst = fmaxf(worst, fmaxf(fabsf(e.x), fabsf(e.y)));
  }
  if (worst > s * 0.499999f) {
    int q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = quant1(f[i], s, inv);
    return make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
  }
  return make_uint2(__byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(m[4], m[5], 0x0040), __byte_perm(m[6], m[7], 0x0040), 0x5410));
}

// s / sqrt(mean x^2 + eps) from the mean square of x / s, which neither overflows
// nor underflows: 1 / sqrt(mean + eps / s^2).  Where eps / s^2 leaves fp32, the
// mean (at most 127^2) is nothing beside it.
__device__ __forceinline__ float rms_scale(float s, float inv, float mean_sq, float eps) {
  if (!(s > 0.f)) return s;  // a row of zeros, or NaN
  const float t = eps * inv * inv;
  return t < 0x1p100f ? rsqrtf(mean_sq + t) : s * rsqrtf(eps);
}

// ------------------------------------------------------------ row quantiser
// TPR threads per row (32 to 256), NV groups of 8 elements per thread in
// registers; width % 8 == 0, rows 16-byte aligned.
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
      v[i].load(xr, c, width / 2);
    else
      v[i].zero();
  }
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) am = max(am, v[i].amax());
  am = __reduce_max_sync(0xFFFFFFFFu, am);
  constexpr int WPR = TPR / 32;                          // warps per row
  const int w0 = (int)threadIdx.x / TPR * WPR;           // the row's first
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = am;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPR; ++w) am = max(am, s_max[w0 + w]);
  }
  const float s = row_scale(am);
  const float inv = inv_scale(s);
  int8_t* cr = codes + (size_t)row * width;
  float2 ss2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + i * TPR;
    if (live && c < nv) {
      float f[8];
      v[i].get(f);
      Vec8<T>::put_codes(cr, c, width / 2, inv > 0.f ? quant8(f, s, inv) : make_uint2(0, 0));
      if (rms_eps > 0.f) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float2 t = mul2(make_float2(f[j], f[j + 1]), make_float2(inv, inv));
          ss2 = fma2(t, t, ss2);
        }
      }
    }
  }
  float ss = 0.f;
  if (rms_eps > 0.f) {
    ss = warp_sum(ss2.x + ss2.y);
    if constexpr (WPR > 1) {
      if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = ss;
      __syncthreads();
      ss = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) ss += s_sum[w0 + w];
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
  int8_t* cr = codes + (size_t)row * width;
  // Squares in chains of 64, 256 of those, and those: equal elements round the
  // same way every time, and one chain over a row of 2^22 was off by 2^-14.
  // (1600 rows of 28672: 82.7 us, 78.7 with one chain.)
  float ss = 0.f, mid = 0.f, low = 0.f;
  int left = 64, groups = 256;
  for (int i = threadIdx.x; i < width; i += 256) {
    const float f = ld_act<T>(xr + i);
    cr[i] = inv > 0.f ? (int8_t)quant1(f, s, inv) : (int8_t)0;
    low = fmaf(f * inv, f * inv, low);
    if (--left == 0) {
      mid += low;
      low = 0.f;
      left = 64;
      if (--groups == 0) {
        ss += mid;
        mid = 0.f;
        groups = 256;
      }
    }
  }
  ss = warp_sum(ss + mid + low);
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
  // As many threads as the row has groups, up to a block: a row is then one round
  // trip (1600 rows of 2048 bf16: 9.6 us with a warp per row, 4.8 with a block).
  // Where the rows fill the SMs more than once anyway, two groups per thread halve
  // the reductions (20000 rows of 1024: 19.8 us with one, 16.7 with two; 4000: 5.5
  // and 5.6; 2000: 3.7 and 4.7).
  if ((long long)rows * nv < (1 << 19)) {
    if (nv > 32 && nv <= 64) return quant_launch<T, 64, 1>(x, ldx, rows, width, eps, codes, scale, st);
    if (nv > 64 && nv <= 128) return quant_launch<T, 128, 1>(x, ldx, rows, width, eps, codes, scale, st);
    if (nv > 128 && nv <= 256) return quant_launch<T, 256, 1>(x, ldx, rows, width, eps, codes, scale, st);
  }
  if (nv <= 32) return quant_launch<T, 32, 1>(x, ldx, rows, width, eps, codes, scale, st);
  if (nv <= 64) return quant_launch<T, 32, 2>(x, ldx, rows, width, eps, codes, scale, st);
  if (nv <= 128) return quant_launch<T, 64, 2>(x, ldx, rows, width, eps, codes, scale, st);
  if (nv <= 256) return quant_launch<T, 128, 2>(x, ldx, rows, width, eps, codes, scale, st);
  if (nv <= 512) return quant_launch<T, 256, 2>(x, ldx, rows, width, eps, codes, scale, st);
  return quant_launch<T, 256, 8>(x, ldx, rows, width, eps, codes, scale, st);
}

// ---------------------------------------------------------------- K/V cache
// Slot and position of packed row t: sequence b = the last with cu[b] <= t
// (binary search; empty sequences have cu[b] == cu[b + 1] and are passed
// over).  Rows outside every sequence, and rows that would fall outside the
// slot, have no place.  The offsets of up to kPlaceSeqs sequences are searched
// in shared memory: a search in global memory is a chain of L2 round trips
// (writing one row for each of 32 sequences took 5.5 us with it).
constexpr int kPlaceSeqs = 1024;
struct PlaceSmem {
  int cu[kPlaceSeqs + 1], start[kPlaceSeqs];
};
__device__ __forceinline__ void place_load(const Kv8Rows& r, PlaceSmem& p) {  // a barrier must follow
  if (!r.cu || r.n_seq > kPlaceSeqs) return;
  for (int i = threadIdx.x; i <= r.n_seq; i += 256) p.cu[i] = __ldg(r.cu + i);
  for (int i = threadIdx.x; i < r.n_seq; i += 256) p.start[i] = r.start ? __ldg(r.start + i) : 0;
}
__device__ __forceinline__ bool kv8_place(const Kv8Rows& r, const PlaceSmem& p, int cap, int t, int& slot, int& pos) {
  int b = 0;
  long long at = t;
  if (r.cu) {
    const bool sh = r.n_seq <= kPlaceSeqs;
    const int* cu = sh ? p.cu : r.cu;
    if (r.n_seq < 1 || t < cu[0] || t >= cu[r.n_seq]) return false;
    int lo = 0, hi = r.n_seq;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;
    at = (long long)t - cu[b];
    if (r.start) at += sh ? p.start[b] : __ldg(r.start + b);
  } else if (r.start) {
    at += __ldg(r.start);
  }
  slot = r.slot0 + b;
  pos = (int)at;
  return at >= 0 && at < cap;
}

// blockIdx.y = KV head; d / 8 lanes per row, K and V of a token loaded before
// either is quantised.
template <typename T, int D, bool ROPE>
__global__ void __launch_bounds__(256)
    k_kv8_write(const Kv8 c, const Kv8Rows r, const Kv8Io io, const float2* __restrict__ rope_cs) {
  constexpr int LPR = D / 8, RPB = 256 / LPR;
  __shared__ PlaceSmem place;
  pdl_launch_dependents();
  pdl_wait();
  place_load(r, place);
  const int sub = threadIdx.x % LPR, head = blockIdx.y;
  const T* kp = static_cast<const T*>(io.k) + head * io.k_head;
  const T* vp = static_cast<const T*>(io.v) + head * io.v_head;
  bool placed = false;  // the offsets are in shared memory
  // whole warps stay in the loop together: the shuffles below need all lanes
  for (long long t0 = (long long)blockIdx.x * RPB; t0 < r.n_rows; t0 += (long long)gridDim.x * RPB) {
    Vec8<T> kv[2];
    const bool in = t0 + threadIdx.x / LPR < r.n_rows;
    const int tok = (int)t0 + threadIdx.x / LPR;
    if (in) {
      kv[0].load(kp + tok * io.k_tok, sub, D / 2);
      kv[1].load(vp + tok * io.v_tok, sub, D / 2);
    } else {
      kv[0].zero();
      kv[1].zero();
    }
    if (!placed) __syncthreads();
    placed = true;
    int slot = 0, pos = 0;
    const bool ok = in && kv8_place(r, place, c.cap, tok, slot, pos);
    const size_t row = ((size_t)slot * c.heads + head) * c.cap + pos;
    if constexpr (ROPE) {
      // Rotate-half: channel i < d/2 pairs with i + d/2, which this lane holds
      // too: a' = a cos - b sin, b' = b cos + a sin.
      float f[8];
      kv[0].get(f);
      const float2* cs = rope_cs + (size_t)(ok ? pos : 0) * (D / 2) + sub * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = cs[i];
        const float x = f[i], y = f[4 + i];
        f[i] = x * t.x - y * t.y;
        f[4 + i] = y * t.x + x * t.y;
      }
      kv[0].put(f);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t am = kv[w].amax();
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
      const float s = row_scale(am);
      const float inv = inv_scale(s);
      if (ok) {
        float f[8];
        kv[w].get(f);
        Vec8<T>::put_codes((w ? c.v : c.k) + row * D, sub, D / 2, inv > 0.f ? quant8(f, s, inv) : make_uint2(0, 0));
        if (sub == 0) (w ? c.v_scale : c.k_scale)[row] = s;
      }
    }
  }
}

// Codes of a word as fp32 times s: byte ^ 0x80 put into the low bits of 2^23
// is 2^23 + 128 + code, exactly.
__device__ __forceinline__ float4 codes4(uint32_t w, float s) {
  const uint32_t u = w ^ 0x80808080u;
  constexpr float kOff = 8388736.f;
  return make_float4((__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)) - kOff) * s,
                     (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441)) - kOff) * s,
                     (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)) - kOff) * s,
                     (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443)) - kOff) * s);
}
__device__ __forceinline__ void put8(float* row, int lane, int half, const uint2 q, float s) {
  reinterpret_cast<float4*>(row)[lane] = codes4(q.x, s);
  reinterpret_cast<float4*>(row + half)[lane] = codes4(q.y, s);
}
__device__ __forceinline__ void put8(bf16* row, int lane, int, const uint2 q, float s) {
  const float4 a = codes4(q.x, s), b = codes4(q.y, s);
  const __nv_bfloat162 w[4] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w),
                               __floats2bfloat162_rn(b.x, b.y), __floats2bfloat162_rn(b.z, b.w)};
  reinterpret_cast<uint4*>(row)[lane] = *reinterpret_cast<const uint4*>(w);
}

// The inverse of k_kv8_write: rows without a place read as zeros.
template <typename T, int D>
__global__ void __launch_bounds__(256) k_kv8_read(const Kv8 c, const Kv8Rows r, const Kv8Io io) {
  constexpr int LPR = D / 8, RPB = 256 / LPR;
  __shared__ PlaceSmem place;
  pdl_launch_dependents();
  pdl_wait();
  place_load(r, place);
  const int sub = threadIdx.x % LPR, head = blockIdx.y;
  T* kp = static_cast<T*>(io.k) + head * io.k_head;
  T* vp = static_cast<T*>(io.v) + head * io.v_head;
  __syncthreads();
  for (long long t = (long long)blockIdx.x * RPB + threadIdx.x / LPR; t < r.n_rows; t += (long long)gridDim.x * RPB) {
    int slot = 0, pos = 0;
    uint2 qk = make_uint2(0, 0), qv = qk;
    float sk = 0.f, sv = 0.f;
    if (kv8_place(r, place, c.cap, (int)t, slot, pos)) {
      const size_t row = ((size_t)slot * c.heads + head) * c.cap + pos;
      qk = Vec8<T>::get_codes(c.k + row * D, sub, D / 2);
      qv = Vec8<T>::get_codes(c.v + row * D, sub, D / 2);
      sk = c.k_scale[row];
      sv = c.v_scale[row];
    }
    put8(kp + t * io.k_tok, sub, D / 2, qk, sk);
    put8(vp + t * io.v_tok, sub, D / 2, qv, sv);
  }
}

// Blocks of 256 threads over tokens (x) and KV heads (y), up to 32 blocks per
// SM (several waves: with 8 resident ones alone the ragged prefixes took 10 %
// longer).
dim3 kv8_grid(const Kv8& c, const Kv8Rows& r) {
  const int per = 256 / (c.d / 8);
  const int need = (r.n_rows - 1) / per + 1, most = std::max(1, 148 * 32 / c.heads);
  return dim3(std::min(need, most), c.heads);
}

template <typename T, bool ROPE>
cudaError_t kv8_write_sel(const Kv8& c, const Kv8Rows& r, const Kv8Io& io, const float2* cs, cudaStream_t st) {
  auto kern = c.d == 64 ? k_kv8_write<T, 64, ROPE> : c.d == 128 ? k_kv8_write<T, 128, ROPE> : k_kv8_write<T, 256, ROPE>;
  return launch_ex(kern, kv8_grid(c, r), dim3(256), 0, st, 1, true, c, r, io, cs);
}

template <typename T>
cudaError_t kv8_read_sel(const Kv8& c, const Kv8Rows& r, const Kv8Io& io, cudaStream_t st) {
  auto kern = c.d == 64 ? k_kv8_read<T, 64> : c.d == 128 ? k_kv8_read<T, 128> : k_kv8_read<T, 256>;
  return launch_ex(kern, kv8_grid(c, r), dim3(256), 0, st, 1, true, c, r, io);
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
