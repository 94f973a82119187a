// Entry points of the 8-bit prefix operators (include/pae.h): argument checks,
// tensor maps and launches.  They need no context and allocate no device
// memory; per device they keep one host-mapped error word and the kernels'
// shared-memory opt-ins, set up by pae_int8_init or the first call.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "int8.h"
#include "pae.h"

namespace pae {

void set_create_error(const char* msg);  // pae_api.cu: message for pae_last_error(NULL)

namespace {

constexpr int kMaxDevices = 64;
constexpr long long kWaitNs = 2000000000LL;  // bound of a device-side wait, as a context's default
constexpr int kMaxCapacity = 1 << 30;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct DeviceState {
  bool ready = false;
  int* err_host = nullptr;
  int* err_dev = nullptr;
  EncodeTiledFn encode = nullptr;
};
std::mutex g_mu;
DeviceState g_dev[kMaxDevices];

pae_status fail(pae_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_create_error(buf);
  return st;
}

// (An error that is reported is also taken from the runtime, or it would fail
// every later call as one that is still pending.)
pae_status cuda_fail(const char* what, cudaError_t e) {
  cudaGetLastError();
  return fail(PAE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

pae_status check_word(const DeviceState* d, const char* fn) {
  const int code = d->err_host ? *(volatile int*)d->err_host : 0;
  if (code == 0) return PAE_OK;
  return fail(PAE_ERR_TIMEOUT, "%s: device error word set (%d): a bounded device wait ran out%s", fn, code,
              code == DEV_DRAIN ? "; copies may still be landing, end the process" : "");
}

// The current device's state, set up on first use.  Setting up allocates
// host-mapped memory, which a stream capture does not allow.
pae_status device_state(const char* fn, pae_stream stream, bool check_stream, DeviceState** out) {
  cudaError_t e = cudaGetLastError();  // (reported once; one that the context does not survive comes back)
  if (e != cudaSuccess) return fail(PAE_ERR_CUDA, "%s: a CUDA error from earlier work is pending (%s)", fn, cudaGetErrorString(e));
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return cuda_fail("cudaGetDevice", e);
  if (dev < 0 || dev >= kMaxDevices) return fail(PAE_ERR_UNSUPPORTED, "%s: device ordinals of 64 and above are not supported", fn);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState& d = g_dev[dev];
  if (!d.ready) {
    if (check_stream) {
      cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
      if (cudaStreamIsCapturing(reinterpret_cast<cudaStream_t>(stream), &cs) != cudaSuccess) cudaGetLastError();
      if (cs != cudaStreamCaptureStatusNone)
        return fail(PAE_ERR_STATE, "%s: the first call on a device may not be captured; call pae_int8_init before", fn);
    }
    cudaDriverEntryPointQueryResult q;
    void* enc = nullptr;
    e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &enc, cudaEnableDefault, &q);
    if (e == cudaSuccess && (!enc || q != cudaDriverEntryPointSuccess)) e = cudaErrorNotSupported;
    if (e == cudaSuccess) e = i8_gemm_init();
    if (e == cudaSuccess) e = kv8_attn_init();
    if (e == cudaSuccess && !d.err_host)
      e = cudaHostAlloc(reinterpret_cast<void**>(&d.err_host), sizeof(int), cudaHostAllocMapped | cudaHostAllocPortable);
    if (e == cudaSuccess) {
      *d.err_host = 0;
      e = cudaHostGetDevicePointer(reinterpret_cast<void**>(&d.err_dev), d.err_host, 0);
    }
    if (e != cudaSuccess) return cuda_fail(fn, e);
    d.encode = reinterpret_cast<EncodeTiledFn>(enc);
    d.ready = true;
  }
  *out = &d;
  return check_word(&d, fn);
}

// [rows][k] signed bytes, boxes of box_rows x 128 bytes, 128-byte swizzle;
// places outside read as zeros.
pae_status make_map(const DeviceState* d, CUtensorMap* m, const void* base, int rows, int k, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)k};
  cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  const CUresult r = d->encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PAE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for [%d][%d] int8", (int)r, rows, k);
  return PAE_OK;
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool known(int dtype) { return dtype == PAE_FP32 || dtype == PAE_BF16; }

pae_status check_cache(const char* fn, const pae_kv8* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return fail(PAE_ERR_ARG, "%s: the cache or one of its pointers is NULL", fn);
  if (c->n_kv_heads > 65535) return fail(PAE_ERR_UNSUPPORTED, "%s: n_kv_heads must be at most 65535", fn);
  if (c->n_slots < 1 || c->n_kv_heads < 1 || c->capacity < 1 || c->capacity > kMaxCapacity)
    return fail(PAE_ERR_ARG, "%s: n_slots, n_kv_heads and capacity must be positive (capacity at most 2^30)", fn);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(PAE_ERR_UNSUPPORTED, "%s: head_dim must be 64, 128 or 256", fn);
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return fail(PAE_ERR_ARG, "%s: codes must start on 16 bytes, scales on 4", fn);
  return PAE_OK;
}

Kv8 view(const pae_kv8* c) {
  return Kv8{reinterpret_cast<int8_t*>(c->k), reinterpret_cast<int8_t*>(c->v), c->k_scale, c->v_scale,
             c->n_slots, c->n_kv_heads, c->capacity, c->head_dim};
}

// Common part of the cache's write and read.
pae_status kv8_io(const char* fn, bool write, const pae_kv8* cache, void* k, void* v, const long long* ks,
                  const long long* vs, const int* cu, const int* start, int n_seq, int n_rows, int dtype,
                  pae_stream stream) {
  pae_status st = check_cache(fn, cache);
  if (st != PAE_OK) return st;
  if (!known(dtype)) return fail(PAE_ERR_ARG, "%s: dtype must be PAE_FP32 or PAE_BF16", fn);
  if (n_rows > kMaxCapacity) return fail(PAE_ERR_UNSUPPORTED, "%s: n_rows must be at most 2^30", fn);
  if (n_rows < 0 || n_seq < 0 || n_seq > cache->n_slots)
    return fail(PAE_ERR_ARG, "%s: n_rows must be >= 0 and n_seq in [0, n_slots]", fn);
  if (!cu && n_seq != 1) return fail(PAE_ERR_ARG, "%s: cu_rows may be NULL only for one sequence", fn);
  if (n_rows == 0) return PAE_OK;
  if (!k || !v) return fail(PAE_ERR_ARG, "%s: k or v is NULL", fn);
  const long long row = (long long)cache->n_kv_heads * cache->head_dim, dense[2] = {row, cache->head_dim};
  if (!ks) ks = dense;
  if (!vs) vs = dense;
  const int unit = dtype == PAE_BF16 ? 8 : 4;  // elements per 16 bytes
  for (int i = 0; i < 2; ++i)
    if (ks[i] < 0 || vs[i] < 0 || ks[i] % unit || vs[i] % unit)
      return fail(PAE_ERR_ARG, "%s: strides must be non-negative and multiples of 16 bytes", fn);
  if (!write && ((n_rows > 1 && (!ks[0] || !vs[0])) || (cache->n_kv_heads > 1 && (!ks[1] || !vs[1]))))
    return fail(PAE_ERR_ARG, "%s: rows that are written may not share their place (stride 0)", fn);
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(PAE_ERR_ARG, "%s: k and v must start on 16 bytes", fn);
  DeviceState* d = nullptr;
  if ((st = device_state(fn, stream, true, &d)) != PAE_OK) return st;
  const Kv8Rows r{cu, start, n_seq, n_rows, 0};
  const Kv8Io io{k, v, ks[0], ks[1], vs[0], vs[1]};
  cudaStream_t sm = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = write ? launch_kv8_write(dtype == PAE_BF16, view(cache), r, io, nullptr, sm)
                              : launch_kv8_read(dtype == PAE_BF16, view(cache), r, io, sm);
  return e == cudaSuccess ? PAE_OK : cuda_fail(fn, e);
}

pae_status plan_attention(const char* fn, const pae_kv8* c, int n_seq, int n_q, int n_q_heads, int n_new, Kv8AttnPlan* p) {
  if (n_seq < 0 || n_seq > c->n_slots || n_q < 0 || n_new < 0)
    return fail(PAE_ERR_ARG, "%s: n_seq must be in [0, n_slots], n_q and n_new >= 0", fn);
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads)
    return fail(PAE_ERR_ARG, "%s: n_q_heads must be a positive multiple of n_kv_heads", fn);
  const long long group = n_q_heads / c->n_kv_heads;
  if ((long long)n_seq * c->n_kv_heads > 65535 || group * std::max(n_q, 1) > (1 << 22) || n_new > kMaxCapacity)
    return fail(PAE_ERR_UNSUPPORTED, "%s: n_seq * n_kv_heads must be at most 65535, n_q * (n_q_heads / n_kv_heads) at most 2^22", fn);
  *p = plan_kv8_attn(std::max(n_seq, 1), c->n_kv_heads, (int)group, std::max(n_q, 1), n_new, c->capacity, c->head_dim);
  return PAE_OK;
}

}  // namespace
}  // namespace pae

using namespace pae;

extern "C" {

pae_status pae_int8_init(void) {
  DeviceState* d = nullptr;
  return device_state("pae_int8_init", nullptr, false, &d);
}

pae_status pae_int8_sync(pae_stream stream) {
  DeviceState* d = nullptr;
  pae_status st = device_state("pae_int8_sync", stream, true, &d);
  if (st != PAE_OK && st != PAE_ERR_TIMEOUT) return st;
  cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail("pae_int8_sync", e);
  return check_word(d, "pae_int8_sync");
}

void pae_int8_clear_error(void) {
  cudaGetLastError();  // one left pending
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return;
  }
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_dev[dev].err_host) return;
  if (cudaDeviceSynchronize() != cudaSuccess) cudaGetLastError();
  if (*(volatile int*)g_dev[dev].err_host != DEV_DRAIN) *(volatile int*)g_dev[dev].err_host = 0;
}

pae_status pae_quantize_rows(const void* x, long long ldx, int rows, int width, int dtype, float rms_eps,
                             signed char* codes, float* scale, pae_stream stream) {
  const char* fn = "pae_quantize_rows";
  if (!known(dtype)) return fail(PAE_ERR_ARG, "%s: dtype must be PAE_FP32 or PAE_BF16", fn);
  if (rows < 0 || width < 1) return fail(PAE_ERR_ARG, "%s: rows must be >= 0 and width >= 1", fn);
  if (rows > kMaxCapacity || width > kMaxCapacity) return fail(PAE_ERR_UNSUPPORTED, "%s: rows and width must be at most 2^30", fn);
  if (!(rms_eps >= 0.f) || std::isinf(rms_eps)) return fail(PAE_ERR_ARG, "%s: rms_eps must be 0 (no norm) or a finite positive number", fn);
  if (rows == 0) return PAE_OK;
  if (!x || !codes || !scale) return fail(PAE_ERR_ARG, "%s: a pointer argument is NULL", fn);
  if (ldx < width) return fail(PAE_ERR_ARG, "%s: ldx must be at least width", fn);
  if (!aligned(x, dtype == PAE_BF16 ? 2 : 4) || !aligned(scale, 4)) return fail(PAE_ERR_ARG, "%s: a pointer is not aligned to its element", fn);
  DeviceState* d = nullptr;
  pae_status st = device_state(fn, stream, true, &d);
  if (st != PAE_OK) return st;
  const cudaError_t e = launch_quantize_rows(dtype == PAE_BF16, x, ldx, rows, width, rms_eps,
                                             reinterpret_cast<int8_t*>(codes), scale, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PAE_OK : cuda_fail(fn, e);
}

pae_status pae_linear_i8(const signed char* x, const float* x_scale, const signed char* w, const float* w_scale,
                         int tokens, int n, int k, void* y, long long ldy, int dtype, pae_stream stream) {
  const char* fn = "pae_linear_i8";
  if (!known(dtype)) return fail(PAE_ERR_ARG, "%s: dtype must be PAE_FP32 or PAE_BF16", fn);
  if (tokens < 0 || n < 1 || k < 1) return fail(PAE_ERR_ARG, "%s: tokens must be >= 0, n and k >= 1", fn);
  if (k % 16 || k > kMaxI8K) return fail(PAE_ERR_UNSUPPORTED, "%s: k must be a multiple of 16 and at most %d (32-bit sums)", fn, kMaxI8K);
  if (tokens > (1 << 24) || n > (1 << 24)) return fail(PAE_ERR_UNSUPPORTED, "%s: tokens and n must be at most 2^24", fn);
  if (tokens == 0) return PAE_OK;
  if (!x || !x_scale || !w || !w_scale || !y) return fail(PAE_ERR_ARG, "%s: a pointer argument is NULL", fn);
  if (ldy < n) return fail(PAE_ERR_ARG, "%s: ldy must be at least n", fn);
  if (!aligned(x, 16) || !aligned(w, 16)) return fail(PAE_ERR_ARG, "%s: codes must start on 16 bytes", fn);
  if (!aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(y, dtype == PAE_BF16 ? 2 : 4))
    return fail(PAE_ERR_ARG, "%s: a pointer is not aligned to its element", fn);
  DeviceState* d = nullptr;
  pae_status st = device_state(fn, stream, true, &d);
  if (st != PAE_OK) return st;
  const I8GemmPlan p = plan_i8_gemm(tokens, n, k, dtype == PAE_BF16 ? 2 : 4);
  CUtensorMap rows, cols, out;
  if ((st = make_map(d, &rows, p.swap ? w : x, p.swap ? n : tokens, k, i8_rows_box(p))) != PAE_OK) return st;
  if ((st = make_map(d, &cols, p.swap ? x : w, p.swap ? tokens : n, k, i8_cols_box(p))) != PAE_OK) return st;
  const size_t es = dtype == PAE_BF16 ? 2 : 4;
  // Whole boxes of 128 bytes per tile: a box may not reach into the next tile's
  // columns.  Whole pieces of 16 bytes per row: a tensor store clips at those, not at
  // the elements, and would write what lies behind a row that ends inside one.
  const bool tma = !p.swap && p.tn % (128 / es) == 0 && aligned(y, 16) && (size_t)n * es % 16 == 0 && (size_t)ldy * es % 16 == 0 &&
                   (size_t)ldy * es < (1ULL << 40);
  if (tma) {
    cuuint64_t dims[2] = {(cuuint64_t)n, (cuuint64_t)tokens};
    cuuint64_t strides[1] = {(cuuint64_t)ldy * es};
    cuuint32_t box[2] = {(cuuint32_t)(128 / es), 32};
    cuuint32_t el[2] = {1, 1};
    const CUresult r = d->encode(&out, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, y, dims,
                                 strides, box, el, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                 CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PAE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for the output", (int)r);
  }
  const I8GemmArgs a{x_scale, w_scale, y, ldy, tokens, n, k, 0, 0, DevErr{d->err_dev, kWaitNs}};
  const cudaError_t e = launch_i8_gemm(dtype == PAE_BF16, &rows, &cols, tma ? &out : nullptr, p, a,
                                       reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PAE_OK : cuda_fail(fn, e);
}

pae_status pae_kv8_write(const pae_kv8* cache, const void* k, const void* v, const long long* k_strides,
                         const long long* v_strides, const int* cu_rows, const int* start, int n_seq, int n_rows,
                         int dtype, pae_stream stream) {
  return kv8_io("pae_kv8_write", true, cache, const_cast<void*>(k), const_cast<void*>(v), k_strides, v_strides, cu_rows,
                start, n_seq, n_rows, dtype, stream);
}

pae_status pae_kv8_read(const pae_kv8* cache, void* k, void* v, const long long* k_strides, const long long* v_strides,
                        const int* cu_rows, const int* start, int n_seq, int n_rows, int dtype, pae_stream stream) {
  return kv8_io("pae_kv8_read", false, cache, k, v, k_strides, v_strides, cu_rows, start, n_seq, n_rows, dtype, stream);
}

pae_status pae_kv8_workspace(const pae_kv8* cache, int n_seq, int n_q, int n_q_heads, int n_new, size_t* bytes) {
  const char* fn = "pae_kv8_workspace";
  if (!bytes) return fail(PAE_ERR_ARG, "%s: bytes is NULL", fn);
  *bytes = 0;
  pae_status st = check_cache(fn, cache);
  if (st != PAE_OK) return st;
  Kv8AttnPlan p;
  if ((st = plan_attention(fn, cache, n_seq, n_q, n_q_heads, n_new, &p)) != PAE_OK) return st;
  if (n_seq > 0 && n_q > 0) *bytes = p.ws_bytes;
  return PAE_OK;
}

pae_status pae_kv8_attention(const pae_kv8* cache, const pae_kv8_query* q, void* workspace, size_t workspace_bytes,
                             pae_stream stream) {
  const char* fn = "pae_kv8_attention";
  pae_status st = check_cache(fn, cache);
  if (st != PAE_OK) return st;
  if (!q) return fail(PAE_ERR_ARG, "%s: the query is NULL", fn);
  Kv8AttnPlan p;
  if ((st = plan_attention(fn, cache, q->n_seq, q->n_q, q->n_q_heads, q->n_new, &p)) != PAE_OK) return st;
  if (q->causal && q->n_new > 0) return fail(PAE_ERR_ARG, "%s: fresh keys cannot be combined with causal", fn);
  if (!std::isfinite(q->scale)) return fail(PAE_ERR_ARG, "%s: scale must be finite (0: 1 / sqrt(head_dim))", fn);
  if (q->n_seq == 0 || q->n_q == 0) return PAE_OK;
  if (!q->lens || !q->q || !q->out) return fail(PAE_ERR_ARG, "%s: lens, q or out is NULL", fn);
  if (q->n_new > 0 && (!q->k_new || !q->v_new)) return fail(PAE_ERR_ARG, "%s: k_new or v_new is NULL with n_new > 0", fn);
  for (int i = 0; i < 3; ++i) {
    const long long s[4] = {q->q_strides[i], q->out_strides[i], q->n_new > 0 ? q->k_new_strides[i] : 0,
                            q->n_new > 0 ? q->v_new_strides[i] : 0};
    for (long long v : s)
      if (v < 0 || v % 8) return fail(PAE_ERR_ARG, "%s: strides must be non-negative multiples of 8 elements", fn);
  }
  if ((q->n_seq > 1 && !q->out_strides[0]) || (q->n_q > 1 && !q->out_strides[1]) || (q->n_q_heads > 1 && !q->out_strides[2]))
    return fail(PAE_ERR_ARG, "%s: output rows may not share their place (stride 0)", fn);
  if (!aligned(q->q, 16) || !aligned(q->out, 16) || (q->n_new > 0 && (!aligned(q->k_new, 16) || !aligned(q->v_new, 16))))
    return fail(PAE_ERR_ARG, "%s: q, out, k_new and v_new must start on 16 bytes", fn);
  if (p.ws_bytes > 0 && (!workspace || workspace_bytes < p.ws_bytes || !aligned(workspace, 16)))
    return fail(PAE_ERR_ARG, "%s: needs a workspace of %zu bytes on 16 bytes (pae_kv8_workspace)", fn, p.ws_bytes);
  DeviceState* d = nullptr;
  if ((st = device_state(fn, stream, true, &d)) != PAE_OK) return st;
  Kv8AttnArgs a{};
  a.c = view(cache);
  a.lens = q->lens;
  a.q = static_cast<const bf16*>(q->q);
  a.q_seq = q->q_strides[0];
  a.q_tok = q->q_strides[1];
  a.q_head = q->q_strides[2];
  a.o = static_cast<bf16*>(q->out);
  a.o_seq = q->out_strides[0];
  a.o_tok = q->out_strides[1];
  a.o_head = q->out_strides[2];
  a.n_seq = q->n_seq;
  a.n_q = q->n_q;
  a.n_new = q->n_new;
  if (q->n_new > 0) {
    a.k_new = static_cast<const bf16*>(q->k_new);
    a.v_new = static_cast<const bf16*>(q->v_new);
    a.kn_seq = q->k_new_strides[0];
    a.kn_tok = q->k_new_strides[1];
    a.kn_head = q->k_new_strides[2];
    a.vn_seq = q->v_new_strides[0];
    a.vn_tok = q->v_new_strides[1];
    a.vn_head = q->v_new_strides[2];
  }
  a.group = q->n_q_heads / cache->n_kv_heads;
  a.causal = q->causal != 0;
  a.scale_log2 = (q->scale == 0.f ? 1.f / std::sqrt((float)cache->head_dim) : q->scale) * 1.4426950408889634f;
  kv8_attn_parts(&a, p, workspace);
  a.err = DevErr{d->err_dev, kWaitNs};
  const cudaError_t e = launch_kv8_attn(p, a, true, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PAE_OK : cuda_fail(fn, e);
}

}  // extern "C"
