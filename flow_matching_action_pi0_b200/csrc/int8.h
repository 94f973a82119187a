// Launch interface of the 8-bit prefix operators (row quantiser, int8
// product, int8 K/V cache, attention over that cache), shared by their entry
// points (pae_int8.cu) and the context (pae_api.cu).  Host-side declarations.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace pae {

// Two fp32 operations in one instruction: (a, b) op (c, d).
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 d, {%6, %7};\n\t"
      "fma.rn.f32x2 c, a, b, d;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 as a pair of 16 bits, lo in the low half: one instruction, round to
// nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// One lane of a converged warp, the same one each time.  (Loops that a whole warp
// walks, one lane issuing, keep addresses and descriptors in uniform registers.)
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// ------------------------------------------------------------ row quantiser
// codes[r][i] = rint(x[r][i] / s_r), s_r = max|x[r]| / 127; scale[r] = s_r, or
// with rms_eps > 0 s_r / sqrt(mean(x[r]^2) + rms_eps): the codes of the
// normalised row are the same, only its scale changes.
cudaError_t launch_quantize_rows(bool in_bf16, const void* x, long long ldx, int rows, int width, float rms_eps,
                                 int8_t* codes, float* scale, cudaStream_t st);

// ------------------------------------------------------------- int8 product
// y[t][f] = (sum_k x[t][k] w[f][k]) sx[t] sw[f], int32 sums.
constexpr int kMaxI8K = 131056;  // the last multiple of 16 at which 2^14 k stays below 2^31
struct I8GemmPlan {
  int cg;       // CTAs per tile (2: pairs of cta_group::2; not with swap)
  int swap;     // 1: weight rows on the MMA's M side, tokens on its N side
  int tn;       // N tile (multiple of 16, 16..256)
  int tiles_m, tiles_n;
  int th;       // swap: weight rows per tile (32, 64 or 128; the MMA always spans 128)
  int splits;   // split-K cluster size (swap only)
  int stages;
  int ctas;     // persistent grid (swap == 0), in tiles in flight
};
I8GemmPlan plan_i8_gemm(int tokens, int n, int k, int out_bytes /* of an output element */);
struct I8GemmArgs {
  const float* sx;
  const float* sw;
  void* y;
  long long ldy;
  int tokens, n, k;
  int tma_out;  // set by the launch
  int w_ready;  // 1: no kernel of the stream still writes the weights, so they may be read before the previous one ends
  DevErr err;
};
cudaError_t i8_gemm_init();
// tm_rows / tm_cols: the operands on the MMA's M and N side, boxes of 128 bytes
// x i8_rows_box / i8_cols_box rows; tm_out (null: plain stores): the output,
// boxes of 32 rows x 128 bytes.
inline int i8_rows_box(const I8GemmPlan& p) { return p.swap ? p.th : 128; }
inline int i8_cols_box(const I8GemmPlan& p) { return p.swap ? p.tn : p.tn / p.cg; }
cudaError_t launch_i8_gemm(bool out_bf16, const CUtensorMap* tm_rows, const CUtensorMap* tm_cols,
                           const CUtensorMap* tm_out, const I8GemmPlan& p, const I8GemmArgs& a, cudaStream_t st);

// ---------------------------------------------------------------- K/V cache
struct Kv8 {
  int8_t *k, *v;            // [slots][heads][cap][d]
  float *k_scale, *v_scale; // [slots][heads][cap]
  int slots, heads, cap, d;
};
struct Kv8Rows {            // packed rows of n_seq sequences: sequence b is rows [cu[b], cu[b + 1])
  const int* cu;            // [n_seq + 1]; null: one sequence of n_rows rows
  const int* start;         // [n_seq] position of each sequence's first row; null: 0
  int n_seq, n_rows, slot0; // sequence b goes to slot slot0 + b
};
struct Kv8Io {              // row (t, head) at p + t * tok + head * head_stride (elements)
  void *k, *v;
  long long k_tok, k_head, v_tok, v_head;
};
// rope_cs (fp32 rows only; null: off): (cos, sin) [position][d / 2]; keys are
// rotated at their position before they are quantised.
cudaError_t launch_kv8_write(bool bf16_rows, const Kv8& c, const Kv8Rows& r, const Kv8Io& io, const float2* rope_cs,
                             cudaStream_t st);
cudaError_t launch_kv8_read(bool bf16_rows, const Kv8& c, const Kv8Rows& r, const Kv8Io& io, cudaStream_t st);

// ---------------------------------------------------------------- attention
// Keys that share the units of one reference at most (a tile's part, a warp's
// share of a row group): contributions in fp16 are off by 2^-28 of the row's
// largest each on tiles, 2^-32 in row groups, 2^-11 of it for all of them.
constexpr long long kTileRefKeys = 1 << 17, kGroupRefKeys = 1 << 21;
struct Kv8AttnPlan {
  int tc;        // 1: tcgen05 tiles of 128 query rows; 0: groups of 8 rows
  int qtiles;    // row tiles (tc) or row groups per (sequence, KV head)
  int splits;    // tc: key splits (a power of two); > 1: partial rows go to the workspace and are merged by a second launch
                 // not tc: blocks that share the keys of all sequences; ws_bytes > 0: merged likewise
  size_t ws_bytes;
};
Kv8AttnPlan plan_kv8_attn(int n_seq, int heads_kv, int group, int n_q, int n_new, int max_keys, int d);
struct Kv8AttnArgs {
  Kv8 c;
  const int* lens;          // [n_seq] valid cached positions of slot b
  const bf16* q;            // strides in elements
  long long q_seq, q_tok, q_head;
  bf16* o;
  long long o_seq, o_tok, o_head;
  const bf16 *k_new, *v_new;  // fresh keys, visible to every query (null: none)
  long long kn_seq, kn_tok, kn_head, vn_seq, vn_tok, vn_head;
  int n_seq, n_q, n_new, group;  // group = query heads per KV head
  int causal;
  float scale_log2;         // softmax scale x log2(e)
  float* part_o;            // averages over the part's keys (see kPartShift): tc [n_seq * heads][splits][rows][d], else [blocks][2][8][d]
  float2* part_ml;          // their weights as (log2, 1), see part_weight
  DevErr err;
};
// Parts are parked as averages x 2^-kPartShift, so that the sum of up to 2^14 of them
// cannot overflow where their average does not.
constexpr float kPartShift = 14.f;
// A part's weight, the log2 of its row sum, as a maximum and a sum for the
// merge: (-inf, 0) where the row saw no key, (0, NaN) where its scores are NaN.
__device__ __forceinline__ float2 part_weight(float lw) {
  return lw == -INFINITY ? make_float2(lw, 0.f) : lw == lw ? make_float2(lw, 1.f) : make_float2(0.f, lw);
}
// Place the partial rows and their statistics in a workspace of p.ws_bytes.
inline void kv8_attn_parts(Kv8AttnArgs* a, const Kv8AttnPlan& p, void* workspace) {
  a->part_o = static_cast<float*>(workspace);
  a->part_ml = reinterpret_cast<float2*>(a->part_o + p.ws_bytes / ((size_t)a->c.d * 4 + 8) * a->c.d);
}
cudaError_t kv8_attn_init();
cudaError_t launch_kv8_attn(const Kv8AttnPlan& p, const Kv8AttnArgs& a, bool pdl, cudaStream_t st);

// parts of launch_kv8_attn
cudaError_t kv8_attn_tc_init();
cudaError_t launch_kv8_attn_tc(const Kv8AttnPlan& p, const Kv8AttnArgs& a, bool pdl, cudaStream_t st);

}  // namespace pae
