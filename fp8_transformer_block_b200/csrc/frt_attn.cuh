// frt_attn.cuh -- what the attention kernels over 4-bit pages share: their
// arguments, one sequence's extent, and the widening of the codes to fp16.
#pragma once

#include <cuda_fp16.h>

#include "frt_paged.cuh"
#include "frt_sm100.cuh"

namespace frt {

constexpr uint64_t kAttnWaitNs = 2000000000ull;  // 2 s per wait
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The least factor from a row's products to its base-2 scores, so that a
// hidden score (-inf) stays hidden: where the scale, or its product with the
// row's power of two, is below it, scores are within 2^-100 of 0 either way.
constexpr float kLeastFactor = 1.17549435e-38f;
__device__ __forceinline__ float score_factor(float scale, float up) {
  const float f = fabsf(scale) * up;
  return f < kLeastFactor ? kLeastFactor : f;   // a NaN stays
}
// the running maximum of a row that has seen no key: below every score, and
// finite, so that a hidden score's distance to it is -inf
constexpr float kNoKey = -3.402823466e38f;
// Weights are 2^(score - m) and go to the tensor cores in fp16.  m is set to
// the largest score so far less kLift, and again once a score passes m by
// kGrow: weights stay below 2^15, and those down to 2^-21 of the largest keep
// all eleven bits (the least step is 2^-31 of it).
constexpr float kLift = 7.0f, kGrow = 15.0f;
// A weight's exponent is one fused multiply-add, factor * product - m, which
// keeps what a rounded m cannot hold of the largest score: up to 2^-24 of it.
// Products are below 2 * 2688 a term (twice that for |q| from 2^127 on); a row
// whose factor could take them past scores of 2^22 has the rounded scores in
// their place, and a factor of 1.
template <int HD>
__device__ __forceinline__ bool is_far(float factor) {
  return factor > 4194304.0f / (HD * 5376);
}

struct AttnArgs {
  int n_seqs, rows, max_q, hq, hkv, group, causal, window;
  int max_pages;
  float sm_scale;
  const uint16_t* q; long ld_q;
  PagePool pool;
  const int* page_table;
  const int* cu_rows;
  const int* kv_len;
  const float* k_scale; const float* v_scale;
  uint16_t* out; long ld_out;
  float* lse;
  int* counters;     // [grid], zero between calls
  float* partials;   // [grid][2] tiles
  int* status;
};

// One sequence: its query rows, its keys, and what its work is cut into.
struct Seq {
  int r0, Lq, L;        // first row, query rows, keys
  int chunk0, chunks;   // the chunks any of its queries sees (one at least)
  int tiles;            // row tiles of each kv head
  __device__ long work(int hkv) const { return long(chunks) * hkv * tiles; }
};

template <int R, int CK>
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int s, bool report) {
  Seq q;
  const long want0 = a.cu_rows ? a.cu_rows[s] : long(s) * a.max_q;
  const long want1 = a.cu_rows ? a.cu_rows[s + 1] : long(s + 1) * a.max_q;
  const long r0 = min(max(want0, 0L), long(a.rows));
  const long r1 = min(min(max(want1, r0), long(a.rows)), r0 + a.max_q);
  const long cap = long(a.max_pages) * a.pool.page_size;
  const long want_l = a.kv_len[s];
  const long L = min(max(want_l, 0L), cap);
  if (report && (r0 != want0 || r1 != want1 || L != want_l)) atomicExch(a.status, FRT_ERANGE);
  q.r0 = int(r0);
  q.Lq = int(r1 - r0);
  q.L = int(L);
  q.tiles = (q.Lq * a.group + R - 1) / R;
  const long first = a.window > 0 ? max(0L, L - q.Lq - a.window + 1) : 0;
  q.chunk0 = int(first / CK);
  q.chunks = max(1, int((L + CK - 1) / CK) - q.chunk0);
  return q;
}

// The biased exponent of the power of two that a row of q is divided by: that
// of its largest, as near as both the power and its inverse are normal numbers
// (so a row is below 2, or below 4 from 2^127 on).
__device__ __forceinline__ int q_exponent(float largest) {
  return min(max(int(__float_as_uint(largest) >> 23), 1), 253);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The four bytes of w, two e2m1 codes each, as fp16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// Two e4m3 codes (low byte first) as an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(h) : "r"(w));
  return h;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The kernels for many query rows (paged_attn_many.cu): workspace, launch.
size_t attn_many_workspace(int hd, int n_seqs, int max_q, int hq, int hkv);
int attn_many_launch(const AttnArgs& a, int hd, void* workspace, cudaStream_t stream);
// Opts a kernel into its dynamic shared memory on the current device.
int allow_smem(const void* kern, int bytes);

}  // namespace frt
