// qk_rope.cu -- rotary tables of scaled frequencies, per-head norms of q and
// k with the rotation, and the paged KV cache's append and read (bf16 and
// 4-bit pages).
//
// All of it is bound by bytes: a head of a row is read once, in 16-byte
// pieces of 8 elements held by neighbouring lanes, normed, rotated and
// written (or quantised into its page) from registers.  See the kernels.
#include <cuda_fp4.h>
#include <math.h>

#include "frt_paged.cuh"

namespace frt {
namespace {

// ------------------------------------------------------------- the table --

struct TableArgs {
  int M, rot, scaling, steps;
  long P;
  double theta, factor, orig_len, low, high, amplitude;
  float* out;
};

// f_i of the header's formula.
__device__ double scaled_frequency(const TableArgs& a, int i) {
  const double e = -2.0 * i / a.rot;
  double f = pow(a.theta, e);
  if (a.scaling == FRT_ROPE_SCALE_LINEAR) f /= a.factor;
  if (a.scaling == FRT_ROPE_SCALE_BASE) f *= pow(a.factor, e * (double(a.rot) / (a.rot - 2)));
  if (a.scaling == FRT_ROPE_SCALE_PARTS) {
    const double turns = a.orig_len * f / 6.283185307179586476925;
    const double keep = fmin(fmax((turns - a.low) / (a.high - a.low), 0.0), 1.0);
    f *= keep + (1.0 - keep) / a.factor;
  }
  return f;
}

// One thread per (pair i, run of `steps` positions): cos and sin of the run's
// first angle and of the frequency itself in fp64.
__global__ void rope_table_scaled_kernel(TableArgs a) {
  const int half = a.rot / 2;
  const long runs = (long(a.M) + a.steps - 1) / a.steps;
  const long g = blockIdx.x * long(blockDim.x) + threadIdx.x;
  if (g >= runs * half) return;
  const int i = int(g % half);
  const long m0 = g / half * a.steps;
  const double f = scaled_frequency(a, i);
  const long m1 = m0 + a.steps < a.M ? m0 + a.steps : a.M;
  for (long m = m0; m < m1; ++m) {
    double s, c;
    sincos(double(a.P + m) * f, &s, &c);
    *reinterpret_cast<float2*>(a.out + m * a.rot + 2 * i) =
        make_float2(float(a.amplitude * c), float(a.amplitude * s));
  }
}

// -------------------------------------------- norm + rotation (+ append) --

struct HeadArgs {
  int rows, hq, hkv, hd, rot, layout;
  int first, heads;     // heads [first, first + heads) of a row are done
  float eps;
  double inv_hd;
  const uint16_t* qkv; long ld_qkv;
  const uint16_t* q_norm; const uint16_t* k_norm;
  const float* rope; int n_pos; const int* positions;
  uint16_t* q_out; long ld_q;
  uint16_t* k_out; long ld_k;
  PagePool pool;
  const long* slots;
  const float* k_scale; const float* v_scale;
  int* status;
};

enum { kToRows = 0, kToBf16Pages = 1, kToFp4Pages = 2 };

// 8 elements of a head (fp32) to 8 e2m1 codes; the two lanes of a 16-element
// block share its scale (header, frt_paged_kv_append); `group`: the lanes of
// the head, all of which call it.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], float rk, uint32_t group,
                                              uint8_t* scale) {
  float y[8], a = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = __fmul_rn(x[j], rk);
    a = fmaxf(a, fabsf(y[j]));  // fmaxf drops NaN
  }
  a = fmaxf(a, __shfl_xor_sync(group, a, 1));
  const __nv_fp8_storage_t s8 =
      __nv_cvt_float_to_fp8(__fdiv_rn(a, 6.0f), __NV_SATFINITE, __NV_E4M3);
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)));
  *scale = s8;
  if (s == 0.0f) return 0;
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 t = make_float2(__fdiv_rn(y[2 * j], s), __fdiv_rn(y[2 * j + 1], s));
    w |= uint32_t(__nv_cvt_float2_to_fp4x2(t, __NV_E2M1, cudaRoundNearest)) << (8 * j);
  }
  return w;
}

// LANES lanes hold a head, 8 elements each (lanes past hd / 8 idle); a group
// of LANES lanes takes U consecutive heads of one row.  Everything the group
// needs is requested before the first use.
template <int LANES, int U, int TO>
__global__ void __launch_bounds__(256) head_kernel(HeadArgs a) {
  const int lane = int(threadIdx.x) % LANES;
  // the group's lanes of the warp: other groups may be at other kinds of heads
  const uint32_t group = (0xffffffffu >> (32 - LANES)) << (threadIdx.x % 32 / LANES * LANES);
  const int parts = (a.heads + U - 1) / U;
  const long unit = (long(blockIdx.x) * blockDim.x + threadIdx.x) / LANES;
  const long row = unit / parts;
  const int h0 = a.first + int(unit - row * parts) * U;
  const int h_end = a.first + a.heads;
  const bool live = row < a.rows;       // the whole group's: it shares a row
  const bool mine = live && lane * 8 < a.hd;
  pdl_trigger();
  pdl_wait();

  long pos = live ? row : 0, slot = -1;
  if (live && a.positions) pos = a.positions[row];
  if constexpr (TO != kToRows) {
    if (live) slot = a.slots[row];
  }
  uint4 xv[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (mine && h0 + u < h_end)
      xv[u] = *reinterpret_cast<const uint4*>(a.qkv + row * a.ld_qkv + long(h0 + u) * a.hd + lane * 8);
    else
      xv[u] = make_uint4(0, 0, 0, 0);

  const bool bad_pos = a.rot > 0 && (pos < 0 || pos >= a.n_pos);
  bool bad_slot = false;
  if constexpr (TO != kToRows) bad_slot = slot >= a.pool.slots();
  if (live && (bad_pos || bad_slot) && lane == 0) atomicExch(a.status, FRT_ERANGE);

  // this lane's (cos, sin): pairs 4*lane.. (adjacent) or 8*lane.. modulo rot/2 (halves)
  const bool rotates = mine && lane * 8 < a.rot && !bad_pos;
  const int half_lanes = a.rot / 16;
  const bool second = lane >= half_lanes;
  float cs[16];
  if (rotates) {
    const float* t = a.rope + pos * a.rot;
    const int n4 = a.layout == FRT_ROPE_HALF ? 4 : 2;
    t += a.layout == FRT_ROPE_HALF ? (second ? lane - half_lanes : lane) * 16 : lane * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n4) {
        const float4 v = *reinterpret_cast<const float4*>(t + 4 * j);
        cs[4 * j] = v.x; cs[4 * j + 1] = v.y; cs[4 * j + 2] = v.z; cs[4 * j + 3] = v.w;
      }
  }
  const int partner = second ? lane - half_lanes : lane + half_lanes;

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u;
    const bool on = h < h_end;
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
    float x[8];
    unpack8(xv[u], x);
    const uint16_t* w = is_v ? nullptr : is_q ? a.q_norm : a.k_norm;
    float r = 1.0f;
    if (w) {  // uniform over the group: it depends on h alone
      // squares of bf16 are exact in fp32; the sum is carried in fp64, so
      // that a key next to a 4-bit border does not depend on its order
      double s = 0.0;
#pragma unroll
      for (int j = 0; j < 8; ++j) s += double(x[j] * x[j]);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1)
        s += __shfl_xor_sync(group, s, o, LANES);
      const float m = __fadd_rn(float(s * a.inv_hd), a.eps);
      r = __frcp_rn(__fsqrt_rn(m));
      float wv[8];
      if (mine) {
        unpack8(*reinterpret_cast<const uint4*>(w + lane * 8), wv);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(__fmul_rn(x[j], r), wv[j]);
      }
    }
    if (!is_v && a.rot > 0) {
      if (a.layout == FRT_ROPE_HALF) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float o = __shfl_sync(group, x[j], partner, LANES);
          if (rotates)
            x[j] = second ? __fadd_rn(__fmul_rn(o, cs[2 * j + 1]), __fmul_rn(x[j], cs[2 * j]))
                          : __fsub_rn(__fmul_rn(x[j], cs[2 * j]), __fmul_rn(o, cs[2 * j + 1]));
        }
      } else if (rotates) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = x[2 * j], x1 = x[2 * j + 1], c = cs[2 * j], s = cs[2 * j + 1];
          x[2 * j] = __fsub_rn(__fmul_rn(x0, c), __fmul_rn(x1, s));
          x[2 * j + 1] = __fadd_rn(__fmul_rn(x0, s), __fmul_rn(x1, c));
        }
      }
    }
    const uint4 o = pack8_bf16(x);
    const bool write = mine && on && !bad_pos;
    if (is_q) {
      if (write) *reinterpret_cast<uint4*>(a.q_out + row * a.ld_q + long(h) * a.hd + lane * 8) = o;
    } else if constexpr (TO == kToRows) {
      if (write)
        *reinterpret_cast<uint4*>(a.k_out + row * a.ld_k + long(h - a.hq) * a.hd + lane * 8) = o;
    } else {
      const int kvh = is_v ? h - a.hq - a.hkv : h - a.hq;
      const bool cached = write && slot >= 0 && !bad_slot;
      uint8_t* rec = cached ? a.pool.record(slot, kvh) : nullptr;
      const int at = cached ? a.pool.row(slot) : 0;
      if constexpr (TO == kToBf16Pages) {
        if (cached)
          *reinterpret_cast<uint4*>(rec + (long(is_v ? a.pool.page_size : 0) + at) * a.hd * 2 + lane * 16) = o;
      } else {
        unpack8(o, x);  // what is cached is the bf16 key
        uint8_t s8;
        const uint32_t codes = quantise8(x, __frcp_rn(*(is_v ? a.v_scale : a.k_scale)), group, &s8);
        if (cached) {
          rec += is_v ? a.pool.record_bytes / 2 : 0;
          *reinterpret_cast<uint32_t*>(rec + long(at) * (a.hd / 2) + lane * 4) = codes;
          if ((lane & 1) == 0)
            rec[a.pool.page_size * (a.hd / 2) + long(at) * (a.hd / 16) + lane / 2] = s8;
        }
      }
    }
  }
}

template <int LANES, int U>
int launch_heads(int to, const HeadArgs& a, cudaStream_t s) {
  const long units = long(a.rows) * ((a.heads + U - 1) / U);
  const long blocks = (units * LANES + 255) / 256;
  FRT_REQUIRE(blocks <= 0x7fffffffL, FRT_ESHAPE, "rows * heads is too large");
  const dim3 grid{unsigned(blocks)}, block{256};
  switch (to) {
    case kToRows: return launch_pdl("frt_qk_norm_rope", head_kernel<LANES, U, kToRows>, grid, block, 0, s, a);
    case kToBf16Pages: return launch_pdl("frt_paged_kv_append", head_kernel<LANES, U, kToBf16Pages>, grid, block, 0, s, a);
    default: return launch_pdl("frt_paged_kv_append", head_kernel<LANES, U, kToFp4Pages>, grid, block, 0, s, a);
  }
}

int launch_heads(int to, const HeadArgs& a, cudaStream_t s) {
  // One head a group while the heads do not fill the GPU (latency), four
  // once they do (the table row and the index arithmetic are shared).
  const int lanes = a.hd <= 64 ? 8 : a.hd <= 128 ? 16 : 32;
  const bool few = long(a.rows) * a.heads * lanes <= num_sms() * 2048L;
  if (lanes == 8) return few ? launch_heads<8, 1>(to, a, s) : launch_heads<8, 4>(to, a, s);
  if (lanes == 16) return few ? launch_heads<16, 1>(to, a, s) : launch_heads<16, 4>(to, a, s);
  return few ? launch_heads<32, 1>(to, a, s) : launch_heads<32, 4>(to, a, s);
}

// ------------------------------------------------------------------ read --

struct ReadArgs {
  int rows, hkv, hd, fp4;
  PagePool pool;
  const long* slots;
  const float* k_scale; const float* v_scale;
  uint16_t* k_out; long ld_k;
  uint16_t* v_out; long ld_v;
  int* status;
};

// One thread per 8 elements of a cached head.
__global__ void __launch_bounds__(256) read_kernel(ReadArgs a) {
  const int hd8 = a.hd / 8;
  const long g = blockIdx.x * 256L + threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const long row = g / (2L * a.hkv * hd8);
  if (row >= a.rows) return;
  const int c = int(g - row * (2L * a.hkv * hd8));
  const int h2 = c / hd8, p = c - h2 * hd8;  // h2: the k heads, then the v heads
  const bool is_v = h2 >= a.hkv;
  const int h = is_v ? h2 - a.hkv : h2;
  uint16_t* out = is_v ? a.v_out : a.k_out;
  if (!out) return;
  const long slot = a.slots[row];
  if (slot < 0) return;
  if (slot >= a.pool.slots()) {
    atomicExch(a.status, FRT_ERANGE);
    return;
  }
  const uint8_t* rec = a.pool.record(slot, h);
  const int at = a.pool.row(slot);
  uint4 o;
  if (a.fp4) {
    rec += is_v ? a.pool.record_bytes / 2 : 0;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + long(at) * (a.hd / 2) + p * 4);
    const __nv_fp8_storage_t s8 = rec[a.pool.page_size * (a.hd / 2) + long(at) * (a.hd / 16) + p / 2];
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)));
    const float k = *(is_v ? a.v_scale : a.k_scale);
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 v(__nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t(w >> (8 * j)), __NV_E2M1));
      x[2 * j] = __fmul_rn(__fmul_rn(__low2float(v), s), k);
      x[2 * j + 1] = __fmul_rn(__fmul_rn(__high2float(v), s), k);
    }
    o = pack8_bf16(x);
  } else {
    o = *reinterpret_cast<const uint4*>(rec + (long(is_v ? a.pool.page_size : 0) + at) * a.hd * 2 + p * 16);
  }
  *reinterpret_cast<uint4*>(out + row * (is_v ? a.ld_v : a.ld_k) + long(h) * a.hd + p * 8) = o;
}

// ---------------------------------------------------------------- checks --

// A row tensor: 16-byte aligned, its stride a multiple of 8 that holds `width`.
int check_rows(const char* name, const void* p, long ld, long width) {
  FRT_REQUIRE(p, FRT_EINVAL, "%s is required", name);
  FRT_REQUIRE(aligned(p, 16) && ld % 8 == 0, FRT_EALIGN,
              "%s must be 16-byte aligned with a row stride that is a multiple of 8", name);
  FRT_REQUIRE(ld >= width, FRT_ESHAPE, "%s: the row stride %ld is less than its %ld columns", name,
              ld, width);
  return FRT_OK;
}

int check_heads(const frt_qk_rope_desc* d) {
  FRT_REQUIRE(d, FRT_EINVAL, "descriptor is NULL");
  FRT_REQUIRE(d->rows >= 0 && d->hq >= 0 && d->hkv >= 0 && d->hq <= 65536 && d->hkv <= 65536,
              FRT_ESHAPE, "bad rows / heads: %d, %d, %d", d->rows, d->hq, d->hkv);
  FRT_REQUIRE(d->hd >= 16 && d->hd <= 256 && d->hd % 8 == 0, FRT_ESHAPE,
              "hd must be a multiple of 8 in [16, 256], got %d", d->hd);
  return FRT_OK;
}

int check_rotation(const frt_qk_rope_desc* d) {
  FRT_REQUIRE(d->rot >= 0 && d->rot <= d->hd && d->rot % 16 == 0, FRT_ESHAPE,
              "rot must be a multiple of 16 in [0, hd], got %d", d->rot);
  FRT_REQUIRE(d->layout == FRT_ROPE_PAIRS || d->layout == FRT_ROPE_HALF, FRT_EINVAL,
              "unknown rotary layout %d", d->layout);
  FRT_REQUIRE(d->eps >= 0.0f, FRT_EINVAL, "eps must be >= 0");
  FRT_REQUIRE((!d->q_norm || aligned(d->q_norm, 16)) && (!d->k_norm || aligned(d->k_norm, 16)),
              FRT_EALIGN, "norm weights must be 16-byte aligned");
  if (d->rot > 0) {
    FRT_REQUIRE(d->rope, FRT_EINVAL, "rope is required when rot > 0");
    FRT_REQUIRE(aligned(d->rope, 16), FRT_EALIGN, "rope must be 16-byte aligned");
    FRT_REQUIRE(d->n_pos >= 1, FRT_ESHAPE, "n_pos must be >= 1, got %d", d->n_pos);
    FRT_REQUIRE(d->positions || d->rows <= d->n_pos, FRT_ERANGE,
                "%d rows without positions exceed the table's %d", d->rows, d->n_pos);
  }
  FRT_REQUIRE(!d->positions || aligned(d->positions, 4), FRT_EALIGN, "positions must be 4-byte aligned");
  return FRT_OK;
}

int check_pool(const frt_qk_rope_desc* d) {
  FRT_REQUIRE(d->hkv >= 1, FRT_ESHAPE, "hkv must be >= 1");
  FRT_REQUIRE(d->format == FRT_PAGE_BF16 || d->format == FRT_PAGE_E2M1, FRT_EINVAL,
              "unknown page format %d", d->format);
  FRT_REQUIRE(frt_kv_record_bytes(d->format, d->page_size, d->hd) > 0, FRT_ESHAPE,
              "no page of format %d with page_size %d and hd %d", d->format, d->page_size, d->hd);
  FRT_REQUIRE(d->n_pages >= 0, FRT_ESHAPE, "n_pages must be >= 0");
  FRT_REQUIRE(d->pool && d->slots, FRT_EINVAL, "pool and slots are required");
  FRT_REQUIRE(aligned(d->pool, 16) && aligned(d->slots, 8), FRT_EALIGN,
              "pool must be 16-byte and slots 8-byte aligned");
  if (d->format == FRT_PAGE_E2M1) {
    FRT_REQUIRE(d->k_scale && d->v_scale, FRT_EINVAL, "k_scale and v_scale are required");
    FRT_REQUIRE(aligned(d->k_scale, 4) && aligned(d->v_scale, 4), FRT_EALIGN,
                "k_scale and v_scale must be 4-byte aligned");
  }
  return FRT_OK;
}

HeadArgs head_args(const frt_qk_rope_desc* d) {
  HeadArgs a{};
  a.rows = d->rows; a.hq = d->hq; a.hkv = d->hkv; a.hd = d->hd; a.rot = d->rot;
  a.layout = d->layout; a.eps = d->eps; a.inv_hd = 1.0 / d->hd;
  a.qkv = d->qkv; a.ld_qkv = d->ld_qkv;
  a.q_norm = d->q_norm; a.k_norm = d->k_norm;
  a.rope = d->rope; a.n_pos = d->n_pos; a.positions = d->positions;
  a.q_out = d->q_out; a.ld_q = d->ld_q; a.k_out = d->k_out; a.ld_k = d->ld_k;
  a.slots = d->slots; a.k_scale = d->k_scale; a.v_scale = d->v_scale;
  a.status = device_status_ptr();
  return a;
}

PagePool page_pool(const frt_qk_rope_desc* d) {
  return make_page_pool(const_cast<void*>(static_cast<const void*>(d->pool)), d->format,
                        d->page_size, d->n_pages, d->hkv, d->hd);
}

}  // namespace
}  // namespace frt

extern "C" int frt_build_rope_table_scaled(int M, int rot, long P, double theta, int scaling,
                                           double factor, double orig_len, double low_turns,
                                           double high_turns, double amplitude, float* rope_out,
                                           void* stream) {
  frt::clear_error();
  FRT_REQUIRE(M >= 0 && P >= 0, FRT_ESHAPE, "M and P must be >= 0");
  FRT_REQUIRE(rot >= 2 && rot <= 65536 && rot % 2 == 0, FRT_ESHAPE,
              "rot must be even and in [2, 65536], got %d", rot);
  FRT_REQUIRE(theta > 0.0 && isfinite(theta), FRT_EINVAL, "theta must be > 0");
  FRT_REQUIRE(scaling >= FRT_ROPE_SCALE_NONE && scaling <= FRT_ROPE_SCALE_PARTS, FRT_EINVAL,
              "unknown frequency scaling %d", scaling);
  FRT_REQUIRE(isfinite(amplitude), FRT_EINVAL, "amplitude must be finite");
  if (scaling != FRT_ROPE_SCALE_NONE)
    FRT_REQUIRE(factor > 0.0 && isfinite(factor), FRT_EINVAL, "factor must be > 0");
  if (scaling == FRT_ROPE_SCALE_BASE)
    FRT_REQUIRE(rot > 2, FRT_ESHAPE, "a scaled base needs rot > 2");
  if (scaling == FRT_ROPE_SCALE_PARTS)
    FRT_REQUIRE(orig_len > 0.0 && isfinite(orig_len) && isfinite(low_turns) &&
                    isfinite(high_turns) && high_turns > low_turns,
                FRT_EINVAL, "scaling by parts needs orig_len > 0 and high_turns > low_turns");
  FRT_REQUIRE(rope_out, FRT_EINVAL, "rope_out is required");
  FRT_REQUIRE(frt::aligned(rope_out, 8), FRT_EALIGN, "rope_out must be 8-byte aligned");
  if (M == 0) return FRT_OK;
  frt::TableArgs a{M, rot, scaling, 1, P, theta, factor, orig_len, low_turns, high_turns, amplitude, rope_out};
  const long threads = (long(M) + a.steps - 1) / a.steps * (rot / 2);
  const long blocks = (threads + 255) / 256;
  FRT_REQUIRE(blocks <= 0x7fffffffL, FRT_ESHAPE, "M * rot is too large");
  frt::rope_table_scaled_kernel<<<unsigned(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return frt::check_launch("frt_build_rope_table_scaled");
}

extern "C" size_t frt_kv_record_bytes(int format, int page_size, int hd) {
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1))) return 0;
  if (hd < 16 || hd > 256) return 0;
  if (format == FRT_PAGE_BF16 && hd % 8 == 0) return size_t(page_size) * hd * 4;
  if (format == FRT_PAGE_E2M1 && hd % 16 == 0) return size_t(page_size) * (hd / 2 + hd / 16) * 2;
  return 0;
}

extern "C" int frt_qk_norm_rope(const frt_qk_rope_desc* d, void* stream) {
  frt::clear_error();
  if (int rc = frt::check_heads(d)) return rc;
  if (int rc = frt::check_rotation(d)) return rc;
  FRT_REQUIRE(d->hq + d->hkv >= 1, FRT_ESHAPE, "there are no heads");
  if (d->rows == 0) return FRT_OK;
  const long hd = d->hd;
  // the row's v heads are not read, so only q and k have to fit the stride
  if (int rc = frt::check_rows("qkv", d->qkv, d->ld_qkv, (d->hq + d->hkv) * hd)) return rc;
  if (d->hq)
    if (int rc = frt::check_rows("q_out", d->q_out, d->ld_q, d->hq * hd)) return rc;
  if (d->hkv)
    if (int rc = frt::check_rows("k_out", d->k_out, d->ld_k, d->hkv * hd)) return rc;
  frt::HeadArgs a = frt::head_args(d);
  FRT_REQUIRE(a.status, FRT_ECUDA, "device status word unavailable");
  a.first = 0;
  a.heads = d->hq + d->hkv;
  return frt::launch_heads(frt::kToRows, a, static_cast<cudaStream_t>(stream));
}

extern "C" int frt_paged_kv_append(const frt_qk_rope_desc* d, void* stream) {
  frt::clear_error();
  if (int rc = frt::check_heads(d)) return rc;
  if (int rc = frt::check_rotation(d)) return rc;
  if (d->rows == 0) return FRT_OK;
  if (int rc = frt::check_pool(d)) return rc;
  const long hd = d->hd;
  if (int rc = frt::check_rows("qkv", d->qkv, d->ld_qkv, (d->hq + 2L * d->hkv) * hd)) return rc;
  if (d->hq && d->q_out)
    if (int rc = frt::check_rows("q_out", d->q_out, d->ld_q, d->hq * hd)) return rc;
  frt::HeadArgs a = frt::head_args(d);
  FRT_REQUIRE(a.status, FRT_ECUDA, "device status word unavailable");
  a.pool = frt::page_pool(d);
  a.first = d->q_out ? 0 : d->hq;
  a.heads = d->hq + 2 * d->hkv - a.first;
  return frt::launch_heads(d->format == FRT_PAGE_BF16 ? frt::kToBf16Pages : frt::kToFp4Pages, a,
                           static_cast<cudaStream_t>(stream));
}

extern "C" int frt_paged_kv_read(const frt_qk_rope_desc* d, void* stream) {
  frt::clear_error();
  if (int rc = frt::check_heads(d)) return rc;
  if (d->rows == 0) return FRT_OK;
  if (int rc = frt::check_pool(d)) return rc;
  FRT_REQUIRE(d->k_out || d->v_out, FRT_EINVAL, "k_out or v_out is required");
  const long width = long(d->hkv) * d->hd;
  if (d->k_out)
    if (int rc = frt::check_rows("k_out", d->k_out, d->ld_k, width)) return rc;
  if (d->v_out)
    if (int rc = frt::check_rows("v_out", d->v_out, d->ld_v, width)) return rc;
  frt::ReadArgs a{d->rows, d->hkv, d->hd, d->format == FRT_PAGE_E2M1, frt::page_pool(d), d->slots,
                  d->k_scale, d->v_scale, d->k_out, d->ld_k, d->v_out, d->ld_v,
                  frt::device_status_ptr()};
  FRT_REQUIRE(a.status, FRT_ECUDA, "device status word unavailable");
  const long blocks = (2L * d->rows * d->hkv * (d->hd / 8) + 255) / 256;
  FRT_REQUIRE(blocks <= 0x7fffffffL, FRT_ESHAPE, "rows * heads is too large");
  return frt::launch_pdl("frt_paged_kv_read", frt::read_kernel, dim3(unsigned(blocks)), dim3(256),
                         0, static_cast<cudaStream_t>(stream), a);
}
