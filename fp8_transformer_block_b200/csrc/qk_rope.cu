// qk_rope.cu -- rotary tables of scaled frequencies, per-head norms of q and
// k with the rotation, and the paged KV cache's append and read (bf16 and
// 4-bit pages).
//
// The floor of all of it is its bytes: a head of a row is read once, in 16-byte
// pieces of 8 elements, normed, rotated and written (or quantised into its
// page) from registers.  What the kernels reach is beside them.
#include <cuda_fp4.h>
#include <math.h>

#include "frt_paged.cuh"

namespace frt {
namespace {

// ------------------------------------------------------------- the table --

struct TableArgs {
  int M, rot, scaling, steps;
  long P;
  double log2_base, log2_base_lo;  // of the (scaled) base, in two parts
  double factor, orig_len, low, high, amplitude;
  float* out;
};

// f_i of the header's formula.  base^(-2i/rot) = 2^(e L): the rounding of the
// exponent e = -2i/rot and of its product with L (up to 2^5) would cost a
// few bits, so both are carried in two parts.
__device__ __forceinline__ double scaled_frequency(const TableArgs& a, int i) {
  const double e = -2.0 * i / a.rot;
  const double e_lo = fma(-e, double(a.rot), -2.0 * i) / a.rot;
  const double x = e * a.log2_base;
  const double x_lo = fma(e, a.log2_base, -x) + (e * a.log2_base_lo + e_lo * a.log2_base);
  double f = exp2(x);
  f = fma(f, x_lo * 0.693147180559945309417, f);
  if (a.scaling == FRT_ROPE_SCALE_LINEAR) f /= a.factor;
  if (a.scaling == FRT_ROPE_SCALE_PARTS) {
    const double turns = a.orig_len * f / 6.283185307179586476925;
    const double keep = fmin(fmax((turns - a.low) / (a.high - a.low), 0.0), 1.0);
    f *= keep + (1.0 - keep) / a.factor;
  }
  return f;
}

// One thread per (pair i, run of `steps` positions).  cos and sin of the
// run's middle angle and of one step are evaluated in fp64; the others
// follow by the addition theorem, outwards in both directions: at most
// steps/2 <= 16 complex products, 2^-53 each, against the 2^-24 of the fp32
// result.  131072 x 128 by parts: 16.4 us, 4.1 TB/s; the floor of its bytes is
// 10.4, and 71 % of the issue slots go to the fp64 of each run's start and the
// products.  Short tables: the latency of exp2 and sincos.
__global__ void __launch_bounds__(256) rope_table_scaled_kernel(TableArgs a) {
  const int half = a.rot / 2;
  const long g = blockIdx.x * 256L + threadIdx.x;
  const long run = g / half;
  const int i = int(g - run * half);
  const long m0 = run * a.steps;
  if (m0 >= a.M) return;
  const double f = scaled_frequency(a, i);
  const long m1 = min(m0 + a.steps, long(a.M)), mid = (m0 + m1) / 2;
  float* out = a.out + 2 * i;
  auto put = [&](long m, double c, double s) {
    *reinterpret_cast<float2*>(out + m * a.rot) =
        make_float2(float(a.amplitude * c), float(a.amplitude * s));
  };
  double s0, c0;
  sincos(double(a.P + mid) * f, &s0, &c0);
  put(mid, c0, s0);
  if (m1 - m0 == 1) return;
  double ds, dc, cu = c0, su = s0, cd = c0, sd = s0;
  sincos(f, &ds, &dc);
  for (int k = 1; k <= mid - m0; ++k) {
    double n = fma(cd, dc, sd * ds);
    sd = fma(sd, dc, -(cd * ds));
    cd = n;
    put(mid - k, cd, sd);
    if (mid + k < m1) {
      n = fma(cu, dc, -(su * ds));
      su = fma(su, dc, cu * ds);
      cu = n;
      put(mid + k, cu, su);
    }
  }
}

// -------------------------------------------- norm + rotation (+ append) --

struct HeadArgs {
  int rows, hq, hkv, hd, rot, layout;
  int q_units;          // groups of U q heads in a row
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

// Where a lane's two pieces of 8 elements lie in a head.  Lane l < rot/16
// holds pieces l and rot/16 + l, which a rotation of halves pairs element by
// element; the others share out what is not rotated.
struct Pieces {
  int turn, rest;  // rot / 16; lanes for the unrotated pieces
  __device__ __forceinline__ int piece(int lane, int slot) const {
    return lane < turn ? lane + slot * turn : 2 * turn + (lane - turn) + slot * rest;
  }
  // the lane and slot that hold a piece
  __device__ __forceinline__ void find(int p, int* lane, int* slot) const {
    const int i = p - 2 * turn;
    *slot = i < 0 ? p >= turn : i >= rest;
    *lane = i < 0 ? p - *slot * turn : turn + i - *slot * rest;
  }
};

__device__ __forceinline__ float absmax8(const uint64_t (&y)[4]) {
  float a = 0.0f;  // fmaxf drops NaN
#pragma unroll
  for (int j = 0; j < 4; ++j) a = absmax2(a, y[j]);
  return a;
}

// The scale of a block whose largest magnitude is `a` (header,
// frt_paged_kv_append).  a / 6 and y / scale below are correctly rounded
// quotients, so that ties fall as the definition says: q = x r with r the
// correctly rounded reciprocal, corrected by its exact remainder (Markstein
// 1990).  a is held to 8192, far past the largest scale's 2688.
__device__ __forceinline__ uint8_t block_scale(float a) {
  a = fminf(a, 8192.0f);
  constexpr float kSixth = 1.0f / 6.0f;
  const float q = __fmul_rn(a, kSixth);
  const float t = __fmaf_rn(__fmaf_rn(q, -6.0f, a), kSixth, q);
  return __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
}

// 8 elements of a block with that scale to e2m1 codes, from their negatives n:
// the remainder q s + n and its product with -r then keep the sign of a zero.
__device__ __forceinline__ uint32_t quantise8(const uint64_t (&n)[4], uint8_t s8) {
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)));
  const float r = s == 0.0f ? 0.0f : __frcp_rn(s);   // scale 0: codes 0
  const uint64_t nr2 = f2_pack(-r, -r), s2 = f2_pack(s, s);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t q = mul2(n[j], nr2);
    const uint64_t t = fma2(fma2(q, s2, n[j]), nr2, q);
    w |= uint32_t(__nv_cvt_float2_to_fp4x2(make_float2(f2_lo(t), f2_hi(t)), __NV_E2M1,
                                           cudaRoundNearest)) << (8 * j);
  }
  return s == 0.0f ? 0 : w;
}

// LANES lanes hold a head, 16 elements each in two pieces (lanes past hd / 16
// idle); a group of LANES lanes takes U consecutive heads of one kind (q, k
// or v) of one row, one after another, the next one's elements under way.
// 8192 rows of 24 + 24 heads of 128, normed and rotated, run in 45 us: 4.5
// TB/s, where the bytes alone would take 31, with 63 % of the issue slots and
// a third of the warps (registers); the waits are fixed latencies, loads and
// the conversions' pipe alike.  24 warps an SM (80 registers) measured better than 16
// with more registers (54 us) and than 32 with spills (63 us), one loop over
// the heads better than U heads in registers at once (58 us).  Into pages, a
// unit's work hangs on its slot as well, and the blocks go from unit to unit
// with the next one's index words and first head under way (16381 rows of 32 +
// 8 + 8 heads of 128 into 4-bit pages: 109 us against 129; the rows form loses
// by it, 51 us against 45).
template <int LANES, int U, int TO>
__global__ void __launch_bounds__(256, U == 1 || TO != kToRows ? 2 : 3) head_kernel(HeadArgs a) {
  const int lane = int(threadIdx.x) % LANES;
  // the group's lanes of the warp: other groups may be at other kinds of heads
  const uint32_t group = (0xffffffffu >> (32 - LANES)) << (threadIdx.x % 32 / LANES * LANES);
  Pieces at;
  at.turn = a.rot / 16;
  at.rest = (a.hd / 8 - 2 * at.turn + 1) / 2;
  const int p0 = at.piece(lane, 0), p1 = at.piece(lane, 1);
  const bool has0 = p0 * 8 < a.hd && lane < at.turn + at.rest;
  const bool has1 = has0 && p1 * 8 < a.hd;
  const bool half = a.layout == FRT_ROPE_HALF;
  // all rows' q heads, then all k heads, then all v heads: a warp's groups
  // are at one kind, and so on one path
  const uint32_t kv_units = (uint32_t(a.hkv) + U - 1) / U;
  const uint32_t n_q = uint32_t(a.rows) * a.q_units, n_k = uint32_t(a.rows) * kv_units;
  const uint32_t n_units = n_q + n_k * (TO == kToRows ? 1 : 2);
  const uint32_t stride = gridDim.x * (256 / LANES);
  uint32_t unit = uint32_t(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;
  pdl_trigger();
  pdl_wait();
  if (unit >= n_units) return;   // the whole group

  // what is loaded ahead for a unit: its row's index words, its first head
  struct Ahead {
    uint32_t row;
    int kind, j0;      // 0 q, 1 k, 2 v; the first of the kind's heads
    int pos;
    long slot;
    const uint16_t* src;
  } next;
  uint4 n0 = make_uint4(0, 0, 0, 0), n1 = n0;   // the next head's pieces
  auto look_ahead = [&](uint32_t x) {
    next.kind = x < n_q ? 0 : x < n_q + n_k ? 1 : 2;
    x -= next.kind == 0 ? 0 : next.kind == 1 ? n_q : n_q + n_k;
    const uint32_t per_row = next.kind == 0 ? uint32_t(a.q_units) : kv_units;
    next.row = x / per_row;
    next.j0 = int(x - next.row * per_row) * U;
    next.pos = a.rot > 0 ? a.positions ? a.positions[next.row] : int(next.row) : 0;
    if constexpr (TO != kToRows) next.slot = a.slots[next.row];
    next.src = a.qkv + long(next.row) * a.ld_qkv +
               long(next.j0 + (next.kind > 0 ? a.hq : 0) + (next.kind > 1 ? a.hkv : 0)) * a.hd;
    if (has0) n0 = *reinterpret_cast<const uint4*>(next.src + p0 * 8);
    if (has1) n1 = *reinterpret_cast<const uint4*>(next.src + p1 * 8);
  };
  look_ahead(unit);

#pragma unroll 1
  for (;;) {
    const Ahead now = next;
    const long row = now.row, slot = TO != kToRows ? now.slot : 0;
    const int j0 = now.j0, pos = now.pos;
    const bool is_q = now.kind == 0, is_v = now.kind == 2;
    const int jn = min(U, (is_q ? a.hq : a.hkv) - j0);
    const uint16_t* src = now.src;
    const uint16_t* w = is_v ? nullptr : is_q ? a.q_norm : a.k_norm;
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    if (w) {
      if (has0) w0 = *reinterpret_cast<const uint4*>(w + p0 * 8);
      if (has1) w1 = *reinterpret_cast<const uint4*>(w + p1 * 8);
    }
    float static_scale = 1.0f;
    if constexpr (TO == kToFp4Pages) static_scale = *(is_v ? a.v_scale : a.k_scale);

    const bool bad_pos = a.rot > 0 && (pos < 0 || pos >= a.n_pos);
    bool bad_slot = false;
    if constexpr (TO != kToRows) bad_slot = slot >= a.pool.slots();
    // this lane's cos and sin: of the 8 pairs (piece 0, piece 1), or of the 4
    // adjacent pairs of each piece
    const bool rotates = lane < at.turn && !bad_pos && !is_v;
    float cs[16];
    if (rotates) {
      const float* t = a.rope + long(pos) * a.rot;
      const int o0 = half ? lane * 16 : p0 * 8, o1 = half ? lane * 16 + 8 : p1 * 8;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(t + (j < 2 ? o0 : o1) + j % 2 * 4);
        cs[4 * j] = v.x; cs[4 * j + 1] = v.y; cs[4 * j + 2] = v.z; cs[4 * j + 3] = v.w;
      }
    }
    if ((bad_pos || bad_slot) && lane == 0) atomicExch(a.status, FRT_ERANGE);

    // a head's pieces; the next one's, or the next unit's first, under way
    const bool more = TO != kToRows && n_units - unit > stride;
    auto advance = [&](int u, uint4& o0, uint4& o1) {
      o0 = n0;
      o1 = n1;
      if (u + 1 < jn) {
        src += a.hd;
        if (has0) n0 = *reinterpret_cast<const uint4*>(src + p0 * 8);
        if (has1) n1 = *reinterpret_cast<const uint4*>(src + p1 * 8);
      } else if (more) {
        look_ahead(unit + stride);
      }
    };
    // the norm and the rotation of one head, rounded to bf16
    auto norm_rotate = [&](uint4& o0, uint4& o1) {
      if (!w && a.rot == 0) return;
      uint64_t y[2][4];
      unpack8_f2(o0, y[0]);
      unpack8_f2(o1, y[1]);
      if (w) {
        // the sum of squares in fp64: a key next to a 4-bit border must not
        // depend on the order of its summands
        double s = 0.0, s1 = 0.0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const double lo = f2_lo(y[i][j]), hi = f2_hi(y[i][j]);
            s = fma(lo, lo, s);
            s1 = fma(hi, hi, s1);
          }
        s += s1;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(group, s, o, LANES);
        const float m = __fadd_rn(float(s * a.inv_hd), a.eps);
        const float r = __frcp_rn(__fsqrt_rn(m));
        uint64_t wv[2][4];
        unpack8_f2(w0, wv[0]);
        unpack8_f2(w1, wv[1]);
        const uint64_t r2 = f2_pack(r, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[0][j] = mul2(mul2(y[0][j], r2), wv[0][j]);
          y[1][j] = mul2(mul2(y[1][j], r2), wv[1][j]);
        }
      }
      if (rotates) {
        // scalar operations with their own roundings: paired products and sums
        // came out fused, and a key next to a 4-bit border must not depend on that
        if (half) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float c = cs[2 * j], s = cs[2 * j + 1];
            uint64_t &v0 = y[0][j / 2], &v1 = y[1][j / 2];
            const float e0 = j % 2 ? f2_hi(v0) : f2_lo(v0), e1 = j % 2 ? f2_hi(v1) : f2_lo(v1);
            const float r0 = __fsub_rn(__fmul_rn(e0, c), __fmul_rn(e1, s));
            const float r1 = __fadd_rn(__fmul_rn(e0, s), __fmul_rn(e1, c));
            v0 = j % 2 ? f2_pack(f2_lo(v0), r0) : f2_pack(r0, f2_hi(v0));
            v1 = j % 2 ? f2_pack(f2_lo(v1), r1) : f2_pack(r1, f2_hi(v1));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint64_t& v = y[j / 4][j % 4];
            const float e0 = f2_lo(v), e1 = f2_hi(v), c = cs[2 * j], s = cs[2 * j + 1];
            v = f2_pack(__fsub_rn(__fmul_rn(e0, c), __fmul_rn(e1, s)),
                        __fadd_rn(__fmul_rn(e0, s), __fmul_rn(e1, c)));
          }
        }
      }
      o0 = pack8_bf16_f2(y[0]);
      o1 = pack8_bf16_f2(y[1]);
    };

    if (TO == kToRows || is_q) {
      uint16_t* dst = (is_q ? a.q_out + row * a.ld_q : a.k_out + row * a.ld_k) + long(j0) * a.hd;
#pragma unroll 1
      for (int u = 0; u < jn; ++u, dst += a.hd) {
        uint4 o0, o1;
        advance(u, o0, o1);
        norm_rotate(o0, o1);
        if (has0 && !bad_pos) *reinterpret_cast<uint4*>(dst + p0 * 8) = o0;
        if (has1 && !bad_pos) *reinterpret_cast<uint4*>(dst + p1 * 8) = o1;
      }
    } else if (slot < 0 || bad_slot || bad_pos) {   // the group's
      if (more) look_ahead(unit + stride);
    } else {
    uint8_t* rec = a.pool.record(slot, j0);
    const long row_in = a.pool.row(slot);
    if constexpr (TO == kToBf16Pages) {
      rec += ((is_v ? a.pool.page_size : 0) + row_in) * a.hd * 2;
#pragma unroll 1
      for (int u = 0; u < jn; ++u, rec += a.pool.record_bytes) {
        uint4 o0, o1;
        advance(u, o0, o1);
        if (!is_v) norm_rotate(o0, o1);
        if (has0) *reinterpret_cast<uint4*>(rec + p0 * 16) = o0;
        if (has1) *reinterpret_cast<uint4*>(rec + p1 * 16) = o1;
      }
    }
    if constexpr (TO == kToFp4Pages) {
      const float rk = -__frcp_rn(static_scale);   // the negatives, for quantise8
      const uint64_t rk2 = f2_pack(rk, rk);
      rec += is_v ? a.pool.record_bytes / 2 : 0;
      const long scales = long(a.pool.page_size) * (a.hd / 2) + row_in * (a.hd / 16);
      // a block of 16 is two neighbouring pieces: who holds the other
      int lane0, lane1, slot0, slot1;
      at.find(p0 ^ 1, &lane0, &slot0);
      at.find(p1 ^ 1, &lane1, &slot1);
#pragma unroll 1
      for (int u = 0; u < jn; ++u, rec += a.pool.record_bytes) {
        uint4 o0, o1;
        advance(u, o0, o1);
        if (!is_v) norm_rotate(o0, o1);
        uint64_t y[2][4];
        unpack8_f2(o0, y[0]);  // what is cached is the bf16 key
        unpack8_f2(o1, y[1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[0][j] = mul2(y[0][j], rk2);
          y[1][j] = mul2(y[1][j], rk2);
        }
        float big0 = absmax8(y[0]), big1 = absmax8(y[1]);
        const float a0 = __shfl_sync(group, big0, lane0, LANES), a1 = __shfl_sync(group, big1, lane0, LANES);
        const float b0 = __shfl_sync(group, big0, lane1, LANES), b1 = __shfl_sync(group, big1, lane1, LANES);
        big0 = fmaxf(big0, slot0 ? a1 : a0);
        big1 = fmaxf(big1, slot1 ? b1 : b0);
        if (__any_sync(group, fmaxf(big0, big1) > 8192.0f)) {
          // far past saturation: keeps infinities out of the remainder
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint64_t& v = y[j / 4][j % 4];
            v = f2_pack(fminf(fmaxf(f2_lo(v), -8192.0f), 8192.0f), fminf(fmaxf(f2_hi(v), -8192.0f), 8192.0f));
          }
        }
        const uint8_t s0 = block_scale(big0), s1 = block_scale(big1);
        uint8_t* codes = rec + row_in * (a.hd / 2);
        if (has0) *reinterpret_cast<uint32_t*>(codes + p0 * 4) = quantise8(y[0], s0);
        if (has1) *reinterpret_cast<uint32_t*>(codes + p1 * 4) = quantise8(y[1], s1);
        if (has0 && (p0 & 1) == 0) rec[scales + p0 / 2] = s0;
        if (has1 && (p1 & 1) == 0) rec[scales + p1 / 2] = s1;
      }
    }
    }
    if (!more) break;
    unit += stride;
  }
}

template <int LANES, int U>
int launch_heads(int to, HeadArgs a, cudaStream_t s) {
  a.q_units = to == kToRows || a.q_out ? (a.hq + U - 1) / U : 0;
  const long units = long(a.rows) * (a.q_units + (a.hkv + U - 1) / U * (to == kToRows ? 1 : 2));
  FRT_REQUIRE(units <= 0x7fffff00L, FRT_ESHAPE, "rows * heads is too large");
  const long blocks = (units * LANES + 255) / 256, most = num_sms() * 2L;
  const bool resident = to != kToRows;   // blocks that go from unit to unit
  const dim3 grid{unsigned(resident && blocks > most ? most : blocks)}, block{256};
  switch (to) {
    case kToRows: return launch_pdl("frt_qk_norm_rope", head_kernel<LANES, U, kToRows>, grid, block, 0, s, a);
    case kToBf16Pages: return launch_pdl("frt_paged_kv_append", head_kernel<LANES, U, kToBf16Pages>, grid, block, 0, s, a);
    default: return launch_pdl("frt_paged_kv_append", head_kernel<LANES, U, kToFp4Pages>, grid, block, 0, s, a);
  }
}

int launch_heads(int to, const HeadArgs& a, cudaStream_t s) {
  // One head a group while the heads do not fill the GPU (latency), four
  // once they do (the table row and the index arithmetic are shared).
  const int lanes = a.hd <= 64 ? 4 : a.hd <= 128 ? 8 : 16;
  const bool few = long(a.rows) * (a.hq + 2 * a.hkv) * lanes <= num_sms() * 2048L;
  constexpr int U = 4;
  if (lanes == 4) return few ? launch_heads<4, 1>(to, a, s) : launch_heads<4, U>(to, a, s);
  if (lanes == 8) return few ? launch_heads<8, 1>(to, a, s) : launch_heads<8, U>(to, a, s);
  return few ? launch_heads<16, 1>(to, a, s) : launch_heads<16, U>(to, a, s);
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

// One thread per 16 elements of a cached head (8 in bf16 pages): a block's
// codes and scale.  16381 rows of 8 + 8 heads of 128 from 4-bit pages: 18.6 us
// for 13.3 of bytes, with 73 % of the issue slots.
__global__ void __launch_bounds__(256) read_kernel(ReadArgs a) {
  const uint32_t pieces = uint32_t(a.hd) / (a.fp4 ? 16 : 8);
  const uint32_t per_row = 2u * a.hkv * pieces;
  const uint32_t g = blockIdx.x * 256u + threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const uint32_t row = g / per_row;
  if (row >= uint32_t(a.rows)) return;
  const uint32_t c = g - row * per_row;
  const uint32_t h2 = c / pieces, p = c - h2 * pieces;  // h2: the k heads, then the v heads
  const bool is_v = h2 >= uint32_t(a.hkv);
  const int h = int(is_v ? h2 - a.hkv : h2);
  uint16_t* out = is_v ? a.v_out : a.k_out;
  if (!out) return;
  const long slot = a.slots[row];
  if (slot < 0) return;
  if (slot >= a.pool.slots()) {
    atomicExch(a.status, FRT_ERANGE);
    return;
  }
  const uint8_t* rec = a.pool.record(slot, h);
  const long at = a.pool.row(slot);
  out += row * (is_v ? a.ld_v : a.ld_k) + long(h) * a.hd;
  if (!a.fp4) {
    reinterpret_cast<uint4*>(out)[p] =
        *reinterpret_cast<const uint4*>(rec + ((is_v ? a.pool.page_size : 0) + at) * a.hd * 2 + p * 16);
    return;
  }
  rec += is_v ? a.pool.record_bytes / 2 : 0;
  const uint2 w = *reinterpret_cast<const uint2*>(rec + at * (a.hd / 2) + p * 8);
  const __nv_fp8_storage_t s8 = rec[long(a.pool.page_size) * (a.hd / 2) + at * (a.hd / 16) + p];
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)));
  const float k = *(is_v ? a.v_scale : a.k_scale);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 v(__nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t((i ? w.y : w.x) >> (8 * j)), __NV_E2M1));
      x[2 * j] = __fmul_rn(__fmul_rn(__low2float(v), s), k);
      x[2 * j + 1] = __fmul_rn(__fmul_rn(__high2float(v), s), k);
    }
    reinterpret_cast<uint4*>(out)[2 * p + i] = pack8_bf16(x);
  }
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

// hq: the descriptor's, or 0 where the call has no q heads
int check_heads(const frt_qk_rope_desc* d, int hq) {
  FRT_REQUIRE(d->rows >= 0 && hq >= 0 && d->hkv >= 0 && hq <= 65536 && d->hkv <= 65536,
              FRT_ESHAPE, "bad rows / heads: %d, %d, %d", d->rows, hq, d->hkv);
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
  frt::TableArgs a{};
  a.M = M; a.rot = rot; a.scaling = scaling; a.P = P; a.factor = factor; a.orig_len = orig_len;
  a.low = low_turns; a.high = high_turns; a.amplitude = amplitude; a.out = rope_out;
  long double base = log2l((long double)theta);
  if (scaling == FRT_ROPE_SCALE_BASE) base += log2l((long double)factor) * rot / (rot - 2);
  a.log2_base = double(base);
  a.log2_base_lo = double(base - a.log2_base);
  // runs as long as the GPU stays full, 32 at most
  const long per_thread = long(M) * (rot / 2) / (frt::num_sms() * 1024L);
  a.steps = per_thread < 1 ? 1 : per_thread > 32 ? 32 : int(per_thread);
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
  FRT_REQUIRE(d, FRT_EINVAL, "descriptor is NULL");
  if (int rc = frt::check_heads(d, d->hq)) return rc;
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
  return frt::launch_heads(frt::kToRows, a, static_cast<cudaStream_t>(stream));
}

extern "C" int frt_paged_kv_append(const frt_qk_rope_desc* d, void* stream) {
  frt::clear_error();
  FRT_REQUIRE(d, FRT_EINVAL, "descriptor is NULL");
  if (int rc = frt::check_heads(d, d->hq)) return rc;
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
  return frt::launch_heads(d->format == FRT_PAGE_BF16 ? frt::kToBf16Pages : frt::kToFp4Pages, a,
                           static_cast<cudaStream_t>(stream));
}

extern "C" int frt_paged_kv_read(const frt_qk_rope_desc* d, void* stream) {
  frt::clear_error();
  FRT_REQUIRE(d, FRT_EINVAL, "descriptor is NULL");
  if (int rc = frt::check_heads(d, 0)) return rc;
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
  const long threads = 2L * d->rows * d->hkv * (d->hd / (a.fp4 ? 16 : 8));
  FRT_REQUIRE(threads <= 0xffffff00L, FRT_ESHAPE, "rows * heads is too large");
  const long blocks = (threads + 255) / 256;
  return frt::launch_pdl("frt_paged_kv_read", frt::read_kernel, dim3(unsigned(blocks)), dim3(256),
                         0, static_cast<cudaStream_t>(stream), a);
}
