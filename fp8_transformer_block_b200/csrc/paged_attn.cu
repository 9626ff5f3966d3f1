// paged_attn.cu -- attention over a paged cache held in 4 bits.
//
// Per (sequence, kv head) the query rows of all its q heads share the keys:
// row r of the unit is token r / G, head r % G of the group (G = hq / hkv).
// A tile of R rows runs over the sequence's keys in chunks, with one pass of
// the running maximum and sum of the softmax.
//
// The codes times their block scales are exact in fp16 (2 + 4 significant
// bits, 2^-10 .. 2688), so the cache is widened in registers to fp16 and the
// products run on the tensor cores with fp32 sums; the static scales are
// applied to the fp32 results.
#include <cmath>
#include <mutex>
#include <set>
#include <utility>

#include "frt_attn.cuh"

namespace frt {

// Before any thread's first launch of the kernel on the device.
int allow_smem(const void* kern, int bytes) {
  static std::mutex mu;
  static std::set<std::pair<int, const void*>> done;
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(mu);
  if (done.count({dev, kern})) return FRT_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();
    return fail(FRT_ECUDA, "frt_paged_attention_fp4: %d bytes of shared memory refused", bytes);
  }
  done.insert({dev, kern});
  return FRT_OK;
}

namespace {

// A position in the list of all (sequence, row tile, kv head, chunk).
template <int R, int CK>
struct Walker {
  Seq q;
  int s, unit, chunk;   // unit = tile * hkv + head

  __device__ void begin(const Seq& seq, int index, long offset) {
    s = index;
    q = seq;
    unit = int(offset / q.chunks);
    chunk = int(offset - long(unit) * q.chunks);
  }
  // Past the unit's last chunk: to the next unit that has any.
  __device__ void next_unit(const AttnArgs& a) {
    chunk = 0;
    if (++unit < a.hkv * q.tiles) return;
    unit = 0;
    do {
      if (++s >= a.n_seqs) return;
      q = load_seq<R, CK>(a, s, false);
    } while (q.tiles == 0);
  }
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int BYTES>
__device__ __forceinline__ void lds(const uint8_t* p, uint32_t (&w)[BYTES / 4]) {
  if constexpr (BYTES == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (BYTES == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  }
}

// ------------------------------------------------------------ few rows ----
//
// Bound by the cache's bytes (hd * 9/8 per key and kv head), if the widening
// keeps up: S^T = K Q^T and O^T = V^T P^T on m16n8k16, the keys (and then
// the head's elements) on the 16 side, so that 8 query rows cost no padding.
// Any order of the summed index is as good as another as long as both
// operands agree, so each lane takes whole runs of a key's codes: lane
// (g = lane / 4, t = lane % 4) widens the quarter t of key g's elements for
// S, and the eighth g of the elements of keys 2t.. for O.
//
// One warp feeds a ring of chunks (bulk copies of page records, or of the
// four parts of a record where the page is longer than the chunk); each of
// the W other warps takes 16 keys of every chunk with a softmax state of its
// own, joined when the unit ends.  The chunks of all units lie on one line
// that is cut into equal runs, one a CTA: a ragged batch loads every SM
// alike.  A unit cut by a run's end leaves partial states in the workspace,
// and the last of its CTAs to finish joins them in order.
//
// 61 sequences of one token and 700 to 16384 keys, 32 q heads on 8 of 128, run
// in 133 to 138 us (93 for the bytes).  No unit is full: on 24 sequences of 8500 keys
// 56 % of the issue slots and 3.6 TB/s.  The 12 computing warps of an SM have
// a chain each from the widening (most of the 331 warp instructions for 16
// keys of a kv head) over the products and the softmax to the next widening,
// and wait for fixed latencies first.  Two groups of 16 keys a warp at once
// hide part of it (one: 154 us), three CTAs an SM (four, with fewer registers:
// 180).

template <int HD, int NT>
struct FewCfg {
  static constexpr int W = 4;                    // computing warps
  static constexpr int R = 8 * NT;               // query rows
  static constexpr int GR = NT == 1 ? 2 : 1;     // groups of 16 keys a warp takes at once
  static constexpr int CK = 16 * GR * W;         // keys of a chunk
  static constexpr int kStage = CK * HD * 9 / 8; // bytes of a chunk
  static constexpr bool kQRegs = HD * NT < 128;
  static constexpr int kJoin = W * R * HD * 4;   // the warps' sums when a unit ends
  static constexpr int kQBytes = kQRegs ? 0 : HD / 16 * NT * 32 * 8;
  static constexpr int kStages = (HD == 256 ? 4 : 6) / GR;
  static constexpr int kThreads = 32 * (W + 1);
  static constexpr int kCtas = HD / 16 * NT <= 8 ? 3 : HD / 16 * NT <= 16 ? 2 : 1;  // per SM
  static constexpr int kTile = R * (HD + 2);     // floats of one partial state
  static constexpr int kSmem = kStages * kStage + kJoin + kQBytes + 2 * W * R * 4 + 1024;
};

template <int HD, int NT>
__global__ void __launch_bounds__(FewCfg<HD, NT>::kThreads, FewCfg<HD, NT>::kCtas)
attn_few_kernel(AttnArgs a) {
  using C = FewCfg<HD, NT>;
  constexpr int W = C::W, R = C::R, CK = C::CK, GR = C::GR;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;
  float* join = reinterpret_cast<float*>(ring + C::kStages * C::kStage);
  uint2* q_smem = reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(join) + C::kJoin);
  float* join_m = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(q_smem) + C::kQBytes);
  float* join_l = join_m + W * R;
  uint64_t* full = reinterpret_cast<uint64_t*>(join_l + W * R);
  uint64_t* empty = full + C::kStages;
  uint32_t* valid = reinterpret_cast<uint32_t*>(empty + C::kStages);
  long* scan = reinterpret_cast<long*>(valid + 8);    // [kThreads / 32] and the start
  volatile int* abort_flag = reinterpret_cast<volatile int*>(scan + 8);
  int* last = reinterpret_cast<int*>(scan + 8) + 1;
  int* units = reinterpret_cast<int*>(scan + 9);
  Seq* start = reinterpret_cast<Seq*>(scan + 10);

  const int tid = int(threadIdx.x), warp = tid / 32, lane = tid % 32;
  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], W);
    }
    *abort_flag = 0;
    *units = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();

  // --- this CTA's run of the line of all chunks ---
  long total = 0, upto = 0;
  Seq mine;
  mine.tiles = mine.chunks = 0;
  for (int base = 0; base < a.n_seqs; base += C::kThreads) {
    const int s = base + tid;
    long n = 0;
    if (s < a.n_seqs) {
      mine = load_seq<R, CK>(a, s, blockIdx.x == 0);
      n = mine.work(a.hkv);
      if (mine.tiles) atomicAdd(units, mine.tiles * a.hkv);
    }
    long inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    long before = 0, all = 0;
    for (int i = 0; i < C::kThreads / 32; ++i) {
      if (i < warp) before += scan[i];
      all += scan[i];
    }
    upto = total + before + inc;
    total += all;
    __syncthreads();
  }
  // A chunk takes a CTA about a microsecond, and joining a unit's shares an
  // eighth of one a share and eight rows: of a unit's n chunks, sqrt(n NT / 8)
  // to a CTA keep the sum of both low (one sequence of 40000 keys: 48 us with
  // a CTA for every chunk, 24 us with this)
  const float mean = float(total) / float(max(*units, 1));
  const long least = max(1L, long(sqrtf(mean * NT / 8) + 0.5f));
  const long most = (total + least - 1) / least;
  const long ctas = most < long(gridDim.x) ? most : long(gridDim.x);
  const long c = blockIdx.x;
  if (c >= ctas) return;
  const long begin = c * total / ctas, end = (c + 1) * total / ctas;
  if (a.n_seqs > C::kThreads) {  // find the start again, block by block
    long run = 0;
    for (int base = 0; base < a.n_seqs; base += C::kThreads) {
      const int s = base + tid;
      long n = 0;
      Seq q;
      if (s < a.n_seqs) {
        q = load_seq<R, CK>(a, s, false);
        n = q.work(a.hkv);
      }
      long inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) scan[warp] = inc;
      __syncthreads();
      long before = 0, all = 0;
      for (int i = 0; i < C::kThreads / 32; ++i) {
        if (i < warp) before += scan[i];
        all += scan[i];
      }
      __syncthreads();
      const long hi = run + before + inc;
      if (n > 0 && begin >= hi - n && begin < hi) {
        scan[6] = s;
        scan[7] = begin - (hi - n);
        *start = q;
      }
      run += all;
    }
  } else if (tid < a.n_seqs) {
    const long n = mine.work(a.hkv);
    if (n > 0 && begin >= upto - n && begin < upto) {
      scan[6] = tid;
      scan[7] = begin - (upto - n);
      *start = mine;
    }
  }
  __syncthreads();
  Walker<R, CK> w;
  w.begin(*start, int(scan[6]), scan[7]);

  const int ps = a.pool.page_size;
  const int sub = ps < CK ? ps : CK;  // keys of one record's piece in a chunk

  if (warp == W) {
    // ------------------------------------------------------------ the feed --
    int stage = 0;
    uint32_t phase = 0;
    const int n_sub = CK / sub;
    const bool parts = ps > CK;
    long issued = 0;
    // lane i looks up piece i of the chunk the walker stands at: one chunk
    // ahead, so that the table's latency is not in the way of the copies
    auto look_up = [&]() {
      const int key0 = (w.q.chunk0 + w.chunk) * CK;
      const int key = parts ? key0 : key0 + lane * sub;
      if (lane >= (parts ? 4 : n_sub) || key >= w.q.L) return -1;
      return __ldg(a.page_table + long(w.s) * a.max_pages + (key >> a.pool.shift));
    };
    int page_next = look_up();
    for (long x = begin; x < end; ++x) {
      int page = page_next;
      const int head = w.unit % a.hkv;
      const int at = (w.q.chunk0 + w.chunk) * CK & (ps - 1);
      const bool in_range = lane < (parts ? 4 : n_sub) &&
                            (w.q.chunk0 + w.chunk) * CK + (parts ? 0 : lane * sub) < w.q.L;
      if (x + 1 < end) {
        if (++w.chunk == w.q.chunks) w.next_unit(a);
        page_next = look_up();
      }
      if (in_range && (page < 0 || page >= a.pool.n_pages)) {
        atomicExch(a.status, FRT_ERANGE);
        page = -1;
      }
      const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
      bool ok = true;
      if (lane == 0) {
        ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, kAttnWaitNs, abort_flag);
        if (!ok) {
          atomicExch(a.status, FRT_ETIMEOUT);
          *abort_flag = 1;
        } else {
          valid[stage] = have;
          const uint32_t bytes = parts ? (have ? C::kStage : 0u)
                                       : __popc(have) * (sub * HD * 9 / 8);
          mbar_arrive_expect_tx(&full[stage], bytes);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      __syncwarp();
      if (page >= 0) {
        const uint8_t* rec = a.pool.base + (long(page) * a.pool.hkv + head) * a.pool.record_bytes;
        uint8_t* dst = ring + stage * C::kStage;
        if (!parts) {
          bulk_load(dst + lane * (sub * HD * 9 / 8), rec, sub * HD * 9 / 8, &full[stage]);
        } else {  // lane 0 .. 3: key codes, key scales, value codes, value scales
          rec += (lane & 2 ? a.pool.record_bytes / 2 : 0) +
                 (lane & 1 ? ps * (HD / 2) + at * (HD / 16) : at * (HD / 2));
          dst += (lane & 2 ? C::kStage / 2 : 0) + (lane & 1 ? CK * (HD / 2) : 0);
          bulk_load(dst, rec, lane & 1 ? CK * (HD / 16) : CK * (HD / 2), &full[stage]);
        }
      }
      ++issued;
      if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
    }
    // after a wait that ran out: no exit with copies in flight
    if (*abort_flag && lane == 0) {
      for (long i = issued - C::kStages < 0 ? 0 : issued - C::kStages; i < issued; ++i)
        mbar_wait_bounded(&full[i % C::kStages], uint32_t(i / C::kStages) & 1u, kAttnWaitNs, nullptr);
    }
    return;
  }

  // ------------------------------------------------------- the arithmetic --
  const int g = lane / 4, t = lane % 4;
  // keys of this lane in a group of 16 (the second eight: + 8): its row of
  // S^T, and the two rows of the summed index of O^T.  The order is the one
  // that spreads both reads over the banks.
  const int key_s = (g & ~1) + ((g ^ (g >> 1)) & 1);
  const int key_o[2] = {2 * t + (t & 1), 2 * t + ((t & 1) ^ 1)};
  // the sign of the scale goes into Q, so that the largest score is that of
  // the largest product
  const float scale = *a.k_scale * a.sm_scale * kLog2e;
  const float vscale = *a.v_scale;
  // where in a stage this lane's bytes of the warp's first group lie, and
  // the way to the next group (in the next record's piece, if that is 16 keys)
  int piece[C::GR];
#pragma unroll
  for (int u = 0; u < C::GR; ++u) piece[u] = ps < CK ? (warp * C::GR + u) * 16 / sub : 0;
  const int in_piece = warp * C::GR * 16 - piece[0] * sub;
  const int at_rec = piece[0] * (sub * HD * 9 / 8);
  const int at_k = at_rec + (in_piece + key_s) * (HD / 2) + t * (HD / 8);
  const int at_ks = at_rec + sub * (HD / 2) + (in_piece + key_s) * (HD / 16) + t * (HD / 64);
  int at_v[2], at_vs[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    at_v[k] = at_rec + sub * (HD / 2 + HD / 16) + (in_piece + key_o[k]) * (HD / 2) + g * (HD / 16);
    at_vs[k] = at_rec + sub * (HD + HD / 16) + (in_piece + key_o[k]) * (HD / 16) + g * HD / 128;
  }
  const int code_step = sub == 16 ? 16 * HD * 9 / 8 : 16 * (HD / 2);
  const int scale_step = sub == 16 ? 16 * HD * 9 / 8 : 16 * (HD / 16);
  int stage = 0;
  uint32_t phase = 0;

  for (long x = begin; x < end;) {
    const long seg0 = x;
    const int n_here = int(min(long(w.q.chunks - w.chunk), end - x));
    const bool from_start = w.chunk == 0, to_end = w.chunk + n_here == w.q.chunks;
    const int head = w.unit % a.hkv, tile = w.unit / a.hkv;
    const int rows_here = w.q.Lq * a.group;

    // Q fragments: row g (+ 8 per nt), elements t * HD/4 .., scaled by a
    // power of two that brings the row's largest below 2
    uint32_t qf[C::kQRegs ? NT : 1][C::kQRegs ? HD / 8 : 1];
    float cq[NT][2], m[NT][2], l[NT][2];
    int lim_hi[NT][2], lim_lo[NT][2];
    int tile_hi = 0, tile_lo = 0x7fffffff, all_hi = 0x7fffffff, all_lo = 0;
    if constexpr (!C::kQRegs) named_bar_sync(1, W * 32);  // the last unit's reads of q_smem
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (!C::kQRegs && nt % W != warp % W && NT >= W) continue;
      const int r = tile * R + nt * 8 + g;
      uint32_t raw[HD / 8];
      float big = 0.0f;
      if (r < rows_here) {
        const int token = r / a.group;
        const uint16_t* src = a.q + long(w.q.r0 + token) * a.ld_q +
                              long(head * a.group + r - token * a.group) * HD + t * (HD / 4);
#pragma unroll
        for (int i = 0; i < HD / 32; ++i) {
          const uint4 v = reinterpret_cast<const uint4*>(src)[i];
          raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) raw[i] = 0;
      }
#pragma unroll
      for (int i = 0; i < HD / 8; ++i)
        big = fmaxf(big, fmaxf(fabsf(__uint_as_float(raw[i] << 16)),
                               fabsf(__uint_as_float(raw[i] & 0xFFFF0000u))));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      const int e = q_exponent(big);
      const float down = copysignf(__uint_as_float(uint32_t(254 - e) << 23), scale);
      const float up = __uint_as_float(uint32_t(e) << 23);
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        raw[i] = pack_f16x2(__uint_as_float(raw[i] << 16) * down,
                            __uint_as_float(raw[i] & 0xFFFF0000u) * down);
        if constexpr (C::kQRegs) qf[nt][i] = raw[i];
      }
      if constexpr (!C::kQRegs) {
#pragma unroll
        for (int j = 0; j < HD / 16; ++j)
          q_smem[(nt * (HD / 16) + j) * 32 + lane] = make_uint2(raw[2 * j], raw[2 * j + 1]);
        if (t == 0) join_m[nt * 8 + g] = up;
      } else {
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2)
          cq[nt][e2] = score_factor(scale, __shfl_sync(0xffffffffu, up, (2 * t + e2) * 4));
      }
    }
    if constexpr (!C::kQRegs) {
      named_bar_sync(1, W * 32);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) cq[nt][e2] = score_factor(scale, join_m[nt * 8 + 2 * t + e2]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        const int r = tile * R + nt * 8 + 2 * t + e2;
        int hi = 0, lo = 0;
        if (r < rows_here) {
          const int place = w.q.L - w.q.Lq + r / a.group;
          hi = a.causal ? min(w.q.L, place + 1) : w.q.L;
          lo = a.window > 0 ? max(0, place - a.window + 1) : 0;
          tile_hi = max(tile_hi, hi);
          tile_lo = min(tile_lo, lo);
          all_hi = min(all_hi, hi);
          all_lo = max(all_lo, lo);
        }
        lim_hi[nt][e2] = hi;
        lim_lo[nt][e2] = lo;
        m[nt][e2] = kNoKey;
        l[nt][e2] = 0.0f;
      }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {  // over t: the tile's limits
      tile_hi = max(tile_hi, __shfl_xor_sync(0xffffffffu, tile_hi, o));
      tile_lo = min(tile_lo, __shfl_xor_sync(0xffffffffu, tile_lo, o));
      all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
      all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
    }
    bool far = false;   // of any of the warp's rows
    float true_cq[C::kQRegs ? NT : 1][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        if constexpr (C::kQRegs) true_cq[nt][e2] = cq[nt][e2];
        if (is_far<HD>(cq[nt][e2])) {
          far = true;
          cq[nt][e2] = 1.0f;
        }
      }
    far = __any_sync(0xffffffffu, far);
    float o_acc[NT][HD / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o_acc[nt][i][j] = 0.0f;

    for (int n = 0; n < n_here; ++n, ++x) {
      const int key0 = (w.q.chunk0 + w.chunk + n) * CK + warp * 16 * GR;
      // every lane waits: each reads what the copies wrote
      const bool got = mbar_wait_bounded(&full[stage], phase, kAttnWaitNs, abort_flag);
      if (!got && lane == 0) {
        atomicExch(a.status, FRT_ETIMEOUT);
        *abort_flag = 1;
      }
      if (__all_sync(0xffffffffu, got) && key0 < tile_hi && key0 + 16 * GR > tile_lo) {
        const uint8_t* st = ring + stage * C::kStage;
        const uint32_t have = valid[stage];
        bool hidden[GR], masked = far || key0 + 16 * GR > all_hi || key0 < all_lo;
#pragma unroll
        for (int u = 0; u < GR; ++u) {  // in a bad page
          hidden[u] = !(have >> piece[u] & 1);
          masked |= hidden[u];
        }

        // S^T, 16 GR keys x 8 NT rows
        float s[GR][NT][4];
#pragma unroll
        for (int u = 0; u < GR; ++u) {
          uint32_t kw[2][HD / 32];
          uint32_t kscl[2][(HD + 127) / 128];  // pairs of block scales, fp16
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            lds<HD / 8>(st + at_k + u * code_step + f * (8 * HD / 2), kw[f]);
            const uint8_t* sp = st + at_ks + u * scale_step + f * (8 * HD / 16);
            if constexpr (HD == 64) {
              kscl[f][0] = e4m3x2_to_f16(*sp);
            } else if constexpr (HD == 128) {
              kscl[f][0] = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(sp));
            } else {
              const uint32_t v = *reinterpret_cast<const uint32_t*>(sp);
              kscl[f][0] = e4m3x2_to_f16(v & 0xFFFFu);
              kscl[f][1] = e4m3x2_to_f16(v >> 16);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][nt][i] = 0.0f;
#pragma unroll
          for (int i = 0; i < HD / 32; ++i) {  // 8 codes of each key: half a block
            uint32_t h[2][4];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              e2m1x8_to_f16(kw[f][i], h[f]);
              const uint32_t sc = __byte_perm(kscl[f][i / 4], 0, i / 2 % 2 ? 0x3232 : 0x1010);
#pragma unroll
              for (int k = 0; k < 4; ++k) h[f][k] = hmul2(h[f][k], sc);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                uint32_t b0, b1;
                if constexpr (C::kQRegs) {
                  b0 = qf[nt][4 * i + 2 * k];
                  b1 = qf[nt][4 * i + 2 * k + 1];
                } else {
                  const uint2 b = q_smem[(nt * (HD / 16) + 2 * i + k) * 32 + lane];
                  b0 = b.x; b1 = b.y;
                }
                mma_f16(s[u][nt], h[0][2 * k], h[1][2 * k], h[0][2 * k + 1], h[1][2 * k + 1], b0, b1);
              }
          }
        }

        // softmax: base-2 scores against a running maximum (kLift below the
        // largest score when it is set) that is raised only when a score
        // passes it by more than kGrow, so most groups pass without the
        // reduction
        if (masked) {
          if (far) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e2 = 0; e2 < 2; ++e2) {
                const float v = C::kQRegs ? true_cq[C::kQRegs ? nt : 0][e2]
                                          : score_factor(scale, join_m[nt * 8 + 2 * t + e2]);
                const float f = is_far<HD>(v) ? v : 1.0f;
#pragma unroll
                for (int u = 0; u < GR; ++u) {
                  s[u][nt][e2] = __fmul_rn(s[u][nt][e2], f);
                  s[u][nt][e2 + 2] = __fmul_rn(s[u][nt][e2 + 2], f);
                }
              }
          }
#pragma unroll
          for (int u = 0; u < GR; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = key0 + 16 * u + key_s + 8 * (i >> 1);
                if (hidden[u] || key >= lim_hi[nt][i & 1] || key < lim_lo[nt][i & 1])
                  s[u][nt][i] = -INFINITY;
              }
        }
        float top[NT][2];
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            float v = fmaxf(s[0][nt][e2], s[0][nt][e2 + 2]);
#pragma unroll
            for (int u = 1; u < GR; ++u) v = fmaxf(v, fmaxf(s[u][nt][e2], s[u][nt][e2 + 2]));
            top[nt][e2] = v * cq[nt][e2];
            grow |= top[nt][e2] > m[nt][e2] + kGrow;
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              float v = top[nt][e2];
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
              v = fmaxf(v - kLift, m[nt][e2]);
              const float f = ex2(m[nt][e2] - v);
              m[nt][e2] = v;
              l[nt][e2] *= f;
#pragma unroll
              for (int i = 0; i < HD / 16; ++i) {
                o_acc[nt][i][e2] *= f;
                o_acc[nt][i][e2 + 2] *= f;
              }
            }
        }
        uint32_t p[GR][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int u = 0; u < GR; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              s[u][nt][i] = ex2(fmaf(s[u][nt][i], cq[nt][i & 1], -m[nt][i & 1]));
              l[nt][i & 1] += s[u][nt][i];
            }
            p[u][nt][0] = movmatrix_trans(pack_f16x2(s[u][nt][0], s[u][nt][1]));
            p[u][nt][1] = movmatrix_trans(pack_f16x2(s[u][nt][2], s[u][nt][3]));
          }
        }

        // O^T += V^T P^T
#pragma unroll
        for (int u = 0; u < GR; ++u) {
          uint32_t vw[2][2][HD / 64];       // [eight][key][words]
          uint32_t vscl[2][HD == 256 ? 2 : 1];  // (key 0, key 1) scales, fp16
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            uint32_t sb[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              lds<HD / 16>(st + at_v[k] + u * code_step + f * (8 * HD / 2), vw[f][k]);
              const uint8_t* sp = st + at_vs[k] + u * scale_step + f * (8 * HD / 16);
              if constexpr (HD == 256) sb[k] = *reinterpret_cast<const uint16_t*>(sp);
              else sb[k] = *sp;
            }
            if (masked) {  // behind the sequence's end the page may hold anything
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (hidden[u] || key0 + 16 * u + key_o[k] + 8 * f >= w.q.L) sb[k] = 0;
            }
            vscl[f][0] = e4m3x2_to_f16(__byte_perm(sb[0], sb[1], 0x0040));
            if constexpr (HD == 256) vscl[f][1] = e4m3x2_to_f16(__byte_perm(sb[0], sb[1], 0x0051));
          }
#pragma unroll
          for (int i = 0; i < HD / 64; ++i) {  // 8 elements of every key
            uint32_t even[2][4], odd[2][4];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const uint32_t w0 = vw[f][0][i], w1 = vw[f][1][i];
              constexpr uint32_t kLow = 0x0F0F0F0Fu;
              e2m1x8_to_f16((w0 & kLow) | ((w1 << 4) & ~kLow), even[f]);
              e2m1x8_to_f16(((w0 >> 4) & kLow) | (w1 & ~kLow), odd[f]);
              const uint32_t sc = vscl[f][HD == 256 ? i / 2 : 0];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                even[f][k] = hmul2(even[f][k], sc);
                odd[f][k] = hmul2(odd[f][k], sc);
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(o_acc[nt][4 * i + k], even[0][k], odd[0][k], even[1][k], odd[1][k],
                        p[u][nt][0], p[u][nt][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
    }

    // --- the unit (or this CTA's share of it) ends: join the warps ---
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][e2] += __shfl_xor_sync(0xffffffffu, l[nt][e2], o);
    named_bar_sync(1, W * 32);  // join_m / join (and its use before) are free
    if (g == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          join_m[warp * R + nt * 8 + 2 * t + e2] = m[nt][e2];
          join_l[warp * R + nt * 8 + 2 * t + e2] = l[nt][e2];
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2)
          *reinterpret_cast<float2*>(join + (warp * R + nt * 8 + 2 * t + e2) * HD + g * (HD / 8) + 2 * i) =
              make_float2(o_acc[nt][i][e2], o_acc[nt][i][e2 + 2]);
    named_bar_sync(1, W * 32);

    const bool whole = from_start && to_end;
    float* part = a.partials + (2 * c + (from_start ? 1 : 0)) * C::kTile;
    // parts of a cut unit: CTAs first .. final
    const long unit0 = seg0 - w.chunk;
    const long first = ((unit0 + 1) * ctas - 1) / total;
    const long final = ((unit0 + w.q.chunks) * ctas - 1) / total;
    for (int i = tid; i < R * (HD / 4); i += W * 32) {
      const int r = i / (HD / 4), d = i % (HD / 4) * 4;
      float mm = kNoKey, ll = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) mm = fmaxf(mm, join_m[k * R + r]);
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const float f = ex2(join_m[k * R + r] - mm);
        const float4 v = *reinterpret_cast<const float4*>(join + (k * R + r) * HD + d);
        ll += join_l[k * R + r] * f;
        acc.x += v.x * f; acc.y += v.y * f; acc.z += v.z * f; acc.w += v.w * f;
      }
      if (!whole) {
        *reinterpret_cast<float4*>(part + r * HD + d) = acc;
        if (d == 0) {
          part[R * HD + r] = mm;
          part[R * HD + R + r] = ll;
        }
        continue;
      }
      const int row = tile * R + r;
      if (row >= rows_here) continue;
      const int token = row / a.group, h = head * a.group + row - token * a.group;
      const float inv = ll > 0.0f ? vscale / ll : ll * vscale;  // no keys: 0; NaN stays
      *reinterpret_cast<uint2*>(a.out + long(w.q.r0 + token) * a.ld_out + long(h) * HD + d) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (d == 0 && a.lse)
        a.lse[long(w.q.r0 + token) * a.hq + h] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    }
    if (!whole) {
      __threadfence();
      named_bar_sync(1, W * 32);
      if (tid == 0) {
        const int before = atomicAdd(&a.counters[first], 1);
        *last = before == int(final - first);
        if (*last) a.counters[first] = 0;
      }
      named_bar_sync(1, W * 32);
      if (*last) {
        __threadfence();
        // the shares' maxima first, a lane each; then their weights (as many
        // at a time as the idle join buffer holds), then the sums with every
        // share's loads under way
        constexpr int kCap = W * HD / 2;
        const int shares = int(final - first) + 1;
        auto share = [&](int k) { return a.partials + (2 * (first + k) + (k == 0)) * C::kTile; };
        // one pass for up to 32 shares; code that runs once is fetched cold,
        // so what follows is kept in loops
#pragma unroll 1
        for (int r = warp; r < R; r += W) {
          float mm = kNoKey, ll = 0.0f;
#pragma unroll 1
          for (int k = lane; k < shares; k += 32) {
            const float* pt = share(k) + R * HD + r;
            const float mk = __ldcg(pt), lk = __ldcg(pt + R);
            const float top = fmaxf(mm, mk);
            ll = ll * ex2(mm - top) + lk * ex2(mk - top);
            mm = top;
          }
          const float top = warp_max(mm);
          ll = warp_sum(ll * ex2(mm - top));
          if (lane == 0) {
            join_m[r] = top;
            join_l[r] = ll;
          }
        }
        constexpr int kItems = R * (HD / 4) / (W * 32);
        float4 acc[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k0 = 0; k0 < shares; k0 += kCap) {
          const int kn = min(kCap, shares - k0);
          named_bar_sync(1, W * 32);   // join_m; the block before
          for (int i = tid; i < R * kn; i += W * 32) {
            const int r = i % R, k = i / R;
            join[r * kCap + k] = ex2(__ldcg(share(k0 + k) + R * HD + r) - join_m[r]);
          }
          named_bar_sync(1, W * 32);
#pragma unroll 4
          for (int k = 0; k < kn; ++k) {
            const float* pt = share(k0 + k);
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
              const int item = i * W * 32 + tid, r = item / (HD / 4);
              const float f = join[r * kCap + k];
              const float4 v = __ldcg(reinterpret_cast<const float4*>(pt + r * HD + item % (HD / 4) * 4));
              acc[i].x += v.x * f; acc[i].y += v.y * f; acc[i].z += v.z * f; acc[i].w += v.w * f;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const int item = i * W * 32 + tid, r = item / (HD / 4), d = item % (HD / 4) * 4;
          const int row = tile * R + r;
          if (row >= rows_here) continue;
          const int token = row / a.group, h = head * a.group + row - token * a.group;
          const float ll = join_l[r];
          const float inv = ll > 0.0f ? vscale / ll : ll * vscale;
          *reinterpret_cast<uint2*>(a.out + long(w.q.r0 + token) * a.ld_out + long(h) * HD + d) =
              make_uint2(pack_bf16x2(acc[i].x * inv, acc[i].y * inv),
                         pack_bf16x2(acc[i].z * inv, acc[i].w * inv));
          if (d == 0 && a.lse)
            a.lse[long(w.q.r0 + token) * a.hq + h] =
                ll == 0.0f ? -INFINITY : (join_m[r] + log2f(ll)) * kLn2;
        }
      }
    }
    w.chunk += n_here;
    if (w.chunk == w.q.chunks && x < end) w.next_unit(a);
  }
}

// ---------------------------------------------------------------- launch --

// Counters of the cut units, at the head of the workspace: no kernel leaves
// anything else there.
constexpr size_t kCounterBytes = 4096;

template <int HD, int NT>
struct Few {
  using C = FewCfg<HD, NT>;
  static int grid() { return num_sms() * C::kCtas; }
  static size_t workspace() { return kCounterBytes + size_t(grid()) * 2 * C::kTile * 4; }
  static int launch(AttnArgs a, void* ws, long most_chunks, cudaStream_t s) {
    FRT_REQUIRE(size_t(grid()) * 4 <= kCounterBytes, FRT_ECUDA, "more SMs than counters");
    auto kern = attn_few_kernel<HD, NT>;
    if (int rc = allow_smem(reinterpret_cast<const void*>(kern), C::kSmem)) return rc;
    a.counters = static_cast<int*>(ws);
    a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kCounterBytes);
    const int n = most_chunks < grid() ? int(most_chunks) : grid();
    return launch_pdl("frt_paged_attention_fp4", kern, dim3(n), dim3(C::kThreads), C::kSmem, s, a);
  }
};

// f(Few<HD, NT>) for the head size and the rows of one kv head.
template <typename F>
auto with_variant(int hd, long rows_per_head, F f) {
  if (hd == 64)
    return rows_per_head <= 8 ? f(Few<64, 1>{}) : rows_per_head <= 16 ? f(Few<64, 2>{}) : f(Few<64, 4>{});
  if (hd == 128)
    return rows_per_head <= 8 ? f(Few<128, 1>{}) : rows_per_head <= 16 ? f(Few<128, 2>{}) : f(Few<128, 4>{});
  return rows_per_head <= 8 ? f(Few<256, 1>{}) : f(Few<256, 2>{});
}

// Which kernel takes the rows of one kv head.  Above 32 rows always the
// tensor-memory one.  For 9 to 32 rows the register kernel streams the cache
// faster, but where the units are few and the keys short, the other's splits
// are done sooner.  Lengths are known on the device only, so the rule goes by
// what the table could hold: 256 keys at most to a split.  Measured with 2 kv
// heads, register kernel / tensor-memory kernel, us:
//                                    hd 64        hd 128       hd 256
//   3 sequences of    16 rows     14.7 / 13.9  18.2 / 16.4  26.4 / 20.2
//   900 to 2000 keys  32 rows     23.6 / 15.0  27.6 / 17.8  27.2 / 22.0
//   12 sequences of   16 rows     16.9 / 18.4  20.0 / 20.8  30.4 / 23.2
//   500 to 1500 keys  32 rows     24.3 / 19.8  28.9 / 22.2  31.8 / 24.9
//   32 sequences of   16 rows     25.3 / 98.4  36.0 / 113   75.5 / 110
//   700 to 8000 keys  32 rows     40.9 / 99.8  66.6 / 120   127 / 108
// With tables just wide enough the rule takes the second kernel for the first
// two and the first for the third (not the faster one at 12 x 16 rows of 64
// and 128, nor at 32 x 32 rows of 256).  A wide table over short sequences
// takes the first.
bool many_rows(long rows_per_head, long units, long keys) {
  if (rows_per_head > 32) return true;
  if (rows_per_head <= 8 || units > num_sms()) return false;
  const long splits = num_sms() / units < 16 ? num_sms() / units : 16;
  return keys <= splits * 256;
}

bool head_counts_ok(int n_seqs, int max_q, int hq, int hkv, int hd) {
  return n_seqs >= 0 && max_q >= 0 && hkv >= 1 && hkv <= 65536 && hq >= hkv && hq <= 65536 &&
         hq % hkv == 0 && (hd == 64 || hd == 128 || hd == 256) &&
         long(max_q) * (hq / hkv) <= 0x40000000L;
}

}  // namespace
}  // namespace frt

extern "C" size_t frt_paged_attention_workspace_size(int n_seqs, int max_q, int hq, int hkv, int hd) {
  if (!frt::head_counts_ok(n_seqs, max_q, hq, hkv, hd)) return 0;
  const long rows = long(max_q) * (hq / hkv);
  const size_t many = rows > 8 ? frt::attn_many_workspace(hd, n_seqs, max_q, hq, hkv) : 0;
  if (rows > 32) return many;
  const size_t few = frt::with_variant(hd, rows, [](auto v) { return v.workspace(); });
  return few > many ? few : many;
}

extern "C" int frt_paged_attention_fp4(const frt_paged_attn_desc* d, void* stream) {
  using frt::aligned;
  frt::clear_error();
  FRT_REQUIRE(d, FRT_EINVAL, "descriptor is NULL");
  FRT_REQUIRE(d->hd == 64 || d->hd == 128 || d->hd == 256, FRT_ESHAPE,
              "hd must be 64, 128 or 256, got %d", d->hd);
  FRT_REQUIRE(d->rows >= 0 && frt::head_counts_ok(d->n_seqs, d->max_q, d->hq, d->hkv, d->hd),
              FRT_ESHAPE, "bad n_seqs / rows / max_q / heads: %d, %d, %d, %d, %d", d->n_seqs,
              d->rows, d->max_q, d->hq, d->hkv);
  const size_t rec = frt_kv_record_bytes(FRT_PAGE_E2M1, d->page_size, d->hd);
  FRT_REQUIRE(rec > 0, FRT_ESHAPE, "page_size must be a power of two in [16, 1024], got %d",
              d->page_size);
  FRT_REQUIRE(d->max_pages >= 0 && d->n_pages >= 0 &&
                  long(d->max_pages) * d->page_size <= 0x40000000L,
              FRT_ESHAPE, "bad max_pages / n_pages: %d, %d", d->max_pages, d->n_pages);
  FRT_REQUIRE(d->window >= 0 && (d->window == 0 || d->causal), FRT_EINVAL,
              "a window must be >= 0 and needs causal");
  FRT_REQUIRE(std::isfinite(d->sm_scale), FRT_EINVAL, "sm_scale must be finite");
  if (d->n_seqs == 0 || d->rows == 0 || d->max_q == 0) return FRT_OK;
  FRT_REQUIRE(d->q && d->out && d->kv_len && d->k_scale && d->v_scale, FRT_EINVAL,
              "q, out, kv_len, k_scale and v_scale are required");
  FRT_REQUIRE(d->max_pages == 0 || (d->pool && d->page_table), FRT_EINVAL,
              "pool and page_table are required");
  FRT_REQUIRE(aligned(d->q, 16) && aligned(d->out, 16) && aligned(d->pool, 16) &&
                  d->ld_q % 8 == 0 && d->ld_out % 8 == 0,
              FRT_EALIGN, "q, out and pool must be 16-byte aligned with row strides that are "
              "multiples of 8");
  FRT_REQUIRE(d->ld_q >= long(d->hq) * d->hd && d->ld_out >= long(d->hq) * d->hd, FRT_ESHAPE,
              "a row stride is less than hq * hd");
  FRT_REQUIRE(aligned(d->page_table, 4) && aligned(d->cu_rows, 4) && aligned(d->kv_len, 4) &&
                  aligned(d->lse, 4) && aligned(d->k_scale, 4) && aligned(d->v_scale, 4),
              FRT_EALIGN, "page_table, cu_rows, kv_len, lse and the scales must be 4-byte aligned");
  const size_t need =
      frt_paged_attention_workspace_size(d->n_seqs, d->max_q, d->hq, d->hkv, d->hd);
  FRT_REQUIRE(d->workspace || need == 0, FRT_EINVAL, "workspace is required");
  FRT_REQUIRE(aligned(d->workspace, 16), FRT_EALIGN, "workspace must be 16-byte aligned");
  FRT_REQUIRE(d->workspace_bytes >= need, FRT_ERANGE, "workspace has %zu bytes, %zu needed",
              d->workspace_bytes, need);
  frt::AttnArgs a{};
  a.n_seqs = d->n_seqs; a.rows = d->rows; a.max_q = d->max_q; a.hq = d->hq; a.hkv = d->hkv;
  a.group = d->hq / d->hkv; a.causal = d->causal != 0;
  // no table holds more than 2^30 keys; place - window then stays in 32 bits
  a.window = d->window < 0x40000000 ? d->window : 0x40000000;
  a.max_pages = d->max_pages; a.sm_scale = d->sm_scale;
  a.q = d->q; a.ld_q = d->ld_q;
  a.pool = frt::make_page_pool(const_cast<void*>(d->pool), FRT_PAGE_E2M1, d->page_size, d->n_pages,
                               d->hkv, d->hd);
  a.page_table = d->page_table; a.cu_rows = d->cu_rows; a.kv_len = d->kv_len;
  a.k_scale = d->k_scale; a.v_scale = d->v_scale;
  a.out = d->out; a.ld_out = d->ld_out; a.lse = d->lse;
  a.status = frt::device_status_ptr();
  FRT_REQUIRE(a.status, FRT_ECUDA, "device status word unavailable");
  const long per_head = long(d->max_q) * a.group;
  if (frt::many_rows(per_head, long(d->n_seqs) * d->hkv, long(d->max_pages) * d->page_size))
    return frt::attn_many_launch(a, d->hd, d->workspace, static_cast<cudaStream_t>(stream));
  return frt::with_variant(d->hd, per_head, [&](auto v) {
    using C = typename decltype(v)::C;
    const long tiles = (per_head + C::R - 1) / C::R;
    const long chunks = (long(d->max_pages) * d->page_size + C::CK - 1) / C::CK;
    const long most = long(d->n_seqs) * d->hkv * tiles;
    // no sequence has fewer than one chunk
    const long all = most >= 0x7fffffffL ? most : most * (chunks > 1 ? chunks : 1);
    return v.launch(a, d->workspace, all, static_cast<cudaStream_t>(stream));
  });
}
