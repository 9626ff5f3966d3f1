// paged_attn_many.cu -- attention over 4-bit pages for many query rows
// (prompts, chunks): both products on tcgen05 tensor cores.
//
// A CTA takes R = 128 QT rows of one (sequence, kv head) -- row r is token
// r / G, head r % G of the group -- and runs over their keys in tiles of KVT:
//   S = Q K^T       Q fp16 (a power of two per row) and K fp16 in shared memory
//   P = 2^(S - m)   written over S in tensor memory as fp16
//   O += P V        P from tensor memory, V fp16 in shared memory
// One thread owns one row of S and O, so the softmax needs no exchange
// between threads.  The two row tiles of a CTA alternate: one's softmax runs
// while the tensor cores work for the other.
//
// Bound by the tensor cores and the exponentials alike: a 128 x 128 tile of
// hd 128 takes 2 x 512 clocks of MMA and 1024 of the 16-a-clock exponential
// unit.  The widening of the codes is shared by all R rows (about a tenth of
// the issue slots at R = 256), which is what the second row tile is for.
// Neither is reached: a causal prompt of 8192 tokens, 32 q heads on 8 of 128,
// runs in 593 us on one input and 607 over changing ones (905 to 927 TFLOP/s),
// because a row tile's chain, in an earlier build of 585 us S to P 2150 clocks
// and P to the next S 1980, is longer than the pipes' shares.
// Tiles of 64 keys with Q K^T one ahead (831 us) and two threads a row (585)
// did not shorten it.
//
// When the units (sequences x heads x row tiles) leave SMs idle, the keys of
// each are cut into `splits`, whose partial states a second kernel joins.
#include <type_traits>

#include "frt_attn.cuh"

namespace frt {
namespace {

template <int HD>
struct ManyCfg {
  static constexpr int QT = HD == 256 ? 1 : 2;     // row tiles of 128
  static constexpr int KVT = HD == 256 ? 64 : 128; // keys of a tile
  static constexpr int R = 128 * QT;
  static constexpr int kWide = HD == 256 ? 256 : 128;  // threads that widen codes
  // four warpgroups: QT of softmax, the rest but one of widening, and the MMAs
  static constexpr int kThreads = 512;
  // registers a thread of each (setmaxnreg), of the launch's 512 x 128
  static constexpr int kRegsSoftmax = 184;
  static constexpr int kRegsWide = QT == 2 ? 80 : 128;
  static constexpr int kRegsMma = 64;
  static_assert(128 * (QT * kRegsSoftmax + (3 - QT) * kRegsWide + kRegsMma) <= 512 * 128,
                "the shares exceed the launch's registers");
  static constexpr int kQBytes = 128 * HD * 2;     // one row tile
  static constexpr int kKvBytes = KVT * HD * 2;    // one K or V tile
  static constexpr int kBlock = KVT * 128;         // its 64-element column block
  static constexpr int kCodeBytes = KVT * (HD / 2 + HD / 16);  // a tile's codes, then its scales
  static constexpr int kRing = 3;                  // code tiles under way, keys and values in turn
  static constexpr int kSmem = QT * kQBytes + 4 * kKvBytes + kRing * kCodeBytes + 1024 + 256;
  // TMEM columns: two S (or P) slots, then O
  static constexpr int kTmem = 512;
  static constexpr int kO = 2 * KVT;
};

// Instruction descriptor, kind::f16: D fp32 (bits 4-5 = 1), A and B f16
// (0), A K-major, B K-major or MN-major (bit 16), N >> 3 at 17, M >> 4 at 24.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
}

// Shared-memory descriptor of an MN-major tile with the 128-byte swizzle:
// atoms of 64 (contiguous) x 8 elements; `lead` bytes between atoms along the
// contiguous dimension, 1024 bytes between groups of 8 along the other.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t smem_addr, uint32_t lead) {
  return uint64_t((smem_addr & 0x3FFFFu) >> 4) | (uint64_t(lead >> 4) << 16) |
         (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// A (128 rows x 16) from tensor memory: two f16 to a column, 8 columns.
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      :: "r"(d), "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// 32 columns of this thread's TMEM lane; the values may be used after
// tmem_wait_ld(r).
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr) : "memory");
}

// The registers pass through the wait, so no use can move ahead of it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
        "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
        "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),
        "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
        "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :: "memory");
}

__device__ __forceinline__ void pass_through(uint32_t (&r)[32]) {
  asm volatile(""
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
        "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
        "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),
        "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
        "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

// Every warp of a warpgroup moves its registers a thread up or down.
template <int N, int FROM = 128>
__device__ __forceinline__ void set_regs() {
  if constexpr (N > FROM) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N));
  if constexpr (N < FROM) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
         "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
         "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The key tiles [begin, end) that row tile rows [row0, row0 + 128) sees.
template <int KVT>
__device__ __forceinline__ void tile_range(const AttnArgs& a, const Seq& q, int row0, int* begin,
                                           int* end) {
  const int rows = q.Lq * a.group;
  *begin = *end = 0;
  if (row0 >= rows) return;
  const int first = q.L - q.Lq + row0 / a.group;
  const int last = q.L - q.Lq + min(row0 + 127, rows - 1) / a.group;
  const int hi = a.causal ? min(q.L, last + 1) : q.L;
  const int lo = a.window > 0 ? max(0, first - a.window + 1) : 0;
  if (hi <= lo) return;
  *begin = lo / KVT;
  *end = (hi + KVT - 1) / KVT;
}

// Partial states: [unit * splits + split] tiles of R rows x HD sums, then
// the rows' maxima and sums of weights.
template <int HD>
__device__ __forceinline__ float* partial_tile(float* base, long index) {
  return base + index * (ManyCfg<HD>::R * (HD + 2));
}

template <int HD>
__global__ void __launch_bounds__(ManyCfg<HD>::kThreads, 1)
attn_many_kernel(AttnArgs a, int splits, int tiles_max) {
  using C = ManyCfg<HD>;
  constexpr int QT = C::QT, KVT = C::KVT, R = C::R;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024 - smem_u32(smem_raw) % 1024) % 1024;
  uint8_t* q_s = smem;
  uint8_t* k_s = q_s + QT * C::kQBytes;
  uint8_t* v_s = k_s + 2 * C::kKvBytes;
  // the rows of Q as they come, before there is a second K tile or a V tile
  uint8_t* q_stage = k_s + C::kKvBytes;
  static_assert(R * (HD * 2 + 16) <= 3 * C::kKvBytes, "Q does not fit its staging");
  uint8_t* code_s = v_s + 2 * C::kKvBytes;      // codes as they come from the pages
  uint64_t* bars = reinterpret_cast<uint64_t*>(code_s + C::kRing * C::kCodeBytes);
  uint64_t *q_in = bars + 23, *q_full = bars, *k_full = bars + 2, *k_empty = bars + 4, *v_full = bars + 6,
           *v_empty = bars + 8, *s_full = bars + 10, *p_full = bars + 12, *pv_done = bars + 14,
           *done = bars + 16, *code_full = bars + 17, *code_empty = bars + 20;
  uint32_t* k_hidden = reinterpret_cast<uint32_t*>(bars + 25);  // [8] 16-key groups in bad pages
  uint32_t* tmem_ptr = k_hidden + 8;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(k_hidden + 9);

  const int tid = int(threadIdx.x), warp = tid / 32, lane = tid % 32;
  pdl_trigger();
  // what needs nothing of the kernel before
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_in[i], 4);
      mbar_init(&q_full[i], 128);
      mbar_init(&k_full[i], C::kWide);
      mbar_init(&v_full[i], C::kWide);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(done, 1);
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(&code_full[i], 1);
      mbar_init(&code_empty[i], C::kWide);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  // ahead of the sequence's lookup, which hides it (when far rows had no loop
  // of their own yet: a prompt of 8192 tokens 591 us against 602, 32 sequences
  // of 1 to 2048 tokens 2176 against 2212; a block without rows pays for it
  // too: 4096 tokens among 63 of one, 916 against 888)
  if (warp == 12) {
    tmem_alloc(tmem_ptr, C::kTmem);
    tmem_relinquish();
  }
  long b = blockIdx.x;
  const long part_index = b;
  const int split = int(b % splits);
  b /= splits;
  const int head = int(b % a.hkv);
  b /= a.hkv;
  const int s = int(b % a.n_seqs);
  // causal tiles with the most keys first
  const int tile = tiles_max - 1 - int(b / a.n_seqs);
  const Seq q = load_seq<R, KVT>(a, s, tile == 0 && head == 0 && split == 0 && tid == 0);
  if (tile >= q.tiles) {   // the sequence is shorter than the longest
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(*tmem_ptr, C::kTmem);
    return;
  }

  int begin[QT], end[QT], lo = 0x7fffffff, hi = 0;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    tile_range<KVT>(a, q, tile * R + t * 128, &begin[t], &end[t]);
    if (begin[t] < end[t]) {
      lo = min(lo, begin[t]);
      hi = max(hi, end[t]);
    }
  }
  const int n_all = max(0, hi - lo);
  const int js = lo + int(long(n_all) * split / splits), je = lo + int(long(n_all) * (split + 1) / splits);
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    begin[t] = max(begin[t], js);
    end[t] = min(end[t], je);
  }
  const int n = n_all ? je - js : 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_ptr;

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_wait_bounded(bar, parity, kAttnWaitNs, abort_flag)) return true;
    atomicExch(a.status, FRT_ETIMEOUT);
    *abort_flag = 1;
    return false;
  };
  // one answer for the warp, whose next steps are warp-wide
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
  };

  if (warp < 4 * QT) {
    // ------------------------------------------------- softmax, one row ----
    set_regs<C::kRegsSoftmax>();
    const int t = warp / 4, r = tid % 128;
    const int row = tile * R + t * 128 + r;
    const bool live = row < q.Lq * a.group;
    const int token = live ? row / a.group : 0;
    const int h = head * a.group + (live ? row - token * a.group : 0);
    const int n_live = max(0, min(32, q.Lq * a.group - (row - lane)));  // of this warp
    const uint32_t lane_base = tmem + (uint32_t(warp % 4 * 32) << 16);

    // Q: a bulk copy of each row (padded, so that the threads' rows start at
    // different banks) into what will be K and V buffers, then fp16 under a
    // power of two that brings the row's largest below 2
    const float scale = *a.k_scale * a.sm_scale * kLog2e;
    uint8_t* in = q_stage + (t * 128 + r) * (HD * 2 + 16);
    if (lane == 0) mbar_arrive_expect_tx(&q_in[t], n_live * HD * 2);
    __syncwarp();
    if (live) bulk_load(in, a.q + long(q.r0 + token) * a.ld_q + long(h) * HD, HD * 2, &q_in[t]);
    const bool got_q = wait_warp(&q_in[t], 0);
    if (!got_q) mbar_wait_bounded(&q_in[t], 0, kAttnWaitNs, nullptr);  // no exit with copies in flight
    float big = 0.0f;
#pragma unroll 4
    for (int i = 0; i < HD / 8; ++i) {
      float f[8];
      unpack8(*reinterpret_cast<const uint4*>(in + i * 16), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) big = fmaxf(big, fabsf(f[k]));
    }
    const int e = q_exponent(big);
    // the sign of the scale goes into Q, so that the largest score is that of
    // the largest product
    const float down = copysignf(__uint_as_float(uint32_t(254 - e) << 23), scale);
    const float factor = score_factor(scale, __uint_as_float(uint32_t(e) << 23));
#pragma unroll 4
    for (int i = 0; i < HD / 8; ++i) {
      float f[8];
      unpack8(*reinterpret_cast<const uint4*>(in + i * 16), f);
      *reinterpret_cast<uint4*>(q_s + t * C::kQBytes + i / 8 * (128 * 128) + r * 128 + ((i % 8) ^ (r & 7)) * 16) =
          make_uint4(pack_f16x2(f[0] * down, f[1] * down), pack_f16x2(f[2] * down, f[3] * down),
                     pack_f16x2(f[4] * down, f[5] * down), pack_f16x2(f[6] * down, f[7] * down));
    }
    fence_proxy_async_smem();
    mbar_arrive(&q_full[t]);

    int lim_hi = 0, lim_lo = 0;
    if (live) {
      const int place = q.L - q.Lq + token;
      lim_hi = a.causal ? min(q.L, place + 1) : q.L;
      lim_lo = a.window > 0 ? max(0, place - a.window + 1) : 0;
    }
    float m = -INFINITY;
    uint64_t l2 = 0;
    int k = 0;
    // a row without a token holds leftovers of shared memory: it is never far
    const float c = live && is_far<HD>(factor) ? 1.0f : factor;
    const uint64_t c2 = f2_pack(c, c);
    // Two loops: with the products of far rows in a branch of one loop, the
    // expert's 50 tokens took 20.6 us (19.5 so and without far rows), a prompt
    // of 8192 594 (592 so, 590 without), 32 sequences of 1 to 2048 tokens 2221
    // (2190 so, 2140 without), 4096 tokens among 63 of one 937 so, 917 without.
    auto attend = [&](auto far) {
    for (int j = begin[t]; got_q && j < end[t]; ++j, ++k) {
      const int slot = QT == 2 ? t : k & 1;
      if (!wait_warp(&s_full[slot], QT == 2 ? k & 1 : (k >> 1) & 1)) break;
      tc_fence_after();
      const uint32_t s_addr = lane_base + slot * KVT;
      const uint32_t hidden = k_hidden[(j - js) & 7];
      const int key0 = j * KVT;
      const int rel_hi = lim_hi - key0, rel_lo = lim_lo - key0;
      const bool masked = __any_sync(0xffffffffu, rel_hi < KVT || rel_lo > 0) || hidden;
      // drop what the row does not see from 32 products
      auto mask32 = [&](uint32_t (&x)[32], int base) {
#pragma unroll
        for (int u = 0; u < 32; ++u)
          if (base + u >= rel_hi || base + u < rel_lo || (hidden >> ((base + u) / 16) & 1)) x[u] = 0xFF800000u;
      };
      auto max32 = [](const uint32_t (&x)[32], float v) {
#pragma unroll
        for (int u = 0; u < 32; u += 2)
          v = fmaxf(fmaxf(v, __uint_as_float(x[u])), __uint_as_float(x[u + 1]));
        return v;
      };
      uint32_t x[KVT / 32][32];
      tmem_ld32_async(s_addr, x[0]);
      tmem_ld32_async(s_addr + 32, x[1]);
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < KVT / 32; i += 2) {
        tmem_wait_ld(x[i]);
        pass_through(x[i + 1]);
        if (i + 2 < KVT / 32) {
          tmem_ld32_async(s_addr + 32 * (i + 2), x[i + 2]);
          tmem_ld32_async(s_addr + 32 * (i + 3), x[i + 3]);
        }
        if constexpr (decltype(far)::value) {
          const float f = c == factor ? 1.0f : factor;
#pragma unroll
          for (int u = 0; u < 32; ++u) {
            x[i][u] = __float_as_uint(__fmul_rn(__uint_as_float(x[i][u]), f));
            x[i + 1][u] = __float_as_uint(__fmul_rn(__uint_as_float(x[i + 1][u]), f));
          }
        }
        if (masked) {
          mask32(x[i], 32 * i);
          mask32(x[i + 1], 32 * i + 32);
        }
        mx = max32(x[i + 1], max32(x[i], mx));
      }
      const float top = mx == -INFINITY ? mx : mx * c;
      // the maximum (kLift below the largest score when it is set) is raised
      // only when a score passes it by more than kGrow, so O is rarely rescaled
      const bool grow = top > m + kGrow;
      if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? ex2(m - (top - kLift)) : 1.0f;
        l2 = mul2(l2, f2_pack(f, f));
        if (grow) m = top - kLift;
        if (k > 0) {
          // S of tile k vouches for the products up to k - 2, and those of
          // k wait for this warp: the parity names those of k - 1
          if (!wait_warp(&pv_done[t], (k - 1) & 1)) break;
          tc_fence_after();
#pragma unroll 1
          for (int i = 0; i < HD / 32; ++i) {
            uint32_t o[32];
            tmem_ld32_async(lane_base + C::kO + t * HD + 32 * i, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t y[16];
#pragma unroll
              for (int w = 0; w < 16; ++w) y[w] = o[16 * u + w];
              tmem_st16(lane_base + C::kO + t * HD + 32 * i + 16 * u, y);
            }
          }
          tmem_wait_st();
        }
      }
      const float base = m == -INFINITY ? 0.0f : -m;
      const uint64_t base2 = f2_pack(base, base);
      auto weigh32 = [&](const uint32_t (&x)[32], int i) {
        uint32_t p[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const uint64_t v = fma2(f2_pack(__uint_as_float(x[2 * u]), __uint_as_float(x[2 * u + 1])), c2, base2);
          const float p0 = ex2(f2_lo(v)), p1 = ex2(f2_hi(v));
          l2 = add2(l2, f2_pack(p0, p1));
          p[u] = pack_f16x2(p0, p1);
        }
        tmem_st16(s_addr + 16 * i, p);
      };
#pragma unroll
      for (int i = 0; i < KVT / 32; ++i) weigh32(x[i], i);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[slot]);
    }
    };
    if (__any_sync(0xffffffffu, live && is_far<HD>(factor))) attend(std::true_type{});
    else attend(std::false_type{});

    // --- the row's result: through shared memory (after `done` every buffer
    // is idle), so that the stores are whole rows ---
    const float l = f2_lo(l2) + f2_hi(l2);
    const bool whole = splits == 1;
    float* part = partial_tile<HD>(a.partials, part_index);
    const float inv = l > 0.0f ? *a.v_scale / l : l * *a.v_scale;
    if (!wait_warp(done, 0)) k = 0;  // every product of the CTA is in
    tc_fence_after();
    const int row_bytes = whole ? HD * 2 : HD * 4;
    const int stride = row_bytes + 16;
    uint8_t* staged = smem + (t * 128 + warp % 4 * 32) * (HD * 4 + 16);
    uint8_t* mine = staged + lane * stride;
#pragma unroll 1
    for (int i = 0; i < HD / 32; ++i) {
      uint32_t x[32];
      tmem_ld32_async(lane_base + C::kO + t * HD + 32 * i, x);
      tmem_wait_ld(x);
      if (k == 0) {  // nothing was summed
#pragma unroll
        for (int u = 0; u < 32; ++u) x[u] = 0;
      }
      if (whole) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float f[8];
#pragma unroll
          for (int w = 0; w < 8; ++w) f[w] = __uint_as_float(x[8 * u + w]) * inv;
          *reinterpret_cast<uint4*>(mine + i * 64 + u * 16) = pack8_bf16(f);
        }
      } else {
#pragma unroll
        for (int u = 0; u < 8; ++u)
          *reinterpret_cast<uint4*>(mine + i * 128 + u * 16) =
              make_uint4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
      }
    }
    uint8_t* dst = whole ? reinterpret_cast<uint8_t*>(a.out + long(q.r0 + token) * a.ld_out + long(h) * HD)
                         : reinterpret_cast<uint8_t*>(part + long(t * 128 + r) * HD);
    __syncwarp();
    constexpr int kShift = HD == 64 ? 3 : HD == 128 ? 4 : 5;   // 16-byte pieces of a bf16 row
    const int shift = whole ? kShift : kShift + 1;
    for (int base = 0; base < n_live << shift; base += 32 * 4) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int x = base + 32 * u + lane, rr = x >> shift, at = (x & ((1 << shift) - 1)) * 16;
        uint8_t* to = reinterpret_cast<uint8_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), rr & 31));
        if (rr < n_live)
          *reinterpret_cast<uint4*>(to + at) = *reinterpret_cast<const uint4*>(staged + rr * stride + at);
      }
    }
    if (live && whole && a.lse)
      a.lse[long(q.r0 + token) * a.hq + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
    if (!whole) {
      part[R * HD + t * 128 + r] = m;
      part[R * HD + R + t * 128 + r] = l;
    }
  } else if (warp < 12) {
    // ------------------------------------------- widening, K then V tiles ----
    set_regs<C::kRegsWide>();
    const int wt = tid - (12 * 32 - C::kWide);
    constexpr int kPieces = KVT * HD / 32;       // 32 codes and two scales
    constexpr int kMine = kPieces / C::kWide;
    // one tile from its codes to fp16; a key behind the sequence's end or in a
    // bad page comes out as zeros, whatever is there
    auto widen = [&](uint8_t* dst, const uint8_t* src, int j, uint32_t hidden) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int flat = i * C::kWide + wt;
        const int key = flat / (HD / 32), piece = flat % (HD / 32);
        const uint4 code = *reinterpret_cast<const uint4*>(src + flat * 16);
        uint32_t sc = *reinterpret_cast<const uint16_t*>(src + KVT * (HD / 2) + flat * 2);
        if (j * KVT + key >= q.L || (hidden >> (key / 16) & 1)) sc = 0;
        sc = e4m3x2_to_f16(sc);
        uint8_t* rowp = dst + piece / 2 * C::kBlock + key * 128;
        uint32_t w[4] = {code.x, code.y, code.z, code.w};
        // eight neighbouring lanes write eight different 16-byte columns:
        // pieces of different column blocks start at different words
        const int turn = HD == 256 ? piece / 2 : HD == 128 ? piece / 2 * 2 : 0;
        if (HD >= 128 && (turn & 2)) {
          uint32_t x = w[0]; w[0] = w[2]; w[2] = x;
          x = w[1]; w[1] = w[3]; w[3] = x;
          sc = __byte_perm(sc, 0, 0x1032);
        }
        if (HD == 256 && (turn & 1)) {
          uint32_t x = w[0]; w[0] = w[1]; w[1] = x;
          x = w[2]; w[2] = w[3]; w[3] = x;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t hv[4];
          e2m1x8_to_f16(w[u], hv);
          const uint32_t s2 = __byte_perm(sc, 0, u < 2 ? 0x1010 : 0x3232);
#pragma unroll
          for (int v = 0; v < 4; ++v) hv[v] = hmul2(hv[v], s2);
          const int col = (piece % 2 * 4 + (u ^ turn)) ^ (key & 7);
          *reinterpret_cast<uint4*>(rowp + col * 16) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
        }
      }
      fence_proxy_async_smem();
    };
    int slot = 0;
    uint32_t turn = 0;
    for (int i = 0; i < 2 * n; ++i) {        // keys and values of tile i / 2
      const int st = i >> 1 & 1;
      const uint32_t ph = i >> 2 & 1;
      const bool v = i & 1;
      if (!wait_warp(&code_full[slot], turn) || !wait_warp(v ? &v_empty[st] : &k_empty[st], ph ^ 1u)) break;
      if (i == 1) {   // from here on, over Q's staging
        bool ok = true;
        for (int t = 0; t < QT; ++t) ok = ok && wait_warp(&q_full[t], 0);
        if (!ok) break;
      }
      widen((v ? v_s : k_s) + st * C::kKvBytes, code_s + slot * C::kCodeBytes, js + i / 2,
            k_hidden[i / 2 & 7]);
      mbar_arrive(v ? &v_full[st] : &k_full[st]);
      mbar_arrive(&code_empty[slot]);
      if (++slot == C::kRing) { slot = 0; turn ^= 1u; }
    }
  } else {
    // ------------------------------------------------------------ the MMAs ----
    set_regs<C::kRegsMma>();
    if (tid == 12 * 32) {
    constexpr uint32_t kQk = idesc_f16(128, KVT, false);
    constexpr uint32_t kPv = idesc_f16(128, HD, true);
    const uint32_t qa = smem_u32(q_s), ka = smem_u32(k_s), va = smem_u32(v_s);
    auto qk = [&](int t, int slot, int st) {
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t off = kk % 4 * 32;
        umma_f16_ss(tmem + slot * KVT, sdesc_k_sw128(qa + t * C::kQBytes + kk / 4 * (128 * 128) + off),
                    sdesc_k_sw128(ka + st * C::kKvBytes + kk / 4 * C::kBlock + off), kQk, kk > 0);
      }
      umma_commit(&s_full[slot]);
    };
    auto pv = [&](int t, int slot, int st, bool more) {
#pragma unroll
      for (int kk = 0; kk < KVT / 16; ++kk)
        umma_f16_ts(tmem + C::kO + t * HD, tmem + slot * KVT + 8 * kk,
                    sdesc_mn_sw128(va + st * C::kKvBytes + kk * 2048, C::kBlock), kPv, more || kk > 0);
      umma_commit(&pv_done[t]);
    };
    bool ok = true;
    int k[QT];     // tiles done by a row tile
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      k[t] = 0;
      // without a key tile too: `done` lets the softmax warps stage results
      // where other warps' rows of Q may still be on their way
      ok = ok && wait(&q_full[t], 0);
    }
    if constexpr (QT == 2) {
      // at tile j, for each row tile: P V of tile j - 1 (its P overlies the
      // S of tile j), then Q K^T of tile j
      bool pending[2] = {false, false};
      for (int i = 0; ok && i <= n; ++i) {
        const int st = i & 1, j = js + i;
        if (i < n) ok = wait(&k_full[st], (i >> 1) & 1);
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (ok && pending[t]) {
            ok = wait(&v_full[st ^ 1], ((i - 1) >> 1) & 1) && wait(&p_full[t], (k[t] - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            pv(t, t, st ^ 1, k[t] > 1);
            pending[t] = false;
          }
          if (ok && i < n && j >= begin[t] && j < end[t]) {
            qk(t, t, st);
            pending[t] = true;
            ++k[t];
          }
        }
        if (ok && i > 0) umma_commit(&v_empty[st ^ 1]);
        if (ok && i < n) umma_commit(&k_empty[st]);
      }
    } else {
      // two S slots: Q K^T of tile j before P V of tile j - 1
      for (int i = 0; ok && i <= n; ++i) {
        const int st = i & 1;
        if (i < n) {
          ok = wait(&k_full[st], (i >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          qk(0, st, st);
          umma_commit(&k_empty[st]);
        }
        if (i > 0) {
          const uint32_t ph = ((i - 1) >> 1) & 1;
          ok = wait(&v_full[st ^ 1], ph) && wait(&p_full[st ^ 1], ph);
          if (!ok) break;
          tc_fence_after();
          pv(0, st ^ 1, st ^ 1, i > 1);
          umma_commit(&v_empty[st ^ 1]);
        }
      }
    }
    // nothing in flight when the tensor memory is freed
    umma_commit(done);
    mbar_wait_bounded(done, 0, kAttnWaitNs, nullptr);
    } else if (warp == 13) {
      // -------------------------------------------- the pages' codes, a tile ----
      const int ps = a.pool.page_size;
      const int span = min(ps, KVT), pieces = KVT / span;   // keys of a piece; lanes at work
      auto look_up = [&](int j) {
        const int key = j * KVT + lane * span;
        if (lane >= pieces || key >= q.L) return -1;
        return __ldg(a.page_table + long(s) * a.max_pages + (key >> a.pool.shift));
      };
      int next = n > 0 ? look_up(js) : -1;
      bool ok = true;
      int slot = 0, sent = 0;
      uint32_t turn = 0;
      for (int i = 0; ok && i < n; ++i) {
        int page = next;
        const int key = (js + i) * KVT + lane * span;
        const bool bad = lane < pieces && key < q.L && (page < 0 || page >= a.pool.n_pages);
        if (bad) {
          atomicExch(a.status, FRT_ERANGE);
          page = -1;
        }
        if (i + 1 < n) next = look_up(js + i + 1);
        const uint32_t groups = ((1u << (span / 16)) - 1) << (lane * span / 16 & 31);
        const uint32_t hidden = __reduce_or_sync(0xffffffffu, bad ? groups : 0u);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, page >= 0)) * span * (HD / 2 + HD / 16);
        const int at = key & (ps - 1);
        for (int half = 0; ok && half < 2; ++half) {   // keys, values
          if (lane == 0) {
            ok = wait(&code_empty[slot], turn ^ 1u);
            if (ok) {
              if (!half) k_hidden[i & 7] = hidden;
              mbar_arrive_expect_tx(&code_full[slot], bytes);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          ++sent;
          if (page >= 0) {
            const uint8_t* rec = a.pool.base + (long(page) * a.pool.hkv + head) * a.pool.record_bytes +
                                 half * (a.pool.record_bytes / 2);
            uint8_t* dst = code_s + slot * C::kCodeBytes;
            bulk_load(dst + lane * span * (HD / 2), rec + at * (HD / 2), span * (HD / 2), &code_full[slot]);
            bulk_load(dst + KVT * (HD / 2) + lane * span * (HD / 16),
                      rec + ps * (HD / 2) + at * (HD / 16), span * (HD / 16), &code_full[slot]);
          }
          if (++slot == C::kRing) { slot = 0; turn ^= 1u; }
        }
      }
      // after a wait that ran out: no exit with copies in flight
      if (*abort_flag && lane == 0)
        for (int i = max(0, sent - C::kRing); i < sent; ++i)
          mbar_wait_bounded(&code_full[i % C::kRing], i / C::kRing & 1, kAttnWaitNs, nullptr);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, C::kTmem);
}

// Joins the splits: one warp a row and head.
template <int HD>
__global__ void __launch_bounds__(256) attn_join_kernel(AttnArgs a, int splits, int tiles_max) {
  using C = ManyCfg<HD>;
  constexpr int V = HD / 32;  // floats a lane
  const int lane = int(threadIdx.x) % 32;
  const long w = (blockIdx.x * 256L + threadIdx.x) / 32;
  pdl_trigger();
  pdl_wait();
  const long per_seq = long(a.max_q) * a.hq;
  const int s = int(w / per_seq);
  if (s >= a.n_seqs) return;
  const int token = int(w % per_seq / a.hq), h = int(w % a.hq);
  const Seq q = load_seq<C::R, C::KVT>(a, s, false);
  if (token >= q.Lq) return;
  const int head = h / a.group;
  const int row = token * a.group + h - head * a.group;
  const long unit = (long(tiles_max - 1 - row / C::R) * a.n_seqs + s) * a.hkv + head;
  const int r = row % C::R;
  // lane i: the maximum, the sum and the weight of split i (16 at most)
  const float* mine = partial_tile<HD>(a.partials, unit * splits + (lane < splits ? lane : 0));
  const float mi = lane < splits ? mine[C::R * HD + r] : -INFINITY;
  const float li = lane < splits ? mine[C::R * HD + C::R + r] : 0.0f;
  const float m = warp_max(mi);
  const float wi = mi == -INFINITY ? 0.0f : ex2(mi - m);  // 0: a share that the row does not see
  const float l = warp_sum(wi * li);
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
#pragma unroll 4
  for (int i = 0; i < splits; ++i) {
    const float* p = partial_tile<HD>(a.partials, unit * splits + i) + long(r) * HD + lane * 2;
    const float f = __shfl_sync(0xffffffffu, wi, i);
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const float2 x = *reinterpret_cast<const float2*>(p + v * 32);
      acc[v] += x.x * f;
      acc[v + 1] += x.y * f;
    }
  }
  const float inv = l > 0.0f ? *a.v_scale / l : l * *a.v_scale;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + long(q.r0 + token) * a.ld_out + long(h) * HD);
#pragma unroll
  for (int v = 0; v < V; v += 2) dst[v / 2 * 32 + lane] = pack_bf16x2(acc[v] * inv, acc[v + 1] * inv);
  if (lane == 0 && a.lse)
    a.lse[long(q.r0 + token) * a.hq + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int HD>
struct Many {
  using C = ManyCfg<HD>;
  static constexpr size_t kHead = 4096;  // the other kernels' counters, which stay zero
  static long tiles(int max_q, int group) { return (long(max_q) * group + C::R - 1) / C::R; }
  static long units(int n_seqs, int max_q, int hq, int hkv) {
    return long(n_seqs) * hkv * tiles(max_q, hq / hkv);
  }
  // As many splits as the idle SMs hold, 16 at most.
  static int splits(int n_seqs, int max_q, int hq, int hkv) {
    const long u = units(n_seqs, max_q, hq, hkv);
    const long n = u > 0 ? num_sms() / u : 1;
    return n < 1 ? 1 : n > 16 ? 16 : int(n);
  }
  static size_t workspace(int n_seqs, int max_q, int hq, int hkv) {
    const int n = splits(n_seqs, max_q, hq, hkv);
    return n == 1 ? 0 : kHead + size_t(units(n_seqs, max_q, hq, hkv)) * n * C::R * (HD + 2) * 4;
  }
  static int launch(AttnArgs a, void* ws, cudaStream_t st) {
    auto kern = attn_many_kernel<HD>;
    if (int rc = allow_smem(reinterpret_cast<const void*>(kern), C::kSmem)) return rc;
    // 128 keys a split at least: with fewer, joining costs what it saves
    const long most = (long(a.max_pages) * a.pool.page_size + 127) / 128;
    int n = splits(a.n_seqs, a.max_q, a.hq, a.hkv);
    if (n > most) n = most < 1 ? 1 : int(most);
    a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kHead);
    const int tm = int(tiles(a.max_q, a.group));
    const long blocks = units(a.n_seqs, a.max_q, a.hq, a.hkv) * n;
    FRT_REQUIRE(blocks <= 0x7fffffffL, FRT_ESHAPE, "n_seqs * max_q * hq is too large");
    if (int rc = launch_pdl("frt_paged_attention_fp4", kern, dim3(unsigned(blocks)), dim3(C::kThreads),
                            C::kSmem, st, a, n, tm))
      return rc;
    if (n == 1) return FRT_OK;
    const long warps = long(a.n_seqs) * a.max_q * a.hq;
    return launch_pdl("frt_paged_attention_fp4", attn_join_kernel<HD>, dim3(unsigned((warps + 7) / 8)),
                      dim3(256), 0, st, a, n, tm);
  }
};

}  // namespace

size_t attn_many_workspace(int hd, int n_seqs, int max_q, int hq, int hkv) {
  return hd == 64    ? Many<64>::workspace(n_seqs, max_q, hq, hkv)
         : hd == 128 ? Many<128>::workspace(n_seqs, max_q, hq, hkv)
                     : Many<256>::workspace(n_seqs, max_q, hq, hkv);
}

int attn_many_launch(const AttnArgs& a, int hd, void* workspace, cudaStream_t stream) {
  return hd == 64    ? Many<64>::launch(a, workspace, stream)
         : hd == 128 ? Many<128>::launch(a, workspace, stream)
                     : Many<256>::launch(a, workspace, stream);
}

}  // namespace frt
