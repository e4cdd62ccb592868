// Attention of few new tokens per sequence (decoding, drafts to verify) over paged keys.
//
// A kv group's rows -- G heads x a few tokens -- are at most NQ = 16 or 32: as rows
// of a 128-row tile they would leave most of the tensor core's rows, and of the
// softmax's lanes, to padding.  Here they are the columns instead:
//   S^T [128 keys x NQ] = K Q^T,   O^T [D x NQ] += V^T P^T
// with K and V as the 128-row A operands straight from the pages and the few rows as B (N = NQ).
// A softmax thread owns a key: it has NQ scores to exponentiate instead of 128, so the
// chain of a block is a few hundred clocks and the kernel runs at the rate of its loads.
// The running maximum of a column runs across threads; it moves only where a weight would exceed
// 2^(SHIFT + TAU), which one barrier with an OR over the warpgroup tells.  Row sums stay per
// thread until the piece ends.  Warps:
//   0-3, 4-7  softmax of the even and the odd blocks (two streams with statistics and
//             accumulator of their own, joined at the piece's end by the first)
//   8         TMA producer of Q (bf16 cache), of K, and of V where a block is few boxes
//   9         tensor memory; issues the S MMAs, up to four blocks ahead of P V, across pieces
//   10        issues the P V MMAs (bf16 cache: writes zeros over V's rows past a sequence's end first)
//   11        scheduler; e4m3 cache: writes Q as two e4m3 terms; pages of less than 64 keys: TMA producer of V
//   12-15     e4m3 cache: V from e4m3 to fp16
// P^T goes to shared memory (the B operand's place), four buffers in turn (two where NQ = 32 and D = 128).
// The weights are rounded to the 16 bits of V's MMA, bf16 or fp16, as the forward rounds them; the row sums add
// the fp32 values.
//
// An MMA of M = 128 and N <= 32 takes 46 clk whatever N is (65 at N = 128), and issuing one about as long: with
// one issuing thread for both products a block took 1800 clk.  e4m3 cache: q is a sum of two
// e4m3 terms (x = hi + lo, hi = e4m3(x), lo = e4m3(x - hi): 8 bits of x), which stand side by side as 2 NQ columns
// of the same MMAs -- half the MMAs of two passes -- and are added in the softmax (the low terms carry a factor of 16).
// The weights are fp16 and V is turned into fp16, exactly, by four more warps.  Two e4m3 terms per weight would end at
// 2^-17 of a row's largest, and what falls below is lost with one sign: with one key 13 nats above 8191 others O was
// 18 % off.  Sixteen warps of six roles fill the instruction cache (120 KB of code).  Kept small for that are the
// conversion (rolled: 32 rows 124 -> 117 us) and the waits (paged_wait), and the scheduler splits q, not the
// converters (stalls for want of an instruction 1.4 per instruction issued, 4.9 with q split there).  The issuers are
// elected, which keeps descriptors uniform (32 rows 127 -> 116 us).
//
// Measured (B200, the whole call on the device): 64 sequences of up to 8192 bf16 keys, 8 kv heads of 128, 1.12 GB:
// 173-180 us, 6.2-6.5 TB/s, bound by DRAM.  4 x 32768 e4m3 keys, 268 MB: 56 us, 4.8 TB/s: 43 us of loads at
// 6.3 TB/s, the rest is start (planning, first loads: 5 us), end and merge.  One sequence of 2000 keys: 12.3-12.7 us,
// nearly all of it latency (planning 2 us, first load 1.5, two blocks 3, end 2, merge 3).  e4m3 in many short units is
// bound by the chain conversion -> P V (1000-1450 clk a block, where the loads take 1400, or 700 at D = 64), and a
// unit's end, 3000 clk, is not overlapped with the next one's P V (64 sequences of up to 4096 keys: 78 us,
// D = 64 65 us; loads alone 46 and 23).
#pragma once

#include "paged_plan.cuh"
#include "paged_tiles.cuh"
#include "sm100_common.cuh"

namespace attn {

template <int D, bool KV8, int NQ>
struct FewLayout {
  static constexpr int BN = 128;
  static constexpr int NBOX = KV8 ? 1 : D / 64;
  static constexpr int ROW_BYTES = KV8 ? D : 128;
  static constexpr int BOX_BYTES = 128 * ROW_BYTES;
  static constexpr int KV_BYTES = NBOX * BOX_BYTES;
  static constexpr int Q_COL = NQ * ROW_BYTES;               // one box column of Q rows (e4m3: the hi or the lo rows)
  static constexpr int Q_BYTES = (KV8 ? 2 : NBOX) * Q_COL;
  static constexpr int P_BYTES = 2 * NQ * 128;               // two 64-key columns of bf16 (e4m3 cache: of fp16)
  // V as the MMA reads it: D / 64 columns of 128-byte rows of 16-bit values (e4m3: written by the converters)
  static constexpr int VM_COL = 128 * 128;
  static constexpr int VM_BYTES = 128 * D * 2;
  static constexpr int VMST = KV8 ? 2 : 0;
  static constexpr int NBUF = 4;                             // score buffers in turn
  // P buffers and Q tiles in turn: fewer where that makes room for another K and V tile (64 sequences of up to 8192
  // bf16 keys, 8 tokens of 4 heads each: 215 us with two tiles, 195 with three)
  static constexpr bool TIGHT = D == 128 && NQ == 32;
  static constexpr int NPB = TIGHT ? 2 : 4, NQB = TIGHT ? 1 : 2;
  static constexpr int NS = KV8 ? 2 * NQ : NQ;               // columns of S^T: e4m3: q's hi terms, then its lo terms
  // as many tiles as shared memory holds
  static constexpr int ROOM = 227 * 1024 - 1024 - NQB * Q_BYTES - NPB * P_BYTES - VMST * VM_BYTES - 5 * 1024;
  static constexpr int ST = ROOM / (2 * KV_BYTES) < 8 ? ROOM / (2 * KV_BYTES) : 8;
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = K_OFF + ST * KV_BYTES;
  static constexpr int VM_OFF = V_OFF + ST * KV_BYTES;
  static constexpr int P_OFF = VM_OFF + VMST * VM_BYTES;
  static constexpr int Q_OFF = P_OFF + NPB * P_BYTES;
  static constexpr int BAR_OFF = Q_OFF + NQB * Q_BYTES;
  static constexpr int NI = 4;
  static constexpr int B_Q_FULL = 0;                    // [NI] by piece: its Q, and the factors of its scores
  static constexpr int B_Q_EMPTY = B_Q_FULL + NI;       // [NQB] by Q tile
  static constexpr int B_K_FULL = B_Q_EMPTY + NQB;      // [ST]
  static constexpr int B_K_EMPTY = B_K_FULL + ST;
  static constexpr int B_V_FULL = B_K_EMPTY + ST;
  static constexpr int B_V_EMPTY = B_V_FULL + ST;
  static constexpr int B_VM_FULL = B_V_EMPTY + ST;      // [VMST] e4m3: converted (four warps)
  static constexpr int B_S_FULL = B_VM_FULL + VMST;     // [NBUF]
  static constexpr int B_P_FULL = B_S_FULL + NBUF;      // [NBUF] four warps
  static constexpr int B_PV_DONE = B_P_FULL + NBUF;     // [NBUF]
  static constexpr int B_O_FINAL = B_PV_DONE + NBUF;
  static constexpr int B_XCHG = B_O_FINAL + 1;          // stream 1's statistics written (four warps)
  static constexpr int B_XCHG_READ = B_XCHG + 1;        // they and both accumulators read (four warps)
  static constexpr int B_ITEM_FULL = B_XCHG_READ + 1;   // [NI]
  static constexpr int B_ITEM_EMPTY = B_ITEM_FULL + NI;
  static constexpr int B_DRAIN = B_ITEM_EMPTY + NI;
  static constexpr int N_BARS = B_DRAIN + 2;
  static constexpr int ITEM_READERS = KV8 ? 15 : 11;  // 8 softmax warps, K's producer, the two issuers, 4 converters
  static constexpr int ITEM_OFF = BAR_OFF + (8 * N_BARS + 15) / 16 * 16;
  static constexpr int CQ_OFF = ITEM_OFF + NI * static_cast<int>(sizeof(PagedItem));  // [NI][NQ] factors of the scores
  static constexpr int STAT_OFF = CQ_OFF + NI * NQ * 4;    // [2 streams][5][NQ]: four warps' sums, the maximum
  static constexpr int WMAX_OFF = STAT_OFF + 2 * 5 * NQ * 4;  // [2 streams][NQ][4 warps]
  static constexpr int MOVED_OFF = WMAX_OFF + 2 * NQ * 4 * 4; // [2 streams][2][NQ]: the maxima in use, the last factors
  static constexpr int FAC_OFF = MOVED_OFF + 2 * 2 * NQ * 4;  // [2][NQ] factors of the accumulators
  static constexpr int POS_OFF = FAC_OFF + 2 * NQ * 4;        // [NQ] position of a column
  static constexpr int TMEM_SLOT_OFF = POS_OFF + NQ * 4;
  static constexpr int ABORT_OFF = TMEM_SLOT_OFF + 4;
  static constexpr int SMEM_USED = ABORT_OFF + 4;
  static constexpr int SMEM_BYTES = (SMEM_USED + 1024) > 122880 ? (SMEM_USED + 1024) : 122880;  // one CTA per SM
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(Q_COL % 1024 == 0 && P_BYTES % 2048 == 0, "operand tiles on swizzle boundaries");
  __device__ static constexpr uint32_t s_col(int b) { return static_cast<uint32_t>(b) * NS; }
  __device__ static constexpr uint32_t o_col(int t) { return static_cast<uint32_t>(NBUF * NS + t * NQ); }
  static constexpr uint32_t TMEM_COLS = NS == 16 ? 128 : (NS == 32 ? 256 : 512);
  static_assert(NBUF * NS + 2 * NQ <= static_cast<int>(TMEM_COLS), "tensor memory columns");
  static constexpr int THREADS = KV8 ? 512 : 384;
  // e4m3: 2 x 128 x 168 + 2 x 128 x 88 = 512 x 128
  static constexpr int REG_LAUNCH = 128, REG_SOFTMAX = 168, REG_OTHER = 88;
  static constexpr int WARP_K = 8, WARP_S = 9, WARP_PV = 10, WARP_SCHED = 11;
  // Weights up to 2^(SHIFT + TAU); a column's largest at 2^SHIFT or more.  bf16 weights have fp32's range.  fp16's end
  // at 65504, and below 2^-14 they step by 2^-24: with the largest at 2^7 to 2^15 a small weight is off by at most
  // 2^-32 of the largest (a row of 32768 keys by 2^-17 of it).
  static constexpr float SHIFT = KV8 ? 7.f : 0.f;
  static constexpr float TAU = 8.f;
  static constexpr float LO = 1.f / 16.f;  // e4m3: what q's lo term stands for
  static constexpr uint32_t HI = ROW_BYTES == 128 ? sdesc_sw128_hi(1024) : sdesc_sw64_hi(512);
  static constexpr uint32_t HI128 = sdesc_sw128_hi(1024);
};

constexpr float kNoKeyYet = -3e38f;  // a column's maximum before its first key

template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t* r) {
  static_assert(N == 16 || N == 32, "columns");
  if constexpr (N == 16) {
    tmem_ld16(taddr, r);
    tmem_ld_wait16(r);
  } else {
    tmem_ld32(taddr, r);
    tmem_ld_wait(r);
  }
}
// Multiplies an accumulator's N columns, 16 at a time, by factors in shared memory.
template <int N>
__device__ __forceinline__ void tmem_scale_cols(uint32_t taddr, const float* alpha) {
#pragma unroll 1
  for (int x = 0; x < N; x += 16) {
    uint32_t r[16];
    tmem_ld_cols<16>(taddr + x, r);
#pragma unroll
    for (int q = 0; q < 16; ++q) r[q] = __float_as_uint(__uint_as_float(r[q]) * alpha[x + q]);
    tmem_st16(taddr + x, r);
  }
  tmem_st_wait();
}

// Barrier of one warpgroup (id 1 or 2), and the same with the OR of a predicate.
__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(x ? 1u : 0u)
      : "memory");
  return r != 0;
}

// One value per column from a warp's 32 x N values: lane q (and q + 16 for N = 16) gets column q's reduction,
// by halving exchanges: each step a lane keeps the half of its columns that its own number names.
template <int N, typename Op>
__device__ __forceinline__ float warp_columns(const float* x, int lane, Op op) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = x[i];
#pragma unroll
  for (int half = N / 2; half > 0; half /= 2) {
    const bool up = (lane & half) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + half], half);
      v[i] = op(up ? v[i + half] : v[i], other);
    }
  }
  if (N == 16) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
  return v[0];
}

template <int D, bool KV8, int NQ>
__global__ void __launch_bounds__(FewLayout<D, KV8, NQ>::THREADS, 1)
    paged_few_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedParams p) {
  using L = FewLayout<D, KV8, NQ>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* const sptr = smem_raw + (sbase - raw);
  auto bar = [&](int slot) -> uint32_t { return sbase + L::BAR_OFF + 8u * slot; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sptr + L::ABORT_OFF);
  const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cta = static_cast<int>(blockIdx.x);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge kernel, which waits for this grid

  // ---- setup
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::N_BARS; ++i) {
      uint32_t n = 1;
      if ((i >= L::B_P_FULL && i < L::B_P_FULL + L::NBUF) || i == L::B_XCHG || i == L::B_XCHG_READ) n = 4;
      if (KV8 && i >= L::B_V_EMPTY && i < L::B_V_EMPTY + L::ST) n = 4;  // read by the converters
      if (KV8 && i >= L::B_VM_FULL && i < L::B_VM_FULL + L::VMST) n = 4;
      if (i >= L::B_ITEM_EMPTY && i < L::B_ITEM_EMPTY + L::NI) n = L::ITEM_READERS;
      mbar_init(bar(i), n);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == L::WARP_S) {
    tmem_alloc(sbase + L::TMEM_SLOT_OFF, L::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == L::WARP_K && lane == 0) {
    if (!KV8) tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // Q rows that no load reaches stay zero (padding columns of the products)
  for (int i = threadIdx.x; i < L::NQB * L::Q_BYTES / 16; i += 256)
    if (warp < 8) *reinterpret_cast<uint4*>(sptr + L::Q_OFF + i * 16) = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < NQ) reinterpret_cast<int*>(sptr + L::POS_OFF)[threadIdx.x] = static_cast<int>(threadIdx.x) / p.group;
  PagedWalk walk;
  if (warp == L::WARP_SCHED) {
    // the CTA's stretch, while the others set up
    paged_walk_start(p, walk, cta, static_cast<int>(gridDim.x), lane);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sptr + L::TMEM_SLOT_OFF);

  auto item_at = [&](int u) -> const volatile PagedItem* {
    return reinterpret_cast<const volatile PagedItem*>(sptr + L::ITEM_OFF + (u % L::NI) * sizeof(PagedItem));
  };
  auto wait_item = [&](int u) { return paged_wait(bar(L::B_ITEM_FULL + u % L::NI), (u / L::NI) & 1, ctl); };
  auto item_done = [&](int u) { return bar(L::B_ITEM_EMPTY + u % L::NI); };
  // One warp loads K and V in turn, unless a tile is many boxes (a warp issues one in about 100 clk): 4 x 32768 e4m3
  // keys in pages of 128 took 59 us with one warp and 63 with two, 64 sequences in pages of 16 211 and 176.
  const bool one_loader = p.box_shift >= 6;

  if constexpr (KV8) {
    static_assert(256 * L::REG_SOFTMAX + (L::THREADS - 256) * L::REG_OTHER <= L::THREADS * L::REG_LAUNCH, "register split");
    if (warp >= 8) setmaxnreg_dec<L::REG_OTHER>();
  }
  if (warp == L::WARP_K) {
    // ===================== TMA producer: Q, K =====================
    int kn = 0, vn = 0, qn = 0;
    int last_q[2] = {0, 0};  // the last pieces whose Q this warp loaded
    bool ok = true;
    for (int u = 0; ok; ++u) {
      if (!(ok = __all_sync(0xffffffffu, wait_item(u)))) break;
      const volatile PagedItem* it = item_at(u);
      const int row0 = it->row0, head = it->head, seq = it->seq, len = it->len, j0 = it->j0, n_loads = it->n_loads;
      mbar_arrive_warp(item_done(u));
      if (row0 < 0) break;
      if (n_loads == 0) {
        if (!KV8 && lane == 0) mbar_arrive(bar(L::B_Q_FULL + u % L::NI));
        continue;
      }
      if constexpr (!KV8) {
        const int qs = qn % L::NQB;
        if (qn >= L::NQB && !(ok = __all_sync(0xffffffffu, paged_wait(bar(L::B_Q_EMPTY + qs), (qn / L::NQB - 1) & 1, ctl))))
          break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(L::B_Q_FULL + u % L::NI), L::NBOX * p.group * p.tile_pos * 128);
#pragma unroll
          for (int x = 0; x < L::NBOX; ++x)
            tma_load_4d(sbase + L::Q_OFF + qs * L::Q_BYTES + x * L::Q_COL, &tm_q, bar(L::B_Q_FULL + u % L::NI), x * 64,
                        head * p.group, row0, 0);
        }
        last_q[1] = last_q[0];
        last_q[0] = u;
        ++qn;
      }
      PageWindow win{-1, -1, 0};
      for (int j = 0; ok && j < n_loads; ++j) {
        const int s = kn % L::ST;
        const uint32_t ph = ((kn / L::ST) - 1) & 1;
        if (kn >= L::ST && !(ok = __all_sync(0xffffffffu, paged_wait(bar(L::B_K_EMPTY + s), ph, ctl)))) break;
#pragma unroll
        for (int v = 0; v < (one_loader ? 2 : 1); ++v) {
          if (v == 1 && vn >= L::ST && !(ok = __all_sync(0xffffffffu, paged_wait(bar(L::B_V_EMPTY + s), ph, ctl)))) break;
          load_block<L::NBOX, L::ROW_BYTES>(p, v == 0 ? &tm_k : &tm_v, sbase + (v == 0 ? L::K_OFF : L::V_OFF) + s * L::KV_BYTES,
                                            bar((v == 0 ? L::B_K_FULL : L::B_V_FULL) + s), win, seq, head, len, j0 + j, lane);
          ++(v == 0 ? kn : vn);
        }
      }
    }
    // Drain: every load this warp issued has landed before the CTA may exit.
    for (int i = 0; i < 2 && i < qn; ++i)
      mbar_wait_drain(bar(L::B_Q_FULL + last_q[i] % L::NI), (last_q[i] / L::NI) & 1, 1000000000ull);
    for (int i = 0; i < L::ST && i < kn; ++i) {
      const int n = kn - 1 - i;
      mbar_wait_drain(bar(L::B_K_FULL + n % L::ST), (n / L::ST) & 1, 1000000000ull);
    }
    for (int i = 0; i < L::ST && i < vn; ++i) {
      const int n = vn - 1 - i;
      mbar_wait_drain(bar(L::B_V_FULL + n % L::ST), (n / L::ST) & 1, 1000000000ull);
    }
  } else if (warp == L::WARP_S) {
    // ===================== S^T = K Q^T =====================
    if (elect_one()) {
      constexpr uint32_t IDESC = KV8 ? idesc_e4m3_f32(128, L::NS) : idesc_bf16_f32(128, L::NS, false, false);
      int g = 0, qi = 0;
      bool ok = true;
      for (int u = 0; ok; ++u) {
        if (!(ok = wait_item(u))) break;
        const volatile PagedItem* it = item_at(u);
        const int row0 = it->row0, n = it->n_loads;
        mbar_arrive(item_done(u));
        if (row0 < 0) break;
        for (int j = 0; j < n; ++j, ++g) {
          const int buf = g % L::NBUF, stage = g % L::ST;
          ok = paged_wait(bar(L::B_K_FULL + stage), (g / L::ST) & 1, ctl);
          // four blocks ago: the scores were read before P was published, and P V is complete, so (with four P buffers)
          // the softmax that S_FULL wakes finds its P buffer free
          if (ok && g >= L::NBUF) ok = paged_wait(bar(L::B_PV_DONE + buf), ((g / L::NBUF) - 1) & 1, ctl);
          if (ok && j == 0) ok = paged_wait(bar(L::B_Q_FULL + u % L::NI), (u / L::NI) & 1, ctl);
          if (!ok) break;
          tc_fence_after();
          const uint32_t kd = sdesc_lo(sbase + L::K_OFF + stage * L::KV_BYTES, 16);
          const uint32_t qd = sdesc_lo(sbase + L::Q_OFF + (qi % L::NQB) * L::Q_BYTES, 16);
          if constexpr (KV8) {
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              umma_ss_f8_h(tmem + L::s_col(buf), kd + (kk * 32 >> 4), L::HI, qd + (kk * 32 >> 4), L::HI, IDESC, kk > 0 ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk & 3) * 32;
              umma_ss_h(tmem + L::s_col(buf), kd + ((kk >> 2) * L::BOX_BYTES + off >> 4), L::HI,
                        qd + ((kk >> 2) * L::Q_COL + off >> 4), L::HI, IDESC, kk > 0 ? 1u : 0u);
            }
          }
          umma_commit(bar(L::B_S_FULL + buf));
          umma_commit(bar(L::B_K_EMPTY + stage));
          if (j == n - 1) {
            umma_commit(bar(L::B_Q_EMPTY + qi % L::NQB));
            ++qi;
          }
        }
      }
      umma_commit(bar(L::B_DRAIN));  // no MMA may still write tensor memory when it is released
      mbar_wait_drain(bar(L::B_DRAIN), 0, 1000000000ull);
    }
  } else if (warp == L::WARP_PV) {
    // ===================== O^T += V^T P^T =====================
    // (bf16's type codes are 1, fp16's 0)
    constexpr uint32_t IDESC = idesc_bf16_f32(D, NQ, true, false) & ~(KV8 ? (1u << 7) | (1u << 10) : 0u);
    // V as the MMAs read it: loaded (bf16), converted (e4m3)
    constexpr int V_READY = KV8 ? L::B_VM_FULL : L::B_V_FULL, V_STAGES = KV8 ? L::VMST : L::ST;
    constexpr int V_PLACE = KV8 ? L::VM_OFF : L::V_OFF;
    // bf16: the whole warp, which may have zeros to write; e4m3: one lane
    auto all = [](bool x) { return KV8 ? x : __all_sync(0xffffffffu, x) != 0; };
    int g = 0;
    const bool issuer = KV8 ? elect_one() : lane == 0;
    bool ok = !KV8 || issuer;
    for (int u = 0; ok; ++u) {
      if (!(ok = all(wait_item(u)))) break;
      const volatile PagedItem* it = item_at(u);
      const int row0 = it->row0, n = it->n_loads, len = it->len, j0 = it->j0;
      if (!KV8) __syncwarp();
      if (issuer) mbar_arrive(item_done(u));
      if (row0 < 0) break;
      for (int j = 0; j < n; ++j, ++g) {
        const int buf = g % L::NBUF, stage = g % V_STAGES;
        if (!(ok = all(paged_wait(bar(V_READY + stage), (g / V_STAGES) & 1, ctl)))) break;
        const int live = len - (j0 + j) * L::BN;  // keys of the block that the sequence has
        if (!KV8 && live < L::BN) zero_tail<L::NBOX, L::ROW_BYTES>(sptr + V_PLACE + stage * L::VM_BYTES, live, lane);
        if (!(ok = all(paged_wait(bar(L::B_P_FULL + buf), (g / L::NBUF) & 1, ctl)))) break;
        if (issuer) {
          tc_fence_after();
          const uint32_t od = tmem + L::o_col(g & 1);
          const uint32_t pd = sdesc_lo(sbase + L::P_OFF + g % L::NPB * L::P_BYTES, 16);
          const uint32_t vd = sdesc_lo(sbase + V_PLACE + stage * L::VM_BYTES, L::VM_COL);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // 16 keys each
            umma_ss_h(od, vd + (kk * 2048 >> 4), L::HI128, pd + ((kk >> 2) * NQ * 128 + (kk & 3) * 32 >> 4), L::HI128, IDESC,
                      (j > 1 || kk > 0) ? 1u : 0u);
          umma_commit(bar(L::B_PV_DONE + buf));
          if (!KV8) umma_commit(bar(L::B_V_EMPTY + stage));  // (e4m3: the converters wait for PV_DONE)
          if (j == n - 1) umma_commit(bar(L::B_O_FINAL));
        }
        if (!KV8) __syncwarp();
      }
    }
    if (issuer) {
      umma_commit(bar(L::B_DRAIN + 1));
      mbar_wait_drain(bar(L::B_DRAIN + 1), 0, 1000000000ull);
    }
  } else if (warp == L::WARP_SCHED) {
    // ===================== scheduler; small pages: TMA producer of V =====================
    if (lane == 0) p.cut[cta] = paged_cut(p, walk, cta);
    int qn = 0, vn = 0;
    bool ok = true;
    for (int u = 0; ok; ++u) {
      const PagedItem it = paged_walk_next(p, walk, cta);
      if (u >= L::NI && !__all_sync(0xffffffffu, paged_wait(item_done(u), ((u / L::NI) - 1) & 1, ctl))) break;
      if (lane == 0) {
        volatile int* dst = reinterpret_cast<volatile int*>(sptr + L::ITEM_OFF + (u % L::NI) * sizeof(PagedItem));
        const int* from = reinterpret_cast<const int*>(&it);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(PagedItem) / 4); ++i) dst[i] = from[i];
        mbar_arrive(bar(L::B_ITEM_FULL + u % L::NI));
      }
      if (it.row0 < 0) break;
      PageWindow win{-1, -1, 0};
      int j = one_loader ? it.n_loads : 0;
      auto load_v = [&] {
        const int s = vn % L::ST;
        if (vn >= L::ST && !(ok = __all_sync(0xffffffffu, paged_wait(bar(L::B_V_EMPTY + s), ((vn / L::ST) - 1) & 1, ctl))))
          return;
        load_block<L::NBOX, L::ROW_BYTES>(p, &tm_v, sbase + L::V_OFF + s * L::KV_BYTES, bar(L::B_V_FULL + s), win, it.seq,
                                          it.head, it.len, it.j0 + j, lane);
        ++vn;
      };
      if constexpr (KV8) {
        if (it.n_loads > 0) {
          for (; j < it.n_loads && vn < L::ST; ++j) load_v();  // (the first blocks, while the ring is empty)
          const int qs = qn % L::NQB;
          if (qn >= L::NQB && !__all_sync(0xffffffffu, paged_wait(bar(L::B_Q_EMPTY + qs), (qn / L::NQB - 1) & 1, ctl))) break;
          ++qn;
          // 16 dims of a row per lane, D / 16 lanes side by side on a row; a loop, not unrolled: this runs once or
          // twice per CTA, and fetching its instructions is what it costs (unrolled over a whole row: 10k clk)
          constexpr int LANES = D / 16;
          uint8_t* const tile = sptr + L::Q_OFF + qs * L::Q_BYTES;
          const int ch = lane % LANES;
#pragma unroll 1
          for (int r = lane / LANES; r < NQ; r += 32 / LANES) {
            const bool real = r < p.group * it.n_pos;
            uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (real) {
              const int pos = r / p.group;
              const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<long long>(it.row0) + pos) * p.q_stride +
                                                                static_cast<long long>(it.head * p.group + r - pos * p.group) * D) +
                                 2 * ch;
              const uint4 w0 = src[0], w1 = src[1];
              x[0] = w0.x, x[1] = w0.y, x[2] = w0.z, x[3] = w0.w, x[4] = w1.x, x[5] = w1.y, x[6] = w1.z, x[7] = w1.w;
            }
            // the power of two that puts the row's largest element into [128, 256)
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) most = max(most, max(x[i] & 0x7f80u, (x[i] >> 16) & 0x7f80u));
#pragma unroll
            for (int off = LANES / 2; off > 0; off >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
            const uint32_t up = q_power(most);
            const float scale = __uint_as_float(up << 23);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t h0, l0, h1, l1;
              split16_e4m3x2(bf_lo(x[2 * i]) * scale, bf_hi(x[2 * i]) * scale, h0, l0);
              split16_e4m3x2(bf_lo(x[2 * i + 1]) * scale, bf_hi(x[2 * i + 1]) * scale, h1, l1);
              hi[i] = h0 | (h1 << 16);
              lo[i] = l0 | (l1 << 16);
            }
            const int sw = L::ROW_BYTES == 128 ? (r & 7) : ((r >> 1) & 3);
            uint8_t* dst = tile + r * L::ROW_BYTES + ((ch ^ sw) * 16);
            *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(dst + L::Q_COL) = make_uint4(lo[0], lo[1], lo[2], lo[3]);  // (16 times the remainder)
            if (ch == 0)
              reinterpret_cast<float*>(sptr + L::CQ_OFF)[(u % L::NI) * NQ + r] = real ? q_factor(p.scale_log2, up) : 0.f;
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(bar(L::B_Q_FULL + u % L::NI));
      }
      for (; ok && j < it.n_loads; ++j) load_v();
    }
    for (int i = 0; i < L::ST && i < vn; ++i) {
      const int n = vn - 1 - i;
      mbar_wait_drain(bar(L::B_V_FULL + n % L::ST), (n / L::ST) & 1, 1000000000ull);
    }
  } else if (KV8 && warp >= 12) {
    // ===================== converters: V from e4m3 to fp16 =====================
    const int tid = threadIdx.x - 384;
    int n = 0;
    bool ok = true;
    for (int u = 0; ok; ++u) {
      if (!(ok = __all_sync(0xffffffffu, wait_item(u)))) break;
      const volatile PagedItem* it = item_at(u);
      const int row0 = it->row0, len = it->len, j0 = it->j0, n_loads = it->n_loads;
      mbar_arrive_warp(item_done(u));
      if (row0 < 0) break;
      for (int j = 0; j < n_loads; ++j, ++n) {
        const int s = n % L::ST, sm = KV8 ? n % max(L::VMST, 1) : 0;
        ok = paged_wait(bar(L::B_V_FULL + s), (n / L::ST) & 1, ctl);
        // P V has read the block converted into the same place
        const int before = n - L::VMST;
        if (ok && before >= 0) ok = paged_wait(bar(L::B_PV_DONE + before % L::NBUF), (before / L::NBUF) & 1, ctl);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const int live = len - (j0 + j) * L::BN;  // rows past the sequence's end become zeros
        convert_block<D>(sptr + L::V_OFF + s * L::KV_BYTES, sptr + L::VM_OFF + sm * L::VM_BYTES, live, tid);
        mbar_arrive_warp(bar(L::B_VM_FULL + sm));
        mbar_arrive_warp(bar(L::B_V_EMPTY + s));
      }
    }
  } else {
    // ===================== softmax warpgroups =====================
    if constexpr (KV8) setmaxnreg_inc<L::REG_SOFTMAX>();
    const int t = warp >> 2, wq = warp & 3;
    const int key = threadIdx.x & 127;  // of the block; == TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>(wq * 32) << 16;
    float* const stat = reinterpret_cast<float*>(sptr + L::STAT_OFF);
    float* const wmax = reinterpret_cast<float*>(sptr + L::WMAX_OFF) + t * NQ * 4;
    float* const moved = reinterpret_cast<float*>(sptr + L::MOVED_OFF) + t * 2 * NQ;
    float* const fac = reinterpret_cast<float*>(sptr + L::FAC_OFF);
    const int* const pos_of = reinterpret_cast<const int*>(sptr + L::POS_OFF);
    // where this thread's key sits in a P row: 64-key columns of 16-bit values
    const uint32_t p_chunk = (key & 63) >> 3;
    const uint32_t p_at = (key >> 6) * (NQ * 128) + (key & 7) * 2;
    int g = 0;             // blocks of the CTA before this piece
    int items = 0;         // pieces with blocks
    // A wait that gave up (ok = false) must not leave the warpgroup's other warps at a barrier: the warp goes on to
    // the next vote (at a piece's start, or in a block), where all of them leave together.
    bool ok = true, failed = false;
    auto wait_for = [&](int slot, int phase) { ok = ok && __all_sync(0xffffffffu, paged_wait(bar(slot), phase & 1, ctl)); };
    for (int u = 0; !failed; ++u) {
      wait_for(L::B_ITEM_FULL + u % L::NI, u / L::NI);
      if (group_any(1 + t, !ok)) break;
      const volatile PagedItem* it = item_at(u);
      if (it->row0 < 0) break;
      const int nb = it->n_loads, len = it->len, d0 = it->d0, j0 = it->j0;
      const int real = p.group * it->n_pos;  // columns in use
      const int lim0 = p.causal ? min(d0, len - 1) : len - 1;  // last key every column sees
      float m[NQ], l[NQ];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        m[q] = q < real ? kNoKeyYet : -kNoKeyYet;
        l[q] = 0.f;
      }
      if (KV8 && nb > 0) wait_for(L::B_Q_FULL + u % L::NI, u / L::NI);  // (the factors of the scores)
      // (the last piece's maxima were read before the vote above)
      if ((threadIdx.x & 127) < NQ) {
        const int q = threadIdx.x & 127;
        moved[q] = q < real ? kNoKeyYet : -kNoKeyYet;
        moved[NQ + q] = 1.f;
      }
      bool first = true;  // no block of this stream yet
      for (int gg = g; gg < g + nb; ++gg) {
        if ((gg & 1) != t) continue;
        const int buf = gg % L::NBUF;
        wait_for(L::B_S_FULL + buf, gg / L::NBUF);
        tc_fence_after();
        uint32_t sr[NQ];
        tmem_ld_cols<NQ>(tmem + lane_addr + L::s_col(buf), sr);
        float* s = reinterpret_cast<float*>(sr);
        if constexpr (KV8) {
#pragma unroll
          for (int x = 0; x < NQ; x += 16) {
            uint32_t lo[16];
            tmem_ld_cols<16>(tmem + lane_addr + L::s_col(buf) + NQ + x, lo);
#pragma unroll
            for (int q = 0; q < 16; ++q) s[x + q] = fmaf(__uint_as_float(lo[q]), L::LO, s[x + q]);
          }
        }
        // scores in base-2 units
        if constexpr (KV8) {
          const float4* cq = reinterpret_cast<const float4*>(sptr + L::CQ_OFF + (u % L::NI) * NQ * 4);
#pragma unroll
          for (int q = 0; q < NQ / 4; ++q) {
            const float4 c = cq[q];
            s[4 * q] *= c.x;
            s[4 * q + 1] *= c.y;
            s[4 * q + 2] *= c.z;
            s[4 * q + 3] *= c.w;
          }
        } else {
#pragma unroll
          for (int q = 0; q < NQ; ++q) s[q] *= p.scale_log2;
        }
        const int kbase = (j0 + gg - g) * L::BN;
        if (kbase + L::BN - 1 > lim0) {
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            const int lim = p.causal ? min(d0 + pos_of[q], len - 1) : len - 1;
            if (kbase + key > lim) s[q] = -INFINITY;
          }
        }
        float over = s[0] - m[0];
#pragma unroll
        for (int q = 1; q < NQ; ++q) over = fmaxf(over, s[q] - m[q]);
        if (group_any(1 + t, over > L::SHIFT + L::TAU || !ok)) {
          if ((failed = group_any(1 + t, !ok))) break;
          // some column's maximum moves: the block's maxima over the four warps; thread q of the stream decides for
          // column q
          const float mine = warp_columns<NQ>(s, lane, [](float x, float y) { return fmaxf(x, y); });
          if (lane < NQ) wmax[lane * 4 + wq] = mine;
          group_sync(1 + t);
          if ((threadIdx.x & 127) < real) {
            const int q = threadIdx.x & 127;
            const float4 w = reinterpret_cast<const float4*>(wmax)[q];
            const float top = fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w));
            const float old = moved[q];
            // (false for a column with no visible key yet: -inf)
            const bool moves = top - old > L::SHIFT + L::TAU;
            const float to = moves ? top - L::SHIFT : old;
            moved[q] = to;
            moved[NQ + q] = moves ? exp2_mufu(old - to) : 1.f;
          }
          group_sync(1 + t);
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            m[q] = moved[q];
            l[q] *= moved[NQ + q];
          }
          if (!first) {
            // the stream's earlier P V must be complete before its accumulator is scaled
            wait_for(L::B_PV_DONE + (gg - 2) % L::NBUF, (gg - 2) / L::NBUF);
            tc_fence_after();
            tmem_scale_cols<NQ>(tmem + lane_addr + L::o_col(t), moved + NQ);
          }
        }
        if (L::NPB == 2 && gg >= 2) wait_for(L::B_PV_DONE + (gg - 2) % L::NBUF, (gg - 2) / L::NBUF);  // its P is read
        uint8_t* const pb = sptr + L::P_OFF + gg % L::NPB * L::P_BYTES + p_at;
#pragma unroll
        for (int q = 0; q < NQ; q += 2) {
          const float e0 = exp2_mufu(s[q] - m[q]), e1 = exp2_mufu(s[q + 1] - m[q + 1]);
          l[q] += e0;
          l[q + 1] += e1;
          uint8_t* const a0 = pb + q * 128 + ((p_chunk ^ (q & 7)) << 4);
          uint8_t* const a1 = pb + (q + 1) * 128 + ((p_chunk ^ ((q + 1) & 7)) << 4);
          const uint32_t w = KV8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
          *reinterpret_cast<uint16_t*>(a0) = static_cast<uint16_t>(w);
          *reinterpret_cast<uint16_t*>(a1) = static_cast<uint16_t>(w >> 16);
        }
        // the first P of a piece lets P V overwrite this stream's accumulator: stream 0 has read it (at the last piece's end)
        if (first && t == 1 && items > 0) wait_for(L::B_XCHG_READ, items - 1);
        first = false;
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive_warp(bar(L::B_P_FULL + buf));
      }
      if (failed) break;
      // ---- the piece's end: both streams' statistics, then O
      if (nb > 0) {
        // stream 1 has no block in this piece: its accumulator is not rewritten, but its place in `stat` is
        if (first && t == 1 && items > 0) wait_for(L::B_XCHG_READ, items - 1);
        const float mine = warp_columns<NQ>(l, lane, [](float x, float y) { return x + y; });
        if (lane < NQ) {
          stat[(t * 5 + wq) * NQ + lane] = mine;
          if (wq == 0) stat[(t * 5 + 4) * NQ + lane] = moved[lane];
        }
        if (t == 1) {
          mbar_arrive_warp(bar(L::B_XCHG));
        } else {
          group_sync(1);
          wait_for(L::B_XCHG, items);
        }
      }
      if (t == 0) {
        const int slot = it->slot;
        const long long row0 = it->row0;
        const int head0 = it->head * p.group;
        const size_t part = static_cast<size_t>(max(slot, 0)) * p.unit_rows;
        if (threadIdx.x < NQ) {
          const int q = threadIdx.x;
          float la = 0.f, lb = 0.f, ma = 0.f, mb = 0.f;
          if (nb > 0) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              la += stat[w * NQ + q];
              lb += stat[(5 + w) * NQ + q];
            }
            ma = stat[4 * NQ + q];
            mb = stat[9 * NQ + q];
          }
          const float top = fmaxf(la > 0.f ? ma : kNoKeyYet, lb > 0.f ? mb : kNoKeyYet);
          const float wa = la > 0.f ? exp2_mufu(ma - top) : 0.f, wb = lb > 0.f ? exp2_mufu(mb - top) : 0.f;
          const float sum = la * wa + lb * wb;
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          fac[q] = wa * inv;
          fac[NQ + q] = wb * inv;
          if (q < real) {
            const float lse2 = sum > 0.f ? top + log2f(sum) : -INFINITY;
            if (slot >= 0)
              p.l_part[part + q] = lse2;
            else
              p.lse[static_cast<long long>(head0 + q - pos_of[q] * p.group) * p.n_tokens + row0 + pos_of[q]] =
                  sum > 0.f ? lse2 * 0.69314718055994531f : -INFINITY;
          }
        }
        group_sync(1);
        // a stream without blocks in the piece has no accumulator (fac 0, not read)
        const bool have_a = nb > 1 || (nb == 1 && (g & 1) == 0), have_b = nb > 1 || (nb == 1 && (g & 1) == 1);
        if (nb > 0) {
          wait_for(L::B_O_FINAL, items);
          tc_fence_after();
        }
        // row d of O^T: TMEM lane d, or lanes 32 g .. 32 g + 15 for rows 16 g .. 16 g + 15 of 64
        const int d = D == 128 ? key : (lane < 16 ? wq * 16 + lane : -1);
        int head = 0;
        long long at = slot >= 0 ? static_cast<long long>(part) * D + d : (row0 * p.H_q + head0) * D + d;
#pragma unroll 1
        for (int c0 = 0; c0 < real; c0 += 16) {  // 16 columns at a time
          __syncwarp();  // the tensor-memory loads take the whole warp, the stores below not every lane
          float x[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) x[q] = 0.f;
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            if (!(st == 0 ? have_a : have_b)) continue;
            uint32_t acc[16];
            tmem_ld_cols<16>(tmem + lane_addr + L::o_col(st) + c0, acc);
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float w = fac[st * NQ + c0 + q];
              if (w > 0.f) x[q] = fmaf(__uint_as_float(acc[q]), w, x[q]);
            }
          }
          if (d < 0) continue;
          if constexpr (KV8) {  // (not in the factors: v_scale / sum may be too small for 32 bits where the product is not)
#pragma unroll
            for (int q = 0; q < 16; ++q) x[q] *= p.v_scale;
          }
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            if (c0 + q >= real) break;
            if (slot >= 0) {
              p.o_part[at] = x[q];
              at += D;
            } else {
              p.o[at] = __float2bfloat16(x[q]);
              at += D;
              if (++head == p.group) {  // the next token's heads
                head = 0;
                at += static_cast<long long>(p.H_q - p.group) * D;
              }
            }
          }
        }
        // stat and the accumulators are read (fac is this stream's own)
        tc_fence_before();
        if (nb > 0) mbar_arrive_warp(bar(L::B_XCHG_READ));
        group_sync(1);  // fac and stat are read by every thread of the stream before the next piece writes them
      }
      g += nb;
      items += nb > 0 ? 1 : 0;
      mbar_arrive_warp(item_done(u));
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == L::WARP_S) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

}  // namespace attn
