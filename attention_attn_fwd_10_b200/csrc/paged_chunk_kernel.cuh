// Attention of chunks of new tokens over paged keys, on the tensor cores.
//
// The forward kernel's pipeline (two 128-row tiles of queries in tensor memory,
// S = Q K^T and O += P V as tcgen05 MMAs, conditional rescaling) fed from pages.  Tile rows are query-major over
// the heads of a kv group -- row r is position r / G, head r % G -- for every
// G, so K and V are read once per group; G need not divide 128 (the rows past
// G * floor(128 / G) are padding).  Warps:
//   0-3, 4-7  softmax of tile 0 and 1 (thread = row)
//   8         TMA producer of Q (bf16 cache) and K
//   9         tensor memory, MMA issue
//   10        TMA producer of V
//   11        scheduler: walks the CTA's stretch of the work list (paged_plan.cuh) and
//             publishes its pieces in a ring of four, ahead of the other roles
// A 128-key block is 128 / box_rows boxes, each within one page; a producer warp's
// lanes hold the page numbers of its next 32 boxes and issue one box each.  Boxes
// wholly past a sequence's end are not loaded.  Slots past the end hold anything
// (NaN too): their scores are masked by selection, and the V producer writes zeros over
// their rows once the block has landed, since 0 x NaN in P V would not be 0.
// A piece whose tokens fit one tile runs as two streams: tile 0 takes its even and tile 1 its
// odd blocks for the same rows, and tile 0 joins both.
//
// e4m3 cache: S runs as kind::f8f6f4 with q as a sum of two e4m3 terms,
//   q = hi + lo,  hi = e4m3(q), lo = e4m3(q - hi):
// the remainder of a bf16 after hi is a multiple of its last bit of at most 8 such steps, so q (scaled per row by a
// power of two into e4m3's range) is represented exactly down to 2^-17 of the row's largest element; two
// MMAs at twice the rate cost what one bf16 MMA does.  The softmax weights are fp16 and V is turned into
// fp16 in shared memory (exactly) by four more warps, 12-15: 128 x D values a block, where splitting the weights as
// well would take 256 x 128 and the time of the busiest warps (a block of two tiles, D = 64: 4.3k clk of softmax
// instead of 2.1k).
//
// Measured (B200, the whole call on the device): 2048 new tokens at the end of 32768 keys, 32 heads over 8 of 128,
// 1.07 TFLOP: 1000-1170 us as the power cap allows, 0.92-1.07 PFLOP/s (e4m3 cache: 1085-1100 us; the contiguous
// forward of the same shape: 1008 us).  Bound, as that one, by the chain softmax -> P V -> S of a tile: 3.7k clk a
// two-tile block, 1.05k of them MMAs.
// The weights are rounded to the 16 bits of V's MMA, bf16 (fp16 over an e4m3 cache); the row sums add the fp32 values.
#pragma once

#include <cuda_fp16.h>

#include "fwd_kernel.cuh"
#include "paged_plan.cuh"
#include "paged_tiles.cuh"
#include "sm100_common.cuh"

namespace attn {

template <int D, bool KV8>
struct ChunkLayout {
  static constexpr int BN = 128;
  static constexpr int ELEM = KV8 ? 1 : 2;
  static constexpr int NBOX = KV8 ? 1 : D / 64;          // boxes across a K / V row
  static constexpr int ROW_BYTES = KV8 ? D : 128;        // bytes of a box row (its swizzle span)
  static constexpr int BOX_BYTES = 128 * ROW_BYTES;      // a 128-row box column
  static constexpr int KV_BYTES = NBOX * BOX_BYTES;      // a K or V tile
  // bf16: a Q tile is NBOX box columns; e4m3: the hi and the lo tile
  static constexpr int Q_BYTES = KV8 ? 2 * KV_BYTES : KV_BYTES;
  static constexpr int KST = KV8 ? (D == 128 ? 4 : 5) : (D == 128 ? 3 : 5);
  static constexpr int VST = KV8 ? (D == 128 ? 2 : 4) : (D == 128 ? 2 : 4);
  // V as the MMA reads it: D / 64 columns of 128-byte rows of 16-bit values (e4m3: written by the converters)
  static constexpr int VM_BYTES = 128 * D * 2;
  static constexpr int VMST = KV8 ? (D == 64 ? 4 : 2) : VST;
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = 2 * Q_BYTES;
  static constexpr int V_OFF = K_OFF + KST * KV_BYTES;   // as loaded
  static constexpr int VM_OFF = KV8 ? V_OFF + VST * KV_BYTES : V_OFF;
  static constexpr int BAR_OFF = VM_OFF + VMST * VM_BYTES;
  static constexpr int NI = 4;  // work item ring
  static constexpr int B_Q_FULL = 0;                 // [t]
  static constexpr int B_Q_EMPTY = B_Q_FULL + 2;     // [t]
  static constexpr int B_K_FULL = B_Q_EMPTY + 2;     // [KST]
  static constexpr int B_K_EMPTY = B_K_FULL + KST;
  static constexpr int B_V_FULL = B_K_EMPTY + KST;   // [VST]
  static constexpr int B_V_EMPTY = B_V_FULL + VST;
  static constexpr int B_V_RAW = B_V_EMPTY + VST;    // bf16: a block to be mended before V_FULL
  static constexpr int B_VM_FULL = B_V_RAW + 1;      // [VMST] e4m3: converted (four warps)
  static constexpr int B_VM_EMPTY = B_VM_FULL + VMST;
  static constexpr int B_S_FULL = B_VM_EMPTY + VMST; // [t]
  static constexpr int B_P_FULL = B_S_FULL + 2;      // [t][half]
  static constexpr int B_O_FINAL = B_P_FULL + 4;     // [t]
  static constexpr int B_XCHG = B_O_FINAL + 2;
  static constexpr int B_XCHG_READ = B_XCHG + 1;
  static constexpr int B_ITEM_FULL = B_XCHG_READ + 1;  // [NI]
  static constexpr int B_ITEM_EMPTY = B_ITEM_FULL + NI;
  static constexpr int B_DRAIN = B_ITEM_EMPTY + NI;
  static constexpr int N_BARS = B_DRAIN + 1;
  static constexpr int ITEM_READERS = KV8 ? 15 : 11;  // 8 softmax warps, two producers, the issuer, 4 converters
  static constexpr int XCHG_OFF = BAR_OFF + (8 * N_BARS + 15) / 16 * 16;  // two streams: tile 1's row statistics
  static constexpr int ITEM_OFF = XCHG_OFF + 1024;
  static constexpr int TMEM_SLOT_OFF = ITEM_OFF + NI * static_cast<int>(sizeof(PagedItem));
  static constexpr int ABORT_OFF = TMEM_SLOT_OFF + 4;
  static constexpr int SMEM_USED = ABORT_OFF + 4;
  // 1 KiB of slack to align the base; at least 120 KiB, so one CTA (512 tensor-memory columns) per SM
  static constexpr int SMEM_BYTES = (SMEM_USED + 1024) > 122880 ? (SMEM_USED + 1024) : 122880;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  __device__ static constexpr uint32_t s_col(int t) { return static_cast<uint32_t>(t) * 128u; }
  __device__ static constexpr uint32_t o_col(int t) { return 256u + static_cast<uint32_t>(t) * D; }
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int THREADS = KV8 ? 512 : 384;
  static constexpr int WARP_K = 8, WARP_MMA = 9, WARP_V = 10, WARP_SCHED = 11;
  // 2 x 128 x 216 + 128 x 72 = 384 x 168; e4m3: 2 x 128 x 200 + 256 x 56 = 512 x 128
  static constexpr int REG_LAUNCH = KV8 ? 128 : 168, REG_SOFTMAX = KV8 ? 200 : 216, REG_OTHER = KV8 ? 56 : 72;
  // Weights up to 2^(SHIFT + TAU), a row's largest at 2^SHIFT or more (paged_few_kernel.cuh says why: fp16's least
  // steps are then 2^-31 of the largest)
  static constexpr float SHIFT = KV8 ? 7.f : 0.f, DOWN = KV8 ? 1.f / 128.f : 1.f;  // 2^-SHIFT
  static constexpr float TAU = 8.f;
  // shared-memory descriptors' high half: K-major Q and K, and V (MN-major)
  static constexpr uint32_t HI = ROW_BYTES == 128 ? sdesc_sw128_hi(1024) : sdesc_sw64_hi(512);
  static constexpr uint32_t HI_V = sdesc_sw128_hi(1024);
};

// A query row (bf16, D values in w) as hi and lo e4m3 terms, scaled by the power of two that puts its largest
// element into [128, 256); written to row `row` of the swizzled tiles at dst and dst + lo_off (nowhere
// where dst is null).  Returns scale_log2 with the power taken back out.
template <int D, int ROW_BYTES>
__device__ __forceinline__ float q_row_to_e4m3x2(const uint4* w, int row, uint8_t* dst, int lo_off, float scale_log2) {
  const uint32_t* x = reinterpret_cast<const uint32_t*>(w);
  uint32_t most = 0;  // the largest exponent field, in place in either half of a word
#pragma unroll
  for (int i = 0; i < D / 2; ++i) most = max(most, max(x[i] & 0x7f80u, (x[i] >> 16) & 0x7f80u));
  const uint32_t up = q_power(most);
  const float scale = __uint_as_float(up << 23);
  if (dst != nullptr) {
#pragma unroll
    for (int ch = 0; ch < D / 16; ++ch) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h0, l0, h1, l1;
        const uint32_t a = x[ch * 8 + 2 * i], b = x[ch * 8 + 2 * i + 1];
        split_e4m3x2(bf_lo(a) * scale, bf_hi(a) * scale, h0, l0);
        split_e4m3x2(bf_lo(b) * scale, bf_hi(b) * scale, h1, l1);
        hi[i] = h0 | (h1 << 16);
        lo[i] = l0 | (l1 << 16);
      }
      const int sw = ROW_BYTES == 128 ? (row & 7) : ((row >> 1) & 3);
      uint8_t* at = dst + row * ROW_BYTES + ((ch ^ sw) * 16);
      *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(at + lo_off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  return q_factor(scale_log2, up);
}

// p = 2^(s c - m) for half of a 128-column score row, packed to pairs of bf16 (F16: of fp16); returns the fp32 sum of
// the unrounded p.  MUFU's ex2 throughout: it maps -inf to an exact 0, so masked and whole blocks run the same code,
// and the row's sum keeps its 32 bits.  (A cubic on the FMA pipe for an eighth of them, 7.5e-5 off, left the lse
// 1.1e-6 off and needs a second copy of the code for masked blocks, which short pieces pay for in instruction
// fetches: 16 sequences of mixed lengths 122.4 us with it, 110 without, bf16 100.3 and 91.0; 2048 tokens over 32768
// 1147 and 1123.)
template <bool F16>
__device__ __forceinline__ float exp_weights(const uint32_t* sr, float c, float m, uint32_t* pk, int half) {
  const uint64_t c2 = f2_pack(c, c);
  const uint64_t nm2 = f2_pack(-m, -m);
  uint64_t acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = 0ull;
#pragma unroll
  for (int q = 0; q < 32; ++q) {
    const int cp = 32 * half + q;
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[2 * cp]), __uint_as_float(sr[2 * cp + 1])), c2, nm2), x0, x1);
    const float e0 = exp2_mufu(x0), e1 = exp2_mufu(x1);
    acc[q & 3] = f2_add(acc[q & 3], f2_pack(e0, e1));
    if constexpr (F16)
      pk[q] = pack_f16x2(e0, e1);
    else
      pk[q] = pack_bf16x2(e0, e1);
  }
  float a0, a1;
  f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a0, a1);
  return a0 + a1;
}

template <int D, bool KV8>
__global__ void __launch_bounds__(ChunkLayout<D, KV8>::THREADS, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedParams p) {
  using L = ChunkLayout<D, KV8>;
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
      if ((i >= L::B_P_FULL && i < L::B_P_FULL + 4) || i == L::B_XCHG || i == L::B_XCHG_READ) n = 4;
      if (KV8 && i >= L::B_Q_FULL && i < L::B_Q_FULL + 2) n = 4;  // written by the four warps of a tile
      if (KV8 && i >= L::B_V_EMPTY && i < L::B_V_EMPTY + L::VST) n = 4;     // read by the converters
      if (KV8 && i >= L::B_VM_FULL && i < L::B_VM_FULL + L::VMST) n = 4;
      if (i >= L::B_ITEM_EMPTY && i < L::B_ITEM_EMPTY + L::NI) n = L::ITEM_READERS;
      mbar_init(bar(i), n);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == L::WARP_MMA) {
    tmem_alloc(sbase + L::TMEM_SLOT_OFF, L::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == L::WARP_K && lane == 0) {
    if (!KV8) tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  PagedWalk walk;
  if (warp == L::WARP_SCHED) {
    // the CTA's stretch, while the others set up
    paged_walk_start(p, walk, cta, static_cast<int>(gridDim.x), lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sptr + L::TMEM_SLOT_OFF);
  static_assert(2 * 128 * L::REG_SOFTMAX + (L::THREADS - 256) * L::REG_OTHER <= L::THREADS * L::REG_LAUNCH,
                "register split");

  // Piece u of the CTA sits in ring slot u % NI once ITEM_FULL completes; every reader arrives on
  // ITEM_EMPTY when it needs it no more.
  auto item_at = [&](int u) -> const volatile PagedItem* {
    return reinterpret_cast<const volatile PagedItem*>(sptr + L::ITEM_OFF + (u % L::NI) * sizeof(PagedItem));
  };
  auto wait_item = [&](int u) { return mbar_wait(bar(L::B_ITEM_FULL + u % L::NI), (u / L::NI) & 1, ctl); };
  auto item_done = [&](int u) { return bar(L::B_ITEM_EMPTY + u % L::NI); };

  if (warp >= 8) setmaxnreg_dec<L::REG_OTHER>();
  if (warp == L::WARP_K) {
    // ===================== TMA producer: Q, K =====================
    int kn = 0, qn0 = 0, qn1 = 0;
    bool ok = true;
    for (int u = 0; ok; ++u) {
      if (!(ok = __all_sync(0xffffffffu, wait_item(u)))) break;
      const volatile PagedItem* it = item_at(u);
      const int row0 = it->row0, head = it->head, seq = it->seq, len = it->len, j0 = it->j0, n_loads = it->n_loads;
      const int nb0 = it->nb0, nb1 = it->nb1, dual = it->dual;
      mbar_arrive_warp(item_done(u));
      if (row0 < 0) break;
      if constexpr (!KV8) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const bool want = t == 0 ? nb0 > 0 : (nb1 > 0 && !dual);
          if (!ok || !want) continue;
          int& qn = t == 0 ? qn0 : qn1;
          // the previous piece's last S_t has read Q_t
          if (qn > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait(bar(L::B_Q_EMPTY + t), (qn - 1) & 1, ctl)))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(L::B_Q_FULL + t), L::NBOX * p.group * p.tile_pos * 128);
#pragma unroll
            for (int x = 0; x < L::NBOX; ++x)
              tma_load_4d(sbase + L::Q_OFF + t * L::Q_BYTES + x * L::BOX_BYTES, &tm_q, bar(L::B_Q_FULL + t), x * 64,
                          head * p.group, row0 + t * p.tile_pos, 0);
          }
          ++qn;
        }
      }
      PageWindow win{-1, -1, 0};
      for (int j = 0; ok && j < n_loads; ++j) {
        const int s = kn % L::KST;
        if (kn >= L::KST && !(ok = __all_sync(0xffffffffu, mbar_wait(bar(L::B_K_EMPTY + s), ((kn / L::KST) - 1) & 1, ctl))))
          break;
        load_block<L::NBOX, L::ROW_BYTES>(p, &tm_k, sbase + L::K_OFF + s * L::KV_BYTES, bar(L::B_K_FULL + s), win, seq, head,
                                           len, j0 + j, lane);
        ++kn;
      }
    }
    // Drain: every load this warp issued has landed before the CTA may exit.
    if (qn0 > 0) mbar_wait_drain(bar(L::B_Q_FULL), (qn0 - 1) & 1, 1000000000ull);
    if (qn1 > 0) mbar_wait_drain(bar(L::B_Q_FULL + 1), (qn1 - 1) & 1, 1000000000ull);
    for (int i = 0; i < L::KST && i < kn; ++i) {
      const int n = kn - 1 - i;
      mbar_wait_drain(bar(L::B_K_FULL + n % L::KST), (n / L::KST) & 1, 1000000000ull);
    }
  } else if (warp == L::WARP_V) {
    // ===================== TMA producer: V =====================
    int vn = 0, raw_n = 0;
    bool ok = true;
    for (int u = 0; ok; ++u) {
      if (!(ok = __all_sync(0xffffffffu, wait_item(u)))) break;
      const volatile PagedItem* it = item_at(u);
      const int row0 = it->row0, head = it->head, seq = it->seq, len = it->len, j0 = it->j0, n_loads = it->n_loads;
      mbar_arrive_warp(item_done(u));
      if (row0 < 0) break;
      PageWindow win{-1, -1, 0};
      for (int j = 0; ok && j < n_loads; ++j) {
        const int s = vn % L::VST;
        if (vn >= L::VST && !(ok = __all_sync(0xffffffffu, mbar_wait(bar(L::B_V_EMPTY + s), ((vn / L::VST) - 1) & 1, ctl))))
          break;
        const uint32_t dst = sbase + L::V_OFF + s * L::KV_BYTES;
        const int live = len - (j0 + j) * L::BN;  // keys of the block that the sequence has
        if (KV8 || live >= L::BN) {
          load_block<L::NBOX, L::ROW_BYTES>(p, &tm_v, dst, bar(L::B_V_FULL + s), win, seq, head, len, j0 + j, lane);
        } else {
          load_block<L::NBOX, L::ROW_BYTES>(p, &tm_v, dst, bar(L::B_V_RAW), win, seq, head, len, j0 + j, lane);
          const bool landed = __all_sync(0xffffffffu, mbar_wait(bar(L::B_V_RAW), raw_n & 1, ctl));
          if (landed) {
            zero_tail<L::NBOX, L::ROW_BYTES>(sptr + (dst - sbase), live, lane);
            if (lane == 0) mbar_arrive(bar(L::B_V_FULL + s));
          }
          ++raw_n;
          ok = landed;
          if (!ok) mbar_wait_drain(bar(L::B_V_RAW), (raw_n - 1) & 1, 1000000000ull);
        }
        if (ok) ++vn;
      }
    }
    for (int i = 0; i < L::VST && i < vn; ++i) {
      const int n = vn - 1 - i;
      mbar_wait_drain(bar(L::B_V_FULL + n % L::VST), (n / L::VST) & 1, 1000000000ull);
    }
  } else if (warp == L::WARP_MMA) {
    // ===================== MMA issuer =====================
    if (lane == 0) {
      constexpr uint32_t IDESC_S = KV8 ? idesc_e4m3_f32(128, 128) : idesc_bf16_f32(128, 128, false, false);
      // (bf16's type codes are 1, fp16's 0)
      constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, false, true) & ~(KV8 ? (1u << 7) | (1u << 10) : 0u);
      auto opaque = [](uint32_t x) {  // keeps the descriptors' arithmetic where it is used (72 registers)
        uint32_t y;
        asm volatile("mov.b32 %0, %1;" : "=r"(y) : "r"(x));
        return y;
      };
      auto issue_s = [&](int t, int q_tile, int stage) {
        const uint32_t base = opaque(sbase);
        const uint32_t qd = sdesc_lo(base + L::Q_OFF + q_tile * L::Q_BYTES, 16);
        const uint32_t kd = sdesc_lo(base + L::K_OFF + stage * L::KV_BYTES, 16);
        if constexpr (KV8) {
#pragma unroll
          for (int kk = 0; kk < 2 * (D / 32); ++kk) {  // the hi terms, then the lo terms; 32 dims (32 bytes) each
            const uint32_t off = (kk % (D / 32)) * 32;
            umma_ss_f8_h(tmem + L::s_col(t), qd + ((kk / (D / 32)) * L::KV_BYTES + off >> 4), L::HI, kd + (off >> 4), L::HI,
                         IDESC_S, kk > 0 ? 1u : 0u);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * L::BOX_BYTES + (kk & 3) * 32;
            umma_ss_h(tmem + L::s_col(t), qd + (off >> 4), L::HI, kd + (off >> 4), L::HI, IDESC_S, kk > 0 ? 1u : 0u);
          }
        }
        umma_commit(bar(L::B_S_FULL + t));
      };
      // PV_t(j) in two halves of 64 keys, each issued once its half of P_t(j) is in tensor memory
      auto issue_pv_half = [&](int t, int stage, bool acc, int hf) {
        const uint32_t vd = sdesc_lo(opaque(sbase) + L::VM_OFF + stage * L::VM_BYTES, 128 * 128);
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          const int kk = 4 * hf + k4;  // 16 keys
          umma_ts_h(tmem + L::o_col(t), tmem + L::s_col(t) + kk * 8, vd + (kk * 2048 >> 4), L::HI_V, IDESC_PV,
                    (acc || kk > 0) ? 1u : 0u);
        }
      };
      // V as the MMAs read it: loaded (bf16), converted (e4m3)
      constexpr int V_READY = KV8 ? L::B_VM_FULL : L::B_V_FULL, V_USED = KV8 ? L::B_VM_EMPTY : L::B_V_EMPTY;
      int kc = 0, vc = 0, qc0 = 0, qc1 = 0, pc0 = 0, pc1 = 0;
      bool ok = true;
      for (int u = 0; ok; ++u) {
        if (!(ok = wait_item(u))) break;
        const volatile PagedItem* it = item_at(u);
        const int row0 = it->row0, nb0 = it->nb0, nb1 = it->nb1, n_loads = it->n_loads;
        const bool dual = it->dual != 0;
        mbar_arrive(item_done(u));
        if (row0 < 0) break;
        if (n_loads == 0) continue;
        auto nblk = [&](int t) { return t == 0 ? nb0 : nb1; };
        const int n_blocks = max(nb0, nb1);
        if (dual) {
          // tile t takes block 2j + t; the S and the PV MMAs each use their ring in load order
          for (int t = 0; ok && t < 2; ++t) {
            if (nblk(t) == 0) continue;
            ok = mbar_wait(bar(L::B_K_FULL + kc % L::KST), (kc / L::KST) & 1, ctl);
            if (ok && t == 0) ok = mbar_wait(bar(L::B_Q_FULL), qc0 & 1, ctl);
            if (!ok) break;
            tc_fence_after();
            issue_s(t, 0, kc % L::KST);
            umma_commit(bar(L::B_K_EMPTY + kc % L::KST));
            ++kc;
          }
          if (ok && n_loads <= 2) umma_commit(bar(L::B_Q_EMPTY));
          for (int j = 0; ok && j < n_blocks; ++j) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok || j >= nblk(t)) continue;
              const int vs = vc % L::VMST;
              const int ph = ((t == 0 ? pc0 : pc1) + j) & 1;
              ok = mbar_wait(bar(V_READY + vs), (vc / L::VMST) & 1, ctl);
              ok = ok && mbar_wait(bar(L::B_P_FULL + 2 * t), ph, ctl);
              if (!ok) break;
              tc_fence_after();
              issue_pv_half(t, vs, j > 0, 0);
              if (!(ok = mbar_wait(bar(L::B_P_FULL + 2 * t + 1), ph, ctl))) break;
              tc_fence_after();
              issue_pv_half(t, vs, j > 0, 1);
              if (j == nblk(t) - 1) umma_commit(bar(L::B_O_FINAL + t));
              umma_commit(bar(V_USED + vs));
              ++vc;
              if (j + 1 < nblk(t)) {
                const int ks = kc % L::KST;
                if (!(ok = mbar_wait(bar(L::B_K_FULL + ks), (kc / L::KST) & 1, ctl))) break;
                tc_fence_after();
                issue_s(t, 0, ks);
                umma_commit(bar(L::B_K_EMPTY + ks));
                if (2 * (j + 1) + t == n_loads - 1) umma_commit(bar(L::B_Q_EMPTY));  // the piece's last S
                ++kc;
              }
            }
          }
        } else {
          ok = mbar_wait(bar(L::B_K_FULL + kc % L::KST), (kc / L::KST) & 1, ctl);
          for (int t = 0; ok && t < 2; ++t) {
            if (nblk(t) == 0) continue;
            if (!(ok = mbar_wait(bar(L::B_Q_FULL + t), (t == 0 ? qc0 : qc1) & 1, ctl))) break;
            tc_fence_after();
            issue_s(t, t, kc % L::KST);
            if (nblk(t) == 1) umma_commit(bar(L::B_Q_EMPTY + t));
          }
          if (!ok) break;
          umma_commit(bar(L::B_K_EMPTY + kc % L::KST));
          ++kc;
          // per block: PV_0(j), S_0(j+1), PV_1(j), S_1(j+1); MMAs of one thread run in issue order, so PV_t(j) has
          // read P_t(j) before S_t(j+1) overwrites it
          for (int j = 0; ok && j < n_blocks; ++j) {
            const int vs = vc % L::VMST;
            const int ks = kc % L::KST;
            if (!(ok = mbar_wait(bar(V_READY + vs), (vc / L::VMST) & 1, ctl))) break;
            bool k_next = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok || j >= nblk(t)) continue;
              const int ph = ((t == 0 ? pc0 : pc1) + j) & 1;
              if (!(ok = mbar_wait(bar(L::B_P_FULL + 2 * t), ph, ctl))) break;
              tc_fence_after();
              issue_pv_half(t, vs, j > 0, 0);
              if (!(ok = mbar_wait(bar(L::B_P_FULL + 2 * t + 1), ph, ctl))) break;
              tc_fence_after();
              issue_pv_half(t, vs, j > 0, 1);
              if (j == nblk(t) - 1) umma_commit(bar(L::B_O_FINAL + t));
              if (j + 1 < nblk(t)) {
                if (!k_next) {
                  if (!(ok = mbar_wait(bar(L::B_K_FULL + ks), (kc / L::KST) & 1, ctl))) break;
                  k_next = true;
                }
                issue_s(t, t, ks);
                if (j + 2 == nblk(t)) umma_commit(bar(L::B_Q_EMPTY + t));
              }
            }
            if (!ok) break;
            umma_commit(bar(V_USED + vs));
            ++vc;
            if (k_next) {
              umma_commit(bar(L::B_K_EMPTY + ks));
              ++kc;
            }
          }
        }
        pc0 += nb0;
        pc1 += nb1;
        qc0 += nb0 > 0 ? 1 : 0;
        qc1 += (nb1 > 0 && !dual) ? 1 : 0;
      }
      umma_commit(bar(L::B_DRAIN));  // no MMA may still write tensor memory when it is released
      mbar_wait_drain(bar(L::B_DRAIN), 0, 1000000000ull);
    }
  } else if (warp == L::WARP_SCHED) {
    // ===================== scheduler =====================
    if (lane == 0) p.cut[cta] = paged_cut(p, walk, cta);
    for (int u = 0;; ++u) {
      const PagedItem it = paged_walk_next(p, walk, cta);
      if (u >= L::NI && !__all_sync(0xffffffffu, mbar_wait(item_done(u), ((u / L::NI) - 1) & 1, ctl))) break;
      if (lane == 0) {
        volatile int* dst = reinterpret_cast<volatile int*>(sptr + L::ITEM_OFF + (u % L::NI) * sizeof(PagedItem));
        const int* src = reinterpret_cast<const int*>(&it);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(PagedItem) / 4); ++i) dst[i] = src[i];
        mbar_arrive(bar(L::B_ITEM_FULL + u % L::NI));
      }
      if (it.row0 < 0) break;
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
        const int s = n % L::VST, sm = n % L::VMST;
        ok = mbar_wait(bar(L::B_V_FULL + s), (n / L::VST) & 1, ctl);
        if (ok && n >= L::VMST) ok = mbar_wait(bar(L::B_VM_EMPTY + sm), ((n / L::VMST) - 1) & 1, ctl);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const int live = len - (j0 + j) * L::BN;  // rows past the sequence's end become zeros
        convert_block<D>(sptr + L::V_OFF + s * L::KV_BYTES, sptr + L::VM_OFF + sm * L::VM_BYTES, live, tid);
        mbar_arrive_warp(bar(L::B_VM_FULL + sm));
        mbar_arrive_warp(bar(L::B_V_EMPTY + s));
      }
    }
  } else {
    // ===================== softmax warpgroups =====================
    setmaxnreg_inc<L::REG_SOFTMAX>();
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;  // == TMEM lane
    const int rpos = row / p.group, rhead = row - rpos * p.group;  // position in the tile, head of the group
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int sc = 0, oc = 0, xc = 0;  // blocks done, O_FINAL phases of this tile, joins
    int oc1 = 0;                 // O_FINAL phases of tile 1
    bool ok = true;
    for (int u = 0; ok; ++u) {
      if (!(ok = __all_sync(0xffffffffu, wait_item(u)))) break;
      const volatile PagedItem* it = item_at(u);
      if (it->row0 < 0) break;
      const int nb = t == 0 ? it->nb0 : it->nb1;
      const int kb0 = it->j0 * L::BN, len = it->len;
      const bool dual = it->dual != 0;
      const int pos0 = dual ? 0 : t * p.tile_pos;     // the tile's first token in the unit
      const int tile_n = min(it->n_pos - pos0, p.tile_pos);  // its tokens
      const bool valid = rpos < tile_n;
      const bool idle = ((warp & 3) * 32) / p.group >= tile_n;  // every row of this warp is padding
      const int lim = p.causal ? min(it->d0 + pos0 + rpos, len - 1) : len - 1;  // last key this row sees
      const int lim_tile = p.causal ? min(it->d0 + pos0, len - 1) : len - 1;    // last key every row of the tile sees
      float c = p.scale_log2;
      if constexpr (KV8) {
        // Q as two e4m3 terms (this row's), scaled by a power of two so that its largest element is in [128, 256)
        if (nb > 0) {
          if (valid) {
            const long long q_row = static_cast<long long>(it->row0) + pos0 + rpos;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + q_row * p.q_stride +
                                                              static_cast<long long>(it->head * p.group + rhead) * D);
            uint4 w[D / 8];
#pragma unroll
            for (int i = 0; i < D / 8; ++i) w[i] = src[i];
            c = q_row_to_e4m3x2<D, L::ROW_BYTES>(w, row, (dual && t == 1) ? nullptr : sptr + L::Q_OFF + t * L::Q_BYTES,
                                                 L::KV_BYTES, p.scale_log2);
          }
          if (!(dual && t == 1)) {
            fence_proxy_async_smem();
            mbar_arrive_warp(bar(L::B_Q_FULL + t));
          }
        }
      }
      float m_used = -INFINITY;
      float l = 0.f;
      for (int j = 0; j < nb; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::B_S_FULL + t), (sc + j) & 1, ctl));
        if (!ok) break;
        if (idle) {  // publish both halves of P(j): their rows only reach padding rows of O
          mbar_arrive_warp(bar(L::B_P_FULL + 2 * t));
          mbar_arrive_warp(bar(L::B_P_FULL + 2 * t + 1));
          continue;
        }
        tc_fence_after();
        uint32_t sr[128];
        const uint32_t s_addr = tmem + lane_addr + L::s_col(t);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) tmem_ld32(s_addr + ch * 32, sr + ch * 32);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) tmem_ld_wait(sr + ch * 32);
        float* s = reinterpret_cast<float*>(sr);
        const int kbase = kb0 + (dual ? 2 * j + t : j) * L::BN;
        const bool need_mask = kbase + L::BN - 1 > lim_tile;
        if (need_mask) {
          const int lim_c = lim - kbase;
#pragma unroll
          for (int cc = 0; cc < 128; ++cc)
            if (cc > lim_c) s[cc] = -INFINITY;
        }
        const float mx = row_max128(sr);
        const float m_new = fmaxf(m_used, mx * c - L::SHIFT);
        const bool resc = (m_new - m_used) > L::TAU;  // false for NaN (-inf - -inf)
        float alpha = 1.f;
        if (resc) {
          alpha = exp2_mufu(m_used - m_new);
          m_used = m_new;
          l *= alpha;
        }
        const float m_eff = (m_used == -INFINITY) ? 0.f : m_used;
        if (j > 0 && __any_sync(0xffffffffu, resc)) {
          const uint32_t o_addr = tmem + lane_addr + L::o_col(t);
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t orr[32];
            tmem_ld32(o_addr + ch * 32, orr);
            tmem_ld_wait(orr);
#pragma unroll
            for (int i = 0; i < 32; ++i) orr[i] = __float_as_uint(__uint_as_float(orr[i]) * alpha);
            tmem_st32(o_addr + ch * 32, orr);
          }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[32];
          l += exp_weights<KV8>(sr, c, m_eff, pk, hf);
          tmem_st32(s_addr + 32 * hf, pk);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive_warp(bar(L::B_P_FULL + 2 * t + hf));
        }
      }
      sc += nb;
      // ---- epilogue: O / l -> bf16 and lse, or the piece's fp32 rows
      if (ok && nb > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::B_O_FINAL + t), oc & 1, ctl));
        ++oc;
      }
      float* xch = reinterpret_cast<float*>(sptr + L::XCHG_OFF);
      if (dual && t == 1) {
        // tile 1's row statistics go to tile 0, which joins both
        xch[row] = m_used;
        xch[128 + row] = l;
        mbar_arrive_warp(bar(L::B_XCHG));
        // the statistics and O_1 may be overwritten only once tile 0 has read them
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::B_XCHG_READ), xc & 1, ctl));
        ++xc;
      } else if (ok) {
        float m_b = -INFINITY, l_b = 0.f;
        const bool have_b = dual && it->nb1 > 0;
        if (dual) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(L::B_XCHG), xc & 1, ctl));
          if (ok && have_b) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::B_O_FINAL + 1), oc1 & 1, ctl));
          m_b = xch[row];
          l_b = xch[128 + row];
        }
        if (ok) {
          tc_fence_after();
          const float mx = fmaxf(m_used, m_b);
          const float w_a = l > 0.f ? exp2_mufu(m_used - mx) : 0.f;
          const float w_b = l_b > 0.f ? exp2_mufu(m_b - mx) : 0.f;
          const float lsum = l * w_a + l_b * w_b;
          const float inv_l = lsum > 0.f ? 1.f / lsum : 0.f;
          const float c_a = w_a * inv_l, c_b = w_b * inv_l;
          // (the power of two taken out first: the logarithm's error grows with its size)
          const float lse2 = lsum > 0.f ? mx + L::SHIFT + __log2f(lsum * L::DOWN) : -INFINITY;
          const uint32_t oa_addr = tmem + lane_addr + L::o_col(t);
          const uint32_t ob_addr = tmem + lane_addr + L::o_col(1);
          const int slot = it->slot;
          const int h = it->head * p.group + rhead;
          const long long orow = static_cast<long long>(it->row0) + pos0 + rpos;
          const size_t part = static_cast<size_t>(max(slot, 0)) * p.unit_rows + t * 128 + row;
#pragma unroll 1
          for (int ch = 0; ch < D / 16; ++ch) {
            __syncwarp();  // the tensor-memory loads take the whole warp, the stores below only real rows
            uint32_t orr[16], obr[16];
            if (nb > 0) {
              tmem_ld16(oa_addr + ch * 16, orr);
              tmem_ld_wait16(orr);
            }
            if (have_b) {
              tmem_ld16(ob_addr + ch * 16, obr);
              tmem_ld_wait16(obr);
            }
            float* ov = reinterpret_cast<float*>(orr);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float v = (nb > 0 && w_a > 0.f) ? __uint_as_float(orr[i]) * c_a : 0.f;
              if (have_b && w_b > 0.f) v += __uint_as_float(obr[i]) * c_b;
              ov[i] = KV8 ? v * p.v_scale : v;
            }
            if (!valid) continue;
            if (slot >= 0) {
              // (256-bit stores: a row chunk's whole sectors at once)
              float* dst = p.o_part + part * D + ch * 16;
              st_global_v8(dst, orr);
              st_global_v8(dst + 8, orr + 8);
            } else {
              uint32_t pkd[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) pkd[i] = pack_bf16x2(ov[2 * i], ov[2 * i + 1]);
              uint4* d4 = reinterpret_cast<uint4*>(p.o + (orow * p.H_q + h) * D + ch * 16);
              d4[0] = make_uint4(pkd[0], pkd[1], pkd[2], pkd[3]);
              d4[1] = make_uint4(pkd[4], pkd[5], pkd[6], pkd[7]);
            }
          }
          if (valid) {
            if (slot >= 0)
              p.l_part[part] = lse2;
            else
              p.lse[static_cast<long long>(h) * p.n_tokens + orow] =
                  lse2 == -INFINITY ? -INFINITY : lse2 * 0.69314718055994531f;
          }
          if (dual) {
            tc_fence_before();
            mbar_arrive_warp(bar(L::B_XCHG_READ));
            ++xc;
          }
        }
      }
      oc1 += it->nb1 > 0 ? 1 : 0;
      mbar_arrive_warp(item_done(u));
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == L::WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

}  // namespace attn
