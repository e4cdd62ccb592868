// The work list of the paged attention, made on the device by each CTA.
//
// Lengths are read when the call runs, so the host cannot lay the work out.  A
// unit is up to `unit_pos` new tokens of one sequence and the query heads of
// one kv head; its steps are the 128-key blocks its last token sees (one block
// where it sees none: its rows still get their zeros), in the chunk kernel two steps a
// block where both tiles work on it (2.2 to 2.3 us) and one where the tokens fit one
// tile (1.0 to 1.2 us).  All units' steps form one line, ordered by sequence, kv head,
// unit; CTA c takes the c-th of gridDim.x equal stretches (units and stretches have an
// even length where a block may be two steps, so no block is cut).  So the loads are
// even whatever the lengths: a ragged batch, one long sequence, chunks beside single
// tokens.  A unit cut by a stretch's end is
// computed in pieces, each left in the workspace as fp32 rows normalized over
// the piece's keys with their log-sum-exp, and joined by paged_merge_kernel.
// Every CTA finds its stretch by itself from the index arrays (two passes of 32
// sequences at a time): no planning launch and no state between calls.
#pragma once

#include <type_traits>

#include "rotary_kernels.cuh"
#include "sm100_common.cuh"

namespace attn {

struct PagedParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  int n_tokens, H_q, H_kv, group;
  long long q_stride;
  int n_pages, page_size, n_seq;
  int room;                    // keys that a row of the page table has pages for
  int box_rows, box_shift;     // keys of one TMA box: the largest power of two that divides page_size, at most 128
  long long table_stride;
  const int *page_table, *seq_len, *q_start;
  float scale_log2;            // scale * k_scale * log2(e)
  float v_scale;
  int causal;
  int tile_pos, unit_pos;      // tokens of a tile, of a unit
  int unit_rows;               // rows of a unit's partial result
  int step_log2;               // a block of a unit of two tiles is 2^step_log2 steps (units of one tile only: 0)
  int unit_extra;              // steps that stand for a unit's start and end (a multiple of 2^step_log2)
  int min_steps;               // least steps of a CTA's stretch (likewise)
  float* o_part;               // [2 gridDim.x, unit_rows, D]
  float* l_part;               // [2 gridDim.x, unit_rows], base-2 log-sum-exp
  int4* cut;                   // [gridDim.x]: the unit that stretch c starts inside of (paged_cut)
  int* status;
  uint64_t wait_limit_ns;
};

// One piece of a unit, as the roles of a CTA read it from shared memory.
struct PagedItem {
  int row0;     // the unit's first token row; -1: no more work
  int n_pos;    // its tokens
  int d0;       // last key its first token sees (causal)
  int len;      // the sequence's keys
  int head;     // kv head
  int seq;
  int j0;       // first key block of the piece
  int nb0, nb1; // steps of tile 0 and tile 1
  int n_loads;  // key blocks loaded, from j0 on
  int dual;     // one tile holds every token: tile 0 takes the even, tile 1 the odd blocks of the piece
  int slot;     // place of the partial result; -1: the piece is the whole unit
};

struct SeqWork {
  int qs, n_new, len, diag, units;
  bool bad;
};

__device__ __forceinline__ SeqWork seq_work(const PagedParams& p, int b) {
  SeqWork w;
  const int qs = p.q_start[b], qe = p.q_start[b + 1], len = p.seq_len[b];
  w.qs = max(0, min(qs, p.n_tokens));
  w.n_new = max(0, min(qe, p.n_tokens) - w.qs);
  w.len = max(0, min(len, p.room));
  w.bad = w.qs != qs || qe < qs || qe > p.n_tokens || w.len != len;
  w.diag = w.len - w.n_new;
  w.units = w.n_new > p.unit_pos ? (w.n_new + p.unit_pos - 1) / p.unit_pos : (w.n_new > 0 ? 1 : 0);
  return w;
}

// Key blocks that the tokens below position `end` (of the sequence's new ones) see.
__device__ __forceinline__ int blocks_to(const PagedParams& p, const SeqWork& w, int end) {
  const int last = p.causal ? min(min(end, w.n_new) - 1 + w.diag, w.len - 1) : w.len - 1;
  return last < 0 ? 0 : (last >> 7) + 1;
}
// Whether unit u's tokens fit one tile.
__device__ __forceinline__ bool one_tile(const PagedParams& p, const SeqWork& w, int u) {
  return w.n_new - u * p.unit_pos <= p.tile_pos;
}
// How a unit's blocks become steps: a number added for its start and end, and the multiple it is rounded up to.
struct UnitSteps {
  int extra, round;
};
__device__ __forceinline__ int unit_steps(const PagedParams& p, const SeqWork& w, int u, UnitSteps as) {
  const int blocks = max(1, blocks_to(p, w, (u + 1) * p.unit_pos));
  int steps = blocks << p.step_log2;
  if (one_tile(p, w, u)) steps = (blocks + p.step_log2) & ~p.step_log2;  // (even where a block may be two steps)
  steps += as.extra;
  return as.round > 1 ? (steps + as.round - 1) / as.round * as.round : steps;
}

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// Steps of one kv head of each lane's sequence (0 past the last): a lane counts few
// units by itself; the warp counts a long chunk's together.
__device__ __forceinline__ long long head_steps(const PagedParams& p, const SeqWork& w, int lane, UnitSteps as) {
  long long mine = 0;
  const bool many = w.units > 8;
  if (!many)
#pragma unroll 1
    for (int u = 0; u < w.units; ++u) mine += unit_steps(p, w, u, as);
  for (unsigned left = __ballot_sync(0xffffffffu, many); left; left &= left - 1) {
    const int src = __ffs(left) - 1;
    SeqWork o;
    o.n_new = __shfl_sync(0xffffffffu, w.n_new, src);
    o.len = __shfl_sync(0xffffffffu, w.len, src);
    o.diag = __shfl_sync(0xffffffffu, w.diag, src);
    o.units = __shfl_sync(0xffffffffu, w.units, src);
    long long part = 0;
#pragma unroll 1
    for (int u = lane; u < o.units; u += 32) part += unit_steps(p, o, u, as);
    part = warp_sum(part);
    if (lane == src) mine = part;
  }
  return mine;
}

// A CTA's walk along its stretch, kept by the scheduler warp (the same in every lane).
struct PagedWalk {
  long long at, end;  // next step, end of the stretch
  long long per;      // steps of a stretch
  UnitSteps as;
  int b, head, u, step;  // where `at` is: sequence, kv head, unit, step of the unit
  SeqWork w;          // sequence b's
};

// x / d for operands that hardly ever need 64 bits (a 64-bit division is some hundred instructions).
__device__ __forceinline__ long long quotient(long long x, long long d) {
  if (((x | d) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(d);
  return x / d;
}

__device__ __forceinline__ void paged_walk_start(const PagedParams& p, PagedWalk& k, int cta, int n_ctas, int lane) {
  long long total = 0, units = 0;
  SeqWork w{};  // the lane's sequence of the 32 read last
  auto read = [&](int b0) {
    w = SeqWork{};
    if (b0 + lane < p.n_seq) w = seq_work(p, b0 + lane);
  };
  k.as = UnitSteps{0, 1};
  for (int b0 = 0; b0 < p.n_seq; b0 += 32) {
    read(b0);
    if (w.bad && cta == 0) atomicExch(p.status, kDevBadIndex);
    total += warp_sum(head_steps(p, w, lane, k.as)) * p.H_kv;
    units += warp_sum(w.units) * p.H_kv;
  }
  k.per = max(quotient(total + n_ctas - 1, n_ctas), static_cast<long long>(p.min_steps));
  k.per = (k.per + p.step_log2) & ~static_cast<long long>(p.step_log2);
  // A second piece costs a CTA about as much as kPieceBlocks blocks.  Few units: if stretches that much longer at
  // most can hold one piece each -- units rounded up to whole stretches -- they do (one sequence of 8000 keys, 8 kv
  // heads: 14.1 us, else 18.1).  Many: a unit's start and end count as steps of their own (64 sequences of up to 1000
  // keys: 49 us without, 38 with four).
  constexpr int kPieceBlocks = 3;
  bool whole = false;
  if (p.n_seq <= 32 && units <= n_ctas && k.per <= 16 << p.step_log2) {
    for (int i = 0; i <= kPieceBlocks && !whole; ++i) {
      const long long per = k.per + (static_cast<long long>(i) << p.step_log2);
      if (per > (1 << 28)) break;
      const UnitSteps as{0, static_cast<int>(per)};
      const long long t = warp_sum(head_steps(p, w, lane, as)) * p.H_kv;
      if (t <= per * n_ctas) {
        whole = true;
        k.as = as;
        k.per = per;
        total = t;
      }
    }
  }
  if (!whole && total >= static_cast<long long>(n_ctas) * p.unit_extra) {
    k.as.extra = p.unit_extra;
    total += units * p.unit_extra;
    k.per = quotient(total + n_ctas - 1, n_ctas);
    k.per = (k.per + p.step_log2) & ~static_cast<long long>(p.step_log2);
  }
  k.at = min(k.per * cta, total);
  k.end = min(k.at + k.per, total);
  k.b = k.head = k.u = k.step = 0;
  if (k.at >= k.end) return;
  long long before = 0;      // steps of the sequences before b0
  long long per_head, upto;  // a head's steps of the lane's sequence, and those of the lanes up to it (inclusive)
  int b0 = 0;
  while (true) {
    if (p.n_seq > 32) read(b0);  // (32 sequences or fewer are still held)
    per_head = head_steps(p, w, lane, k.as);
    upto = per_head * p.H_kv;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += x;
    }
    if (__any_sync(0xffffffffu, before + upto > k.at) || b0 + 32 >= p.n_seq) break;
    before += __shfl_sync(0xffffffffu, upto, 31);
    b0 += 32;
  }
  const unsigned past = __ballot_sync(0xffffffffu, before + upto > k.at);
  // Lengths that change while the call runs may make this reading differ from the one that gave `total`: such a
  // stretch is left out, so that no place outside the tensors follows from it.
  bool torn = past == 0;
  const int src = past == 0 ? 0 : __ffs(past) - 1;
  const long long ph = max(1ll, __shfl_sync(0xffffffffu, per_head, src));
  long long r = k.at - before - (__shfl_sync(0xffffffffu, upto, src) - ph * p.H_kv);
  k.b = b0 + src;
  const long long head = quotient(r, ph);
  torn |= head >= p.H_kv;
  k.head = torn ? 0 : static_cast<int>(head);
  r -= ph * k.head;
  k.w.qs = __shfl_sync(0xffffffffu, w.qs, src);
  k.w.n_new = __shfl_sync(0xffffffffu, w.n_new, src);
  k.w.len = __shfl_sync(0xffffffffu, w.len, src);
  k.w.diag = __shfl_sync(0xffffffffu, w.diag, src);
  k.w.units = __shfl_sync(0xffffffffu, w.units, src);
  // the unit that holds step r of the head: 32 units at a time
  for (int u0 = 0;; u0 += 32) {
    const int steps = u0 + lane < k.w.units ? unit_steps(p, k.w, u0 + lane, k.as) : 0;
    int sum = steps;
    if (k.w.units > 1) {
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += x;
      }
    }
    const unsigned in = __ballot_sync(0xffffffffu, sum > r);
    if (in == 0 && u0 + 32 < k.w.units) {
      r -= __shfl_sync(0xffffffffu, sum, 31);
      continue;
    }
    torn |= in == 0;
    const int lu = in == 0 ? 0 : __ffs(in) - 1;
    k.u = u0 + lu;
    k.step = static_cast<int>(r - (__shfl_sync(0xffffffffu, sum, lu) - __shfl_sync(0xffffffffu, steps, lu)));
    break;
  }
  if (torn) {
    if (lane == 0) atomicExch(p.status, kDevBadIndex);
    k.end = k.at;
  }
}

// The next piece of the stretch (row0 = -1 when it is used up).
__device__ __forceinline__ PagedItem paged_walk_next(const PagedParams& p, PagedWalk& k, int cta) {
  PagedItem it{};
  it.row0 = -1;
  it.slot = -1;
  if (k.at >= k.end) return it;
  const int steps = unit_steps(p, k.w, k.u, k.as);
  const int take = static_cast<int>(min(static_cast<long long>(steps - k.step), k.end - k.at));
  it.dual = one_tile(p, k.w, k.u);
  const int scale = it.dual ? 0 : p.step_log2;  // log2 of the steps of a block
  const int q0 = k.u * p.unit_pos;
  it.row0 = k.w.qs + q0;
  it.n_pos = min(p.unit_pos, k.w.n_new - q0);
  it.d0 = q0 + k.w.diag;
  it.len = k.w.len;
  it.head = k.head;
  it.seq = k.b;
  it.j0 = k.step >> scale;
  const int j1 = (k.step + take) >> scale;
  const int all = min(blocks_to(p, k.w, q0 + p.unit_pos), j1);
  if (it.dual) {
    const int n = max(all - it.j0, 0);
    it.nb0 = (n + 1) / 2;
    it.nb1 = n / 2;
    it.n_loads = n;
  } else {
    it.nb0 = max(min(blocks_to(p, k.w, q0 + p.tile_pos), j1) - it.j0, 0);
    it.nb1 = max(all - it.j0, 0);
    it.n_loads = max(it.nb0, it.nb1);
  }
  if (take < steps) it.slot = 2 * cta + (k.step == 0 ? 1 : 0);
  // advance
  k.at += take;
  k.step += take;
  if (k.step == steps) {
    k.step = 0;
    if (++k.u == k.w.units) {
      k.u = 0;
      if (++k.head == p.H_kv) {
        k.head = 0;
        if (k.at < k.end) {
          do {
            ++k.b;
            k.w = seq_work(p, min(k.b, p.n_seq - 1));
          } while (k.w.units == 0 && k.b < p.n_seq - 1);
        }
      }
    }
  }
  return it;
}

// The unit that a stretch starts inside of, for the merge: its first token row, tokens, kv head and
// last CTA, or row0 = -1 where the stretch starts a unit, is empty, or is not
// the first one to start inside the unit (an earlier one merges it).
__device__ __forceinline__ int4 paged_cut(const PagedParams& p, const PagedWalk& k, int cta) {
  if (k.at >= k.end || k.step == 0) return make_int4(-1, 0, 0, 0);
  const long long start = k.at - k.step;
  if (start < (cta - 1) * k.per) return make_int4(-1, 0, 0, 0);
  const int q0 = k.u * p.unit_pos;
  const long long last = quotient(start + unit_steps(p, k.w, k.u, k.as) - 1, k.per);
  const long long end = static_cast<long long>(gridDim.x) - 1;  // (`last` is beyond only where lengths change meanwhile)
  return make_int4(k.w.qs + q0, min(p.unit_pos, k.w.n_new - q0), k.head, static_cast<int>(min(last, end)));
}

// Joins the pieces of the units that were cut.  Block (c, y): rows 8 y .. 8 y + 7 of the unit
// that stretch c + 1 starts inside of: pieces 2 c + 1 and 2 c', c' = c + 1 .. last.
//   lse = log2 sum_s 2^(lse_s),   O = sum_s 2^(lse_s - lse) O_s
// It is a chain of reads (the record, then the pieces), so their latency counts: a warp asks for the pieces of
// its rows, W at a time each, together (four rows a warp for the chunk kernel's 256-row units: one row
// a warp took 30 us for 147 cut units, in eight waves of blocks).  More than 2 W pieces (a long sequence over
// many CTAs) are shared out among the block's eight warps, row by row.  The order of the sums depends on the
// lengths only.
template <int D, int ROWS, int W>
struct MergeRows {
  static constexpr int PER = D / 32;
  using Vec = typename std::conditional<PER == 4, float4, float2>::type;
  float m[ROWS], sum[ROWS], acc[ROWS][PER];

  __device__ __forceinline__ MergeRows() {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      m[i] = -INFINITY;
      sum[i] = 0.f;
#pragma unroll
      for (int x = 0; x < PER; ++x) acc[i][x] = 0.f;
    }
  }

  // adds pieces first, first + step, ... below n (at most W of them) of rows r, r + 1, ...
  template <typename Place>
  __device__ __forceinline__ void add(const PagedParams& p, int r, int lane, int first, int step, int n, Place place) {
    float l[ROWS][W];
    Vec v[ROWS][W];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int s = first + j * step;
        l[i][j] = -INFINITY;
        if (s < n) {
          const size_t at = static_cast<size_t>(place(s)) * p.unit_rows + r + i;
          l[i][j] = p.l_part[at];
          v[i][j] = *reinterpret_cast<const Vec*>(p.o_part + at * D + lane * PER);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      float top = m[i];
#pragma unroll
      for (int j = 0; j < W; ++j) top = fmaxf(top, l[i][j]);
      if (top == -INFINITY) continue;  // no piece so far saw a key
      const float old = m[i] == -INFINITY ? 0.f : exp2_mufu(m[i] - top);
      sum[i] *= old;
#pragma unroll
      for (int x = 0; x < PER; ++x) acc[i][x] *= old;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if (l[i][j] == -INFINITY) continue;
        const float w = exp2_mufu(l[i][j] - top);
        sum[i] += w;
#pragma unroll
        for (int x = 0; x < PER; ++x) acc[i][x] += w * reinterpret_cast<const float*>(&v[i][j])[x];
      }
      m[i] = top;
    }
  }
};

// Where row r of a unit is (tile rows are position-major): its token and head; false for padding.
template <int TILE_ROWS>
__device__ __forceinline__ bool unit_row(const PagedParams& p, int r, int n_pos, int& pos, int& head) {
  const int rr = r % TILE_ROWS;
  pos = rr / p.group;
  head = rr - pos * p.group;
  const bool real = pos < p.tile_pos;
  pos += r / TILE_ROWS * p.tile_pos;
  return real && pos < n_pos;
}

__host__ __device__ constexpr int merge_rows(int tile_rows) { return tile_rows == 128 ? 4 : 1; }  // rows of a warp

template <int D, int TILE_ROWS>
__global__ void __launch_bounds__(256) paged_merge_kernel(const PagedParams p) {
  constexpr int PER = D / 32, ROWS = merge_rows(TILE_ROWS), W = ROWS == 1 ? 8 : 4;
  __shared__ __align__(16) float red_o[8][D];
  __shared__ float red_m[8], red_l[8];
  // a programmatic dependent of the attention kernel: waits for its results
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x + 1;
  const int4 cut = p.cut[c];
  if (cut.x < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = cut.w - c + 2;  // pieces
  auto place = [&](int s) { return s == 0 ? 2 * c - 1 : 2 * (c + s - 1); };
  auto finish = [&](int r, float m, float sum, const float* acc) {
    int pos, head;
    if (!unit_row<TILE_ROWS>(p, r, cut.y, pos, head)) return;
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int h = cut.z * p.group + head;
    const long long at = static_cast<long long>(cut.x) + pos;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (at * p.H_q + h) * D + lane * PER);
#pragma unroll
    for (int x = 0; x < PER / 2; ++x) dst[x] = pack_bf16x2(acc[2 * x] * inv, acc[2 * x + 1] * inv);
    if (lane == 0)
      p.lse[static_cast<long long>(h) * p.n_tokens + at] = sum > 0.f ? (m + log2f(sum)) * 0.69314718055994531f : -INFINITY;
  };
  const int r0 = blockIdx.y * 8 * ROWS;
  int pos, head;
  if (n <= 2 * W) {
    const int r = r0 + warp * ROWS;
    bool any = false;  // (padding rows hold no partial result: they are read, and dropped)
#pragma unroll
    for (int i = 0; i < ROWS; ++i) any |= unit_row<TILE_ROWS>(p, r + i, cut.y, pos, head);
    if (!any) return;
    MergeRows<D, ROWS, W> rows;
    rows.add(p, r, lane, 0, 1, n, place);
    if (n > W) rows.add(p, r, lane, W, 1, n, place);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) finish(r + i, rows.m[i], rows.sum[i], rows.acc[i]);
    return;
  }
  for (int r = r0; r < r0 + 8 * ROWS; ++r) {
    if (!unit_row<TILE_ROWS>(p, r, cut.y, pos, head)) continue;  // (the same for the whole block)
    MergeRows<D, 1, 4> row;
    for (int s = warp; s < n; s += 32) row.add(p, r, lane, s, 8, n, place);
#pragma unroll
    for (int x = 0; x < PER; ++x) red_o[warp][lane * PER + x] = row.acc[0][x];
    if (lane == 0) {
      red_m[warp] = row.m[0];
      red_l[warp] = row.sum[0];
    }
    __syncthreads();
    if (warp == 0) {
      float top = red_m[0], sum = 0.f, acc[PER];
#pragma unroll
      for (int g = 1; g < 8; ++g) top = fmaxf(top, red_m[g]);
#pragma unroll
      for (int x = 0; x < PER; ++x) acc[x] = 0.f;
      if (top > -INFINITY) {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float w = exp2_mufu(red_m[g] - top);
          sum += w * red_l[g];
#pragma unroll
          for (int x = 0; x < PER; ++x) acc[x] += w * red_o[g][lane * PER + x];
        }
      }
      finish(r, top, sum, acc);
    }
    __syncthreads();
  }
}

}  // namespace attn
