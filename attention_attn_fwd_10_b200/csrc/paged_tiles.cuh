// Loading a paged cache's 128-key blocks, turning e4m3 values into fp16, and e4m3 pairs: shared by the paged
// attention kernels.
#pragma once

#include "paged_plan.cuh"
#include "sm100_common.cuh"

namespace attn {

// True in one lane of a converged warp.  A branch on it, unlike one on the lane's number, keeps what it issues in
// uniform registers: the MMAs of a block leave sooner.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// mbar_wait in fewer instructions: where many warps of different roles wait inside loops, the copies of its code
// fill the instruction cache.
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, const WaitCtl& ctl) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t it = 0; !mbar_try_wait(bar, parity); ++it) {
    if ((it & 15u) != 0) continue;
    if (*ctl.abort_flag) return false;
    const uint64_t now = globaltimer_ns();
    if (it == 0) t0 = now;
    if (now - t0 > ctl.limit_ns) {
      *ctl.abort_flag = 1;
      atomicExch(ctl.status, kDevWaitTimeout);
      return false;
    }
  }
  return true;
}

// x as a sum of two e4m3 values, pairs of them in the low 16 bits (the first value in the low byte):
//   hi = e4m3(x), lo = e4m3((x - hi) * factor).
// fp16 holds the remainder exactly: hi takes the leading four bits of at most eleven.
template <bool TIMES16>
__device__ __forceinline__ void split_e4m3x2_any(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  uint32_t h2, b2;
  uint16_t h, l;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h2) : "f"(x1), "f"(x0));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(h2));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b2) : "h"(h));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h2) : "r"(h2), "r"(b2));
  if (TIMES16) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h2) : "r"(h2), "r"(0x4c004c00u));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(h2));
  hi = h;
  lo = l;
}
__device__ __forceinline__ void split_e4m3x2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  split_e4m3x2_any<false>(x0, x1, hi, lo);
}
__device__ __forceinline__ void split16_e4m3x2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  split_e4m3x2_any<true>(x0, x1, hi, lo);
}

// A query row's power of two for its e4m3 terms: `most` is the largest element's exponent field as it sits in a bf16
// (bits 7 .. 14); the power (as an fp32 exponent field) puts that element into [128, 256).  At most 2^73: rows
// below 2^-66 have scores of 0 all the same, and the factor taken back out stays a normal number.
__device__ __forceinline__ uint32_t q_power(uint32_t most) {
  return static_cast<uint32_t>(min(261 - static_cast<int>(most >> 7), 200));
}
__device__ __forceinline__ float q_factor(float scale_log2, uint32_t power) {
  return fmaxf(scale_log2 * __uint_as_float((254u - power) << 23), 1.17549435e-38f);
}

// A producer warp's page numbers: lane l holds the page of box base + l of the current sequence.
struct PageWindow {
  int base;  // first box held; -1: none
  int page, slot;  // the lane's box: its page, its first slot there
};

// The page of box `box` of sequence `seq` (all lanes call with their own box, within one window of 32 boxes that
// starts at a multiple of 32); -1 past the table or for an entry outside the cache (reported).
__device__ __forceinline__ void window_load(const PagedParams& p, PageWindow& w, int seq, int base, int n_boxes, int lane) {
  w.base = base;
  w.page = -1;
  w.slot = 0;
  const int box = base + lane;
  if (box < n_boxes) {
    const int j = (box << p.box_shift) / p.page_size;
    w.slot = (box << p.box_shift) - j * p.page_size;
    const int page = p.page_table[seq * p.table_stride + j];
    if (page >= 0 && page < p.n_pages)
      w.page = page;
    else
      atomicExch(p.status, kDevBadIndex);
  }
}

// Loads block `blk` (128 keys) of a sequence's cache into shared memory at `dst`: box i of the block by lane i of
// the warp (lane i + boxes: its second 128-byte column); `full` completes when all of them have landed.
// NBOX columns of ROW_BYTES; boxes wholly past the sequence's end are left out.  A warp issues a TMA instruction
// in about 100 clk (lane by lane or in a loop of one lane alike), so pages of 16 keys, 16 boxes a tile, take 1.6k
// clk a tile: K and V have a warp each.
template <int NBOX, int ROW_BYTES>
__device__ __forceinline__ void load_block(const PagedParams& p, const CUtensorMap* map, uint32_t dst, uint32_t full,
                                           PageWindow& win, int seq, int head, int len, int blk, int lane) {
  const int boxes_log2 = 7 - p.box_shift;  // of a block
  const int n_boxes = (len + p.box_rows - 1) >> p.box_shift;
  const int first = blk << boxes_log2;
  if (win.base != (first & ~31)) window_load(p, win, seq, first & ~31, n_boxes, lane);
  const int n = min(1 << boxes_log2, n_boxes - first);
  if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(n) * NBOX * p.box_rows * ROW_BYTES);
  __syncwarp();
  const int i = lane & ((1 << boxes_log2) - 1), x = lane >> boxes_log2;
  const int page = __shfl_sync(0xffffffffu, win.page, (first + i) & 31);
  const int slot = __shfl_sync(0xffffffffu, win.slot, (first + i) & 31);
  if (i < n && x < NBOX)
    tma_load_4d(dst + x * 128 * ROW_BYTES + i * p.box_rows * ROW_BYTES, map, full, x * 64, head, slot, page);
}

// Writes zeros over the rows of a landed block that lie past the sequence's end (`live` keys are the sequence's), by
// the whole warp, visible to the tensor cores.  Whole rows: the swizzle moves 16-byte chunks within a row only.
template <int NBOX, int ROW_BYTES>
__device__ __forceinline__ void zero_tail(uint8_t* tile, int live, int lane) {
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int x = 0; x < NBOX; ++x)
    for (int c = live * (ROW_BYTES / 16) + lane; c < 128 * ROW_BYTES / 16; c += 32)
      *reinterpret_cast<uint4*>(tile + x * 128 * ROW_BYTES + c * 16) = zero;
  fence_proxy_async_smem();
  __syncwarp();
}

// Turns a landed e4m3 block of V into fp16 (exactly), by 128 threads: src as loaded, one column of D-byte rows;
// dst D / 64 columns of 128-byte rows, swizzled as the MMAs read them.  Rows past the sequence's end (`live` keys are
// its own) become zeros.  Visible to the tensor cores.
//
// A thread takes 16 dims of a key at a time: a 16-byte chunk in, two out.  Eight lanes that access shared memory
// together have four chunks of two keys.  D = 128: keys k and k ^ 5, whose swizzles set the chunks apart both as read
// (bit 2 of the key) and as written (bit 0); one key's eight chunks would meet in the banks as they are written, four to
// each of the two columns.  A thread's keys are 32 apart, so that all its swizzles are the same and every address is a
// constant off four bases: the warps of this loop share the instruction cache with four other roles.
template <int D>
__device__ __forceinline__ void convert_block(const uint8_t* src, uint8_t* dst, int live, int tid) {
  const int key0 = D == 128 ? tid / 32 * 8 + ((tid >> 3 & 3) ^ ((tid >> 2 & 1) * 5)) : tid / 4, c = tid & 3;
  const int sw = D == 128 ? (key0 & 7) : ((key0 >> 1) & 3);
  const uint8_t* const in = src + key0 * D + ((c ^ sw) * 16);
  const uint8_t* const in4 = src + key0 * D + (((c + 4) ^ sw) * 16);  // D = 128: chunk c + 4
  uint8_t* const out0 = dst + key0 * 128 + (((2 * c) ^ (key0 & 7)) * 16);
  uint8_t* const out1 = dst + key0 * 128 + (((2 * c + 1) ^ (key0 & 7)) * 16);
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int col = 0; col < D / 64; ++col) {
      const uint4 x = *reinterpret_cast<const uint4*>((col == 0 ? in : in4) + i * 32 * D);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t y[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y[2 * k]) : "h"(static_cast<uint16_t>(w[k])));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y[2 * k + 1]) : "h"(static_cast<uint16_t>(w[k] >> 16)));
      }
      const int at = col * (128 * 128) + i * 32 * 128;
      *reinterpret_cast<uint4*>(out0 + at) = make_uint4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint4*>(out1 + at) = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
  if (live < 128) {  // the thread's own rows past the end
#pragma unroll 1
    for (int i = 0; i < 4 * (D / 64); ++i) {
      const int at = i / 4 * (128 * 128) + (i & 3) * 32 * 128;
      if (key0 + (i & 3) * 32 < live) continue;
      *reinterpret_cast<uint4*>(out0 + at) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(out1 + at) = make_uint4(0, 0, 0, 0);
    }
  }
  fence_proxy_async_smem();
}

// Two weights as a pair of fp16.
__device__ __forceinline__ uint32_t pack_f16x2(float x0, float x1) {
  uint32_t w;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(x1), "f"(x0));
  return w;
}

}  // namespace attn
