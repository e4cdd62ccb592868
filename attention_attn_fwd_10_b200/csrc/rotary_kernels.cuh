// Rotary positions and the paged cache's append: one kernel.
//
// A token's row is a list of heads -- q's, then k's, then (append) v's -- and a
// CTA takes `tok` tokens x `hpc` heads of that list.  Per token it needs the
// angles a_i = position * inv_freq[i]; they are shared by all heads, so the CTA
// computes cos and sin once per (token, frequency) into shared memory.  The
// product position * inv_freq / 2 pi is formed in 64 bits and reduced to
// [-1/2, 1/2] turns there (at position 10^6 an fp32 product has lost 6 of 24
// bits of the turn), then cospi/sinpi run in fp32 on the remainder.
//
// The work is bytes: each element is read and written once.  An item is two
// chunks of VEC elements (16 bytes each for VEC = 8) that hold VEC whole pairs:
// chunks (i, i + n_freq / VEC) of a head in the half layout, (2i, 2i + 1) in the
// interleaved one.  A thread holds ITEMS = 4 items, all loads issued before the
// angles are computed, so their latency overlaps; four CTAs of 256 threads per SM.  It is
// also near the issue rate (68 % with a division per item and access), so a thread's items share one.
// q and k of 2 x 8192 tokens x 16 heads x 128, 269 MB: 44.2 us, 6.1 TB/s, 93 % of the measured copy rate
// (3, 5, 6 CTAs per SM: 45.6, 50.2, 56.9 us; 2 items per thread: 50.6 us; 8: 56.7 us).
#pragma once

#include <cuda_fp8.h>

#include "sm100_common.cuh"

namespace attn {

constexpr int kDevBadIndex = 7;  // matches ATTN_ERR_BAD_INDEX

struct RotaryParams {
  const __nv_bfloat16* src[3];  // q, k, v (q, v may be null: no heads)
  void* dst[3];                 // rope: q_out, k_out; append: q_out, cache k, cache v
  long long src_stride[3];      // elements between tokens
  long long dst_stride[3];      // (dense outputs)
  int heads[3];
  int n_heads;                  // sum of heads
  int hpc, tok;                 // heads and tokens of a CTA
  long long n_tokens;
  long long period;             // rope with positions = nullptr: position = token % period
  // rotation
  const float* inv_freq;
  const int* positions;         // [n_axes, n_tokens] or nullptr
  int n_freq;                   // 0: no rotation
  int sec_end[4];               // frequencies below sec_end[a] (and not below sec_end[a - 1]) are axis a's
  float sign;                   // -1: inverse
  // paged cache (append)
  int n_pages, page_size, max_pages, n_seq;
  long long page_stride, token_stride, head_stride, table_stride;
  float scale[3];               // e4m3: value = stored * scale
  const int* page_table;
  const int* seq_len;
  const int* q_start;
  int* status;
};

// The sequence that owns token t: the number of starts at or below t, less one,
// found by the whole warp 32 ways at a time (one load per level: 32 levels-1
// sequences, 1024 at two).  Returns -1 where no sequence owns t.
__device__ __forceinline__ int owner_of(long long t, const int* q_start, int n_seq, int lane) {
  int lo = 0, n = n_seq + 1;  // the last start at or below t is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool below = lane * step < n && q_start[i] <= t;
    const unsigned m = __ballot_sync(0xffffffffu, below);
    const int c = __popc(m);
    if (c == 0) return -1;
    const int first = (c - 1) * step;
    n = min(step, n - first);
    lo += first;
  }
  const int b = lo;
  if (b >= n_seq) return -1;
  return q_start[b] <= t && t < q_start[b + 1] ? b : -1;
}

template <int VEC>
struct RotVec;
template <>
struct RotVec<8> {
  using T = uint4;
  static constexpr int W = 4;
};
template <>
struct RotVec<4> {
  using T = uint2;
  static constexpr int W = 2;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// x / scale as e4m3 (round to nearest even, saturating), VEC values.
template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t* dst, const float* x, float scale) {
  uint32_t w[VEC / 4];
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i)
    w[i] = pack_e4m3x4(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale), __fdiv_rn(x[4 * i + 2], scale),
                       __fdiv_rn(x[4 * i + 3], scale));
  if constexpr (VEC == 8)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = w[0];
}

template <int VEC>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* dst, const float* x) {
  typename RotVec<VEC>::T o;
  uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<typename RotVec<VEC>::T*>(dst) = o;
}

constexpr int kRotThreads = 256;
constexpr int kRotMaxTok = 8;    // tokens of a CTA: one warp looks each one's sequence up

template <int D, int VEC, int ITEMS, bool INTERLEAVED, bool PAGED, bool E4M3>
__global__ void __launch_bounds__(kRotThreads, 4) rotary_kernel(const RotaryParams p) {
  using V = typename RotVec<VEC>::T;
  constexpr int PER_HEAD = D / (2 * VEC);  // items of a head
  __shared__ __align__(16) float s_cos[kRotMaxTok * D / 2], s_sin[kRotMaxTok * D / 2];
  __shared__ long long s_slot[kRotMaxTok];  // append: the token's place in the cache, -1 = none
  __shared__ int s_key[kRotMaxTok];         // append: its key's index in the sequence
  __shared__ int s_owned[kRotMaxTok];       // append: some sequence owns the token
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long t0 = static_cast<long long>(blockIdx.x) * p.tok;
  const int nt = static_cast<int>(min(static_cast<long long>(p.tok), p.n_tokens - t0));
  const int h0 = blockIdx.y * p.hpc;
  const int nh = min(p.hpc, p.n_heads - h0);
  const int fv = p.n_freq / VEC;  // rotated items of a head

  // Item u of a thread: the same chunks ca, cb of (token, head list entry) number pair0 + u STEP of the CTA, so that
  // one division places all of them.
  constexpr int STEP = kRotThreads / PER_HEAD;
  static_assert(kRotThreads % PER_HEAD == 0, "a thread's items have the same chunks");
  const int i = tid % PER_HEAD, pair0 = tid / PER_HEAD;
  const int n_pairs = nt * nh;
  int ca, cb;
  if (INTERLEAVED || i >= fv) {
    ca = 2 * i;  // (past the rotated ones, half layout: 2 fv + 2 (i - fv))
    cb = ca + 1;
  } else {
    ca = i;
    cb = i + fv;
  }
  struct Place {
    int tau, h;            // token of the CTA, entry of its head range
    int which, head;       // q, k or v, and the head there
  };
  auto settle = [&](Place& w) {
    while (w.h >= nh) {
      w.h -= nh;
      ++w.tau;
    }
    w.which = 0;
    w.head = h0 + w.h;
    if (w.head >= p.heads[0]) {
      w.head -= p.heads[0];
      w.which = 1;
      if (w.head >= p.heads[1]) {
        w.head -= p.heads[1];
        w.which = 2;
      }
    }
  };
  Place first;
  first.tau = pair0 / nh;
  first.h = pair0 - first.tau * nh;

  V xa[ITEMS], xb[ITEMS];
  {
    Place w = first;
#pragma unroll
    for (int u = 0; u < ITEMS; ++u, w.h += STEP) {
      if (pair0 + u * STEP >= n_pairs) break;
      settle(w);
      const __nv_bfloat16* src = p.src[w.which] + (t0 + w.tau) * p.src_stride[w.which] + w.head * D;
      xa[u] = *reinterpret_cast<const V*>(src + ca * VEC);
      xb[u] = *reinterpret_cast<const V*>(src + cb * VEC);
    }
  }

  if (PAGED) {
    // Ranges and lengths, owned by a token or not (the look-up below meets only those that are), by the grid's
    // threads from each CTA's last warp on: the first ones have tokens to look up.
    if (blockIdx.y == 0) {
      for (long long b = static_cast<long long>(blockIdx.x) * kRotThreads + (kRotThreads - 1 - tid); b < p.n_seq;
           b += static_cast<long long>(gridDim.x) * kRotThreads) {
        const int start = p.q_start[b], end = p.q_start[b + 1], len = p.seq_len[b];
        if (start < 0 || end < start || end > p.n_tokens || len < 0 ||
            len > static_cast<long long>(p.max_pages) * p.page_size)
          atomicExch(p.status, kDevBadIndex);
      }
    }
    if (warp < nt) {
      const long long t = t0 + warp;
      const int b = owner_of(t, p.q_start, p.n_seq, lane);
      if (lane == 0) {
        long long slot = -1;
        int key = 0;
        if (b >= 0) {
          const int q_end = p.q_start[b + 1];
          const long long key_ll = static_cast<long long>(p.seq_len[b]) - (q_end - t);
          bool ok = p.q_start[b] >= 0 && q_end <= p.n_tokens && key_ll >= 0 &&
                    key_ll < static_cast<long long>(p.max_pages) * p.page_size;
          if (ok) {
            key = static_cast<int>(key_ll);
            const int j = key / p.page_size;
            const int page = p.page_table[b * p.table_stride + j];
            ok = page >= 0 && page < p.n_pages;
            if (ok) slot = page * p.page_stride + (key - j * p.page_size) * p.token_stride;
          }
          if (!ok) atomicExch(p.status, kDevBadIndex);
        }
        s_slot[warp] = slot;
        s_key[warp] = key;
        s_owned[warp] = b >= 0;
      }
    }
    __syncthreads();
  }
  if (p.n_freq > 0) {
    for (int e = tid; e < nt * p.n_freq; e += kRotThreads) {
      const int tau = e / p.n_freq, f = e - tau * p.n_freq;
      const int axis = (f >= p.sec_end[0]) + (f >= p.sec_end[1]) + (f >= p.sec_end[2]);
      int pos;
      if (p.positions != nullptr)
        pos = p.positions[axis * p.n_tokens + t0 + tau];
      else
        pos = PAGED ? s_key[tau] : static_cast<int>((t0 + tau) % p.period);
      double turns = static_cast<double>(pos) * static_cast<double>(p.inv_freq[f]) * 0.15915494309189533577;
      turns -= rint(turns);
      float s, c;
      sincospif(2.f * static_cast<float>(turns), &s, &c);
      s_cos[tau * p.n_freq + f] = c;
      s_sin[tau * p.n_freq + f] = s * p.sign;
    }
    __syncthreads();
  }

  Place w = first;
#pragma unroll
  for (int u = 0; u < ITEMS; ++u, w.h += STEP) {
    if (pair0 + u * STEP >= n_pairs) break;
    settle(w);
    if (PAGED && !s_owned[w.tau]) continue;
    const uint32_t* wa = reinterpret_cast<const uint32_t*>(&xa[u]);
    const uint32_t* wb = reinterpret_cast<const uint32_t*>(&xb[u]);
    float a[VEC], b[VEC];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      a[2 * i] = bf_lo(wa[i]);
      a[2 * i + 1] = bf_hi(wa[i]);
      b[2 * i] = bf_lo(wb[i]);
      b[2 * i + 1] = bf_hi(wb[i]);
    }
    if (w.which < 2 && i < fv) {
      const float* cs = s_cos + w.tau * p.n_freq + i * VEC;
      const float* sn = s_sin + w.tau * p.n_freq + i * VEC;
      float c[VEC], s[VEC];
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        reinterpret_cast<float4*>(c)[i] = reinterpret_cast<const float4*>(cs)[i];
        reinterpret_cast<float4*>(s)[i] = reinterpret_cast<const float4*>(sn)[i];
      }
      if (INTERLEAVED) {
        // pair j: elements 2j, 2j + 1 of the item's 2 VEC consecutive ones
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          const float x0 = a[2 * j], x1 = a[2 * j + 1], y0 = b[2 * j], y1 = b[2 * j + 1];
          a[2 * j] = x0 * c[j] - x1 * s[j];
          a[2 * j + 1] = x1 * c[j] + x0 * s[j];
          b[2 * j] = y0 * c[VEC / 2 + j] - y1 * s[VEC / 2 + j];
          b[2 * j + 1] = y1 * c[VEC / 2 + j] + y0 * s[VEC / 2 + j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float x = a[j], y = b[j];
          a[j] = x * c[j] - y * s[j];
          b[j] = y * c[j] + x * s[j];
        }
      }
    }
    if (!PAGED || w.which == 0) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.dst[w.which]) + (t0 + w.tau) * p.dst_stride[w.which] + w.head * D;
      store_bf16<VEC>(dst + ca * VEC, a);
      store_bf16<VEC>(dst + cb * VEC, b);
    } else {
      const long long slot = s_slot[w.tau];
      if (slot < 0) continue;
      const long long at = slot + w.head * p.head_stride;
      if constexpr (E4M3) {
        uint8_t* dst = static_cast<uint8_t*>(p.dst[w.which]) + at;
        store_e4m3<VEC>(dst + ca * VEC, a, p.scale[w.which]);
        store_e4m3<VEC>(dst + cb * VEC, b, p.scale[w.which]);
      } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.dst[w.which]) + at;
        store_bf16<VEC>(dst + ca * VEC, a);
        store_bf16<VEC>(dst + cb * VEC, b);
      }
    }
  }
}

}  // namespace attn
