// Attention of each sequence's new tokens over its paged keys.
#pragma once

#include <cuda_fp8.h>

#include "rotary_kernels.cuh"
#include "sm100_common.cuh"

namespace attn {

struct PagedParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const void *k, *v;
  int n_tokens, H_q, H_kv, group;
  long long q_stride;
  int n_pages, page_size, max_pages, n_seq;
  long long page_stride, token_stride, head_stride, table_stride;
  const int *page_table, *seq_len, *q_start;
  float scale_log2;  // scale * k_scale * log2(e)
  float v_scale;
  int causal;
  int* status;
};

__device__ __forceinline__ float cell(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float cell(const __nv_fp8_e4m3* p) { return static_cast<float>(*p); }

// The plain form: one warp per (token, query head), one key at a time.
template <int D, typename Cell>
__global__ void __launch_bounds__(256) paged_plain_kernel(const PagedParams p) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (w >= static_cast<long long>(p.n_tokens) * p.H_q) return;
  const long long t = w / p.H_q;
  const int h = static_cast<int>(w - t * p.H_q);
  const int b = owner_of(t, p.q_start, p.n_seq, lane);
  if (b < 0) return;
  const int len = p.seq_len[b];
  const long long room = static_cast<long long>(p.max_pages) * p.page_size;
  const int n = static_cast<int>(max(0ll, min(static_cast<long long>(len), room)));
  bool bad = n != len || p.q_start[b] < 0 || p.q_start[b + 1] > p.n_tokens;
  const long long last = p.causal ? static_cast<long long>(len) - (p.q_start[b + 1] - t) : len - 1ll;
  const int end = static_cast<int>(max(0ll, min(static_cast<long long>(n), last + 1)));
  float q[PER], acc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    q[i] = __bfloat162float(p.q[t * p.q_stride + static_cast<long long>(h) * D + lane * PER + i]);
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const long long head = h / p.group * p.head_stride + lane * PER;
  for (int j = 0; j < end; ++j) {
    const int page = p.page_table[b * p.table_stride + j / p.page_size];
    if (page < 0 || page >= p.n_pages) {
      bad = true;
      continue;
    }
    const long long at = page * p.page_stride + j % p.page_size * p.token_stride + head;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) s += q[i] * cell(static_cast<const Cell*>(p.k) + at + i);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float x = s * p.scale_log2;
    const float mn = fmaxf(m, x);
    const float a = m == -INFINITY ? 0.f : exp2f(m - mn), e = exp2f(x - mn);
    m = mn;
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = acc[i] * a + e * cell(static_cast<const Cell*>(p.v) + at + i);
  }
  const float inv = l > 0.f ? p.v_scale / l : 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    p.o[(t * p.H_q + h) * D + lane * PER + i] = __float2bfloat16(acc[i] * inv);
  if (lane == 0) {
    p.lse[static_cast<long long>(h) * p.n_tokens + t] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    if (bad) atomicExch(p.status, kDevBadIndex);
  }
}

}  // namespace attn
