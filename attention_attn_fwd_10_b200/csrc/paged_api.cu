// C-ABI entry points of rotary positions, the paged cache's append and the
// attention over it (declared in include/attn.h): argument checks and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "api_internal.h"
#include "paged_chunk_kernel.cuh"
#include "paged_few_kernel.cuh"
#include "paged_plan.cuh"
#include "rotary_kernels.cuh"

namespace attn {
namespace {

constexpr int kNumSms = 148;  // B200

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// ---------------------------------------------------------------------------- rotation

// Checks a rotation and puts it into the kernel's parameters.
attn_status_t set_rotary(RotaryParams* p, const attn_rotary_t* r, int D, bool inverse) {
  if (!r->inv_freq) return ATTN_ERR_INVALID_ARG;
  if (r->n_freq < 4 || r->n_freq % 4 != 0 || r->n_freq > D / 2) return ATTN_ERR_INVALID_ARG;
  if (r->n_axes < 1 || r->n_axes > 4 || (r->interleaved != 0 && r->interleaved != 1)) return ATTN_ERR_INVALID_ARG;
  if (!r->positions && r->n_axes != 1) return ATTN_ERR_INVALID_ARG;
  if (!aligned(r->inv_freq, 4) || !aligned(r->positions, 4)) return ATTN_ERR_MISALIGNED;
  int end = 0;
  for (int a = 0; a < r->n_axes; ++a) {
    if (r->section[a] < 0 || r->section[a] > r->n_freq) return ATTN_ERR_INVALID_ARG;
    end += r->section[a];
    p->sec_end[a] = end;
  }
  if (end != r->n_freq) return ATTN_ERR_INVALID_ARG;
  for (int a = r->n_axes - 1; a < 4; ++a) p->sec_end[a] = r->n_freq;  // no frequency beyond the last axis
  p->inv_freq = r->inv_freq;
  p->positions = r->positions;
  p->n_freq = r->n_freq;
  p->sign = inverse ? -1.f : 1.f;
  return ATTN_OK;
}

template <int D, int VEC, bool INTERLEAVED, bool PAGED, bool E4M3>
cudaError_t launch_rotary(RotaryParams p, cudaStream_t s) {
  constexpr int ITEMS = 4;
  constexpr int PER_HEAD = D / (2 * VEC);
  constexpr int MOST = kRotThreads * ITEMS / PER_HEAD;  // (token, head) pairs of a CTA
  // Whole tokens per CTA (their angles are computed once), as many as fit; fewer,
  // down to a head range of one token, while the grid would leave SMs idle.
  int tok = std::max(1, std::min(kRotMaxTok, MOST / p.n_heads));
  int hpc = std::min(p.n_heads, MOST);
  auto ctas = [&] { return (p.n_tokens + tok - 1) / tok * ((p.n_heads + hpc - 1) / hpc); };
  while (tok > 1 && ctas() < 2 * kNumSms) tok = (tok + 1) / 2;
  while (hpc > 8 && ctas() < kNumSms) hpc = (hpc + 1) / 2;
  p.tok = tok;
  p.hpc = hpc;
  const long long gx = (p.n_tokens + tok - 1) / tok;
  const int gy = (p.n_heads + hpc - 1) / hpc;
  if (gx > 2147483647ll || gy > 65535) return cudaErrorInvalidConfiguration;
  rotary_kernel<D, VEC, ITEMS, INTERLEAVED, PAGED, E4M3>
      <<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), kRotThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// 16-byte chunks need frequencies in eights; else (rotated dims such as 24) 8-byte ones.
template <bool PAGED, bool E4M3>
cudaError_t launch_rotary_any(const RotaryParams& p, int D, bool interleaved, cudaStream_t s) {
  const bool wide = p.n_freq % 8 == 0;
  if (D == 128) {
    if (wide)
      return interleaved ? launch_rotary<128, 8, true, PAGED, E4M3>(p, s) : launch_rotary<128, 8, false, PAGED, E4M3>(p, s);
    return interleaved ? launch_rotary<128, 4, true, PAGED, E4M3>(p, s) : launch_rotary<128, 4, false, PAGED, E4M3>(p, s);
  }
  if (wide)
    return interleaved ? launch_rotary<64, 8, true, PAGED, E4M3>(p, s) : launch_rotary<64, 8, false, PAGED, E4M3>(p, s);
  return interleaved ? launch_rotary<64, 4, true, PAGED, E4M3>(p, s) : launch_rotary<64, 4, false, PAGED, E4M3>(p, s);
}

bool good_stride(long long stride, int H, int D) {
  return stride % 8 == 0 && stride >= static_cast<long long>(H) * D && stride < (1ll << 40);
}

// ---------------------------------------------------------------------------- paged cache

attn_status_t check_cache(const attn_paged_kv_t* c, int n_tokens) {
  if (!c) return ATTN_ERR_INVALID_ARG;
  if (!c->k || !c->v || !c->page_table || !c->seq_len || !c->q_start) return ATTN_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->H_kv < 1 || c->max_pages < 1 || c->n_seq < 1 || n_tokens < 0) return ATTN_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size % 16 != 0) return ATTN_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return ATTN_ERR_UNSUPPORTED;
  if (c->e4m3 != 0 && c->e4m3 != 1) return ATTN_ERR_INVALID_ARG;
  if (!(std::isfinite(c->k_scale) && c->k_scale > 0.f && std::isfinite(c->v_scale) && c->v_scale > 0.f))
    return ATTN_ERR_INVALID_ARG;
  if (!c->e4m3 && (c->k_scale != 1.f || c->v_scale != 1.f)) return ATTN_ERR_INVALID_ARG;
  if (c->table_stride < c->max_pages) return ATTN_ERR_INVALID_ARG;
  // key indices are 32-bit, with room for a tile past the end
  if (static_cast<long long>(c->max_pages) * c->page_size > 2147483647ll - 1024) return ATTN_ERR_UNSUPPORTED;
  if (c->H_kv > 65535 || c->n_seq > (1 << 24)) return ATTN_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4) || !aligned(c->seq_len, 4) ||
      !aligned(c->q_start, 4))
    return ATTN_ERR_MISALIGNED;
  const int per16 = c->e4m3 ? 16 : 8;
  struct Dim {
    long long stride;
    long long size;
  } d[3] = {{c->page_stride, c->n_pages}, {c->token_stride, c->page_size}, {c->head_stride, c->H_kv}};
  for (const Dim& x : d) {
    if (x.size > 1 && x.stride < c->D) return ATTN_ERR_INVALID_ARG;
    if (x.stride < 0 || x.stride >= (1ll << 38)) return ATTN_ERR_INVALID_ARG;
    if (x.stride % per16 != 0) return ATTN_ERR_MISALIGNED;
  }
  // no two elements share a place: each dim steps over the whole of the smaller ones
  std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  long long extent = c->D;
  for (const Dim& x : d) {
    if (x.size == 1) continue;
    if (x.stride < extent) return ATTN_ERR_INVALID_ARG;
    extent = x.stride * (x.size - 1) + extent;
  }
  return ATTN_OK;
}

// The cache viewed as (D, H_kv, page_size, n_pages); boxes of one head, box_rows slots of one page, and
// 128 bytes (or a whole e4m3 row of 64) across.
bool make_cache_map(CUtensorMap* map, const attn_paged_kv_t* c, void* ptr, int box_rows) {
  EncodeTiledFn enc = api_encode_tiled();
  if (!enc) return false;
  const long long eb = c->e4m3 ? 1 : 2;
  auto bytes = [&](long long stride, int size) {  // a dim of one element may have any stride
    return static_cast<cuuint64_t>((size > 1 ? stride : c->D) * eb);
  };
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->D), static_cast<cuuint64_t>(c->H_kv),
                              static_cast<cuuint64_t>(c->page_size), static_cast<cuuint64_t>(c->n_pages)};
  const cuuint64_t strides[3] = {bytes(c->head_stride, c->H_kv), bytes(c->token_stride, c->page_size),
                                 bytes(c->page_stride, c->n_pages)};
  // What L2 fetches at a time: no more than the bytes that lie together.  With 256 bytes, the 128-byte rows of an
  // e4m3 cache [pages, slots, heads, 128] brought in the next head's row too: 393 MB of DRAM reads for 268.
  const long long together = c->page_size > 1 && c->token_stride == c->D ? 256 : c->D * eb;
  const CUtensorMapL2promotion promotion = together >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                           : together >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                             : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  const cuuint32_t across = static_cast<cuuint32_t>(c->e4m3 ? c->D : 64);
  const cuuint32_t box[4] = {across, 1, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  return enc(map, c->e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, ptr, dims, strides, box,
             estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
             across * eb == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, promotion,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The token rows viewed as (D, H_q, tokens); boxes of one kv group's heads x `positions` tokens x 64 dims.
bool make_q_map(CUtensorMap* map, const void* q, int n_tokens, int H_q, int D, long long q_stride, int group, int positions) {
  EncodeTiledFn enc = api_encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H_q), static_cast<cuuint64_t>(n_tokens), 1};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(q_stride) * 2,
                                 static_cast<cuuint64_t>(q_stride) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(positions), 1};
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kPagedCtas = kNumSms;  // persistent: one CTA per SM

// Workspace: the cut units' records, the pieces' log-sum-exps, their fp32 rows (two pieces per CTA).
struct PagedWorkspace {
  size_t l_off, o_off, bytes;
};
PagedWorkspace paged_workspace(int unit_rows, int D) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  PagedWorkspace w;
  const size_t rows = 2ull * kPagedCtas * unit_rows;
  w.l_off = up(kPagedCtas * sizeof(int4));
  w.o_off = w.l_off + up(rows * sizeof(float));
  w.bytes = w.o_off + up(rows * D * sizeof(float));
  return w;
}

// Lays the workspace out, encodes the maps and launches `kern` (one CTA per SM), then the merge.
template <int D, bool KV8, int TILE_ROWS, typename L>
cudaError_t launch_paged(void (*kern)(CUtensorMap, CUtensorMap, CUtensorMap, PagedParams), const attn_paged_kv_t* c,
                         PagedParams p, int tiles, void* workspace, CUcontext* seen, cudaStream_t s) {
  p.tile_pos = TILE_ROWS / p.group;
  p.unit_pos = tiles * p.tile_pos;
  p.unit_rows = tiles * TILE_ROWS;
  p.step_log2 = tiles - 1;
  p.unit_extra = tiles == 2 ? 2 : 4;
  p.min_steps = 2;
  const PagedWorkspace w = paged_workspace(p.unit_rows, D);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.cut = reinterpret_cast<int4*>(ws);
  p.l_part = reinterpret_cast<float*>(ws + w.l_off);
  p.o_part = reinterpret_cast<float*>(ws + w.o_off);
  CUtensorMap mq{}, mk, mv;
  if (!KV8 && !make_q_map(&mq, p.q, p.n_tokens, p.H_q, D, p.q_stride, p.group, p.tile_pos)) return cudaErrorUnknown;
  if (!make_cache_map(&mk, c, c->k, p.box_rows) || !make_cache_map(&mv, c, c->v, p.box_rows)) return cudaErrorUnknown;
  cudaError_t e = api_smem_opt_in(reinterpret_cast<const void*>(kern), L::SMEM_BYTES, seen);
  if (e != cudaSuccess) return e;
  kern<<<kPagedCtas, L::THREADS, L::SMEM_BYTES, s>>>(mq, mk, mv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the merge: a programmatic dependent, so that its launch overlaps the attention's tail (it waits on the device for
  // that grid, and so for everything before it)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kPagedCtas - 1, static_cast<unsigned>(p.unit_rows / (8 * merge_rows(TILE_ROWS))));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, TILE_ROWS>, p);
}

// The kernel by the rows that a sequence's new tokens make in a kv group (max_new, or the mean where it is not
// known, times the group's heads): up to 32 as MMA columns, more as tiles of 128 rows.  64 sequences of up to 4096
// keys, 8 kv heads, head dim 128, bf16 / e4m3 cache, in us: 16 rows as 16 columns 106 / 85, as 32 columns 105 / 101,
// as tiles 116 / 171; 32 rows as 32 columns 107 / 118, as tiles 115 / 161 (and 33 rows would be two column units).
// Head dim 64: 70 / 69, 72 / 94, 98 / 131; 78 / 102, 94 / 122.  (The mean misjudges one long chunk among single
// tokens: right, but as column units that each read the chunk's keys.)
template <int D, bool KV8>
cudaError_t launch_attend(const attn_paged_kv_t* c, const PagedParams& p, int max_new, void* workspace, cudaStream_t s) {
  static CUcontext seen[3][kApiMaxDevices] = {};
  const long long rows = static_cast<long long>(max_new > 0 ? max_new : (p.n_tokens + p.n_seq - 1) / p.n_seq) * p.group;
  if (rows <= 16)
    return launch_paged<D, KV8, 16, FewLayout<D, KV8, 16>>(paged_few_kernel<D, KV8, 16>, c, p, 1, workspace, seen[0], s);
  if (rows <= 32)
    return launch_paged<D, KV8, 32, FewLayout<D, KV8, 32>>(paged_few_kernel<D, KV8, 32>, c, p, 1, workspace, seen[1], s);
  return launch_paged<D, KV8, 128, ChunkLayout<D, KV8>>(paged_chunk_kernel<D, KV8>, c, p, 2, workspace, seen[2], s);
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

attn_status_t attn_rope(const void* q, const void* k, void* q_out, void* k_out, long long n_tokens, int H_q, int H_k,
                        int D, long long q_stride, long long k_stride, long long q_out_stride,
                        long long k_out_stride, long long period, const attn_rotary_t* rotary, int inverse,
                        void* stream) {
  if (!rotary || n_tokens < 0 || H_q < 1 || (inverse != 0 && inverse != 1)) return ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
  if (!q || !q_out || !good_stride(q_stride, H_q, D) || !good_stride(q_out_stride, H_q, D)) return ATTN_ERR_INVALID_ARG;
  if (k && (!k_out || H_k < 1 || !good_stride(k_stride, H_k, D) || !good_stride(k_out_stride, H_k, D)))
    return ATTN_ERR_INVALID_ARG;
  if ((q == q_out && q_stride != q_out_stride) || (k && k == k_out && k_stride != k_out_stride))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(q_out, 16) || (k && (!aligned(k, 16) || !aligned(k_out, 16))))
    return ATTN_ERR_MISALIGNED;
  RotaryParams p{};
  const attn_status_t st = set_rotary(&p, rotary, D, inverse != 0);
  if (st != ATTN_OK) return st;
  if (!rotary->positions && (period < 1 || period > 2147483647ll)) return ATTN_ERR_INVALID_ARG;
  if (n_tokens > 2147483647ll || H_q > 65535 || (k && H_k > 65535)) return ATTN_ERR_UNSUPPORTED;
  if (n_tokens == 0) return ATTN_OK;
  p.src[0] = static_cast<const __nv_bfloat16*>(q);
  p.dst[0] = q_out;
  p.src_stride[0] = q_stride;
  p.dst_stride[0] = q_out_stride;
  p.heads[0] = H_q;
  if (k) {
    p.src[1] = static_cast<const __nv_bfloat16*>(k);
    p.dst[1] = k_out;
    p.src_stride[1] = k_stride;
    p.dst_stride[1] = k_out_stride;
    p.heads[1] = H_k;
  }
  p.n_heads = p.heads[0] + p.heads[1];
  p.n_tokens = n_tokens;
  p.period = period;
  return launch_rotary_any<false, false>(p, D, rotary->interleaved != 0, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

attn_status_t attn_paged_append(const attn_paged_kv_t* c, const void* q, const void* k, const void* v, void* q_out,
                                int n_tokens, int H_q, long long q_stride, long long k_stride, long long v_stride,
                                const attn_rotary_t* rotary, void* stream) {
  attn_status_t st = check_cache(c, n_tokens);
  if (st != ATTN_OK) return st;
  if (!k || !v || !good_stride(k_stride, c->H_kv, c->D) || !good_stride(v_stride, c->H_kv, c->D))
    return ATTN_ERR_INVALID_ARG;
  if (q && (!rotary || !q_out || H_q < 1 || !good_stride(q_stride, H_q, c->D))) return ATTN_ERR_INVALID_ARG;
  const long long q_dense = static_cast<long long>(H_q) * c->D;
  if (q && q == q_out && q_stride != q_dense) return ATTN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || (q && (!aligned(q, 16) || !aligned(q_out, 16)))) return ATTN_ERR_MISALIGNED;
  if (q && H_q > 65535) return ATTN_ERR_UNSUPPORTED;
  RotaryParams p{};
  if (rotary) {
    st = set_rotary(&p, rotary, c->D, false);
    if (st != ATTN_OK) return st;
  }
  if (n_tokens == 0) return ATTN_OK;
  p.status = api_status_ptr();
  if (!p.status) return ATTN_ERR_CUDA;
  if (q) {
    p.src[0] = static_cast<const __nv_bfloat16*>(q);
    p.dst[0] = q_out;
    p.src_stride[0] = q_stride;
    p.dst_stride[0] = q_dense;
    p.heads[0] = H_q;
  }
  p.src[1] = static_cast<const __nv_bfloat16*>(k);
  p.src[2] = static_cast<const __nv_bfloat16*>(v);
  p.dst[1] = c->k;
  p.dst[2] = c->v;
  p.src_stride[1] = k_stride;
  p.src_stride[2] = v_stride;
  p.heads[1] = p.heads[2] = c->H_kv;
  p.scale[1] = c->k_scale;
  p.scale[2] = c->v_scale;
  p.n_heads = p.heads[0] + 2 * c->H_kv;
  p.n_tokens = n_tokens;
  p.n_pages = c->n_pages;
  p.page_size = c->page_size;
  p.max_pages = c->max_pages;
  p.n_seq = c->n_seq;
  p.page_stride = c->page_stride;
  p.token_stride = c->token_stride;
  p.head_stride = c->head_stride;
  p.table_stride = c->table_stride;
  p.page_table = c->page_table;
  p.seq_len = c->seq_len;
  p.q_start = c->q_start;
  const bool il = rotary && rotary->interleaved;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      c->e4m3 ? launch_rotary_any<true, true>(p, c->D, il, s) : launch_rotary_any<true, false>(p, c->D, il, s);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

size_t attn_fwd_paged_workspace_size(int H_q, int H_kv, int D) {
  if (H_q < 1 || H_kv < 1 || H_q % H_kv != 0 || H_q / H_kv > 128 || (D != 64 && D != 128)) return 0;
  return paged_workspace(256, D).bytes;
}

attn_status_t attn_fwd_paged(const attn_paged_kv_t* c, const void* q, void* o, float* lse, void* workspace,
                             int n_tokens, int H_q, long long q_stride, int max_new, int causal, float scale,
                             void* stream) {
  attn_status_t st = check_cache(c, n_tokens);
  if (st != ATTN_OK) return st;
  if (!q || !o || !lse || !workspace || H_q < 1 || H_q % c->H_kv != 0 || !good_stride(q_stride, H_q, c->D))
    return ATTN_ERR_INVALID_ARG;
  if (max_new < 0 || (causal != 0 && causal != 1) || !std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  // what turns a product of q and a stored key into a score in base-2 units
  const double scale_log2 = static_cast<double>(scale) * c->k_scale * 1.4426950408889634;
  if (scale_log2 > 3.4028234e38) return ATTN_ERR_INVALID_ARG;
  if (H_q / c->H_kv > 128) return ATTN_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 16) || !aligned(workspace, 32)) return ATTN_ERR_MISALIGNED;
  if (n_tokens == 0) return ATTN_OK;
  PagedParams p{};
  p.status = api_status_ptr();
  if (!p.status) return ATTN_ERR_CUDA;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.n_tokens = n_tokens;
  p.H_q = H_q;
  p.H_kv = c->H_kv;
  p.group = H_q / c->H_kv;
  p.q_stride = q_stride;
  p.n_pages = c->n_pages;
  p.page_size = c->page_size;
  p.room = c->max_pages * c->page_size;
  p.n_seq = c->n_seq;
  while (p.box_shift < 7 && c->page_size % (2 << p.box_shift) == 0) ++p.box_shift;
  p.box_rows = 1 << p.box_shift;
  p.table_stride = c->table_stride;
  p.page_table = c->page_table;
  p.seq_len = c->seq_len;
  p.q_start = c->q_start;
  p.scale_log2 = std::max(static_cast<float>(scale_log2), 1.17549435e-38f);
  p.v_scale = c->v_scale;
  p.causal = causal;
  p.wait_limit_ns = api_wait_limit_ns();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (c->e4m3)
    e = c->D == 128 ? launch_attend<128, true>(c, p, max_new, workspace, s) : launch_attend<64, true>(c, p, max_new, workspace, s);
  else
    e = c->D == 128 ? launch_attend<128, false>(c, p, max_new, workspace, s)
                    : launch_attend<64, false>(c, p, max_new, workspace, s);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
