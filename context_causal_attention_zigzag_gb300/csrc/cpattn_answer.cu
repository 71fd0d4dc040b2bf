// C-ABI layer of the answering calls: argument checks and dispatch.
// Declarations and the meaning of every argument are in include/cpattn.h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "cpattn.h"
#include "cpattn_internal.h"

using namespace cpattn;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// CPATTN_OK, or why these heads and types are not taken.
int check_heads(int H, int Hkv, int D, int dtype) {
  if (dtype == CPATTN_F32) return CPATTN_ERR_UNSUPPORTED;
  if (dtype != CPATTN_BF16 && dtype != CPATTN_F16) return CPATTN_ERR_INVALID_ARG;
  if (H < 1 || Hkv < 1 || H % Hkv != 0 || H / Hkv > 128 || H > 65535)
    return CPATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return CPATTN_ERR_INVALID_ARG;
  return CPATTN_OK;
}

// Rows of [heads, D] elements, `stride` apart: 16-byte steps, no overlap.
bool check_rows(const void* p, int64_t stride, int heads, int D) {
  return p != nullptr && aligned(p, 16) && stride % 8 == 0 && stride >= (int64_t)heads * D &&
         stride < ((int64_t)1 << 38);
}

// Whether `rows` rows of [heads, D] 16-bit values, `stride` apart, and n bytes
// at `out` share memory.
bool overlaps(const void* p, int64_t stride, int64_t rows, int heads, int D, const void* out,
              int64_t n) {
  const char *a = static_cast<const char*>(p), *b = static_cast<const char*>(out);
  return a < b + n && b < a + 2 * ((rows - 1) * stride + (int64_t)heads * D);
}

// The same for a cache, from its first value to its last.
bool overlaps(const void* p, const CacheShape& c, int Hkv, int D, const void* out, int64_t n) {
  const __int128 a = reinterpret_cast<intptr_t>(p), b = reinterpret_cast<intptr_t>(out);
  const __int128 values = (__int128)(c.num_pages - 1) * c.page_stride +
                          (__int128)(c.page_size - 1) * c.token_stride +
                          (__int128)(Hkv - 1) * c.head_stride + D;
  return a < b + n && b < a + 2 * values;
}

bool page_size_ok(int P) {
  return P == 16 || P == 32 || P == 64 || (P >= 128 && P <= 1024 && P % 128 == 0);
}

bool check_cache(const void* k, const void* v, const CacheShape& c, int D) {
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return false;
  if (!page_size_ok(c.page_size) || c.num_pages < 1 || c.num_pages > INT32_MAX / c.page_size)
    return false;
  for (int64_t s : {c.page_stride, c.token_stride, c.head_stride})
    if (s < D || s % 8 != 0 || s >= ((int64_t)1 << 38)) return false;
  return true;
}

// Rows of a packed tensor, positions of a request in the cache and requests (the
// empty ones are passed one by one): within these an item, and the way to it, take
// less than the kernels' bounded waits allow (2 s), some of which last a whole item.
// A key tile of packed keys takes 1.6 us at 1.9 GHz and 2.1 us at 1.5, where a GPU at
// its power limit was seen: 2^19 of them 1.1 s.  In pages of 16 it takes 2.0 us (items
// of 128 rows behind 131072 positions), 2.5 us at 1.5 GHz: 1.3 s.
constexpr int kMostRows = 1 << 26;
constexpr int kMostPositions = 1 << 26;
constexpr int kMostRequests = 1 << 20;

bool scale_ok(float s) { return s <= 0.f || isfinite(s); }

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

int status(cudaError_t e) { return e == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA; }

}  // namespace

namespace cpattn {

bool encode_tiled(CUtensorMap* m, bool bf16, int rank, const void* ptr, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
             const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool rows_map(CUtensorMap* m, const void* ptr, bool bf16, int heads, int D, int64_t stride,
              int64_t rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)kTcTile};
  return encode_tiled(m, bf16, 3, ptr, dims, strides, box);
}

}  // namespace cpattn

extern "C" {

int cpattn_page_tables(const int32_t* ctx_lens, const int32_t* new_lens, int R, int page_size,
                       const int32_t* free_pages, int num_free, int32_t* block_table,
                       int table_width, int64_t table_stride, int32_t* cu_new, int64_t* slots,
                       int64_t num_slots, int32_t* used, cpattn_stream_t stream) {
  // The kernel steps through the requests in an int.
  if (R < 0 || R > (1 << 30) || !page_size_ok(page_size) || num_free < 0 || table_width < 0 ||
      table_stride < table_width || num_slots < 0 || num_slots > INT32_MAX)
    return CPATTN_ERR_INVALID_ARG;
  if (!cu_new || !used || (R > 0 && (!ctx_lens || !new_lens)) || (num_free > 0 && !free_pages) ||
      (R > 0 && table_width > 0 && !block_table) || (num_slots > 0 && !slots))
    return CPATTN_ERR_INVALID_ARG;
  for (const void* p : {(const void*)ctx_lens, (const void*)new_lens, (const void*)free_pages,
                        (const void*)block_table, (const void*)cu_new, (const void*)used})
    if (!aligned(p, 4)) return CPATTN_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return CPATTN_ERR_INVALID_ARG;
  int* err = device_error_word();
  if (err == nullptr) return CPATTN_ERR_CUDA;
  TablesArgs a = {ctx_lens,     new_lens, R,     page_size, free_pages, num_free, block_table,
                  table_width, table_stride, cu_new, slots, num_slots, used,  err};
  return status(launch_page_tables(a, (cudaStream_t)stream));
}

int cpattn_cache_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                       const int64_t* slots, int64_t N, void* k_cache, void* v_cache,
                       int64_t num_pages, int page_size, int64_t page_stride,
                       int64_t token_stride, int64_t head_stride, int Hkv, int D, int dtype,
                       cpattn_stream_t stream) {
  int rc = check_heads(Hkv, Hkv, D, dtype);
  if (rc != CPATTN_OK) return rc;
  if (N < 0 || N > INT32_MAX) return CPATTN_ERR_INVALID_ARG;
  CacheShape c = {num_pages, page_size, page_stride, token_stride, head_stride};
  if (!check_cache(k_cache, v_cache, c, D)) return CPATTN_ERR_INVALID_ARG;
  if (N == 0) return CPATTN_OK;
  if (!check_rows(k, k_stride, Hkv, D) || !check_rows(v, v_stride, Hkv, D) || !slots ||
      !aligned(slots, 8))
    return CPATTN_ERR_INVALID_ARG;
  int* err = device_error_word();
  if (err == nullptr) return CPATTN_ERR_CUDA;
  CacheWriteArgs a = {k, v, k_stride, v_stride, slots, N, k_cache, v_cache, c, Hkv, D, err};
  return status(launch_cache_write(a, (cudaStream_t)stream));
}

size_t cpattn_tree_attn_workspace_bytes(int N, int H, int Hkv, int D) {
  if (N < 0 || check_heads(H, Hkv, D, CPATTN_BF16) != CPATTN_OK) return 0;
  return tree_workspace_bytes(N, H, Hkv, D);
}

int cpattn_tree_attn(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                     int64_t num_pages, int page_size, int64_t page_stride, int64_t token_stride,
                     int64_t head_stride, const int32_t* block_table, int table_width,
                     int64_t table_stride, const int32_t* ctx_lens, const int32_t* cu_new,
                     const uint64_t* tree, void* out, float* lse, int R, int N, int H, int Hkv,
                     int D, int dtype, float softmax_scale, void* workspace,
                     size_t workspace_bytes, cpattn_stream_t stream) {
  int rc = check_heads(H, Hkv, D, dtype);
  if (rc != CPATTN_OK) return rc;
  if (R < 0 || R > kMostRequests || N < 0 || N > (1 << 30) || !scale_ok(softmax_scale))
    return CPATTN_ERR_INVALID_ARG;
  CacheShape c = {num_pages, page_size, page_stride, token_stride, head_stride};
  if (!check_cache(k_cache, v_cache, c, D)) return CPATTN_ERR_INVALID_ARG;
  if (table_width < 0 || table_stride < table_width || table_width > kMostPositions / page_size)
    return CPATTN_ERR_INVALID_ARG;
  if (R == 0 || N == 0) return CPATTN_OK;
  if (!check_rows(q, q_stride, H, D) || !check_rows(out, (int64_t)H * D, H, D) || !lse ||
      !aligned(lse, 4) || (table_width > 0 && !block_table) || !ctx_lens || !cu_new)
    return CPATTN_ERR_INVALID_ARG;
  if (!aligned(block_table, 4) || !aligned(ctx_lens, 4) || !aligned(cu_new, 4) ||
      !aligned(tree, 8))
    return CPATTN_ERR_INVALID_ARG;
  if (overlaps(q, q_stride, N, H, D, out, 2 * (int64_t)N * H * D)) return CPATTN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < tree_workspace_bytes(N, H, Hkv, D))
    return CPATTN_ERR_WORKSPACE;
  const int64_t out_bytes = 2 * (int64_t)N * H * D;
  if (overlaps(k_cache, c, Hkv, D, out, out_bytes) || overlaps(v_cache, c, Hkv, D, out, out_bytes))
    return CPATTN_ERR_INVALID_ARG;
  int* err = device_error_word();
  if (err == nullptr) return CPATTN_ERR_CUDA;
  TreeArgs a;
  a.q = q;
  a.q_stride = q_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.cache = c;
  a.table = block_table;
  a.width = table_width;
  a.table_stride = table_stride;
  a.ctx = ctx_lens;
  a.cu = cu_new;
  a.tree = reinterpret_cast<const unsigned long long*>(tree);
  a.out = out;
  a.lse = lse;
  a.R = R;
  a.N = N;
  a.H = H;
  a.Hkv = Hkv;
  a.D = D;
  a.scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)D);
  a.scale_log2 = a.scale * 1.4426950408889634f;
  a.workspace = workspace;
  a.err = err;
  a.cu_k = nullptr;
  a.k_stride = a.v_stride = 0;
  a.Nk = a.causal = a.above = 0;
  return status(launch_tree_attn(a, dtype, (cudaStream_t)stream));
}

size_t cpattn_prompt_attn_workspace_bytes(int R, int Nq, int H, int D) {
  if (R < 0 || Nq < 0 || check_heads(H, H, D, CPATTN_BF16) != CPATTN_OK) return 0;
  return prompt_workspace_bytes(R, Nq, H, D);
}

int cpattn_prompt_attn(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                       const void* v, int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k,
                       void* out, float* lse, int R, int Nq, int Nk, int H, int Hkv, int D,
                       int causal, int dtype, float softmax_scale, void* workspace,
                       size_t workspace_bytes, cpattn_stream_t stream) {
  int rc = check_heads(H, Hkv, D, dtype);
  if (rc != CPATTN_OK) return rc;
  if (R < 0 || R > kMostRequests || Nq < 0 || Nk < 0 || Nq > kMostRows || Nk > kMostRows ||
      (causal != 0 && causal != 1) || !scale_ok(softmax_scale))
    return CPATTN_ERR_INVALID_ARG;
  // Work items are numbered in an int, with room for the CTAs that ask past the end.
  if (((int64_t)Nq / 128 + R) * H > INT32_MAX / 2) return CPATTN_ERR_INVALID_ARG;
  if (R == 0 || Nq == 0) return CPATTN_OK;
  if (!check_rows(q, q_stride, H, D) || !check_rows(out, (int64_t)H * D, H, D) || !lse ||
      !aligned(lse, 4) || !cu_q || !cu_k || !aligned(cu_q, 4) || !aligned(cu_k, 4))
    return CPATTN_ERR_INVALID_ARG;
  if (Nk > 0 && (!check_rows(k, k_stride, Hkv, D) || !check_rows(v, v_stride, Hkv, D)))
    return CPATTN_ERR_INVALID_ARG;
  const int64_t out_bytes = 2 * (int64_t)Nq * H * D;
  if (overlaps(q, q_stride, Nq, H, D, out, out_bytes) ||
      (Nk > 0 && (overlaps(k, k_stride, Nk, Hkv, D, out, out_bytes) ||
                  overlaps(v, v_stride, Nk, Hkv, D, out, out_bytes))))
    return CPATTN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < prompt_workspace_bytes(R, Nq, H, D))
    return CPATTN_ERR_WORKSPACE;
  int* err = device_error_word();
  if (err == nullptr) return CPATTN_ERR_CUDA;
  PromptArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.out = out;
  a.lse = lse;
  a.R = R;
  a.Nq = Nq;
  a.Nk = Nk;
  a.H = H;
  a.Hkv = Hkv;
  a.D = D;
  a.causal = causal;
  a.scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)D);
  a.scale_log2 = a.scale * 1.4426950408889634f;
  a.workspace = workspace;
  a.err = err;
  return status(launch_prompt_attn(a, dtype, (cudaStream_t)stream));
}

}  // extern "C"
