// Attention of the answering calls on CUDA cores: one warp per (row, head),
// its query spread over the lanes, one key at a time with the running maximum
// and sum of the softmax in float32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cpattn_internal.h"

namespace cpattn {
namespace {

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half(x); }

template <typename T, int D>
struct Row {
  static constexpr int E = D / 32;
  float q[E], o[E], m = -INFINITY, l = 0.f;
  __device__ void load(const T* p, float scale) {
    for (int e = 0; e < E; ++e) q[e] = to_f(p[(threadIdx.x & 31) * E + e]) * scale;
    for (int e = 0; e < E; ++e) o[e] = 0.f;
  }
  __device__ void key(const T* k, const T* v) {
    const int at = (threadIdx.x & 31) * E;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += q[e] * to_f(k[at + e]);
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float mn = fmaxf(m, s), a = m == -INFINITY ? 0.f : expf(m - mn), p = expf(s - mn);
    l = l * a + p;
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + p * to_f(v[at + e]);
    m = mn;
  }
  __device__ void store(T* out, float* lse) {
    const int at = (threadIdx.x & 31) * E;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int e = 0; e < E; ++e) put(out + at + e, o[e] * inv);
    if ((threadIdx.x & 31) == 0) *lse = l == 0.f ? -INFINITY : m + logf(l);
  }
};

// The sequence of row i by its offsets; false when the row lies in none.
__device__ __forceinline__ bool find_row(const int* cu, int R, int total, int i, int& r, int& first,
                                         int& n, int* err) {
  int lo = 0, hi = R;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (cu[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  r = lo;
  if (!packed_rows(cu, r, total, first, n)) atomicExch(err, kErrBadTables);
  return i >= first && i < first + n;
}

__device__ __forceinline__ void check_rows(const int* cu, int R, int total, int* err) {
  int first, n;
  for (int r = threadIdx.x; r < R; r += blockDim.x)
    if (!packed_rows(cu, r, total, first, n)) atomicExch(err, kErrBadTables);
}

template <typename T, int D>
__global__ void __launch_bounds__(128) tree_simt_kernel(const TreeArgs a) {
  if (blockIdx.x == 0) check_rows(a.cu, a.R, a.N, a.err);
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int i = (int)(w / a.H), h = (int)(w % a.H);
  if (i >= a.N) return;
  int r, first, n;
  if (!find_row(a.cu, a.R, a.N, i, r, first, n, a.err)) return;
  int ctx = a.ctx[r];
  const int64_t cap = (int64_t)a.width * a.cache.page_size;
  if (ctx < 0 || (int64_t)ctx + n > cap || (a.tree != nullptr && n > 64)) atomicExch(a.err, kErrBadTables);
  ctx = ctx < 0 ? 0 : ctx;
  const int total = (int)min((int64_t)ctx + n, cap);
  const unsigned long long bits = a.tree != nullptr ? a.tree[i] : 0;
  const int P = a.cache.page_size, t = i - first;
  Row<T, D> row;
  row.load(static_cast<const T*>(a.q) + i * a.q_stride + h * D, a.scale);
  const int64_t hoff = (int64_t)(h / (a.H / a.Hkv)) * a.cache.head_stride;
  for (int j = 0; j < total; ++j) {
    const int d = j - ctx;
    if (d >= 0 && !(a.tree != nullptr ? (d < 64 && (bits >> d & 1)) : d <= t)) continue;
    const int page = a.table[r * a.table_stride + j / P];
    if (page < 0 || page >= a.cache.num_pages) {
      atomicExch(a.err, kErrBadTables);
      continue;
    }
    const int64_t off = page * a.cache.page_stride + (j % P) * a.cache.token_stride + hoff;
    row.key(static_cast<const T*>(a.k_cache) + off, static_cast<const T*>(a.v_cache) + off);
  }
  row.store(static_cast<T*>(a.out) + ((int64_t)i * a.H + h) * D, a.lse + (int64_t)h * a.N + i);
}

int grid_of(int rows, int H) { return (int)(((int64_t)rows * H + 3) / 4); }

}  // namespace

size_t tree_workspace_bytes(int N, int H, int Hkv, int D) { return 256; }

#define CPATTN_BY_TYPE(kernel, rows)                                                        \
  if (dtype == CPATTN_BF16 && a.D == 128)                                                   \
    kernel<__nv_bfloat16, 128><<<grid_of(rows, a.H), 128, 0, stream>>>(a);                  \
  else if (dtype == CPATTN_BF16)                                                            \
    kernel<__nv_bfloat16, 64><<<grid_of(rows, a.H), 128, 0, stream>>>(a);                   \
  else if (a.D == 128)                                                                      \
    kernel<__half, 128><<<grid_of(rows, a.H), 128, 0, stream>>>(a);                         \
  else                                                                                      \
    kernel<__half, 64><<<grid_of(rows, a.H), 128, 0, stream>>>(a);                          \
  return cudaGetLastError()

cudaError_t launch_tree_attn(const TreeArgs& a, int dtype, cudaStream_t stream) {
  CPATTN_BY_TYPE(tree_simt_kernel, a.N);
}

}  // namespace cpattn
