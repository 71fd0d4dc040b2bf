// The paged cache's bookkeeping and its write: block tables and slot maps from
// request lengths, and the copy of new keys and values into their slots.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "cpattn_internal.h"

namespace cpattn {
namespace {

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
  return n > 0 ? n : 148;
}

// ---------------------------------------------------------------------------
// Tables.  With have_r = ceil(ctx_r / P) and need_r = ceil((ctx_r + new_r) / P)
// two exclusive sums over the requests say everything: cu_r = sum new gives a
// token's request and position, start_r = sum (need - have) the pages of the
// free list that the request takes.  A token's slot needs no other block's
// writes (its page is either the request's last old page or a page of the free
// list), so one launch does it all: every block runs the sums itself -- R
// lengths from L2, a chunk of 1024 at a time -- and then fills its share of
// the slots and table entries.  The call is bound by its latency: a launch,
// two dependent loads and the block's sum.
// ---------------------------------------------------------------------------
constexpr int kTabThreads = 1024;

// Exclusive sums of two values over the block; tot gets the block's sums.
__device__ __forceinline__ void block_sums(long long& a, long long& b, long long (*part)[32],
                                           long long& tot_a, long long& tot_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = a, y = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, d), w = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) {
      x += u;
      y += w;
    }
  }
  if (lane == 31) {
    part[0][warp] = x;
    part[1][warp] = y;
  }
  __syncthreads();
  if (warp < 2) {
    const long long own = part[warp][lane];
    long long z = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, z, d);
      if (lane >= d) z += u;
    }
    part[warp][lane] = z - own;  // exclusive
    if (lane == 31) part[2][warp] = z;
  }
  __syncthreads();
  a = x - a + part[0][warp];
  b = y - b + part[1][warp];
  tot_a = part[2][0];
  tot_b = part[2][1];
}

// Last index i in [0, n) with pre[i] <= x (pre[0] <= x, non-decreasing).
__device__ __forceinline__ int last_at_or_below(const uint32_t* pre, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreads) page_tables_kernel(const TablesArgs a) {
  __shared__ long long part[3][32];
  // Exclusive sums within the chunk, in 32 bits (sums that pass them are an
  // error already; they stay in order).
  __shared__ uint32_t s_tok[kTabThreads], s_page[kTabThreads];
  __shared__ int s_ctx[kTabThreads];
  const int tid = threadIdx.x;
  const long long P = a.page_size;
  const long long stride = (long long)gridDim.x * kTabThreads;
  const long long mine = (long long)blockIdx.x * kTabThreads + tid;
  long long tok0 = 0, page0 = 0;  // sums of the chunks before
  bool bad = false;
  for (int r0 = 0; r0 < a.R; r0 += kTabThreads) {
    const int r = r0 + tid, nr = min(kTabThreads, a.R - r0);
    long long ctx = 0, n = 0;
    if (r < a.R) {
      ctx = a.ctx[r];
      n = a.fresh[r];
      if (ctx < 0 || n < 0) {
        bad = true;
        ctx = ctx < 0 ? 0 : ctx;
        n = 0;
      }
    }
    long long tok = n, page = (ctx + n + P - 1) / P - (ctx + P - 1) / P, ntok, npage;
    block_sums(tok, page, part, ntok, npage);
    s_tok[tid] = (uint32_t)(tok < 0xffffffffll ? tok : 0xffffffffll);
    s_page[tid] = (uint32_t)(page < 0xffffffffll ? page : 0xffffffffll);
    s_ctx[tid] = (int)ctx;
    if (blockIdx.x == 0 && r < a.R)
      a.cu[r] = (int)(tok0 + tok < INT_MAX ? tok0 + tok : INT_MAX);
    __syncthreads();
    // New table entries: page x of the free list goes to one request.
    long long x = mine < page0 ? mine + (page0 - mine + stride - 1) / stride * stride : mine;
    const long long page_end = page0 + npage < a.num_free ? page0 + npage : a.num_free;
    for (; x < page_end; x += stride) {
      const int i = last_at_or_below(s_page, nr, (uint32_t)(x - page0));
      const long long col =
          ((uint32_t)s_ctx[i] + (uint32_t)P - 1) / (uint32_t)P + (x - page0 - s_page[i]);
      if (col < a.width)
        a.table[(int64_t)(r0 + i) * a.table_stride + col] = a.free_pages[x];
      else
        bad = true;
    }
    bad = bad || page0 + npage > a.num_free || tok0 + ntok > a.num_slots;
    // Slots.
    x = mine < tok0 ? mine + (tok0 - mine + stride - 1) / stride * stride : mine;
    const long long tok_end = tok0 + ntok < a.num_slots ? tok0 + ntok : a.num_slots;
    for (; x < tok_end; x += stride) {
      const int i = last_at_or_below(s_tok, nr, (uint32_t)(x - tok0));
      const uint32_t c = s_ctx[i], pos = c + ((uint32_t)(x - tok0) - s_tok[i]);
      const uint32_t p = (uint32_t)P, col = pos / p, have = (c + p - 1) / p;
      long long id = -1;
      if (col < (uint32_t)a.width) {
        if (col < have) {
          id = a.table[(int64_t)(r0 + i) * a.table_stride + col];
        } else {
          const long long f = page0 + s_page[i] + (col - have);
          if (f < a.num_free) id = a.free_pages[f];
        }
      }
      if (id < 0) bad = true;
      a.slots[x] = id < 0 ? -1 : id * P + (pos - col * p);
    }
    tok0 += ntok;
    page0 += npage;
    __syncthreads();  // the next chunk overwrites the sums
  }
  for (long long x = mine < tok0 ? mine + (tok0 - mine + stride - 1) / stride * stride : mine;
       x < a.num_slots; x += stride)
    a.slots[x] = -1;
  if (mine == 0) {
    a.cu[a.R] = (int)(tok0 < INT_MAX ? tok0 : INT_MAX);
    *a.used = (int)(page0 < INT_MAX ? page0 : INT_MAX);
  }
  if (bad) atomicExch(a.err, kErrBadTables);
}

// ---------------------------------------------------------------------------
// Write.  One warp per token: its slot is read once, then the token's key and
// value rows move in 16-byte vectors, all loads of a round before its stores.
// Bound by HBM: 2 rows read and 2 rows written a token.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheWriteArgs a) {
  constexpr int kVec = D / 8;  // 16-byte vectors of a head's row
  constexpr int U = 8;
  const int lane = threadIdx.x & 31;
  const int row_vecs = a.Hkv * kVec;
  const int64_t slots = a.cache.num_pages * a.cache.page_size;
  const int64_t nwarps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < a.N;
       i += nwarps) {
    const int64_t slot = a.slots[i];
    if (slot < 0) continue;
    if (slot >= slots) {
      if (lane == 0) atomicExch(a.err, kErrBadTables);
      continue;
    }
    const int page = (int)slot / a.cache.page_size;
    const int64_t dst0 = page * a.cache.page_stride +
                         ((int)slot - page * a.cache.page_size) * a.cache.token_stride;
    const uint16_t* k = static_cast<const uint16_t*>(a.k) + i * a.k_stride;
    const uint16_t* v = static_cast<const uint16_t*>(a.v) + i * a.v_stride;
    uint16_t* kc = static_cast<uint16_t*>(a.k_cache) + dst0;
    uint16_t* vc = static_cast<uint16_t*>(a.v_cache) + dst0;
    for (int e0 = lane; e0 < 2 * row_vecs; e0 += 32 * U) {
      uint4 val[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int e = e0 + u * 32;
        if (e < 2 * row_vecs)
          val[u] = *reinterpret_cast<const uint4*>(e < row_vecs ? k + e * 8
                                                                : v + (e - row_vecs) * 8);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int e = e0 + u * 32;
        if (e < 2 * row_vecs) {
          const int w = e < row_vecs ? e : e - row_vecs;
          const int64_t off = (w / kVec) * a.cache.head_stride + (w % kVec) * 8;
          *reinterpret_cast<uint4*>((e < row_vecs ? kc : vc) + off) = val[u];
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_page_tables(const TablesArgs& a, cudaStream_t stream) {
  const int64_t want = (a.num_slots + kTabThreads - 1) / kTabThreads;
  const int sms = sm_count();
  const int grid = (int)(want < 1 ? 1 : (want < sms ? want : sms));
  page_tables_kernel<<<grid, kTabThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_write(const CacheWriteArgs& a, cudaStream_t stream) {
  const int64_t want = (a.N + 7) / 8, cap = (int64_t)sm_count() * 8;
  const int grid = (int)(want < cap ? want : cap);
  if (a.D == 128)
    cache_write_kernel<128><<<grid, 256, 0, stream>>>(a);
  else
    cache_write_kernel<64><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace cpattn
