// Eviction: each request and kv head keeps the heaviest positions of its cache,
// which move as little as possible.
//
// A cluster of CTAs takes one kv head of one request.  With f, t, cut and keep of
// the call, M = c - t - f positions lie between the first and the last ones and m
// = cut - f of them stay:
//  1. Each CTA takes a run of those positions, and turns their scores into
//     integers of the same order in shared memory (read again where a run is too
//     long for it).
//  2. The m-th largest is found digit by digit (11, 11 and 10 bits): each CTA
//     counts the digits of its run that begin as the ones found so far, and all of
//     them add up the cluster's counts through distributed shared memory and take
//     the digit in which the m-th lies.  Counts are integers: nothing depends on
//     the order of additions.
//  3. What is above it stays, and of its equals as many as are left, from the
//     lowest position on.  Counts of a thread's positions, summed over the CTA and
//     the cluster, number the places below the cut that become free and the
//     positions behind it that stay; both go into lists, so that the n-th place is
//     filled by the n-th position.
//  4. The pairs of the lists are copied, a warp a pair (key and value at once);
//     sources lie behind the cut and destinations before it, so no order matters.
//  5. The last t move to the cut, a wave at a time: all CTAs read the wave into
//     registers, meet, and write it.
// Bound by HBM for long caches (scores once, moved rows once in and out); for short
// ones by its chain of meetings.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "cpattn.h"
#include "cpattn_internal.h"

namespace cg = cooperative_groups;

namespace cpattn {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kRun = 16384;  // scores of a CTA's run in shared memory
constexpr int kMaxCluster = 8;

struct Shared {
  uint32_t run[kRun];
  int count[2][kBins];  // of the digits, by turns
  int meet[4];          // this CTA's counts, read by the others
  int warp[2][kWarps];
  int pick[2];
};

// Integers in the order of the scores: NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t ordered(float s) {
  if (s != s) return 0;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// What a call asks of one request, the same for all its heads; false if it is broken.
struct Plan {
  int c, keep, f, t, cut;
};
__device__ __forceinline__ bool plan_of(const EvictArgs& a, int r, Plan& p) {
  const int cap = a.width * a.cache.page_size;
  const int c = a.ctx[r], keep = a.keep[r];
  p.c = c < 0 ? 0 : (c > cap ? cap : c);
  p.keep = p.c;
  p.f = p.t = 0;
  p.cut = p.c;
  if (c < 0 || c > cap || keep < 0 || min(c, keep) > a.most) return false;
  if (keep >= c) return true;
  p.keep = keep;
  p.f = min(a.first, keep);
  p.t = min(a.recent, keep - p.f);
  p.cut = keep - p.t;
  return true;
}

// Exclusive sums of two values over the block; the block's in tot.
__device__ __forceinline__ void block_sums(int& x, int& y, int (*part)[kWarps], int& tot_x,
                                           int& tot_y) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int u = x, v = y;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int p = __shfl_up_sync(0xffffffffu, u, d), q = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) {
      u += p;
      v += q;
    }
  }
  __syncthreads();  // the sums before are read
  if (lane == 31) {
    part[0][warp] = u;
    part[1][warp] = v;
  }
  __syncthreads();
  tot_x = tot_y = 0;
  int bx = 0, by = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) {
      bx = tot_x;
      by = tot_y;
    }
    tot_x += part[0][w];
    tot_y += part[1][w];
  }
  x = bx + u - x;
  y = by + v - y;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int item = blockIdx.x / C, r = item / a.Hkv, g = item % a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = a.cache.page_size;
  const int* table = a.table + (int64_t)r * a.table_stride;
  int* kept = a.kept + ((int64_t)r * a.Hkv + g) * a.most;
  const int everyone = C * kThreads, me = rank * kThreads + tid;

  Plan p;
  bool good = plan_of(a, r, p);
  // Every CTA of the request looks at its pages, so that all decide alike.
  if (good && p.keep < p.c) {
    bool bad = false;
    for (int i = tid; i < (p.c + P - 1) / P; i += kThreads) {
      const int page = table[i];
      bad |= page < 0 || page >= a.cache.num_pages;
    }
    good = !__syncthreads_or(bad);
  }
  if (!good) {
    p.keep = p.c;
    if (tid == 0) atomicExch(a.err, kErrBadTables);
  }
  if (g == 0 && rank == 0 && tid == 0) a.new_lens[r] = good ? p.keep : a.ctx[r];
  if (p.keep == p.c) {
    for (int i = me; i < a.most; i += everyone) kept[i] = i < p.c ? i : -1;
    return;
  }
  for (int i = me; i < a.most; i += everyone)
    if (i < p.f || i >= p.cut) kept[i] = i < p.f ? i : (i < p.keep ? i + (p.c - p.keep) : -1);

  // The run of positions [lo, hi) of this CTA.
  const int M = p.c - p.t - p.f, m = p.cut - p.f;
  const int per = (M + C - 1) / C;
  const int lo = p.f + min(M, rank * per), hi = p.f + min(M, (rank + 1) * per), n = hi - lo;
  const bool held = per <= kRun;
  auto score = [&](int pos) {
    const int page = table[pos / P];
    return ordered(a.scores[((int64_t)page * a.Hkv + g) * P + pos % P]);
  };
  auto key_of = [&](int i) { return held ? s.run[i] : score(lo + i); };
  if (held)
    for (int i = tid; i < n; i += kThreads) s.run[i] = score(lo + i);
  for (int i = tid; i < 2 * kBins; i += kThreads) (&s.count[0][0])[i] = 0;
  __syncthreads();

  // The m-th largest, `found` being its leading bits and `left` its rank among those that
  // begin alike.
  uint32_t found = 0;
  int left = m, shift = 32;
  if (m > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10;
      int* count = s.count[pass & 1];
      if (pass == 2) {  // read by all two meetings ago
        for (int i = tid; i < kBins; i += kThreads) count[i] = 0;
        __syncthreads();
      }
      const int above = shift;
      shift -= bits;
      for (int i = tid; i < n; i += kThreads) {
        const uint32_t k = key_of(i);
        if (pass == 0 || k >> above == found)
          atomicAdd(&count[k >> shift & ((1u << bits) - 1)], 1);
      }
      cluster.sync();
      // Four bins a thread from the highest down: thread 0 holds the last ones.
      int mine[kBins / kThreads], sum = 0, none = 0;
#pragma unroll
      for (int j = 0; j < kBins / kThreads; ++j) {
        const int b = kBins - 1 - (tid * (kBins / kThreads) + j);
        mine[j] = 0;
        for (int c = 0; c < C; ++c) mine[j] += cluster.map_shared_rank(count, c)[b];
        sum += mine[j];
      }
      int before = sum, t0, t1;
      block_sums(before, none, s.warp, t0, t1);
      if (before < left && left <= before + sum) {
        int x = before;
#pragma unroll
        for (int j = 0; j < kBins / kThreads; ++j) {
          if (x < left && left <= x + mine[j]) {
            s.pick[0] = kBins - 1 - (tid * (kBins / kThreads) + j);
            s.pick[1] = left - x;
          }
          x += mine[j];
        }
      }
      __syncthreads();
      found = found << bits | (uint32_t)s.pick[0];
      left = s.pick[1];
      __syncthreads();
    }
  }
  // Of the equals of `found` the first `left` stay.  Which are in this run: by the runs before.
  int equal = 0, none = 0, mine_equal, t1;
  const int chunk = (n + kThreads - 1) / kThreads;  // positions a thread, one after another
  const int i0 = min(n, tid * chunk), i1 = min(n, i0 + chunk);
  if (m > 0)
    for (int i = i0; i < i1; ++i) equal += key_of(i) == found;
  int rank_equal = equal;
  block_sums(rank_equal, none, s.warp, mine_equal, t1);
  if (tid == 0) s.meet[0] = mine_equal;
  cluster.sync();
  int quota = left;
  for (int c = 0; c < rank; ++c) quota -= *cluster.map_shared_rank(&s.meet[0], c);
  auto stays = [&](int i, int& nth) {
    const uint32_t k = key_of(i);
    if (k != found) return k > found;
    return nth++ < quota;
  };
  // Places that become free below the cut, and positions that stay behind it.
  int holes = 0, late = 0, nth = rank_equal;
  for (int i = i0; i < i1; ++i) {
    const bool stay = m > 0 && stays(i, nth);
    if (lo + i < p.cut)
      holes += !stay;
    else
      late += stay;
  }
  int all_holes, all_late;
  int hole0 = holes, late0 = late;
  block_sums(hole0, late0, s.warp, all_holes, all_late);
  if (tid == 0) {
    s.meet[1] = all_holes;
    s.meet[2] = all_late;
  }
  cluster.sync();
  int fills = 0;
  for (int c = 0; c < C; ++c) {
    const int h = cluster.map_shared_rank(s.meet, c)[1], l = cluster.map_shared_rank(s.meet, c)[2];
    if (c < rank) {
      hole0 += h;
      late0 += l;
    }
    fills += h;
  }
  int* to = a.lists + 2 * ((int64_t)r * a.Hkv + g) * a.list_cap;
  int* from = to + a.list_cap;
  nth = rank_equal;
  for (int i = i0; i < i1; ++i) {
    const int pos = lo + i;
    const bool stay = m > 0 && stays(i, nth);
    if (pos < p.cut) {
      if (stay)
        kept[pos] = pos;
      else
        to[hole0++] = pos;
    } else if (stay) {
      from[late0++] = pos;
    }
  }
  __threadfence();
  cluster.sync();

  // Copies.  A lane takes 16 bytes of the key (the first lanes of a row) or value.
  const int vecs = a.D / 8, rows = 32 / (2 * vecs);  // of a warp at a time
  const int which = lane % (2 * vecs) / vecs, col = lane % vecs * 8, sub = lane / (2 * vecs);
  uint16_t* base = static_cast<uint16_t*>(which ? a.v_cache : a.k_cache) +
                   g * a.cache.head_stride + col;
  auto at = [&](int pos) {
    return base + table[pos / P] * a.cache.page_stride + pos % P * a.cache.token_stride;
  };
  auto weight = [&](int pos) {
    return a.weights + ((int64_t)table[pos / P] * a.Hkv + g) * P + pos % P;
  };
  const bool first = lane % (2 * vecs) == 0;
  constexpr int U = 4;
  const int step = C * kWarps * rows, begin = (rank * kWarps + warp) * rows + sub;
  for (int h0 = begin; h0 < fills; h0 += step * U) {
    uint4 v[U];
    float x[U];
    int dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * step;
      if (h < fills) {
        const int src = __ldcg(from + h);
        dst[u] = __ldcg(to + h);
        v[u] = *reinterpret_cast<const uint4*>(at(src));
        if (first) {
          x[u] = *weight(src);
          kept[dst[u]] = src;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h0 + u * step < fills) {
        *reinterpret_cast<uint4*>(at(dst[u])) = v[u];
        if (first) *weight(dst[u]) = x[u];
      }
  }
  // The last ones: no wave is written before all of it, and what the copies above
  // read from its places, has been read.
  const int shift_by = p.c - p.keep;
  for (int w0 = p.cut; w0 < p.keep; w0 += step * U) {
    uint4 v[U];
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int pos = w0 + begin + u * step;
      if (pos < p.keep) {
        v[u] = *reinterpret_cast<const uint4*>(at(pos + shift_by));
        if (first) x[u] = *weight(pos + shift_by);
      }
    }
    cluster.sync();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int pos = w0 + begin + u * step;
      if (pos < p.keep) {
        *reinterpret_cast<uint4*>(at(pos)) = v[u];
        if (first) *weight(pos) = x[u];
      }
    }
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

// ---------------------------------------------------------------------------
// The pages that became free, in request order.  Each block sums the requests
// and fills its share of the list.
// ---------------------------------------------------------------------------
constexpr int kFreedThreads = 512;

__global__ void __launch_bounds__(kFreedThreads) freed_kernel(const EvictArgs a) {
  __shared__ int part[2][kFreedThreads / 32];
  __shared__ int pre[kFreedThreads], have[kFreedThreads], gone[kFreedThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P = a.cache.page_size;
  long long done = 0;  // pages of the requests before
  const long long stride = (long long)gridDim.x * kFreedThreads;
  const long long mine = (long long)blockIdx.x * kFreedThreads + tid;
  for (int r0 = 0; r0 < a.R; r0 += kFreedThreads) {
    const int r = r0 + tid;
    int first = 0, n = 0;
    if (r < a.R) {
      const int c = a.ctx[r], k = a.new_lens[r];
      first = (k + P - 1) / P;
      n = k < c ? (c + P - 1) / P - first : 0;
    }
    int sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += u;
    }
    if (lane == 31) part[0][warp] = sum;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < kFreedThreads / 32; ++w) {
      if (w == warp) before = total;
      total += part[0][w];
    }
    pre[tid] = before + sum - n;
    have[tid] = first;
    gone[tid] = n;
    __syncthreads();
    const long long end = done + total < a.num_freed_max ? done + total : a.num_freed_max;
    for (long long x = mine < done ? mine + (done - mine + stride - 1) / stride * stride : mine;
         x < end; x += stride) {
      const int y = (int)(x - done);
      int l = 0, h = kFreedThreads;  // the last request that begins at y or before
      while (h - l > 1) {
        const int mid = (l + h) / 2;
        if (pre[mid] <= y)
          l = mid;
        else
          h = mid;
      }
      a.freed[x] = a.table[(int64_t)(r0 + l) * a.table_stride + have[l] + (y - pre[l])];
    }
    done += total;
    __syncthreads();
  }
  for (long long x = mine < done ? mine + (done - mine + stride - 1) / stride * stride : mine;
       x < a.num_freed_max; x += stride)
    a.freed[x] = -1;
  if (mine == 0) {
    *a.num_freed = (int)(done < a.num_freed_max ? done : a.num_freed_max);
    if (done > a.num_freed_max) atomicExch(a.err, kErrBadTables);
  }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  static DeviceOnce allowed;
  e = allowed.shared_memory(reinterpret_cast<const void*>(evict_kernel), dev, sizeof(Shared));
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)a.R * a.Hkv;
  int C = kMaxCluster;
  while (C > 1 && items * C > 2 * sms) C /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_kernel, a);
  if (e != cudaSuccess) return e;
  const int64_t want = (a.num_freed_max + kFreedThreads - 1) / kFreedThreads;
  const int grid = (int)(want < 1 ? 1 : (want < sms ? want : sms));
  freed_kernel<<<grid, kFreedThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace cpattn
