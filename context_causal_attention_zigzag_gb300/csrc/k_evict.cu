// Eviction: each request and kv head keeps the heaviest positions of its cache,
// which move as little as possible.  With f, t, cut and keep of the call, M = c - t - f
// positions lie between the first and the last ones and m = cut - f of them stay.
//
// evict_select_kernel, a CTA (long tables: a cluster of them) for each head of a request:
//  1. Each CTA takes a run of those positions, and turns their scores into
//     integers of the same order in shared memory (read again where a run is too
//     long for it).
//  2. The m-th largest is found digit by digit (11, 11 and 10 bits): each CTA
//     counts the digits of its run that begin as the ones found so far; the first
//     one adds the counts up (through distributed shared memory) and finds the digit in
//     which the m-th lies.  Counts are integers: no order of additions matters.
//  3. What is above it stays, and of its equals as many as are left, from the
//     lowest position on.  A thread has which of its positions stay as bits.  Their counts,
//     summed over the CTA and the cluster, number the places below the cut that become free
//     and the positions behind it that stay; both go into lists, so that the n-th place is
//     filled by the n-th position.
// evict_fill_kernel copies the pairs of the lists: a lane looks up a pair's pages and moves
// its weight, then the warp copies the pairs' rows, key and value at once.  Sources lie
// behind the cut and destinations before it, so no order matters.
// evict_shift_kernel moves the last t to the cut, over what the fills have read by then:
// a CTA takes 64 bytes of each row, a wave of rows at a time, read whole before any is
// written (the last ones may move within themselves).  It also lists the pages that
// became free.
//
// Bound by HBM for many positions (scores once, moved rows once in and out), by the
// chain of its steps for few.  Measured, 8 heads of 128 in bfloat16: 1100 positions cut to 990
// in 16.4 us; 16 requests of 1000-8192 to the half in 56 us (172 MB, 25 at the copy rate: the
// longest one's CTA selects for 16, fills for 21, shifts for 14); 131072 to 16384 in 59 us (select
// 25, fill 21 at 5.5 TB/s of rows in and out, shift 5).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cpattn.h"
#include "cpattn_internal.h"
#include "tc_ptx.cuh"

namespace cg = cooperative_groups;

namespace cpattn {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kRun = 16384;  // scores of a CTA's run in shared memory
constexpr int kMaxCluster = 8;
constexpr int kAllLongest = 2048;

struct Shared {
  uint32_t run[kRun];
  int count[kBins];  // of the digits
  int total[kBins];  // the cluster's, in its first CTA
  int meet[4];       // this CTA's counts, read by the others
  int warp[5][kWarps];
  int pick[3][3];    // of each pass
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

__device__ __forceinline__ int warp_sums(int x) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, d);
    if ((threadIdx.x & 31) >= d) x += u;
  }
  return x;
}

// The sum of the warps' values before this warp's; the block's in tot.  `part` is used once.
__device__ __forceinline__ int warps_before(int x, int* part, int& tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) part[warp] = x;
  __syncthreads();
  const int mine = part[lane], upto = warp_sums(mine);
  tot = __shfl_sync(0xffffffffu, upto, 31);
  return __shfl_sync(0xffffffffu, upto - mine, warp);
}

// Runs `chunk`, chunk + chunks, .. of `pairs` (at most 32) of the item's lists, by this warp: a
// lane looks up a pair's pages and moves its weight, the warp copies the rows.
template <int D>
__device__ __forceinline__ void fill_places(const EvictArgs& a, int item, const int* to,
                                            const int* from, int fills, int pairs, int chunk,
                                            int chunks) {
  constexpr int kLanes = D / 4;       // of a pair of rows, 16 bytes each
  constexpr int kRows = 32 / kLanes;  // of a warp at a time
  constexpr int U = 4;                // turns of a set
  const int lane = threadIdx.x & 31, r = item / a.Hkv, g = item % a.Hkv, P = a.cache.page_size;
  const PageDiv div = a.pages;
  const int* table = a.table + (int64_t)r * a.table_stride;
  const int sub = lane / kLanes, l = lane % kLanes;
  // The first half of a pair's lanes copies the key, the second the value.
  uint16_t* base = static_cast<uint16_t*>(l < kLanes / 2 ? a.k_cache : a.v_cache) +
                   g * a.cache.head_stride + l % (kLanes / 2) * 8;
  for (int h0 = chunk * pairs; h0 < fills; h0 += chunks * pairs) {
    const int n = min(pairs, fills - h0);
    int64_t src = 0, dst = 0;
    if (lane < n) {
      const int x = from[h0 + lane], y = to[h0 + lane];
      const int ix = div.page(x), iy = div.page(y), ox = div.place(x, ix), oy = div.place(y, iy);
      const int px = table[ix], py = table[iy];
      a.kept[(int64_t)item * a.most + y] = x;
      a.weights[((int64_t)py * a.Hkv + g) * P + oy] =
          a.weights[((int64_t)px * a.Hkv + g) * P + ox];
      src = px * a.cache.page_stride + ox * a.cache.token_stride;
      dst = py * a.cache.page_stride + oy * a.cache.token_stride;
    }
    // Two sets by turns: one is stored while the other's loads are in flight.
    uint4 v[2][U];
    auto load = [&](uint4 (&v)[U], int j0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * kRows + sub;
        const int64_t at = __shfl_sync(0xffffffffu, src, j & 31);
        if (j < n) v[u] = *reinterpret_cast<const uint4*>(base + at);
      }
    };
    auto store = [&](const uint4 (&v)[U], int j0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * kRows + sub;
        const int64_t at = __shfl_sync(0xffffffffu, dst, j & 31);
        if (j < n) *reinterpret_cast<uint4*>(base + at) = v[u];
      }
    };
    load(v[0], 0);
    for (int j0 = 0; j0 < n; j0 += 2 * U * kRows) {
      load(v[1], j0 + U * kRows);
      store(v[0], j0);
      load(v[0], j0 + 2 * U * kRows);
      store(v[1], j0 + U * kRows);
    }
  }
}

// Vectors [vec0, vec0 + vecs) of 16 bytes of the last rows (key and value side by side; vecs a
// power of two) to the cut, a wave of rows at a time; vector 0 brings their weights.
template <int kCta>
__device__ __forceinline__ void shift_rows(const EvictArgs& a, int item, const Plan& p, int vec0,
                                           int vecs) {
  constexpr int U = 4;
  const int r = item / a.Hkv, g = item % a.Hkv, P = a.cache.page_size;
  const int* table = a.table + (int64_t)r * a.table_stride;
  const int by = p.c - p.keep, tid = threadIdx.x, rows = kCta / vecs;
  const int vec = vec0 + tid % vecs, half = a.D / 8;
  uint16_t* base = static_cast<uint16_t*>(vec < half ? a.k_cache : a.v_cache) +
                   g * a.cache.head_stride + vec % half * 8;
  const PageDiv div = a.pages;
  for (int w0 = p.cut; w0 < p.keep; w0 += U * rows) {
    uint4 v[U];
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int pos = w0 + u * rows + tid / vecs;
      if (pos < p.keep) {
        const int i = div.page(pos + by), o = div.place(pos + by, i), page = table[i];
        v[u] = *reinterpret_cast<const uint4*>(base + page * a.cache.page_stride +
                                               o * a.cache.token_stride);
        if (vec == 0) x[u] = a.weights[((int64_t)page * a.Hkv + g) * P + o];
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int pos = w0 + u * rows + tid / vecs;
      if (pos < p.keep) {
        const int i = div.page(pos), o = div.place(pos, i), page = table[i];
        *reinterpret_cast<uint4*>(base + page * a.cache.page_stride + o * a.cache.token_stride) =
            v[u];
        if (vec == 0) a.weights[((int64_t)page * a.Hkv + g) * P + o] = x[u];
      }
    }
  }
}

// Whether a request's pages can be used, where its positions are brought down.
__device__ __forceinline__ bool pages_ok(const EvictArgs& a, int r, const Plan& p) {
  const int* table = a.table + (int64_t)r * a.table_stride;
  const int n = (p.c + a.cache.page_size - 1) / a.cache.page_size;
  bool ok = true;
#pragma unroll 4
  for (int i = 0; i < n; ++i) ok &= table[i] >= 0 && table[i] < a.cache.num_pages;
  return ok;
}

// The pages that became free, in request order: each of `blocks` blocks sums the requests and
// fills its share of the list.  new_lens: nullptr where they are not written yet.
constexpr int kShiftThreads = 512;

template <int kCta>
__device__ __forceinline__ void list_freed(const EvictArgs& a, int block, int blocks,
                                           const int* new_lens) {
  __shared__ int part[kCta / 32];
  __shared__ int pre[kCta], have[kCta];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P = a.cache.page_size;
  long long done = 0;  // pages of the requests before
  const long long stride = (long long)blocks * kCta;
  const long long mine = (long long)block * kCta + tid;
  for (int r0 = 0; r0 < a.R; r0 += kCta) {
    const int r = r0 + tid;
    int first = 0, n = 0;
    if (r < a.R) {
      const int c = a.ctx[r];
      int k = c;
      if (new_lens != nullptr) {
        k = new_lens[r];
      } else {
        Plan p;
        if (plan_of(a, r, p) && p.keep < p.c && pages_ok(a, r, p)) k = p.keep;
      }
      first = (k + P - 1) / P;
      n = k < c ? (c + P - 1) / P - first : 0;
    }
    int sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += u;
    }
    if (lane == 31) part[warp] = sum;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < kCta / 32; ++w) {
      if (w == warp) before = total;
      total += part[w];
    }
    pre[tid] = before + sum - n;
    have[tid] = first;
    __syncthreads();
    const long long end = done + total < a.num_freed_max ? done + total : a.num_freed_max;
    for (long long x = mine < done ? mine + (done - mine + stride - 1) / stride * stride : mine;
         x < end; x += stride) {
      const int y = (int)(x - done);
      int l = 0, h = kCta;  // the last request that begins at y or before
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

// kAll: a CTA does all for its head; blocks behind those of the heads list the freed pages.
template <bool kAll>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x;
  tc::launch_dependents();
  if (kAll && blockIdx.x == (unsigned)(a.R * a.Hkv)) {
    list_freed<kThreads>(a, 0, 1, nullptr);
    return;
  }
  const int item = blockIdx.x / C, r = item / a.Hkv, g = item % a.Hkv;
  const int P = a.cache.page_size;
  const int* table = a.table + (int64_t)r * a.table_stride;
  int* kept = a.kept + ((int64_t)r * a.Hkv + g) * a.most;
  const int everyone = C * kThreads, me = rank * kThreads + tid;
  auto together = [&]() {
    if (C > 1)
      cluster.sync();
    else
      __syncthreads();
  };
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
    if (rank == 0 && tid == 0) a.fills[item] = -1;  // nothing moves
    for (int i = me; i < a.most; i += everyone) kept[i] = i < p.c ? i : -1;
    return;
  }
  // (The fills put in what comes from elsewhere.)
  for (int i = me; i < a.most; i += everyone)
    kept[i] = i < p.cut ? i : (i < p.keep ? i + (p.c - p.keep) : -1);

  // The run of positions [lo, lo + n) of this CTA.
  const int M = p.c - p.t - p.f, m = p.cut - p.f;
  const int per = (M + C - 1) / C;
  const int lo = p.f + min(M, rank * per), n = p.f + min(M, (rank + 1) * per) - lo;
  const bool held = per <= kRun;
  const PageDiv div = a.pages;
  auto score = [&](int pos) {
    const int i = div.page(pos);
    return ordered(a.scores[((int64_t)table[i] * a.Hkv + g) * P + div.place(pos, i)]);
  };
  auto key_of = [&](int i) { return held ? s.run[i] : score(lo + i); };
  if (held) {
#pragma unroll 8
    for (int i = tid; i < n; i += kThreads) s.run[i] = score(lo + i);
  }
  for (int i = tid; i < kBins; i += kThreads) s.count[i] = s.total[i] = 0;
  together();

  // The m-th largest, `found` being its leading bits and `left` its rank among those that
  // begin alike.
  uint32_t found = 0;
  int left = m, shift = 32;
  bool plain = true;  // all that begin like `found` stay
  if (m > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10;
      const int above = shift;
      shift -= bits;
      for (int i = tid; i < n; i += kThreads) {
        const uint32_t k = key_of(i);
        if (pass == 0 || k >> above == found)
          atomicAdd(&s.count[k >> shift & ((1u << bits) - 1)], 1);
      }
      __syncthreads();
      int* sums = s.count;
      if (C > 1) {
        int* first = cluster.map_shared_rank(s.total, 0);
        for (int i = tid; i < kBins; i += kThreads)
          if (s.count[i] > 0) atomicAdd(&first[i], s.count[i]);
        cluster.sync();
        sums = s.total;
      }
      if (rank == 0) {
        // Two bins a thread from the highest down.
        const int b = kBins - 1 - 2 * tid, hi = sums[b], lo2 = sums[b - 1];
        const int upto = warp_sums(hi + lo2);
        int all;
        const int before = upto - hi - lo2 +
                           warps_before(__shfl_sync(0xffffffffu, upto, 31), s.warp[pass], all);
        int digit = -1, rest = 0, alike = 0;
        if (before < left && left <= before + hi) {
          digit = b;
          rest = left - before;
          alike = hi;
        } else if (before + hi < left && left <= before + hi + lo2) {
          digit = b - 1;
          rest = left - before - hi;
          alike = lo2;
        }
        if (digit >= 0)
          for (int c = 0; c < C; ++c) {
            int* pick = C > 1 ? cluster.map_shared_rank(s.pick[pass], c) : s.pick[pass];
            pick[0] = digit;
            pick[1] = rest;
            pick[2] = rest == alike;
          }
        __syncthreads();
        if (C > 1)
          for (int i = tid; i < kBins; i += kThreads) s.total[i] = 0;
      }
      if (C > 1) cluster.sync();
      for (int i = tid; i < kBins; i += kThreads) s.count[i] = 0;
      found = found << bits | (uint32_t)s.pick[pass][0];
      left = s.pick[pass][1];
      plain = s.pick[pass][2];
      __syncthreads();
      if (plain) break;
    }
  }
  // Of those whose leading bits equal `found` the first `left` stay: how many of them are in
  // this run, by the runs before.
  const int lane = tid & 31, warp = tid >> 5;
  const bool some = m > 0;
  auto lead_of = [&](uint32_t key) { return shift < 32 ? key >> shift : 0u; };
  int quota = left;
  if (C > 1 && !plain) {
    int equal = 0, all;
    for (int i = tid; i < n; i += kThreads) equal += lead_of(key_of(i)) == found;
    const int upto = warp_sums(equal);
    warps_before(__shfl_sync(0xffffffffu, upto, 31), s.warp[3], all);
    if (tid == 0) s.meet[0] = all;
    cluster.sync();
    for (int c = 0; c < rank; ++c) quota -= *cluster.map_shared_rank(&s.meet[0], c);
  }
  // The run in windows of what shared memory holds (one, unless a run is too long for it).  A
  // thread takes q positions of a window, q odd for the banks, as bits: which of them become free
  // below the cut, and which stay behind it; the block's counts of both in one word, before this
  // thread and in all.
  uint32_t free_ = 0, go = 0;
  int first = 0, before = 0, all = 0, seen = 0;
  auto window = [&](int w0) {
    const int len = min(kRun, n - w0), q = (len + kThreads - 1) / kThreads | 1;
    if (!held) {
      __syncthreads();  // the window before has been read
#pragma unroll 4
      for (int i = tid; i < len; i += kThreads) s.run[i] = score(lo + w0 + i);
      __syncthreads();
    }
    const int i0 = min(len, tid * q), mine = min(len, i0 + q) - i0;
    uint32_t above = 0, same = 0;
    for (int j = 0; j < mine; ++j) {
      const uint32_t k = lead_of(s.run[i0 + j]);
      above |= (uint32_t)(k > found) << j;
      same |= (uint32_t)(k == found) << j;
    }
    if (!plain) {  // the lowest of the block's equals, as far as the quota goes
      int tot;
      const int upto = warp_sums(__popc(same));
      const int base = warps_before(__shfl_sync(0xffffffffu, upto, 31), s.warp[3], tot);
      int over = min(__popc(same), max(0, seen + base + upto - quota));
      for (; over > 0; --over) same &= ~(0x80000000u >> __clz(same));
      seen += tot;
    }
    const uint32_t stay = some ? above | same : 0, live = (1u << mine) - 1;
    first = lo + w0 + i0;
    const int e = min(mine, max(0, p.cut - first));
    const uint32_t early = (1u << e) - 1;
    free_ = early & ~stay;
    go = stay & live & ~early;
    const int x = __popc(free_) | __popc(go) << 16, upto = warp_sums(x);
    before = upto - x + warps_before(__shfl_sync(0xffffffffu, upto, 31), s.warp[4], all);
  };
  int holes = 0, late = 0;
  for (int w0 = 0; w0 == 0 || w0 < n; w0 += kRun) {
    window(w0);
    holes += all & 0xffff;
    late += all >> 16;
  }
  int hole0 = 0, late0 = 0, fills = holes;
  if (C > 1) {
    if (tid == 0) {
      s.meet[1] = holes;
      s.meet[2] = late;
    }
    cluster.sync();
    fills = 0;
    for (int c = 0; c < C; ++c) {
      const int h = cluster.map_shared_rank(s.meet, c)[1], l = cluster.map_shared_rank(s.meet, c)[2];
      if (c < rank) {
        hole0 += h;
        late0 += l;
      }
      fills += h;
    }
  }
  if (rank == 0 && tid == 0) a.fills[item] = fills;
  // A window's lists take the scores' place; where other kernels read them they go out from
  // there (straight from the bits a CTA of 14000 free places took 7 us).
  int* const free_list = reinterpret_cast<int*>(s.run);
  int* const go_list = free_list + (kAll ? kRun / 2 : 0);  // (neither is longer than half of a run)
  seen = 0;
  for (int w0 = 0; w0 == 0 || w0 < n; w0 += kRun) {
    if (!held) window(w0);
    const int frees = all & 0xffff, goes = all >> 16;
    int h = before & 0xffff, l = (before >> 16) + (kAll ? 0 : frees);
    for (; free_ != 0; free_ &= free_ - 1) free_list[h++] = first + __ffs(free_) - 1;
    for (; go != 0; go &= go - 1) go_list[l++] = first + __ffs(go) - 1;
    if constexpr (!kAll) {
      int* to = a.lists + 2 * (int64_t)item * a.list_cap;
      int* from = to + a.list_cap + late0;
      to += hole0;
      __syncthreads();
      for (int i = tid; i < frees; i += kThreads) to[i] = free_list[i];
      for (int i = tid; i < goes; i += kThreads) from[i] = go_list[frees + i];
      hole0 += frees;
      late0 += goes;
    }
  }
  if (C > 1) cluster.sync();  // no CTA leaves while another reads its shared memory
  if constexpr (kAll) {
    __syncthreads();
    const int pairs = min(32, max(4, (fills + kWarps - 1) / kWarps));
    if (a.D == 128)
      fill_places<128>(a, item, free_list, go_list, fills, pairs, warp, kWarps);
    else
      fill_places<64>(a, item, free_list, go_list, fills, pairs, warp, kWarps);
    __syncthreads();  // the fills have read what the shift writes over
    shift_rows<kThreads>(a, item, p, 0, a.D / 4);
  }
}

// ---------------------------------------------------------------------------
// Blocks (part, item): a warp takes 32 pairs of the item's lists at a time.
// ---------------------------------------------------------------------------
constexpr int kFillWarps = 4;
// Pairs a warp looks up at a time, all their rows in flight at once (4 requests of 4000, half
// kept: 19 us, with 32 pairs 22; 131072 positions take the same either way).
constexpr int kFillPairs = 8;

template <int D>
__global__ void __launch_bounds__(kFillWarps * 32, 8) evict_fill_kernel(const EvictArgs a) {
  tc::launch_dependents();
  tc::wait_prior_grid();
  const int item = a.item0 + blockIdx.y;
  const int* to = a.lists + 2 * (int64_t)item * a.list_cap;
  fill_places<D>(a, item, to, to + a.list_cap, a.fills[item], kFillPairs,
                 blockIdx.x * kFillWarps + (threadIdx.x >> 5), gridDim.x * kFillWarps);
}

// ---------------------------------------------------------------------------
// Blocks (slice, item): 64 bytes of each of the last rows (slice 0 their weights, too).
// The blocks behind those list the pages that became free.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kShiftThreads)
    evict_shift_kernel(const EvictArgs a, int slices, int freed_blocks) {
  tc::wait_prior_grid();
  const int64_t shifts = (int64_t)a.R * a.Hkv * slices;
  if (blockIdx.x >= shifts) {
    list_freed<kShiftThreads>(a, (int)(blockIdx.x - shifts), freed_blocks, a.new_lens);
    return;
  }
  const int item = blockIdx.x / slices, slice = blockIdx.x % slices;
  if (a.fills[item] < 0) return;
  Plan p;
  plan_of(a, item / a.Hkv, p);
  shift_rows<kShiftThreads>(a, item, p, slice * 4, 4);
}

// A launch that may begin while the one before it ends.
template <typename... Args>
cudaError_t launch_behind(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t stream,
                          Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  static DeviceOnce allowed;
  e = allowed.shared_memory(reinterpret_cast<const void*>(evict_select_kernel<false>), dev, sizeof(Shared));
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)a.R * a.Hkv, longest = (int64_t)a.width * a.cache.page_size;
  const int freed_blocks = a.num_freed_max / (8 * kShiftThreads) < sms
                               ? a.num_freed_max / (8 * kShiftThreads) + 1
                               : sms;
  // A CTA a head does all where the heads fill the SMs, or where that is so little that the host
  // (5 us more for three launches than for one) decides.  Measured (us on the device, one launch /
  // three; 8 heads a request, keys and values of 128, half kept of):
  //    1 request of 1000: 14 / 12    1 of 2000: 17 / 14     1 of 4000: 28 / 16
  //    8 requests of 1000: 15 / 16   8 of 4000: 27 / 25     8 of 8000: 49 / 47
  //   12 requests of 1000: 15 / 19  12 of 4000: 32 / 38    12 of 8000: 57 / 63
  if (items > 0 && longest <= kRun && (longest <= kAllLongest || 2 * items >= sms)) {
    static DeviceOnce all_allowed;
    e = all_allowed.shared_memory(reinterpret_cast<const void*>(evict_select_kernel<true>), dev,
                                  sizeof(Shared));
    if (e != cudaSuccess) return e;
    // The block that lists the freed pages looks at the tables itself, if they are few.
    const bool with_freed = (int64_t)a.R * a.width <= 8192 && a.width <= 128;
    evict_select_kernel<true>
        <<<(unsigned)(items + with_freed), kThreads, sizeof(Shared), stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || with_freed) return e;
    return launch_behind(evict_shift_kernel, dim3(freed_blocks), kShiftThreads, stream, a, 0,
                         freed_blocks);
  }
  const int slices = a.D * 4 / 64;
  if (items > 0) {
    // A CTA whose shared memory holds the scores that a request can have, or a cluster; a wider
    // one where it finds room at once.  Measured (us, clusters of 1, 2, 4 and 8; 8 heads a request):
    //   1 request of  8000: 20, 22, 20, 20     4 requests of  8000: 25, 27, 26, 47
    //   1 request of 16000: 28, 26, 21, 22     4 requests of 16000: 51, 49, 47, 70
    //   1 request of 32000: 65, 35, 30, 29     2 requests of 32000: 92, 55, 49, 62
    int C = 1;
    if (longest > kRun / 2 && 4 * items <= sms) C = 4;
    if (longest > kRun * 2 && 16 * items <= sms) C = 8;
    while (C < kMaxCluster && C * (int64_t)kRun < longest) C *= 2;
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
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel<false>, a);
    if (e != cudaSuccess) return e;
    // Warps for all the pairs that there can be, as far as the SMs can hold them.
    const int64_t pairs = (a.list_cap + kFillWarps * kFillPairs - 1) / (kFillWarps * kFillPairs);
    int64_t parts = (int64_t)sms * 16 / items + 1;
    if (parts > pairs) parts = pairs > 0 ? pairs : 1;
    // (65535 blocks in y at most.)
    for (int64_t i0 = 0; i0 < items; i0 += 65535) {
      EvictArgs b = a;
      const int64_t n = items - i0 < 65535 ? items - i0 : 65535;
      b.item0 = (int)i0;
      const dim3 grid((unsigned)parts, (unsigned)n);
      e = a.D == 128 ? launch_behind(evict_fill_kernel<128>, grid, kFillWarps * 32, stream, b)
                     : launch_behind(evict_fill_kernel<64>, grid, kFillWarps * 32, stream, b);
      if (e != cudaSuccess) return e;
    }
  }
  return launch_behind(evict_shift_kernel, dim3((unsigned)(items * slices + freed_blocks)),
                       kShiftThreads, stream, a, slices, freed_blocks);
}

}  // namespace cpattn
