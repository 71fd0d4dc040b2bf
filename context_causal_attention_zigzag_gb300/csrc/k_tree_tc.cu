// Attention of new tokens over the paged cache on the tensor cores (sm_103a).
//
//   o_i = sum_j p_ij v_j,  p_ij = exp(scale q_i k_j - lse_i)
//
// over the positions j of the row's own request: all that were there before
// the new tokens, and of the new ones those its tree word names.
//
// The call reads each key and value once and multiplies it with the few rows
// that share its kv head (new tokens x query heads of the kv head), so it is
// bound by HBM up to about 100 rows.  Everything follows from that:
//  * The rows that share a kv head are packed into one 128-row tile (token
//    major, 128 / G tokens), which one walk over the cache serves.
//  * The walk is cut without regard to requests: all key tiles (128 positions)
//    of all (request, kv head) items stand in one line, and CTA c of N takes
//    the c-th N-th of it.  Contexts of any lengths keep every SM loading to
//    the end, and a single long one is spread over all of them.  An item that
//    a cut divides leaves float32 partials (normalised O, lse), at most two a
//    CTA, which tree_merge_kernel joins; its launch overlaps this kernel's
//    tail.  The lengths stay on the device: each CTA sums them itself.
//  * TMA brings the pages of a tile, one box a page and 64 columns, into a
//    ring of 160 KB per SM.
//  * The two softmax warpgroups take turns on the key tiles (even, odd), each
//    with its own running maximum, sum and O in TMEM, joined at the end of the
//    piece; so one tile's softmax hides behind the other's products.
//  * More than 128 rows (large trees, parts of prompts): an item has two row
//    tiles, the warpgroups take one each, and each key tile is loaded once for
//    both.
// Pages hold whatever was left in them behind a request's last position:
// scores there are replaced by -inf, and the V rows, which enter the product
// with weight 0, are zeroed in shared memory first (0 * NaN is NaN).  Pages
// that lie wholly behind it are not read.
//
// CTA = 384 threads: warp 0 loads, warp 1 owns TMEM and issues the products
// S_i = Q_i K^T (SS) and O_i += P_i V (TS, P over S in TMEM), warps 4-7 and
// 8-11 are the warpgroups, one thread per row.  TMEM: S0 [0,128) S1 [128,256)
// O0 [256,384) O1 [384,512).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cpattn_internal.h"
#include "tc_ptx.cuh"

namespace cpattn {
namespace {

using namespace tc;

constexpr int kT = 128;  // tile edge (rows, keys)
constexpr int kBoxBytes = kT * 64 * 2;
constexpr int kThreads = 384;
constexpr int kMaxCtas = 160;  // partials are laid out for so many
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kBoxBytes;
  static constexpr int kSlots = D == 128 ? 5 : 10;  // K(x), V(x) take consecutive slots
  static constexpr int kOffQ = 0;                   // two row tiles
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kOffBar = kOffRing + kSlots * kTileBytes;
  static constexpr int kBarQ = 0;
  static constexpr int kBarFull = 1;
  static constexpr int kBarEmpty = kBarFull + kSlots;
  static constexpr int kBarS = kBarEmpty + kSlots;
  static constexpr int kBarP = kBarS + 2;
  static constexpr int kBarO = kBarP + 2;
  static constexpr int kBarMeet = kBarO + 2;  // [2] the warpgroups meet
  static constexpr int kBarDrain = kBarMeet + 2;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffSums = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr int kSmemBytes = kOffSums + 192 + 1024;  // + slack for 1024-B alignment
};

__host__ __device__ constexpr uint32_t col_s(int i) { return 128u * (uint32_t)i; }
__host__ __device__ constexpr uint32_t col_o(int i) { return 256u + 128u * (uint32_t)i; }

// What one request asks for, held to the buffers whatever its lengths say.
struct Req {
  int q0, n;   // its rows of q
  int ctx;     // positions before them
  int total;   // positions in all
};

__device__ __forceinline__ bool load_req(const TreeArgs& a, int r, Req& x) {
  bool ok = packed_rows(a.cu, r, a.N, x.q0, x.n);
  const int ctx = a.ctx[r];
  const int cap = a.width * a.cache.page_size;
  x.ctx = ctx < 0 ? 0 : (ctx > cap ? cap : ctx);
  ok = ok && ctx >= 0 && (long long)ctx + x.n <= cap && (a.tree == nullptr || x.n <= 64);
  x.total = (int)((long long)x.ctx + x.n < cap ? (long long)x.ctx + x.n : cap);
  return ok;
}

// An item is a kv head of a request and up to two row tiles of `tpt` tokens.
__device__ __forceinline__ int items_of(const Req& x, int tpt) {
  return (x.n + 2 * tpt - 1) / (2 * tpt);
}
// Key tiles of the request's m-th item (at least one, so that its rows are
// written); without a tree no row sees behind the item's last token.
__device__ __forceinline__ int tiles_of(const Req& x, int tpt, bool chain, int m) {
  const int last = min(x.n, (m + 1) * 2 * tpt);
  const int end = chain ? min(x.total, x.ctx + last) : x.total;
  return end > 0 ? (end + kT - 1) / kT : 1;
}
__device__ __forceinline__ long long head_tiles(const Req& x, int tpt, bool chain) {
  long long s = 0;
  for (int m = 0, e = items_of(x, tpt); m < e; ++m) s += tiles_of(x, tpt, chain, m);
  return s;
}

// Where the c-th CTA's part of T tiles begins, and whose a tile is.
__device__ __forceinline__ long long part_begin(long long c, long long T, int n) {
  return c * T / n;
}
__device__ __forceinline__ int part_of(long long t, long long T, int n) {
  return (int)(((t + 1) * n - 1) / T);
}

// A run of key tiles [t0, t1) of one item.
struct Piece {
  Req x;
  int r, g, m, t0, t1, tiles;
  long long at;  // the line's index of tile t0
  bool pair;     // two row tiles
};

// Walks the pieces of one CTA.
struct Walk {
  Piece p;
  long long left;
  int off;  // tile within the item
  int items;

  __device__ __forceinline__ void init(const TreeArgs& a, int tpt, int r, long long in_req,
                                       long long at, long long n) {
    p.r = r;
    p.at = at;
    left = n;
    if (left <= 0) return;
    load_req(a, r, p.x);
    items = items_of(p.x, tpt);
    const long long per = head_tiles(p.x, tpt, a.tree == nullptr);
    p.g = (int)(in_req / per);
    long long rest = in_req - p.g * per;
    p.m = 0;
    while (true) {
      const int t = tiles_of(p.x, tpt, a.tree == nullptr, p.m);
      if (rest < t) break;
      rest -= t;
      ++p.m;
    }
    off = (int)rest;
    p.t1 = off;
    p.tiles = 0;  // the first call of next() stays on this item
  }
  __device__ __forceinline__ bool next(const TreeArgs& a, int tpt) {
    if (left <= 0) return false;
    if (p.tiles != 0 && p.t1 == p.tiles) {
      off = 0;
      if (++p.m == items) {
        p.m = 0;
        if (++p.g == a.Hkv) {
          p.g = 0;
          do {
            ++p.r;
            load_req(a, p.r, p.x);
          } while (p.x.n == 0);
          items = items_of(p.x, tpt);
        }
      }
    }
    p.tiles = tiles_of(p.x, tpt, a.tree == nullptr, p.m);
    p.t0 = off;
    const int n = (int)(left < p.tiles - off ? left : p.tiles - off);
    p.t1 = off + n;
    p.pair = p.x.n - p.m * 2 * tpt > tpt;
    left -= n;
    return true;
  }
  __device__ __forceinline__ void done() { p.at += p.t1 - p.t0; }
};

// The partials: per CTA two places (0: of an item begun by an earlier CTA, 1:
// of one that goes on in the next), each `rows` rows of O [D] and lse; and per
// CTA a record of the item begun there and cut.
struct Cut {
  int last;    // CTA that holds the item's end; -1: nothing was cut here
  int token0;  // the item's first row of q
  int n;       // its tokens
  int g;
};
struct Partials {
  Cut* cuts;
  float* lse;  // [kMaxCtas][2][rows], in log2
  float* o;    // [kMaxCtas][2][rows][D]
  int rows;    // rows of a place: those of an item, tile by tile
};

__host__ __device__ inline int64_t place_of(const Partials& w, int cta, int which, int row) {
  return ((int64_t)cta * 2 + which) * w.rows + row;
}

// The 128 columns that a row sees of the key tile at position k0, as a bit mask.
// Positions below ctx are seen; of the new ones those in `bits` (bit j: the
// j-th), or without a tree the first `upto` of them.
__device__ __forceinline__ void seen_columns(uint32_t* vis, int k0, int ctx, bool chain,
                                             unsigned long long bits, int upto) {
  typedef unsigned __int128 u128;
  const u128 ones = ~(u128)0;
  const int sf = (chain ? ctx + upto : ctx) - k0;  // columns below: seen
  u128 v = sf >= kT ? ones : (sf <= 0 ? (u128)0 : (((u128)1 << sf) - 1));
  if (!chain) {
    if (sf >= 0 && sf < kT) v |= (u128)bits << sf;
    if (sf < 0 && sf > -64) v |= (u128)(bits >> -sf);
  }
  vis[0] = (uint32_t)v;
  vis[1] = (uint32_t)(v >> 32);
  vis[2] = (uint32_t)(v >> 64);
  vis[3] = (uint32_t)(v >> 96);
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const TreeArgs a, const Partials w) {
  using C = Cfg<D>;
  constexpr int kSlots = C::kSlots;
  constexpr uint32_t kIdescQK = idesc_f16(kBf16, 128, 128, false, false);
  constexpr uint32_t kIdescPV = idesc_f16(kBf16, 128, D, false, true);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t sQ = base + C::kOffQ, sRing = base + C::kOffRing;
  const uint32_t bars = base + C::kOffBar;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  long long* sums = reinterpret_cast<long long*>(smem + C::kOffSums);  // [12] warps, T, in_req, r

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{abort_flag, a.err};
  const int G = a.H / a.Hkv, tpt = kT / G;
  const bool chain = a.tree == nullptr;

  launch_dependents();  // the merge sets itself up; it waits for this kernel's end
  if (threadIdx.x == 0) {
    mbar_init(bar(C::kBarQ), 256);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar(C::kBarFull + s), 1);
      mbar_init(bar(C::kBarEmpty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kBarS + i), 1);
      mbar_init(bar(C::kBarP + i), 128);
      mbar_init(bar(C::kBarO + i), 1);
      mbar_init(bar(C::kBarMeet + i), 256);
    }
    mbar_init(bar(C::kBarDrain), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // Where this CTA's part of the line begins: each thread sums a run of
  // requests, the block sums the threads, and the thread whose run holds the
  // beginning finds the request.
  const int per = (a.R + kThreads - 1) / kThreads;
  const int r_lo = min(a.R, (int)threadIdx.x * per), r_hi = min(a.R, r_lo + per);
  long long own = 0;
  bool bad = false;
  for (int r = r_lo; r < r_hi; ++r) {
    Req x;
    bad |= !load_req(a, r, x);
    own += head_tiles(x, tpt, chain) * a.Hkv;
  }
  if (bad && blockIdx.x == 0) atomicExch(a.err, kErrBadTables);
  long long upto = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += u;
  }
  if (lane == 31) sums[warp] = upto;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long T = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i == warp) upto += T;
    T += sums[i];
  }
  const int n_ctas = (int)(T < (long long)gridDim.x ? T : (long long)gridDim.x);
  const int cta = blockIdx.x;
  long long begin = 0, count = 0;
  if (cta < n_ctas) {
    begin = part_begin(cta, T, n_ctas);
    count = part_begin(cta + 1, T, n_ctas) - begin;
    if (begin >= upto - own && begin < upto) {
      long long at = upto - own;
      for (int r = r_lo; r < r_hi; ++r) {
        Req x;
        load_req(a, r, x);
        const long long t = head_tiles(x, tpt, chain) * a.Hkv;
        if (begin < at + t) {
          sums[13] = begin - at;
          sums[14] = r;
          break;
        }
        at += t;
      }
    }
  }
  if (threadIdx.x == 0) w.cuts[cta].last = -1;
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  Walk walk;
  walk.init(a, tpt, (int)sums[14], sums[13], begin, count);
  Piece& p = walk.p;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA
    // All lanes hold page numbers (a window of 32 pages, the next one fetched
    // ahead) and issue the copies of a tile between them.
    const int P = a.cache.page_size;
    const int box = P < kT ? P : kT;      // rows of a copy
    const int ppt = kT / box;             // copies of a tile and 64 columns
    const int npages = (int)a.cache.num_pages;
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    auto wwait = [&](uint32_t bar_addr, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar_addr, parity, wc));
    };
    uint32_t seq = 0, armed[kSlots] = {0};
    bool ok = true;
    while (ok && walk.next(a, tpt)) {
      const int* table = a.table + (int64_t)p.r * a.table_stride;
      const int used = (p.x.total + P - 1) / P;  // pages that hold positions
      auto page_at = [&](int i) { return i < used ? table[i] : 0; };
      int win = p.t0 * kT / P;
      int now = page_at(win + lane), ahead = page_at(win + 32 + lane);
      for (int t = p.t0; ok && t < p.t1; ++t) {
        const int first = t * kT / P;
        if (first + ppt > win + 32) {
          // ppt divides 32 and the window began on a tile, so it ends on one.
          win += 32;
          now = ahead;
          ahead = page_at(win + 32 + lane);
        }
        // Lane c * halves + half issues copy c of the tile, columns 64 * half.
        const int c = lane / C::kHalves, half = lane % C::kHalves;
        const int id = __shfl_sync(0xffffffffu, now, (first - win + (c < ppt ? c : 0)) & 31);
        const bool mine = c < ppt && first + c < used;
        const bool good = mine && id >= 0 && id < npages;
        if (mine && !good) atomicExch(a.err, kErrBadTables);
        const uint32_t copies = __popc(__ballot_sync(0xffffffffu, good));
        const int row = (t * kT) % P;  // within the page (0 for pages up to a tile)
        for (int which = 0; which < 2; ++which) {  // K(t), then V(t)
          const uint32_t n = seq++;
          const int sl = n % kSlots;
          if (!wwait(bar(C::kBarEmpty + sl), ((n / kSlots) & 1) ^ 1)) {
            ok = false;
            break;
          }
          ++armed[sl];
          if (lane == 0) mbar_arrive_expect_tx(bar(C::kBarFull + sl), copies * box * 128);
          __syncwarp();
          if (good)
            tma_load_4d(sRing + sl * C::kTileBytes + half * kBoxBytes + c * box * 128,
                        which == 0 ? &tm_k : &tm_v, bar(C::kBarFull + sl), half * 64, p.g, row, id);
        }
      }
      walk.done();
    }
    if (!ok) {
      // Let the copies already issued land before the CTA exits.
      for (int s = 0; s < kSlots; ++s)
        if (armed[s]) mbar_drain(bar(C::kBarFull + s), (armed[s] - 1) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    // Row tile i's s-th product takes key tile s of the piece (two row tiles)
    // or 2 s + i (one row tile, the warpgroups taking turns).
    const bool leader = elect_one();
    auto wwait = [&](uint32_t bar_addr, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar_addr, parity, wc));
    };
    const uint64_t d_q = sdesc_sw128(sQ, 16, 1024);
    const uint64_t d_k = sdesc_sw128(sRing, 16, 1024);
    const uint64_t d_v = sdesc_sw128(sRing, kBoxBytes, 1024);
    auto slot_off = [](uint32_t n) { return (n % kSlots) * (uint32_t)C::kTileBytes; };
    uint32_t kv = 0, p_ph[2] = {0, 0};
    bool ok = true;
    for (int k = 0; ok && walk.next(a, tpt); ++k) {
      if (!wwait(bar(C::kBarQ), k & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool pair = p.pair;
      const int nt = p.t1 - p.t0;
      const int steps[2] = {pair ? nt : (nt + 1) / 2, pair ? nt : nt / 2};
      auto key_entry = [&](int i, int s) {
        return 2 * (kv + (uint32_t)(pair ? s : 2 * s + i));
      };
      auto scores = [&](int i, int s) {  // S_i of step s; K is freed after its last reader
        const uint32_t n = key_entry(i, s);
        if (!wwait(bar(C::kBarFull + n % kSlots), (n / kSlots) & 1)) return false;
        tc_fence_after();
        if (leader) {
          const uint64_t a0 = sdesc_advance(d_q, pair ? i * C::kTileBytes : 0);
          const uint64_t b0 = sdesc_advance(d_k, slot_off(n));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kBoxBytes + (kk & 3) * 32;
            mma_ss(tmem + col_s(i), sdesc_advance(a0, off), sdesc_advance(b0, off), kIdescQK,
                   kk > 0);
          }
          mma_commit(bar(C::kBarS + i));
          if (!pair || i == 1) mma_commit(bar(C::kBarEmpty + n % kSlots));
        }
        return true;
      };
      for (int i = 0; ok && i < 2; ++i)
        if (steps[i] > 0) ok = scores(i, 0);
      for (int s = 0; ok && s < steps[0]; ++s) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!ok || s >= steps[i]) continue;
          const uint32_t n = key_entry(i, s) + 1;
          ok = wwait(bar(C::kBarFull + n % kSlots), (n / kSlots) & 1) &&
               wwait(bar(C::kBarP + i), p_ph[i]);
          if (!ok) continue;
          p_ph[i] ^= 1;
          tc_fence_after();
          if (leader) {
            const uint64_t bv = sdesc_advance(d_v, slot_off(n));
#pragma unroll
            for (int kk = 0; kk < kT / 16; ++kk)
              mma_ts(tmem + col_o(i), tmem + col_s(i) + kk * 8, sdesc_advance(bv, kk * 2048),
                     kIdescPV, (s > 0) | (kk > 0));
            if (!pair || i == 1) mma_commit(bar(C::kBarEmpty + n % kSlots));
          }
          if (s + 1 < steps[i]) ok = scores(i, s + 1);
        }
      }
      if (!ok) break;
      if (leader) {
        mma_commit(bar(C::kBarO + 0));
        if (steps[1] > 0) mma_commit(bar(C::kBarO + 1));
      }
      kv += nt;
      walk.done();
    }
    if (!ok) {
      // Let every MMA already issued retire before TMEM is released.
      if (leader) mma_commit(bar(C::kBarDrain));
      mbar_drain(bar(C::kBarDrain), 0);
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- softmax
    const int ti = (warp - 4) >> 2;
    const int wq = warp & 3;         // TMEM sub-partition = rows 32*wq ..
    const int row = wq * 32 + lane;  // row within the tile
    const uint32_t tl = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t colS = col_s(ti), colO = col_o(ti);
    const float sl2 = a.scale_log2;
    const int tok = row / G, head = row - tok * G;
    // (m, l) of both warpgroups; in the second row tile's place, which has no
    // use while they share one.
    float2* ml = reinterpret_cast<float2*>(smem + C::kOffQ + C::kTileBytes);
    uint32_t s_ph = 0, o_ph[2] = {0, 0}, kv = 0;
    bool ok = true;
    auto wwait = [&](uint32_t bar_addr, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar_addr, parity, wc));
    };
    for (int k = 0; ok && walk.next(a, tpt); ++k) {
      const bool pair = p.pair;
      const int nt = p.t1 - p.t0;
      const int item_tok = p.m * 2 * tpt;
      const int mine = (pair ? ti * tpt : 0) + tok;  // token within the item
      const int token = item_tok + mine;             // within the request
      const bool live = tok < tpt && token < p.x.n;
      // Q rows: of the shared tile the warpgroups load half the columns each.
      if (live) {
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.q) + (p.x.q0 + token) * a.q_stride + (p.g * G + head) * D);
        uint8_t* dst = smem + C::kOffQ + (pair ? ti * C::kTileBytes : 0) + row * 128;
        constexpr int kHalf = D / 16;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          if (!pair && c / kHalf != ti) continue;
          *reinterpret_cast<uint4*>(dst + (c >> 3) * kBoxBytes + (((c & 7) ^ (row & 7)) << 4)) =
              src[c];
        }
      }
      unsigned long long bits = 0;
      if (!chain && live) {
        bits = a.tree[p.x.q0 + token];
        if (p.x.n < 64) bits &= (1ull << p.x.n) - 1;
      }
      fence_async_shared();
      mbar_arrive(bar(C::kBarQ));
      const bool warp_live = __any_sync(0xffffffffu, live);
      float m = -INFINITY, l = 0.f;
      const int step = pair ? 1 : 2;
      for (int x = pair ? 0 : ti; x < nt; x += step) {
        const int k0 = (p.t0 + x) * kT;
        if (!wwait(bar(C::kBarS + ti), s_ph)) {
          ok = false;
          break;
        }
        s_ph ^= 1;
        tc_fence_after();
        if (warp_live) {
          uint32_t r[128];
          tmem_ld32(tl + colS + 0, r + 0);
          tmem_ld32(tl + colS + 32, r + 32);
          tmem_ld32(tl + colS + 64, r + 64);
          tmem_ld32(tl + colS + 96, r + 96);
          tmem_wait_ld_regs(r);
          reg_fence32(r + 32);
          reg_fence32(r + 64);
          reg_fence32(r + 96);
          if (k0 + kT > p.x.ctx) {
            uint32_t vis[4];
            seen_columns(vis, k0, p.x.ctx, chain, bits, token + 1);
#pragma unroll
            for (int j = 0; j < 128; ++j)
              if (!(vis[j >> 5] >> (j & 31) & 1)) r[j] = __float_as_uint(-INFINITY);
          }
          float mx0 = __uint_as_float(r[0]), mx1 = __uint_as_float(r[1]);
          float mx2 = __uint_as_float(r[2]), mx3 = __uint_as_float(r[3]);
#pragma unroll
          for (int j = 4; j < 128; j += 4) {
            mx0 = fmaxf(mx0, __uint_as_float(r[j]));
            mx1 = fmaxf(mx1, __uint_as_float(r[j + 1]));
            mx2 = fmaxf(mx2, __uint_as_float(r[j + 2]));
            mx3 = fmaxf(mx3, __uint_as_float(r[j + 3]));
          }
          const float m_tile = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * sl2;
          const float m_new = fmaxf(m, m_tile);
          const bool rescale = __any_sync(0xffffffffu, m_new > m + kRescaleThreshold);
          float alpha = 1.f;
          if (rescale) {
            // A row that has seen no key yet keeps m = -inf and alpha = 1.
            alpha = m_new == -INFINITY ? 1.f : ex2(m - m_new);
            l *= alpha;
            m = m_new;
          }
          const float nm = m == -INFINITY ? 0.f : -m;
          float l0 = 0.f, l1 = 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t e[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float a0 = ex2(fmaf(__uint_as_float(r[64 * h + 2 * j]), sl2, nm));
              const float a1 = ex2(fmaf(__uint_as_float(r[64 * h + 2 * j + 1]), sl2, nm));
              l0 += a0;
              l1 += a1;
              e[j] = pack16<kBf16>(a0, a1);
            }
            tmem_st32(tl + colS + 32 * h, e);
          }
          l += l0 + l1;
          if (rescale && x >= step) {
            // O <- O * 2^(m_old - m_new).  This tile's S barrier also covers the
            // previous product into O; the next is issued after the P barrier.
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t o[32];
              tmem_ld32(tl + colO + cc * 32, o);
              tmem_wait_ld_regs(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tmem_st32(tl + colO + cc * 32, o);
            }
          }
        }
        const int valid = p.x.total - k0;
        if (valid < kT && (!pair || ti == 0)) {
          // V rows behind the last position.  With two row tiles the first
          // one's warpgroup clears them: the second's product is issued later.
          const uint32_t n = 2 * (kv + x) + 1;
          if (!wwait(bar(C::kBarFull + n % kSlots), (n / kSlots) & 1)) {
            ok = false;
            break;
          }
          if (row >= valid) {
            uint8_t* v = smem + C::kOffRing + (n % kSlots) * C::kTileBytes + row * 128;
#pragma unroll
            for (int half = 0; half < C::kHalves; ++half)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(v + half * kBoxBytes + c * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_shared();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::kBarP + ti));
      }
      if (!ok) break;
      // ------------------------------------------------------------ epilogue
      // o = (f0 O0 + f1 O1) / L: of one row tile each warpgroup joins and
      // writes half the columns, of two its own rows.
      const bool two = !pair && nt > 1;  // both warpgroups hold a part of the row
      float f0, f1 = 0.f, L, M;
      if (!pair) {
        ml[ti * kT + row] = make_float2(m, l);
        mbar_arrive(bar(C::kBarMeet + 0));
        ok = wwait(bar(C::kBarMeet + 0), k & 1) && wwait(bar(C::kBarO + 0), o_ph[0]) &&
             (!two || wwait(bar(C::kBarO + 1), o_ph[1]));
        if (!ok) break;
        o_ph[0] ^= 1;
        if (two) o_ph[1] ^= 1;
        const float2 x0 = ml[row], x1 = ml[kT + row];
        M = fmaxf(x0.x, x1.x);
        f0 = x0.x == -INFINITY ? 0.f : ex2(x0.x - M);
        f1 = x1.x == -INFINITY ? 0.f : ex2(x1.x - M);
        L = x0.y * f0 + x1.y * f1;
      } else {
        mbar_arrive(bar(C::kBarMeet + 0));  // keeps the barriers' phases in step with the pieces
        // Each warpgroup waits for both products, so that both count the phases.
        ok = wwait(bar(C::kBarO + 0), o_ph[0]) && wwait(bar(C::kBarO + 1), o_ph[1]);
        if (!ok) break;
        o_ph[0] ^= 1;
        o_ph[1] ^= 1;
        M = m;
        L = l;
        f0 = 1.f;
      }
      tc_fence_after();
      const float inv = L == 0.f ? 0.f : 1.f / L;  // a row that sees nothing: 0
      f0 *= inv;
      f1 *= inv;
      const float lse2 = L == 0.f ? -INFINITY : M + log2f(L);
      const bool whole = p.t0 == 0 && p.t1 == p.tiles;
      const int which = p.t0 == 0 ? 1 : 0;
      const int64_t place = place_of(w, cta, which, (pair ? ti * tpt * G : 0) + row);
      const int64_t out_row = (int64_t)(p.x.q0 + token) * a.H + p.g * G + head;
      const int c_lo = pair ? 0 : ti * (D / 2), c_hi = pair ? D : c_lo + D / 2;
      if (warp_live) {
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          if (cc * 32 < c_lo || cc * 32 >= c_hi) continue;
          uint32_t o[32];
          tmem_ld32(tl + (pair ? colO : col_o(0)) + cc * 32, o);
          tmem_wait_ld_regs(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f0);
          if (two) {
            uint32_t u[32];
            tmem_ld32(tl + col_o(1) + cc * 32, u);
            tmem_wait_ld_regs(u);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              o[j] = __float_as_uint(fmaf(__uint_as_float(u[j]), f1, __uint_as_float(o[j])));
          }
          if (live && whole) {
            uint4* op = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + out_row * D + cc * 32);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint4 v;
              v.x = pack16<kBf16>(__uint_as_float(o[8 * j + 0]), __uint_as_float(o[8 * j + 1]));
              v.y = pack16<kBf16>(__uint_as_float(o[8 * j + 2]), __uint_as_float(o[8 * j + 3]));
              v.z = pack16<kBf16>(__uint_as_float(o[8 * j + 4]), __uint_as_float(o[8 * j + 5]));
              v.w = pack16<kBf16>(__uint_as_float(o[8 * j + 6]), __uint_as_float(o[8 * j + 7]));
              op[j] = v;
            }
          } else if (live) {
            uint4* op = reinterpret_cast<uint4*>(w.o + place * D + cc * 32);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              op[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
          __syncwarp();
        }
      }
      if (live && (pair || ti == 0)) {
        if (whole)
          a.lse[(int64_t)(p.g * G + head) * a.N + p.x.q0 + token] =
              L == 0.f ? -INFINITY : lse2 * kLn2;
        else
          w.lse[place] = lse2;
      }
      if (!whole && p.t0 == 0 && warp == 4 && lane == 0) {
        Cut c;
        c.last = part_of(p.at + p.tiles - 1, T, n_ctas);
        c.token0 = p.x.q0 + item_tok;
        c.n = min(p.x.n - item_tok, 2 * tpt);
        c.g = p.g;
        w.cuts[cta] = c;
      }
      // The next piece overwrites Q, (m, l) and O: not before both are through.
      tc_fence_before();
      mbar_arrive(bar(C::kBarMeet + 1));
      ok = wwait(bar(C::kBarMeet + 1), k & 1);
      tc_fence_after();
      kv += nt;
      walk.done();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Joins the partials of each item that was cut: with L = log2 sum_c 2^lse_c,
// o = sum_c 2^(lse_c - L) o_c.  Block (c, y) takes rows y, y + gridDim.y, ... of
// the item begun by CTA c; its warps share the row's partials and join theirs
// through shared memory.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 8;

template <bool kBf16, int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const TreeArgs a,
                                                                      const Partials w) {
  constexpr int E = D / 32;
  __shared__ float s_o[kMergeWarps][D], s_m[kMergeWarps], s_l[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.H / a.Hkv;
  wait_prior_grid();
  const int c0 = blockIdx.x;
  const Cut cut = w.cuts[c0];
  if (cut.last <= c0) return;
  const int parts = cut.last - c0 + 1;
  for (int row = blockIdx.y; row < cut.n * G; row += gridDim.y) {
    float m = -INFINITY, l = 0.f, o[E] = {};
    for (int i = warp; i < parts; i += kMergeWarps) {
      const int64_t at = place_of(w, c0 + i, i == 0 ? 1 : 0, row);
      const float x = w.lse[at];
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = w.o[at * D + e * 32 + lane];
      const float mn = fmaxf(m, x);
      const float f = m == -INFINITY ? 0.f : ex2(m - mn), g = x == -INFINITY ? 0.f : ex2(x - mn);
      l = l * f + g;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + v[e] * g;
      m = mn;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][e * 32 + lane] = o[e];
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY;
    for (int i = 0; i < kMergeWarps; ++i) M = fmaxf(M, s_m[i]);
    float L = 0.f, f[kMergeWarps];
#pragma unroll
    for (int i = 0; i < kMergeWarps; ++i) {
      f[i] = s_m[i] == -INFINITY ? 0.f : ex2(s_m[i] - M);
      L += s_l[i] * f[i];
    }
    const int token = cut.token0 + row / G, head = cut.g * G + row % G;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    if (threadIdx.x < D / 2) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int i = 0; i < kMergeWarps; ++i) {
        x += s_o[i][2 * threadIdx.x] * f[i];
        y += s_o[i][2 * threadIdx.x + 1] * f[i];
      }
      reinterpret_cast<uint32_t*>(a.out)[((int64_t)token * a.H + head) * (D / 2) + threadIdx.x] =
          pack16<kBf16>(x * inv, y * inv);
    }
    if (threadIdx.x == 0)
      a.lse[(int64_t)head * a.N + token] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// The cache as a 4-D tensor (d, head, token of the page, page), box 64 columns
// of up to 128 tokens of one page and head.
bool make_map(CUtensorMap* m, const void* ptr, bool bf16, const CacheShape& c, int Hkv, int D) {
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)c.page_size,
                        (cuuint64_t)c.num_pages};
  cuuint64_t strides[3] = {(cuuint64_t)c.head_stride * 2, (cuuint64_t)c.token_stride * 2,
                           (cuuint64_t)c.page_stride * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)(c.page_size < kT ? c.page_size : kT), 1};
  return encode_tiled(m, bf16, 4, ptr, dims, strides, box);
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Rows of a place: an item's, at most two tiles of 128 / G tokens.
int place_rows(int N, int G) {
  const int64_t most = 2 * (int64_t)(kT / G) * G, have = (int64_t)N * G;
  return (int)(have < most ? have : most);
}

template <bool kBf16, int D>
cudaError_t run(const TreeArgs& a, cudaStream_t stream) {
  const int G = a.H / a.Hkv;
  CUtensorMap mk, mv;
  if (!make_map(&mk, a.k_cache, kBf16, a.cache, a.Hkv, D) ||
      !make_map(&mv, a.v_cache, kBf16, a.cache, a.Hkv, D))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int smem = Cfg<D>::kSmemBytes;
  e = cudaFuncSetAttribute(tree_kernel<kBf16, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem);
  if (e != cudaSuccess) return e;
  Partials w;
  w.rows = place_rows(a.N, G);
  char* ws = static_cast<char*>(a.workspace);
  w.cuts = reinterpret_cast<Cut*>(ws);
  ws += align256(kMaxCtas * sizeof(Cut));
  w.lse = reinterpret_cast<float*>(ws);
  ws += align256((size_t)kMaxCtas * 2 * w.rows * sizeof(float));
  w.o = reinterpret_cast<float*>(ws);
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  tree_kernel<kBf16, D><<<grid, kThreads, smem, stream>>>(mk, mv, a, w);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, w.rows < 8 ? w.rows : 8);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<kBf16, D>, a, w);
}

}  // namespace

size_t tree_workspace_bytes(int N, int H, int Hkv, int D) {
  const size_t rows = (size_t)place_rows(N, H / Hkv);
  return align256(kMaxCtas * sizeof(Cut)) +
         align256((size_t)kMaxCtas * 2 * rows * sizeof(float)) +
         align256((size_t)kMaxCtas * 2 * rows * D * sizeof(float));
}

cudaError_t launch_tree_attn(const TreeArgs& a, int dtype, cudaStream_t stream) {
  if (dtype == CPATTN_BF16) return a.D == 128 ? run<true, 128>(a, stream) : run<true, 64>(a, stream);
  return a.D == 128 ? run<false, 128>(a, stream) : run<false, 64>(a, stream);
}

}  // namespace cpattn
