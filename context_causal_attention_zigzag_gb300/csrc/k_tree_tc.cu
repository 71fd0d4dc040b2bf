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
//    A piece also costs its start and its end, so an item counts kItemCost
//    tiles more than it has when the line is cut.
//  * TMA brings the pages of a tile, one box a page and 64 columns, into a
//    ring of 192 KB per SM.
//  * The two softmax warpgroups take turns on the key tiles (even, odd), each
//    with its own running maximum, sum and O in TMEM, joined at the end of the
//    piece; so one tile's softmax hides behind the other's products.
//  * Between pieces nothing stands still: the next piece's pages and Q rows
//    load and its first scores are computed while the last one's epilogue runs.
//  * More than 128 rows (large trees, parts of prompts; kPair): an item has two
//    row tiles, the warpgroups take one each, and each key tile is loaded once
//    for both.
// With packed keys instead of a cache (kPaged false) it answers prompts of few
// rows and many keys.
// Measured (H = 32, Hkv = 8, D = 128): 64 single tokens over 100-8192 cached ones
// 183-188 us (6.0-6.2 TB/s, 90 % of the copy rate), two trees of 6-8 tokens over
// 100000-131072 158-163 us, 16 trees of 5-31 tokens over 500-5000 in pages of
// 16 54 us (3.4 TB/s: half of it start, first loads and merge), one token over 1000
// 13 us.
// Pages hold whatever was left in them behind a request's last position:
// scores there are replaced by -inf, and the V rows, which enter the product
// with weight 0, are zeroed in shared memory first (0 * NaN is NaN).  Pages
// that lie wholly behind it are not read.
//
// CTA = 384 threads: warp 0 loads K and V, warp 2 Q, warp 1 owns TMEM and
// issues the products S_i = Q_i K^T (SS) and O_i += P_i V (TS, P over S in
// TMEM), warps 4-7 and 8-11 are the warpgroups, one thread per row.  TMEM: S0
// [0,128) S1 [128,256) O0 [256,384) O1 [384,512).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "answer_way.h"
#include "cpattn_internal.h"
#include "line_walk.h"
#include "tc_ptx.cuh"

namespace cpattn {
namespace {

using namespace tc;
using namespace line;

constexpr int kT = kTcTile;  // tile edge (rows, keys)
constexpr int kBoxBytes = kT * 64 * 2;
constexpr int kThreads = 384;
constexpr int kMaxCtas = 160;  // partials are laid out for so many
constexpr float kLn2 = 0.6931471805599453f;

template <int D, bool kPair>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kBoxBytes;
  static constexpr int kRowTiles = kPair ? 2 : 1;
  static constexpr int kSlots = (D == 128 ? 1 : 2) * (kPair ? 5 : 6);
  static constexpr int kOffQ = 0;
  static constexpr int kOffRing = kRowTiles * kTileBytes;
  static constexpr int kOffBar = kOffRing + kSlots * kTileBytes;
  static constexpr int kBarQFull = 0;
  static constexpr int kBarQEmpty = 1;
  static constexpr int kBarFull = 2;
  static constexpr int kBarEmpty = kBarFull + kSlots;
  static constexpr int kBarS = kBarEmpty + kSlots;
  static constexpr int kBarP = kBarS + 2;
  static constexpr int kBarO = kBarP + 2;
  static constexpr int kBarMeet = kBarO + 2;  // [2] the warpgroups meet
  static constexpr int kBarDrain = kBarMeet + 2;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  // The prologue's sums; then (m, l) of both warpgroups.
  static constexpr int kOffSums = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr int kSmemBytes = kOffSums + 2 * kT * 8;
};

__host__ __device__ constexpr uint32_t col_s(int i) { return 128u * (uint32_t)i; }
__host__ __device__ constexpr uint32_t col_o(int i) { return 256u + 128u * (uint32_t)i; }

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

// The 128 columns that a row sees of the key tile at position k0, as a bit mask:
// the positions below `limit` and, of those from ctx on, the ones in `bits`.
__device__ __forceinline__ void seen_columns(uint32_t* vis, int k0, int limit, int ctx,
                                             unsigned long long bits) {
  typedef unsigned __int128 u128;
  const int lo = limit - k0, sf = ctx - k0;
  u128 v = lo >= kT ? ~(u128)0 : (lo <= 0 ? (u128)0 : (((u128)1 << lo) - 1));
  if (sf >= 0 && sf < kT) v |= (u128)bits << sf;
  if (sf < 0 && sf > -64) v |= (u128)(bits >> -sf);
  vis[0] = (uint32_t)v;
  vis[1] = (uint32_t)(v >> 32);
  vis[2] = (uint32_t)(v >> 64);
  vis[3] = (uint32_t)(v >> 96);
}

template <bool kBf16, int D, bool kPair, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const TreeArgs a, const Partials w, const int q_box) {
  using C = Cfg<D, kPair>;
  constexpr int kSlots = C::kSlots;
  constexpr uint32_t kIdescQK = idesc_f16(kBf16, 128, 128, false, false);
  constexpr uint32_t kIdescPV = idesc_f16(kBf16, 128, D, false, true);
  extern __shared__ __align__(1024) uint8_t smem[];
  // The compiler is kept from folding the address into every operand descriptor:
  // with the descriptors as immediates the issuing warp is 2 % slower.
  const uint32_t base = opaque(smem_u32(smem));
  if (base & 1023u) {  // the swizzled tiles need it; shared memory has no room for slack
    if (threadIdx.x == 0) {
      atomicExch(a.err, kErrLaunch);
      w.cuts[blockIdx.x].last = -1;
    }
    return;
  }
  const uint32_t sQ = base + C::kOffQ, sRing = base + C::kOffRing;
  const uint32_t bars = base + C::kOffBar;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  // [12] of the warps; then where this CTA begins: in_req, r and the request.
  long long* sums = reinterpret_cast<long long*>(smem + C::kOffSums);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{abort_flag, a.err};
  const int G = a.H / a.Hkv, tpt = kT / G, span = tpt * C::kRowTiles;
  const bool chain = a.tree == nullptr;

  launch_dependents();  // the merge sets itself up; it waits for this kernel's end
  if (threadIdx.x == 0) {
    mbar_init(bar(C::kBarQFull), 1);
    mbar_init(bar(C::kBarQEmpty), 1);
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
  // beginning finds the request.  Lengths that break the rules could name the
  // same rows over and over: nothing is computed then.
  const int per = (a.R + kThreads - 1) / kThreads;
  const int r_lo = min(a.R, (int)threadIdx.x * per), r_hi = min(a.R, r_lo + per);
  long long own = 0;
  bool bad = false;
  Req x;
  for (int r = r_lo; r < r_hi; ++r) bad |= !load_line_req<kPaged>(a, r, x);
  if (bad && blockIdx.x == 0) atomicExch(a.err, kErrBadTables);
  if (!__syncthreads_or(bad)) {
    for (int r = r_lo; r < r_hi; ++r) {
      if (per > 1) load_line_req<kPaged>(a, r, x);
      own += head_cost(x, span, chain) * a.Hkv;
    }
  }
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
  const long long parts = (T + kMinPart - 1) / kMinPart;
  const int n_ctas = (int)(parts < (long long)gridDim.x ? parts : (long long)gridDim.x);
  const int cta = blockIdx.x;
  Cuts cuts;
  cuts.init(T, n_ctas);
  long long begin = 0, count = 0;
  if (cta < n_ctas) {
    begin = cuts.begin(cta);
    count = cuts.begin(cta + 1) - begin;
    if (begin >= upto - own && begin < upto) {
      long long at = upto - own;
      int r = r_lo;
      while (per > 1) {
        load_line_req<kPaged>(a, r, x);
        const long long t = head_cost(x, span, chain) * a.Hkv;
        if (begin < at + t) break;
        at += t;
        ++r;
      }
      sums[13] = begin - at;
      sums[14] = r;
      *reinterpret_cast<Req*>(sums + 16) = x;
    }
  }
  if (threadIdx.x == 0) w.cuts[cta].last = -1;
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  Walk<kPaged> walk;
  walk.init(a, span, (int)sums[14], *reinterpret_cast<const Req*>(sums + 16), sums[13], begin,
            count);
  __syncthreads();  // the sums' place is used again
  Piece& p = walk.p;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    auto wwait = [&](uint32_t bar_addr, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait_short(bar_addr, parity, wc));
    };
    uint32_t seq = 0;  // ring entries asked for
    bool ok = true;
    // Fills the next two ring entries, K then V; `copy` issues this lane's share.
    auto fill = [&](uint32_t bytes, auto copy) {
#pragma unroll 1
      for (int which = 0; ok && which < 2; ++which) {
        const uint32_t n = seq;
        const int sl = n % kSlots;
        ok = wwait(bar(C::kBarEmpty + sl), ((n / kSlots) & 1) ^ 1);
        if (!ok) break;
        ++seq;
        if (lane == 0) mbar_arrive_expect_tx(bar(C::kBarFull + sl), bytes);
        __syncwarp();
        copy(which == 0 ? &tm_k : &tm_v, sRing + sl * C::kTileBytes, bar(C::kBarFull + sl));
      }
    };
    if constexpr (!kPaged) {
      while (ok && walk.next(a, span))
        for (int t = p.t0; ok && t < p.t1; ++t)
          fill(C::kTileBytes, [&](const CUtensorMap* map, uint32_t dst, uint32_t full) {
            if (lane < C::kHalves)
              tma_load_3d(dst + lane * kBoxBytes, map, full, lane * 64, p.g, p.x.k0 + t * kT);
          });
    } else {
      // All lanes hold page numbers (a window of 32 pages, the next one fetched
      // ahead) and issue the copies of a tile between them.
      const int P = a.cache.page_size;
      const int box = P < kT ? P : kT;      // rows of a copy
      const int ppt = kT / box;             // copies of a tile and 64 columns
      const int npages = (int)a.cache.num_pages;
      while (ok && walk.next(a, span)) {
        const int* table = a.table + (int64_t)p.r * a.table_stride;
        const int used = (p.x.total + P - 1) / P;  // pages that hold positions
        auto page_at = [&](int i) { return i < used ? table[i] : 0; };
        int win = p.t0 * kT / P;
        int now = page_at(win + lane), ahead = page_at(win + 32 + lane);
        const int c = lane / C::kHalves, half = lane % C::kHalves;
        for (int t = p.t0; ok && t < p.t1; ++t) {
          const int first = t * kT / P;
          if (first + ppt > win + 32) {
            // ppt divides 32 and the window began on a tile, so it ends on one.
            win += 32;
            now = ahead;
            ahead = page_at(win + 32 + lane);
          }
          // Lane c * halves + half issues copy c of the tile, columns 64 * half.
          const int id = __shfl_sync(0xffffffffu, now, (first - win + (c < ppt ? c : 0)) & 31);
          const bool mine = c < ppt && first + c < used;
          const bool good = mine && id >= 0 && id < npages;
          if (mine && !good) atomicExch(a.err, kErrBadTables);
          const uint32_t copies = __popc(__ballot_sync(0xffffffffu, good));
          const int row = (t * kT) % P;  // within the page (0 for pages up to a tile)
          fill(copies * box * 128, [&](const CUtensorMap* map, uint32_t dst, uint32_t full) {
            if (good)
              tma_load_4d(dst + half * kBoxBytes + c * box * 128, map, full, half * 64, p.g, row, id);
          });
        }
      }
    }
    if (!ok) {
      // Let the copies already issued land before the CTA exits.
      for (uint32_t n = seq > (uint32_t)kSlots ? seq - kSlots : 0; n < seq; ++n)
        mbar_drain(bar(C::kBarFull + n % kSlots), (n / kSlots) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    // Stream i's s-th step takes key tile s of the piece (two row tiles) or
    // 2 s + i (one row tile, the warpgroups taking turns).
    const bool leader = elect_one();
    auto wwait = [&](uint32_t bar_addr, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait_short(bar_addr, parity, wc));
    };
    const uint64_t d_q = sdesc_sw128(sQ, 16, 1024);
    const uint64_t d_k = sdesc_sw128(sRing, 16, 1024);
    const uint64_t d_v = sdesc_sw128(sRing, kBoxBytes, 1024);
    auto slot_off = [](uint32_t n) { return (n % kSlots) * (uint32_t)C::kTileBytes; };
    struct Run {
      uint32_t kv;  // ring entries before the piece's
      int nt;
      bool pair;
      __device__ __forceinline__ int steps(int i) const {
        return pair ? nt : (nt + 1 - i) / 2;
      }
    };
    Run cur{0, 0, false}, nxt;
    uint32_t entries = 0, p_ph = 0, q_ph = 0;  // p_ph: bit i
    bool ok = true;
    auto next_run = [&](Run& u) {
      if (!walk.next(a, span)) {
        u.nt = 0;  // no steps
        u.pair = false;
        return false;
      }
      u.kv = entries;
      u.nt = p.t1 - p.t0;
      u.pair = kPair && p.x.n - p.m * span > tpt;
      entries += 2 * u.nt;
      return true;
    };
    // The piece's key tile x has K in ring entry kv + 2 x and V behind it.
    auto key_entry = [&](const Run& u, int i, int s) {
      return u.kv + 2u * (uint32_t)(u.pair ? s : 2 * s + i);
    };
    auto full = [&](uint32_t n) { return wwait(bar(C::kBarFull + n % kSlots), (n / kSlots) & 1); };
    // S_i of step s.  K is freed after its last reader, Q after the piece's last
    // scores.
    auto scores = [&](const Run& u, int i, int s) {
      const uint32_t n = key_entry(u, i, s);
      if (!full(n)) return false;
      tc_fence_after();
      if (leader) {
        const uint64_t a0 = sdesc_advance(d_q, u.pair ? i * C::kTileBytes : 0);
        const uint64_t b0 = sdesc_advance(d_k, slot_off(n));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kBoxBytes + (kk & 3) * 32;
          mma_ss(tmem + col_s(i), sdesc_advance(a0, off), sdesc_advance(b0, off), kIdescQK,
                 kk > 0);
        }
        mma_commit(bar(C::kBarS + i));
        if (!u.pair || i == 1) mma_commit(bar(C::kBarEmpty + n % kSlots));
        if (u.pair ? i == 1 && s + 1 == u.nt : 2 * s + i + 1 == u.nt)
          mma_commit(bar(C::kBarQEmpty));
      }
      return true;
    };
    // O_i += P_i V of the piece's step s; V is freed after its last reader.
    auto values = [&](const Run& u, int i, int s) {
      const uint32_t n = key_entry(u, i, s) + 1;
      if (!full(n) || !wwait(bar(C::kBarP + i), p_ph >> i & 1)) return false;
      p_ph ^= 1u << i;
      tc_fence_after();
      if (leader) {
        const uint64_t bv = sdesc_advance(d_v, slot_off(n));
#pragma unroll
        for (int kk = 0; kk < kT / 16; ++kk)
          mma_ts(tmem + col_o(i), tmem + col_s(i) + kk * 8, sdesc_advance(bv, kk * 2048), kIdescPV,
                 (s > 0) | (kk > 0));
        if (!u.pair || i == 1) mma_commit(bar(C::kBarEmpty + n % kSlots));
        if (s + 1 == u.steps(i)) mma_commit(bar(C::kBarO + i));
      }
      return true;
    };
    // Behind each product come the stream's next scores; at a piece's end they
    // are the next piece's first, which its softmax finds when it leaves the
    // epilogue.  The walk begins behind an empty piece.  The steps within a
    // piece are unrolled; its end and the next one's begin share one copy of the
    // code (what runs once a piece misses the instruction cache).
    bool more = next_run(nxt);
    while (ok && (cur.nt > 0 || more)) {
      const int last = cur.steps(0) - 1, steps1 = cur.steps(1);
      for (int s = 0; s < last; ++s) {
        if (!values(cur, 0, s) || !scores(cur, 0, s + 1) || !values(cur, 1, s) ||
            (s + 1 < steps1 && !scores(cur, 1, s + 1))) {
          ok = false;
          break;
        }
      }
#pragma unroll 1
      for (int i = 0; ok && i < 2; ++i)
        if (last >= 0 && last < cur.steps(i)) ok = values(cur, i, last);
      if (ok && more) {
        ok = wwait(bar(C::kBarQFull), q_ph);
        q_ph ^= 1;
      }
#pragma unroll 1
      for (int i = 0; ok && more && i < 2; ++i)
        if (nxt.steps(i) > 0) ok = scores(nxt, i, 0);
      cur = nxt;
      more = more && next_run(nxt);
    }
    if (!ok) {
      // Let every MMA already issued retire before TMEM is released.
      if (leader) mma_commit(bar(C::kBarDrain));
      mbar_drain(bar(C::kBarDrain), 0);
    }
  } else if (warp == 2) {
    // -------------------------------------------------------------------- Q
    // The rows of each piece, as soon as the scores of the piece before are
    // done: boxes of q_box tokens and 64 columns, one a lane.  A box may reach
    // into another request's rows; theirs are computed and not stored.
    if (lane == 0) tma_prefetch_desc(&tm_q);
    const int box_bytes = q_box * G * 128;
    bool ok = true;
    int k = 0;
    for (; ok && walk.next(a, span); ++k) {
      ok = __all_sync(0xffffffffu, mbar_wait_short(bar(C::kBarQEmpty), (k & 1) ^ 1, wc));
      if (!ok) break;
      const int tok0 = p.m * span, ntok = min(span, p.x.n - tok0);
      const int boxes = (ntok + q_box - 1) / q_box;  // q_box divides tpt, or one is a tile
      if (lane == 0) mbar_arrive_expect_tx(bar(C::kBarQFull), boxes * C::kHalves * box_bytes);
      __syncwarp();
      for (int e = lane; e < boxes * C::kHalves; e += 32) {
        const int half = e % C::kHalves, t = e / C::kHalves * q_box;
        const int tile = kPair && t >= tpt ? 1 : 0;
        tma_load_3d(sQ + tile * C::kTileBytes + half * kBoxBytes + (t - tile * tpt) * G * 128, &tm_q,
                    bar(C::kBarQFull), half * 64, p.g * G, p.x.q0 + tok0 + t);
      }
    }
    if (!ok && k > 0) mbar_drain(bar(C::kBarQFull), (k - 1) & 1);
  } else if (warp >= 4) {
    // -------------------------------------------------------------- softmax
    const int ti = (warp - 4) >> 2;
    const int wq = warp & 3;         // TMEM sub-partition = rows 32*wq ..
    const int row = wq * 32 + lane;  // row within the tile
    const uint32_t tl = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t colS = col_s(ti), colO = col_o(ti);
    const float sl2 = a.scale_log2;
    const int g_magic = (65535 + G) / G;  // r / G = r * g_magic >> 16 for r < 256, G <= 128
    const int tok = row / G, head = row - tok * G;
    float2* ml = reinterpret_cast<float2*>(smem + C::kOffSums);  // of both warpgroups
    uint32_t s_ph = 0, o_ph[2] = {0, 0}, entries = 0;
    bool ok = true;
    auto wwait = [&](uint32_t bar_addr, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait_short(bar_addr, parity, wc));
    };
    bool more = walk.next(a, span);
    for (int k = 0; ok && more; ++k) {
      const int item_tok = p.m * span;
      const bool pair = kPair && p.x.n - item_tok > tpt;
      const int nt = p.t1 - p.t0;
      const int token = item_tok + (pair ? ti * tpt : 0) + tok;  // within the request
      const bool live = tok < tpt && token < p.x.n;
      unsigned long long bits = 0;
      if (!chain && live) {
        bits = a.tree[p.x.q0 + token];
        if (p.x.n < 64) bits &= (1ull << p.x.n) - 1;
      }
      // Without a tree a row sees the new positions up to itself.
      const int upto = chain && (kPaged || a.causal) ? token + 1 : 0;
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
            seen_columns(vis, k0, p.x.ctx + upto, p.x.ctx, bits);
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
          const float m_tile =
              best_score<kBf16>(fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)), sl2);
          // Only rows that are stored have a say: what the others hold may change
          // from call to call, and a rescale changes the rounding.
          const bool rescale = __any_sync(0xffffffffu, live && m_tile - m > kWeightLag<kBf16>);
          float alpha = 1.f;
          if (rescale) {
            const float m_new = fmaxf(m, new_reference<kBf16>(m_tile));
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
#pragma unroll 1
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
          const uint32_t n = entries + 2 * x + 1;
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
      const Piece q = p;
      entries += 2 * nt;
      more = walk.next(a, span);  // the next piece's lengths load meanwhile
      float f0, f1 = 0.f, L, M;
      if (!pair) ml[ti * kT + row] = make_float2(m, l);
      mbar_arrive(bar(C::kBarMeet + 0));
      // Both warpgroups wait for every product, so that both count the phases.
      ok = wwait(bar(C::kBarMeet + 0), k & 1) && wwait(bar(C::kBarO + 0), o_ph[0]) &&
           (nt == 1 && !pair || wwait(bar(C::kBarO + 1), o_ph[1]));
      if (!ok) break;
      o_ph[0] ^= 1;
      if (nt > 1 || pair) o_ph[1] ^= 1;
      if (!pair) {
        const float2 x0 = ml[row], x1 = ml[kT + row];
        M = fmaxf(x0.x, x1.x);
        f0 = x0.x == -INFINITY ? 0.f : ex2(x0.x - M);
        f1 = x1.x == -INFINITY ? 0.f : ex2(x1.x - M);
        L = x0.y * f0 + x1.y * f1;
      } else {
        M = m;
        L = l;
        f0 = 1.f;
      }
      tc_fence_after();
      const float inv = L == 0.f ? 0.f : 1.f / L;  // a row that sees nothing: 0
      f0 *= inv;
      f1 *= inv;
      const float lse2 = L == 0.f ? -INFINITY : M + log2f(L);
      const bool whole = q.t0 == 0 && q.t1 == q.tiles;
      const int which = q.t0 == 0 ? 1 : 0;
      const int tile_tok = pair ? ti * tpt : 0;  // first token of the tile within the item
      const int64_t place = place_of(w, cta, which, tile_tok * G);
      if (warp_live) {
        // After the transpose this lane writes a piece of each of the quad's
        // four rows; where, and whether they are live.
        int64_t at[4];
        bool writes[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = row - (lane & 3) + j, t = (r * g_magic) >> 16;
          const int64_t to = whole ? (int64_t)(q.x.q0 + item_tok + tile_tok + t) * a.H + q.g * G +
                                         (r - t * G)
                                   : place + r;
          at[j] = to * D;
          writes[j] = t < tpt && item_tok + tile_tok + t < q.x.n;
        }
        const int cc_lo = pair ? 0 : ti * (D / 64), cc_hi = pair ? D / 32 : cc_lo + D / 64;
#pragma unroll 1
        for (int cc = cc_lo; cc < cc_hi; ++cc) {
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
          if (whole) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[j].x = pack16<kBf16>(__uint_as_float(o[8 * j + 0]), __uint_as_float(o[8 * j + 1]));
              v[j].y = pack16<kBf16>(__uint_as_float(o[8 * j + 2]), __uint_as_float(o[8 * j + 3]));
              v[j].z = pack16<kBf16>(__uint_as_float(o[8 * j + 4]), __uint_as_float(o[8 * j + 5]));
              v[j].w = pack16<kBf16>(__uint_as_float(o[8 * j + 6]), __uint_as_float(o[8 * j + 7]));
            }
            quad_transpose(v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (writes[j])
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at[j] + cc * 32 +
                                          (lane & 3) * 8) = v[j];
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint4 v[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int b = h * 16 + j * 4;
                v[j] = make_uint4(o[b], o[b + 1], o[b + 2], o[b + 3]);
              }
              quad_transpose(v);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (writes[j])
                  *reinterpret_cast<uint4*>(w.o + at[j] + cc * 32 + h * 16 + (lane & 3) * 4) = v[j];
            }
          }
          __syncwarp();
        }
      }
      if (live && (pair || ti == 0)) {
        if (whole)
          a.lse[(int64_t)(q.g * G + head) * a.N + q.x.q0 + token] =
              L == 0.f ? -INFINITY : lse2 * kLn2;
        else
          w.lse[place + row] = lse2;
      }
      if (!whole && q.t0 == 0 && warp == 4 && lane == 0) {
        Cut c;
        c.last = cuts.of(q.item_at + kItemCost + q.tiles - 1);
        c.token0 = q.x.q0 + item_tok;
        c.n = min(q.x.n - item_tok, span);
        c.g = q.g;
        w.cuts[cta] = c;
      }
      // The next piece overwrites (m, l) and O: not before both are through.
      tc_fence_before();
      mbar_arrive(bar(C::kBarMeet + 1));
      ok = wwait(bar(C::kBarMeet + 1), k & 1);
      tc_fence_after();
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
// o = sum_c 2^(lse_c - L) o_c.  Blocks (c, y) take the rows of the item begun by
// CTA c.  Up to kFew partials a warp takes a row, eight partials' loads at a
// time; more (one long context spread over the SMs) are shared by the block's
// warps and joined through shared memory.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 4;
constexpr int kMergeRows = 16;  // blocks of an item at most
constexpr int kFew = 16;

template <bool kBf16, int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const TreeArgs a,
                                                                      const Partials w) {
  constexpr int E = D / 32, U = 8;
  __shared__ float s_o[kMergeWarps][D], s_m[kMergeWarps], s_l[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.H / a.Hkv;
  wait_prior_grid();
  const int c0 = blockIdx.x;
  const Cut cut = w.cuts[c0];
  if (cut.last <= c0) return;
  const int parts = cut.last - c0 + 1, rows = cut.n * G;
  const bool few = parts <= kFew;
  const int step = few ? 1 : kMergeWarps;
  for (int base = blockIdx.y * (few ? kMergeWarps : 1); base < rows;
       base += gridDim.y * (few ? kMergeWarps : 1)) {
    const int row = base + (few ? warp : 0);
    float m = -INFINITY, l = 0.f, o[E] = {};
    if (row < rows) {
      for (int i0 = few ? 0 : warp; i0 < parts; i0 += U * step) {
        float x[U], v[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * step;
          x[u] = -INFINITY;
          if (i < parts) {
            const int64_t at = place_of(w, c0 + i, i == 0 ? 1 : 0, row);
            x[u] = w.lse[at];
            if constexpr (E == 4) {
              const float4 f = reinterpret_cast<const float4*>(w.o + at * D)[lane];
              v[u][0] = f.x;
              v[u][1] = f.y;
              v[u][2] = f.z;
              v[u][3] = f.w;
            } else {
              const float2 f = reinterpret_cast<const float2*>(w.o + at * D)[lane];
              v[u][0] = f.x;
              v[u][1] = f.y;
            }
          }
        }
        float mn = m;
#pragma unroll
        for (int u = 0; u < U; ++u) mn = fmaxf(mn, x[u]);
        const float f = m == -INFINITY ? 0.f : ex2(m - mn);
        l *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (i0 + u * step >= parts) continue;
          const float g = x[u] == -INFINITY ? 0.f : ex2(x[u] - mn);
          l += g;
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = fmaf(v[u][e], g, o[e]);
        }
        m = mn;
      }
    }
    if (!few) {
      __syncthreads();  // the row before is through
#pragma unroll
      for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
      if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
      }
      __syncthreads();
      if (warp != 0) continue;
      float mn = -INFINITY;
#pragma unroll
      for (int i = 0; i < kMergeWarps; ++i) mn = fmaxf(mn, s_m[i]);
      l = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
      for (int i = 0; i < kMergeWarps; ++i) {
        const float f = s_m[i] == -INFINITY ? 0.f : ex2(s_m[i] - mn);
        l += s_l[i] * f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(s_o[i][lane * E + e], f, o[e]);
      }
      m = mn;
    }
    if (row < rows) {
      const int token = cut.token0 + row / G, head = cut.g * G + row % G;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint32_t* out = static_cast<uint32_t*>(a.out) + ((int64_t)token * a.H + head) * (D / 2) +
                      lane * (E / 2);
      if constexpr (E == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(pack16<kBf16>(o[0] * inv, o[1] * inv),
                                                    pack16<kBf16>(o[2] * inv, o[3] * inv));
      else
        *out = pack16<kBf16>(o[0] * inv, o[1] * inv);
      if (lane == 0)
        a.lse[(int64_t)head * a.N + token] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Two row tiles an item where the requests have more than a tile's rows (128)
// on the average; each request is right either way, one row tile reads a large
// request's keys once for each 128 rows.
bool use_pairs(int R, int N, int G) { return (int64_t)N * G > (int64_t)R * kT; }

// Rows of a place: an item's, at most two tiles of 128 / G tokens.
int place_rows(int N, int G) {
  const int64_t most = 2 * (int64_t)(kT / G) * G, have = (int64_t)N * G;
  return (int)(have < most ? have : most);
}

template <bool kBf16, int D, bool kPair, bool kPaged>
cudaError_t run(const TreeArgs& a, int dev, int sms, cudaStream_t stream) {
  const int G = a.H / a.Hkv;
  CUtensorMap mq, mk, mv;
  const int box = query_box(a.R, a.N, G);
  if (!query_map(&mq, a, kBf16, G, D, box)) return cudaErrorInvalidValue;
  if constexpr (kPaged) {
    if (!cache_map(&mk, a.k_cache, kBf16, a.cache, a.Hkv, D) ||
        !cache_map(&mv, a.v_cache, kBf16, a.cache, a.Hkv, D))
      return cudaErrorInvalidValue;
  } else {
    if (!rows_map(&mk, a.k_cache, kBf16, a.Hkv, D, a.k_stride, a.Nk) ||
        !rows_map(&mv, a.v_cache, kBf16, a.Hkv, D, a.v_stride, a.Nk))
      return cudaErrorInvalidValue;
  }
  const int smem = Cfg<D, kPair>::kSmemBytes;
  static DeviceOnce allowed;
  cudaError_t e = allowed.shared_memory(reinterpret_cast<const void*>(tree_kernel<kBf16, D, kPair, kPaged>), dev, smem);
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
  tree_kernel<kBf16, D, kPair, kPaged><<<grid, kThreads, smem, stream>>>(mq, mk, mv, a, w, box);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, w.rows < kMergeRows ? w.rows : kMergeRows);
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

// The cache as a 4-D tensor (d, head, token of the page, page), box 64 columns
// of up to 128 tokens of one page and head.
bool cache_map(CUtensorMap* m, const void* ptr, bool bf16, const CacheShape& c, int Hkv, int D) {
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)c.page_size,
                        (cuuint64_t)c.num_pages};
  cuuint64_t strides[3] = {(cuuint64_t)c.head_stride * 2, (cuuint64_t)c.token_stride * 2,
                           (cuuint64_t)c.page_stride * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)(c.page_size < kT ? c.page_size : kT), 1};
  return encode_tiled(m, bf16, 4, ptr, dims, strides, box);
}

// Tokens of a box of Q: about what a request has on the average, so that little
// is read for nothing, but whole swizzle groups of 8 rows and a part of a tile
// (else a tile).
int query_box(int R, int N, int G) {
  const int tpt = kT / G;
  const int64_t mean = ((int64_t)N + R - 1) / R;
  for (int t = 1; t < tpt; t *= 2)
    if (t >= mean && t * G % 8 == 0 && tpt % t == 0) return t;
  return tpt;
}

// Q as a 3-D tensor (d, head, token), box 64 columns, the heads of a kv head and
// `tokens` tokens.
bool query_map(CUtensorMap* m, const TreeArgs& a, bool bf16, int G, int D, int tokens) {
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.H, (cuuint64_t)a.N};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.q_stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)tokens};
  return encode_tiled(m, bf16, 3, a.q, dims, strides, box);
}

namespace {
size_t places_bytes(size_t rows, int D) {
  return align256(kMaxCtas * sizeof(Cut)) +
         align256((size_t)kMaxCtas * 2 * rows * sizeof(float)) +
         align256((size_t)kMaxCtas * 2 * rows * D * sizeof(float));
}
}  // namespace

size_t tree_workspace_bytes(int N, int H, int Hkv, int D) {
  return places_bytes((size_t)place_rows(N, H / Hkv), D);
}

size_t line_workspace_bytes(int N, int H, int D) {
  const int64_t have = (int64_t)N * H;
  return places_bytes((size_t)(have < 2 * kT ? have : 2 * kT), D);
}

cudaError_t launch_line_attn(const TreeArgs& a, int dtype, int dev, int sms, cudaStream_t stream) {
  const bool pair = use_pairs(a.R, a.N, a.H / a.Hkv);
#define CPATTN_TREE(paged)                                                          \
  if (dtype == CPATTN_BF16) {                                                       \
    if (a.D == 128)                                                                 \
      return pair ? run<true, 128, true, paged>(a, dev, sms, stream)                          \
                  : run<true, 128, false, paged>(a, dev, sms, stream);                        \
    return pair ? run<true, 64, true, paged>(a, dev, sms, stream)                             \
                : run<true, 64, false, paged>(a, dev, sms, stream);                           \
  }                                                                                 \
  if (a.D == 128)                                                                   \
    return pair ? run<false, 128, true, paged>(a, dev, sms, stream)                           \
                : run<false, 128, false, paged>(a, dev, sms, stream);                         \
  return pair ? run<false, 64, true, paged>(a, dev, sms, stream)                              \
              : run<false, 64, false, paged>(a, dev, sms, stream)
  if (a.cu_k == nullptr) {
    CPATTN_TREE(true);
  }
  CPATTN_TREE(false);
#undef CPATTN_TREE
}

// The keys of a request are only bounded here (the table's width): a table much
// wider than its requests sends small calls to the tensor cores, which costs
// what the table in answer_way.h says.
cudaError_t launch_tree_attn(const TreeArgs& a, int dtype, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t keys = (int64_t)a.width * a.cache.page_size;
  if (small_attn_us(a, keys, sms) < line_attn_us(a, keys))
    return launch_small_attn(a, dtype, sms, stream);
  return launch_line_attn(a, dtype, dev, sms, stream);
}

}  // namespace cpattn
