// The attention weight of cached positions on the tensor cores (sm_103a).
//
//   w_j <- decay w_j + sum_i exp(scale q_i k_j - lse_i)
//
// With the normalisers known the sum needs no running maximum and no second
// product: S = K Q^T has a key a row, so a thread of the epilogue holds one key and
// adds up its row, exp by exp, and nothing is exchanged.
//  * An item is 256 keys of a kv head: two key tiles, which share the tiles of 128 rows
//    (tokens x query heads).  Both lie in shared memory; TMA loads pages and rows.
//  * Many rows (prompts): bound by the tensor cores and the exponentials.  Three
//    warpgroups take the steps (a tile of rows each) by turns and walk both key tiles'
//    rows of products; at the item's end their sums meet in shared memory.
//  * Few rows (single tokens, drafts): bound by HBM, which the ring of key tiles keeps
//    loading.  A warpgroup takes a key tile, and the rows of a request and kv head stay in
//    shared memory from one item to the next.
//  * The work is cut without regard to requests and items: all products of all items
//    stand in one line and CTA c of N takes the c-th N-th of it.  An item that a cut
//    divides leaves float32 sums, joined in order by weights_merge_kernel, so that
//    two runs give the same bits.
// Sums: a tile's 128 terms in four accumulators, tiles in one with compensation
// (a prompt of 16384 tokens adds 65536 terms to a weight).
// Rows of keys behind a request's last position hold whatever was there; they are
// rows of S of their own, which nobody stores.  Columns of tokens behind its last one,
// or that do not see a key, are passed over by selection.
//
// Threads: warp 0 (where keys stream, 4 too) loads K and Q, warps 1 and 2 issue the
// products of a key tile each, warp 3 writes down the pieces and the normalisers, the last
// 8 or 12 warps are the warpgroups, a key a thread.  TMEM: two places of 128 columns for
// each key tile's products.
//
// Measured (H = 32, Hkv = 8, D = 128): 64 single tokens over 100-8192 positions 94 us (5.1
// TB/s, HBM at 75 %: an item takes a CTA about as long to walk, issue and add up as to load);
// 16 prompts of 100-2000, D = 64, float16 112 us (the warpgroups' way through the rows:
// exponentials 42 % of the time, issue slots 51 %); one of 16384 855-915 us (1.2-1.3 PFLOP/s; 1965 cycles a
// step of two products of 128 x 128 x 128, which as instructions of their own take 1712).
// Two key tiles an item, so that a tile of rows is loaded for 256 keys.  Not faster: four
// warpgroups (924-978 us), products' rows read 64 columns at a time or a read ahead (spills).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cpattn.h"
#include "cpattn_internal.h"
#include "tc_ptx.cuh"
#include "weights_line.h"

namespace cpattn {
namespace {

using namespace tc;
using namespace wline;

constexpr int kT = kTcTile;
constexpr int kBoxBytes = kT * 64 * 2;
constexpr int kMaxCtas = 160;  // sums are laid out for so many
constexpr float kLog2e = 1.4426950408889634f;
// What the warpgroups need to know of a piece; warp 3 writes it down, so that their
// registers are left to the products.
struct __align__(16) Note {
  int q0, n, ctx, total;
  int r, g, m, q0t;
  int s0, s1, begins[2];
  int more, last, fresh, whole;  // more: another piece follows
  int end_cta;                   // that holds the item's last step
  int in_page[2];                // where a key tile begins within its page
  int pad;
  int page[16];                  // of each 128 / page_size-th of the tiles (a tile each from 128 on)
};
constexpr int kNotes = 4;

// kDeep: few rows a request, deeper rings of keys, else of rows.  Each key tile of the
// pair has a ring of its own: the warpgroups that take it then see every phase of its
// barriers (of a shared ring's they would miss those of the other's tiles, and take one
// for the next but one).
template <int D, bool kDeep>
struct Cfg {
  static constexpr int kGroups = kDeep ? 2 : 3;  // warpgroups
  static constexpr int kHands = 128 * kGroups;   // their threads
  static constexpr int kCtl = kDeep ? 8 : 4;  // warps before them
  static constexpr int kThreads = 32 * kCtl + kHands;
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kBoxBytes;
  static constexpr int kDepth = kDeep ? (D == 128 ? 3 : 6) : (D == 128 ? 1 : 2);  // of a key tile's ring
  static constexpr int kKeys = 2 * kDepth;
  static constexpr int kRows = kDeep ? 1 : (D == 128 ? 4 : 8);
  // Of normalisers: more than the warpgroups that take the steps by turns, so that none waits
  // for a place of which it has not seen the phase before.
  static constexpr int kNorms = kRows < 4 ? 4 : kRows;
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = kKeys * kTileBytes;
  static constexpr int kOffL = kOffQ + kRows * kTileBytes;  // also the prologue's sums
  static constexpr int kOffX = kOffL + kNorms * kT * 4;  // sums, by turns
  static constexpr int kOffBar = kOffX + (kDeep ? 0 : 2 * kGroups * kPair * 4);
  static constexpr int kBarKFull = 0;
  static constexpr int kBarKEmpty = kBarKFull + kKeys;
  static constexpr int kBarQFull = kBarKEmpty + kKeys;
  static constexpr int kBarQEmpty = kBarQFull + kRows;
  static constexpr int kBarLFull = kBarQEmpty + kRows;
  static constexpr int kBarLEmpty = kBarLFull + kNorms;
  static constexpr int kBarS = kBarLEmpty + kNorms;      // [2][2][3] products are there, for a reader
  static constexpr int kBarSFree = kBarS + 12;          // [2][2] and have been read
  static constexpr int kBarPFull = kBarSFree + 4;       // a piece's notes
  static constexpr int kBarPEmpty = kBarPFull + kNotes;
  static constexpr int kBarXFull = kBarPEmpty + kNotes;  // [2] the warpgroups' sums
  static constexpr int kBarXEmpty = kBarXFull + 2;
  static constexpr int kBarDrain = kBarXEmpty + 2;
  static constexpr int kNumBars = kBarDrain + 2;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffNotes = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr int kSmemBytes = kOffNotes + kNotes * (int)sizeof(Note);
  static_assert(kSmemBytes <= 232448 && kNorms <= 8, "shared memory");
};

// TMEM: two places of products for each key tile.
__device__ constexpr uint32_t col_s(int place) { return 128u * (uint32_t)place; }

// The sums of items that were cut: per CTA two places (0: of an item begun by an
// earlier CTA, 1: of one that goes on in the next), and a record of the item begun
// there and cut.
struct Cut {
  int last;  // CTA that holds the item's end; -1: nothing was cut here
  int r, g, m;
};
struct Sums {
  Cut* cuts;
  float* sums;  // [kMaxCtas][2][kPair]
};

// Two float32 values in a register pair: an instruction for both.
typedef unsigned long long Two;
__device__ __forceinline__ Two two(float x, float y) {
  Two p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ Two two(uint32_t x, uint32_t y) {
  return two(__uint_as_float(x), __uint_as_float(y));
}
__device__ __forceinline__ float2 apart(Two p) {
  float2 x;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x.x), "=f"(x.y) : "l"(p));
  return x;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void exps(float& x, float& y, Two p) {
  const float2 f = apart(p);
  x = ex2(f.x);
  y = ex2(f.y);
}

template <bool kBf16, int D, bool kDeep>
__global__ void __launch_bounds__(Cfg<D, kDeep>::kThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const WeightsArgs args, const Sums out, const int q_box) {
  using C = Cfg<D, kDeep>;
  constexpr int kThreads = C::kThreads;
  const TreeArgs& a = args.t;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = opaque(smem_u32(smem));
  if (base & 1023u) {  // the swizzled tiles need it; shared memory has no room for slack
    if (threadIdx.x == 0) {
      atomicExch(a.err, kErrLaunch);
      out.cuts[blockIdx.x].last = -1;
    }
    return;
  }
  const uint32_t bars = base + C::kOffBar;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  // Of each place for normalisers: whether a row there gives nothing (its lse is -inf).
  volatile uint8_t* some_void = smem + C::kOffMisc + 8;
  // [20] of the warps; then where this CTA begins: in_req, r and the request.
  long long* sums = reinterpret_cast<long long*>(smem + C::kOffL);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{abort_flag, a.err};
  const int G = a.H / a.Hkv, tpt = kT / G;
  const bool chain = a.tree == nullptr;

  launch_dependents();  // the merge sets itself up; it waits for this kernel's end
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kKeys; ++s) {
      mbar_init(bar(C::kBarKFull + s), 1);
      mbar_init(bar(C::kBarKEmpty + s), 1);
    }
    for (int s = 0; s < C::kRows; ++s) {
      mbar_init(bar(C::kBarQFull + s), 1);
      mbar_init(bar(C::kBarQEmpty + s), 2);
    }
    for (int s = 0; s < C::kNorms; ++s) {
      mbar_init(bar(C::kBarLFull + s), 32);
      mbar_init(bar(C::kBarLEmpty + s), kDeep ? 256 : 128);
    }
    for (int i = 0; i < 12; ++i) mbar_init(bar(C::kBarS + i), 1);
    for (int i = 0; i < 4; ++i) mbar_init(bar(C::kBarSFree + i), 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kBarXFull + i), C::kHands);
      mbar_init(bar(C::kBarXEmpty + i), 256);
    }
    for (int i = 0; i < kNotes; ++i) {
      mbar_init(bar(C::kBarPFull + i), 32);
      mbar_init(bar(C::kBarPEmpty + i), C::kHands);
    }
    mbar_init(bar(C::kBarDrain), 1);
    mbar_init(bar(C::kBarDrain + 1), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // Where this CTA's part of the line begins: each thread sums a run of requests, the
  // block sums the threads, and the thread whose run holds the beginning finds the
  // request.  Lengths that break the rules could name the same rows over and over:
  // nothing is computed then.
  const int per = (a.R + kThreads - 1) / kThreads;
  const int r_lo = min(a.R, (int)threadIdx.x * per), r_hi = min(a.R, r_lo + per);
  long long own = 0;
  bool bad = false;
  Req x;
  for (int r = r_lo; r < r_hi; ++r) bad |= !load_req<true>(a, r, x);
  if (bad && blockIdx.x == 0) atomicExch(a.err, kErrBadTables);
  if (!__syncthreads_or(bad)) {
    for (int r = r_lo; r < r_hi; ++r) {
      if (per > 1) load_req<true>(a, r, x);
      own += head_cost(x, tpt, chain) * a.Hkv;
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
        load_req<true>(a, r, x);
        const long long t = head_cost(x, tpt, chain) * a.Hkv;
        if (begin < at + t) break;
        at += t;
        ++r;
      }
      sums[20] = begin - at;
      sums[21] = r;
      *reinterpret_cast<Req*>(sums + 22) = x;
    }
  }
  if (threadIdx.x == 0) out.cuts[cta].last = -1;
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  Walk walk;
  walk.init(a, tpt, (int)sums[21], *reinterpret_cast<const Req*>(sums + 22), sums[20], begin, count);
  __syncthreads();  // the sums' place is used again
  Piece& p = walk.p;

  // Pages of up to a tile are powers of two.
  const int P = a.cache.page_size, P_log = P <= kT ? 31 - __clz(P) : 0;
  auto page_index = [&](int pos) { return P <= kT ? pos >> P_log : pos / P; };
  auto in_page = [&](int tile_pos) { return P <= kT ? 0 : tile_pos % P; };  // of a tile's begin

  auto wwait = [&](uint32_t bar_addr, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_short(bar_addr, parity, wc));
  };

  if (warp == 0 || (kDeep && warp == 4)) {
    // -------------------------------------------------------------- K and Q
    // Deep: warp 0 loads the first key tile and Q, warp 4 the second (one for both took
    // longer to walk and to issue than HBM to bring them).
    // Lane l holds the page number of copy l of the pair (the next pair's are fetched
    // ahead); lane c * halves + half issues copy c of a tile, columns 64 * half.
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_q);
    }
    const int box_bytes = q_box * G * 128;
    uint32_t rows = 0;
    const int box = P < kT ? P : kT;  // rows of a copy
    const int ppt = kT / box;         // copies of a tile and 64 columns
    const int npages = (int)a.cache.num_pages;
    auto page_of = [&](const Piece& u) {
      const int at = u.m * kPair + lane * box;
      return lane < 2 * ppt && at < u.x.total ? a.table[(int64_t)u.r * a.table_stride + page_index(at)] : -1;
    };
    const int c = lane / C::kHalves, half = lane % C::kHalves;
    uint32_t seq[2] = {0, 0};
    bool ok = true;
    int ahead = walk.more ? page_of(walk.ahead) : -1;
    while (ok && walk.next(a, tpt, kDeep)) {
      const int now = ahead;
      if (walk.more) ahead = page_of(walk.ahead);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!ok || (kDeep && i != warp / 4) || p.begins(i, tpt, chain) == p.s1) continue;
        const int k0 = p.m * kPair + i * kT;
        const int id = __shfl_sync(0xffffffffu, now, (i * ppt + (c < ppt ? c : 0)) & 31);
        const bool mine = c < ppt && k0 + c * box < p.x.total;
        const bool good = mine && id >= 0 && id < npages;
        if (mine && !good) atomicExch(a.err, kErrBadTables);
        const uint32_t copies = __popc(__ballot_sync(0xffffffffu, good));
        const int sl = i * C::kDepth + seq[i] % C::kDepth;
        ok = wwait(bar(C::kBarKEmpty + sl), ((seq[i] / C::kDepth) & 1) ^ 1);
        if (!ok) continue;
        ++seq[i];
        if (lane == 0) mbar_arrive_expect_tx(bar(C::kBarKFull + sl), copies * box * 128);
        __syncwarp();
        if (good)
          tma_load_4d(base + C::kOffK + sl * C::kTileBytes + half * kBoxBytes + c * box * 128, &tm_k,
                      bar(C::kBarKFull + sl), half * 64, p.g, in_page(k0), id);
      }
      // The rows: boxes of q_box tokens and 64 columns, one a lane.  A box may reach into
      // another request's rows; their columns are passed over.
      for (int s = p.s0; ok && warp == 0 && p.fresh && s < p.s1; ++s) {
        const int sl = rows % C::kRows;
        ok = wwait(bar(C::kBarQEmpty + sl), ((rows / C::kRows) & 1) ^ 1);
        if (!ok) break;
        ++rows;
        const int tok0 = (p.q0t + s) * tpt;
        const int boxes = (min(tpt, p.x.n - tok0) + q_box - 1) / q_box;  // q_box divides tpt
        if (lane == 0)
          mbar_arrive_expect_tx(bar(C::kBarQFull + sl), boxes * C::kHalves * box_bytes);
        __syncwarp();
        for (int e = lane; e < boxes * C::kHalves; e += 32) {
          const int half = e % C::kHalves, t = e / C::kHalves * q_box;
          tma_load_3d(base + C::kOffQ + sl * C::kTileBytes + half * kBoxBytes + t * G * 128, &tm_q,
                      bar(C::kBarQFull + sl), half * 64, p.g * G, p.x.q0 + tok0 + t);
        }
      }
    }
    if (!ok) {
      // Let the copies already issued land before the CTA exits.
      for (int i = 0; i < 2; ++i)
        for (uint32_t n = seq[i] > (uint32_t)C::kDepth ? seq[i] - C::kDepth : 0; n < seq[i]; ++n)
          mbar_drain(bar(C::kBarKFull + i * C::kDepth + n % C::kDepth), (n / C::kDepth) & 1);
      for (uint32_t n = rows > (uint32_t)C::kRows ? rows - C::kRows : 0; n < rows; ++n)
        mbar_drain(bar(C::kBarQFull + n % C::kRows), (n / C::kRows) & 1);
    }
  } else if (warp < 3) {
    // ------------------------------------------------------------------ MMA
    // A warp issues the products of a key tile.  (One warp for both took longer to issue
    // them, two waits and eight instructions each, than the tensor cores to compute.)
    const bool leader = elect_one();
    const int i = warp - 1;
    const uint64_t d_q = sdesc_sw128(base + C::kOffQ, 16, 1024);
    const uint64_t d_k = sdesc_sw128(base + C::kOffK, 16, 1024);
    uint32_t rows = 0, keys = 0, used = 0;
    int group = C::kGroups - 1;  // rows stream: that takes this step
    bool ok = true;
    while (ok && walk.next(a, tpt, kDeep)) {
      const int from = p.begins(i, tpt, chain), s1 = p.s1;
      for (int s = p.s0; s < s1; ++s) {
        rows += p.fresh;
        group = group == C::kGroups - 1 ? 0 : group + 1;
        const uint32_t slot = (rows - 1) % C::kRows;
        ok = wwait(bar(C::kBarQFull + slot), ((rows - 1) / C::kRows) & 1);
        if (ok && s >= from) {
          if (s == from) {
            ok = wwait(bar(C::kBarKFull + i * C::kDepth + keys % C::kDepth), (keys / C::kDepth) & 1);
            ++keys;
          }
          const int sl = i * C::kDepth + (keys - 1) % C::kDepth, at = 2 * i + (used & 1);
          ok = ok && wwait(bar(C::kBarSFree + at), (used >> 1 & 1) ^ 1);
          ++used;
          if (ok) {
            tc_fence_after();
            // All 128 columns, or the live ones to a multiple of 32.
            const int live = min(tpt, p.x.n - (p.q0t + s) * tpt) * G;
            const uint32_t idesc = idesc_f16(kBf16, 128, 128, false, false) -
                                   ((uint32_t)((kT - (live + 31) / 32 * 32) >> 3) << 17);
            if (leader) {
              const uint64_t a0 = sdesc_advance(d_k, sl * C::kTileBytes);
              const uint64_t b0 = sdesc_advance(d_q, slot * C::kTileBytes);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * kBoxBytes + (kk & 3) * 32;
                mma_ss(tmem + col_s(at), sdesc_advance(a0, off), sdesc_advance(b0, off), idesc, kk > 0);
              }
              // A barrier for each place and reader: so a reader sees all its phases, and none
              // ends before the one before it has been seen.
              mma_commit(bar(C::kBarS + 3 * at + (kDeep ? 0 : group)));
              if (s + 1 == s1) mma_commit(bar(C::kBarKEmpty + sl));
            }
          }
        }
        if (!ok) break;
        if (leader && (p.last || s + 1 < s1)) mma_commit(bar(C::kBarQEmpty + slot));
      }
    }
    if (!ok) {
      // Let every product already issued retire before TMEM is released.
      if (leader) mma_commit(bar(C::kBarDrain + i));
      mbar_drain(bar(C::kBarDrain + i), 0);
    }
  } else if (warp == 3) {
    // ---------------------------------------------------- notes and normalisers
    // The pieces' notes, each before the normalisers of the piece before it (the
    // warpgroups look one piece ahead); -lse log2(e) of each row (infinity: it gives nothing,
    // whatever its products are), four rows a lane, a step's values fetched while the step
    // before is handed over.
    int tok[4], head[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      tok[j] = (lane * 4 + j) / G;
      head[j] = lane * 4 + j - tok[j] * G;
    }
    float v[4];
    struct At {
      int q0, n, g, q0t, s, s1;
      bool fresh;
    } at = {}, then = {};  // the piece whose normalisers go out, and the next
    // Lane l holds the page number of the l-th part of the pair, the next pair's ahead.
    const int box = P < kT ? P : kT, parts_of_pair = 2 * (kT / box);
    auto page_of = [&](const Piece& u) {
      const int pos = u.m * kPair + lane * box;
      return lane < parts_of_pair && pos < u.x.total
                 ? a.table[(int64_t)u.r * a.table_stride + page_index(pos)]
                 : -1;
    };
    int pages_ahead = walk.more ? page_of(walk.ahead) : -1;
    uint32_t noted = 0, rows = 0;
    bool ok = true, more = true;
    // Writes down the next piece, and keeps it in `then`.
    auto note = [&]() {
      more = walk.next(a, tpt, kDeep);
      if (!more) return true;
      const int page = pages_ahead;
      if (walk.more) pages_ahead = page_of(walk.ahead);
      const int sl = noted % kNotes;
      if (!wwait(bar(C::kBarPEmpty + sl), ((noted / kNotes) & 1) ^ 1)) return false;
      ++noted;
      Note& c = *reinterpret_cast<Note*>(smem + C::kOffNotes + sl * sizeof(Note));
      if (lane < 16) c.page[lane] = page >= 0 && page < a.cache.num_pages ? page : -1;
      if (lane == 0) {
        c.q0 = p.x.q0;
        c.n = p.x.n;
        c.ctx = p.x.ctx;
        c.total = p.x.total;
        c.r = p.r;
        c.g = p.g;
        c.m = p.m;
        c.q0t = p.q0t;
        c.s0 = p.s0;
        c.s1 = p.s1;
        c.begins[0] = p.begins(0, tpt, chain);
        c.begins[1] = p.begins(1, tpt, chain);
        c.more = walk.more;
        c.last = p.last;
        c.fresh = p.fresh;
        c.whole = p.whole();
        c.in_page[0] = in_page(p.m * kPair);
        c.in_page[1] = in_page(p.m * kPair + kT);
        c.end_cta = c.whole || p.s0 > 0 ? -1 : cuts.of(p.item_at + kItemCost + p.steps - 1);
      }
      mbar_arrive(bar(C::kBarPFull + sl));
      then = {p.x.q0, p.x.n, p.g, p.q0t, p.s0, p.s1, p.fresh};
      return true;
    };
    auto fetch = [&](const At& u) {
      const int tok0 = (u.q0t + u.s) * tpt;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = INFINITY;
        if (tok[j] < tpt && tok0 + tok[j] < u.n)
          v[j] = args.lse[(int64_t)(u.g * G + head[j]) * a.N + u.q0 + tok0 + tok[j]];
      }
    };
    ok = note();
    bool some = more;
    if (some) fetch(then);
    while (ok && some) {
      at = then;
      ok = note();
      // `then` holds the next piece, or (more false) this one.
      if (!at.fresh) {
        some = more;
        if (some) fetch(then);
        continue;
      }
      for (; ok && at.s < at.s1; ) {
        const float4 l = {-kLog2e * v[0], -kLog2e * v[1], -kLog2e * v[2], -kLog2e * v[3]};
        const bool none = __any_sync(0xffffffffu, l.x == INFINITY || l.y == INFINITY ||
                                                      l.z == INFINITY || l.w == INFINITY);
        ++at.s;
        if (at.s < at.s1)
          fetch(at);
        else if (more)
          fetch(then);
        const int sl = rows % C::kNorms;
        ok = wwait(bar(C::kBarLEmpty + sl), ((rows / C::kNorms) & 1) ^ 1);
        if (!ok) break;
        ++rows;
        reinterpret_cast<float4*>(smem + C::kOffL + sl * kT * 4)[lane] = l;
        if (lane == 0) some_void[sl] = none;
        mbar_arrive(bar(C::kBarLFull + sl));
      }
      some = more;
    }
  } else if (warp >= C::kCtl) {
    // -------------------------------------------------------------- the sums
    // Deep: a warpgroup a key tile.  Else the warpgroups take the steps by turns, both key
    // tiles of each, and add up their sums at the piece's end.
    const int group = (warp - C::kCtl) >> 2;
    const int row = (warp & 3) * 32 + lane;  // TMEM lane, key of the tile
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t rows = 0, used = 0, made1 = 0;  // made1: all products of key tile 1
    uint32_t phases = 0;                     // of this warpgroup's barriers of the places
    int behind = group;  // steps until this warpgroup's next
    bool ok = true;
    auto note_of = [&](uint32_t k) -> const Note& {
      return *reinterpret_cast<const Note*>(smem + C::kOffNotes + (k % kNotes) * sizeof(Note));
    };
    // The weight that this thread stores (of key tile `group`), and what it holds so far.
    auto weight_of = [&](const Note& u, float& old) -> float* {
      if (group > 1) return nullptr;
      const int pos = u.m * kPair + group * kT + row;
      const int page = u.page[P < kT ? (group * kT + row) >> P_log : group];
      if (pos >= u.total || page < 0) return nullptr;
      float* to = args.weights + ((int64_t)page * a.Hkv + u.g) * P +
                  (P < kT ? row & (P - 1) : u.in_page[group] + row);
      if (u.whole && pos < u.ctx) old = *to;
      return to;
    };
    const Two sl2 = two(a.scale_log2, a.scale_log2);
    Two t0, t1;
    // Adds up 32 columns from c on of a key's row of products with the tile of rows at tok0, of
    // which all (whole) or those that see the key count.
    auto columns = [&](const uint32_t* r, const float* nl, int c, bool whole, bool voids, int ahead_by,
                       int tok0, int ntok, int n, int q0) {
      float y[32];
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(nl + c + j);
        exps(y[j], y[j + 1], fma2(two(r[j], r[j + 1]), sl2, l.x));
        exps(y[j + 2], y[j + 3], fma2(two(r[j + 2], r[j + 3]), sl2, l.y));
      }
      if (!whole) {
        // Which of the columns see this key: of the live ones those of the key's own token
        // and later ones, or those whose word names it.
        const int hi = ntok * G - c;
        uint32_t seen = hi >= 32 ? 0xffffffffu : (1u << hi) - 1;
        const int lo = (chain && ahead_by > tok0 ? min(ahead_by - tok0, tpt) * G : 0) - c;
        if (lo > 0) seen = lo >= 32 ? 0u : seen >> lo << lo;
        if (!chain && ahead_by >= 0) {
          uint32_t named = 0;
          for (int t = c / G; t < ntok && t * G < c + 32; ++t) {
            const unsigned long long word = a.tree[q0 + tok0 + t];
            if (ahead_by < n && ahead_by < 64 && (word >> ahead_by & 1)) {
              const int b = max(t * G - c, 0), e = min(t * G + G - c, 32);
              named |= (e - b >= 32 ? 0xffffffffu : (1u << (e - b)) - 1) << b;
            }
          }
          seen &= named;
        }
        if (voids) {  // (some row of the tile: seldom)
#pragma unroll 1
          for (int j = 0; j < 32; ++j)
            if (nl[c + j] == INFINITY) seen &= ~(1u << j);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j] = seen >> j & 1 ? y[j] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        t0 = add2(t0, two(y[j], y[j + 1]));
        t1 = add2(t1, two(y[j + 2], y[j + 3]));
      }
    };
    // The whole row; frees the products' place.  Columns that none of the warp's keys (the first
    // is `first` new tokens on) sees are passed over, those that all see need no selection: of a
    // key tile's steps along the diagonal only one in four selects in a warp (16 prompts of
    // 100-2000 tokens 113.3 -> 112.1 us, 64 single tokens 94.9 -> 93.8; one of 16384 872 -> 875).
    auto row_sum = [&](uint32_t at, int free_bar, const float* nl, bool voids, int first, int tok0, int n,
                       int q0) {
      t0 = t1 = two(0.f, 0.f);
      const int ntok = min(tpt, n - tok0), live = ntok * G;
      const int any = chain ? max(0, min(first - tok0, tpt)) * G : 0;
      const int all = chain ? max(0, min(first + 31 - tok0, tpt)) * G : (first + 31 < 0 ? 0 : kT);
      int c = any & ~31;
      if (c >= live) {
        tc_fence_before();
        mbar_arrive(bar(free_bar));
      }
#pragma unroll 1
      for (; c < live; c += 32) {
        uint32_t r[32];
        tmem_ld32(at + c, r);
        tmem_wait_ld_regs(r);
        if (c + 32 >= live) {
          tc_fence_before();
          mbar_arrive(bar(free_bar));
        }
        columns(r, nl, c, c >= all && c + 32 <= live && !voids, voids, first + lane, tok0, ntok, n, q0);
      }
      const float2 x0 = apart(t0), x1 = apart(t1);
      return (x0.x + x0.y) + (x1.x + x1.y);
    };
    // total + x, with what the rounding leaves out in `lost`.
    auto plus = [](float& total, float& lost, float x) {
      const float term = x - lost, sum = total + term;
      lost = fabsf(sum) < INFINITY ? __fadd_rn(__fadd_rn(sum, -total), -term) : 0.f;
      total = sum;
    };
    bool more = walk.more;
    float old_ahead = 0.f;
    float* to_ahead = nullptr;
    if (more) {
      ok = wwait(bar(C::kBarPFull), 0);
      if (ok) to_ahead = weight_of(note_of(0), old_ahead);
    }
    for (uint32_t k = 0; ok && more; ++k) {
      const Note& u = note_of(k);
      float* const to = to_ahead;
      const float old = old_ahead;
      more = u.more;
      if (more) {
        ok = wwait(bar(C::kBarPFull + (k + 1) % kNotes), ((k + 1) / kNotes) & 1);
        if (!ok) break;
        to_ahead = weight_of(note_of(k + 1), old_ahead);
      }
      const int s0 = u.s0, s1 = u.s1, n = u.n, q0 = u.q0, ctx = u.ctx, q0t = u.q0t;
      const int from0 = u.begins[0], from1 = u.begins[1];
      const int ahead_by = u.m * kPair + row - ctx;  // >= 0: the new token of key tile 0's position
      const int first = ahead_by - lane;             // of the warp's first key
      float total0 = 0.f, lost0 = 0.f, total1 = 0.f, lost1 = 0.f;
      if constexpr (kDeep) {
        const bool last = u.last;
        for (int s = s0; s < s1; ++s) {
          rows += u.fresh;
          const uint32_t slot = (rows - 1) % C::kNorms;
          ok = wwait(bar(C::kBarLFull + slot), ((rows - 1) / C::kNorms) & 1);
          if (!ok) break;
          const bool voids = some_void[slot];
          if (s >= (group == 0 ? from0 : from1)) {
            const int at = 2 * group + (used & 1), tok0 = (q0t + s) * tpt;
            ok = wwait(bar(C::kBarS + 3 * at), used >> 1 & 1);
            if (!ok) break;
            ++used;
            tc_fence_after();
            plus(total0, lost0,
                 row_sum(tl + col_s(at), C::kBarSFree + at,
                         reinterpret_cast<const float*>(smem + C::kOffL + slot * kT * 4), voids,
                         first + group * kT, tok0, n, q0));
          }
          if (last || s + 1 < s1) mbar_arrive(bar(C::kBarLEmpty + slot));
        }
      } else {
        // Step s0 + behind is this warpgroup's, then each kGroups-th.
        int s = s0 + behind;
        for (; s < s1; s += C::kGroups) {
          const uint32_t step = rows + (s - s0), slot = step % C::kNorms;
          const int tok0 = (q0t + s) * tpt;
          const float* nl = reinterpret_cast<const float*>(smem + C::kOffL + slot * kT * 4);
          ok = wwait(bar(C::kBarLFull + slot), (step / C::kNorms) & 1);
          const bool voids = some_void[slot];
#pragma unroll 1
          for (int i = 0; ok && i < (s >= from1 ? 2 : 1); ++i) {
            const int at = 2 * i + ((i == 0 ? step : made1 + (uint32_t)(s - from1)) & 1);
            ok = wwait(bar(C::kBarS + 3 * at + group), phases >> at & 1);
            if (!ok) break;
            phases ^= 1u << at;
            tc_fence_after();
            const float x =
                row_sum(tl + col_s(at), C::kBarSFree + at, nl, voids, first + i * kT, tok0, n, q0);
            plus(i == 0 ? total0 : total1, i == 0 ? lost0 : lost1, x);
          }
          if (!ok) break;
          mbar_arrive(bar(C::kBarLEmpty + slot));
        }
        behind = s - s1;
        made1 += s1 - from1;
        rows += s1 - s0;
      }
      if (!ok) break;
      float total = total0;
      if constexpr (!kDeep) {
        // Two places by turns: the sums of the piece before the last have been read.
        float* x = reinterpret_cast<float*>(smem + C::kOffX) + (k & 1) * C::kGroups * kPair + row;
        ok = wwait(bar(C::kBarXEmpty + (k & 1)), (k >> 1 & 1) ^ 1);
        if (!ok) break;
        x[group * kPair] = total0;
        x[group * kPair + kT] = total1;
        mbar_arrive(bar(C::kBarXFull + (k & 1)));
        if (group < 2) {
          ok = wwait(bar(C::kBarXFull + (k & 1)), k >> 1 & 1);
          if (!ok) break;
          total = 0.f;
#pragma unroll
          for (int w = 0; w < C::kGroups; ++w) total += x[w * kPair + group * kT];
          mbar_arrive(bar(C::kBarXEmpty + (k & 1)));
        }
      }
      if (group < 2) {
        if (u.whole) {
          if (to) *to = ahead_by + group * kT < 0 ? fmaf(args.decay, old, total) : total;
        } else {
          const int which = u.s0 == 0 ? 1 : 0;
          out.sums[((int64_t)cta * 2 + which) * kPair + group * kT + row] = total;
          if (which == 1 && group == 0 && row == 0) {
            Cut c;
            c.last = u.end_cta;
            c.r = u.r;
            c.g = u.g;
            c.m = u.m;
            out.cuts[cta] = c;
          }
        }
      }
      mbar_arrive(bar(C::kBarPEmpty + k % kNotes));
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
// Adds up the sums of each item that was cut, in the CTAs' order: block c those of the
// item begun by CTA c, a thread a key.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPair) weights_merge_kernel(const WeightsArgs args, const Sums out) {
  const TreeArgs& a = args.t;
  wait_prior_grid();
  const int c0 = blockIdx.x;
  const Cut cut = out.cuts[c0];
  if (cut.last <= c0) return;
  Req x;
  load_req<true>(a, cut.r, x);
  const int pos = cut.m * kPair + (int)threadIdx.x, P = a.cache.page_size;
  if (pos >= x.total) return;
  const int page = a.table[(int64_t)cut.r * a.table_stride + pos / P];
  if (page < 0 || page >= a.cache.num_pages) return;
  float* to = args.weights + ((int64_t)page * a.Hkv + cut.g) * P + pos % P;
  const float old = pos < x.ctx ? *to : 0.f;
  float sum = 0.f;
  for (int c = c0; c <= cut.last; ++c)
    sum += out.sums[((int64_t)c * 2 + (c == c0)) * kPair + threadIdx.x];
  *to = pos < x.ctx ? fmaf(args.decay, old, sum) : sum;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <bool kBf16, int D, bool kDeep>
cudaError_t run(const WeightsArgs& w, int dev, int sms, cudaStream_t stream) {
  const TreeArgs& a = w.t;
  const int G = a.H / a.Hkv, box = query_box(a.R, a.N, G);
  CUtensorMap mq, mk;
  if (!query_map(&mq, a, kBf16, G, D, box) ||
      !cache_map(&mk, a.k_cache, kBf16, a.cache, a.Hkv, D))
    return cudaErrorInvalidValue;
  const int smem = Cfg<D, kDeep>::kSmemBytes;
  static DeviceOnce allowed;
  cudaError_t e = allowed.shared_memory(
      reinterpret_cast<const void*>(weights_kernel<kBf16, D, kDeep>), dev, smem);
  if (e != cudaSuccess) return e;
  Sums out;
  char* ws = static_cast<char*>(a.workspace);
  out.cuts = reinterpret_cast<Cut*>(ws);
  out.sums = reinterpret_cast<float*>(ws + align256(kMaxCtas * sizeof(Cut)));
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  weights_kernel<kBf16, D, kDeep><<<grid, Cfg<D, kDeep>::kThreads, smem, stream>>>(mq, mk, w, out, box);
  e = cudaGetLastError();
  // No request has more than one tile of rows: no item has two steps, none is cut.
  if (e != cudaSuccess || a.N <= kT / G) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kPair);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weights_merge_kernel, w, out);
}

template <bool kBf16, int D>
cudaError_t run_deep(const WeightsArgs& w, int dev, int sms, cudaStream_t stream) {
  const bool deep = keys_stream(w.t.R, w.t.N, w.t.H / w.t.Hkv);
  return deep ? run<kBf16, D, true>(w, dev, sms, stream) : run<kBf16, D, false>(w, dev, sms, stream);
}

}  // namespace

size_t weights_workspace_bytes() {
  return align256(kMaxCtas * sizeof(Cut)) + (size_t)kMaxCtas * 2 * kPair * sizeof(float);
}

cudaError_t launch_tc_weights(const WeightsArgs& w, int dtype, int dev, int sms,
                              cudaStream_t stream) {
  if (dtype == CPATTN_BF16)
    return w.t.D == 128 ? run_deep<true, 128>(w, dev, sms, stream)
                        : run_deep<true, 64>(w, dev, sms, stream);
  return w.t.D == 128 ? run_deep<false, 128>(w, dev, sms, stream)
                      : run_deep<false, 64>(w, dev, sms, stream);
}

}  // namespace cpattn
