// The attention weight of cached positions on the tensor cores (sm_103a).
//
//   w_j <- decay w_j + sum_i exp(scale q_i k_j - lse_i)
//
// With the normalisers known the sum needs no running maximum and no second
// product: S = K Q^T has a key a row, so a thread of the epilogue holds one key and
// adds up its row, exp by exp, and nothing is exchanged.
//  * An item is 256 keys of a kv head: two key tiles, whose products with a tile of
//    128 rows (tokens x query heads) alternate.  A key tile is the products' left
//    operand and stays in TMEM for all of them (a product from shared memory runs at
//    60 % of the tensor rate, from TMEM at 86 %); only the rows stream, by TMA.
//  * Many rows (prompts): bound by the tensor cores.  Few rows (single tokens, drafts):
//    by HBM, which the ring of key tiles keeps loading; the rows of a request and kv
//    head then stay in shared memory from one item to the next.
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
// CTA = 384 threads: warp 0 loads K, warp 2 Q, warp 3 the normalisers (and notes down the pieces), warp 1 owns
// TMEM and issues the products, warps 4-7 and 8-11 take a key tile each: they move it from
// shared memory to TMEM and read the products' rows.  TMEM: S0 [0,128) S1 [128,256), then
// two places for each key tile [256,512).
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
constexpr int kThreads = 384;
constexpr int kMaxCtas = 160;  // sums are laid out for so many
constexpr float kLog2e = 1.4426950408889634f;
// Registers per thread of the control warps and of the warpgroups, which hold a row of
// products (setmaxnreg); the launch gives 384 threads x 168.
constexpr int kRegCtl = 128, kRegSum = 184;
static_assert(128 * kRegCtl + 256 * kRegSum <= kThreads * 168, "register split");

template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// What the warpgroups need to know of a piece; warp 3 writes it down, so that their
// registers are left to the products.
struct __align__(16) Note {
  int q0, n, ctx, total;
  int r, g, m, q0t;
  int s0, s1, begins[2];
  int more, last, fresh, whole;  // more: another piece follows
  int end_cta;                   // that holds the item's last step
  int pad[3];
};
constexpr int kNotes = 4;

// kDeep: deeper rings of keys (few rows a request), else of rows.  Each key tile of the
// pair has a ring of its own: the warpgroup that takes it then sees every phase of its
// barriers (of a shared ring's it would miss those of the other's tiles, and take one
// for the next but one).
template <int D, bool kDeep>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kBoxBytes;
  static constexpr int kDepth = (D == 128 ? 1 : 2) * (kDeep ? 2 : 1);  // of a key tile's ring
  static constexpr int kKeys = 2 * kDepth;
  static constexpr int kRows = (D == 128 ? 1 : 2) * (kDeep ? 2 : 4);
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = kKeys * kTileBytes;
  static constexpr int kOffL = kOffQ + kRows * kTileBytes;  // also the prologue's sums
  static constexpr int kOffBar = kOffL + kRows * kT * 4;
  static constexpr int kBarKFull = 0;
  static constexpr int kBarKEmpty = kBarKFull + kKeys;
  static constexpr int kBarQFull = kBarKEmpty + kKeys;
  static constexpr int kBarQEmpty = kBarQFull + kRows;
  static constexpr int kBarLFull = kBarQEmpty + kRows;
  static constexpr int kBarLEmpty = kBarLFull + kRows;
  static constexpr int kBarS = kBarLEmpty + kRows;    // [2] products of a tile are there
  static constexpr int kBarSFree = kBarS + 2;         // [2] and have been read
  static constexpr int kBarA = kBarSFree + 2;         // [2][2] a key tile is in its place
  static constexpr int kBarPFull = kBarA + 4;      // a piece's notes
  static constexpr int kBarPEmpty = kBarPFull + kNotes;
  static constexpr int kBarDrain = kBarPEmpty + kNotes;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffNotes = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr int kSmemBytes = kOffNotes + kNotes * (int)sizeof(Note);
  static_assert(kSmemBytes <= 232448, "shared memory");
};

__host__ __device__ constexpr uint32_t col_s(int i) { return 128u * (uint32_t)i; }
__host__ __device__ constexpr uint32_t col_a(int i, int which) {
  return 256u + 128u * (uint32_t)i + 64u * (uint32_t)which;
}

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

template <bool kBf16, int D, bool kDeep>
__global__ void __launch_bounds__(kThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const WeightsArgs args, const Sums out, const int q_box) {
  using C = Cfg<D, kDeep>;
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
  // [12] of the warps; then where this CTA begins: in_req, r and the request.
  long long* sums = reinterpret_cast<long long*>(smem + C::kOffL);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{abort_flag, a.err};
  const int G = a.H / a.Hkv, tpt = kT / G;
  const bool chain = a.tree == nullptr;

  launch_dependents();  // the merge sets itself up; it waits for this kernel's end
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kKeys; ++s) {
      mbar_init(bar(C::kBarKFull + s), 1);
      mbar_init(bar(C::kBarKEmpty + s), 128);
    }
    for (int s = 0; s < C::kRows; ++s) {
      mbar_init(bar(C::kBarQFull + s), 1);
      mbar_init(bar(C::kBarQEmpty + s), 1);
      mbar_init(bar(C::kBarLFull + s), 32);
      mbar_init(bar(C::kBarLEmpty + s), 256);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kBarS + i), 1);
      mbar_init(bar(C::kBarSFree + i), 128);
      mbar_init(bar(C::kBarA + 2 * i), 128);
      mbar_init(bar(C::kBarA + 2 * i + 1), 128);
    }
    for (int i = 0; i < kNotes; ++i) {
      mbar_init(bar(C::kBarPFull + i), 32);
      mbar_init(bar(C::kBarPEmpty + i), 256);
    }
    mbar_init(bar(C::kBarDrain), 1);
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
      sums[13] = begin - at;
      sums[14] = r;
      *reinterpret_cast<Req*>(sums + 16) = x;
    }
  }
  if (threadIdx.x == 0) out.cuts[cta].last = -1;
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  Walk walk;
  walk.init(a, tpt, (int)sums[14], *reinterpret_cast<const Req*>(sums + 16), sums[13], begin, count);
  __syncthreads();  // the sums' place is used again
  Piece& p = walk.p;

  auto wwait = [&](uint32_t bar_addr, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_short(bar_addr, parity, wc));
  };

  if (warp < 4) {
  reg_dec<kRegCtl>();
  if (warp == 0) {
    // -------------------------------------------------------------------- K
    // Lane l holds the page number of copy l of the pair (the next pair's are fetched
    // ahead); lane c * halves + half issues copy c of a tile, columns 64 * half.
    if (lane == 0) tma_prefetch_desc(&tm_k);
    const int P = a.cache.page_size;
    const int box = P < kT ? P : kT;  // rows of a copy
    const int ppt = kT / box;         // copies of a tile and 64 columns
    const int npages = (int)a.cache.num_pages;
    auto page_of = [&](const Piece& u) {
      const int at = u.m * kPair + lane * box;
      return lane < 2 * ppt && at < u.x.total ? a.table[(int64_t)u.r * a.table_stride + at / P] : -1;
    };
    const int c = lane / C::kHalves, half = lane % C::kHalves;
    uint32_t seq[2] = {0, 0};
    bool ok = true;
    int ahead = walk.more ? page_of(walk.ahead) : -1;
    while (ok && walk.next(a, tpt)) {
      const int now = ahead;
      if (walk.more) ahead = page_of(walk.ahead);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!ok || p.begins(i, tpt, chain) == p.s1) continue;
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
                      bar(C::kBarKFull + sl), half * 64, p.g, k0 % P, id);
      }
    }
    if (!ok) {
      // Let the copies already issued land before the CTA exits.
      for (int i = 0; i < 2; ++i)
        for (uint32_t n = seq[i] > (uint32_t)C::kDepth ? seq[i] - C::kDepth : 0; n < seq[i]; ++n)
          mbar_drain(bar(C::kBarKFull + i * C::kDepth + n % C::kDepth), (n / C::kDepth) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    const bool leader = elect_one();
    const uint64_t d_q = sdesc_sw128(base + C::kOffQ, 16, 1024);
    uint32_t rows = 0, staged[2] = {0, 0}, used[2] = {0, 0};
    bool ok = true;
    while (ok && walk.next(a, tpt)) {
      const int from[2] = {p.begins(0, tpt, chain), p.begins(1, tpt, chain)};
      for (int s = p.s0; ok && s < p.s1; ++s) {
        if (p.fresh) {
          ok = wwait(bar(C::kBarQFull + rows % C::kRows), (rows / C::kRows) & 1);
          if (!ok) break;
          ++rows;
        }
        const uint32_t slot = (rows - 1) % C::kRows;
        const int live = min(tpt, p.x.n - (p.q0t + s) * tpt) * G;
        const uint32_t idesc = idesc_f16(kBf16, 128, 128, false, false) -
                               ((uint32_t)((kT - (live + 31) / 32 * 32) >> 3) << 17);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (s < from[i]) continue;
          if (s == from[i]) {
            ok = ok && wwait(bar(C::kBarA + 2 * i + (staged[i] & 1)), (staged[i] >> 1) & 1);
            ++staged[i];
          }
          ok = ok && wwait(bar(C::kBarSFree + i), (used[i] & 1) ^ 1);
          if (!ok) break;
          ++used[i];
          tc_fence_after();
          if (leader) {
            const uint64_t b0 = sdesc_advance(d_q, slot * C::kTileBytes);
            const uint32_t at = tmem + col_a(i, (staged[i] - 1) & 1);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ts(tmem + col_s(i), at + kk * 8,
                     sdesc_advance(b0, (kk >> 2) * kBoxBytes + (kk & 3) * 32), idesc, kk > 0);
            mma_commit(bar(C::kBarS + i));
          }
        }
        if (ok && leader && (p.last || s + 1 < p.s1)) mma_commit(bar(C::kBarQEmpty + slot));
      }
    }
    if (!ok) {
      // Let every product already issued retire before TMEM is released.
      if (leader) mma_commit(bar(C::kBarDrain));
      mbar_drain(bar(C::kBarDrain), 0);
    }
  } else if (warp == 2) {
    // -------------------------------------------------------------------- Q
    // Boxes of q_box tokens and 64 columns, one a lane.  A box may reach into another
    // request's rows; their columns are passed over.
    if (lane == 0) tma_prefetch_desc(&tm_q);
    const int box_bytes = q_box * G * 128;
    uint32_t rows = 0;
    bool ok = true;
    while (ok && walk.next(a, tpt)) {
      if (!p.fresh) continue;
      for (int s = p.s0; s < p.s1; ++s) {
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
      for (uint32_t n = rows > (uint32_t)C::kRows ? rows - C::kRows : 0; n < rows; ++n)
        mbar_drain(bar(C::kBarQFull + n % C::kRows), (n / C::kRows) & 1);
    }
  } else if (warp == 3) {
    // ---------------------------------------------------- notes and normalisers
    // The pieces' notes, each before the normalisers of the piece before it (the
    // warpgroups look one piece ahead); -lse log2(e) of each row, -inf for those that
    // give nothing, four rows a lane, a step's values fetched while the step before is
    // handed over.
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
    uint32_t noted = 0, rows = 0;
    bool ok = true, more = true;
    // Writes down the next piece, and keeps it in `then`.
    auto note = [&]() {
      more = walk.next(a, tpt);
      if (!more) return true;
      const int sl = noted % kNotes;
      if (!wwait(bar(C::kBarPEmpty + sl), ((noted / kNotes) & 1) ^ 1)) return false;
      ++noted;
      if (lane == 0) {
        Note c;
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
        c.end_cta = c.whole || p.s0 > 0 ? -1 : cuts.of(p.item_at + kItemCost + p.steps - 1);
        *reinterpret_cast<Note*>(smem + C::kOffNotes + sl * sizeof(Note)) = c;
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
        float4 l;
        l.x = v[0] == -INFINITY ? -INFINITY : -kLog2e * v[0];
        l.y = v[1] == -INFINITY ? -INFINITY : -kLog2e * v[1];
        l.z = v[2] == -INFINITY ? -INFINITY : -kLog2e * v[2];
        l.w = v[3] == -INFINITY ? -INFINITY : -kLog2e * v[3];
        ++at.s;
        if (at.s < at.s1)
          fetch(at);
        else if (more)
          fetch(then);
        const int sl = rows % C::kRows;
        ok = wwait(bar(C::kBarLEmpty + sl), ((rows / C::kRows) & 1) ^ 1);
        if (!ok) break;
        ++rows;
        reinterpret_cast<float4*>(smem + C::kOffL + sl * kT * 4)[lane] = l;
        mbar_arrive(bar(C::kBarLFull + sl));
      }
      some = more;
    }
  }
  } else {
    reg_inc<kRegSum>();
    // -------------------------------------------------------------- the sums
    const int ti = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;  // TMEM lane, key of the tile
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float sl2 = a.scale_log2;
    const int P = a.cache.page_size, npages = (int)a.cache.num_pages;
    uint32_t staged = 0, used = 0, rows = 0;
    bool ok = true;
    auto note_of = [&](uint32_t k) -> const Note& {
      return *reinterpret_cast<const Note*>(smem + C::kOffNotes + (k % kNotes) * sizeof(Note));
    };
    // Moves this warpgroup's key tile of a piece from its ring to its place in TMEM.
    auto stage = [&](const Note& u) {
      if (u.begins[ti] == u.s1) return true;
      const int sl = ti * C::kDepth + staged % C::kDepth;
      if (!wwait(bar(C::kBarKFull + sl), (staged / C::kDepth) & 1)) return false;
      const uint8_t* from = smem + C::kOffK + sl * C::kTileBytes + row * 128;
      const uint32_t to = tl + col_a(ti, staged & 1);
#pragma unroll
      for (int half = 0; half < C::kHalves; ++half) {
        uint32_t r[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 v =
              *reinterpret_cast<const uint4*>(from + half * kBoxBytes + ((c ^ (row & 7)) * 16));
          r[4 * c] = v.x;
          r[4 * c + 1] = v.y;
          r[4 * c + 2] = v.z;
          r[4 * c + 3] = v.w;
        }
        tmem_st32(to + half * 32, r);
      }
      mbar_arrive(bar(C::kBarKEmpty + sl));
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(C::kBarA + 2 * ti + (staged & 1)));
      ++staged;
      return true;
    };
    auto page_of = [&](const Note& u) {
      const int pos = u.m * kPair + ti * kT + row;
      return pos < u.total ? a.table[(int64_t)u.r * a.table_stride + pos / P] : -1;
    };
    int page_ahead = -1;
    bool more = walk.more;
    if (more) {
      ok = wwait(bar(C::kBarPFull), 0);
      if (ok) {
        page_ahead = page_of(note_of(0));
        ok = stage(note_of(0));
      }
    }
    for (uint32_t k = 0; ok && more; ++k) {
      const Note& u = note_of(k);
      const int page = page_ahead;
      more = u.more;
      if (more) {
        ok = wwait(bar(C::kBarPFull + (k + 1) % kNotes), ((k + 1) / kNotes) & 1);
        if (!ok) break;
        page_ahead = page_of(note_of(k + 1));
      }
      const int s1 = u.s1, from = u.begins[ti];
      const bool fresh = u.fresh, last = u.last, whole = u.whole;
      const int pos = u.m * kPair + ti * kT + row, ahead_by = pos - u.ctx;
      float* to = nullptr;
      if (pos < u.total && page >= 0 && page < npages)
        to = args.weights + ((int64_t)page * a.Hkv + u.g) * P + pos % P;
      float old = 0.f;
      if (to && whole && ahead_by < 0) old = *to;
      if (from == s1 && more) ok = stage(note_of(k + 1));
      float total = 0.f, lost = 0.f;  // lost: what total's roundings left out
      int tok0 = (u.q0t + u.s0) * tpt;
#pragma unroll 1
      for (int s = u.s0; ok && s < s1; ++s, tok0 += tpt) {
        rows += fresh;
        const uint32_t slot = (rows - 1) % C::kRows;
        if (s < from) {
          // Another key tile's step: its normalisers pass by.
          ok = wwait(bar(C::kBarLFull + slot), ((rows - 1) / C::kRows) & 1);
          if (!ok) break;
        } else {
          // The next tile goes to its place while this one's last product runs.
          if (s + 1 == s1 && more) ok = stage(note_of(k + 1));
          ok = ok && wwait(bar(C::kBarLFull + slot), ((rows - 1) / C::kRows) & 1) &&
               wwait(bar(C::kBarS + ti), used & 1);
          if (!ok) break;
          ++used;
          tc_fence_after();
          const int ntok = min(tpt, u.n - tok0), live = ntok * G;
          const float* nl = reinterpret_cast<const float*>(smem + C::kOffL + slot * kT * 4);
          uint32_t r[128];
          tmem_ld32(tl + col_s(ti) + 0, r + 0);
          tmem_ld32(tl + col_s(ti) + 32, r + 32);
          tmem_ld32(tl + col_s(ti) + 64, r + 64);
          tmem_ld32(tl + col_s(ti) + 96, r + 96);
          tmem_wait_ld_regs(r);
          reg_fence32(r + 32);
          reg_fence32(r + 64);
          reg_fence32(r + 96);
          tc_fence_before();
          mbar_arrive(bar(C::kBarSFree + ti));
          float t0 = 0.f, t1 = 0.f, t2 = 0.f, t3 = 0.f;
          // The tile's last key against the tile's first token.
          const int edge = ahead_by - row + kT - 1;
          if (live == kT && (chain ? edge <= tok0 : edge < 0)) {
#pragma unroll
            for (int j = 0; j < kT; j += 4) {
              const float4 l = *reinterpret_cast<const float4*>(nl + j);
              t0 += ex2(fmaf(__uint_as_float(r[j]), sl2, l.x));
              t1 += ex2(fmaf(__uint_as_float(r[j + 1]), sl2, l.y));
              t2 += ex2(fmaf(__uint_as_float(r[j + 2]), sl2, l.z));
              t3 += ex2(fmaf(__uint_as_float(r[j + 3]), sl2, l.w));
            }
          } else {
            // The columns that see this key, as a bit mask: of the live ones those of
            // the key's own token and later ones, or those whose word names it.
            typedef unsigned __int128 u128;
            u128 v = live >= kT ? ~(u128)0 : (((u128)1 << live) - 1);
            if (chain) {
              const int first = ahead_by > tok0 ? min(ahead_by - tok0, tpt) * G : 0;
              v = first >= kT ? 0 : v >> first << first;
            } else if (ahead_by >= 0) {
              v = 0;
              for (int t = 0; t < ntok; ++t) {
                const unsigned long long word = a.tree[u.q0 + tok0 + t];
                const u128 cols = G >= kT ? ~(u128)0 : (((u128)1 << G) - 1);
                if (ahead_by < u.n && ahead_by < 64 && (word >> ahead_by & 1)) v |= cols << (t * G);
              }
            }
            const uint32_t vis[4] = {(uint32_t)v, (uint32_t)(v >> 32), (uint32_t)(v >> 64),
                                     (uint32_t)(v >> 96)};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c * 32 >= live) break;
#pragma unroll
              for (int j = c * 32; j < c * 32 + 32; j += 4) {
                const float4 l = *reinterpret_cast<const float4*>(nl + j);
                const float y0 = ex2(fmaf(__uint_as_float(r[j]), sl2, l.x));
                const float y1 = ex2(fmaf(__uint_as_float(r[j + 1]), sl2, l.y));
                const float y2 = ex2(fmaf(__uint_as_float(r[j + 2]), sl2, l.z));
                const float y3 = ex2(fmaf(__uint_as_float(r[j + 3]), sl2, l.w));
                t0 += vis[c] >> (j & 31) & 1 ? y0 : 0.f;
                t1 += vis[c] >> ((j & 31) + 1) & 1 ? y1 : 0.f;
                t2 += vis[c] >> ((j & 31) + 2) & 1 ? y2 : 0.f;
                t3 += vis[c] >> ((j & 31) + 3) & 1 ? y3 : 0.f;
              }
            }
          }
          const float term = ((t0 + t1) + (t2 + t3)) - lost;
          const float sum = total + term;
          lost = fabsf(sum) < INFINITY ? __fadd_rn(__fadd_rn(sum, -total), -term) : 0.f;
          total = sum;
        }
        if (last || s + 1 < s1) mbar_arrive(bar(C::kBarLEmpty + slot));
      }
      if (!ok) break;
      if (whole) {
        if (to) *to = ahead_by < 0 ? fmaf(args.decay, old, total) : total;
      } else {
        const int which = u.s0 == 0 ? 1 : 0;
        out.sums[((int64_t)cta * 2 + which) * kPair + ti * kT + row] = total;
        if (which == 1 && ti == 0 && row == 0) {
          Cut c;
          c.last = u.end_cta;
          c.r = u.r;
          c.g = u.g;
          c.m = u.m;
          out.cuts[cta] = c;
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
  weights_kernel<kBf16, D, kDeep><<<grid, kThreads, smem, stream>>>(mq, mk, w, out, box);
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
  // Few rows a request on the average: keys are what streams.
  const bool deep = (int64_t)w.t.N * (w.t.H / w.t.Hkv) <= (int64_t)w.t.R * kT;
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
