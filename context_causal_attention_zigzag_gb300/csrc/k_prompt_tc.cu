// Attention over packed prompts on the tensor cores (sm_103a): tcgen05.mma
// with TMEM accumulators, TMA-staged tiles, warp-specialised, persistent.
//
//   o_i = sum_j p_ij v_j,  p_ij = exp(scale q_i k_j - lse_i),  j <= i + nk - nq
//
// for each sequence by itself, by one pass over its keys with the running
// maximum and sum of the softmax.  Compute bound from a few hundred tokens on:
// 4 D flops per visible pair and head against one K and V tile of 64 KB that
// 256 query rows share.
//
// A work item is two 128-row query tiles that walk the same key tiles.  With
// an even number of query heads per kv head they are the same 128 rows of two
// neighbouring heads: both see the same keys, so no tile is loaded or
// multiplied for one of them alone, and an item is as small as 128 rows (a
// short prompt fills it).  With an odd number they are 256 rows of one head.
// Items are sorted by their number of key tiles (prompt_plan_kernel) and taken in
// that order, in the cost bands of the ring forward (banded_item), by whichever
// CTA is free; one sequence needs no sorting and is dealt in snake order; a call
// of no more items than SMs is neither (prompt_way()).
//
// What bounds it: from some hundred tokens on the rate of the tensor cores'
// instructions (16 SS and 16 TS of 128 x 128 x 16 per key tile and item, 1.52 us at
// 1.9 GHz against 1.57-1.62 measured per tile), below that what an item costs
// around its tiles (about 2.5 us: the last product, the epilogue, the first
// softmax) and the start (6-8 us).  16384 tokens, H = 32, Hkv = 8, D = 128: 1.39-1.46
// ms (1.51-1.59 PFLOP/s); 16 prompts of 100-2000: 0.222 ms (1.08 PFLOP/s).
//
// Sequences start at any row: TMA takes any first row, and a tile's rows
// behind the sequence's end belong to others.  Their scores are replaced by
// -inf, and their V rows, which enter the product with weight 0, are zeroed in
// shared memory by the softmax threads before the product, since 0 * NaN is
// NaN.  Only a sequence's last tile pays for that.
//
// Roles of a CTA (384 threads) as in the ring forward: warp 0 loads (Q tiles once
// per item, K(j), V(j) in consecutive slots of one ring), warp 1 owns TMEM and
// issues the products S_i = Q_i K^T (SS) and O_i += P_i V (TS, P in TMEM over
// S), warp 2 finds the items, warps 4-7 and 8-11 are the softmax of tile 0 and 1,
// one thread per row.
// MMA order per key tile: PV0(j), S0(j+1), PV1(j), S1(j+1), across items too, so
// that the next item's scores are ready when the softmax leaves the epilogue.
// (An epilogue in four warps of its own held the products up: at 512 threads
// the issuing warp has too few registers for its descriptors, and the 16384-token
// prompt went from 1.31 to 1.46 ms.)
// The weights are rounded to the input type for the second product
// (their sum is taken before rounding, in float32): the tensor cores take 16-bit
// operands, and the rounding is as large as that of the output itself (float16's
// smallest step: kWeightLag in tc_ptx.cuh).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "answer_way.h"
#include "cpattn_internal.h"
#include "tc_ptx.cuh"

namespace cpattn {
namespace {

using namespace tc;

constexpr int kT = 128;  // tile edge (rows, keys)
constexpr int kBoxBytes = kT * 64 * 2;
constexpr int kThreads = 384;
constexpr float kLn2 = 0.6931471805599453f;

// One block of query rows of a sequence, as the plan lists it.
struct __align__(16) Block {
  int qrow;   // its first row of q
  int nrows;  // rows of the sequence from there on
  int krow;   // the sequence's first row of k and v
  int nk;     // its keys
  int diag;   // keys that the block's first row sees under the causal rule (may be <= 0)
  int pad[3];
};

// Number of key tiles that rows [at, at + n) of a block see (n <= 0: none).
__device__ __forceinline__ int key_tiles(const Block& b, int causal, int at, int n) {
  const int last = min(at + n, b.nrows) - 1;  // last row
  if (last < at) return 0;
  const int end = causal ? min(b.nk, b.diag + last) : b.nk;
  return end > 0 ? (end + kT - 1) / kT : 0;
}

// ---------------------------------------------------------------------------
// Plan: the blocks of all sequences in order of falling cost.  One CTA; a
// counting sort over kBins costs.  The order inside a bin varies from run to
// run; results do not (each block's arithmetic is its own).
// ---------------------------------------------------------------------------
constexpr int kBins = 1024;

struct Plan {
  int nblocks;
  int next;  // items that CTAs have taken after their first
  int pad[62];
};

__device__ __forceinline__ Block make_block(int q0, int nq, int k0, int nk, int at) {
  Block b;
  b.qrow = q0 + at;
  b.nrows = nq - at;
  b.krow = k0;
  b.nk = nk;
  b.diag = at + nk - nq + 1;
  b.pad[0] = b.pad[1] = b.pad[2] = 0;
  return b;
}

__global__ void __launch_bounds__(1024) prompt_plan_kernel(const PromptArgs a, int rows, int cap,
                                                           Plan* plan, Block* list) {
  __shared__ int s_bin[kBins], s_warp[32], s_most;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  launch_dependents();
  s_bin[tid] = 0;
  if (tid == 0) {
    s_most = 1;
    plan->next = 0;
  }
  __syncthreads();
  int q0, nq, k0, nk, most = 1;
  bool bad = false;
  for (int r = tid; r < a.R; r += 1024) {
    bad |= !packed_rows(a.cu_q, r, a.Nq, q0, nq);
    bad |= !packed_rows(a.cu_k, r, a.Nk, k0, nk);
    most = max(most, (nk + kT - 1) / kT);
  }
  atomicMax(&s_most, most);
  if (bad) atomicExch(a.err, kErrBadTables);
  // Broken offsets may name the same rows over and over: nothing is computed then.
  if (__syncthreads_or(bad)) {
    if (tid == 0) plan->nblocks = 0;
    return;
  }
  most = s_most;
  // Largest cost first: bin 0 holds the blocks with the most key tiles.
  auto bin_of = [&](const Block& b) {
    const int c = key_tiles(b, a.causal, 0, rows);
    return (int)((long long)(most - c) * (kBins - 1) / most);
  };
  for (int pass = 0; pass < 2; ++pass) {
    for (int r = warp; r < a.R; r += 32) {
      packed_rows(a.cu_q, r, a.Nq, q0, nq);
      packed_rows(a.cu_k, r, a.Nk, k0, nk);
      for (int at = lane * rows; at < nq; at += 32 * rows) {
        const Block b = make_block(q0, nq, k0, nk, at);
        const int x = atomicAdd(&s_bin[bin_of(b)], 1);
        if (pass == 1 && x < cap) list[x] = b;  // more only if the offsets changed under the call
      }
    }
    __syncthreads();
    if (pass == 1) break;
    // Exclusive sums of the bins, in place: where each bin's blocks start.
    const int own = s_bin[tid];
    int x = own;
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += u;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int z = s_warp[lane];
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, z, d);
        if (lane >= d) z += u;
      }
      s_warp[lane] = z;
    }
    __syncthreads();
    s_bin[tid] = x - own + (warp > 0 ? s_warp[warp - 1] : 0);
    if (tid == 1023) plan->nblocks = min(s_bin[tid] + own, cap);
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// The attention kernel.
// ---------------------------------------------------------------------------
constexpr int kFeed = 2;      // items handed out ahead
constexpr int kReaders = 10;  // warps that read them

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kBoxBytes;
  static constexpr int kSlots = D == 128 ? 5 : 8;  // K(j), V(j) take consecutive slots
  static constexpr int kOffQ = 0;
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kOffBar = kOffRing + kSlots * kTileBytes;
  static constexpr int kBarQFull = 0;   // [2] per query tile
  static constexpr int kBarQEmpty = 2;  // [2]
  static constexpr int kBarFull = 4;
  static constexpr int kBarEmpty = kBarFull + kSlots;
  // Per query tile.  With a third S buffer a tile's scores and weights run one
  // step ahead of their product, so two barriers take turns: a single one could
  // be a phase behind or ahead, and its parity pass for the one waited for.
  static constexpr int kTurns = D == 128 ? 1 : 2;
  static constexpr int kBarS = kBarEmpty + kSlots;
  static constexpr int kBarP = kBarS + 2 * kTurns;
  static constexpr int kBarO = kBarP + 2 * kTurns;
  static constexpr int kBarFeedFull = kBarO + 2 * kTurns;  // [kFeed]
  static constexpr int kBarFeedEmpty = kBarFeedFull + kFeed;
  static constexpr int kBarDrain = kBarFeedEmpty + kFeed;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffFeed = (kOffMisc + 16 + 15) / 16 * 16;  // items, 48 bytes each
  static constexpr int kSmemBytes = kOffFeed + kFeed * 48 + 1024;  // + slack for 1024-B alignment

  // Barrier and parity of query tile i's c-th step.
  static __device__ __forceinline__ int turn(int bar0, int i, uint32_t c) {
    return bar0 + i * kTurns + (kTurns == 2 ? (int)(c & 1) : 0);
  }
  static __device__ __forceinline__ uint32_t parity(uint32_t c) {
    return kTurns == 2 ? c >> 1 & 1 : c & 1;
  }
};

// TMEM.  D = 128: S0 [0,128) S1 [128,256) O0 [256,384) O1 [384,512).  D = 64
// leaves room for a third S buffer: the scores of step n = 2 * (key tile) +
// (query tile) go to buffer n % 3, which lets a tile's next scores be computed
// while its softmax still runs (O0 [384,448) O1 [448,512)).
template <int D>
__host__ __device__ constexpr uint32_t col_s(int i, uint32_t step) {
  return D == 128 ? 128u * (uint32_t)i : 128u * ((2 * step + (uint32_t)i) % 3);
}
template <int D>
__host__ __device__ constexpr uint32_t col_o(int i) {
  return D == 128 ? 256u + 128u * (uint32_t)i : 384u + 64u * (uint32_t)i;
}

struct Work {
  const Plan* plan;   // nullptr: one sequence, decoded in closed form, or direct
  const Block* list;
  int direct;         // at most an item a CTA: each finds its own
  int rows;           // rows of a block: 128 (two heads an item) or 256 (two row tiles)
  int inner;          // items per block and kv head
};

// The only item of a direct call's CTA: the warp sums the sequences' blocks, 32 at
// a time, up to its own.
__device__ __forceinline__ bool find_direct(const PromptArgs& a, const Work& w, Block& b, int& g,
                                            int& h0) {
  const int lane = threadIdx.x & 31, per = a.Hkv * w.inner;
  const int mine = (int)blockIdx.x / per, sub = (int)blockIdx.x - mine * per;
  g = sub / w.inner;
  h0 = g * (a.H / a.Hkv) + (sub - g * w.inner) * (w.rows == kT ? 2 : 1);
  int before = 0;
  for (int r0 = 0; r0 < a.R; r0 += 32) {
    int q0, k0, nk, n = 0, nb = 0;
    if (r0 + lane < a.R) {
      packed_rows(a.cu_q, r0 + lane, a.Nq, q0, n);
      nb = (n + w.rows - 1) / w.rows;
    }
    int upto = nb;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += u;
    }
    const int at = mine - before;
    const uint32_t found = __ballot_sync(0xffffffffu, at >= upto - nb && at < upto);
    if (found != 0) {
      const int src = __ffs(found) - 1;
      const int skip = __shfl_sync(0xffffffffu, upto - nb, src);
      packed_rows(a.cu_q, r0 + src, a.Nq, q0, n);
      packed_rows(a.cu_k, r0 + src, a.Nk, k0, nk);
      b = make_block(q0, n, k0, nk, (at - skip) * w.rows);
      return true;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// One warp finds the items of a CTA and hands them to the others through shared
// memory: finding one takes several divisions and dependent loads, which would
// otherwise stand between two items of every role.
struct Items {
  const PromptArgs& a;
  const Work& w;
  int nblocks, n_items, k;
  int band_size, band_items;   // the cost bands of banded_item
  int q0, nq, k0, nk;          // the single sequence

  __device__ __forceinline__ Items(const PromptArgs& a_, const Work& w_) : a(a_), w(w_) {
    k = 0;
    const int per = a.Hkv * w.inner;
    if (w.plan != nullptr) {
      nblocks = w.plan->nblocks;
    } else {
      packed_rows(a.cu_q, 0, a.Nq, q0, nq);
      packed_rows(a.cu_k, 0, a.Nk, k0, nk);
      nblocks = (nq + w.rows - 1) / w.rows;
    }
    n_items = nblocks * per;
    if (n_items > 0) {
      const int nb = cost_band_count(nblocks * w.inner, nblocks, gridDim.x, 0);
      band_size = (nblocks + nb - 1) / nb;
      band_items = band_size * per;
    }
  }
  // The next item: its block, kv head g and first query head h0.  A planned call
  // takes them in turn, largest first, whichever CTA is free; a single sequence
  // is dealt in snake order (its items' costs fall evenly).
  __device__ __forceinline__ bool next(Block& b, int& g, int& h0) {
    const int grp = a.H / a.Hkv, heads = w.rows == kT ? 2 : 1;
    int idx;
    if (w.plan != nullptr) {
      idx = blockIdx.x;
      if (k++ > 0) {
        if ((threadIdx.x & 31) == 0) idx = gridDim.x + atomicAdd(&const_cast<Plan*>(w.plan)->next, 1);
        idx = __shfl_sync(0xffffffffu, idx, 0);
      }
    } else {
      const long long x = (long long)k * gridDim.x +
                          ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      ++k;
      idx = x < n_items ? (int)x : n_items;
    }
    if (idx >= n_items) return false;
    const int band = idx / band_items;
    int rest = idx - band * band_items;
    const int here = min(band_size, nblocks - band * band_size) * w.inner;  // of a kv head
    g = rest / here;
    rest -= g * here;
    const int r = rest / w.inner;
    const int rank = band * band_size + r;
    h0 = g * grp + (rest - r * w.inner) * heads;
    if (w.plan != nullptr) {
      const int4* p = reinterpret_cast<const int4*>(w.list + rank);
      const int4 x = p[0];
      b.qrow = x.x;
      b.nrows = x.y;
      b.krow = x.z;
      b.nk = x.w;
      b.diag = p[1].x;
    } else {
      b = make_block(q0, nq, k0, nk, (nblocks - 1 - rank) * w.rows);
    }
    return true;
  }
};

template <bool kBf16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const PromptArgs a, const Work w) {
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{abort_flag, a.err};
  const int row_step = w.rows == kT ? 0 : kT;   // second query tile: rows further on,
  const int head_step = w.rows == kT ? 1 : 0;   // or the next head

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar(C::kBarFull + s), 1);
      mbar_init(bar(C::kBarEmpty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kBarQFull + i), 1);
      mbar_init(bar(C::kBarQEmpty + i), 1);
      for (int t = 0; t < C::kTurns; ++t) {
        mbar_init(bar(C::turn(C::kBarS, i, t)), 1);
        mbar_init(bar(C::turn(C::kBarP, i, t)), 128);
        mbar_init(bar(C::turn(C::kBarO, i, t)), 1);
      }
    }
    for (int f = 0; f < kFeed; ++f) {
      mbar_init(bar(C::kBarFeedFull + f), 1);
      mbar_init(bar(C::kBarFeedEmpty + f), kReaders);
    }
    mbar_init(bar(C::kBarDrain), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (w.plan != nullptr) {
    wait_prior_grid();  // the plan
  } else if (blockIdx.x == 0) {
    int x, y;
    for (int r = threadIdx.x; r < a.R; r += kThreads)
      if (!packed_rows(a.cu_q, r, a.Nq, x, y) || !packed_rows(a.cu_k, r, a.Nk, x, y))
        atomicExch(a.err, kErrBadTables);
  }

  int4* slots = reinterpret_cast<int4*>(smem + C::kOffFeed);
  Block b;
  int g, h0, nt0, nt1;  // nt0, nt1: key tiles that the two query tiles see
  // The next item, for one of the reading warps: from the shared ring, until one
  // that says there is none; of a direct call each warp finds the only one.
  uint32_t fed = 0;
  auto next_item = [&](bool& ok) {
    if (w.direct) {
      if (fed++ != 0 || !find_direct(a, w, b, g, h0)) return false;
      nt0 = key_tiles(b, a.causal, 0, kT);
      nt1 = key_tiles(b, a.causal, row_step, kT);
      return true;
    }
    const uint32_t s = fed % kFeed;
    if (!__all_sync(0xffffffffu,
                    mbar_wait_short(bar(C::kBarFeedFull + s), (fed / kFeed) & 1, wc))) {
      ok = false;
      return false;
    }
    ++fed;
    const int4 x = slots[3 * s], y = slots[3 * s + 1];
    const int2 z = *reinterpret_cast<const int2*>(slots + 3 * s + 2);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::kBarFeedEmpty + s));
    b.qrow = x.x;
    b.nrows = x.y;
    b.krow = x.z;
    b.nk = x.w;
    b.diag = y.x;
    g = y.y;
    h0 = y.z;
    nt0 = z.x;
    nt1 = z.y;
    return y.w != 0;
  };
  if (warp == 0) {
    // ------------------------------------------------------------------ TMA
    const bool leader = elect_one();
    auto wwait = [&](uint32_t bar_addr, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait_short(bar_addr, parity, wc));
    };
    if (leader) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    uint32_t seq = 0, q_armed[2] = {0, 0};  // ring entries and Q tiles asked for
    bool ok = true;
    while (ok && next_item(ok)) {
      const int nt = max(nt0, nt1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!ok || (i == 0 ? nt0 : nt1) == 0) continue;  // a tile without keys is not multiplied
        ok = wwait(bar(C::kBarQEmpty + i), (q_armed[i] & 1) ^ 1);
        if (!ok) continue;
        ++q_armed[i];
        if (leader) {
          mbar_arrive_expect_tx(bar(C::kBarQFull + i), C::kTileBytes);
          for (int half = 0; half < C::kHalves; ++half)
            tma_load_3d(sQ + i * C::kTileBytes + half * kBoxBytes, &tm_q, bar(C::kBarQFull + i),
                        half * 64, h0 + i * head_step, b.qrow + i * row_step);
        }
      }
      for (int m = 0; ok && m < nt; ++m) {
        for (int which = 0; which < 2; ++which) {  // K(m), then V(m)
          const uint32_t n = seq;
          const int sl = n % kSlots;
          if (!wwait(bar(C::kBarEmpty + sl), ((n / kSlots) & 1) ^ 1)) {
            ok = false;
            break;
          }
          ++seq;
          if (leader) {
            mbar_arrive_expect_tx(bar(C::kBarFull + sl), C::kTileBytes);
            for (int half = 0; half < C::kHalves; ++half)
              tma_load_3d(sRing + sl * C::kTileBytes + half * kBoxBytes, which == 0 ? &tm_k : &tm_v,
                          bar(C::kBarFull + sl), half * 64, g, b.krow + m * kT);
          }
        }
      }
    }
    if (!ok) {
      // Let the copies already issued land before the CTA exits.
      for (int i = 0; i < 2; ++i)
        if (q_armed[i]) mbar_drain(bar(C::kBarQFull + i), (q_armed[i] - 1) & 1);
      for (uint32_t n = seq > (uint32_t)kSlots ? seq - kSlots : 0; n < seq; ++n)
        mbar_drain(bar(C::kBarFull + n % kSlots), (n / kSlots) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    const bool leader = elect_one();
    auto wwait = [&](uint32_t bar_addr, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait_short(bar_addr, parity, wc));
    };
    uint32_t kv_it = 0, s_n[2] = {0, 0}, p_n[2] = {0, 0}, q_ph[2] = {0, 0};
    bool ok = true;
    // Operand descriptors, computed once and advanced by byte offsets.
    const uint64_t d_q = sdesc_sw128(sQ, 16, 1024);
    const uint64_t d_k = sdesc_sw128(sRing, 16, 1024);
    const uint64_t d_v = sdesc_sw128(sRing, kBoxBytes, 1024);
    auto slot_off = [](uint32_t n) { return (n % kSlots) * (uint32_t)C::kTileBytes; };
    // S_i = Q_i K^T, K in ring entry kn (key tile kn / 2 of all).
    auto scores = [&](int i, uint32_t kn) {
      const uint32_t d = tmem + col_s<D>(i, kn / 2);
      const uint64_t a0 = sdesc_advance(d_q, i * C::kTileBytes);
      const uint64_t b0 = sdesc_advance(d_k, slot_off(kn));
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kBoxBytes + (kk & 3) * 32;
        mma_ss(d, sdesc_advance(a0, off), sdesc_advance(b0, off), kIdescQK, kk > 0);
      }
      mma_commit(bar(C::turn(C::kBarS, i, s_n[i])));
    };
    auto values = [&](int i, uint32_t vn, uint32_t accumulate) {  // O_i += P_i V
      const uint32_t p = tmem + col_s<D>(i, vn / 2);
      const uint64_t bv = sdesc_advance(d_v, slot_off(vn));
#pragma unroll
      for (int kk = 0; kk < kT / 16; ++kk)
        mma_ts(tmem + col_o<D>(i), p + kk * 8, sdesc_advance(bv, kk * 2048), kIdescPV,
               accumulate | (kk > 0));
    };
    auto full = [&](uint32_t n) { return wwait(bar(C::kBarFull + n % kSlots), (n / kSlots) & 1); };
    // An item's first scores of query tile i, which sees nti > 0 key tiles.
    // After a tile's last scores its next Q may load.
    auto first_scores = [&](int i, uint32_t kn, int nti) {
      if (!wwait(bar(C::kBarQFull + i), q_ph[i]) || !full(kn)) return false;
      q_ph[i] ^= 1;
      tc_fence_after();
      if (leader) {
        scores(i, kn);
        if (nti == 1) mma_commit(bar(C::kBarQEmpty + i));
      }
      ++s_n[i];
      return true;
    };
    // An item as the tiles its two query tiles see.  Items without keys are met
    // in turn like the others: looking past them for the next one would wait for
    // roles that are still at this one.
    int cur[2], nxt[2];
    auto next_tiles = [&](int (&nt)[2]) {
      const bool some = next_item(ok);
      nt[0] = some ? nt0 : 0;
      nt[1] = some ? nt1 : 0;
      return some;
    };
    bool have = next_tiles(cur), started = false;  // started: cur's first scores are issued
    // K(m) is ring entry 2 * kv_it, V(m) entry 2 * kv_it + 1.  Behind each query
    // tile's product come its next scores (D = 64: before it).
    while (ok && have) {
      const bool more = next_tiles(nxt);
      const int nt = max(cur[0], cur[1]);
      if (nt > 0 && !started) {
        const uint32_t kn = 2 * kv_it;
        for (int i = 0; ok && i < 2; ++i)
          if (cur[i] > 0) ok = first_scores(i, kn, cur[i]);
        if (ok && leader) mma_commit(bar(C::kBarEmpty + kn % kSlots));
        if (!ok) break;
      }
      started = nt > 0 && max(nxt[0], nxt[1]) > 0;
      for (int m = 0; m + 1 < nt; ++m) {
        const uint32_t vn = 2 * kv_it + 1, nkn = 2 * kv_it + 2;
        if (!full(vn)) {
          ok = false;
          break;
        }
        tc_fence_after();
        bool k_ready = false;
        auto product = [&](int i) {
          if (m < cur[i]) {
            if (!wwait(bar(C::turn(C::kBarP, i, p_n[i])), C::parity(p_n[i]))) {
              return false;
            }
            ++p_n[i];
            tc_fence_after();
            if (leader) {
              values(i, vn, m > 0);
              if (D == 64 || m + 1 == cur[i])
                mma_commit(bar(C::turn(C::kBarO, i, p_n[i] - 1)));
            }
          }
          return true;
        };
        auto next_scores = [&](int i) {
          if (m + 1 < cur[i]) {
            if (!k_ready) {
              if (!full(nkn)) {
                return false;
              }
              tc_fence_after();
              k_ready = true;
            }
            if (leader) {
              scores(i, nkn);
              if (m + 2 == cur[i]) mma_commit(bar(C::kBarQEmpty + i));
            }
            ++s_n[i];
          }
          return true;
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ok = D == 128 ? product(i) && next_scores(i) : next_scores(i) && product(i);
          if (!ok) break;
        }
        if (!ok) break;
        if (leader) {
          mma_commit(bar(C::kBarEmpty + vn % kSlots));
          mma_commit(bar(C::kBarEmpty + nkn % kSlots));
        }
        ++kv_it;
      }
      if (!ok) break;
      if (nt > 0) {
        // The item's last key tile: behind its products come the next item's first
        // scores, so that the softmax finds them when it leaves the epilogue.
        const uint32_t vn = 2 * kv_it + 1, nkn = 2 * kv_it + 2;
        ok = full(vn);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (ok && nt == cur[i]) {
            ok = wwait(bar(C::turn(C::kBarP, i, p_n[i])), C::parity(p_n[i]));
            ++p_n[i];
            tc_fence_after();
            if (ok && leader) {
              values(i, vn, nt > 1);
              mma_commit(bar(C::turn(C::kBarO, i, p_n[i] - 1)));
            }
          }
          if (ok && nxt[i] > 0) ok = first_scores(i, nkn, nxt[i]);
        }
        if (ok && leader) {
          mma_commit(bar(C::kBarEmpty + vn % kSlots));
          if (started) mma_commit(bar(C::kBarEmpty + nkn % kSlots));
        }
        ++kv_it;
      }
      cur[0] = nxt[0];
      cur[1] = nxt[1];
      have = more;
    }
    if (!ok) {
      // Let every MMA already issued retire before TMEM is released.
      if (leader) mma_commit(bar(C::kBarDrain));
      mbar_drain(bar(C::kBarDrain), 0);
    }
  } else if (warp == 2 && !w.direct) {
    // ---------------------------------------------------------------- items
    Items items(a, w);
    bool some = true;
    for (uint32_t k = 0; some; ++k) {
      const uint32_t s = k % kFeed;
      if (!__all_sync(0xffffffffu, mbar_wait_short(bar(C::kBarFeedEmpty + s),
                                                   ((k / kFeed) & 1) ^ 1, wc)))
        break;
      some = items.next(b, g, h0);
      if (lane == 0) {
        slots[3 * s] = make_int4(b.qrow, b.nrows, b.krow, b.nk);
        slots[3 * s + 1] = make_int4(b.diag, g, h0, some);
        slots[3 * s + 2] = make_int4(key_tiles(b, a.causal, 0, kT),
                                     key_tiles(b, a.causal, row_step, kT), 0, 0);
        mbar_arrive(bar(C::kBarFeedFull + s));
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- softmax
    const int ti = (warp - 4) >> 2;  // query tile of this warpgroup
    const int wq = warp & 3;         // TMEM sub-partition = rows 32*wq ..
    const int row = wq * 32 + lane;  // row within the tile
    const uint32_t tl = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t colO = col_o<D>(ti);
    const float sl2 = a.scale_log2;
    uint32_t step = 0, o_ph = 0, kv_it = 0;
    bool ok = true;
    while (ok && next_item(ok)) {
      const int nt = ti == 0 ? nt0 : nt1;
      const int at = ti * row_step + row;  // row within the block
      const int end = a.causal ? min(b.nk, b.diag + at) : b.nk;  // keys that the row sees
      const bool live = at < b.nrows;
      float m = -INFINITY, l = 0.f;
      for (int t = 0; t < nt; ++t) {
        const int see = end - t * kT;  // visible columns of the tile
        const uint32_t colS = col_s<D>(ti, kv_it + t);
        if (!__all_sync(0xffffffffu, mbar_wait_short(bar(C::turn(C::kBarS, ti, step)),
                                                     C::parity(step), wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t r[128];
        tmem_ld32(tl + colS + 0, r + 0);
        tmem_ld32(tl + colS + 32, r + 32);
        tmem_ld32(tl + colS + 64, r + 64);
        tmem_ld32(tl + colS + 96, r + 96);
        tmem_wait_ld_regs(r);
        reg_fence32(r + 32);
        reg_fence32(r + 64);
        reg_fence32(r + 96);
        if (see < kT) {
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (j >= see) r[j] = __float_as_uint(-INFINITY);
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
        // Only the sequence's own rows have a say: a rescale changes the rounding.
        const bool need = live && m_tile - m > kWeightLag<kBf16>;
        const bool rescale = __any_sync(0xffffffffu, need);
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
          uint32_t p[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float a0 = ex2(fmaf(__uint_as_float(r[64 * h + 2 * j]), sl2, nm));
            const float a1 = ex2(fmaf(__uint_as_float(r[64 * h + 2 * j + 1]), sl2, nm));
            l0 += a0;
            l1 += a1;
            p[j] = pack16<kBf16>(a0, a1);
          }
          tmem_st32(tl + colS + 32 * h, p);
        }
        l += l0 + l1;
        if (rescale && t > 0) {
          // Softmax-state correction: O <- O * 2^(m_old - m_new).  The S
          // barrier of this tile also covers the previous P V product (D = 64:
          // it does not, and O's barrier completes with every product), and the
          // next one is issued only after the P barrier below.
          if (D == 64) {
            if (!__all_sync(0xffffffffu,
                            mbar_wait_short(bar(C::turn(C::kBarO, ti, step - 1)),
                                            C::parity(step - 1), wc))) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
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
        const int valid = b.nk - t * kT;
        if (valid < kT && (ti == 0 || t >= nt0)) {
          // V rows behind the sequence's end.  The warpgroup of the first
          // query tile that uses the V tile clears them: the other's product
          // is issued after its product.
          const uint32_t vn = 2 * (kv_it + t) + 1;
          if (!__all_sync(0xffffffffu,
                          mbar_wait_short(bar(C::kBarFull + vn % kSlots), (vn / kSlots) & 1, wc))) {
            ok = false;
            break;
          }
          if (row >= valid) {
            uint8_t* p = smem + C::kOffRing + (vn % kSlots) * C::kTileBytes + row * 128;
#pragma unroll
            for (int half = 0; half < C::kHalves; ++half)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(p + half * kBoxBytes + c * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_shared();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::turn(C::kBarP, ti, step)));
        ++step;
      }
      if (!ok) break;
      kv_it += max(nt0, nt1);
      // ------------------------------------------------------------ epilogue
      const int64_t qrow = b.qrow + at;
      const int head = h0 + ti * head_step;
      uint4* op = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                           (qrow * a.H + head) * D);
      float* lp = a.lse + (int64_t)head * a.Nq + qrow;
      if (nt == 0) {
        if (live) {
          for (int j = 0; j < D / 8; ++j) op[j] = make_uint4(0u, 0u, 0u, 0u);
          *lp = -INFINITY;
        }
        continue;
      }
      // D = 64: of the last product.
      if (!__all_sync(0xffffffffu,
                      mbar_wait_short(bar(C::turn(C::kBarO, ti, step - 1)),
                                      D == 128 ? o_ph : C::parity(step - 1), wc))) {
        ok = false;
        break;
      }
      o_ph ^= 1;
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing: 0
      // After the transpose this lane writes piece lane % 4 of each 64 bytes of
      // the quad's four rows.
      const int quad_at = at - (lane & 3);
      uint16_t* quad_out = static_cast<uint16_t*>(a.out) +
                           ((int64_t)(b.qrow + quad_at) * a.H + head) * D + (lane & 3) * 8;
      const int64_t row_step_out = (int64_t)a.H * D;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        tmem_ld32(tl + colO + cc * 32, o);
        tmem_wait_ld_regs(o);
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j].x = pack16<kBf16>(__uint_as_float(o[8 * j + 0]) * inv, __uint_as_float(o[8 * j + 1]) * inv);
          v[j].y = pack16<kBf16>(__uint_as_float(o[8 * j + 2]) * inv, __uint_as_float(o[8 * j + 3]) * inv);
          v[j].z = pack16<kBf16>(__uint_as_float(o[8 * j + 4]) * inv, __uint_as_float(o[8 * j + 5]) * inv);
          v[j].w = pack16<kBf16>(__uint_as_float(o[8 * j + 6]) * inv, __uint_as_float(o[8 * j + 7]) * inv);
        }
        quad_transpose(v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (quad_at + j < b.nrows)
            *reinterpret_cast<uint4*>(quad_out + j * row_step_out + cc * 32) = v[j];
        __syncwarp();
      }
      if (live) *lp = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
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
// host side
// ---------------------------------------------------------------------------

// Blocks that the plan may list: a sequence's last block of `rows` may be short.
int64_t most_blocks(int R, int Nq) { return (int64_t)Nq / kT + R; }

template <bool kBf16, int D>
cudaError_t run(const PromptArgs& a, Way by, int dev, int sms, cudaStream_t stream) {
  const int grp = a.H / a.Hkv;
  Work w;
  w.rows = grp % 2 == 0 ? kT : 2 * kT;
  w.inner = grp % 2 == 0 ? grp / 2 : grp;
  w.plan = nullptr;
  w.list = nullptr;
  w.direct = 0;
  CUtensorMap mq, mk, mv;
  // No keys at all: every item has no tiles, nothing is read through the maps.
  const bool keys = a.Nk > 0;
  if (!rows_map(&mq, a.q, kBf16, a.H, D, a.q_stride, a.Nq) ||
      !rows_map(&mk, keys ? a.k : a.q, kBf16, keys ? a.Hkv : a.H, D, keys ? a.k_stride : a.q_stride,
                keys ? a.Nk : a.Nq) ||
      !rows_map(&mv, keys ? a.v : a.q, kBf16, keys ? a.Hkv : a.H, D, keys ? a.v_stride : a.q_stride,
                keys ? a.Nk : a.Nq))
    return cudaErrorInvalidValue;
  const int smem = Cfg<D>::kSmemBytes;
  static DeviceOnce allowed;
  cudaError_t e = allowed.shared_memory(reinterpret_cast<const void*>(prompt_kernel<kBf16, D>), dev, smem);
  if (e != cudaSuccess) return e;
  const int64_t most = (a.Nq / w.rows + (int64_t)a.R) * a.Hkv * w.inner;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most < sms ? most : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  if (by == kDirect) {
    w.direct = 1;
  } else if (a.R > 1) {
    // The plan goes first; this kernel sets itself up meanwhile.
    Plan* plan = static_cast<Plan*>(a.workspace);
    Block* list = reinterpret_cast<Block*>(plan + 1);
    const int cap = (int)most_blocks(a.R, a.Nq);
    prompt_plan_kernel<<<1, 1024, 0, stream>>>(a, w.rows, cap, plan, list);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    w.plan = plan;
    w.list = list;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, prompt_kernel<kBf16, D>, mq, mk, mv, a, w);
}

}  // namespace

size_t prompt_workspace_bytes(int R, int Nq, int H, int D) {
  const size_t plan = sizeof(Plan) + (size_t)most_blocks(R, Nq) * sizeof(Block);
  const size_t line = line_workspace_bytes(Nq, H, D);
  return plan > line ? plan : line;
}

cudaError_t launch_prompt_attn(const PromptArgs& a, int dtype, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  TreeArgs t = {};
  t.q = a.q;
  t.q_stride = a.q_stride;
  t.k_cache = a.k;
  t.v_cache = a.v;
  t.cu = a.cu_q;
  t.out = a.out;
  t.lse = a.lse;
  t.R = a.R;
  t.N = a.Nq;
  t.H = a.H;
  t.Hkv = a.Hkv;
  t.D = a.D;
  t.scale = a.scale;
  t.scale_log2 = a.scale_log2;
  t.workspace = a.workspace;
  t.err = a.err;
  t.cu_k = a.cu_k;
  t.k_stride = a.k_stride;
  t.v_stride = a.v_stride;
  t.Nk = a.Nk;
  t.causal = a.causal;
  const auto [by, above] = prompt_way(t, sms);
  if (by == kSmall) {
    t.above = above;
    e = launch_small_attn(t, dtype, sms, stream);
    return e != cudaSuccess || above == 0 ? e : launch_line_attn(t, dtype, dev, sms, stream);
  }
  if (by == kLine) return launch_line_attn(t, dtype, dev, sms, stream);
  if (dtype == CPATTN_BF16)
    return a.D == 128 ? run<true, 128>(a, by, dev, sms, stream)
                      : run<true, 64>(a, by, dev, sms, stream);
  return a.D == 128 ? run<false, 128>(a, by, dev, sms, stream)
                    : run<false, 64>(a, by, dev, sms, stream);
}

}  // namespace cpattn
