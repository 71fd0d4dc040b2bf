// The line of products that the CTAs of k_weights_tc.cu share: which items there
// are, what each counts, where a CTA's part begins and which pieces of which items
// it walks.  Host and device, so that the CPU can check it.
#pragma once

#include <stdint.h>

#include "cpattn_internal.h"

namespace cpattn {
namespace wline {

// An item is 256 key positions of a kv head of a request; its steps are the tiles
// of `tpt` tokens that see any of them.
constexpr int kPair = 2 * kTcTile;
// What starting and ending an item costs, in steps.
constexpr int kItemCost = 1;
// Least part of the line for a CTA.
constexpr int kMinPart = 2;

// Which form of the kernel takes a call of N new tokens of R requests, G query heads a kv head:
// keys that stream past a request's rows (a deep ring of key tiles, one place for rows), or rows
// that stream past two key tiles.  The lengths themselves are on the device, so the mean decides.
// Measured (us, keys stream / rows stream; H = 32, Hkv = 8, D = 128, pages of 64):
//   32 requests of 16 tokens over 4000   68 / 84     64 single tokens over 1000-8192     127 / 170
//   32 of 30 (a tile of rows at most)    74 / 88     63 of them and a prompt of 100      152 / 170
//   32 of 33 (two tiles)                108 / 107    63 and a prompt of 500              246 / 174
//   32 of 100                           180 / 164    63 and a prompt of 2000             266 / 195
// So requests of more than one tile of rows are better off where rows stream; a prompt beside
// enough single tokens is not told apart from drafts of the same mean.
// Where keys stream a step of a request of several tiles waits for its rows: 1.7 us, and the
// loading of the key tile behind it waits for the item.  Up to kMostKeyRows rows that is 0.3 s
// at 1.5 GHz, where the bounded waits allow 2; the rows of the most that a call takes (2^27)
// stream past an item's keys in 1.4 s.
constexpr int64_t kMostKeyRows = (int64_t)1 << 24;
inline bool keys_stream(int R, int N, int G) {
  const int64_t rows = (int64_t)N * G;
  return rows <= (int64_t)R * kTcTile && rows <= kMostKeyRows;
}

__host__ __device__ inline int tiles_of(const Req& x, int tpt) { return (x.n + tpt - 1) / tpt; }
__host__ __device__ inline int items_of(const Req& x) { return (x.total + kPair - 1) / kPair; }
// First tile of tokens that sees position p or one behind it.
__host__ __device__ inline int first_tile(const Req& x, int tpt, bool chain, int p) {
  return chain && p > x.ctx ? (p - x.ctx) / tpt : 0;
}

// sum of floor((a i + b) / m) over i in [0, n), all >= 0 and m > 0: whole parts of a
// and b add up at once, and what is left counts the lattice points under a line, which
// are those of the line seen from the other axis.
__host__ __device__ inline long long floor_sum(long long n, long long m, long long a, long long b) {
  long long sum = 0;
  while (n > 0) {
    if (a >= m) {
      sum += n * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += n * (b / m);
      b %= m;
    }
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const long long t = m;
    m = a;
    a = t;
  }
  return sum;
}

// What the first m items of a kv head of the request count.
__host__ __device__ inline long long cost_upto(const Req& x, int tpt, bool chain, int m) {
  const int tiles = tiles_of(x, tpt);
  long long sum = (long long)m * (kItemCost + tiles);
  const int old = (x.ctx + kPair - 1) / kPair;  // items that begin within the old positions
  if (chain && tiles > 1 && m > old)
    sum -= floor_sum(m - old, tpt, kPair, (long long)old * kPair - x.ctx);
  return sum;
}
__host__ __device__ inline long long head_cost(const Req& x, int tpt, bool chain) {
  return x.n > 0 ? cost_upto(x, tpt, chain, items_of(x)) : 0;
}

// The line of length T is cut into n parts, part c beginning at floor(c T / n).
struct Cuts {
  long long q;
  int e, n;
  __host__ __device__ inline void init(long long T, int n_) {
    n = n_;
    q = n > 0 ? T / n : 0;
    e = (int)(T - q * n);
  }
  __host__ __device__ inline long long begin(int c) const {
    return c * q + (n > 0 ? (long long)c * e / n : 0);
  }
  // The part that holds unit t.
  __host__ __device__ inline int of(long long t) const {
    return (int)(((t + 1) * n - 1) / (q * n + e));
  }
};

// Steps [s0, s1) of an item of `steps`, step s being tile q0t + s of tokens.
struct Piece {
  Req x;
  int r, g, m, q0t, s0, s1, steps;
  long long item_at;  // where the item begins on the line
  bool last;   // the next piece's tile of tokens is not the one that this one ends on
  bool fresh;  // nor is this one's that of the piece before
  __host__ __device__ inline bool whole() const { return s0 == 0 && s1 == steps; }
  // First step of the piece that needs key tile i (0, 1); s1: none does.
  __host__ __device__ inline int begins(int i, int tpt, bool chain) const {
    const int p = m * kPair + i * kTcTile;
    if (p >= x.total) return s1;
    const int s = i == 0 ? s0 : first_tile(x, tpt, chain, p) - q0t;
    return s < s0 ? s0 : (s > s1 ? s1 : s);
  }
};

// Walks the pieces of one CTA, one piece ahead.
struct Walk {
  Piece p, ahead;
  bool more;       // ahead is a piece
  int tiles, items;  // of ahead's request (a division for each piece would hold up its warp)
  long long left;  // of the CTA's part
  int off;         // where it goes on within the item; -1: at the next item

  __host__ __device__ inline bool load(const TreeArgs& a) {
    do {
      if (++ahead.r >= a.R) return false;  // only if the lengths changed under the call
      load_req<true>(a, ahead.r, ahead.x);
    } while (ahead.x.n == 0);
    return true;
  }
  __host__ __device__ inline void request(int tpt) {
    tiles = tiles_of(ahead.x, tpt);
    items = items_of(ahead.x);
  }
  __host__ __device__ inline void item(int tpt, bool chain) {
    ahead.q0t = tiles > 1 ? first_tile(ahead.x, tpt, chain, ahead.m * kPair) : 0;
    ahead.steps = tiles - ahead.q0t;
  }
  // The part of n units begins in request r (x), `in_req` behind the request's begin,
  // at `at` on the line.
  __host__ __device__ inline void init(const TreeArgs& a, int tpt, int r, const Req& x,
                                       long long in_req, long long at, long long n) {
    const bool chain = a.tree == nullptr;
    left = n;
    more = false;
    // Every field has a value from the start.
    p = Piece();
    ahead = Piece();
    p.last = true;
    off = tiles = items = 0;
    if (left <= 0) return;
    ahead.r = r;
    ahead.x = x;
    const long long per = head_cost(x, tpt, chain);
    ahead.g = (int)(in_req / per);
    const long long rest = in_req - ahead.g * per;
    // The last item that begins at `rest` or before.
    const long long each = kItemCost + tiles_of(x, tpt);
    int lo, hi = items_of(x);
    if (!chain || tiles_of(x, tpt) == 1) {
      lo = (int)(rest / each);
    } else {
      lo = 0;
      while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (cost_upto(x, tpt, chain, mid) <= rest)
          lo = mid;
        else
          hi = mid;
      }
    }
    ahead.m = lo;
    off = (int)(rest - cost_upto(x, tpt, chain, lo));
    ahead.item_at = at - off;
    request(tpt);
    item(tpt, chain);
    advance(a, tpt);
  }
  __host__ __device__ inline void advance(const TreeArgs& a, int tpt) {
    const bool chain = a.tree == nullptr;
    more = false;
    while (left > 0) {
      if (off < 0) {
        off = 0;
        ahead.item_at += kItemCost + ahead.steps;
        if (++ahead.m == items) {
          ahead.m = 0;
          if (++ahead.g == a.Hkv) {
            ahead.g = 0;
            if (!load(a)) {
              left = 0;
              return;
            }
            request(tpt);
          }
        }
        item(tpt, chain);
      }
      const int rest = kItemCost + ahead.steps - off;
      const int n = (int)(left < rest ? left : rest);
      ahead.s0 = off > kItemCost ? off - kItemCost : 0;
      ahead.s1 = off + n > kItemCost ? off + n - kItemCost : 0;
      left -= n;
      off = n == rest ? -1 : off + n;
      if (ahead.s1 > ahead.s0) {
        more = true;
        return;
      }
    }
  }
  // keep: a tile of tokens that is its request's only one serves the next piece too.
  __host__ __device__ inline bool next(const TreeArgs& a, int tpt, bool keep) {
    if (!more) return false;
    const bool fresh = p.last, only = tiles == 1;
    p = ahead;
    p.fresh = fresh;
    advance(a, tpt);
    p.last = !(keep && more && ahead.r == p.r && ahead.g == p.g && only);
    return true;
  }
};

}  // namespace wline
}  // namespace cpattn
