// The line of key tiles that the CTAs of k_tree_tc.cu share: which items there
// are, what each counts, where a CTA's part begins and which pieces of which
// items it walks.  Host and device, so that the CPU can check it.
#pragma once

#include <stdint.h>

#include "cpattn_internal.h"

namespace cpattn {
namespace line {

// What starting and ending an item costs, in key tiles.  64 single tokens over
// 100-8192 cached ones (H = 32, Hkv = 8, D = 128): 205 us at 1, 196 at 2, 192 at 3.
constexpr int kItemCost = 3;
// Least part of the line for a CTA (one token over 1000: 13.9 us at 1, 14.4 at 2).
constexpr int kMinPart = 1;

// An item is a kv head of a request and `span` of its tokens.
__host__ __device__ inline int items_of(const Req& x, int span) { return (x.n + span - 1) / span; }
// Key tiles of the request's m-th item (at least one, so that its rows are
// written); without a tree no row sees behind the item's last token.
__host__ __device__ inline int tiles_of(const Req& x, int span, bool chain, int m) {
  const int last = x.n < (m + 1) * span ? x.n : (m + 1) * span;
  const int end = chain && x.ctx + last < x.total ? x.ctx + last : x.total;
  return end > 0 ? (end + kTcTile - 1) / kTcTile : 1;
}
// What a kv head of the request counts on the line.
__host__ __device__ inline long long head_cost(const Req& x, int span, bool chain) {
  long long s = 0;
  for (int m = 0, e = items_of(x, span); m < e; ++m) s += kItemCost + tiles_of(x, span, chain, m);
  return s;
}

// The line of length T is cut into n parts, part c beginning at floor(c T / n)
// = c q + floor(c e / n) with T = q n + e (small numbers but for one division).
__host__ __device__ inline long long div_small(long long x, int n) {
  return x <= 0xffffffffll ? (long long)((uint32_t)x / (uint32_t)n) : x / n;
}
struct Cuts {
  long long q;
  int e, n;
  __host__ __device__ inline void init(long long T, int n_) {
    n = n_;
    q = n > 0 ? div_small(T, n) : 0;
    e = (int)(T - q * n);
  }
  __host__ __device__ inline long long begin(int c) const {
    return c * q + (n > 0 ? c * e / n : 0);
  }
  // The part that holds unit t.
  __host__ __device__ inline int of(long long t) const {
    return (int)(((t + 1) * n - 1) / (q * n + e));
  }
};

// A run of key tiles [t0, t1) of one item.
struct Piece {
  Req x;
  int r, g, m, t0, t1, tiles;
  long long item_at;  // where the item begins on the line
};

// Walks the pieces of one CTA.
template <bool kPaged>
struct Walk {
  Piece p;
  long long left;  // of the CTA's part
  int off;         // where it goes on within the item; -1: at the next item
  int items;

  // The part begins in request r (x), `in_req` behind the request's begin, at
  // `at` on the line.
  __host__ __device__ inline void init(const TreeArgs& a, int span, int r, const Req& x,
                                       long long in_req, long long at, long long n) {
    left = n;
    if (left <= 0) return;
    p.r = r;
    p.x = x;
    items = items_of(x, span);
    const long long per = head_cost(x, span, a.tree == nullptr);
    p.g = per <= 0x7fffffffll ? (int)div_small(in_req, (int)per) : (int)(in_req / per);
    long long rest = in_req - p.g * per;
    p.m = 0;
    while (true) {
      const int t = kItemCost + tiles_of(x, span, a.tree == nullptr, p.m);
      if (rest < t) break;
      rest -= t;
      ++p.m;
    }
    off = (int)rest;
    p.item_at = at - rest;
    p.tiles = 0;
  }
  __host__ __device__ inline bool next(const TreeArgs& a, int span) {
    while (left > 0) {
      if (off < 0) {
        off = 0;
        p.item_at += kItemCost + p.tiles;
        if (++p.m == items) {
          p.m = 0;
          if (++p.g == a.Hkv) {
            p.g = 0;
            do {
              if (++p.r >= a.R) {  // only if the lengths changed under the call
                left = 0;
                return false;
              }
              load_line_req<kPaged>(a, p.r, p.x);
            } while (p.x.n == 0);
            items = items_of(p.x, span);
          }
        }
      }
      p.tiles = tiles_of(p.x, span, a.tree == nullptr, p.m);
      const int rest = kItemCost + p.tiles - off;
      const int n = (int)(left < rest ? left : rest);
      p.t0 = off > kItemCost ? off - kItemCost : 0;
      p.t1 = off + n > kItemCost ? off + n - kItemCost : 0;
      left -= n;
      off = n == rest ? -1 : off + n;
      if (p.t1 > p.t0) return true;
    }
    return false;
  }
};

}  // namespace line
}  // namespace cpattn
