// Which kernel answers a call, from its sizes (the lengths themselves are on the
// device), and what the kernels are estimated to take.  Host only; its choices are
// checked without a GPU.
#pragma once

#include <math.h>
#include <stdint.h>

#include "cpattn_internal.h"

namespace cpattn {

// The CUDA-core kernel.  Few blocks: eight warps a block, two heads and four keys' loads at a time.
// Many: four warps, four heads (fewer blocks read a key twice), two keys.
inline bool few_blocks(const TreeArgs& a, int sms) {
  const int G = a.H / a.Hkv;
  return (int64_t)a.N * a.Hkv * ((G + 1) / 2) <= 2 * sms;
}

// What it and the tensor cores' cut line take for `keys` keys a request (us,
// estimated).  Measured, one token a request, H = 32, Hkv = 8, D = 128 (us, CUDA cores
// / cut line), by requests and keys:
//            1 key        16          64         256        1000
//     1    4.5 / 11.8  4.8 / 11.4  6.2 / 11.4  11 / 13    29 / 13
//     8    5.0 / 13.8  5.7 / 13.5  7.0 / 13.5  12 / 17    34 / 21
//    64    5.8 / 28    7.7 / 27     13 / 28    34 / 41   109 / 60
//   256     16 / 79     23 / 77     44 / 77   121 / 119  418 / 181
// The estimates below follow these within a fifth.
inline float small_attn_us(const TreeArgs& a, int64_t keys, int sms) {
  const int G = a.H / a.Hkv, heads = G < 4 ? G : 4;
  const float kd = (float)keys * a.D;
  if (few_blocks(a, sms)) return 4.6f + 1.6f * ceilf(kd / 8192.f);
  const float blocks = (float)a.N * a.Hkv * ((G + heads - 1) / heads);
  const float latency = 4.6f + kd / 2048.f;
  const float work = 5.f + blocks * (0.0052f + 1.52e-6f * kd * (0.35f + 0.1625f * heads));
  return latency > work ? latency : work;
}

inline float line_attn_us(const TreeArgs& a, int64_t keys) {
  const int64_t rows = (int64_t)a.N * (a.H / a.Hkv) / a.R;  // of a request and kv head
  const float items = (float)a.R * a.Hkv * (1 + rows / 256);
  return 12.f + items * (0.032f + 0.0095f * ceilf((float)keys / 128.f) * a.D / 128.f);
}

// How a call is done, from its means (the lengths themselves are on the device).
//  kSmall: a block a token and kv head on CUDA cores (k_answer_small.cu).
//  kDirect: at most an item a CTA; each CTA finds its own, nothing is planned.
//  kLine: few rows and many keys a sequence; the keys of an item are shared
//    among CTAs and a kv head's query heads share a row tile (k_tree_tc.cu).
//  kSorted: the rest.
// Measured (us, H = 32, Hkv = 8, D = 128; direct or sorted / line), for sequences
// of nq queries behind 1 to n keys:
//   1 x   1, n 1000: 10.8 / 12.8    4 x  1, n 1000: 19.0 / 14.2   16 x  1, n 8000: 99 / 54
//   1 x   1, n 8000: 20.2 / 13.7    4 x 32, n 1000: 18.6 / 18.3   16 x 32, n    1: 17.6 / 15.0
//   4 x 128, n 8000: 82.5 / 57.5    4 x 64, n 1000: 18.5 / 25.1   16 x 64, n 1000: 29.6 / 42.9
// and without keys in front (small / direct, line or sorted):
//   1 x 16:  5.3 /  9.4    8 x  4:  5.3 / 10.8    64 x  4: 15 / 28
//   1 x 64:  9.2 /  9.4    8 x 16:  9.6 / 10.8    64 x 16: 49 / 31
enum Way : int { kSmall, kDirect, kLine, kSorted };

struct PromptWay {
  Way by;
  int above;  // kSmall: sequences of so many keys and more go to the cut line (0: none do)
};

// Only the means are known, and one block or CTA of kSmall and kDirect walks all keys of
// its rows: in an uneven batch, or one padded with empty sequences, the longest
// decides.  So both are also taken at their worst, all keys in one sequence.
//  - kDirect, where that could cost more than the choice wins: the cut line.
//  - kSmall, where it could take more than three times as long as the next best: sequences
//    with several times the mean of keys are left to the cut line, a second kernel (and
//    its merge) behind the first.
// Measured (us, this choice / by the means alone; H = 32, Hkv = 8, D = 128):
//   one of 400 among 63 of 1: 28 / 92          256 x 1, one behind 16384: 30 / 660
//   one of 2000 in 512 slots: 86 / 1690        4 x 128, one behind 4000: 29 / 58
//   38 x 1, one behind 19000, H = 8, Hkv = 1: 15 / 235
// and what an even batch pays for it:
//   64 x 1 behind 16: 10.5 / 5.2    64 x 8: 28 / 22    4 x 64 behind 1000: 25 / 19
inline PromptWay prompt_way(const TreeArgs& a, int sms) {
  if (a.Nk == 0) return {kSorted, 0};
  const int G = a.H / a.Hkv;
  const int64_t items = ((int64_t)a.N / kTcTile + a.R) * (G % 2 == 0 ? a.H / 2 : a.H);
  const int64_t rows = (int64_t)a.N * G / a.R, keys = a.Nk / a.R;
  auto direct_us = [](int64_t n) { return 8.f + 1.5f * (float)(n / kTcTile + 1); };
  Way by = items <= sms ? kDirect : kSorted;
  const float tiles = (float)(keys / kTcTile + 1);  // of the longest rows
  float us = by == kDirect ? direct_us(keys) : 14.f + items * (3.f + 1.6f * tiles) / sms;
  if (rows <= kTcTile) {
    const float line = line_attn_us(a, keys);
    if (keys > 512 || by == kSorted || (a.R > 1 && direct_us(a.Nk) > 2.f * line)) {
      by = kLine;
      us = line;
    }
  } else if (by == kDirect) {
    // Whether the CTAs without an item would help more than the sharing costs.
    const float mean = a.causal && a.Nk == a.N ? 0.5f * tiles : tiles;
    const float line = 20.f + 1.7f * mean * a.N * a.H / (2 * kTcTile) / sms;
    if (line < us || (a.R > 1 && us * direct_us(a.Nk) > line * line)) {
      by = kLine;
      us = line;
    }
  }
  // Under the causal rule a row sees about the keys in front of its sequence's
  // queries and half of those among them.
  const int64_t all = a.causal ? (a.Nk > a.N ? a.Nk - a.N / 2 : a.Nk / 2) : a.Nk;
  if (small_attn_us(a, all / a.R + 1, sms) >= us) return {by, 0};
  const bool even = small_attn_us(a, all + 1, sms) <= 3.f * us;
  return {kSmall, even || a.R == 1 ? 0 : (int)(keys < 8 ? 32 : 4 * keys)};
}

}  // namespace cpattn
