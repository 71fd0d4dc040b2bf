// Rotary positions: q and k (or their gradients) turned on their way into or out
// of the ring, and a step's tokens turned on their way into the paged cache.
//
//   (a, b) -> (m (a cos pf - s b sin pf), m (s a sin pf + b cos pf)),  s = +-1
//
// for each pair of the first `rot` values of a head; the rest is copied.
//
// The angle p f of a far position has lost its fraction in float32 (p = 10^6: off
// by 0.03).  Here a frequency is held as the fraction of a turn a position, in
// units of 2^-64 of a turn, to the nearest; its product with the position, modulo
// 2^64, is the angle without the whole turns, off by half a unit a position (2^-22
// at 2^40), at the price of three 32-bit products.  It is split at the nearest
// quarter turn, so that sine and cosine are taken of at most an eighth of one.
// For float32 they come from sincospif; for 16-bit outputs from __sinf and
// __cosf, whose 2^-21 (absolute) moves a value by 2^-21 (|a| + |b|) at most: far below
// half a step (2^-12) of a value as large as its pair, not of one that nearly cancels.
//
// Both calls are bound by HBM: each value is read and written once, in 16-byte
// vectors where rot allows it.  A thread holds the same vectors of each head (both
// partners of their pairs), so its sines and cosines serve several heads of a token.
// Measured: 131072 tokens of 32 heads of 128 into the ring's order in bfloat16 316 us
// (6.8 TB/s, the copy rate), 2 x 16384 in float32 out of it 163 us (6.6 TB/s); 32001
// tokens of 32 + 8 + 8 heads into the cache 126 us (6.2 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "cpattn.h"
#include "cpattn_internal.h"
#include "tc_ptx.cuh"

namespace cpattn {
namespace {

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
  return n > 0 ? n : 148;
}

constexpr int kThreads = 256;
// Blocks an SM (registers allow what is in flight): 131072 tokens of 32 heads of 128 in
// bfloat16 take 437 us with 2, 316 with 3, 551 with 4 (which spills).
constexpr int kResident = 3;
// Threads an SM from which on a thread takes more heads (and fewer sines).
constexpr int kEnough = 2048;
constexpr int kMostPairs = 128;  // of a head (D at most 256)

// kVec values as they lie in memory.
template <int kBytes>
struct Raw;
template <>
struct Raw<16> {
  typedef uint4 type;
};
template <>
struct Raw<8> {
  typedef uint2 type;
};
template <>
struct Raw<4> {
  typedef uint32_t type;
};
template <>
struct Raw<2> {
  typedef uint16_t type;
};

// Two 16-bit values as they lie in a word.
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float x, float y) {
  return tc::pack16<std::is_same<T, __nv_bfloat16>::value>(x, y);
}

// kVec values as 32-bit words.
template <typename T, int kVec>
struct Values {
  static constexpr int kBytes = sizeof(T) * kVec, kWords = kBytes < 4 ? 1 : kBytes / 4;
  typedef typename Raw<kBytes>::type Raw_;
  uint32_t w[kWords];
  __device__ __forceinline__ void read(const T* p) {
    const Raw_ r = *reinterpret_cast<const Raw_*>(p);
    if constexpr (kBytes == 2)
      w[0] = r;
    else
      memcpy(w, &r, kBytes);
  }
  __device__ __forceinline__ void write(T* p) const {
    Raw_ r;
    if constexpr (kBytes == 2)
      r = (uint16_t)w[0];
    else
      memcpy(&r, w, kBytes);
    *reinterpret_cast<Raw_*>(p) = r;
  }
};

// Fraction of a turn a position, in units of 2^-64, to the nearest: 1 / 2 pi and its product
// with f as sums of two (a product rounded to 53 bits is off by up to 2^-53 of the angle: 2^-22
// at position 2^31, 2^-13 at 2^40).
__device__ __forceinline__ unsigned long long turns(double f) {
  const double inv = 0.15915494309189535, inv_rest = -9.839338337591243e-18;
  const double t = __dmul_rn(f, inv), rest = __fma_rn(f, inv, -t) + f * inv_rest;
  double part = t - rint(t);  // exact
  if (part >= 0.5) part -= 1.0;
  const double units = part * 18446744073709551616.0, whole = rint(units);
  return (unsigned long long)(__double2ll_rn(whole) +
                              __double2ll_rn((units - whole) + rest * 18446744073709551616.0));
}

// Sine and cosine of `phase` units of 2^-64 turns.
template <bool kPrecise>
__device__ __forceinline__ void sine_cosine(unsigned long long phase, float& s, float& c) {
  const uint32_t p = (uint32_t)(phase >> 32);
  const uint32_t quarter = (p + 0x20000000u) >> 30;
  const float r = (float)(int)(p - (quarter << 30));  // within an eighth of a turn
  float s0, c0;
  if constexpr (kPrecise) {
    sincospif(r * 4.656612873077393e-10f, &s0, &c0);  // 2^-31
  } else {
    const float a = r * 1.4629180792671596e-09f;  // 2 pi 2^-32
    s0 = __sinf(a);
    c0 = __cosf(a);
  }
  s = quarter & 1 ? c0 : s0;
  c = quarter & 1 ? s0 : c0;
  if (quarter & 2) s = -s;
  if ((quarter + 1) & 2) c = -c;
}

// What a thread does with each head: the vectors at `at` (both partners, split by
// rot / 2, unless the pairs lie side by side) or, behind the first rot values, a copy.
template <typename T, int kVec, bool kInterleaved>
struct Turn {
  static constexpr int kPairs = kInterleaved ? kVec / 2 : kVec;
  static constexpr int kVecs = kInterleaved ? 1 : 2;
  float c[kPairs], s[kPairs];
  const unsigned long long* f;  // of its first pair, in shared memory
  int at, half;
  bool turns_;

  // Units of a head: those that turn, then those that copy.
  __host__ __device__ static int turning(int rot) { return rot / (kVec * kVecs); }
  __host__ __device__ static int units(int D, int rot) { return turning(rot) + (D - rot) / kVec; }

  // table: rot / 2 values, filled by the block.
  __device__ __forceinline__ void init(int unit, int rot, const double* freqs,
                                       unsigned long long* table) {
    for (int i = threadIdx.x; i < rot / 2; i += kThreads) table[i] = turns(freqs[i]);
    __syncthreads();
    const int n = turning(rot);
    turns_ = unit < n;
    half = rot / 2;
    at = turns_ ? unit * kVec : rot + (unit - n) * kVec;
    f = table + unit * kPairs;
  }
  __device__ __forceinline__ void angles(long long position, float magnitude, float sign) {
    if (!turns_) return;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      sine_cosine<sizeof(T) == 4>(f[i] * (unsigned long long)position, s[i], c[i]);
      s[i] *= magnitude * sign;
      c[i] *= magnitude;
    }
  }
  __device__ __forceinline__ void load(const T* x, Values<T, kVec> (&v)[kVecs]) const {
    v[0].read(x + at);
    if (kVecs == 2 && turns_) v[kVecs - 1].read(x + at + half);
  }
  __device__ __forceinline__ void pair(int i, float& x, float& y) const {
    const float u = x;
    x = u * c[i] - y * s[i];
    y = u * s[i] + y * c[i];
  }
  __device__ __forceinline__ void turn(Values<T, kVec> (&v)[kVecs]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        uint32_t& a = kInterleaved ? v[0].w[2 * i] : v[0].w[i];
        uint32_t& b = kInterleaved ? v[0].w[2 * i + 1] : v[kVecs - 1].w[i];
        float x = __uint_as_float(a), y = __uint_as_float(b);
        pair(i, x, y);
        a = __float_as_uint(x);
        b = __float_as_uint(y);
      }
    } else if constexpr (kInterleaved) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        float2 x = unpack<T>(v[0].w[i]);
        pair(i, x.x, x.y);
        v[0].w[i] = pack<T>(x.x, x.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < Values<T, kVec>::kWords; ++i) {
        float2 x = unpack<T>(v[0].w[i]), y = unpack<T>(v[kVecs - 1].w[i]);
        pair(kVec > 1 ? 2 * i : 0, x.x, y.x);
        if (kVec > 1) pair(kVec > 1 ? 2 * i + 1 : 0, x.y, y.y);
        v[0].w[i] = pack<T>(x.x, x.y);
        v[kVecs - 1].w[i] = pack<T>(y.x, y.y);
      }
    }
  }
  // n heads from `from` to `to`, turned or as they are; all loads of four before their stores.
  template <typename Step>
  __device__ __forceinline__ void move(const T* from, Step from_step, T* to, Step to_step, int n,
                                       bool turned) const {
    constexpr int U = 4;
    for (int h = 0; h < n; h += U) {
      Values<T, kVec> v[U][kVecs];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (h + j < n) load(from + (h + j) * from_step, v[j]);
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (h + j < n) {
          if (turned) turn(v[j]);
          store(to + (h + j) * to_step, v[j]);
        }
    }
  }
  __device__ __forceinline__ void store(T* x, const Values<T, kVec> (&v)[kVecs]) const {
    v[0].write(x + at);
    if (kVecs == 2 && turns_) v[kVecs - 1].write(x + at + half);
  }
};

// ---------------------------------------------------------------------------
// In and out of the ring.  Consecutive threads take the units of a token, then
// the token's groups of heads, then the next tokens of out; a block steps through
// out's tokens.  In place nothing is copied (units of a head: `units`).
// ---------------------------------------------------------------------------
template <typename T, int kVec, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kResident) rotary_kernel(const RotaryArgs a, int units, int groups,
                                                          int per_group) {
  typedef Turn<T, kVec, kInterleaved> Unit;
  // The unit and the group are the same in each step: the stride is a multiple of
  // units * groups threads.
  const int per_token = units * groups;
  const int tokens = kThreads / per_token;  // of a step of the block
  const int lane = threadIdx.x % per_token;
  __shared__ unsigned long long table[kMostPairs];
  Unit u;
  u.init(lane % units, a.rot, a.freqs, table);
  if ((int)threadIdx.x >= tokens * per_token) return;
  const int h0 = lane / units * per_group, h1 = min(a.H, h0 + per_group);
  const long long total = (long long)a.B * a.S_out;
  for (long long i = (long long)blockIdx.x * tokens + threadIdx.x / per_token; i < total;
       i += (long long)gridDim.x * tokens) {
    const int b = (int)(i / a.S_out), p = (int)(i - (long long)b * a.S_out);
    const int n = a.to_sharded ? natural_pos(a.ring, p) : p;
    T* out = static_cast<T*>(a.out) + i * a.out_stride;
    if (n >= a.S_nat) {  // padding
      Values<T, kVec> zero[Unit::kVecs] = {};
      for (int h = h0; h < h1; ++h) u.store(out + h * a.D, zero);
      continue;
    }
    const long long from = (long long)b * a.S_in + (a.from_sharded ? sharded_pos(a.ring, n) : n);
    const T* x = static_cast<const T*>(a.x) + from * a.x_stride;
    u.angles(a.positions ? a.positions[b * a.positions_stride + n] : a.offset + n, a.magnitude,
             a.sign);
    u.move(x + h0 * a.D, a.D, out + h0 * a.D, a.D, h1 - h0, u.turns_);
  }
}

template <typename T, int kVec, bool kInterleaved>
cudaError_t run(const RotaryArgs& a, cudaStream_t stream) {
  typedef Turn<T, kVec, kInterleaved> Unit;
  const bool in_place = a.x == a.out && a.S_nat == a.S_out;
  const int units = in_place ? Unit::turning(a.rot) : Unit::units(a.D, a.rot);
  // All heads a thread where that leaves threads enough for the SMs.
  const long long total = (long long)a.B * a.S_out;
  const long long full = (long long)sm_count() * kEnough;
  int per_group = a.H;
  while (per_group > 1 &&
         total * units * ((a.H + per_group - 1) / per_group) < full &&
         units * ((a.H + (per_group + 1) / 2 - 1) / ((per_group + 1) / 2)) <= kThreads)
    per_group = (per_group + 1) / 2;
  const int groups = (a.H + per_group - 1) / per_group;
  const int tokens = kThreads / (units * groups);
  long long grid = (total + tokens - 1) / tokens;
  const long long cap = (long long)sm_count() * 16;
  if (grid > cap) grid = cap;
  rotary_kernel<T, kVec, kInterleaved><<<(unsigned)grid, kThreads, 0, stream>>>(a, units, groups,
                                                                               per_group);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// A step's tokens.  A thread holds the same vectors of `per_group` heads of q, of k or
// of v: consecutive threads take the units, then the groups, then the next tokens.
// ---------------------------------------------------------------------------
constexpr int kWriteThreads = 384;  // three groups of the narrowest units (127) at least
// Heads a thread has in flight: 32001 tokens of 32 + 8 + 8 heads of 128 take 175 us with 1,
// 126 with 2, 152 with 4 (which spills); with two blocks an SM that step through the tokens.
// 142 with sixteen times as many (each makes the table of frequencies).
constexpr int kMostHeads = 2;

template <typename T, int kVec, bool kInterleaved>
__global__ void __launch_bounds__(kWriteThreads, 2)
    rotary_write_kernel(const RotaryWriteArgs a, int units, int q_groups, int groups, int per_group) {
  typedef Turn<T, kVec, kInterleaved> Unit;
  const int per_token = units * groups;
  const int tokens = kWriteThreads / per_token;
  const int lane = threadIdx.x % per_token;
  __shared__ unsigned long long table[kMostPairs];
  Unit u;
  u.init(lane % units, a.rot, a.freqs, table);
  if ((int)threadIdx.x >= tokens * per_token) return;
  int group = lane / units, kind = 0;  // 0: q, 1: k, 2: v
  if (group >= q_groups) {
    const int kv_groups = (groups - q_groups) / 2;
    group -= q_groups;
    kind = group < kv_groups ? 1 : 2;
    if (kind == 2) group -= kv_groups;
  }
  const int heads = kind == 0 ? a.H : a.Hkv, h0 = group * per_group, n = min(per_group, heads - h0);
  const T* x = static_cast<const T*>(kind == 0 ? a.q : (kind == 1 ? a.k : a.v)) + h0 * a.D;
  const int64_t x_stride = kind == 0 ? a.q_stride : (kind == 1 ? a.k_stride : a.v_stride);
  const int64_t step = kind == 0 ? a.D : a.cache.head_stride;
  T* to = static_cast<T*>(kind == 0 ? a.out : (kind == 1 ? a.k_cache : a.v_cache)) + h0 * step;
  // In place nothing is copied.
  const bool turned = u.turns_ && kind < 2, idle = kind == 0 && !u.turns_ && a.q == a.out;
  const long long places = a.cache.num_pages * a.cache.page_size;
  for (long long i = (long long)blockIdx.x * tokens + threadIdx.x / per_token; i < a.N;
       i += (long long)gridDim.x * tokens) {
    if (idle) continue;
    const T* from = x + i * x_stride;
    const long long slot = kind != 0 ? a.slots[i] : 0;
    if (turned) u.angles(a.positions[i], a.magnitude, 1.f);
    T* row = to + i * a.out_stride;
    if (kind != 0) {
      if (slot >= places && kind == 1 && h0 == 0 && lane % units == 0)
        atomicExch(a.err, kErrBadTables);
      if (slot < 0 || slot >= places) continue;
      const int page = (int)slot / a.cache.page_size;
      row = to + page * a.cache.page_stride +
            ((int)slot - page * a.cache.page_size) * a.cache.token_stride;
    }
    for (int h = 0; h < n; h += kMostHeads) {
      Values<T, kVec> v[kMostHeads][Unit::kVecs];
#pragma unroll
      for (int j = 0; j < kMostHeads; ++j)
        if (h + j < n) u.load(from + (h + j) * a.D, v[j]);
#pragma unroll
      for (int j = 0; j < kMostHeads; ++j) {
        if (h + j < n) {
          if (turned) u.turn(v[j]);
          u.store(row, v[j]);
        }
        row += step;
      }
    }
  }
}

template <typename T, int kVec, bool kInterleaved>
cudaError_t run(const RotaryWriteArgs& a, cudaStream_t stream) {
  typedef Turn<T, kVec, kInterleaved> Unit;
  const int units = Unit::units(a.D, a.rot);
  // Few heads a thread where there are few tokens; more where a token needs more threads
  // than a block has.
  const long long full = (long long)sm_count() * kEnough;
  int per_group = 1, q_groups, groups;
  while (true) {
    q_groups = (a.H + per_group - 1) / per_group;
    groups = q_groups + 2 * ((a.Hkv + per_group - 1) / per_group);
    if (units * groups <= kWriteThreads &&
        (per_group >= kMostHeads || a.N * units * groups <= full))
      break;
    per_group *= 2;
  }
  const int tokens = kWriteThreads / (units * groups);
  long long grid = (a.N + tokens - 1) / tokens;
  const long long cap = (long long)sm_count() * 2;
  if (grid > cap) grid = cap;
  rotary_write_kernel<T, kVec, kInterleaved><<<(unsigned)grid, kWriteThreads, 0, stream>>>(
      a, units, q_groups, groups, per_group);
  return cudaGetLastError();
}

// The widest vectors (16 bytes down to one pair's share) that rot and rot / 2 allow.
template <typename T, typename Args>
cudaError_t run_vec(const Args& a, bool interleaved, cudaStream_t stream) {
  constexpr int kMost = 16 / sizeof(T);
  const int step = interleaved ? a.rot : a.rot / 2;
  if (interleaved) {
    if (step % kMost == 0) return run<T, kMost, true>(a, stream);
    return run<T, 2, true>(a, stream);
  }
  if (step % kMost == 0) return run<T, kMost, false>(a, stream);
  if (step % 2 == 0) return run<T, 2, false>(a, stream);
  return run<T, 1, false>(a, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, bool interleaved, cudaStream_t stream) {
  if (dtype == CPATTN_F32) return run_vec<float>(a, interleaved, stream);
  if (dtype == CPATTN_BF16) return run_vec<__nv_bfloat16>(a, interleaved, stream);
  return run_vec<__half>(a, interleaved, stream);
}

cudaError_t launch_rotary_write(const RotaryWriteArgs& a, int dtype, bool interleaved,
                                cudaStream_t stream) {
  if (dtype == CPATTN_BF16) return run_vec<__nv_bfloat16>(a, interleaved, stream);
  return run_vec<__half>(a, interleaved, stream);
}

}  // namespace cpattn
