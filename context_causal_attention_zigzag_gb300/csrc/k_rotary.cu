// Rotary positions: q and k (or their gradients) turned on their way into or out
// of the ring, and a step's tokens turned on their way into the paged cache.
//
//   (a, b) -> (m (a cos pf - s b sin pf), m (s a sin pf + b cos pf)),  s = +-1
//
// for each pair of the first `rot` values of a head; the rest is copied.
//
// The angle p f of a far position has lost its fraction in float32 (p = 10^6: off
// by 0.03).  Here a frequency is held as the fraction of a turn a position, in
// units of 2^-64 of a turn; its product with the position, modulo 2^64, is the
// angle without the whole turns, exact but for the frequency's own rounding
// (2^-53), at the price of three 32-bit products.  It is split at the nearest
// quarter turn, so that sine and cosine are taken of at most an eighth of one.
// For float32 they come from sincospif; for 16-bit outputs from __sinf and
// __cosf, whose 2^-21 is far below half a step of the output (2^-12).
//
// Both calls are bound by HBM: each value is read and written once, in 16-byte
// vectors where rot allows it.  A thread holds the same vectors of each head (both
// partners of their pairs), so its sines and cosines serve all heads of a token.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cpattn.h"
#include "cpattn_internal.h"

namespace cpattn {
namespace {

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
  return n > 0 ? n : 148;
}

constexpr int kThreads = 256;

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

template <typename T>
__device__ __forceinline__ float to_float(T x) {
  return static_cast<float>(x);
}
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x) {
  return __float2half_rn(x);
}

template <typename T, int kVec>
union Values {
  typename Raw<sizeof(T) * kVec>::type raw;
  T v[kVec];
  __device__ __forceinline__ Values() {}
};

// Fraction of a turn a position, in units of 2^-64.
__device__ __forceinline__ unsigned long long turns(double f) {
  const double t = f * 0.15915494309189535;  // 1 / 2 pi
  return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
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
  unsigned long long f[kPairs];
  float c[kPairs], s[kPairs];
  int at, half;
  bool turns_;

  // Units of a head: those that turn, then those that copy.
  __host__ __device__ static int turning(int rot) { return rot / (kVec * kVecs); }
  __host__ __device__ static int units(int D, int rot) { return turning(rot) + (D - rot) / kVec; }

  __device__ __forceinline__ void init(int unit, int rot, const double* freqs) {
    const int n = turning(rot);
    turns_ = unit < n;
    half = rot / 2;
    at = turns_ ? unit * kVec : rot + (unit - n) * kVec;
    if (turns_) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) f[i] = turns(freqs[unit * kPairs + i]);
    }
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
    v[0].raw = *reinterpret_cast<const decltype(v[0].raw)*>(x + at);
    if (kVecs == 2 && turns_)
      v[kVecs - 1].raw = *reinterpret_cast<const decltype(v[0].raw)*>(x + at + half);
  }
  __device__ __forceinline__ void turn(Values<T, kVec> (&v)[kVecs]) const {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      T& a = kInterleaved ? v[0].v[2 * i] : v[0].v[i];
      T& b = kInterleaved ? v[0].v[2 * i + 1] : v[kVecs - 1].v[i];
      const float x = to_float(a), y = to_float(b);
      a = from_float<T>(x * c[i] - y * s[i]);
      b = from_float<T>(x * s[i] + y * c[i]);
    }
  }
  __device__ __forceinline__ void store(T* x, const Values<T, kVec> (&v)[kVecs]) const {
    *reinterpret_cast<decltype(v[0].raw)*>(x + at) = v[0].raw;
    if (kVecs == 2 && turns_)
      *reinterpret_cast<decltype(v[0].raw)*>(x + at + half) = v[kVecs - 1].raw;
  }
};

// ---------------------------------------------------------------------------
// In and out of the ring.  Consecutive threads take the units of a token, then
// the token's groups of heads, then the next tokens of out; a block steps through
// out's tokens.  In place nothing is copied (units of a head: `units`).
// ---------------------------------------------------------------------------
template <typename T, int kVec, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, int units, int groups,
                                                          int per_group) {
  typedef Turn<T, kVec, kInterleaved> Unit;
  constexpr int U = 4;
  // The unit and the group are the same in each step: the stride is a multiple of
  // units * groups threads.
  const int per_token = units * groups;
  const int tokens = kThreads / per_token;  // of a step of the block
  const int lane = threadIdx.x % per_token;
  if ((int)threadIdx.x >= tokens * per_token) return;
  Unit u;
  u.init(lane % units, a.rot, a.freqs);
  const int h0 = lane / units * per_group, h1 = min(a.H, h0 + per_group);
  const long long total = (long long)a.B * a.S_out;
  for (long long i = (long long)blockIdx.x * tokens + threadIdx.x / per_token; i < total;
       i += (long long)gridDim.x * tokens) {
    const int b = (int)(i / a.S_out), p = (int)(i - (long long)b * a.S_out);
    const int n = a.to_sharded ? natural_pos(a.ring, p) : p;
    T* out = static_cast<T*>(a.out) + i * a.out_stride;
    if (n >= a.S_nat) {  // padding
      Values<T, kVec> zero[Unit::kVecs];
#pragma unroll
      for (int j = 0; j < kVec; ++j)
#pragma unroll
        for (int e = 0; e < Unit::kVecs; ++e) zero[e].v[j] = from_float<T>(0.f);
      for (int h = h0; h < h1; ++h) u.store(out + h * a.D, zero);
      continue;
    }
    const long long from = (long long)b * a.S_in + (a.from_sharded ? sharded_pos(a.ring, n) : n);
    const T* x = static_cast<const T*>(a.x) + from * a.x_stride;
    u.angles(a.positions ? a.positions[b * a.positions_stride + n] : a.offset + n, a.magnitude,
             a.sign);
    for (int h = h0; h < h1; h += U) {
      Values<T, kVec> v[U][Unit::kVecs];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (h + j < h1) u.load(x + (h + j) * a.D, v[j]);
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (h + j < h1) {
          if (u.turns_) u.turn(v[j]);
          u.store(out + (h + j) * a.D, v[j]);
        }
    }
  }
}

template <typename T, int kVec, bool kInterleaved>
cudaError_t run(const RotaryArgs& a, cudaStream_t stream) {
  typedef Turn<T, kVec, kInterleaved> Unit;
  const bool in_place = a.x == a.out && a.S_nat == a.S_out;
  const int units = in_place ? Unit::turning(a.rot) : Unit::units(a.D, a.rot);
  // All heads a thread where that leaves threads enough for the SMs.
  const long long total = (long long)a.B * a.S_out;
  const long long full = (long long)sm_count() * 1024;
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
// A step's tokens: "heads" 0 .. H - 1 are q's, then k's, then v's.
// ---------------------------------------------------------------------------
template <typename T, int kVec, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rotary_write_kernel(const RotaryWriteArgs a, int units,
                                                                int groups, int per_group) {
  typedef Turn<T, kVec, kInterleaved> Unit;
  constexpr int U = 4;
  const int per_token = units * groups;
  const int tokens = kThreads / per_token;
  const int lane = threadIdx.x % per_token;
  if ((int)threadIdx.x >= tokens * per_token) return;
  Unit u;
  u.init(lane % units, a.rot, a.freqs);
  const int all = a.H + 2 * a.Hkv;
  const int h0 = lane / units * per_group, h1 = min(all, h0 + per_group);
  const long long places = a.cache.num_pages * a.cache.page_size;
  for (long long i = (long long)blockIdx.x * tokens + threadIdx.x / per_token; i < a.N;
       i += (long long)gridDim.x * tokens) {
    long long slot = a.slots[i];
    if (slot >= places) {
      if (lane == 0) atomicExch(a.err, kErrBadTables);
      slot = -1;
    }
    const int page = slot < 0 ? 0 : (int)slot / a.cache.page_size;
    const int64_t row = page * a.cache.page_stride +
                        (slot < 0 ? 0 : (int)slot - page * a.cache.page_size) * a.cache.token_stride;
    const T* q = static_cast<const T*>(a.q) + i * a.q_stride;
    const T* k = static_cast<const T*>(a.k) + i * a.k_stride;
    const T* v = static_cast<const T*>(a.v) + i * a.v_stride;
    T* out = static_cast<T*>(a.out) + i * a.out_stride;
    T* kc = static_cast<T*>(a.k_cache) + row;
    T* vc = static_cast<T*>(a.v_cache) + row;
    u.angles(a.positions[i], a.magnitude, 1.f);
    const bool in_place = a.q == a.out;
    for (int h = h0; h < h1; h += U) {
      Values<T, kVec> w[U][Unit::kVecs];
      T* to[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        to[j] = nullptr;
        int g = h + j;
        if (g >= h1) continue;
        const T* from;
        if (g < a.H) {
          from = q + g * a.D;
          if (u.turns_ || !in_place) to[j] = out + g * a.D;
        } else {
          g -= a.H;
          const bool key = g < a.Hkv;
          if (!key) g -= a.Hkv;
          from = (key ? k : v) + g * a.D;
          if (slot >= 0) to[j] = (key ? kc : vc) + g * a.cache.head_stride;
        }
        if (to[j]) u.load(from, w[j]);
      }
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (to[j]) {
          if (u.turns_ && h + j < a.H + a.Hkv) u.turn(w[j]);
          u.store(to[j], w[j]);
        }
    }
  }
}

template <typename T, int kVec, bool kInterleaved>
cudaError_t run(const RotaryWriteArgs& a, cudaStream_t stream) {
  typedef Turn<T, kVec, kInterleaved> Unit;
  const int units = Unit::units(a.D, a.rot), all = a.H + 2 * a.Hkv;
  const long long full = (long long)sm_count() * 1024;
  int per_group = all;
  while (per_group > 1 &&
         a.N * units * ((all + per_group - 1) / per_group) < full &&
         units * ((all + (per_group + 1) / 2 - 1) / ((per_group + 1) / 2)) <= kThreads)
    per_group = (per_group + 1) / 2;
  const int groups = (all + per_group - 1) / per_group;
  const int tokens = kThreads / (units * groups);
  long long grid = (a.N + tokens - 1) / tokens;
  const long long cap = (long long)sm_count() * 16;
  if (grid > cap) grid = cap;
  rotary_write_kernel<T, kVec, kInterleaved><<<(unsigned)grid, kThreads, 0, stream>>>(
      a, units, groups, per_group);
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
