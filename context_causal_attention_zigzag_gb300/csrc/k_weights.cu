// The attention weight that the new tokens of a call gave to each cached position:
//
//   w_j <- decay w_j + sum_i exp(scale q_i k_j - lse_i)
//
// over the rows i (new tokens x query heads of the kv head) that see position j.
//
// On CUDA cores, for calls of few rows and keys (the rest: k_weights_tc.cu): a thread holds a
// key's row and walks the rows of q, which lie in shared memory as float32 a few at a time;
// the block's keys share them.  Bound by that chain: 6 us on the device (of many calls in a
// graph) for one token of 32 + 8 heads over 1000 positions, where the tensor cores' kernel needs
// 8 for its start.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cpattn.h"
#include "cpattn_internal.h"
#include "tc_ptx.cuh"

namespace cpattn {
namespace {

using tc::ex2;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKeys = 128;   // of a block, a thread each
constexpr int kStage = 16;   // rows of q in shared memory at a time

template <bool kBf16>
__device__ __forceinline__ float2 pair_of(uint32_t w) {
  if constexpr (kBf16) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kKeys) weights_kernel(const WeightsArgs w, int tiles) {
  const TreeArgs& a = w.t;
  __shared__ __align__(16) float s_q[kStage][D];
  __shared__ float s_l[kStage];
  const int G = a.H / a.Hkv, P = a.cache.page_size;
  const long long items = (long long)a.R * a.Hkv * tiles;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int tile = (int)(item % tiles);
    const int g = (int)(item / tiles % a.Hkv), r = (int)(item / tiles / a.Hkv);
    Req x;
    if (!load_req<true>(a, r, x) && threadIdx.x == 0) atomicExch(a.err, kErrBadTables);
    const int k0 = tile * kKeys, p = k0 + (int)threadIdx.x;
    if (x.n == 0 || k0 >= x.total) continue;
    int page = -1;
    if (p < x.total) {
      page = a.table[(int64_t)r * a.table_stride + p / P];
      if (page < 0 || page >= a.cache.num_pages) {
        page = -1;
        atomicExch(a.err, kErrBadTables);
      }
    }
    uint4 key[D / 8];
    if (page >= 0) {
      const uint16_t* k = static_cast<const uint16_t*>(a.k_cache) + page * a.cache.page_stride +
                          (p % P) * a.cache.token_stride + g * a.cache.head_stride;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) key[i] = reinterpret_cast<const uint4*>(k)[i];
    }
    float sum = 0.f;
    // Rows of tokens that see none of the block's keys are passed over.
    const int t0 = a.tree == nullptr && k0 > x.ctx ? k0 - x.ctx : 0;
    const int rows = x.n * G;
    for (int i0 = t0 * G; i0 < rows; i0 += kStage) {
      const int n = min(kStage, rows - i0);
      __syncthreads();
      for (int e = threadIdx.x; e < n * (D / 2); e += kKeys) {
        const int i = i0 + e / (D / 2), d = e % (D / 2), t = i / G, h = g * G + i - t * G;
        const uint32_t raw = *reinterpret_cast<const uint32_t*>(
            static_cast<const uint16_t*>(a.q) + (int64_t)(x.q0 + t) * a.q_stride + h * D + 2 * d);
        reinterpret_cast<float2*>(s_q[e / (D / 2)])[d] = pair_of<kBf16>(raw);
        if (d == 0) s_l[e / (D / 2)] = -kLog2e * w.lse[(int64_t)h * a.N + x.q0 + t];
      }
      __syncthreads();
      if (page < 0) continue;
      for (int i = 0; i < n; ++i) {
        const int t = (i0 + i) / G;
        const bool seen =
            p < x.ctx || (a.tree == nullptr ? p - x.ctx <= t
                                            : p - x.ctx < x.n && p - x.ctx < 64 &&
                                                  (a.tree[x.q0 + t] >> (p - x.ctx) & 1));
        if (!seen) continue;
        float y = 0.f;
#pragma unroll
        for (int e = 0; e < D / 8; ++e) {
          const uint32_t raw[4] = {key[e].x, key[e].y, key[e].z, key[e].w};
          const float4 q0 = reinterpret_cast<const float4*>(s_q[i])[2 * e];
          const float4 q1 = reinterpret_cast<const float4*>(s_q[i])[2 * e + 1];
          float2 v = pair_of<kBf16>(raw[0]);
          y = fmaf(v.x, q0.x, y);
          y = fmaf(v.y, q0.y, y);
          v = pair_of<kBf16>(raw[1]);
          y = fmaf(v.x, q0.z, y);
          y = fmaf(v.y, q0.w, y);
          v = pair_of<kBf16>(raw[2]);
          y = fmaf(v.x, q1.x, y);
          y = fmaf(v.y, q1.y, y);
          v = pair_of<kBf16>(raw[3]);
          y = fmaf(v.x, q1.z, y);
          y = fmaf(v.y, q1.w, y);
        }
        sum += s_l[i] == INFINITY ? 0.f : ex2(fmaf(y, a.scale_log2, s_l[i]));
      }
    }
    if (page >= 0) {
      float* to = w.weights + ((int64_t)page * a.Hkv + g) * P + p % P;
      *to = p < x.ctx ? fmaf(w.decay, *to, sum) : sum;
    }
  }
}

template <bool kBf16>
cudaError_t run(const WeightsArgs& w, int sms, cudaStream_t stream) {
  const int64_t keys = (int64_t)w.t.width * w.t.cache.page_size;
  const int tiles = (int)((keys + kKeys - 1) / kKeys);
  const int64_t items = (int64_t)w.t.R * w.t.Hkv * tiles, cap = (int64_t)sms * 16;
  if (items == 0) return cudaSuccess;
  const int grid = (int)(items < cap ? items : cap);
  if (w.t.D == 128)
    weights_kernel<kBf16, 128><<<grid, kKeys, 0, stream>>>(w, tiles);
  else
    weights_kernel<kBf16, 64><<<grid, kKeys, 0, stream>>>(w, tiles);
  return cudaGetLastError();
}

// Whether the CUDA cores are faster, from a call's sizes (the lengths themselves are on the
// device; a table much wider than its requests makes both estimates too high).  Measured (us,
// CUDA cores / tensor cores; H = 32, Hkv = 8, D = 128), by requests x tokens and keys a request:
//              16          64         256        1000        4000
//    1 x 1  5.0 / 6.8   5.1 / 6.8   5.6 / 8.1  5.8 / 8.3   7.3 / 8.9
//    8 x 1  5.2 / 7.9   5.3 / 7.9   7.3 / 8.7   14 / 12     34 / 22
//   64 x 1  9.1 / 15     11 / 16     25 / 24    70 / 40    273 / 119
//    1 x 8   19 / 6.9    19 / 7.1    19 / 8.2   20 / 8.3    24 / 8.8
// Many rows are left to the tensor cores however they are spread: a thread here walks all those
// of its request.
bool small_weights(const TreeArgs& a) {
  const int64_t rows = (int64_t)a.N * (a.H / a.Hkv), keys = (int64_t)a.width * a.cache.page_size;
  if (rows > 32) return false;
  const float mean = (float)rows / a.R, heads = (float)a.R * a.Hkv;
  const float latency = 4.2f + 0.46f * mean;
  const float work = 5.f + heads * ((keys + 127) / 128) * (0.009f + 0.0018f * mean);
  return (latency > work ? latency : work) < 7.5f + 0.0148f * heads * ((keys + 255) / 256);
}

}  // namespace

cudaError_t launch_cache_weights(const WeightsArgs& w, int dtype, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (small_weights(w.t))
    return dtype == CPATTN_BF16 ? run<true>(w, sms, stream) : run<false>(w, sms, stream);
  return launch_tc_weights(w, dtype, dev, sms, stream);
}

}  // namespace cpattn
