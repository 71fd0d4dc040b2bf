// Attention of the answering calls where there is little to do: one block per
// token and kv head on CUDA cores, in one launch.
//
// The tensor-core kernels take about 10 us whatever they are given (barriers,
// TMEM, tensor maps, a pipeline to fill, a merge), and an SM holds one of their
// blocks.  With a few dozen keys a row all of that is latency; here it is a
// launch, the request's lengths, the keys and one exchange between the warps.
//
// D / 8 lanes hold a key's row, 8 values (16 bytes) each, so a warp reads 2 (D =
// 128) or 4 keys at a time, and each lane keeps its 8 columns of q and o for up
// to kHeads query heads, which share the loads.  Scores and weights stay in
// float32 with the running maximum and sum of the softmax; the block's warps
// take turns on the keys and join their parts through shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "answer_way.h"
#include "cpattn_internal.h"
#include "tc_ptx.cuh"

namespace cpattn {
namespace {

using tc::ex2;
using tc::pack16;

constexpr int kPages = 512;  // page numbers kept in shared memory
constexpr float kLn2 = 0.6931471805599453f;

template <bool kBf16>
__device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x;
    if constexpr (kBf16) {
      x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    } else {
      x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    }
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

template <bool kBf16, int D, int kHeads, int kWarps, int U, bool kPaged>
__global__ void __launch_bounds__(kWarps * 32) small_kernel(const TreeArgs a) {
  constexpr int kThreads = kWarps * 32;
  constexpr int kLanes = D / 8;         // of a key
  constexpr int kKeys = 32 / kLanes;    // of a warp at a time
  __shared__ float s_o[kWarps][kHeads][D], s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  __shared__ int s_r, s_page[kPaged ? kPages : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / kLanes, col = (lane % kLanes) * 8;
  const int i = blockIdx.x, G = a.H / a.Hkv;
  const int chunks = (G + kHeads - 1) / kHeads;
  const int g = blockIdx.y / chunks, h0 = (blockIdx.y - g * chunks) * kHeads;
  const int nh = min(kHeads, G - h0);
  // The token's request: each thread looks at some.
  if (threadIdx.x == 0) s_r = -1;
  __syncthreads();
  const bool reports = blockIdx.x == 0 && blockIdx.y == 0;
  for (int r = threadIdx.x; r < a.R; r += kThreads) {
    const int lo = a.cu[r], hi = a.cu[r + 1];
    if (lo <= i && i < hi) s_r = r;
    if (reports) {
      Req x;
      if (!load_req<kPaged>(a, r, x)) atomicExch(a.err, kErrBadTables);
    }
  }
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + i * a.q_stride + (g * G + h0) * D + col;
  float q[kHeads][8], o[kHeads][8], m[kHeads], l[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (h < nh) v = *reinterpret_cast<const uint4*>(qp + h * D);
    unpack<kBf16>(v, q[h]);
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      q[h][e] *= a.scale_log2;
      o[h][e] = 0.f;
    }
  }
  __syncthreads();
  const int r = s_r;
  if (r < 0) return;  // behind the last request: left as it is
  Req x;
  load_req<kPaged>(a, r, x);
  if (!kPaged && a.above > 0 && x.total >= a.above) return;  // the cut line's
  const int t = i - x.q0;
  const bool chain = a.tree == nullptr;
  unsigned long long bits = 0;
  if (!chain) {
    bits = a.tree[i];
    if (x.n < 64) bits &= (1ull << x.n) - 1;
  }
  // Seen: the positions below `limit`, and of those from ctx on the ones in bits.
  const int limit = chain ? min(x.total, x.ctx + (kPaged || a.causal ? t + 1 : 0)) : x.ctx;
  const int end = chain ? limit : x.total;
  const int P = a.cache.page_size;
  const int* table = kPaged ? a.table + (int64_t)r * a.table_stride : nullptr;
  if constexpr (kPaged) {
    for (int p = threadIdx.x; p < kPages && p * P < end; p += kThreads) s_page[p] = table[p];
    __syncthreads();
  }
  const uint16_t* kp = static_cast<const uint16_t*>(a.k_cache) + col;
  const uint16_t* vp = static_cast<const uint16_t*>(a.v_cache) + col;
  bool bad = false;
  for (int j0 = warp * kKeys + sub; j0 - sub < end; j0 += kWarps * kKeys * U) {
    uint4 kv[U], vv[U];
    bool on[U];
    int64_t at_k[U], at_v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * kWarps * kKeys, d = j - x.ctx;
      on[u] = j < limit || (!chain && j < end && d >= 0 && d < 64 && (bits >> d & 1));
      at_k[u] = at_v[u] = 0;
      if (on[u]) {
        if constexpr (kPaged) {
          const int p = j / P, page = p < kPages ? s_page[p] : table[p];
          if (page < 0 || page >= a.cache.num_pages) {
            on[u] = false;
            bad = true;
          }
          at_k[u] = at_v[u] = page * a.cache.page_stride + (j % P) * a.cache.token_stride +
                              g * a.cache.head_stride;
        } else {
          at_k[u] = (int64_t)(x.k0 + j) * a.k_stride + g * D;
          at_v[u] = (int64_t)(x.k0 + j) * a.v_stride + g * D;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      kv[u] = vv[u] = make_uint4(0, 0, 0, 0);
      if (on[u]) {
        kv[u] = *reinterpret_cast<const uint4*>(kp + at_k[u]);
        vv[u] = *reinterpret_cast<const uint4*>(vp + at_v[u]);
      }
    }
    float s[U][kHeads];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8];
      unpack<kBf16>(kv[u], f);
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        float y = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) y = fmaf(q[h][e], f[e], y);
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) y += __shfl_xor_sync(0xffffffffu, y, d);
        s[u][h] = on[u] ? y : -INFINITY;
      }
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      float mn = m[h];
#pragma unroll
      for (int u = 0; u < U; ++u) mn = fmaxf(mn, s[u][h]);
      const float c = mn == -INFINITY ? 0.f : mn;  // nothing seen yet
      const float f = ex2(m[h] - c);
      m[h] = mn;
      l[h] *= f;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[h][e] *= f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u][h] = ex2(s[u][h] - c);
        l[h] += s[u][h];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8];
      unpack<kBf16>(vv[u], f);
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[h][e] = fmaf(s[u][h], f[e], o[h][e]);
    }
  }
  if (bad) atomicExch(a.err, kErrBadTables);
  // Join the warp's keys, then the warps.
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
#pragma unroll
    for (int d = kLanes; d < 32; d <<= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m[h], d);
      const float lo = __shfl_xor_sync(0xffffffffu, l[h], d);
      const float mn = fmaxf(m[h], mo), c = mn == -INFINITY ? 0.f : mn;
      const float f = ex2(m[h] - c), fo = ex2(mo - c);
      l[h] = l[h] * f + lo * fo;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[h][e] = o[h][e] * f + __shfl_xor_sync(0xffffffffu, o[h][e], d) * fo;
      m[h] = mn;
    }
    if (sub == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s_o[warp][h][col + e] = o[h][e];
      if (lane == 0) {
        s_m[warp][h] = m[h];
        s_l[warp][h] = l[h];
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < nh * (D / 2); e += kThreads) {
    const int h = e / (D / 2), c = e % (D / 2) * 2;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
    float L = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = M == -INFINITY ? 0.f : ex2(s_m[w][h] - M);
      L += s_l[w][h] * f;
      y0 = fmaf(s_o[w][h][c], f, y0);
      y1 = fmaf(s_o[w][h][c + 1], f, y1);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;  // a row that sees nothing: 0
    const int head = g * G + h0 + h;
    reinterpret_cast<uint32_t*>(a.out)[((int64_t)i * a.H + head) * (D / 2) + c / 2] =
        pack16<kBf16>(y0 * inv, y1 * inv);
    if (c == 0) a.lse[(int64_t)head * a.N + i] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
  }
}

template <bool kBf16, int D, int kHeads, int kWarps, int U>
void run(const TreeArgs& a, cudaStream_t stream) {
  const int G = a.H / a.Hkv;
  const dim3 grid(a.N, a.Hkv * ((G + kHeads - 1) / kHeads));
  if (a.cu_k == nullptr)
    small_kernel<kBf16, D, kHeads, kWarps, U, true><<<grid, kWarps * 32, 0, stream>>>(a);
  else
    small_kernel<kBf16, D, kHeads, kWarps, U, false><<<grid, kWarps * 32, 0, stream>>>(a);
}

template <bool kBf16, int D>
void run_heads(const TreeArgs& a, int sms, cudaStream_t stream) {
  const int G = a.H / a.Hkv;
  if (few_blocks(a, sms)) {
    if (G == 1)
      run<kBf16, D, 1, 8, 4>(a, stream);
    else
      run<kBf16, D, 2, 8, 4>(a, stream);
  } else if (G == 1) {
    run<kBf16, D, 1, 4, 2>(a, stream);
  } else if (G == 2) {
    run<kBf16, D, 2, 4, 2>(a, stream);
  } else {
    run<kBf16, D, 4, 4, 2>(a, stream);
  }
}

}  // namespace

cudaError_t launch_small_attn(const TreeArgs& a, int dtype, int sms, cudaStream_t stream) {
  if (dtype == CPATTN_BF16) {
    if (a.D == 128)
      run_heads<true, 128>(a, sms, stream);
    else
      run_heads<true, 64>(a, sms, stream);
  } else {
    if (a.D == 128)
      run_heads<false, 128>(a, sms, stream);
    else
      run_heads<false, 64>(a, sms, stream);
  }
  return cudaGetLastError();
}

}  // namespace cpattn
