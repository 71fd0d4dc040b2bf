// Inline-PTX building blocks for the sm_103a tensor-core kernels: mbarriers
// with bounded waits, TMA tile loads, TMEM allocation, tcgen05.mma issue and
// commit, tcgen05.ld / tcgen05.st, and the shared-memory matrix descriptors.
//
// Operand layouts used throughout (bf16, 128-byte swizzle):
//  * a [rows x 64] bf16 box written by TMA with SWIZZLE_128B is rows of 128 B,
//    grouped in 8-row / 1024-B swizzle atoms (16-B chunk c of row r stored at
//    chunk c ^ (r % 8)); every box starts on a 1024-B boundary.
//  * K-major operand (contraction dim contiguous, e.g. Q and K for Q K^T):
//    stride between 8-row groups (SBO) = 1024 B; the contraction dim advances
//    by moving the start address 32 B per 16 elements inside a 128-B row and
//    to the next box every 64 elements.
//  * MN-major operand (output dim contiguous, e.g. V for P V): SBO = 1024 B
//    between 8-row groups along the contraction dim, LBO = box size between
//    64-column blocks along the output dim.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace cpattn {
namespace tc {

// A device-side wait gives up after this long (nanoseconds of %globaltimer).
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// The same value, which the compiler no longer knows.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  asm volatile("" : "+r"(x));
  return x;
}

__device__ __forceinline__ uint64_t global_timer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// ---------------------------------------------------------------------------
// mbarrier
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Shared state of the bounded waits of one CTA.
struct WaitCtl {
  volatile int* abort;              // shared flag: some wait of this CTA gave up
  int* err;                         // device error word (global)
  uint64_t limit_ns = kWaitLimitNs;  // how long a wait may spin
};

// Waits for the phase of `bar` with the given parity to complete.  Returns
// false (after raising the CTA's abort flag and the device error word) if it
// does not within w.limit_ns, or if another wait of the CTA already gave up.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, const WaitCtl& w) {
  if (mbar_test(bar, parity)) return true;
  const uint64_t t0 = global_timer();
  while (true) {
    if (mbar_test(bar, parity)) return true;
    if (*w.abort) return false;
    if (global_timer() - t0 > w.limit_ns) {
      *w.abort = 1;
      atomicExch(w.err, 1);
      return false;
    }
  }
}

// The same wait for chains of short steps: the abort flag and the global timer,
// whose reading takes longer than such a step, are looked at once in 64 polls.
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity, const WaitCtl& w) {
  if (mbar_test(bar, parity)) return true;
  uint64_t t0 = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_test(bar, parity)) return true;
    if (*w.abort) return false;
    const uint64_t t = global_timer();
    if (t0 == 0) {
      t0 = t;
    } else if (t - t0 > w.limit_ns) {
      *w.abort = 1;
      atomicExch(w.err, 1);
      return false;
    }
  }
}

// Same, without raising the abort flag: the bounded drain at teardown.
__device__ __forceinline__ bool mbar_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer();
  while (!mbar_test(bar, parity)) {
    if (global_timer() - t0 > kWaitLimitNs) return false;
  }
  return true;
}

// ---------------------------------------------------------------------------
// TMA
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// 3-D tiled load into shared memory; completion is reported to `bar` as
// transaction bytes.  c0 is the innermost coordinate.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// The same for a 4-D tensor.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

// True in exactly one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred != 0;
}

// Asks for a 3-D tile of the tensor to be brought into L2 ahead of its load
// (nothing lands in shared memory, nothing to wait for).
__device__ __forceinline__ void tma_prefetch_l2_3d(const CUtensorMap* map, int c0, int c1,
                                                   int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// ---------------------------------------------------------------------------
// TMEM and tcgen05
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive (once) on `bar` when every tcgen05 operation this thread issued so
// far has completed.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

#define CPATTN_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), \
                     "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define CPATTN_W8(i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), \
                     "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// Each thread of the warp reads 32 consecutive 32-bit columns of its lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : CPATTN_R8(0), CPATTN_R8(8), CPATTN_R8(16), CPATTN_R8(24)
      : "r"(taddr));
}

// Each thread of the warp writes 32 consecutive 32-bit columns of its lane.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          taddr),
      CPATTN_W8(0), CPATTN_W8(8), CPATTN_W8(16), CPATTN_W8(24)
      : "memory");
}

#define CPATTN_RW8(i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), \
                      "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])

// tcgen05.ld writes its destination registers asynchronously; they are valid
// after tcgen05.wait::ld.  Waits, then ties the 32 registers to the wait so
// that no use of them is scheduled before it.
__device__ __forceinline__ void tmem_wait_ld_regs(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : CPATTN_RW8(0), CPATTN_RW8(8), CPATTN_RW8(16), CPATTN_RW8(24)
               :
               : "memory");
}

// Ties 32 registers to this point without emitting code.
__device__ __forceinline__ void reg_fence32(uint32_t* r) {
  asm volatile(""
               : CPATTN_RW8(0), CPATTN_RW8(8), CPATTN_RW8(16), CPATTN_RW8(24)
               :
               : "memory");
}

#undef CPATTN_R8
#undef CPATTN_W8
#undef CPATTN_RW8

// ---------------------------------------------------------------------------
// Descriptors
// ---------------------------------------------------------------------------

// Shared-memory matrix descriptor, 128-byte swizzle.
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version of tcgen05
  d |= (uint64_t)2 << 61;  // SWIZZLE_128B
  return d;
}

// The descriptor of the operand `bytes` further on in shared memory (a
// multiple of 16): the start-address field holds address / 16 in its low 14
// bits, and shared-memory addresses stay below 2^18, so the add never
// carries out of the field.
__device__ __forceinline__ uint64_t sdesc_advance(uint64_t desc, uint32_t bytes) {
  return desc + (uint64_t)(bytes >> 4);
}

// Instruction descriptor, kind::f16: bf16 (or both fp16) A and B, fp32
// accumulator, M x N.
// a_mn / b_mn: operand is MN-major (output dim contiguous) instead of K-major.
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4)                          // D format: f32
         | ((bf16 ? 1u : 0u) << 7)          // A format: bf16 or fp16
         | ((bf16 ? 1u : 0u) << 10)         // B format
         | ((a_mn ? 1u : 0u) << 15)         // A major
         | ((b_mn ? 1u : 0u) << 16)         // B major
         | ((uint32_t)(N >> 3) << 17)       // N / 8
         | ((uint32_t)(M >> 4) << 24);      // M / 16
}
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return idesc_f16(true, M, N, a_mn, b_mn);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Two values of one 16-bit type, rounded to nearest.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (kBf16) {
    return pack_bf16(lo, hi);
  } else {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
}

// The reference m of the softmax weights 2^(s - m), in log2, is corrected when a
// tile's best score passes it by more than kWeightLag; it then becomes that score
// (bfloat16), or 7 less (float16).  float16 weights so reach from 2^15 down to the
// type's smallest step: the row's largest is 2^7 at least, one keeps its 11 bits down
// to 2^-21 of the largest and has a step of 2^-31 below that.  With the score itself
// as the reference, those below 2^-25 vanished from O while the float32 sum of the
// weights kept them (16383 keys 17 nats below the row's best: O 44 % off).
// In float16 the score and the reference are rounded up, so that no weight passes
// 2^15 whatever the scores' size: beyond 2^24 their own rounding would make one
// overflow.
template <bool kBf16>
constexpr float kWeightLag = kBf16 ? 8.f : 15.f;

template <bool kBf16>
__device__ __forceinline__ float best_score(float max, float sl2) {
  return kBf16 ? max * sl2 : __fmul_ru(max, sl2);
}
template <bool kBf16>
__device__ __forceinline__ float new_reference(float best) {
  return kBf16 ? best : __fadd_ru(best, -7.f);
}

// Transposes 4 x 4 16-byte pieces within each quad of lanes: v[j] of lane q
// becomes what v[q] of the quad's lane j was.  A thread that holds 64
// consecutive bytes of its own row then holds one piece of four rows, and the
// quad writes each row's 64 bytes together (8 rows a warp store instead of
// 32, each of which costs the load/store unit a cycle).
__device__ __forceinline__ void quad_transpose(uint4 (&v)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 1; b <= 2; b <<= 1) {
    const bool up = lane & b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & b) continue;
      uint4 x = up ? v[j] : v[j | b];
      x.x = __shfl_xor_sync(0xffffffffu, x.x, b);
      x.y = __shfl_xor_sync(0xffffffffu, x.y, b);
      x.z = __shfl_xor_sync(0xffffffffu, x.z, b);
      x.w = __shfl_xor_sync(0xffffffffu, x.w, b);
      if (up)
        v[j] = x;
      else
        v[j | b] = x;
    }
  }
}

// Orders this thread's shared-memory writes before later accesses of the
// tensor cores and TMA (the async proxy).
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Programmatic launches: lets the next kernel of the stream start, and waits
// until the one before has finished and its writes are visible.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_prior_grid() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace tc
}  // namespace cpattn
