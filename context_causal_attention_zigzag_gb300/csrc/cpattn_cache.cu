// C-ABI layer of the rotary and cache calls: argument checks and dispatch.
// Declarations and the meaning of every argument are in include/cpattn.h.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "answer_checks.h"
#include "cpattn.h"
#include "cpattn_internal.h"

using namespace cpattn;
using namespace cpattn::checks;

namespace {

// Rows of `width` values of `elt` bytes, `stride` apart: 16-byte steps, no overlap.
bool rotary_rows(const void* p, int64_t stride, int64_t width, int elt) {
  return p != nullptr && aligned(p, 16) && stride * elt % 16 == 0 && stride >= width &&
         stride < ((int64_t)1 << 38);
}

// Whether na rows of wa bytes, sa bytes apart, and nb rows of wb bytes share memory.  Slices of
// one fused projection (equal strides, side by side) do not.
typedef __int128 Bytes;
bool rows_meet(const void* pa, Bytes sa, Bytes na, Bytes wa, const void* pb, Bytes sb, Bytes nb,
               Bytes wb) {
  const Bytes a = reinterpret_cast<intptr_t>(pa), b = reinterpret_cast<intptr_t>(pb);
  if (na == 0 || nb == 0 || a >= b + (nb - 1) * sb + wb || b >= a + (na - 1) * sa + wa)
    return false;
  if (sa != sb) return true;
  Bytes d = (a - b) % sa;  // where a row of a begins in a period of b's
  if (d < 0) d += sa;
  return d < wb || d + wa > sa;
}

// A stretch of memory.
struct Stretch {
  const void* p;
  Bytes n;
};
// Whether one that is written meets another, or one that is read.  Kernels read lengths, tables
// and lists again, and go by what they found the first time: another value there could lead
// them out of the cache.
template <int kW, int kR>
bool any_meet(const Stretch (&written)[kW], const Stretch (&read)[kR]) {
  auto meet = [](const Stretch& x, const Stretch& y) {
    return rows_meet(x.p, x.n, x.n > 0, x.n, y.p, y.n, y.n > 0, y.n);
  };
  for (int i = 0; i < kW; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(written[i], written[j])) return true;
    for (int j = 0; j < kR; ++j)
      if (meet(written[i], read[j])) return true;
  }
  return false;
}
// From a table's first byte to its last.
Stretch table_stretch(const int32_t* table, int R, int width, int64_t stride) {
  return {table, R > 0 && width > 0 ? 4 * ((Bytes)(R - 1) * stride + width) : 0};
}

// From a cache's first byte to its last.
Bytes cache_bytes(const CacheShape& c, int Hkv, int D) {
  return 2 * ((Bytes)(c.num_pages - 1) * c.page_stride +
              (Bytes)(c.page_size - 1) * c.token_stride + (Bytes)(Hkv - 1) * c.head_stride + D);
}

// Whether rows of `width` bytes, `stride` apart, and a stretch share memory.
bool row_meets(const void* p, Bytes stride, Bytes rows, Bytes width, const Stretch& x) {
  return rows_meet(p, stride, rows, width, x.p, stride, x.n > 0, x.n);
}

// Whether the keys and values of a cache share memory: both have its strides, and may lie by
// turns in one tensor.  With the axes from the widest stride down, an axis cannot make up for
// more than a step of those before it, so that of each only the steps around what is left matter.
bool caches_meet(const void* k, const void* v, const CacheShape& c, int Hkv, int D) {
  struct Axis {
    int64_t stride, n;
  } axes[3] = {{2 * c.page_stride, c.num_pages}, {2 * c.token_stride, c.page_size}, {2 * c.head_stride, Hkv}};
  std::sort(axes, axes + 3, [](const Axis& x, const Axis& y) { return x.stride > y.stride; });
  int64_t left[8] = {reinterpret_cast<intptr_t>(v) - reinterpret_cast<intptr_t>(k)};
  const Bytes all = cache_bytes(c, Hkv, D);
  if (left[0] >= all || -left[0] >= all) return false;
  int ways = 1;
  for (const Axis& x : axes) {
    if (x.n == 1) continue;  // its stride says nothing
    int next = 0;
    int64_t then[8];
    for (int i = 0; i < ways; ++i) {
      int64_t m = left[i] / x.stride;
      if (m * x.stride > left[i]) --m;
      for (int j = 0; j < 2; ++j, ++m)
        if (m < x.n && -m < x.n) then[next++] = left[i] - m * x.stride;
    }
    ways = next;
    for (int i = 0; i < ways; ++i) left[i] = then[i];
  }
  for (int i = 0; i < ways; ++i)
    if (left[i] < 2 * D && -left[i] < 2 * D) return true;
  return false;
}

bool turn_ok(int D, int rot, int interleaved, const double* freqs, float magnitude) {
  return rot >= 2 && rot <= D && rot % 2 == 0 && (interleaved == 0 || interleaved == 1) && freqs &&
         aligned(freqs, 8) && isfinite(magnitude);
}

}  // namespace

extern "C" {

int cpattn_rotary_frequencies(double* freqs, double* magnitude, int rot, double base, int scaling,
                              double factor, double original, double low, double high) {
  if (!freqs || !magnitude || rot < 2 || rot % 2 != 0 || !isfinite(base) || !(base > 1.0) ||
      scaling < CPATTN_ROTARY_PLAIN || scaling > CPATTN_ROTARY_PARTS || !isfinite(factor) ||
      !(factor >= 1.0))
    return CPATTN_ERR_INVALID_ARG;
  if (scaling == CPATTN_ROTARY_BASE && rot == 2) return CPATTN_ERR_INVALID_ARG;
  if (scaling == CPATTN_ROTARY_PARTS &&
      (!isfinite(original) || !(original > 0.0) || !(low >= 0.0) || !(high > low) ||
       !isfinite(high)))
    return CPATTN_ERR_INVALID_ARG;
  if (scaling == CPATTN_ROTARY_BASE) base *= pow(factor, (double)rot / (rot - 2));
  for (int i = 0; i < rot / 2; ++i) {
    double f = pow(base, -2.0 * i / rot);
    if (scaling == CPATTN_ROTARY_LINEAR) f /= factor;
    if (scaling == CPATTN_ROTARY_PARTS) {
      const double turns = original * f / 6.283185307179586;
      double g = (turns - low) / (high - low);
      g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
      f = (1.0 - g) * f / factor + g * f;
    }
    freqs[i] = f;
  }
  *magnitude = scaling == CPATTN_ROTARY_PARTS ? 0.1 * log(factor) + 1.0 : 1.0;
  return CPATTN_OK;
}

int cpattn_rotary(const void* x, int64_t x_stride, void* out, int64_t out_stride, int B, int S_nat,
                  int S, int H, int D, int rot, int interleaved, const double* freqs,
                  float magnitude, int transposed, const int32_t* positions,
                  int64_t positions_stride, int64_t offset, int cp_size, int layout,
                  int from_sharded, int to_sharded, int dtype, cpattn_stream_t stream) {
  if (dtype != CPATTN_F32 && dtype != CPATTN_BF16 && dtype != CPATTN_F16)
    return CPATTN_ERR_INVALID_ARG;
  if (B < 0 || B > 65535 || S_nat < 0 || S < S_nat || S > (1 << 30) || H < 1 || H > 65535 ||
      D < 8 || D > 256 || D % 8 != 0 || cp_size < 1)
    return CPATTN_ERR_INVALID_ARG;
  if (layout != CPATTN_LAYOUT_CONTIGUOUS && layout != CPATTN_LAYOUT_ZIGZAG)
    return CPATTN_ERR_INVALID_ARG;
  if ((from_sharded | to_sharded | transposed) & ~1) return CPATTN_ERR_INVALID_ARG;
  const int per = layout == CPATTN_LAYOUT_ZIGZAG ? 2 : 1;
  // Two natural tensors know no chunks.
  if ((from_sharded || to_sharded) && S % ((int64_t)cp_size * per) != 0)
    return CPATTN_ERR_INVALID_ARG;
  if (!turn_ok(D, rot, interleaved, freqs, magnitude)) return CPATTN_ERR_INVALID_ARG;
  RotaryArgs a;
  memset(&a, 0, sizeof(a));
  a.S_in = from_sharded ? S : S_nat;
  a.S_out = to_sharded ? S : S_nat;
  if ((int64_t)B * a.S_out == 0) return CPATTN_OK;
  const int elt = dtype == CPATTN_F32 ? 4 : 2;
  const int64_t width = (int64_t)H * D;
  if (!rotary_rows(out, out_stride, width, elt) ||
      ((int64_t)B * a.S_in > 0 && !rotary_rows(x, x_stride, width, elt)))
    return CPATTN_ERR_INVALID_ARG;
  if (positions && (!aligned(positions, 4) || (positions_stride != 0 && positions_stride < S_nat)))
    return CPATTN_ERR_INVALID_ARG;
  const bool same = x == out && x_stride == out_stride && from_sharded == to_sharded;
  if (!same && rows_meet(x, x_stride * elt, (int64_t)B * a.S_in, width * elt, out,
                         out_stride * elt, (int64_t)B * a.S_out, width * elt))
    return CPATTN_ERR_INVALID_ARG;
  // (Several blocks read these while others write.)
  const Stretch read[] = {
      {positions, positions && S_nat > 0 ? 4 * ((Bytes)(B - 1) * positions_stride + S_nat) : 0},
      {freqs, 4 * (Bytes)rot}};
  for (const Stretch& r : read)
    if (row_meets(out, out_stride * elt, (Bytes)B * a.S_out, width * elt, r))
      return CPATTN_ERR_INVALID_ARG;
  a.x = x;
  a.out = out;
  a.x_stride = x_stride;
  a.out_stride = out_stride;
  a.B = B;
  a.S_nat = S_nat;
  a.H = H;
  a.D = D;
  a.rot = rot;
  a.freqs = freqs;
  a.magnitude = magnitude;
  a.sign = transposed ? -1.f : 1.f;
  a.positions = positions;
  a.positions_stride = positions_stride;
  a.offset = offset;
  a.ring.S = S;
  a.ring.cp = cp_size;
  a.ring.per_rank = per;
  a.ring.L = S / cp_size;
  a.ring.c = a.ring.L / per;
  a.from_sharded = from_sharded != 0;
  a.to_sharded = to_sharded != 0;
  return status(launch_rotary(a, dtype, interleaved != 0, (cudaStream_t)stream));
}

int cpattn_rotary_cache_write(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                              const void* v, int64_t v_stride, void* out, int64_t out_stride,
                              const int32_t* positions, const int64_t* slots, int64_t N, int rot,
                              int interleaved, const double* freqs, float magnitude, void* k_cache,
                              void* v_cache, int64_t num_pages, int page_size, int64_t page_stride,
                              int64_t token_stride, int64_t head_stride, int H, int Hkv, int D,
                              int dtype, cpattn_stream_t stream) {
  int rc = check_heads(H, Hkv, D, dtype);
  if (rc != CPATTN_OK) return rc;
  if (N < 0 || N > INT32_MAX || !turn_ok(D, rot, interleaved, freqs, magnitude))
    return CPATTN_ERR_INVALID_ARG;
  CacheShape c = {num_pages, page_size, page_stride, token_stride, head_stride};
  if (!check_cache(k_cache, v_cache, c, D)) return CPATTN_ERR_INVALID_ARG;
  if (N == 0) return CPATTN_OK;
  if (!check_rows(q, q_stride, H, D) || !check_rows(k, k_stride, Hkv, D) ||
      !check_rows(v, v_stride, Hkv, D) || !check_rows(out, out_stride, H, D) || !slots ||
      !aligned(slots, 8) || !positions || !aligned(positions, 4))
    return CPATTN_ERR_INVALID_ARG;
  const Bytes wq = 2 * (Bytes)H * D, wk = 2 * (Bytes)Hkv * D, wc = cache_bytes(c, Hkv, D);
  if (!(q == out && q_stride == out_stride) &&
      rows_meet(q, 2 * q_stride, N, wq, out, 2 * out_stride, N, wq))
    return CPATTN_ERR_INVALID_ARG;
  if (rows_meet(k, 2 * k_stride, N, wk, out, 2 * out_stride, N, wq) ||
      rows_meet(v, 2 * v_stride, N, wk, out, 2 * out_stride, N, wq) ||
      rows_meet(k_cache, wc, 1, wc, out, 2 * out_stride, N, wq) ||
      rows_meet(v_cache, wc, 1, wc, out, 2 * out_stride, N, wq))
    return CPATTN_ERR_INVALID_ARG;
  if (caches_meet(k_cache, v_cache, c, Hkv, D)) return CPATTN_ERR_INVALID_ARG;
  const Stretch lists[] = {{positions, 4 * (Bytes)N}, {slots, 8 * (Bytes)N}, {freqs, 4 * (Bytes)rot}};
  for (const Stretch& x : lists)
    if (row_meets(out, 2 * out_stride, N, wq, x)) return CPATTN_ERR_INVALID_ARG;
  const Stretch caches[] = {{k_cache, wc}, {v_cache, wc}};
  for (const Stretch& x : caches) {
    const Stretch one[] = {x};
    if (any_meet(one, lists) || row_meets(q, 2 * q_stride, N, wq, x) ||
        row_meets(k, 2 * k_stride, N, wk, x) || row_meets(v, 2 * v_stride, N, wk, x))
      return CPATTN_ERR_INVALID_ARG;
  }
  int* err = device_error_word();
  if (err == nullptr) return CPATTN_ERR_CUDA;
  RotaryWriteArgs a = {q,     k,         v,         out,  q_stride, k_stride, v_stride, out_stride,
                       positions, slots, N,         H,    Hkv,      D,        rot,      freqs,
                       magnitude, k_cache, v_cache, c,    err};
  return status(launch_rotary_write(a, dtype, interleaved != 0, (cudaStream_t)stream));
}

size_t cpattn_cache_weights_workspace_bytes(int N, int H, int Hkv, int D) {
  if (N < 0 || check_heads(H, Hkv, D, CPATTN_BF16) != CPATTN_OK) return 0;
  return weights_workspace_bytes();
}

int cpattn_cache_weights(const void* q, int64_t q_stride, const void* k_cache, int64_t num_pages,
                         int page_size, int64_t page_stride, int64_t token_stride,
                         int64_t head_stride, const int32_t* block_table, int table_width,
                         int64_t table_stride, const int32_t* ctx_lens, const int32_t* cu_new,
                         const uint64_t* tree, const float* lse, float* weights, float decay, int R,
                         int N, int H, int Hkv, int D, int dtype, float softmax_scale,
                         void* workspace, size_t workspace_bytes, cpattn_stream_t stream) {
  int rc = check_heads(H, Hkv, D, dtype);
  if (rc != CPATTN_OK) return rc;
  // An item's steps are its tiles of whole tokens: 2^20 of 128 rows take 1.1 s at 1.9 GHz.
  if (R < 0 || R > kMostRequests || N < 0 || N > (int64_t)(kTcTile / (H / Hkv)) << 20 ||
      !scale_ok(softmax_scale) || !isfinite(decay))
    return CPATTN_ERR_INVALID_ARG;
  CacheShape c = {num_pages, page_size, page_stride, token_stride, head_stride};
  if (!check_cache(k_cache, k_cache, c, D)) return CPATTN_ERR_INVALID_ARG;
  if (table_width < 0 || table_stride < table_width || table_width > kMostPositions / page_size)
    return CPATTN_ERR_INVALID_ARG;
  if (R == 0 || N == 0) return CPATTN_OK;
  if (!check_rows(q, q_stride, H, D) || !lse || !aligned(lse, 4) || !weights ||
      !aligned(weights, 4) || (table_width > 0 && !block_table) || !ctx_lens || !cu_new ||
      !aligned(block_table, 4) || !aligned(ctx_lens, 4) || !aligned(cu_new, 4) ||
      !aligned(tree, 8))
    return CPATTN_ERR_INVALID_ARG;
  const Stretch written[] = {{weights, 4 * (Bytes)num_pages * Hkv * page_size}};
  const Stretch read[] = {{k_cache, cache_bytes(c, Hkv, D)},
                          {q, 2 * ((Bytes)(N - 1) * q_stride + (Bytes)H * D)},
                          {lse, 4 * (Bytes)H * N},
                          {ctx_lens, 4 * (Bytes)R},
                          {cu_new, 4 * ((Bytes)R + 1)},
                          {tree, tree ? 8 * (Bytes)N : 0},
                          table_stretch(block_table, R, table_width, table_stride)};
  if (any_meet(written, read)) return CPATTN_ERR_INVALID_ARG;
  const size_t need = weights_workspace_bytes();
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need)
    return CPATTN_ERR_WORKSPACE;
  const Stretch both[] = {written[0], {workspace, (Bytes)need}};
  if (any_meet(both, read)) return CPATTN_ERR_INVALID_ARG;
  int* err = device_error_word();
  if (err == nullptr) return CPATTN_ERR_CUDA;
  WeightsArgs w;
  memset(&w, 0, sizeof(w));
  TreeArgs& a = w.t;
  a.q = q;
  a.q_stride = q_stride;
  a.k_cache = k_cache;
  a.cache = c;
  a.table = block_table;
  a.width = table_width;
  a.table_stride = table_stride;
  a.ctx = ctx_lens;
  a.cu = cu_new;
  a.tree = reinterpret_cast<const unsigned long long*>(tree);
  a.R = R;
  a.N = N;
  a.H = H;
  a.Hkv = Hkv;
  a.D = D;
  a.scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)D);
  a.scale_log2 = a.scale * 1.4426950408889634f;
  a.workspace = workspace;
  a.err = err;
  w.lse = lse;
  w.weights = weights;
  w.decay = decay;
  return status(launch_cache_weights(w, dtype, (cudaStream_t)stream));
}

namespace {
// Shapes that the workspace can be asked for.
bool evict_shape_ok(int R, int Hkv, int width, int P, int most) {
  return R >= 0 && R <= 65535 && Hkv >= 1 && Hkv <= 65535 && (int64_t)R * Hkv <= (1 << 24) &&
         width >= 0 && page_size_ok(P) && width <= kMostPositions / P && most >= 1 &&
         most <= kMostPositions && (int64_t)R * Hkv * most < ((int64_t)1 << 40);
}
// No list is longer than what can be kept of a request.
int64_t evict_list(int width, int P, int most) {
  const int64_t cap = (int64_t)width * P;
  return cap < most ? cap : most;
}
}  // namespace

size_t cpattn_cache_evict_workspace_bytes(int R, int Hkv, int table_width, int page_size,
                                          int most) {
  if (!evict_shape_ok(R, Hkv, table_width, page_size, most)) return 0;
  const size_t items = (size_t)R * Hkv;
  return (items + items * 2 * evict_list(table_width, page_size, most)) * sizeof(int);
}

int cpattn_cache_evict(float* weights, const float* scores, void* k_cache, void* v_cache,
                       int64_t num_pages, int page_size, int64_t page_stride, int64_t token_stride,
                       int64_t head_stride, const int32_t* block_table, int table_width,
                       int64_t table_stride, const int32_t* ctx_lens, const int32_t* keep,
                       int first, int recent, int most, int32_t* new_lens, int32_t* kept,
                       int32_t* freed, int num_freed_max, int32_t* num_freed, int R, int Hkv,
                       int D, int dtype, void* workspace, size_t workspace_bytes,
                       cpattn_stream_t stream) {
  int rc = check_heads(Hkv, Hkv, D, dtype);
  if (rc != CPATTN_OK) return rc;
  CacheShape c = {num_pages, page_size, page_stride, token_stride, head_stride};
  if (!check_cache(k_cache, v_cache, c, D) ||
      !evict_shape_ok(R, Hkv, table_width, page_size, most) || table_stride < table_width ||
      first < 0 || recent < 0 || num_freed_max < 0)
    return CPATTN_ERR_INVALID_ARG;
  if (!num_freed || !aligned(num_freed, 4) || (num_freed_max > 0 && !freed) || !aligned(freed, 4))
    return CPATTN_ERR_INVALID_ARG;
  if (R > 0 && (!weights || !aligned(weights, 4) || !aligned(scores, 4) ||
                (table_width > 0 && !block_table) || !aligned(block_table, 4) || !ctx_lens ||
                !aligned(ctx_lens, 4) || !keep || !aligned(keep, 4) || !new_lens ||
                !aligned(new_lens, 4) || !kept || !aligned(kept, 4)))
    return CPATTN_ERR_INVALID_ARG;
  const size_t need = cpattn_cache_evict_workspace_bytes(R, Hkv, table_width, page_size, most);
  const Bytes rows = 4 * (Bytes)R, wc = R > 0 ? cache_bytes(c, Hkv, D) : 0,
              ww = R > 0 ? 4 * (Bytes)num_pages * Hkv * page_size : 0;
  // Keys and values may lie side by side in one tensor, but share nothing: the shift moves both.
  if (R > 0 && caches_meet(k_cache, v_cache, c, Hkv, D)) return CPATTN_ERR_INVALID_ARG;
  const Stretch caches[] = {{k_cache, wc}, {v_cache, wc}};
  const Stretch written[] = {{weights, ww},
                             {new_lens, rows},
                             {kept, rows * Hkv * most},
                             {freed, 4 * (Bytes)num_freed_max},
                             {num_freed, 4}};
  const Stretch read[] = {{ctx_lens, rows},
                          {keep, rows},
                          {scores != weights ? scores : nullptr, scores != weights && scores ? ww : 0},
                          table_stretch(block_table, R, table_width, table_stride)};
  if (any_meet(written, read) || any_meet(written, caches)) return CPATTN_ERR_INVALID_ARG;
  for (const Stretch& x : caches) {
    const Stretch one[] = {x};
    if (any_meet(one, read)) return CPATTN_ERR_INVALID_ARG;
  }
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return CPATTN_ERR_WORKSPACE;
  const Stretch scratch[] = {{workspace, (Bytes)need}};
  if (any_meet(scratch, read) || any_meet(scratch, written) || any_meet(scratch, caches))
    return CPATTN_ERR_INVALID_ARG;
  int* err = device_error_word();
  if (err == nullptr) return CPATTN_ERR_CUDA;
  EvictArgs a = {PageDiv(page_size)};
  a.weights = weights;
  a.scores = scores ? scores : weights;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.cache = c;
  a.table = block_table;
  a.width = table_width;
  a.table_stride = table_stride;
  a.ctx = ctx_lens;
  a.keep = keep;
  a.first = first;
  a.recent = recent;
  a.most = most;
  a.new_lens = new_lens;
  a.kept = kept;
  a.freed = freed;
  a.num_freed_max = num_freed_max;
  a.num_freed = num_freed;
  a.R = R;
  a.Hkv = Hkv;
  a.D = D;
  a.fills = static_cast<int*>(workspace);
  a.lists = a.fills + (int64_t)R * Hkv;
  a.item0 = 0;
  a.list_cap = evict_list(table_width, page_size, most);
  a.err = err;
  return status(launch_cache_evict(a, (cudaStream_t)stream));
}

}  // extern "C"
