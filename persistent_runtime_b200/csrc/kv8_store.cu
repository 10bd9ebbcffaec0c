// mk_kv8_store: quantise new K/V rows into the blocks of an 8-bit paged cache.
//
// One warp (or the 2 to 8 warps that its rows fill) owns one touched block of K
// or of V for one kv head: it alone decides the block's scale, so there are no
// atomics and the result is a function of the inputs only.  A block's new rows
// stay in registers, as they were loaded, between the maximum and the rounding:
// rows are read once and codes written once.  Bound by HBM (element size + 1
// bytes per element) from some thousand rows on, by launch latency for a decode
// step.  The warps of a CTA take neighbouring heads of the same rows, which lie
// next to each other in the usual [rows][heads][head_dim]: 98k bf16 rows of 8
// heads (604 MB) took 347 us with a CTA per head, 156 us with a CTA that went
// through the heads one after the other, 143 us side by side and 102 us (5.9 TB/s)
// with packed products and no divisions.  Eight octets of a lane instead of 16
// (twice the warps for a block) were slower, 137 against 116 us.
//
// Slots: a sequence with n rows at any offset touches at most floor(n / T) + 2
// blocks, so with f(s) = floor(row_start[s] / T) + 2 s the slots
// [f(s), f(s + 1)) hold the blocks of sequence s and a warp finds its sequence
// by a 32-ary search, without a pass over all lengths.
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "kv8.cuh"

namespace mk {
namespace {

constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126: its reciprocal is finite

struct StoreArgs {
  mk_kv8_cache c;
  mk_batch b;
  mk_rows x[2];  // K, V
  int layer;
  const int32_t *gate;
  int t_log2, split_log2;  // of block, and of the warps of a block
};

// Eight row elements as they lie in memory.
template <int DT>
struct Octet {
  uint4 w[DT == MK_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const char *at) {
    w[0] = __ldg(reinterpret_cast<const uint4 *>(at));
    if constexpr (DT == MK_F32) w[1] = __ldg(reinterpret_cast<const uint4 *>(at) + 1);
  }
  // The larger of `top` and the largest magnitude, as bits: the order of the
  // magnitudes, with NaN above infinity.  16-bit types: two maxima in halves.
  __device__ __forceinline__ uint32_t max_bits(uint32_t top) const {
    if constexpr (DT == MK_F32) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        top = max(max(max(top, w[i].x & 0x7fffffffu), max(w[i].y & 0x7fffffffu, w[i].z & 0x7fffffffu)), w[i].w & 0x7fffffffu);
      return top;
    } else {
      using H2 = typename std::conditional<DT == MK_BF16, __nv_bfloat162, __half2>::type;
      const uint32_t u[4] = {w[0].x & 0x7fff7fffu, w[0].y & 0x7fff7fffu, w[0].z & 0x7fff7fffu, w[0].w & 0x7fff7fffu};
      H2 m = *reinterpret_cast<const H2 *>(&top);
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __hmax2_nan(m, *reinterpret_cast<const H2 *>(&u[i]));
      return *reinterpret_cast<const uint32_t *>(&m);
    }
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    if constexpr (DT == MK_F32) {
      const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = DT == MK_BF16 ? make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u))
                                       : __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
};

// The largest magnitude in fp32, from max_bits() reduced over threads.
template <int DT>
__device__ __forceinline__ float max_value(uint32_t top) {
  if constexpr (DT == MK_F32) return __uint_as_float(top);
  const uint32_t h = max(top & 0xffffu, top >> 16);
  if constexpr (DT == MK_BF16) return __uint_as_float(h << 16);
  return __half2float(__ushort_as_half((unsigned short)h));
}

// Two products in one instruction.  (A packed sum behind it would be fused with
// it, in one rounding.)
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// The codes of eight values x over a scale, given its reciprocal: the product
// is rounded to fp32, then to nearest even.  It is at most qmax, up to its own
// rounding.  int8: adding 1.5 2^23 rounds to an integer whose lowest byte is
// the code.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t w[2];
  const float2 by = make_float2(inv, inv);
  constexpr float kMagic = 12582912.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float2 y[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) y[j] = mul2(make_float2(x[4 * i + 2 * j], x[4 * i + 2 * j + 1]), by);
    if constexpr (FMT == MK_KV8_INT8) {
      w[i] = __byte_perm(__byte_perm(__float_as_uint(__fadd_rn(y[0].x, kMagic)), __float_as_uint(__fadd_rn(y[0].y, kMagic)), 0x0040),
                         __byte_perm(__float_as_uint(__fadd_rn(y[1].x, kMagic)), __float_as_uint(__fadd_rn(y[1].y, kMagic)), 0x0040),
                         0x5410);
    } else {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(y[0], __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(y[1], __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
  }
  return make_uint2(w[0], w[1]);
}

template <int FMT>
__device__ __forceinline__ void decode8(uint2 q, float (&y)[8]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t byte = (w[i >> 2] >> (8 * (i & 3))) & 0xffu;
    if constexpr (FMT == MK_KV8_INT8) {
      y[i] = (float)(int8_t)byte;
    } else {
      y[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
    }
  }
}

// The last sequence with f(s) <= slot, by all lanes of a warp together: each
// looks at one of 32 places between lo and hi.
__device__ __forceinline__ int find_seq(const mk_batch &b, int t_log2, int slot) {
  int lo = 0, hi = b.n_seqs;  // f(lo) <= slot, or lo = 0; f(hi) > slot, or hi = n_seqs
  const int lane = threadIdx.x & 31;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int s = lo + lane * step;
    const bool le = s < hi && (b.d_row_start[s] >> t_log2) + 2ll * s <= slot;
    const int n = __popc(__ballot_sync(0xffffffffu, le));  // f increases: the first n lanes
    const int at = lo + max(0, n - 1) * step;
    hi = min(hi, at + step);
    lo = at;
  }
  return lo;
}

// A warp holds PASSES x 32 octets of 8 elements; 2^split_log2 warps make one block
// of T x D elements.
template <int FMT, int DT, int PASSES>
__global__ void __launch_bounds__(256) kv8_store_kernel(const __grid_constant__ StoreArgs a) {
  pdl_trigger();
  pdl_wait();
  if (gated(a.gate)) return;
  const int T = a.c.block, P = a.c.page_size, D = a.c.head_dim;
  const int slot = blockIdx.x, which = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.y == 0 && which == 0 && threadIdx.x == 0 && slot < a.b.n_seqs) {
    // the grid has at least n_seqs slots: every sequence is checked once,
    // also one that a row_start out of order hides from the search
    const SeqRows mine = seq_rows(a.b, P, slot);
    if (mine.bad) record_status(a.c.d_status, MK_ERR_DEVICE, slot, mine.value(a.b), mine.bad);
  }
  const int s = a.b.d_row_start ? find_seq(a.b, a.t_log2, slot) : slot;  // without: one block per sequence
  const SeqRows q = seq_rows(a.b, P, s);
  const int i = a.b.d_row_start ? (int)(slot - ((q.r0 >> a.t_log2) + 2ll * s)) : 0;
  // slots behind the blocks of a sequence: rows behind the last one, or a row_start out of order
  if (q.bad || q.n == 0 || i < 0 || i > (q.n >> a.t_log2) + 1) return;
  const int first = ((q.c >> a.t_log2) + i) << a.t_log2;  // first position of the block
  const int end = q.c + q.n;
  if (first >= end) return;
  const int entry = first / P, in_page = first - entry * P;
  const int page = a.b.d_page_table[(int64_t)s * a.b.max_pages + entry];
  const int h = (int)(blockIdx.y * (blockDim.x >> 5) + warp) >> a.split_log2;
  const bool on = h < a.c.n_kv_heads;  // the last CTA's warps may be too many
  const mk_rows &x = a.x[which];
  const int row_log2 = D == 128 ? 4 : 3;  // octets of a row
  const int n_old = max(0, q.c - first);  // rows of the block that are there already
  const int n_end = on ? min(T, end - first) : 0;  // rows [n_old, n_end) are new
  const int sub = warp & ((1 << a.split_log2) - 1);
  const int row_step = 32 >> row_log2 << a.split_log2;  // rows of a pass
  const int row0 = (sub << 5 | lane) >> row_log2;
  const int d0 = (lane & ((1 << row_log2) - 1)) * 8;
  constexpr int kSize = DT == MK_F32 ? 4 : 2;
  const char *src = static_cast<const char *>(x.data) +
                    ((q.r0 + (int64_t)(first + row0 - q.c)) * x.row_stride + h * x.head_stride + d0) * kSize;
  const int64_t src_step = row_step * x.row_stride * kSize;
  const unsigned n_new = (unsigned)max(0, n_end - n_old);
  Octet<DT> v[PASSES];
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    if ((unsigned)(row0 + p * row_step - n_old) < n_new) v[p].load(src);
    else v[p] = Octet<DT>{};
    src += src_step;
  }
  if (page < 0 || page >= a.c.n_pages) {
    if (threadIdx.x == 0) record_status(a.c.d_status, MK_ERR_DEVICE, s, page, MK_CHECK_PAGE);
    return;
  }
  const int64_t slab = kv8_slab(a.c, a.layer, page, on ? h : 0);
  uint8_t *codes = static_cast<uint8_t *>(which ? a.c.d_v : a.c.d_k) + (slab * P + in_page) * D;
  float *scale = (which ? a.c.d_v_scale : a.c.d_k_scale) + ((slab * P + in_page) >> a.t_log2);
  const float old = n_old > 0 ? *scale : 0.0f;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) top = v[p].max_bits(top);
  if constexpr (DT != MK_F32) top = max(top & 0xffffu, top >> 16);
  top = __reduce_max_sync(0xffffffffu, top);
  __shared__ uint32_t tops[8];
  if (a.split_log2 > 0) {
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    for (int w = warp - sub; w < warp - sub + (1 << a.split_log2); ++w) top = max(top, tops[w]);
  }

  const float a_max = max_value<DT>(top);
  const float inv_qmax = FMT == MK_KV8_INT8 ? 1.0f / 127.0f : 1.0f / 448.0f;
  float sc = fmaxf(__fmul_rn(a_max, inv_qmax), kScaleMin);
  bool nan = !(a_max < INFINITY);
  if (n_old > 0) {
    nan = nan || isnan(old);
    sc = fmaxf(sc, old);
  }
  const float inv = __frcp_rn(sc);
  if (n_old > 0 && !nan && sc != old) {
    // the block's earlier codes follow the larger scale
    const float ratio = __fmul_rn(old, inv);
    for (int row = row0; row < min(n_old, n_end); row += row_step) {
      uint2 *at = reinterpret_cast<uint2 *>(codes + (int64_t)row * D + d0);
      float y[8];
      decode8<FMT>(*at, y);
      *at = encode8<FMT>(y, ratio);
    }
  }
  uint8_t *dst = codes + row0 * D + d0;
  const int dst_step = row_step * D;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    if ((unsigned)(row0 + p * row_step - n_old) < n_new) {
      float y[8];
      v[p].values(y);
      *reinterpret_cast<uint2 *>(dst) = nan ? make_uint2(0, 0) : encode8<FMT>(y, inv);
    }
    dst += dst_step;
  }
  // All lanes have read the old scale: other warps' before the barrier above, this one's
  // before this one (the reduction orders no memory).
  __syncwarp();
  if (on && lane == 0 && sub == 0) *scale = nan ? __int_as_float(0x7fc00000) : sc;
}

template <int FMT, int DT>
cudaError_t launch_store(StoreArgs a, cudaStream_t st) {
  // octets of a lane if one warp takes a block: 4 .. 64; at most 64 registers of rows
  const int octets = a.c.block * a.c.head_dim / 8 / 32;
  constexpr int kMost = DT == MK_F32 ? 8 : 16;
  const int passes = octets < kMost ? octets : kMost;
  const int split = octets / passes;
  a.split_log2 = __builtin_ctz((unsigned)split);
  a.t_log2 = __builtin_ctz((unsigned)a.c.block);
  const int warps = std::min(8, a.c.n_kv_heads * split);
  const int64_t slots = a.b.d_row_start ? (int64_t)a.b.n_rows / a.c.block + 2ll * a.b.n_seqs
                                        : (int64_t)a.b.n_seqs;
  const int heads = warps / split;
  const dim3 grid((unsigned)slots, (unsigned)((a.c.n_kv_heads + heads - 1) / heads), 2);
  const int threads = heads * split * 32;
  const auto kernel = passes == 4   ? kv8_store_kernel<FMT, DT, 4>
                      : passes == 8 ? kv8_store_kernel<FMT, DT, 8>
                                    : kv8_store_kernel<FMT, DT, kMost>;
  return pdl_launch(kernel, grid, threads, 0, st, a);
}

template <int FMT>
cudaError_t launch_store(const StoreArgs &a, cudaStream_t st) {
  switch (a.x[0].dtype) {
    case MK_F32: return launch_store<FMT, MK_F32>(a, st);
    case MK_BF16: return launch_store<FMT, MK_BF16>(a, st);
    default: return launch_store<FMT, MK_F16>(a, st);
  }
}

}  // namespace

cudaError_t kv8_store_launch(const mk_kv8_cache &cache, int layer, const mk_rows &k, const mk_rows &v,
                             const mk_batch &batch, const int32_t *gate, cudaStream_t stream) {
  const StoreArgs a{cache, batch, {k, v}, layer, gate, 0, 0};
  return cache.format == MK_KV8_INT8 ? launch_store<MK_KV8_INT8>(a, stream)
                                     : launch_store<MK_KV8_E4M3>(a, stream);
}

}  // namespace mk

extern "C" mk_status mk_kv8_store(const mk_kv8_cache *cache, int layer, const mk_rows *k,
                                  const mk_rows *v, const mk_batch *batch, void *stream) {
  using namespace mk;
  const char *why = check_kv8_cache(cache, layer);
  if (!why) why = check_batch(batch, cache->page_size);
  if (!why && batch->n_rows == 0) return MK_OK;
  if (!why) why = check_rows(k);
  if (!why) why = check_rows(v);
  if (!why && k->dtype != v->dtype) why = "k and v rows differ in element type";
  if (why) return ops_fail(MK_ERR_ARG, "mk_kv8_store", why);
  DeviceGuard guard(cache->device);
  if (guard.error() != cudaSuccess) return ops_cuda_fail(guard.error(), "mk_kv8_store");
  const cudaError_t e = kv8_store_launch(*cache, layer, *k, *v, *batch, nullptr,
                                         static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return ops_cuda_fail(e, "mk_kv8_store");
  return MK_OK;
}
