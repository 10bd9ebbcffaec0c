// mk_kv8_store: quantise new K/V rows into the blocks of an 8-bit paged cache.
//
// One CTA owns one (touched block, kv head) of K or of V: it alone decides the
// block's scale, so there are no atomics and the result is a function of the
// inputs only.  A CTA keeps the block's new rows in registers as fp32 between
// the maximum and the rounding, so rows are read once and codes written once:
// the call is bound by HBM (element size + 1 bytes per element) once it has
// some thousand rows, and by launch latency for a decode step.
//
// Slots: a sequence with n rows at any offset touches at most floor(n / T) + 2
// blocks, so with f(s) = floor(row_start[s] / T) + 2 s the slots
// [f(s), f(s + 1)) hold the blocks of sequence s and a CTA finds its sequence
// by bisection, without a pass over all lengths.
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

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
};

// Eight row elements as fp32.
template <int DT>
__device__ __forceinline__ void load8(const void *base, int64_t at, float (&x)[8]) {
  if constexpr (DT == MK_F32) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (DT == MK_BF16) {
        f = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
      } else {
        f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
      }
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// Eight scaled values as codes: to nearest even, clamped.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&y)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (FMT == MK_KV8_INT8) {
      uint32_t v = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int q = max(-127, min(127, __float2int_rn(y[4 * i + j])));
        v |= (uint32_t)(q & 0xff) << (8 * j);
      }
      w[i] = v;
    } else {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i], y[4 * i + 1]),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2], y[4 * i + 3]),
                                                   __NV_SATFINITE, __NV_E4M3);
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

// PASSES x blockDim.x octets of 8 elements make one block of T x D elements.
template <int FMT, int DT, int PASSES>
__global__ void __launch_bounds__(256) kv8_store_kernel(const __grid_constant__ StoreArgs a) {
  if (gated(a.gate)) return;
  const int T = a.c.block, P = a.c.page_size, D = a.c.head_dim;
  const int slot = blockIdx.x, h = blockIdx.y, which = blockIdx.z;
  // the last sequence with f(s) <= slot
  int s = 0;
  if (a.b.d_row_start) {
    int hi = a.b.n_seqs - 1;
    while (s < hi) {
      const int mid = (s + hi + 1) >> 1;
      if ((int64_t)a.b.d_row_start[mid] / T + 2ll * mid <= slot) s = mid;
      else hi = mid - 1;
    }
  } else {
    s = slot;  // one row, one block per sequence
  }
  if (h == 0 && which == 0 && threadIdx.x == 0 && slot < a.b.n_seqs) {
    // the grid has at least n_seqs slots: every sequence is checked once,
    // also one that a row_start out of order hides from the bisection
    const SeqRows mine = seq_rows(a.b, P, slot);
    if (mine.bad) record_status(a.c.d_status, MK_ERR_DEVICE, slot, mine.value(a.b), mine.bad);
  }
  const SeqRows q = seq_rows(a.b, P, s);
  const int i = a.b.d_row_start ? (int)(slot - ((int64_t)q.r0 / T + 2ll * s)) : 0;
  if (q.bad || q.n == 0 || i < 0) return;
  const int first = (q.c / T + i) * T;  // first position of the block
  const int end = q.c + q.n;
  if (first >= end) return;
  const int page = a.b.d_page_table[(int64_t)s * a.b.max_pages + first / P];
  if (page < 0 || page >= a.c.n_pages) {
    if (threadIdx.x == 0) record_status(a.c.d_status, MK_ERR_DEVICE, s, page, MK_CHECK_PAGE);
    return;
  }
  const int64_t slab = kv8_slab(a.c, a.layer, page, h);
  uint8_t *codes = static_cast<uint8_t *>(which ? a.c.d_v : a.c.d_k) + (slab * P + first % P) * D;
  float *scale = (which ? a.c.d_v_scale : a.c.d_k_scale) + slab * (P / T) + (first % P) / T;
  const mk_rows &x = a.x[which];
  const int per_row = D / 8;
  const int n_old = max(0, q.c - first);     // rows of the block that are there already
  const int n_end = min(T, end - first);     // rows [n_old, n_end) are new
  const float old = n_old > 0 ? *scale : 0.0f;

  float v[PASSES][8];
  uint32_t top = 0;  // bits of the largest magnitude: above those of infinity for a NaN
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int o = p * blockDim.x + threadIdx.x;
    const int row = o / per_row, d = (o - row * per_row) * 8;
    if (row >= n_old && row < n_end) {
      const int64_t r = q.r0 + (first + row - q.c);
      load8<DT>(x.data, r * x.row_stride + h * x.head_stride + d, v[p]);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[p][j]) & 0x7fffffffu);
    }
  }
  __shared__ uint32_t warp_top[8];
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
  __syncthreads();
  for (int w = 0; w < (int)blockDim.x / 32; ++w) top = max(top, warp_top[w]);

  const float inv_qmax = FMT == MK_KV8_INT8 ? 1.0f / 127.0f : 1.0f / 448.0f;
  float sc = fmaxf(__fmul_rn(__uint_as_float(top), inv_qmax), kScaleMin);
  bool nan = top >= 0x7f800000u;
  if (n_old > 0) {
    nan = nan || isnan(old);
    sc = fmaxf(sc, old);
  }
  const float inv = __frcp_rn(sc);
  if (n_old > 0 && !nan && sc != old) {
    // the block's earlier codes follow the larger scale
    const float ratio = __fmul_rn(old, inv);
    for (int o = threadIdx.x; o < n_old * per_row; o += blockDim.x) {
      uint2 *at = reinterpret_cast<uint2 *>(codes + (int64_t)o * 8);
      float y[8];
      decode8<FMT>(*at, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(y[j], ratio);
      *at = encode8<FMT>(y);
    }
  }
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int o = p * blockDim.x + threadIdx.x;
    const int row = o / per_row;
    if (row >= n_old && row < n_end) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = nan ? 0.0f : __fmul_rn(v[p][j], inv);
      *reinterpret_cast<uint2 *>(codes + (int64_t)o * 8) = encode8<FMT>(y);
    }
  }
  // every thread has read the old scale: the barrier above orders that before this
  if (threadIdx.x == 0) *scale = nan ? __int_as_float(0x7fc00000) : sc;
}

template <int FMT, int DT>
cudaError_t launch_store(const StoreArgs &a, cudaStream_t st) {
  const int octets = a.c.block * a.c.head_dim / 8;  // 128 .. 2048
  const int threads = octets < 256 ? octets : 256;
  const int64_t slots = a.b.d_row_start ? (int64_t)a.b.n_rows / a.c.block + 2ll * a.b.n_seqs
                                        : (int64_t)a.b.n_seqs;
  const dim3 grid((unsigned)slots, (unsigned)a.c.n_kv_heads, 2);
  switch (octets / threads) {
    case 1: kv8_store_kernel<FMT, DT, 1><<<grid, threads, 0, st>>>(a); break;
    case 2: kv8_store_kernel<FMT, DT, 2><<<grid, threads, 0, st>>>(a); break;
    case 4: kv8_store_kernel<FMT, DT, 4><<<grid, threads, 0, st>>>(a); break;
    default: kv8_store_kernel<FMT, DT, 8><<<grid, threads, 0, st>>>(a); break;
  }
  return cudaGetLastError();
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
  const StoreArgs a{cache, batch, {k, v}, layer, gate};
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
