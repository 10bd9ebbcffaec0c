// mk_decode_step_kv8: the decode step, one grid per operator, over an 8-bit
// paged cache.  Every operator but attention runs the task bodies of the
// worker kernel, as mk_decode_step_perop does; attention becomes
//   qkv_norm_rope   the per-head norms and RoPE of the QKV projection's rows,
//   mk_kv8_store    the new K/V rows into the cache,
//   mk_kv8_attention,
// and at batch >= 2 a pass that lays the result out as the O projection's
// operand.  A device-side failure sets the handle's status word before
// anything of the caller's is written; every later launch of the step looks
// at that word first.
#include <cuda_runtime.h>

#include <algorithm>

#include "kv8.cuh"
#include "mk_handle.hpp"

namespace mk {
namespace {

struct RopeArgs {
  const float *qkv;  // [B][Hkv][rep + 2][D]: q heads, k, v of a kv head
  const uint16_t *q_norm, *k_norm;
  const float *rope;  // [positions][D / 2][2] cos, sin
  const int32_t *kv_len;
  const int32_t *page_table;
  int32_t *status;
  float *q, *k, *v;  // [B][Hq][D], [B][Hkv][D], [B][Hkv][D]
  int hkv, rep, capacity, page_size, max_pages, n_pages;
  bool check;  // the step's first launch of this kind: look at the page table
  float eps;
};

__device__ __forceinline__ float bf(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// One CTA per sequence and kv head, one warp per row of its group.  Bound by
// latency: a few KB per CTA.
template <int D>
__global__ void __launch_bounds__(256) qkv_norm_rope(const __grid_constant__ RopeArgs a) {
  pdl_trigger();
  pdl_wait();
  if (*(volatile const int32_t *)a.status != 0) return;
  const int g = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31;
  const int pos = a.kv_len[b];
  if (pos < 0 || pos >= a.capacity) return;  // the step's other launches report it
  if (a.check && g == 0) {
    // pages of the positions 0 .. pos
    for (int j = threadIdx.x; j <= pos / a.page_size; j += blockDim.x) {
      const int page = a.page_table[(int64_t)b * a.max_pages + j];
      if ((page < 0 || page >= a.n_pages) && atomicCAS(a.status, kDevOk, kDevBadInput) == kDevOk) {
        a.status[1] = -1;
        a.status[2] = b;
        a.status[3] = (int)blockIdx.x;
      }
    }
  }
  constexpr int N = D / 32;
  for (int row = threadIdx.x >> 5; row < a.rep + 2; row += blockDim.x >> 5) {
    const float *src = a.qkv + (((int64_t)b * a.hkv + g) * (a.rep + 2) + row) * D;
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = src[lane + 32 * i];
    if (row <= a.rep) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      const float inv = rsqrtf(ss / (float)D + a.eps);
      const uint16_t *gain = row < a.rep ? a.q_norm : a.k_norm;
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] *= inv * bf(gain[lane + 32 * i]);
      const float *rope = a.rope + (int64_t)pos * D;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {  // dims lane + 32 i and lane + 32 i + D / 2
        const float c = rope[2 * (lane + 32 * i)], s = rope[2 * (lane + 32 * i) + 1];
        const float x0 = x[i], x1 = x[i + N / 2];
        x[i] = x0 * c - x1 * s;
        x[i + N / 2] = x1 * c + x0 * s;
      }
    }
    float *dst = row < a.rep ? a.q + (((int64_t)b * a.hkv + g) * a.rep + row) * D
                             : (row == a.rep ? a.k : a.v) + ((int64_t)b * a.hkv + g) * D;
#pragma unroll
    for (int i = 0; i < N; ++i) dst[lane + 32 * i] = x[i];
  }
}

__device__ __forceinline__ uint16_t to_bf(float f) {  // round to nearest even
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
  return r;
}

// The attention output [B][K] as the batched O projection's operand: two bf16
// terms (x = hi + lo) of element (k, b), hi at the place below and lo 4
// elements further, in 512-byte blocks per (16 k, 8 sequences), the order of
// the worker kernel's B fragments.
__global__ void attention_operand(const float *att, uint16_t *opnd, int K, int nn,
                                  const int32_t *status) {
  pdl_trigger();
  pdl_wait();
  const int k = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y, kk = k & 15;
  if (k >= K || *(volatile const int32_t *)status != 0) return;
  const float x = att[(int64_t)b * K + k];
  const int64_t at = ((int64_t)(k >> 4) * nn + (b >> 3)) * 256 + ((b & 7) * 4 + ((kk & 7) >> 1)) * 8 +
                     (kk >> 3) * 2 + (kk & 1);
  const uint16_t hi = to_bf(x);
  opnd[at] = hi;
  opnd[at + 4] = to_bf(x - bf(hi));
}

mk_status refuse(mk_handle *h, mk_status s, const char *text) noexcept {
  try {
    h->err = text;
  } catch (...) {  // no memory for the text: the status still says what happened
  }
  return s;
}

// The step's rows in its workspace, then the attention's own.
struct StepPlaces {
  int64_t q, k, v, att, attention, total;
};

mk_batch step_batch(const mk_handle *h, const int32_t *kv_len, const int32_t *table, int max_pages) {
  mk_batch b{};
  b.n_seqs = b.n_rows = h->cfg.batch;
  b.max_rows = 1;
  b.max_pages = max_pages;
  b.d_kv_len = kv_len;
  b.d_page_table = table;
  return b;
}

// Checks what the workspace size depends on; MK_OK and the places, or a refusal.
mk_status step_places(mk_handle *h, const mk_kv8_cache *c, int max_pages, StepPlaces *out) {
  if (h->host_only) return refuse(h, MK_ERR_ARG, "handle was made by mk_plan_graph");
  const char *why = check_kv8_cache(c, 0);
  if (why) return refuse(h, MK_ERR_ARG, why);
  const mk_model_config &m = h->cfg;
  if (c->device != h->device) return refuse(h, MK_ERR_ARG, "the cache is on another device than the handle");
  if (c->n_layers != m.n_layers || c->n_kv_heads != m.n_kv_heads || c->head_dim != m.head_dim)
    return refuse(h, MK_ERR_ARG, "the cache has other layers, kv heads or head_dim than the handle");
  static const int32_t any = 0;  // the sizes do not depend on the pointers
  const mk_batch b = step_batch(h, &any, &any, max_pages);
  why = check_batch(&b, c->page_size);
  if (why) return refuse(h, MK_ERR_ARG, why);
  if ((int64_t)max_pages * c->page_size < m.kv_capacity)
    return refuse(h, MK_ERR_ARG, "the page table covers fewer than kv_capacity positions");
  int64_t attention = 0;
  if (mk_kv8_attention_workspace(c, m.n_q_heads, MK_F32, &b, &attention) != MK_OK)
    return refuse(h, MK_ERR_ARG, mk_last_error(nullptr));
  const int64_t q = 4ll * m.batch * m.n_q_heads * m.head_dim, kv = 4ll * m.batch * m.n_kv_heads * m.head_dim;
  *out = StepPlaces{0, q, q + kv, q + 2 * kv, 2 * q + 2 * kv, 2 * q + 2 * kv + attention};
  return MK_OK;
}

}  // namespace
}  // namespace mk

extern "C" mk_status mk_decode_step_kv8_workspace(mk_handle *h, const mk_kv8_cache *cache,
                                                  int max_pages, int64_t *bytes) {
  if (!h) return mk::ops_fail(MK_ERR_ARG, "mk_decode_step_kv8_workspace", "null handle");
  if (!bytes) return mk::refuse(h, MK_ERR_ARG, "null result");
  mk::StepPlaces w{};
  const mk_status s = mk::step_places(h, cache, max_pages, &w);
  if (s == MK_OK) *bytes = w.total;
  return s;
}

extern "C" mk_status mk_decode_step_kv8(mk_handle *h, const int32_t *d_tokens_in,
                                        int32_t *d_tokens_out, int32_t *d_kv_len,
                                        const mk_kv8_cache *cache, const int32_t *d_page_table,
                                        int max_pages, float *d_logits, void *d_workspace,
                                        int64_t workspace_bytes, void *stream) {
  using namespace mk;
  if (!h) return ops_fail(MK_ERR_ARG, "mk_decode_step_kv8", "null handle");
  StepPlaces w{};
  const mk_status s = step_places(h, cache, max_pages, &w);
  if (s != MK_OK) return s;
  if (!h->loaded) return refuse(h, MK_ERR_NOT_LOADED, "mk_load_weights has not been called");
  if (!d_tokens_in || !d_tokens_out || !d_kv_len || !d_page_table)
    return refuse(h, MK_ERR_ARG, "null buffer");
  if (ops_workspace("mk_decode_step_kv8", d_workspace, workspace_bytes, w.total) != MK_OK)
    return refuse(h, MK_ERR_ARG, mk_last_error(nullptr));
  DeviceGuard guard(h->device);
  if (guard.error() != cudaSuccess) {
    ops_cuda_fail(guard.error(), "mk_decode_step_kv8");
    return refuse(h, MK_ERR_CUDA, cudaGetErrorString(guard.error()));
  }

  const mk_model_config &m = h->cfg;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  Params p = h->base;
  p.tokens_in = d_tokens_in;
  p.tokens_out = d_tokens_out;
  p.kv_len = d_kv_len;
  p.logits = d_logits;
  p.persistent = 0;
  p.dispatch = 0;
  p.page_size = 0;  // the other operators read no cache
  char *base = static_cast<char *>(d_workspace);
  float *q = reinterpret_cast<float *>(base + w.q), *k = reinterpret_cast<float *>(base + w.k);
  float *v = reinterpret_cast<float *>(base + w.v), *att = reinterpret_cast<float *>(base + w.att);
  mk_kv8_cache c = *cache;
  c.d_status = nullptr;  // what they check has been checked for the handle's status word
  const mk_batch batch = step_batch(h, d_kv_len, d_page_table, max_pages);
  const int D = m.head_dim, rep = m.n_q_heads / m.n_kv_heads;
  const mk_rows q_rows{q, MK_F32, (int64_t)m.n_q_heads * D, D};
  const mk_rows k_rows{k, MK_F32, (int64_t)m.n_kv_heads * D, D};
  const mk_rows v_rows{v, MK_F32, (int64_t)m.n_kv_heads * D, D};
  bool first = true;
  for (int o = 0; o + 1 < (int)h->op_offset.size(); ++o) {
    const int n = h->op_offset[o + 1] - h->op_offset[o];
    if (n == 0) continue;
    const int task = h->graph.op_tasks[o][0];
    cudaError_t e = cudaSuccess;
    if (h->graph.type[task] != kAttn) {
      p.task_list = h->d_op_tasks + h->op_offset[o];
      e = launch_tasks(p, n, h->smem, st);
    } else {
      const int layer = h->graph.layer[task];
      const DevLayer &L = h->layers[layer];
      const RopeArgs r{L.qkv, L.q_norm, L.k_norm, p.rope, d_kv_len, d_page_table, p.status, q, k, v,
                       m.n_kv_heads, rep, m.kv_capacity, c.page_size, max_pages, c.n_pages, first, m.rms_eps};
      first = false;
      const dim3 grid(m.n_kv_heads, m.batch);
      e = pdl_launch(D == 128 ? qkv_norm_rope<128> : qkv_norm_rope<64>, grid, 256, 0, st, r);
      if (e == cudaSuccess) e = kv8_store_launch(c, layer, k_rows, v_rows, batch, p.status, st);
      if (e == cudaSuccess)
        e = kv8_attention_launch(c, layer, q_rows, m.n_q_heads, p.attn_scale, m.batch > 1 ? att : L.att,
                                 nullptr, batch, base + w.attention, p.status, st);
      if (e == cudaSuccess && m.batch > 1) {
        const int K = m.n_q_heads * D;
        e = pdl_launch(attention_operand, dim3((K + 255) / 256, m.batch), 256, 0, st, (const float *)att, L.attb, K,
                       p.nn, (const int32_t *)p.status);
      }
    }
    if (e != cudaSuccess) {
      ops_cuda_fail(e, "mk_decode_step_kv8");
      return refuse(h, MK_ERR_CUDA, cudaGetErrorString(e));
    }
  }
  return MK_OK;
}
