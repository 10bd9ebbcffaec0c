// Shared by the translation units of the 8-bit paged caches and of the page
// calls: argument checks, device guard, status words, small device helpers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "mk.h"

namespace mk {

// Records "call: text" for mk_last_error(NULL) and returns `s`; never throws.
mk_status ops_fail(mk_status s, const char *call, const char *text) noexcept;
mk_status ops_cuda_fail(cudaError_t e, const char *call) noexcept;
// MK_OK if `workspace` is fit for `need` bytes.
mk_status ops_workspace(const char *call, const void *workspace, int64_t have, int64_t need) noexcept;

// Makes `device` current for the duration of a call and the previous device
// current again after it.
class DeviceGuard {
 public:
  explicit DeviceGuard(int device) {
    err_ = cudaGetDevice(&prev_);
    if (err_ == cudaSuccess && prev_ != device) {
      err_ = cudaSetDevice(device);
      changed_ = err_ == cudaSuccess;
    }
  }
  ~DeviceGuard() {
    if (changed_) cudaSetDevice(prev_);
  }
  DeviceGuard(const DeviceGuard &) = delete;
  DeviceGuard &operator=(const DeviceGuard &) = delete;
  cudaError_t error() const { return err_; }

 private:
  cudaError_t err_ = cudaSuccess;
  int prev_ = 0;
  bool changed_ = false;
};

// SM count of a device (looked up once per device); 1 if it is unknown.
int sm_count(int device);

// The checks that the calls on an 8-bit cache share: null, or the reason.
const char *check_kv8_cache(const mk_kv8_cache *c, int layer);
const char *check_batch(const mk_batch *b, int page_size);
const char *check_rows(const mk_rows *r);

// The launches of the two calls, for arguments that have been checked; with
// `gate` they do nothing once *gate (on the device) is not 0.
cudaError_t kv8_store_launch(const mk_kv8_cache &cache, int layer, const mk_rows &k, const mk_rows &v,
                             const mk_batch &batch, const int32_t *gate, cudaStream_t stream);
cudaError_t kv8_attention_launch(const mk_kv8_cache &cache, int layer, const mk_rows &q, int n_q_heads,
                                 float scale, void *out, float *lse, const mk_batch &batch,
                                 void *workspace, const int32_t *gate, cudaStream_t stream);

#ifdef __CUDACC__
// ---------------------------------------------------------------------------
// Device side
// ---------------------------------------------------------------------------
// One failure is kept: the first one whose exchange succeeds.
__device__ __forceinline__ void record_status(int32_t *status, int code, int which, int value,
                                              int check) {
  if (!status) return;
  if (atomicCAS(status, 0, code) == 0) {
    status[1] = which;
    status[2] = value;
    status[3] = check;
  }
}

// Place of layer `layer`, head h of page `page` in the pools, in units of one
// (page, layer, head): 64 bits, a pool may hold more than 2^31 codes.
__device__ __forceinline__ int64_t kv8_slab(const mk_kv8_cache &c, int layer, int page, int h) {
  return ((int64_t)page * c.n_layers + layer) * c.n_kv_heads + h;
}

// The new rows of sequence s and its cached length, as far as the device can
// check them.
struct SeqRows {
  int s, r0, n, c;  // sequence, first row, rows, positions cached before them
  int bad;          // 0 or the check that failed
  __device__ int value(const mk_batch &b) const {  // what a failure reports
    return bad == MK_CHECK_ROWS ? b.d_row_start[s + 1] : c;
  }
};

__device__ __forceinline__ SeqRows seq_rows(const mk_batch &b, int page_size, int s) {
  SeqRows q{s, s, 1, b.d_kv_len[s], 0};
  if (b.d_row_start) {
    q.r0 = b.d_row_start[s];
    const int r1 = b.d_row_start[s + 1];
    if (q.r0 < 0 || r1 < q.r0 || r1 > b.n_rows) {
      q.bad = MK_CHECK_ROWS;
      q.n = 0;  // not even the rows are known
      return q;
    }
    q.n = r1 - q.r0;
    if (q.n > b.max_rows) q.bad = MK_CHECK_ROWS;
  }
  if (q.n > 0 && (q.c < 0 || (int64_t)q.c + q.n > (int64_t)b.max_pages * page_size))
    q.bad = MK_CHECK_LENGTH;
  return q;
}

__device__ __forceinline__ bool gated(const int32_t *gate) {
  return gate && *(volatile const int32_t *)gate != 0;
}

// Launches that may get ready before the one in front of them has ended (its
// kernel calls pdl_trigger, or ends) and wait for its end with pdl_wait, before
// they read or write anything.
template <typename... Params, typename... Args>
cudaError_t pdl_launch(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                       const Args &...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

}  // namespace mk
