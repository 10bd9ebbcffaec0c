"""Python binding of libmk.so, the decode-step megakernel (C ABI in include/mk.h).

Argument marshalling only: every step of the decode path runs in the library's
CUDA kernels.  torch is used for device memory and streams.  If libmk.so is
missing the import of the binding fails loudly: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmk.so")

MK_OK, MK_ERR_ARG, MK_ERR_CUDA, MK_ERR_OOM, MK_ERR_GRAPH = 0, -1, -2, -3, -4
MK_ERR_NOT_LOADED, MK_ERR_TIMEOUT, MK_ERR_DEVICE = -5, -6, -7
TASK_NAMES = {0: "GENERIC", 1: "EMBED", 2: "QKV", 3: "ATTN", 4: "MERGE", 5: "OPROJ",
              6: "GATEUP", 7: "DOWN", 8: "LMHEAD", 9: "ARGMAX", 10: "EMPTY"}

# Every symbol declared in include/mk.h.
EXPORTS = ("mk_plan_graph", "mk_graph_from_edges", "mk_build_graph", "mk_load_weights",
           "mk_decode_step", "mk_decode_steps", "mk_decode_steps_paged", "mk_decode_step_perop",
           "mk_decode_step_noalloc",
           "mk_sync_status", "mk_reset",
           "mk_graph_export", "mk_get_info", "mk_final_hidden", "mk_debug_set_event_count",
           "mk_set_trace", "mk_set_timeout_us", "mk_last_error", "mk_destroy",
           "mk_kv8_store", "mk_kv8_attention", "mk_kv8_attention_workspace",
           "mk_pages_workspace", "mk_pages_fork", "mk_pages_free", "mk_pages_reserve",
           "mk_pages_compact", "mk_pages_copy", "mk_decode_step_kv8",
           "mk_decode_step_kv8_workspace")

MK_KV8_INT8, MK_KV8_E4M3 = 0, 1
MK_F32, MK_BF16, MK_F16 = 0, 1, 2
MK_KV8_MAX_ROWS, MK_MAX_POOLS = 16, 8
# status word 3 of the calls on 8-bit caches and pages: which check failed
CHECKS = {1: "row_start", 2: "kv_len", 3: "page table entry", 4: "sequence or page of a list",
          5: "fork into a sequence that holds pages", 6: "free pages"}


class MkError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"mk status {status}: {msg}")
        self.status = status


class ModelConfig(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("hidden", ctypes.c_int), ("n_q_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int),
                ("vocab", ctypes.c_int), ("tied_embeddings", ctypes.c_int),
                ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_double),
                ("batch", ctypes.c_int), ("kv_capacity", ctypes.c_int)]


class Tuning(ctypes.Structure):
    _fields_ = [("num_workers", ctypes.c_int), ("col_align", ctypes.c_int),
                ("attn_tasks_per_worker", ctypes.c_int), ("attn_min_chunk", ctypes.c_int),
                ("ring_stages", ctypes.c_int),
                ("ring_stage_bytes", ctypes.c_int), ("l2_prefetch_bytes", ctypes.c_int),
                ("wait_timeout_us", ctypes.c_uint), ("kv_page_size", ctypes.c_int),
                ("l2_stream_policy", ctypes.c_int), ("attn_jit", ctypes.c_int),
                ("dispatch", ctypes.c_int)]


_PP = ctypes.POINTER(ctypes.c_void_p)


class Weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p),
                ("lm_head", ctypes.c_void_p)] + [
        (n, _PP) for n in ("attn_norm", "wq", "wk", "wv", "q_norm", "k_norm", "wo", "mlp_norm",
                           "w_gate", "w_up", "w_down")]


_I32P = ctypes.POINTER(ctypes.c_int32)


class GraphView(ctypes.Structure):
    _fields_ = [("n_tasks", ctypes.c_int32), ("n_events", ctypes.c_int32),
                ("n_edges", ctypes.c_int32), ("num_workers", ctypes.c_int32)] + [
        (n, _I32P) for n in ("task_type", "task_op", "task_layer", "task_idx", "task_dep",
                             "task_trig", "event_count", "event_first", "event_last",
                             "edge_src", "edge_dst")] + [
        (n, ctypes.c_int32) for n in ("qkv_rows", "o_rows", "gu_rows", "down_rows", "lm_rows",
                                      "attn_splits", "attn_chunk")] + [
        ("mma_mb", ctypes.c_int32 * 5), ("mma_kcb", ctypes.c_int32 * 5)]


class Info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("device", "num_workers", "n_tasks", "n_events",
                                               "n_ops", "smem_bytes", "ring_stages",
                                               "ring_stage_bytes")] + [
        ("weight_bytes", ctypes.c_int64), ("act_bytes", ctypes.c_int64)]


class Kv8Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("device", "format", "n_layers", "n_kv_heads", "head_dim",
                                            "page_size", "block", "n_pages")] + [
        (n, ctypes.c_void_p) for n in ("d_k", "d_v", "d_k_scale", "d_v_scale", "d_status")]


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class Batch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("n_seqs", "n_rows", "max_rows", "max_pages")] + [
        (n, ctypes.c_void_p) for n in ("d_row_start", "d_kv_len", "d_page_table")]


class Pages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("device", "n_pages", "n_seqs", "max_pages", "page_size",
                                            "n_pools")] + [
        ("d_pool", ctypes.c_void_p * MK_MAX_POOLS), ("page_bytes", ctypes.c_int64 * MK_MAX_POOLS),
        ("d_page_table", ctypes.c_void_p), ("d_ref", ctypes.c_void_p),
        ("d_status", ctypes.c_void_p)]


_lib = None


def lib():
    """The loaded libmk.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: run `python -m persistent_runtime_b200.build`"
                          " (there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_int
    H = ctypes.POINTER(vp)
    sig = {
        "mk_plan_graph": ([ctypes.POINTER(ModelConfig), ctypes.POINTER(Tuning), i32, H], st),
        "mk_graph_from_edges": ([i32, vp, vp, i32, vp, vp, H], st),
        "mk_build_graph": ([ctypes.POINTER(ModelConfig), ctypes.POINTER(Tuning), i32, H], st),
        "mk_load_weights": ([vp, ctypes.POINTER(Weights), vp], st),
        "mk_decode_step": ([vp, vp, vp, vp, vp, vp, vp, vp], st),
        "mk_decode_step_perop": ([vp, vp, vp, vp, vp, vp, vp, vp], st),
        "mk_decode_steps": ([vp, i32, vp, vp, vp, vp, vp, vp, vp], st),
        "mk_decode_steps_paged": ([vp, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp], st),
        "mk_decode_step_noalloc": ([vp, vp, vp, vp, vp, vp, vp, vp], st),
        "mk_sync_status": ([vp, vp, vp], st),
        "mk_reset": ([vp, vp], st),
        "mk_graph_export": ([vp, ctypes.POINTER(GraphView)], st),
        "mk_get_info": ([vp, ctypes.POINTER(Info)], st),
        "mk_final_hidden": ([vp, ctypes.POINTER(vp)], st),
        "mk_debug_set_event_count": ([vp, i32, i32, vp], st),
        "mk_set_trace": ([vp, vp, ctypes.c_int64], st),
        "mk_set_timeout_us": ([vp, ctypes.c_uint], st),
        "mk_last_error": ([vp], ctypes.c_char_p),
        "mk_destroy": ([vp], None),
        "mk_kv8_store": ([vp, i32, vp, vp, vp, vp], st),
        "mk_kv8_attention": ([vp, i32, vp, i32, ctypes.c_float, vp, vp, vp, vp, ctypes.c_int64, vp],
                             st),
        "mk_kv8_attention_workspace": ([vp, i32, i32, vp, vp], st),
        "mk_decode_step_kv8": ([vp, vp, vp, vp, vp, vp, i32, vp, vp, ctypes.c_int64, vp], st),
        "mk_decode_step_kv8_workspace": ([vp, vp, i32, vp], st),
        "mk_pages_workspace": ([vp, i32, vp], st),
        "mk_pages_fork": ([vp, i32, vp, vp, vp, ctypes.c_int64, vp], st),
        "mk_pages_free": ([vp, i32, vp, vp, ctypes.c_int64, vp], st),
        "mk_pages_reserve": ([vp, vp, vp, vp, ctypes.c_int64, vp], st),
        "mk_pages_compact": ([vp, vp, ctypes.c_int64, vp], st),
        "mk_pages_copy": ([vp, i32, vp, vp, vp, ctypes.c_int64, vp], st),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _check(rc: int, h=None):
    if rc != MK_OK:
        msg = lib().mk_last_error(h)
        raise MkError(rc, msg.decode() if msg else "")


def make_config(w, kv_capacity: int) -> ModelConfig:
    """ModelConfig from any object with the workload attributes (see synth.Workload)."""
    return ModelConfig(w.n_layers, w.hidden, w.n_q_heads, w.n_kv_heads, w.head_dim, w.ffn,
                       w.vocab, int(w.tied_embeddings), w.rms_eps, w.rope_theta, w.batch,
                       kv_capacity)


def make_tuning(**kw) -> Tuning:
    t = Tuning()
    for k, v in kw.items():
        setattr(t, k, v)
    return t


@dataclass
class Graph:
    """Host copy of a graph's tables (same field names as the oracle's)."""
    task_type: np.ndarray
    task_op: np.ndarray
    task_layer: np.ndarray
    task_idx: np.ndarray
    task_dep: np.ndarray
    task_trig: np.ndarray
    event_count: np.ndarray
    event_first: np.ndarray
    event_last: np.ndarray
    edge_src: np.ndarray
    edge_dst: np.ndarray
    num_workers: int
    tiling: tuple
    mma_tiling: tuple = ()  # ((mb, kcb) of QKV, O, GATE_UP, DOWN, LM_HEAD) at batch >= 2

    @property
    def n_tasks(self):
        return int(self.task_type.size)

    @property
    def n_events(self):
        return int(self.event_count.size)


def _export(h) -> Graph:
    v = GraphView()
    _check(lib().mk_graph_export(h, ctypes.byref(v)), h)

    def arr(p, n):
        return np.ctypeslib.as_array(p, shape=(n,)).copy() if n else np.zeros(0, np.int32)

    return Graph(*(arr(getattr(v, f), v.n_tasks) for f in
                   ("task_type", "task_op", "task_layer", "task_idx", "task_dep", "task_trig")),
                 *(arr(getattr(v, f), v.n_events) for f in
                   ("event_count", "event_first", "event_last")),
                 arr(v.edge_src, v.n_edges), arr(v.edge_dst, v.n_edges), v.num_workers,
                 (v.qkv_rows, v.o_rows, v.gu_rows, v.down_rows, v.lm_rows, v.attn_splits,
                  v.attn_chunk),
                 tuple((int(v.mma_mb[i]), int(v.mma_kcb[i])) for i in range(5)))


def plan_graph(w, kv_capacity: int, num_workers: int, **tuning) -> Graph:
    """Host-only graph construction (mk_plan_graph)."""
    h = ctypes.c_void_p()
    cfg = make_config(w, kv_capacity)
    t = make_tuning(**tuning)
    _check(lib().mk_plan_graph(ctypes.byref(cfg), ctypes.byref(t), num_workers, ctypes.byref(h)))
    try:
        return _export(h)
    finally:
        lib().mk_destroy(h)


def graph_from_edges(task_op, task_idx, edges) -> Graph:
    op = np.ascontiguousarray(task_op, dtype=np.int32)
    idx = np.ascontiguousarray(task_idx, dtype=np.int32)
    e = np.asarray(edges, dtype=np.int32).reshape(-1, 2)
    src, dst = np.ascontiguousarray(e[:, 0]), np.ascontiguousarray(e[:, 1])
    h = ctypes.c_void_p()
    _check(lib().mk_graph_from_edges(op.size, op.ctypes.data, idx.ctypes.data, src.size,
                                     src.ctypes.data, dst.ctypes.data, ctypes.byref(h)))
    try:
        return _export(h)
    finally:
        lib().mk_destroy(h)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr()


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


class Megakernel:
    """One handle: graph + device state for one model shape and batch."""

    def __init__(self, w, kv_capacity: int, device: int = 0, **tuning):
        self.w = w
        self.kv_capacity = kv_capacity
        self.device = device
        self._h = ctypes.c_void_p()
        cfg = make_config(w, kv_capacity)
        t = make_tuning(**tuning)
        _check(lib().mk_build_graph(ctypes.byref(cfg), ctypes.byref(t), device,
                                    ctypes.byref(self._h)))
        self._keep = []

    def close(self):
        if self._h:
            lib().mk_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def load_weights(self, weights: dict, stream=None):
        """weights: torch tensors (bf16 or int16/uint16 bit patterns), same keys as synth."""
        Ly = self.w.n_layers
        arrays = {}
        for name in ("attn_norm", "wq", "wk", "wv", "q_norm", "k_norm", "wo", "mlp_norm",
                     "w_gate", "w_up", "w_down"):
            arr = (ctypes.c_void_p * Ly)(*[weights["layers"][l][name].data_ptr() for l in range(Ly)])
            arrays[name] = arr
        W = Weights(weights["embed"].data_ptr(), weights["final_norm"].data_ptr(),
                    None if weights.get("lm_head") is None else weights["lm_head"].data_ptr(),
                    *[ctypes.cast(arrays[n], _PP) for n in
                      ("attn_norm", "wq", "wk", "wv", "q_norm", "k_norm", "wo", "mlp_norm",
                       "w_gate", "w_up", "w_down")])
        _check(lib().mk_load_weights(self._h, ctypes.byref(W), _stream_ptr(stream)), self._h)

    def decode_step(self, tokens_in, tokens_out, kv_len, k_cache, v_cache, logits=None,
                    stream=None):
        _check(lib().mk_decode_step(self._h, _ptr(tokens_in), _ptr(tokens_out), _ptr(kv_len),
                                    _ptr(k_cache), _ptr(v_cache), _ptr(logits),
                                    _stream_ptr(stream)), self._h)

    def decode_steps(self, n_steps, tokens_in, tokens_out, kv_len, k_cache, v_cache, logits=None,
                     stream=None):
        """n_steps steps in one launch; tokens_out holds n_steps x batch tokens."""
        _check(lib().mk_decode_steps(self._h, n_steps, _ptr(tokens_in), _ptr(tokens_out),
                                     _ptr(kv_len), _ptr(k_cache), _ptr(v_cache), _ptr(logits),
                                     _stream_ptr(stream)), self._h)

    def decode_steps_paged(self, n_steps, tokens_in, tokens_out, kv_len, k_pool, v_pool,
                           n_pages, page_table, logits=None, stream=None):
        """n_steps steps on paged K/V pools [n_pages][Ly][Hkv][P][D] with a page table
        [batch][ceil(kv_capacity / P)] (handle built with kv_page_size = P)."""
        _check(lib().mk_decode_steps_paged(self._h, n_steps, _ptr(tokens_in), _ptr(tokens_out),
                                           _ptr(kv_len), _ptr(k_pool), _ptr(v_pool), n_pages,
                                           _ptr(page_table), _ptr(logits), _stream_ptr(stream)),
               self._h)

    def decode_step_perop(self, tokens_in, tokens_out, kv_len, k_cache, v_cache, logits=None,
                          stream=None):
        _check(lib().mk_decode_step_perop(self._h, _ptr(tokens_in), _ptr(tokens_out),
                                          _ptr(kv_len), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(logits), _stream_ptr(stream)), self._h)

    def decode_step_noalloc(self, tokens_in, tokens_out, kv_len, k_cache, v_cache, logits=None,
                            stream=None):
        """mk_decode_step with its working buffers in the library's static region."""
        _check(lib().mk_decode_step_noalloc(self._h, _ptr(tokens_in), _ptr(tokens_out),
                                            _ptr(kv_len), _ptr(k_cache), _ptr(v_cache),
                                            _ptr(logits), _stream_ptr(stream)), self._h)

    def decode_step_kv8(self, tokens_in, tokens_out, kv_len, cache, page_table, logits=None,
                        stream=None):
        """One step, a grid per operator, over an 8-bit paged cache (a KV8Cache with this
        model's layers, kv heads and head_dim) and its int32 page table [batch][max_pages]."""
        import torch
        batch = self.w.batch
        if page_table.dim() != 2 or page_table.shape[0] != batch:
            _refuse(f"page_table must be [{batch}][max_pages]")
        cache._int32(page_table, None, "page_table")
        for t, what in ((tokens_in, "tokens_in"), (tokens_out, "tokens_out"), (kv_len, "kv_len")):
            cache._int32(t, None, what)
            if t.numel() < batch:
                _refuse(f"{what} must have {batch} entries")
        if logits is not None and (logits.dtype is not torch.float32 or not logits.is_contiguous()
                                   or logits.get_device() != cache._index
                                   or logits.numel() < batch * self.w.vocab):
            _refuse(f"logits must be a contiguous float32 tensor [{batch}][{self.w.vocab}] on "
                    f"{cache.device}")
        size = ctypes.c_int64()
        max_pages = page_table.shape[1]
        _check(lib().mk_decode_step_kv8_workspace(self._h, cache._ref, max_pages,
                                                  ctypes.byref(size)), self._h)
        if stream is None:
            stream = torch.cuda.current_stream(cache.device)
        with cache._given(stream):
            ws = torch.empty(size.value, dtype=torch.uint8, device=cache.device)
        _check(lib().mk_decode_step_kv8(self._h, _ptr(tokens_in), _ptr(tokens_out), _ptr(kv_len),
                                        cache._ref, page_table.data_ptr(), max_pages, _ptr(logits),
                                        ws.data_ptr(), size.value, _stream_ptr(stream)), self._h)

    def sync_status(self, stream=None):
        """Returns (status, detail[4]); status 0 = ok."""
        d = (ctypes.c_int32 * 4)()
        rc = lib().mk_sync_status(self._h, _stream_ptr(stream), d)
        return rc, list(d)

    def reset(self, stream=None):
        _check(lib().mk_reset(self._h, _stream_ptr(stream)), self._h)

    def graph(self) -> Graph:
        return _export(self._h)

    def info(self) -> Info:
        i = Info()
        _check(lib().mk_get_info(self._h, ctypes.byref(i)), self._h)
        return i

    def final_hidden_ptr(self) -> int:
        p = ctypes.c_void_p()
        _check(lib().mk_final_hidden(self._h, ctypes.byref(p)), self._h)
        return p.value

    def set_event_count(self, event: int, count: int, stream=None):
        _check(lib().mk_debug_set_event_count(self._h, event, count, _stream_ptr(stream)),
               self._h)

    def set_trace(self, buf=None):
        """buf: int64/uint64 torch tensor with >= 8 * n_tasks elements, or None."""
        if buf is None:
            _check(lib().mk_set_trace(self._h, None, 0), self._h)
        else:
            _check(lib().mk_set_trace(self._h, buf.data_ptr(), buf.numel() * buf.element_size()),
                   self._h)

    def set_timeout_us(self, us: int):
        _check(lib().mk_set_timeout_us(self._h, us), self._h)


# ----------------------------------------------------------------------------
# 8-bit paged caches and the pages of a cache (no handle, caller-owned tensors)
# ----------------------------------------------------------------------------
def _refuse(why: str):
    raise MkError(MK_ERR_ARG, why)


class _Status:
    """The device status words of a cache or of a set of pages."""

    def _new_status(self):
        import torch
        self.status = torch.zeros(4, dtype=torch.int32, device=self.device)

    def sync_status(self):
        """Waits for the device's work; returns (status, [status, which, value, check]), status
        0 = ok, and leaves the words as they are until reset()."""
        import torch
        torch.cuda.synchronize(self.device)
        d = self.status.tolist()
        return d[0], d

    def reset(self):
        self.status.zero_()

    def check(self):
        """Raises MkError for a failure that the device has recorded."""
        rc, d = self.sync_status()
        if rc != 0:
            raise MkError(rc, f"the device refused: {CHECKS.get(d[3], d[3])} (entry {d[1]}, "
                              f"value {d[2]})")

    def _int32(self, t, n, what):
        """Address of a contiguous int32 tensor of n entries (n None: any) on this device."""
        if t.dtype is not self._i32 or t.get_device() != self._index or not t.is_contiguous():
            _refuse(f"{what} must be a contiguous int32 tensor on {self.device}")
        if n is not None and t.numel() != n:
            _refuse(f"{what} must have {n} entries")
        return t.data_ptr()

    def _stream(self, stream):
        """The raw stream: the given one, or the device's current one."""
        return self._raw_stream(self._index) if stream is None else stream.cuda_stream

    def _given(self, stream):
        """A context in which `stream` is the current one: what a call allocates for itself must
        be free on the stream that uses it, not only on the one that is current."""
        import torch
        if stream.device_index != self._index:
            _refuse(f"the stream is not one of {self.device}")
        return torch.cuda.stream(stream)

    def _bind(self, device):
        import torch
        if device.type != "cuda":
            _refuse(f"tensors must be on a CUDA device, not {device}")
        self.device, self._index = device, device.index
        self._i32 = torch.int32
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        # new tensors on the device, from sizes given one by one: the shortest way
        self._bytes = torch.empty(0, dtype=torch.uint8, device=device).new_empty
        self._floats = torch.empty(0, dtype=torch.float32, device=device).new_empty
        self._lib = lib()


class KV8Cache(_Status):
    """A paged K/V cache in 8 bits with a scale for every `block` positions of a (page, layer,
    kv head), on the caller's tensors:

    k, v              int8 or float8_e4m3fn [n_pages][n_layers][n_kv_heads][page_size][head_dim]
    k_scale, v_scale  float32 [n_pages][n_layers][n_kv_heads][page_size / block]

    The pages belong to sequences as in Megakernel.decode_steps_paged: position p of sequence s
    is row p % page_size of page page_table[s][p // page_size].  Calls are asynchronous on the
    current (or the given) stream of the cache's device; use one object per thread.  With
    `stream` the caller's tensors must be ready on that stream, and stay alive (or be recorded
    there with Tensor.record_stream) until the call has run; what a call returns is recorded."""

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        self._bind(k.device)
        formats = {torch.int8: MK_KV8_INT8, torch.float8_e4m3fn: MK_KV8_E4M3}
        if k.dim() != 5 or k.dtype not in formats:
            _refuse("k must be int8 or float8_e4m3fn [n_pages][n_layers][n_kv_heads][page_size]"
                    "[head_dim]")
        if k_scale.dim() != 4 or tuple(k_scale.shape[:3]) != tuple(k.shape[:3]) \
                or k_scale.shape[3] < 1 or k.shape[3] % k_scale.shape[3]:
            _refuse("k_scale must be [n_pages][n_layers][n_kv_heads][page_size / block]")
        if v.shape != k.shape or v.dtype != k.dtype or v_scale.shape != k_scale.shape:
            _refuse("k and v differ in shape or type")
        if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
            _refuse("scales must be float32")
        for t in (k, v, k_scale, v_scale):
            if t.device != k.device or not t.is_contiguous():
                _refuse("k, v and their scales must be contiguous and on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self._new_status()
        n_pages, n_layers, n_kv_heads, page_size, head_dim = k.shape
        self.n_pages, self.n_layers, self.n_kv_heads = n_pages, n_layers, n_kv_heads
        self.page_size, self.head_dim = page_size, head_dim
        self.block = page_size // k_scale.shape[3]
        self._c = Kv8Cache(k.device.index, formats[k.dtype], n_layers, n_kv_heads, head_dim,
                           page_size, self.block, n_pages, k.data_ptr(), v.data_ptr(),
                           k_scale.data_ptr(), v_scale.data_ptr(), self.status.data_ptr())
        self._dtypes = {torch.float32: MK_F32, torch.bfloat16: MK_BF16, torch.float16: MK_F16}
        self._workspaces = {}
        # the argument structures of a call, refilled by every call
        self._ref = ctypes.addressof(self._c)
        self._args = tuple(x() for x in (Rows, Rows, Batch))
        self._at = tuple(ctypes.addressof(x) for x in self._args)
        self._batch_args = self._args[2]
        # the library's own checks of the cache
        self._fill_batch(None, 1, 1, 1, 1, self.status.data_ptr(), self.status.data_ptr())
        _check(self._lib.mk_kv8_attention_workspace(self._ref, n_kv_heads, MK_BF16, self._at[2],
                                                    ctypes.byref(ctypes.c_int64())))

    @classmethod
    def empty(cls, n_pages, n_layers, n_kv_heads, head_dim, page_size=64, block=64, dtype=None,
              device="cuda"):
        """A cache on new tensors; dtype torch.int8 (default) or torch.float8_e4m3fn."""
        import torch
        if block < 1 or page_size % block:
            _refuse("page_size must be a multiple of block")
        shape = (n_pages, n_layers, n_kv_heads, page_size, head_dim)
        scales = shape[:3] + (page_size // block,)
        dtype = torch.int8 if dtype is None else dtype
        return cls(*(torch.empty(shape, dtype=dtype, device=device) for _ in range(2)),
                   *(torch.ones(scales, dtype=torch.float32, device=device) for _ in range(2)))

    def pools(self):
        """The tensors whose first dimension are pages, for PagePool."""
        return [self.k, self.v, self.k_scale, self.v_scale]

    def _rows(self, slot, x, n_heads, what):
        """Fills argument structure `slot` with the rows x; returns their number."""
        shape, stride = x.shape, x.stride()
        if len(shape) != 3 or (n_heads and shape[1] != n_heads) or shape[2] != self.head_dim \
                or (stride[2] != 1 and shape[0]):
            _refuse(f"{what} must be [rows][{n_heads or 'heads'}][{self.head_dim}] with contiguous "
                    "head_dim")
        dtype = self._dtypes.get(x.dtype)
        if dtype is None or x.get_device() != self._index:
            _refuse(f"{what} must be float32, bfloat16 or float16 on {self.device}")
        r = self._args[slot]
        r.data, r.dtype = x.data_ptr(), dtype
        # the stride of a single row or head is never used, and may be anything
        r.row_stride = stride[0] if shape[0] > 1 else 0
        r.head_stride = stride[1] if shape[1] > 1 else 0
        return shape[0]

    def _fill_batch(self, start, n_seqs, n_rows, max_rows, max_pages, kv_len, page_table):
        b = self._batch_args
        b.n_seqs, b.n_rows, b.max_rows, b.max_pages = n_seqs, n_rows, max_rows, max_pages
        b.d_row_start, b.d_kv_len, b.d_page_table = start, kv_len, page_table

    def _batch(self, page_table, kv_len, row_start, n_rows, max_rows):
        shape = page_table.shape
        if len(shape) != 2 or shape[1] < 1:
            _refuse("page_table must be [n_seqs][max_pages]")
        n, max_pages = shape
        if row_start is None:
            if n_rows != n:
                _refuse("without row_start there is one row per sequence")
            start = None
        else:
            start = self._int32(row_start, n + 1, "row_start")
        self._fill_batch(start, n, n_rows, max_rows, max_pages, self._int32(kv_len, n, "kv_len"),
                         self._int32(page_table, None, "page_table"))
        return n, max_pages

    def store(self, layer, k, v, page_table, kv_len, row_start=None, stream=None):
        """mk_kv8_store: quantise the new rows k, v [n_rows][n_kv_heads][head_dim] (float32,
        bfloat16 or float16) and append them to layer `layer`; rows row_start[s] to
        row_start[s + 1] - 1 (row s without row_start) go to the positions from kv_len[s]."""
        n_rows = self._rows(0, k, self.n_kv_heads, "k")
        if self._rows(1, v, self.n_kv_heads, "v") != n_rows or v.dtype is not k.dtype:
            _refuse("k and v differ in shape or type")
        self._batch(page_table, kv_len, row_start, n_rows, n_rows or 1)
        if n_rows:
            rk, rv, b = self._at
            rc = self._lib.mk_kv8_store(self._ref, layer, rk, rv, b, self._stream(stream))
            if rc:
                _check(rc)

    def attention(self, layer, q, page_table, kv_len, row_start=None, max_rows=None, scale=None,
                  out=None, return_lse=False, stream=None):
        """mk_kv8_attention: q [n_rows][n_q_heads][head_dim]; row i of sequence s sees the
        positions 0 to kv_len[s] + i.  max_rows bounds the rows of one sequence (1 without
        row_start; at most MK_KV8_MAX_ROWS).  Returns the output in q's type (in `out` if given,
        which must not overlap q), and with return_lse also the float32 log-sum-exp
        [n_rows][n_q_heads]."""
        if stream is not None:
            import torch
            now = torch.cuda.current_stream(self.device)
            with self._given(stream):
                got = self.attention(layer, q, page_table, kv_len, row_start, max_rows, scale, out,
                                     return_lse)
            # both streams may still use what is returned when the caller drops it
            for t in got if return_lse else (got,):
                t.record_stream(stream)
                t.record_stream(now)
            return got
        n_rows = self._rows(0, q, 0, "q")
        n_heads = q.shape[1]
        if max_rows is None:
            if row_start is not None:
                _refuse("max_rows is needed with row_start")
            max_rows = 1
        n, max_pages = self._batch(page_table, kv_len, row_start, n_rows, max_rows)
        if out is None:
            out = q.new_empty(n_rows, n_heads, self.head_dim)
        elif out.shape != q.shape or out.dtype != q.dtype or out.device != self.device \
                or not out.is_contiguous() or out.data_ptr() == q.data_ptr():
            _refuse("out must be contiguous, with the shape, type and device of q, and not q itself")
        lse = self._floats(n_rows, n_heads) if return_lse else None
        if n == n_rows == 0:
            return (out, lse) if return_lse else out
        rq, _, b = self._at
        # the workspace's size follows from the sizes alone
        key = (n_heads, q.dtype, n, max_rows, max_pages)
        size = self._workspaces.get(key)
        if size is None:
            bytes_ = ctypes.c_int64()
            _check(self._lib.mk_kv8_attention_workspace(self._ref, n_heads, self._args[0].dtype, b,
                                                        ctypes.byref(bytes_)))
            size = self._workspaces[key] = bytes_.value
        if n_rows:
            # a workspace of its own for every call: calls on other streams and
            # captured graphs do not meet in it
            ws = self._bytes(size) if size else None
            rc = self._lib.mk_kv8_attention(
                self._ref, layer, rq, n_heads, self.head_dim ** -0.5 if scale is None else scale,
                out.data_ptr(), lse.data_ptr() if return_lse else None, b,
                ws.data_ptr() if size else None, size, self._stream(None))
            if rc:
                _check(rc)
        return (out, lse) if return_lse else out


class PagePool(_Status):
    """The pages of a cache and who holds them, on the caller's tensors:

    page_table  int32 [n_seqs][max_pages], -1 = no page
    ref_count   int32 [n_pages], page table entries that name the page
    pools       tensors whose first dimension are the pages: the K and V pools of
                Megakernel.decode_steps_paged, or KV8Cache.pools()

    Calls are asynchronous and take a stream as KV8Cache's do; use one object per thread."""

    def __init__(self, page_table, ref_count, page_size, pools):
        self._bind(page_table.device)
        if page_table.dim() != 2 or ref_count.dim() != 1:
            _refuse("page_table must be [n_seqs][max_pages] and ref_count [n_pages]")
        if len(pools) > MK_MAX_POOLS:
            _refuse(f"more than {MK_MAX_POOLS} pools")
        self.page_table, self.ref_count, self.page_size = page_table, ref_count, page_size
        self.pools = list(pools)
        self._new_status()
        n_pages = ref_count.numel()
        if n_pages < 1:
            _refuse("ref_count must have an entry for every page")
        p = self._c = Pages(page_table.device.index, n_pages, page_table.shape[0],
                            page_table.shape[1], page_size, len(pools))
        for i, x in enumerate(self.pools):
            if x.dim() < 1 or x.shape[0] != n_pages or x.device != self.device \
                    or not x.is_contiguous():
                _refuse(f"pool {i} must be contiguous, on {self.device}, with {n_pages} pages")
            p.d_pool[i] = x.data_ptr()
            p.page_bytes[i] = x.numel() // n_pages * x.element_size()
        p.d_page_table = self._int32(page_table, None, "page_table")
        p.d_ref = self._int32(ref_count, None, "ref_count")
        p.d_status = self.status.data_ptr()
        self._ref = ctypes.addressof(p)
        self._sizes = {}
        self._workspace(0)

    @classmethod
    def empty(cls, n_seqs, max_pages, page_size, pools):
        """Nobody holds a page yet."""
        import torch
        if not len(pools):
            _refuse("no pools")
        device = pools[0].device
        return cls(torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(pools[0].shape[0], dtype=torch.int32, device=device), page_size,
                   pools)

    def _workspace(self, n):
        size = self._sizes.get(n)
        if size is None:
            b = ctypes.c_int64()
            _check(self._lib.mk_pages_workspace(self._ref, n, ctypes.byref(b)))
            size = self._sizes[n] = b.value
        return size

    def _call(self, fn, n, args, stream):
        if stream is not None:
            with self._given(stream):
                return self._call(fn, n, args, None)
        size = self._workspace(n)
        ws = self._bytes(size)
        rc = fn(self._ref, *args, ws.data_ptr(), size, self._stream(None))
        if rc:
            _check(rc)

    def fork(self, src, dst, stream=None):
        """mk_pages_fork: sequences dst take (and share) the pages of sequences src."""
        n = src.numel()
        self._call(self._lib.mk_pages_fork, n, (n, self._int32(src, None, "src"),
                                                self._int32(dst, n, "dst")), stream)

    def free(self, seqs, stream=None):
        """mk_pages_free: the sequences give their pages back."""
        n = seqs.numel()
        self._call(self._lib.mk_pages_free, n, (n, self._int32(seqs, None, "seqs")), stream)

    def reserve(self, kv_len, n_new, stream=None):
        """mk_pages_reserve: pages that only their sequence holds under the positions kv_len[s]
        to kv_len[s] + n_new[s] - 1 of every sequence."""
        n = self._c.n_seqs
        self._call(self._lib.mk_pages_reserve, 0, (self._int32(kv_len, n, "kv_len"),
                                                   self._int32(n_new, n, "n_new")), stream)

    def compact(self, stream=None):
        """mk_pages_compact: the pages in use move to the lowest page numbers."""
        self._call(self._lib.mk_pages_compact, 0, (), stream)

    def copy(self, src, dst, stream=None):
        """mk_pages_copy: pages dst of every pool take the contents of pages src."""
        n = src.numel()
        self._call(self._lib.mk_pages_copy, n, (n, self._int32(src, None, "src"),
                                                self._int32(dst, n, "dst")), stream)
