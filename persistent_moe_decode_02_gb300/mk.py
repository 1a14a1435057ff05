"""Thin ctypes binding of libmk.so (include/mk.h): argument marshalling only.

Every step of the decode path runs inside the library's CUDA kernel; this
module never computes any of it.  It fails loudly when libmk.so is missing
(build it with ``persistent_moe_decode_02_gb300.build.build()``)."""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmk.so")

MK_OK, MK_ERR_INVALID, MK_ERR_CUDA, MK_ERR_DEP_TIMEOUT, MK_ERR_CAPACITY, MK_ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5
MK_DBG_HIDDEN, MK_DBG_EXPERT_IDS, MK_DBG_GATES, MK_DBG_ROUTER_LOGITS, MK_DBG_SEQ_LENS, MK_DBG_UNION = 1, 2, 3, 4, 5, 6
MK_DBG_TASKS, MK_DBG_TRACE, MK_DBG_STAGE_TRACE = 7, 8, 9
TRACE_SLOTS = ["fetch", "dep", "act", "stages", "done", "p_first", "p_last", "p_start", "s_first", "s_last",
               "mid1", "mid2"]

EXPORTS = [
    "mk_plan_create", "mk_decode_step", "mk_decode_steps", "mk_decode_step_host", "mk_plan_update", "mk_plan_sync",
    "mk_plan_read_debug", "mk_plan_info", "mk_plan_destroy", "mk_status_string", "mk_plan_inspect",
    "mk_last_error", "mk_decode_step_noalloc", "mk_plan_set_sampling", "mk_plan_set_top_p", "mk_sched_create", "mk_sched_submit", "mk_sched_next",
    "mk_sched_commit", "mk_sched_abandon", "mk_sched_result", "mk_sched_forget", "mk_sched_stats",
    "mk_sched_destroy", "mk_serve_step", "mk_sched_next_rows", "mk_sched_set_prefill", "mk_plan_update_rows",
    "mk_sched_peek_rows", "mk_chunk_create", "mk_chunk_update", "mk_chunk_append", "mk_chunk_attend", "mk_chunk_read",
    "mk_chunk_sync", "mk_chunk_info", "mk_chunk_destroy", "mk_chunk_inspect", "mk_probs", "mk_verify", "mk_norm",
    "mk_quantize", "mk_route", "mk_experts_create", "mk_experts_up", "mk_experts_down", "mk_experts_sync",
    "mk_experts_set_debug", "mk_experts_destroy",
]
MK_KV_BF16, MK_KV_E4M3 = 0, 1
MK_ROWS_BF16, MK_ROWS_F32, MK_ROWS_E4M3 = 0, 1, 2


class MkModelDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("n_layers", "hidden", "n_q_heads", "n_kv_heads", "head_dim",
                                            "n_experts", "top_k", "expert_ffn", "vocab", "page_size")] + \
               [("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float)]


_PP = ctypes.POINTER(ctypes.c_void_p)


class MkWeights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p), ("lm_head", ctypes.c_void_p),
                ("attn_norm", _PP), ("wqkv", _PP), ("wo", _PP), ("ffn_norm", _PP), ("router", _PP),
                ("w_gate_up", _PP), ("w_down", _PP)]


class MkKv(ctypes.Structure):
    _fields_ = [("kv_pool", _PP), ("num_pages", ctypes.c_int)]


class MkPlanOpts(ctypes.Structure):
    _fields_ = [("timeout_us", ctypes.c_int), ("num_ctas", ctypes.c_int), ("max_batch", ctypes.c_int),
                ("split_pages", ctypes.c_int), ("debug_drop_task", ctypes.c_int), ("trace", ctypes.c_int),
                ("temperature", ctypes.c_float), ("seed", ctypes.c_ulonglong), ("top_p", ctypes.c_float),
                ("chunk_first", ctypes.POINTER(ctypes.c_int)), ("tc_off", ctypes.c_int)]


class MkError(RuntimeError):
    def __init__(self, fn: str, code: int):
        detail = lib().mk_last_error().decode()
        super().__init__(f"{fn} failed: {code} ({status_string(code)})" + (f": {detail}" if detail else ""))
        self.code = code


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it first "
                              "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, p_int = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_int)
        L.mk_plan_create.argtypes = [ctypes.POINTER(MkModelDims), ctypes.POINTER(MkWeights), ctypes.POINTER(MkKv),
                                     i32, p_int, p_int, i32, ctypes.POINTER(MkPlanOpts), ctypes.POINTER(vp)]
        L.mk_decode_step.argtypes = [vp, vp, vp, vp, vp]
        L.mk_decode_steps.argtypes = [vp, vp, i32, vp, vp, vp]
        L.mk_decode_step_host.argtypes = [vp, p_int, ctypes.POINTER(ctypes.c_float), p_int, vp]
        L.mk_plan_update.argtypes = [vp, i32, p_int, p_int, i32, vp]
        L.mk_plan_sync.argtypes = [vp, vp]
        L.mk_plan_read_debug.argtypes = [vp, i32, vp, ctypes.c_size_t, vp]
        L.mk_plan_info.argtypes = [vp, p_int, i32]
        L.mk_plan_destroy.argtypes = [vp]
        L.mk_plan_destroy.restype = None
        L.mk_status_string.argtypes = [i32]
        L.mk_status_string.restype = ctypes.c_char_p
        L.mk_last_error.argtypes = []
        L.mk_last_error.restype = ctypes.c_char_p
        L.mk_plan_inspect.argtypes = [ctypes.POINTER(MkModelDims), i32, p_int, i32, i32, p_int, i32, p_int]
        L.mk_decode_step_noalloc.argtypes = [ctypes.POINTER(MkModelDims), ctypes.POINTER(MkWeights),
                                             ctypes.POINTER(MkKv), i32, p_int, p_int, i32, vp, vp, vp, vp, vp]
        i64, p_i64 = ctypes.c_longlong, ctypes.POINTER(ctypes.c_longlong)
        L.mk_plan_set_sampling.argtypes = [vp, ctypes.c_float, ctypes.c_ulonglong]
        L.mk_plan_set_top_p.argtypes = [vp, ctypes.c_float]
        L.mk_sched_create.argtypes = [i32, i32, i32, i32, ctypes.POINTER(vp)]
        L.mk_sched_submit.argtypes = [vp, i64, p_int, i32, i32, i32]
        L.mk_sched_next.argtypes = [vp, p_int, p_int, p_int, p_int, p_i64, p_int]
        L.mk_sched_next_rows.argtypes = [vp, p_int, p_int, p_int, p_int, p_i64, p_int, p_int]
        L.mk_sched_set_prefill.argtypes = [vp, i32]
        L.mk_sched_peek_rows.argtypes = [vp, p_int, p_int, p_int, p_int, p_i64, p_int]
        L.mk_plan_update_rows.argtypes = [vp, i32, p_int, p_int, i32, p_int, vp]
        L.mk_sched_commit.argtypes = [vp, p_int]
        L.mk_sched_abandon.argtypes = [vp]
        L.mk_sched_result.argtypes = [vp, i64, p_int, i32, p_int, p_int]
        L.mk_sched_forget.argtypes = [vp, i64]
        L.mk_sched_stats.argtypes = [vp, p_int, i32]
        L.mk_sched_destroy.argtypes = [vp]
        L.mk_sched_destroy.restype = None
        L.mk_serve_step.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(MkModelDims), ctypes.POINTER(MkWeights),
                                    ctypes.POINTER(MkKv), ctypes.POINTER(MkPlanOpts), vp]
        L.mk_chunk_create.argtypes = [ctypes.POINTER(MkModelDims), i32, i32, i32, p_int, p_int, p_int, i32,
                                      ctypes.POINTER(vp)]
        L.mk_chunk_update.argtypes = [vp, i32, p_int, p_int, p_int, i32, vp]
        L.mk_chunk_append.argtypes = [vp, vp, i32, i64, vp, vp, vp]
        L.mk_chunk_attend.argtypes = [vp, vp, vp, vp, vp]
        L.mk_chunk_read.argtypes = [vp, vp, vp, vp]
        L.mk_chunk_sync.argtypes = [vp, vp]
        L.mk_chunk_info.argtypes = [vp, p_int, i32]
        L.mk_chunk_destroy.argtypes = [vp]
        L.mk_chunk_destroy.restype = None
        L.mk_chunk_inspect.argtypes = [ctypes.POINTER(MkModelDims), i32, p_int, p_int, i32, p_int, i32]
        L.mk_probs.argtypes = [vp, i32, i32, i64, ctypes.c_float, vp, vp]
        L.mk_verify.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.mk_norm.argtypes = [i32, i32, vp, i32, i64, vp, i32, i32, vp, ctypes.c_float, vp, vp, i32, vp, vp]
        L.mk_quantize.argtypes = [i32, i32, vp, i32, i64, vp, vp, vp]
        L.mk_route.argtypes = [i32, i32, i32, vp, i64, vp, vp, vp, vp, vp]
        L.mk_experts_create.argtypes = [ctypes.POINTER(MkModelDims), i32, ctypes.POINTER(vp)]
        L.mk_experts_up.argtypes = [vp, i32] + [vp] * 9
        L.mk_experts_down.argtypes = [vp, i32] + [vp] * 9
        L.mk_experts_sync.argtypes = [vp, vp]
        L.mk_experts_set_debug.argtypes = [vp, i32, i32]
        L.mk_experts_destroy.argtypes = [vp]
        L.mk_experts_destroy.restype = None
        for f in ("mk_plan_create", "mk_decode_step", "mk_decode_steps", "mk_decode_step_host", "mk_plan_update", "mk_plan_sync",
                  "mk_plan_read_debug", "mk_plan_info", "mk_plan_inspect", "mk_decode_step_noalloc",
                  "mk_plan_set_sampling", "mk_plan_set_top_p", "mk_sched_create", "mk_sched_submit", "mk_sched_next", "mk_sched_commit", "mk_sched_abandon",
                  "mk_sched_result", "mk_sched_forget", "mk_sched_stats", "mk_serve_step", "mk_sched_next_rows",
                  "mk_sched_set_prefill", "mk_plan_update_rows", "mk_sched_peek_rows", "mk_chunk_create",
                  "mk_chunk_update", "mk_chunk_append", "mk_chunk_attend", "mk_chunk_read", "mk_chunk_sync",
                  "mk_chunk_info", "mk_chunk_inspect", "mk_probs", "mk_verify", "mk_norm", "mk_quantize", "mk_route",
                  "mk_experts_create", "mk_experts_up", "mk_experts_down", "mk_experts_sync", "mk_experts_set_debug"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().mk_status_string(code).decode()


def dims_struct(D) -> MkModelDims:
    return MkModelDims(D.n_layers, D.hidden, D.n_q_heads, D.n_kv_heads, D.head_dim, D.n_experts, D.top_k,
                       D.expert_ffn, D.vocab, D.page_size, D.rms_eps, D.rope_theta)


def _int_array(vals: Sequence[int]):
    return (ctypes.c_int * len(vals))(*[int(v) for v in vals])


def _ptr_array(tensors):
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def inspect_tasks(D, seq_lens: Sequence[int], num_ctas: int, split_pages: int = 0):
    """Host-only task list: returns (tasks [n, 12] int tensor, cta_start list)."""
    dims = dims_struct(D)
    sl = _int_array(seq_lens)
    n = lib().mk_plan_inspect(ctypes.byref(dims), len(seq_lens), sl, num_ctas, split_pages, None, 0, None)
    if n < 0:
        raise MkError("mk_plan_inspect", n)
    buf = (ctypes.c_int * (12 * n))()
    cs = (ctypes.c_int * (num_ctas + 1))()
    n2 = lib().mk_plan_inspect(ctypes.byref(dims), len(seq_lens), sl, num_ctas, split_pages, buf, n, cs)
    assert n2 == n
    return torch.tensor(list(buf), dtype=torch.int64).view(n, 12), list(cs)


def _weight_structs(D, weights: dict, kv_pools):
    """ctypes views of the weight and KV pointers (the arrays must outlive the call)."""
    arrays = {k: _ptr_array(weights[k]) for k in
              ("attn_norm", "wqkv", "wo", "ffn_norm", "router", "w_gate_up", "w_down")}
    kvp = _ptr_array(kv_pools)
    cast = lambda a: ctypes.cast(a, _PP)
    w = MkWeights(weights["embed"].data_ptr(), weights["final_norm"].data_ptr(), weights["lm_head"].data_ptr(),
                  *[cast(arrays[k]) for k in ("attn_norm", "wqkv", "wo", "ffn_norm", "router", "w_gate_up",
                                              "w_down")])
    kv = MkKv(cast(kvp), int(kv_pools[0].shape[0]))
    return w, kv, (arrays, kvp)


def decode_step_noalloc(D, weights: dict, kv_pools, seq_lens: Sequence[int], page_table, max_pages: int,
                        tokens: torch.Tensor, next_token: torch.Tensor, logits: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, stream=None) -> int:
    """One step through mk_decode_step_noalloc (no plan, no allocation inside
    the library).  Returns the enqueue status; the device status goes to
    `status` (int32[4] on the device) when given."""
    w, kv, keep = _weight_structs(D, weights, kv_pools)
    dims = dims_struct(D)
    ptr = lambda t: ctypes.c_void_p(t.data_ptr() if t is not None else 0)
    pt = [int(x) for x in page_table]
    rc = lib().mk_decode_step_noalloc(ctypes.byref(dims), ctypes.byref(w), ctypes.byref(kv), len(seq_lens),
                                      _int_array(seq_lens), _int_array(pt), max_pages, ptr(tokens), ptr(logits),
                                      ptr(next_token), ptr(status), _stream(stream))
    del keep
    return rc


class Plan:
    """Owns an mk_plan.  Weight/KV tensors are referenced, not copied.

    weights: dict with 'embed', 'final_norm', 'lm_head' tensors and per-layer
    lists 'attn_norm', 'wqkv', 'wo', 'ffn_norm', 'router', 'w_gate_up',
    'w_down' (bf16 CUDA tensors in the layout of include/mk.h).
    kv_pools: per-layer bf16 [num_pages, nkv, 2, head_dim, page_size] (per page
    and KV head the K block, then the V block, each stored transposed, slot
    fastest)."""

    def __init__(self, D, weights: dict, kv_pools, seq_lens: Sequence[int], page_table,
                 max_pages: int, timeout_us: int = 0, num_ctas: int = 0, max_batch: int = 0,
                 split_pages: int = 0, debug_drop_task: int = 0, trace: int = 0, tc_off: bool = False):
        self.D = D
        self._keep = (weights, kv_pools)
        self._arrays = {k: _ptr_array(weights[k]) for k in
                        ("attn_norm", "wqkv", "wo", "ffn_norm", "router", "w_gate_up", "w_down")}
        self._kvp = _ptr_array(kv_pools)
        cast = lambda a: ctypes.cast(a, _PP)
        self._w = MkWeights(weights["embed"].data_ptr(), weights["final_norm"].data_ptr(),
                            weights["lm_head"].data_ptr(), *[cast(self._arrays[k]) for k in
                                                             ("attn_norm", "wqkv", "wo", "ffn_norm", "router",
                                                              "w_gate_up", "w_down")])
        self._kv = MkKv(cast(self._kvp), int(kv_pools[0].shape[0]))
        self._dims = dims_struct(D)
        opts = MkPlanOpts(timeout_us, num_ctas, max_batch, split_pages, debug_drop_task, int(trace))
        opts.tc_off = int(bool(tc_off))
        self.batch = len(seq_lens)
        pt = [int(x) for x in page_table]
        h = ctypes.c_void_p()
        rc = lib().mk_plan_create(ctypes.byref(self._dims), ctypes.byref(self._w), ctypes.byref(self._kv),
                                  self.batch, _int_array(seq_lens), _int_array(pt), max_pages,
                                  ctypes.byref(opts), ctypes.byref(h))
        if rc != MK_OK:
            raise MkError("mk_plan_create", rc)
        self.h = h

    def step(self, tokens: torch.Tensor, next_token: torch.Tensor, logits: Optional[torch.Tensor] = None,
             stream=None) -> int:
        """Enqueue one decode step (device buffers).  Returns the status code."""
        return lib().mk_decode_step(self.h, ctypes.c_void_p(tokens.data_ptr()),
                                    ctypes.c_void_p(logits.data_ptr() if logits is not None else 0),
                                    ctypes.c_void_p(next_token.data_ptr()), _stream(stream))

    def steps(self, tokens: torch.Tensor, n_steps: int, next_tokens: torch.Tensor,
              logits: Optional[torch.Tensor] = None, stream=None) -> int:
        """Enqueue n_steps decode steps in one launch (device buffers):
        next_tokens int32 [n_steps, batch], logits float32 [n_steps, batch,
        vocab] or None.  Returns the status code."""
        return lib().mk_decode_steps(self.h, ctypes.c_void_p(tokens.data_ptr()), int(n_steps),
                                     ctypes.c_void_p(logits.data_ptr() if logits is not None else 0),
                                     ctypes.c_void_p(next_tokens.data_ptr()), _stream(stream))

    def step_host(self, tokens, next_token, logits=None, stream=None) -> int:
        """One step with host buffers (int32 / float32 CPU tensors, contiguous)."""
        tp = ctypes.cast(tokens.data_ptr(), ctypes.POINTER(ctypes.c_int))
        np_ = ctypes.cast(next_token.data_ptr(), ctypes.POINTER(ctypes.c_int))
        lp = ctypes.cast(logits.data_ptr(), ctypes.POINTER(ctypes.c_float)) if logits is not None else None
        return lib().mk_decode_step_host(self.h, tp, lp, np_, _stream(stream))

    def update_rows(self, seq_lens: Sequence[int], page_table, max_pages: int, chunk_first: Sequence[int],
                    stream=None) -> None:
        """Replace the batch with rows of which some are prefill chunks (include/mk.h)."""
        self.batch = len(seq_lens)
        pt = [int(x) for x in page_table]
        rc = lib().mk_plan_update_rows(self.h, self.batch, _int_array(seq_lens), _int_array(pt), max_pages,
                                       _int_array(chunk_first), _stream(stream))
        if rc != MK_OK:
            raise MkError("mk_plan_update_rows", rc)

    def update(self, seq_lens: Sequence[int], page_table, max_pages: int, stream=None) -> None:
        # int32 host arrays handed over by pointer (a numpy array or CPU tensor is not copied)
        sl = np.ascontiguousarray(np.asarray(seq_lens), dtype=np.int32)
        pt = np.ascontiguousarray(np.asarray(page_table), dtype=np.int32)
        p_int = ctypes.POINTER(ctypes.c_int)
        rc = lib().mk_plan_update(self.h, len(sl), sl.ctypes.data_as(p_int), pt.ctypes.data_as(p_int), max_pages,
                                  _stream(stream))
        if rc != MK_OK:
            raise MkError("mk_plan_update", rc)
        self.batch = len(seq_lens)

    def sync(self, stream=None) -> int:
        return lib().mk_plan_sync(self.h, _stream(stream))

    def set_sampling(self, temperature: float, seed: int = 0) -> None:
        """Temperature sampling for the following steps (0: greedy); see include/mk.h."""
        rc = lib().mk_plan_set_sampling(self.h, float(temperature), int(seed) & (2 ** 64 - 1))
        if rc != MK_OK:
            raise MkError("mk_plan_set_sampling", rc)

    def set_top_p(self, top_p: float) -> None:
        """Nucleus sampling (0 < top_p < 1) for the following sampled steps; 1: off."""
        rc = lib().mk_plan_set_top_p(self.h, float(top_p))
        if rc != MK_OK:
            raise MkError("mk_plan_set_top_p", rc)

    def read_debug(self, what: int, out: torch.Tensor, stream=None) -> torch.Tensor:
        rc = lib().mk_plan_read_debug(self.h, what, ctypes.c_void_p(out.data_ptr()),
                                      out.numel() * out.element_size(), _stream(stream))
        if rc != MK_OK:
            raise MkError("mk_plan_read_debug", rc)
        return out

    def timeline(self, stream=None):
        """(tasks int32 [n, 12], stamps int64 [n, 10]) of the last step (needs trace=True)."""
        n = self.info()["num_tasks"]
        tasks = torch.empty(n, 12, dtype=torch.int32)
        self.read_debug(MK_DBG_TASKS, tasks, stream)
        stamps = torch.empty(n, len(TRACE_SLOTS), dtype=torch.int64)
        self.read_debug(MK_DBG_TRACE, stamps, stream)
        self.sync(stream)
        return tasks, stamps

    def stage_timeline(self, stream=None) -> torch.Tensor:
        """int64 [num_ctas, 4096, 6] of the last step: per CTA and ring stage, the
        copy issue, landing and release stamps (ns, 0 = none), the task index, and
        the SM clock at landing and release (needs trace=2)."""
        out = torch.empty(self.info()["num_ctas"], 4096, 6, dtype=torch.int64)
        self.read_debug(MK_DBG_STAGE_TRACE, out, stream)
        self.sync(stream)
        return out

    def info(self) -> dict:
        buf = (ctypes.c_int * 12)()
        lib().mk_plan_info(self.h, buf, 12)
        keys = ["num_ctas", "num_tasks", "nstages", "stage_bytes", "smem_bytes", "batch", "attn_tasks",
                "gu_tasks", "lm_tiles", "replans", "tc_gate_up", "tc_proj"]
        return dict(zip(keys, list(buf)))

    def close(self):
        if getattr(self, "h", None):
            lib().mk_plan_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Scheduler:
    """Owns an mk_sched: the host-side request queue, batch and KV page
    allocator of continuous batching (include/mk.h describes the policy)."""

    def __init__(self, num_pages: int, page_size: int, max_batch: int, max_pages: int):
        h = ctypes.c_void_p()
        rc = lib().mk_sched_create(num_pages, page_size, max_batch, max_pages, ctypes.byref(h))
        if rc != MK_OK:
            raise MkError("mk_sched_create", rc)
        self.h, self.max_batch, self.max_pages = h, max_batch, max_pages

    def submit(self, rid: int, prompt: Sequence[int], max_new_tokens: int, eos_token: int = -1) -> None:
        rc = lib().mk_sched_submit(self.h, rid, _int_array(prompt), len(prompt), max_new_tokens, eos_token)
        if rc != MK_OK:
            raise MkError("mk_sched_submit", rc)

    def set_prefill(self, max_chunk: int) -> None:
        """Prompt tokens a request may feed per step as consecutive rows (1: one token per step)."""
        rc = lib().mk_sched_set_prefill(self.h, int(max_chunk))
        if rc != MK_OK:
            raise MkError("mk_sched_set_prefill", rc)

    def next(self):
        """The next batch's rows as a dict (seq_lens, page_table, tokens, rids,
        chunk_first, changed), or None when idle."""
        cap, mp = self.max_batch, self.max_pages
        b, ch = ctypes.c_int(), ctypes.c_int()
        sl, pt, tk = (ctypes.c_int * cap)(), (ctypes.c_int * (cap * mp))(), (ctypes.c_int * cap)()
        rids, cf = (ctypes.c_longlong * cap)(), (ctypes.c_int * cap)()
        rc = lib().mk_sched_next_rows(self.h, ctypes.byref(b), sl, pt, tk, rids, cf, ctypes.byref(ch))
        if rc != MK_OK:
            raise MkError("mk_sched_next_rows", rc)
        n = b.value
        if n == 0:
            return None
        return {"seq_lens": list(sl[:n]), "page_table": list(pt[:n * mp]), "tokens": list(tk[:n]),
                "rids": list(rids[:n]), "chunk_first": list(cf[:n]), "changed": bool(ch.value)}

    def peek(self):
        """The rows next() would return after the pending batch committed with no end token, or None."""
        cap, mp = self.max_batch, self.max_pages
        b = ctypes.c_int()
        sl, pt, tk = (ctypes.c_int * cap)(), (ctypes.c_int * (cap * mp))(), (ctypes.c_int * cap)()
        rids, cf = (ctypes.c_longlong * cap)(), (ctypes.c_int * cap)()
        rc = lib().mk_sched_peek_rows(self.h, ctypes.byref(b), sl, pt, tk, rids, cf)
        if rc != MK_OK:
            raise MkError("mk_sched_peek_rows", rc)
        n = b.value
        if n == 0:
            return None
        return {"seq_lens": list(sl[:n]), "page_table": list(pt[:n * mp]), "tokens": list(tk[:n]),
                "rids": list(rids[:n]), "chunk_first": list(cf[:n])}

    def commit(self, next_tokens: Sequence[int]) -> None:
        rc = lib().mk_sched_commit(self.h, _int_array(next_tokens))
        if rc != MK_OK:
            raise MkError("mk_sched_commit", rc)

    def abandon(self) -> None:
        rc = lib().mk_sched_abandon(self.h)
        if rc != MK_OK:
            raise MkError("mk_sched_abandon", rc)

    def result(self, rid: int):
        """(output tokens, done) of request rid."""
        n, d = ctypes.c_int(), ctypes.c_int()
        rc = lib().mk_sched_result(self.h, rid, None, 0, ctypes.byref(n), ctypes.byref(d))
        if rc != MK_OK:
            raise MkError("mk_sched_result", rc)
        buf = (ctypes.c_int * max(1, n.value))()
        rc = lib().mk_sched_result(self.h, rid, buf, n.value, ctypes.byref(n), ctypes.byref(d))
        if rc != MK_OK:
            raise MkError("mk_sched_result", rc)
        return list(buf[:n.value]), bool(d.value)

    def forget(self, rid: int) -> None:
        rc = lib().mk_sched_forget(self.h, rid)
        if rc != MK_OK:
            raise MkError("mk_sched_forget", rc)

    def stats(self) -> dict:
        buf = (ctypes.c_int * 5)()
        lib().mk_sched_stats(self.h, buf, 5)
        return dict(zip(["queued", "active", "retired", "free_pages", "steps"], list(buf)))

    def close(self):
        if getattr(self, "h", None):
            lib().mk_sched_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Server:
    """The serving loop: a Scheduler plus the plan it drives (created by the
    first mk_serve_step).  kv_pools: the KV pool the scheduler's pages index
    (every page of it is the scheduler's)."""

    def __init__(self, D, weights: dict, kv_pools, max_batch: int, max_pages: int, timeout_us: int = 0,
                 num_ctas: int = 0, split_pages: int = 0, temperature: float = 0.0, seed: int = 0,
                 prefill: int = 8):
        self.D = D
        self._keep = (weights, kv_pools)
        self._w, self._kv, self._arrays = _weight_structs(D, weights, kv_pools)
        self._dims = dims_struct(D)
        self._opts = MkPlanOpts(timeout_us, num_ctas, max_batch, split_pages, 0, 0, float(temperature),
                                int(seed) & (2 ** 64 - 1))
        self.sched = Scheduler(int(kv_pools[0].shape[0]), D.page_size, max_batch, max_pages)
        if prefill > 1:   # prompts enter the cache in chunks of up to `prefill` tokens per step
            self.sched.set_prefill(min(prefill, 8))
        self.plan = ctypes.c_void_p()

    def submit(self, rid: int, prompt: Sequence[int], max_new_tokens: int, eos_token: int = -1) -> None:
        self.sched.submit(rid, prompt, max_new_tokens, eos_token)

    def step(self, stream=None) -> int:
        """One serving step; returns the batch size that ran (0: idle)."""
        rc = lib().mk_serve_step(self.sched.h, ctypes.byref(self.plan), ctypes.byref(self._dims),
                                 ctypes.byref(self._w), ctypes.byref(self._kv), ctypes.byref(self._opts),
                                 _stream(stream))
        if rc < 0:
            raise MkError("mk_serve_step", rc)
        return rc

    def run(self, max_steps: int = 1 << 30, stream=None) -> int:
        """Step until nothing is queued or admitted (or max_steps); returns the steps run."""
        n = 0
        while n < max_steps and self.step(stream) > 0:
            n += 1
        return n

    def result(self, rid: int):
        return self.sched.result(rid)

    def close(self):
        if getattr(self, "plan", None) and self.plan.value:
            lib().mk_plan_destroy(self.plan)
            self.plan = ctypes.c_void_p()
        if getattr(self, "sched", None) is not None:
            self.sched.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _here(name: str, t: torch.Tensor, dtype, shape, dev: int) -> int:
    """The address of a contiguous tensor of the current device, checked."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != dev:
        raise ValueError(f"{name}: a tensor of the current CUDA device is wanted, got {t.device}")
    raise ValueError(f"{name}: {t.dtype} of {tuple(t.shape)}{'' if t.is_contiguous() else ', not contiguous'}; wanted "
                     f"contiguous {dtype} of {tuple(shape)}")


# These calls take microseconds, so the current device and stream are asked for without the objects around them.
def _device() -> int:
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else torch.cuda.current_device()


def _on(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _chunk_dims(D) -> MkModelDims:
    return MkModelDims(n_q_heads=D.n_q_heads, n_kv_heads=D.n_kv_heads, head_dim=D.head_dim, page_size=D.page_size,
                       rope_theta=D.rope_theta)


_BF16, _U8, _F32, _I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


class Chunk:
    """Owns an mk_chunk: the operators over a chunk of new tokens of each
    request (include/mk.h) - append to the paged cache, causal attention over
    it, and reading it back.

    D: dims with n_q_heads, n_kv_heads, head_dim, page_size and rope_theta (0:
    no rotation).  kv_type: "bf16" (pools as Plan's: bf16 [num_pages, nkv, 2,
    head_dim, page_size]) or "e4m3" (uint8 [num_pages, nkv, 2, head_dim + 1,
    page_size]: codes, then the slots' scale exponents + 127)."""

    def __init__(self, D, kv_type: str, num_pages: int, seq_lens: Sequence[int], new_lens: Sequence[int], page_table,
                 max_pages: int):
        kinds = {"bf16": MK_KV_BF16, "e4m3": MK_KV_E4M3}
        if kv_type not in kinds:
            raise ValueError(f"kv_type: {kv_type!r}, wanted one of {tuple(kinds)}")
        self._dims = _chunk_dims(D)
        self.kv_type, self.num_pages = kv_type, int(num_pages)
        self.nq, self.nkv, self.d = D.n_q_heads, D.n_kv_heads, D.head_dim
        h = ctypes.c_void_p()
        rc = lib().mk_chunk_create(ctypes.byref(self._dims), kinds[kv_type], num_pages,
                                   *self._batch(seq_lens, new_lens, page_table, max_pages), ctypes.byref(h))
        if rc != MK_OK:
            raise MkError("mk_chunk_create", rc)
        self.h = h
        self._lens(seq_lens, new_lens)
        self._pool = torch.Size((self.num_pages, self.nkv, 2, self.d + (kv_type == "e4m3"), D.page_size))
        self._pool_type = _U8 if kv_type == "e4m3" else _BF16

    def _batch(self, seq_lens, new_lens, page_table, max_pages):
        def ints(x):
            x = np.asarray(x)
            if x.size and (x.dtype.kind not in "iu" or x.min() < -2 ** 31 or x.max() >= 2 ** 31):
                raise ValueError("seq_lens, new_lens and page_table hold 32-bit integers")
            return np.ascontiguousarray(x, dtype=np.int32)

        sl, nl, pt = ints(seq_lens), ints(new_lens), ints(page_table)
        if sl.ndim != 1 or nl.shape != sl.shape or pt.size != len(sl) * max_pages:
            raise ValueError("seq_lens, new_lens and page_table do not describe one batch")
        p_int = ctypes.POINTER(ctypes.c_int)
        self._host = (sl, nl, pt)    # outlive the call
        return (len(sl), sl.ctypes.data_as(p_int), nl.ctypes.data_as(p_int), pt.ctypes.data_as(p_int), int(max_pages))

    def _lens(self, seq_lens, new_lens):
        self.rows = int(sum(int(x) for x in new_lens))
        self.tokens = self.rows + int(sum(int(x) for x in seq_lens))
        self._q = torch.Size((self.rows, self.nq, self.d))
        self._kv = torch.Size((self.tokens, self.nkv, 2, self.d))

    def update(self, seq_lens: Sequence[int], new_lens: Sequence[int], page_table, max_pages: int, stream=None) -> None:
        """Another batch for this chunk (uploaded on the stream)."""
        rc = lib().mk_chunk_update(self.h, *self._batch(seq_lens, new_lens, page_table, max_pages), _stream(stream))
        if rc != MK_OK:
            raise MkError("mk_chunk_update", rc)
        self._lens(seq_lens, new_lens)

    def append(self, qkv: torch.Tensor, kv_pool: torch.Tensor, q: Optional[torch.Tensor] = None, stream=None) -> None:
        """Rotate and append the rows qkv [rows, nkv, G + 2, head_dim] (or [rows, nkv * (G + 2) * head_dim]; bf16 or
        float32, rows may lie apart) to one layer's pool; the rotated queries to q [rows, nq, head_dim] (bf16)."""
        width, n = (self.nq + 2 * self.nkv) * self.d, 1
        shape, steps = qkv.shape, qkv.stride()
        fits = len(shape) > 1 and shape[0] == self.rows
        for i in range(len(shape) - 1, 0, -1):     # what follows the first dimension is one contiguous row
            fits = fits and (steps[i] == n or shape[i] == 1)
            n *= shape[i]
        if not fits or n != width:
            raise ValueError(f"qkv: shape {tuple(shape)}, wanted {self.rows} contiguous rows of {width}")
        dev = _device()
        if qkv.get_device() != dev or qkv.dtype not in (_BF16, _F32):
            raise ValueError(f"qkv: a bf16 or float32 tensor of the current CUDA device is wanted, got {qkv.dtype} on "
                             f"{qkv.device}")
        if (q is None) != (self.nq == 0):
            raise ValueError("q: wanted exactly when the chunk has query heads")
        stride = steps[0] if self.rows > 1 else width
        rc = lib().mk_chunk_append(self.h, qkv.data_ptr(), int(qkv.dtype is _F32), stride,
                                   _here("kv_pool", kv_pool, self._pool_type, self._pool, dev),
                                   None if q is None else _here("q", q, _BF16, self._q, dev), _on(stream, dev))
        if rc != MK_OK:
            raise MkError("mk_chunk_append", rc)

    def attend(self, q: torch.Tensor, kv_pool: torch.Tensor, out: torch.Tensor, stream=None) -> None:
        """Causal attention of the rows q [rows, nq, head_dim] over the pages; out like q (bf16)."""
        dev = _device()
        rc = lib().mk_chunk_attend(self.h, _here("q", q, _BF16, self._q, dev),
                                   _here("kv_pool", kv_pool, self._pool_type, self._pool, dev),
                                   _here("out", out, _BF16, self._q, dev), _on(stream, dev))
        if rc != MK_OK:
            raise MkError("mk_chunk_attend", rc)

    def read(self, kv_pool: torch.Tensor, out: torch.Tensor, stream=None) -> None:
        """Every cached and new position of every request, out [tokens, nkv, 2, head_dim] (bf16)."""
        dev = _device()
        rc = lib().mk_chunk_read(self.h, _here("kv_pool", kv_pool, self._pool_type, self._pool, dev),
                                 _here("out", out, _BF16, self._kv, dev), _on(stream, dev))
        if rc != MK_OK:
            raise MkError("mk_chunk_read", rc)

    def sync(self, stream=None) -> int:
        """Wait for the stream; the device status."""
        return lib().mk_chunk_sync(self.h, _stream(stream))

    def info(self) -> dict:
        buf = (ctypes.c_int * 7)()
        lib().mk_chunk_info(self.h, buf, 7)
        return dict(zip(["batch", "rows", "tokens", "tasks", "split_tasks", "joined_rows", "num_ctas"], list(buf)))

    def close(self):
        if getattr(self, "h", None):
            lib().mk_chunk_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def inspect_chunk(D, seq_lens: Sequence[int], new_lens: Sequence[int], num_ctas: int) -> torch.Tensor:
    """Host-only attention task list of a chunk: int tensor [n, 8] (request, KV head, first row, rows, first
    64-key tile, tiles, first split row or -1, CTA)."""
    dims, n = _chunk_dims(D), len(seq_lens)
    if len(new_lens) != n:
        raise ValueError("seq_lens and new_lens do not describe one batch")
    args = (ctypes.byref(dims), n, _int_array(seq_lens), _int_array(new_lens), num_ctas)
    count = lib().mk_chunk_inspect(*args, None, 0)
    if count < 0:
        raise MkError("mk_chunk_inspect", count)
    buf = (ctypes.c_int * (8 * count))()
    lib().mk_chunk_inspect(*args, buf, count)
    return torch.tensor(list(buf), dtype=torch.int64).view(count, 8)


def probs(logits: torch.Tensor, temperature: float, out: torch.Tensor, stream=None) -> None:
    """softmax(logits / temperature) of float32 rows [rows, vocab] (rows may lie apart) into out [rows, vocab];
    temperature 0: 1 at the largest logit."""
    dev = _device()
    if logits.dim() != 2 or logits.dtype is not _F32 or logits.get_device() != dev or (
            logits.numel() and logits.stride(1) != 1 and logits.shape[1] != 1):
        raise ValueError("logits: float32 rows [rows, vocab] of the current CUDA device are wanted")
    rows, vocab = logits.shape
    rc = lib().mk_probs(logits.data_ptr() if rows else None, rows, vocab, logits.stride(0) if rows > 1 else vocab,
                        float(temperature), _here("out", out, _F32, logits.shape, dev) if rows else None, _on(stream, dev))
    if rc != MK_OK:
        raise MkError("mk_probs", rc)


def verify(target: torch.Tensor, draft: Optional[torch.Tensor], drafts: torch.Tensor, u: torch.Tensor, r: torch.Tensor,
           tokens: torch.Tensor, accepted: torch.Tensor, n_draft: Optional[torch.Tensor] = None, stream=None) -> None:
    """Verify drafted tokens (include/mk.h): target float32 [batch, k + 1, vocab], draft float32 [batch, k, vocab] or
    None (certain drafts), drafts int32 [batch, k], u float32 [batch, k], r float32 [batch], n_draft int32 [batch] or
    None (k each); out: tokens int32 [batch, k + 1], accepted int32 [batch]."""
    if target.dim() != 3:
        raise ValueError("target: float32 [batch, k + 1, vocab] is wanted")
    b, k1, v = target.shape
    dev, each, row = _device(), (b, k1 - 1), (b,)
    rc = lib().mk_verify(b, k1 - 1, v, _here("target", target, _F32, target.shape, dev),
                         None if draft is None else _here("draft", draft, _F32, (b, k1 - 1, v), dev),
                         _here("drafts", drafts, _I32, each, dev),
                         None if n_draft is None else _here("n_draft", n_draft, _I32, row, dev),
                         _here("u", u, _F32, each, dev), _here("r", r, _F32, row, dev),
                         _here("tokens", tokens, _I32, (b, k1), dev), _here("accepted", accepted, _I32, row, dev),
                         _on(stream, dev))
    if rc != MK_OK:
        raise MkError("mk_verify", rc)


_E4M3 = torch.float8_e4m3fn
_ROWS, _F32_ROWS = {_BF16: MK_ROWS_BF16, _F32: MK_ROWS_F32}, {_F32: MK_ROWS_F32}


def _rows(name: str, t: torch.Tensor, kinds):
    """Device, type, shape and row stride of rows [rows, n] that may lie apart."""
    dev, kind, shape = t.get_device(), kinds.get(t.dtype), t.shape
    if kind is not None and dev >= 0 and len(shape) == 2 and dev == torch._C._cuda_getDevice():
        if t.is_contiguous():
            return dev, kind, shape, shape[1]
        steps = t.stride()
        if steps[1] == 1 or shape[1] == 1:
            return dev, kind, shape, steps[0] if shape[0] > 1 else shape[1]
    raise ValueError(f"{name}: {' or '.join(str(k) for k in kinds)} rows [rows, n] of the current CUDA device are wanted")


def _scales(t: Optional[torch.Tensor], shape, dev: int) -> int:
    """The address of 8-bit rows' scales: uint8, a 32nd of the last dimension."""
    if t is None:
        raise ValueError("8-bit rows come with their scales")
    return _here("scales", t, _U8, shape, dev)


def norm(x: torch.Tensor, gamma: Optional[torch.Tensor], eps: float, out: Optional[torch.Tensor],
         add: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
         stream=None) -> None:
    """t = x + add summed over its terms (fp32), out = t / sqrt(mean(t^2) + eps) * gamma (include/mk.h).  x bf16 or
    float32 [rows, n] (rows may lie apart); add bf16 or float32 [rows, n] or [rows, terms, n]; gamma bf16 [n] or None;
    out bf16, float32 or (with scales uint8 [rows, n / 32]) float8_e4m3fn [rows, n], or None; total like x, packed, or
    None; it may be x itself."""
    dev, kind, shape, stride = _rows("x", x, _ROWS)
    rows, n = shape
    terms, a, a_kind = 0, None, 0
    if add is not None:
        a_type = add.dtype
        if a_type not in _ROWS or add.dim() not in (2, 3):
            raise ValueError("add: bf16 or float32 [rows, n] or [rows, terms, n] is wanted")
        terms, a_kind = add.shape[1] if add.dim() == 3 else 1, _ROWS[a_type]
        a = _here("add", add, a_type, (rows, terms, n) if add.dim() == 3 else shape, dev)
    o, s, o_kind = None, None, 0
    if out is not None:
        o_type = out.dtype
        if o_type is _E4M3:
            s, o_kind = _scales(scales, (rows, n // 32), dev), MK_ROWS_E4M3
        elif o_type in _ROWS:
            o_kind = _ROWS[o_type]
        else:
            raise ValueError("out: bf16, float32 or float8_e4m3fn is wanted")
        o = _here("out", out, o_type, shape, dev)
    if s is None and scales is not None:
        raise ValueError("scales: only with an 8-bit out")
    if not rows:
        return
    rc = lib().mk_norm(rows, n, x.data_ptr(), kind, stride, a, a_kind, terms,
                       None if gamma is None else _here("gamma", gamma, _BF16, (n,), dev), eps,
                       None if total is None else _here("total", total, x.dtype, shape, dev), o, o_kind, s,
                       _on(stream, dev))
    if rc != MK_OK:
        raise MkError("mk_norm", rc)


def quantize(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """Rows x [rows, n] (bf16 or float32, rows may lie apart) to 8 bits: codes float8_e4m3fn [rows, n], scales uint8
    [rows, n / 32] (include/mk.h).  Contiguous weights of more dimensions go as x.view(-1, n)."""
    dev, kind, shape, stride = _rows("x", x, _ROWS)
    rows, n = shape
    c, s = _here("codes", codes, _E4M3, shape, dev), _scales(scales, (rows, n // 32), dev)
    if not rows:
        return
    rc = lib().mk_quantize(rows, n, x.data_ptr(), kind, stride, c, s, _on(stream, dev))
    if rc != MK_OK:
        raise MkError("mk_quantize", rc)


def route(logits: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor, first: torch.Tensor, order: torch.Tensor,
          stream=None) -> None:
    """Each row's experts and the rows of each expert (include/mk.h): logits float32 [rows, experts] (rows may lie
    apart); out: ids int32 and gates float32 [rows, top_k], first int32 [experts + 1], order int32 [rows * top_k]."""
    dev, _, (rows, experts), stride = _rows("logits", logits, _F32_ROWS)
    if ids.dim() != 2:
        raise ValueError("ids: int32 [rows, top_k] is wanted")
    k = ids.shape[1]
    each = (rows, k)
    rc = lib().mk_route(rows, experts, k, logits.data_ptr() if rows else None, stride, _here("ids", ids, _I32, each, dev),
                        _here("gates", gates, _F32, each, dev), _here("first", first, _I32, (experts + 1,), dev),
                        _here("order", order, _I32, (rows * k,), dev), _on(stream, dev))
    if rc != MK_OK:
        raise MkError("mk_route", rc)


class Experts:
    """Owns an mk_experts: the experts' products over a chunk's rows
    (include/mk.h).

    D: dims with hidden, n_experts, top_k and expert_ffn.  rows_type: "bf16", or
    "e4m3" (rows, weights and up's results as float8_e4m3fn codes with uint8
    scales of a 32nd of their last dimension).  timeout_us, debug_drop: limits
    and losses for tests (mk_experts_set_debug)."""

    def __init__(self, D, rows_type: str, timeout_us: int = 0, debug_drop: int = 0):
        kinds = {"bf16": MK_ROWS_BF16, "e4m3": MK_ROWS_E4M3}
        if rows_type not in kinds:
            raise ValueError(f"rows_type: {rows_type!r}, wanted one of {tuple(kinds)}")
        dims = MkModelDims(hidden=D.hidden, n_experts=D.n_experts, top_k=D.top_k, expert_ffn=D.expert_ffn)
        h = ctypes.c_void_p()
        rc = lib().mk_experts_create(ctypes.byref(dims), kinds[rows_type], ctypes.byref(h))
        if rc != MK_OK:
            raise MkError("mk_experts_create", rc)
        self.h, self.e4m3 = h, rows_type == "e4m3"
        if timeout_us or debug_drop:
            rc = lib().mk_experts_set_debug(h, timeout_us, debug_drop)
            if rc != MK_OK:
                raise MkError("mk_experts_set_debug", rc)
        self.hidden, self.experts, self.top_k, self.ffn = e = D.hidden, D.n_experts, D.top_k, D.expert_ffn
        self._first, self._up, self._down = (e[1] + 1,), (e[1], 2 * e[3], e[0]), (e[1], e[0], e[3]) if self.e4m3 else (e[1], e[3], e[0])

    def _lists(self, first, order):
        """Device, rows, pairs and the lists' addresses."""
        dev, pairs = order.get_device(), order.numel()
        if dev < 0 or dev != torch._C._cuda_getDevice() or pairs % self.top_k:
            raise ValueError(f"order: a multiple of {self.top_k} pairs on the current CUDA device is wanted, got {pairs} on "
                             f"{order.device}")
        return (dev, pairs // self.top_k, pairs, _here("first", first, _I32, self._first, dev),
                _here("order", order, _I32, (pairs,), dev))

    def up(self, x: torch.Tensor, w: torch.Tensor, first: torch.Tensor, order: torch.Tensor, h: torch.Tensor,
           x_scales: Optional[torch.Tensor] = None, w_scales: Optional[torch.Tensor] = None,
           h_scales: Optional[torch.Tensor] = None, stream=None) -> None:
        """Gate and up products with SwiGLU: x [rows, hidden], w [experts, 2 ffn, hidden] (rows interleaved), first and
        order of route(); h [rows * top_k, ffn] in the sorted order."""
        dev, rows, pairs, f, o = self._lists(first, order)
        h8, f8, kind, sa, sb, sc = self.hidden // 32, self.ffn // 32, _BF16, None, None, None
        if self.e4m3:
            kind, sa, sc = _E4M3, _scales(x_scales, (rows, h8), dev), _scales(h_scales, (pairs, f8), dev)
            sb = _scales(w_scales, (self.experts, 2 * self.ffn, h8), dev)
        elif x_scales is not None or w_scales is not None or h_scales is not None:
            raise ValueError("scales are of 8-bit rows")
        rc = lib().mk_experts_up(self.h, rows, _here("x", x, kind, (rows, self.hidden), dev), sa,
                                 _here("w", w, kind, self._up, dev), sb, f, o,
                                 _here("h", h, kind, (pairs, self.ffn), dev), sc, _on(stream, dev))
        if rc != MK_OK:
            raise MkError("mk_experts_up", rc)

    def down(self, h: torch.Tensor, w: torch.Tensor, first: torch.Tensor, order: torch.Tensor,
             gates: Optional[torch.Tensor], y: torch.Tensor, h_scales: Optional[torch.Tensor] = None,
             w_scales: Optional[torch.Tensor] = None, stream=None) -> None:
        """Down products times the gates: h [rows * top_k, ffn] of up(), w [experts, ffn, hidden] (8 bits: [experts,
        hidden, ffn]), gates float32 [rows, top_k] or None; y bf16 [rows, top_k, hidden] (or [rows * top_k, hidden])."""
        dev, rows, pairs, f, o = self._lists(first, order)
        f8, kind, sa, sb = self.ffn // 32, _BF16, None, None
        if self.e4m3:
            kind, sa = _E4M3, _scales(h_scales, (pairs, f8), dev)
            sb = _scales(w_scales, (self.experts, self.hidden, f8), dev)
        elif h_scales is not None or w_scales is not None:
            raise ValueError("scales are of 8-bit rows")
        g = None if gates is None else _here("gates", gates, _F32, (rows, self.top_k), dev)
        rc = lib().mk_experts_down(self.h, rows, _here("h", h, kind, (pairs, self.ffn), dev), sa,
                                   _here("w", w, kind, self._down, dev), sb, f, o, g,
                                   _here("y", y, _BF16, (rows, self.top_k, self.hidden) if y.dim() == 3 else (pairs, self.hidden),
                                         dev), _on(stream, dev))
        if rc != MK_OK:
            raise MkError("mk_experts_down", rc)

    def sync(self, stream=None) -> int:
        """Wait for the stream; MK_OK, or MK_ERR_DEP_TIMEOUT if a wait of the products ran out since this stream last asked."""
        return lib().mk_experts_sync(self.h, _stream(stream))

    def close(self):
        if getattr(self, "h", None):
            lib().mk_experts_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
