"""ctypes binding of libstage.so: the C ABI of include/stage.h with the same names.

Argument marshalling only.  Every step of the stage forward runs in the library's CUDA
kernels; nothing here computes.  Device buffers are PyTorch tensors (PyTorch provides
device memory and the stream); host arrays are numpy arrays.  If the library has not
been built this module raises on load: there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional, Sequence

import numpy as np

from . import build as _build

STAGE_OK = 0
STAGE_E_INVALID = -1
STAGE_E_DOES_NOT_FIT = -2
STAGE_E_HANDOFF = -3
STAGE_E_POSITION = -4
STAGE_E_BUSY = -5
STAGE_E_NOT_LAST = -6
STAGE_E_CUDA = -7
STAGE_E_STATE = -8
STAGE_E_INJECTED = -9
STAGE_E_HOST = -10
STAGE_F32, STAGE_F16, STAGE_BF16 = 0, 1, 2
STAGE_ROPE_PLAIN, STAGE_ROPE_LINEAR, STAGE_ROPE_BASE, STAGE_ROPE_BANDS, STAGE_ROPE_PARTS = 0, 1, 2, 3, 4
STAGE_LOGPROBS_MAX_TOP = 32
STAGE_KV4_SCRATCH_MAX = 64 << 20
STAGE_KV4_ERROR_AT = 2048
STAGE_PLAN_OK, STAGE_PLAN_NO_PAGES, STAGE_PLAN_BAD_LEN, STAGE_PLAN_NO_ROOM = 0, 1, 2, 3
ERROR_NAMES = {0: "STAGE_OK", -1: "STAGE_E_INVALID", -2: "STAGE_E_DOES_NOT_FIT", -3: "STAGE_E_HANDOFF",
               -4: "STAGE_E_POSITION", -5: "STAGE_E_BUSY", -6: "STAGE_E_NOT_LAST", -7: "STAGE_E_CUDA",
               -8: "STAGE_E_STATE", -9: "STAGE_E_INJECTED", -10: "STAGE_E_HOST"}


class StageError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERROR_NAMES.get(code, code)}: {msg}")
        self.code = code


class stage_model_cfg(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("n_layers", "hidden", "n_q_heads", "n_kv_heads", "head_dim", "ffn", "vocab",
                                       "n_experts", "top_k", "expert_ffn")] + \
               [("rms_eps", C.c_float), ("rope_theta", C.c_float)] + \
               [(n, C.c_int) for n in ("max_seqs", "max_seq_len", "max_tokens", "gemm_bf16_min_tokens", "shared_ffn")]


class stage_layer_range(C.Structure):
    _fields_ = [("begin", C.c_int), ("end", C.c_int)]


class stage_q8(C.Structure):
    _fields_ = [("q", C.c_void_p), ("scale", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64)]


class stage_layer_w(C.Structure):
    _fields_ = [("attn_norm", C.c_void_p), ("ffn_norm", C.c_void_p)] + \
               [(n, stage_q8) for n in ("wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down", "router")] + \
               [("e_gate", C.c_void_p), ("e_up", C.c_void_p), ("e_down", C.c_void_p)] + \
               [(n, stage_q8) for n in ("shared_score", "shared_gate", "shared_up", "shared_down")]


class stage_weights(C.Structure):
    _fields_ = [("embed", stage_q8), ("final_norm", C.c_void_p), ("lm_head", stage_q8), ("layers", C.c_void_p)]


class stage_act(C.Structure):
    _fields_ = [("data", C.c_void_p), ("rows", C.c_int), ("cols", C.c_int)]


_lib = None

_SIGS = {
    "stage_required_bytes": (C.c_size_t, [C.POINTER(stage_model_cfg), stage_layer_range]),
    "stage_plan_placement": (C.c_int, [C.POINTER(stage_model_cfg), C.c_int, C.POINTER(C.c_size_t),
                                       C.POINTER(C.c_int32), C.POINTER(C.c_size_t)]),
    "stage_create": (C.c_int, [C.POINTER(stage_model_cfg), stage_layer_range, C.c_void_p, C.c_size_t, C.c_void_p,
                               C.POINTER(C.c_void_p)]),
    "stage_load_layer": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p]),
    "stage_load_endpoints": (C.c_int, [C.c_void_p, C.c_void_p]),
    "stage_prefill": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "stage_decode": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "stage_logits": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p]),
    "stage_commit": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p]),
    "stage_truncate": (C.c_int, [C.c_void_p, C.c_int, C.c_int]),
    "stage_reset": (C.c_int, [C.c_void_p]),
    "stage_committed_len": (C.c_int, [C.c_void_p, C.c_int, C.POINTER(C.c_int)]),
    "stage_gemm_mode": (C.c_int, [C.c_void_p, C.c_int, C.POINTER(C.c_int)]),
    "stage_read_kv": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p]),
    "stage_write_kv": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p]),
    "stage_last_error": (C.c_char_p, [C.c_void_p]),
    "stage_create_error": (C.c_char_p, []),
    "stage_destroy": (None, [C.c_void_p]),
    "stage_debug_inject": (C.c_int, [C.c_void_p, C.c_int, C.c_int]),
    "stage_pipeline_create": (C.c_int, [C.c_void_p, C.c_int, C.POINTER(C.c_void_p)]),
    "stage_pipeline_step": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                      C.c_void_p, C.c_void_p, C.c_void_p]),
    "stage_pipeline_generate": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p]),
    "stage_pipeline_handoff_stats": (C.c_int, [C.c_void_p, C.c_int, C.POINTER(C.c_int64), C.POINTER(C.c_int64)]),
    "stage_pipeline_kernel_timing": (C.c_int, [C.c_void_p, C.c_int]),
    "stage_pipeline_kernel_time": (C.c_int, [C.c_void_p, C.POINTER(C.c_float), C.POINTER(C.c_int)]),
    "stage_pipeline_last_error": (C.c_char_p, [C.c_void_p]),
    "stage_pipeline_destroy": (None, [C.c_void_p]),
    "stage_op_q8_device_bytes": (C.c_int, [C.c_int64, C.c_int64, C.POINTER(C.c_size_t), C.POINTER(C.c_size_t)]),
    "stage_op_q8_pack": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p]),
    "stage_op_embed": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_void_p, C.c_int, C.c_void_p,
                                 C.c_void_p]),
    "stage_op_gemv": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_void_p, C.c_int, C.c_void_p,
                                C.c_float, C.c_void_p, C.c_void_p]),
    "stage_op_attention_workspace_bytes": (C.c_size_t, [C.c_int] * 5),
    "stage_op_gemm_bf16": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_void_p, C.c_int64, C.c_int64,
                                     C.c_void_p, C.c_void_p]),
    "stage_op_attention_decode": (C.c_int, [C.c_void_p] * 5 + [C.c_int] * 6 + [C.c_void_p, C.c_void_p, C.c_size_t,
                                                                              C.c_void_p]),
    "stage_op_attention_decode_static": (C.c_int, [C.c_void_p] * 5 + [C.c_int] * 6 + [C.c_void_p, C.c_void_p]),
    "stage_op_last_error": (C.c_char_p, []),
    "stage_op_kv4_cache_bytes": (C.c_size_t, [C.c_int64, C.c_int, C.c_int, C.c_int]),
    "stage_op_kv4_plan": (C.c_int, [C.c_int, C.c_int, C.c_int64] + [C.c_void_p] * 4 + [C.c_int, C.c_void_p, C.c_int] +
                          [C.c_void_p] * 3 + [C.c_int] + [C.c_void_p] * 6),
    "stage_op_kv4_append": (C.c_int, [C.c_void_p, C.c_int64, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p, C.c_int,
                                      C.c_int64, C.c_void_p, C.c_int, C.c_void_p]),
    "stage_op_kv4_read": (C.c_int, [C.c_void_p, C.c_int64, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_void_p,
                                    C.c_void_p, C.c_int, C.c_int64, C.c_void_p]),
    "stage_op_kv4_attention_workspace_bytes": (C.c_size_t, [C.c_int] * 6),
    "stage_op_kv4_attention_many": (C.c_int, [C.c_int] * 8),
    "stage_op_kv4_debug_stall": (C.c_int, [C.c_int]),
    "stage_op_kv4_attention": (C.c_int, [C.c_void_p, C.c_int64, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_int64,
                                         C.c_int, C.c_int] + [C.c_void_p] * 3 + [C.c_int] * 4 +
                               [C.c_void_p, C.c_int64, C.c_void_p, C.c_size_t, C.c_void_p]),
    "stage_op_norm_f8": (C.c_int, [C.c_void_p, C.c_int, C.c_int64] * 2 + [C.c_void_p, C.c_int64, C.c_void_p, C.c_float,
                                                                         C.c_int, C.c_int] +
                         [C.c_void_p, C.c_int64] * 3 + [C.c_void_p]),
    "stage_op_f8_gemm": (C.c_int, [C.c_void_p, C.c_int64] * 3 + [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int,
                                                                 C.c_int64, C.c_void_p, C.c_void_p]),
    "stage_op_f8_debug_stall": (C.c_int, [C.c_int]),
    "stage_op_f8_debug_late": (C.c_int, [C.c_int]),
    "stage_op_rope_freqs": (C.c_int, [C.c_int, C.c_double, C.c_int] + [C.c_double] * 4 + [C.POINTER(C.c_double),
                                                                                        C.POINTER(C.c_float)]),
    "stage_op_rope": (C.c_int, [C.c_void_p, C.c_int64, C.c_int] * 2 + [C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_void_p,
                                                                      C.c_int, C.c_int, C.c_float] +
                      [C.c_void_p, C.c_int64] * 2 + [C.c_void_p]),
    "stage_op_logprobs": (C.c_int, [C.c_void_p, C.c_int, C.c_int64, C.c_int, C.c_int] + [C.c_void_p] * 4 +
                          [C.c_int, C.c_void_p, C.c_void_p, C.c_void_p]),
}


def declared_symbols() -> list:
    """Every function the headers in include/ declare (parsed from the headers)."""
    import re
    names = []
    inc = os.path.join(_build.ROOT, "include")
    for h in sorted(os.listdir(inc)):
        if h.endswith(".h"):
            names += re.findall(r"^STAGE_API [^(]*?\b(stage_\w+)\(", open(os.path.join(inc, h)).read(), flags=re.M)
    return names


def lib():
    """Load libstage.so (built by __graft_entry__.build()).  Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.LIB):
            raise ImportError(f"{_build.LIB} is not built: run __graft_entry__.build() (nvcc, sm_103a)")
        # make libcudart resolvable even when PyTorch has not loaded it yet
        try:
            C.CDLL(os.path.join(_build.cuda_lib_dir(), "libcudart.so"), mode=C.RTLD_GLOBAL)
        except OSError:
            pass
        L = C.CDLL(_build.LIB)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


# ----------------------------------------------------------------------------- marshalling

def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _ptr(a: Optional[np.ndarray]):
    return None if a is None else a.ctypes.data


def make_cfg(model, max_seqs: int, max_seq_len: int, max_tokens: int, gemm_bf16_min_tokens: int = 0) -> stage_model_cfg:
    """stage_model_cfg from any object with the model's shape fields (e.g. synth.ModelCfg)."""
    return stage_model_cfg(model.n_layers, model.hidden, model.n_q_heads, model.n_kv_heads, model.head_dim,
                           model.ffn, model.vocab, model.n_experts, model.top_k, model.expert_ffn,
                           model.rms_eps, model.rope_theta, max_seqs, max_seq_len, max_tokens, gemm_bf16_min_tokens,
                           getattr(model, "shared_ffn", 0))


class _Keep:
    """Holds the numpy arrays behind a stage_weights so their memory outlives the call."""

    def __init__(self):
        self.refs = []

    def q8(self, m) -> stage_q8:
        if m is None:
            return stage_q8(None, None, 0, 0)
        q = np.ascontiguousarray(m.q, dtype=np.int8)
        s = np.ascontiguousarray(m.s, dtype=np.uint16)
        self.refs += [q, s]
        return stage_q8(q.ctypes.data, s.ctypes.data, q.shape[0], q.shape[1])

    def f32(self, a):
        if a is None:
            return None
        a = np.ascontiguousarray(a, dtype=np.float32)
        self.refs.append(a)
        return a.ctypes.data

    def layer(self, lw) -> stage_layer_w:
        w = stage_layer_w()
        w.attn_norm, w.ffn_norm = self.f32(lw.attn_norm), self.f32(lw.ffn_norm)
        for n in ("wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down", "router", "shared_score", "shared_gate",
                  "shared_up", "shared_down"):
            setattr(w, n, self.q8(getattr(lw, n, None)))
        for n in ("e_gate", "e_up", "e_down"):
            mats = getattr(lw, n, None) or []
            if mats:
                arr = (stage_q8 * len(mats))(*[self.q8(m) for m in mats])
                self.refs.append(arr)
                setattr(w, n, C.cast(arr, C.c_void_p))
            else:
                setattr(w, n, None)
        return w

    def weights(self, sw) -> stage_weights:
        w = stage_weights()
        w.embed = self.q8(sw.embed)
        w.final_norm = self.f32(sw.final_norm)
        w.lm_head = self.q8(sw.lm_head)
        if sw.layers:
            arr = (stage_layer_w * len(sw.layers))(*[self.layer(l) for l in sw.layers])
            self.refs.append(arr)
            w.layers = C.cast(arr, C.c_void_p)
        return w


def _act(t) -> Optional[stage_act]:
    if t is None:
        return None
    if t.dtype.__str__() != "torch.float32" or not t.is_cuda or not t.is_contiguous() or t.dim() != 2:
        raise StageError(STAGE_E_HANDOFF, "hidden activations are contiguous float32 CUDA tensors [n, hidden]")
    return stage_act(t.data_ptr(), t.shape[0], t.shape[1])


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return int(stream) if not hasattr(stream, "cuda_stream") else stream.cuda_stream


# ----------------------------------------------------------------------------- functions (same names as the C ABI)

def stage_required_bytes(cfg: stage_model_cfg, begin: int, end: int) -> int:
    return int(lib().stage_required_bytes(C.byref(cfg), stage_layer_range(begin, end)))


def stage_plan_placement(cfg: stage_model_cfg, budgets) -> tuple:
    """Block bounds [n_devices + 1] and each stage's required bytes for the given per-device
    budgets (see include/stage.h); raises StageError (DoesNotFit when no placement is legal)."""
    n = len(budgets)
    bud = (C.c_size_t * max(n, 1))(*[int(b) for b in budgets])
    bounds = (C.c_int32 * (n + 1))()
    req = (C.c_size_t * max(n, 1))()
    rc = lib().stage_plan_placement(C.byref(cfg), n, bud, bounds, req)
    if rc != STAGE_OK:
        raise StageError(rc, "no legal placement" if rc == STAGE_E_DOES_NOT_FIT else "invalid placement request")
    return [int(b) for b in bounds], [int(r) for r in req[:n]]


def stage_create(cfg: stage_model_cfg, begin: int, end: int, weights=None, budget: Optional[int] = None, stream=None):
    """Returns a stage handle (int).  ``weights``: an object shaped like synth.StageWeights or None."""
    keep = _Keep()
    wp = C.byref(keep.weights(weights)) if weights is not None else None
    h = C.c_void_p()
    budget = (1 << 62) if budget is None else int(budget)
    rc = lib().stage_create(C.byref(cfg), stage_layer_range(begin, end), wp, budget, _stream(stream), C.byref(h))
    if rc != STAGE_OK:
        raise StageError(rc, lib().stage_create_error().decode())
    return h.value


def _check(st, rc):
    if rc != STAGE_OK:
        raise StageError(rc, lib().stage_last_error(st).decode())


def stage_load_layer(st, global_layer: int, layer_weights) -> None:
    keep = _Keep()
    lw = keep.layer(layer_weights)
    _check(st, lib().stage_load_layer(st, global_layer, C.byref(lw)))


def stage_load_endpoints(st, weights) -> None:
    keep = _Keep()
    w = keep.weights(weights)
    _check(st, lib().stage_load_endpoints(st, C.byref(w)))


def _fwd(fn, st, seq_ids, positions, tokens, hidden_in, hidden_out):
    seq, pos = _i32(seq_ids), _i32(positions)
    tok = None if tokens is None else _i32(tokens)
    hin, hout = _act(hidden_in), _act(hidden_out)
    rc = fn(st, len(pos), _ptr(seq), _ptr(pos), _ptr(tok), C.byref(hin) if hin else None,
            C.byref(hout) if hout else None)
    _check(st, rc)


def stage_prefill(st, seq_ids, positions, tokens=None, hidden_in=None, hidden_out=None) -> None:
    _fwd(lib().stage_prefill, st, seq_ids, positions, tokens, hidden_in, hidden_out)


def stage_decode(st, seq_ids, positions, tokens=None, hidden_in=None, hidden_out=None) -> None:
    _fwd(lib().stage_decode, st, seq_ids, positions, tokens, hidden_in, hidden_out)


def stage_logits(st, row_index: Sequence[int], logits_out=None, argmax_out=None) -> None:
    rows = _i32(row_index)
    lp = None if logits_out is None else logits_out.data_ptr()
    ap = None if argmax_out is None else argmax_out.data_ptr()
    _check(st, lib().stage_logits(st, len(rows), _ptr(rows), lp, ap))


def stage_commit(st, seq_ids, new_len) -> None:
    s, n = _i32(seq_ids), _i32(new_len)
    _check(st, lib().stage_commit(st, len(s), _ptr(s), _ptr(n)))


def stage_truncate(st, seq_id: int, length: int) -> None:
    _check(st, lib().stage_truncate(st, seq_id, length))


def stage_reset(st) -> None:
    _check(st, lib().stage_reset(st))


def stage_committed_len(st, seq_id: int) -> int:
    v = C.c_int()
    _check(st, lib().stage_committed_len(st, seq_id, C.byref(v)))
    return v.value


def stage_read_kv(st, global_layer: int, seq_id: int, n_pos: int, n_kv_heads: int, head_dim: int):
    """(K, V) of one owned block and sequence as float16 [n_kv_heads, n_pos, head_dim]."""
    k = np.zeros((n_kv_heads, n_pos, head_dim), dtype=np.uint16)
    v = np.zeros_like(k)
    _check(st, lib().stage_read_kv(st, global_layer, seq_id, n_pos, _ptr(k), _ptr(v)))
    return k.view(np.float16), v.view(np.float16)


def stage_write_kv(st, global_layer: int, seq_id: int, pos0: int, k, v) -> None:
    """Write (K, V) float16 [n_kv_heads, n_pos, head_dim] at positions pos0.. of one owned
    block and sequence."""
    k = np.ascontiguousarray(np.asarray(k, dtype=np.float16)).view(np.uint16)
    v = np.ascontiguousarray(np.asarray(v, dtype=np.float16)).view(np.uint16)
    if k.shape != v.shape or k.ndim != 3:
        raise ValueError("k and v must both be [n_kv_heads, n_pos, head_dim]")
    _check(st, lib().stage_write_kv(st, global_layer, seq_id, pos0, k.shape[1], _ptr(k), _ptr(v)))


def stage_gemm_mode(st, n_tokens: int) -> int:
    v = C.c_int()
    _check(st, lib().stage_gemm_mode(st, n_tokens, C.byref(v)))
    return v.value


def stage_last_error(st) -> str:
    return lib().stage_last_error(st).decode()


def stage_create_error() -> str:
    return lib().stage_create_error().decode()


def stage_destroy(st) -> None:
    lib().stage_destroy(st)


def stage_debug_inject(st, what: int, value: int) -> None:
    _check(st, lib().stage_debug_inject(st, what, value))


def _pcheck(p, rc):
    if rc != STAGE_OK:
        raise StageError(rc, lib().stage_pipeline_last_error(p).decode())


def stage_pipeline_create(stages: Sequence[int]):
    arr = (C.c_void_p * len(stages))(*stages)
    h = C.c_void_p()
    rc = lib().stage_pipeline_create(arr, len(stages), C.byref(h))
    if rc != STAGE_OK:
        raise StageError(rc, "stages must tile [0, n_layers) in order with one model, device and stream")
    return h.value


def stage_pipeline_step(p, is_prefill: bool, seq_ids, positions, tokens, row_index=(), logits_out=None,
                        want_tokens: bool = True):
    seq, pos, tok = _i32(seq_ids), _i32(positions), _i32(tokens)
    rows = _i32(row_index)
    nxt = np.zeros(len(rows), dtype=np.int32) if (want_tokens and len(rows)) else None
    lp = None if logits_out is None else logits_out.data_ptr()
    rc = lib().stage_pipeline_step(p, int(bool(is_prefill)), len(pos), _ptr(seq), _ptr(pos), _ptr(tok), len(rows),
                                   _ptr(rows) if len(rows) else None, lp, _ptr(nxt))
    _pcheck(p, rc)
    return nxt


def stage_pipeline_generate(p, seq_ids, first_tokens, n_steps: int, use_graph: bool = True) -> np.ndarray:
    seq, tok = _i32(seq_ids), _i32(first_tokens)
    out = np.zeros((n_steps, len(seq)), dtype=np.int32)
    _pcheck(p, lib().stage_pipeline_generate(p, len(seq), _ptr(seq), _ptr(tok), n_steps, int(bool(use_graph)), _ptr(out)))
    return out


def stage_pipeline_handoff_stats(p, boundary: int):
    c, b = C.c_int64(), C.c_int64()
    _pcheck(p, lib().stage_pipeline_handoff_stats(p, boundary, C.byref(c), C.byref(b)))
    return c.value, b.value


def stage_pipeline_kernel_timing(p, enable: bool) -> None:
    _pcheck(p, lib().stage_pipeline_kernel_timing(p, int(bool(enable))))


def stage_pipeline_kernel_time(p):
    """(mean microseconds, count) of the FFN up-projection launches of the last timed step."""
    m, n = C.c_float(), C.c_int()
    _pcheck(p, lib().stage_pipeline_kernel_time(p, C.byref(m), C.byref(n)))
    return m.value, n.value


def stage_pipeline_last_error(p) -> str:
    return lib().stage_pipeline_last_error(p).decode()


def stage_pipeline_destroy(p) -> None:
    lib().stage_pipeline_destroy(p)


# ----------------------------------------------------------------------------- kernel-level entry points

def stage_op_last_error() -> str:
    return lib().stage_op_last_error().decode()


def _opcheck(rc):
    if rc != STAGE_OK:
        raise StageError(rc, lib().stage_op_last_error().decode())


def stage_op_q8_device_bytes(rows: int, cols: int):
    qb, sb = C.c_size_t(), C.c_size_t()
    _opcheck(lib().stage_op_q8_device_bytes(rows, cols, C.byref(qb), C.byref(sb)))
    return qb.value, sb.value


def stage_op_q8_pack(m, q_dev, s_dev) -> None:
    keep = _Keep()
    h = keep.q8(m)
    _opcheck(lib().stage_op_q8_pack(C.byref(h), q_dev.data_ptr(), s_dev.data_ptr()))


def stage_op_embed(q_dev, s_dev, rows: int, cols: int, tok, out, stream=None) -> None:
    """tok: int32 device tensor [n_tok]; out: f32 device tensor [n_tok, cols]."""
    _opcheck(lib().stage_op_embed(q_dev.data_ptr(), s_dev.data_ptr(), rows, cols, tok.data_ptr(), tok.shape[0],
                                  out.data_ptr(), _stream(stream)))


def stage_op_gemv(q_dev, s_dev, rows: int, cols: int, x, y, gamma=None, eps: float = 1e-5, stream=None) -> None:
    _opcheck(lib().stage_op_gemv(q_dev.data_ptr(), s_dev.data_ptr(), rows, cols, x.data_ptr(), x.shape[0],
                                 None if gamma is None else gamma.data_ptr(), eps, y.data_ptr(), _stream(stream)))


def stage_op_gemm_bf16(a_bits, q_dev, s_dev, rows: int, cols: int, y, stream=None) -> None:
    """a_bits: int16/uint16 device tensor [M, lda] of bf16 bit patterns; y: f32 [M, rows]."""
    M, lda = a_bits.shape
    _opcheck(lib().stage_op_gemm_bf16(a_bits.data_ptr(), lda, M, q_dev.data_ptr(), s_dev.data_ptr(), rows, cols,
                                      y.data_ptr(), _stream(stream)))


def stage_op_attention_workspace_bytes(n_tok, n_q_heads, n_kv_heads, head_dim, n_chunks) -> int:
    return int(lib().stage_op_attention_workspace_bytes(n_tok, n_q_heads, n_kv_heads, head_dim, n_chunks))


def stage_op_attention_decode(q, k_cache, v_cache, seq, pos, out, n_chunks: int, workspace, stream=None) -> None:
    """q [n_tok, Hq, D] f32; k/v_cache [seqs, Hkv, max_len, D] f16; seq/pos int32 [n_tok] (device tensors)."""
    n_tok, hq, d = q.shape
    hkv, max_len = k_cache.shape[1], k_cache.shape[2]
    _opcheck(lib().stage_op_attention_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), seq.data_ptr(),
                                             pos.data_ptr(), n_tok, hq, hkv, d, max_len, n_chunks, out.data_ptr(),
                                             workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                             _stream(stream)))


def stage_op_attention_decode_static(q, k_cache, v_cache, seq, pos, out, n_chunks: int, stream=None) -> None:
    """stage_op_attention_decode without a workspace: scratch is the library's fixed array
    (no device allocation; calls must not overlap on the GPU)."""
    n_tok, hq, d = q.shape
    hkv, max_len = k_cache.shape[1], k_cache.shape[2]
    _opcheck(lib().stage_op_attention_decode_static(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                                    seq.data_ptr(), pos.data_ptr(), n_tok, hq, hkv, d, max_len,
                                                    n_chunks, out.data_ptr(), _stream(stream)))


# ----------------------------------------------------------------------------- the paged 4-bit KV cache
# A cache is a contiguous uint8 tensor [n_pages, n_kv_heads, page_len / 16, 18 * head_dim] (stage_op_kv4_cache_shape):
# the entry points take its sizes from the shape.  Unlike the entry points above, which take raw buffers, these
# check types, shapes and devices: an index array of another type would be read as garbage.

# They are called once per block and step, so the checks are kept short.

_torch = None
_KV4_DTYPE: dict = {}


def _load_torch():
    global _torch
    import torch
    _KV4_DTYPE.update({torch.float32: STAGE_F32, torch.float16: STAGE_F16, torch.bfloat16: STAGE_BF16})
    _torch = torch
    return torch


def _invalid(msg: str):
    raise StageError(STAGE_E_INVALID, msg)


def _kv4_cache(cache):
    torch = _torch or _load_torch()
    shape = cache.shape
    if len(shape) != 4 or cache.dtype is not torch.uint8 or not cache.is_contiguous():
        _invalid("cache must be a contiguous uint8 tensor [n_pages, n_kv_heads, page_len / 16, 18 * head_dim]")
    n_pages, hkv, tiles, nb = shape
    if nb % 18:
        _invalid("the cache's last dimension must be 18 * head_dim")
    return cache.data_ptr(), n_pages, tiles * 16, hkv, nb // 18


def _kv4_launch(stream, *tensors) -> int:
    """The stream to launch on, once every tensor is known to be on the current device: a launch goes there."""
    torch = _torch or _load_torch()
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev:
            _invalid("tensors on several devices")
    if dev < 0:
        _invalid("device tensors are needed")
    if dev != torch.cuda.current_device():
        _invalid(f"tensors on device {dev}, but the current one is {torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _i32dev(t, what: str, n: int) -> int:
    if t.dtype is not _torch.int32 or not t.is_contiguous():
        _invalid(f"{what} must be a contiguous int32 tensor")
    if t.numel() != n:
        _invalid(f"{what} has {t.numel()} entries, not {n}")
    return t.data_ptr()


def _rows(t, heads: int, head_dim: int, what: str):
    """(pointer, dtype, row stride) of rows [n, heads, head_dim], which may lie apart (a slice of a fused output)."""
    dt = _KV4_DTYPE.get(t.dtype)
    if dt is None:
        _invalid(f"{what} must be float32, float16 or bfloat16")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != head_dim:
        _invalid(f"{what} must be [n_tok, {heads}, {head_dim}]")
    s0, s1, s2 = t.stride()
    if shape[0] and (s2 != 1 or (heads > 1 and s1 != head_dim)):
        _invalid(f"the heads of a row of {what} must lie side by side")
    return t.data_ptr(), dt, s0 if shape[0] > 1 else heads * head_dim


def _beyond_c_int(*sizes) -> bool:  # it would drop what lies above its bits
    return any(not -1 << 31 <= s < 1 << 31 for s in sizes)


def stage_op_kv4_cache_bytes(n_pages: int, page_len: int, n_kv_heads: int, head_dim: int) -> int:
    if not 0 < n_pages < 1 << 31 or _beyond_c_int(page_len, n_kv_heads, head_dim):
        return 0
    return int(lib().stage_op_kv4_cache_bytes(n_pages, page_len, n_kv_heads, head_dim))


def stage_op_kv4_cache_shape(n_pages: int, page_len: int, n_kv_heads: int, head_dim: int) -> tuple:
    """Shape of the uint8 tensor that holds a cache."""
    if not stage_op_kv4_cache_bytes(n_pages, page_len, n_kv_heads, head_dim):
        _invalid("no cache of these sizes")
    return n_pages, n_kv_heads, page_len // 16, 18 * head_dim


def stage_op_kv4_plan(page_len: int, seq_len, new_len, table, free_ring, free_state, seq_len_out, free_state_out, cu_new,
                      slot, pos, seq, status, keep_len=None, n_pages: Optional[int] = None, stream=None) -> None:
    """Block tables and slot maps of one step (include/stage_kv4.h).  Device int32 tensors: seq_len, keep_len,
    new_len, seq_len_out [n]; table [n, stride]; free_ring; free_state, free_state_out [2]; cu_new [n + 1];
    slot, pos, seq [n_tok]; status [1].  n_pages: the cache's pages (default: as many as the ring holds)."""
    if not 16 <= page_len <= 4096:  # a C int would drop what lies above its bits
        _invalid("page_len must lie in [16, 4096]")
    tensors = (seq_len, new_len, table, free_ring, free_state, seq_len_out, free_state_out, cu_new, slot, pos, seq, status)
    stream = _kv4_launch(stream, *tensors) if keep_len is None else _kv4_launch(stream, *tensors, keep_len)
    n, n_tok, ring_len = seq_len.numel(), slot.numel(), free_ring.numel()
    if table.dim() != 2 or table.shape[0] != n:
        _invalid("table must be [n_seqs, stride]")
    sizes = (n, n, table.numel(), ring_len, 2, n, 2, n + 1, n_tok, n_tok, n_tok, 1)
    i32 = _torch.int32
    for t, size in zip(tensors, sizes):
        if t.dtype is not i32 or t.numel() != size or not t.is_contiguous():
            _invalid("plan takes contiguous int32 tensors: seq_len, new_len, seq_len_out [n], table [n, stride], free_ring, "
                     "free_state, free_state_out [2], cu_new [n + 1], slot, pos, seq [n_tok], status [1]")
    p = [t.data_ptr() for t in tensors]
    rc = (_lib or lib()).stage_op_kv4_plan(
        n, page_len, ring_len if n_pages is None else n_pages, p[0],
        None if keep_len is None else _i32dev(keep_len, "keep_len", n), p[1], p[2], table.shape[1], p[3], ring_len, p[4], p[5],
        p[6], n_tok, p[7], p[8], p[9], p[10], p[11], stream)
    if rc:
        _opcheck(rc)


def stage_op_kv4_append(cache, k, v, slot, stream=None) -> None:
    """Quantise rows k, v [n_tok, n_kv_heads, head_dim] (float32, float16 or bfloat16; rows may lie apart) and write
    them to their slots (int32 [n_tok]; outside the cache: skipped)."""
    ptr, n_pages, page_len, hkv, d = _kv4_cache(cache)
    stream = _kv4_launch(stream, cache, k, v, slot)
    kp, kt, ks = _rows(k, hkv, d, "k")
    vp, vt, vs = _rows(v, hkv, d, "v")
    n_tok = k.shape[0]
    if v.shape[0] != n_tok or kt != vt or ks != vs:
        _invalid("k and v must have one length, type and row stride")
    rc = (_lib or lib()).stage_op_kv4_append(ptr, n_pages, page_len, hkv, d, kp, vp, kt, ks, _i32dev(slot, "slot", n_tok),
                                             n_tok, stream)
    if rc:
        _opcheck(rc)


def stage_op_kv4_read(cache, slot, k_out, v_out, stream=None) -> None:
    """Rows at the slots (int32 [n_tok]) as values into k_out, v_out [n_tok, n_kv_heads, head_dim]; rows of slots
    outside the cache stay as they were."""
    ptr, n_pages, page_len, hkv, d = _kv4_cache(cache)
    stream = _kv4_launch(stream, cache, k_out, v_out, slot)
    kp, kt, ks = _rows(k_out, hkv, d, "k_out")
    vp, vt, vs = _rows(v_out, hkv, d, "v_out")
    n_tok = k_out.shape[0]
    if v_out.shape[0] != n_tok or kt != vt or ks != vs:
        _invalid("k_out and v_out must have one length, type and row stride")
    rc = (_lib or lib()).stage_op_kv4_read(ptr, n_pages, page_len, hkv, d, _i32dev(slot, "slot", n_tok), n_tok, kp, vp, kt,
                                           ks, stream)
    if rc:
        _opcheck(rc)


def stage_op_kv4_attention_workspace_bytes(n_seqs: int, n_q_heads: int, n_kv_heads: int, head_dim: int, max_q: int,
                                           max_len: int) -> int:
    if _beyond_c_int(n_seqs, n_q_heads, n_kv_heads, head_dim, max_q, max_len):
        return 0
    return int(lib().stage_op_kv4_attention_workspace_bytes(n_seqs, n_q_heads, n_kv_heads, head_dim, max_q, max_len))


def stage_op_kv4_attention_many(n_seqs: int, n_tok: int, n_q_heads: int, n_kv_heads: int, head_dim: int, dtype, max_q: int,
                                max_len: int) -> bool:
    """Whether a call with these sizes (dtype: a torch type) runs on the kernel for many columns."""
    _torch or _load_torch()
    if _beyond_c_int(n_seqs, n_tok, n_q_heads, n_kv_heads, head_dim, max_q, max_len):
        _invalid("no attention of these sizes")
    rc = lib().stage_op_kv4_attention_many(n_seqs, n_tok, n_q_heads, n_kv_heads, head_dim, _KV4_DTYPE.get(dtype, -1), max_q, max_len)
    if rc < 0:
        _opcheck(rc)
    return bool(rc)


def stage_op_kv4_debug_stall(calls: int) -> None:
    """The next calls of this thread on the kernel for many columns run out of time (tests of that path)."""
    _opcheck(lib().stage_op_kv4_debug_stall(calls))


def stage_op_kv4_attention(cache, q, cu_q, seq_len, table, out, max_q: int, max_len: int, workspace, stream=None) -> None:
    """q, out [n_tok, n_q_heads, head_dim] of one type; cu_q int32 [n_seqs + 1], seq_len int32 [n_seqs], table int32
    [n_seqs, stride]; max_q, max_len bound the query tokens and the length of a sequence; workspace: a tensor of
    stage_op_kv4_attention_workspace_bytes(...) bytes, zero before its first use; the 32-bit word STAGE_KV4_ERROR_AT bytes into
    it is 1 once a call has given up waiting (its rows are NaN)."""
    if not (0 < max_q <= 1 << 20 and 0 < max_len <= 1 << 30):  # a C int would drop what lies above its bits
        _invalid("max_q must lie in [1, 2^20] and max_len in [1, 2^30]")
    ptr, n_pages, page_len, hkv, d = _kv4_cache(cache)
    stream = _kv4_launch(stream, cache, q, cu_q, seq_len, table, out, workspace)
    if q.dim() != 3 or out.shape != q.shape:
        _invalid("q and out must be [n_tok, n_q_heads, head_dim]")
    n_tok, hq, _ = q.shape
    qp, qt, qs = _rows(q, hq, d, "q")
    op, ot, os_ = _rows(out, hq, d, "out")
    n = seq_len.numel()
    if ot != qt:
        _invalid("q and out must have one type")
    if table.dim() != 2 or table.shape[0] != n or not workspace.is_contiguous():
        _invalid("table must be [n_seqs, stride], and workspace contiguous")
    stride = table.shape[1]
    rc = (_lib or lib()).stage_op_kv4_attention(
        ptr, n_pages, page_len, hkv, d, qp, qt, qs, n_tok, hq, _i32dev(cu_q, "cu_q", n + 1),
        _i32dev(seq_len, "seq_len", n), _i32dev(table, "table", n * stride), stride, n, max_q, max_len, op, os_,
        workspace.data_ptr(), workspace.nbytes, stream)
    if rc:
        _opcheck(rc)


# ----------------------------------------------------------------------------- a step's operators around the projections
# include/stage_step.h.  8-bit rows are torch.float8_e4m3fn tensors (or uint8 codes); like the 4-bit cache's entry points
# these check types, shapes and devices.

# They are called several times per block, so they read each property of a tensor once.

_TOO_MANY = "a size beyond 31 bits"  # a C int would drop what lies above its bits


def _launch_on(stream, dev: int) -> int:
    """The stream to launch on, for tensors that are all on device `dev`: the current one, since a launch goes there."""
    if dev < 0:
        _invalid("device tensors are needed, all on one device")
    current = _torch._C._cuda_getDevice()
    if dev != current:
        _invalid(f"tensors on device {dev}, but the current one is {current}")
    return _torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _f8(t, shape, dev: int, what: str):
    """(pointer, row stride) of 8-bit rows, which may lie apart."""
    dt = t.dtype
    if dt is not _torch.float8_e4m3fn and dt is not _torch.uint8:
        _invalid(f"{what} must be float8_e4m3fn (or uint8 codes)")
    if t.shape != shape or t.get_device() != dev:
        _invalid(f"{what} must be {list(shape)}, on the device of the others")
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        _invalid(f"the columns of {what} must lie side by side")
    return t.data_ptr(), s0 if shape[0] > 1 else -(-shape[1] // 16) * 16


def _matrix(t, shape, dev: int, what: str):
    """(pointer, dtype, row stride) of rows [n, k] of a float type, which may lie apart."""
    dt = _KV4_DTYPE.get(t.dtype)
    if dt is None:
        _invalid(f"{what} must be float32, float16 or bfloat16")
    if t.shape != shape or t.get_device() != dev:
        _invalid(f"{what} must be {list(shape)}, on the device of the others")
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        _invalid(f"the columns of {what} must lie side by side")
    return t.data_ptr(), dt, s0 if shape[0] > 1 else shape[1]


def _scales(t, shape, dev: int, what: str):
    """(pointer, stride) of float32 scales [blocks, n]."""
    if t.dtype is not _torch.float32 or t.shape != shape or t.get_device() != dev:
        _invalid(f"{what} must be float32 {list(shape)}, on the device of the others")
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        _invalid(f"the columns of {what} must lie side by side")
    return t.data_ptr(), s0 if shape[0] > 1 else shape[1]


def _array(t, dtype, n: int, dev: int, what: str) -> int:
    """Pointer of n entries side by side."""
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != dev:
        _invalid(f"{what} must be a contiguous {dtype} tensor of {n} entries, on the device of the others")
    return t.data_ptr()


def stage_op_norm_f8(x, q=None, scale=None, gamma=None, eps: float = 1e-5, resid=None, resid_out=None, y=None, stream=None) -> None:
    """Rows x [n_tok, n] plus resid (if given; the sum goes to resid_out, which may be resid), RMS norm with gamma (float32 [n]; None:
    no norm), as 8-bit rows q [n_tok, n] with scales [ceil(n / 128), n_tok] and/or as rows y of x's type."""
    torch = _torch or _load_torch()
    shape, dev = x.shape, x.get_device()
    if len(shape) != 2:
        _invalid("x must be [n_tok, n]")
    if (resid is None) != (resid_out is None) or (q is None) != (scale is None):
        _invalid("resid and resid_out go together, and so do q and scale")
    stream = _launch_on(stream, dev)
    n_tok, n = shape
    if (n_tok | n) >> 31:
        _invalid(_TOO_MANY)
    xp, xt, xs = _matrix(x, shape, dev, "x")
    gp = None
    rp = rt = rs = op = os_ = qp = qs = sp = ss = yp = ys = 0
    if resid is not None:
        rp, rt, rs = _matrix(resid, shape, dev, "resid")
        op, ot, os_ = _matrix(resid_out, shape, dev, "resid_out")
        if ot != rt:
            _invalid("resid and resid_out must have one type")
    if gamma is not None:
        gp = _array(gamma, torch.float32, n, dev, "gamma")
    if q is not None:
        qp, qs = _f8(q, shape, dev, "q")
        sp, ss = _scales(scale, ((n + 127) // 128, n_tok), dev, "scale")
    if y is not None:
        yp, yt, ys = _matrix(y, shape, dev, "y")
        if yt != xt:
            _invalid("y must have x's type")
    rc = (_lib or lib()).stage_op_norm_f8(xp, xt, xs, rp, rt, rs, op, os_, gp, eps, n_tok, n, qp, qs, sp, ss, yp, ys, stream)
    if rc:
        _opcheck(rc)


def stage_op_f8_gemm(a, a_scale, w, w_scale, out, error=None, stream=None) -> None:
    """out [M, N] (float32, float16 or bfloat16) = a w^T of 8-bit rows a [M, K] and w [N, K] (row strides of multiples of 16 bytes) with
    scales a_scale [ceil(K / 128), M] and w_scale [ceil(N / 128), ceil(K / 128)]; error: int32 [1], set to 1 once a call has
    given up waiting (what misses something is NaN)."""
    torch = _torch or _load_torch()
    sa, sw, dev = a.shape, w.shape, a.get_device()
    if len(sa) != 2 or len(sw) != 2 or sa[1] != sw[1]:
        _invalid("a must be [M, K] and w [N, K]")
    stream = _launch_on(stream, dev)
    m, k = sa
    n = sw[0]
    if (m | n | k) >> 31:
        _invalid(_TOO_MANY)
    kb = (k + 127) // 128
    ap, as_ = _f8(a, sa, dev, "a")
    wp, ws = _f8(w, sw, dev, "w")
    sp, ss = _scales(a_scale, (kb, m), dev, "a_scale")
    if w_scale.dtype is not torch.float32 or w_scale.shape != ((n + 127) // 128, kb) or not w_scale.is_contiguous() or w_scale.get_device() != dev:
        _invalid(f"w_scale must be contiguous float32 [{(n + 127) // 128}, {kb}], on the device of the others")
    yp, yt, ys = _matrix(out, (m, n), dev, "out")
    rc = (_lib or lib()).stage_op_f8_gemm(ap, as_, sp, ss, wp, ws, w_scale.data_ptr(), m, n, k, yp, yt, ys,
                                          None if error is None else _array(error, torch.int32, 1, dev, "error"), stream)
    if rc:
        _opcheck(rc)


def stage_op_f8_debug_stall(calls: int) -> None:
    """The next calls of stage_op_f8_gemm by this thread run out of time (tests of that path)."""
    if _beyond_c_int(calls):
        _invalid("calls outside [0, 16]")
    _opcheck(lib().stage_op_f8_debug_stall(calls))


def stage_op_f8_debug_late(calls: int) -> None:
    """In the next calls of stage_op_f8_gemm by this thread a warp of each SM gives up just before its product comes (tests of that path)."""
    if _beyond_c_int(calls):
        _invalid("calls outside [0, 16]")
    _opcheck(lib().stage_op_f8_debug_late(calls))


def stage_op_rope_freqs(rot_dim: int, theta: float = 10000.0, scaling: int = STAGE_ROPE_PLAIN, factor: float = 1.0,
                        first_len: float = 1.0, low: float = 1.0, high: float = 32.0):
    """(frequencies float64 [rot_dim / 2] on the host, scale) for stage_op_rope."""
    if _beyond_c_int(rot_dim, scaling):
        _invalid("rot_dim or scaling out of range")
    f, scale = np.zeros(max(1, min(rot_dim, 1024) // 2), dtype=np.float64), C.c_float()
    _opcheck(lib().stage_op_rope_freqs(rot_dim, theta, scaling, factor, first_len, low, high, f.ctypes.data_as(C.POINTER(C.c_double)),
                                       C.byref(scale)))
    return f, scale.value


def _heads(t, n_tok: int, d: int, dt: int, dev: int, what: str):
    """(pointer, row stride, heads) of rows [n_tok, heads, d] whose heads lie side by side."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != n_tok or shape[2] != d or _KV4_DTYPE.get(t.dtype) != dt or t.get_device() != dev:
        _invalid(f"{what} must be [{n_tok}, heads, {d}], of q's type and on its device")
    heads = shape[1]
    s0, s1, s2 = t.stride()
    if n_tok and (s2 != 1 or (s1 != d and heads > 1)):
        _invalid(f"the heads of a row of {what} must lie side by side")
    return t.data_ptr(), s0 if n_tok > 1 else heads * d, heads


def stage_op_rope(q, k, pos, freqs, q_out=None, k_out=None, interleaved: bool = False, scale: float = 1.0, stream=None) -> None:
    """Rotary positions of the heads q [n_tok, n_q_heads, head_dim] and k [n_tok, n_k_heads, head_dim] (or None) at pos (int32 [n_tok];
    negative: padding, not written) with freqs (float64 [rot_dim / 2], radians per position), into q_out and k_out (default: in
    place).  Rows may lie apart; the heads of a row lie side by side."""
    torch = _torch or _load_torch()
    shape, dt, dev = q.shape, _KV4_DTYPE.get(q.dtype), q.get_device()
    if len(shape) != 3 or dt is None:
        _invalid("q must be [n_tok, n_q_heads, head_dim], float32, float16 or bfloat16")
    stream = _launch_on(stream, dev)
    n_tok, _, d = shape
    qp, qs, hq = qop, qos, _ = _heads(q, n_tok, d, dt, dev, "q")
    kp = ks = kop = kos = hk = 0
    if q_out is not None:
        qop, qos, h = _heads(q_out, n_tok, d, dt, dev, "q_out")
        if h != hq:
            _invalid("q_out must have q's heads")
    if k is not None:
        kp, ks, hk = kop, kos, _ = _heads(k, n_tok, d, dt, dev, "k")
        if k_out is not None:
            kop, kos, h = _heads(k_out, n_tok, d, dt, dev, "k_out")
            if h != hk:
                _invalid("k_out must have k's heads")
    elif k_out is not None:
        _invalid("k_out without k")
    half = freqs.numel()
    if (n_tok | hq | hk | d | half << 1) >> 31:
        _invalid(_TOO_MANY)
    rc = (_lib or lib()).stage_op_rope(qp, qs, hq, kp, ks, hk, d, dt, _array(pos, torch.int32, n_tok, dev, "pos"), n_tok,
                                       _array(freqs, torch.float64, half, dev, "freqs"), 2 * half, 1 if interleaved else 0, scale, qop,
                                       qos, kop, kos, stream)
    if rc:
        _opcheck(rc)


def stage_op_logprobs(logits, tokens=None, logprob=None, entropy=None, rank=None, top_ids=None, top_logprobs=None, stream=None) -> None:
    """From rows of logits [n, vocab] (which may lie apart): logprob (float32 [n]) and rank (int32 [n]) of tokens (int32 [n]), entropy
    (float32 [n]), and the k likeliest tokens top_ids (int32 [n, k]) with top_logprobs (float32 [n, k]); each may be None."""
    torch = _torch or _load_torch()
    shape, dev = logits.shape, logits.get_device()
    if len(shape) != 2:
        _invalid("logits must be [n, vocab]")
    stream = _launch_on(stream, dev)
    n, vocab = shape
    zp, zt, zs = _matrix(logits, shape, dev, "logits")
    i32, f32 = torch.int32, torch.float32
    tp = lp = ep = rp = ip = bp = None
    if tokens is not None:
        tp = _array(tokens, i32, n, dev, "tokens")
    if logprob is not None:
        lp = _array(logprob, f32, n, dev, "logprob")
    if entropy is not None:
        ep = _array(entropy, f32, n, dev, "entropy")
    if rank is not None:
        rp = _array(rank, i32, n, dev, "rank")
    top = 0
    if top_ids is not None:
        if top_ids.dim() != 2 or top_ids.shape[0] != n:
            _invalid(f"top_ids must be [{n}, k]")
        top = top_ids.shape[1]
        ip = _array(top_ids, i32, n * top, dev, "top_ids")
    if top_logprobs is not None:
        if top_logprobs.dim() != 2 or top_logprobs.shape[0] != n or (top_ids is not None and top_logprobs.shape[1] != top):
            _invalid(f"top_logprobs must be [{n}, k], k that of top_ids")
        top = top_logprobs.shape[1]
        bp = _array(top_logprobs, f32, n * top, dev, "top_logprobs")
    if (n | vocab | top) >> 31:
        _invalid(_TOO_MANY)
    rc = (_lib or lib()).stage_op_logprobs(zp, zt, zs, n, vocab, tp, lp, ep, rp, top, ip, bp, stream)
    if rc:
        _opcheck(rc)
