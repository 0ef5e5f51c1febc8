"""Thin ctypes binding of libmk.so (include/mk.h): argument marshalling only.

Every step of the decode path runs in the library's CUDA kernels; this module
turns torch tensors into device pointers and Python lists into host arrays.
PyTorch is used for device memory and streams only. There is no fallback: if
libmk.so is missing or fails to load, every entry point raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmk.so")

MK_OK, MK_ERR_INVALID, MK_ERR_CUDA, MK_ERR_TIMEOUT, MK_ERR_OOM = 0, 1, 2, 3, 4
OPS = {1: "QKV", 2: "ATTN", 3: "RED", 4: "OPROJ", 5: "GATEUP", 6: "DOWN", 7: "LMHEAD"}
OP_QKV, OP_ATTN, OP_RED, OP_OPROJ, OP_GATEUP, OP_DOWN, OP_LMHEAD = range(1, 8)

# exported entry points (the C-ABI surface declared in include/mk.h)
EXPORTS = ("mk_create", "mk_decode_step", "mk_decode_step_multilaunch", "mk_get_status",
           "mk_destroy", "mk_last_error", "mk_read_counters", "mk_set_timeout",
           "mk_debug_inject_unsatisfiable_wait", "mk_set_trace", "mk_schedule_build",
           "mk_decode_step_noalloc", "mk_debug_use_generic_kernel", "mk_decode_greedy",
           "mk_create_paged", "mk_decode_step_paged", "mk_decode_greedy_persistent",
           "mk_debug_permute_queues", "mk_set_dynamic", "mk_schedule_build_dynamic",
           "mk_schedule_build_steps", "mk_prefill",
           # operators over a KV cache
           "mk_rope_init", "mk_rope_append", "mk_norm_rope_append", "mk_tree_attention",
           "mk_tree_attention_workspace", "mk_prefix_attention", "mk_prefix_attention_workspace",
           "mk_tree_accept", "mk_tree_accept_workspace", "mk_tree_verify", "mk_cache_compact",
           "mk_cache_copy_blocks", "mk_pages_create", "mk_pages_destroy", "mk_pages_resize",
           "mk_pages_fork", "mk_pages_compact", "mk_pages_read")

MAX_STEPS_PER_LAUNCH = 32  # MK_MAX_STEPS_PER_LAUNCH

MAX_GREEDY_STEPS = 1024  # MK_MAX_GREEDY_STEPS


class MkError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"mk error {code}: {msg}")
        self.code = code


class MkConfig(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("hidden", ctypes.c_int), ("n_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int),
                ("vocab", ctypes.c_int), ("tied_embeddings", ctypes.c_int),
                ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float),
                ("batch", ctypes.c_int), ("kv_capacity", ctypes.c_int)]


_vpp = ctypes.POINTER(ctypes.c_void_p)


class MkWeights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("lm_head", ctypes.c_void_p),
                ("final_norm", ctypes.c_void_p), ("attn_norm", _vpp), ("wq", _vpp), ("wk", _vpp),
                ("wv", _vpp), ("wo", _vpp), ("mlp_norm", _vpp), ("wgate", _vpp), ("wup", _vpp),
                ("wdown", _vpp)]


class MkInstr(ctypes.Structure):
    _fields_ = [("op", ctypes.c_int16), ("layer", ctypes.c_int16), ("a0", ctypes.c_int32),
                ("a1", ctypes.c_int32), ("a2", ctypes.c_int32), ("wait_ctr", ctypes.c_int32),
                ("wait_target", ctypes.c_int32), ("sig_ctr", ctypes.c_int32),
                ("sig_amount", ctypes.c_int32)]


class MkCache(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("n_blocks", ctypes.c_int),
                ("block_size", ctypes.c_int), ("batch", ctypes.c_int),
                ("table_entries", ctypes.c_int), ("block_table", ctypes.c_void_p),
                ("k", _vpp), ("v", _vpp)]


class MkRopeConfig(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("rotary_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("scaling", ctypes.c_int),
                ("theta", ctypes.c_double), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("original_length", ctypes.c_int),
                ("magnitude", ctypes.c_float)]


class MkRope(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("rotary_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("magnitude", ctypes.c_float),
                ("turns", ctypes.c_uint64 * 64)]


INSTR_DTYPE = np.dtype([("op", "<i2"), ("layer", "<i2"), ("a0", "<i4"), ("a1", "<i4"),
                        ("a2", "<i4"), ("wait_ctr", "<i4"), ("wait_target", "<i4"),
                        ("sig_ctr", "<i4"), ("sig_amount", "<i4")])
TRACE_DTYPE = np.dtype([("sm", "<u4"), ("index", "<u4"), ("op", "<i4"), ("layer", "<i4"),
                        ("t_start", "<u8"), ("t_ready", "<u8"), ("t_end", "<u8"),
                        ("t_stored", "<u8"), ("res_wait_ns", "<u4"), ("stage_ns", "<u4"),
                        ("t_issue_first", "<u8"), ("t_issue_last", "<u8"),
                        ("page_wait_ns", "<u4"), ("reserved", "<u4")])

_lib = None


def lib():
    """Loads libmk.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run decode_megakernel_03_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32p = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32)
        L.mk_create.argtypes = [ctypes.POINTER(MkConfig), ctypes.POINTER(MkWeights), _vpp, _vpp,
                                ctypes.POINTER(vp)]
        L.mk_decode_step.argtypes = [vp, i32p, i32p, vp, vp]
        L.mk_decode_step_multilaunch.argtypes = [vp, i32p, i32p, vp, vp, ctypes.c_int]
        L.mk_decode_greedy.argtypes = [vp, i32p, i32p, ctypes.c_int, vp, vp, vp]
        L.mk_create_paged.argtypes = [ctypes.POINTER(MkConfig), ctypes.POINTER(MkWeights), _vpp,
                                      _vpp, ctypes.c_int, ctypes.c_int, ctypes.POINTER(vp)]
        L.mk_decode_step_paged.argtypes = [vp, i32p, i32p, i32p, vp, vp]
        L.mk_decode_greedy_persistent.argtypes = [vp, i32p, i32p, ctypes.c_int, vp, vp, vp]
        L.mk_get_status.argtypes = [vp, vp]
        L.mk_destroy.argtypes = [vp]
        L.mk_last_error.argtypes = [vp]
        L.mk_last_error.restype = ctypes.c_char_p
        L.mk_read_counters.argtypes = [vp, i32p, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
        L.mk_set_timeout.argtypes = [vp, ctypes.c_uint64]
        L.mk_debug_inject_unsatisfiable_wait.argtypes = [vp, ctypes.c_int]
        L.mk_debug_use_generic_kernel.argtypes = [vp, ctypes.c_int]
        L.mk_debug_permute_queues.argtypes = [vp, ctypes.c_uint32]
        L.mk_set_dynamic.argtypes = [vp, ctypes.c_int]
        L.mk_prefill.argtypes = [vp, i32p, ctypes.c_int, ctypes.c_int, vp, vp]
        L.mk_schedule_build_steps.argtypes = [ctypes.POINTER(MkConfig), ctypes.c_int, i32p,
                                              ctypes.c_int, ctypes.POINTER(MkInstr),
                                              ctypes.c_int, ctypes.POINTER(ctypes.c_int), i32p,
                                              i32p, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
        L.mk_schedule_build_dynamic.argtypes = [ctypes.POINTER(MkConfig), ctypes.c_int, i32p,
                                                ctypes.c_int, ctypes.POINTER(MkInstr),
                                                ctypes.c_int, ctypes.POINTER(ctypes.c_int), i32p,
                                                i32p, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
        L.mk_set_trace.argtypes = [vp, vp, ctypes.c_int]
        L.mk_schedule_build.argtypes = [ctypes.POINTER(MkConfig), ctypes.c_int, i32p,
                                        ctypes.POINTER(MkInstr), ctypes.c_int,
                                        ctypes.POINTER(ctypes.c_int), i32p, i32p, ctypes.c_int,
                                        ctypes.POINTER(ctypes.c_int)]
        L.mk_decode_step_noalloc.argtypes = [ctypes.POINTER(MkConfig), ctypes.POINTER(MkWeights),
                                             _vpp, _vpp, i32p, i32p, vp, vp, ctypes.c_char_p,
                                             ctypes.c_size_t]
        i, i64, size, sizep = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.POINTER(
            ctypes.c_size_t)
        ip, cachep = ctypes.POINTER(ctypes.c_int), ctypes.POINTER(MkCache)
        L.mk_rope_init.argtypes = [ctypes.POINTER(MkRopeConfig), ctypes.POINTER(MkRope)]
        L.mk_rope_append.argtypes = [ctypes.POINTER(MkRope), cachep, i, i, i, i, i, vp, i64, vp,
                                     i64, vp, i64, vp, i64, vp, vp, vp, vp]
        L.mk_norm_rope_append.argtypes = [ctypes.POINTER(MkRope), vp, vp, ctypes.c_float,
                                          *L.mk_rope_append.argtypes[1:]]
        L.mk_tree_attention.argtypes = [cachep, i, i, i, i, i, ctypes.c_float, vp, i64, vp, vp, vp,
                                        vp, i64, vp, size, vp]
        L.mk_tree_attention_workspace.argtypes = [cachep, i, i, i, i, sizep]
        L.mk_prefix_attention.argtypes = [cachep, i, i, i, i, i, ctypes.c_float, vp, i64, i, vp, vp, vp,
                                          vp, vp, vp, i64, vp, size, vp]
        L.mk_prefix_attention_workspace.argtypes = [cachep, i, i, i, i, i, sizep]
        L.mk_tree_accept.argtypes = [i, i, i, i, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, size, vp]
        L.mk_tree_accept_workspace.argtypes = [i, i, i, sizep]
        L.mk_tree_verify.argtypes = [i, i, i, i, vp, i64, i, vp, i64, vp, vp, vp, vp, vp, vp, i64, vp,
                                     vp, vp, vp]
        L.mk_cache_compact.argtypes = [cachep, i, i, vp, vp, vp, vp]
        L.mk_cache_copy_blocks.argtypes = [cachep, vp, i, vp]
        L.mk_pages_create.argtypes = [i, i, i, i, ctypes.POINTER(vp)]
        L.mk_pages_destroy.argtypes = [vp]
        L.mk_pages_resize.argtypes = [vp, i, vp, vp, vp, i, ip]
        L.mk_pages_fork.argtypes = [vp, i, vp, vp]
        L.mk_pages_compact.argtypes = [vp, vp, i, ip]
        L.mk_pages_read.argtypes = [vp, vp, vp, ip]
        _lib = L
    return _lib


def _err(h) -> str:
    s = lib().mk_last_error(h)
    return s.decode() if s else ""


def _check(rc: int, h=None):
    if rc != MK_OK:
        raise MkError(rc, _err(h))


def make_config(shape, batch: int, capacity: int) -> MkConfig:
    return MkConfig(shape.n_layers, shape.hidden, shape.n_heads, shape.n_kv_heads, shape.head_dim,
                    shape.ffn, shape.vocab, int(bool(shape.tied)), float(shape.rms_eps),
                    float(shape.rope_theta), int(batch), int(capacity))


def _i32(vals, n: int | None = None):
    """A host int32 array of vals; n: the length the library will read."""
    if n is not None and len(vals) != n:
        raise MkError(MK_ERR_INVALID, f"expected {n} values, got {len(vals)}")
    a = (ctypes.c_int32 * len(vals))(*[int(v) for v in vals])
    return a


def _dev(t, n: int, dtype: str, what: str) -> ctypes.c_void_p:
    """The device pointer of tensor t after checking that the library may
    write n elements of dtype there (it cannot check that itself)."""
    if not t.is_cuda or str(t.dtype) != "torch." + dtype or not t.is_contiguous():
        raise MkError(MK_ERR_INVALID, f"{what} must be a contiguous CUDA {dtype} tensor")
    if t.numel() < n:
        raise MkError(MK_ERR_INVALID, f"{what} holds {t.numel()} elements, {n} are written")
    return ctypes.c_void_p(t.data_ptr())


DYN_LMHEAD = 1  # MK_DYN_LMHEAD


def schedule(shape, batch: int, capacity: int, n_sm: int, positions, dyn: int = 0):
    """Host-only schedule: (instrs structured array, sm_offsets, counter targets).
    dyn: MK_DYN_* flags (0: the static plan)."""
    cfg = make_config(shape, batch, capacity)
    n_instr, n_ctr = ctypes.c_int(0), ctypes.c_int(0)
    pos = _i32(positions)
    rc = lib().mk_schedule_build_dynamic(ctypes.byref(cfg), n_sm, pos, int(dyn), None, 0,
                                         ctypes.byref(n_instr), None, None, 0,
                                         ctypes.byref(n_ctr))
    _check(rc)
    instrs = (MkInstr * n_instr.value)()
    offs = (ctypes.c_int32 * (n_sm + 1))()
    tg = (ctypes.c_int32 * n_ctr.value)()
    rc = lib().mk_schedule_build_dynamic(ctypes.byref(cfg), n_sm, pos, int(dyn), instrs,
                                         n_instr.value, ctypes.byref(n_instr), offs, tg,
                                         n_ctr.value, ctypes.byref(n_ctr))
    _check(rc)
    arr = np.frombuffer(bytes(instrs), dtype=INSTR_DTYPE).copy()
    return arr, np.array(offs, dtype=np.int64), np.array(tg, dtype=np.int64)


def schedule_steps(shape, batch: int, capacity: int, n_sm: int, positions, n_steps: int):
    """Host-only schedule of n_steps greedy steps in one launch (the plan of
    mk_decode_greedy_persistent): (instrs, sm_offsets, counter targets)."""
    cfg = make_config(shape, batch, capacity)
    n_instr, n_ctr = ctypes.c_int(0), ctypes.c_int(0)
    pos = _i32(positions)
    rc = lib().mk_schedule_build_steps(ctypes.byref(cfg), n_sm, pos, int(n_steps), None, 0,
                                       ctypes.byref(n_instr), None, None, 0, ctypes.byref(n_ctr))
    _check(rc)
    instrs = (MkInstr * n_instr.value)()
    offs = (ctypes.c_int32 * (n_sm + 1))()
    tg = (ctypes.c_int32 * n_ctr.value)()
    rc = lib().mk_schedule_build_steps(ctypes.byref(cfg), n_sm, pos, int(n_steps), instrs,
                                       n_instr.value, ctypes.byref(n_instr), offs, tg,
                                       n_ctr.value, ctypes.byref(n_ctr))
    _check(rc)
    arr = np.frombuffer(bytes(instrs), dtype=INSTR_DTYPE).copy()
    return arr, np.array(offs, dtype=np.int64), np.array(tg, dtype=np.int64)


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _model_structs(shape, weights: dict, k_cache: list, v_cache: list, batch: int):
    """ctypes mk_config / mk_weights / cache pointer arrays for torch tensors;
    the last element keeps the host arrays alive."""
    L = shape.n_layers
    arrs = {}
    for name in ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm", "wgate", "wup", "wdown"):
        arrs[name] = (ctypes.c_void_p * L)(*[t.data_ptr() for t in weights[name]])
    lm = weights.get("lm_head")
    w = MkWeights(weights["embed"].data_ptr(), lm.data_ptr() if lm is not None else None,
                  weights["final_norm"].data_ptr(),
                  *[ctypes.cast(arrs[n], _vpp) for n in ("attn_norm", "wq", "wk", "wv", "wo",
                                                         "mlp_norm", "wgate", "wup", "wdown")])
    kc = (ctypes.c_void_p * L)(*[t.data_ptr() for t in k_cache])
    vc = (ctypes.c_void_p * L)(*[t.data_ptr() for t in v_cache])
    cfg = make_config(shape, batch, int(k_cache[0].shape[2]))
    return cfg, w, kc, vc, (arrs, weights, k_cache, v_cache)


def decode_step_noalloc(shape, weights: dict, k_cache: list, v_cache: list, batch: int, tokens,
                        positions, logits, stream=None):
    """mk_decode_step_noalloc: one decode step with no handle and no device
    allocation (scratch in the library's static device array). Synchronous.
    Returns (status code, message)."""
    cfg, w, kc, vc, keep = _model_structs(shape, weights, k_cache, v_cache, batch)
    msg = ctypes.create_string_buffer(512)
    rc = lib().mk_decode_step_noalloc(ctypes.byref(cfg), ctypes.byref(w), ctypes.cast(kc, _vpp),
                                      ctypes.cast(vc, _vpp), _i32(tokens, batch),
                                      _i32(positions, batch),
                                      _dev(logits, batch * shape.vocab, "float32", "logits"),
                                      _stream_ptr(stream), msg, len(msg))
    del keep
    return rc, msg.value.decode()


class Decoder:
    """One handle: a model (weights on the device), a batch and its KV cache.

    weights: dict of torch bf16 CUDA tensors as produced by synth.make_weights
    (per-layer lists for the layer matrices); k_cache / v_cache: lists of
    [B][nkv][S][D] bf16 CUDA tensors, updated in place by every step.
    """

    def __init__(self, shape, weights: dict, k_cache: list, v_cache: list, batch: int,
                 paged=None):
        """paged = (block_size, n_blocks, kv_capacity): k_cache / v_cache are
        block pools [n_blocks][nkv][block_size][D] (mk_create_paged), stepped
        with step_paged."""
        self.shape = shape
        self.batch = batch
        self.capacity = int(k_cache[0].shape[2]) if paged is None else int(paged[2])
        # block-table entries per sequence of a paged handle
        self.max_blocks = 0 if paged is None else -(-self.capacity // int(paged[0]))
        L = shape.n_layers
        self._keep = (weights, k_cache, v_cache)
        arrs = {}
        for name in ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm", "wgate", "wup", "wdown"):
            arrs[name] = (ctypes.c_void_p * L)(*[t.data_ptr() for t in weights[name]])
        self._arrs = arrs
        lm = weights.get("lm_head")
        self._w = MkWeights(weights["embed"].data_ptr(), lm.data_ptr() if lm is not None else None,
                            weights["final_norm"].data_ptr(),
                            *[ctypes.cast(arrs[n], _vpp) for n in ("attn_norm", "wq", "wk", "wv",
                                                                   "wo", "mlp_norm", "wgate",
                                                                   "wup", "wdown")])
        self._kc = (ctypes.c_void_p * L)(*[t.data_ptr() for t in k_cache])
        self._vc = (ctypes.c_void_p * L)(*[t.data_ptr() for t in v_cache])
        self.cfg = make_config(shape, batch, self.capacity)
        h = ctypes.c_void_p()
        if paged is None:
            rc = lib().mk_create(ctypes.byref(self.cfg), ctypes.byref(self._w),
                                 ctypes.cast(self._kc, _vpp), ctypes.cast(self._vc, _vpp),
                                 ctypes.byref(h))
        else:
            rc = lib().mk_create_paged(ctypes.byref(self.cfg), ctypes.byref(self._w),
                                       ctypes.cast(self._kc, _vpp), ctypes.cast(self._vc, _vpp),
                                       int(paged[0]), int(paged[1]), ctypes.byref(h))
        _check(rc, None)
        self.h = h

    # -- decode ----------------------------------------------------------
    def _logits(self, logits, rows: int | None = None) -> ctypes.c_void_p:
        n = (self.batch if rows is None else rows) * self.shape.vocab
        return _dev(logits, n, "float32", "logits")

    def _tokens_out(self, t, n_steps: int, most: int) -> ctypes.c_void_p:
        # a step count out of range is refused by the library before it
        # writes anything, so only a valid count sizes the check
        n = n_steps * self.batch if 1 <= n_steps <= most else 0
        return _dev(t, n, "int32", "tokens_out")

    def step(self, tokens, positions, logits, stream=None) -> int:
        rc = lib().mk_decode_step(self.h, _i32(tokens, self.batch), _i32(positions, self.batch),
                                  self._logits(logits), _stream_ptr(stream))
        _check(rc, self.h)
        return rc

    def prefill(self, tokens, start_pos: int, logits, stream=None) -> int:
        """mk_prefill: the prompt into sequence 0 of the cache, in chunks of
        `batch` tokens; logits (device fp32 [vocab]) receives the logits after
        the last prompt token."""
        rc = lib().mk_prefill(self.h, _i32(tokens), len(tokens), int(start_pos),
                              self._logits(logits, 1), _stream_ptr(stream))
        _check(rc, self.h)
        return rc

    def step_paged(self, tokens, positions, block_table, logits, stream=None) -> int:
        """mk_decode_step_paged; block_table: int32 numpy array
        [batch][ceil(kv_capacity / block_size)] on the host."""
        tbl = np.ascontiguousarray(block_table, dtype=np.int32)
        if self.max_blocks and tbl.size != self.batch * self.max_blocks:
            raise MkError(MK_ERR_INVALID, f"block_table must hold batch x {self.max_blocks} entries")
        rc = lib().mk_decode_step_paged(self.h, _i32(tokens, self.batch),
                                        _i32(positions, self.batch),
                                        tbl.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                        self._logits(logits), _stream_ptr(stream))
        _check(rc, self.h)
        return rc

    def decode_greedy(self, tokens, positions, n_steps: int, tokens_out, logits,
                      stream=None) -> int:
        """mk_decode_greedy: n_steps greedy steps, the tokens fed back on the
        device; tokens_out is a device int32 tensor of n_steps * batch."""
        rc = lib().mk_decode_greedy(self.h, _i32(tokens, self.batch), _i32(positions, self.batch),
                                    int(n_steps), self._tokens_out(tokens_out, n_steps,
                                                                   MAX_GREEDY_STEPS),
                                    self._logits(logits), _stream_ptr(stream))
        _check(rc, self.h)
        return rc

    def decode_greedy_persistent(self, tokens, positions, n_steps: int, tokens_out, logits,
                                 stream=None) -> int:
        """mk_decode_greedy_persistent: n_steps greedy steps in one launch."""
        rc = lib().mk_decode_greedy_persistent(
            self.h, _i32(tokens, self.batch), _i32(positions, self.batch), int(n_steps),
            self._tokens_out(tokens_out, n_steps, MAX_STEPS_PER_LAUNCH), self._logits(logits),
            _stream_ptr(stream))
        _check(rc, self.h)
        return rc

    def step_multilaunch(self, tokens, positions, logits, stream=None, graph: bool = False) -> int:
        rc = lib().mk_decode_step_multilaunch(self.h, _i32(tokens, self.batch),
                                              _i32(positions, self.batch), self._logits(logits),
                                              _stream_ptr(stream), int(bool(graph)))
        _check(rc, self.h)
        return rc

    def status(self, stream=None) -> int:
        """mk_get_status: returns the code (does not raise on MK_ERR_TIMEOUT)."""
        return lib().mk_get_status(self.h, _stream_ptr(stream))

    def counters(self) -> np.ndarray:
        n = ctypes.c_int(0)
        lib().mk_read_counters(self.h, None, 0, ctypes.byref(n))
        buf = (ctypes.c_int32 * n.value)()
        _check(lib().mk_read_counters(self.h, buf, n.value, ctypes.byref(n)), self.h)
        return np.array(buf, dtype=np.int64)

    def set_timeout(self, ns: int):
        _check(lib().mk_set_timeout(self.h, int(ns)), self.h)

    def use_generic_kernel(self, enable: bool):
        """Test hook: launch the instantiation that reads the head shape at run time."""
        _check(lib().mk_debug_use_generic_kernel(self.h, int(bool(enable))), self.h)

    def set_dynamic(self, flags: int):
        """mk_set_dynamic: MK_DYN_* flags (0: the static plan)."""
        _check(lib().mk_set_dynamic(self.h, int(flags)), self.h)

    def permute_queues(self, seed: int):
        """Test hook: hand the per-SM queues to the CTAs in a seeded order."""
        _check(lib().mk_debug_permute_queues(self.h, int(seed)), self.h)

    def inject_unsatisfiable_wait(self, enable: bool):
        _check(lib().mk_debug_inject_unsatisfiable_wait(self.h, int(bool(enable))), self.h)

    def set_trace(self, buf=None):
        """buf: a torch uint8 CUDA tensor of n * TRACE_DTYPE.itemsize bytes, or
        None to disable."""
        if buf is None:
            _check(lib().mk_set_trace(self.h, None, 0), self.h)
        else:
            _check(lib().mk_set_trace(self.h, ctypes.c_void_p(buf.data_ptr()),
                                      buf.numel() // TRACE_DTYPE.itemsize), self.h)

    def last_error(self) -> str:
        return _err(self.h)

    def close(self):
        if getattr(self, "h", None):
            lib().mk_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- operators over a KV cache -------------------------------------------------------

MAX_TREE = 64  # MK_MAX_TREE
TYPE_BF16, TYPE_FP32 = 0, 1
ROPE_SCALINGS = {"none": 0, "linear": 1, "bands": 2, "yarn": 3}  # MK_ROPE_*


def _bad(msg: str) -> MkError:
    return MkError(MK_ERR_INVALID, msg)


class Cache:
    """A model's KV cache as the operators see it (mk_cache).

    k, v: each layer's bf16 CUDA tensor, contiguous: caches [B][nkv][S][D], or
    block pools [n_blocks][nkv][block_size][D] with block_table, a contiguous
    int32 CUDA tensor [batch][entries]. The tensors are updated in place; the
    table may be rewritten between calls (in stream order).
    """

    def __init__(self, k: list, v: list, block_table=None):
        _use_torch()
        k, v = list(k), list(v)
        if not k or len(k) != len(v):
            raise _bad("k and v must hold a tensor for each layer")
        shape, device = k[0].shape, k[0].device
        if device.type != "cuda" or len(shape) != 4:
            raise _bad("k and v must be CUDA tensors [blocks][nkv][block_size][D]")
        for t in k + v:
            if (t.dtype != torch.bfloat16 or t.shape != shape or t.device != device
                    or not t.is_contiguous()):
                raise _bad("k and v must be contiguous bfloat16 tensors, alike in every layer")
        self.n_layers = len(k)
        self.n_blocks, self.n_kv_heads, self.block_size, self.head_dim = map(int, shape)
        self.device = device
        self.batch, entries, ptr = self.n_blocks, 0, None
        if block_table is not None:
            # (an empty table has no pointer, which would read as a contiguous cache)
            if len(block_table.shape) != 2 or 0 in block_table.shape:
                raise _bad("block_table must be [batch][entries], at least one of each")
            ptr = _ints(block_table, self.device, "block_table", block_table.shape)
            self.batch, entries = map(int, block_table.shape)
        self.k, self.v, self.block_table = k, v, block_table
        n = self.n_layers
        self._k = (ctypes.c_void_p * n)(*[t.data_ptr() for t in k])
        self._v = (ctypes.c_void_p * n)(*[t.data_ptr() for t in v])
        self.struct = MkCache(n, self.n_kv_heads, self.head_dim, self.n_blocks, self.block_size,
                              self.batch, entries, ptr, ctypes.cast(self._k, _vpp),
                              ctypes.cast(self._v, _vpp))
        self.ref = ctypes.byref(self.struct)
        self.workspaces = {}  # bytes of workspace by call shape


class Rope:
    """A plan of rotary positions (mk_rope_init). rotary_dim: the head's first
    dimensions that turn (default: all); interleaved: pairs (2i, 2i + 1)
    instead of (i, i + rotary_dim / 2); scaling: "none", "linear", "bands" or
    "yarn"; magnitude None: 1, or 0.1 ln(factor) + 1 for "yarn"."""

    def __init__(self, head_dim: int, theta: float = 10000.0, rotary_dim: int | None = None,
                 interleaved: bool = False, scaling: str = "none", factor: float = 1.0,
                 low: float = 1.0, high: float = 4.0, original_length: int = 0,
                 magnitude: float | None = None):
        if scaling not in ROPE_SCALINGS:
            raise _bad(f"scaling must be one of {', '.join(ROPE_SCALINGS)}")
        if magnitude is not None and not magnitude > 0:
            raise _bad("magnitude must be positive")
        cfg = MkRopeConfig(head_dim, head_dim if rotary_dim is None else rotary_dim,
                           int(bool(interleaved)), ROPE_SCALINGS[scaling], theta, factor, low,
                           high, original_length, magnitude or 0.0)
        self.struct = MkRope()
        self.ref = ctypes.byref(self.struct)
        _check(lib().mk_rope_init(ctypes.byref(cfg), self.ref))


torch = None  # see _use_torch


def _use_torch():
    """Imports torch where the first tensor comes in (schedules, page tables and
    rotary plans need none)."""
    global torch, _TYPES, _current_raw, _current_device
    if torch is not None:
        return
    import torch as t
    _TYPES = {t.bfloat16: TYPE_BF16, t.float32: TYPE_FP32}
    # the current stream's handle and device without making objects (a few
    # microseconds less per call), where this torch has the short ways
    _current_raw = getattr(t._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: t.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(t._C, "_cuda_getDevice", None) or t.cuda.current_device
    torch = t


def _elsewhere(device, stream):
    """None where a call on `device` can launch at once on the current stream;
    else a context that makes the device (and the stream) current, inside which
    the call starts again: its launch, and the tensors that it allocates,
    belong to that stream then."""
    if stream is None:
        return None if _current_device() == device.index else torch.cuda.device(device)
    if stream.device != device:
        raise _bad("stream and tensors are on different devices")
    return torch.cuda.stream(stream)


def _ints(t, device, what: str, shape):
    """The pointer of an int32 index tensor (contiguous, on `device`)."""
    if t is None:
        return None
    if getattr(t, "dtype", None) != torch.int32 or t.device != device or not t.is_contiguous():
        raise _bad(f"{what} must be a contiguous int32 tensor on {device}")
    if t.shape != shape:
        raise _bad(f"{what} has the shape {tuple(t.shape)}, not {shape}")
    return t.data_ptr()


def _type_of(t, what: str) -> int:
    kind = _TYPES.get(getattr(t, "dtype", None))
    if kind is None:
        raise _bad(f"{what} must be bfloat16 or float32")
    return kind


def _queries(q, cache) -> tuple:
    """(shape, type, row stride) of q [B][T][nh][D]."""
    shape = getattr(q, "shape", ())
    if len(shape) != 4 or shape[3] != cache.head_dim:
        raise _bad("q must be [batch][tokens][heads][head_dim], the cache's head_dim")
    return shape, _type_of(q, "q"), _heads(q, shape, q.dtype, cache.device, "q")


def _heads(t, shape, dtype, device, what: str) -> int:
    """The row stride of t [B][T][heads][D]: heads packed, rows evenly spaced."""
    if getattr(t, "dtype", None) != dtype or t.device != device or t.shape != shape:
        has = f"{t.dtype} {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor) else repr(t)
        raise _bad(f"{what} must be a {dtype} tensor of the shape {tuple(shape)} on {device}, not {has}")
    b, n, h, d = shape
    sb, sn, sh, sd = t.stride()
    if sd != 1 or (h > 1 and sh != d):
        raise _bad(f"{what}: a row's heads must be packed")
    if n == 1:
        return sb if b > 1 else h * d
    if b > 1 and sb != n * sn:
        raise _bad(f"{what}: rows must be evenly spaced over batch and tokens")
    return sn


def _new(shape, dtype, device, zero: bool):
    return (torch.zeros if zero else torch.empty)(shape, dtype=dtype, device=device)


def _rope_args(cache: Cache, q, k, v, starts, parents, counts, q_out):
    """What the calls of the library share from n_tokens on, up to the stream; q_out."""
    dev = cache.device
    shape, kind, qs = _queries(q, cache)
    b, n, nh, d = shape
    kv, dtype = (b, n, cache.n_kv_heads, d), q.dtype
    ks, vs = _heads(k, kv, dtype, dev, "k"), _heads(v, kv, dtype, dev, "v")
    sp = _ints(starts, dev, "starts", (b,))
    pp, cp = _ints(parents, dev, "parents", (b, n)), _ints(counts, dev, "counts", (b,))
    if q_out is None:
        q_out, os_ = _new(shape, dtype, dev, counts is not None), nh * d
    else:
        os_ = _heads(q_out, shape, dtype, dev, "q_out")
    return (b, n, nh, kind, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
            q_out.data_ptr(), os_, sp, pp, cp, _current_raw(dev.index)), q_out


def rope_append(rope: Rope, cache: Cache, layer: int, q, k, v, starts, parents=None, counts=None,
                q_out=None, stream=None):
    """mk_rope_append: q [B][T][nh][D], k, v [B][T][nkv][D] (bf16 or fp32; views
    into a fused projection's rows are fine), starts [B], parents [B][T],
    counts [B] int32, all on the device. Returns the rotated queries (q_out,
    which may be q; else a new tensor, whose rows behind counts are 0)."""
    if (other := _elsewhere(cache.device, stream)) is not None:
        with other:
            return rope_append(rope, cache, layer, q, k, v, starts, parents, counts, q_out)
    args, q_out = _rope_args(cache, q, k, v, starts, parents, counts, q_out)
    _check(lib().mk_rope_append(rope.ref, cache.ref, layer, *args))
    return q_out


def _norm_weights(t, cache: Cache, what: str):
    if t is None:
        return None
    if getattr(t, "dtype", None) != torch.bfloat16 or t.device != cache.device or not t.is_contiguous():
        raise _bad(f"{what} must be a contiguous bfloat16 tensor on {cache.device}")
    if t.shape != (cache.head_dim,):
        raise _bad(f"{what} has the shape {tuple(t.shape)}, not {(cache.head_dim,)}")
    return t.data_ptr()


def norm_rope_append(rope: Rope, cache: Cache, layer: int, q, k, v, q_norm, k_norm, starts,
                     parents=None, counts=None, eps: float = 1e-6, q_out=None, stream=None):
    """mk_norm_rope_append: rope_append of queries and keys whose heads are first
    divided by their root mean square and multiplied by q_norm, k_norm (bf16 [D]
    on the device; None: ones)."""
    if (other := _elsewhere(cache.device, stream)) is not None:
        with other:
            return norm_rope_append(rope, cache, layer, q, k, v, q_norm, k_norm, starts, parents,
                                    counts, eps, q_out)
    qn, kn = _norm_weights(q_norm, cache, "q_norm"), _norm_weights(k_norm, cache, "k_norm")
    args, q_out = _rope_args(cache, q, k, v, starts, parents, counts, q_out)
    _check(lib().mk_norm_rope_append(rope.ref, qn, kn, eps, cache.ref, layer, *args))
    return q_out


def tree_attention(cache: Cache, layer: int, q, starts, parents=None, counts=None, scale=None,
                   out=None, stream=None):
    """mk_tree_attention: q [B][T][nh][D] (bf16 or fp32) over `layer` of the
    cache, whose slots starts[b] + t hold the nodes' rows. scale None:
    1 / sqrt(D). Returns out (given, or new; new rows behind counts are 0). The
    workspace is allocated for the call on its stream."""
    dev = cache.device
    if (other := _elsewhere(dev, stream)) is not None:
        with other:
            return tree_attention(cache, layer, q, starts, parents, counts, scale, out)
    shape, kind, qs = _queries(q, cache)
    b, n, nh, d = shape
    sp = _ints(starts, dev, "starts", (b,))
    pp, cp = _ints(parents, dev, "parents", (b, n)), _ints(counts, dev, "counts", (b,))
    size = cache.workspaces.get((b, n, nh, kind))
    if size is None:
        need = ctypes.c_size_t()
        _check(lib().mk_tree_attention_workspace(cache.ref, b, n, nh, kind, ctypes.byref(need)))
        size = cache.workspaces[b, n, nh, kind] = need.value
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    if out is None:
        out, os_ = _new(shape, q.dtype, dev, counts is not None), nh * d
    else:
        os_ = _heads(out, shape, q.dtype, dev, "out")
    _check(lib().mk_tree_attention(cache.ref, layer, b, n, nh, kind,
                                   d ** -0.5 if scale is None else scale, q.data_ptr(), qs, sp, pp,
                                   cp, out.data_ptr(), os_, ws.data_ptr(), size,
                                   _current_raw(dev.index)))
    return out


def prefix_attention(cache: Cache, layer: int, q, first, prefix, starts, parents=None, counts=None,
                     scale=None, out=None, stream=None):
    """mk_prefix_attention: tree_attention of a batch whose groups share a prefix.
    first, prefix [n_groups] int32 on the device: each group's first sequence, and how
    many of its slots the group shares (the first sequence's rows are read)."""
    dev = cache.device
    if (other := _elsewhere(dev, stream)) is not None:
        with other:
            return prefix_attention(cache, layer, q, first, prefix, starts, parents, counts, scale, out)
    shape, kind, qs = _queries(q, cache)
    b, n, nh, d = shape
    if len(getattr(first, "shape", ())) != 1:
        raise _bad("first must be a tensor [groups]")
    groups = first.shape[0]
    fp, xp = _ints(first, dev, "first", (groups,)), _ints(prefix, dev, "prefix", (groups,))
    sp = _ints(starts, dev, "starts", (b,))
    pp, cp = _ints(parents, dev, "parents", (b, n)), _ints(counts, dev, "counts", (b,))
    size = cache.workspaces.get((b, n, nh, kind, groups))
    if size is None:
        need = ctypes.c_size_t()
        _check(lib().mk_prefix_attention_workspace(cache.ref, b, n, nh, kind, groups,
                                                   ctypes.byref(need)))
        size = cache.workspaces[b, n, nh, kind, groups] = need.value
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    if out is None:
        out, os_ = _new(shape, q.dtype, dev, counts is not None), nh * d
    else:
        os_ = _heads(out, shape, q.dtype, dev, "out")
    _check(lib().mk_prefix_attention(cache.ref, layer, b, n, nh, kind,
                                     d ** -0.5 if scale is None else scale, q.data_ptr(), qs, groups,
                                     fp, xp, sp, pp, cp, out.data_ptr(), os_, ws.data_ptr(), size,
                                     _current_raw(dev.index)))
    return out


def _logits(t) -> tuple:
    """(device, shape) of logits [B][T][V]."""
    if not getattr(t, "is_cuda", False) or len(t.shape) != 3:
        raise _bad("logits must be a CUDA tensor [batch][tokens][vocab]")
    return t.device, t.shape


def _rows(t, shape, what: str) -> int:
    """The row stride of t [B][T][V]: rows packed and evenly spaced."""
    b, n, vocab = shape
    sb, sn, sv = t.stride()
    if (vocab > 1 and sv != 1) or (n > 1 and b > 1 and sb != n * sn):
        raise _bad(f"{what}: rows must be packed and evenly spaced")
    return (sb if b > 1 else vocab) if n == 1 else sn


def tree_accept(logits, tokens, parents=None, counts=None, stream=None):
    """mk_tree_accept: logits [B][T][V] (bf16 or fp32), tokens [B][T] int32.
    Returns int32 (choices [B][T], path [B][T], accepted [B], next [B])."""
    _use_torch()
    dev, shape = _logits(logits)
    if (other := _elsewhere(dev, stream)) is not None:
        with other:
            return tree_accept(logits, tokens, parents, counts)
    kind = _type_of(logits, "logits")
    b, n, vocab = shape
    stride = _rows(logits, shape, "logits")
    tp = _ints(tokens, dev, "tokens", (b, n))
    pp, cp = _ints(parents, dev, "parents", (b, n)), _ints(counts, dev, "counts", (b,))
    need = ctypes.c_size_t()
    _check(lib().mk_tree_accept_workspace(b, n, vocab, ctypes.byref(need)))
    # one allocation: the workspace (tens of KB), then the outputs behind it
    first, rows = -(-need.value // 4), b * n
    buf = torch.empty(first + 2 * rows + 2 * b, dtype=torch.int32, device=dev)
    ws = buf.data_ptr()
    at = ws + 4 * first
    _check(lib().mk_tree_accept(b, n, vocab, kind, logits.data_ptr(), stride, tp, pp, cp, at,
                                at + 4 * rows, at + 8 * rows, at + 8 * rows + 4 * b, ws,
                                need.value, _current_raw(dev.index)))
    last = first + 2 * rows
    return (buf.as_strided((b, n), (n, 1), first), buf.as_strided((b, n), (n, 1), first + rows),
            buf.as_strided((b,), (1,), last), buf.as_strided((b,), (1,), last + b))


def _floats(t, device, what: str, shape):
    """The pointer of an fp32 tensor (contiguous, on `device`)."""
    if t is None:
        return None
    if (getattr(t, "dtype", None) != torch.float32 or t.device != device
            or not t.is_contiguous()):
        raise _bad(f"{what} must be a contiguous float32 tensor on {device}")
    if t.shape != shape:
        raise _bad(f"{what} has the shape {tuple(t.shape)}, not {shape}")
    return t.data_ptr()


def tree_verify(logits, tokens, uniform, noise, parents=None, counts=None, draft=None,
                temperature=None, stream=None):
    """mk_tree_verify: logits [B][T][V] (bf16 or fp32), tokens [B][T] int32,
    uniform [B][T] fp32 in [0, 1), noise [B][V] fp32 (exponential, mean 1; its rows
    packed); draft [B][T][V] (bf16 or fp32) the distributions that each node's children
    were sampled from, or None; temperature [B] fp32. Returns int32 (path [B][T],
    accepted [B], next [B])."""
    _use_torch()
    dev, shape = _logits(logits)
    if (other := _elsewhere(dev, stream)) is not None:
        with other:
            return tree_verify(logits, tokens, uniform, noise, parents, counts, draft, temperature)
    kind = _type_of(logits, "logits")
    b, n, vocab = shape
    stride = _rows(logits, shape, "logits")
    draft_kind, draft_at, draft_stride = 0, None, 0
    if draft is not None:
        if getattr(draft, "device", None) != dev or draft.shape != shape:
            raise _bad(f"draft must be a tensor of the shape {tuple(shape)} on {dev}")
        draft_kind, draft_stride = _type_of(draft, "draft"), _rows(draft, shape, "draft")
        draft_at = draft.data_ptr()
    if getattr(noise, "dtype", None) != torch.float32 or noise.device != dev or noise.shape != (b, vocab) or (
            vocab > 1 and noise.stride(1) != 1):
        raise _bad(f"noise must be a float32 tensor of the shape {(b, vocab)} on {dev}, its rows packed")
    tp, up = _ints(tokens, dev, "tokens", (b, n)), _floats(uniform, dev, "uniform", (b, n))
    pp, cp = _ints(parents, dev, "parents", (b, n)), _ints(counts, dev, "counts", (b,))
    hp = _floats(temperature, dev, "temperature", (b,))
    rows = b * n
    buf = torch.empty(rows + 2 * b, dtype=torch.int32, device=dev)
    at = buf.data_ptr()
    _check(lib().mk_tree_verify(b, n, vocab, kind, logits.data_ptr(), stride, draft_kind, draft_at,
                                draft_stride, hp, tp, pp, cp, up, noise.data_ptr(),
                                noise.stride(0) if b > 1 else vocab, at, at + 4 * rows,
                                at + 4 * rows + 4 * b, _current_raw(dev.index)))
    return (buf.as_strided((b, n), (n, 1), 0), buf.as_strided((b,), (1,), rows),
            buf.as_strided((b,), (1,), rows + b))


def cache_compact(cache: Cache, starts, path, accepted, stream=None):
    """mk_cache_compact: the accepted nodes' rows moved down behind the context
    in every layer; starts [B], path [B][T], accepted [B] as tree_accept gives
    them."""
    dev = cache.device
    if (other := _elsewhere(dev, stream)) is not None:
        with other:
            return cache_compact(cache, starts, path, accepted)
    if len(getattr(path, "shape", ())) != 2:
        raise _bad("path must be [batch][tokens]")
    b, n = path.shape
    sp = _ints(starts, dev, "starts", (b,))
    pp, ap = _ints(path, dev, "path", (b, n)), _ints(accepted, dev, "accepted", (b,))
    _check(lib().mk_cache_compact(cache.ref, b, n, sp, pp, ap, _current_raw(dev.index)))


def _host_ints(x) -> np.ndarray:
    """A contiguous host int32 array of x (whole numbers only)."""
    if type(x) is np.ndarray and x.dtype == np.int32 and x.flags.c_contiguous:
        return x
    a = np.asarray(x)
    if a.dtype != np.int32:
        if a.size and (a.dtype.kind not in "iu" or a.min() < -2**31 or a.max() >= 2**31):
            raise _bad("host arrays must hold 32-bit whole numbers")
        a = a.astype(np.int32)
    return np.ascontiguousarray(a)


def _at(a: np.ndarray) -> int:
    return a.__array_interface__["data"][0]


def cache_copy_blocks(cache: Cache, copies, stream=None):
    """mk_cache_copy_blocks: copies [n][3] on the host, (src, dst, rows) each, as
    the calls of Pages return them."""
    if (other := _elsewhere(cache.device, stream)) is not None:
        with other:
            return cache_copy_blocks(cache, copies)
    c = _host_ints(copies)
    if c.size and (c.ndim != 2 or c.shape[1] != 3):
        raise _bad("copies must be [n][3]")
    _check(lib().mk_cache_copy_blocks(cache.ref, _at(c), c.size // 3,
                                      _current_raw(cache.device.index)))


class Pages:
    """The page tables of a paged cache, on the host (mk_pages_*): which blocks
    each of n_seqs sequences holds. resize and compact return the copies
    ([n][3] int32) that cache_copy_blocks has to make, one call for each result
    and in order, before the pages are written; table() is what Decoder.step_paged takes."""

    def __init__(self, n_blocks: int, block_size: int, n_seqs: int, kv_capacity: int):
        self.h = ctypes.c_void_p()
        self.n_blocks, self.n_seqs = n_blocks, n_seqs
        _check(lib().mk_pages_create(n_blocks, block_size, n_seqs, kv_capacity,
                                     ctypes.byref(self.h)))
        self.entries = -(-kv_capacity // block_size)

    @staticmethod
    def _pair(a, b, what: str):
        a, b = _host_ints(a), _host_ints(b)
        if a.size != b.size:
            raise _bad(f"{what} must be two lists of the same length")
        return a, b

    def resize(self, seqs, lengths) -> np.ndarray:
        """mk_pages_resize (0: gives a sequence's pages back)."""
        s, n = self._pair(seqs, lengths, "seqs, lengths")
        copies, made = np.empty((s.size, 3), np.int32), ctypes.c_int()
        _check(lib().mk_pages_resize(self.h, s.size, _at(s), _at(n), _at(copies), s.size,
                                     ctypes.byref(made)))
        return copies[:made.value]

    def fork(self, parents, children):
        """mk_pages_fork: each empty child becomes a fork of its parent."""
        p, c = self._pair(parents, children, "parents, children")
        _check(lib().mk_pages_fork(self.h, p.size, _at(p), _at(c)))

    def compact(self) -> np.ndarray:
        """mk_pages_compact: the pages in use renumbered to the lowest ones."""
        copies, made = np.empty((self.n_blocks, 3), np.int32), ctypes.c_int()
        _check(lib().mk_pages_compact(self.h, _at(copies), self.n_blocks, ctypes.byref(made)))
        return copies[:made.value]

    def table(self) -> np.ndarray:
        """[n_seqs][entries] int32, -1 behind a sequence's pages."""
        t = np.empty((self.n_seqs, self.entries), np.int32)
        _check(lib().mk_pages_read(self.h, _at(t), None, None))
        return t

    def lengths(self) -> np.ndarray:
        n = np.empty(self.n_seqs, np.int32)
        _check(lib().mk_pages_read(self.h, None, _at(n), None))
        return n

    def n_free(self) -> int:
        n = ctypes.c_int()
        _check(lib().mk_pages_read(self.h, None, None, ctypes.byref(n)))
        return n.value

    def close(self):
        if getattr(self, "h", None):
            lib().mk_pages_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
