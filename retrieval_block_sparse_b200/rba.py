"""Python binding of librba.so (include/rba.h): argument marshalling only.

Every computation runs in the CUDA library.  torch supplies device memory
(caller-owned pools, outputs, workspaces) and the current CUDA stream.  If
the library is missing the calls raise; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "librba.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_BOUNDS = range(7)
F32, BF16 = 0, 1
MODES = {"mean": 0, "topr_attn": 1, "external": 2, "embed_cosine": 3, "identity": 4}
SCORE_REDUCE = {"sum": 0, "max": 1}

_c_i32, _c_i64, _c_f32, _c_size, _p = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                        ctypes.c_size_t, ctypes.c_void_p)

# name -> (restype, argtypes), mirroring include/rba.h
SIGNATURES = {
    "rba_store_create": (_c_i32, [_p, _p, _p, _p, _p, _p, ctypes.POINTER(_p)]),
    "rba_store_destroy": (_c_i32, [_p]),
    "rba_store_set_score_reduce": (_c_i32, [_p, _c_i32]),
    "rba_store_set_wait_limit_ns": (_c_i32, [_p, ctypes.c_uint64]),
    "rba_store_set_decode_step_one_launch": (_c_i32, [_p, _c_i32]),
    "rba_candidates": (_c_i32, [_p, _c_i64, _c_i32, _c_i32, ctypes.POINTER(_c_i32),
                                ctypes.POINTER(_c_i32)]),
    "rba_memorize": (_c_i32, [_p, _p, _p, _c_i64, _c_i32, _p, _c_i32, _c_f32, _p]),
    "rba_score": (_c_i32, [_p, _p, _c_i32, _c_i64, _c_i32, _c_i32, _p, _p, _p]),
    "rba_topk": (_c_i32, [_p, _c_i32, _c_i32, _c_i32, _c_i32, _p, _p, _c_size, _p]),
    "rba_topk_workspace_size": (_c_size, [_c_i32, _c_i32, _c_i32]),
    "rba_attend": (_c_i32, [_p, _p, _p, _c_i32, _c_i64, _c_i32, _c_i32, _c_f32, _p, _p, _p,
                            _c_size, _p]),
    "rba_attend_workspace_size": (_c_size, [_p, _c_i32, _c_i64, _c_i32, _c_i32]),
    "rba_attend_noalloc": (_c_i32, [_p, _p, _p, _c_i32, _c_i64, _c_i32, _c_i32, _c_f32, _p, _p,
                                    _p]),
    "rba_attend_landmark_gated": (_c_i32, [_p, _p, _p, _c_i32, _c_i64, _c_i32, _c_i32, _c_f32,
                                           _p, _p, _p]),
    "rba_attend_prefill": (_c_i32, [_p, _p, _c_i32, _c_i32, _p, _c_i32, _c_i32, _c_i64, _c_i32,
                                    _c_i32, _p, _p, _c_f32, _p, _p, _p, _c_size, _p]),
    "rba_attend_prefill_workspace_size": (_c_size, [_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i64,
                                                    _c_i32, _c_i32]),
    "rba_decode_step": (_c_i32, [_p, _p, _c_i32, _c_i64, _c_i32, _c_i32, _c_f32, _p, _p, _p, _p,
                                 _p, _c_size, _p]),
    "rba_decode_step_workspace_size": (_c_size, [_p, _c_i32, _c_i64, _c_i32, _c_i32]),
    "rba_decode_step_plan": (_c_i32, [_p, _c_i32, _c_i64, _c_i32, _c_i32]),
    "rba_decode_step_launches": (_c_i32, [_p, _c_i32, _c_i64, _c_i32, _c_i32]),
    "rba_stream_step": (_c_i32, [_p, _p, _p, _p, _c_i64, _c_i32, _c_i32, _c_i32, _c_f32, _p,
                                 _c_i32, _p, _p, _p, ctypes.POINTER(_c_i32), _p, _c_size, _p]),
    "rba_group_means": (_c_i32, [_p, _c_i64, _c_i32, _c_i32, _p, _p]),
    "rba_approx_select": (_c_i32, [_p, _p, _c_i64, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _p,
                                   _p, _p, _p, _p, _c_size, _p]),
    "rba_approx_select_workspace_size": (_c_size, [_p, _c_i64, _c_i32, _c_i32, _c_i32, _c_i32,
                                                   _c_i32]),
    "rba_memory_rule": (_c_i32, [_c_i64, ctypes.POINTER(_c_i64), ctypes.POINTER(_c_i64),
                                 ctypes.POINTER(_c_i64)]),
    "rba_memory_units": (_c_i32, [_p]),
    "rba_count_retrievals": (_c_i32, [_p, _p, _c_i32, _c_i32, _p, _p]),
    "rba_memory_update": (_c_i32, [_p, _c_i64, _c_i32, _c_i64, _c_i64, _c_i64, _p, _p,
                                   ctypes.POINTER(_c_i64), _p]),
    "rba_decode_step_host": (_c_i32, [_p, _p, _p, _c_i32, _c_i64, _c_i32, _c_i32, _c_f32, _p, _p,
                                      _p, _p, _p, _p, _p, _c_size, _p]),
    "rba_paged_create": (_c_i32, [_p, _p, ctypes.POINTER(_p)]),
    "rba_paged_destroy": (_c_i32, [_p]),
    "rba_paged_strip_bytes": (_c_i32, [_c_i32]),
    "rba_paged_extend": (_c_i32, [_p, _p, _c_i32, _p, _c_i32, _p, _p]),
    "rba_paged_truncate": (_c_i32, [_p, _p, _c_i32, _p]),
    "rba_paged_append": (_c_i32, [_p, _p, _c_i32, _p, _c_i64, _c_i64, _p, _c_i64, _c_i64, _p]),
    "rba_paged_read": (_c_i32, [_p, _p, _c_i32, _p, _p, _p]),
    "rba_paged_select": (_c_i32, [_p, _p, _c_i64, _c_i64, _c_i32, _c_i32, _c_i32, _c_i32, _p, _p,
                                  _c_size, _p]),
    "rba_paged_select_workspace_size": (_c_size, [_p]),
    "rba_paged_attend": (_c_i32, [_p, _p, _c_i64, _c_i64, _c_i32, _p, _c_i32, _c_i32, _c_i32,
                                  _c_f32, _p, _p, _p, _c_size, _p]),
    "rba_paged_attend_workspace_size": (_c_size, [_p]),
    "rba_paged_step_check": (_c_i32, [_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _p, _c_size, _p,
                                      _c_size]),
    "rba_paged_check": (_c_i32, [_p, _p]),
    "rba_store_check": (_c_i32, [_p, _p]),
    "rba_row_pitch": (_c_i32, [_c_i32]),
    "rba_status_string": (ctypes.c_char_p, [_c_i32]),
    "rba_version": (_c_i32, []),
}

_LIB = None


class RbaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """Loads librba.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m retrieval_block_sparse_b200.build`"
                " (the CUDA library is required; there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def status_string(s: int) -> str:
    return lib().rba_status_string(s).decode()


def _check(s: int, where: str):
    if s != OK:
        raise RbaError(s, where)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _tdtype(dtype: int):
    return torch.bfloat16 if dtype == BF16 else torch.float32


class _Desc(ctypes.Structure):
    _fields_ = [("batch", _c_i32), ("n_q_heads", _c_i32), ("n_kv_heads", _c_i32),
                ("head_dim", _c_i32), ("block_size", _c_i32), ("n_rep", _c_i32),
                ("d_ret", _c_i32), ("capacity_tokens", _c_i64), ("dtype", _c_i32),
                ("mode", _c_i32)]


class Store:
    """A block store: caller-owned device pools described to the library.

    Pools (allocated here with torch, owned by this object), rows of P =
    rba_row_pitch(D) elements (P = D for D = 64 or 128; else the first D are
    the row and the rest stay zero -- write rows through `kv_rows`):
      k, v     [B][Hkv][capacity][P]         store dtype
      rep      mean: fp32 [B][Hkv][cap_blocks][1][P]; topr_attn / external:
               dtype [B][Hkv][cap_blocks][r][P]; embed_cosine: fp32
               [B][cap_blocks][d_ret]; identity: none
      rep_pos  int32 [B][Hkv][cap_blocks][r] (topr_attn)
      status   int32[4] device status word
    score_reduce: "sum" (default) or "max" -- how a block's r representative
    keys combine into its score (rba_store_set_score_reduce).
    """

    def __init__(self, *, batch, n_q_heads, n_kv_heads, head_dim, block_size, capacity_tokens,
                 dtype="bf16", mode="mean", n_rep=1, d_ret=0, device="cuda", score_reduce="sum"):
        self.dtype = BF16 if dtype in ("bf16", torch.bfloat16) else F32
        self.mode = mode
        self.B, self.Hq, self.Hkv, self.D = batch, n_q_heads, n_kv_heads, head_dim
        self.bs, self.r, self.d_ret, self.cap = block_size, n_rep, d_ret, capacity_tokens
        self.cap_blocks = capacity_tokens // block_size
        # pool rows hold `pitch` elements: the head dim, then zero padding
        self.pitch = lib().rba_row_pitch(head_dim)
        if self.pitch < 0:
            raise RbaError(ERR_UNSUPPORTED, f"head_dim {head_dim}")
        P = self.pitch
        td = _tdtype(self.dtype)
        dev = torch.device(device)
        self.k = torch.zeros((batch, n_kv_heads, capacity_tokens, P), dtype=td, device=dev)
        self.v = torch.zeros_like(self.k)
        self.rep = None
        self.rep_pos = None
        if mode == "mean":
            self.rep = torch.zeros((batch, n_kv_heads, self.cap_blocks, 1, P),
                                   dtype=torch.float32, device=dev)
        elif mode in ("topr_attn", "external"):
            self.rep = torch.zeros((batch, n_kv_heads, self.cap_blocks, n_rep, P), dtype=td,
                                   device=dev)
            if mode == "topr_attn":
                self.rep_pos = torch.full((batch, n_kv_heads, self.cap_blocks, n_rep), -1,
                                          dtype=torch.int32, device=dev)
        elif mode == "embed_cosine":
            self.rep = torch.zeros((batch, self.cap_blocks, d_ret), dtype=torch.float32, device=dev)
        elif mode != "identity":
            raise ValueError(mode)
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)
        d = _Desc(batch, n_q_heads, n_kv_heads, head_dim, block_size, n_rep, d_ret,
                  capacity_tokens, self.dtype, MODES[mode])
        h = _p()
        _check(lib().rba_store_create(ctypes.byref(d), _ptr(self.k), _ptr(self.v), _ptr(self.rep),
                                      _ptr(self.rep_pos), _ptr(self.status), ctypes.byref(h)),
               "rba_store_create")
        self.handle = h
        if score_reduce != "sum":
            _check(lib().rba_store_set_score_reduce(h, SCORE_REDUCE[score_reduce]),
                   "rba_store_set_score_reduce")
        self.score_reduce = score_reduce

    def set_wait_limit_ns(self, ns):
        """Bound of the one-launch decode step's device waits (0: the default 2 s)."""
        _check(lib().rba_store_set_wait_limit_ns(self.handle, int(ns)),
               "rba_store_set_wait_limit_ns")

    def set_decode_step_one_launch(self, on=True):
        """Let decode_step run as one cooperative launch where eligible (plan 3)."""
        _check(lib().rba_store_set_decode_step_one_launch(self.handle, int(bool(on))),
               "rba_store_set_decode_step_one_launch")

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _LIB is not None:
            _LIB.rba_store_destroy(h)
            self.handle = None

    @property
    def tdtype(self):
        return _tdtype(self.dtype)

    def kv_rows(self, t):
        """The first D elements of every row of a pool tensor (a view to write into)."""
        return t[..., :self.D]

    # -- geometry ------------------------------------------------------------
    def candidates(self, T, sink, window):
        f, n = _c_i32(), _c_i32()
        _check(lib().rba_candidates(self.handle, T, sink, window, ctypes.byref(f), ctypes.byref(n)),
               "rba_candidates")
        return f.value, n.value

    # -- memorise --------------------------------------------------------------
    def memorize(self, k_src=None, v_src=None, *, first_block=0, n_blocks=None, aux=None,
                 scale=None):
        if n_blocks is None:
            n_blocks = k_src.shape[2] // self.bs if k_src is not None else aux.shape[2]
        n_aux = 0
        if aux is not None and self.mode == "topr_attn":
            n_aux = aux.shape[1]
        if scale is None:
            scale = 1.0 / math.sqrt(self.D)
        _check(lib().rba_memorize(self.handle, _ptr(k_src), _ptr(v_src), first_block, n_blocks,
                                  _ptr(aux), n_aux, scale, _stream()), "rba_memorize")

    # -- score -------------------------------------------------------------------
    def score(self, q, T, sink, window, *, n_q=None, out=None, qsum_ws=None):
        first, nc = self.candidates(T, sink, window)
        if self.mode == "embed_cosine":
            n_q = q.shape[0]
            shape = (n_q, nc)
        else:
            n_q = 1 if q.dim() == 3 else q.shape[2]
            shape = (self.B, self.Hkv, nc)
            if (self.Hq // self.Hkv) * n_q > 64 and qsum_ws is None:
                qsum_ws = torch.empty((self.B, self.Hkv, self.D), dtype=torch.float32,
                                      device=q.device)
        if out is None:
            out = torch.empty(shape, dtype=torch.float32, device=q.device)
        _check(lib().rba_score(self.handle, _ptr(q), n_q, T, sink, window, _ptr(out),
                               _ptr(qsum_ws), _stream()), "rba_score")
        return out

    # -- attend ----------------------------------------------------------------
    def attend_workspace(self, k, T, sink, window):
        n = lib().rba_attend_workspace_size(self.handle, k, T, sink, window)
        return torch.zeros(max(n, 16), dtype=torch.uint8, device=self.k.device)

    def attend(self, q, idx, T, sink, window, *, scale=None, out=None, lse=None, workspace=None):
        k = idx.shape[-1] if idx is not None else 0
        if scale is None:
            scale = 1.0 / math.sqrt(self.D)
        if out is None:
            out = torch.empty((self.B, self.Hq, self.D), dtype=torch.float32, device=q.device)
        if lse is None:
            lse = torch.empty((self.B, self.Hq), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = self.attend_workspace(k, T, sink, window)
        _check(lib().rba_attend(self.handle, _ptr(q), _ptr(idx), k, T, sink, window, scale,
                                _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                                _stream()), "rba_attend")
        return out, lse

    def attend_gated(self, q, idx, T, sink, window, *, scale=None, out=None, lse=None):
        """Landmark-gated attention (landmark stores): each retrieved block enters
        the softmax once, with its landmark's logit (see rba.h)."""
        k = idx.shape[-1] if idx is not None else 0
        if scale is None:
            scale = 1.0 / math.sqrt(self.D)
        if out is None:
            out = torch.empty((self.B, self.Hq, self.D), dtype=torch.float32, device=q.device)
        if lse is None:
            lse = torch.empty((self.B, self.Hq), dtype=torch.float32, device=q.device)
        _check(lib().rba_attend_landmark_gated(self.handle, _ptr(q), _ptr(idx), k, T, sink,
                                               window, scale, _ptr(out), _ptr(lse), _stream()),
               "rba_attend_landmark_gated")
        return out, lse

    def prefill_workspace(self, n_chunks, chunk_len, n_sel, k, T, sink, window):
        n = lib().rba_attend_prefill_workspace_size(self.handle, n_chunks, chunk_len, n_sel, k, T,
                                                    sink, window)
        return torch.zeros(max(n, 16), dtype=torch.uint8, device=self.k.device)

    def attend_prefill(self, q, idx, chunk_k, chunk_v, T, sink, window, *, scale=None, out=None,
                       lse=None, workspace=None):
        n_chunks, _, chunk_len, _ = q.shape
        n_sel, k = idx.shape[1], idx.shape[2]
        if scale is None:
            scale = 1.0 / math.sqrt(self.D)
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        if lse is None:
            lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = self.prefill_workspace(n_chunks, chunk_len, n_sel, k, T, sink, window)
        _check(lib().rba_attend_prefill(self.handle, _ptr(q), n_chunks, chunk_len, _ptr(idx), n_sel,
                                        k, T, sink, window, _ptr(chunk_k), _ptr(chunk_v), scale,
                                        _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                                        _stream()), "rba_attend_prefill")
        return out, lse

    # -- whole decode step -----------------------------------------------------------
    def decode_workspace(self, k, T, sink, window):
        n = lib().rba_decode_step_workspace_size(self.handle, k, T, sink, window)
        return torch.zeros(max(n, 16), dtype=torch.uint8, device=self.k.device)

    def decode_plan(self, k, T, sink, window):
        """3: the whole step in one cooperative launch; 2: score -> top-k ->
        whole-block tensor-core attention kernel, overlapped (programmatic
        dependent launches); 1: the same with the CUDA-core attention kernel;
        0: score -> top-k -> split-K in stream order; <0: see rba.h."""
        return lib().rba_decode_step_plan(self.handle, k, T, sink, window)

    def decode_launches(self, k, T, sink, window):
        """Kernels one decode_step enqueues (-4: invalid arguments)."""
        return lib().rba_decode_step_launches(self.handle, k, T, sink, window)

    def decode_step(self, q, k, T, sink, window, *, scale=None, workspace=None, out=None,
                    lse=None, idx=None, scores=None):
        if scale is None:
            scale = 1.0 / math.sqrt(self.D)
        dev = q.device
        if out is None:
            out = torch.empty((self.B, self.Hq, self.D), dtype=torch.float32, device=dev)
        if lse is None:
            lse = torch.empty((self.B, self.Hq), dtype=torch.float32, device=dev)
        if idx is None:
            idx = torch.empty((self.B, self.Hkv, k), dtype=torch.int32, device=dev)
        if workspace is None:
            workspace = self.decode_workspace(k, T, sink, window)
        _check(lib().rba_decode_step(self.handle, _ptr(q), k, T, sink, window, scale, _ptr(scores),
                                     _ptr(idx), _ptr(out), _ptr(lse), _ptr(workspace),
                                     workspace.numel(), _stream()), "rba_decode_step")
        return idx, out, lse

    def stream_step(self, q, k_new, v_new, T, k, sink, window, *, aux=None, scale=None,
                    workspace=None, out=None, lse=None, idx=None):
        """Append one token's K/V at position T, memorise the block it completes,
        decode q over T + 1 tokens.  Returns (idx [B][Hkv][k'], out, lse) with
        k' = min(k, candidates at T + 1)."""
        if scale is None:
            scale = 1.0 / math.sqrt(self.D)
        dev = q.device
        if out is None:
            out = torch.empty((self.B, self.Hq, self.D), dtype=torch.float32, device=dev)
        if lse is None:
            lse = torch.empty((self.B, self.Hq), dtype=torch.float32, device=dev)
        if idx is None:
            idx = torch.empty((self.B, self.Hkv, max(k, 1)), dtype=torch.int32, device=dev)
        if workspace is None:
            workspace = self.decode_workspace(k, T + 1, sink, window)
        n_aux = aux.shape[1] if (aux is not None and self.mode == "topr_attn") else 0
        used = ctypes.c_int32(0)
        _check(lib().rba_stream_step(self.handle, _ptr(q), _ptr(k_new), _ptr(v_new), T, k, sink,
                                     window, scale, _ptr(aux), n_aux, _ptr(idx), _ptr(out),
                                     _ptr(lse), ctypes.byref(used), _ptr(workspace),
                                     workspace.numel(), _stream()), "rba_stream_step")
        kk = used.value
        sel = idx.reshape(-1)[: self.B * self.Hkv * kk].reshape(self.B, self.Hkv, kk)
        return sel, out, lse

    # -- two-stage approximate token retrieval (block size 1) ---------------------
    def group_means(self, group, *, first_group=0, n_groups=None, out=None):
        """Mean key of every group of `group` consecutive tokens (fp32 index
        [B][Hkv][capacity // group][P]); groups [first_group, first_group + n_groups)."""
        cap_groups = self.cap // group
        if n_groups is None:
            n_groups = cap_groups - first_group
        if out is None:
            out = torch.zeros((self.B, self.Hkv, cap_groups, self.pitch), dtype=torch.float32,
                              device=self.k.device)
        _check(lib().rba_group_means(self.handle, first_group, n_groups, group, _ptr(out),
                                     _stream()), "rba_group_means")
        return out

    def approx_select(self, q, T, sink, window, group, groups_kept, k, means, *, idx=None,
                      groups_out=None, scanned=None, workspace=None):
        """Two-stage selection of k tokens per (batch, kv head).  Returns
        (idx [B][Hkv][k], kept groups [B][Hkv][groups_kept], keys read [B][Hkv])."""
        dev = q.device
        if idx is None:
            idx = torch.empty((self.B, self.Hkv, k), dtype=torch.int32, device=dev)
        if groups_out is None:
            groups_out = torch.empty((self.B, self.Hkv, groups_kept), dtype=torch.int32,
                                     device=dev)
        if scanned is None:
            scanned = torch.empty((self.B, self.Hkv), dtype=torch.int32, device=dev)
        if workspace is None:
            n = lib().rba_approx_select_workspace_size(self.handle, T, sink, window, group,
                                                       groups_kept, k)
            workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
        _check(lib().rba_approx_select(self.handle, _ptr(q), T, sink, window, group,
                                       groups_kept, k, _ptr(means), _ptr(idx), _ptr(groups_out),
                                       _ptr(scanned), _ptr(workspace), workspace.numel(),
                                       _stream()), "rba_approx_select")
        return idx, groups_out, scanned

    # -- dynamic memory update ---------------------------------------------------
    def memory_units(self):
        """Memory units U: B * Hkv (dot modes) or B (cosine bank)."""
        return lib().rba_memory_units(self.handle)

    def new_counters(self):
        """Zeroed retrieval counters [U][cap_blocks] (uint32 in the library; held
        here as int32 with the same bits)."""
        return torch.zeros((self.memory_units(), self.cap_blocks), dtype=torch.int32,
                           device=self.k.device)

    def count_retrievals(self, idx, counters):
        """Adds the selection idx ([..., U, k] int32, row r -> unit r % U) to counters."""
        k = idx.shape[-1]
        rows = idx.numel() // k if k else 0
        _check(lib().rba_count_retrievals(self.handle, _ptr(idx), rows, k, _ptr(counters),
                                          _stream()), "rba_count_retrievals")

    def memory_update(self, T, counters, *, pinned_blocks=0, keep_newest=None, drop_oldest=None,
                      keep_total=None, keep_map=None):
        """Counter-driven prune and in-place compaction of the T tokens held.
        Counts not given follow memory_rule(n) for the n = T // bs - pinned_blocks
        entries.  Returns (T_new, keep_map [U][keep_total])."""
        n = T // self.bs - pinned_blocks
        rule = memory_rule(max(n, 0))
        keep_newest = rule[0] if keep_newest is None else keep_newest
        drop_oldest = rule[1] if drop_oldest is None else drop_oldest
        keep_total = rule[2] if keep_total is None else keep_total
        if keep_map is None:
            keep_map = torch.empty((self.memory_units(), max(keep_total, 1)), dtype=torch.int32,
                                   device=self.k.device)
        t_new = _c_i64(0)
        _check(lib().rba_memory_update(self.handle, T, pinned_blocks, keep_newest, drop_oldest,
                                       keep_total, _ptr(counters), _ptr(keep_map),
                                       ctypes.byref(t_new), _stream()), "rba_memory_update")
        return t_new.value, keep_map[:, :keep_total]

    def decode_step_host(self, q_host, k, T, sink, window, *, q_dev, idx_dev, out_dev, lse_dev,
                         out_host, lse_host=None, idx_host=None, workspace, scale=None):
        """Host buffers in and out; synchronises the current stream."""
        if scale is None:
            scale = 1.0 / math.sqrt(self.D)
        hp = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        _check(lib().rba_decode_step_host(self.handle, hp(q_host), _ptr(q_dev), k, T, sink, window,
                                          scale, _ptr(idx_dev), _ptr(out_dev), _ptr(lse_dev),
                                          hp(out_host), hp(lse_host), hp(idx_host),
                                          _ptr(workspace), workspace.numel(), _stream()),
               "rba_decode_step_host")

    def check(self):
        """Synchronises and raises if a kernel recorded a device-side error."""
        _check(lib().rba_store_check(self.handle, _stream()), "device status")


class _PagedDesc(ctypes.Structure):
    _fields_ = [("n_q_heads", _c_i32), ("n_kv_heads", _c_i32), ("head_dim", _c_i32),
                ("page_size", _c_i32), ("n_pages", _c_i32), ("max_requests", _c_i32),
                ("max_pages", _c_i32), ("dtype", _c_i32)]


class _PagedBuffers(ctypes.Structure):
    _fields_ = [(n, _p) for n in ("pool", "rep", "table", "lens", "free_pages", "n_free",
                                  "status")]


_MOST = 2 ** 31 - 1


def _fits(**numbers):
    """Refuses numbers that the library would take for others (ctypes cuts them to 32 bits)."""
    for name, x in numbers.items():
        if not -_MOST - 1 <= x <= _MOST:
            raise ValueError(f"{name}: expected a 32-bit number, got {x}")


class PagedStore:
    """A paged memory in 4 bits for requests of different lengths (rba_paged_* in rba.h).

    A page is a memory block of `page_size` tokens.  Lengths, page tables and the free list
    live on the device and are read there by every call, so a decode step (extend, append,
    select, attend) can be captured once and replayed while the requests grow.

    Buffers (allocated here, or the caller's own where given; contiguous, on one device):
      pool    uint8 [n_pages][Hkv][strips][strip_bytes]   rep   fp32 [n_pages][Hkv][P]
      table   int32 [max_requests][max_pages]             lens  int32 [max_requests]
      free    int32 [n_pages] (a stack)                   n_free int32 [1]
    table, lens, free and n_free belong together: all of them are given, or none.
    Work runs on the store's device, on torch's current stream there.
    """

    def __init__(self, *, n_q_heads, n_kv_heads, head_dim, page_size, n_pages, max_requests,
                 max_pages, dtype="bf16", device="cuda", pool=None, rep=None, table=None,
                 lens=None, free=None, n_free=None):
        if dtype not in ("bf16", "f32", torch.bfloat16, torch.float32):
            raise ValueError(f"dtype: expected bf16 or f32, got {dtype}")
        _fits(n_q_heads=n_q_heads, n_kv_heads=n_kv_heads, head_dim=head_dim, page_size=page_size,
              n_pages=n_pages, max_requests=max_requests, max_pages=max_pages)
        self.dtype = BF16 if dtype in ("bf16", torch.bfloat16) else F32
        self.Hq, self.Hkv, self.D, self.page_size = n_q_heads, n_kv_heads, head_dim, page_size
        self.n_pages, self.max_requests, self.max_pages = n_pages, max_requests, max_pages
        L = lib()
        self.pitch = L.rba_row_pitch(head_dim)
        if self.pitch < 0:
            raise RbaError(ERR_UNSUPPORTED, f"head_dim {head_dim}")
        self.strip_bytes = L.rba_paged_strip_bytes(head_dim)
        strips = -(-page_size // 16) if page_size > 0 else 0
        given = [t for t in (pool, rep, table, lens, free, n_free) if t is not None]
        dev = given[0].device if given else torch.device(device)

        def buf(name, t, shape, dt, fill):
            if t is None:
                return fill(shape, dt)
            if tuple(t.shape) != shape or t.dtype != dt or t.device != dev:
                raise ValueError(f"{name}: expected {dt} {shape} on {dev}, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device}")
            _ptr(t)
            return t

        def zeros(shape, dt):
            return torch.zeros(shape, dtype=dt, device=dev)

        if len({t is None for t in (table, lens, free, n_free)}) > 1:
            # (a free list made anew holds pages that the table's requests hold)
            raise ValueError("table, lens, free and n_free are given together")
        self.pool = buf("pool", pool, (n_pages, n_kv_heads, strips, self.strip_bytes),
                        torch.uint8, zeros)
        self.rep = buf("rep", rep, (n_pages, n_kv_heads, self.pitch), torch.float32, zeros)
        self.table = buf("table", table, (max_requests, max_pages), torch.int32, zeros)
        self.lens = buf("lens", lens, (max_requests,), torch.int32, zeros)
        self.free = buf("free", free, (n_pages,), torch.int32,
                        lambda s, dt: torch.arange(n_pages - 1, -1, -1, dtype=dt, device=dev))
        self.n_free = buf("n_free", n_free, (1,), torch.int32,
                          lambda s, dt: torch.full(s, n_pages, dtype=dt, device=dev))
        self.device = self.pool.device
        if not self.pool.is_cuda:
            raise ValueError("expected CUDA tensors")
        self._index, self._td = self.device.index, _tdtype(self.dtype)
        self.status = zeros((8,), torch.int32)
        d = _PagedDesc(n_q_heads, n_kv_heads, head_dim, page_size, n_pages, max_requests,
                       max_pages, self.dtype)
        b = _PagedBuffers(*(_ptr(t) for t in (self.pool, self.rep, self.table, self.lens,
                                              self.free, self.n_free, self.status)))
        h = _p()
        with torch.cuda.device(self.device):
            _check(L.rba_paged_create(ctypes.byref(d), ctypes.byref(b), ctypes.byref(h)),
                   "rba_paged_create")
        self.handle = h

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _LIB is not None:
            _LIB.rba_paged_destroy(h)
            self.handle = None

    @property
    def tdtype(self):
        return _tdtype(self.dtype)

    # -- marshalling (a decode step makes four calls: host time counts) ----------
    def _call(self, name, *args):
        """One library call on the store's device and torch's current stream there."""
        i = self._index
        stream = torch._C._cuda_getCurrentRawStream(i)
        if torch._C._cuda_getDevice() == i:
            s = getattr(_LIB, name)(self.handle, *args, stream)
        else:
            with torch.cuda.device(i):
                s = getattr(_LIB, name)(self.handle, *args, stream)
        if s != OK:
            raise RbaError(s, name)

    def _refuse(self, name, t, shape, dt):
        raise ValueError(f"{name}: expected a {dt} tensor {shape} on {self.device} with dense "
                         f"dims, got {t.dtype} {tuple(t.shape)}, strides {t.stride()}, on "
                         f"{t.device}")

    def _arg(self, name, t, shape, dt):
        """Pointer of a contiguous tensor of exactly this shape, type and device."""
        if t.dtype is not dt or t.shape != shape or t.get_device() != self._index or \
                not t.is_contiguous():
            self._refuse(name, t, shape, dt)
        return t.data_ptr()

    def _rows(self, name, t, n, heads):
        """(pointer, row stride, head stride) of rows [n][heads][D] with dense dims."""
        sn, sh, sd = t.stride() if t.dim() == 3 else (0, 0, 0)
        if t.dtype is not self._td or t.shape != (n, heads, self.D) or sd != 1 or \
                t.get_device() != self._index:
            self._refuse(name, t, (n, heads, self.D), self._td)
        return t.data_ptr(), sn, sh

    def _bytes(self, t):
        """(pointer, bytes) of a workspace."""
        if t.dtype is not torch.uint8 or t.get_device() != self._index or not t.is_contiguous():
            self._refuse("workspace", t, tuple(t.shape), torch.uint8)
        return t.data_ptr(), t.numel()

    def _out(self, name, t, shape, dt):
        """(t, pointer) of an output: the caller's, checked, or a new one."""
        if t is None:
            t = self.lens.new_empty(shape, dtype=dt)  # (cheaper on the host than torch.empty)
            return t, t.data_ptr()
        return t, self._arg(name, t, shape, dt)

    # -- page tables -------------------------------------------------------------
    def extend(self, n_new, n_slots, *, slots=None, starts=None):
        """Grows request r by n_new[r] tokens.  Returns (slots [n_slots], -1 past the new
        tokens; starts [R + 1], the first new token of each request)."""
        R = n_new.shape[0]
        if R > _MOST or n_slots > _MOST:
            _fits(requests=R, n_slots=n_slots)
        slots, sp = self._out("slots", slots, (n_slots,), torch.int32)
        starts, tp = self._out("starts", starts, (R + 1,), torch.int32)
        self._call("rba_paged_extend", self._arg("n_new", n_new, (R,), torch.int32), R, sp, n_slots,
                   tp)
        return slots, starts

    def truncate(self, keep):
        """Cuts request r back to at most keep[r] tokens (0: the request is over)."""
        R = keep.shape[0]
        if R > _MOST:
            _fits(requests=R)
        self._call("rba_paged_truncate", self._arg("keep", keep, (R,), torch.int32), R)

    # -- rows ----------------------------------------------------------------------
    def append(self, slots, k, v):
        """Writes rows k, v [n][Hkv][D] in 4 bits at their slots, and the mean keys of the
        pages they complete.  Rows may be strided views (a fused projection's slices)."""
        n = slots.shape[0]
        if n > _MOST:
            _fits(rows=n)
        kp, kt, kh = self._rows("k", k, n, self.Hkv)
        vp, vt, vh = self._rows("v", v, n, self.Hkv)
        self._call("rba_paged_append", self._arg("slots", slots, (n,), torch.int32), n, kp, kt,
                   kh, vp, vt, vh)

    def read(self, slots, *, k=None, v=None):
        """Rows at the slots as the values held there: (k, v), each [n][Hkv][D]."""
        n = slots.shape[0]
        if n > _MOST:
            _fits(rows=n)
        shape = (n, self.Hkv, self.D)
        k, kp = self._out("k", k, shape, self._td)
        v, vp = self._out("v", v, shape, self._td)
        self._call("rba_paged_read", self._arg("slots", slots, (n,), torch.int32), n, kp, vp)
        return k, v

    # -- select, attend --------------------------------------------------------------
    def select_workspace(self):
        n = lib().rba_paged_select_workspace_size(self.handle)
        return torch.empty(max(n, 16), dtype=torch.uint8, device=self.device)

    def select(self, q, k, sink, window, *, idx=None, workspace=None):
        """The k best pages of each (request, kv head) for q [R][Hq][D]: idx [R][Hkv][k],
        ascending, -1 past a request's candidates."""
        R = q.shape[0]
        if not (k <= _MOST and -1 < sink <= _MOST and -1 < window <= _MOST):
            _fits(k=k, sink=sink, window=window)
        qp, qr, qh = self._rows("q", q, R, self.Hq)
        idx, ip = self._out("idx", idx, (R, self.Hkv, k), torch.int32)
        if workspace is None:
            workspace = self.select_workspace()
        self._call("rba_paged_select", qp, qr, qh, R, k, sink, window, ip, *self._bytes(workspace))
        return idx

    def attend_workspace(self):
        """Workspace of attend; one serves every call, one call at a time."""
        with torch.cuda.device(self.device):
            n = lib().rba_paged_attend_workspace_size(self.handle)
        return torch.empty(max(n, 16), dtype=torch.uint8, device=self.device)

    def attend(self, q, idx, sink, window, *, scale=None, out=None, lse=None, workspace=None):
        """Attention of one token of each request, q [R][Hq][D], over its sink tokens, the
        pages idx (None: no pages) and its window.  Returns (out fp32 [R][Hq][D], lse)."""
        R = q.shape[0]
        qp, qr, qh = self._rows("q", q, R, self.Hq)
        k = idx.shape[-1] if idx is not None else 0
        if not (k <= _MOST and -1 < sink <= _MOST and -1 < window <= _MOST):
            _fits(k=k, sink=sink, window=window)
        ip = self._arg("idx", idx, (R, self.Hkv, k), torch.int32) if k else None
        scale = 1.0 / math.sqrt(self.D) if scale is None else float(scale)
        out, op = self._out("out", out, (R, self.Hq, self.D), torch.float32)
        lse, lp = self._out("lse", lse, (R, self.Hq), torch.float32)
        if workspace is None:
            workspace = self.attend_workspace()
        self._call("rba_paged_attend", qp, qr, qh, R, ip, k, sink, window, scale, op, lp,
                   *self._bytes(workspace))
        return out, lse

    # -- whole decode step -----------------------------------------------------------
    def decode_step(self, q, k_new, v_new, n_new, k, sink, window, *, scale=None, slots=None,
                    starts=None, idx=None, out=None, lse=None, select_workspace=None,
                    workspace=None):
        """One step of every request: request r grows by n_new[r] tokens, whose rows are packed in
        k_new, v_new [n][Hkv][D] (n may be larger: rows past them are ignored), then q [R][Hq][D]
        attends to sink, its k best pages and window.  Returns (idx, out, lse).  With every
        buffer given it can be captured once and replayed.  A step refused with an exception has
        changed nothing; one whose extension the device refuses (too few free pages) writes no row,
        attends to what is held, and is reported by check()."""
        # everything is checked before the first call: a refused step leaves the store as it was
        n, R, i32, f32 = k_new.shape[0], n_new.shape[0], torch.int32, torch.float32
        _fits(rows=n, k=k, sink=sink, window=window)
        scale = None if scale is None else float(scale)
        if min(k, sink, window) < 0:
            raise ValueError(f"k, sink, window: expected 0 or more, got {k}, {sink}, {window}")
        self._rows("k_new", k_new, n, self.Hkv)
        self._rows("v_new", v_new, n, self.Hkv)
        self._rows("q", q, R, self.Hq)
        for name, t, shape, dt in (("n_new", n_new, (R,), i32), ("slots", slots, (n,), i32),
                                   ("starts", starts, (R + 1,), i32),
                                   ("idx", idx, (R, self.Hkv, k), i32),
                                   ("out", out, (R, self.Hq, self.D), f32),
                                   ("lse", lse, (R, self.Hq), f32)):
            if t is not None:
                self._arg(name, t, shape, dt)
        if select_workspace is None and k:
            select_workspace = self.select_workspace()
        if workspace is None:
            workspace = self.attend_workspace()
        spaces = (*(self._bytes(select_workspace) if k else (None, 0)), *self._bytes(workspace))
        with torch.cuda.device(self.device):  # (the library's own limits)
            _check(_LIB.rba_paged_step_check(self.handle, R, n, k, sink, window, *spaces),
                   "decode_step")
        slots, _ = self.extend(n_new, k_new.shape[0], slots=slots, starts=starts)
        self.append(slots, k_new, v_new)
        idx = self.select(q, k, sink, window, idx=idx, workspace=select_workspace) if k else None
        out, lse = self.attend(q, idx, sink, window, scale=scale, out=out, lse=lse,
                               workspace=workspace)
        return idx, out, lse

    def check(self):
        """Synchronises and raises if a kernel recorded a device-side error."""
        self._call("rba_paged_check")


def memory_rule(n):
    """(keep_newest, drop_oldest, keep_total) for n memory entries (host only)."""
    a, b, c = _c_i64(), _c_i64(), _c_i64()
    _check(lib().rba_memory_rule(n, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)),
           "rba_memory_rule")
    return a.value, b.value, c.value


def topk(scores, k, *, index_base=0, out=None, workspace=None):
    """Top-k per row of a 2-D (or [..., n]) fp32 score tensor; ascending positions."""
    n = scores.shape[-1]
    rows = scores.numel() // n if n else 0
    if out is None:
        out = torch.empty(scores.shape[:-1] + (k,), dtype=torch.int32, device=scores.device)
    if workspace is None:
        nb = lib().rba_topk_workspace_size(rows, n, k)
        workspace = torch.empty(max(nb, 16), dtype=torch.uint8, device=scores.device)
    _check(lib().rba_topk(_ptr(scores), rows, n, k, index_base, _ptr(out), _ptr(workspace),
                          workspace.numel(), _stream()), "rba_topk")
    return out
