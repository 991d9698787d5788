"""AB-Attention (Accurate Block Attention) hot path on NVIDIA B200.

Python binding of the C ABI in ``include/ab.h`` (library ``libab.so`` in this
package).  This module only marshals arguments: it checks tensor shapes and
dtypes, allocates outputs with torch on the caller's device and passes raw
pointers and the current CUDA stream to the library.  Every step of the path
runs in the library's CUDA kernels; there is no CPU fallback, and calling any
op without the built library raises ``RuntimeError``.

Names follow the C ABI: ``ab_select`` (IBCS), ``ab_sample`` (SIP),
``ab_attention`` (the packed 1/pi-weighted sparse attention),
``ab_attention_dense``, ``ab_forward`` and ``ab_forward_host``; before the path
``ab_qk_norm_rope`` (norms of queries and keys, position rotation) and
``ab_forward_qkv``; for models that produce their sequences step by step, a paged
key-value cache: ``ab_paged_plan``, ``ab_paged_append``, ``ab_paged_select``,
``ab_paged_topk``, ``ab_attention_paged`` and ``ab_paged_forward``.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libab.so")

AB_OK = 0
STATUS_NAMES = {0: "AB_OK", 1: "AB_ERR_INVALID_ARG", 2: "AB_ERR_UNSUPPORTED", 3: "AB_ERR_CUDA",
                4: "AB_ERR_CAPACITY", 5: "AB_ERR_TIMEOUT", 6: "AB_ERR_WORKSPACE"}

# every symbol include/ab.h declares
EXPORTS = ("ab_budget", "ab_workspace_size", "ab_select", "ab_sample", "ab_sample_systematic", "ab_sample_topk", "ab_attention",
           "ab_attention_dense", "ab_forward", "ab_forward_host", "ab_get_device_error",
           "ab_status_string", "ab_select_static", "ab_forward_slice", "ab_select_sample",
           "ab_qk_norm_rope", "ab_forward_qkv", "ab_paged_workspace_size", "ab_paged_plan", "ab_paged_append",
           "ab_paged_select", "ab_paged_topk", "ab_attention_paged", "ab_paged_forward")


class AbError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class ab_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("L", ctypes.c_int32),
                ("d", ctypes.c_int32), ("q_block", ctypes.c_int32), ("kv_block", ctypes.c_int32),
                ("C", ctypes.c_int32), ("kmeans_iters", ctypes.c_int32),
                ("keep_ratio", ctypes.c_float), ("L_kv", ctypes.c_int32), ("seed", ctypes.c_uint64)]


@dataclass(frozen=True)
class Params:
    """Problem description (mirrors ``ab_params``).  ``L`` is the number of
    queries per (b, h); ``L_kv`` the number of keys and values (0: the same as
    ``L``, i.e. self-attention)."""

    B: int
    H: int
    L: int
    d: int
    q_block: int = 128
    kv_block: int = 16
    C: int = 8
    kmeans_iters: int = 3
    keep_ratio: float = 0.1
    seed: int = 42
    L_kv: int = 0

    @property
    def Lk(self) -> int:
        return self.L_kv if self.L_kv > 0 else self.L

    @property
    def Nq(self) -> int:
        return -(-self.L // self.q_block)

    @property
    def Nkv(self) -> int:
        return -(-self.Lk // self.kv_block)

    def c(self) -> ab_params:
        return ab_params(self.B, self.H, self.L, self.d, self.q_block, self.kv_block, self.C,
                         self.kmeans_iters, float(self.keep_ratio), int(self.L_kv),
                         int(self.seed) & (2**64 - 1))

    @staticmethod
    def of(w, seed: int = 42, **kw) -> "Params":
        """From a ``synthetic.Workload``."""
        args = dict(B=w.B, H=w.H, L=w.L, d=w.d, q_block=w.q_block, kv_block=w.kv_block, C=w.C,
                    kmeans_iters=w.kmeans_iters, keep_ratio=w.keep_ratio, seed=seed,
                    L_kv=w.Lk if w.Lk != w.L else 0)
        args.update(kw)
        return Params(**args)


class ab_norm_rope(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
                ("n_pos", ctypes.c_int32), ("wq", ctypes.c_void_p), ("wk", ctypes.c_void_p),
                ("cos_table", ctypes.c_void_p), ("sin_table", ctypes.c_void_p)]


class ab_tokens(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("batch", ctypes.c_int64), ("token", ctypes.c_int64),
                ("head", ctypes.c_int64)]


class ab_paged_params(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("page", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("recent", ctypes.c_int32), ("keep_ratio", ctypes.c_float)]


NORMS = {"none": 0, "head": 1, "token": 2}


class NormRope:
    """Norm and rotation of queries and keys (mirrors ``ab_norm_rope``): ``norm``
    is "none", "head" (mean square over each head's d) or "token" (over all
    heads); ``wq`` and ``wk`` fp32 weights [d] or [heads, d] (None: ones);
    ``cos`` and ``sin`` fp32 [n_pos, d/2] (both None: no rotation);
    ``interleaved``: pairs (2i, 2i+1), else (i, i + d/2).  All tensors are
    contiguous on one CUDA device and are kept; their values may change, a
    NormRope's attributes cannot."""

    def __init__(self, norm="head", interleaved=True, eps=1e-6, wq=None, wk=None, cos=None, sin=None):
        if norm not in NORMS:
            raise ValueError(f"norm must be one of {sorted(NORMS)}, got {norm!r}")
        if (cos is None) != (sin is None):
            raise ValueError("cos and sin come together")
        self.__dict__.update(norm=norm, interleaved=bool(interleaved), eps=float(eps), wq=wq, wk=wk, cos=cos, sin=sin)
        self._bind()

    def _bind(self):
        """The library's copy, from the tensors as they are."""
        import torch
        wq, wk, cos, sin = self.wq, self.wk, self.cos, self.sin
        tensors = [t for t in (wq, wk, cos, sin) if t is not None]
        for t in tensors:
            if t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda:
                raise ValueError(f"weights and tables must be contiguous fp32 CUDA tensors, got {t.dtype} on {t.device}")
            if t.device != tensors[0].device:
                raise ValueError("weights and tables must be on one device")
        for t in (wq, wk):
            if t is not None and t.dim() != (2 if self.norm == "token" else 1):
                raise ValueError(f"weights of norm {self.norm!r} have shape [{'heads, ' if self.norm == 'token' else ''}d], "
                                 f"got {tuple(t.shape)}")
        if cos is not None and (cos.dim() != 2 or cos.shape != sin.shape or cos.shape[0] < 1):
            raise ValueError("cos and sin must be [n_pos, d/2], with one row at least")
        n_pos = 0 if cos is None else cos.shape[0]
        at = [0 if t is None else t.data_ptr() for t in (wq, wk, cos, sin)]
        self.__dict__.update(
            n_pos=n_pos, device=tensors[0].device if tensors else None, _index=tensors[0].get_device() if tensors else None,
            _fits=None, _where=[t.data_ptr for t in tensors], _at=[t.data_ptr() for t in tensors],
            _c=ab_norm_rope(NORMS[self.norm], int(self.interleaved), self.eps, n_pos, *at))

    def __setattr__(self, name, value):
        raise AttributeError(f"cannot assign to {name!r}: make another NormRope")

    def __delattr__(self, name):
        raise AttributeError(f"cannot delete {name!r}: make another NormRope")

    def check(self, Hq: int, Hk: int, d: int, index: int):
        """The weights and tables belong to Hq query and Hk key heads of d on CUDA device `index`."""
        if self._at != [where() for where in self._where]:  # a tensor has other storage now (`.data = ...`)
            self._bind()
        if self._fits == (Hq, Hk, d, index):
            return
        for t, H in ((self.wq, Hq), (self.wk, Hk)):
            if t is not None and tuple(t.shape) != ((H, d) if self.norm == "token" else (d,)):
                raise ValueError(f"norm weights {tuple(t.shape)} do not fit {H} heads of {d}")
        if self.cos is not None and self.cos.shape[1] != d // 2:
            raise ValueError(f"cos and sin have {self.cos.shape[1]} columns, {d // 2} expected")
        if self._index is not None and self._index != index:
            raise ValueError(f"weights and tables are on {self.device}, the tokens on cuda:{index}")
        self.__dict__["_fits"] = (Hq, Hk, d, index)


@dataclass(frozen=True)
class PagedParams:
    """A paged key-value cache (mirrors ``ab_paged_params``): ``S`` sequences with
    up to ``max_pages`` of the ``num_pages`` pages of ``page`` tokens each;
    ``keep_ratio`` and ``recent`` are ``ab_paged_topk``'s."""

    S: int
    Hq: int
    Hkv: int
    d: int
    page: int
    num_pages: int
    max_pages: int
    keep_ratio: float = 0.1
    recent: int = 1

    def c(self) -> ab_paged_params:
        c = self.__dict__.get("_c")
        if c is None:
            c = ab_paged_params(self.S, self.Hq, self.Hkv, self.d, self.page, self.num_pages, self.max_pages, self.recent,
                                float(self.keep_ratio))
            object.__setattr__(self, "_c", c)
        return c


_lib = None


def lib(path: str = LIB_PATH):
    """The loaded ``libab.so``; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"libab.so not built ({path}); run block_sparse_attention_queries_b200/build.py")
        L = ctypes.CDLL(path)
        P = ctypes.POINTER(ab_params)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        L.ab_budget.argtypes = [P]
        L.ab_budget.restype = ctypes.c_int32
        L.ab_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        L.ab_select.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ab_sample.argtypes = [P, vp, vp, vp, vp, vp]
        L.ab_sample_topk.argtypes = [P, vp, vp, vp, vp, vp]
        L.ab_sample_systematic.argtypes = [P, vp, vp, vp, vp, vp]
        L.ab_attention.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp]
        L.ab_attention_dense.argtypes = [P, vp, vp, vp, vp, vp]
        L.ab_forward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ab_forward_host.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ab_select_sample.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ab_forward_slice.argtypes = [P, ctypes.c_int32, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                       vp]
        L.ab_select_static.argtypes = [P, vp, vp, vp, vp, vp, vp]
        L.ab_get_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_int32)]
        L.ab_status_string.argtypes = [ctypes.c_int]
        L.ab_status_string.restype = ctypes.c_char_p
        NR, TK, PP, i32 = (ctypes.POINTER(ab_norm_rope), ctypes.POINTER(ab_tokens), ctypes.POINTER(ab_paged_params),
                           ctypes.c_int32)
        L.ab_qk_norm_rope.argtypes = [P, NR, TK, TK, TK, vp, vp, vp, vp, vp, vp]
        L.ab_forward_qkv.argtypes = [P, NR, TK, TK, TK, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ab_paged_workspace_size.argtypes = [PP, i32, ctypes.POINTER(ctypes.c_size_t)]
        L.ab_paged_plan.argtypes = [PP, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.ab_paged_append.argtypes = [PP, NR, i32, TK, TK, TK, vp, vp, vp, vp, vp, vp, vp]
        L.ab_paged_select.argtypes = [PP, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ab_paged_topk.argtypes = [PP, vp, vp, vp, vp, vp]
        L.ab_attention_paged.argtypes = [PP, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ab_paged_forward.argtypes = [PP, NR, i32, TK, TK, TK, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                       sz, vp]
        for name in ("ab_qk_norm_rope", "ab_forward_qkv", "ab_paged_workspace_size", "ab_paged_plan",
                     "ab_paged_append", "ab_paged_select", "ab_paged_topk", "ab_attention_paged", "ab_paged_forward"):
            getattr(L, name).restype = ctypes.c_int
        for name in ("ab_workspace_size", "ab_select", "ab_sample", "ab_sample_systematic", "ab_sample_topk", "ab_attention",
                     "ab_attention_dense",
                     "ab_forward", "ab_forward_host", "ab_get_device_error", "ab_select_static",
                     "ab_forward_slice", "ab_select_sample"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != AB_OK:
        raise AbError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check_bf16(t, shape):
    import torch
    if t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"expected contiguous bf16 {list(shape)}, got {t.dtype} {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")


def _check_qkv(p: Params, Q, *kv):
    """Q (and O) are [B, H, L, d]; K and V are [B, H, Lk, d]."""
    _check_bf16(Q, (p.B, p.H, p.L, p.d))
    for t in kv:
        _check_bf16(t, (p.B, p.H, p.Lk, p.d))


def budget(p: Params) -> int:
    return int(lib().ab_budget(ctypes.byref(p.c())))


def workspace_size(p: Params) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ab_workspace_size(ctypes.byref(p.c()), ctypes.byref(n)), "ab_workspace_size")
    return int(n.value)


def alloc_workspace(p: Params, device):
    import torch
    return torch.empty(workspace_size(p), dtype=torch.uint8, device=device)


def ab_select(p: Params, Q, K, workspace=None, want_centroids=False):
    """IBCS: returns P [B,H,Nq,Nkv] fp32 (and centroids [B,H,Nq,C,d] fp32, counts [B,H,Nq,C] int32)."""
    import torch
    _check_qkv(p, Q, K)
    dev = Q.device
    P = torch.empty(p.B, p.H, p.Nq, p.Nkv, dtype=torch.float32, device=dev)
    cent = torch.empty(p.B, p.H, p.Nq, p.C, p.d, dtype=torch.float32, device=dev) if want_centroids else None
    cnt = torch.empty(p.B, p.H, p.Nq, p.C, dtype=torch.int32, device=dev) if want_centroids else None
    ws = alloc_workspace(p, dev) if workspace is None else workspace
    _check(lib().ab_select(ctypes.byref(p.c()), _ptr(Q), _ptr(K), _ptr(P), _ptr(cent), _ptr(cnt), _ptr(ws),
                           ws.numel(), _stream(dev)), "ab_select")
    return (P, cent, cnt) if want_centroids else P


def ab_select_static(p: Params, Q, K, want_centroids=False):
    """ab_select with the library's own fixed device scratch: no workspace is
    allocated (the outputs still are, here, by torch).  For callers that
    cannot allocate device memory; see include/ab.h for the size limit and the
    rule that overlapping calls race."""
    import torch
    _check_qkv(p, Q, K)
    dev = Q.device
    P = torch.empty(p.B, p.H, p.Nq, p.Nkv, dtype=torch.float32, device=dev)
    cent = torch.empty(p.B, p.H, p.Nq, p.C, p.d, dtype=torch.float32, device=dev) if want_centroids else None
    cnt = torch.empty(p.B, p.H, p.Nq, p.C, dtype=torch.int32, device=dev) if want_centroids else None
    _check(lib().ab_select_static(ctypes.byref(p.c()), _ptr(Q), _ptr(K), _ptr(P), _ptr(cent), _ptr(cnt),
                                  _stream(dev)), "ab_select_static")
    return (P, cent, cnt) if want_centroids else P


def _list_outputs(p: Params, P, out):
    """Checks P and returns (idx, pi_q32, count): `out` if given (checked), else new zeroed tensors."""
    import torch
    if P.dtype != torch.float32 or tuple(P.shape) != (p.B, p.H, p.Nq, p.Nkv) or not P.is_contiguous():
        raise ValueError("P must be contiguous fp32 [B,H,Nq,Nkv]")
    dev = P.device
    if out is None:
        return (torch.zeros(p.B, p.H, p.Nq, p.Nkv, dtype=torch.int32, device=dev),
                torch.zeros(p.B, p.H, p.Nq, p.Nkv, dtype=torch.int32, device=dev),
                torch.zeros(p.B, p.H, p.Nq, dtype=torch.int32, device=dev))
    for t, shape in zip(out, ((p.B, p.H, p.Nq, p.Nkv), (p.B, p.H, p.Nq, p.Nkv), (p.B, p.H, p.Nq))):
        if t.dtype not in (torch.int32, torch.uint32) or tuple(t.shape) != shape or not t.is_contiguous() \
                or t.device != dev:
            raise ValueError(f"list output must be contiguous int32 {shape} on {dev}")
    return tuple(out)


def _lists_call(fn_name, p: Params, P, out=None):
    idx, piq, cnt = _list_outputs(p, P, out)
    _check(getattr(lib(), fn_name)(ctypes.byref(p.c()), _ptr(P), _ptr(idx), _ptr(piq), _ptr(cnt),
                                   _stream(P.device)), fn_name)
    return idx, piq, cnt


def ab_select_sample(p: Params, Q, K, workspace=None, out=None):
    """ab_select then ab_sample in one call (the scoring kernel samples the
    rows it scores when rows have at most 2048 KV blocks); returns
    (P, idx, pi_q32, count), bit-identical to the two calls in a row.
    `out` = (P, idx, pi_q32, count) writes into caller-owned tensors."""
    import torch
    _check_qkv(p, Q, K)
    if out is None:
        P = torch.empty(p.B, p.H, p.Nq, p.Nkv, dtype=torch.float32, device=Q.device)
        idx, piq, cnt = _list_outputs(p, P, None)
    else:
        P, idx, piq, cnt = out
        if P.dtype != torch.float32 or tuple(P.shape) != (p.B, p.H, p.Nq, p.Nkv) or not P.is_contiguous():
            raise ValueError("P must be contiguous float32 [B, H, Nq, Nkv]")
        idx, piq, cnt = _list_outputs(p, P, (idx, piq, cnt))
    ws = alloc_workspace(p, Q.device) if workspace is None else workspace
    _check(lib().ab_select_sample(ctypes.byref(p.c()), _ptr(Q), _ptr(K), _ptr(P), _ptr(idx), _ptr(piq), _ptr(cnt),
                                  _ptr(ws), ws.numel(), _stream(Q.device)), "ab_select_sample")
    return P, idx, piq, cnt


def ab_sample(p: Params, P, out=None):
    """SIP: returns idx [B,H,Nq,Nkv] int32, pi_q32 [B,H,Nq,Nkv] uint32 (as int32 storage), count [B,H,Nq].
    `out` = (idx, pi_q32, count) writes into caller-owned tensors instead."""
    return _lists_call("ab_sample", p, P, out)


def ab_sample_systematic(p: Params, P, out=None):
    """Systematic sampling with SIP's inclusion probabilities: same outputs as ab_sample."""
    return _lists_call("ab_sample_systematic", p, P, out)


def ab_sample_topk(p: Params, P, out=None):
    """Truncation (top-Kb by P, ties to the lower block, pi = 1): same outputs as ab_sample."""
    return _lists_call("ab_sample_topk", p, P, out)


def ab_attention(p: Params, Q, K, V, idx, pi_q32, count, out=None):
    """Packed 1/pi-weighted block-sparse attention; Q [B,H,L,d], K and V
    [B,H,Lk,d]; returns O [B,H,L,d] bf16."""
    import torch
    _check_qkv(p, Q, K, V)
    for t, shape in ((idx, (p.B, p.H, p.Nq, p.Nkv)), (pi_q32, (p.B, p.H, p.Nq, p.Nkv)), (count, (p.B, p.H, p.Nq))):
        if t.dtype not in (torch.int32, torch.uint32) or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"list tensor must be contiguous int32 {shape}")
    O = torch.empty_like(Q) if out is None else out
    _check_bf16(O, (p.B, p.H, p.L, p.d))
    _check(lib().ab_attention(ctypes.byref(p.c()), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx), _ptr(pi_q32),
                              _ptr(count), _ptr(O), _stream(Q.device)), "ab_attention")
    return O


def ab_attention_dense(p: Params, Q, K, V, out=None):
    """Dense softmax(QK^T/sqrt(d))V with the same kernel family; returns O."""
    import torch
    _check_qkv(p, Q, K, V)
    O = torch.empty_like(Q) if out is None else out
    _check_bf16(O, (p.B, p.H, p.L, p.d))
    _check(lib().ab_attention_dense(ctypes.byref(p.c()), _ptr(Q), _ptr(K), _ptr(V), _ptr(O),
                                    _stream(Q.device)), "ab_attention_dense")
    return O


class Buffers:
    """Device buffers of one layer (P, lists, output, workspace)."""

    def __init__(self, p: Params, device):
        import torch
        self.P = torch.empty(p.B, p.H, p.Nq, p.Nkv, dtype=torch.float32, device=device)
        self.idx = torch.zeros(p.B, p.H, p.Nq, p.Nkv, dtype=torch.int32, device=device)
        self.pi_q32 = torch.zeros(p.B, p.H, p.Nq, p.Nkv, dtype=torch.int32, device=device)
        self.count = torch.zeros(p.B, p.H, p.Nq, dtype=torch.int32, device=device)
        self.O = torch.empty(p.B, p.H, p.L, p.d, dtype=torch.bfloat16, device=device)
        self.ws = alloc_workspace(p, device)


def ab_forward(p: Params, Q, K, V, bufs: Buffers | None = None) -> Buffers:
    """ab_select -> ab_sample -> ab_attention on device buffers."""
    _check_qkv(p, Q, K, V)
    b = Buffers(p, Q.device) if bufs is None else bufs
    _check(lib().ab_forward(ctypes.byref(p.c()), _ptr(Q), _ptr(K), _ptr(V), _ptr(b.P), _ptr(b.idx),
                            _ptr(b.pi_q32), _ptr(b.count), _ptr(b.O), _ptr(b.ws), b.ws.numel(),
                            _stream(Q.device)), "ab_forward")
    return b


def head_slices(B: int, H: int, world: int):
    """Contiguous near-equal partition of a layer's B * H heads among `world`
    ranks: [(bh0, nbh), ...], rank r taking flattened heads [bh0, bh0 + nbh)
    (the first B*H % world ranks take one head more).  Every rank gets at
    least one head, so world must not exceed B * H."""
    n = B * H
    if not 1 <= world <= n:
        raise ValueError(f"cannot split {n} heads among {world} ranks")
    base, extra = divmod(n, world)
    out, bh0 = [], 0
    for r in range(world):
        nbh = base + (1 if r < extra else 0)
        out.append((bh0, nbh))
        bh0 += nbh
    return out


def slice_rows(p: Params, bh0: int, nbh: int):
    """(b, h, i) in the whole problem of every row of a slice's per-row
    buffers (P, idx, pi_q32: [nbh, Nq, ...]; count: [nbh, Nq]), in their
    order: local row r is row bh0 * Nq + r of the whole [B, H, Nq] layout.
    These are the counters SIP draws a slice's rows with (the library derives
    the same from the slice's first row and the whole problem's H)."""
    out = []
    for lb in range(nbh):
        b, h = divmod(bh0 + lb, p.H)
        out.extend((b, h, i) for i in range(p.Nq))
    return out


def slice_params(p: Params, nbh: int) -> Params:
    """The problem of one slice of nbh heads (B = 1, H = nbh): its buffer
    shapes and workspace size.  The whole problem's Params stay the ones
    passed to ab_forward_slice."""
    from dataclasses import replace
    return replace(p, B=1, H=nbh)


def ab_forward_slice(p: Params, bh0: int, nbh: int, Q, K, V, bufs: Buffers | None = None) -> Buffers:
    """ab_forward on heads [bh0, bh0 + nbh) of the problem `p` (flattened b * H
    + h): Q [1, nbh, L, d], K and V [1, nbh, Lk, d]; the buffers are the
    slice's (Buffers(slice_params(p, nbh))).  The draws use the whole
    problem's counters, so the result equals those heads of ab_forward(p)."""
    ps = slice_params(p, nbh)
    _check_qkv(ps, Q, K, V)
    b = Buffers(ps, Q.device) if bufs is None else bufs
    _check(lib().ab_forward_slice(ctypes.byref(p.c()), int(bh0), int(nbh), _ptr(Q), _ptr(K), _ptr(V), _ptr(b.P),
                                  _ptr(b.idx), _ptr(b.pi_q32), _ptr(b.count), _ptr(b.O), _ptr(b.ws), b.ws.numel(),
                                  _stream(Q.device)), "ab_forward_slice")
    return b


def ab_forward_host(p: Params, Qh, Kh, Vh, Oh, Qd, Kd, Vd, bufs: Buffers, device):
    """Host bf16 Qh [B,H,L,d], Kh and Vh [B,H,Lk,d] -> host out Oh [B,H,L,d];
    Qd/Kd/Vd are device staging buffers of the same shapes."""
    for t, n in ((Qh, p.L), (Kh, p.Lk), (Vh, p.Lk), (Oh, p.L), (Qd, p.L), (Kd, p.Lk), (Vd, p.Lk)):
        if tuple(t.shape) != (p.B, p.H, n, p.d) or not t.is_contiguous():
            raise ValueError(f"expected contiguous [{p.B},{p.H},{n},{p.d}], got {tuple(t.shape)}")
    _check(lib().ab_forward_host(ctypes.byref(p.c()), _ptr(Qh), _ptr(Kh), _ptr(Vh), _ptr(Oh), _ptr(Qd),
                                 _ptr(Kd), _ptr(Vd), _ptr(bufs.P), _ptr(bufs.idx), _ptr(bufs.pi_q32),
                                 _ptr(bufs.count), _ptr(bufs.O), _ptr(bufs.ws), bufs.ws.numel(),
                                 _stream(device)), "ab_forward_host")


# ------------------------------------------- norm and rotation, paged cache
_marshal_module = None


def _m():
    """The built checks of tensors (csrc/marshal.cpp)."""
    global _marshal_module
    if _marshal_module is None:
        import torch  # its libraries are loaded first
        try:
            from . import _marshal
        except ImportError as e:
            raise RuntimeError("_marshal.so not built; run block_sparse_attention_queries_b200/build.py") from e
        if getattr(_marshal, "built_for", None) != f"AB_TORCH={torch.__version__};":
            raise RuntimeError("_marshal.so was built for another torch; run block_sparse_attention_queries_b200/build.py")
        _marshal_module = _marshal
    return _marshal_module


_fns = {}


def _fn(fn_name):
    """The library's function with every pointer as an address or bytes."""
    ref = getattr(lib(), fn_name)
    fn = lib()[fn_name]
    scalars = (ctypes.c_int32, ctypes.c_size_t)
    fn.argtypes = [t if t in scalars or t in (ctypes.POINTER(ab_params), ctypes.POINTER(ab_paged_params),
                                              ctypes.POINTER(ab_norm_rope)) else ctypes.c_void_p for t in ref.argtypes]
    fn.restype = ref.restype
    _fns[fn_name] = fn
    return fn


def _call(fn_name, index, *args):
    """The library's function on CUDA device `index` and its current stream."""
    import torch
    fn = _fns.get(fn_name) or _fn(fn_name)
    if index == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != AB_OK:
        raise AbError(status, fn_name)


def _cuda_index(t):
    index = t.get_device()
    if index < 0:
        raise ValueError("expected a CUDA tensor")
    return index


def _c(p: Params) -> ab_params:
    """p.c(), made once (Params are immutable)."""
    c = p.__dict__.get("_c")
    if c is None:
        c = p.c()
        object.__setattr__(p, "_c", c)
    return c


def _dense_tokens(p: Params, nr: NormRope, q, k, v, pos_q, pos_k):
    """Checked arguments of the calls from the projections' layout: device, tokens, positions."""
    import torch
    first = q if q is not None else k if k is not None else v
    if first is None:
        raise ValueError("none of q, k, v is given")
    dev = _cuda_index(first)
    nr.check(p.H, p.H, p.d, dev)
    m, L, Lk = _m(), p.L, p.Lk
    kv = (p.B, Lk, p.H, p.d)
    tok = (None if q is None else m.tokens(dev, q, (p.B, L, p.H, p.d), "q"), None if k is None else m.tokens(dev, k, kv, "k"),
           None if v is None else m.tokens(dev, v, kv, "v"))
    pos = (None, None) if pos_q is None and pos_k is None else \
        m.tensors(dev, pos_q, torch.int32, (p.B, L), "pos_q", pos_k, torch.int32, (p.B, Lk), "pos_k")
    return dev, tok, pos


def ab_qk_norm_rope(p: Params, nr: NormRope, q, k=None, v=None, pos_q=None, pos_k=None, out=None):
    """Norm and rotation from the projections' layout to the attention's: q
    [B, L, H, d], k and v [B, Lk, H, d] bf16 (any strides that are multiples of
    8, e.g. slices of a fused projection; each may be None); returns
    (Q, K, V) [B, H, L or Lk, d] bf16 (None for what was not given), ready for
    ``ab_forward``.  pos_q [B, L], pos_k [B, Lk] int32 are the tokens' rows in
    the tables (None: 0, 1, 2, ...).  `out` = (Q, K, V) writes into caller-owned
    tensors."""
    import torch
    bf16 = torch.bfloat16
    dev, tok, pos = _dense_tokens(p, nr, q, k, v, pos_q, pos_k)
    sq, sk = (p.B, p.H, p.L, p.d), (p.B, p.H, p.Lk, p.d)
    if out is None:
        out = tuple(torch.empty(s, dtype=bf16, device=dev) if t is not None else None for t, s in ((q, sq), (k, sk), (v, sk)))
    else:
        out = tuple(o if t is not None else None for t, o in zip((q, k, v), out))
    ptrs = _m().tensors(dev, out[0], bf16, sq, "Q", out[1], bf16, sk, "K", out[2], bf16, sk, "V")
    _call("ab_qk_norm_rope", dev, _c(p), nr._c, *tok, *pos, *ptrs)
    return out


def ab_forward_qkv(p: Params, nr: NormRope, q, k, v, pos_q=None, pos_k=None, bufs: Buffers | None = None) -> Buffers:
    """``ab_qk_norm_rope`` then ``ab_forward``: the path from the projections q
    [B, L, H, d], k and v [B, Lk, H, d].  The rotated tensors are the returned
    buffers' Q, K and V (made on the first call if `bufs` has none)."""
    import torch
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    dev, tok, pos = _dense_tokens(p, nr, q, k, v, pos_q, pos_k)
    if None in tok:
        raise ValueError("q, k and v are all needed")
    b = Buffers(p, q.device) if bufs is None else bufs
    for name, n in (("Q", p.L), ("K", p.Lk), ("V", p.Lk)):
        if getattr(b, name, None) is None:
            setattr(b, name, torch.empty(p.B, p.H, n, p.d, dtype=bf16, device=dev))
    sq, sk, rows = (p.B, p.H, p.L, p.d), (p.B, p.H, p.Lk, p.d), (p.B, p.H, p.Nq, p.Nkv)
    ptrs = _m().tensors(dev, b.Q, bf16, sq, "Q", b.K, bf16, sk, "K", b.V, bf16, sk, "V", b.P, f32, rows, "P", b.idx, i32, rows,
                        "idx", b.pi_q32, b.pi_q32.dtype, rows, "pi_q32", b.count, i32, rows[:3], "count", b.O, bf16, sq, "O",
                        b.ws, torch.uint8, (b.ws.numel(),), "ws")
    _call("ab_forward_qkv", dev, _c(p), nr._c, *tok, *pos, *ptrs, b.ws.numel())
    return b


def paged_workspace_size(pp: PagedParams, select=True) -> int:
    """Bytes of workspace for ab_attention_paged, and with `select` for
    ab_paged_select and ab_paged_forward too."""
    n = ctypes.c_size_t(0)
    _check(lib().ab_paged_workspace_size(pp.c(), int(bool(select)), n), "ab_paged_workspace_size")
    return int(n.value)


def alloc_paged_workspace(pp: PagedParams, device, select=True):
    import torch
    return torch.empty(paged_workspace_size(pp, select), dtype=torch.uint8, device=device)


class PagedCache:
    """A cache's tensors: K, V [num_pages, Hkv, page, d] and ksum
    [num_pages, Hkv, d] bf16, the block table [S, max_pages], the sequences'
    lengths, the list of free pages with its count, and a workspace.  All
    sequences are empty, all pages free."""

    def __init__(self, pp: PagedParams, device, select=True):
        import torch
        kv = (pp.num_pages, pp.Hkv, pp.page, pp.d)
        self.K, self.V = (torch.empty(kv, dtype=torch.bfloat16, device=device) for _ in range(2))
        self.ksum = torch.empty(pp.num_pages, pp.Hkv, pp.d, dtype=torch.bfloat16, device=device)
        self.table = torch.zeros(pp.S, pp.max_pages, dtype=torch.int32, device=device)
        self.lens = torch.zeros(pp.S, dtype=torch.int32, device=device)
        self.free_pages = torch.arange(pp.num_pages - 1, -1, -1, dtype=torch.int32, device=device)
        self.free_count = torch.full((1,), pp.num_pages, dtype=torch.int32, device=device)
        self.ws = alloc_paged_workspace(pp, device, select)


def ab_paged_plan(pp: PagedParams, n_new, lens, table, free_pages, free_count, T=None, lens_out=None,
                  free_count_out=None, out=None):
    """Block tables and slot maps of one step: n_new [S] int32 new tokens per
    sequence (-1: the sequence has ended), lens [S], table [S, max_pages],
    free_pages [num_pages], free_count [1] int32; no page may stand in two rows
    of the table, or in one and the list of free pages.  Updates table and free_pages,
    lens and free_count too (or writes lens_out, free_count_out instead);
    returns (cu_new [S + 1], slots [T], positions [T]).  T: length of the slot
    map (at least the number of new tokens; None with `out`: that of out's
    slots).  `out` = (cu_new, slots, positions) writes into caller-owned
    tensors."""
    import torch
    dev = _cuda_index(n_new)
    i32, seqs, one = torch.int32, (pp.S,), (1,)
    if out is None:
        if T is None:
            raise ValueError("T or out is needed")
        out = (torch.empty(pp.S + 1, dtype=i32, device=dev), torch.empty(T, dtype=i32, device=dev),
               torch.empty(T, dtype=i32, device=dev))
    elif T is None:
        T = out[1].numel()
    ptrs = _m().tensors(dev, n_new, i32, seqs, "n_new", lens, i32, seqs, "lens",
                        lens if lens_out is None else lens_out, i32, seqs, "lens_out",
                        table, i32, (pp.S, pp.max_pages), "table", free_pages, i32, (pp.num_pages,), "free_pages",
                        free_count, i32, one, "free_count", free_count if free_count_out is None else free_count_out, i32, one,
                        "free_count_out", out[0], i32, (pp.S + 1,), "cu_new", out[1], i32, (T,), "slots",
                        out[2], i32, (T,), "positions")
    _call("ab_paged_plan", dev, pp.c(), T, *ptrs)
    return out


def _paged_tokens(pp: PagedParams, nr: NormRope, q, k, v):
    """Checked new tokens: device, their number, the library's arguments."""
    dev = _cuda_index(q)
    T, Hq, Hkv, d = q.shape[0], pp.Hq, pp.Hkv, pp.d
    nr.check(Hq, Hkv, d, dev)
    m, kv = _m(), (T, Hkv, d)
    return dev, T, (m.tokens(dev, q, (T, Hq, d), "q"), m.tokens(dev, k, kv, "k"), m.tokens(dev, v, kv, "v"))


def ab_paged_append(pp: PagedParams, nr: NormRope, q, k, v, slots, positions, K, V, ksum=None, out=None):
    """Norm and rotation of new tokens q [T, Hq, d], k and v [T, Hkv, d] bf16
    (strides as for ab_qk_norm_rope), keys and values written to their slots of
    the cache, the touched pages' means to ksum (None: not kept); returns the
    queries Q [T, Hq, d] (`out` if given; rows of skipped tokens are left as they
    were, in a new Q not set)."""
    import torch
    bf16, i32 = torch.bfloat16, torch.int32
    dev, T, tok = _paged_tokens(pp, nr, q, k, v)
    rows, kv = (T, pp.Hq, pp.d), (pp.num_pages, pp.Hkv, pp.page, pp.d)
    Q = torch.empty(rows, dtype=bf16, device=dev) if out is None else out
    ptrs = _m().tensors(dev, slots, i32, (T,), "slots", positions, i32, (T,), "positions", Q, bf16, rows, "Q", K, bf16, kv, "K",
                        V, bf16, kv, "V", ksum, bf16, (pp.num_pages, pp.Hkv, pp.d), "ksum")
    if T:
        _call("ab_paged_append", dev, pp.c(), nr._c, T, *tok, *ptrs)
    return Q


def _query_rows(pp: PagedParams, Q, cu_new) -> int:
    T = Q.shape[0]
    if cu_new is None and T != pp.S:
        raise ValueError(f"Q has {T} rows, {pp.S} expected without cu_new")
    return T


def ab_paged_select(pp: PagedParams, Q, ksum, table, lens, cu_new=None, workspace=None, out=None):
    """Every page's estimated share P [S, Hkv, max_pages] fp32 of the attention
    mass of each sequence's newest token (entries behind a sequence's last page
    are left as they were, 0 in a new P).  Q [S, Hq, d], or [T, Hq, d] with
    cu_new [S + 1] as ab_paged_plan returns it (T = 0: nothing is done)."""
    import torch
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    dev, T = _cuda_index(Q), _query_rows(pp, Q, cu_new)
    shape = (pp.S, pp.Hkv, pp.max_pages)
    P = torch.zeros(shape, dtype=f32, device=dev) if out is None else out
    ws = alloc_paged_workspace(pp, dev, True) if workspace is None else workspace
    n = ws.numel()
    ptrs = _m().tensors(dev, Q, bf16, (T, pp.Hq, pp.d), "Q", ksum, bf16, (pp.num_pages, pp.Hkv, pp.d), "ksum",
                        table, i32, (pp.S, pp.max_pages), "table", lens, i32, (pp.S,), "lens", cu_new, i32, (pp.S + 1,), "cu_new",
                        P, f32, shape, "P", ws, torch.uint8, (n,), "workspace")
    if T:
        _call("ab_paged_select", dev, pp.c(), T, *ptrs, n)
    return P


def ab_paged_topk(pp: PagedParams, P, lens, out=None):
    """The pages to attend to: (idx [S, Hkv, max_pages], count [S, Hkv]) int32,
    the newest `recent` pages and those of largest P, keep_ratio of them in all."""
    import torch
    i32 = torch.int32
    dev = _cuda_index(P)
    shape = (pp.S, pp.Hkv, pp.max_pages)
    if out is None:
        out = (torch.zeros(shape, dtype=i32, device=dev), torch.zeros(shape[:2], dtype=i32, device=dev))
    ptrs = _m().tensors(dev, P, torch.float32, shape, "P", lens, i32, (pp.S,), "lens", out[0], i32, shape, "idx",
                        out[1], i32, shape[:2], "count")
    _call("ab_paged_topk", dev, pp.c(), *ptrs)
    return out


def ab_attention_paged(pp: PagedParams, Q, K, V, table, lens, idx=None, count=None, cu_new=None, workspace=None,
                       out=None):
    """Attention of each sequence's newest token over the cache (all pages, or
    the listed ones); Q as for ab_paged_select; returns O [S, Hq, d] bf16 (rows
    of sequences without a new token are left as they were, 0 in a new O)."""
    import torch
    bf16, i32 = torch.bfloat16, torch.int32
    dev, T = _cuda_index(Q), _query_rows(pp, Q, cu_new)
    if (idx is None) != (count is None):
        raise ValueError("idx and count come together")
    kv, shape, lists = (pp.num_pages, pp.Hkv, pp.page, pp.d), (pp.S, pp.Hq, pp.d), (pp.S, pp.Hkv, pp.max_pages)
    O = torch.zeros(shape, dtype=bf16, device=dev) if out is None else out
    ws = alloc_paged_workspace(pp, dev, False) if workspace is None else workspace
    n = ws.numel()
    ptrs = _m().tensors(dev, Q, bf16, (T, pp.Hq, pp.d), "Q", K, bf16, kv, "K", V, bf16, kv, "V",
                        table, i32, (pp.S, pp.max_pages), "table", lens, i32, (pp.S,), "lens", cu_new, i32, (pp.S + 1,), "cu_new",
                        idx, i32, lists, "idx", count, i32, lists[:2], "count", O, bf16, shape, "O",
                        ws, torch.uint8, (n,), "workspace")
    if T:
        _call("ab_attention_paged", dev, pp.c(), T, *ptrs, n)
    return O


class PagedBuffers:
    """Outputs of ab_paged_forward: Q [T, Hq, d], P, idx, count and O [S, Hq, d]."""

    def __init__(self, pp: PagedParams, T: int, device):
        import torch
        shape = (pp.S, pp.Hkv, pp.max_pages)
        self.Q = torch.zeros(T, pp.Hq, pp.d, dtype=torch.bfloat16, device=device)
        self.P = torch.zeros(shape, dtype=torch.float32, device=device)
        self.idx = torch.zeros(shape, dtype=torch.int32, device=device)
        self.count = torch.zeros(shape[:2], dtype=torch.int32, device=device)
        self.O = torch.zeros(pp.S, pp.Hq, pp.d, dtype=torch.bfloat16, device=device)


def ab_paged_forward(pp: PagedParams, nr: NormRope, q, k, v, cache: PagedCache, cu_new, slots, positions,
                     bufs: PagedBuffers | None = None) -> PagedBuffers:
    """One step of sparse attention over the cache for new tokens q [T, Hq, d], k
    and v [T, Hkv, d], after ab_paged_plan: append, select, top-k, attention of
    each sequence's newest token.  T = 0 (requests only end): nothing is done."""
    import torch
    bf16, i32 = torch.bfloat16, torch.int32
    if cu_new is None:
        raise ValueError("cu_new is needed")
    dev, T, tok = _paged_tokens(pp, nr, q, k, v)
    c, b = cache, PagedBuffers(pp, T, dev) if bufs is None else bufs
    kv, shape = (pp.num_pages, pp.Hkv, pp.page, pp.d), (pp.S, pp.Hkv, pp.max_pages)
    n = c.ws.numel()
    ptrs = _m().tensors(dev, slots, i32, (T,), "slots", positions, i32, (T,), "positions",
                        c.table, i32, (pp.S, pp.max_pages), "table", c.lens, i32, (pp.S,), "lens", cu_new, i32, (pp.S + 1,), "cu_new",
                        b.Q, bf16, (T, pp.Hq, pp.d), "Q", c.K, bf16, kv, "K", c.V, bf16, kv, "V",
                        c.ksum, bf16, (pp.num_pages, pp.Hkv, pp.d), "ksum", b.P, torch.float32, shape, "P", b.idx, i32, shape, "idx",
                        b.count, i32, shape[:2], "count", b.O, bf16, (pp.S, pp.Hq, pp.d), "O", c.ws, torch.uint8, (n,), "workspace")
    if T:
        _call("ab_paged_forward", dev, pp.c(), nr._c, T, *tok, *ptrs, n)
    return b


def device_error(device=None) -> int:
    """Reads and clears the library's device error word (0 = none)."""
    code = ctypes.c_int32(0)
    _check(lib().ab_get_device_error(_stream(device), ctypes.byref(code)), "ab_get_device_error")
    return int(code.value)


def status_string(code: int) -> str:
    return lib().ab_status_string(int(code)).decode()
