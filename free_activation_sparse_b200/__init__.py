"""Weight-informed activation-sparse linear layer for LLM decode on B200 (sm_100a).

A thin ctypes binding of ``libwina.so`` (the C ABI in ``include/wina.h``). Every step
of the computation runs in the library's CUDA kernels; this module only checks tensor
dtypes/devices, allocates outputs and workspaces through PyTorch, passes raw device
pointers and the current CUDA stream, and turns status codes into exceptions.
Importing it fails if the library has not been built
(``python free_activation_sparse_b200/build.py``).
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

__all__ = [
    "WinaError", "lib", "LIB_PATH", "F32", "BF16", "GATE_TOPK", "GATE_STAT", "GATE_DENSE",
    "abi_version", "normal_quantile", "workspace_size", "Workspace", "FfnWeights",
    "pack_in_major", "col_norms", "select_topk", "stat_topk_threshold", "sparse_matvec",
    "sparse_ffn_swiglu", "ffn_ws_view", "ffn_prepare", "declared_symbols", "sparse_matvec_noalloc",
    "dense_matvec", "dense_ffn_swiglu", "spark_ffn", "ds_channel_absmean", "ds_calibrate_channels",
    "ds_label_build", "ds_decode_attention", "Kv8Cache", "kv8_cache", "kv8_plan", "kv8_write", "kv8_read",
    "kv8_attention",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libwina.so")
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "wina.h")

# enums of wina.h
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED_DTYPE, ERR_WORKSPACE, ERR_CAPACITY, ERR_CUDA, ERR_TIMEOUT = range(7)
F32, BF16 = 0, 1
LAYOUT_OUT_IN, LAYOUT_IN_MAJOR = 0, 1
GATE_TOPK, GATE_STAT, GATE_DENSE = 0, 1, 2
OP_SELECT_TOPK, OP_STAT_THRESHOLD, OP_SPARSE_MATVEC, OP_FFN_SWIGLU, OP_SPARK_FFN, OP_DENSE_FFN = 0, 1, 2, 3, 4, 5
OP_KV8_ATTENTION = 6
KV8_INT8, KV8_E4M3 = 0, 1


class WinaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = int(code)
        super().__init__(f"{where}: {lib.wina_status_string(code).decode()} (status {code})")


class _FfnT(ctypes.Structure):
    _fields_ = [
        ("wt_gate", ctypes.c_void_p), ("wt_up", ctypes.c_void_p), ("wt_down", ctypes.c_void_p),
        ("wdt", ctypes.c_int), ("c_gate", ctypes.c_void_p), ("c_up", ctypes.c_void_p),
        ("c_down", ctypes.c_void_p), ("d", ctypes.c_int64), ("ffn", ctypes.c_int64),
    ]


class _FfnView(ctypes.Structure):
    _fields_ = [("h", ctypes.c_size_t), ("keep_gate", ctypes.c_size_t), ("keep_up", ctypes.c_size_t),
                ("keep_down", ctypes.c_size_t), ("stamps", ctypes.c_size_t), ("cta_t", ctypes.c_size_t)]


class _Kv8T(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("format", ctypes.c_int), ("n_pages", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("page", ctypes.c_int64), ("dh", ctypes.c_int64)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python free_activation_sparse_b200/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I32, D, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double, ctypes.c_size_t
    E = ctypes.c_int
    sig = {
        "wina_abi_version": (I32, []),
        "wina_set_wait_limit_ns": (None, [ctypes.c_uint64]),
        "wina_status_string": (ctypes.c_char_p, [E]),
        "wina_normal_quantile": (D, [D]),
        "wina_workspace_size": (SZ, [E, I64, I64, I64, I64]),
        "wina_ffn_ws_view": (E, [I64, I64, I64, ctypes.POINTER(_FfnView)]),
        "wina_pack_in_major": (E, [P, E, I64, I64, P, P]),
        "wina_col_norms": (E, [P, E, I64, I64, E, P, P]),
        "wina_select_topk": (E, [P, E, P, I64, I64, I64, P, P, P, P]),
        "stat_topk_threshold": (E, [P, E, I64, D, I64, P, P, P, P, I64, P, P]),
        "sparse_matvec": (E, [P, E, I64, I64, P, P, I64, P, I64, I64, P, P, SZ, P, P]),
        "sparse_matvec_noalloc": (E, [P, E, I64, I64, P, P, I64, P, I64, I64, P, P, P]),
        "sparse_ffn_swiglu": (E, [ctypes.POINTER(_FfnT), P, E, I64, E, I64, I64, I64, D, P, P, SZ, P, P]),
        "wina_dense_matvec": (E, [P, E, I64, I64, P, E, P, P, P]),
        "spark_ffn_swiglu": (E, [P, P, P, E, I64, I64, P, E, D, P, P, P, P, P, SZ, P, P]),
        "wina_dense_ffn_swiglu": (E, [P, P, P, E, I64, I64, P, E, P, P, SZ, P, P]),
        "ds_channel_absmean": (E, [P, E, I64, I64, I64, I64, P, P, P]),
        "ds_label_build": (E, [P, E, I64, I64, I64, I64, P, P, I64, I64, I64, P, P]),
        "ds_decode_smem_bytes": (SZ, [I64, I64, I64]),
        "ds_decode_attention": (E, [P, E, P, P, P, E, P, I64, I64, I64, I64, I64, I64, P, I64, ctypes.c_float, P, P, P,
                                    P]),
        "kv8_plan": (E, [P, P, I64, I64, P, I64, P, I64, P, I64, P, P, P, P, P, P, P]),
        "kv8_write": (E, [ctypes.POINTER(_Kv8T), P, P, E, I64, I64, I64, P, P, P]),
        "kv8_read": (E, [ctypes.POINTER(_Kv8T), P, I64, P, P, E, P, P]),
        "kv8_attention": (E, [ctypes.POINTER(_Kv8T), P, E, I64, I64, I64, P, I64, P, P, I64, I64, ctypes.c_float, I64,
                              ctypes.c_float, P, P, SZ, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


lib = _load()


def declared_symbols() -> list[str]:
    """Function names declared in include/wina.h (parsed from the header text)."""
    import re
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(\w+)\s*\(", text, flags=re.M)) - {"defined"})


# ------------------------------------------------------------------------------------
# marshalling helpers (no arithmetic of the method here)
# ------------------------------------------------------------------------------------


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dt(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _cuda(t, name):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check(code: int, where: str):
    if code != OK:
        raise WinaError(code, where)


def abi_version() -> int:
    return int(lib.wina_abi_version())


def normal_quantile(p: float) -> float:
    """Phi^-1(p), computed by the library's host code."""
    return float(lib.wina_normal_quantile(float(p)))


def workspace_size(op: int, n: int, m: int, k: int, batch: int) -> int:
    return int(lib.wina_workspace_size(int(op), int(n), int(m), int(k), int(batch)))


class Workspace:
    """A zero-filled device scratch buffer for one op and size (reusable across calls
    of that op on one stream)."""

    def __init__(self, op: int, n: int, m: int, k: int, batch: int, device=None):
        torch = _torch()
        nbytes = max(workspace_size(op, n, m, k, batch), 256)
        self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")
        self.nbytes = nbytes

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())


# ------------------------------------------------------------------------------------
# public calls
# ------------------------------------------------------------------------------------


def pack_in_major(W):
    """W[m][n] -> Wt[n][m] (input-channel-major), same dtype."""
    torch = _torch()
    _cuda(W, "W")
    m, n = W.shape
    Wt = torch.empty((n, m), dtype=W.dtype, device=W.device)
    _check(lib.wina_pack_in_major(_ptr(W), _dt(W), m, n, _ptr(Wt), _stream()), "wina_pack_in_major")
    return Wt


def col_norms(W, layout: str = "out_in"):
    """float32 column norms c[n] of W[m][n] ('out_in') or of the packed Wt[n][m] ('in_major')."""
    torch = _torch()
    _cuda(W, "W")
    if layout == "out_in":
        m, n = W.shape
        lay = LAYOUT_OUT_IN
    elif layout == "in_major":
        n, m = W.shape
        lay = LAYOUT_IN_MAJOR
    else:
        raise ValueError(layout)
    c = torch.empty(n, dtype=torch.float32, device=W.device)
    _check(lib.wina_col_norms(_ptr(W), _dt(W), m, n, lay, _ptr(c), _stream()), "wina_col_norms")
    return c


def select_topk(x, c, k: int, want_scores: bool = False):
    """Top-k gate per token: returns (idx int32 [B][k] ascending, xs float32 [B][k]
    [, scores float32 [B][n]])."""
    torch = _torch()
    _cuda(x, "x")
    _cuda(c, "c")
    x2 = x.reshape(1, -1) if x.dim() == 1 else x
    B, n = x2.shape
    idx = torch.empty((B, k), dtype=torch.int32, device=x.device)
    xs = torch.empty((B, k), dtype=torch.float32, device=x.device)
    sc = torch.empty((B, n), dtype=torch.float32, device=x.device) if want_scores else None
    _check(lib.wina_select_topk(_ptr(x2), _dt(x2), _ptr(c), n, k, B, _ptr(idx), _ptr(xs), _ptr(sc), _stream()),
           "wina_select_topk")
    return (idx, xs, sc) if want_scores else (idx, xs)


def stat_topk_threshold(v, s: float, cap: int | None = None, status=None):
    """Spark statistical gate per row of v: returns (idx [B][cap], xs [B][cap],
    count [B], t [B]). Entries past count are unspecified."""
    torch = _torch()
    _cuda(v, "v")
    v2 = v.reshape(1, -1) if v.dim() == 1 else v
    B, n = v2.shape
    cap = n if cap is None else int(cap)
    idx = torch.empty((B, max(cap, 1)), dtype=torch.int32, device=v.device)
    xs = torch.empty((B, max(cap, 1)), dtype=torch.float32, device=v.device)
    count = torch.empty(B, dtype=torch.int32, device=v.device)
    t = torch.empty(B, dtype=torch.float32, device=v.device)
    _check(lib.stat_topk_threshold(_ptr(v2), _dt(v2), n, float(s), B, _ptr(idx), _ptr(xs), _ptr(count), _ptr(t),
                                   cap, _ptr(status), _stream()), "stat_topk_threshold")
    return idx[:, :cap], xs[:, :cap], count, t


def sparse_matvec(Wt, idx, xs, k: int | None = None, count=None, ws: Workspace | None = None, status=None, y=None):
    """y[b] = sum_r xs[b][r] * Wt[idx[b][r]] over the first k (or count[b]) entries."""
    torch = _torch()
    for t_, nm in ((Wt, "Wt"), (idx, "idx"), (xs, "xs"), (count, "count")):
        _cuda(t_, nm)
    if idx.dtype != torch.int32 or xs.dtype != torch.float32:
        raise TypeError("idx must be int32 and xs float32")
    idx2 = idx.reshape(1, -1) if idx.dim() == 1 else idx
    xs2 = xs.reshape(1, -1) if xs.dim() == 1 else xs
    n, m = Wt.shape
    B, ld = idx2.shape
    if k is None and count is None:
        k = ld
    kk = -1 if k is None else int(k)
    if ws is None:
        ws = Workspace(OP_SPARSE_MATVEC, n, m, ld, B, device=Wt.device)
    if y is None:
        y = torch.empty((B, m), dtype=torch.float32, device=Wt.device)
    _check(lib.sparse_matvec(_ptr(Wt), _dt(Wt), n, m, _ptr(idx2), _ptr(xs2), kk, _ptr(count), ld, B, _ptr(y),
                             ws.ptr, ws.nbytes, _ptr(status), _stream()), "sparse_matvec")
    return y


def sparse_matvec_noalloc(Wt, idx, xs, k: int | None = None, count=None, status=None, y=None):
    """sparse_matvec without a workspace: the library's own fixed scratch is used (for
    callers that cannot allocate device memory; see include/wina.h for its limit and
    the rule that such calls must not overlap)."""
    torch = _torch()
    for t_, nm in ((Wt, "Wt"), (idx, "idx"), (xs, "xs"), (count, "count")):
        _cuda(t_, nm)
    if idx.dtype != torch.int32 or xs.dtype != torch.float32:
        raise TypeError("idx must be int32 and xs float32")
    idx2 = idx.reshape(1, -1) if idx.dim() == 1 else idx
    xs2 = xs.reshape(1, -1) if xs.dim() == 1 else xs
    n, m = Wt.shape
    B, ld = idx2.shape
    if k is None and count is None:
        k = ld
    kk = -1 if k is None else int(k)
    if y is None:
        y = torch.empty((B, m), dtype=torch.float32, device=Wt.device)
    _check(lib.sparse_matvec_noalloc(_ptr(Wt), _dt(Wt), n, m, _ptr(idx2), _ptr(xs2), kk, _ptr(count), ld, B,
                                     _ptr(y), _ptr(status), _stream()), "sparse_matvec_noalloc")
    return y


@dataclass
class FfnWeights:
    """Packed SwiGLU FFN: wt_gate/wt_up [d][ffn], wt_down [ffn][d] (input-major), and
    the float32 column norms of W_gate, W_up (length d) and W_down (length ffn)."""
    wt_gate: object
    wt_up: object
    wt_down: object
    c_gate: object
    c_up: object
    c_down: object

    @property
    def d(self) -> int:
        return int(self.wt_gate.shape[0])

    @property
    def ffn(self) -> int:
        return int(self.wt_gate.shape[1])

    def _struct(self) -> _FfnT:
        key = (self.wt_gate.data_ptr(), self.wt_up.data_ptr(), self.wt_down.data_ptr(), self.c_gate.data_ptr(),
               self.c_up.data_ptr(), self.c_down.data_ptr())
        cached = self.__dict__.get("_cstruct")
        if cached is None or cached[0] != key:
            st = _FfnT(key[0], key[1], key[2], _dt(self.wt_gate), key[3], key[4], key[5], self.d, self.ffn)
            self.__dict__["_cstruct"] = cached = (key, st)
        return cached[1]


def ffn_prepare(W_gate, W_up, W_down) -> FfnWeights:
    """Offline preparation of one FFN from W_gate, W_up [ffn][d] and W_down [d][ffn]
    (output-major, as multiplied by x): pack input-major and take column norms."""
    return FfnWeights(pack_in_major(W_gate), pack_in_major(W_up), pack_in_major(W_down),
                      col_norms(W_gate), col_norms(W_up), col_norms(W_down))


def sparse_ffn_swiglu(f: FfnWeights, x, mode: int = GATE_TOPK, k_gate: int = 0, k_up: int = 0, k_down: int = 0,
                      s: float = 0.08, ws: Workspace | None = None, status=None, y=None):
    """Gated SwiGLU FFN for x [B][d]: returns y float32 [B][d]."""
    torch = _torch()
    _cuda(x, "x")
    x2 = x.reshape(1, -1) if x.dim() == 1 else x
    B = x2.shape[0]
    if ws is None:
        ws = Workspace(OP_FFN_SWIGLU, f.d, f.ffn, 0, B, device=x.device)
    if y is None:
        y = torch.empty((B, f.d), dtype=torch.float32, device=x.device)
    _check(lib.sparse_ffn_swiglu(ctypes.byref(f._struct()), _ptr(x2), _dt(x2), B, int(mode), int(k_gate), int(k_up),
                                 int(k_down), float(s), _ptr(y), ws.ptr, ws.nbytes, _ptr(status), _stream()),
           "sparse_ffn_swiglu")
    return y


def dense_matvec(W, x, y=None, xbuf=None):
    """The dense comparator y = W x on the output-major W [m][n] (one token)."""
    torch = _torch()
    _cuda(W, "W")
    _cuda(x, "x")
    m, n = W.shape
    if y is None:
        y = torch.empty(m, dtype=torch.float32, device=W.device)
    if xbuf is None:
        xbuf = torch.empty(n, dtype=torch.float32, device=W.device)
    _check(lib.wina_dense_matvec(_ptr(W), _dt(W), m, n, _ptr(x), _dt(x), _ptr(y), _ptr(xbuf), _stream()),
           "wina_dense_matvec")
    return y


def dense_ffn_swiglu(W_gate, W_up, W_down, x, y=None, ws: Workspace | None = None, status=None):
    """The dense comparator of the FFN on the output-major weights (one token): returns y [d]."""
    torch = _torch()
    for t_, nm in ((W_gate, "W_gate"), (W_up, "W_up"), (W_down, "W_down"), (x, "x")):
        _cuda(t_, nm)
    ffn, d = W_gate.shape
    if y is None:
        y = torch.empty(d, dtype=torch.float32, device=x.device)
    if ws is None:
        ws = Workspace(OP_DENSE_FFN, d, ffn, 0, 1, device=x.device)
    _check(lib.wina_dense_ffn_swiglu(_ptr(W_gate), _ptr(W_up), _ptr(W_down), _dt(W_gate), d, ffn, _ptr(x), _dt(x),
                                     _ptr(y), ws.ptr, ws.nbytes, _ptr(status) if status is not None else None,
                                     _stream()), "wina_dense_ffn_swiglu")
    return y


def spark_ffn(W_gate, W_up, Wt_down, x, s: float = 0.08, ws: Workspace | None = None, status=None, y=None):
    """The Spark FFN as a key-value lookup for one token: W_gate, W_up output-major [ffn][d],
    Wt_down input-major [ffn][d]. Returns (y [d], g [ffn], idx [ffn] (first count valid),
    count [1])."""
    torch = _torch()
    for t_, nm in ((W_gate, "W_gate"), (W_up, "W_up"), (Wt_down, "Wt_down"), (x, "x")):
        _cuda(t_, nm)
    ffn, d = W_gate.shape
    if ws is None:
        ws = Workspace(OP_SPARK_FFN, d, ffn, 0, 1, device=x.device)
    if y is None:
        y = torch.empty(d, dtype=torch.float32, device=x.device)
    g = torch.empty(ffn, dtype=torch.float32, device=x.device)
    idx = torch.empty(ffn, dtype=torch.int32, device=x.device)
    count = torch.empty(1, dtype=torch.int32, device=x.device)
    _check(lib.spark_ffn_swiglu(_ptr(W_gate), _ptr(W_up), _ptr(Wt_down), _dt(W_gate), d, ffn, _ptr(x), _dt(x),
                                float(s), _ptr(y), _ptr(g), _ptr(idx), _ptr(count), ws.ptr, ws.nbytes, _ptr(status),
                                _stream()), "spark_ffn_swiglu")
    return y, g, idx, count


def ffn_ws_view(ws: Workspace, d: int, ffn: int, batch: int) -> dict:
    """Views of the intermediate results a sparse_ffn_swiglu call leaves in `ws`:
    h [B][ffn] float32; keep_gate, keep_up [B][d] and keep_down [B][ffn] as 0/1 bytes;
    the single-token kernel's phase clock stamps [16] (int64 SM cycles of CTA 0) and
    per-CTA phase end times cta_t [296][4] (int64 ns)."""
    torch = _torch()
    v = _FfnView()
    _check(lib.wina_ffn_ws_view(d, ffn, batch, ctypes.byref(v)), "wina_ffn_ws_view")
    buf = ws.buf

    def take(off, count, dtype, shape):
        nb = count * torch.empty(0, dtype=dtype).element_size()
        return buf[off: off + nb].view(dtype).view(*shape)

    return dict(
        h=take(v.h, batch * ffn, torch.float32, (batch, ffn)),
        keep_gate=take(v.keep_gate, batch * d, torch.uint8, (batch, d)),
        keep_up=take(v.keep_up, batch * d, torch.uint8, (batch, d)),
        keep_down=take(v.keep_down, batch * ffn, torch.uint8, (batch, ffn)),
        stamps=take(v.stamps, 16, torch.int64, (16,)),
        cta_t=take(v.cta_t, 296 * 4, torch.int64, (296, 4)),
    )


# ------------------------------------------------------------------------------------
# Double Sparsity decode attention
# ------------------------------------------------------------------------------------


def ds_channel_absmean(K, seq_len):
    """Mean |K| per (key/value head, channel) over the valid tokens: K [B][Hkv][Tmax][dh],
    seq_len int32 [B] -> float32 [Hkv][dh]."""
    torch = _torch()
    _cuda(K, "K")
    _cuda(seq_len, "seq_len")
    B, Hkv, Tmax, dh = K.shape
    out = torch.empty((Hkv, dh), dtype=torch.float32, device=K.device)
    _check(lib.ds_channel_absmean(_ptr(K), _dt(K), B, Hkv, Tmax, dh, _ptr(seq_len), _ptr(out), _stream()),
           "ds_channel_absmean")
    return out


def ds_calibrate_channels(K, seq_len, r: int):
    """The K-outlier channels: the r channels of largest mean |K| per key/value head,
    ascending (int32 [Hkv][r]); the means go through the top-K gate kernel."""
    a = ds_channel_absmean(K, seq_len)
    idx, _ = select_topk(a, None, r)
    return idx


def ds_label_build(K, seq_len, channels, t0: int = 0, t1: int | None = None, label=None):
    """The label cache [B][Hkv][Tmax][r] (K's dtype) for tokens [t0, t1)."""
    torch = _torch()
    for t_, nm in ((K, "K"), (seq_len, "seq_len"), (channels, "channels")):
        _cuda(t_, nm)
    B, Hkv, Tmax, dh = K.shape
    r = channels.shape[1]
    if t1 is None:
        t1 = Tmax
    if label is None:
        label = torch.zeros((B, Hkv, Tmax, r), dtype=K.dtype, device=K.device)
    _check(lib.ds_label_build(_ptr(K), _dt(K), B, Hkv, Tmax, dh, _ptr(seq_len), _ptr(channels), r, t0, t1,
                              _ptr(label), _stream()), "ds_label_build")
    return label


def ds_decode_attention(q, K, V, label, channels, seq_len, k: int, scale: float = 0.0, out=None,
                        want_idx: bool = False, want_scores: bool = False, status=None):
    """One Double Sparsity decode step: q [B][Hq][dh] -> out float32 [B][Hq][dh]; with
    want_idx / want_scores also the kept tokens [B][Hq][k] and the approximate scores
    [B][Hq][Tmax]. Returns (out, idx or None, scores or None)."""
    torch = _torch()
    for t_, nm in ((q, "q"), (K, "K"), (V, "V"), (label, "label"), (channels, "channels"), (seq_len, "seq_len")):
        _cuda(t_, nm)
    B, Hq, dh = q.shape
    _, Hkv, Tmax, _ = K.shape
    r = channels.shape[1]
    if out is None:
        out = torch.empty((B, Hq, dh), dtype=torch.float32, device=q.device)
    idx = torch.full((B, Hq, k), -1, dtype=torch.int32, device=q.device) if want_idx else None
    sc = torch.zeros((B, Hq, Tmax), dtype=torch.float32, device=q.device) if want_scores else None
    _check(lib.ds_decode_attention(_ptr(q), _dt(q), _ptr(K), _ptr(V), _ptr(label), _dt(K), _ptr(channels), B, Hq,
                                   Hkv, Tmax, dh, r, _ptr(seq_len), k, float(scale), _ptr(out),
                                   _ptr(idx) if idx is not None else None, _ptr(sc) if sc is not None else None,
                                   _ptr(status) if status is not None else None, _stream()), "ds_decode_attention")
    return out, idx, sc


# ------------------------------------------------------------------------------------
# the 8-bit paged key/value cache
# ------------------------------------------------------------------------------------


def _on(dev, names, *tensors):
    """Every tensor given (named in `names`) is a contiguous int32 tensor on `dev`."""
    i32 = _torch().int32
    for i, t in enumerate(tensors):
        if t is not None and not (t.dtype is i32 and t.device == dev and t.is_contiguous()):
            name = names.split()[i]
            if t.dtype is not i32:
                raise TypeError(f"{name} must be int32, not {t.dtype}")
            raise ValueError(f"{name} must be contiguous and on {dev} (is on {t.device})")


def _addr(t):
    return None if t is None else t.data_ptr()


def _launch(dev, where, fn, *args):
    """Call `fn` with the current stream of `dev` as its last argument, `dev` being current."""
    if dev.type != "cuda":
        raise ValueError(f"{where}: tensors must be on a CUDA device")
    torch, index = _torch(), dev.index
    # the stream as a number: the Stream object would cost 2 us of a call's 12
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch._C._cuda_getDevice():
        code = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, stream)
    if code != OK:
        raise WinaError(code, where)


@dataclass
class Kv8Cache:
    """The pages of an 8-bit key/value cache: k, v int8 or float8_e4m3fn
    [n_pages][heads][page][dh], and one float32 scale per page and head, k_scale and v_scale
    [n_pages][heads]; a value is scale * byte."""
    k: object
    v: object
    k_scale: object
    v_scale: object

    @property
    def n_pages(self) -> int:
        return int(self.k.shape[0])

    @property
    def heads(self) -> int:
        return int(self.k.shape[1])

    @property
    def page(self) -> int:
        return int(self.k.shape[2])

    @property
    def dh(self) -> int:
        return int(self.k.shape[3])

    def _struct(self) -> _Kv8T:
        torch = _torch()
        k, v = self.k, self.v
        dt = k.dtype
        if v.dtype is not dt or (dt is not torch.int8 and dt is not torch.float8_e4m3fn):
            raise TypeError("k and v must both be int8 or both float8_e4m3fn")
        fmt, shape = KV8_INT8 if dt is torch.int8 else KV8_E4M3, k.shape
        if len(shape) != 4 or v.shape != shape:
            raise ValueError("k and v must be [n_pages][heads][page][dh], of one shape")
        n, h, page, dh = shape
        dev = k.device
        for t in (self.k_scale, self.v_scale):
            if t.dtype is not torch.float32:
                raise TypeError("k_scale and v_scale must be float32")
            if t.shape != (n, h) or not t.is_contiguous() or t.device != dev:
                raise ValueError(f"k_scale and v_scale must be contiguous [n_pages][heads] on {dev}")
        if v.device != dev or not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("k and v must be contiguous and on one device")
        return _Kv8T(k.data_ptr(), v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(), fmt, n, h, page, dh)


def kv8_cache(n_pages: int, heads: int, page: int, dh: int, dtype=None, device=None) -> Kv8Cache:
    """A zero-filled 8-bit cache (dtype: int8, the default, or float8_e4m3fn)."""
    torch = _torch()
    dtype = torch.int8 if dtype is None else dtype
    if dtype not in (torch.int8, torch.float8_e4m3fn):
        raise TypeError("dtype must be int8 or float8_e4m3fn")
    dev = device or "cuda"
    k, v = (torch.zeros((n_pages, heads, page, dh), dtype=torch.int8, device=dev).view(dtype) for _ in range(2))
    ks, vs = (torch.zeros((n_pages, heads), dtype=torch.float32, device=dev) for _ in range(2))
    return Kv8Cache(k, v, ks, vs)


def kv8_plan(seq_len, new_len, table, free_pages, n_free, page: int, tokens: int, kv_len=None, cu_q=None, slots=None,
             positions=None, n_free_out=None, status=None):
    """Where one step's tokens go. seq_len, new_len int32 [B] (new_len < 0 ends a request);
    table int32 [B][width], free_pages int32 [cells] and its count n_free int32 [1] are the
    page tables and the stack of free pages, updated in place (the count into n_free_out).
    Returns (kv_len [B], cu_q [B + 1], slots [tokens], positions [tokens], n_free_out [1]),
    allocated where not given; kv_len may be seq_len itself and n_free_out n_free."""
    torch = _torch()
    i32, dev = torch.int32, seq_len.device
    B = seq_len.shape[0]
    new = lambda n: torch.empty(n, dtype=i32, device=dev)  # noqa: E731
    kv_len = new(B) if kv_len is None else kv_len
    cu_q = new(B + 1) if cu_q is None else cu_q
    slots = new(tokens) if slots is None else slots
    positions = new(tokens) if positions is None else positions
    n_free_out = new(1) if n_free_out is None else n_free_out
    _on(dev, "seq_len new_len table free_pages n_free kv_len cu_q slots positions n_free_out status", seq_len, new_len,
        table, free_pages, n_free, kv_len, cu_q, slots, positions, n_free_out, status)
    if seq_len.dim() != 1 or new_len.shape != seq_len.shape or table.dim() != 2 or table.shape[0] != B:
        raise ValueError("seq_len and new_len must be [B] and table [B][width]")
    if kv_len.numel() != B or cu_q.numel() != B + 1 or slots.numel() != tokens or positions.numel() != tokens or \
            n_free.numel() != 1 or n_free_out.numel() != 1:
        raise ValueError("kv_len [B], cu_q [B + 1], slots and positions [tokens], n_free and n_free_out [1]")
    _launch(dev, "kv8_plan", lib.kv8_plan, _addr(seq_len), _addr(new_len), B, page, _addr(table), table.shape[1],
            _addr(free_pages), free_pages.numel(), _addr(n_free), tokens, _addr(kv_len), _addr(cu_q), _addr(slots),
            _addr(positions), _addr(n_free_out), _addr(status))
    return kv_len, cu_q, slots, positions, n_free_out


def _rows(t, name, heads, dh):
    """The row stride of t [T][heads][dh], whose rows are contiguous and may lie apart."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dh:
        raise ValueError(f"{name} must be [T][{heads}][{dh}]")
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != dh):
        raise ValueError(f"{name}'s rows must be contiguous (a token's heads side by side)")
    return s[0] if t.shape[0] > 1 else heads * dh


def kv8_write(cache: Kv8Cache, k, v, slots, status=None) -> Kv8Cache:
    """New keys and values [T][heads][dh] (bf16 or float32, rows may be slices of a wider
    tensor's) into the pages of `cache`, at slots int32 [T] (negative: skipped)."""
    c = cache._struct()
    dev = cache.k.device
    dt = _dt(k)
    if v.dtype != k.dtype:
        raise TypeError("k and v must have one dtype")
    if k.device != dev or v.device != dev:
        raise ValueError(f"k and v must be on {dev}")
    ld_k, ld_v = _rows(k, "k", c.heads, c.dh), _rows(v, "v", c.heads, c.dh)
    _on(dev, "slots status", slots, status)
    T = k.shape[0]
    if v.shape[0] != T or slots.numel() != T:
        raise ValueError("k, v and slots must have one length")
    _launch(dev, "kv8_write", lib.kv8_write, ctypes.byref(c), _addr(k), _addr(v), dt, T, ld_k, ld_v, _addr(slots),
            _addr(status))
    return cache


def kv8_read(cache: Kv8Cache, slots, dtype=None, k=None, v=None, status=None):
    """The cached rows at slots int32 [T] as (k, v) [T][heads][dh] of dtype (bf16, the
    default, or float32; that of k and v where they are given); zeros for negative slots."""
    torch = _torch()
    c = cache._struct()
    dev, T = cache.k.device, slots.numel()
    shape = (T, c.heads, c.dh)
    if k is None:
        k = torch.empty(shape, dtype=dtype or (torch.bfloat16 if v is None else v.dtype), device=dev)
    if v is None:
        v = torch.empty(shape, dtype=k.dtype, device=dev)
    dt = _dt(k)
    if dtype is not None and k.dtype != dtype:
        raise TypeError(f"k must be {dtype}")
    _on(dev, "slots status", slots, status)
    if v.dtype is not k.dtype:
        raise TypeError("k and v must have one dtype")
    for t in (k, v):
        if t.shape != shape or t.device != dev or not t.is_contiguous():
            raise ValueError(f"k and v must be contiguous {list(shape)} on {dev}")
    _launch(dev, "kv8_read", lib.kv8_read, ctypes.byref(c), _addr(slots), T, _addr(k), _addr(v), dt, _addr(status))
    return k, v


def kv8_attention(cache: Kv8Cache, q, table, kv_len, cu_q=None, max_q: int = 1, scale: float = 0.0, window: int = 0,
                  softcap: float = 0.0, ws: Workspace | None = None, out=None, status=None):
    """Causal attention of q [T][Hq][dh] (bf16 or float32; rows may be slices of a wider
    tensor's) over the pages: request b's queries are rows cu_q[b] .. cu_q[b + 1] - 1 (at
    most max_q; cu_q None: one row each), the last of them at key kv_len[b] - 1. Returns out
    [T][Hq][dh] in q's dtype; with `out` given, rows behind the last request stay as they were."""
    torch = _torch()
    c = cache._struct()
    dev = cache.k.device
    dt = _dt(q)
    if q.device != dev:
        raise ValueError(f"q must be on {dev}")
    if q.dim() != 3:
        raise ValueError("q must be [T][Hq][dh]")
    T, Hq = q.shape[0], q.shape[1]
    ld_q = _rows(q, "q", Hq, c.dh)
    B = kv_len.numel()
    if out is None:
        out = torch.zeros((T, Hq, c.dh), dtype=q.dtype, device=dev)
    _on(dev, "table kv_len cu_q status", table, kv_len, cu_q, status)
    if out.dtype is not q.dtype:
        raise TypeError(f"out must be {q.dtype}")
    if table.dim() != 2 or table.shape[0] != B or (cu_q is not None and cu_q.numel() != B + 1):
        raise ValueError("table must be [B][width], kv_len [B] and cu_q [B + 1]")
    if out.shape != (T, Hq, c.dh) or out.device != dev or not out.is_contiguous():
        raise ValueError(f"out must be contiguous {[T, Hq, c.dh]} on {dev}")
    if Hq < 1 or Hq % c.heads:
        raise ValueError(f"{Hq} query heads over {c.heads} key/value heads")
    if ws is None:
        ws = Workspace(OP_KV8_ATTENTION, c.dh, max_q * (Hq // c.heads), 0, B, device=dev)
    elif ws.buf.device != dev:
        raise ValueError(f"ws must be on {dev}")
    _launch(dev, "kv8_attention", lib.kv8_attention, ctypes.byref(c), _addr(q), dt, T, ld_q, Hq, _addr(table),
            table.shape[1], _addr(kv_len), _addr(cu_q), B, max_q, scale, window, softcap, _addr(out), ws.buf.data_ptr(),
            ws.nbytes, _addr(status))
    return out
