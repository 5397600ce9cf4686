"""Host-side checks of the 8-bit cache's entry points (CPU only, no kernel launches): bad
arguments return the documented codes before any CUDA call, and the binding's own checks
raise."""

from __future__ import annotations

import ctypes
import shutil
import subprocess

import pytest
import torch

import free_activation_sparse_b200 as W
from free_activation_sparse_b200 import build

FAKE = 1 << 20  # a 16-byte-aligned address that is never dereferenced
ODD = FAKE + 2
BIG = 1 << 62


def desc(**kw):
    a = dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, fmt=W.KV8_INT8, n_pages=100, heads=8, page=16, dh=128)
    a.update(kw)
    return W._Kv8T(a["k"], a["v"], a["ks"], a["vs"], a["fmt"], a["n_pages"], a["heads"], a["page"], a["dh"])


BAD_CACHES = [dict(k=None), dict(vs=None), dict(page=8), dict(page=48), dict(page=256), dict(page=0), dict(dh=32),
              dict(dh=96), dict(n_pages=0), dict(n_pages=1 << 27), dict(n_pages=BIG), dict(heads=0), dict(heads=1025),
              dict(k=ODD), dict(ks=FAKE + 1)]


def test_plan_rejects_bad_arguments():
    def call(seq=FAKE, B=4, page=16, width=8, cells=100, tokens=4, slots=FAKE, pos=None, out=FAKE, status=None, cu=FAKE):
        return W.lib.kv8_plan(seq, FAKE, B, page, FAKE, width, FAKE, cells, FAKE, tokens, FAKE, cu, slots, pos, out, status,
                              None)

    for kw in (dict(seq=None), dict(seq=FAKE + 1), dict(B=0), dict(B=8193), dict(B=BIG), dict(page=0), dict(page=17),
               dict(width=0), dict(width=1 << 27), dict(width=BIG), dict(cells=0), dict(cells=(1 << 30) + 1),
               dict(tokens=-1), dict(tokens=BIG), dict(slots=None), dict(slots=FAKE + 4), dict(pos=FAKE + 8),
               dict(out=None), dict(status=FAKE + 1), dict(cu=None)):
        assert call(**kw) == W.ERR_INVALID_ARG, kw


def test_write_and_read_reject_bad_arguments():
    def write(c=desc(), k=FAKE, v=FAKE, dt=W.BF16, T=4, ld_k=1024, ld_v=1024, slots=FAKE, status=None):
        return W.lib.kv8_write(ctypes.byref(c) if c is not None else None, k, v, dt, T, ld_k, ld_v, slots, status, None)

    def read(c=desc(), slots=FAKE, T=4, k=FAKE, v=FAKE, dt=W.BF16, status=None):
        return W.lib.kv8_read(ctypes.byref(c) if c is not None else None, slots, T, k, v, dt, status, None)

    for call in (write, read):
        assert call(c=None) == W.ERR_INVALID_ARG
        for kw in BAD_CACHES:
            assert call(c=desc(**kw)) == W.ERR_INVALID_ARG, kw
        assert call(c=desc(fmt=2)) == W.ERR_UNSUPPORTED_DTYPE
        assert call(dt=7) == W.ERR_UNSUPPORTED_DTYPE
        for kw in (dict(T=-1), dict(T=BIG), dict(slots=None), dict(slots=FAKE + 1), dict(k=ODD), dict(status=FAKE + 1)):
            assert call(**kw) == W.ERR_INVALID_ARG, kw
        assert call(T=0) == W.OK  # nothing to do: nothing is launched
    for kw in (dict(k=None), dict(v=ODD), dict(ld_k=1023), dict(ld_v=1000), dict(ld_k=1025), dict(ld_k=1028),
               dict(ld_k=BIG), dict(ld_v=-1024)):
        assert write(**kw) == W.ERR_INVALID_ARG, kw
    assert read(k=None, v=None) == W.OK


def test_attention_rejects_bad_arguments():
    need = W.workspace_size(W.OP_KV8_ATTENTION, 128, 4, 0, 3)
    assert need > 0

    def call(c=desc(), q=FAKE, dt=W.BF16, T=3, ld=4096, Hq=32, table=FAKE, width=8, kv=FAKE, cu=None, B=3, max_q=1,
             scale=0.0, window=0, cap=0.0, out=FAKE, ws=FAKE, n=need, status=None):
        return W.lib.kv8_attention(ctypes.byref(c) if c is not None else None, q, dt, T, ld, Hq, table, width, kv, cu, B,
                                   max_q, scale, window, cap, out, ws, n, status, None)

    assert call(c=None) == W.ERR_INVALID_ARG
    for kw in BAD_CACHES:
        assert call(c=desc(**kw)) == W.ERR_INVALID_ARG, kw
    assert call(dt=5) == W.ERR_UNSUPPORTED_DTYPE
    nan, inf = float("nan"), float("inf")
    for kw in (dict(q=None), dict(q=ODD), dict(T=-1), dict(T=(1 << 24) + 1, cu=FAKE), dict(ld=4095), dict(ld=4100),
               dict(ld=BIG), dict(Hq=0), dict(Hq=12), dict(Hq=8 * 65), dict(table=None), dict(width=0),
               dict(width=1 << 27), dict(kv=None), dict(B=0), dict(B=8193, T=8193), dict(T=4), dict(max_q=2),
               dict(max_q=0, cu=FAKE), dict(max_q=BIG, cu=FAKE), dict(scale=nan), dict(scale=inf), dict(window=-1),
               dict(cap=-1.0), dict(cap=nan), dict(cap=inf), dict(out=None), dict(out=ODD), dict(ws=None),
               dict(ws=FAKE + 4), dict(status=FAKE + 2), dict(cu=FAKE + 2)):
        assert call(**kw) == W.ERR_INVALID_ARG, kw
    assert call(n=need - 1) == W.ERR_WORKSPACE
    assert call(n=0) == W.ERR_WORKSPACE
    assert call(T=0, cu=FAKE) == W.OK


def test_workspace_size_grows_with_the_rows():
    a = W.workspace_size(W.OP_KV8_ATTENTION, 128, 1, 0, 1)
    b = W.workspace_size(W.OP_KV8_ATTENTION, 256, 8192, 0, 64)
    assert 0 < a <= b < 1 << 28
    assert W.workspace_size(W.OP_KV8_ATTENTION, 0, 1, 0, 1) == 0


def cache(dev="cpu", dtype=torch.int8, **kw):
    a = dict(n=4, h=2, p=16, d=64)
    a.update(kw)
    k = torch.zeros((a["n"], a["h"], a["p"], a["d"]), dtype=torch.int8, device=dev).view(dtype)
    s = torch.ones((a["n"], a["h"]), device=dev)
    return W.Kv8Cache(k, k.clone(), s, s.clone())


def test_binding_raises_on_bad_tensors():
    i32 = torch.int32
    z = lambda *s, dt=i32: torch.zeros(s, dtype=dt)  # noqa: E731
    c = cache()
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # CPU tensors
        W.kv8_write(c, x, x, z(3))
    with pytest.raises(ValueError):
        W.kv8_read(c, z(3))
    with pytest.raises(ValueError):
        W.kv8_plan(z(2), z(2), z(2, 4), z(9), z(1), 16, 5)
    with pytest.raises(TypeError):  # dtypes
        W.kv8_write(c, x.half(), x.half(), z(3))
    with pytest.raises(TypeError):
        W.kv8_write(c, x, x.float(), z(3))
    with pytest.raises(TypeError):
        W.kv8_write(c, x, x, z(3, dt=torch.int64))
    with pytest.raises(TypeError):
        W.kv8_write(cache(dtype=torch.uint8), x, x, z(3))
    with pytest.raises(TypeError):
        W.kv8_plan(z(2, dt=torch.int64), z(2), z(2, 4), z(9), z(1), 16, 5)
    with pytest.raises(TypeError):
        W.kv8_cache(4, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):  # shapes and strides
        W.kv8_write(c, x, x, z(4))
    with pytest.raises(ValueError):
        W.kv8_write(c, x[:, :1], x[:, :1], z(3))
    with pytest.raises(ValueError):
        W.kv8_write(c, x.transpose(0, 1).contiguous().transpose(0, 1), x, z(3))
    with pytest.raises(ValueError):
        W.kv8_read(c, z(3), k=torch.zeros((2, 2, 64)), v=torch.zeros((2, 2, 64)))
    with pytest.raises(ValueError):
        W.kv8_plan(z(2), z(3), z(2, 4), z(9), z(1), 16, 5)
    with pytest.raises(ValueError):
        W.kv8_plan(z(2), z(2), z(3, 4), z(9), z(1), 16, 5)
    with pytest.raises(ValueError):
        W.kv8_plan(z(2), z(2), z(2, 4), z(9), z(1), 16, 5, slots=z(4))
    with pytest.raises(ValueError):
        W.kv8_plan(z(2), z(2), z(2, 8)[:, ::2], z(9), z(1), 16, 5)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    for bad in (lambda: W.kv8_attention(c, q[:, :3], z(2, 4), z(2)), lambda: W.kv8_attention(c, q[0], z(2, 4), z(2)),
                lambda: W.kv8_attention(c, q, z(3, 4), z(2)), lambda: W.kv8_attention(c, q, z(2, 4), z(2), cu_q=z(2)),
                lambda: W.kv8_attention(c, q, z(2, 4), z(2), out=torch.zeros((2, 4, 128), dtype=torch.bfloat16)),
                lambda: W.kv8_attention(c, q.transpose(1, 2), z(2, 4), z(2))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        W.kv8_attention(c, q, z(2, 4), z(2), out=torch.zeros((2, 4, 64)))
    with pytest.raises(ValueError):
        W.Kv8Cache(c.k, c.v[:2], c.k_scale, c.v_scale)._struct()
    with pytest.raises(ValueError):
        W.Kv8Cache(c.k, c.v, c.k_scale[:2], c.v_scale)._struct()


def test_no_write_kernel_is_built_that_no_call_reaches():
    """kv8_write shares a run among warps where a page is more than four times the rows of 8 (bf16)
    or 4 (float32) passes of a warp, and pages have 128 places at most: not for bf16 rows of 64."""
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("no nm")
    names = subprocess.run([nm, "-C", build.LIB], capture_output=True, text=True, check=True).stdout
    for bf16 in (True, False):
        for e4m3 in ("true", "false"):
            for dh in (64, 128, 256):
                rows = (8 if bf16 else 4) * (32 // (dh // 8))
                name = f"k_kv8_write_shared<{str(bf16).lower()}, {e4m3}, {dh}>"
                assert (name in names) == (128 > 4 * rows), name
                assert name.replace("_shared", "") in names
