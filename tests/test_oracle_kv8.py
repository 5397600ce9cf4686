"""Pins of the 8-bit cache's oracle (CPU): worked examples and independent routines."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O


def test_scale_is_the_smallest_power_of_two_that_holds():
    # 127 = 127 * 2^0; just above it the next power is needed; 448 likewise for e4m3
    assert O.kv8_scale(127.0, "int8") == 1.0
    assert O.kv8_scale(np.nextafter(127.0, 200.0), "int8") == 2.0
    assert O.kv8_scale(63.5, "int8") == 0.5
    assert O.kv8_scale(448.0, "e4m3") == 1.0
    assert O.kv8_scale(449.0, "e4m3") == 2.0
    assert O.kv8_scale(0.0, "int8") == 2.0 ** -120
    assert O.kv8_scale(3.4028235e38, "int8") == 2.0 ** 122


def test_rounding_to_the_formats():
    assert O.kv8_round([0.5, 1.5, -2.5, 126.5], "int8").tolist() == [0.0, 2.0, -2.0, 126.0]
    x = np.concatenate([np.random.default_rng(0).normal(size=4000) * 100, np.linspace(-0.05, 0.05, 999),
                        [448.0, 447.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(O.kv8_round(x, "e4m3"), want)


def test_plan_worked_example():
    """Pages of 16. Request 0: 16 + 1 tokens, one more page; 1 ended with two pages; 2: 5 + 20,
    one more; 3: 0 + 0. The stack [7, 8] gets 3, 4 pushed; 0 pops 4, 2 pops 3."""
    t = np.array([[1, -1, -1], [3, 4, -1], [6, -1, -1], [-1, -1, -1]])
    r = O.kv8_plan([16, 17, 5, 0], [1, -1, 20, 0], t, np.array([7, 8, -1, -1, -1]), 2, 16, 23)
    assert r["kv_len"].tolist() == [17, 0, 25, 0] and r["cu_q"].tolist() == [0, 1, 1, 21, 21]
    assert r["table"].tolist() == [[1, 4, -1], [3, 4, -1], [6, 3, -1], [-1, -1, -1]]
    assert r["free_pages"].tolist() == [7, 8, 3, 4, -1] and r["n_free"] == 2
    assert r["slots"].tolist() == [64] + [6 * 16 + i for i in range(5, 16)] + [3 * 16 + i for i in range(9)] + [-1, -1]
    assert r["positions"].tolist() == [16] + list(range(5, 25)) + [0, 0]
    assert not r["short"] and not r["bad"]


def test_write_growth_and_fresh_pages():
    val, scale = np.zeros((2, 1, 16, 1)), np.zeros((2, 1))
    val, scale = O.kv8_write(val, scale, np.array([[[127.0]], [[3.0]]]), [16, 17], 16, "int8")
    assert scale[1, 0] == 1.0 and val[1, 0, :2, 0].tolist() == [127.0, 3.0]
    # 128 needs scale 2: 127 / 2 = 63.5 -> 64, 3 / 2 = 1.5 -> 2 (ties to even)
    val, scale = O.kv8_write(val, scale, np.array([[[128.0]]]), [18], 16, "int8")
    assert scale[1, 0] == 2.0 and val[1, 0, :3, 0].tolist() == [64.0, 2.0, 64.0]
    # place 0 written: the page starts anew, later places keep their bytes
    val, scale = O.kv8_write(val, scale, np.array([[[1.0]]]), [16], 16, "int8")
    assert scale[1, 0] == 2.0 ** -6 and val[1, 0, :3, 0].tolist() == [64.0, 2.0, 64.0]
    assert scale[0, 0] == 0 and not val[0].any()


@pytest.mark.parametrize("n,kv,hq,hkv", [(1, 40, 4, 2), (7, 40, 2, 2), (12, 12, 3, 1)])
def test_attention_is_sdpa(n, kv, hq, hkv):
    g = np.random.default_rng(n)
    q, K, V = g.normal(size=(n, hq, 32)), g.normal(size=(kv, hkv, 32)), g.normal(size=(kv, hkv, 32))
    for window in (0, 5):
        out, mass, size = O.kv8_attention(q, K, V, window=window)
        d = torch.arange(kv - n, kv)[:, None] - torch.arange(kv)[None]
        mask = (d >= 0) & ((d < window) if window else (d >= 0))
        r = lambda x: torch.from_numpy(x).transpose(0, 1).repeat_interleave(hq // x.shape[1], 0)  # noqa: E731
        want = torch.nn.functional.scaled_dot_product_attention(r(q), r(K), r(V), attn_mask=mask).transpose(0, 1).numpy()
        assert np.abs(out - want).max() < 1e-12
        assert (mass >= np.abs(out) - 1e-12).all()
    # more queries than keys: the early ones see nothing
    out, _, _ = O.kv8_attention(np.ones((3, 1, 32)), np.ones((1, 1, 32)), np.ones((1, 1, 32)))
    assert not out[:2].any() and np.allclose(out[2], 1)


def test_softcap_is_applied_before_the_softmax():
    q, K = np.array([[[2.0, 0.0]]]), np.array([[[4.0, 0.0]], [[-4.0, 0.0]]])
    V = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])
    out, _, _ = O.kv8_attention(q, K, V, scale=1.0, softcap=2.0)
    z = 2 * np.tanh(4.0)
    assert np.allclose(out[0, 0], [1 / (1 + np.exp(-2 * z)), 1 / (1 + np.exp(2 * z))], atol=1e-14)


def test_what_is_stored_stands_for_a_finite_number():
    big = float(np.finfo(np.float32).max)
    for fmt, top in (("int8", 63.0 * 2.0 ** 122), ("e4m3", 240.0 * 2.0 ** 120)):
        val, scale = np.zeros((1, 1, 16, 1)), np.zeros((1, 1))
        val, scale = O.kv8_write(val, scale, np.array([[[big]], [[-big]], [[top]]]), [0, 1, 2], 16, fmt)
        assert (val[0, 0, :3, 0] * scale[0, 0]).tolist() == [top, -top, top]
    # older rows that are rounded again: 127 * 2^121 is a tie between 63 and 64 times 2^122
    val, scale = O.kv8_write(np.zeros((1, 1, 16, 1)), np.zeros((1, 1)), np.array([[[127.0 * 2.0 ** 121]]]), [0], 16, "int8")
    assert scale[0, 0] == 2.0 ** 121 and val[0, 0, 0, 0] == 127.0
    val, scale = O.kv8_write(val, scale, np.array([[[big]]]), [1], 16, "int8")
    assert scale[0, 0] == 2.0 ** 122 and val[0, 0, :2, 0].tolist() == [63.0, 63.0]
