"""GPU parity of the 8-bit paged key/value cache against its float64 oracle.

* Plans are whole numbers and exact; so are the bytes and scales of a write (the scales are
  powers of two, so each byte is one rounding of an exact quotient) and the values read.
* Attention, per element: the output's rounding, half a step of its type relative to it, plus
  the weights' errors, which scale with mass = sum_j p_j |v_j|:
    - a weight's own rounding: float16, 2^-11 (bf16 queries), or two float16 parts, 2^-22;
    - a score's error es on both sides of the quotient p_j / sum p, e^(2 es) - 1, where
      es = size * (dh + 8) * 2^-23 + softcap * 2^-21: a float32 dot product of dh terms, each
      addition off by at most 2^-23 of size = sum_c |q_c k_c| * scale, a few roundings of the
      factors, and tanh to 4 steps;
    - 2^-21 for the exponential, and keys * 2^-23 for the float32 sums.
  And in relative L2 over a request: 1e-5 for float32, the bound of the other products here;
  for bf16 the half step 2^-8, plus the weights' 2^-11.
"""

from __future__ import annotations

import numpy as np
import pytest

import oracle as O
import free_activation_sparse_b200 as W
from tests.gpu_util import dev_f32, dev_i32, host, rel_l2, status_word, torch

pytestmark = pytest.mark.gpu

FMT = {"int8": "int8", "e4m3": "float8_e4m3fn"}


def dtype_of(name):
    t = torch()
    return {"bf16": t.bfloat16, "f32": t.float32, "int8": t.int8, "e4m3": t.float8_e4m3fn}[name]


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def rows(rng, shape, dtype):
    """Random rows in dtype and as the float64 values they hold."""
    x = torch().from_numpy(rng.normal(size=shape).astype(np.float32)).cuda().to(dtype_of(dtype))
    return x, f64(x)


# ------------------------------------------------------------------------------------
# kv8_plan
# ------------------------------------------------------------------------------------


def plan_case(rng, B, page, width, new_max, ended, tokens_pad=0, spare=7):
    seq = rng.integers(0, width * page - new_max + 1, size=B)
    seq[rng.random(B) < 0.15] = 0
    new = rng.integers(0, new_max + 1, size=B)
    new[rng.choice(B, size=ended, replace=False)] = -1
    have = -(-seq // page)
    total = int(have.sum()) + int((-(-(seq + np.maximum(new, 0)) // page) - have).sum()) + spare
    order = rng.permutation(total)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    cells = np.full(total + 3, -5)
    cells[:total - at] = order[at:]
    return seq, new, table, cells, total - at, int(np.maximum(new, 0).sum()) + tokens_pad


def check_plan(seq, new, table, cells, n_free, page, tokens, alias=False):
    want = O.kv8_plan(seq, new, table, cells, n_free, page, tokens)
    d_seq, d_new, d_table, d_cells, d_n = (dev_i32(np.asarray(v)) for v in (seq, new, table, cells, [n_free]))
    st = status_word()
    kw = dict(kv_len=d_seq, n_free_out=d_n) if alias else {}
    got = W.kv8_plan(d_seq, d_new, d_table, d_cells, d_n, page, tokens, status=st, **kw)
    for name, g in zip(("kv_len", "cu_q", "slots", "positions"), got):
        assert np.array_equal(host(g), want[name]), name
    assert int(host(got[4])[0]) == want["n_free"]
    assert np.array_equal(host(d_table), want["table"])
    assert np.array_equal(host(d_cells), want["free_pages"])
    codes = ([W.ERR_CAPACITY] if want["short"] else []) + ([W.ERR_INVALID_ARG] if want["bad"] else [])
    assert int(host(st)[0]) in (codes or [0])
    return want


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("B,page,width,new_max,ended,pad", [
    (1, 16, 4, 1, 0, 0), (1, 128, 9, 700, 0, 5), (2, 32, 3, 1, 1, 3), (33, 16, 40, 1, 5, 0), (64, 64, 12, 300, 9, 1),
    (513, 16, 20, 3, 60, 0), (999, 16, 33, 40, 100, 13), (1024, 32, 8, 9, 0, 2), (8192, 16, 5, 2, 900, 0),
    (5, 16, 2000, 9000, 1, 4), (40, 16, 30, 0, 40, 6)])
def test_plan_matches_oracle(B, page, width, new_max, ended, pad, alias):
    rng = np.random.default_rng(B * 7 + page + new_max)
    check_plan(*(lambda s, n, t, c, f, k: (s, n, t, c, f, page, k))(*plan_case(rng, B, page, width, new_max, ended, pad)),
               alias=alias)


def test_plan_short_of_pages_or_places():
    rng = np.random.default_rng(3)
    for B, new_max in ((7, 90), (600, 30)):
        seq, new, table, cells, n_free, tokens = plan_case(rng, B, 16, 30, new_max, B // 7)
        full = check_plan(seq, new, table, cells, n_free, 16, tokens)
        assert not full["short"]
        # pushed pages count as free ones, so take away more than those
        few = max(0, n_free - int(n_free * 0.7))
        assert check_plan(seq, new, table, cells, few, 16, tokens)["n_free"] >= 0
        assert check_plan(seq, new, table, cells, n_free, 16, tokens // 2)["short"]
        check_plan(seq, new, table, cells, 0, 16, tokens)
        check_plan(seq, new, table, cells, n_free, 16, 0)


def test_plan_out_of_range_inputs():
    rng = np.random.default_rng(4)
    seq, new, table, cells, n_free, tokens = plan_case(rng, 12, 16, 10, 20, 2, 4)
    seq[3], seq[7], new[9] = -5, 161, 200
    new[9], seq[9] = 200, 10
    want = check_plan(seq, new, table, cells, n_free, 16, tokens + 400)
    assert want["bad"]
    seq[1], new[1] = 100, 2 ** 31 - 1  # sums past 32 bits
    seq[2], new[2] = 100, 2 ** 31 - 1
    check_plan(seq, new, table, cells, n_free, 16, tokens)
    seq, new, table, cells, n_free, tokens = plan_case(rng, 12, 16, 10, 20, 2, 4)
    for wrong in (-1, len(cells) + 1):
        want = O.kv8_plan(seq, new, table, cells, wrong, 16, tokens)
        st = status_word()
        got = W.kv8_plan(dev_i32(seq), dev_i32(new), dev_i32(table), dev_i32(cells), dev_i32(np.array([wrong])), 16, tokens,
                         status=st)
        assert int(host(st)[0]) != 0 and np.array_equal(host(got[0]), want["kv_len"])


def test_plan_pushes_past_the_last_cell():
    """A stack too small for the pages that come back: the rest is lost, and said so."""
    seq, new = np.array([64, 40, 3]), np.array([-1, -1, 1])
    table = np.arange(12).reshape(3, 4)
    want = check_plan(seq, new, table, np.array([50, 51, -1, -1]), 2, 16, 1)
    assert want["short"] and want["n_free"] == 4


# ------------------------------------------------------------------------------------
# kv8_write, kv8_read
# ------------------------------------------------------------------------------------


class Mirror:
    """A cache on the GPU and the oracle's two sides of it."""

    def __init__(self, n, heads, page, dh, fmt, seed=0):
        rng = np.random.default_rng(seed)
        self.fmt, self.page = fmt, page
        self.c = W.kv8_cache(n, heads, page, dh, dtype=dtype_of(fmt))
        # what recycled pages hold: old bytes under old scales
        raw = O.kv8_round(np.clip(rng.normal(size=(2, n, heads, page, dh)) * 40, -120, 120), fmt)
        for x, at in ((raw[0], self.c.k), (raw[1], self.c.v)):
            at.view(torch().int8).copy_(torch().from_numpy(x.astype(np.float32)).cuda().to(dtype_of(fmt)).view(torch().int8))
        scales = np.ldexp(1.0, rng.integers(-9, 2, size=(2, n, heads)))
        self.c.k_scale.copy_(dev_f32(scales[0]))
        self.c.v_scale.copy_(dev_f32(scales[1]))
        self.k, self.v = (raw[0], scales[0]), (raw[1], scales[1])

    def write(self, k, v, kf, vf, slots):
        st = status_word()
        W.kv8_write(self.c, k, v, dev_i32(slots), status=st)
        self.k = O.kv8_write(*self.k, kf, slots, self.page, self.fmt)
        self.v = O.kv8_write(*self.v, vf, slots, self.page, self.fmt)
        return int(host(st)[0])

    def check(self):
        for (val, scale), raw, sc in ((self.k, self.c.k, self.c.k_scale), (self.v, self.c.v, self.c.v_scale)):
            assert np.array_equal(f64(sc), scale, equal_nan=True)
            assert np.array_equal(f64(raw), val)


def run_slots(starts, lens, page):
    return np.concatenate([np.arange(s, s + n) for s, n in zip(starts, lens)] or [np.zeros(0)]).astype(np.int64)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,page,dh", [(1, 16, 64), (8, 16, 128), (3, 32, 256), (5, 64, 128), (2, 128, 64),
                                           (2, 128, 256), (32, 16, 128)])
def test_write_matches_oracle_bit_for_bit(fmt, dtype, heads, page, dh):
    rng = np.random.default_rng(heads * 1000 + page + dh)
    m = Mirror(24, heads, page, dh, fmt, seed=page)
    # whole pages, a page from its middle, single places, a page's last place
    pages = rng.permutation(24)
    starts = [pages[0] * page, pages[1] * page + 5, pages[2] * page + page - 1, pages[3] * page, pages[4] * page + 1]
    lens = [page, page - 5, 1, 1, page - 1]
    slots = run_slots(starts, lens, page)
    T = len(slots)
    # one buffer of q | k | v rows, as a fused projection leaves it
    loud = np.exp(rng.normal(size=(T, 1, 1)))
    both = torch().from_numpy((rng.normal(size=(T, 3 * heads, dh)) * loud).astype(np.float32)).cuda().to(dtype_of(dtype))
    k, v = both[:, heads:2 * heads], both[:, 2 * heads:]
    assert m.write(k, v, f64(k), f64(v), slots) == 0
    m.check()
    # one more token each where there is room, twice as loud every time: scales grow
    for step in range(3):
        more = np.array([pages[3] * page + 1 + step, pages[5] * page + step])
        k, kf = rows(rng, (2, heads, dh), dtype)
        k = (k.float() * 2.0 ** (2 * step)).to(k.dtype)
        m.write(k, k, f64(k), f64(k), more)
        m.check()


def test_write_skips_and_refuses_slots():
    rng = np.random.default_rng(5)
    m = Mirror(6, 2, 16, 64, "int8")
    slots = np.array([-1, 16, 17, -1, -7, 40, 41, 95, -1])
    k, kf = rows(rng, (9, 2, 64), "bf16")
    assert m.write(k, k, kf, kf, slots) == 0
    m.check()
    slots[5:8] = [96, 97, 2 ** 31 - 1]  # outside the cache
    assert m.write(k, k, kf, kf, slots) == W.ERR_INVALID_ARG
    m.check()
    W.kv8_write(m.c, k[:0], k[:0], dev_i32(slots[:0]))
    m.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("T", [150, 2500])
def test_write_many_tokens_per_cta(T, fmt):
    """Several runs and parts of runs in one CTA's stretch of tokens."""
    rng = np.random.default_rng(T)
    n = T // 4
    m = Mirror(n, 2, 16, 64, fmt)
    pages, slots = list(rng.permutation(n)), []
    while len(slots) < T and pages:
        p, a = pages.pop(), int(rng.integers(0, 16)) if rng.random() < 0.5 else 0
        slots += range(p * 16 + a, p * 16 + a + int(rng.integers(1, 17 - a)))
        if rng.random() < 0.1:
            slots.append(-1)
    slots = np.array(slots[:T])
    k, kf = rows(rng, (len(slots), 2, 64), "bf16")
    v, vf = rows(rng, (len(slots), 2, 64), "bf16")
    assert m.write(k, v, kf, vf, slots) == 0
    m.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_write_extreme_values(fmt):
    """Zero rows, subnormal and largest numbers; infinities and NaN turn that page and head's
    scale into NaN until the page starts anew."""
    m = Mirror(8, 2, 16, 64, fmt)
    x = np.zeros((6, 2, 64), dtype=np.float32)
    x[1] = 1e-44
    x[2, 0], x[2, 1] = 3.4028235e38, -3.4028235e38
    x[3, 0, 5], x[4, 1, 0] = np.nan, -np.inf
    x[5] = 448.0
    k = dev_f32(x)
    slots = np.array([0, 16, 32, 48, 64, 80])
    m.write(k, k, x, x, slots)
    m.check()
    assert np.isnan(host(m.c.k_scale)[3, 0]) and np.isfinite(host(m.c.k_scale)[3, 1])
    x[:] = 1.0
    m.write(k.fill_(1.0), k, x, x, slots + 1)  # behind the NaN: still NaN
    m.check()
    m.write(k, k, x, x, slots)  # anew
    m.check()
    assert np.isfinite(host(m.c.k_scale)[:6]).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,page,dh,T", [(1, 16, 64, 1), (3, 32, 256, 77), (32, 128, 128, 300), (4, 64, 64, 2049)])
def test_read_matches_oracle(fmt, dtype, heads, page, dh, T):
    rng = np.random.default_rng(T)
    m = Mirror(40, heads, page, dh, fmt)
    slots = rng.integers(0, 40 * page, size=T)
    slots[rng.random(T) < 0.1] = -1
    if T > 1:
        slots[1] = slots[0]  # the same slot twice
    st = status_word()
    k, v = W.kv8_read(m.c, dev_i32(slots), dtype=dtype_of(dtype), status=st)
    # a byte times a power of two is exact in either type
    assert np.array_equal(f64(k), O.kv8_read(*m.k, slots, page)) and np.array_equal(f64(v), O.kv8_read(*m.v, slots, page))
    assert int(host(st)[0]) == 0
    slots[0] = 40 * page
    k, _ = W.kv8_read(m.c, dev_i32(slots), status=st)
    assert int(host(st)[0]) == W.ERR_INVALID_ARG and not f64(k)[0].any()
    assert W.kv8_read(m.c, dev_i32(slots[:0]))[0].shape == (0, heads, dh)


def test_read_rounds_once_to_bf16():
    """Scales that are no powers of two (a cache from elsewhere): one rounding."""
    m = Mirror(4, 2, 16, 64, "int8")
    m.c.k_scale.mul_(1.37)
    slots = np.arange(64)
    k, _ = W.kv8_read(m.c, dev_i32(slots))
    want = m.c.k.float() * m.c.k_scale[:, :, None, None]
    want = want.permute(0, 2, 1, 3).reshape(64, 2, 64).to(k.dtype)
    assert torch().equal(k, want)


# ------------------------------------------------------------------------------------
# kv8_attention
# ------------------------------------------------------------------------------------


def attention_case(seed, kv, q_lens, hq, hkv, dh, page, fmt, dtype, pad=0, extra_width=1):
    rng = np.random.default_rng(seed)
    have = [-(-n // page) for n in kv]
    n = sum(have) + 2
    m = Mirror(n, hkv, page, dh, fmt, seed=seed)
    # modest scores: scales about 2^-5 for bytes about 40
    m.k = (m.k[0], np.ldexp(1.0, rng.integers(-7, -4, size=(n, hkv))))
    m.c.k_scale.copy_(dev_f32(m.k[1]))
    order = rng.permutation(n)
    table = np.full((len(kv), max(have) + extra_width), -1)
    at = 0
    for b, h in enumerate(have):
        table[b, :h] = order[at:at + h]
        at += h
    T = sum(q_lens) + pad
    wide = torch().from_numpy(rng.normal(size=(T, hq + 2 * hkv, dh)).astype(np.float32)).cuda().to(dtype_of(dtype))
    return m, wide[:, :hq], table, np.concatenate([[0], np.cumsum(q_lens)])


def cached(m, table, b, n):
    """The first n cached rows of request b, as float64 (K, V)."""
    s = np.array([table[b, j // m.page] * m.page + j % m.page for j in range(n)], dtype=np.int64)
    return O.kv8_read(*m.k, s, m.page), O.kv8_read(*m.v, s, m.page)


def check_attention(out, m, q, table, kv, cu, dtype, sample=None, **kw):
    out, qf = f64(out), f64(q)
    dh = qf.shape[2]
    half, weight, l2 = (2.0 ** -8, 2.0 ** -11, 2.0 ** -8 + 2.0 ** -11) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -22, 1e-5)
    for b in range(len(kv)):
        a, e = int(cu[b]), int(cu[b + 1])
        if e == a:
            continue
        K, V = cached(m, table, b, kv[b])
        want, mass, size = O.kv8_attention(qf[a:e], K, V, **kw)
        es = size[:, :, None] * (dh + 8) * 2.0 ** -23 + kw.get("softcap", 0.0) * 2.0 ** -21
        tol = half * np.abs(want) + mass * (weight + np.expm1(2 * es) + 2.0 ** -21 + kv[b] * 2.0 ** -23)
        off = np.abs(out[a:e] - want)
        assert (off <= tol).all(), (b, float((off - tol).max()), np.argwhere(off > tol)[:5].tolist())
        assert rel_l2(out[a:e], want) <= l2, (b, rel_l2(out[a:e], want))


# Long bf16 rows take the tensor-core kernel where there are enough of them: `pad` more rows behind
# the last request (as a padded batch has them) send short tests there too.
PADS = pytest.mark.parametrize("pad", [0, 5200])

SHAPES = [
    # kv lengths, query lengths, hq, hkv, dh, page
    ([1], [1], 1, 1, 64, 16), ([5], [1], 4, 2, 128, 16), ([33], [1], 8, 1, 256, 32), ([1000], [1], 32, 32, 128, 16),
    ([16, 17, 0, 31, 129], [1] * 5, 8, 2, 128, 16), ([700, 3, 2500], [1] * 3, 7, 1, 64, 64),
    ([128, 127, 400], [1] * 3, 16, 1, 128, 128), ([60, 1500], [1, 1], 3, 3, 256, 16),
    # spans and prompts, causal within themselves
    ([9], [9], 2, 2, 64, 16), ([40, 300, 7], [3, 5, 1], 8, 4, 256, 64), ([130, 64], [17, 64], 12, 4, 128, 32),
    ([600, 200, 50], [1, 130, 50], 8, 2, 128, 16), ([300], [300], 10, 2, 64, 128), ([400, 333], [333, 100], 4, 4, 256, 16),
    # a request without queries, one with more queries than keys, one without keys
    ([50, 20, 0, 300], [0, 33, 4, 2], 8, 8, 128, 16)]


@PADS
@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("e4m3", "bf16"), ("int8", "f32"), ("e4m3", "f32")])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attention_matches_oracle(shape, fmt, dtype, pad):
    kv, ql, hq, hkv, dh, page = SHAPES[shape]
    one = all(n == 1 for n in ql)
    if pad and (one or dtype == "f32"):
        pytest.skip("one kernel takes these, padded or not")
    m, q, table, cu = attention_case(shape, kv, ql, hq, hkv, dh, page, fmt, dtype, pad=pad)
    st = status_word()
    args = {} if one else dict(cu_q=dev_i32(cu), max_q=max(ql))
    out = W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), status=st, **args)
    assert int(host(st)[0]) == 0 and out.dtype == q.dtype
    check_attention(out, m, q, table, kv, cu, dtype)
    again = W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), **args)
    assert torch().equal(out, again)  # fixed-order sums
    if one:  # the same through offsets
        out2 = W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), cu_q=dev_i32(cu), max_q=1)
        check_attention(out2, m, q, table, kv, cu, dtype)


@PADS
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,softcap,scale", [(1, 0.0, 0.0), (16, 0.0, 0.0), (100, 30.0, 0.0), (0, 5.0, 0.3),
                                                  (10 ** 12, 0.0, 0.02), (257, 50.0, 0.0)])
def test_attention_window_softcap_scale(window, softcap, scale, dtype, pad):
    for seed, (kv, ql, hq, hkv, dh, page) in enumerate([([900, 40, 1, 0], [1, 1, 1, 1], 8, 4, 256, 64),
                                                        ([700, 90], [60, 90], 8, 2, 128, 16)]):
        m, q, table, cu = attention_case(seed + 50, kv, ql, hq, hkv, dh, page, "int8", dtype, pad=pad)
        args = dict(scale=scale, window=window, softcap=softcap)
        out = W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), cu_q=dev_i32(cu), max_q=max(ql), **args)
        check_attention(out, m, q, table, kv, cu, dtype, **args)


def test_calls_without_tokens():
    """A step in which no request brings a token (and one in which all end)."""
    t = torch()
    m, q, table, cu = attention_case(30, [20, 30], [1, 1], 4, 2, 64, 16, "int8", "bf16")
    lens, none = dev_i32(np.array([20, 30])), dev_i32(np.zeros(2))
    r = W.kv8_plan(lens, none, dev_i32(table), dev_i32(np.arange(4)), dev_i32(np.array([4])), 16, 0)
    assert host(r[0]).tolist() == [20, 30] and host(r[1]).tolist() == [0, 0, 0] and r[2].numel() == 0
    r = W.kv8_plan(lens, none - 1, dev_i32(table), dev_i32(np.arange(9)), dev_i32(np.array([4])), 16, 0)
    assert host(r[0]).tolist() == [0, 0] and int(host(r[4])[0]) == 4 + 2 + 2
    assert W.kv8_attention(m.c, q[:0], dev_i32(table), lens, cu_q=r[1], max_q=7).shape == (0, 4, 64)
    W.kv8_write(m.c, q[:0, :2], q[:0, 2:], r[2])
    assert W.kv8_read(m.c, r[2])[1].shape == (0, 2, 64)
    # rows, but no request has any: left as they were
    out = t.full((3, 4, 64), 7.0, dtype=t.bfloat16, device="cuda")
    W.kv8_attention(m.c, t.ones_like(out), dev_i32(table), lens, cu_q=r[1], max_q=1, out=out)
    assert (f64(out) == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_leaves_rows_behind_the_last_request(dtype):
    for ql, pad in (([1, 1, 1], 5), ([3, 1, 2], 5), ([150, 1, 40], 5), ([150, 1, 40], 900)):
        kv = [200, 17, 64]
        m, q, table, cu = attention_case(9, kv, ql, 8, 2, 128, 16, "e4m3", dtype, pad=pad)
        out = torch().full(tuple(q.shape), 7.0, dtype=q.dtype, device="cuda")
        W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), cu_q=dev_i32(cu), max_q=max(ql), out=out)
        check_attention(out, m, q, table, kv, cu, dtype)
        assert (f64(out)[cu[-1]:] == 7.0).all()


@PADS
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ql", [[1, 1, 1], [40, 3, 129]])
def test_attention_ignores_what_lies_behind_the_keys(dtype, ql, pad):
    """NaN bytes, NaN and infinite scales and bad page indices in places that no query sees."""
    kv = [200, 17, 130]
    m, q, table, cu = attention_case(10, kv, ql, 8, 2, 128, 16, "e4m3", dtype, pad=pad)
    args = dict(cu_q=dev_i32(cu), max_q=max(ql))
    base = W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), **args)[:cu[-1]]
    seen = np.zeros((m.c.n_pages, 16), dtype=bool)
    for b, n in enumerate(kv):
        for j in range(n):
            seen[table[b, j // 16], j % 16] = True
    bad = torch().from_numpy(~seen).cuda()[:, None, :, None].expand(m.c.k.shape)
    m.c.k.view(torch().int8)[bad] = 0x7f
    m.c.v.view(torch().int8)[bad] = -1
    unused = torch().from_numpy(~seen.any(1)).cuda()
    m.c.k_scale[unused] = float("nan")
    m.c.v_scale[unused] = float("inf")
    wide = np.where(table < 0, 10 ** 9, table)
    st = status_word()
    got = W.kv8_attention(m.c, q, dev_i32(wide), dev_i32(np.array(kv)), status=st, **args)
    assert int(host(st)[0]) == 0 and torch().equal(got[:cu[-1]], base)


@PADS
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ql", [[1, 1], [37, 130]])
def test_attention_nan_where_a_seen_page_is_nan(dtype, ql, pad):
    kv = [90, 200]
    m, q, table, cu = attention_case(11, kv, ql, 4, 2, 64, 16, "int8", dtype, pad=pad)
    m.c.v_scale[table[1, 2], 0] = float("nan")
    out = f64(W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), cu_q=dev_i32(cu), max_q=max(ql)))
    assert np.isfinite(out[:cu[1]]).all() and np.isfinite(out[cu[1]:cu[2], 2:]).all()
    assert np.isnan(out[cu[2] - 1, :2]).all()


@PADS
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ql", [[1, 1], [37, 130]])
def test_attention_bad_indices_are_reported_and_never_followed(dtype, ql, pad):
    kv = [90, 200]
    m, q, table, cu = attention_case(12, kv, ql, 4, 2, 64, 16, "int8", dtype, pad=pad)
    args = dict(cu_q=dev_i32(cu), max_q=max(ql))
    for wrong in (-1, m.c.n_pages, 2 ** 31 - 1, -2 ** 31):
        t2 = table.copy()
        t2[1, 3] = wrong
        st = status_word()
        out = f64(W.kv8_attention(m.c, q, dev_i32(t2), dev_i32(np.array(kv)), status=st, **args))
        assert int(host(st)[0]) == W.ERR_INVALID_ARG and np.isfinite(out).all()
        # the page's tokens are left out
        K, V = cached(m, table, 1, 200)
        keep = np.r_[0:48, 64:200]
        last = O.kv8_attention(f64(q)[cu[2] - 1:cu[2]], K[keep], V[keep])[0]
        assert rel_l2(out[cu[2] - 1], last[0]) <= 2.0 ** -7
    # lengths past the table are clamped; queries past max_q are left unwritten; offsets are bounded
    st = status_word()
    out = W.kv8_attention(m.c, q, dev_i32(table[:, :13]), dev_i32(np.array([90, 10 ** 9])), status=st, **args)
    assert int(host(st)[0]) == W.ERR_INVALID_ARG
    if max(ql) > 1:
        st = status_word()
        part = torch().full(tuple(q.shape), 7.0, dtype=q.dtype, device="cuda")
        W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), cu_q=dev_i32(cu), max_q=100, out=part, status=st)
        assert int(host(st)[0]) == W.ERR_INVALID_ARG
        assert (f64(part)[cu[1] + 100:] == 7.0).all()
        check_attention(part, m, q, table, kv[:1], cu, dtype)
    for offs in ([0, -3, 5], [0, 10 ** 9, -10 ** 9], [5, 2, 1]):
        st = status_word()
        W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), cu_q=dev_i32(np.array(offs)), max_q=max(ql), status=st)
        assert int(host(st)[0]) == W.ERR_INVALID_ARG


@PADS
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_wide_range_of_scales(dtype, pad):
    """Value scales 2^20 apart: a loud page that gets no weight must not cost the quiet ones
    their digits (and the other way round)."""
    kv, ql = [300, 400], [1, 140]
    m, q, table, cu = attention_case(13, kv, ql, 4, 2, 128, 16, "int8", dtype, pad=pad)
    rng = np.random.default_rng(1)
    m.v = (m.v[0], np.ldexp(1.0, rng.integers(-24, -4, size=m.v[1].shape)))
    m.c.v_scale.copy_(dev_f32(m.v[1]))
    out = W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), cu_q=dev_i32(cu), max_q=140)
    check_attention(out, m, q, table, kv, cu, dtype)
    # query magnitudes far from 1
    for f in (2.0 ** -40, 2.0 ** 20):
        q2 = (q.float() * f).to(q.dtype)
        out = W.kv8_attention(m.c, q2, dev_i32(table), dev_i32(np.array(kv)), cu_q=dev_i32(cu), max_q=140, scale=0.1 / f)
        check_attention(out, m, q2, table, kv, cu, dtype, scale=0.1 / f)


@pytest.mark.parametrize("dtype,fmt", [("bf16", "int8"), ("bf16", "e4m3"), ("f32", "int8")])
@pytest.mark.parametrize("B,kv_max,hq,hkv,q_max", [(1, 20000, 4, 1, 1), (70, 900, 8, 8, 1), (300, 60, 4, 2, 1), (3, 9000, 8, 2, 4),
                                                   (2, 5000, 16, 2, 64), (40, 700, 4, 1, 30)])
def test_attention_large_batches_and_long_contexts(B, kv_max, hq, hkv, q_max, dtype, fmt):
    """Work split over a long axis and joined; many requests to a CTA. Sampled requests."""
    rng = np.random.default_rng(B)
    kv = rng.integers(kv_max // 2, kv_max + 1, size=B).tolist()
    ql = [int(min(n, rng.integers(1, q_max + 1))) for n in kv]
    m, q, table, cu = attention_case(B, kv, ql, hq, hkv, 128, 16, fmt, dtype)
    out = W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), cu_q=dev_i32(cu), max_q=q_max)
    assert np.isfinite(f64(out)).all()
    for b in sorted({0, B // 2, B - 1}):
        check_attention(out[int(cu[b]):int(cu[b + 1])], m, q[int(cu[b]):int(cu[b + 1])], table[b:b + 1], kv[b:b + 1],
                        [0, ql[b]], dtype)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("B,kv_max,hq,hkv,q_max,dh", [(40, 3000, 8, 2, 80, 128), (25, 4000, 8, 8, 140, 128), (4, 6000, 32, 8, 1500, 128),
                                                      (30, 2500, 16, 2, 33, 64), (300, 500, 4, 4, 70, 64)])
def test_attention_bf16_prompts_agree_with_float32_everywhere(B, kv_max, hq, hkv, q_max, dh, fmt):
    """Long lines of tiles of every height, many to a CTA: every row of the bf16 path against the
    float32 path (another kernel) on the same numbers, within bf16's half step of a result and
    2^-11 of each weight; the rows' sizes stand in for their mass."""
    rng = np.random.default_rng(B + q_max)
    kv = rng.integers(kv_max // 3, kv_max + 1, size=B).tolist()
    ql = [int(min(n, rng.integers(1, q_max + 1))) for n in kv]
    m, q, table, cu = attention_case(B + 1, kv, ql, hq, hkv, dh, 16, fmt, "bf16")
    args = (dev_i32(table), dev_i32(np.array(kv)))
    a = W.kv8_attention(m.c, q, *args, cu_q=dev_i32(cu), max_q=max(ql)).float()
    b = W.kv8_attention(m.c, q.float(), *args, cu_q=dev_i32(cu), max_q=max(ql))
    rel = ((a - b).norm(dim=2) / b.norm(dim=2)).max()
    assert float(rel) <= 2.0 ** -7, float(rel)  # 2^-8, and as much again for the weights' errors against the norm


@pytest.mark.parametrize("dtype,dh,hq,hkv,q_max", [("bf16", 128, 4, 1, 1), ("f32", 128, 16, 1, 1), ("f32", 64, 2, 2, 1),
                                                    ("bf16", 256, 2, 1, 5), ("bf16", 128, 40, 1, 3)])
def test_attention_most_requests(dtype, dh, hq, hkv, q_max):
    """8192 requests: the largest shared memory of every shape; sampled requests."""
    rng = np.random.default_rng(dh)
    kv = rng.integers(0, 40, size=8192).tolist()
    ql = [int(min(max(n, 1), rng.integers(1, q_max + 1))) for n in kv]
    m, q, table, cu = attention_case(3, kv, ql, hq, hkv, dh, 16, "int8", dtype)
    st = status_word()
    out = W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), cu_q=dev_i32(cu), max_q=q_max, status=st)
    assert int(host(st)[0]) == 0
    for b in sorted({0, 1, 2, 8190, 8191, *rng.integers(0, 8192, size=40).tolist()}):
        a, e = int(cu[b]), int(cu[b + 1])
        check_attention(out[a:e], m, q[a:e], table[b:b + 1], kv[b:b + 1], [0, e - a], dtype)


def test_attention_offsets_past_32_bits():
    """A cache of more than 2^32 bytes a side whose last pages are the ones in use."""
    t = torch()
    n, heads, page, dh = (1 << 32) // (8 * 128 * 128) + 40, 8, 128, 128
    c = W.kv8_cache(n, heads, page, dh)
    rng = np.random.default_rng(2)
    pages = np.array([n - 1, 3, n - 7, 0])
    for raw in (c.k, c.v):
        raw[t.from_numpy(pages).cuda()] = t.from_numpy(rng.integers(-90, 91, size=(4, heads, page, dh)).astype(np.int8)).cuda()
    c.k_scale.fill_(2.0 ** -6)
    c.v_scale.fill_(2.0 ** -4)
    m = Mirror(1, heads, page, dh, "int8")
    m.c, m.k, m.v = c, None, None
    for ql in (1, 130):
        q, qf = rows(rng, (ql + 600, 8, dh), "bf16")
        qf = qf[:ql]
        out = W.kv8_attention(c, q, dev_i32(pages[None]), dev_i32(np.array([500])), cu_q=dev_i32(np.array([0, ql])), max_q=ql)[:ql]
        slots = dev_i32(np.concatenate([p * page + np.arange(page) for p in pages])[:500])
        K, V = W.kv8_read(c, slots)
        want, _, _ = O.kv8_attention(qf, f64(K), f64(V))
        assert rel_l2(f64(out), want) <= 2.0 ** -8 + 2.0 ** -11
    # and written there
    x, xf = rows(rng, (5, heads, dh), "bf16")
    at = np.arange(n * page - 5, n * page)
    c.k_scale[n - 1] = 0
    W.kv8_write(c, x, x, dev_i32(at))
    val, sc = O.kv8_write(np.zeros((1, heads, page, dh)), np.zeros((1, heads)), xf, at - (n - 1) * page, page, "int8")
    assert np.array_equal(f64(c.k[n - 1])[:, -5:], val[0][:, -5:]) and np.array_equal(f64(c.k_scale[n - 1]), sc[0])


# ------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------


class Server:
    """The calls of a serving loop over fixed buffers, with room for `T` tokens a step."""

    def __init__(self, B, T, hq, hkv, dh, page, pages, width, fmt, dtype, max_q):
        t = torch()
        i32 = lambda *s: t.zeros(s, dtype=t.int32, device="cuda")  # noqa: E731
        self.c = W.kv8_cache(pages, hkv, page, dh, dtype=dtype_of(fmt))
        self.hq, self.hkv, self.max_q, self.T, self.page = hq, hkv, max_q, T, page
        self.len, self.new, self.table = i32(B), i32(B), i32(B, width).fill_(-1)
        self.free, self.n_free = t.arange(pages, dtype=t.int32, device="cuda"), i32(1).fill_(pages)
        self.cu, self.slots, self.pos, self.status = i32(B + 1), i32(T), i32(T), i32(1)
        self.qkv = t.zeros((T, hq + 2 * hkv, dh), dtype=dtype_of(dtype), device="cuda")
        self.out = t.zeros((T, hq, dh), dtype=dtype_of(dtype), device="cuda")
        self.ws = W.Workspace(W.OP_KV8_ATTENTION, dh, max_q * hq // hkv, 0, B)

    def step(self):
        W.kv8_plan(self.len, self.new, self.table, self.free, self.n_free, self.page, self.T, kv_len=self.len, cu_q=self.cu,
                   slots=self.slots, positions=self.pos, n_free_out=self.n_free, status=self.status)
        W.kv8_write(self.c, self.qkv[:, self.hq:self.hq + self.hkv], self.qkv[:, self.hq + self.hkv:], self.slots,
                    status=self.status)
        W.kv8_attention(self.c, self.qkv[:, :self.hq], self.table, self.len, cu_q=self.cu, max_q=self.max_q, ws=self.ws,
                        out=self.out, status=self.status)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("fmt,dtype,dh,page,max_q", [("int8", "bf16", 128, 16, 40), ("e4m3", "bf16", 64, 32, 1),
                                                     ("int8", "f32", 128, 16, 3), ("e4m3", "bf16", 128, 64, 200),
                                                     ("int8", "bf16", 64, 64, 280)])
def test_serving_loop(fmt, dtype, dh, page, max_q, graph):
    """Requests come, grow by prompts and single tokens, end and give their pages back, in a
    padded batch; the same loop captured once and replayed. Every step's attention against the
    oracle on the oracle's own cache, pages included."""
    t = torch()
    rng = np.random.default_rng(page + max_q)
    B, hq, hkv = 5, 4, 2
    T = B * max_q + 3
    s = Server(B, T, hq, hkv, dh, page, 60, 14, fmt, dtype, max_q)
    run = s.step
    if graph:
        s.step()  # no tokens yet: nothing changes
        side = t.cuda.Stream()
        side.wait_stream(t.cuda.current_stream())
        g = t.cuda.CUDAGraph()
        with t.cuda.stream(side):
            with t.cuda.graph(g, stream=side):
                s.step()
        t.cuda.current_stream().wait_stream(side)
        run = g.replay
    ref = dict(len=np.zeros(B, dtype=np.int64), table=host(s.table).astype(np.int64), free=host(s.free).astype(np.int64),
               n=60)
    k = v = (np.zeros((60, hkv, page, dh)), np.zeros((60, hkv)))
    for step in range(9):
        new = np.where(rng.random(B) < 0.4, 1, rng.integers(0, max_q + 1, size=B))
        new[(ref["len"] > 0) & (rng.random(B) < 0.15)] = -1
        new = np.where(ref["len"] + new > 14 * page, -1, new)
        x, xf = rows(rng, tuple(s.qkv.shape), dtype)
        s.qkv.copy_(x)
        s.new.copy_(dev_i32(new))
        s.out.fill_(7.0)
        run()
        t.cuda.synchronize()
        assert int(host(s.status)[0]) == 0
        p = O.kv8_plan(ref["len"], new, ref["table"], ref["free"], ref["n"], page, T)
        assert not p["short"] and np.array_equal(host(s.slots), p["slots"]) and np.array_equal(host(s.table), p["table"])
        assert int(host(s.n_free)[0]) == p["n_free"] and np.array_equal(host(s.len), p["kv_len"])
        k = O.kv8_write(*k, xf[:, hq:hq + hkv], p["slots"], page, fmt)
        v = O.kv8_write(*v, xf[:, hq + hkv:], p["slots"], page, fmt)
        m = Mirror.__new__(Mirror)
        m.page, m.k, m.v = page, k, v
        check_attention(s.out, m, s.qkv[:, :hq], p["table"], p["kv_len"].tolist(), p["cu_q"], dtype)
        assert (f64(s.out)[p["cu_q"][-1]:] == 7.0).all()
        ref = dict(len=p["kv_len"], table=p["table"], free=p["free_pages"], n=p["n_free"])


def test_calls_on_another_stream_and_two_workspaces_at_once():
    """Two attentions side by side, each on its own stream with its own workspace."""
    t = torch()
    m, q, table, cu = attention_case(20, [4000, 3000], [1, 1], 8, 2, 128, 16, "int8", "bf16")
    m2, q2, table2, cu2 = attention_case(21, [500, 90], [200, 90], 8, 2, 128, 16, "e4m3", "bf16")
    d = [dev_i32(x) for x in (table, np.array([4000, 3000]), table2, np.array([500, 90]), cu2)]
    want = W.kv8_attention(m.c, q, d[0], d[1])
    want2 = W.kv8_attention(m2.c, q2, d[2], d[3], cu_q=d[4], max_q=200)
    s1, s2 = t.cuda.Stream(), t.cuda.Stream()
    w1 = W.Workspace(W.OP_KV8_ATTENTION, 128, 4, 0, 2)
    w2 = W.Workspace(W.OP_KV8_ATTENTION, 128, 800, 0, 2)
    t.cuda.synchronize()
    outs = []
    for _ in range(20):
        with t.cuda.stream(s1):
            a = W.kv8_attention(m.c, q, d[0], d[1], ws=w1)
        with t.cuda.stream(s2):
            b = W.kv8_attention(m2.c, q2, d[2], d[3], cu_q=d[4], max_q=200, ws=w2)
        outs.append((a, b))
    t.cuda.synchronize()
    assert all(t.equal(a, want) and t.equal(b, want2) for a, b in outs)


def test_double_sparsity_is_calibrated_from_the_cache():
    """kv8_read feeds the Double Sparsity calls: the labels of a cached sequence are its key
    rows' channels."""
    t = torch()
    m = Mirror(10, 2, 16, 64, "int8", seed=3)
    slots = np.concatenate([p * 16 + np.arange(16) for p in (7, 2, 9, 0)])[:60]
    k, _ = W.kv8_read(m.c, dev_i32(slots), dtype=t.float32)
    K = t.zeros((1, 2, 64, 64), device="cuda")
    K[0, :, :60] = k.transpose(0, 1)
    seq = dev_i32(np.array([60]))
    C = W.ds_calibrate_channels(K, seq, 8)
    rows64 = O.kv8_read(*m.k, slots, 16)
    for g in range(2):
        assert host(C)[g].tolist() == O.ds_calibrate_channels(rows64[:, g], 8).tolist()
    lab = host(W.ds_label_build(K, seq, C))
    assert np.array_equal(lab[0, 1, :60], rows64[:, 1][:, host(C)[1]])


# ------------------------------------------------------------------------------------
# calls that go past what the tests above reach
# ------------------------------------------------------------------------------------


# Requests with fewer keys than queries, so that whole tiles of query rows see no key, in every
# kernel and kind of team: kv length, queries, requests, hq, hkv, dh, rows behind the last request.
BLIND = [(100, 2048, 1, 32, 8, 128, 0), (5, 300, 1, 32, 8, 128, 0), (5, 300, 3, 8, 8, 64, 5200),  # tensor-core kernel
         (20, 64, 1, 8, 8, 128, 0), (20, 64, 1, 4, 2, 256, 0), (5, 60, 1, 8, 2, 64, 0), (100, 300, 1, 4, 2, 256, 0),  # CTAs
         (5, 300, 1, 16, 8, 128, 0), (5, 300, 1, 32, 8, 64, 0), (30, 200, 4, 8, 4, 256, 0)]  # one-warp teams


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kv,n,B,hq,hkv,dh,pad", BLIND)
def test_attention_tiles_that_see_no_key(kv, n, B, hq, hkv, dh, pad, dtype):
    """Their rows are zeros, whatever lay in `out`, and the workspace is left as a call has to
    find it: a call whose tiles are cut, on the same workspace, gives what it gives on a new one."""
    t = torch()
    m, q, table, cu = attention_case(kv + n, [kv] * B, [n] * B, hq, hkv, dh, 16, "int8", dtype, pad=pad)
    ws = W.Workspace(W.OP_KV8_ATTENTION, dh, n * hq // hkv, 0, B)
    out = t.full(tuple(q.shape), 7.0, dtype=q.dtype, device="cuda")
    st = status_word()
    args = dict(cu_q=dev_i32(cu), max_q=n)
    W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array([kv] * B)), ws=ws, out=out, status=st, **args)
    assert int(host(st)[0]) == 0
    for b in range(B):
        assert not f64(out)[cu[b]:cu[b + 1] - kv].any(), b
    check_attention(out, m, q, table, [kv] * B, cu, dtype)
    assert (f64(out)[cu[-1]:] == 7.0).all()
    W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array([kv] * B)), ws=ws, out=out.fill_(7.0), softcap=5.0, **args)
    for b in range(B):
        assert not f64(out)[cu[b]:cu[b + 1] - kv].any(), b
    check_attention(out, m, q, table, [kv] * B, cu, dtype, softcap=5.0)
    assert not ws.buf[:160 * 12 * 4].any()  # the teams' arrival counters, which lead the workspace
    m2, q2, table2, cu2 = attention_case(n, [3000] * B, [min(n, 200)] * B, hq, hkv, dh, 16, "int8", dtype, pad=pad)
    args = dict(cu_q=dev_i32(cu2), max_q=n)
    want = W.kv8_attention(m2.c, q2, dev_i32(table2), dev_i32(np.array([3000] * B)), **args)
    for _ in range(2):
        got = W.kv8_attention(m2.c, q2, dev_i32(table2), dev_i32(np.array([3000] * B)), ws=ws, **args)
        assert t.equal(got, want)


def test_serving_step_that_runs_out_of_pages():
    """kv8_plan leaves requests out: their lengths stay, their new tokens keep their rows. The
    others' rows are right, and so are the next step's on the same workspace."""
    t = torch()
    rng = np.random.default_rng(8)
    B, hq, hkv, dh, page, max_q = 3, 8, 2, 64, 16, 600
    s = Server(B, B * max_q, hq, hkv, dh, page, 50, 50, "int8", "bf16", max_q)
    k = v = (np.zeros((50, hkv, page, dh)), np.zeros((50, hkv)))
    ref = dict(len=np.zeros(B, dtype=np.int64), table=host(s.table).astype(np.int64), free=host(s.free).astype(np.int64), n=50)
    # the second step finds 9 pages free: the last request's 600 tokens do not fit behind its 40
    for new, short in (([400, 200, 40], False), ([2, 1, 600], True), ([3, 1, 100], False)):
        new = np.array(new)
        x, xf = rows(rng, tuple(s.qkv.shape), "bf16")
        s.qkv.copy_(x)
        s.new.copy_(dev_i32(new))
        s.out.fill_(7.0)
        s.status.zero_()
        s.step()
        t.cuda.synchronize()
        p = O.kv8_plan(ref["len"], new, ref["table"], ref["free"], ref["n"], page, B * max_q)
        assert p["short"] == short and int(host(s.status)[0]) == (W.ERR_CAPACITY if short else 0)
        assert np.array_equal(host(s.len), p["kv_len"]) and np.array_equal(host(s.cu), p["cu_q"])
        k = O.kv8_write(*k, xf[:, hq:hq + hkv], p["slots"], page, "int8")
        v = O.kv8_write(*v, xf[:, hq + hkv:], p["slots"], page, "int8")
        m = Mirror.__new__(Mirror)
        m.page, m.k, m.v = page, k, v
        check_attention(s.out, m, s.qkv[:, :hq], p["table"], p["kv_len"].tolist(), p["cu_q"], "bf16")
        assert (f64(s.out)[p["cu_q"][-1]:] == 7.0).all()
        ref = dict(len=p["kv_len"], table=p["table"], free=p["free_pages"], n=p["n_free"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,dh,kv,ql,hq,hkv,pad", [
    (16, 64, [10], [1], 4, 2, 0), (16, 256, [100], [1], 4, 2, 0), (32, 128, [10], [1], 8, 2, 0), (32, 64, [100], [3], 4, 2, 0),
    (64, 128, [100], [1], 2, 2, 0), (128, 256, [700], [2], 8, 2, 0), (128, 64, [700], [1], 4, 2, 0),
    (32, 128, [900] * 64, [1] * 64, 16, 8, 0), (64, 64, [130] * 64, [1] * 64, 16, 8, 0), (64, 256, [130] * 64, [1] * 64, 16, 8, 0),
    (64, 128, [300, 400], [100, 130], 4, 2, 5200), (128, 64, [300, 400], [100, 130], 4, 2, 5200)])
def test_attention_carries_nan(page, dh, kv, ql, hq, hkv, pad, dtype):
    """A page whose key scale is NaN (kv8_write met an infinity or a NaN there) gives NaN to every
    row that sees a key of it, wherever the page lies among the kernels' chunks and warps; a query
    with a NaN or an infinity gives NaN to its own row of that head."""
    m, q, table, cu = attention_case(77, kv, ql, hq, hkv, dh, page, "int8", dtype, pad=pad)
    args = (dev_i32(table), dev_i32(np.array(kv)))
    more = dict(cu_q=dev_i32(cu), max_q=max(ql))
    base = f64(W.kv8_attention(m.c, q, *args, **more))
    G, b = hq // hkv, len(kv) - 1
    assert np.isfinite(base).all()
    pages = -(-kv[b] // page)
    for at in sorted({0, pages // 2, pages - 1}):
        keep = m.c.k_scale.clone()
        m.c.k_scale[int(table[b, at]), 1] = float("nan")
        out = f64(W.kv8_attention(m.c, q, *args, **more))
        m.c.k_scale.copy_(keep)
        want = np.zeros(out.shape, dtype=bool)
        for i in range(ql[b]):
            want[cu[b] + i, G:2 * G] = kv[b] - ql[b] + i >= at * page
        assert np.array_equal(np.isnan(out), want), at
        assert np.array_equal(out[~want], base[~want])
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        row, head = int(cu[b]) + ql[b] // 2, hq - 1
        q2[row, head, 3] = bad
        out = f64(W.kv8_attention(m.c, q2, *args, **more))
        want = np.zeros(out.shape, dtype=bool)
        want[row, head] = True
        assert np.array_equal(np.isnan(out), want), bad
        assert np.array_equal(out[~want], base[~want])


@PADS
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [1, 80])
def test_attention_nan_values_reach_rows_that_hardly_weigh_them(B, dtype, pad):
    """A page whose value scale is NaN, its keys' weights far below float32's smallest number: as
    with the values themselves, 0 * NaN is NaN."""
    kv, ql = [300] * B, [2] * (B - 1) + [130]
    m, q, table, cu = attention_case(78, kv, ql, 8, 4, 64, 16, "int8", dtype, pad=pad)
    m.c.k_scale.mul_(256.0)  # scores apart by hundreds
    args = (dev_i32(table), dev_i32(np.array(kv)))
    more = dict(cu_q=dev_i32(cu), max_q=130)
    base = f64(W.kv8_attention(m.c, q, *args, **more))
    assert np.isfinite(base).all()
    for b in {0, B - 1}:
        for at in (0, 3):
            keep = m.c.v_scale.clone()
            m.c.v_scale[int(table[b, at]), 2] = float("nan")
            out = f64(W.kv8_attention(m.c, q, *args, **more))
            m.c.v_scale.copy_(keep)
            assert np.isnan(out[cu[b]:cu[b + 1], 4:6]).all()
            out[cu[b]:cu[b + 1], 4:6] = base[cu[b]:cu[b + 1], 4:6]
            assert np.array_equal(out, base)


@pytest.mark.parametrize("dtype,dh,hq,n,kv", [("bf16", 256, 8, 4096, 71000), ("f32", 256, 8, 4096, 71000), ("f32", 64, 16, 3000, 140000)])
def test_attention_long_chunk_over_a_long_context(dtype, dh, hq, n, kv):
    """One request with more pieces of keys than 2^32 over a CTA's threads. Sampled rows."""
    m, q, table, cu = attention_case(31, [kv], [n], hq, 1, dh, 128, "int8", dtype)
    st = status_word()
    out = torch().full(tuple(q.shape), 7.0, dtype=q.dtype, device="cuda")
    W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array([kv])), cu_q=dev_i32(cu), max_q=n, out=out, status=st)
    assert int(host(st)[0]) == 0
    K, V = cached(m, table, 0, kv)
    half = 2.0 ** -8 + 2.0 ** -11 if dtype == "bf16" else 1e-5
    for i in (0, 1, n // 2, n - 1):
        want, _, _ = O.kv8_attention(f64(q[i:i + 1]), K[:kv - n + i + 1], V[:kv - n + i + 1])
        assert rel_l2(f64(out[i:i + 1]), want) <= half


def test_attention_that_would_run_for_hours_is_refused():
    """A table that names one page 2^23 times over: 2^34 pieces of keys for the head (2^33 for
    the tensor-core kernel), and with fewer rows but 1024 heads 2^37 over all. Nothing is computed."""
    t = torch()
    table = t.zeros((1, (1 << 30) // 128), dtype=t.int32, device="cuda")
    for dtype, dh, heads, hq, n, kv in (("bf16", 256, 1, 64, 32, 1 << 30), ("f32", 256, 1024, 1024, 9, 1 << 30),
                                        ("bf16", 64, 1, 64, 4096, 1 << 30)):
        c = W.kv8_cache(1, heads, 128, dh)
        q, out = (t.full((n, hq, dh), 7.0, dtype=dtype_of(dtype), device="cuda") for _ in range(2))
        st = status_word()
        W.kv8_attention(c, q, table, dev_i32(np.array([kv])), cu_q=dev_i32(np.array([0, n])), max_q=n, out=out, status=st)
        assert int(host(st)[0]) == W.ERR_INVALID_ARG and bool((out == 7.0).all())


@PADS
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("exponent", [119, -120])
@pytest.mark.parametrize("kv,ql", [([300], [1]), ([9000], [130]), ([200] * 80, [1] * 79 + [30]), ([40, 500], [7, 100])])
def test_attention_values_at_the_ends_of_float32(kv, ql, exponent, dtype, pad):
    """Values near float32's largest and smallest numbers: results of their size, whole tiles and
    joined parts."""
    m, q, table, cu = attention_case(79, kv, ql, 8, 4, 128, 32, "int8", dtype, pad=pad)
    m.v = (m.v[0], np.full(m.v[1].shape, 2.0 ** exponent))
    m.c.v_scale.copy_(dev_f32(m.v[1]))
    out = W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array(kv)), cu_q=dev_i32(cu), max_q=130)
    assert np.isfinite(f64(out)).all()
    check_attention(out, m, q, table, kv, cu, dtype)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,dh", [(16, 64), (128, 256)])
def test_write_of_finite_numbers_reads_back_finite(page, dh, dtype, fmt):
    """Numbers around those whose byte would stand for 2^128, new and rounded again; the long run
    goes through both write kernels' loops."""
    t = torch()
    m = Mirror(8, 2, page, dh, fmt)
    rng = np.random.default_rng(4)
    top = t.finfo(dtype_of(dtype)).max
    edge = np.array([1.0, 0.9999, 1.984375 / 2, 1.9843 / 2, 1.9375 / 2, 1.937 / 2, 1.75 / 2, 0.5, 0.25, 2.0 ** -7, 0.0])
    for slots, most in ((np.arange(0, page), 1.0), (page + np.arange(5), 0.4), (page + 5 + np.arange(3), 1.0),
                        (np.array([2 * page]), 0.4961), (np.array([2 * page + 1]), 1.0), (np.array([2 * page + 2]), 0.9)):
        x = rng.choice(edge, size=(len(slots), 2, dh)) * rng.choice([-1.0, 1.0], size=(len(slots), 2, dh)) * float(top) * most
        x[:, :, 0] = float(top) * most
        k = dev_f32(x.astype(np.float32)).to(dtype_of(dtype)).clamp(-top, top)
        assert bool(t.isfinite(k).all())
        m.write(k, k.neg(), f64(k), -f64(k), slots)
        m.check()
        # every place written so far (the ones behind hold a recycled page's bytes, which nobody sees)
        seen = slots if slots[0] % page == 0 else np.arange(slots[0] // page * page, slots[-1] + 1)
        k2, v2 = W.kv8_read(m.c, dev_i32(seen), dtype=dtype_of(dtype))
        assert bool(t.isfinite(k2).all()) and bool(t.isfinite(v2).all())
        if len(slots) > 1:  # half a step of the byte, or a whole one where it is held down
            rel = ((W.kv8_read(m.c, dev_i32(slots), dtype=t.float32)[0].double() - k.double()).abs() / k.double().abs().clamp(min=1e30))[k.abs() > 0.2 * top]
            assert float(rel.max()) <= 2.0 ** -3


def test_plan_reports_entries_that_are_no_pages():
    """On the stack and in a request's table: the tokens get no slot, and the status says why."""
    seq, new, table = np.array([5, 20, 0, 3]), np.array([1, 30, 4, 0]), np.full((4, 4), -1)
    table[0, 0], table[1, :2], table[3, 0] = 3, (1, 2), -9  # request 3 brings no token: nobody looks
    cells = np.array([6, 5, 4, 7, -1])
    assert not check_plan(seq, new, table, cells, 4, 16, 40)["bad"]
    for wrong in (-1, -2 ** 31, 2 ** 27, 2 ** 31 - 1):
        for at in (2, 3):  # popped by request 2 and by request 1
            c2 = cells.copy()
            c2[at] = wrong
            want = check_plan(seq, new, table, c2, 4, 16, 40)
            assert want["bad"] and (want["slots"][:35] < 0).any() and (want["slots"][:35] >= 0).any()
        t2 = table.copy()
        t2[1, 1] = wrong
        assert check_plan(seq, new, t2, cells, 4, 16, 40)["bad"]
    # one wrong entry past 4096 tokens, where a cluster shares the plan
    rng = np.random.default_rng(6)
    seq, new, table, cells, n_free, tokens = plan_case(rng, 60, 16, 40, 300, 4, 5)
    assert tokens > 4096 and not check_plan(seq, new, table, cells, n_free, 16, tokens)["bad"]
    pushed = int((-(-seq // 16))[new < 0].sum())  # popped first
    need = int((-(-(seq + np.maximum(new, 0)) // 16) + -seq // 16)[new >= 0].sum())
    assert need > pushed + 50
    cells[n_free - 1 - (need - pushed) // 2] = -1
    assert check_plan(seq, new, table, cells, n_free, 16, tokens)["bad"]


@pytest.mark.parametrize("fmt,apart", [("int8", 27), ("e4m3", 18)])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("at", [1, 3])
def test_attention_prompt_tile_with_a_page_louder_by_the_stated_range(at, side, fmt, apart):
    """The tensor-core kernel holds a tile's bytes against its loudest page. Up to the stated quotient
    that is exact: rows that see quiet pages only (those before page `at`, in one tile with rows
    that see it) are as without it, and values of every row are within the usual bounds."""
    kv, n, page = 200, 200, 16
    m, q, table, cu = attention_case(80 + at, [kv], [n], 8, 2, 128, page, fmt, "bf16", pad=5200)
    args = (dev_i32(table), dev_i32(np.array([kv])))
    more = dict(cu_q=dev_i32(cu), max_q=n)
    assert at * page < 256 // 4  # the tile of the first 64 queries
    (val, scale), dev = (m.k, m.c.k_scale) if side == "k" else (m.v, m.c.v_scale)
    scale = np.full(scale.shape, 2.0 ** -6)
    scale[table[0, at]] = 2.0 ** (apart - 6)
    dev.copy_(dev_f32(scale))
    if side == "k":
        m.k = (val, scale)
    else:
        m.v = (val, scale)
    out = W.kv8_attention(m.c, q, *args, **more)
    rows_ = at * page
    check_attention(out[:rows_], m, q[:rows_], table, [rows_], [0, rows_], "bf16")
    if side == "v":
        check_attention(out, m, q, table, [kv], cu, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [64, 128, 256])
def test_attention_short_tile_with_a_page_far_louder(dh, dtype):
    """The kernel of short rows: weights are within 2^-39 of the row's largest, times the loud
    page's scale over a quiet one's, in rows that do not see it as well."""
    kv, n, page, apart = 40, 12, 32, 18
    m, q, table, cu = attention_case(90, [kv], [n], 1, 1, dh, page, "int8", dtype)
    scale = np.full(m.v[1].shape, 2.0 ** -6)
    scale[table[0, 1]] = 2.0 ** (apart - 6)
    m.v = (m.v[0], scale)
    m.c.v_scale.copy_(dev_f32(scale))
    half, weight = (2.0 ** -8, 2.0 ** -11) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -22)
    for length, loud in ((kv, 2.0 ** apart), (page, 1.0)):  # of 40 keys, the first 4 queries see 32 at most
        out = f64(W.kv8_attention(m.c, q, dev_i32(table), dev_i32(np.array([length])), cu_q=dev_i32(cu), max_q=n))
        K, V = cached(m, table, 0, length)
        want, mass, size = O.kv8_attention(f64(q), K, V)
        es = size[:, :, None] * (dh + 8) * 2.0 ** -23
        tol = half * np.abs(want) + mass * (weight + np.expm1(2 * es) + 2.0 ** -21 + length * 2.0 ** -23)
        # 2^-39 of the largest weight, for each key that the row sees
        tol += 2.0 ** -39 * loud * np.stack([np.abs(V[:length - n + i + 1]).sum(0) for i in range(n)])
        assert (np.abs(out - want) <= tol).all(), length


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("page,dh", [(16, 128), (128, 64), (128, 256)])
def test_write_leaves_older_rows_whose_scale_stays(page, dh, fmt):
    """Also under the largest scales, and bytes that no write of this library would leave there."""
    rng = np.random.default_rng(5)
    m = Mirror(4, 2, page, dh, fmt)
    big = np.full(m.k[1].shape, 2.0 ** 122)
    m.k, m.v = (m.k[0], big), (m.v[0], big)
    m.c.k_scale.copy_(dev_f32(big))
    m.c.v_scale.copy_(dev_f32(big))
    for slots in (np.arange(3, page), page + np.array([page - 1]), 2 * page + np.arange(2, 12)):
        for dtype in ("f32", "bf16"):
            k, kf = rows(rng, (len(slots), 2, dh), dtype)
            m.write(k, k, kf, kf, slots)
            m.check()
