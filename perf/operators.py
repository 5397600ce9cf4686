"""The 8-bit paged key/value cache: what its operators are measured on.

A case is one call of an operator as a decode server makes it. `run` makes the framework's
calls where `own` is true, and computes the same in elementary torch operations otherwise.

  plan       request lengths -> page table, slots, positions, query offsets
  write      a step's keys and values into 8-bit pages, read back as the values they stand for
  read       cached tokens back as rows of numbers
  attention  a step's queries over the pages (single tokens, short spans, prompt chunks)

Shapes: 32 heads of 128 (Llama-7B), 32 / 8 heads of 128 (Llama-3-8B), 8 / 4 heads of 256
(Gemma-2-2B), and odd ones in `draw`.
"""

import math
import random

import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}
E_MIN, E_MAX = -120, 122  # exponents of the scales


def _dt(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[name]


# ------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------


def listed():
    return [
        # one decode step of 64 requests: the smallest call, all latency
        dict(name="plan, 64 decode requests", op="plan", B=64, page=16, kv_max=4096, new_max=1, ended=3, mix=1),
        # a step that mixes prompts with decoding, odd request count, some requests done
        dict(name="plan, 999 mixed requests", op="plan", B=999, page=16, kv_max=16384, new_max=64, ended=37, mix=2),
        # one decode step of 8 sequences, Llama-7B heads: each token goes to a page of its own
        dict(name="write, 8 decode tokens", op="write", B=8, hkv=32, dh=128, page=16, fmt="int8", dtype="bf16",
             kv_max=64, q_max=1, mix=3),
        # prompts of a Llama-3-8B server: 5 requests, ragged, behind cached prefixes
        dict(name="write, 5 prompts e4m3", op="write", B=5, hkv=8, dh=128, page=32, fmt="e4m3", dtype="bf16",
             kv_max=512, q_max=5000, mix=4),
        # Gemma-2-2B heads in float32
        dict(name="write, 3 prompts f32", op="write", B=3, hkv=4, dh=256, page=64, fmt="int8", dtype="f32",
             kv_max=300, q_max=1500, mix=5),
        # a cached prefix read back: labels and calibration of Double Sparsity, prefix reuse
        dict(name="read, 1 prefix of 1000", op="read", B=1, hkv=32, dh=128, page=16, fmt="int8", dtype="bf16",
             kv_min=1000, kv_max=1000, mix=6),
        dict(name="read, 12 prefixes f32", op="read", B=12, hkv=8, dh=128, page=64, fmt="e4m3", dtype="f32",
             kv_min=200, kv_max=6000, mix=7),
        # one sequence of 4096 tokens, Llama-7B heads: few rows, the cache's axis has to be split
        dict(name="decode, 1 x 4096, 32 heads", op="attention", B=1, pad=0, hq=32, hkv=32, dh=128, page=16,
             fmt="int8", dtype="bf16", kv_min=4096, kv_max=4096, q_max=1, window=0, softcap=0.0, mix=8),
        # a Llama-3-8B server's ragged batch, two empty places at its end
        dict(name="decode, 16 ragged, 32/8 heads", op="attention", B=16, pad=2, hq=32, hkv=8, dh=128, page=32,
             fmt="e4m3", dtype="bf16", kv_min=100, kv_max=9000, q_max=1, window=0, softcap=0.0, mix=9),
        # the largest cache: 64 long contexts
        dict(name="decode, 64 long, 32/8 heads", op="attention", B=64, pad=0, hq=32, hkv=8, dh=128, page=16,
             fmt="int8", dtype="bf16", kv_min=4000, kv_max=16384, q_max=1, window=0, softcap=0.0, mix=10),
        # Gemma-2-2B's local layers in float32, spans of up to 5 tokens (drafts being checked)
        dict(name="spans, 6 windowed f32, 8/4 heads", op="attention", B=6, pad=0, hq=8, hkv=4, dh=256, page=64,
             fmt="int8", dtype="f32", kv_min=500, kv_max=8000, q_max=5, window=4096, softcap=50.0, mix=11),
        # prompt chunks of a Llama-3-8B server behind cached prefixes: the most arithmetic
        dict(name="prompts, 4 chunks, 32/8 heads", op="attention", B=4, pad=0, hq=32, hkv=8, dh=128, page=16,
             fmt="e4m3", dtype="bf16", kv_min=2100, kv_max=8192, q_max=2048, window=0, softcap=0.0, mix=12),
    ]


HEADS = [(32, 32), (32, 8), (8, 4), (10, 2), (7, 1), (12, 4), (3, 3), (16, 1)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "read", "attention", "attention", "attention"])
    page, fmt, dtype = rng.choice([16, 32, 64, 128]), rng.choice(["int8", "e4m3"]), rng.choice(["bf16", "bf16", "f32"])
    mix = rng.randrange(1 << 20)
    hq, hkv = rng.choice(HEADS)
    dh = rng.choice([64, 128, 128, 256])
    if op == "plan":
        B = _log(rng, 1, 999)
        return dict(op=op, B=B, page=page, kv_max=_log(rng, 16, 16384), new_max=_log(rng, 1, max(1, 32000 // B)),
                    ended=rng.randrange(B // 8 + 1), mix=mix)
    if op == "write":
        B = _log(rng, 1, 64)
        most = max(1, min(5000, 12000 * 1024 // (hkv * dh) // B))
        return dict(op=op, B=B, hkv=hkv, dh=dh, page=page, fmt=fmt, dtype=dtype, kv_max=_log(rng, 1, 500),
                    q_max=_log(rng, 1, most), mix=mix)
    if op == "read":
        B = _log(rng, 1, 24)
        most = max(2, min(6000, 32000 * 1024 // (hkv * dh) // B))
        hi = _log(rng, 1, most)
        return dict(op=op, B=B, hkv=hkv, dh=dh, page=page, fmt=fmt, dtype=dtype, kv_min=rng.randint(1, hi), kv_max=hi,
                    mix=mix)
    B = _log(rng, 1, 64)
    hi = _log(rng, 16, min(16384, 600000 * 1024 // (hkv * dh) // B))
    spans = rng.choice(["one", "short", "prompt"])
    q_max = 1 if spans == "one" else rng.randint(2, 16) if spans == "short" else _log(rng, 17, 2048)
    # products of at most the largest listed prompts', scores of at most 2^30 numbers
    q_max = max(1, min(q_max, hi, (1 << 30) // (B * hq * hi), 4 * 2048 * 8192 * 32 * 128 // (B * hi * hq * dh)))
    return dict(op=op, B=B, pad=rng.choice([0, 0, 1, 3]), hq=hq, hkv=hkv, dh=dh, page=page, fmt=fmt, dtype=dtype,
                kv_min=rng.randint(q_max, hi), kv_max=hi, q_max=q_max, window=rng.choice([0, 0, 0, rng.randint(1, hi)]),
                softcap=rng.choice([0.0, 0.0, 30.0]), mix=mix)


def _lengths(case):
    """(cached before, new) tokens of every request: of the case, not of the seed."""
    r = random.Random(case["mix"])
    op, B = case["op"], case["B"]
    if op == "plan":
        seq = [r.randint(0, case["kv_max"]) for _ in range(B)]
        # most requests decode one token, every eighth brings a prompt
        new = [r.randint(1, case["new_max"]) if i % 8 == 7 else 1 for i in range(B)]
        for i in r.sample(range(B), case["ended"]):
            new[i] = -1
        return seq, new
    if op == "write":
        return [r.randint(0, case["kv_max"]) for _ in range(B)], [r.randint((case["q_max"] + 1) // 2, case["q_max"]) for _ in range(B)]
    kv = [r.randint(case["kv_min"], case["kv_max"]) for _ in range(B)]
    if op == "read":
        return kv, [0] * B
    q = [r.randint((case["q_max"] + 1) // 2, case["q_max"]) for _ in range(B)]
    kv, q = kv + [0] * case["pad"], q + [min(1, case["q_max"])] * case["pad"]  # empty places: a query, no keys
    return [a - b if a >= b else 0 for a, b in zip(kv, q)], q


def _pairs(kv, q, window):
    """Query-key pairs of one request, whose last query is at the last key."""
    n = 0
    for i in range(q):
        pos = kv - q + i
        n += max(0, pos + 1 - (max(0, pos - window + 1) if window else 0))
    return n


def work(case):
    seq, new = _lengths(case)
    if case["op"] == "plan":
        P, T = case["page"], sum(max(0, n) for n in new)
        taken = sum(-(-(s + n) // P) - -(-s // P) for s, n in zip(seq, new) if n > 0)
        back = sum(-(-s // P) for s, n in zip(seq, new) if n < 0)
        return {"bytes": 16 * len(seq) + 8 * (taken + back) + 8 * T, "flops": 0}
    row = case["hkv"] * case["dh"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "write":  # read the new rows, write them as bytes; read the touched pages back
        T, P = sum(new), case["page"]
        back = sum(s + n - s // P * P for s, n in zip(seq, new))
        return {"bytes": 2 * row * (T * (e + 1) + back * (1 + e)), "flops": 0}
    if case["op"] == "read":
        return {"bytes": 2 * row * sum(seq) * (1 + e), "flops": 0}
    T, D = sum(new), case["hq"] * case["dh"]
    w, keys, pairs = case["window"], 0, 0
    for s, n in zip(seq, new):
        kv = s + n if s else n if case["kv_min"] and s + n >= case["kv_min"] else 0
        keys += min(kv, w + n - 1) if w else kv
        pairs += _pairs(kv, n, w)
    scales = 2 * 4 * case["hkv"] * keys // case["page"]
    return {"bytes": 2 * row * keys + scales + 2 * T * D * e, "flops": 4 * pairs * D}


# ------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------


def _pow2(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scale_of(amax, fmt):
    """The smallest power of two s with amax <= qmax s, for float32 amax >= 0."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 127 / 128, x - 7, x - 6) if fmt == "int8" else torch.where(m <= 0.875, x - 9, x - 8)
    return _pow2(torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX))


def _round8(x, fmt):
    return torch.round(x).to(torch.int8) if fmt == "int8" else x.to(torch.float8_e4m3fn)


def _filled(case, pages, g):
    """Pages of keys or values with a few loud channels per head, as trained models have, and
    pages of different loudness; the scales that quantising them gives."""
    H, P, D, fmt = case["hkv"], case["page"], case["dh"], case["fmt"]
    chan = torch.where(torch.rand((H, 1, D), device="cuda", generator=g) < 0.06, 4.0, 1.0)
    loud = torch.exp(0.3 * torch.randn((pages, H, 1, 1), device="cuda", generator=g))
    out = torch.empty((pages, H, P, D), dtype=_dt(fmt), device="cuda")
    scale = torch.empty((pages, H), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (H * P * D))
    for a in range(0, pages, step):
        x = torch.randn((min(step, pages - a), H, P, D), device="cuda", generator=g) * chan * loud[a:a + step]
        s = _scale_of(x.abs().amax((2, 3)), fmt)
        scale[a:a + step] = s
        out[a:a + step] = _round8(x / s[:, :, None, None], fmt)
    return out, scale, chan


def _table(kv, page, width, pages, g):
    """Page tables over shuffled pages: [len(kv)][width], -1 behind a request's pages."""
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    have = [-(-n // page) for n in kv]
    table = torch.full((len(kv), width), -1, dtype=torch.int32)
    order = order.cpu()
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = order[at:at + n]
        at += n
    return table.cuda(), order[at:]


def _slots(kv, page, table, first=None):
    """Slots of every request's cached tokens from `first` on (all of them by default)."""
    first = first or [0] * len(kv)
    b = torch.tensor([i for i, n in enumerate(kv) for _ in range(first[i], n)], dtype=torch.int64)
    t = torch.tensor([j for i, n in enumerate(kv) for j in range(first[i], n)], dtype=torch.int64)
    return (table.cpu()[b, t // page].to(torch.int64) * page + t % page).to(torch.int32).cuda()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    seq, new = _lengths(case)
    P = case["page"]
    s = {"case": case}
    if case["op"] == "plan":
        B, T = case["B"], sum(max(0, n) for n in new)
        ends = [a + max(0, n) for a, n in zip(seq, new)]
        width = -(-max(ends) // P) + 3
        pages = sum(-(-e // P) for e in ends) + B
        s["table"], rest = _table(seq, P, width, pages, g)
        back = sum(-(-a // P) for a, n in zip(seq, new) if n < 0)
        s["free"] = torch.cat([rest, torch.full((back + 5,), -1, dtype=torch.int32)]).cuda()
        s["n_free"] = _i32([len(rest)])
        s["seq"], s["new"], s["tokens"] = _i32(seq), _i32(new), T + 13  # a padded batch
        # the buffers of a server's step
        s["out"] = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (B, B + 1, T + 13, T + 13, 1)]
        return s
    kv = [a + n for a, n in zip(seq, new)]
    if case["op"] == "attention":
        kv = [n if n >= case["kv_min"] else 0 for n in kv]
    pages = sum(-(-n // P) for n in kv) + 2
    width = -(-max(kv) // P) + 1
    s["k"], s["k_scale"], chan = _filled(case, pages, g)
    s["v"], s["v_scale"], _ = _filled(case, pages, g)
    s["table"], _ = _table(kv, P, width, pages, g)
    H, D, T, dt = case["hkv"], case["dh"], sum(new), _dt(case["dtype"])
    if case["op"] == "read":
        s["slots"] = _slots(kv, P, s["table"])
        s["out"] = [torch.empty((sum(kv), H, D), dtype=dt, device="cuda") for _ in range(2)]
    elif case["op"] == "write":
        # keys and values as the projections leave them: one row of q | k | v for each token
        s["slots"] = _slots(kv, P, s["table"], seq)
        s["back"] = _slots(kv, P, s["table"], [a // P * P for a in seq])
        x = torch.randn((T, 3, H, D), device="cuda", generator=g) * torch.exp(0.5 * torch.randn((T, 1, 1, 1), device="cuda", generator=g))
        s["new"] = (x * chan.view(1, 1, H, D)).to(dt)
        s["out"] = [torch.empty((s["back"].numel(), H, D), dtype=dt, device="cuda") for _ in range(2)]
    else:
        G = case["hq"] // H
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        loud = chan.view(H, 1, D).expand(H, G, D).reshape(1, case["hq"], D)
        s["q"] = (torch.randn((T, case["hq"], D), device="cuda", generator=g) * loud).to(dt)
        s["kv_len"], s["cu_q"] = _i32(kv), _i32(cu) if case["q_max"] > 1 else None
        s["max_q"], s["max_kv"] = max(new), max(kv)  # known where the batch is put together
        s["out"] = torch.empty_like(s["q"])
        if own:  # the scratch that a server keeps for its attention
            import free_activation_sparse_b200 as W
            s["ws"] = W.Workspace(W.OP_KV8_ATTENTION, D, max(new) * G, 0, len(kv))
    return s


# ------------------------------------------------------------------------------------
# the calls
# ------------------------------------------------------------------------------------


def run(s):
    case = s["case"]
    if own:
        import free_activation_sparse_b200 as W
        if case["op"] == "plan":
            kv_len, cu_q, slots, positions, n_free = s["out"]
            W.kv8_plan(s["seq"], s["new"], s["table"], s["free"], s["n_free"], case["page"], s["tokens"], kv_len=kv_len,
                       cu_q=cu_q, slots=slots, positions=positions, n_free_out=n_free)
            return [kv_len, cu_q, slots, positions, n_free, s["table"], s["free"]]
        cache = W.Kv8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if case["op"] == "write":
            W.kv8_write(cache, s["new"][:, 1], s["new"][:, 2], s["slots"])
            k, v = W.kv8_read(cache, s["back"], k=s["out"][0], v=s["out"][1])
            return [k, v, s["k_scale"], s["v_scale"]]
        if case["op"] == "read":
            return list(W.kv8_read(cache, s["slots"], k=s["out"][0], v=s["out"][1]))
        return W.kv8_attention(cache, s["q"], s["table"], s["kv_len"], cu_q=s["cu_q"], max_q=s["max_q"],
                               window=case["window"], softcap=case["softcap"], ws=s["ws"], out=s["out"])
    if case["op"] == "plan":
        return _plan(s["seq"], s["new"], s["table"], s["free"], s["n_free"], case["page"], s["tokens"])
    if case["op"] == "write":
        s["k_scale"] = _write(s["k"], s["k_scale"], s["new"][:, 1], s["slots"], case["fmt"])
        s["v_scale"] = _write(s["v"], s["v_scale"], s["new"][:, 2], s["slots"], case["fmt"])
        dt = s["new"].dtype
        return [_read(s["k"], s["k_scale"], s["back"], dt), _read(s["v"], s["v_scale"], s["back"], dt), s["k_scale"], s["v_scale"]]
    if case["op"] == "read":
        dt = _dt(case["dtype"])
        return [_read(s["k"], s["k_scale"], s["slots"], dt), _read(s["v"], s["v_scale"], s["slots"], dt)]
    return _attention(s)


def _plan(seq, new, table, free, n_free, P, tokens):
    """Ended requests (new < 0) push their pages onto the free stack; then the others pop theirs."""
    ended = new < 0
    count = new.clamp(min=0)
    have = (seq + P - 1) // P
    kv_len = torch.where(ended, 0, seq + count)
    need = torch.where(ended, 0, (kv_len + P - 1) // P - have)
    back = torch.where(ended, have, 0)
    cu = torch.cumsum(count, 0)
    cu_q = torch.cat([torch.zeros_like(cu[:1]), cu]).to(torch.int32)
    col = torch.arange(table.shape[1], device=table.device)[None]
    # push: the cells behind the stack's top, in the order of requests and pages
    at = n_free + (torch.cumsum(back, 0) - back)[:, None] + col
    pushed = ended[:, None] & (col < have[:, None])
    stack = torch.cat([free, free[:1]])  # a cell more, for what is not pushed
    stack.scatter_(0, torch.where(pushed, at, free.numel()).reshape(-1), table.reshape(-1))
    top = n_free + back.sum()
    # pop
    j = (torch.cumsum(need, 0) - need)[:, None] + col - have[:, None]
    taken = ~ended[:, None] & (col >= have[:, None]) & (col < (have + need)[:, None])
    table = torch.where(taken, stack[(top - 1 - j).clamp(0, free.numel() - 1)], table)
    t = torch.arange(tokens, device=seq.device)
    b = torch.searchsorted(cu, t, right=True)
    real = b < seq.numel()
    b = b.clamp(max=seq.numel() - 1)
    pos = torch.where(real, seq[b] + t - cu_q[b], 0)
    slots = torch.where(real, table[b, pos // P] * P + pos % P, -1)
    return [kv_len.to(torch.int32), cu_q, slots.to(torch.int32), pos.to(torch.int32), (top - need.sum()).to(torch.int32),
            table, stack[:-1]]


def _write(pages, scale, x, slots, fmt):
    """New rows into their pages, in place; returns the new scales. A page that is written from
    its first place on starts anew; any other keeps its older rows, rounded again where its
    scale grows."""
    n, H, P, D = pages.shape
    x = x.float()
    slots = slots.long()
    page, off = slots // P, slots % P
    amax = torch.zeros((n, H), device=x.device).index_reduce_(0, page, x.abs().amax(2), "amax")
    first = torch.full((n,), P, dtype=torch.int64, device=x.device).scatter_reduce_(0, page, off, "amin")
    fresh = (first == 0)[:, None]
    grown = torch.where(fresh, _scale_of(amax, fmt), torch.maximum(scale, _scale_of(amax, fmt)))
    grown = torch.where((first < P)[:, None], grown, scale)
    older = (torch.arange(P, device=x.device)[None] < first[:, None]) & (first < P)[:, None] & (first > 0)[:, None]
    again = _round8(pages.float() * (scale / grown)[:, :, None, None], fmt)
    # bytes are moved by their bits: not every operation takes 8-bit floats
    raw = torch.where(older[:, None, :, None], again.view(torch.int8), pages.view(torch.int8))
    raw[page, :, off] = _round8(x / grown[page][:, :, None], fmt).view(torch.int8)
    pages.view(torch.int8).copy_(raw)
    return grown


def _read(pages, scale, slots, dt):
    P = pages.shape[2]
    page, off = slots.long() // P, slots.long() % P
    bits = pages.view(torch.int8)[page, :, off]
    return (bits.view(pages.dtype).float() * scale[page][:, :, None]).to(dt)


def _attention(s):
    """Padded to the longest request: [request][kv head][query x group][key]."""
    case, q, table, kv_len = s["case"], s["q"], s["table"], s["kv_len"].long()
    T, Hq, D = q.shape
    B, H, P, nq, nk = kv_len.numel(), case["hkv"], case["page"], s["max_q"], s["max_kv"]
    G = Hq // H
    cu = s["cu_q"].long() if s["cu_q"] is not None else torch.arange(B + 1, device=q.device)
    width = -(-nk // P)
    at = table[:, :width].long().clamp(min=0)

    def dense(pages, scale):  # [B][H][keys][D]
        x = pages.view(torch.int8)[at].view(pages.dtype).float() * scale[at][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, width * P, D)[:, :, :nk]

    i = torch.arange(nq, device=q.device)
    n_q = cu[1:] - cu[:-1]
    rows = (cu[:-1, None] + i).clamp(max=T - 1)
    x = q.float()[rows].reshape(B, nq, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, nq * G, D)
    score = (x / math.sqrt(D)) @ dense(s["k"], s["k_scale"]).transpose(2, 3)
    if case["softcap"]:
        score = case["softcap"] * torch.tanh(score / case["softcap"])
    pos = (kv_len - n_q)[:, None] + i
    j = torch.arange(nk, device=q.device)
    seen = (j <= pos[:, :, None]) & (j < kv_len[:, None, None])
    if case["window"]:
        seen = seen & (j > pos[:, :, None] - case["window"])
    seen = seen[:, None, :, None, :].expand(B, 1, nq, G, nk).reshape(B, 1, nq * G, nk)
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(3, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    total = p.sum(3, keepdim=True)
    o = (p @ dense(s["v"], s["v_scale"])) / torch.where(total > 0, total, 1.0)
    o = o.reshape(B, H, nq, G, D).permute(0, 2, 1, 3, 4).reshape(B, nq, Hq, D)
    t = torch.arange(T, device=q.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return o[b, t - cu[b]].to(q.dtype)


# ------------------------------------------------------------------------------------
# the definition, in 64 bits
# ------------------------------------------------------------------------------------


def _two(e):
    """2^e exactly, for whole e from -1000 to 1000."""
    return torch.tensor([math.ldexp(1.0, i) for i in range(-1000, 1001)], dtype=torch.float64, device=e.device)[e.long() + 1000]


def _scale64(amax, fmt):
    """The least e with qmax 2^e >= amax, found by trying the neighbours of its logarithm."""
    top = QMAX[fmt]
    e = torch.floor(torch.log2((amax / top).clamp(min=1e-290)))
    for _ in range(2):
        e = torch.where(top * _two(e) < amax, e + 1, e)
    for _ in range(2):
        e = torch.where(top * _two(e - 1) >= amax, e - 1, e)
    return _two(torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX))


def _near8(x, fmt):
    """The nearest number that the format holds, ties to even, for |x| <= qmax."""
    if fmt == "int8":
        return torch.round(x)
    top = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    top = torch.where(_two(top) > x.abs().clamp(min=2.0 ** -6), top - 1, top)
    top = torch.where(_two(top + 1) <= x.abs(), top + 1, top)
    step = _two(top - 3)
    return torch.round(x / step) * step


def _write64(pages, scale, x, slots, back, page, fmt):
    """Page by page, as the definition reads: the values at the places `back`, and the scales."""
    val, scale, x = pages.float().double(), scale.double(), x.double()
    at = slots.long()
    starts = [0] + [i for i in range(1, at.numel()) if int(at[i]) // page != int(at[i - 1]) // page]
    for a, b in zip(starts, starts[1:] + [at.numel()]):
        p, off = int(at[a]) // page, int(at[a]) % page
        rows = x[a:b]
        s = _scale64(rows.abs().amax((0, 2)), fmt)
        if off:
            s = torch.maximum(s, scale[p])
            val[p, :, :off] = _near8(val[p, :, :off] * (scale[p] / s)[:, None, None], fmt)
        scale[p] = s
        val[p, :, off:off + b - a] = _near8((rows / s[:, None]).permute(1, 0, 2), fmt)
    back = back.long()
    return val[back // page, :, back % page] * scale[back // page][:, :, None], scale


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    P = case["page"]
    if case["op"] == "read":
        at = s["slots"].long()
        return [s[n].float().double()[at // P, :, at % P] * s[n + "_scale"].double()[at // P][:, :, None] for n in ("k", "v")]
    if case["op"] == "write":
        at, back = s["slots"].cpu(), s["back"]
        k = _write64(s["k"], s["k_scale"], s["new"][:, 1], at, back, P, case["fmt"])
        v = _write64(s["v"], s["v_scale"], s["new"][:, 2], at, back, P, case["fmt"])
        return [k[0], v[0], k[1], v[1]]
    # attention: request by request, and some queries at a time
    T, Hq, D = s["q"].shape
    H = case["hkv"]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    seq, new = _lengths(case)
    a = 0
    for b, n in enumerate(new):
        kv = int(s["kv_len"][b])
        if kv:
            pages = s["table"][b, : -(-kv // P)].long()

            def rows(x, f):
                x = x[pages].float().double() * f[pages].double()[:, :, None, None]
                return x.transpose(0, 1).reshape(H, -1, D)[:, :kv].repeat_interleave(Hq // H, 0)

            K, V = rows(s["k"], s["k_scale"]), rows(s["v"], s["v_scale"])
            some = max(1, (1 << 27) // (Hq * kv))
            for i in range(0, n, some):
                m = min(some, n - i)
                z = torch.einsum("qhd,hkd->hqk", s["q"][a + i:a + i + m].double(), K) * D ** -0.5
                if case["softcap"]:
                    z = torch.tanh(z / case["softcap"]) * case["softcap"]
                back = torch.arange(kv - n + i, kv - n + i + m, device="cuda")[:, None] - torch.arange(kv, device="cuda")
                z[:, (back < 0) | ((back >= case["window"]) if case["window"] else (back < 0))] = -math.inf
                out[a + i:a + i + m] = torch.einsum("hqk,hkd->qhd", torch.softmax(z, -1), V)
        a += n
    return out
