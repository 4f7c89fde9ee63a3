"""The token-mixing operators of a decode layer, as measured cases.

Between the QKV matrix product and the O matrix product of a layer stand
  append   the rotation of the queries and keys by their positions, and the
           keys' and values' way into a paged cache;
  attend   attention of each sequence's new tokens over that cache;
  linear   in a layer of the other kind, linear attention with a decay for
           each head, over a state that takes the cache's place.

`run` computes one of them: in elementary torch operations where `own` is
false, through the library's calls where it is true.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
CHUNK = 128        # tokens of one step of the plain linear attention


# ---- cases ------------------------------------------------------------------

def _append(name, seqs, new, ctx, q_heads, kv_heads, dim, page, dtype, rot, **more):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "ctx": ctx, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "rot": rot,
            "interleaved": False, "factor": 1.0, "head_major": False, **more}


def _attend(name, seqs, new, ctx, q_heads, kv_heads, dim, page, dtype, **more):
    return {"name": name, "op": "attend", "seqs": seqs, "new": new, "ctx": ctx, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "window": 0,
            "head_major": False, **more}


def _linear(name, seqs, new, qk_heads, v_heads, k_dim, v_dim, dtype, **more):
    return {"name": name, "op": "linear", "seqs": seqs, "new": new, "qk_heads": qk_heads,
            "v_heads": v_heads, "k_dim": k_dim, "v_dim": v_dim, "dtype": dtype, "fixed": False, **more}


def listed():
    return [
        # One user's next token: the 7168 outputs of a 27B-shaped layer's QKV product (40 query, 8 key
        # and 8 value heads of 128). Latency is all of it.
        _append("append_token", 1, 1, 4095, 40, 8, 128, 16, "f16", 128),
        # A batch of users, one token each, far into long contexts: interleaved pairs over a quarter
        # of the head, positions scaled past the trained length.
        _append("append_batch_far", 48, 1, 200000, 32, 4, 256, 64, "bf16", 64, interleaved=True, factor=8.0),
        # Prompts of several users at once, of all lengths up to 2048 tokens.
        _append("append_prompts", 6, 2048, 500, 40, 8, 128, 16, "f16", 128, head_major=True),
        # One user's next token after 4095 others.
        _attend("attend_token", 1, 1, 4095, 40, 8, 128, 16, "f16"),
        # Thirty-two users' next tokens, contexts of all lengths up to 16384: the cache's bytes bound it.
        _attend("attend_batch", 32, 1, 16383, 40, 8, 128, 64, "bf16"),
        # Four drafted tokens each to verify, behind a sliding window.
        _attend("attend_verify_window", 7, 4, 30000, 16, 2, 64, 32, "f16", window=4096, head_major=True),
        # A fresh prompt of 169 tokens.
        _attend("attend_prompt", 1, 169, 0, 40, 8, 128, 16, "f16"),
        # Chunks of several users' prompts; pages of 24 tokens end inside every tile.
        _attend("attend_chunks", 4, 1024, 8192, 16, 4, 64, 24, "bf16"),
        # A chunk of 4096 tokens at the end of a context of 16384.
        _attend("attend_chunk_long", 1, 4096, 12288, 40, 8, 128, 64, "f16"),
        # One user's next token in a layer with a state: 8 query and key heads, 40 value heads
        # (7168 outputs of the QKV product again), the decay computed from the token.
        _linear("linear_token", 1, 1, 8, 40, 128, 128, "f16"),
        # Ninety-six users' next tokens: the states' bytes bound it.
        _linear("linear_batch", 96, 1, 8, 40, 128, 128, "bf16"),
        # Three long prompts, up to 16384 tokens, fixed decays.
        _linear("linear_prompts", 3, 16384, 8, 40, 128, 128, "f16", fixed=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    tops = {}
    for c in listed():
        w = work(c)
        tops[c["op"]] = {k: max(tops.get(c["op"], {}).get(k, 0), w[k]) for k in w}
    op = rng.choice(["append", "attend", "attend", "linear"])
    while True:
        c = _drawn(rng, op)
        w = work(c)
        if w["bytes"] <= tops[op]["bytes"] and w["flops"] <= tops[op]["flops"] and _plain_room(c):
            return c


def _drawn(rng, op):
    dtype = rng.choice(["f16", "bf16"])
    if op == "linear":
        qk = rng.choice([1, 2, 3, 4, 8])
        step = rng.random() < 0.4                            # single tokens, or prompts
        return _linear("", _log_int(rng, 1, 96 if step else 6), 1 if step else _log_int(rng, 2, 16384), qk,
                       qk * rng.choice([1, 2, 3, 5]), rng.choice([64, 128]), rng.choice([64, 128]), dtype,
                       fixed=rng.random() < 0.5)
    kv = rng.choice([1, 2, 3, 4, 8])
    q = kv * rng.choice([1, 2, 3, 4, 5, 6, 8])
    dim = rng.choice([64, 64, 80, 96, 128, 128, 256])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 100, 128])
    form = rng.choice(["token", "verify", "prompt"])
    seqs = _log_int(rng, 1, 64 if form == "token" else 16)
    new = 1 if form == "token" else rng.randint(2, 8) if form == "verify" else _log_int(rng, 9, 4096)
    ctx = rng.choice([0, _log_int(rng, 1, 16384), _log_int(rng, 512, 16384), _log_int(rng, 512, 16384)])
    head_major = rng.random() < 0.5
    if op == "append":
        return _append("", seqs, new, rng.choice([ctx, _log_int(rng, 1, 1000000)]), q, kv, dim, page, dtype,
                       2 * rng.randint(1, dim // 2) if rng.random() < 0.3 else rng.choice([dim, dim // 2]),
                       interleaved=rng.random() < 0.5, factor=rng.choice([1.0, 1.0, 4.0, 16.0]),
                       head_major=head_major)
    window = rng.choice([0, 0, _log_int(rng, 1, 8192)])
    return _attend("", seqs, new, ctx, q, kv, dim, page, dtype, window=window, head_major=head_major)


def _plain_room(c):
    """Whether the plain form's padded intermediate values stay near the largest listed case's."""
    if c["op"] == "attend":
        new, length = _lengths(c)
        return c["seqs"] * max(length) * max(c["q_heads"] * max(new), 2 * c["kv_heads"] * c["dim"]) <= 2.8e9
    if c["op"] == "append":
        new, length = _lengths(c)
        return sum(length) // c["page"] <= 20_000_000
    return True


def _lengths(c):
    """(new tokens, tokens with the new ones) of each sequence: the first has the case's full
    counts, the others any count up to them, now and then no new token."""
    r = random.Random("%d/%d/%d" % (c["seqs"], c["new"], c.get("ctx", 0)))
    new, length = [], []
    for s in range(c["seqs"]):
        n = c["new"] if s == 0 else 0 if s > 1 and r.random() < 0.06 else r.randint(1, c["new"])
        new.append(n)
        length.append(n + (c.get("ctx", 0) if s == 0 else r.randint(0, c.get("ctx", 0))))
    return new, length


def _seen(n, length, window):
    """Pairs of a new token and a token that it attends to, of one sequence."""
    w = window or length
    first = length - n + 1                                   # tokens that the first new one sees
    full = max(0, min(n, w - first))                         # new tokens whose window is not full
    return full * first + full * (full - 1) // 2 + (n - full) * min(w, length)


def work(c):
    new, length = _lengths(c)
    rows = sum(new)
    if c["op"] == "append":
        per_row = 2 * 2 * (c["q_heads"] + 2 * c["kv_heads"]) * c["dim"]
        return {"bytes": rows * per_row, "flops": rows * (c["q_heads"] + c["kv_heads"]) * c["rot"] * 3}
    if c["op"] == "attend":
        w = c["window"]
        keys = sum(min(l, w + n - 1) if w else l for n, l in zip(new, length) if n)
        pairs = sum(_seen(n, l, w) for n, l in zip(new, length) if n)
        return {"bytes": 2 * 2 * (rows * c["q_heads"] + keys * c["kv_heads"]) * c["dim"],
                "flops": 4 * pairs * c["q_heads"] * c["dim"]}
    qk, v = c["qk_heads"] * c["k_dim"], c["v_heads"] * c["v_dim"]
    gates = c["v_heads"] if c["fixed"] else rows * c["v_heads"]
    state = c["seqs"] * c["k_dim"] * v
    return {"bytes": 2 * 2 * rows * (qk + v) + 4 * gates + 2 * 4 * state, "flops": 4 * rows * c["k_dim"] * v}


# ---- inputs -----------------------------------------------------------------

def _freqs(rot, base, factor, trained):
    """Radians per position of each rotated pair, in 64 bits. With a factor the slow pairs (under
    1 turn in the trained length) turn that much slower, the fast ones (over 32) as before."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor != 1.0:
        turns = trained * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0, dt=dtype):
        x = torch.empty(shape, dtype=dt, device=dev).normal_(generator=gen)
        return x.mul_(scale) if scale != 1.0 else x

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    new, length = _lengths(case)
    rows, seqs = sum(new), case["seqs"]
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    st = {"case": case, "start": ints(start), "max_new": max(new), "max_len": max(length)}
    if case["op"] == "linear":
        hk, hv, dk, dv = case["qk_heads"], case["v_heads"], case["k_dim"], case["v_dim"]
        qkv = randn(rows, 2 * hk * dk + hv * dv)             # rows of the QKV product
        qkv[:, :2 * hk * dk] *= dk ** -0.5
        st["q"] = qkv[:, :hk * dk].view(rows, hk, dk)
        st["k"] = qkv[:, hk * dk:2 * hk * dk].view(rows, hk, dk)
        st["v"] = qkv[:, 2 * hk * dk:].view(rows, hv, dv)
        rate = 2.0 ** -(1 + 8 * torch.arange(hv, device=dev, dtype=torch.float32) / hv)
        if case["fixed"]:
            st["log_decay"] = (-rate).expand(rows, hv)
        else:
            u = torch.empty(rows, hv, device=dev).uniform_(0.25, 1.75, generator=gen)
            st["log_decay"] = -(rate * u)
        st["state"] = randn(seqs, hv, dk, dv, scale=0.5, dt=torch.float32)
        st["state_out"] = torch.zeros_like(st["state"])
        st["slots"] = torch.randperm(seqs, generator=gen, device=dev).to(torch.int32)
        st["out"] = torch.zeros(rows, hv, dv, dtype=dtype, device=dev)
        return st

    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    st["length"] = ints(length)
    st["out"] = torch.zeros(rows, hq, d, dtype=dtype, device=dev)
    n_pages = [(l + page - 1) // page for l in length]
    width = max(n_pages + [1])
    if case["op"] == "append":
        # Only the pages that the new tokens go to are a sequence's own; what lies before is not touched.
        first = [(l - n) // page for l, n in zip(length, new)]
        touched = [p - f if n else 0 for p, f, n in zip(n_pages, first, new)]
    else:
        first, touched = [0] * seqs, n_pages
    pool = sum(touched) + 3
    order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(seqs, width, dtype=torch.int32, device=dev)
    at = 0
    for s in range(seqs):
        table[s, first[s]:first[s] + touched[s]] = order[at:at + touched[s]]
        at += touched[s]
    shape = (pool, hkv, page, d) if case["head_major"] else (pool, page, hkv, d)
    k, v = randn(*shape), randn(*shape)
    st["k_cache"], st["v_cache"] = (k.transpose(1, 2), v.transpose(1, 2)) if case["head_major"] else (k, v)
    st["table"] = table
    if case["op"] == "append":
        qkv = randn(rows, (hq + 2 * hkv) * d)                # rows of the QKV product
        st["q"] = qkv[:, :hq * d].view(rows, hq, d)
        st["k"] = qkv[:, hq * d:(hq + hkv) * d].view(rows, hkv, d)
        st["v"] = qkv[:, (hq + hkv) * d:].view(rows, hkv, d)
        st["freqs"] = _freqs(case["rot"], 1e6, case["factor"], 32768.0).to(dev)
        st["amp"] = 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0
    else:
        st["q"] = randn(rows, hq, d, scale=2.0)
        st["scale"] = d ** -0.5
    return st


# ---- one pass ---------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "linear": _own_linear}[op](state)
    return {"append": _plain_append, "attend": _plain_attend, "linear": _plain_linear}[op](state)


def _rows(st):
    """Sequence of each row, and its place among the sequence's new tokens."""
    start = st["start"].long()
    r = torch.arange(st["q"].shape[0], device=start.device)
    s = torch.searchsorted(start[1:], r, right=True)
    return s, r - start[s]


def _plain_append(st):
    c = st["case"]
    s, i = _rows(st)
    length, start = st["length"].long(), st["start"].long()
    pos = length[s] - (start[s + 1] - start[s]) + i
    angle = pos.double()[:, None] * st["freqs"]
    cos, sin = ((st["amp"] * f(angle)).float()[:, None, :] for f in (torch.cos, torch.sin))

    def rotate(x):
        x = x.float()
        head, tail = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["interleaved"]:
            a, b = head[..., 0::2], head[..., 1::2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = head.chunk(2, -1)
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((turned, tail), -1)

    page = st["table"].long()[s, pos // c["page"]]
    st["out"].copy_(rotate(st["q"]))
    st["k_cache"][page, pos % c["page"]] = rotate(st["k"]).to(st["k_cache"].dtype)
    st["v_cache"][page, pos % c["page"]] = st["v"]
    return {"q": st["out"], "k": st["k_cache"], "v": st["v_cache"]}


def _plain_attend(st):
    c = st["case"]
    hq, hkv, d, n, m, top = c["q_heads"], c["kv_heads"], c["dim"], c["seqs"], st["max_new"], st["max_len"]
    dev = st["q"].device
    s, i = _rows(st)
    length, start = st["length"].long(), st["start"].long()
    q = torch.zeros(n, m, hq, d, device=dev)
    q[s, i] = st["q"].float()
    q = q.view(n, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    j = torch.arange(top, device=dev)
    there = j < length[:, None]                                                  # [n, top]
    page = st["table"].long()[:, j // c["page"]]

    def cached(x):
        x = torch.where(there[..., None, None], x[page, j % c["page"]].float(), 0.0)
        return x.permute(0, 2, 1, 3)                                             # [n, hkv, top, d]

    pos = (length - (start[1:] - start[:-1]))[:, None] + torch.arange(m, device=dev)
    seen = there[:, None, :] & (j <= pos[..., None])                             # [n, m, top]
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    score = torch.matmul(q, cached(st["k_cache"]).transpose(2, 3)).mul_(st["scale"])
    score = score.view(n, hkv, hq // hkv, m, top).masked_fill_(~seen[:, None, None], -math.inf)
    high = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(high.isfinite(), high, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, hkv, -1, top), cached(st["v_cache"])).view(n, hkv, hq // hkv, m, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n, m, hq, d)
    return o[s, i].to(st["q"].dtype)


def _plain_linear(st):
    c = st["case"]
    hv, n = c["v_heads"], c["seqs"]
    dev, m = st["q"].device, st["max_new"]
    s, i = _rows(st)

    def padded(x, dt=torch.float32):
        y = torch.zeros(n, m, *x.shape[1:], device=dev, dtype=dt)
        y[s, i] = x.to(dt)
        return y.transpose(1, 2)                                                 # [n, heads, m, ...]

    each = hv // c["qk_heads"]
    q, k = (padded(st[x]).repeat_interleave(each, 1) for x in "qk")
    v, g = padded(st["v"]), padded(st["log_decay"], torch.float64)
    state = st["state"][st["slots"].long()]
    outs = []
    for t in range(0, m, CHUNK):
        qc, kc, vc, gc = (x[:, :, t:t + CHUNK] for x in (q, k, v, g))
        b = gc.cumsum(-1)                                                        # 64 bits
        span = b[..., :, None] - b[..., None, :]
        low = torch.ones(b.shape[-1], b.shape[-1], dtype=torch.bool, device=dev).tril()
        w = torch.where(low, span, -math.inf).exp().float()
        o = torch.matmul(torch.matmul(qc, kc.transpose(2, 3)) * w, vc)
        outs.append(o + torch.matmul(qc * b.exp().float()[..., None], state))
        left = (b[..., -1:] - b).exp().float()[..., None]
        state = state * b[..., -1].exp().float()[..., None, None] + torch.matmul((kc * left).transpose(2, 3), vc)
    st["state_out"][st["slots"].long()] = state
    return {"out": torch.cat(outs, 2).transpose(1, 2)[s, i].to(st["q"].dtype), "state": st["state_out"]}


# ---- the library's calls ----------------------------------------------------

_engines = {}


def _engine(device):
    import q4_quantized_decode_b200 as q4
    if device.index not in _engines:
        _engines[device.index] = q4.Q4Gemv(device.index or 0)
    return _engines[device.index]


def _cache(st):
    import q4_quantized_decode_b200 as q4
    if "cache" not in st:                                    # a program makes it once, with its pools
        st["cache"] = q4.PagedKV(st["k_cache"], st["v_cache"], st["table"])
    return st["cache"]


def _own_append(st):
    c = st["case"]
    _engine(st["q"].device).kv_append(_cache(st), st["start"], st["length"], st["k"], st["v"], q=st["q"],
                                      q_out=st["out"], freqs=st["freqs"], interleaved=c["interleaved"],
                                      amp=st["amp"])
    return {"q": st["out"], "k": st["k_cache"], "v": st["v_cache"]}


def _own_attend(st):
    return _engine(st["q"].device).attn_paged(_cache(st), st["start"], st["length"], st["q"], scale=st["scale"],
                                              window=st["case"]["window"], max_new=st["max_new"], out=st["out"])


def _own_linear(st):
    out, state = _engine(st["q"].device).linattn(st["q"], st["k"], st["v"], st["log_decay"], st["start"],
                                                 st["state"], state_out=st["state_out"], slots=st["slots"],
                                                 max_new=st["max_new"], out=st["out"])
    return {"out": out, "state": state}


# ---- the definition, in 64 bits ---------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "linear": _exact_linear}[case["op"]](case, st)


def _exact_append(case, st):
    new, length = _lengths(case)
    pos = [p for n, l in zip(new, length) for p in range(l - n, l)]
    seq = [s for s, n in enumerate(new) for _ in range(n)]
    dev, rot = st["q"].device, case["rot"]
    at = torch.tensor(pos, dtype=torch.float64, device=dev)
    turn = torch.polar(torch.full((len(pos), rot // 2), st["amp"], dtype=torch.float64, device=dev),
                       torch.outer(at, st["freqs"]))[:, None]

    def rotate(x):
        x = x.double().clone()
        first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
        second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    ix = torch.tensor([[s, p // case["page"], p % case["page"]] for s, p in zip(seq, pos)], device=dev).view(-1, 3)
    page = st["table"][ix[:, 0], ix[:, 1]].long()
    k, v = st["k_cache"].double(), st["v_cache"].double()
    k[page, ix[:, 2]] = rotate(st["k"])
    v[page, ix[:, 2]] = st["v"].double()
    return {"q": rotate(st["q"]), "k": k, "v": v}


def _exact_attend(case, st):
    new, length = _lengths(case)
    each = case["q_heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    row = 0
    for s, (n, l) in enumerate(zip(new, length)):
        if n == 0:
            continue
        pages = st["table"][s, :(l + case["page"] - 1) // case["page"]].long()
        p = torch.arange(l - n, l, device=out.device)[:, None]
        j = torch.arange(l, device=out.device)[None]
        hidden = (j > p) | (j <= p - case["window"] if case["window"] else j < 0)
        for h in range(case["kv_heads"]):
            k = st["k_cache"][pages, :, h].reshape(-1, case["dim"])[:l].double()
            v = st["v_cache"][pages, :, h].reshape(-1, case["dim"])[:l].double()
            for g in range(h * each, (h + 1) * each):
                a = st["q"][row:row + n, g].double() @ k.T * case["dim"] ** -0.5
                a[hidden] = -math.inf
                out[row:row + n, g] = torch.softmax(a, 1) @ v
        row += n
    return out


def _exact_linear(case, st):
    new, _ = _lengths(case)
    if max(new) * case["seqs"] * case["v_heads"] * case["k_dim"] * case["v_dim"] > 1e11:
        return None
    each = case["v_heads"] // case["qk_heads"]
    head = torch.arange(case["v_heads"], device=st["q"].device) // each
    start = [sum(new[:s]) for s in range(case["seqs"])]
    slots = st["slots"].long()
    state = st["state"].double()[slots]
    out = torch.zeros(st["v"].shape, dtype=torch.float64, device=st["q"].device)
    by_len = sorted(range(case["seqs"]), key=lambda s: -new[s])                  # the longest first
    state = state[by_len]
    for t in range(max(new)):
        live = [s for s in by_len if new[s] > t]
        r = torch.tensor([start[s] + t for s in live], device=out.device)
        a = st["log_decay"][r].double().exp()[..., None, None]
        now = state[:len(live)]
        now.mul_(a).add_(st["k"][r].double()[:, head, :, None] * st["v"][r].double()[:, :, None, :])
        out[r] = (st["q"][r].double()[:, head, None, :] @ now)[:, :, 0]
    full = torch.zeros_like(state)
    full[slots[torch.tensor(by_len, device=out.device)]] = state
    return {"out": out, "state": full}
