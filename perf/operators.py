"""Workloads of the paged-cache operators: M-RoPE append into a paged KV cache,
attention over that cache, and attention of candidates that share a prompt.

``listed()`` names the workloads, ``draw(rng)`` makes more of the same ranges,
``prepare(case, seed)`` makes a case's inputs on the GPU, ``run(state)`` makes
one pass (in plain torch operations, or, where ``own`` is true, through the
package's entry points), ``exact(case, seed)`` gives the same outputs from the
definitions in 64 bits, and ``work(case)`` the bytes and operations that a pass
cannot do without.

Sizes follow the package's 1.7B-parameter speech decoder (16 query heads, 8 key
heads of 128, M-RoPE sections 24/20/20, theta 1e6, 5 or 256 candidates).
"""
import math
import random

import torch

own = False

THETA = 1.0e6
EPS = 1.0e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _append(name, **kw):
    case = {"name": name, "op": "append", "dtype": "bf16", "hq": 16, "hk": 8, "d": 128, "page": 16,
            "norm": True, "seqs": 5, "new_lo": 1, "new_hi": 1, "past_lo": 0, "past_hi": 0, "order": 1}
    case.update(kw)
    return case


def _attend(name, **kw):
    case = {"name": name, "op": "attend", "dtype": "bf16", "hq": 16, "hk": 8, "d": 128, "page": 16,
            "seqs": 5, "new_lo": 1, "new_hi": 1, "past_lo": 0, "past_hi": 0, "cap": 0.0, "window": 0,
            "slopes": False, "bidir": 0, "order": 1}
    case.update(kw)
    return case


def _shared(name, **kw):
    case = {"name": name, "op": "shared", "dtype": "bf16", "hq": 16, "hk": 8, "d": 128, "page": 16,
            "groups": 1, "members_lo": 5, "members_hi": 5, "prefix_lo": 1000, "prefix_hi": 1000,
            "past_lo": 1, "past_hi": 300, "cap": 0.0, "window": 0, "slopes": False, "order": 1}
    case.update(kw)
    return case


def listed():
    return [
        # one decode step's append for 5 candidates of one utterance: latency
        _append("append_decode_5", seqs=5, past_lo=100, past_hi=1200),
        # a ragged batch of prompts entering the cache, out of a packed q/k/v projection
        _append("append_prompts", seqs=9, new_lo=37, new_hi=1500, page=32),
        # one decode step's attention for 5 candidates: latency
        _attend("decode_5", seqs=5, past_lo=200, past_hi=1500),
        # a full serving batch in the middle of its utterances
        _attend("decode_256", seqs=256, past_lo=60, past_hi=4100),
        # a few very long sessions: few rows, a long axis
        _attend("decode_long", seqs=3, past_lo=60000, past_hi=131000, page=64),
        # several prompts prefilled together, lengths as they come
        _attend("prompts_ragged", seqs=9, new_lo=37, new_hi=1500, page=32),
        # one long prompt
        _attend("prompt_16384", seqs=1, new_lo=16384, new_hi=16384, page=64),
        # a chunk of a prompt on a long cache, capped scores and a distance bias
        _attend("chunk_capped", seqs=2, new_lo=90, new_hi=130, past_lo=12000, past_hi=21000, cap=30.0,
                slopes=True),
        # 32-bit storage, heads of 64, odd sizes, a sliding window, a bidirectional prompt start
        _attend("window_f32", dtype="f32", hq=12, hk=4, d=64, page=24, seqs=7, new_lo=1, new_hi=333,
                past_lo=0, past_hi=2500, window=700, bidir=50),
        # 5 candidates of one prompt: latency
        _shared("candidates_5", prefix_lo=1100, prefix_hi=1100),
        # many requests of 5 candidates each, prompts of their own
        _shared("requests_of_5", groups=51, prefix_lo=200, prefix_hi=2200),
        # one long prompt (a voice and style description) under a full batch
        _shared("candidates_256", members_lo=256, members_hi=256, prefix_lo=8192, prefix_hi=8192,
                past_hi=600, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges: decode steps and prompts, short and
    long caches, both types, other head layouts, odd sizes, every score option."""
    op = rng.choice(("append", "attend", "attend", "shared"))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    hq, hk = rng.choice(((16, 8), (16, 8), (12, 4), (16, 2), (7, 7), (24, 3), (8, 1)))
    d = rng.choice((128, 128, 64, 96, 80))
    page = rng.choice((16, 16, 32, 64, 128, 24, 20, 1 if op == "append" else 8))
    order = rng.randrange(1, 1 << 30)
    kw = {"dtype": dtype, "hq": hq, "hk": hk, "d": d, "page": page, "order": order}
    if op == "append":
        kw["norm"] = rng.random() < 0.6
        if rng.random() < 0.5:
            kw.update(seqs=_log_int(rng, 1, 300), past_lo=rng.randrange(0, 50), past_hi=_log_int(rng, 60, 3000))
        else:
            seqs = _log_int(rng, 1, 30)
            hi = max(2, _log_int(rng, 20, 8000) // seqs)
            kw.update(seqs=seqs, new_lo=1, new_hi=hi, past_lo=0, past_hi=rng.randrange(0, 300))
        return _append("", **kw)
    kw["cap"] = rng.choice((0.0, 0.0, 0.0, 20.0, 50.0))
    kw["window"] = rng.choice((0, 0, 0, _log_int(rng, 30, 3000)))
    kw["slopes"] = rng.random() < 0.25
    per_key = hk * d * (8 if dtype == "f32" else 4)  # bytes of keys and values a position
    if op == "shared":
        groups = _log_int(rng, 1, 40)
        members = _log_int(rng, 1, max(2, 256 // groups))
        prefix = _log_int(rng, 50, 9000 if groups < 4 else 1500)
        kw.update(groups=groups, members_lo=rng.randrange(1, members + 1), members_hi=members,
                  prefix_lo=rng.randrange(1, prefix + 1), prefix_hi=prefix,
                  past_lo=rng.randrange(0, 3), past_hi=_log_int(rng, 4, 700))
        return _shared("", **kw)
    kind = rng.random()
    if kind < 0.5:  # decode; 600 MB of cache at most
        seqs = _log_int(rng, 1, 256)
        most = max(40, min(100000, 600_000_000 // (per_key * seqs)))
        hi = _log_int(rng, 30, most)
        kw.update(seqs=seqs, past_lo=rng.randrange(0, hi), past_hi=hi)
        if rng.random() < 0.2:  # a few tokens checked at once
            kw.update(new_lo=1, new_hi=rng.randrange(2, 9))
    else:  # prompts, chunks
        budget = 1000 if dtype == "f32" else 6000
        seqs = _log_int(rng, 1, 20)
        hi = max(3, _log_int(rng, 20, budget) // seqs)
        kw.update(seqs=seqs, new_lo=rng.randrange(1, hi), new_hi=hi, past_lo=0,
                  past_hi=_log_int(rng, 1, 4000))
        if rng.random() < 0.3:
            kw["bidir"] = rng.randrange(1, 400)
    return _attend("", **kw)


def _spread(rng, n, lo, hi):
    """n lengths in [lo, hi], the ends among them where there are several."""
    v = [rng.randint(lo, hi) for _ in range(n)]
    if n > 1:
        v[rng.randrange(n)] = hi
    return v


def _lengths(case):
    """The case's lengths: (new, past) tokens of every sequence, and for shared
    prompts the members and prefix length of every group."""
    rng = random.Random(case["order"])
    if case["op"] == "shared":
        members = _spread(rng, case["groups"], case["members_lo"], case["members_hi"])
        prefix = _spread(rng, case["groups"], case["prefix_lo"], case["prefix_hi"])
        n = sum(members)
        return [1] * n, _spread(rng, n, case["past_lo"], case["past_hi"]), members, prefix
    n = case["seqs"]
    new = _spread(rng, n, case["new_lo"], case["new_hi"])
    past = _spread(rng, n, case["past_lo"], case["past_hi"])
    return new, past, None, None


def _visible(case, i, length):
    """(first, last + 1) of the keys that query position i of `length` sees."""
    last = min(length, max(i + 1, case.get("bidir", 0)))
    first = max(0, i - case["window"] + 1) if case["window"] else 0
    return first, max(first, last)


def work(case):
    new, past, members, prefix = _lengths(case)
    e = 2 if case["dtype"] == "bf16" else 4
    hq, hk, d = case["hq"], case["hk"], case["d"]
    tokens = sum(new)
    if case["op"] == "append":
        # q, k, v read, q written, k and v written to their slots, positions and table read
        nbytes = tokens * (2 * hq + 4 * hk) * d * e + tokens * 12 + len(new) * 8
        # rotation: 6 operations a pair; norm: 4 an element
        flops = tokens * (hq + hk) * d * (3 + (4 if case["norm"] else 0))
        return {"bytes": nbytes, "flops": flops}
    pairs, keys = 0, 0
    if case["op"] == "shared":
        s = 0
        for m, p in zip(members, prefix):
            lowest = p
            for _ in range(m):
                length = p + past[s]
                first, last = _visible(case, length - 1, length)
                pairs += last - first
                keys += max(0, length - max(first, p))
                lowest = min(lowest, first)
                s += 1
            keys += p - lowest
    else:
        for n, p in zip(new, past):
            length = n + p
            lo, hi = length, 0
            for i in range(p, length):
                first, last = _visible(case, i, length)
                pairs += last - first
                lo, hi = min(lo, first), max(hi, last)
            keys += max(0, hi - lo)
    nbytes = 2 * tokens * hq * d * e + 2 * keys * hk * d * e + 4 * (keys // case["page"] + 2 * len(new))
    return {"bytes": nbytes, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _pages_for(lens, page, order, pad):
    """Block table [n, max_pages] int32: pages handed out from a shuffled pool;
    entries past a sequence's pages hold 0."""
    counts = [-(-n // page) for n in lens]
    table = torch.zeros(len(lens), max(1, max(counts)) + pad, dtype=torch.int32)
    at = 0
    for s, c in enumerate(counts):
        table[s, :c] = order[at:at + c]
        at += c
    return table, at


def _sections(d):
    half = d // 2
    h = (half * 20) // 64
    return (half - 2 * h, h, h)


def prepare(case, seed):
    dev = torch.device("cuda")
    dt = DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    shuffle = torch.Generator().manual_seed(int(seed))
    new, past, members, prefix = _lengths(case)
    hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
    tokens = sum(new)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * std).to(dt)

    def pool(pages):
        t = torch.empty(pages, hk, page, d, dtype=dt, device=dev)
        return t.normal_(generator=gen)

    st = {"case": dict(case)}
    if case["op"] == "shared":
        lens, own_lens = list(past), list(past)
        need = sum(-(-p // page) for p in prefix) + sum(-(-n // page) for n in own_lens)
        order = torch.randperm(need + 3, generator=shuffle).to(torch.int32)
        ptab, at = _pages_for(prefix, page, order, 1)
        tab, _ = _pages_for(own_lens, page, order[at:], 1)
        start = [0]
        for m in members:
            start.append(start[-1] + m)
        st.update(group_start=torch.tensor(start, dtype=torch.int32).to(dev),
                  prefix_lens=torch.tensor(prefix, dtype=torch.int32).to(dev),
                  prefix_table=ptab.to(dev), host_members=members, host_prefix=prefix)
        pages = need + 3
    else:
        lens = [n + p for n, p in zip(new, past)]
        need = sum(-(-n // page) for n in lens)
        order = torch.randperm(need + 3, generator=shuffle).to(torch.int32)
        tab, _ = _pages_for(lens, page, order, 1)
        pages = need + 3
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    st.update(k_pages=pool(pages), v_pages=pool(pages), block_table=tab.to(dev),
              kv_lens=torch.tensor(lens, dtype=torch.int32).to(dev),
              q_start=torch.tensor(start, dtype=torch.int32).to(dev),
              host_new=new, host_lens=lens)
    if case["op"] == "append":
        # q, k and v are slices of one packed projection
        qkv = normal(tokens, (hq + 2 * hk) * d)
        st["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        st["k"] = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        st["v"] = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
        st["q_out"] = torch.empty(tokens, hq, d, dtype=dt, device=dev)
        # text and audio positions: row t runs on, rows h and w wrap around
        base = torch.cat([torch.arange(p, p + n) for n, p in zip(new, past)]).to(torch.int32)
        st["pos"] = torch.stack([base, base % 97, base % 61]).contiguous().to(dev)
        st["gamma_q"] = (1 + 0.1 * normal(d).float()).to(dt) if case["norm"] else None
        st["gamma_k"] = (1 + 0.1 * normal(d).float()).to(dt) if case["norm"] else None
        return st
    st["q"] = normal(tokens, hq, d, std=2.0)
    st["out"] = torch.zeros(tokens, hq, d, dtype=dt, device=dev)
    st["slopes"] = (torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32).to(dev)
                    if case["slopes"] else None)
    st["bidir"] = (torch.full((len(new),), case["bidir"], dtype=torch.int32, device=dev)
                   if case.get("bidir") else None)
    if own:
        import swiglu_ar_tts_b200 as ops

        st["workspace"] = ops.attention_prepare(torch.empty(
            ops.attention_workspace(tokens, hq, d), dtype=torch.uint8, device=dev))
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    if op == "append":
        return _plain_append(state)
    if op == "attend":
        return _plain_attend(state)
    return _plain_shared(state)


def _own(op, st):
    import swiglu_ar_tts_b200 as ops

    case = st["case"]
    if op == "append":
        ops.mrope_paged_append(st["q"], st["k"], st["v"], st["pos"], st["q_start"], st["kv_lens"],
                               st["block_table"], st["k_pages"], st["v_pages"],
                               sections=_sections(case["d"]), theta=THETA, gamma_q=st["gamma_q"],
                               gamma_k=st["gamma_k"], eps=EPS, q_out=st["q_out"])
        return st["q_out"], st["k_pages"], st["v_pages"]
    if op == "attend":
        return ops.paged_attention(st["q"], st["k_pages"], st["v_pages"], st["q_start"], st["kv_lens"],
                                   st["block_table"], softcap=case["cap"], window=case["window"],
                                   slopes=st["slopes"], bidir_lens=st["bidir"],
                                   workspace=st["workspace"], out=st["out"])
    return ops.shared_prefix_attention(st["q"], st["k_pages"], st["v_pages"], st["group_start"],
                                       st["prefix_lens"], st["prefix_table"], st["kv_lens"],
                                       st["block_table"], softcap=case["cap"], window=case["window"],
                                       slopes=st["slopes"], workspace=st["workspace"], out=st["out"])


def _plain_append(st):
    case = st["case"]
    d, page = case["d"], case["page"]
    q, k, v, pos = st["q"], st["k"], st["v"], st["pos"]
    dt = q.dtype
    starts, lens = st["q_start"].long(), st["kv_lens"].long()
    tokens = q.shape[0]
    t = torch.arange(tokens, device=q.device)
    seq = torch.searchsorted(starts, t, right=True) - 1
    at = lens[seq] - (starts[seq + 1] - t)
    where = st["block_table"].long()[seq, at // page]
    half = d // 2
    j = torch.arange(half, device=q.device)
    s0, s1, _ = _sections(d)
    row = (j >= s0).long() + (j >= s0 + s1).long()
    angle = pos.double()[row, :].t() * (THETA ** (-2.0 * j.double() / d))  # [tokens, half]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def rotate(x, gamma):
        x = x.float()
        if gamma is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(dt)

    st["q_out"].copy_(rotate(q, st["gamma_q"]))
    st["k_pages"][where, :, at % page] = rotate(k, st["gamma_k"])
    st["v_pages"][where, :, at % page] = v
    return st["q_out"], st["k_pages"], st["v_pages"]


def _gather(pages, table_row, length, page):
    """Positions 0..length of one sequence, in 32 bits: [hk, length, d]."""
    n = -(-length // page)
    x = pages[table_row[:n].long()].transpose(0, 1)
    return x.reshape(x.shape[0], n * page, x.shape[3])[:, :length].float()


def _scores(case, st, q, k, qpos, kpos, length, bidir):
    """Scores in 32 bits with everything unseen at -inf: q [hq, n, d] at
    positions qpos against k [hk, m, d] at positions kpos."""
    hq, hk = case["hq"], case["hk"]
    n = q.shape[1]
    s = q.reshape(hk, (hq // hk) * n, -1) @ k.transpose(1, 2)
    s = s.reshape(hq, n, -1) * (1.0 / math.sqrt(case["d"]))
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    gap = qpos[:, None] - kpos[None, :]
    if st["slopes"] is not None:
        s = s - st["slopes"][:, None, None] * gap.abs().float()
    seen = (kpos[None, :] < length) & ((gap >= 0) | (kpos[None, :] < bidir))
    if case["window"]:
        seen = seen & (gap < case["window"])
    return s.masked_fill(~seen, -math.inf)


def _softmax(s):
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _plain_attend(st):
    case = st["case"]
    hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
    out, at = st["out"], 0
    for s, (new, length) in enumerate(zip(st["host_new"], st["host_lens"])):
        k = _gather(st["k_pages"], st["block_table"][s], length, page)
        v = _gather(st["v_pages"], st["block_table"][s], length, page)
        kpos = torch.arange(length, device=out.device)
        step = max(1, (1 << 28) // (hq * max(1, length)))
        for r in range(0, new, step):
            n = min(step, new - r)
            q = st["q"][at + r:at + r + n].float().transpose(0, 1)
            qpos = length - new + r + torch.arange(n, device=out.device)
            p = _softmax(_scores(case, st, q, k, qpos, kpos, length, case["bidir"]))
            o = p.reshape(hk, (hq // hk) * n, length) @ v
            out[at + r:at + r + n] = o.reshape(hq, n, d).transpose(0, 1).to(out.dtype)
        at += new
    return out


def _plain_shared(st):
    case = st["case"]
    hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
    g = hq // hk
    out, s = st["out"], 0
    for gr, (members, prefix) in enumerate(zip(st["host_members"], st["host_prefix"])):
        k0 = _gather(st["k_pages"], st["prefix_table"][gr], prefix, page)
        v0 = _gather(st["v_pages"], st["prefix_table"][gr], prefix, page)
        kpos0 = torch.arange(prefix, device=out.device)
        lens = st["host_lens"][s:s + members]
        qpos = prefix - 1 + st["kv_lens"][s:s + members].long()
        q = st["q"][s:s + members].float().transpose(0, 1)
        shared = _scores(case, st, q, k0, qpos, kpos0, prefix, 0)  # [hq, members, prefix]
        for i, length in enumerate(lens):
            k = _gather(st["k_pages"], st["block_table"][s + i], length, page)
            v = _gather(st["v_pages"], st["block_table"][s + i], length, page)
            kpos = prefix + torch.arange(length, device=out.device)
            rest = _scores(case, st, q[:, i:i + 1], k, qpos[i:i + 1], kpos, prefix + length, 0)
            p = _softmax(torch.cat([shared[:, i:i + 1], rest], -1))
            p = p.reshape(hk, g, prefix + length)
            o = p[..., :prefix] @ v0 + p[..., prefix:] @ v
            out[s + i] = o.reshape(hq, d).to(out.dtype)
        s += members
    return out


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] != "append" and work(case)["flops"] > 6e12:
        return None
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    return _exact_attention(st)


def _exact_append(st):
    case = st["case"]
    d, page = case["d"], case["page"]
    s0, s1, s2 = _sections(d)
    rows = torch.tensor([0] * s0 + [1] * s1 + [2] * s2, device="cuda")
    freq = torch.tensor([math.exp(-2.0 * i / d * math.log(THETA)) for i in range(d // 2)],
                        dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                       st["pos"].double().index_select(0, rows).mul(freq[:, None])).t()  # [tokens, d/2]

    def rotated(x, gamma):
        x = x.double()
        if gamma is not None:
            x = x * gamma.double() * ((x.square().sum(-1, keepdim=True) / d) + EPS).rsqrt()
        z = torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous()) * turn[:, None]
        return torch.cat([z.real, z.imag], -1)

    q, k, v = rotated(st["q"], st["gamma_q"]), rotated(st["k"], st["gamma_k"]), st["v"].double()
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    table, t = st["block_table"].tolist(), 0
    for s, (new, length) in enumerate(zip(st["host_new"], st["host_lens"])):
        for first in range(length - new, length):
            if first % page and first != length - new:
                continue
            last = min(length, (first // page + 1) * page)
            pg, a, b = table[s][first // page], first % page, (last - 1) % page + 1
            kp[pg, :, a:b] = k[t:t + last - first].transpose(0, 1)
            vp[pg, :, a:b] = v[t:t + last - first].transpose(0, 1)
            t += last - first
    return q, kp, vp


def _exact_attention(st):
    """Head by head over one list of (page, slot) a sequence, whatever the
    operator: a shared prompt's positions come first in its members' lists."""
    case = st["case"]
    hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    table = st["block_table"].long()
    at, group, left = 0, -1, 0
    prompt = None
    for s, new in enumerate(st["host_new"]):
        pos = torch.arange(st["host_lens"][s], device="cuda")
        slots = table[s, pos // page] * page + pos % page
        if case["op"] == "shared":
            while left == 0:
                group += 1
                left = st["host_members"][group]
                ppos = torch.arange(st["host_prefix"][group], device="cuda")
                prompt = st["prefix_table"].long()[group, ppos // page] * page + ppos % page
            left -= 1
            slots = torch.cat([prompt, slots])
        length = slots.numel()
        if length == 0:
            at += new
            continue
        rows = torch.arange(length - new, length, device="cuda").double()[:, None]
        cols = torch.arange(length, device="cuda").double()[None, :]
        pg, sl = slots // page, slots % page
        step = max(1, (1 << 27) // length)
        for h in range(hk):
            kh, vh = st["k_pages"][pg, h, sl].double(), st["v_pages"][pg, h, sl].double()
            for head in range(h * (hq // hk), (h + 1) * (hq // hk)):
                for r in range(0, new, step):
                    n = min(step, new - r)
                    w = torch.einsum("id,jd->ij", st["q"][at + r:at + r + n, head].double(), kh) / math.sqrt(d)
                    i = rows[r:r + n]
                    if case["cap"]:
                        w = torch.tanh(w / case["cap"]) * case["cap"]
                    if st["slopes"] is not None:
                        w = w - float(st["slopes"][head]) * (i - cols).abs()
                    hidden = (cols > i) & (cols >= case.get("bidir", 0))
                    if case["window"]:
                        hidden = hidden | (cols <= i - case["window"])
                    w[hidden] = -math.inf
                    w = w - w.max(1, keepdim=True).values.clamp(min=-1e300)
                    w = w.exp_()
                    norm = w.sum(1, keepdim=True)
                    norm[norm == 0] = 1.0
                    out[at + r:at + r + n, head] = (w @ vh) / norm
        at += new
    return out
