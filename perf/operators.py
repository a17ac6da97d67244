"""Performance cases of the operators around a cached, rotated attention: the rotary
positions of queries and keys with their per-head norms, the page plan of a key-value
cache, and attention of one new token over that cache.

Every case runs in a plain form (elementary torch operations, 32-bit arithmetic, 64-bit
angles) or, with ``own`` set, through the calls of ``ffn_long_video_b200``.

Kinds of cases:

``rope``    queries and keys of a prompt: per-head RMSNorm (optional) and rotation
``append``  the same for the new tokens of a decoding step, the rotated keys and the values
            written into a paged cache
``grad``    the gradient of ``rope``
``plan``    a step's slots, positions and block tables from the sequences' lengths, and the
            step that takes it back
``decode``  attention of one new token per sequence over the paged cache
"""
import math

import torch

own = False

EPS = 1e-6
MAGNITUDE = 1.25   # factor of the rotated part (long-context scaling of the positions)
BASE = 1.0e6       # rotary base


# ------------------------------------------------------------------------------- cases
def listed():
    def rope(name, kind, **kw):
        c = dict(name=name, kind=kind, dtype="bf16", tokens=1, hq=28, hkv=4, d=128, rot=128,
                 interleaved=False, norm=False, axes=1)
        return dict(c, **kw)

    def decode(name, **kw):
        c = dict(name=name, kind="decode", dtype="bf16", seqs=1, lo=1, hi=1, page=16, hq=28,
                 hkv=4, d=128, heads_outer=False)
        return dict(c, **kw)

    return [
        # the 64K-token layer's prompt: video tokens in cube order with three position axes
        rope("rope 64K video", "rope", tokens=65792, axes=3),
        # a 3B-width layer with normalised heads, text positions, an odd token count
        rope("rope 18K norm", "rope", tokens=18559, hq=16, hkv=2, norm=True),
        # one sequence decoding: latency alone
        rope("append 1", "append", norm=True),
        # a batch of decoding sequences, part of the head rotated
        rope("append 200 part", "append", tokens=200, hq=16, hkv=2, rot=64, interleaved=True),
        # fine-tuning: gradient at the 18K layer, norms' weights included
        rope("grad 18K norm", "grad", tokens=18560, hq=16, hkv=2, norm=True),
        # fp32, small heads, interleaved pairs, part of the head, no norm
        rope("grad 5K fp32", "grad", dtype="fp32", tokens=4999, hq=4, hkv=1, d=64, rot=32,
             interleaved=True),
        # a decoding step of 64 sequences: a token or a few drafted ones for each
        dict(name="plan 64 step", kind="plan", seqs=64, page=16, hi=32768, grow=4, turnover=0),
        # admission and release: prompts enter where finished sequences leave
        dict(name="plan 300 turnover", kind="plan", seqs=300, page=64, hi=16384, grow=8,
             turnover=3),
        # one short sequence: latency alone
        decode("decode 1x500", hi=500),
        # one long video: 64K tokens of one sequence over the whole GPU
        decode("decode 1x65793", hi=65793, page=64),
        # a ragged batch, pages of 16, one KV head's pages side by side
        decode("decode 61 ragged", seqs=61, lo=0, hi=9001, hq=16, hkv=2, heads_outer=True),
        # a full batch of long sequences in fp32: the largest
        decode("decode 24x30K fp32", dtype="fp32", seqs=24, lo=20000, hi=30001, page=128),
    ]


_HEADS = ((4, 1), (8, 2), (16, 2), (28, 4), (6, 3), (4, 4), (16, 1), (12, 1))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("rope", "append", "grad", "plan", "decode", "decode"))
    hq, hkv = rng.choice(_HEADS)
    d = rng.choice((64, 128))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if kind == "plan":
        seqs = _log(rng, 1, 1000)
        return dict(kind=kind, seqs=seqs, page=rng.choice((1, 16, 48, 64, 256)),
                    hi=_log(rng, 16, min(65536, 4_800_000 // seqs)), grow=_log(rng, 1, 64),
                    turnover=rng.choice((0, 0, 2, 5)))
    if kind == "decode":
        seqs = _log(rng, 1, 256)
        hi = _log(rng, 1, min(131072, 600_000 // seqs))
        return dict(kind=kind, dtype=dtype, seqs=seqs, lo=rng.choice((0, 1, hi // 2, hi)), hi=hi,
                    page=rng.choice((1, 16, 23, 64, 256)), hq=hq, hkv=hkv, d=d,
                    heads_outer=rng.random() < 0.5)
    top = {"rope": 40000, "append": 2000, "grad": 20000}[kind]
    axes = rng.choice((1, 3)) if kind != "append" else 1
    rot = rng.choice((d, d, d // 2, 32))
    return dict(kind=kind, dtype=dtype, tokens=_log(rng, 1, top), hq=hq, hkv=hkv, d=d, rot=rot,
                interleaved=rng.random() < 0.5, norm=rng.random() < 0.5, axes=axes)


# ------------------------------------------------------------------------------ inputs
def _lengths(c):
    """Lengths spread over lo..hi, the same for every seed: the work follows the case."""
    span = c["hi"] - c["lo"] + 1
    n = [c["lo"] + int(span * math.modf((i + 1) * 0.6180339887498949)[0]) for i in range(c["seqs"])]
    n[-1] = c["hi"]
    return n


def _steps(c):
    """Lengths before and after a plan step: most sequences gain a few tokens; with a
    turnover of k every k-th one is finished, and the one after it enters with its prompt."""
    old, new = [], []
    for i, n in enumerate(_lengths(dict(c, lo=1))):
        k = c["turnover"]
        if k and i % k == 0:
            old.append(n), new.append(0)
        elif k and i % k == 1:
            old.append(0), new.append(n)
        else:
            old.append(n), new.append(n + 1 + i % c["grow"])
    return old, new


def _pages(n, page):
    return -(-n // page)


def _sections(c):
    """Pairs per position axis: a quarter in time, the rest over height and width."""
    h = c["rot"] // 2
    return (h // 4, (h - h // 4) // 2, h - h // 4 - (h - h // 4) // 2)


def _positions(c, dev, g):
    n = c["tokens"]
    if c["axes"] == 1:
        if c["kind"] == "append":   # sequences of any length, far ones among them
            return torch.randint(0, 1 << 20, (n,), generator=g, device=dev, dtype=torch.int32)
        start = torch.randint(0, 4096, (1,), generator=g, device=dev, dtype=torch.int32)
        return torch.arange(n, device=dev, dtype=torch.int32) + start
    # cube-major video tokens: 4x4x4 cubes of a 32x32 grid, then text tokens
    n_vis = n // 64 * 64
    i = torch.arange(n, device=dev)
    cube, r = i // 64, i % 64
    t = cube // 64 * 4 + r // 16
    h = cube // 8 % 8 * 4 + r // 4 % 4
    w = cube % 8 * 4 + r % 4
    text = torch.clamp(t[n_vis - 1] if n_vis else t[0] * 0, min=31) + 1 + i - n_vis
    pos = torch.where(i < n_vis, torch.stack((t, h, w)), text)
    shift = torch.randint(0, 64, (1,), generator=g, device=dev)
    return (pos + shift).to(torch.int32)


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def rand(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if c["kind"] == "plan":
        old, new = _steps(c)
        cols = _pages(max(old + new), c["page"])
        held = [_pages(n, c["page"]) for n in old]
        n_pages = sum(max(_pages(n, c["page"]), m) for n, m in zip(new, held)) + 7
        ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        po = ints(held)
        first = torch.cumsum(po, 0) - po
        j = torch.arange(cols, device=dev)
        at = torch.clamp(first[:, None] + j, max=n_pages - 1)
        table = torch.where(j < po[:, None], ids[at], -1).to(torch.int32).contiguous()
        free = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
        n_free = n_pages - sum(held)
        free[:n_free] = ids[sum(held):]
        rows = [sum(max(b - a, 0) for a, b in zip(x, y)) for x, y in ((old, new), (new, old))]
        return dict(c=c, old=ints(old), new=ints(new), table=table, free=free,
                    n_free=ints([n_free]), rows=max(1, rows[0]), back=max(1, rows[1]))

    dt = _dtype(c)
    if c["kind"] == "decode":
        n = _lengths(c)
        cols = max(1, _pages(max(n), c["page"]))
        held = [_pages(x, c["page"]) for x in n]
        n_pages = sum(held) + 3
        ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        po = ints(held)
        first = torch.cumsum(po, 0) - po
        j = torch.arange(cols, device=dev)
        at = torch.clamp(first[:, None] + j, max=n_pages - 1)
        table = torch.where(j < po[:, None], ids[at], -1).to(torch.int32).contiguous()
        shape = (n_pages, c["hkv"], c["page"], c["d"]) if c["heads_outer"] else \
            (n_pages, c["page"], c["hkv"], c["d"])
        k, v = rand(*shape, dtype=dt), rand(*shape, dtype=dt)
        if c["heads_outer"]:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        return dict(c=c, q=rand(c["seqs"], c["hq"], c["d"], dtype=dt), k=k, v=v, table=table,
                    lens=ints(n))

    n, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["d"]
    qkv = rand(n, (hq + 2 * hkv) * d, dtype=dt)   # one fused projection: Q, K, V are its parts
    s = dict(c=c, Q=qkv[:, :hq * d].view(n, hq, d),
             K=qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d),
             V=qkv[:, (hq + hkv) * d:].view(n, hkv, d), pos=_positions(c, dev, g))
    s["freq"] = BASE ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
    s["sections"] = _sections(c) if c["axes"] == 3 else None
    s["axis"] = torch.tensor([a for a in range(3) for _ in range(_sections(c)[a])], device=dev)
    s["wq"] = (1 + 0.2 * rand(d)).to(dt) if c["norm"] else None
    s["wk"] = (1 + 0.2 * rand(d)).to(dt) if c["norm"] else None
    if c["kind"] == "grad":   # gradients as the attention's backward pass gives them
        s["dq"], s["dk"] = rand(n, hq, d), rand(n, hkv, d)
    if c["kind"] == "append":
        pages = _pages(2 * n, 16) + 1
        # a page more than the cache has: where the plain form puts what is not to be kept
        s["k_all"], s["v_all"] = (rand(pages + 1, 16, hkv, d, dtype=dt) for _ in range(2))
        slots = torch.randperm(pages * 16, generator=g, device=dev)[:n].to(torch.int32)
        pad = torch.arange(n, device=dev) >= max(1, n - n // 16)   # rows that pad the batch
        s["slots"] = torch.where(pad, -1, slots).to(torch.int32)
        s["k_cache"], s["v_cache"] = s["k_all"][:pages], s["v_all"][:pages]
    return s


# ---------------------------------------------------------------------------- one pass
def run(state):
    c = state["c"]
    if own:
        return _own(state, c)
    return {"rope": _rope, "append": _append, "grad": _grad, "plan": _plan,
            "decode": _decode}[c["kind"]](state, c)


def _own(s, c):
    import ffn_long_video_b200 as fb
    if c["kind"] == "plan":
        slots, pos, start, _ = fb.kv_plan(s["old"], s["new"], s["table"], s["free"], s["n_free"],
                                          c["page"], s["rows"])
        slots2, pos2, start2, _ = fb.kv_plan(s["new"], s["old"], s["table"], s["free"],
                                             s["n_free"], c["page"], s["back"])
        return (slots, pos, start, slots2, pos2, start2, s["table"], s["free"], s["n_free"])
    if c["kind"] == "decode":
        out, lse, _ = fb.decode_attn(s["q"], s["k"], s["v"], s["table"], s["lens"])
        return out, lse
    kw = dict(w_q=s["wq"], w_k=s["wk"], eps=EPS, interleaved=c["interleaved"],
              sections=s["sections"], magnitude=MAGNITUDE)
    if c["kind"] == "rope":
        return fb.qk_rope(s["Q"], s["K"], s["pos"], s["freq"], **kw)
    if c["kind"] == "append":
        q = fb.qk_rope_append(s["Q"], s["K"], s["V"], s["pos"], s["freq"], s["slots"],
                              s["k_cache"], s["v_cache"], **kw)
        return q, s["k_cache"], s["v_cache"]
    dq, dk, dwq, dwk, _ = fb.qk_rope_backward(s["dq"], s["dk"], s["pos"], s["freq"], Q=s["Q"],
                                              K=s["K"], **kw)
    return (dq, dk, dwq, dwk) if c["norm"] else (dq, dk)


# ------------------------------------------------------------------------- plain forms
def _cos_sin(s, c):
    """cos and sin of every token's pairs, times the magnitude: [tokens, 1, rot/2]."""
    if c["axes"] == 3:
        at = s["pos"][s["axis"]].t()
    else:
        at = s["pos"][:, None]
    angle = at.double() * s["freq"]
    return (torch.cos(angle) * MAGNITUDE).float()[:, None], \
        (torch.sin(angle) * MAGNITUDE).float()[:, None]


def _turn(x, c, cos, sin):
    """The rotation of the first rot elements of each head (fp32)."""
    rot = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1) if rot < c["d"] else y


def _inverse_rms(x):
    return 1.0 / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + EPS)


def _head(x, w, c, cos, sin):
    x = x.float()
    if w is not None:
        x = x * _inverse_rms(x) * w.float()
    return _turn(x, c, cos, sin)


def _rope(s, c):
    cos, sin = _cos_sin(s, c)
    return _head(s["Q"], s["wq"], c, cos, sin).to(s["Q"].dtype), \
        _head(s["K"], s["wk"], c, cos, sin).to(s["K"].dtype)


def _append(s, c):
    q, k = _rope(s, c)
    spare = s["k_cache"].shape[0] * s["k_cache"].shape[1]
    at = torch.where(s["slots"] >= 0, s["slots"], spare).long()
    s["k_all"].view(-1, c["hkv"], c["d"])[at] = k
    s["v_all"].view(-1, c["hkv"], c["d"])[at] = s["V"]
    return q, s["k_cache"], s["v_cache"]


def _grad_head(dy, x, w, c, cos, sin):
    g = _turn(dy.float(), c, cos, -sin)
    if w is None:
        return g, None
    x = x.float()
    r = _inverse_rms(x)
    xhat = x * r
    dw = (g * xhat).sum(dim=(0, 1))
    g = g * w.float()
    return r * (g - xhat * (g * xhat).mean(dim=-1, keepdim=True)), dw


def _grad(s, c):
    cos, sin = _cos_sin(s, c)
    dq, dwq = _grad_head(s["dq"], s["Q"], s["wq"], c, cos, sin)
    dk, dwk = _grad_head(s["dk"], s["K"], s["wk"], c, cos, sin)
    return (dq, dk, dwq, dwk) if c["norm"] else (dq, dk)


def _plan_step(old, new, table, free, n_free, page, rows):
    """One step: pages that shrinking sequences give back go onto the free list, growing ones
    take theirs from its end; then the slot and the position of every new token."""
    dev = old.device
    po, pn = (old + page - 1) // page, (new + page - 1) // page
    give, take = torch.clamp(po - pn, min=0), torch.clamp(pn - po, min=0)
    g0, t0 = torch.cumsum(give, 0) - give, torch.cumsum(take, 0) - take
    F, R, T = n_free.long(), give.sum(), take.sum()
    j = torch.arange(table.shape[1], device=dev)[None]
    given, taken = (j >= pn[:, None]) & (j < po[:, None]), (j >= po[:, None]) & (j < pn[:, None])
    stack = torch.cat((free, torch.zeros(1, dtype=torch.int32, device=dev)))
    spare = free.shape[0]
    at = torch.where(given, F + R - 1 - (g0[:, None] + j - pn[:, None]), spare)
    stack[at.reshape(-1)] = table.reshape(-1)
    at = torch.where(taken, F + R - 1 - (t0[:, None] + j - po[:, None]), spare)
    table.copy_(torch.where(taken, stack[at], table))
    left = F + R - T
    free.copy_(torch.where(torch.arange(spare, device=dev) < left, stack[:spare], free))
    n_free.copy_(left)
    more = torch.clamp(new - old, min=0)
    start = torch.cat((torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(more, 0)))
    r = torch.arange(rows, device=dev)
    seq = torch.clamp(torch.searchsorted(start, r, right=True) - 1, max=old.shape[0] - 1)
    pos = old[seq] + (r - start[seq])
    real = r < start[-1]
    pos = torch.where(real, pos, 0)
    slot = table[seq, torch.clamp(pos // page, max=table.shape[1] - 1)] * page + pos % page
    return torch.where(real, slot, -1).to(torch.int32), pos.to(torch.int32), start.to(torch.int32)


def _plan(s, c):
    args = (s["table"], s["free"], s["n_free"], c["page"])
    a = _plan_step(s["old"], s["new"], *args, s["rows"])
    b = _plan_step(s["new"], s["old"], *args, s["back"])
    return (*a, *b, s["table"], s["free"], s["n_free"])


def _decode(s, c):
    n, hkv, d, page = c["seqs"], c["hkv"], c["d"], c["page"]
    at = torch.clamp(s["table"], min=0).long()
    L = at.shape[1] * page
    k = s["k"][at].reshape(n, L, hkv, d).float().permute(0, 2, 3, 1)
    v = s["v"][at].reshape(n, L, hkv, d).float().transpose(1, 2)
    q = s["q"].float().view(n, hkv, c["hq"] // hkv, d)
    there = (torch.arange(L, device=at.device) < s["lens"][:, None])[:, None, None]
    z = torch.matmul(q * d ** -0.5, k).masked_fill(~there, float("-inf"))
    top = torch.clamp(z.amax(dim=-1, keepdim=True), min=torch.finfo(torch.float32).min)
    e = torch.exp(z - top)
    total = e.sum(dim=-1, keepdim=True)
    o = torch.matmul(e, torch.where(there.transpose(-1, -2), v, 0.0))
    o = torch.where(total > 0, o / total, 0.0).view(n, c["hq"], d).to(s["q"].dtype)
    lse = torch.where(total > 0, top + torch.log(total), float("-inf"))
    return o, lse.view(n, c["hq"])


# ----------------------------------------------------------------------- what it takes
def work(case):
    c = case
    if c["kind"] == "plan":
        old, new = _steps(c)
        rows = sum(abs(a - b) for a, b in zip(old, new))
        moved = sum(abs(_pages(a, c["page"]) - _pages(b, c["page"])) for a, b in zip(old, new))
        # both calls: lengths in, starts out; a slot and a position for each new token; a table
        # entry read or written and a list entry written or read for each page that moves
        return {"bytes": 2 * (12 * c["seqs"] + 4) + 8 * rows + 2 * 8 * moved, "flops": 0}
    es = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] == "decode":
        keys = sum(_lengths(c))
        return {"bytes": 2 * keys * c["hkv"] * c["d"] * es + 2 * c["seqs"] * c["hq"] * c["d"] * es
                + 4 * c["seqs"] * c["hq"] + 4 * sum(_pages(x, c["page"]) for x in _lengths(c)),
                "flops": 4 * keys * c["hq"] * c["d"]}
    n, d, heads = c["tokens"], c["d"], c["hq"] + c["hkv"]
    flops = n * heads * (3 * c["rot"] + (4 * d if c["norm"] else 0))
    move = 2 * es * n * heads * d
    if c["kind"] == "append":
        move += 2 * es * n * c["hkv"] * d + 4 * n
    if c["kind"] == "grad":
        move = (8 + (es if c["norm"] else 0)) * n * heads * d
        flops *= 2
    return {"bytes": move + 4 * c["axes"] * n, "flops": flops}


# ----------------------------------------------------------------- the definitions, 64 bit
def exact(case, seed):
    c = case
    if c["kind"] == "plan":
        return None      # whole numbers
    s = prepare(c, seed)
    if c["kind"] == "decode":
        # softmax over each sequence's own keys, a sequence and a KV head at a time
        outs, lses = [], []
        for b, n in enumerate(_lengths(c)):
            pages = s["table"][b, :_pages(n, c["page"])].long()
            k = s["k"][pages].double().reshape(-1, c["hkv"], c["d"])[:n]
            v = s["v"][pages].double().reshape(-1, c["hkv"], c["d"])[:n]
            q = s["q"][b].double().reshape(c["hkv"], -1, c["d"])
            z = torch.einsum("hgd,nhd->hgn", q, k) / math.sqrt(c["d"])
            p = torch.softmax(z, dim=-1) if n else z
            outs.append(torch.einsum("hgn,nhd->hgd", p, v).reshape(c["hq"], c["d"]))
            lses.append(torch.logsumexp(z, dim=-1).reshape(c["hq"]))
        return torch.stack(outs), torch.stack(lses)
    # each rotated pair as a complex number times the unit number of its angle
    n, rot, half = c["tokens"], c["rot"], c["rot"] // 2
    first = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else half)
    pos = s["pos"].double().view(c["axes"], n)
    if c["axes"] == 3:
        a, b, _ = s["sections"]
        pair = torch.arange(half, device="cuda")
        pos = pos[(pair >= a).long() + (pair >= a + b).long()].T
    else:
        pos = pos[0][:, None].expand(n, half)
    unit = torch.polar(torch.full((n, half), MAGNITUDE, dtype=torch.float64, device="cuda"),
                       pos * s["freq"])[:, None]

    def turned(x, u):
        z = torch.complex(x[..., first], x[..., second]) * u
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def normed(x, w):
        if w is None:
            return x
        ms = torch.linalg.vector_norm(x, dim=-1, keepdim=True).square() / c["d"]
        return x / torch.sqrt(ms + EPS) * w

    Q, K = s["Q"].double(), s["K"].double()
    wq, wk = (None if w is None else w.double() for w in (s["wq"], s["wk"]))
    if c["kind"] != "grad":
        q, k = turned(normed(Q, wq), unit), turned(normed(K, wk), unit)
        if c["kind"] == "rope":
            return q, k
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        keep = s["slots"] >= 0
        at = s["slots"][keep].long()
        kc[at // 16, at % 16], vc[at // 16, at % 16] = k[keep], s["V"].double()[keep]
        return q, kc, vc
    # the gradient by differentiating the definition
    leaves = [x.requires_grad_() for x in (Q, K, wq, wk) if x is not None]
    y = (turned(normed(Q, wq), unit), turned(normed(K, wk), unit))
    return torch.autograd.grad(y, leaves, (s["dq"].double(), s["dk"].double()))
