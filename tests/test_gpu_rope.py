"""Rotary positions with per-head norms, into outputs and into the paged cache,
and their gradient, against the float64 statement (needs a B200).

Tolerances, with u = 2^-24 (half a step of fp32) and R the length of an
element's rotated pair after the norm (its own magnitude where nothing turns):
the turn is rounded once (pi u on the angle, 1.6 u after its range), sine and
cosine have 2 ulp (2 u), the magnitude 1 u, the norm's sum of 16 products and 3
exchanges 19 u, halved by the root, its inverse root 2 ulp (4 u), two products
2 u, rotation two products and a sum 3 u: 24 u on each of two terms, 34 u R
together.  An output rounded to its type adds half a step, eps / 2 relative."""
import numpy as np
import pytest
import torch

import ffn_long_video_b200 as fb
from oracle import generation_ref as gen

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


def _f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def _rand(g, *shape, dtype=FP32, scale=1.0):
    return (scale * torch.randn(shape, generator=g)).to(dtype).cuda()


def _radius(x, rot, il):
    """Length of each element's pair."""
    r = np.abs(x).copy()
    f, s = gen.rope_pairs(x.shape[-1], rot, il)
    r[..., f] = r[..., s] = np.hypot(x[..., f], x[..., s])
    return r


def _close(got, want, bound, what):
    d = np.abs(_f64(got) - want)
    assert np.all(d <= bound), (what, float((d - bound).max()), float((d / np.maximum(bound, 1e-300)).max()))


def _inputs(n, hq, hkv, d, dtype, layout, seed=7, scale=1.0):
    """Q, K, V as the parts of one projection, as dense tensors, or heads outermost."""
    g = torch.Generator().manual_seed(seed)
    if layout == "fused":
        x = _rand(g, n, (hq + 2 * hkv) * d, dtype=dtype, scale=scale)
        q, k, v = x.split([hq * d, hkv * d, hkv * d], dim=1)
        return q.view(n, hq, d), k.view(n, hkv, d), v.view(n, hkv, d)
    if layout == "heads":
        return tuple(_rand(g, h, n, d, dtype=dtype, scale=scale).transpose(0, 1)
                     for h in (hq, hkv, hkv))
    return tuple(_rand(g, n, h, d, dtype=dtype, scale=scale) for h in (hq, hkv, hkv))


def _positions(n, axes, seed=3, far=False):
    r = np.random.default_rng(seed)
    hi = 2 ** 31 if far else 5000
    p = r.integers(-hi, hi, (axes, n) if axes == 3 else n).astype(np.int32)
    p.flat[0] = 0
    return p


def _sections(rot, axes):
    h = rot // 2
    return (h // 4, h // 2 - h // 4, h - h // 2) if axes == 3 else None


# n, hq, hkv, d, dtype, rot, interleaved, norm, axes, layout
CASES = [
    (1, 28, 4, 128, BF16, 128, False, "qk", 1, "fused"),
    (37, 28, 4, 128, BF16, 128, False, "qk", 3, "fused"),
    (300, 16, 2, 128, BF16, 128, False, None, 3, "dense"),
    (65, 6, 3, 128, FP32, 64, True, "qk", 1, "heads"),
    (129, 4, 1, 64, FP32, 64, False, None, 1, "fused"),
    (33, 8, 2, 64, BF16, 32, True, "q", 3, "dense"),
    (18, 5, 5, 64, BF16, 16, False, "k", 1, "heads"),
    (7, 1, 1, 128, FP32, 112, True, "qk", 1, "dense"),
    (7, 1, 1, 128, FP32, 112, False, "qk", 1, "dense"),
    (50, 16, 1, 128, BF16, 0, False, "qk", 1, "fused"),
    (2500, 7, 7, 64, FP32, 64, True, "qk", 1, "dense"),
    (5001, 12, 2, 128, BF16, 96, False, "qk", 3, "fused"),
    (4300, 5, 5, 128, BF16, 128, True, "k", 1, "heads"),
    (3700, 3, 1, 64, FP32, 64, False, None, 3, "fused"),
]


def _case(c, far=False, seed=7):
    n, hq, hkv, d, dtype, rot, il, norm, axes, layout = c
    Q, K, V = _inputs(n, hq, hkv, d, dtype, layout, seed)
    g = torch.Generator().manual_seed(seed + 1)
    wq = (1 + _rand(g, d, scale=0.3)).to(dtype) if norm in ("qk", "q") else None
    wk = (1 + _rand(g, d, scale=0.3)).to(dtype) if norm in ("qk", "k") else None
    pos = _positions(n, axes, far=far)
    freq = 1e6 ** (-np.arange(0, rot, 2) / rot) if rot else None
    sec = _sections(rot, axes) if rot else None
    kw = dict(w_q=wq, w_k=wk, eps=1e-5, interleaved=il, sections=sec, magnitude=1.3)
    args = (torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda()) if rot else (None, None)
    ang = gen.rope_angles(pos, freq, sec) if rot else np.zeros((n, 0))
    return Q, K, V, wq, wk, args, kw, ang


def _expected(x, w, ang, c):
    """(value, bound) of the rotated heads of x."""
    rot, il = c[5], c[6]
    x = _f64(x)
    w = None if w is None else _f64(w)
    want = gen.qk_rope(x, ang, rot, il, w, 1e-5, 1.3)
    nx = gen.head_norm(x, w, 1e-5)[0]
    R = _radius(nx, rot, il)
    R[..., :rot] *= 1.3
    eps = torch.finfo(c[4]).eps / 2
    return want, eps * np.abs(want) + 34 * U * R * (1 + eps)


@pytest.mark.parametrize("c", CASES, ids=str)
def test_forward(c):
    Q, K, _, wq, wk, args, kw, ang = _case(c)
    q, k = fb.qk_rope(Q, K, *args, **kw)
    _close(q, *_expected(Q, wq, ang, c), "q")
    _close(k, *_expected(K, wk, ang, c), "k")
    # the same bits again, into given outputs with heads outside tokens
    n, hq, hkv, d = c[:4]
    oq = torch.empty(hq, n, d, dtype=c[4], device="cuda").transpose(0, 1)
    ok = torch.empty(n, hkv + 3, d, dtype=c[4], device="cuda")[:, 1:1 + hkv]
    fb.qk_rope(Q, K, *args, out_q=oq, out_k=ok, **kw)
    assert torch.equal(oq, q) and torch.equal(ok, k)


@pytest.mark.parametrize("c", [CASES[1], CASES[3], CASES[5]], ids=str)
def test_in_place(c):
    Q, K, V, _, _, args, kw, _ = _case(c)
    q, k = fb.qk_rope(Q, K, *args, **kw)
    v0 = V.clone()
    fb.qk_rope(Q, K, *args, out_q=Q, out_k=K, **kw)
    assert torch.equal(Q, q) and torch.equal(K, k) and torch.equal(V, v0)


@pytest.mark.parametrize("c", [CASES[1], CASES[4]], ids=str)
def test_far_and_negative_positions(c):
    """Positions over all of int32: a turn is reduced in 64 bits, so the bound
    grows by 2^31 radians * 2^-53 * 3 roundings = 7e-7 = 12 u alone."""
    Q, K, _, wq, wk, args, kw, ang = _case(c, far=True)
    q, k = fb.qk_rope(Q, K, *args, **kw)
    for got, x, w in ((q, Q, wq), (k, K, wk)):
        want, bound = _expected(x, w, ang, c)
        R = _radius(gen.head_norm(_f64(x), None if w is None else _f64(w), 1e-5)[0], c[5], c[6])
        # the float64 statement rounds its angles as well: twice
        _close(got, want, bound + 24 * 1.3 * U * R, "far")


def test_a_bad_row_stays_alone():
    """NaN and infinities in one head reach no other head, zeros stay zeros."""
    c = CASES[1]
    Q, K, _, wq, wk, args, kw, ang = _case(c)
    q0, k0 = fb.qk_rope(Q, K, *args, **kw)
    Q[3, 5, 9], Q[4, 6, 0], K[2, 1, 77], Q[6, 1] = float("nan"), float("inf"), float("-inf"), 0.0
    q, k = fb.qk_rope(Q, K, *args, **kw)
    keep = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    keep[3, 5] = keep[4, 6] = keep[6, 1] = False
    assert torch.equal(q[keep], q0[keep]) and torch.all(q[6, 1] == 0)
    assert torch.isnan(q[3, 5]).any() and torch.isnan(q[4, 6]).any()
    keep = torch.ones(k.shape[:2], dtype=torch.bool, device="cuda")
    keep[2, 1] = False
    assert torch.equal(k[keep], k0[keep])


@pytest.mark.parametrize("n", [3, 9000])
@pytest.mark.parametrize("il", [False, True])
def test_a_bad_element_reaches_its_pair_alone(n, il):
    """Without a norm a NaN or an infinity spoils its pair; the rest of the head,
    the part beyond the rotation too, is as without it. 9000 tokens: the walk
    over tokens, 3: a warp per step."""
    c = (n, 4, 2, 64, FP32, 32, il, None, 1, "dense")
    Q, K, _, _, _, args, kw, _ = _case(c)
    q0, k0 = fb.qk_rope(Q, K, *args, **kw)
    bad = [(0, 1, 40, float("inf")), (n - 1, 3, 63, float("nan")), (1, 0, 5, float("inf"))]
    for t, h, e, x in bad:
        Q[t, h, e] = x
        K[t, h % 2, e] = x
    q, k = fb.qk_rope(Q, K, *args, **kw)
    for got, want, heads in ((q, q0, 4), (k, k0, 2)):
        keep = torch.ones_like(got, dtype=torch.bool)
        for t, h, e, _ in bad:
            pair = ([e] if e >= 32 else [e & ~1, e | 1] if il else [e % 16, e % 16 + 16])
            keep[t, h % heads, pair] = False
        assert torch.equal(got[keep], want[keep]) and not torch.isfinite(got[~keep]).any()


# --------------------------------------------------------------------- into the cache
@pytest.mark.parametrize("heads_outer", [False, True])
@pytest.mark.parametrize("page", [1, 16, 23])
@pytest.mark.parametrize("c", [CASES[0], CASES[1], CASES[3], CASES[5], CASES[9], CASES[10],
                               CASES[11], CASES[12], CASES[13]], ids=str)
def test_append(c, page, heads_outer):
    """The outputs of qk_rope, bit for bit, at their slots; every other element
    of the cache as it was; slots outside the cache written nowhere."""
    n, hq, hkv, d, dtype = c[:5]
    Q, K, V, wq, wk, args, kw, _ = _case(c)
    q0, k0 = fb.qk_rope(Q, K, *args, **kw)
    pages = -(-(2 * n + 3) // page)
    shape = (pages, hkv, page, d) if heads_outer else (pages, page, hkv, d)
    kc, vc = (torch.full(shape, s, dtype=dtype, device="cuda") for s in (11.0, 12.0))
    kv, vv = (x.transpose(1, 2) if heads_outer else x for x in (kc, vc))
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(5))[:n]
    slots = slots.to(torch.int32).cuda()
    if n > 4:
        slots[1], slots[2], slots[4] = -1, pages * page, -2 ** 31
    q = fb.qk_rope_append(Q, K, V, *args, slots, kv, vv, **kw)
    assert torch.equal(q, q0)
    want_k, want_v = torch.full_like(kv, 11.0), torch.full_like(vv, 12.0)
    ok = (slots >= 0) & (slots < pages * page)
    s = slots[ok].long()
    want_k[s // page, s % page], want_v[s // page, s % page] = k0[ok], V[ok]
    assert torch.equal(kv, want_k) and torch.equal(vv, want_v)
    # the same tokens as they are
    kc.fill_(11.0), vc.fill_(12.0)
    fb.kv_append(k0, V, slots, kv, vv)
    assert torch.equal(kv, want_k) and torch.equal(vv, want_v)


def test_append_far_slots():
    """Cache offsets past 2^32 elements' bytes and past 2^31 elements: pages at
    the end of a cache of 2.2e9 elements each for keys and values."""
    hkv, d, page = 4, 128, 64
    pages = 2 ** 31 // (hkv * d * page) + 2000
    kc = torch.empty(pages, page, hkv, d, dtype=BF16, device="cuda")
    vc = torch.empty_like(kc)
    g = torch.Generator().manual_seed(1)
    K, V = _rand(g, 40, hkv, d, dtype=BF16), _rand(g, 40, hkv, d, dtype=BF16)
    slots = torch.arange(40, dtype=torch.int32, device="cuda") * 3 + (pages - 2) * page
    kc[-3:] = 0
    vc[-3:] = 0
    fb.kv_append(K, V, slots, kc, vc)
    s = slots.long()
    assert torch.equal(kc[s // page, s % page], K) and torch.equal(vc[s // page, s % page], V)
    assert int((kc[-3:] != 0).any(dim=-1).sum()) == 40 * hkv


@pytest.mark.parametrize("n,h,d,dtype", [(1, 1, 64, BF16), (1000, 3, 64, FP32), (513, 7, 128, BF16),
                                         (3001, 2, 128, FP32), (77, 40, 128, BF16)])
def test_append_of_shared_and_strided_rows(n, h, d, dtype):
    """Keys shared by all heads (head stride 0), values a part of wider rows."""
    g = torch.Generator().manual_seed(n)
    K = _rand(g, n, 1, d, dtype=dtype).expand(n, h, d)
    V = _rand(g, n, h + 2, d + 16, dtype=dtype)[:, 1:h + 1, 16:]
    pages = -(-n // 5) + 1
    kc, vc = (torch.zeros(pages, 5, h, d, dtype=dtype, device="cuda") for _ in range(2))
    slots = torch.randperm(pages * 5, generator=g)[:n].to(torch.int32).cuda()
    fb.kv_append(K, V, slots, kc, vc)
    s = slots.long()
    want_k, want_v = torch.zeros_like(kc), torch.zeros_like(vc)
    want_k[s // 5, s % 5], want_v[s // 5, s % 5] = K, V
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_many_tokens_are_the_same_as_a_few(dtype, norm):
    """Tokens do not depend on each other: a long call, in whatever form its size
    selects, gives the bits of calls on its parts; so does the gradient's dx."""
    n, hq, hkv, d = 20003, 28, 4, 128
    g = torch.Generator().manual_seed(2)
    Q, K = _rand(g, n, hq, d, dtype=dtype), _rand(g, n, hkv, d, dtype=dtype)
    w = dict(w_q=_rand(g, d, dtype=dtype), w_k=_rand(g, d, dtype=dtype)) if norm else {}
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 7
    freq = torch.from_numpy(fb.rope_frequencies(d)[0]).cuda()
    q, k = fb.qk_rope(Q, K, pos, freq, **w)
    dQ, dK, *_ = fb.qk_rope_backward(q, k, pos, freq, Q, K, **w)
    for a, b in ((0, 1), (1, 200), (200, 7000), (7000, n)):
        q2, k2 = fb.qk_rope(Q[a:b], K[a:b], pos[a:b], freq, **w)
        assert torch.equal(q[a:b], q2) and torch.equal(k[a:b], k2)
        dq2, dk2, *_ = fb.qk_rope_backward(q2, k2, pos[a:b], freq, Q[a:b], K[a:b], **w)
        assert torch.equal(dQ[a:b], dq2) and torch.equal(dK[a:b], dk2)


# -------------------------------------------------------------------------- gradient
def _grad_bound(dy, x, w, ang, c, dy_rot):
    """Bounds of dx and of one dw term.  g carries 34 u of its pair's length G,
    r 13.5 u and x r one product more; dx = r (g w - x r mean(g w x r)):
    34 + 13.5 + 2 u on the first term, 34 + 29 + 13.5 + 19 (sum) + 4 u on the
    second: 100 u covers both."""
    rot, il = c[5], c[6]
    G = _radius(_f64(dy), rot, il)
    G[..., :rot] *= 1.3
    if w is None:
        return 34 * U * G, None
    w = np.abs(_f64(w))
    _, r = gen.head_norm(_f64(x), None, 1e-5)
    xh = np.abs(_f64(x)) * r
    return 100 * U * r * (G * w + xh * np.mean(G * w * xh, -1, keepdims=True)), G * xh


@pytest.mark.parametrize("dy_dtype", [FP32, BF16])
@pytest.mark.parametrize("c", CASES, ids=str)
def test_backward(c, dy_dtype):
    n, hq, hkv, d, dtype, rot, il = c[:7]
    Q, K, _, wq, wk, args, kw, ang = _case(c)
    g = torch.Generator().manual_seed(21)
    dq, dk = _rand(g, n, hq, d, dtype=dy_dtype), _rand(g, n, hkv, d, dtype=dy_dtype)
    gq, gk, dwq, dwk, ws = fb.qk_rope_backward(dq, dk, *args, Q=Q, K=K, **kw)
    for got, gw, dy, x, w, what in ((gq, dwq, dq, Q, wq, "q"), (gk, dwk, dk, K, wk, "k")):
        want, want_w = gen.qk_rope_backward(_f64(dy), _f64(x), ang, rot, il,
                                            None if w is None else _f64(w), 1e-5, 1.3)
        bound, terms = _grad_bound(dy, x, w, ang, c, rot)
        _close(got, want, bound, "d" + what)
        if w is None:
            assert gw is None
            continue
        # whatever the split, no term passes more sums than its lane's share of the terms (no
        # lane has over a quarter of the tokens), 32 lanes' sums of a block, 32 rows of blocks
        # and 32 of their sums, each of half a step
        depth = -(-n // 4) * (hq + hkv) + 96
        _close(gw, want_w, (50 + depth) * U * terms.sum((0, 1)), "dw_" + what)
    # the same bits again; in place where the upstream gradient is fp32
    again = fb.qk_rope_backward(dq, dk, *args, Q=Q, K=K, workspace=ws,
                                dQ=dq if dy_dtype == FP32 else None,
                                dK=dk if dy_dtype == FP32 else None, **kw)
    for a, b in zip((gq, gk, dwq, dwk), again):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("c", [CASES[2], CASES[3], CASES[5]], ids=str)
def test_backward_against_differences(c):
    """The gradient along a random direction v against central differences of
    the float64 forward: sum(grad v) = (L(x + h v) - L(x - h v)) / 2h up to the
    gradient's own error (100 u of the sum of its bounds, here 1e-5 relative to
    the sum of the terms' magnitudes) and the differences' (h^2)."""
    n, hq, hkv, d, dtype, rot, il = c[:7]
    Q, K, _, wq, wk, args, kw, ang = _case(c)
    g = torch.Generator().manual_seed(22)
    dq, dk = _rand(g, n, hq, d), _rand(g, n, hkv, d)
    gq, gk, dwq, _, _ = fb.qk_rope_backward(dq, dk, *args, Q=Q, K=K, **kw)
    w = None if wq is None else _f64(wq)
    r = np.random.default_rng(23)
    v, vw = r.standard_normal(Q.shape), r.standard_normal(d)
    h = 1e-4

    def loss(x, w_):
        return float((gen.qk_rope(x, ang, rot, il, w_, 1e-5, 1.3) * _f64(dq)).sum())

    x = _f64(Q)
    got, terms = (_f64(gq) * v).sum(), np.abs(_f64(gq) * v).sum()
    want = (loss(x + h * v, w) - loss(x - h * v, w)) / (2 * h)
    assert abs(got - want) <= 1e-5 * terms
    if w is not None:
        got, terms = (_f64(dwq) * vw).sum(), np.abs(_f64(dwq) * vw).sum()
        want = (loss(x, w + h * vw) - loss(x, w - h * vw)) / (2 * h)
        assert abs(got - want) <= 1e-4 * terms


def test_no_tokens():
    Q, K = torch.empty(0, 8, 128, device="cuda"), torch.empty(0, 2, 128, device="cuda")
    w = torch.ones(128, device="cuda")
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    freq = torch.ones(64, dtype=torch.float64, device="cuda")
    q, k = fb.qk_rope(Q, K, pos, freq, w_q=w, w_k=w)
    assert q.shape == Q.shape and k.shape == K.shape
    dw = torch.full((128,), 5.0, device="cuda")
    fb.qk_rope_backward(Q, K, pos, freq, Q=Q, K=K, w_q=w, w_k=w, dw_q=dw)
    assert torch.all(dw == 0)


def test_graph_replay_on_another_stream():
    """Captured on a stream of its own, replayed with other inputs in place."""
    c = CASES[11]
    Q, K, _, wq, wk, args, kw, _ = _case(c)
    Q2, K2 = _case(c, seed=8)[:2]
    g = torch.Generator().manual_seed(2)
    dq, dk = _rand(g, *Q.shape), _rand(g, *K.shape)
    q, k = torch.empty(Q.shape, dtype=BF16, device="cuda"), torch.empty(K.shape, dtype=BF16, device="cuda")
    ws = torch.empty(fb.qk_rope_backward_workspace_bytes(*Q.shape[:2], K.shape[1], 128),
                     dtype=torch.uint8, device="cuda")
    out = [torch.empty(s, device="cuda") for s in (Q.shape, K.shape, (128,), (128,))]

    def step(stream=None):
        fb.qk_rope(Q, K, *args, out_q=q, out_k=k, stream=stream, **kw)
        fb.qk_rope_backward(dq, dk, *args, Q=Q, K=K, dQ=out[0], dK=out[1], dw_q=out[2], dw_k=out[3],
                            workspace=ws, stream=stream, **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    Q.copy_(Q2), K.copy_(K2)
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (q, k, *out)]
    for x in (q, k, *out):
        x.zero_()
    s.wait_stream(torch.cuda.current_stream())
    step(stream=s)
    torch.cuda.synchronize()
    for a, b in zip(got, (q, k, *out)):
        assert torch.equal(a, b)


def test_binding_refusals():
    Q, K, V, _, _, args, kw, _ = _case(CASES[1])
    pos, freq = args
    bad = [
        lambda: fb.qk_rope(Q[:, :, ::2], K, pos, freq),                 # strided elements
        lambda: fb.qk_rope(Q, K.float(), pos, freq),                    # another type
        lambda: fb.qk_rope(Q, K[:5], pos, freq),                        # another length
        lambda: fb.qk_rope(Q, K, pos.long(), freq),                     # 64-bit positions
        lambda: fb.qk_rope(Q, K, pos, freq.float()),                    # 32-bit frequencies
        lambda: fb.qk_rope(Q, K, pos[0], freq, sections=(16, 24, 24)),  # one axis
        lambda: fb.qk_rope(Q, K, None, freq),
        lambda: fb.qk_rope(Q, K, pos, freq, sections=(32, 32)),
        lambda: fb.qk_rope(Q, K, pos, freq, w_q=torch.ones(64, dtype=BF16, device="cuda")),
        lambda: fb.qk_rope_backward(Q, K, pos, freq, w_q=torch.ones(128, dtype=BF16, device="cuda")),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        fb.qk_rope(Q.half(), K.half(), pos, freq)
    # expanded outputs share memory: refused by the library
    with pytest.raises(fb.AdasparkError):
        fb.qk_rope(Q, K, pos, freq, sections=kw["sections"],
                   out_q=Q[:1].expand(Q.shape[0], -1, -1))
    # expanded inputs are only read
    q, _ = fb.qk_rope(Q[:1].expand(Q.shape[0], -1, -1), K, pos, freq, sections=kw["sections"])
    q2, _ = fb.qk_rope(Q[:1].repeat(Q.shape[0], 1, 1), K, pos, freq, sections=kw["sections"])
    assert torch.equal(q, q2)


@pytest.mark.parametrize("n", [0, 1, 5000])
def test_backward_workspace_has_a_clear_status(n):
    g = torch.Generator().manual_seed(4)
    Q, K = _rand(g, n, 4, 64, dtype=BF16), _rand(g, n, 2, 64, dtype=BF16)
    w = torch.ones(64, dtype=BF16, device="cuda")
    ws = torch.full((fb.qk_rope_backward_workspace_bytes(n, 4, 2, 64),), 255, dtype=torch.uint8,
                    device="cuda")
    freq = torch.from_numpy(fb.rope_frequencies(64)[0]).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    *_, ws2 = fb.qk_rope_backward(Q, K, pos, freq, Q, K, w_q=w, workspace=ws)
    assert ws2.data_ptr() == ws.data_ptr() and fb.read_device_status(ws2) == (fb.OK, 0)


@pytest.mark.parametrize("axes", [3, 0])
def test_norms_alone_look_at_no_axes(axes):
    """Without a rotation the C calls read neither positions nor sections, whatever
    the number of axes: the bits of the calls with one axis."""
    import ctypes
    L, n, hq, hkv, d = fb.lib(), 50, 4, 2, 128
    g = torch.Generator().manual_seed(6)
    Q, K, V = (_rand(g, n, h, d, dtype=BF16) for h in (hq, hkv, hkv))
    w = _rand(g, d, dtype=BF16)
    want = fb.qk_rope(Q, K, None, None, w_q=w, w_k=w)
    dQ, dK = _rand(g, n, hq, d), _rand(g, n, hkv, d)
    want_g = fb.qk_rope_backward(dQ, dK, None, None, Q, K, w_q=w, w_k=w)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rope = (None, axes, None, None, 0, 0, 1.0, p(w), p(w), 1e-6, n, hq, hkv, d)
    qs, ks = (hq * d, d), (hkv * d, d)
    q, k = torch.zeros_like(Q), torch.zeros_like(K)
    assert L.adaspark_qk_rope(p(Q), *qs, p(K), *ks, fb.BF16, *rope, p(q), *qs, p(k), *ks,
                              stream) == fb.OK
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    kc, vc = (torch.zeros(n, 1, hkv, d, dtype=BF16, device="cuda") for _ in range(2))
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    q.zero_()
    assert L.adaspark_qk_rope_append(p(Q), *qs, p(K), *ks, p(V), *ks, fb.BF16, *rope, p(slots), p(kc),
                                     p(vc), hkv * d, hkv * d, d, n, 1, p(q), *qs, stream) == fb.OK
    assert torch.equal(q, want[0]) and torch.equal(kc[:, 0], want[1]) and torch.equal(vc[:, 0], V)
    out = [torch.zeros_like(t) for t in want_g[:4]]
    ws = want_g[4]
    assert L.adaspark_qk_rope_backward(p(dQ), *qs, p(dK), *ks, fb.FP32, p(Q), *qs, p(K), *ks, fb.BF16,
                                       *rope, *map(p, out), p(ws), ws.numel(), stream) == fb.OK
    for a, b in zip(out, want_g):
        assert torch.equal(a, b)


# n beyond one walk of the warps (1776), so that some take a token more than others; the last
# case takes 6 walks
@pytest.mark.parametrize("n,hq,hkv,d,dtype", [(5001, 12, 2, 128, BF16), (4300, 5, 5, 128, BF16),
                                              (2500, 7, 7, 64, FP32), (1777, 3, 1, 64, BF16),
                                              (9000, 6, 1, 64, FP32)])
def test_weight_gradients_count_every_row(n, hq, hkv, d, dtype):
    """Heads of ones with signs have the inverse root 1, so without a rotation an element of
    dw is a sum of n * heads signs, a whole number: a row that is lost, or counted twice, moves
    it by 1.  r = rsqrt(1) may be off by 2 ulp (4 u), its product with x rounds 1 u; every sum
    adds half a step: a lane's steps over its tokens, the lanes of a block at one element
    (4 warps of 32 / (d/8) heads), the blocks' rows in 128 chains and 7 halvings. Below a half
    all told."""
    g = torch.Generator().manual_seed(n)
    sign = lambda *s: (2.0 * torch.randint(0, 2, s, generator=g) - 1)  # noqa: E731
    Q, K = sign(n, hq, d), sign(n, hkv, d)
    dQ, dK = sign(n, hq, d), sign(n, hkv, d)
    w = torch.ones(d, dtype=dtype, device="cuda")
    dev = lambda t: t.to(dtype).cuda()  # noqa: E731
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    per = 256 // d                                   # heads of a warp's step
    walks = -(-n // (4 * 3 * sms))
    for rows in (slice(None), slice(n - 1, n), slice(n - 7, n - 3)):
        mq, mk = torch.zeros_like(dQ), torch.zeros_like(dK)
        mq[rows], mk[rows] = dQ[rows], dK[rows]
        *_, dwq, dwk, _ = fb.qk_rope_backward(mq.cuda(), mk.cuda(), None, None, dev(Q), dev(K),
                                              w_q=w, w_k=w, eps=0.0)
        for got, x, dy, h in ((dwq, Q, mq, hq), (dwk, K, mk, hkv)):
            want = (x.double() * dy.double()).sum((0, 1)).numpy()
            depth = walks * -(-h // per) + 4 * per + -(-3 * sms // 128) + 7
            bound = (5 + depth) * U * n * h
            assert bound < 0.5
            assert np.abs(_f64(got) - want).max() <= bound
