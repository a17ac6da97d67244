"""The calls around the key-value cache without a GPU: what pins their float64
statements (oracle/generation_ref.py), rotary frequencies, and refusals before
any device work."""
import ctypes
import math

import numpy as np
import pytest
import torch

import ffn_long_video_b200 as fb
from oracle import generation_ref as gen


# ------------------------------------------------------------------ oracle pins
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(16, 16), (16, 8), (64, 32)])
def test_rotation_is_a_complex_product(d, rot, interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, d))
    ang = gen.rope_angles(rng.integers(-50, 1000, 5), 10.0 ** -np.arange(rot // 2))
    y = gen.rotate(x, ang, rot, interleaved, 1.5)
    f, s = gen.rope_pairs(d, rot, interleaved)
    z = (x[..., f] + 1j * x[..., s]) * 1.5 * np.exp(1j * ang)[:, None]
    assert np.allclose(y[..., f], z.real, atol=1e-12)
    assert np.allclose(y[..., s], z.imag, atol=1e-12)
    assert np.array_equal(y[..., rot:], x[..., rot:])
    # the transpose undoes it up to the squared magnitude
    back = gen.rotate(y, -ang, rot, interleaved, 1.5)
    assert np.allclose(back[..., :rot], 2.25 * x[..., :rot], atol=1e-12)


def test_rotated_scores_depend_on_distance_alone():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 64))
    freq, _ = fb.rope_frequencies(64, 10000.0)
    dots = [float((gen.qk_rope(q, gen.rope_angles([a + 17], freq), 64, False)
                   * gen.qk_rope(k, gen.rope_angles([a], freq), 64, False)).sum())
            for a in (0, 5, 100000)]
    assert np.allclose(dots, dots[0], atol=1e-9)


def test_axes_follow_their_sections():
    pos = np.array([[3, 4], [10, 20], [7, 9]])
    ang = gen.rope_angles(pos, np.ones(8), (2, 3, 3))
    assert np.array_equal(ang, [[3, 3, 10, 10, 10, 7, 7, 7], [4, 4, 20, 20, 20, 9, 9, 9]])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_gradient_matches_central_differences(interleaved, norm):
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((2, 2, 2, 16))
    w = 1 + 0.3 * rng.standard_normal(16) if norm else None
    ang = gen.rope_angles([3, 50], 0.3 ** np.arange(4))
    args = (ang, 8, interleaved)
    loss = lambda x_, w_: float((gen.qk_rope(x_, *args, w_, 1e-3, 1.2) * dy).sum())  # noqa: E731
    dx, dw = gen.qk_rope_backward(dy, x, *args, w, 1e-3, 1.2)
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        # central differences: rounding 1e-16 * |loss| / h ~ 1e-9, curvature h^2
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    if norm:
        for i in range(16):
            e = np.zeros(16)
            e[i] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_plan_steps_keep_every_page_once_and_can_be_undone():
    rng = np.random.default_rng(4)
    n, cols, page, pool = 9, 12, 4, 60
    table, free = np.full((n, cols), -1), rng.permutation(pool)
    n_free, lens = pool, np.zeros(n, int)
    for step in range(40):
        new = np.where(rng.random(n) < 0.3, rng.integers(0, cols * page + 1, n),
                       np.minimum(lens + rng.integers(0, 4, n), cols * page))
        got = gen.kv_plan(lens, new, table, free, n_free, page, 500)
        if got is None:
            assert sum(-(-new // page)) > pool
            continue
        held = [p for i in range(n) for p in got[0][i, :-(-new[i] // page)]]
        assert sorted(held + list(got[1][:got[2]])) == list(range(pool))
        assert got[5][-1] == np.maximum(new - lens, 0).sum()
        back = gen.kv_plan(new, lens, got[0], got[1], got[2], page, 500)
        assert back[2] == n_free and np.array_equal(back[1][:n_free], free[:n_free])
        for i in range(n):
            assert np.array_equal(back[0][i, :-(-lens[i] // page)],
                                  table[i, :-(-lens[i] // page)])
        table, free, n_free, lens = got[0], got[1], got[2], new


def test_decode_closed_forms():
    q = np.zeros((3, 2, 64))
    k = np.random.default_rng(5).standard_normal((4, 2, 1, 64))
    v = np.arange(8.0).reshape(4, 2, 1, 1) * np.ones(64)
    out, lse = gen.decode_attn(q, k, v, [[2, 0], [1, 3], [1, 9]], [3, 0, 4])
    # equal scores: the mean of the keys' values, the logarithm of their number
    assert np.allclose(out[0], (4 + 5 + 0) / 3) and np.allclose(lse[0], math.log(3))
    assert np.all(out[1] == 0) and np.all(np.isneginf(lse[1]))
    assert np.allclose(out[2], 2.5) and np.allclose(lse[2], math.log(2))   # page 9 is not there
    # one score far above the others takes everything
    q[0, 0] = 100 * k[2, 1, 0]
    assert np.allclose(gen.decode_attn(q, k, v, [[2, 0]] * 3, [3, 0, 0])[0][0, 0], 5)


# -------------------------------------------------------------- rotary frequencies
def test_rope_frequencies():
    f, m = fb.rope_frequencies(128, 1e6)
    assert np.allclose(f, 1e6 ** (-np.arange(0, 128, 2) / 128), rtol=1e-14) and m == 1.0
    g, m = fb.rope_frequencies(128, 1e6, fb.ROPE_LINEAR, 4.0)
    assert np.allclose(g, f / 4, rtol=1e-14) and m == 1.0
    g, m = fb.rope_frequencies(64, 1e4, fb.ROPE_NTK, 8.0)
    f64, _ = fb.rope_frequencies(64, 1e4)
    # the fastest pair keeps its frequency, the slowest is divided by the factor
    assert g[0] == 1.0 and np.isclose(g[-1], f64[-1] / 8, rtol=1e-12) and m == 1.0
    g, m = fb.rope_frequencies(64, 1e4, fb.ROPE_YARN, 8.0, 4000)
    turns = 4000 * f64 / (2 * np.pi)
    assert np.allclose(g[turns >= 32], f64[turns >= 32], rtol=1e-14)
    assert np.allclose(g[turns <= 1], f64[turns <= 1] / 8, rtol=1e-14)
    assert np.all((g <= f64) & (g >= f64 / 8)) and np.isclose(m, 0.1 * math.log(8) + 1)
    # factor 1 changes nothing
    for mode in (fb.ROPE_LINEAR, fb.ROPE_NTK, fb.ROPE_YARN):
        g, m = fb.rope_frequencies(64, 1e4, mode, 1.0, 100)
        assert np.allclose(g, f64, rtol=1e-14) and m == 1.0


@pytest.mark.parametrize("args", [
    (0, 1e4), (63, 1e4), (-2, 1e4), (64, 1.0), (64, float("nan")), (64, float("inf")),
    (64, 1e4, 4, 2.0), (64, 1e4, -1, 2.0), (64, 1e4, 1, 0.5), (64, 1e4, 1, float("nan")),
    (2, 1e4, 2, 2.0), (64, 1e4, 3, 2.0, 0)])
def test_rope_frequencies_refusals(args):
    with pytest.raises(fb.AdasparkError):
        fb.rope_frequencies(*args)


# ----------------------------------------------------- refusals before device work
P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4100)
SEC = (ctypes.c_int32 * 3)(16, 24, 24)
BAD_SEC = (ctypes.c_int32 * 3)(16, 24, 25)
NEG_SEC = (ctypes.c_int32 * 3)(-16, 56, 24)


def _call(name, order, base, change):
    a = dict(base, **change)
    return getattr(fb.lib(), "adaspark_" + name)(*[a[k] for k in order.split()])


ROPE_ORDER = ("Q q_ts q_hs K k_ts k_hs dtype pos axes sec freq rot il mag wq wk eps n hq hkv d "
              "Qo qo_ts qo_hs Ko ko_ts ko_hs stream")
ROPE = dict(Q=P, q_ts=1024, q_hs=128, K=P, k_ts=256, k_hs=128, dtype=fb.BF16, pos=P, axes=3,
            sec=SEC, freq=P, rot=128, il=0, mag=1.0, wq=P, wk=P, eps=1e-6, n=7, hq=8, hkv=2,
            d=128, Qo=P, qo_ts=1024, qo_hs=128, Ko=P, ko_ts=256, ko_hs=128, stream=None)
ROPE_BAD = [dict(Q=None), dict(K=None), dict(pos=None), dict(freq=None), dict(n=-1), dict(hq=7),
            dict(hq=0), dict(hkv=0), dict(d=96), dict(dtype=2), dict(rot=8), dict(rot=136),
            dict(rot=-16), dict(axes=2), dict(axes=3, sec=BAD_SEC), dict(axes=3, sec=NEG_SEC),
            dict(axes=3, sec=None), dict(eps=-1.0), dict(eps=float("nan")),
            dict(mag=float("inf")), dict(Q=ODD), dict(q_ts=1028), dict(k_hs=132), dict(wq=ODD),
            dict(hq=8192, hkv=2), dict(n=(1 << 30) + 1)]
ROPE_OUT_BAD = [dict(Qo=None), dict(Qo=ODD), dict(qo_ts=1028),
                dict(qo_ts=512), dict(qo_hs=64), dict(qo_ts=0)]   # rows that share memory
CACHE = dict(slots=P, kc=P, vc=P, c_ps=4096, c_ts=256, c_hs=128, pages=50, page=16)
CACHE_BAD = [dict(slots=None), dict(kc=None), dict(vc=None), dict(kc=ODD), dict(c_ps=4000),
             dict(c_ts=128), dict(c_hs=64), dict(c_ts=260), dict(pages=0), dict(page=0),
             dict(pages=1 << 20, page=1 << 12)]


@pytest.mark.parametrize("change", ROPE_BAD + ROPE_OUT_BAD
                         + [dict(Ko=None), dict(Ko=ODD), dict(ko_ts=128)])
def test_qk_rope_refusals(change):
    assert _call("qk_rope", ROPE_ORDER, ROPE, change) == fb.EINVAL


def test_no_tokens_is_no_work():
    assert _call("qk_rope", ROPE_ORDER, ROPE, dict(n=0)) == fb.OK
    assert _call("kv_append", "K k_ts k_hs V v_ts v_hs dtype n hkv d slots kc vc c_ps c_ts c_hs "
                 "pages page stream", dict(ROPE, V=P, v_ts=256, v_hs=128, **CACHE),
                 dict(n=0)) == fb.OK


APPEND_ORDER = ("Q q_ts q_hs K k_ts k_hs V v_ts v_hs dtype pos axes sec freq rot il mag wq wk eps "
                "n hq hkv d slots kc vc c_ps c_ts c_hs pages page Qo qo_ts qo_hs stream")


@pytest.mark.parametrize("change", ROPE_BAD + ROPE_OUT_BAD + CACHE_BAD
                         + [dict(V=None), dict(V=ODD), dict(v_ts=260)])
def test_qk_rope_append_refusals(change):
    base = dict(ROPE, V=P, v_ts=256, v_hs=128, **CACHE)
    assert _call("qk_rope_append", APPEND_ORDER, base, change) == fb.EINVAL


@pytest.mark.parametrize("change", CACHE_BAD + [dict(K=None), dict(V=None), dict(K=ODD),
                                                dict(v_hs=4), dict(n=-1), dict(hkv=0), dict(d=32),
                                                dict(dtype=5)])
def test_kv_append_refusals(change):
    base = dict(ROPE, V=P, v_ts=256, v_hs=128, **CACHE)
    assert _call("kv_append", "K k_ts k_hs V v_ts v_hs dtype n hkv d slots kc vc c_ps c_ts c_hs "
                 "pages page stream", base, change) == fb.EINVAL


@pytest.mark.parametrize("change", [dict(gQ=None), dict(gK=None), dict(dQ=None), dict(dK=None),
                                    dict(dwq=None), dict(dwk=None), dict(ws=None),
                                    dict(ws=ctypes.c_void_p(4097)), dict(wsb=16), dict(dy=3),
                                    dict(gQ=ODD), dict(gq_ts=1025), dict(dQ=ODD)]
                         + [c for c in ROPE_BAD])
def test_qk_rope_backward_refusals(change):
    base = dict(ROPE, gQ=P, gq_ts=1024, gq_hs=128, gK=P, gk_ts=256, gk_hs=128, dy=fb.FP32, dQ=P,
                dK=P, dwq=P, dwk=P, ws=P,
                wsb=fb.qk_rope_backward_workspace_bytes(7, 8, 2, 128, fb.BF16))
    assert base["wsb"] > 0
    order = ("gQ gq_ts gq_hs gK gk_ts gk_hs dy Q q_ts q_hs K k_ts k_hs dtype pos axes sec freq rot "
             "il mag wq wk eps n hq hkv d dQ dK dwq dwk ws wsb stream")
    assert _call("qk_rope_backward", order, base, change) == fb.EINVAL


BWD_ORDER = ("gQ gq_ts gq_hs gK gk_ts gk_hs dy Q q_ts q_hs K k_ts k_hs dtype pos axes sec freq rot "
             "il mag wq wk eps n hq hkv d dQ dK dwq dwk ws wsb stream")
LAYER_ORDER = ("x Wq Wk Wv Wo Wg Wu Wd dtype ids off text C nv n hq hkv d D F pa pf pos axes sec "
               "freq rot il mag wq wk eps y ws wsb stream")


@pytest.mark.parametrize("mag", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("name", ["qk_rope", "qk_rope_append", "qk_rope_backward", "layer_rope"])
def test_a_magnitude_that_is_not_finite_is_refused_without_a_rotation_too(name, mag):
    base = dict(ROPE, rot=0, pos=None, freq=None, mag=mag, V=P, v_ts=256, v_hs=128, **CACHE)
    if name == "qk_rope_backward":
        base.update(gQ=P, gq_ts=1024, gq_hs=128, gK=P, gk_ts=256, gk_hs=128, dy=fb.FP32, dQ=P,
                    dK=P, dwq=P, dwk=P, ws=P,
                    wsb=fb.qk_rope_backward_workspace_bytes(7, 8, 2, 128, fb.BF16))
    if name == "layer_rope":
        base.update(x=P, Wq=P, Wk=P, Wv=P, Wo=P, Wg=P, Wu=P, Wd=P, ids=P, off=P, text=P, C=16,
                    nv=512, n=544, hq=4, hkv=1, D=256, F=512, pa=0.7, pf=0.7, y=P, ws=P,
                    wsb=fb.layer_workspace_bytes(544, 512, 16, 4, 1, 128, 256, 512))
    order = dict(qk_rope=ROPE_ORDER, qk_rope_append=APPEND_ORDER, qk_rope_backward=BWD_ORDER,
                 layer_rope=LAYER_ORDER)[name]
    assert _call(name, order, base, {}) == fb.EINVAL


PLAN_ORDER = "old new ns page table ts cols free pages nf starts slots pos rows ws wsb stream"


@pytest.mark.parametrize("change", [{k: None} for k in "old new table free nf starts slots pos ws".split()]
                         + [{k: 0} for k in "ns page cols pages rows wsb".split()]
                         + [dict(ts=7), dict(old=ctypes.c_void_p(4097)),
                            dict(ws=ctypes.c_void_p(4097)), dict(pages=1 << 20, page=1 << 12),
                            dict(ns=(1 << 24) + 1, wsb=1 << 40), dict(rows=(1 << 30) + 1),
                            dict(pages=(1 << 30) + 1, page=1)])
def test_kv_plan_refusals(change):
    base = dict(old=P, new=P, ns=5, page=16, table=P, ts=8, cols=8, free=P, pages=64, nf=P,
                starts=P, slots=P, pos=P, rows=40, ws=P, wsb=fb.kv_plan_workspace_bytes(5),
                stream=None)
    assert _call("kv_plan", PLAN_ORDER, base, change) == fb.EINVAL


DECODE_ORDER = ("Q q_ts q_hs kc vc c_ps c_ts c_hs pages page dtype table ts cols lens ns hq hkv d "
                "scale out lse ws wsb stream")


@pytest.mark.parametrize("change", [dict(Q=None), dict(table=None), dict(lens=None), dict(out=None),
                                    dict(ws=None), dict(wsb=100), dict(ns=0), dict(cols=0),
                                    dict(scale=float("nan")), dict(hq=9), dict(d=256), dict(Q=ODD),
                                    dict(q_ts=1028), dict(out=ODD), dict(dtype=3),
                                    dict(cols=1 << 28), dict(ws=ctypes.c_void_p(4097)),
                                    dict(ns=(1 << 24) + 1, wsb=1 << 40),
                                    dict(ns=1 << 23, cols=1 << 16, wsb=1 << 40)]
                         + CACHE_BAD[1:])
def test_decode_attn_refusals(change):
    base = dict(Q=P, q_ts=1024, q_hs=128, dtype=fb.BF16, table=P, ts=8, cols=8, lens=P, ns=5, hq=8,
                hkv=2, d=128, scale=0.1, out=P, lse=P, ws=P,
                wsb=fb.decode_attn_workspace_bytes(5, 8, 2, 128, fb.BF16), stream=None, **CACHE)
    assert base["wsb"] > 0
    assert _call("decode_attn", DECODE_ORDER, base, change) == fb.EINVAL


@pytest.mark.parametrize("change", [dict(pos=None), dict(freq=None), dict(rot=8), dict(axes=2),
                                    dict(sec=BAD_SEC), dict(sec=None), dict(eps=-1.0),
                                    dict(mag=float("nan")), dict(wq=ODD), dict(x=None),
                                    dict(ws=None), dict(wsb=8)])
def test_layer_rope_refusals(change):
    base = dict(ROPE, x=P, Wq=P, Wk=P, Wv=P, Wo=P, Wg=P, Wu=P, Wd=P, ids=P, off=P, text=P, C=16,
                nv=512, n=544, hq=4, hkv=1, D=256, F=512, pa=0.7, pf=0.7, y=P, ws=P,
                wsb=fb.layer_workspace_bytes(544, 512, 16, 4, 1, 128, 256, 512))
    order = ("x Wq Wk Wv Wo Wg Wu Wd dtype ids off text C nv n hq hkv d D F pa pf pos axes sec freq "
             "rot il mag wq wk eps y ws wsb stream")
    assert _call("layer_rope", order, base, change) == fb.EINVAL


def test_workspace_queries_of_bad_sizes_are_zero():
    assert fb.kv_plan_workspace_bytes(0) == 0
    assert fb.qk_rope_backward_workspace_bytes(-1, 8, 2, 128) == 0
    assert fb.qk_rope_backward_workspace_bytes(5, 8, 3, 128) == 0
    assert fb.decode_attn_workspace_bytes(0, 8, 2, 128) == 0
    assert fb.decode_attn_workspace_bytes(1, 8, 2, 96) == 0


def test_binding_refuses_host_tensors():
    x, kv = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    i = torch.zeros(3, dtype=torch.int32)
    c = torch.zeros(2, 16, 2, 64)
    f = torch.zeros(32, dtype=torch.float64)
    for call in (lambda: fb.qk_rope(x, kv, i, f),
                 lambda: fb.qk_rope_append(x, kv, kv, i, f, i, c, c),
                 lambda: fb.kv_append(kv, kv, i, c, c),
                 lambda: fb.qk_rope_backward(x, kv, i, f),
                 lambda: fb.kv_plan(i, i, torch.zeros(3, 2, dtype=torch.int32), i, i[:1], 16, 4),
                 lambda: fb.decode_attn(x, c, c, torch.zeros(3, 2, dtype=torch.int32), i)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("given", [dict(positions=torch.zeros(4, dtype=torch.int32)),
                                   dict(sections=(16, 24, 24)),
                                   dict(positions=torch.zeros(4, dtype=torch.int32),
                                        w_qnorm=torch.ones(128))])
def test_layer_refuses_positions_without_frequencies(given):
    """They would be dropped: the layer would run without its positions."""
    with pytest.raises(ValueError, match="freq"):
        fb.layer(*[torch.zeros(4, 4)] * 11, 2, 1, 1, 0.7, 0.7, **given)


@pytest.mark.parametrize("scale", [3.4e38, -2.4e38, float("inf"), float("nan")])
def test_decode_refuses_a_scale_beyond_its_logarithm_base(scale):
    """The scores are kept in base 2: a scale whose product with log2(e) overflows would make
    a score of 0 NaN."""
    base = dict(Q=P, q_ts=1024, q_hs=128, dtype=fb.BF16, table=P, ts=8, cols=8, lens=P, ns=5, hq=8,
                hkv=2, d=128, scale=scale, out=P, lse=P, ws=P,
                wsb=fb.decode_attn_workspace_bytes(5, 8, 2, 128, fb.BF16), stream=None, **CACHE)
    assert _call("decode_attn", DECODE_ORDER, base, {}) == fb.EINVAL
