"""Attention of one new token over the paged cache against the float64
statement (needs a B200).

Tolerances, with u = 2^-24: a score is a sum of d products in fp32.  fp32 inputs:
a lane adds d / 32 products, five exchanges follow: under 12 u of scale
sum|q k|.  bf16 inputs: the products are exact, and the sum may run over all d
terms in hardware that keeps at least fp32 and may cut instead of round: 2 d u.
The scaled score, its difference to the maximum (2 u |z| each, |z - max| taken
as 2 max|z|), exp2 (2 ulp) and the factor log2(e) give 8 u max|z| + 4 u.  With
dz that sum, a weight is off by dz relative, against a sum of weights off by
the same: 2 dz.  A weight kept as two bf16 parts adds 2^-16.  Sums run over a
quarter of the keys and the joins: (n / 4 + 700) u.  So
  |out - want| <= (2 dz + 2^-16 [bf16] + (n / 4 + 700) u) sum p |v| + eps / 2 |want|
  |lse - want| <= dz + (n / 4 + 700) u + 4 u |want|."""
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


def _make(lens, hq, hkv, d, dtype, page, heads_outer=False, seed=0, spare_cols=0, spare_pages=2,
          garbage=True, scale=1.0):
    """Q, cache, table of sequences on scattered pages; what no sequence holds is NaN."""
    g = torch.Generator().manual_seed(seed)
    lens = [int(n) for n in lens]
    held = [-(-n // page) for n in lens]
    cols = max(1, max(held)) + spare_cols
    pool = sum(held) + spare_pages
    ids = torch.randperm(pool, generator=g).tolist()
    table = torch.full((len(lens), cols), 2 ** 30, dtype=torch.int32)
    shape = (pool, page, hkv, d)
    k = torch.full(shape, float("nan")) if garbage else torch.zeros(shape)
    v = k.clone()
    at = 0
    for i, n in enumerate(lens):
        p = torch.tensor(ids[at:at + held[i]], dtype=torch.long)
        at += held[i]
        table[i, :held[i]] = p.to(torch.int32)
        j = torch.arange(n)
        k[p[j // page], j % page] = scale * torch.randn(n, hkv, d, generator=g)
        v[p[j // page], j % page] = torch.randn(n, hkv, d, generator=g)
    q = torch.randn(len(lens), hq, d, generator=g)
    k, v, q = (x.to(dtype).cuda() for x in (k, v, q))
    if heads_outer:
        k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    return q, k, v, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def _check(q, k, v, table, lens, out, lse, scale=None, want=None):
    hq, d = q.shape[1:]
    hkv, page = k.shape[2], k.shape[1]
    bf16 = q.dtype == BF16
    want, want_lse = want or gen.decode_attn(_f64(q), _f64(k), _f64(v), table.cpu().numpy(),
                                             lens.tolist(), scale)
    sc = abs(d ** -0.5 if scale is None else scale)
    out, lse, Q = _f64(out), _f64(lse), _f64(q)
    for i, n in enumerate(lens.tolist()):
        if n == 0:
            assert np.all(out[i] == 0) and np.all(np.isneginf(lse[i]))
            continue
        j = np.arange(n)
        t = table[i].cpu().numpy()[j // page]
        there = (t >= 0) & (t < k.shape[0])
        t, j = torch.from_numpy(t[there]).long().cuda(), torch.from_numpy(j[there] % page).cuda()
        K, V = _f64(k[t, j]), _f64(v[t, j])
        for h in range(hq):
            kh, vh = K[:, h // (hq // hkv)], np.abs(V[:, h // (hq // hkv)])
            z = kh @ Q[i, h] * (d ** -0.5 if scale is None else scale)
            dot = (np.abs(kh) @ np.abs(Q[i, h])).max() * sc
            dz = (2 * d if bf16 else 12) * U * dot + 8 * U * np.abs(z).max() + 4 * U
            p = np.exp(z - want_lse[i, h])
            sums = (len(z) / 4 + 700) * U
            rel = 2 * dz + sums + (2.0 ** -16 if bf16 else 0)
            eps = torch.finfo(q.dtype).eps / 2
            err = np.abs(out[i, h] - want[i, h])
            bound = rel * (p @ vh) * (1 + eps) + eps * np.abs(want[i, h])
            assert np.all(err <= bound), (i, h, n, float((err / bound).max()))
            e = abs(lse[i, h] - want_lse[i, h])
            assert e <= dz + sums + 4 * U * abs(want_lse[i, h]), (i, h, n, e)


def _run(*a, scale=None, **kw):
    out, lse, ws = fb.decode_attn(*a, scale=scale, **kw)
    code, det = fb.read_device_status(ws)
    assert code == fb.OK, hex(det)
    return out, lse


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 300, 0, 513]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("hq,hkv,d", [(28, 4, 128), (16, 2, 128), (4, 1, 64), (6, 3, 64), (3, 3, 128),
                                      (16, 1, 128), (9, 1, 64), (24, 2, 128),
                                      (20, 1, 128), (40, 1, 64)])
@pytest.mark.parametrize("spare_cols", [0, 3000])
def test_lengths_and_heads(hq, hkv, d, dtype, spare_cols):
    """Tables as long as the longest sequence (a cluster of blocks per run), and
    far longer ones (the line of tiles over the GPU)."""
    case = _make(LENS, hq, hkv, d, dtype, 16, seed=hq, spare_cols=spare_cols)
    _check(*case, *_run(*case))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n_seqs,longest", [(1, 1), (1, 64), (1, 65), (2, 129), (1, 500), (5, 256),
                                            (3, 1000), (1, 2048), (1, 2049), (60, 70), (100, 33)])
def test_few_short_sequences(n_seqs, longest, dtype):
    """Clusters of 1 to 8 blocks per run and their borders: runs of one tile to
    four a block, blocks without a tile, sequences without keys."""
    r = np.random.default_rng(longest)
    lens = r.integers(0, longest + 1, n_seqs)
    lens[-1] = longest
    case = _make(lens, 7, 1, 128, dtype, 16, seed=longest)
    out, lse = _run(*case)
    _check(*case, out, lse)
    o, l = _run(*case)
    assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (FP32, 128), (FP32, 64)])
@pytest.mark.parametrize("page", [1, 5, 23, 64, 100, 256, 1000])
@pytest.mark.parametrize("heads_outer", [False, True])
def test_pages_and_layouts(page, dtype, d, heads_outer):
    case = _make([700, 3, 0, 257, 99, 64, 1], 8, 2, d, dtype, page, heads_outer, seed=page,
                 spare_cols=page % 3)
    _check(*case, *_run(*case))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,hq,hkv", [(5000, 7, 1), (20011, 7, 1), (9000, 12, 1), (4000, 2, 2),
                                      (3000, 32, 2)])
def test_one_long_sequence(n, hq, hkv, dtype):
    """Cut over all blocks and joined."""
    case = _make([n], hq, hkv, 128, dtype, 64, seed=n)
    _check(*case, *_run(*case))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_ragged_batch(dtype):
    r = np.random.default_rng(0)
    case = _make(r.integers(0, 900, 70), 8, 2, 128, dtype, 16, seed=2)
    out, lse = _run(*case)
    _check(*case, out, lse)
    for _ in range(3):       # the same bits each time
        o, l = _run(*case)
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_more_sequences_than_threads():
    r = np.random.default_rng(1)
    lens = r.integers(0, 9, 1500)
    lens[700:900] = 0
    case = _make(lens, 2, 1, 64, BF16, 4, seed=3)
    _check(*case, *_run(*case))


def test_all_sequences_empty():
    case = _make([0] * 5, 8, 2, 128, BF16, 16)
    out, lse = _run(*case)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
@pytest.mark.parametrize("spare_cols", [0, 3000])
def test_scales(scale, spare_cols):
    case = _make([100, 7], 8, 2, 64, FP32, 16, seed=4, spare_cols=spare_cols)
    _check(*case, *_run(*case, scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_large_scores(dtype):
    """Scores in the thousands: one key takes (nearly) all; the running maximum
    moves at every tile."""
    q, k, v, table, lens = _make([400, 150], 8, 2, 128, dtype, 16, seed=5, garbage=False)
    k = (k.float() * torch.linspace(1, 60, k.shape[0], device="cuda")[:, None, None, None]).to(dtype)
    q = (q.float() * 8).to(dtype)
    _check(q, k, v, table, lens, *_run(q, k, v, table, lens))


@pytest.mark.parametrize("spare_cols", [0, 3000])
def test_infinite_scores(spare_cols):
    """Every score -inf: nothing is left of the row (0, -inf).  Some: those keys
    weigh nothing.  A NaN or +inf score makes its row NaN and no other."""
    q, k, v, table, lens = _make([40, 40, 40, 40], 4, 4, 64, FP32, 8, seed=6, garbage=False,
                                 spare_cols=spare_cols)
    q.fill_(1.0)
    # key j of sequence i on its page, head i only
    def key(i, j):
        return (int(table[i, j // 8]), j % 8, i)
    for j in range(40):
        k[key(0, j)] = float("-inf")
    k[key(1, 3)] = float("-inf")
    k[key(2, 5)] = float("nan")
    k[key(3, 30)] = float("inf")
    out, lse, ws = fb.decode_attn(q, k, v, table, lens)
    want, want_lse = gen.decode_attn(_f64(q), np.nan_to_num(_f64(k), nan=0, posinf=0, neginf=-1e300),
                                     _f64(v), table.cpu().numpy(), lens.tolist())
    assert torch.all(out[0, 0] == 0) and torch.isneginf(lse[0, 0])
    assert torch.all(torch.isnan(out[2, 2])) and torch.all(torch.isnan(out[3, 3]))
    ok = np.ones((4, 4), bool)
    ok[0, 0] = ok[2, 2] = ok[3, 3] = False
    assert np.allclose(_f64(out)[ok], want[ok], atol=1e-4)
    assert np.allclose(_f64(lse)[ok], want_lse[ok], atol=1e-4)


def test_strides_and_given_outputs():
    """Q as part of a projection, K and V as the halves of one cache, a table
    with longer rows; results into given buffers."""
    q, k, v, table, lens = _make([77, 300, 5], 8, 2, 128, BF16, 16, seed=7)
    want = _run(q, k, v, table, lens)
    both = torch.stack((k, v), dim=1)
    wide = torch.full((3, 12, 128), float("nan"), dtype=BF16, device="cuda")
    wide[:, :8] = q
    rows = torch.full((3, table.shape[1] + 5), -3, dtype=torch.int32, device="cuda")
    rows[:, :table.shape[1]] = table
    out = torch.full_like(q, float("nan"))
    lse = torch.full((3, 8), float("nan"), device="cuda")
    ws = torch.randint(0, 255, (fb.decode_attn_workspace_bytes(3, 8, 2, 128),), dtype=torch.uint8,
                       device="cuda")
    fb.decode_attn(wide[:, :8], both[:, 0], both[:, 1], rows[:, :table.shape[1]], lens, out=out,
                   lse=lse, workspace=ws)
    assert fb.read_device_status(ws)[0] == fb.OK
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 6, 7, 10, 11, 17, 23])
@pytest.mark.parametrize("spare_cols", [0, 3000])
def test_every_group_size_in_fp32(group, d, spare_cols):
    """Query heads per KV head, which fp32 cuts into runs of 2 to 8."""
    x = _make([0, 1, 70, 333], 2 * group, 2, d, FP32, 16, spare_cols=spare_cols, seed=group)
    _check(*x, *_run(*x))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lens,spare_cols", [([300, 0, 77], 0), ([300, 0, 4000], 3000),
                                             ([30] * 200, 0)])
def test_output_over_the_queries(lens, spare_cols, dtype):
    """out may be Q itself: the same results as apart."""
    x = _make(lens, 16, 2, 128, dtype, 16, spare_cols=spare_cols)
    out, lse = _run(*x)
    q = x[0].clone()
    over, lse2 = _run(q, *x[1:], out=q)
    assert over.data_ptr() == q.data_ptr()
    assert torch.equal(out, q) and torch.equal(lse, lse2)


@pytest.mark.parametrize("spare_cols", [0, 3000])
def test_bad_lengths_and_pages_are_flagged(spare_cols):
    """A length the table cannot hold counts as 0, a page that is not there holds
    no keys; both are reported, and other sequences are as without them."""
    case = _make([40, 60, 50], 8, 2, 128, BF16, 16, seed=8, spare_cols=spare_cols)
    q, k, v, table, lens = case
    want = _run(*case)
    for bad in (-1, table.shape[1] * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        lens2 = lens.clone()
        lens2[1] = bad
        out, lse, ws = fb.decode_attn(q, k, v, table, lens2)
        code, det = fb.read_device_status(ws)
        assert code == fb.EDEVICE and det & 0xff == fb.DEV_BAD_LAYOUT
        assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))
        # another cut of the work: equal up to the joins' rounding
        for i in (0, 2):
            assert torch.allclose(lse[i], want[1][i], rtol=0, atol=1e-5)
    for bad in (-1, k.shape[0], 2 ** 31 - 1, -2 ** 31):
        t2 = table.clone()
        t2[1, 2] = bad
        out, lse, ws = fb.decode_attn(q, k, v, t2, lens)
        code, det = fb.read_device_status(ws)
        assert code == fb.EDEVICE and det & 0xff == fb.DEV_BAD_LAYOUT
        _check(q, k, v, t2, lens, out, lse)
    assert torch.equal(_run(*case)[0], want[0])     # the next call is clean


def test_far_pages():
    """Pages past 2^31 elements of a cache."""
    hkv, d, page = 4, 128, 64
    pages = 2 ** 31 // (hkv * d * page) + 2000
    kc, vc = (torch.empty(pages, page, hkv, d, dtype=BF16, device="cuda") for _ in range(2))
    q, k, v, table, lens = _make([300, 130], 28, hkv, d, BF16, page, seed=9)
    want = _run(q, k, v, table, lens)
    n = k.shape[0]
    kc[-n:], vc[-n:] = k, v
    out, lse = _run(q, kc, vc, torch.where(table < n, table + (pages - n), table), lens)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_captured_calls_share_a_workspace():
    """Two captured calls on one workspace, replayed in turn while the lengths
    grow in place, equal the eager calls."""
    q, k, v, table, lens = _make([300, 64, 0, 129], 8, 2, 128, BF16, 16, seed=10)
    q2 = torch.randn(q.shape, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    ws = torch.empty(fb.decode_attn_workspace_bytes(4, 8, 2, 128), dtype=torch.uint8, device="cuda")
    n = lens.clone()
    res = [(torch.empty_like(q), torch.empty(4, 8, device="cuda")) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, x, (o, l) in zip(graphs, (q, q2), res):
        with torch.cuda.graph(g):
            fb.decode_attn(x, k, v, table, n, out=o, lse=l, workspace=ws)
    for cut in (0, 1, 40, 200):
        n.copy_(torch.clamp(lens - cut, min=0))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert fb.read_device_status(ws)[0] == fb.OK
        for x, (o, l) in zip((q, q2), res):
            eo, el = _run(x, k, v, table, n)
            assert torch.equal(o, eo) and torch.equal(l, el)


def test_two_streams():
    """Calls on two streams with workspaces of their own."""
    case = _make([2000, 100], 8, 2, 128, BF16, 16, seed=11)
    want = _run(*case)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            got.append(fb.decode_attn(*case, stream=s))
    torch.cuda.synchronize()
    for out, lse, ws in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_binding_refusals():
    q, k, v, table, lens = _make([40, 60], 8, 2, 128, BF16, 16)
    bad = [
        lambda: fb.decode_attn(q, k, v[:, :8], table, lens),
        lambda: fb.decode_attn(q, k, v.transpose(0, 1), table, lens),
        lambda: fb.decode_attn(q, k.float(), v.float(), table, lens),
        lambda: fb.decode_attn(q, k[0], v[0], table, lens),
        lambda: fb.decode_attn(q, k, v, table.long(), lens),
        lambda: fb.decode_attn(q, k, v, table[:1], lens),
        lambda: fb.decode_attn(q, k, v, table.t().contiguous().t(), lens),
        lambda: fb.decode_attn(q, k, v, table, lens[:1]),
        lambda: fb.decode_attn(q, k, v, table, lens, out=q.float()),
        lambda: fb.decode_attn(q, k, v, table, lens, workspace=lens),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fb.AdasparkError):
        fb.decode_attn(q, k, v, table, lens, scale=float("inf"))
    with pytest.raises(fb.AdasparkError):
        fb.decode_attn(q, k, v, table, lens, workspace=torch.empty(256, dtype=torch.uint8,
                                                                  device="cuda"))
