"""The calls as they are used together (needs a B200): a video prompt through
rotary positions and AdaS-Attn, its keys and values into the paged cache, then
text tokens one at a time - plan, rotate and append, attend.  A text token of
AdaS-Attn attends densely to every earlier token, so each step's output is held
to the prefill's row of the same token."""
import numpy as np
import pytest
import torch

import ffn_long_video_b200 as fb
import workloads
from oracle import generation_ref as gen
from tests import parity

pytestmark = pytest.mark.gpu

CASES = {
    "bf16": workloads.small_config(name="gen-bf16", grid=(4, 8, 8), cube=(4, 4, 4), n_text=24,
                                   D=256, hq=8, hkv=2, F=256, seed=71),
    "fp32-d64": workloads.small_config(name="gen-fp32", grid=(4, 8, 8), cube=(4, 4, 2), n_text=17,
                                       D=256, hq=4, hkv=1, d=64, F=256, dtype="fp32", seed=72),
}


def video_positions(cfg):
    """[3, N]: (t, h, w) of the video tokens in cube order, then text positions."""
    T, H, W = cfg.grid
    ch, cw, ct = cfg.cube
    perm, _, _ = fb.cube_partition(T, H, W, ch, cw, ct, cfg.n_text)
    t, rest = perm // (H * W), perm % (H * W)
    vis = np.stack((t, rest // W, rest % W))
    text = vis.max() + 1 + np.arange(cfg.n_text)
    return np.concatenate((vis, np.broadcast_to(text, (3, cfg.n_text))), axis=1).astype(np.int32)


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("graph", [False, True])
def test_decoding_continues_the_prompt(name, graph):
    cfg = CASES[name]
    case = parity.make_case(cfg)
    t, N, n_new, page, d = case["t"], cfg.n_tokens, 9, 16, cfg.d
    sections = (d // 8, 3 * d // 16, 3 * d // 16)
    freq, mag = fb.rope_frequencies(d, 1e6)
    freq = torch.from_numpy(freq).cuda()
    pos = torch.from_numpy(video_positions(cfg)).cuda()
    w = torch.ones(d, dtype=t["Q"].dtype, device="cuda")
    kw = dict(w_q=w, w_k=w, sections=sections, magnitude=mag)
    Qr, Kr = fb.qk_rope(t["Q"], t["K"], pos, freq, **kw)
    want, ws = fb.cube_attn(Qr, Kr, t["V"], case["ids"], case["off"], cfg.n_vis, cfg.p)
    assert fb.read_device_status(ws)[0] == fb.OK

    # a batch of two sequences: the prompt twice, the second one shorter by three text tokens
    lens = [N - n_new, N - n_new - 3]
    cols = -(-N // page)
    pool = 2 * cols + 3
    table = torch.full((2, cols), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pool, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    n_free = torch.tensor([pool], dtype=torch.int32, device="cuda")
    k_cache = torch.full((pool, page, cfg.hkv, d), float("nan"), dtype=Kr.dtype, device="cuda")
    v_cache = torch.full_like(k_cache, float("nan"))
    cur = torch.zeros(2, dtype=torch.int32, device="cuda")
    nxt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    slots, prompt_pos, starts, pws = fb.kv_plan(cur, nxt, table, free, n_free, page, sum(lens) + 5)
    assert fb.read_device_status(pws)[0] == fb.OK
    row = prompt_pos[:sum(lens)].long()
    fb.kv_append(Kr[row], t["V"][row], slots[:sum(lens)].contiguous(), k_cache, v_cache)
    cur.copy_(nxt)

    # the step's buffers, as a captured loop keeps them; one padding row
    rows = 3
    q_in, k_in, v_in = (torch.zeros(rows, x.shape[1], d, dtype=x.dtype, device="cuda")
                        for x in (t["Q"], t["K"], t["V"]))
    pos3 = torch.zeros(3, rows, dtype=torch.int32, device="cuda")
    b = {k: torch.empty(s, dtype=torch.int32, device="cuda")
         for k, s in (("slots", rows), ("positions", rows), ("token_starts", 3))}
    qr = torch.empty_like(q_in)
    out = torch.empty(2, cfg.hq, d, dtype=Qr.dtype, device="cuda")
    lse = torch.empty(2, cfg.hq, device="cuda")
    dt = fb.BF16 if cfg.dtype == "bf16" else fb.FP32
    dws = torch.empty(fb.decode_attn_workspace_bytes(2, cfg.hq, cfg.hkv, d, dt), dtype=torch.uint8,
                      device="cuda")

    def step():
        fb.kv_plan(cur, nxt, table, free, n_free, page, rows, workspace=pws, **b)
        fb.qk_rope_append(q_in, k_in, v_in, pos3, freq, b["slots"], k_cache, v_cache, out_q=qr, **kw)
        fb.decode_attn(qr[:2], k_cache, v_cache, table, nxt, out=out, lse=lse, workspace=dws)
        cur.copy_(nxt)

    captured = None
    outs = []
    for i in range(n_new):
        at = [lens[0] + i, lens[1] + i]
        nxt.copy_(torch.tensor([x + 1 for x in at], dtype=torch.int32))
        for buf, src in ((q_in, t["Q"]), (k_in, t["K"]), (v_in, t["V"])):
            buf[:2] = src[at]
        pos3[:, :2] = pos[:, at]
        if graph and captured is None:
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
        if graph:
            captured.replay()
        else:
            step()
        for x in (pws, dws):
            assert fb.read_device_status(x)[0] == fb.OK
        assert b["positions"].tolist() == at + [0] and b["slots"][2] == -1
        # the rotated rows are the prefill's, so the cache holds the prompt's keys
        assert torch.equal(qr[:2], Qr[at])
        outs.append(out.clone())
        if cfg.dtype == "bf16":
            tol = dict(atol=2e-2, rtol=2.0 ** -7)     # two roundings of bf16, and the protocol's 2e-2
        else:
            tol = dict(atol=1e-4, rtol=1e-5)
        assert torch.allclose(out.float(), want[at].float(), **tol), (i, (out - want[at]).abs().max())
    # the last step against the float64 statement over the prefill's own keys
    full = lambda x, n: x[:n].unsqueeze(0)  # noqa: E731
    for s, n in enumerate((N, N - 3)):
        o, l = gen.decode_attn(Qr[n - 1:n].cpu(), full(Kr, n).cpu().float().numpy(),
                               full(t["V"], n).cpu().float().numpy(), np.zeros((1, 1), int), [n])
        assert np.abs(lse[s].double().cpu().numpy() - l[0]).max() <= 1e-4
        assert np.abs(out[s].double().cpu().numpy() - o[0]).max() <= (2e-2 if dt == fb.BF16 else 1e-4)


@pytest.mark.parametrize("rotate,norm", [(True, True), (True, False), (False, True)])
def test_layer_with_positions(rotate, norm):
    """The layer's own path through qk_rope: its Q and K are the rotated
    projections and its attention the standalone call's, bit for bit."""
    cfg = workloads.small_config(name="gen-layer", grid=(4, 8, 8), cube=(4, 4, 4), n_text=23, D=256,
                                 hq=6, hkv=3, F=256, seed=73)
    t = {k: v.cuda() for k, v in workloads.make_stack(cfg, 0).items()}
    W = [t[k].t().contiguous() for k in ("W_q", "W_k", "W_v", "W_o")]
    ids, off, text, _ = parity.layout_tensors(cfg, "cuda")
    args = (t["x"], *W, t["W_gate"], t["W_up"], t["W_down"], ids, off, text, cfg.n_vis, cfg.hq,
            cfg.hkv, 0.7, 0.7)
    sizes = (cfg.n_tokens, cfg.n_vis, cfg.n_cubes, cfg.hq, cfg.hkv, cfg.d, cfg.D, cfg.F)
    _, ws = fb.layer(*args)
    plain = {k: v.clone() for k, v in fb.layer_buffers(ws, *sizes).items() if k in "QKV"}
    kw = {}
    g = torch.Generator().manual_seed(4)
    pos = torch.from_numpy(video_positions(cfg)).cuda()
    freq = torch.from_numpy(fb.rope_frequencies(cfg.d, 1e6)[0]).cuda()
    w = (1 + 0.2 * torch.randn(2, cfg.d, generator=g)).to(torch.bfloat16).cuda()
    if rotate:
        kw.update(positions=pos, freq=freq, sections=(16, 24, 24), magnitude=1.1)
    if norm:
        kw.update(w_qnorm=w[0].contiguous(), w_knorm=w[1].contiguous())
    y, ws = fb.layer(*args, **kw)
    assert fb.read_device_status(ws)[0] == fb.OK
    buf = fb.layer_buffers(ws, *sizes)
    Q, K = fb.qk_rope(plain["Q"], plain["K"], kw.get("positions"), kw.get("freq"),
                      w_q=kw.get("w_qnorm"), w_k=kw.get("w_knorm"), sections=kw.get("sections"),
                      magnitude=kw.get("magnitude", 1.0))
    assert torch.equal(buf["Q"], Q) and torch.equal(buf["K"], K)
    assert torch.equal(buf["V"], plain["V"])
    out, _ = fb.cube_attn(Q, K, plain["V"], ids, off, cfg.n_vis, 0.7)
    assert torch.equal(buf["a"], out) and torch.isfinite(y).all()
    with pytest.raises(ValueError):
        fb.layer(*args, freq=freq)
    with pytest.raises(fb.AdasparkError):
        fb.layer(*args, freq=freq, positions=pos, sections=(16, 24, 23))


def test_layer_with_norms_looks_at_no_axes():
    """The C call of a layer with norms and no rotation, three axes named and no sections:
    the bits of the call with one axis."""
    import ctypes
    cfg = workloads.small_config(name="gen-norms", grid=(4, 8, 8), cube=(4, 4, 4), n_text=23, D=256,
                                 hq=6, hkv=3, F=256, seed=74)
    t = {k: v.cuda() for k, v in workloads.make_stack(cfg, 0).items()}
    W = [t[k].t().contiguous() for k in ("W_q", "W_k", "W_v", "W_o")]
    ids, off, text, _ = parity.layout_tensors(cfg, "cuda")
    w = torch.linspace(0.5, 1.5, cfg.d).to(torch.bfloat16).cuda()
    want, ws = fb.layer(t["x"], *W, t["W_gate"], t["W_up"], t["W_down"], ids, off, text, cfg.n_vis,
                        cfg.hq, cfg.hkv, 0.7, 0.7, w_qnorm=w, w_knorm=w)
    y = torch.zeros_like(want)
    p = lambda x: ctypes.c_void_p(x.data_ptr())  # noqa: E731
    args = [p(x) for x in (t["x"], *W, t["W_gate"], t["W_up"], t["W_down"])]
    rc = fb.lib().adaspark_layer_rope(
        *args, fb.BF16, p(ids), p(off), p(text), cfg.n_cubes, cfg.n_vis, cfg.n_tokens, cfg.hq,
        cfg.hkv, cfg.d, cfg.D, cfg.F, 0.7, 0.7, None, 3, None, None, 0, 0, 1.0, p(w), p(w), 1e-6,
        p(y), p(ws), ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == fb.OK and fb.read_device_status(ws)[0] == fb.OK
    assert torch.equal(y, want)


def test_rotary_positions_after_a_video_lie_an_offset_from_the_plan():
    """Tokens after a video prompt: the plan's positions count tokens; with the sequence's
    offset, on one axis, they rotate as the prompt's three equal axes do, bit for bit."""
    cfg = CASES["bf16"]
    g = torch.Generator().manual_seed(5)
    pos = torch.from_numpy(video_positions(cfg)).cuda()
    d, sections = cfg.d, (cfg.d // 8, 3 * cfg.d // 16, 3 * cfg.d // 16)
    freq = torch.from_numpy(fb.rope_frequencies(d, 1e6)[0]).cuda()
    Q, K, V = (torch.randn(cfg.n_tokens, h, d, generator=g).to(torch.bfloat16).cuda()
               for h in (cfg.hq, cfg.hkv, cfg.hkv))
    want_q, want_k = fb.qk_rope(Q, K, pos, freq, sections=sections)
    # two sequences: the video alone, and the video with five text tokens
    at = [cfg.n_vis, cfg.n_vis + 5]
    offset = torch.stack([pos[:, :n].max() + 1 - n for n in at]).to(torch.int32)
    assert offset[0] == offset[1] < -32
    lens, page = torch.tensor(at, dtype=torch.int32, device="cuda"), 16
    cols = -(-cfg.n_tokens // page)
    table = torch.full((2, cols), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(2 * cols, dtype=torch.int32, device="cuda")
    n_free = torch.tensor([2 * cols], dtype=torch.int32, device="cuda")
    fb.kv_plan(lens * 0, lens, table, free, n_free, page, sum(at))
    slots, places, _, ws = fb.kv_plan(lens, lens + 1, table, free, n_free, page, 2)
    assert fb.read_device_status(ws) == (fb.OK, 0) and places.tolist() == at
    kc, vc = (torch.zeros(2 * cols, page, cfg.hkv, d, dtype=Q.dtype, device="cuda") for _ in range(2))
    q = fb.qk_rope_append(Q[at], K[at], V[at], places + offset, freq, slots, kc, vc)
    s = slots.long()
    assert torch.equal(q, want_q[at]) and torch.equal(kc[s // page, s % page], want_k[at])
    # the places themselves would not do
    assert not torch.equal(fb.qk_rope(Q[at], K[at], places, freq)[0], want_q[at])
