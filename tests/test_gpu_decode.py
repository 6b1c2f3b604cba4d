"""moe_decode / moe_decode_mxfp4: the whole layer for a few tokens in one launch, against 64 bits.

Routing is compared with the oracle's gate by the rule of parity.py; the outputs with the layer's
formula in fp64 on the experts that the call chose.  Tolerance of y, before any run: the kernel
rounds twice to bf16 (h and y, each off by at most 2^-8 relative, half a step) and accumulates in
fp32, so element by element

    |err| <= 2^-8 |y| (1 + 2^-8) + 2^-8 A + 2^-14 A,   A = sum_j |w_j| (|h_j| . |w2_j|^T) + |h_s| . |w2_s|^T

where 2^-14 A covers the fp32 sums: at most 7168 + 2048 terms each off by 2^-24 of the running sum of
magnitudes if every rounding went the same way ((7168 + 2048) 2^-24 < 2^-10 of A in the worst order;
pairwise over warps, lanes and MMA blocks the depth is below 2^9 additions, 2^9 * 2^-24 = 2^-15), and
the fast exponential and division in silu (a few 2^-23).  Values near the end of fp32's range add an
absolute term: silu(g) = g / (1 + e^-g) is flushed to zero once 1 + e^-g > 2^126 (the fast division's
documented range), that is for g < -87.3, where |g| e^g < 88 * 2^-126 < 2^-119; so h = silu(g) v is off
by at most 2^-119 |v| there, y by 2^-119 F with F = sum_j |w_j| (|v_j| . |w2_j|^T) + |v_s| . |w2_s|^T, and
bf16's own smallest step below 2^-126 is 2^-133.  In norm, two independent roundings give at
most sqrt(2) * 2^-8 / sqrt(3) < 2^-8 relative to the parts they round; 2^-8 of |y| + |y's h part|.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
from mixture_experts_routing_gate_b200 import build as B
from mixture_experts_routing_gate_b200 import workloads as W
from parity import compare_routing, np64, oracle_gate_of

pytestmark = pytest.mark.gpu

TINY = W.CONFIGS["tiny"]
V3 = W.CONFIGS["v3_decode"]


@pytest.fixture(scope="module")
def M():
    B.build()
    from mixture_experts_routing_gate_b200 import moe
    return moe


def _layer(cfg, mxfp4=False):
    li = W.make_layer(cfg, device="cuda", bf16_experts=not mxfp4)
    w4 = W.make_mxfp4_weights(cfg, device="cuda") if mxfp4 else None
    return li, w4


def _decode(M, cfg, li, w4, ws=None, table=None, ids=None, stream=None, outs=None):
    desc = M.layer_desc(cfg)
    T = li.x.shape[0]
    ws = ws or M.Workspace(desc, T)
    y = torch.full_like(li.x, float("nan"))
    w = torch.full((T, cfg.topk), -1.0, dtype=torch.float32, device="cuda")
    idx = torch.full((T, cfg.topk), -1, dtype=torch.int32, device="cuda")
    cnt = torch.full((cfg.n_experts,), -1, dtype=torch.int32, device="cuda")
    kw = dict(bias=li.bias, logit_offset=li.logit_offset, token_ids=ids, tid2eid=table, weights_out=w, indices_out=idx,
              counts_out=cnt, stream=stream)
    if w4 is not None:
        M.moe_decode_mxfp4(desc, li.x, li.w_gate, w4, y, ws, **kw)
    else:
        M.moe_decode(desc, li.x, li.w_gate, li.w1, li.w3, li.w2, y, ws, **kw)
    return y, w, idx, cnt, ws


def _weights64(li, w4, e):
    if w4 is None:
        return li.w1[e].double(), li.w3[e].double(), li.w2[e].double()
    f = lambda c, s: torch.from_numpy(O.mxfp4_dequant(c[e].cpu().numpy(), s[e].cpu().numpy())).double().cuda()
    return f(w4.w1, w4.w1s), f(w4.w3, w4.w3s), f(w4.w2, w4.w2s)


def _reference(cfg, li, w4, idx, w):
    """(y, A, F) in fp64 for the given experts and weights."""
    x = li.x.double()
    y = torch.zeros_like(x)
    A = torch.zeros_like(x)
    F = torch.zeros_like(x)

    def add(e, rows, scale):
        w1, w3, w2 = _weights64(li, w4, e)
        g, v = x[rows] @ w1.t(), x[rows] @ w3.t()
        if cfg.swiglu_limit > 0:
            g, v = g.clamp(max=cfg.swiglu_limit), v.clamp(-cfg.swiglu_limit, cfg.swiglu_limit)
        h = g * torch.sigmoid(g) * v
        y[rows] += (h @ w2.t()) * scale
        A[rows] += (h.abs() @ w2.abs().t()) * scale.abs()
        F[rows] += (v.abs() @ w2.abs().t()) * scale.abs()

    T = x.shape[0]
    add(cfg.n_experts, list(range(T)), torch.ones((T, 1), dtype=torch.float64, device="cuda"))
    idx = idx.tolist()
    for e in sorted({e for row in idx for e in row}):
        rows = [t for t in range(T) if e in idx[t]]
        scale = [sum(float(w[t, j]) for j in range(cfg.topk) if idx[t][j] == e) for t in rows]
        add(e, rows, torch.tensor(scale, dtype=torch.float64, device="cuda")[:, None])
    return y, A, F


def _check(M, cfg, li, w4, y, w, idx, cnt, ws):
    M.check_device_errors(ws, "moe_decode")
    ref, A, F = _reference(cfg, li, w4, idx, w.double())
    err = (y.double() - ref).abs()
    lim = 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8) + (2.0 ** -8 + 2.0 ** -14) * A + 2.0 ** -119 * F + 2.0 ** -133
    assert bool((err <= lim).all()), f"max err / limit {float((err / lim).max())}"
    part = float((ref.norm() ** 2 + (2.0 ** -8 * A).norm() ** 2) ** 0.5)
    assert float(err.norm()) <= 2.0 ** -8 * part, float(err.norm()) / part
    assert np.array_equal(cnt.cpu().numpy(), np.bincount(idx.cpu().numpy().reshape(-1), minlength=cfg.n_experts))


def _check_gated(M, cfg, li, w4=None, ws=None):
    y, w, idx, cnt, ws = _decode(M, cfg, li, w4, ws)
    g = oracle_gate_of(cfg, li.x, li.w_gate, li.bias, li.logit_offset)
    compare_routing(cfg, g, idx.cpu().numpy(), w.cpu().numpy(), None if li.bias is None else li.bias.cpu().numpy())
    _check(M, cfg, li, w4, y, w, idx, cnt, ws)


CASES = {
    "smallest": TINY.replace(T=1, dim=128, n_experts=16, n_groups=1, n_limited_groups=1, topk=1, inter_dim=128),
    "tiny_1": TINY.replace(T=1), "tiny_2": TINY.replace(T=2), "tiny_3": TINY.replace(T=3), "tiny_7": TINY.replace(T=7),
    "tiny_8": TINY.replace(T=8), "tiny_9": TINY.replace(T=9), "tiny_16": TINY.replace(T=16),
    # last k chunk of 128 in the up projection, of 384 in the down projection
    "tails": TINY.replace(T=5, dim=640, inter_dim=384),
    "tails_16": TINY.replace(T=16, dim=1664, inter_dim=896, n_groups=1, n_limited_groups=1, topk=8),
    # more stages of k in a tile than the weight ring holds, in the up and in the down projection
    "long_up": TINY.replace(T=2, dim=8192 + 128, n_groups=1, n_limited_groups=1, topk=8),
    "long_down": TINY.replace(T=2, inter_dim=8192 + 640, n_groups=1, n_limited_groups=1, topk=8),
    # every token on the same few experts: rows of one expert up to T
    "crowded": TINY.replace(T=16, n_groups=1, n_limited_groups=1, topk=8, logit_offset_std=30.0, bias_std=None),
    "no_bias_groups": TINY.replace(T=11, bias_std=None),
    "softmax": TINY.replace(T=6, score_func="softmax", bias_std=None, route_scale=2.0),
    "sqrtsoftplus": TINY.replace(T=6, score_func="sqrtsoftplus", gate_general_fp32=False),
    "e48_groups_3": TINY.replace(T=4, n_experts=48, n_groups=3, n_limited_groups=2, topk=5),
    "e80": TINY.replace(T=4, n_experts=80, n_groups=1, n_limited_groups=1, topk=8),
    "groups_16": V3.replace(T=13, dim=512, inter_dim=256, n_groups=16, n_limited_groups=5),
    "groups_32": TINY.replace(T=13, n_experts=256, n_groups=32, n_limited_groups=9, topk=8),
    "one_group_kept": TINY.replace(T=16, n_experts=64, n_groups=8, n_limited_groups=1, topk=8),
    "e512_k8": TINY.replace(T=16, n_experts=512, n_groups=8, n_limited_groups=4, topk=8, dim=512),
    "offset_384": W.CONFIGS["v4_skew"].replace(T=10, dim=512, inter_dim=256),
    "clamp_inside": TINY.replace(T=9, swiglu_limit=0.05, weight_in_expert=True, route_scale=2.5, w_std=0.1),
}


@pytest.mark.parametrize("name", list(CASES))
def test_decode_bf16(M, name):
    cfg = CASES[name]
    _check_gated(M, cfg, _layer(cfg)[0])


MX_CASES = {
    "mx_1": TINY.replace(T=1, dim=512, inter_dim=512), "mx_8": TINY.replace(T=8, dim=1024, inter_dim=512),
    "mx_16": TINY.replace(T=16, dim=1536, inter_dim=1024, topk=4),
    "mx_crowded": TINY.replace(T=16, dim=512, inter_dim=512, n_groups=1, n_limited_groups=1, topk=8, logit_offset_std=30.0,
                               bias_std=None),
    "mx_long": TINY.replace(T=3, dim=20480, inter_dim=512, topk=2),
    "mx_clamp_inside": TINY.replace(T=9, dim=512, inter_dim=1536, swiglu_limit=0.05, weight_in_expert=True, w_std=0.1),
}


@pytest.mark.parametrize("name", list(MX_CASES))
def test_decode_mxfp4(M, name):
    cfg = MX_CASES[name]
    li, w4 = _layer(cfg, mxfp4=True)
    _check_gated(M, cfg, li, w4)


def test_decode_mxfp4_every_code_and_scale(M):
    # one-hot tokens pick single columns of w1 / w3; scales over their whole range in w2 (the sum stays
    # finite in fp32: codes up to 6, h around 1, scales up to 2^100), each output row one block scale
    cfg = TINY.replace(T=4, dim=512, inter_dim=512, n_groups=1, n_limited_groups=1, topk=1)
    li, w4 = _layer(cfg, mxfp4=True)
    byte = torch.arange(256, dtype=torch.uint8, device="cuda")
    w4.w1[:, :, :] = byte.repeat(cfg.dim // 2 // 256 * cfg.inter_dim).view(cfg.inter_dim, cfg.dim // 2)
    w4.w1s.fill_(127)
    rows = torch.arange(cfg.dim, device="cuda")
    w4.w2s[:, :, :] = (2 + rows % 226).to(torch.uint8)[None, :, None]
    _check_gated(M, cfg, li, w4)


def _hash_case(M, cfg, vocab, seed, duplicates):
    rng = np.random.default_rng(seed)
    table = np.stack([rng.choice(cfg.n_experts, size=cfg.topk, replace=duplicates) for _ in range(vocab)]).astype(np.int32)
    if duplicates:
        table[::3] = table[::3, :1]     # rows that name one expert k times
    ids = rng.integers(0, vocab, cfg.T).astype(np.int32)
    return table, ids


@pytest.mark.parametrize("mxfp4", [False, True])
@pytest.mark.parametrize("inside", [False, True])
@pytest.mark.parametrize("duplicates", [False, True])
def test_decode_hash(M, duplicates, inside, mxfp4):
    cfg = TINY.replace(T=16, dim=512, inter_dim=512, n_groups=1, n_limited_groups=1, topk=6, bias_std=None,
                       weight_in_expert=inside)
    li, w4 = _layer(cfg, mxfp4)
    table, ids = _hash_case(M, cfg, 50, 3, duplicates)
    y, w, idx, cnt, ws = _decode(M, cfg, li, w4, table=torch.from_numpy(table).cuda(), ids=torch.from_numpy(ids).cuda())
    i_ora, w_ora = O.hash_gate(ids, table, np64(li.x), np64(li.w_gate), cfg.route_scale)
    assert np.array_equal(idx.cpu().numpy(), i_ora)
    np.testing.assert_allclose(w.cpu().numpy(), w_ora, rtol=2e-5, atol=2e-6)
    _check(M, cfg, li, w4, y, w, idx, cnt, ws)


def test_decode_flags_bad_ids_and_scales(M):
    cfg = TINY.replace(T=3, dim=512, inter_dim=512, n_groups=1, n_limited_groups=1, topk=2, bias_std=None)
    li, w4 = _layer(cfg, mxfp4=True)
    table = torch.zeros((10, 2), dtype=torch.int32, device="cuda")
    table[:, 1] = 5
    good = torch.tensor([0, 9, 4], dtype=torch.int32, device="cuda")
    ws = _decode(M, cfg, li, w4, table=table, ids=good)[4]
    assert M.moe_get_error(ws) == (M.MOE_OK, 0)
    _decode(M, cfg, li, w4, ws, table, torch.tensor([0, 17, 4], dtype=torch.int32, device="cuda"))
    assert M.moe_get_error(ws) == (M.MOE_ERR_DEVICE, 17)
    table[4, 1] = -2
    _decode(M, cfg, li, w4, ws, table, good)
    assert M.moe_get_error(ws) == (M.MOE_ERR_DEVICE, -2)
    table[4, 1] = 5
    w4.w2s[5, 77, 3] = 255
    _decode(M, cfg, li, w4, ws, table, good)
    assert M.moe_get_error(ws) == (M.MOE_ERR_DEVICE, 0x10000 + 255)
    w4.w2s[5, 77, 3] = 120
    y, w, idx, cnt, ws = _decode(M, cfg, li, w4, ws, table, good)
    _check(M, cfg, li, w4, y, w, idx, cnt, ws)


@pytest.mark.parametrize("T", [1, 2, 3, 16])
def test_decode_flags_the_bad_id_of_any_token(M, T):
    cfg = TINY.replace(T=T, n_groups=1, n_limited_groups=1, topk=2, bias_std=None)
    li, _ = _layer(cfg)
    table = torch.tensor([[0, 3], [9, 1]], dtype=torch.int32, device="cuda")
    ws = M.Workspace(M.layer_desc(cfg), T)
    for t in range(T):
        ids = torch.ones(T, dtype=torch.int32, device="cuda")
        ids[t] = 1000 + t
        idx = _decode(M, cfg, li, None, ws, table, ids)[2]
        assert M.moe_get_error(ws) == (M.MOE_ERR_DEVICE, 1000 + t)
        assert idx.tolist() == [[9, 1]] * T      # clamped to the last row
    bad = torch.tensor([[0, 3], [16, -1]], dtype=torch.int32, device="cuda")
    idx = _decode(M, cfg, li, None, ws, bad, torch.ones(T, dtype=torch.int32, device="cuda"))[2]
    st, info = M.moe_get_error(ws)
    assert st == M.MOE_ERR_DEVICE and info in (16, -1)
    assert idx.tolist() == [[15, 0]] * T


def test_decode_not_a_number_stays_in_its_token(M):
    cfg = TINY.replace(T=5)
    li, _ = _layer(cfg)
    want = _decode(M, cfg, li, None)[0]
    li.x[2, 17] = float("nan")
    li.x[4, 3] = float("inf")
    y, w, idx, cnt, ws = _decode(M, cfg, li, None)
    M.check_device_errors(ws)
    assert bool((idx >= 0).all()) and bool((idx < cfg.n_experts).all())
    for t in (0, 1, 3):
        assert torch.equal(y[t], want[t])
    assert bool(torch.isnan(y[2]).all())


@pytest.mark.parametrize("mxfp4", [False, True])
def test_decode_together_with_the_other_entry_points(M, mxfp4):
    # a serving program's mix on one workspace: a prompt through moe_forward, then decode steps of
    # falling batch size, then the stages again; every result as from a fresh workspace
    cfg = TINY.replace(T=64, dim=512, inter_dim=512)
    li, w4 = _layer(cfg, mxfp4)
    desc = M.layer_desc(cfg)
    ws = M.Workspace(desc, 64)

    def forward(space):
        y = torch.empty_like(li.x)
        if mxfp4:
            M.moe_forward_mxfp4(desc, li.x, li.w_gate, w4, y, space, bias=li.bias)
        else:
            M.moe_forward(desc, li.x, li.w_gate, li.w1, li.w3, li.w2, y, space, bias=li.bias)
        return y

    first = forward(ws)
    import dataclasses
    for T in (16, 9, 8, 3, 1, 16):
        part = dataclasses.replace(li, x=li.x[:T].contiguous())
        c = cfg.replace(T=T)
        y = _decode(M, c, part, w4, ws)[0]
        assert torch.equal(y, _decode(M, c, part, w4)[0])
        _check_gated(M, c, part, w4, ws)
        if not mxfp4:   # the same layer: both within the layer's output bar of each other
            rms = float(first.float().pow(2).mean().sqrt())
            assert float((y.float() - first[:T].float()).abs().max()) <= 4e-2 * rms
    assert torch.equal(forward(ws), first)
    M.check_device_errors(ws)


def test_decode_repeats_bit_identically_and_leaves_neighbours(M):
    cfg = V3.replace(T=7, dim=1024, inter_dim=512)
    li, _ = _layer(cfg)
    desc = M.layer_desc(cfg)
    ws = M.Workspace(desc, 7)
    buf = torch.full((9, cfg.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[1:8]
    want = _decode(M, cfg, li, None)[0]
    for i in range(300):
        M.moe_decode(desc, li.x, li.w_gate, li.w1, li.w3, li.w2, y, ws, bias=li.bias)
        if i % 60 == 0 or i == 299:
            assert torch.equal(y, want)
    assert bool((buf[0] == 7.0).all()) and bool((buf[8] == 7.0).all())
    M.check_device_errors(ws)


def test_decode_in_a_graph_and_on_two_streams(M):
    import dataclasses
    cfg = TINY.replace(T=6, dim=512, inter_dim=256)
    li, _ = _layer(cfg)
    desc = M.layer_desc(cfg)
    xs = [W.normal_bf16((6, cfg.dim), 1.0, 50 + i, W.TID_X, device="cuda") for i in range(4)]
    want = [_decode(M, cfg, dataclasses.replace(li, x=x), None)[0] for x in xs]
    torch.cuda.synchronize()

    # captured once, replayed on new inputs in the same buffers; two graphs share the workspace
    ws, x, y = M.Workspace(desc, 6), xs[0].clone(), torch.empty_like(xs[0])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                M.moe_decode(desc, x, li.w_gate, li.w1, li.w3, li.w2, y, ws, bias=li.bias)
        graphs.append(g)
    for i, src in enumerate(xs):
        x.copy_(src)
        graphs[i % 2].replay()
        assert torch.equal(y, want[i])

    # two streams at once, a workspace each
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [M.Workspace(desc, 6) for _ in range(2)]
    outs = [[torch.empty_like(y) for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for s in range(2):
            M.moe_decode(desc, xs[(i + s) % 4], li.w_gate, li.w1, li.w3, li.w2, outs[s][i], spaces[s], bias=li.bias,
                         stream=streams[s])
    torch.cuda.synchronize()
    for s in range(2):
        for i in range(20):
            assert torch.equal(outs[s][i], want[(i + s) % 4])
        M.check_device_errors(spaces[s])


def test_decode_of_no_tokens(M):
    cfg = TINY.replace(T=4)
    li, _ = _layer(cfg)
    desc = M.layer_desc(cfg)
    cnt = torch.full((cfg.n_experts,), 9, dtype=torch.int32, device="cuda")
    x = li.x[:0]
    M.moe_decode(desc, x, li.w_gate, li.w1, li.w3, li.w2, torch.empty_like(x), M.Workspace(desc, 0), counts_out=cnt)
    assert int(cnt.abs().sum()) == 0


def test_decode_binding_refusals(M):
    cfg = TINY.replace(T=4)
    li, _ = _layer(cfg)
    desc = M.layer_desc(cfg)
    ws = M.Workspace(desc, 4)
    y = torch.empty_like(li.x)
    call = lambda **kw: M.moe_decode(*({"desc": desc, "x": li.x, "w_gate": li.w_gate, "w1": li.w1, "w3": li.w3, "w2": li.w2,
                                        "y": y, "ws": ws} | {k: v for k, v in kw.items() if k in ("x", "w_gate", "w1", "w2", "y", "ws")}).values(),
                                     **{k: v for k, v in kw.items() if k not in ("x", "w_gate", "w1", "w2", "y", "ws")})
    call()
    for bad in (dict(x=li.x.float()), dict(x=li.x[:, :128]), dict(y=y[:3]), dict(w1=li.w1[:-1]), dict(w2=li.w1),
                dict(w_gate=li.w_gate.t()), dict(bias=li.bias[:8]), dict(x=li.x.cpu()),
                dict(counts_out=torch.empty(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(M.MoeError):
        call(ws=M.Workspace(desc, 1))
    big = TINY.replace(T=17)
    l17, _ = _layer(big)
    with pytest.raises(M.MoeError) as e:
        M.moe_decode(desc, l17.x, l17.w_gate, l17.w1, l17.w3, l17.w2, torch.empty_like(l17.x), M.Workspace(desc, 17))
    assert e.value.status == M.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("mxfp4", [False, True])
def test_decode_stall_times_out_and_the_workspace_recovers(M, monkeypatch, mxfp4):
    # the test build's producers issue no loads: every wait runs out, the kernel returns and its
    # counters are back at zero, so that the same workspace serves the next call
    hooks = M.load_library(B.build(test_hooks=True))
    hooks.moe_test_set_stall.argtypes = [ctypes.c_int]
    hooks.moe_test_set_stall.restype = None
    cfg = TINY.replace(T=4, dim=512, inter_dim=512)
    li, w4 = _layer(cfg, mxfp4)
    with monkeypatch.context() as m:
        m.setattr(M, "lib", hooks)
        ws = M.Workspace(M.layer_desc(cfg), 4)
        hooks.moe_test_set_stall(1)
        try:
            _decode(M, cfg, li, w4, ws)
            st, info = M.moe_get_error(ws)
        finally:
            hooks.moe_test_set_stall(0)
        assert st == M.MOE_ERR_TIMEOUT and 400 <= info <= 410, (st, info)
        _check_gated(M, cfg, li, w4, ws)


@pytest.mark.parametrize("mxfp4", [False, True])
@pytest.mark.parametrize("T", [2, 16])
@pytest.mark.parametrize("stall", [2, 3, 4])
def test_decode_waits_given_up_midway(M, monkeypatch, stall, T, mxfp4):
    # the test build: the lists never come (2), or the copies end in the middle of a tile, in every CTA (3) or in
    # the first alone (4).  The call ends with a timeout and writes its outputs at most; the next ones are right
    hooks = M.load_library(B.build(test_hooks=True))
    hooks.moe_test_set_stall.argtypes = [ctypes.c_int]
    hooks.moe_test_set_stall.restype = None
    cfg = TINY.replace(T=T, dim=8192, inter_dim=1024)
    li, w4 = _layer(cfg, mxfp4)
    with monkeypatch.context() as m:
        m.setattr(M, "lib", hooks)
        desc = M.layer_desc(cfg)
        ws = M.Workspace(desc, T)
        behind = ws.buf[ws.tensor.data_ptr() - ws.buf.data_ptr() + ws.nbytes:]
        behind.fill_(165)
        buf = torch.full((T + 2, cfg.dim), 7.0, dtype=torch.bfloat16, device="cuda")
        y = buf[1:T + 1]
        weights = (w4,) if mxfp4 else (li.w1, li.w3, li.w2)
        call = M.moe_decode_mxfp4 if mxfp4 else M.moe_decode
        hooks.moe_test_set_stall(stall)
        try:
            call(desc, li.x, li.w_gate, *weights, y, ws, bias=li.bias)
            st, info = M.moe_get_error(ws)
        finally:
            hooks.moe_test_set_stall(0)
        assert st == M.MOE_ERR_TIMEOUT and 400 <= info <= 411, (st, info)
        assert bool((buf[0] == 7.0).all()) and bool((buf[T + 1] == 7.0).all()) and bool((behind == 165).all())
        assert int(ws.tensor[:4096].count_nonzero()) == 0    # the control words of the next call
        for _ in range(2):
            _check_gated(M, cfg, li, w4, ws)


@pytest.mark.parametrize("T", [1, 16])
def test_decode_leaves_the_control_words_at_zero(M, T):
    # calls one after another on one workspace find the grid's counters at zero, and so does what follows
    cfg = TINY.replace(T=T, n_experts=64, inter_dim=512)
    li, _ = _layer(cfg)
    desc = M.layer_desc(cfg)
    ws = M.Workspace(desc, T)
    y = torch.empty_like(li.x)
    left = torch.zeros(400, dtype=torch.int64, device="cuda")
    for i in range(400):
        M.moe_decode(desc, li.x, li.w_gate, li.w1, li.w3, li.w2, y, ws, bias=li.bias)
        left[i] = ws.tensor[:4096].count_nonzero()
    assert int(left.sum()) == 0
    _check_gated(M, cfg, li, None, ws)


@pytest.mark.parametrize("mxfp4", [False, True])
def test_decode_on_the_workspace_of_a_larger_batch(M, mxfp4):
    import dataclasses
    cfg = TINY.replace(T=17, dim=512, inter_dim=512)
    li, w4 = _layer(cfg, mxfp4)
    ws = M.Workspace(M.layer_desc(cfg), 17)
    for T in (16, 1):
        part = dataclasses.replace(li, x=li.x[:T].contiguous())
        _check_gated(M, cfg.replace(T=T), part, w4, ws)


# The precision of h, where y's own rounding does not hide it: features in pairs whose values are almost alike and
# whose w2 columns are opposite, so that y is small beside what it is a sum of.  The roundings of h are independent
# of each other, each below u |h| (u = 2^-16 for two bf16 parts, 2^-11 for f16; one bf16 would be off by 2^-9.3 in the
# mean square), so in norm their sum is below u B, B^2 = sum_j w_j^2 (h_j^2 . (w2_j^T)^2) + h_s^2 . (w2_s^T)^2.  y is
# rounded once more, 2^-8 |y|, and the fp32 sums and the fast exponential leave 2^-17 A as a worst case: sums of up
# to 2^6 additions a lane, truncated by up to 2^-23 each.
@pytest.mark.parametrize("mxfp4", [False, True])
@pytest.mark.parametrize("T,dim,inter", [(1, 512, 512), (3, 1024, 512), (7, 512, 1024), (16, 512, 512), (1, 2048, 2048), (6, 2048, 2048),
                                         (16, 2048, 2048)])
def test_decode_holds_h_to_more_than_bf16(M, T, dim, inter, mxfp4):
    cfg = TINY.replace(T=T, dim=dim, inter_dim=inter)
    li, w4 = _layer(cfg, mxfp4)
    if mxfp4:
        for name in ("w1", "w1s", "w3", "w3s"):
            t = getattr(w4, name)
            t[:, 1::2] = t[:, 0::2]
        w4.w3[:, 1::2, 5] ^= 1                                  # one code of the row
        w4.w2.copy_((w4.w2 & 0x0f) | ((w4.w2 & 0x0f) << 4) ^ 0x80)   # the second code of a byte: the first's opposite
    else:
        li.w1[:, 1::2] = li.w1[:, 0::2]
        li.w3[:, 1::2] = li.w3[:, 0::2] * (1 + 2.0 ** -6)
        li.w2[:, :, 1::2] = -li.w2[:, :, 0::2]
    y, w, idx, cnt, ws = _decode(M, cfg, li, w4)
    M.check_device_errors(ws, "moe_decode")
    ref, A, _ = _reference(cfg, li, w4, idx, w.double())
    B2 = torch.zeros_like(ref)
    x = li.x.double()
    for e in sorted({e for row in idx.tolist() for e in row} | {cfg.n_experts}):
        w1, w3, w2 = _weights64(li, w4, e)
        scale = torch.tensor([1.0 if e == cfg.n_experts else sum(float(w[t, j]) for j in range(cfg.topk) if idx[t, j] == e)
                              for t in range(T)], dtype=torch.float64, device="cuda")[:, None]
        g = x @ w1.t()
        B2 += scale ** 2 * ((g * torch.sigmoid(g) * (x @ w3.t())) ** 2 @ (w2 ** 2).t())
    u = 2.0 ** -11 if mxfp4 else 2.0 ** -16
    err = float((y.double() - ref).norm())
    lim = u * float(B2.sqrt().norm()) + 2.0 ** -8 * float(ref.norm()) + 2.0 ** -17 * float(A.norm())
    assert lim < 2.0 ** -10 * float(B2.sqrt().norm())    # else the case would not tell
    assert err <= lim, err / lim


def test_decode_mxfp4_spread_inside_a_block_of_x(M):
    # x in f16 blocks of 32 is exact down to 2^-31 of the block's largest value; a value of that size is all that the
    # weights see of its block here (the largest one meets zero codes)
    cfg = TINY.replace(T=2, dim=512, inter_dim=512, n_groups=1, n_limited_groups=1, topk=1)
    li, w4 = _layer(cfg, mxfp4=True)
    li.x[:] = 0
    li.x[:, 64] = 1.0
    li.x[0, 65], li.x[1, 95] = 2.0 ** -31 * (255 / 128), -2.0 ** -31
    for name in ("w1", "w3"):
        getattr(w4, name)[:] = 0
        getattr(w4, name)[:, :, 32] = 0x70      # column 65: 6
        getattr(w4, name)[:, :, 47] = 0x50      # column 95: 3
        getattr(w4, name + "s").fill_(127 + 25)
    _check_gated(M, cfg, li, w4)


def test_decode_mxfp4_scales_of_the_up_projections(M):
    # w1's and w3's scales over 200 powers of two, opposite to each other so that h stays in range
    cfg = TINY.replace(T=3, dim=512, inter_dim=1024, n_groups=1, n_limited_groups=1, topk=2)
    li, w4 = _layer(cfg, mxfp4=True)
    r = (torch.arange(cfg.inter_dim, device="cuda") // 32 * 7 % 200 - 100)[None, :, None]
    w4.w1s[:] = (127 + r).to(torch.uint8)
    w4.w3s[:] = (127 - r).to(torch.uint8)
    _check_gated(M, cfg, li, w4)


@pytest.mark.parametrize("mxfp4", [False, True])
def test_decode_infinity_and_nan_stay_in_their_token(M, mxfp4):
    # every expert for every token, so that routing (and with it the order of sums) cannot differ
    cfg = TINY.replace(T=5, dim=512, inter_dim=512, n_groups=1, n_limited_groups=1, topk=4, bias_std=None)
    li, w4 = _layer(cfg, mxfp4)
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None].contiguous()
    ids = torch.zeros(5, dtype=torch.int32, device="cuda")
    want = _decode(M, cfg, li, w4, table=table, ids=ids)[0]
    li.x[1, 40], li.x[3, 500] = float("inf"), float("nan")
    y, _, _, _, ws = _decode(M, cfg, li, w4, table=table, ids=ids)
    M.check_device_errors(ws)
    for t in (0, 2, 4):
        assert torch.equal(y[t], want[t])
    assert not bool(torch.isfinite(y[1]).any()) and bool(torch.isnan(y[3]).all())


@pytest.mark.parametrize("groups", [1, 4])
def test_decode_with_experts_switched_off_by_their_bias(M, groups):
    cfg = TINY.replace(T=16, n_groups=groups, n_limited_groups=min(groups, 2), topk=3)
    li, _ = _layer(cfg)
    off = torch.tensor([0, 5, 6, 9, 15], device="cuda")
    li.bias[off] = float("-inf")
    y, w, idx, cnt, ws = _decode(M, cfg, li, None)
    assert not bool(torch.isin(idx, off.to(torch.int32)).any())
    _check(M, cfg, li, None, y, w, idx, cnt, ws)
    if groups == 1:      # as with a bias below every other
        li.bias[off] = -1e4
        again = _decode(M, cfg, li, None)
        assert torch.equal(again[2], idx) and torch.equal(again[0], y)


def test_decode_results_do_not_depend_on_the_batch(M):
    # one token alone, among 7 and among 16 on the same experts: the same bits, whichever columns h's parts take
    import dataclasses
    cfg = TINY.replace(T=16, dim=512, inter_dim=1024, n_groups=1, n_limited_groups=1, topk=4, bias_std=None)
    li, _ = _layer(cfg)
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None].contiguous()
    ys = []
    for T in (16, 8, 7, 4, 2, 1):
        part = dataclasses.replace(li, x=li.x[:T].contiguous())
        ys.append(_decode(M, cfg.replace(T=T), part, None, table=table, ids=torch.zeros(T, dtype=torch.int32, device="cuda"))[0])
    for y in ys:
        assert torch.equal(y[:1], ys[0][:1])
        assert torch.equal(y, ys[0][:len(y)])
