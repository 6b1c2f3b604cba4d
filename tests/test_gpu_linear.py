"""moe_linear against y = act(x w^T + bias) + residual in 64 bits.

Tolerance, before any run.  With A = |x| |w|^T the fp32 sum of K products is off by at most a few 2^-24 of
A for each of the additions on its longest chain; the chains here are at most K / 8 + 64 long (lanes,
warps and MMA steps add in parallel), and roundings to nearest of random sign grow with the root of
that, so 2^-24 * 4 sqrt(K) * A bounds them with room to spare; truncating accumulators (one-sided) are
covered by adding K * 2^-27 * A.  bias, activation and residual are a handful of fp32 operations on values
below |z| + |bias| + |r| (an activation's slope is below 1.13, its fast exponential good to 2^-21 of the
result for |z| < 16): 2^-20 of each.  bf16 outputs add half a step, 2^-8 |y|.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from mixture_experts_routing_gate_b200 import build as B
from mixture_experts_routing_gate_b200 import workloads as W

pytestmark = pytest.mark.gpu
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module")
def M():
    B.build()
    from mixture_experts_routing_gate_b200 import moe
    return moe


def _normal(shape, std, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _act64(z, act):
    return {"none": lambda v: v, "relu": lambda v: torch.where(v < 0, 0.0, v), "silu": lambda v: v * torch.sigmoid(v),
            "gelu": lambda v: 0.5 * v * torch.erfc(-v / math.sqrt(2)),
            "gelu_tanh": lambda v: v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))}[act](z)


def _check(y, x, w, act, bias, residual):
    K = x.shape[1]
    x64, w64 = x.double(), w.double()
    z = x64 @ w64.t()
    A = x64.abs() @ w64.abs().t()
    b = torch.zeros(w.shape[0], dtype=torch.float64, device="cuda") if bias is None else bias.double()
    r = torch.zeros_like(z) if residual is None else residual.double()
    want = _act64(z + b, act) + r
    lim = 1.13 * 2.0 ** -24 * (4 * math.sqrt(K) + K / 8) * A + 2.0 ** -20 * (z.abs() + b.abs() + r.abs()) + 2.0 ** -126
    if y.dtype == torch.bfloat16:
        lim = lim * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    err = (y.double() - want).abs()
    assert bool((err <= lim).all()), f"max err / limit {float((err / lim).max())} at {int((err / lim).argmax())} of {tuple(y.shape)}"


def _run(M, T, K, N, act="none", bias=False, residual=False, out=torch.bfloat16, xpad=0, ypad=0, rpad=0, seed=1):
    x = _normal((T, K + xpad), 1.0, seed)[:, :K]
    w = _normal((N, K), 1.0 / math.sqrt(K), seed + 1)
    b = _normal((N,), 0.5, seed + 2, torch.float32) if bias else None
    r = _normal((T, N + rpad), 1.0, seed + 3)[:, :N] if residual else None
    whole = torch.full((T + 2, N + ypad), 77.0, dtype=out, device="cuda")
    y = whole[1:T + 1, :N]
    desc = M.linear_desc(K, N, act, out)
    ws = M.LinearWorkspace(desc, T)
    M.moe_linear(desc, x, w, y, ws, bias=b, residual=r)
    M.check_device_errors(ws, "moe_linear")
    _check(y, x, w, act, b, r)
    # the rows before and after, and what lies between the rows, are left as they were
    assert bool((whole[0] == 77.0).all()) and bool((whole[T + 1] == 77.0).all()) and bool((whole[:, N:] == 77.0).all())
    again = torch.empty_like(y)
    for _ in range(3):
        M.moe_linear(desc, x, w, again, ws, bias=b, residual=r)
        assert torch.equal(again, y)
    return x, w, b, r, y


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16])
@pytest.mark.parametrize("K,N", [(8, 1), (128, 64), (136, 65), (1000, 63), (7168, 512), (512, 7168), (2048, 129)])
def test_stream(M, T, K, N):
    _run(M, T, K, N, ACTS[(T + N) % 5], bias=T % 2 == 0, residual=N % 2 == 1, xpad=8 * (T % 3), ypad=T % 4)


@pytest.mark.parametrize("T", [1, 16])
def test_stream_with_a_full_ring_behind_every_tile(M, T):
    # each CTA's run crosses a tile's end while the weight ring is full behind it: warps that are late with
    # the next tile's first stage must still find it
    K = N = 7168
    x, w = _normal((T, K), 1.0, 3), _normal((N, K), 1.0 / math.sqrt(K), 4)
    desc = M.linear_desc(K, N, out_dtype=torch.float32)
    ws = M.LinearWorkspace(desc, T)
    outs = [torch.empty((T, N), dtype=torch.float32, device="cuda") for _ in range(60)]
    for y in outs:
        M.moe_linear(desc, x, w, y, ws)
    _check(outs[0], x, w, "none", None, None)
    assert all(torch.equal(y, outs[0]) for y in outs)


@pytest.mark.parametrize("T", [17, 33, 64, 127, 128, 129, 300, 513])
@pytest.mark.parametrize("K,N", [(8, 1), (64, 128), (72, 130), (1000, 255), (2048, 257), (512, 1536), (7168, 40)])
def test_tiles(M, T, K, N):
    _run(M, T, K, N, ACTS[(T + K) % 5], bias=T % 2 == 1, residual=N % 2 == 0, xpad=8 * (T % 3), ypad=T % 4, rpad=N % 3)


@pytest.mark.parametrize("T,K,N", [(2048, 512, 2048), (4096, 1024, 768), (1000, 256, 5000), (5000, 128, 700), (64, 512, 60000)])
def test_many_tiles(M, T, K, N):
    _run(M, T, K, N, "silu", bias=True, residual=True)


@pytest.mark.parametrize("T", [3, 100, 700])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_epilogues(M, T, act, out):
    for bias in (False, True):
        for residual in (False, True):
            _run(M, T, 264, 200, act, bias, residual, out, ypad=8, rpad=8)
            _run(M, T, 264, 201, act, bias, residual, out, ypad=2, rpad=3)


@pytest.mark.parametrize("T", [5, 40, 600])
def test_into_the_residual_itself(M, T):
    K, N = 512, 384
    x, w = _normal((T, K), 1.0, 3), _normal((N, K), 1.0 / math.sqrt(K), 4)
    y = _normal((T, N), 1.0, 5)
    r = y.clone()
    desc = M.linear_desc(K, N)
    M.moe_linear(desc, x, w, y, M.LinearWorkspace(desc, T), residual=y)
    _check(y, x, w, "none", None, r)


@pytest.mark.parametrize("T", [4, 50, 400])
def test_not_a_number_stays_in_its_row_and_column(M, T):
    K, N = 264, 320
    x, w = _normal((T, K), 1.0, 3), _normal((N, K), 1.0, 4)
    desc = M.linear_desc(K, N, "relu", torch.float32)
    ws = M.LinearWorkspace(desc, T)
    want, y = (torch.empty((T, N), dtype=torch.float32, device="cuda") for _ in range(2))
    M.moe_linear(desc, x, w, want, ws)
    x[2, 5] = float("nan")
    w[7, K - 1] = float("nan")
    M.moe_linear(desc, x, w, y, ws)
    keep = torch.ones((T, N), dtype=torch.bool, device="cuda")
    keep[2] = False
    keep[:, 7] = False
    assert torch.equal(y[keep], want[keep])
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[:, 7]).all())


def test_one_workspace_many_shapes_and_a_graph(M):
    # a decoder block's projections on one workspace, then captured and replayed on new inputs
    shapes = [(4, 512, 1536, "none"), (4, 1536, 512, "gelu"), (40, 512, 1536, "silu"), (300, 1536, 512, "relu"), (16, 512, 64, "none")]
    descs = [M.linear_desc(K, N, act) for _, K, N, act in shapes]
    ws = max((M.LinearWorkspace(d, s[0]) for d, s in zip(descs, shapes)), key=lambda w: w.nbytes)
    xs = [_normal((T, K), 1.0, 20 + i) for i, (T, K, _, _) in enumerate(shapes)]
    ww = [_normal((N, K), 1.0 / math.sqrt(K), 40 + i) for i, (_, K, N, _) in enumerate(shapes)]
    ys = [torch.empty((T, N), dtype=torch.bfloat16, device="cuda") for T, _, N, _ in shapes]

    def block():
        for d, x, w, y in zip(descs, xs, ww, ys):
            M.moe_linear(d, x, w, y, ws)

    block()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):   # two graphs sharing the workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            block()
        graphs.append(g)
    for r in range(4):
        for i, x in enumerate(xs):
            x.copy_(_normal(tuple(x.shape), 1.0, 100 + 10 * r + i))
        graphs[r % 2].replay()
        for (_, _, _, act), x, w, y in zip(shapes, xs, ww, ys):
            _check(y, x, w, act, None, None)
    M.check_device_errors(ws)


def test_two_streams_a_workspace_each(M):
    T, K, N = 200, 2048, 256      # few tiles: K is cut
    desc = M.linear_desc(K, N)
    x, w = _normal((T, K), 1.0, 3), _normal((N, K), 1.0 / math.sqrt(K), 4)
    want = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    M.moe_linear(desc, x, w, want, M.LinearWorkspace(desc, T))
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [M.LinearWorkspace(desc, T) for _ in range(2)]
    outs = [[torch.empty_like(want) for _ in range(30)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(30):
        for s in range(2):
            M.moe_linear(desc, x, w, outs[s][i], spaces[s], stream=streams[s])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for side in outs for o in side)


def test_no_tokens_and_binding_refusals(M):
    desc = M.linear_desc(64, 32)
    x, w = _normal((4, 64), 1.0, 1), _normal((32, 64), 1.0, 2)
    y = torch.empty((4, 32), dtype=torch.bfloat16, device="cuda")
    ws = M.LinearWorkspace(desc, 4)
    M.moe_linear(desc, x[:0], w, y[:0], ws)
    M.moe_linear(desc, x, w, y, ws)
    wide = _normal((4, 128), 1.0, 3)
    for bad in (dict(x=x.float()), dict(x=wide), dict(x=wide[:, ::2]), dict(w=w.t()), dict(w=w[:16]), dict(y=y.float()),
                dict(y=y[:3]), dict(y=y[:1].expand(4, 32)), dict(bias=torch.zeros(31, device="cuda")), dict(residual=y[:2]),
                dict(x=x.cpu())):
        a = {"x": x, "w": w, "y": y} | bad
        with pytest.raises(ValueError):
            M.moe_linear(desc, a["x"], a["w"], a["y"], ws, bias=a.get("bias"), residual=a.get("residual"))
    with pytest.raises(M.MoeError) as e:      # rows of x that do not start on 16 bytes
        M.moe_linear(desc, _normal((4, 68), 1.0, 1)[:, :64], w, y, ws)
    assert e.value.status == M.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("T", [4, 100, 700])
def test_stall_times_out_and_the_workspace_recovers(M, monkeypatch, T):
    hooks = M.load_library(B.build(test_hooks=True))
    hooks.moe_test_set_stall.argtypes = [ctypes.c_int]
    hooks.moe_test_set_stall.restype = None
    K, N = 1024, 300
    x, w = _normal((T, K), 1.0, 3), _normal((N, K), 1.0 / math.sqrt(K), 4)
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    with monkeypatch.context() as m:
        m.setattr(M, "lib", hooks)
        desc = M.linear_desc(K, N)
        ws = M.LinearWorkspace(desc, T)
        hooks.moe_test_set_stall(1)
        try:
            M.moe_linear(desc, x, w, y, ws)
            st, info = M.moe_get_error(ws)
        finally:
            hooks.moe_test_set_stall(0)
        assert st == M.MOE_ERR_TIMEOUT and 500 <= info <= 520, (st, info)
        M.moe_linear(desc, x, w, y, ws)
        M.check_device_errors(ws)
        _check(y, x, w, "none", None, None)


def test_decode_step_of_a_block(M):
    # the operators as they are used together: a projection into the residual stream, the layer on the
    # normalised stream, its result added by the next projection, logits of the head
    import dataclasses
    cfg = W.CONFIGS["tiny"].replace(T=5, dim=512, inter_dim=512)
    li = W.make_layer(cfg, device="cuda")
    T, d, V = 5, cfg.dim, 1000
    attn, wo = _normal((T, d), 1.0, 7), _normal((d, d), 1.0 / math.sqrt(d), 8)
    stream = _normal((T, d), 1.0, 9)
    head = _normal((V, d), 1.0 / math.sqrt(d), 10)
    to_d, to_v = M.linear_desc(d, d), M.linear_desc(d, V, out_dtype=torch.float32)
    wl, wd = M.LinearWorkspace(to_v, T), M.Workspace(M.layer_desc(cfg), T)
    r0 = stream.clone()
    M.moe_linear(to_d, attn, wo, stream, wl, residual=stream)
    _check(stream, attn, wo, "none", None, r0)
    x = (stream.float() * torch.rsqrt(stream.float().pow(2).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    M.moe_decode(M.layer_desc(cfg), x, li.w_gate, li.w1, li.w3, li.w2, y, wd, bias=li.bias)
    logits = torch.empty((T, V), dtype=torch.float32, device="cuda")
    M.moe_linear(to_v, y, head, logits, wl)
    _check(logits, y, head, "none", None, None)
    M.moe_forward(M.layer_desc(cfg), x, li.w_gate, li.w1, li.w3, li.w2, y2, wd, bias=li.bias)
    rms = float(y2.float().pow(2).mean().sqrt())
    assert float((y.float() - y2.float()).abs().max()) <= 4e-2 * rms
    M.check_device_errors(wd)
    M.check_device_errors(wl)


@pytest.mark.parametrize("T,K,N", [(3, 7168, 7168), (16, 7168, 7168), (20, 7168, 64), (100, 7168, 300), (700, 2048, 5000),
                                   (4096, 1024, 4096)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_waits_given_up_midway(M, monkeypatch, T, K, N, out):
    # the test build's producers stop inside a tile: the call ends with a timeout, writes y at most, and the
    # same workspace serves the next one
    hooks = M.load_library(B.build(test_hooks=True))
    hooks.moe_test_set_stall.argtypes = [ctypes.c_int]
    hooks.moe_test_set_stall.restype = None
    x, w = _normal((T, K), 1.0, 3), _normal((N, K), 1.0 / math.sqrt(K), 4)
    buf = torch.full((T + 2, N + 8), 7.0, dtype=out, device="cuda")
    y = buf[1:T + 1, :N]
    with monkeypatch.context() as m:
        m.setattr(M, "lib", hooks)
        desc = M.linear_desc(K, N, out_dtype=out)
        ws = M.LinearWorkspace(desc, T)
        hooks.moe_test_set_stall(3)
        try:
            M.moe_linear(desc, x, w, y, ws)
            st, info = M.moe_get_error(ws)
        finally:
            hooks.moe_test_set_stall(0)
        assert st == M.MOE_ERR_TIMEOUT and 500 <= info <= 520, (st, info)
        assert int(ws.tensor[:4096].count_nonzero()) == 0
        for _ in range(2):
            M.moe_linear(desc, x, w, y, ws)
            M.check_device_errors(ws)
            _check(y, x, w, "none", None, None)
        assert bool((buf[0] == 7.0).all()) and bool((buf[T + 1] == 7.0).all()) and bool((buf[:, N:] == 7.0).all())


def test_small_batches_on_the_workspace_of_a_large_one(M):
    K, N = 1024, 1032
    desc = M.linear_desc(K, N)
    ws = M.LinearWorkspace(desc, 300)
    w = _normal((N, K), 1.0 / math.sqrt(K), 4)
    for T in (1, 16, 17, 300, 1):
        x, y = _normal((T, K), 1.0, 3 + T), torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        M.moe_linear(desc, x, w, y, ws)
        M.check_device_errors(ws)
        _check(y, x, w, "none", None, None)


@pytest.mark.parametrize("T", [1, 9, 40, 300, 5000])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_fp32_outputs_take_the_accurate_exponential(M, T, act):
    # one-hot rows, so that z is exact: what remains is the activation.  expf is good to 2^-23, the sum and the
    # division round 2^-24 each: 2^-22.  gelu_tanh's exponent a has seven roundings of 2^-24 (no cancellation), which
    # e^a turns into 7 |a| 2^-24.  Where e^a passes fp32's range, 2^128, z / (1 + e^a) is zero instead of less than
    # |z| 2^-128 (a = 88.7 at z = -10.1, where that is 2.5 times the smallest normal number, 2^-126).
    K, N = 8, 512
    w = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    w[:, 3] = torch.linspace(-30.0, 30.0, N, device="cuda").to(torch.bfloat16)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    x[:, 3] = 1.0
    desc = M.linear_desc(K, N, act, torch.float32)
    y = torch.empty((T, N), dtype=torch.float32, device="cuda")
    M.moe_linear(desc, x, w, y, M.LinearWorkspace(desc, T))
    z = w[:, 3].double().expand(T, N)
    want = _act64(z, act)
    a = torch.zeros_like(z) if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    lim = (2.0 ** -22 + 7 * a.abs() * 2.0 ** -24) * want.abs() + 2.0 ** -126 + z.abs() * 2.0 ** -128
    assert bool(((y.double() - want).abs() <= lim).all())


@pytest.mark.parametrize("T", [1, 16, 33, 300])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_infinity_goes_through_as_in_the_formula(M, T, out):
    # an infinite product stays in its row; ReLU clears the negative one
    K, N = 64, 136
    x, w = _normal((T, K), 1.0, 3), _normal((N, K), 1.0, 4)
    want, y = (torch.empty((T, N), dtype=out, device="cuda") for _ in range(2))
    for act in ("none", "relu"):
        desc = M.linear_desc(K, N, act, out)
        ws = M.LinearWorkspace(desc, T)
        clean = x.clone()
        M.moe_linear(desc, clean, w, want, ws)
        clean[0, 7] = float("inf")
        M.moe_linear(desc, clean, w, y, ws)
        assert torch.equal(y[1:], want[1:])
        s = torch.sign(w[:, 7].float())
        first = torch.where(s > 0, float("inf"), 0.0 if act == "relu" else float("-inf"))
        assert torch.equal(y[0].float()[s != 0], first[s != 0]) and bool(y[0].isnan()[s == 0].all())
