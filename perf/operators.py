"""Timed cases of the serving operators: the MoE layer for a few tokens and the linear projection.

Two operators, each in a plain form (elementary torch operations in 32 bits, routing in 64) and as the
calls of the library's Python binding:

* ``layer``: one whole mixture-of-experts layer (gate, routed SwiGLU experts, combine, shared expert)
  for 1 to 16 tokens -- ``moe_decode`` (bf16 experts) and ``moe_decode_mxfp4`` (MXFP4 experts);
* ``linear``: y = act(x . w^T + bias) + residual for any number of tokens -- ``moe_linear``.

``own`` selects the form that ``run`` computes; the inputs are the same for both.
"""
import math
from types import SimpleNamespace

import numpy as np
import torch

own = False

# E2M1 magnitudes by code (bits 2-1 exponent, bit 0 mantissa; bit 3 is the sign)
FP4_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _layer(name, T, d, E, G, g, k, I, score, scale, bias, offset, vocab, w_std, mxfp4=False):
    return dict(name=name, op="layer", T=T, d=d, E=E, G=G, g=g, k=k, I=I, score=score, scale=scale, bias=bias,
                offset=offset, vocab=vocab, w_std=w_std, mxfp4=mxfp4)


def _linear(name, T, K, N, act="none", bias=False, residual=False, out="bf16", pad=0):
    return dict(name=name, op="linear", T=T, K=K, N=N, act=act, bias=bias, residual=residual, out=out, pad=pad)


def listed():
    return [
        # the smallest layer of the repository, one token: launch and synchronisation latency alone
        _layer("layer tiny T1", 1, 256, 16, 4, 2, 4, 128, "sigmoid", 1.0, True, False, 0, 0.02),
        # one sequence decoding through the 256-expert layer: nine experts' weights streamed
        _layer("layer v3 T1", 1, 7168, 256, 8, 4, 8, 2048, "sigmoid", 2.5, True, False, 0, 0.006),
        # four sequences on the hash-routed layer: experts from the token-id table
        _layer("layer hash T4", 4, 4096, 256, 1, 1, 6, 2048, "sigmoid", 1.0, False, False, 129280, 0.01),
        # a small serving batch on the layer whose experts are unevenly popular
        _layer("layer v4 T16", 16, 5120, 384, 1, 1, 6, 1536, "sqrtsoftplus", 1.5, True, True, 0, 0.01),
        # one and eight sequences with the experts held in 4 bits
        _layer("layer v3 mxfp4 T1", 1, 7168, 256, 8, 4, 8, 2048, "sigmoid", 2.5, True, False, 0, 0.006, True),
        _layer("layer v3 mxfp4 T8", 8, 7168, 256, 8, 4, 8, 2048, "sigmoid", 2.5, True, False, 0, 0.006, True),
        # a projection back into the residual stream for one token: a matrix-vector product
        _linear("linear T1 residual", 1, 7168, 7168, residual=True),
        # a ragged small batch, an odd number of features, rows of x inside wider rows
        _linear("linear T33 odd", 33, 4104, 1999, act="gelu", bias=True, residual=True, pad=56),
        # the output head over the vocabulary for a decode batch, logits in fp32
        _linear("linear head T64", 64, 7168, 129280, out="fp32"),
        # a dense up projection for a short prompt
        _linear("linear T300 silu", 300, 5120, 1536, act="silu", bias=True),
        # prefill: the widths of the 4096-token layer, and the largest batch of the repository
        _linear("linear T4096", 4096, 7168, 2048, act="gelu_tanh", bias=True),
        _linear("linear T16384", 16384, 5120, 5120, bias=True, residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        mxfp4 = rng.random() < 0.4
        step = 512 if mxfp4 else 128
        d = step * rng.randint(2 if not mxfp4 else 1, 7168 // step)
        I = step * rng.randint(1, 2048 // step)
        E = rng.choice([16, 32, 48, 64, 96, 128, 256, 384])
        while (E + 1) * d * I > 257 * 7168 * 2048:
            E //= 2
            E -= E % 16
        vocab = rng.choice([0, 0, 0, 1000, 129280])
        G = 1 if vocab else rng.choice([v for v in (1, 2, 4, 8, 16) if E % v == 0 and E // v >= 2])
        g = rng.randint(1, G)
        k = rng.randint(1, min(8, g * (E // G)))
        T = _log_int(rng, 1, 16)
        while T > 1 and T * k * d * I > 64 * 7168 * 2048:
            T -= 1
        score = "sigmoid" if vocab else rng.choice(["sigmoid", "sqrtsoftplus", "softmax"])
        bias = not vocab and score != "softmax" and rng.random() < 0.7
        return _layer("", T, d, E, G, g, k, I, score, rng.choice([1.0, 1.5, 2.5]), bias, not vocab and rng.random() < 0.3,
                      vocab, rng.choice([0.006, 0.01, 0.02]), mxfp4) | {"name": "drawn layer"}
    T, K, N = _log_int(rng, 1, 16384), 8 * _log_int(rng, 16, 896), _log_int(rng, 1, 129280)
    while T * K * N > 16384 * 5120 * 5120 or T * N > 16384 * 7168:
        if T > N:
            T = T * 2 // 3 + 1
        else:
            N = N * 2 // 3 + 1
    return _linear("drawn linear", T, K, N, rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), rng.random() < 0.5,
                   rng.random() < 0.4, rng.choice(["bf16", "bf16", "fp32"]), rng.choice([0, 0, 8, 136]))


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _normal(gen, shape, std, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = SimpleNamespace(**case)
    s = {"case": c}
    if c.op == "linear":
        s["x"] = _normal(gen, (c.T, c.K + c.pad), 1.0)[:, :c.K]
        s["w"] = _normal(gen, (c.N, c.K), 1.0 / math.sqrt(c.K))
        s["bias"] = _normal(gen, (c.N,), 0.5, torch.float32) if c.bias else None
        s["residual"] = _normal(gen, (c.T, c.N), 1.0) if c.residual else None
        return s
    s["x"] = _normal(gen, (c.T, c.d), 1.0)
    s["w_gate"] = _normal(gen, (c.E, c.d), c.w_std, torch.float32)
    s["bias"] = _normal(gen, (c.E,), 0.01, torch.float32) if c.bias else None
    s["offset"] = _normal(gen, (c.E,), 1.0, torch.float32) if c.offset else None
    if c.vocab:
        # k distinct experts for every token id; ids by Zipf frequencies
        s["table"] = torch.rand((c.vocab, c.E), generator=gen, device="cuda").topk(c.k, dim=1).indices.to(torch.int32)
        cdf = torch.arange(1, c.vocab + 1, dtype=torch.float64, device="cuda").pow(-1.1).cumsum(0)
        u = torch.rand((c.T,), generator=gen, device="cuda", dtype=torch.float64) * cdf[-1]
        s["ids"] = torch.searchsorted(cdf, u, right=True).clamp_(max=c.vocab - 1).to(torch.int32)
    if c.mxfp4:
        base = 127 + round(math.log2(c.w_std / 2.93))   # 2.93: root mean square of the sixteen codes
        w = SimpleNamespace()
        for name, rows, cols in (("w1", c.I, c.d), ("w3", c.I, c.d), ("w2", c.d, c.I)):
            setattr(w, name, torch.randint(0, 256, (c.E + 1, rows, cols // 2), generator=gen, device="cuda", dtype=torch.uint8))
            setattr(w, name + "s", torch.randint(base - 1, base + 2, (c.E + 1, rows, cols // 32), generator=gen, device="cuda",
                                                 dtype=torch.uint8))
        s["w"] = w
    else:
        s["w1"] = _normal(gen, (c.E + 1, c.I, c.d), c.w_std)
        s["w3"] = _normal(gen, (c.E + 1, c.I, c.d), c.w_std)
        s["w2"] = _normal(gen, (c.E + 1, c.d, c.I), c.w_std)
    return s


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------
def _act(z, act):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    z = _act(z, c.act)
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(torch.float32 if c.out == "fp32" else torch.bfloat16)


def _scores(c, logits):
    if c.score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    if c.score == "sqrtsoftplus":
        return torch.sqrt(torch.clamp(logits, min=0.0) + torch.log1p(torch.exp(-logits.abs())))
    e = torch.exp(logits - logits.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _routing(s):
    """Experts [T, k] and gate weights [T, k], in 64 bits (the selection is by comparison)."""
    c = s["case"]
    logits = s["x"].double() @ s["w_gate"].double().t()
    if s["offset"] is not None:
        logits = logits + s["offset"].double()
    score = _scores(c, logits)
    if c.vocab:
        idx = s["table"][s["ids"].long()].long()
    else:
        b = score if s["bias"] is None else score + s["bias"].double()
        if c.G > 1:
            by = b.view(c.T, c.G, c.E // c.G)
            of_group = by.amax(-1) if s["bias"] is None else by.topk(2, dim=-1).values.sum(-1)
            kept = torch.sort(of_group, dim=-1, descending=True, stable=True).indices[:, :c.g]
            mask = torch.zeros((c.T, c.G), dtype=torch.bool, device=b.device).scatter_(1, kept, True)
            b = torch.where(mask[:, :, None], by, -math.inf).view(c.T, c.E)
        idx = torch.sort(b, dim=-1, descending=True, stable=True).indices[:, :c.k]
    w = score.gather(1, idx)
    if c.score != "softmax":
        w = w / w.sum(-1, keepdim=True)
    return idx, w * c.scale


def _matrix(s, name, which):
    """Rows `which` of a stacked weight in 32 bits."""
    if not s["case"].mxfp4:
        return s[name][which].float()
    code = getattr(s["w"], name)[which]
    scale = torch.exp2(getattr(s["w"], name + "s")[which].float() - 127.0)
    value = torch.tensor(FP4_VALUES, dtype=torch.float32, device=code.device)
    pairs = torch.stack((value[torch.arange(256, device=code.device) % 16], value[torch.arange(256, device=code.device) // 16]), dim=-1)
    v = pairs[code.int()].flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)


def _experts(s, x, which):
    """SwiGLU of the experts `which` [n], on x [n, d, t]."""
    g = _matrix(s, "w1", which) @ x
    h = g / (1.0 + torch.exp(-g)) * (_matrix(s, "w3", which) @ x)
    return _matrix(s, "w2", which) @ h


def _plain_layer(s):
    c = s["case"]
    idx, w = _routing(s)
    x = s["x"].float()
    rows = _experts(s, x.repeat_interleave(c.k, dim=0)[:, :, None], idx.reshape(-1))       # [T * k, d, 1]
    shared = _experts(s, x.t()[None], torch.full((1,), c.E, device=x.device))[0].t()       # [T, d]
    y = (rows.view(c.T, c.k, c.d) * w.float()[:, :, None]).sum(1) + shared
    counts = torch.zeros((c.E,), dtype=torch.int32, device=x.device)
    counts.index_add_(0, idx.reshape(-1), torch.ones((c.T * c.k,), dtype=torch.int32, device=x.device))
    return {"y": y.to(torch.bfloat16), "counts": counts}


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def _handle(s):
    """What a serving program keeps for one layer: descriptor, workspace and output buffers."""
    from mixture_experts_routing_gate_b200 import moe as M
    c = s["case"]
    if c.op == "linear":
        desc = M.linear_desc(c.K, c.N, activation=c.act, out_dtype=torch.float32 if c.out == "fp32" else torch.bfloat16)
        ws = M.LinearWorkspace(desc, c.T)
        y = torch.empty((c.T, c.N), dtype=torch.float32 if c.out == "fp32" else torch.bfloat16, device="cuda")
        return SimpleNamespace(M=M, desc=desc, ws=ws, y=y)
    cfg = SimpleNamespace(dim=c.d, n_experts=c.E, n_groups=c.G, n_limited_groups=c.g, topk=c.k, inter_dim=c.I,
                          score_func=c.score, route_scale=c.scale)
    desc = M.layer_desc(cfg)
    return SimpleNamespace(M=M, desc=desc, ws=M.Workspace(desc, c.T), y=torch.empty_like(s["x"]),
                           counts=torch.empty((c.E,), dtype=torch.int32, device="cuda"))


def run(state):
    s = state
    if not own:
        return _plain_linear(s) if s["case"].op == "linear" else _plain_layer(s)
    if "handle" not in s:
        s["handle"] = _handle(s)
    h = s["handle"]
    if s["case"].op == "linear":
        h.M.moe_linear(h.desc, s["x"], s["w"], h.y, h.ws, bias=s["bias"], residual=s["residual"])
        return h.y
    route = dict(bias=s["bias"], logit_offset=s["offset"], token_ids=s.get("ids"), tid2eid=s.get("table"), counts_out=h.counts)
    if s["case"].mxfp4:
        h.M.moe_decode_mxfp4(h.desc, s["x"], s["w_gate"], s["w"], h.y, h.ws, **route)
    else:
        h.M.moe_decode(h.desc, s["x"], s["w_gate"], s["w1"], s["w3"], s["w2"], h.y, h.ws, **route)
    return {"y": h.y, "counts": h.counts}


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def _active_experts(c):
    """Distinct routed experts of a batch, as the mean over a few simulated routings."""
    rng = np.random.default_rng(0)
    found = []
    for _ in range(8):
        if c.vocab:
            p = np.arange(1, c.vocab + 1) ** -1.1
            ids = np.unique(rng.choice(c.vocab, size=c.T, p=p / p.sum()))
            idx = np.concatenate([rng.permutation(c.E)[:c.k] for _ in ids])
        else:
            b = rng.standard_normal((c.T, c.E)) * c.w_std * math.sqrt(c.d)
            if c.offset:
                b += rng.standard_normal(c.E)
            by = b.reshape(c.T, c.G, -1)
            best = np.sort(by, axis=2)[:, :, -2:].sum(2) if c.bias else by.max(2)
            cut = np.sort(best, axis=1)[:, c.G - c.g][:, None]
            idx = np.argsort(np.where((best >= cut)[:, :, None], by, -np.inf).reshape(c.T, c.E), axis=1)[:, -c.k:]
        found.append(len(np.unique(idx)))
    return sum(found) / len(found)


def work(case):
    c = SimpleNamespace(**case)
    if c.op == "linear":
        out = 4 if c.out == "fp32" else 2
        return {"bytes": 2 * c.T * c.K + 2 * c.N * c.K + c.T * c.N * (out + (2 if c.residual else 0)) + (4 * c.N if c.bias else 0),
                "flops": 2 * c.T * c.K * c.N}
    weight = (0.5 + 1 / 32) if c.mxfp4 else 2
    experts = _active_experts(c) + 1
    return {"bytes": experts * 3 * c.d * c.I * weight + 4 * c.E * c.d + 4 * c.T * c.d + 4 * c.E,
            "flops": 6 * c.T * (c.k + 1) * c.d * c.I + 2 * c.T * c.E * c.d}


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    x = s["x"].double()
    if c.op == "linear":
        y = torch.empty((c.T, c.N), dtype=torch.float64, device="cuda")
        for n in range(0, c.N, 16384):
            z = x @ s["w"][n:n + 16384].double().t()
            if c.bias:
                z += s["bias"][n:n + 16384].double()
            f = torch.nn.functional
            z = {"none": lambda v: v, "relu": f.relu, "silu": f.silu, "gelu": f.gelu,
                 "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[c.act](z)
            if c.residual:
                z += s["residual"][:, n:n + 16384].double()
            y[:, n:n + 16384] = z
        return y

    def weight(name, e):
        if not c.mxfp4:
            return s[name][e].double()
        byte = getattr(s["w"], name)[e].long()
        code = torch.stack((byte & 15, byte >> 4), dim=-1).flatten(-2)
        exponent, mantissa = (code >> 1) & 3, code & 1
        size = torch.where(exponent == 0, 0.5 * mantissa.double(), (1.0 + 0.5 * mantissa) * torch.exp2(exponent.double() - 1.0))
        scale = torch.exp2(getattr(s["w"], name + "s")[e].double() - 127.0).repeat_interleave(32, dim=-1)
        return torch.where(code >= 8, -size, size) * scale

    def ffn(e, rows):
        return (torch.nn.functional.silu(rows @ weight("w1", e).t()) * (rows @ weight("w3", e).t())) @ weight("w2", e).t()

    logits = x @ s["w_gate"].double().t()
    if c.offset:
        logits = logits + s["offset"].double()
    score = {"sigmoid": torch.sigmoid, "softmax": lambda v: torch.softmax(v, -1),
             "sqrtsoftplus": lambda v: torch.nn.functional.softplus(v, threshold=700.0).sqrt()}[c.score](logits)
    y = ffn(c.E, x)
    chosen = [[] for _ in range(c.E)]
    for t in range(c.T):
        if c.vocab:
            experts = s["table"][int(s["ids"][t])].tolist()
        else:
            b = (score[t] + s["bias"].double() if c.bias else score[t]).tolist()
            per = c.E // c.G
            best = [sum(sorted(b[i * per:(i + 1) * per], reverse=True)[:2 if c.bias else 1]) for i in range(c.G)]
            kept = sorted(range(c.G), key=lambda i: (-best[i], i))[:c.g]
            experts = sorted((e for i in kept for e in range(i * per, (i + 1) * per)), key=lambda e: (-b[e], e))[:c.k]
        w = score[t, experts]
        if c.score != "softmax":
            w = w / w.sum()
        for e, v in zip(experts, (w * c.scale).tolist()):
            chosen[e].append((t, v))
    for e, rows in enumerate(chosen):
        if rows:
            tokens = [t for t, _ in rows]
            y[tokens] += ffn(e, x[tokens]) * torch.tensor([v for _, v in rows], dtype=torch.float64, device="cuda")[:, None]
    return {"y": y, "counts": None}
