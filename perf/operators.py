"""Cases of the operators around the expert products: routing with a balance
bias, the 8-bit integer product with token and channel scales, and the norms
around a block with its gate and residual scale.

``own`` False computes each operator in elementary torch operations; ``own``
True calls the library's entry points on the same inputs.
"""
import math

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------- cases

def _route(name, T, E, k, sigmoid, n_group, topk_group, group_top, renorm, factor, scaled):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "sigmoid": sigmoid,
            "n_group": n_group, "topk_group": topk_group, "group_top": group_top,
            "renorm": renorm, "factor": factor, "scaled": scaled}


def _norm(name, T, H, after, gate, token_gate, before, codes, alpha, beta):
    return {"name": name, "op": "norm", "T": T, "H": H, "after": after, "gate": gate,
            "token_gate": token_gate, "before": before, "codes": codes, "alpha": alpha,
            "beta": beta}


def _linear(name, T, K, N, gated, gelu, quantize):
    return {"name": name, "op": "linear", "T": T, "K": K, "N": N, "gated": gated, "gelu": gelu,
            "quantize": quantize}


def listed():
    return [
        # one decoded token through a 256-expert sigmoid router, 8 groups of which 4 are kept
        _route("route_t1_e256_groups", 1, 256, 8, True, 8, 4, 2, True, 2.5, False),
        # a decode batch through the 128-expert softmax router with per-expert scales
        _route("route_t64_e128", 64, 128, 8, False, 1, 1, 1, True, 1.0, True),
        # a ragged prefill chunk through the grouped 256-expert router
        _route("route_t4095_e256_groups", 4095, 256, 8, True, 8, 4, 2, True, 2.5, False),
        # the skewed workload's 16384 tokens, 64 experts, weights left as the softmax gives them
        _route("route_t16384_e64", 16384, 64, 6, False, 1, 1, 1, False, 1.0, False),
        # one decoded token: the norm after a block, channel gate, residual and the next norm
        _norm("norm_t1_h2816", 1, 2816, True, True, False, True, False, 1.0, 1.0),
        # a decode batch with only the norm ahead of a block (the first of the stack)
        _norm("norm_t257_h4096_before", 257, 4096, False, False, False, True, False, 1.0, 1.0),
        # a prefill: both norms, channel gate and residual scale
        _norm("norm_t8192_h2816", 8192, 2816, True, True, False, True, False, 0.75, 1.25),
        # the longest prefill: token gate of a shared expert, codes for an int8 product
        _norm("norm_t16383_h2048_codes", 16383, 2048, True, False, True, True, True, 1.0, 0.5),
        # one decoded token through the dense MLP's gated product (I = 2112)
        _linear("linear_t1_gated", 1, 2816, 4224, True, True, False),
        # a decode batch through its down product, from bf16 rows
        _linear("linear_t16_down", 16, 2112, 2816, False, False, True),
        # a ragged batch through a wide plain product
        _linear("linear_t257_wide", 257, 4096, 14336, False, False, False),
        # a prefill through the wide gated product, from bf16 rows
        _linear("linear_t4096_gated", 4096, 4096, 28672, True, False, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "linear"])
    if op == "route":
        T = _log_int(rng, 1, 16384)
        n_group = rng.choice([1, 1, 2, 4, 8])
        size = max(2, _log_int(rng, 8, 512) // n_group)
        topk_group = rng.randint(1, n_group)
        k = rng.randint(1, min(16, topk_group * size))
        c = _route("", T, n_group * size, k, rng.random() < 0.5, n_group, topk_group,
                   rng.choice([1, 2]), rng.random() < 0.7, rng.choice([1.0, 2.5]),
                   rng.random() < 0.5)
    elif op == "norm":
        H = 8 * _log_int(rng, 32, 1024)
        T = min(_log_int(rng, 1, 16384), 16383 * 2048 // H)
        after = rng.random() < 0.7
        before = not after or rng.random() < 0.8
        c = _norm("", T, H, after, after and rng.random() < 0.5, after and rng.random() < 0.5,
                  before, before and rng.random() < 0.5, rng.choice([1.0, 0.75]),
                  rng.choice([1.0, 0.5, 1.25]))
    else:
        gated = rng.random() < 0.5
        K = 16 * _log_int(rng, 16, 512)
        N = _log_int(rng, 256, 14336)
        N = 2 * N if gated else N
        T = min(_log_int(rng, 1, 8192), 4096 * 4096 * 28672 // (N * K))
        c = _linear("", T, K, N, gated, gated and rng.random() < 0.5, rng.random() < 0.5)
    del c["name"]
    return c


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 8 * T * k + 8 * E + (4 * E if case["scaled"] else 0),
                "flops": 10 * T * E}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        row = 2 * H  # the residual
        per_channel = 0
        if case["after"]:
            row += 2 * H + 2 * H  # the block's output in, the new residual out
            row += 4 if case["token_gate"] else 0
            per_channel += 2 * H * (2 if case["gate"] else 1)
        if case["before"]:
            row += 2 * H
            per_channel += 2 * H
        if case["codes"]:
            row += H + 4
        return {"bytes": T * row + per_channel, "flops": 12 * T * H}
    T, K, N = case["T"], case["K"], case["N"]
    x = T * K * (2 if case["quantize"] else 1) + (0 if case["quantize"] else 4 * T)
    out = 2 * T * (N // 2 if case["gated"] else N)
    return {"bytes": x + N * K + 4 * N + out, "flops": 2 * T * K * N}


# ------------------------------------------------------------------ inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE)


def _quantized_normal(gen, rows, cols):
    """int8 codes and row scales of N(0,1) rows (round to nearest even)."""
    v = _normal(gen, rows, cols)
    s = v.abs().amax(dim=1).clamp_min(1e-20) / 127.0
    return torch.round(v / s[:, None]).clamp_(-127, 127).to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    st = dict(case)
    bf, f32, dev = torch.bfloat16, torch.float32, DEVICE
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = _normal(gen, T, E) + 0.5 * _normal(gen, E)
        # the bias has settled near what evens the load out: small next to the scores
        st["bias"] = _normal(gen, E) * (0.05 if case["sigmoid"] else 0.5 / E)
        st["scale"] = 0.5 + torch.rand(E, generator=gen, device=dev) if case["scaled"] else None
        st["ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
        st["w"] = torch.empty(T, k, dtype=f32, device=dev)
        st["load"] = torch.empty(E, dtype=torch.int32, device=dev)
    elif case["op"] == "norm":
        T, H = case["T"], case["H"]
        st["r"] = (2.0 * _normal(gen, T, H)).to(bf)
        st["y"] = _normal(gen, T, H).to(bf) if case["after"] else None
        gamma = lambda: (1.0 + 0.1 * _normal(gen, H)).to(bf)  # noqa: E731
        st["post_w"] = gamma() if case["after"] else None
        st["pre_w"] = gamma() if case["before"] else None
        st["gate_w"] = (0.5 + 0.1 * _normal(gen, H)).to(bf) if case["gate"] else None
        st["token_w"] = torch.sigmoid(_normal(gen, T)) if case["token_gate"] else None
        st["r_out"] = torch.empty(T, H, dtype=bf, device=dev) if case["after"] else None
        st["a"] = torch.empty(T, H, dtype=bf, device=dev) if case["before"] else None
        st["q"] = torch.empty(T, H, dtype=torch.int8, device=dev) if case["codes"] else None
        st["q_scale"] = torch.empty(T, dtype=f32, device=dev) if case["codes"] else None
        st["q_value"] = torch.empty(T, H, dtype=bf, device=dev) if case["codes"] else None
    else:
        T, K, N = case["T"], case["K"], case["N"]
        if case["quantize"]:
            st["x"] = _normal(gen, T, K).to(bf)
            st["xq"] = torch.empty(T, K, dtype=torch.int8, device=dev)
            st["xs"] = torch.empty(T, dtype=f32, device=dev)
        else:
            st["xq"], st["xs"] = _quantized_normal(gen, T, K)
        st["wq"], ws = _quantized_normal(gen, N, K)
        st["ws"] = ws * K ** -0.5  # outputs near unit size
        st["out"] = torch.empty(T, N // 2 if case["gated"] else N, dtype=bf, device=dev)
        st["work"] = torch.zeros(256, dtype=torch.uint8, device=dev)
    return st


# -------------------------------------------------------------- plain forms

def _plain_route(st):
    T, E, k = st["T"], st["E"], st["k"]
    z = st["logits"].double()
    if st["sigmoid"]:
        s = 1.0 / (1.0 + torch.exp(-z))
    else:
        e = torch.exp(z - z.amax(dim=1, keepdim=True))
        s = e / e.sum(dim=1, keepdim=True)
    c = s + st["bias"].double()
    G = st["n_group"]
    if G > 1:
        best = torch.sort(c.view(T, G, E // G), dim=2, descending=True, stable=True).values
        score = best[:, :, :st["group_top"]].sum(dim=2)
        order = torch.sort(score, dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, G, dtype=torch.bool, device=c.device)
        keep.scatter_(1, order[:, :st["topk_group"]], True)
        c = torch.where(keep.repeat_interleave(E // G, dim=1), c, -math.inf)
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(s, 1, ids)
    if st["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = w * st["factor"]
    if st["scale"] is not None:
        w = w * st["scale"].double()[ids]
    load = torch.zeros(E, dtype=torch.int32, device=c.device)
    load.index_add_(0, ids.reshape(-1), torch.ones(T * k, dtype=torch.int32, device=c.device))
    return {"ids": ids.to(torch.int32), "w": w.float(), "load": load}


def _plain_rms(v, eps):
    mean = v.double().square().mean(dim=1, keepdim=True).float()
    return v * (1.0 / torch.sqrt(mean + eps))


def _plain_codes(v):
    """Codes (as float values) and scale of each row, s = amax / 127."""
    amax = v.abs().amax(dim=1, keepdim=True)
    s = torch.where(amax > 0, amax / 127.0, torch.ones_like(amax))
    return torch.round(v / s).clamp(-127.0, 127.0), s


def _plain_norm(st):
    out = {}
    r = st["r"].float()
    if st["after"]:
        t = _plain_rms(st["y"].float(), 1e-6) * st["post_w"].float()
        if st["gate"]:
            t = t * st["gate_w"].float()
        m = torch.full((st["T"], 1), st["beta"], dtype=torch.float32, device=r.device)
        if st["token_gate"]:
            m = m * st["token_w"][:, None]
        r = (st["alpha"] * r + m * t).to(torch.bfloat16)
        out["r"] = r
        r = r.float()
    if st["before"]:
        a = (_plain_rms(r, 1e-6) * st["pre_w"].float()).to(torch.bfloat16)
        out["a"] = a
        if st["codes"]:
            q, s = _plain_codes(a.float())
            out["q"] = (q * s).to(torch.bfloat16)
    return out


def _plain_act(st, g):
    if st["gelu"]:
        c = math.sqrt(2.0 / math.pi)
        return 0.5 * g * (1.0 + torch.tanh(c * (g + 0.044715 * g * g * g)))
    return g / (1.0 + torch.exp(-g))


def _plain_linear(st):
    if st["quantize"]:
        q, s = _plain_codes(st["x"].float())
        s = s[:, 0]
    else:
        q, s = st["xq"].float(), st["xs"]
    acc = q @ st["wq"].float().t()
    v = acc * (s[:, None] * st["ws"][None, :])
    if st["gated"]:
        I = st["N"] // 2
        v = _plain_act(st, v[:, :I]) * v[:, I:]
    return {"out": v.to(torch.bfloat16)}


# --------------------------------------------------------- the library's own

def _own_route(st):
    from mixture_experts_ffn_06_b200 import api
    if "shape" not in st:  # a program makes these once, with its buffers
        st["shape"] = api.make_shape(T=st["T"], H=64, E=st["E"], k=st["k"], I=64)
        st["opts"] = api.balance_opts(
            scoring=api.SCORE_SIGMOID if st["sigmoid"] else api.SCORE_SOFTMAX,
            n_group=st["n_group"], topk_group=st["topk_group"], group_top=st["group_top"],
            renorm=st["renorm"], factor=st["factor"])
    api.moe_route_balanced(st["shape"], st["logits"], st["bias"], st["scale"], st["ids"],
                           st["w"], load=st["load"], opts=st["opts"])
    return {"ids": st["ids"], "w": st["w"], "load": st["load"]}


def _own_norm(st):
    from mixture_experts_ffn_06_b200 import api
    api.moe_block_norm(st["r"], y=st["y"], post_w=st["post_w"], gate=st["gate_w"],
                       token_gate=st["token_w"], alpha=st["alpha"], beta=st["beta"],
                       post_eps=1e-6, pre_w=st["pre_w"], pre_eps=1e-6, r_out=st["r_out"],
                       a=st["a"], codes=st["q"], scales=st["q_scale"])
    out = {}
    if st["after"]:
        out["r"] = st["r_out"]
    if st["before"]:
        out["a"] = st["a"]
        if st["codes"]:  # the bf16 values that the codes stand for
            out["q"] = torch.mul(st["q"], st["q_scale"][:, None], out=st["q_value"])
    return out


def _own_linear(st):
    from mixture_experts_ffn_06_b200 import api
    if st["quantize"]:
        api.moe_quantize_rows_i8(st["x"], st["xq"], st["xs"])
    act = (api.ACT_GELU_TANH if st["gelu"] else api.ACT_SILU) if st["gated"] else None
    api.moe_linear_i8(st["xq"], st["xs"], st["wq"], st["ws"], st["out"], st["work"], gate_act=act)
    return {"out": st["out"]}


def run(state):
    if own:
        return {"route": _own_route, "norm": _own_norm, "linear": _own_linear}[state["op"]](state)
    return {"route": _plain_route, "norm": _plain_norm, "linear": _plain_linear}[state["op"]](state)


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    if case["op"] == "route":
        z, b = st["logits"].to(d), st["bias"].to(d)
        s = torch.sigmoid(z) if case["sigmoid"] else torch.softmax(z, dim=1)
        c = s + b
        E, G = case["E"], case["n_group"]
        if G > 1:
            top = c.reshape(-1, G, E // G).topk(min(case["group_top"], E // G), dim=2).values
            kept = top.sum(dim=2).topk(case["topk_group"], dim=1).indices
            group = torch.arange(E, device=c.device) // (E // G)
            inside = (kept[:, :, None] == group).any(dim=1)
            c = c.masked_fill(~inside, -math.inf)
        ids = c.topk(case["k"], dim=1).indices
        w = s.gather(1, ids)
        if case["renorm"]:
            w = w / w.sum(dim=1, keepdim=True)
        w = w * case["factor"]
        if case["scaled"]:
            w = w * st["scale"].to(d)[ids]
        return {"ids": None, "w": w, "load": None}
    if case["op"] == "norm":
        r = st["r"].to(d)
        out = {}
        if case["after"]:
            y = st["y"].to(d)
            y = y * torch.rsqrt((y * y).mean(dim=1, keepdim=True) + 1e-6) * st["post_w"].to(d)
            if case["gate"]:
                y = y * st["gate_w"].to(d)
            if case["token_gate"]:
                y = y * st["token_w"].to(d)[:, None]
            r = case["alpha"] * r + case["beta"] * y
            out["r"] = r
            r = r.to(torch.bfloat16).to(d)  # the stored stream is what the next norm reads
        if case["before"]:
            out["a"] = r * torch.rsqrt((r * r).mean(dim=1, keepdim=True) + 1e-6) * st["pre_w"].to(d)
            if case["codes"]:
                out["q"] = None  # a code is a rounding decision, not a computed number
        return out
    if case["quantize"]:  # the codes are fixed by fp32 division and rounding
        x = st["x"].float()
        top = x.abs().max(dim=1, keepdim=True).values
        s = torch.where(top > 0, top / 127.0, 1.0)
        q, s = torch.round(x / s).clamp(-127, 127).to(d), s.to(d)
    else:
        q, s = st["xq"].to(d), st["xs"].to(d)[:, None]
    v = (q @ st["wq"].to(d).t()) * s * st["ws"].to(d)
    if case["gated"]:
        g, u = v.chunk(2, dim=1)
        if case["gelu"]:
            g = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))
        else:
            g = g * torch.sigmoid(g)
        v = g * u
    return {"out": v}
