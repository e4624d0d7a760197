"""moe_block_norm and moe_quantize_rows_i8 on the GPU.

Their definition fixes a chain of IEEE fp32 operations (the means in 64 bits),
so against that chain every output has to be equal to the bit.  Against the
formula in 64 bits: one bf16 rounding (2^-8 of the value) and, before it, at
most eight fp32 roundings of terms no larger than |alpha r| + |m t| (2^-24 each;
the inverse norm's own three are among them)."""
import numpy as np
import pytest
import torch

import operators_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_ffn_06_b200 import api as a
    return a


def _bf(g, *shape, mul=1.0, add=0.0):
    return (torch.randn(*shape, generator=g) * mul + add).to(torch.bfloat16)


def _np(t):
    return None if t is None else t.float().cpu().numpy()


def _inputs(T, H, seed, after, gate, token_gate, before):
    g = torch.Generator().manual_seed(seed)
    d = dict(r=_bf(g, T, H, mul=2.0))
    if after:
        d["y"] = _bf(g, T, H)
        if after != "plain":
            d["post_w"] = _bf(g, H, mul=0.1, add=1.0)
    if gate:
        d["gate"] = _bf(g, H, mul=0.3, add=0.5)
    if token_gate:
        d["token_gate"] = torch.rand(T, generator=g)
    if before:
        d["pre_w"] = _bf(g, H, mul=0.1, add=1.0)
    return d


def _run(api, d, a=True, codes=False, **kw):
    T, H = d["r"].shape
    c = {n: t.cuda() for n, t in d.items()}
    r_out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda") if "y" in d else None
    av = torch.empty(T, H, dtype=torch.bfloat16, device="cuda") if a and "pre_w" in d else None
    q = torch.empty(T, H, dtype=torch.int8, device="cuda") if codes else None
    s = torch.empty(T, device="cuda") if codes else None
    api.moe_block_norm(c.pop("r"), r_out=r_out, a=av, codes=q, scales=s, **c, **kw)
    torch.cuda.synchronize()
    return r_out, av, q, s


def _check(d, got, **kw):
    r_out, a, q, s = got
    want_r, want_a = ref.block_norm(**{n: _np(t) for n, t in d.items()}, **kw)
    if r_out is not None:
        assert np.array_equal(_np(r_out), want_r, equal_nan=True)
        base, t = ref.block_norm64(**{n: _np(v) for n, v in d.items() if n != "pre_w"},
                                   **{n: v for n, v in kw.items() if n != "pre_eps"})
        err = np.abs(_np(r_out) - (base + t))
        bound = 2.0 ** -8 * np.abs(base + t) + 8 * 2.0 ** -24 * (np.abs(base) + np.abs(t))
        assert (err <= bound * (1 + 2.0 ** -8)).all()
    if a is not None:
        assert np.array_equal(_np(a), want_a, equal_nan=True)
    if q is not None:
        qc, qs = ref.quantize_i8(want_a)
        assert np.array_equal(q.cpu().numpy(), qc)
        assert np.array_equal(s.cpu().numpy(), qs, equal_nan=True)


SIZES = [(1, 8), (1, 2816), (3, 256), (37, 200), (64, 2048), (130, 2816), (5, 4096), (7, 8192),
         (2, 14336), (3, 32768), (1025, 1032), (2000, 264), (300, 32000), (310, 32768), (500, 5632),
         (301, 1024), (999, 8)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("after,gate,token_gate,before,codes,alpha,beta", [
    (True, True, False, True, True, 0.75, 1.25),
    (True, False, True, True, False, 1.0, 0.5),
    (True, True, True, False, False, 1.0, 1.0),
    ("plain", False, True, True, True, -1.0, 2.0),
    ("plain", False, False, False, False, 0.0, 1.0),
    (False, False, False, True, True, 1.0, 1.0),
    (False, False, False, True, False, 1.0, 1.0),
])
def test_matches_the_definition(api, T, H, after, gate, token_gate, before, codes, alpha, beta):
    d = _inputs(T, H, T + H, after, gate, token_gate, before)
    kw = dict(alpha=alpha, beta=beta) if after else {}
    _check(d, _run(api, d, codes=codes, **kw), **kw)


def test_codes_without_the_normalised_row(api):
    d = _inputs(33, 704, 3, True, False, False, True)
    _check(d, _run(api, d, a=False, codes=True))


def test_eps_and_extreme_rows(api):
    d = _inputs(12, 512, 4, True, True, True, True)
    d["y"][0] = 0.0
    d["r"][0] = 0.0                       # nothing in the row: norm 0, scale 1
    d["y"][1] = 3e38                      # squares overflow fp32, not fp64
    d["y"][2] = 1e-38
    d["r"][3] = 3e38
    d["token_gate"][4] = 0.0              # a closed gate leaves the residual
    d["r"][5, 7] = float("inf")
    d["r"][6, 9] = float("nan")
    d["y"][7, 3] = float("nan")
    kw = dict(post_eps=1e-5, pre_eps=1e-3)
    got = _run(api, d, codes=True, **kw)
    want_r, want_a = ref.block_norm(**{n: _np(t) for n, t in d.items()}, **kw)
    assert np.array_equal(_np(got[0]), want_r, equal_nan=True)
    assert np.array_equal(_np(got[1]), want_a, equal_nan=True)
    q, s = got[2].cpu().numpy(), got[3].cpu().numpy()
    qc, qs = ref.quantize_i8(want_a)
    assert np.array_equal(q, qc) and np.array_equal(s, qs, equal_nan=True)
    assert torch.equal(got[0][4].cpu(), d["r"][4])
    assert s[0] == 1.0 and not np.isfinite(s[[5, 6, 7]]).any() and (q[[5, 6, 7]] == 0).all()


def test_the_residual_is_updated_in_place(api):
    d = _inputs(50, 640, 5, True, False, False, True)
    c = {n: t.cuda() for n, t in d.items()}
    a = torch.empty_like(c["r"])
    api.moe_block_norm(c["r"], y=c["y"], post_w=c["post_w"], pre_w=c["pre_w"], r_out=c["r"], a=a)
    _check(d, (c["r"], a, None, None))


def test_an_empty_batch(api):
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    api.moe_block_norm(e, pre_w=w, a=e.clone())
    api.moe_quantize_rows_i8(e, e.to(torch.int8), torch.empty(0, device="cuda"))


def test_rows_past_32_bit_offsets(api):
    T, H = 800_000, 2816   # 2.25e9 values
    d = _inputs(64, H, 6, True, True, False, True)
    c = {n: t.cuda() for n, t in d.items()}
    r = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    y = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(T, H, dtype=torch.int8, device="cuda")
    s = torch.empty(T, device="cuda")
    r[-64:], y[-64:] = c["r"], c["y"]
    api.moe_block_norm(r, y=y, post_w=c["post_w"], gate=c["gate"], pre_w=c["pre_w"], r_out=r, a=y,
                       codes=q, scales=s)
    _check(d, (r[-64:], y[-64:], q[-64:], s[-64:]))


def test_captured_and_replayed(api):
    d = _inputs(40, 2816, 7, True, True, True, True)
    c = {n: t.cuda() for n, t in d.items()}
    r_out, a = torch.empty_like(c["r"]), torch.empty_like(c["r"])
    q = torch.empty(40, 2816, dtype=torch.int8, device="cuda")
    s = torch.empty(40, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_block_norm(r_out=r_out, a=a, codes=q, scales=s, **c)
    for seed in (8, 9):
        d = _inputs(40, 2816, seed, True, True, True, True)
        for n, t in d.items():
            c[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        _check(d, (r_out, a, q, s))


# ------------------------------------------------------------- quantiser

@pytest.mark.parametrize("R,C", [(1, 8), (1, 2112), (3, 704), (16, 2816), (33, 4096), (5, 14336),
                                 (2, 32768), (3001, 72)])
def test_quantiser_is_exact(api, R, C):
    g = torch.Generator().manual_seed(R + C)
    x = _bf(g, R, C, mul=3.0)
    if R > 2:
        x[0] = 0.0
        x[1] = 9.2e-41                    # the smallest bf16 value: a subnormal scale
        x[2] = 3.3e38
    q = torch.empty(R, C, dtype=torch.int8, device="cuda")
    s = torch.empty(R, device="cuda")
    api.moe_quantize_rows_i8(x.cuda(), q, s)
    qc, qs = ref.quantize_i8(_np(x))
    assert np.array_equal(q.cpu().numpy(), qc) and np.array_equal(s.cpu().numpy(), qs)


def test_quantiser_ties_and_non_finite_rows(api):
    # amax 127: scale 1, so halves are ties, to the even code
    x = torch.zeros(4, 16)
    x[0] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 3.5, 4.5, -126.5] + [0.0] * 6)
    x[1, 3] = float("inf")
    x[2, 4] = float("nan")
    x[3, 5], x[3, 6] = float("-inf"), float("nan")
    q = torch.empty(4, 16, dtype=torch.int8, device="cuda")
    s = torch.empty(4, device="cuda")
    api.moe_quantize_rows_i8(x.to(torch.bfloat16).cuda(), q, s)
    assert q[0].tolist()[:10] == [127, 0, 2, 2, 0, -2, -2, 4, 4, -126]
    assert (q[1:] == 0).all()
    assert s[1].item() == float("inf") and torch.isnan(s[2:]).all()
