"""Gated int8 products into bf16 alone, on every form: neighbouring lanes swap
channels there for 4-byte stores, where an fp32 output keeps each lane to its own.
Both ways hold the same fp32 value, so the bf16 rows have to be equal to the bit."""
import pytest
import torch

from linear_forms import FORMS

pytestmark = pytest.mark.gpu

RTOL, ATOL = 2.0 ** -13, 1e-30   # of the fp32 output, as derived in test_gpu_linear_i8.py
BAND = 2048                      # values in front of and behind an output


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_ffn_06_b200 import api as a
    return a


def _inputs(T, N, K):
    g = torch.Generator(device="cuda").manual_seed(T + N + K)
    x, w = (torch.randint(-128, 128, (n, K), dtype=torch.int8, device="cuda", generator=g) for n in (T, N))
    xs = (0.5 + torch.rand(T, device="cuda", generator=g)) / 127
    ws = (0.5 + torch.rand(N, device="cuda", generator=g)) / 127 / K ** 0.5
    return x, xs, w, ws


@pytest.mark.parametrize("T,N,K", FORMS)
def test_bf16_alone(api, T, N, K):
    x, xs, w, ws = _inputs(T, N, K)
    n = N // 2
    work = torch.zeros(256, dtype=torch.uint8, device="cuda")
    v = (x.double() @ w.double().T).float() * (xs[:, None] * ws)
    for act in (api.ACT_SILU, api.ACT_GELU_TANH):
        o32 = torch.full((T, n), float("nan"), device="cuda")
        both = torch.full((T, n), float("nan"), dtype=torch.bfloat16, device="cuda")
        api.moe_linear_i8(x, xs, w, ws, both, work, gate_act=act, out_f32=o32)
        raw = torch.full((BAND + T * n + BAND,), float("nan"), dtype=torch.bfloat16, device="cuda")
        alone = raw[BAND:BAND + T * n].view(T, n)
        api.moe_linear_i8(x, xs, w, ws, alone, work, gate_act=act)
        assert api.moe_read_error(work) == 0
        g = v[:, :n].double()
        if act == api.ACT_GELU_TANH:
            g = g / (1 + torch.exp(-2 * (2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
        else:
            g = g / (1 + torch.exp(-g))
        want = g * v[:, n:].double()
        assert bool(((o32 - want).abs() <= RTOL * want.abs() + ATOL).all())
        assert torch.equal(both, o32.to(torch.bfloat16))
        assert torch.equal(alone, both)
        assert bool(raw[:BAND].isnan().all()) and bool(raw[BAND + T * n:].isnan().all())


def test_short_tiles_one_launch_behind_the_other(api):
    # more tiles of one k-block than SMs have TMEM columns for at once
    T, N, K = 100, 128256, 128
    x, xs, w, ws = _inputs(T, N, K)
    work = torch.zeros(256, dtype=torch.uint8, device="cuda")
    outs = [torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    for o in outs:
        api.moe_linear_i8(x, xs, w, ws, o, work)
    want = ((x.double() @ w.double().T).float() * (xs[:, None] * ws)).to(torch.bfloat16)
    assert api.moe_read_error(work) == 0
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("T,N,K", [(5, 2048, 256), (40, 2048, 256), (100, 2048, 2064), (700, 2048, 256)])
def test_gated_fp32_output_within_the_stated_error(api, T, N, K):
    # gates from a hundredth to some hundreds: sigmoid arguments far out on both sides
    x, xs, w, ws = _inputs(T, N, K)
    n = N // 2
    ws[:n] *= torch.logspace(-1, 3, n, device="cuda")
    work = torch.zeros(256, dtype=torch.uint8, device="cuda")
    v = (x.double() @ w.double().T).float() * (xs[:, None] * ws)
    g, u = v[:, :n].double(), v[:, n:].double()
    for act, c in ((api.ACT_SILU, 1.2), (api.ACT_GELU_TANH, 4.2)):
        o32 = torch.empty(T, n, device="cuda")
        api.moe_linear_i8(x, xs, w, ws, None, work, gate_act=act, out_f32=o32)
        e = (8 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3) if act == api.ACT_GELU_TANH else g
        want = g / (1 + torch.exp(-e)) * u
        assert float(e.min()) < -100 and float(e.max()) > 100
        bound = (5 + c * (-e).clamp(0, 90)) * 2.0 ** -23 * want.abs() + (g * u).abs() * 2.0 ** -126 + 2.0 ** -149
        assert bool(((o32 - want).abs() <= bound).all())
