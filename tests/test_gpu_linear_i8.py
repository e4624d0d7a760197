"""moe_linear_i8 on the GPU.

Plain: the integer sums are exact and the two fp32 products are fixed, so
out_f32 has to equal the definition to the bit and out be its bf16 rounding.
Gated: Act(g) * u from fp32 g and u.  g carries three roundings (2^-24 each) and
the activation's exponent |2v| <= 88 (beyond it the value is below 1e-36)
multiplies the relative error of g by at most 3 |2v|, its own evaluation adds a
few ulps and |2v| ulps of the exponential: 88 (3 * 3 + 4) 2^-24 < 2^-13 in all."""
import numpy as np
import pytest
import torch

import operators_ref as ref

pytestmark = pytest.mark.gpu

GATED_RTOL, GATED_ATOL = 2.0 ** -13, 1e-30


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_ffn_06_b200 import api as a
    return a


def _inputs(T, N, K, seed):
    g = np.random.default_rng(seed)
    x = g.integers(-128, 128, (T, K), dtype=np.int8)
    w = g.integers(-128, 128, (N, K), dtype=np.int8)
    xs = (0.5 + g.random(T)).astype(np.float32) / 127
    ws = (0.5 + g.random(N)).astype(np.float32) / 127 / np.float32(K ** 0.5) * 2
    return x, xs, w, ws


def _ws():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def _run(api, x, xs, w, ws, act=None, bf16=True, fp32=True):
    c = [torch.from_numpy(v).cuda() for v in (x, xs, w, ws)]
    T, n = x.shape[0], w.shape[0] // (1 if act is None else 2)
    out = torch.full((T, n), float("nan"), dtype=torch.bfloat16, device="cuda") if bf16 else None
    o32 = torch.full((T, n), float("nan"), device="cuda") if fp32 else None
    work = _ws()
    api.moe_linear_i8(*c, out, work, gate_act=act, out_f32=o32)
    torch.cuda.synchronize()
    assert api.moe_read_error(work) == 0
    return out, o32


def _check(got, want, act=None):
    out, o32 = got
    v = o32.cpu().numpy()
    if act is None:
        assert np.array_equal(v, want)
    else:
        assert (np.abs(v - want) <= GATED_RTOL * np.abs(want) + GATED_ATOL).all()
    if out is not None:
        assert torch.equal(out, o32.to(torch.bfloat16))


SIZES = [(1, 1, 16), (1, 64, 64), (1, 2816, 2112), (2, 130, 272), (8, 1408, 2816), (9, 96, 704),
         (16, 2816, 2112), (17, 250, 1040), (31, 4224, 528), (33, 512, 128), (64, 704, 2816),
         (65, 260, 400), (100, 1000, 1000 // 16 * 16), (128, 256, 256), (129, 258, 144),
         (257, 1030, 2048), (300, 77, 96), (511, 4096, 512), (1000, 514, 4112), (2100, 300, 16)]


@pytest.mark.parametrize("T,N,K", SIZES)
def test_plain_product_is_exact(api, T, N, K):
    x, xs, w, ws = _inputs(T, N, K, T + N + K)
    _check(_run(api, x, xs, w, ws), ref.linear_i8(x, xs, w, ws))


@pytest.mark.parametrize("T,N,K", [(T, 2 * ((N + 1) // 2), K) for T, N, K in SIZES])
@pytest.mark.parametrize("act", [0, 1])
def test_gated_product(api, T, N, K, act):
    if N < 2:
        N = 2
    x, xs, w, ws = _inputs(T, N, K, T + N + K + 1)
    _check(_run(api, x, xs, w, ws, act), ref.linear_i8(x, xs, w, ws, act), act)


# sizes that reach the forms the small ones do not: many small blocks, unsplit K
# at few tokens, several tiles to a CTA and to a CTA pair, two token sub-tiles to a
# weight tile on single CTAs and on pairs
FORMS = [(8, 14336, 64), (3, 20000, 48), (12, 9000, 128), (40, 20000, 128), (700, 14000, 640),
         (600, 14336, 256), (2000, 16384, 256), (257, 14336, 2064), (512, 18944, 2704),
         (1024, 18944, 4112), (1030, 18944, 2704), (5000, 640, 1040),
         (512, 18944, 8192), (1024, 18944, 8192),
         # few tokens: eight warps to a block, K too long for them, too many of them
         (6, 5000, 4096), (8, 9000, 208), (1, 20000, 5008), (7, 200, 4112), (16, 20000, 64),
         # K split over clusters, with one token tile and several
         (100, 130, 2064), (130, 130, 2064), (260, 514, 4112), (1025, 300, 2832), (390, 2500, 4112),
         (1100, 780, 8192), (25, 4400, 8192), (128, 4500, 2064),
         # fewer tiles than SMs, K too short to split
         (20, 2000, 256), (100, 2000, 256), (128, 9000, 400)]


@pytest.mark.parametrize("T,N,K", FORMS)
@pytest.mark.parametrize("act", [None, 0])
def test_every_form(api, T, N, K, act):
    g = torch.Generator(device="cuda").manual_seed(T + N + K)
    x, w = (torch.randint(-128, 128, (n, K), dtype=torch.int8, device="cuda", generator=g) for n in (T, N))
    xs = (0.5 + torch.rand(T, device="cuda", generator=g)) / 127
    ws = (0.5 + torch.rand(N, device="cuda", generator=g)) / 127 / K ** 0.5
    n = N if act is None else N // 2
    out = torch.full((T, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    o32 = torch.full((T, n), float("nan"), device="cuda")
    work = _ws()
    api.moe_linear_i8(x, xs, w, ws, out, work, gate_act=act, out_f32=o32)
    assert api.moe_read_error(work) == 0
    v = (x.double() @ w.double().T).float() * (xs[:, None] * ws)   # the sums are exact
    if act is None:
        assert torch.equal(o32, v)
    else:
        want = v[:, :n].double()
        want = want / (1 + torch.exp(-want)) * v[:, n:].double()
        assert bool(((o32 - want).abs() <= GATED_RTOL * want.abs() + GATED_ATOL).all())
    assert torch.equal(out, o32.to(torch.bfloat16))


@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_extreme_codes_at_the_longest_k(api, T):
    # every product is 128 * 128: the largest sum that 32 bits hold
    K, N = api.LINEAR_MAX_K, 130
    x = np.full((T, K), -128, np.int8)
    w = np.full((N, K), -128, np.int8)
    w[1] = 127
    xs, ws = np.ones(T, np.float32), np.ones(N, np.float32)
    _, o32 = _run(api, x, xs, w, ws)
    want = np.full((T, N), np.float32(16384.0 * K))
    want[:, 1] = np.float32(-128.0 * 127.0 * K)
    assert np.array_equal(o32.cpu().numpy(), want)


def test_gate_extremes_and_scales_that_are_not_finite(api):
    x, xs, w, ws = _inputs(6, 64, 32, 3)
    ws[:16] *= 1000.0                     # gates far out on both sides
    xs[1] = np.nan                        # a row that could not be quantised
    xs[2] = np.inf
    x[2] = 0
    for act in (0, 1):
        _, o32 = _run(api, x, xs, w, ws, act)
        v = o32.cpu().numpy()
        assert np.isnan(v[[1, 2]]).all()
        rows = [0, 3, 4, 5]
        want = ref.linear_i8(x[rows], xs[rows], w, ws, act)
        assert (np.abs(v[rows] - want) <= GATED_RTOL * np.abs(want) + GATED_ATOL).all()


@pytest.mark.parametrize("T,N,K,act", [(3, 66, 48, None), (70, 132, 160, 0), (300, 258, 272, None)])
def test_one_output_at_a_time(api, T, N, K, act):
    x, xs, w, ws = _inputs(T, N, K, 11)
    out, o32 = _run(api, x, xs, w, ws, act)
    assert torch.equal(_run(api, x, xs, w, ws, act, fp32=False)[0], out)
    assert torch.equal(_run(api, x, xs, w, ws, act, bf16=False)[1], o32)


def test_the_plain_constant_is_the_plain_product(api):
    T, N, K = 5, 48, 64
    x, xs, w, ws = _inputs(T, N, K, 17)
    assert torch.equal(_run(api, x, xs, w, ws, fp32=False)[0],
                       _run_plain_constant(api, x, xs, w, ws, N))
    with pytest.raises(ValueError, match="out: expected"):
        _run_plain_constant(api, x, xs, w, ws, N // 2)  # room for a gated product alone


def _run_plain_constant(api, x, xs, w, ws, n):
    out = torch.zeros(x.shape[0], n, dtype=torch.bfloat16, device="cuda")
    api.moe_linear_i8(*[torch.from_numpy(v).cuda() for v in (x, xs, w, ws)], out, _ws(),
                      gate_act=api.LINEAR_PLAIN)
    return out


class Guarded:
    """A buffer between two bands of a known byte."""

    def __init__(self, shape, dtype, band=4096):
        n = int(np.prod(shape)) * torch.tensor([], dtype=dtype).element_size()
        self.raw = torch.full((band + n + band,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.raw[band:band + n].view(dtype).view(*shape)
        self.band, self.n = band, n

    def intact(self):
        torch.cuda.synchronize()
        return bool((self.raw[:self.band] == 0xA5).all() and
                    (self.raw[self.band + self.n:] == 0xA5).all())


@pytest.mark.parametrize("T,N,K,act", [(1, 66, 48, None), (7, 2816, 2112, None), (33, 130, 400, 1),
                                       (130, 258, 528, None), (301, 514, 272, 0), (600, 77, 64, None)])
def test_writes_only_its_outputs(api, T, N, K, act):
    x, xs, w, ws = _inputs(T, N, K, 12)
    c = [torch.from_numpy(v).cuda() for v in (x, xs, w, ws)]
    n = N if act is None else N // 2
    out, o32, work = Guarded((T, n), torch.bfloat16), Guarded((T, n), torch.float32), Guarded((256,), torch.uint8)
    work.t.zero_()
    for _ in range(2):
        api.moe_linear_i8(*c, out.t, work.t, gate_act=act, out_f32=o32.t)
    assert out.intact() and o32.intact() and work.intact()
    _check((out.t, o32.t), ref.linear_i8(x, xs, w, ws, api.LINEAR_PLAIN if act is None else act), act)


def test_inputs_and_outputs_past_32_bit_offsets(api):
    g = np.random.default_rng(13)
    for T, N, K in ((160_000, 14336, 16), (4_400_000, 32, 512)):
        x = torch.ones(T, K, dtype=torch.int8, device="cuda")
        tail = g.integers(-128, 128, (200, K), dtype=np.int8)
        x[-200:] = torch.from_numpy(tail).cuda()
        xs = torch.ones(T, device="cuda")
        w = g.integers(-128, 128, (N, K), dtype=np.int8)
        out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        api.moe_linear_i8(x, xs, torch.from_numpy(w).cuda(), torch.ones(N, device="cuda"), out, _ws())
        want = ref.linear_i8(tail, np.ones(200, np.float32), w, np.ones(N, np.float32))
        assert np.array_equal(out[-200:].float().cpu().numpy(), ref.to_bf16(want))
        first = ref.linear_i8(np.ones((1, K), np.int8), np.ones(1, np.float32), w, np.ones(N, np.float32))
        assert np.array_equal(out[:1].float().cpu().numpy(), ref.to_bf16(first))
        del x, xs, out


@pytest.mark.parametrize("T,N,K,act", [(1, 4224, 2816, 1), (24, 2816, 2112, None), (700, 512, 256, 0)])
def test_captured_replayed_and_on_two_streams_at_once(api, T, N, K, act):
    x, xs, w, ws = _inputs(T, N, K, 14)
    c = [torch.from_numpy(v).cuda() for v in (x, xs, w, ws)]
    n = N if act is None else N // 2
    want = _run(api, x, xs, w, ws, act)[0]
    work = _ws()   # two graphs share the error word
    outs = [torch.zeros(T, n, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.moe_linear_i8(*c, o, work, gate_act=act)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert api.moe_read_error(work) == 0
