"""moe_route_balanced on the GPU against its definition in 64 bits.

ids and load have to be equal.  A weight is formed in fp64 and rounded once
(relative 2^-24); without renorm the softmax's denominator is a sum of fp32
exponentials, each within a few ulps of 2^-23, so 1e-6 relative covers both; a
weight below fp32's normal range is rounded to a multiple of 2^-149."""
import numpy as np
import pytest
import torch

import operators_ref as ref

pytestmark = pytest.mark.gpu

RTOL, ATOL = 1e-6, 2.0 ** -149


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_ffn_06_b200 import api as a
    return a


def _cuda(v):
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v, np.float32)).cuda()


def _run(api, z, k, bias=None, scale=None, with_load=True, **opts):
    T, E = z.shape
    ids = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    load = torch.full((E,), -5, dtype=torch.int32, device="cuda") if with_load else None
    api.moe_route_balanced(api.make_shape(T=T, H=8, E=E, k=k, I=8), _cuda(z), _cuda(bias),
                           _cuda(scale), ids, w, load=load,
                           opts=api.balance_opts(**opts) if opts else None)
    torch.cuda.synchronize()
    return ids, w, load


def _check(got, want):
    ids, w, load = got
    rid, rw, rload = want
    assert np.array_equal(ids.cpu().numpy(), rid)
    w = w.cpu().numpy().astype(np.float64)
    assert (np.abs(w - rw) <= RTOL * np.abs(rw) + ATOL).all()
    if load is not None:
        assert np.array_equal(load.cpu().numpy(), rload)


# T, E, k, scoring, n_group, topk_group, group_top, renorm, factor
CASES = [
    (1, 256, 8, 1, 8, 4, 2, True, 2.5),     # DeepSeek-V3 routing, one token
    (130, 256, 8, 1, 8, 4, 2, True, 2.5),
    (77, 128, 8, 0, 1, 1, 1, True, 1.0),
    (64, 8, 2, 0, 1, 1, 1, False, 1.0),
    (33, 64, 6, 0, 1, 1, 1, False, 16.0),
    (9, 160, 6, 0, 8, 3, 1, False, 16.0),   # groups by their best expert
    (41, 40, 5, 1, 20, 7, 2, True, 1.0),    # groups of two
    (41, 66, 4, 1, 22, 5, 2, False, -1.5),  # groups of three; a negative factor
    (37, 32, 4, 1, 32, 4, 2, True, 1.0),    # groups of one expert
    (19, 512, 32, 1, 32, 32, 2, True, 1.0),  # the largest E, k and n_group
    (5, 1, 1, 0, 1, 1, 1, True, 1.0),       # one expert
    (23, 33, 32, 0, 1, 1, 1, True, 1.0),    # nearly every expert chosen
    (12, 500, 31, 0, 4, 1, 1, True, 1.0),   # one kept group
    (2049, 96, 3, 1, 3, 2, 2, False, 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d-E%d-k%d-s%d-g%d" % c[:5])
@pytest.mark.parametrize("with_bias", [True, False])
def test_matches_the_definition(api, case, with_bias):
    T, E, k, scoring, n_group, topk_group, group_top, renorm, factor = case
    g = np.random.default_rng(E * 7 + T)
    z = g.standard_normal((T, E)).astype(np.float32)
    bias = (0.1 * g.standard_normal(E)).astype(np.float32) if with_bias else None
    scale = (0.5 + g.random(E)).astype(np.float32) if with_bias else None
    opts = dict(scoring=scoring, n_group=n_group, topk_group=topk_group, group_top=group_top,
                renorm=renorm, factor=factor)
    _check(_run(api, z, k, bias, scale, **opts), ref.route(z, k, bias, scale, **opts))


# many tokens: 8 or 16 lanes to a token, experts read in quads or one by one
MANY = [
    (3701, 8, 2, 0, 1, 1, 1, True, 1.0),
    (3701, 64, 6, 0, 1, 1, 1, False, 1.0),
    (3703, 66, 8, 1, 1, 1, 1, True, 1.0),
    (3600, 128, 8, 1, 1, 1, 1, True, 1.0),
    (3700, 256, 8, 1, 8, 4, 2, True, 2.5),
    (3700, 250, 8, 0, 1, 1, 1, True, 1.0),
    (3700, 256, 8, 0, 4, 3, 1, False, 1.0),
    (3700, 512, 8, 1, 1, 1, 1, True, 1.0),
    (3700, 500, 7, 1, 5, 2, 2, True, 1.0),
    (3700, 96, 8, 1, 3, 1, 2, True, 1.0),
    (3700, 160, 6, 0, 16, 5, 2, True, 1.0),
    (3700, 510, 8, 1, 17, 9, 2, True, 1.0),
    (3700, 128, 12, 0, 1, 1, 1, True, 1.0),
    (20000, 32, 4, 1, 1, 1, 1, True, 1.0),
    # 16 lanes to a token for up to 16 experts, a warp for more
    (3700, 24, 16, 0, 1, 1, 1, True, 1.0),
    (3701, 256, 16, 1, 8, 4, 2, True, 2.5),
    (3700, 510, 9, 1, 1, 1, 1, False, 1.0),
    (3700, 512, 16, 0, 4, 2, 2, True, 1.0),
    (3700, 64, 17, 1, 1, 1, 1, True, 1.0),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "T%d-E%d-k%d-s%d-g%d" % c[:5])
def test_many_tokens(api, case):
    test_matches_the_definition(api, case, True)


@pytest.mark.parametrize("T", [40, 3700])
@pytest.mark.parametrize("scoring", [0, 1])
@pytest.mark.parametrize("spread", [0.0, 1e-7, 1e-3])
@pytest.mark.parametrize("k", [8, 15])
def test_the_largest_together(api, T, scoring, spread, k):
    # the largest logits on the experts that one lane holds, apart by nothing, by less
    # than fp32 tells and by more; and more near equals than a candidate list takes
    g = np.random.default_rng(11)
    E = 256
    z = g.standard_normal((T, E)).astype(np.float32)
    one_lane = [q * 32 + i for q in range(8) for i in range(4)]
    for t in range(T):
        at = one_lane[:9 + t % 20] if t % 2 else g.permutation(E)[:6 + t % 30]
        z[t, at] = (4.0 + spread * g.standard_normal(len(at))).astype(np.float32)
    for n_group in (1, 8):
        opts = dict(scoring=scoring, n_group=n_group, topk_group=4 if n_group > 1 else 1, group_top=2)
        _check(_run(api, z, k, **opts), ref.route(z, k, **opts))


@pytest.mark.parametrize("T", [70, 3700])
@pytest.mark.parametrize("off_logits,off_bias", [(1, 0), (0, 3), (2, 1)])
def test_rows_off_a_16_byte_boundary(api, T, off_logits, off_bias):
    g = np.random.default_rng(29)
    E, k = 256, 8
    z = g.standard_normal((T, E)).astype(np.float32)
    bias = (0.1 * g.standard_normal(E)).astype(np.float32)
    zd = torch.zeros(T * E + 4, device="cuda")[off_logits:off_logits + T * E].view(T, E)
    bd = torch.zeros(E + 4, device="cuda")[off_bias:off_bias + E]
    zd.copy_(torch.from_numpy(z))
    bd.copy_(torch.from_numpy(bias))
    opts = dict(scoring=1, n_group=8, topk_group=4, group_top=2)
    ids = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    load = torch.full((E,), -5, dtype=torch.int32, device="cuda")
    api.moe_route_balanced(api.make_shape(T=T, H=8, E=E, k=k, I=8), zd, bd, None, ids, w,
                           load=load, opts=api.balance_opts(**opts))
    _check((ids, w, load), ref.route(z, k, bias, None, **opts))


def test_defaults_without_options_and_load(api):
    z = np.random.default_rng(0).standard_normal((50, 24)).astype(np.float32)
    _check(_run(api, z, 3, with_load=False), ref.route(z, 3))


@pytest.mark.parametrize("T", [300, 3700])
@pytest.mark.parametrize("scoring", [0, 1])
def test_close_choices_are_ranked_as_real_numbers(api, scoring, T):
    # scores that fp32 cannot tell apart: logits one ulp apart, with biases that
    # bring far scores together to within 1e-9
    g = np.random.default_rng(5)
    E, k = 64, 8
    z = np.full((T, E), 0.5, np.float32)
    steps = g.permuted(np.tile(np.arange(E), (T, 1)), axis=1)
    z = (z.view(np.uint32) + steps.astype(np.uint32)).view(np.float32)
    _check(_run(api, z, k, scoring=scoring), ref.route(z, k, scoring=scoring))
    z = g.standard_normal((T, E)).astype(np.float32)
    z[1:] = z[0] + 1e-7 * g.standard_normal((T - 1, E)).astype(np.float32)
    s = 1.0 / (1.0 + np.exp(-z[0].astype(np.float64)))
    if scoring == 0:
        s = np.exp(z[0].astype(np.float64))
        s /= s.sum()
    bias = (1.0 - s).astype(np.float32)
    _check(_run(api, z, k, bias, scoring=scoring), ref.route(z, k, bias, scoring=scoring))


@pytest.mark.parametrize("n_group,topk_group,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("scoring", [0, 1])
@pytest.mark.parametrize("T", [200, 3700])
def test_equal_values_go_to_the_lower_id(api, T, scoring, n_group, topk_group, group_top):
    g = np.random.default_rng(6)
    z = g.integers(-1, 2, (T, 48)).astype(np.float32)  # many equal logits
    z[0] = 0.0
    z[1] = -0.0
    z[2] = 60.0   # sigmoid is 1 in fp64
    opts = dict(scoring=scoring, n_group=n_group, topk_group=topk_group, group_top=group_top)
    _check(_run(api, z, 5, **opts), ref.route(z, 5, **opts))


@pytest.mark.parametrize("n_group,topk_group,group_top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
@pytest.mark.parametrize("scoring", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T", [40, 3700])
def test_masked_and_special_logits(api, T, scoring, renorm, n_group, topk_group, group_top):
    g = np.random.default_rng(7)
    E, k = 64, 6
    z = g.standard_normal((T, E)).astype(np.float32)
    z[0] = -np.inf                       # nothing available
    z[1] = np.nan
    z[2, :E - 3] = -np.inf               # fewer available than k
    z[3, ::2] = np.nan
    z[4, 5] = np.inf
    z[5, [7, 40]] = np.inf
    z[6] = np.finfo(np.float32).min      # the type's lowest value is available
    z[7, 1:] = np.finfo(np.float32).min
    z[8] = np.float32(-800.0)            # scores underflow in fp64
    z[9, 3] = 300.0
    z[10, 8:] = -np.inf                  # one available group
    z[11, 1:] = -np.inf                  # one available expert
    z[12] = np.inf
    z[13, :32] = -np.inf
    z[13, 32:] = np.nan
    bias = (0.05 * g.standard_normal(E)).astype(np.float32)
    opts = dict(scoring=scoring, renorm=renorm, n_group=n_group, topk_group=topk_group,
                group_top=group_top)
    for b in (None, bias):
        ids, w, load = _run(api, z, k, b, **opts)
        _check((ids, w, load), ref.route(z, k, b, **opts))
        got = np.sort(ids.cpu().numpy(), axis=1)
        assert (got >= 0).all() and (got < E).all() and (np.diff(got, axis=1) > 0).all()
        assert (w[[0, 1, 13]] == 0).all()


def test_a_bias_that_is_not_finite(api):
    g = np.random.default_rng(8)
    z = g.standard_normal((30, 32)).astype(np.float32)
    bias = (0.1 * g.standard_normal(32)).astype(np.float32)
    bias[3], bias[4], bias[9] = np.inf, -np.inf, np.nan
    for n_group in (1, 4):
        opts = dict(scoring=1, n_group=n_group, topk_group=2 if n_group > 1 else 1, group_top=2)
        _check(_run(api, z, 4, bias, **opts), ref.route(z, 4, bias, **opts))


def test_the_bias_moves_the_choice_and_never_the_weight(api):
    z = np.zeros((3, 4), np.float32)
    z[:] = [0.0, 1.0, 2.0, 3.0]
    ids, w, load = _run(api, z, 2, np.array([5.0, 4.0, 0.0, 0.0], np.float32), scoring=1)
    assert ids.tolist() == [[0, 1]] * 3 and load.tolist() == [3, 3, 0, 0]
    s = 1 / (1 + np.exp(-np.array([0.0, 1.0])))
    assert np.allclose(w.cpu().numpy(), s / s.sum(), rtol=RTOL, atol=0)


@pytest.mark.parametrize("T", [8, 9, 17, 25, 33, 41, 49, 57, 64, 65])
def test_the_load_of_one_to_nine_blocks(api, T):
    z = np.random.default_rng(T).standard_normal((T, 300)).astype(np.float32)
    for _ in range(3):
        _check(_run(api, z, 8), ref.route(z, 8))


def test_an_empty_batch_clears_the_load(api):
    load = torch.full((16,), 9, dtype=torch.int32, device="cuda")
    e = torch.empty(0, device="cuda")
    api.moe_route_balanced(api.make_shape(T=0, H=8, E=16, k=2, I=8), e, None, None,
                           e.to(torch.int32), e, load=load)
    assert load.tolist() == [0] * 16


def test_rows_past_32_bit_offsets(api):
    T, E, k = 8_400_000, 256, 8   # 2.15e9 logits
    z = torch.zeros(T, E, device="cuda")
    z[:, 17] = 1.0
    tail = torch.randn(100, E, device="cuda")
    z[-100:] = tail
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    load = torch.empty(E, dtype=torch.int32, device="cuda")
    api.moe_route_balanced(api.make_shape(T=T, H=8, E=E, k=k, I=8), z, None, None, ids, w,
                           load=load)
    _check((ids[-100:], w[-100:], None), ref.route(tail.cpu().numpy(), k))
    assert int(load.sum(dtype=torch.int64)) == T * k and int(load[17]) >= T - 100


def test_captured_and_replayed(api):
    g = np.random.default_rng(9)
    T, E, k = 700, 128, 8
    opts = dict(scoring=1, n_group=8, topk_group=4, group_top=2)
    bias = (0.1 * g.standard_normal(E)).astype(np.float32)
    z = torch.zeros(T, E, device="cuda")
    b = _cuda(bias)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    load = torch.empty(E, dtype=torch.int32, device="cuda")
    s, o = api.make_shape(T=T, H=8, E=E, k=k, I=8), api.balance_opts(**opts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_route_balanced(s, z, b, None, ids, w, load=load, opts=o)
    for _ in range(2):
        new = g.standard_normal((T, E)).astype(np.float32)
        z.copy_(torch.from_numpy(new))
        graph.replay()
        torch.cuda.synchronize()
        _check((ids, w, load), ref.route(new, k, bias, **opts))


def test_repeated_calls_agree_bit_for_bit_on_another_stream(api):
    z = np.random.default_rng(10).standard_normal((5000, 64)).astype(np.float32)
    first = _run(api, z, 6, scoring=0, renorm=False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = _run(api, z, 6, scoring=0, renorm=False)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
