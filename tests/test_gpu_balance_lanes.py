"""Balanced routing where few lanes hold all that can be chosen: one or two kept groups, of
which a lane may have to give eight experts and more."""
import numpy as np
import pytest
import torch

import operators_ref as ref

pytestmark = pytest.mark.gpu

RTOL, ATOL = 2.0 ** -23, 2.0 ** -149   # fp64 weights, rounded once


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_ffn_06_b200 import api as a
    return a


# E, k, n_group, topk_group
CASES = [(256, 8, 8, 1), (256, 8, 8, 2), (256, 8, 4, 1), (256, 16, 8, 1), (512, 8, 32, 1),
         (512, 16, 32, 1), (512, 16, 8, 1), (512, 16, 8, 2), (512, 16, 8, 4), (512, 16, 2, 1),
         (510, 9, 17, 1), (500, 8, 5, 1), (96, 8, 3, 1), (512, 32, 16, 1), (256, 7, 8, 1),
         (256, 12, 8, 4), (256, 13, 8, 4)]


@pytest.mark.parametrize("E,k,n_group,topk_group", CASES)
@pytest.mark.parametrize("T", [1, 40, 3700])
@pytest.mark.parametrize("scoring", [0, 1])
def test_few_lanes_in_play(api, E, k, n_group, topk_group, T, scoring):
    g = np.random.default_rng(E + k + n_group + T)
    z = g.standard_normal((T, E)).astype(np.float32)
    bias = (0.1 * g.standard_normal(E)).astype(np.float32)
    ids = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    load = torch.full((E,), -5, dtype=torch.int32, device="cuda")
    opts = dict(scoring=scoring, n_group=n_group, topk_group=topk_group, group_top=2)
    api.moe_route_balanced(api.make_shape(T=T, H=8, E=E, k=k, I=8), torch.from_numpy(z).cuda(),
                           torch.from_numpy(bias).cuda(), None, ids, w, load=load,
                           opts=api.balance_opts(**opts))
    want_ids, want, want_load = ref.route(z, k, bias, None, **opts)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert np.array_equal(load.cpu().numpy(), want_load)
    assert (np.abs(w.cpu().numpy().astype(np.float64) - want) <= RTOL * want + ATOL).all()


@pytest.mark.parametrize("T", [9, 33, 64])
def test_the_load_of_few_blocks_called_and_replayed(api, T):
    # called they are a cluster that sums the counts, in a graph they add to zeros
    E, k = 128, 8
    g = np.random.default_rng(T)
    z = torch.zeros(T, E, device="cuda")
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    load = torch.full((E,), -5, dtype=torch.int32, device="cuda")
    s = api.make_shape(T=T, H=8, E=E, k=k, I=8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.moe_route_balanced(s, z, None, None, ids, w, load=load)
    for _ in range(3):
        new = g.standard_normal((T, E)).astype(np.float32)
        want_ids, _, want_load = ref.route(new, k)
        z.copy_(torch.from_numpy(new))
        for go in (graph.replay, lambda: api.moe_route_balanced(s, z, None, None, ids, w, load=load)):
            ids.fill_(-5)
            load.fill_(-5)
            go()
            assert np.array_equal(ids.cpu().numpy(), want_ids)
            assert np.array_equal(load.cpu().numpy(), want_load)
