"""The weights of moe_route_balanced that are not renormalised, to the last bits.

A weight is exp / denominator in fp64 and rounded once (2^-24).  The denominator's terms
are 2^n (1 + r + q) with 1 + r exact, r at most 0.347 and q below 0.071: the series stops
below 2^-27 of a term, q takes three roundings and its sum with the rest two, each 2^-24 of 0.071,
0.36 x 2^-24 in all and over a term of at least 0.7 half a rounding: 2^-25."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

RTOL, ATOL = 2.0 ** -24 + 2.0 ** -25, 2.0 ** -149


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_ffn_06_b200 import api as a
    return a


def _logits(kind, T, E):
    g = np.random.default_rng(T + E)
    z = g.standard_normal((T, E))
    if kind == "wide":
        z = g.uniform(-200, 200, (T, E))
    elif kind == "level":
        z = 0.01 * z
    elif kind == "offset":
        z = 1.0e4 + 3.0 * z
    z = (4 * z if kind == "normal" else z).astype(np.float32)
    if kind == "holes":
        z[g.random((T, E)) < 0.5] = -np.inf
        z[g.random((T, E)) < 0.1] = np.nan
        z[0], z[1], z[2, 1:] = -np.inf, np.nan, np.finfo(np.float32).min
        z[3], z[4, E // 2] = np.finfo(np.float32).max, np.inf
        z[5] = np.finfo(np.float32).min
    return z


def _definition(z, k):
    """ids and weights of the softmax over what is available, in 64 bits."""
    z = np.minimum(z, np.finfo(np.float32).max).astype(np.float64)
    avail = z > -np.inf
    top = np.max(np.where(avail, z, -np.inf), axis=1, keepdims=True)
    e = np.zeros_like(z)
    np.exp(np.subtract(z, np.where(avail, top, 0.0), where=avail, out=np.zeros_like(z)), where=avail, out=e)
    s = e / np.maximum(e.sum(axis=1, keepdims=True), np.finfo(np.float64).tiny)
    ids = np.argsort(-np.where(avail, s, -np.inf), axis=1, kind="stable")[:, :k]
    return ids, np.take_along_axis(s, ids, 1)


@pytest.mark.parametrize("kind", ["normal", "wide", "level", "offset", "holes"])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (8, 8), (33, 4), (64, 6), (255, 16), (512, 8)])
@pytest.mark.parametrize("T", [6, 3700, 16384])
def test_weights_of_the_whole_softmax(api, kind, E, k, T):
    z = _logits(kind, T, E)
    ids = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    api.moe_route_balanced(api.make_shape(T=T, H=8, E=E, k=k, I=8), torch.from_numpy(z).cuda(), None,
                           None, ids, w, opts=api.balance_opts(renorm=False))
    want_ids, want = _definition(z, k)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert (np.abs(w.cpu().numpy().astype(np.float64) - want) <= RTOL * want + ATOL).all()
