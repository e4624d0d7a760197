"""Rows whose sum of squares lies on the border between two fp32 means: the order of the
sum, which depends on the number of rows, may decide between the two, and nothing else."""
import numpy as np
import pytest
import torch

import operators_ref as ref

pytestmark = pytest.mark.gpu

H, N = 2048, 400


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_ffn_06_b200 import api as a
    return a


def border_rows():
    """Squares that sum to 2048 + 2^-13, half way between the means 1 and 1 + 2^-23, and some
    2^-50 to 2^-42 more in small ones."""
    g = np.random.default_rng(31)
    rows = np.zeros((N, H), np.float32)
    for t in range(N):
        tiny = 30 + int(g.integers(0, 400))
        # with ones and a few twos: n ones + 4 m = 2048, n + m + 2 + tiny = H
        m = -(-(2 + tiny) // 3)
        v = np.concatenate([np.full(m, 2.0), np.full(2048 - 4 * m, 1.0), np.full(2, 2.0 ** -7)])
        v = np.concatenate([v, np.full(H - len(v), 2.0 ** -25)]).astype(np.float32)
        rows[t] = g.permutation(v)
    return rows


def test_the_border_rows_lie_on_the_border():
    v = border_rows().astype(np.float64)
    small = (v * v).copy()
    small[small > 2.0 ** -20] = 0.0
    assert ((v * v).sum(1) >= 2048.0 + 2.0 ** -13).all()
    assert (np.sort(v * v, 1)[:, ::-1].sum(1) - 2048.0 - 2.0 ** -13 < 2.0 ** -40).all()
    assert (small.sum(1) > 0).all()


def test_the_order_of_the_sum_moves_a_row_to_the_next_mean_at_most(api):
    rows = border_rows()
    x = torch.from_numpy(rows).to(torch.bfloat16).cuda()
    w = (1.0 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16)
    wf = w.float().numpy()
    inv = [np.float32(1) / np.sqrt(np.float32(m) + np.float32(1e-6)) for m in (1.0, 1.0 + 2.0 ** -23)]
    want = [ref.to_bf16((rows * i) * wf) for i in inv]

    def run(r):
        a = torch.empty_like(r)
        api.moe_block_norm(r, pre_w=w.cuda(), a=a)
        return a

    many = run(x)
    assert torch.equal(many, run(x))
    for got in (many, torch.cat([run(x[i:i + 100]) for i in range(0, N, 100)]), run(x.repeat(3, 1))[N:2 * N]):
        g = got.float().cpu().numpy()
        assert ((g == want[0]).all(1) | (g == want[1]).all(1)).all()
