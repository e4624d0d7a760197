"""Int8 products on the forms that the small sizes do not reach."""
import pytest
import torch

pytestmark = pytest.mark.gpu


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
