"""A tensor that is left out is refused by name, not by an attribute of None."""
import pytest
import torch


@pytest.fixture(scope="module")
def api():
    from mixture_experts_ffn_06_b200 import build
    build.build()
    from mixture_experts_ffn_06_b200 import api as a
    return a


def test_missing_tensors_are_named(api):
    z, i8 = torch.zeros, torch.int8
    s = api.make_shape(T=4, H=8, E=16, k=2, I=8)
    rows, codes, ws = z(4, 64, dtype=torch.bfloat16), z(4, 64, dtype=i8), z(256, dtype=torch.uint8)
    calls = {
        "logits": lambda: api.moe_route_balanced(s, None, None, None, z(4, 2), z(4, 2)),
        "src": lambda: api.moe_quantize_rows_i8(None, codes, z(4)),
        "x": lambda: api.moe_linear_i8(None, z(4), codes, z(4), rows, ws),
        "w": lambda: api.moe_linear_i8(codes, z(4), None, z(4), rows, ws),
        "ws": lambda: api.moe_linear_i8(codes, z(4), codes, z(4), rows, None),
        "r": lambda: api.moe_block_norm(None, pre_w=rows[0], a=rows),
    }
    for name, call in calls.items():
        with pytest.raises(ValueError, match=f"^{name}: expected"):
            call()
