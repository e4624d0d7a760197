"""Refusals of the operators next to the expert products, on the host before any
launch: no GPU needed, the pointers are never dereferenced."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
FAKE, ODD8, ODD4 = P(1 << 20), P((1 << 20) + 8), P((1 << 20) + 4)

FIELDS = {
    "moe_balance_opts": ["scoring", "n_group", "topk_group", "group_top", "renorm", "factor"],
    "moe_block_norm_params": ["y", "r", "post_w", "gate", "token_gate", "pre_w", "alpha", "beta",
                              "post_eps", "pre_eps", "r_out", "a", "codes", "scales"],
}


@pytest.fixture(scope="module")
def api():
    from mixture_experts_ffn_06_b200 import build
    build.build()
    from mixture_experts_ffn_06_b200 import api as a
    return a


def test_ctypes_mirrors_match_the_header(api, tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe.h"', "int main(void) {"]
    for st, fields in FIELDS.items():
        lines.append(f'  printf("{st} size %zu\\n", sizeof({st}));')
        lines += [f'  printf("{st} {f} %zu\\n", offsetof({st}, {f}));' for f in fields]
    lines += ['  printf("c max_row %d\\n", MOE_MAX_ROW);', '  printf("c max_k %d\\n", MOE_LINEAR_MAX_K);',
              '  printf("c plain %d\\n", MOE_LINEAR_PLAIN);', "  return 0;", "}"]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines) + "\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe),
                           str(src)])
    table = {}
    for line in subprocess.check_output([str(exe)], text=True).splitlines():
        st, f, v = line.split()
        table[(st, f)] = int(v)
    for st, fields in FIELDS.items():
        cls = getattr(api, st)
        assert ctypes.sizeof(cls) == table[(st, "size")]
        for f in fields:
            assert getattr(cls, f).offset == table[(st, f)], (st, f)
    assert (api.MAX_ROW, api.LINEAR_MAX_K, api.LINEAR_PLAIN) == tuple(
        table[("c", n)] for n in ("max_row", "max_k", "plain"))


@pytest.mark.parametrize("kw,status", [
    (dict(scoring=2), 1), (dict(scoring=-1), 1), (dict(n_group=-1), 1),
    (dict(n_group=33, topk_group=1), 2), (dict(n_group=3), 1),          # 16 % 3
    (dict(n_group=4, topk_group=0), 1), (dict(n_group=4, topk_group=5), 1),
    (dict(n_group=4, topk_group=2, group_top=0), 1),
    (dict(n_group=4, topk_group=2, group_top=3), 1),
    (dict(n_group=16, topk_group=1, group_top=2), 1),                   # k = 2 of one expert
    (dict(factor=float("nan")), 1), (dict(factor=float("inf")), 1),
])
def test_balanced_routing_refuses_bad_options(api, kw, status):
    s = api.make_shape(T=4, H=64, E=16, k=2, I=8)
    f = api.lib.moe_route_balanced
    assert f(s, FAKE, FAKE, FAKE, api.balance_opts(**kw), FAKE, FAKE, None, None) == status


def test_balanced_routing_refuses_bad_arguments(api):
    f = api.lib.moe_route_balanced
    s = api.make_shape(T=4, H=64, E=16, k=2, I=8)
    assert f(None, FAKE, None, None, None, FAKE, FAKE, None, None) == 1
    assert f(s, None, None, None, None, FAKE, FAKE, None, None) == 1
    assert f(s, FAKE, None, None, None, None, FAKE, None, None) == 1
    assert f(s, FAKE, None, None, None, FAKE, None, None, None) == 1
    for kw, status in ((dict(E=513), 2), (dict(E=64, k=33), 2), (dict(k=17), 1), (dict(T=-1), 1),
                       (dict(T=1 << 24), 2)):
        bad = api.make_shape(**{**dict(T=4, H=64, E=16, k=2, I=8), **kw})
        assert f(bad, FAKE, None, None, None, FAKE, FAKE, None, None) == status
    empty = api.make_shape(T=0, H=64, E=16, k=2, I=8)
    assert f(empty, None, None, None, None, None, None, None, None) == 0


def test_i8_quantiser_refuses_bad_arguments(api):
    f = api.lib.moe_quantize_rows_i8
    assert f(FAKE, 4, 12, FAKE, FAKE, None) == 1
    assert f(FAKE, -1, 16, FAKE, FAKE, None) == 1
    assert f(FAKE, 4, 0, FAKE, FAKE, None) == 1
    assert f(FAKE, 4, api.MAX_ROW + 8, FAKE, FAKE, None) == 2
    assert f(FAKE, 1 << 31, 16, FAKE, FAKE, None) == 2
    assert f(None, 4, 16, FAKE, FAKE, None) == 1
    assert f(FAKE, 4, 16, None, FAKE, None) == 1
    assert f(FAKE, 4, 16, FAKE, None, None) == 1
    assert f(ODD8, 4, 16, FAKE, FAKE, None) == 1
    assert f(FAKE, 4, 16, ODD4, FAKE, None) == 1
    assert f(None, 0, 16, None, None, None) == 0


def test_linear_i8_refuses_bad_arguments(api):
    f = api.lib.moe_linear_i8
    good = dict(T=4, N=32, K=64, x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, act=-1, out=FAKE, o32=None,
                work=FAKE, n=256)

    def call(**kw):
        a = {**good, **kw}
        return f(a["T"], a["N"], a["K"], a["x"], a["xs"], a["w"], a["ws"], a["act"], a["out"],
                 a["o32"], a["work"], a["n"], None)

    for kw in (dict(T=-1), dict(N=0), dict(K=0), dict(act=2), dict(act=-2), dict(act=0, N=31),
               dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(out=None),
               dict(work=None), dict(work=ODD8), dict(x=ODD8), dict(w=ODD8), dict(out=ODD8),
               dict(o32=ODD8)):
        assert call(**kw) == 1, kw
    for kw in (dict(K=24), dict(K=api.LINEAR_MAX_K + 16), dict(T=1 << 24), dict(N=1 << 22)):
        assert call(**kw) == 2, kw
    assert call(n=255) == 3
    assert call(T=0, x=None, out=None) == 0


def test_block_norm_refuses_bad_arguments(api):
    good = dict(y=FAKE, r=FAKE, post_w=FAKE, gate=FAKE, token_gate=FAKE, pre_w=FAKE, alpha=1.0,
                beta=1.0, post_eps=1e-6, pre_eps=1e-6, r_out=FAKE, a=FAKE, codes=FAKE, scales=FAKE)

    def call(T=4, H=64, **kw):
        a = {**good, **kw}
        return api.lib.moe_block_norm(T, H, api.moe_block_norm_params(*(a[n] for n in good)), None)

    assert api.lib.moe_block_norm(4, 64, None, None) == 1
    for kw in (dict(T=-1), dict(H=0), dict(r=None), dict(r_out=None), dict(y=None),
               dict(y=None, post_w=None, gate=None, token_gate=None),
               dict(y=None, post_w=None, gate=None, r_out=None), dict(pre_w=None),
               dict(pre_w=None, a=None), dict(pre_w=None, a=None, codes=None),
               dict(a=None, codes=None, scales=None), dict(codes=None), dict(scales=None),
               dict(y=None, post_w=None, gate=None, token_gate=None, r_out=None, pre_w=None, a=None,
                    codes=None, scales=None),
               dict(alpha=float("inf")), dict(beta=float("nan")), dict(post_eps=-1.0),
               dict(pre_eps=float("nan")), dict(pre_eps=float("inf"))):
        assert call(**kw) == 1, kw
    for n in ("y", "r", "post_w", "gate", "pre_w", "r_out", "a"):
        assert call(**{n: ODD8}) == 1, n
    assert call(codes=ODD4) == 1
    for kw in (dict(H=60), dict(H=api.MAX_ROW + 8), dict(T=1 << 24)):
        assert call(**kw) == 2, kw
    assert call(T=0) == 0


def test_the_binding_refuses_wrong_tensors(api):
    bf, i8 = torch.bfloat16, torch.int8
    r = torch.zeros(4, 64, dtype=bf)
    w = torch.ones(64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        api.moe_block_norm(r, pre_w=w, a=r.clone())
    with pytest.raises(ValueError, match="y: expected a contiguous"):
        api.moe_block_norm(r, y=r[:3], pre_w=w, a=r)
    with pytest.raises(ValueError, match="src"):
        api.moe_quantize_rows_i8(r.float(), r.to(i8), torch.zeros(4))
    with pytest.raises(ValueError, match="src"):
        api.moe_quantize_rows_i8(torch.zeros(64, 4, dtype=bf).t(), r.to(i8), torch.zeros(4))
    s = api.make_shape(T=4, H=8, E=16, k=2, I=8)
    with pytest.raises(ValueError, match="logits"):
        api.moe_route_balanced(s, torch.zeros(4, 15), None, None, torch.zeros(4, 2), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="x"):
        api.moe_linear_i8(r, torch.zeros(4), r, torch.zeros(4), r, torch.zeros(256, dtype=torch.uint8))


def test_the_binding_refuses_sizes_past_32_bits(api):
    # as a C int they would arrive as 16 (no memory behind these tensors)
    def meta(dtype, *shape):
        return torch.empty(shape, dtype=dtype, device="meta")

    big, i8, bf, f32 = (1 << 32) + 16, torch.int8, torch.bfloat16, torch.float32
    ws = meta(torch.uint8, 256)
    for call in (lambda: api.moe_linear_i8(meta(i8, 1, big), meta(f32, 1), meta(i8, 1, big),
                                           meta(f32, 1), meta(bf, 1, 1), ws),
                 lambda: api.moe_linear_i8(meta(i8, 1, 16), meta(f32, 1), meta(i8, big, 16),
                                           meta(f32, big), meta(bf, 1, big), ws),
                 lambda: api.moe_quantize_rows_i8(meta(bf, 1, big), meta(i8, 1, big), meta(f32, 1)),
                 lambda: api.moe_block_norm(meta(bf, 1, big), pre_w=meta(bf, big), a=meta(bf, 1, big))):
        with pytest.raises(api.MoEError) as e:
            call()
        assert e.value.status == 2
