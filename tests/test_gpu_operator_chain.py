"""The operators next to the expert products run together, as the feed-forward
half of a decoder layer with an INT8 dense MLP and routed experts uses them:

  moe_block_norm (norm before the MLP, int8 codes) -> moe_linear_i8 gated ->
  moe_quantize_rows_i8 -> moe_linear_i8 -> moe_block_norm (norm after, gate,
  residual, norm before the experts) -> router logits -> moe_route_balanced ->
  moe_permute -> moe_expert_ffn -> moe_combine -> moe_block_norm (norm after,
  residual scale, the next layer's norm and codes)

Each step is held to its definition on the inputs it was given (to the bit where the
definition fixes it; the experts' sum within 2e-2 of its RMS, the layer's bar), and
the captured chain to the eager one."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import operators_ref as ref
from parity_util import OUT_TOL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_ffn_06_b200 import api as a
    return a


class Chain:
    def __init__(self, api, T, H, E, k, I, I_dense, seed):
        self.api, self.T, self.H, self.E, self.k, self.I, self.D = api, T, H, E, k, I, I_dense
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        bf = torch.bfloat16
        gamma = lambda: (1 + 0.1 * n(H)).to(bf)  # noqa: E731
        self.r = n(T, H).to(bf)
        self.w_mlp, self.w_mlp_post, self.w_moe, self.w_moe_post, self.w_next = (gamma() for _ in range(5))
        self.gate = (0.5 + 0.1 * n(H)).to(bf)
        self.q13, self.s13 = self.weight(n(2 * I_dense, H) * H ** -0.5)
        self.q2, self.s2 = self.weight(n(H, I_dense) * I_dense ** -0.5)
        self.router_w, self.router_s = n(E, H).to(bf), (0.5 + torch.rand(H, generator=g, device="cuda")).to(bf)
        self.bias = 0.05 * n(E)
        self.w13 = (n(E, 2 * I, H) * 0.02).to(bf)
        self.w2 = (n(E, H, I) * 0.02).to(bf)
        e = lambda *s, dt=bf: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        i8, i32, f32 = torch.int8, torch.int32, torch.float32
        self.shape = api.make_shape(T=T, H=H, E=E, k=k, I=I)
        cap = api.moe_layout_capacity(self.shape)
        self.a_q, self.a_s = e(T, H, dt=i8), e(T, dt=f32)
        self.h, self.h_q, self.h_s = e(T, I_dense), e(T, I_dense, dt=i8), e(T, dt=f32)
        self.y_mlp, self.r1, self.a1 = e(T, H), e(T, H), e(T, H)
        self.logits, self.ids, self.w = e(T, E, dt=f32), e(T, k, dt=i32), e(T, k, dt=f32)
        self.load = e(E, dt=i32)
        self.offsets, self.slots, self.rows = e(E + 1, dt=i32), e(cap, dt=i32), e(T, k, dt=i32)
        self.y_rows, self.y_moe = e(cap, H, dt=f32), e(T, H)
        self.r2, self.a2, self.q2_out, self.s2_out = e(T, H), e(T, H), e(T, H, dt=i8), e(T, dt=f32)
        self.ws = api.alloc_workspace(self.shape)
        self.opts = api.balance_opts(scoring=api.SCORE_SIGMOID, n_group=4, topk_group=2, group_top=2,
                                     factor=2.5)

    def weight(self, w):
        q = torch.empty(w.shape, dtype=torch.int8, device="cuda")
        s = torch.empty(w.shape[0], device="cuda")
        self.api.moe_quantize_rows_i8(w.to(torch.bfloat16), q, s)
        return q, s

    def run(self):
        a, s = self.api, self.shape
        a.moe_block_norm(self.r, pre_w=self.w_mlp, codes=self.a_q, scales=self.a_s)
        a.moe_linear_i8(self.a_q, self.a_s, self.q13, self.s13, self.h, self.ws, gate_act=a.ACT_GELU_TANH)
        a.moe_quantize_rows_i8(self.h, self.h_q, self.h_s)
        a.moe_linear_i8(self.h_q, self.h_s, self.q2, self.s2, self.y_mlp, self.ws)
        a.moe_block_norm(self.r, y=self.y_mlp, post_w=self.w_mlp_post, gate=self.gate, pre_w=self.w_moe,
                         r_out=self.r1, a=self.a1)
        a.moe_router_logits(s, self.r1, self.router_w, self.router_s, 1e-6, self.logits)
        a.moe_route_balanced(s, self.logits, self.bias, None, self.ids, self.w, load=self.load, opts=self.opts)
        a.moe_permute(s, self.ids, self.offsets, self.slots, self.rows, self.ws)
        a.moe_expert_ffn(s, self.a1, self.offsets, self.slots, self.w13, self.w2, None, None, self.y_rows,
                         self.ws)
        a.moe_combine(s, self.y_rows, self.rows, self.w, self.y_moe)
        a.moe_block_norm(self.r1, y=self.y_moe, post_w=self.w_moe_post, alpha=0.75, beta=1.25,
                         pre_w=self.w_next, r_out=self.r2, a=self.a2, codes=self.q2_out, scales=self.s2_out)

    OUTPUTS = ("a_q", "a_s", "h", "y_mlp", "r1", "a1", "logits", "ids", "w", "load", "y_moe", "r2", "a2",
               "q2_out", "s2_out")

    def outputs(self):
        torch.cuda.synchronize()
        assert self.api.moe_read_error(self.ws) == 0
        return {n: getattr(self, n).clone() for n in self.OUTPUTS}

    def check(self):
        f = lambda t: t.float().cpu().numpy()  # noqa: E731
        i = lambda t: t.cpu().numpy()  # noqa: E731
        q, s = ref.quantize_i8(ref.block_norm(f(self.r), pre_w=f(self.w_mlp))[1])
        assert np.array_equal(i(self.a_q), q) and np.array_equal(i(self.a_s), s)
        h = ref.linear_i8(q, s, i(self.q13), i(self.s13), ref.GELU)
        # one bf16 rounding on top of the gated product's own error
        assert (np.abs(f(self.h) - h) <= (2.0 ** -8 + 2.0 ** -12) * np.abs(h) + 1e-30).all()
        q, s = ref.quantize_i8(f(self.h))
        assert np.array_equal(i(self.h_q), q)
        y = ref.to_bf16(ref.linear_i8(q, s, i(self.q2), i(self.s2)))
        assert np.array_equal(f(self.y_mlp), y)
        r1, a1 = ref.block_norm(f(self.r), y=y, post_w=f(self.w_mlp_post), gate=f(self.gate),
                                pre_w=f(self.w_moe))
        assert np.array_equal(f(self.r1), r1) and np.array_equal(f(self.a1), a1)
        ids, w, load = ref.route(i(self.logits), self.k, i(self.bias), scoring=1, n_group=4, topk_group=2,
                                 group_top=2, factor=2.5)
        assert np.array_equal(i(self.ids), ids) and np.array_equal(i(self.load), load)
        assert (np.abs(i(self.w) - w) <= 1e-6 * np.abs(w)).all()
        want = torch.zeros(self.T, self.H, dtype=torch.float64, device="cuda")
        for e in range(self.E):
            t, j = (self.ids == e).nonzero(as_tuple=True)
            x = self.a1[t].double() @ self.w13[e].double().T
            x = torch.nn.functional.silu(x[:, :self.I]) * x[:, self.I:]
            want.index_add_(0, t, (x @ self.w2[e].double().T) * self.w[t, j].double()[:, None])
        rms = float(want.square().mean().sqrt())
        err = (self.y_moe.double() - want).abs() - 2.0 ** -8 * want.abs()
        assert float(err.max()) <= OUT_TOL * rms
        r2, a2 = ref.block_norm(r1, y=f(self.y_moe), post_w=f(self.w_moe_post), alpha=0.75, beta=1.25,
                                pre_w=f(self.w_next))
        assert np.array_equal(f(self.r2), r2) and np.array_equal(f(self.a2), a2)
        q, s = ref.quantize_i8(a2)
        assert np.array_equal(i(self.q2_out), q) and np.array_equal(i(self.s2_out), s)


@pytest.mark.parametrize("T", [1, 13, 70, 333])
def test_feed_forward_half_of_a_layer(api, T):
    c = Chain(api, T, H=512, E=16, k=4, I=96, I_dense=352, seed=T)
    c.run()
    eager = c.outputs()
    c.check()
    # the same, captured once and replayed on other residual rows
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    graph.replay()
    again = c.outputs()
    for n, v in eager.items():
        assert torch.equal(again[n], v), n
    c.r.copy_(torch.randn(c.T, c.H, device="cuda").to(torch.bfloat16))
    graph.replay()
    c.outputs()
    c.check()


FIRST_CALLS = """
import torch
from mixture_experts_ffn_06_b200 import api
g = torch.Generator(device="cuda").manual_seed(1)
T, H, N, E, k = 64, 2048, 512, 64, 6
r = torch.randn(T, H, device="cuda", generator=g).bfloat16()
one = torch.ones(H, device="cuda", dtype=torch.bfloat16)
w = torch.randint(-128, 128, (N, H), dtype=torch.int8, device="cuda", generator=g)
w_s = torch.rand(N, device="cuda", generator=g)
z = torch.randn(T, E, device="cuda", generator=g)
shape = api.make_shape(T=T, H=H, E=E, k=k, I=8)
ws = torch.zeros(256, dtype=torch.uint8, device="cuda")


def buffers():
    return (torch.zeros(T, H, dtype=torch.int8, device="cuda"), torch.zeros(T, device="cuda"),
            torch.zeros(T, N, dtype=torch.bfloat16, device="cuda"),
            torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda"),
            torch.zeros(E, dtype=torch.int32, device="cuda"))


def run(b):
    api.moe_block_norm(r, pre_w=one, codes=b[0], scales=b[1])
    api.moe_quantize_rows_i8(r, b[0], b[1])
    api.moe_linear_i8(b[0], b[1], w, w_s, b[2], ws)
    api.moe_route_balanced(shape, z, None, None, b[3], b[4], load=b[5])


captured, eager = buffers(), buffers()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run(captured)
graph.replay()
run(eager)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, eager))
assert int(captured[5].sum()) == T * k and api.moe_read_error(ws) == 0
"""


def test_first_calls_of_a_process_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, check=True, timeout=300)
