"""The three operators in a row, as a mixture-of-experts layer runs them: the
8-bit norm, the router on its logits, the experts, the combine step. Eager and
as a CUDA graph. Needs a GPU."""

import numpy as np
import pytest
import torch

import reduce_rmsnorm_gb300 as tw
import synth
from norm_parity import bits16, check_bf16, check_residual, y_error
from oracle import experts as oracle
from test_gpu_q8 import outputs, same

pytestmark = pytest.mark.gpu
EPS = synth.EPS


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from reduce_rmsnorm_gb300 import build
    build.build()
    tw.lib()
    tw.tw_device_status(reset=True)
    yield
    assert tw.tw_device_status(reset=True) == 0


class Layer:
    """T tokens, E experts that each scale a token by a vector of their own."""

    def __init__(self, T, H, E, K, N, seed):
        p, r, g = synth.make_inputs(T, H, N, 0.2, seed=seed)
        gen = torch.Generator().manual_seed(seed)
        self.T, self.H, self.E, self.K = T, H, E, K
        self.P, self.R0, self.G = p.cuda(), r.cuda(), g.cuda()
        self.R = self.R0.clone()
        self.router = (torch.randn(H, E, generator=gen) / H ** 0.5).cuda()
        self.expert = torch.randn(E, H, generator=gen).bfloat16().cuda()
        self.bias = (0.01 * torch.randn(E, generator=gen)).cuda()
        self.q, self.s = outputs(T, H, 32, "e8m0")
        self.logits = torch.empty(T, E, device="cuda")
        self.w = torch.empty(T, K, device="cuda")
        self.ids = torch.empty(T, K, device="cuda", dtype=torch.int32)
        self.rows = torch.arange(T * K, device="cuda", dtype=torch.int32).view(T, K)
        self.x = torch.empty(T * K, H, device="cuda", dtype=torch.bfloat16)
        self.out = torch.empty(T, H, device="cuda", dtype=torch.bfloat16)
        torch.cuda.synchronize()

    def step(self):
        T, H = self.T, self.H
        tw.tw_fused_reduce_residual_rmsnorm_q8(self.P, self.R, self.G, EPS, self.q, self.s, group=32)
        y = self.q.float().view(T, -1, 32) * self.s.float().unsqueeze(2)
        y = y.view(T, H)
        torch.matmul(y, self.router, out=self.logits)
        tw.tw_route_experts(self.logits, self.w, self.ids, bias=self.bias, scoring="sigmoid",
                            n_groups=4, top_groups=2, group_top=2, scale=2.0)
        self.x.copy_((y[:, None, :] * self.expert[self.ids.long()]).view(-1, H))
        self.mid = self.R.clone()
        tw.tw_combine_residual_rmsnorm(self.x, self.rows, self.w, self.R, self.G, EPS, self.out)


def test_layer_against_the_oracle():
    m = Layer(70, 1024, 16, 3, 2, seed=1)
    m.step()
    torch.cuda.synchronize()
    want, _ = oracle.route(m.logits.cpu().double().numpy(), 3, m.bias.cpu().double().numpy(),
                           scoring="sigmoid", n_groups=4, top_groups=2, group_top=2, scale=2.0)
    assert np.array_equal(m.ids.cpu().numpy(), want)
    z, y, absum = oracle.combine(bits16(m.x), m.rows.cpu().numpy(), m.w.cpu().numpy(), [],
                                 bits16(m.mid), bits16(m.G), EPS)
    check_residual(z, absum, 4, m.R)
    check_bf16(y, y_error(z, y, absum, 4, bits16(m.G), EPS), m.out)


def test_two_captured_layers_replay_as_eager_runs():
    """Two layers captured into two graphs, replayed in turn and at once on
    two streams; the operators keep no workspace that they could share."""
    layers = [Layer(40, 512, 16, 3, 2, seed=2), Layer(90, 2048, 16, 4, 1, seed=3)]
    eager = []
    for m in layers:
        m.step()
        torch.cuda.synchronize()
        eager.append((m.q.clone(), m.s.clone(), m.ids.clone(), m.w.clone(), m.R.clone(), m.out.clone()))
    graphs = []
    for m in layers:
        m.R.copy_(m.R0)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.R.copy_(m.R0)
            m.step()
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for m in layers:
            m.out.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for m, (q, s, ids, w, R, out) in zip(layers, eager):
            assert same(m.q, q) and same(m.s, s) and torch.equal(m.ids, ids)
            assert torch.equal(m.w, w) and torch.equal(m.R, R) and torch.equal(m.out, out)


def test_prepared_calls_equal_the_plain_ones():
    T, H, E, K = 30, 1024, 32, 4
    m = Layer(T, H, E, K, 2, seed=5)
    m.x.normal_()
    m.logits.normal_()
    torch.cuda.synchronize()

    def fresh():
        R = m.R0.clone()
        q, s = outputs(T, H, 128, "f32")
        return R, q, s, torch.empty_like(m.out), torch.empty_like(m.w), torch.empty_like(m.ids)

    R, q, s, out, w, ids = fresh()
    tw.tw_fused_reduce_residual_rmsnorm_q8(m.P, R, m.G, EPS, q, s, group=128)
    tw.tw_route_experts(m.logits, w, ids, bias=m.bias)
    tw.tw_combine_residual_rmsnorm(m.x, m.rows, w, R, m.G, EPS, out, partials=m.P)
    R2, q2, s2, out2, w2, ids2 = fresh()
    calls = [tw.FusedQ8Call(m.P, R2, m.G, EPS, q2, s2, group=128),
             tw.RouteCall(m.logits, w2, ids2, bias=m.bias),
             tw.CombineCall(m.x, m.rows, w2, R2, m.G, EPS, out2, partials=m.P)]
    for c in calls:
        c()
    torch.cuda.synchronize()
    assert same(q, q2) and same(s, s2) and torch.equal(w, w2) and torch.equal(ids, ids2)
    assert torch.equal(out, out2) and torch.equal(R, R2)
    q3, s3 = outputs(T, H, 128, "f32")
    q4, s4 = outputs(T, H, 128, "f32")
    Ra, Rb = m.R0.clone(), m.R0.clone()
    tw.tw_combine_residual_rmsnorm_q8(m.x, m.rows, w, Ra, m.G, EPS, q3, s3, group=128)
    tw.CombineQ8Call(m.x, m.rows, w, Rb, m.G, EPS, q4, s4, group=128)()
    torch.cuda.synchronize()
    assert same(q3, q4) and same(s3, s4) and torch.equal(Ra, Rb)
