"""The 8-bit step (tw_fused_reduce_residual_rmsnorm_q8) against the fp64
oracle and against the bf16 step. Needs a GPU."""

import numpy as np
import pytest
import torch

import reduce_rmsnorm_gb300 as tw
import synth
from norm_parity import bits16, check_q8, y_error
from oracle import fused, quant8
from parity import to_gpu

pytestmark = pytest.mark.gpu
EPS = synth.EPS
SCALES = {"f32": torch.float32, "e8m0": torch.float8_e8m0fnu}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from reduce_rmsnorm_gb300 import build
    build.build()
    tw.lib()
    tw.tw_device_status(reset=True)
    yield
    assert tw.tw_device_status(reset=True) == 0


def outputs(T, H, group, kind, fill=0x5A):
    """An output pair filled with a pattern, so that a missed write shows."""
    q = torch.full((T, H), fill, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    n = H // group if group else 1
    if kind == "f32":
        return q, torch.full((T, n), -7.0, device="cuda")
    return q, torch.full((T, n), fill, device="cuda", dtype=torch.uint8).view(SCALES[kind])


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def run(p, r, g, group, kind, **kw):
    P, R, G = to_gpu(p, r, g)
    q, s = outputs(*r.shape, group, kind)
    tw.tw_fused_reduce_residual_rmsnorm_q8(P, R, G, EPS, q, s, group=group, **kw)
    torch.cuda.synchronize()
    return q, s, R


def check(p, r, g, q, s, group):
    pb, rb, gb = synth.bits(p), synth.bits(r), synth.bits(g)
    z, y = fused.reduce_residual_rmsnorm(pb, rb, gb, EPS)
    absum = np.abs(fused.reduce_residual(np.abs(pb.astype(np.int32) & 0x7FFF), rb & 0x7FFF))
    check_q8(y, y_error(z, y, absum, pb.shape[0], gb, EPS), q, s, group)


# one token to more rows than the GPU holds at once; one vector per row to the
# largest row; ragged rows; few and many partials
SHAPES = [(1, 32, 1), (1, 8192, 8), (3, 128, 2), (5, 4096, 16), (2, 32768, 9), (17, 2048, 5),
          (130, 1152, 3), (200, 5120, 4), (160, 4096, 2), (1000, 8192, 1), (700, 8192, 4),
          (640, 1024, 12), (9, 16384, 8), (470, 16384, 2), (33, 12288, 7), (3000, 256, 2)]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("T,H,N", SHAPES)
def test_q8_parity(T, H, N, group, kind):
    if group and H % group:
        pytest.skip("H is no multiple of the group")
    p, r, g = synth.make_inputs(T, H, N, 0.3, seed=T + H + N)
    q, s, R = run(p, r, g, group, kind)
    check(p, r, g, q, s, group)
    # the residual is bitwise the bf16 step's
    P, R2, G = to_gpu(p, r, g)
    tw.tw_fused_reduce_residual_rmsnorm(P, R2, G, EPS, torch.empty_like(R2))
    assert torch.equal(R.view(torch.int16), R2.view(torch.int16))


@pytest.mark.parametrize("T,H,N,group", [(5, 64, 2, 64), (40, 8, 1, 0), (40, 264, 3, 0), (7, 5000, 3, 0),
                                         (300, 10 * 64, 6, 64), (152, 24, 8, 0), (3, 32760, 2, 0)])
def test_q8_parity_odd_sizes(T, H, N, group):
    p, r, g = synth.make_inputs(T, H, N, 0.3, seed=T + H)
    for kind in SCALES:
        q, s, _ = run(p, r, g, group, kind)
        check(p, r, g, q, s, group)


@pytest.mark.parametrize("T,H,N", [(1024, 8192, 8), (300, 8192, 4), (90, 8192, 12), (64, 32768, 2),
                                   (500, 1056, 3), (1300, 256, 1), (2000, 1056, 3), (700, 4096, 8),
                                   (1300, 2816, 2), (700, 4992, 3), (400, 1024, 14),
                                   (320, 12000, 3), (200, 8704, 8), (170, 16352, 12)])
@pytest.mark.parametrize("group,kind", [(0, "f32"), (32, "e8m0")])
def test_q8_is_bitwise_the_same_under_every_budget_and_shard(T, H, N, group, kind):
    p, r, g = synth.make_inputs(T, H, N, 0.1, seed=5)
    r[:, ::7] = -0.0                   # sums of zeros keep their sign in every form
    p[:, :, ::14] = -0.0
    q0, s0, R0 = run(p, r, g, group, kind)
    for budget in (1, 4, 40):
        q, s, R = run(p, r, g, group, kind, sm_budget=budget)
        assert same(q, q0) and same(s, s0) and torch.equal(R, R0), budget
    P, R, G = to_gpu(p, r, g)
    q, s = outputs(T, H, group, kind)
    cut = T // 3 + 1
    for a, b in ((0, cut), (cut, T)):
        tw.tw_fused_reduce_residual_rmsnorm_q8([P[i, a:b] for i in range(N)], R[a:b], G, EPS, q[a:b],
                                               s[a:b], group=group)
    torch.cuda.synchronize()
    assert same(q, q0) and same(s, s0) and torch.equal(R, R0)


def test_q8_one_outlier_sets_its_groups_scale_only():
    T, H = 4, 1024
    r = torch.full((T, H), 0.01).bfloat16()
    r[:, 100] = 1000.0
    p, g = torch.zeros(1, T, H).bfloat16(), torch.ones(H).bfloat16()
    q, s, _ = run(p, r, g, 32, "f32")
    check(p, r, g, q, s, 32)
    s = s.cpu()
    assert torch.all(s[:, 3] > 1000 * s[:, 0]) and torch.all(s[:, 0] == s[:, 31])
    q, s, _ = run(p, r, g, 0, "f32")
    check(p, r, g, q, s, 0)


def test_q8_zero_rows_tiny_rows_and_zero_gamma():
    T, H = 6, 256
    r = torch.zeros(T, H).bfloat16()
    r[1] = 1e-38                       # normalised by eps: far below the smallest scale's range
    r[2:] = torch.randn(T - 2, H).bfloat16()
    g = torch.ones(H).bfloat16()
    g[64:128] = 0.0                    # two whole groups of zeros in every row
    p = torch.zeros(2, T, H).bfloat16()
    for kind in SCALES:
        for group in (0, 32):
            q, s, _ = run(p, r, g, group, kind)
            check(p, r, g, q, s, group)
            v = quant8.decode(q.cpu().view(torch.uint8).numpy())
            assert not np.isnan(v).any() and not v[0].any() and not v[:, 64:128].any()
        assert torch.all(s.float()[:, 2:4] == 2.0 ** -126)  # 0 / 448, held at the smallest


def test_q8_power_of_two_scales_at_the_border():
    """A row of ones with eps = 0 has r = 1, so y = gamma exactly: the largest
    values of the groups sit at, next below and next above 448 * 2^k."""
    a = torch.tensor([1.734375, 1.7421875, 1.75, 1.7578125, 1.765625, 1.9921875, 1.0, 3.5, 448.0,
                      450.0, 0.02734375, 2.0 ** -120])
    H = 32 * len(a)
    g = torch.zeros(H).bfloat16()
    g[::32] = a.bfloat16()
    P, R, G = to_gpu(torch.zeros(1, 3, H).bfloat16(), torch.ones(3, H).bfloat16(), g)
    q, s = outputs(3, H, 32, "e8m0")
    tw.tw_fused_reduce_residual_rmsnorm_q8(P, R, G, 0.0, q, s, group=32)
    torch.cuda.synchronize()
    want = quant8.scale(g[::32].double().numpy(), "e8m0")
    got = quant8.decode_scales(s.cpu().view(torch.uint8).numpy(), "e8m0")
    assert np.array_equal(got, np.tile(want, (3, 1)))
    codes = quant8.decode(q.cpu().view(torch.uint8).numpy())[:, ::32]
    assert np.all(np.abs(codes) <= 448.0)
    assert np.all(np.abs(codes * got - g[::32].double().numpy()) <=
                  got * quant8.half_step(codes))


def test_q8_nan_and_infinity():
    T, H = 5, 128
    r = torch.randn(T, H).bfloat16()
    r[1, 7] = float("nan")             # the whole row's norm is NaN
    r[2, 9] = float("inf")             # scale 0: inf * 0 is NaN, the rest 0
    g = torch.ones(H).bfloat16()
    g[40] = float("inf")               # an infinite value in the second group of 32
    p = torch.zeros(1, T, H).bfloat16()
    for kind in SCALES:
        q, s, _ = run(p, r, g, 32, kind)
        v = quant8.decode(q.cpu().view(torch.uint8).numpy())
        s64 = quant8.decode_scales(s.cpu().view(torch.uint8).numpy() if kind == "e8m0" else
                                   s.cpu().numpy(), kind)
        assert np.isnan(v[1]).all()
        assert np.isnan(v[2, 9]) and not np.nan_to_num(v[2, np.arange(H) != 40]).any()
        with np.errstate(invalid="ignore"):
            back = v * np.repeat(s64, 32, axis=1)
        for t in (0, 3, 4):
            assert np.isnan(back[t, 32:64]).all(), kind   # its group reads back as NaN
            assert np.isfinite(back[t, :32]).all() and np.isfinite(back[t, 64:]).all()


def test_q8_eight_byte_aligned_output_and_untouched_neighbours():
    T, H, N = 13, 24, 2
    p, r, g = synth.make_inputs(T, H, N, 0.2, seed=2)
    P, R, G = to_gpu(p, r, g)
    raw = torch.full((T * H + 24,), 0x11, device="cuda", dtype=torch.uint8)
    sc = torch.full((T + 2,), 3.0, device="cuda")
    q = raw[8:8 + T * H].view(T, H).view(torch.float8_e4m3fn)
    s = sc[1:1 + T].view(T, 1)
    tw.tw_fused_reduce_residual_rmsnorm_q8(P, R, G, EPS, q, s)
    torch.cuda.synchronize()
    check(p, r, g, q, s, 0)
    assert torch.all(raw[:8] == 0x11) and torch.all(raw[8 + T * H:] == 0x11)
    assert sc[0] == 3.0 and sc[-1] == 3.0


def test_q8_repeats_bitwise_and_follows_its_stream():
    p, r, g = synth.make_inputs(500, 4096, 4, 0.1, seed=8)
    q0, s0, R0 = run(p, r, g, 128, "f32")
    side = torch.cuda.Stream()
    q1, s1, R1 = run(p, r, g, 128, "f32", stream=side)
    assert same(q0, q1) and same(s0, s1) and torch.equal(R0, R1)
    # aliased partials: one buffer four times
    P, R, G = to_gpu(p, r, g)
    q, s = outputs(500, 4096, 128, "f32")
    tw.tw_fused_reduce_residual_rmsnorm_q8([P[0]] * 4, R, G, EPS, q, s, group=128)
    torch.cuda.synchronize()
    check(torch.stack([p[0]] * 4), r, g, q, s, 128)
    assert bits16(R).shape == (500, 4096)
