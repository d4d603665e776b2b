"""The expert router against the fp64 oracle. Needs a GPU.

The experts have to be those of the oracle, in order. A weight's relative error:
u = 2^-24; expf's argument is rounded at |x - m| u (the row's range), expf is
within 2 ulp (4 u), and the sum of at most 1024 scores, the division and the
scale add at most 48 u (each lane adds 32, then 5 steps). 2 (range + 64) u
covers both the numerator and the sum."""

import math

import numpy as np
import pytest
import torch

import reduce_rmsnorm_gb300 as tw
from oracle import experts

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from reduce_rmsnorm_gb300 import build
    build.build()
    tw.lib()
    tw.tw_device_status(reset=True)
    yield
    assert tw.tw_device_status(reset=True) == 0


def route(x, k, bias=None, **kw):
    T = x.shape[0]
    w = torch.full((T, k), -3.0, device="cuda")
    ids = torch.full((T, k), -9, device="cuda", dtype=torch.int32)
    b = None if bias is None else bias.cuda()
    tw.tw_route_experts(x.cuda().contiguous(), w, ids, bias=b, **kw)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy()


def check(x, k, bias=None, **kw):
    kw.pop("stream", None)
    ids, w = route(x, k, bias, **kw)
    x64 = x.double().numpy()
    want, w64 = experts.route(x64, k, None if bias is None else bias.double().numpy(), **kw)
    assert np.array_equal(ids, want), np.argwhere(ids != want)[:5]
    finite = np.where(np.isfinite(x64), np.abs(x64), 0.0)
    span = 2 * np.minimum(finite.max(axis=1, keepdims=True, initial=0.0), 1000.0)
    # 2^-149: below it fp32 has nothing
    tol = 2 * (span + 64) * U * np.abs(w64) + 2.0 ** -149
    assert np.all(np.abs(w - w64) <= tol), np.abs(w - w64).max()
    return ids, w


def logits(T, E, seed, sigma=1.5, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * sigma).to(dtype)


SIZES = [(1, 1, 1), (1, 256, 8), (3, 7, 7), (129, 100, 3), (2, 1024, 32), (65, 33, 2), (300, 8, 2),
         (50, 64, 6), (40, 128, 8), (21, 160, 6), (10, 977, 11), (9, 512, 16), (1000, 16, 4),
         (11, 40, 32), (2, 31, 31)]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", SIZES)
def test_route_parity(T, E, K, dtype, scoring):
    x = logits(T, E, seed=E + K, dtype=dtype)
    bias = logits(1, E, seed=3, sigma=0.05)[0]
    for renormalize in (True, False):
        check(x, K, scoring=scoring, renormalize=renormalize, scale=2.5)
        check(x, K, bias, scoring=scoring, renormalize=renormalize)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,G,top", [(256, 8, 8, 4), (160, 6, 8, 3), (64, 4, 32, 7), (96, 5, 3, 2),
                                       (1024, 32, 16, 2), (330, 9, 11, 5), (8, 2, 4, 1), (12, 2, 2, 2)])
def test_route_groups(E, K, G, top, scoring):
    for dtype in (torch.float32, torch.bfloat16):
        x = logits(60, E, seed=E, dtype=dtype)
        for bias in (None, logits(1, E, seed=4, sigma=0.05)[0], torch.zeros(E)):
            for group_top in (1, 2):
                check(x, K, bias, scoring=scoring, n_groups=G, top_groups=top, group_top=group_top)


def test_route_groups_of_one_expert():
    x = logits(20, 32, seed=1)
    check(x, 5, scoring="sigmoid", n_groups=32, top_groups=6, group_top=1)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_equal_values_go_to_the_lowest_index(scoring):
    for E in (5, 32, 300):
        ids, _ = check(torch.full((3, E), 0.75), min(E, 6), scoring=scoring)
        assert np.array_equal(ids[0], np.arange(min(E, 6)))
        check(torch.full((2, E), -2.0), 4, torch.full((E,), 0.25), scoring=scoring)
    x = logits(200, 64, seed=2, sigma=1.0).round()  # a few distinct values, -0 and +0 among them
    check(x, 8, scoring=scoring)
    check(x, 8, torch.zeros(64), scoring=scoring, n_groups=8, top_groups=3, group_top=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_values_that_fp32_cannot_tell_apart(scoring):
    """The biases undo the scores' differences but for parts of 2^-30 and less,
    so that the order of most candidates is below fp32's resolution."""
    g = torch.Generator().manual_seed(11)
    E, T = 64, 30
    x = torch.randn(T, E, generator=g)
    x[:] = x[0]
    s = torch.softmax(x[0].double(), 0) if scoring == "softmax" else torch.sigmoid(x[0].double())
    bias = (0.5 - s).float()  # s + bias = 0.5 up to half an fp32 step of the bias
    check(x, 16, bias, scoring=scoring)
    check(x, 8, bias, scoring=scoring, n_groups=8, top_groups=4, group_top=2)
    # saturated scores: 1 / (1 + e^-x) is 1 in fp32 from x = 17 on
    big = 20.0 + 0.25 * torch.randn(T, E, generator=g)
    check(big, 8, torch.zeros(E), scoring=scoring)
    check(big, 8, scoring=scoring, n_groups=8, top_groups=2, group_top=2)
    low = -95.0 + 0.25 * torch.randn(T, E, generator=g)
    check(low, 8, scoring=scoring, n_groups=8, top_groups=2, group_top=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_near_values_with_fewer_experts_than_slots(scoring):
    """Candidates that only fp64 can order, some rows with fewer than K of them."""
    g = torch.Generator().manual_seed(12)
    for E, K in ((64, 8), (64, 20), (256, 8), (300, 8), (6, 6)):
        x = torch.randn(12, E, generator=g)
        x[:] = x[0]
        s = torch.softmax(x[0].double(), 0) if scoring == "softmax" else torch.sigmoid(x[0].double())
        bias = (0.5 - s).float()
        for t in range(8):
            x[t, t + 1:] = -math.inf
        if scoring == "softmax":  # the scores of the masked rows differ: no near values there
            check(x[8:], K, bias, scoring=scoring)
        check(x, K, bias, scoring=scoring)
        check(x, K, bias, scoring=scoring, renormalize=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,top", [(64, 8, 3), (128, 8, 4), (256, 8, 4), (256, 4, 2), (96, 12, 5)])
def test_route_near_group_values(scoring, E, G, top):
    """Group values that differ by less than fp32 holds, and groups that tie."""
    g = torch.Generator().manual_seed(13)
    size = E // G
    x = torch.randn(4000, size, generator=g).repeat(1, G)
    # one expert of each group moves by a few fp32 steps, in some rows not at all
    x[::2, ::size] += 3e-7 * torch.randint(-2, 3, (2000, G), generator=g)
    for bias in (None, torch.zeros(E), 0.01 * torch.randn(size, generator=g).repeat(G)):
        for group_top in (1, 2):
            check(x[:60], 4, bias, scoring=scoring, n_groups=G, top_groups=top, group_top=group_top)
    ids, _ = route(x, 4, torch.zeros(E), scoring=scoring, n_groups=G, top_groups=top, group_top=2)
    assert ids.min() >= 0


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_masked_experts_and_rows(scoring):
    inf = math.inf
    x = logits(8, 40, seed=5)
    x[0] = -inf                         # nothing left
    x[1, :38] = -inf                    # two of six left
    x[2] = math.nan
    x[3, 5] = math.nan
    x[4, 7] = inf
    x[4, 9] = inf                       # two infinite logits tie
    x[5] = torch.finfo(torch.float32).min
    x[6] = -inf
    x[6, 39] = -300.0
    for renormalize in (True, False):
        ids, w = check(x, 6, scoring=scoring, renormalize=renormalize)
        assert np.all(ids[0] == -1) and np.all(ids[2] == -1) and not w[0].any() and not w[2].any()
        assert np.all(ids[1, 2:] == -1) and not w[1, 2:].any() and 5 not in ids[3]
        assert ids[4, 0] == 7 and ids[4, 1] == 9 and ids[6, 0] == 39
        check(x, 6, scoring=scoring, renormalize=renormalize, n_groups=4, top_groups=2, group_top=2)
        bias = torch.zeros(40)
        bias[3], bias[8], bias[11] = -inf, math.nan, inf
        ids, _ = check(x, 6, bias, scoring=scoring, renormalize=renormalize)
        assert 3 not in ids and 8 not in ids and np.all(ids[[3, 4, 5, 7], 0] == 11)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_logits_of_the_types_extremes(scoring):
    big = torch.finfo(torch.bfloat16).max
    x = torch.tensor([[big, -big, 0.0, 1.0], [-big, -big, -big, -big], [100.0, -100.0, 88.0, -88.0],
                      [-200.0, -201.0, -300.0, -1000.0]], dtype=torch.bfloat16)
    for dtype in (torch.bfloat16, torch.float32):
        check(x.to(dtype), 3, scoring=scoring)
        check(x.to(dtype), 3, torch.tensor([0.1, 0.2, 0.3, 0.4]), scoring=scoring)


def test_route_zero_scale_and_negative_scale():
    x = logits(5, 20, seed=6)
    check(x, 3, scale=0.0)
    check(x, 3, scale=-1.5, scoring="sigmoid")


def test_route_unaligned_rows_streams_and_neighbours():
    """Odd E and bases aligned to the type only; neighbours of the outputs stay."""
    T, E, K = 37, 51, 5
    for dtype in (torch.float32, torch.bfloat16):
        flat = torch.zeros(T * E + 3, device="cuda", dtype=dtype)
        x = logits(T, E, seed=7, dtype=dtype)
        view = flat[1:1 + T * E].view(T, E)
        view.copy_(x)
        w = torch.full((T * K + 2,), -3.0, device="cuda")
        ids = torch.full((T * K + 2,), -9, device="cuda", dtype=torch.int32)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        tw.tw_route_experts(view, w[1:-1].view(T, K), ids[1:-1].view(T, K), stream=side)
        side.synchronize()
        want, _ = experts.route(x.double().numpy(), K)
        assert np.array_equal(ids[1:-1].view(T, K).cpu().numpy(), want)
        assert w[0] == -3 and w[-1] == -3 and ids[0] == -9 and ids[-1] == -9


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K,G,top", [(256, 8, 1, 1), (256, 8, 8, 4), (96, 3, 1, 1), (128, 8, 4, 2),
                                       (224, 7, 1, 1), (192, 8, 6, 3)])
def test_route_long_batches(E, K, G, top, dtype, scoring):
    """Enough tokens that rows of more than 64 experts share a warp. The batch
    repeats 150 tokens, so that every place in a warp meets every one of them;
    some are masked, some equal everywhere."""
    x = logits(150, E, seed=E, dtype=dtype)
    x[3], x[4, : E - 2], x[5], x[6, ::2] = -math.inf, -math.inf, 0.5, x[6, 1::2]
    x[7] = math.nan
    bias = logits(1, E, seed=2, sigma=0.05)[0]
    many = x.repeat(220, 1)[:32797]
    for b in (None, bias):
        for renormalize in (True, False):
            kw = dict(scoring=scoring, renormalize=renormalize, n_groups=G, top_groups=top,
                      group_top=2, scale=1.5)
            ids, w = check(x, K, b, **kw)
            ids2, w2 = route(many, K, b, **kw)
            assert np.array_equal(ids2, np.tile(ids, (220, 1))[:32797])
            # other lanes add the weights' sum in another order
            assert np.allclose(w2, np.tile(w, (220, 1))[:32797], rtol=2 * 64 * U, atol=0)


def test_route_many_tokens_repeat_bitwise_and_independent_of_the_batch():
    x = logits(40000, 64, seed=8)
    bias = logits(1, 64, seed=9, sigma=0.05)[0]
    kw = dict(scoring="sigmoid", n_groups=8, top_groups=4, group_top=2)
    ids, w = route(x, 6, bias, **kw)
    again, w2 = route(x, 6, bias, **kw)
    assert np.array_equal(ids, again) and np.array_equal(w, w2)
    part, w3 = route(x[777:1001], 6, bias, **kw)
    assert np.array_equal(ids[777:1001], part) and np.array_equal(w[777:1001], w3)
    want, _ = experts.route(x[:2000].double().numpy(), 6, bias.double().numpy(), **kw)
    assert np.array_equal(ids[:2000], want)
