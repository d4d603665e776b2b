"""The combine step (gathered weighted expert rows + partials + residual, then
RMSNorm in bf16 or e4m3) against the fp64 oracle. Needs a GPU."""

import numpy as np
import pytest
import torch

import reduce_rmsnorm_gb300 as tw
import synth
from norm_parity import bits16, check_bf16, check_q8, check_residual, y_error
from oracle import bf16, experts
from test_gpu_q8 import SCALES, outputs, same

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


def inputs(T, H, K, N, M, seed=0, dropped=0.0):
    """Host tensors of one call; rows may repeat and may be dropped."""
    rng = np.random.Generator(np.random.PCG64(seed))
    p, r, g = synth.make_inputs(T, H, max(N, 1), 0.2, seed=seed)
    x, _, _ = synth.make_inputs(max(M, 1), H, 1, 1.0, seed=seed + 1)
    rows = rng.integers(0, max(M, 1), size=(T, K)).astype(np.int32)
    rows[rng.random((T, K)) < dropped] = -1
    w = rng.random((T, K)).astype(np.float32)
    return dict(x=x[0][:M], rows=torch.from_numpy(rows), w=torch.from_numpy(w), p=p[:N], r=r, g=g)


def gpu(h):
    d = {k: v.cuda().contiguous() for k, v in h.items()}
    torch.cuda.synchronize()
    return d


def call(d, out, scales=None, group=0, **kw):
    args = (d["x"], d["rows"], d["w"], d["r"], d["g"], EPS, out)
    if scales is None:
        tw.tw_combine_residual_rmsnorm(*args, partials=d["p"], **kw)
    else:
        tw.tw_combine_residual_rmsnorm_q8(*args, scales, group=group, partials=d["p"], **kw)
    torch.cuda.synchronize()


def oracle(h):
    pb = [bits16(v) for v in h["p"]]
    z, y, absum = experts.combine(bits16(h["x"]), h["rows"].numpy(), h["w"].numpy(), pb,
                                  bits16(h["r"]), bits16(h["g"]), EPS)
    n = h["rows"].shape[1] + len(pb) + 1
    return z, y, absum, n, y_error(z, y, absum, n, bits16(h["g"]), EPS)


def check(h, d, out):
    z, y, absum, n, err = oracle(h)
    check_residual(z, absum, n, d["r"])
    check_bf16(y, err, out)


SHAPES = [(1, 8, 1, 0, 1), (1, 4096, 8, 0, 8), (1, 32768, 2, 1, 5), (3, 264, 32, 0, 40),
          (64, 8192, 8, 1, 512), (40, 2048, 2, 16, 80), (200, 1032, 5, 2, 333),
          (700, 256, 6, 0, 64), (150, 4096, 4, 1, 1000), (33, 16384, 3, 2, 50),
          (5, 24576, 9, 1, 11), (2500, 64, 2, 1, 5000), (17, 5000, 1, 0, 3)]


@pytest.mark.parametrize("T,H,K,N,M", SHAPES)
def test_combine_parity(T, H, K, N, M):
    h = inputs(T, H, K, N, M, seed=T + H, dropped=0.15)
    d = gpu(h)
    out = torch.full((T, H), 7.0, device="cuda", dtype=torch.bfloat16)
    call(d, out)
    check(h, d, out)


@pytest.mark.parametrize("kind", sorted(SCALES))
@pytest.mark.parametrize("T,H,K,N,M,group", [(1, 4096, 8, 0, 8, 32), (64, 8192, 8, 1, 512, 32),
                                             (200, 1032, 5, 2, 333, 0), (700, 256, 6, 0, 64, 128),
                                             (150, 4160, 4, 1, 1000, 64), (3, 32768, 2, 1, 4, 128),
                                             (9, 96, 3, 0, 20, 32), (20, 10240, 2, 0, 30, 0)])
def test_combine_q8_parity(T, H, K, N, M, group, kind):
    h = inputs(T, H, K, N, M, seed=T + H, dropped=0.1)
    d = gpu(h)
    q, s = outputs(T, H, group, kind)
    call(d, q, s, group)
    z, y, absum, n, err = oracle(h)
    check_residual(z, absum, n, d["r"])
    check_q8(y, err, q, s, group)
    # the residual is bitwise that of the bf16 form
    d2 = gpu(h)
    call(d2, torch.empty_like(d2["r"]))
    assert torch.equal(d["r"].view(torch.int16), d2["r"].view(torch.int16))


def test_combine_with_nothing_kept_is_the_norm_of_the_residual():
    h = inputs(6, 512, 4, 0, 3, seed=3)
    h["rows"][:] = -1
    h["w"][:] = float("nan")           # a dropped slot's weight is not used
    d = gpu(h)
    out = torch.empty_like(d["r"])
    call(d, out)
    check(h, d, out)
    assert torch.equal(d["r"].cpu().view(torch.int16), h["r"].view(torch.int16))
    # no expert rows at all
    h["x"] = h["x"][:0]
    d = gpu(h)
    call(d, out)
    check(h, d, out)


def test_combine_a_row_index_outside_the_expert_rows_is_left_out_and_reported():
    M = 5
    h = inputs(7, 256, 3, 1, M, seed=4)
    h["rows"][2, 1] = M
    h["rows"][4, 0] = -2
    h["rows"][6, 2] = 2 ** 31 - 1
    d = gpu(h)
    out = torch.empty_like(d["r"])
    call(d, out)
    check(h, d, out)
    assert tw.tw_device_status(reset=True) == 8
    assert tw.tw_device_status(reset=True) == 0


def test_combine_same_row_in_every_slot_and_non_finite_rows():
    h = inputs(4, 128, 5, 0, 3, seed=6)
    h["rows"][0] = 1
    h["x"][2] = float("nan")           # a row that no slot names is not read into any
    h["rows"][h["rows"] == 2] = 0
    h["rows"][3] = 2
    d = gpu(h)
    out = torch.empty_like(d["r"])
    call(d, out)
    assert torch.isnan(out[3]).all() and torch.isfinite(out[:3].float()).all()
    for k in ("rows", "w", "r"):
        h[k] = h[k][:3]
    z, y, absum, n, err = oracle(h)
    check_bf16(y, err, out[:3])


def test_combine_output_over_a_partial_and_untouched_inputs():
    h = inputs(50, 1024, 4, 2, 60, seed=7)
    d = gpu(h)
    keep = {k: d[k].clone() for k in ("x", "rows", "w", "g")}
    other = d["p"][0].clone()
    call(d, d["p"][1])
    check(h, d, d["p"][1])
    assert torch.equal(d["p"][0], other)
    for k, v in keep.items():
        assert torch.equal(d[k], v), k


@pytest.mark.parametrize("T,H,K,N", [(300, 4096, 8, 1), (100, 8192, 2, 0), (20, 16384, 4, 1),
                                     (200, 1032, 3, 2)])
def test_combine_bitwise_under_budgets_shards_and_repeats(T, H, K, N):
    h = inputs(T, H, K, N, 2 * T, seed=8, dropped=0.1)
    d0 = gpu(h)
    out0 = torch.empty_like(d0["r"])
    call(d0, out0)
    for kw in (dict(), dict(sm_budget=1), dict(sm_budget=7), dict(stream=torch.cuda.Stream())):
        d = gpu(h)
        out = torch.empty_like(d["r"])
        torch.cuda.synchronize()
        call(d, out, **kw)
        assert torch.equal(out, out0) and torch.equal(d["r"], d0["r"]), kw
    d = gpu(h)
    out = torch.empty_like(d["r"])
    cut = T // 2 + 1
    for a, b in ((0, cut), (cut, T)):
        tw.tw_combine_residual_rmsnorm(d["x"], d["rows"][a:b], d["w"][a:b], d["r"][a:b], d["g"], EPS,
                                       out[a:b], partials=[v[a:b] for v in d["p"]])
    torch.cuda.synchronize()
    assert torch.equal(out, out0) and torch.equal(d["r"], d0["r"])


def test_combine_expert_rows_beyond_32_bit_offsets():
    """Rows whose element offset does not fit in 32 bits: 2^31 / 8192 rows and
    a few more (4.3 GB)."""
    H, T, K = 8192, 3, 2
    M = 2 ** 31 // H + 8
    x = torch.empty(M, H, device="cuda", dtype=torch.bfloat16)
    h = inputs(T, H, K, 0, 8, seed=9)
    last = torch.arange(M - 8, M)
    x[last.cuda()] = h["x"].cuda()
    d = gpu(dict(h, rows=(h["rows"] + (M - 8)).to(torch.int32)))
    d["x"] = x
    out = torch.empty_like(d["r"])
    call(d, out)
    check(h, d, out)


def test_bf16_bits_helper_reads_values():
    v = torch.tensor([1.5, -2.0]).bfloat16()
    assert bf16.decode(bits16(v)).tolist() == [1.5, -2.0]
