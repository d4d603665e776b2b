"""The 8-bit step, the combine step and the router on the CPU: the oracle's
pins, and the argument checks of the C ABI (fake addresses that validation
never dereferences) and of the binding."""

import ctypes
import math

import numpy as np
import pytest
import torch

import reduce_rmsnorm_gb300 as tw
import synth
from oracle import bf16, experts, fused, quant8

BASE = 0x7F0000000000


@pytest.fixture(scope="module")
def L():
    from reduce_rmsnorm_gb300 import build
    build.build()
    return tw.lib()


# ------------------------------------------------------------------ oracle pins


def test_e4m3_decoding_is_the_format():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(quant8.decode(codes), want, equal_nan=True)
    assert np.nanmax(want) == quant8.E4M3_MAX


def test_half_step_is_half_the_gap_between_codes():
    values = np.sort(quant8.decode(np.arange(127, dtype=np.uint8)))  # 0 .. 448, finite
    gaps = np.diff(values)
    assert np.array_equal(quant8.half_step(values[:-1]), gaps / 2)


def test_scale_rules():
    s = quant8.scale(np.array([448.0, 896.0, 0.0, 1e-60]), "f32")
    assert np.array_equal(s, [1.0, 2.0, 2.0 ** -126, 2.0 ** -126])
    s = quant8.scale(np.array([448.0, 448.0001, 224.0, 0.0]), "e8m0")
    assert np.array_equal(s, [1.0, 2.0, 0.5, 2.0 ** -126])


def test_route_oracle_by_hand():
    # four experts in two groups; group values 0.6 + 0.5 and 0.9 + 0.1
    p = np.array([[0.6, 0.5, 0.9, 0.1]])
    x = np.log(p / (1 - p))  # sigmoid gives p back
    ids, w = experts.route(x, 2, scoring="sigmoid", n_groups=2, top_groups=1, group_top=2,
                           renormalize=False)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[0.6, 0.5]])
    ids, w = experts.route(x, 2, scoring="sigmoid", n_groups=2, top_groups=1, group_top=1)
    assert ids.tolist() == [[2, 3]] and np.allclose(w, [[0.9, 0.1]])
    # the bias moves the choice, not the weights
    ids, w = experts.route(x, 1, bias=[0, 0, 0, 1.0], scoring="sigmoid", renormalize=False)
    assert ids.tolist() == [[3]] and np.allclose(w, [[0.1]])
    ids, w = experts.route(np.array([[-math.inf, 2.0], [-math.inf, -math.inf]]), 2)
    assert ids.tolist() == [[1, -1], [-1, -1]] and w.tolist() == [[1, 0], [0, 0]]


def test_combine_oracle_is_the_fused_step_for_unit_weights():
    p, r, g = synth.make_inputs(5, 64, 3, 0.5, seed=1)
    pb, rb, gb = synth.bits(p), synth.bits(r), synth.bits(g)
    z, y = fused.reduce_residual_rmsnorm(pb, rb, gb, 1e-5)
    flat = pb.reshape(-1, 64)  # row n * T + t is partial n's row t
    rows = np.array([[n * 5 + t for n in range(3)] + [-1] for t in range(5)])
    z2, y2, _ = experts.combine(flat, rows, np.ones((5, 4)), [], rb, gb, 1e-5)
    assert np.allclose(z, z2, rtol=1e-14) and np.allclose(y, y2, rtol=1e-14)
    assert bf16.decode(rb).shape == z2.shape


# ------------------------------------------------------------------ C-ABI checks


def _at(i):
    return BASE + (i << 24)


def _ptrs(values):
    return (ctypes.c_void_p * max(1, len(values)))(*values)


def _q8(L, N=2, T=4, H=256, eps=1e-5, group=32, scale_type=0, sm_budget=0, **at):
    a = dict(partials=[_at(i + 1) for i in range(max(N, 0))], residual=_at(40), gamma=_at(41),
             out=_at(42), scales=_at(43))
    a.update(at)
    return L.tw_fused_reduce_residual_rmsnorm_q8(_ptrs(a["partials"]), N, a["residual"], a["gamma"],
                                                 eps, T, H, a["out"], a["scales"], group,
                                                 scale_type, None, sm_budget)


def _combine(L, q8=False, N=1, K=2, M=8, T=4, H=256, eps=1e-5, group=32, scale_type=0,
             sm_budget=0, **at):
    a = dict(partials=[_at(i + 1) for i in range(max(N, 0))], residual=_at(40), gamma=_at(41),
             out=_at(42), scales=_at(43), experts=_at(44), rows=_at(45), weights=_at(46))
    a.update(at)
    parts = None if a["partials"] is None else _ptrs(a["partials"])
    head = (a["experts"], M, a["rows"], a["weights"], K, parts, N, a["residual"], a["gamma"], eps,
            T, H, a["out"])
    if q8:
        return L.tw_combine_residual_rmsnorm_q8(*head, a["scales"], group, scale_type, None,
                                                sm_budget)
    return L.tw_combine_residual_rmsnorm(*head, None, sm_budget)


def _route(L, dtype=0, bias=None, T=4, E=64, K=4, scoring=0, n_groups=1, top_groups=1, group_top=1,
           renormalize=1, scale=1.0, **at):
    a = dict(logits=_at(1), weights=_at(2), ids=_at(3))
    a.update(at)
    return L.tw_route_experts(a["logits"], dtype, bias, T, E, K, scoring, n_groups, top_groups,
                              group_top, renormalize, scale, a["weights"], a["ids"], None)


INVALID, ALIGN, UNSUPPORTED = tw.TW_ERR_INVALID_ARG, tw.TW_ERR_ALIGN, tw.TW_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad,want", [
    (dict(N=0), INVALID), (dict(N=17), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID),
    (dict(H=260), ALIGN), (dict(H=32776, group=0), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(eps=math.inf), INVALID), (dict(eps=math.nan), INVALID), (dict(sm_budget=-1), INVALID),
    (dict(group=16), INVALID), (dict(group=-32), INVALID), (dict(group=256), INVALID),
    (dict(H=264, group=128), ALIGN), (dict(H=264, group=32), ALIGN), (dict(scale_type=2), INVALID),
    (dict(scale_type=-1), INVALID), (dict(T=1 << 60), INVALID),
    (dict(residual=None), INVALID), (dict(gamma=None), INVALID), (dict(out=None), INVALID),
    (dict(scales=None), INVALID), (dict(partials=[_at(1), None]), INVALID),
    (dict(residual=_at(40) + 8), ALIGN), (dict(gamma=_at(41) + 2), ALIGN),
    (dict(partials=[_at(1), _at(2) + 8]), ALIGN), (dict(out=_at(42) + 4), ALIGN),
    (dict(scales=_at(43) + 2), ALIGN),
    (dict(out=_at(1)), INVALID), (dict(out=_at(40)), INVALID), (dict(scales=_at(42) + 512), INVALID),
    (dict(scales=_at(2)), INVALID), (dict(residual=_at(1)), INVALID), (dict(scales=_at(41)), INVALID),
])
def test_q8_refusals(L, bad, want):
    assert _q8(L, **bad) == want


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("bad,want", [
    (dict(N=-1), INVALID), (dict(N=17), INVALID), (dict(K=0), INVALID), (dict(K=33), INVALID),
    (dict(M=-1), INVALID), (dict(M=1 << 31), INVALID), (dict(T=-1), INVALID), (dict(H=260), ALIGN),
    (dict(H=32776, group=0), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(sm_budget=-1), INVALID),
    (dict(T=1 << 60), INVALID), (dict(T=1 << 55, H=8, group=0, K=32), INVALID),
    (dict(experts=None), INVALID), (dict(rows=None), INVALID), (dict(weights=None), INVALID),
    (dict(residual=None), INVALID), (dict(gamma=None), INVALID), (dict(out=None), INVALID),
    (dict(partials=None), INVALID), (dict(partials=[None]), INVALID),
    (dict(experts=_at(44) + 8), ALIGN), (dict(rows=_at(45) + 2), ALIGN),
    (dict(weights=_at(46) + 1), ALIGN), (dict(residual=_at(40) + 8), ALIGN),
    (dict(partials=[_at(1) + 8]), ALIGN), (dict(out=_at(42) + 4), ALIGN),
    (dict(out=_at(44)), INVALID), (dict(residual=_at(44) + 512), INVALID),
    (dict(out=_at(40) + 512), INVALID), (dict(out=_at(45)), INVALID), (dict(residual=_at(46)), INVALID),
    (dict(out=_at(1) + 512), INVALID), (dict(residual=_at(1)), INVALID), (dict(out=_at(41)), INVALID),
])
def test_combine_refusals(L, q8, bad, want):
    assert _combine(L, q8, **bad) == want


@pytest.mark.parametrize("bad,want", [
    (dict(group=16), INVALID), (dict(H=264, group=32), ALIGN), (dict(scale_type=2), INVALID),
    (dict(scale_type=-1), INVALID), (dict(scales=None), INVALID), (dict(scales=_at(43) + 1), ALIGN),
    (dict(scales=_at(44)), INVALID), (dict(out=_at(1)), INVALID), (dict(scales=_at(40)), INVALID),
])
def test_combine_q8_refusals(L, bad, want):
    assert _combine(L, True, **bad) == want


@pytest.mark.parametrize("bad,want", [
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(scoring=2), INVALID),
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(K=0), INVALID), (dict(K=33), INVALID),
    (dict(E=3, K=4), INVALID), (dict(n_groups=0), INVALID), (dict(n_groups=33, E=66), INVALID),
    (dict(n_groups=5), INVALID), (dict(n_groups=4, top_groups=5), INVALID),
    (dict(n_groups=4, top_groups=0), INVALID), (dict(group_top=0), INVALID),
    (dict(group_top=3), INVALID), (dict(E=32, n_groups=32, top_groups=8, group_top=2), INVALID),
    (dict(n_groups=32, top_groups=1, K=3), INVALID), (dict(scale=math.inf), INVALID),
    (dict(scale=math.nan), INVALID), (dict(E=1025), UNSUPPORTED), (dict(T=1 << 60), INVALID),
    (dict(logits=None), INVALID), (dict(weights=None), INVALID), (dict(ids=None), INVALID),
    (dict(logits=_at(1) + 2), ALIGN), (dict(dtype=1, logits=_at(1) + 1), ALIGN),
    (dict(weights=_at(2) + 2), ALIGN), (dict(ids=_at(3) + 1), ALIGN), (dict(bias=_at(9) + 2), ALIGN),
    (dict(ids=_at(2) + 32), INVALID), (dict(ids=_at(1) + 64), INVALID),
    (dict(weights=_at(1) + 1020), INVALID), (dict(bias=_at(2) + 60), INVALID),
])
def test_route_refusals(L, bad, want):
    assert _route(L, **bad) == want


def test_empty_batches_are_no_ops(L):
    assert _q8(L, T=0) == tw.TW_OK
    assert _combine(L, T=0) == tw.TW_OK
    assert _combine(L, True, T=0, N=0, partials=None, experts=None, M=0) == tw.TW_OK
    assert _route(L, T=0, logits=None, weights=None, ids=None) == tw.TW_OK


# ------------------------------------------------------------------ binding checks


def _host_inputs():
    T, H, K, M = 4, 256, 2, 8
    h = dict(P=torch.zeros(2, T, H, dtype=torch.bfloat16), R=torch.zeros(T, H, dtype=torch.bfloat16),
             G=torch.ones(H, dtype=torch.bfloat16), X=torch.zeros(M, H, dtype=torch.bfloat16),
             rows=torch.zeros(T, K, dtype=torch.int32), w=torch.zeros(T, K),
             out=torch.empty(T, H, dtype=torch.bfloat16),
             q=torch.empty(T, H, dtype=torch.float8_e4m3fn), s=torch.empty(T, H // 32))
    return h


def test_binding_refuses_host_tensors():
    h = _host_inputs()
    calls = (lambda: tw.tw_fused_reduce_residual_rmsnorm_q8(h["P"], h["R"], h["G"], 1e-5, h["q"],
                                                            h["s"], group=32),
             lambda: tw.tw_combine_residual_rmsnorm(h["X"], h["rows"], h["w"], h["R"], h["G"], 1e-5,
                                                    h["out"], partials=h["P"]),
             lambda: tw.tw_combine_residual_rmsnorm_q8(h["X"], h["rows"], h["w"], h["R"], h["G"],
                                                       1e-5, h["q"], h["s"], group=32),
             lambda: tw.tw_route_experts(h["w"], h["w"], h["rows"]))
    for call in calls:
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


class _Fake:
    """The attributes of a CUDA tensor that the binding reads."""

    def __init__(self, shape, dtype, index=0, ptr=0x10000):
        self.shape, self.dtype, self.is_cuda = torch.Size(shape), dtype, True
        self.device, self._ptr = torch.device("cuda", index), ptr

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return self._ptr

    def get_device(self):
        return self.device.index


def _fakes(bad=None, **other):
    T, H, K, M, E = 4, 256, 2, 8, 16
    b16, f32 = torch.bfloat16, torch.float32
    spec = dict(p=((T, H), b16), R=((T, H), b16), G=((H,), b16), X=((M, H), b16),
                rows=((T, K), torch.int32), w=((T, K), f32), out=((T, H), b16),
                q=((T, H), torch.float8_e4m3fn), s=((T, H // 32), f32), x=((T, E), f32),
                b=((E,), f32), ids=((T, K), torch.int32))
    spec.update(other)
    return {k: _Fake(v[0], v[1], 1 if k == bad else 0) for k, v in spec.items()}


def _calls(f):
    return dict(
        q8=lambda: tw.tw_fused_reduce_residual_rmsnorm_q8([f["p"]], f["R"], f["G"], 1e-5, f["q"],
                                                          f["s"], group=32),
        combine=lambda: tw.tw_combine_residual_rmsnorm(f["X"], f["rows"], f["w"], f["R"], f["G"],
                                                       1e-5, f["out"], partials=[f["p"]]),
        combine_q8=lambda: tw.tw_combine_residual_rmsnorm_q8(f["X"], f["rows"], f["w"], f["R"],
                                                             f["G"], 1e-5, f["q"], f["s"], group=32,
                                                             partials=[f["p"]]),
        route=lambda: tw.tw_route_experts(f["x"], f["w"], f["ids"], bias=f["b"]))


USES = dict(q8="p R G q s", combine="p R G X rows w out", combine_q8="p R G X rows w q s",
            route="x w ids b")


@pytest.fixture
def no_library(monkeypatch):
    def refuse():
        raise AssertionError("library called before the checks")
    monkeypatch.setattr(tw, "lib", refuse)
    monkeypatch.setattr(tw, "_current_device", lambda: 0)
    monkeypatch.setattr(torch, "Tensor", (torch.Tensor, _Fake))  # isinstance only


def test_binding_refuses_tensors_on_another_device(no_library):
    for op, names in USES.items():
        for bad in names.split():
            with pytest.raises(ValueError, match="current device is cuda:0"):
                _calls(_fakes(bad))[op]()


def test_binding_refuses_wrong_types_and_shapes(no_library):
    T, H, K = 4, 256, 2
    wrong = [("q8", "q", ((T, H), torch.bfloat16)), ("q8", "s", ((T, 1), torch.float32)),
             ("q8", "s", ((T, H // 32), torch.uint8)), ("q8", "q", ((T, H + 8), torch.float8_e4m3fn)),
             ("combine", "X", ((8, H + 8), torch.bfloat16)), ("combine", "X", ((8, H), torch.float16)),
             ("combine", "rows", ((T, K), torch.int64)), ("combine", "rows", ((T + 1, K), torch.int32)),
             ("combine", "w", ((T, K), torch.bfloat16)), ("combine", "w", ((T, K + 1), torch.float32)),
             ("combine", "out", ((T, H), torch.float32)), ("combine", "p", ((T + 1, H), torch.bfloat16)),
             ("combine_q8", "s", ((T, H // 64), torch.float32)),
             ("route", "x", ((T, 16), torch.float16)), ("route", "b", ((8,), torch.float32)),
             ("route", "b", ((16,), torch.bfloat16)), ("route", "ids", ((T, K), torch.int64)),
             ("route", "ids", ((T, K + 1), torch.int32)), ("route", "w", ((T + 1, K), torch.float32))]
    for op, name, spec in wrong:
        with pytest.raises(ValueError):
            _calls(_fakes(None, **{name: spec}))[op]()
    f = _fakes()
    with pytest.raises(ValueError, match="scoring"):
        tw.tw_route_experts(f["x"], f["w"], f["ids"], scoring="argmax")


def test_binding_refuses_streams_on_another_device(no_library):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0
    f = _fakes()
    for call in (lambda: tw.FusedQ8Call([f["p"]], f["R"], f["G"], 1e-5, f["q"], f["s"], 32, Stream()),
                 lambda: tw.CombineCall(f["X"], f["rows"], f["w"], f["R"], f["G"], 1e-5, f["out"],
                                        stream=Stream()),
                 lambda: tw.RouteCall(f["x"], f["w"], f["ids"], stream=Stream())):
        with pytest.raises(ValueError, match="stream"):
            call()
