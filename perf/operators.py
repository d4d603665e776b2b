"""What the 8-bit norm step, the expert router and the expert combine are
measured on: their cases, their plain forms and their work.

The three operators surround the experts of a mixture-of-experts layer:

  q8       z = sum of N partials + residual; residual <- bf16(z); RMSNorm(z)
           in e4m3 with one scale per row or per group of 32, 64 or 128
  route    scores of E experts per token -> the K best and their weights
  combine  z = K weighted expert rows + N partials + residual; residual <-
           bf16(z); RMSNorm(z) in bf16, or in e4m3 as above

``own`` False: plain torch in 32 bits (64 where the choice of an expert or a
power-of-two scale sits next to a border). ``own`` True: the framework's calls.
"""

import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126  # the smallest scale: a group of zeros has it
DEVICE = "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------ cases


def _q8(name, T, H, N, group, scale):
    return dict(name=name, op="q8", T=T, H=H, N=N, group=group, scale=scale)


def _combine(name, T, H, K, N, dropped, group=-1, scale=""):
    """group -1: bf16 output; otherwise e4m3 with that group and scale type."""
    return dict(name=name, op="combine", T=T, H=H, K=K, N=N, dropped=dropped, group=group,
                scale=scale)


def _route(name, T, E, K, dtype, scoring, bias, n_groups, top_groups, group_top, renormalize,
           scale, masked):
    return dict(name=name, op="route", T=T, E=E, K=K, dtype=dtype, scoring=scoring, bias=bias,
                n_groups=n_groups, top_groups=top_groups, group_top=group_top,
                renormalize=renormalize, scale=scale, masked=masked)


def listed():
    return [
        # one token of a decode step before an 8-bit product, one scale per token
        _q8("q8 one token", 1, 8192, 8, 0, "f32"),
        # a batch and a hidden size that fill no power of two, per-token scales
        _q8("q8 ragged", 333, 5000, 3, 0, "f32"),
        # one chunk of a prompt at the benchmark's layer shape, block scales of 32
        _q8("q8 layer", 1024, 8192, 8, 32, "e8m0"),
        # the benchmark's largest layer shape, group scales
        _q8("q8 large", 8192, 16384, 8, 128, "f32"),
        # one token of a decode step: eight experts' rows
        _combine("combine one token", 1, 4096, 8, 0, 0.0),
        # a decode batch with a shared expert, 8-bit output for the next product
        _combine("combine decode q8", 64, 8192, 8, 1, 0.0, 32, "e8m0"),
        # odd sizes, five experts, two partials, a fifth of the slots dropped by capacity
        _combine("combine ragged", 1000, 2056, 5, 2, 0.2),
        # a prompt of two experts per token beside a shared expert
        _combine("combine prompt", 8192, 8192, 2, 1, 0.0),
        # one token: sigmoid scores, a bias for balance, four of eight groups
        _route("route one token", 1, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5, 0.0),
        # a decode batch over an odd number of experts, some masked, scores as they are
        _route("route ragged", 129, 100, 3, "bf16", "softmax", False, 1, 1, 1, False, 1.0, 0.1),
        # a long prompt, softmax over the chosen
        _route("route softmax", 32768, 64, 6, "bf16", "softmax", False, 1, 1, 1, True, 1.0, 0.0),
        # a long prompt, sigmoid scores with bias and groups
        _route("route groups", 16384, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5, 0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _divisors(n, most):
    return [d for d in range(1, min(n, most) + 1) if n % d == 0]


def draw(rng):
    op = rng.choice(("q8", "combine", "route"))
    if op == "route":
        E = _log_int(rng, 4, 1024)
        T = _log_int(rng, 1, min(65536, (1 << 25) // E))
        K = rng.randint(1, min(E, 16))
        scoring = rng.choice(("softmax", "sigmoid"))
        G = rng.choice(_divisors(E, 32))
        top = rng.randint(1, G)
        while E // G * top < K:  # the chosen groups hold K experts
            top += 1
        return _drop_name(_route("", T, E, K, rng.choice(("f32", "bf16")), scoring,
                                 rng.random() < 0.5, G, top,
                                 rng.choice((1, 2)) if E // G >= 2 else 1, rng.random() < 0.5,
                                 rng.choice((1.0, 2.5)), rng.choice((0.0, 0.0, 0.3))))
    group = rng.choice((0, 32, 64, 128))
    unit = group or 8
    H = unit * _log_int(rng, max(1, 256 // unit), 32768 // unit)
    scale = rng.choice(("f32", "e8m0"))
    if op == "q8":
        N = rng.randint(1, 16)
        T = _log_int(rng, 1, max(2, min(16384, (1 << 30) // (H * (N + 2)))))
        return _drop_name(_q8("", T, H, N, group, scale))
    K, N = rng.randint(1, 16), rng.randint(0, 4)
    T = _log_int(rng, 1, max(2, min(16384, (1 << 30) // (H * (K + N + 2)))))
    if rng.random() < 0.5:
        group, scale = -1, ""
    return _drop_name(_combine("", T, H, K, N, rng.choice((0.0, 0.1)), group, scale))


def _drop_name(case):
    case.pop("name")
    return case


# ------------------------------------------------------------------ inputs


def _randn(g, *shape):
    return torch.randn(shape, device=DEVICE, generator=g)


def _norm_inputs(g, s, T, H, N):
    """Partials, residual and gamma of a layer: small partials, a residual
    stream whose channels differ in size, a gamma near one."""
    s["partials"] = torch.randn((N, T, H), device=DEVICE, generator=g,
                                dtype=torch.bfloat16).mul_(0.05)
    channel = torch.exp(0.5 * _randn(g, H))
    s["residual"] = (_randn(g, T, H) * channel).to(torch.bfloat16)
    s["gamma"] = (1.0 + 0.1 * _randn(g, H)).to(torch.bfloat16)


def _out_buffers(s, T, H, group, scale):
    if group < 0:
        s["out"] = torch.empty((T, H), device=DEVICE, dtype=torch.bfloat16)
        s["scales"] = None
        return
    s["out"] = torch.empty((T, H), device=DEVICE, dtype=torch.float8_e4m3fn)
    s["scales"] = torch.empty((T, H // group if group else 1), device=DEVICE,
                              dtype=torch.float32 if scale == "f32" else torch.float8_e8m0fnu)


def prepare(case, seed):
    """Inputs, output buffers and, for the framework's calls, the prepared
    call: a decode loop marshals its arguments once and then only launches."""
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    s = dict(case=case)
    T = case["T"]
    if case["op"] == "route":
        E, K = case["E"], case["K"]
        x = 1.5 * _randn(g, T, E)
        if case["masked"]:
            x = torch.where(torch.rand((T, E), device=DEVICE, generator=g) < case["masked"],
                            -math.inf, x)
        s["logits"] = x.to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        s["bias"] = 0.05 * _randn(g, E) if case["bias"] else None
        s["weights"] = torch.empty((T, K), device=DEVICE, dtype=torch.float32)
        s["ids"] = torch.empty((T, K), device=DEVICE, dtype=torch.int32)
    else:
        H, N = case["H"], case["N"]
        _norm_inputs(g, s, T, H, N)
        _out_buffers(s, T, H, case["group"], case["scale"])
        if case["op"] == "combine":
            K = case["K"]
            M = T * K  # every slot's row, in the order in which the experts wrote them
            s["experts"] = torch.randn((M, H), device=DEVICE, generator=g, dtype=torch.bfloat16)
            rows = torch.randperm(M, device=DEVICE, generator=g).to(torch.int32).view(T, K)
            if case["dropped"]:
                gone = torch.rand((T, K), device=DEVICE, generator=g) < case["dropped"]
                rows = torch.where(gone, -1, rows)
            s["rows"] = rows.contiguous()
            s["weights"] = torch.softmax(_randn(g, T, K), 1)
    if own:
        s["call"] = _prepared(s)
    return s


def _prepared(s):
    import reduce_rmsnorm_gb300 as tw
    case = s["case"]
    if case["op"] == "route":
        return tw.RouteCall(s["logits"], s["weights"], s["ids"], bias=s["bias"],
                            scoring=case["scoring"], n_groups=case["n_groups"],
                            top_groups=case["top_groups"], group_top=case["group_top"],
                            renormalize=case["renormalize"], scale=case["scale"])
    if case["op"] == "q8":
        return tw.FusedQ8Call(s["partials"], s["residual"], s["gamma"], EPS, s["out"], s["scales"],
                              group=case["group"])
    if case["group"] < 0:
        return tw.CombineCall(s["experts"], s["rows"], s["weights"], s["residual"], s["gamma"],
                              EPS, s["out"], partials=s["partials"])
    return tw.CombineQ8Call(s["experts"], s["rows"], s["weights"], s["residual"], s["gamma"], EPS,
                            s["out"], s["scales"], group=case["group"], partials=s["partials"])


# ------------------------------------------------------------------ one pass


def run(state):
    case = state["case"]
    if own:
        state["call"]()
        if case["op"] == "route":
            return dict(weights=state["weights"], ids=state["ids"])
        out = dict(out=state["out"], residual=state["residual"])
        if state["scales"] is not None:
            out["scales"] = state["scales"]
        return out
    return _plain_route(state) if case["op"] == "route" else _plain_norm(state)


def _plain_norm(s):
    case = s["case"]
    z = s["residual"].float()
    if case["N"]:
        z = s["partials"].float().sum(0) + z
    if case["op"] == "combine":
        rows = s["rows"].long()
        picked = s["experts"][rows.clamp(min=0)].float()
        w = torch.where(rows >= 0, s["weights"], 0.0)
        z = (picked * w[:, :, None]).sum(1) + z
    s["residual"].copy_(z)  # the step updates the residual in place
    y = z * torch.rsqrt((z * z).mean(1, keepdim=True) + EPS) * s["gamma"].float()
    out = dict(residual=s["residual"])
    if case["group"] < 0:
        out["out"] = y.to(torch.bfloat16)
        return out
    T, H = y.shape
    y = y.view(T, -1, case["group"] or H)
    amax = y.abs().amax(2)
    if case["scale"] == "f32":
        scale = (amax / E4M3_MAX).clamp(min=SCALE_MIN)
    else:  # 448 = 0.875 * 2^9: the smallest power of two that keeps amax within it
        m, e = torch.frexp(amax)
        k = torch.where(m <= 0.875, e - 9, e - 8)
        k = torch.where(amax > 0, k, torch.full_like(k, -126)).clamp(-126, 127)
        scale = torch.ldexp(torch.ones_like(amax), k)
    q = (y / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    out["out"] = q.to(torch.float8_e4m3fn).view(T, H)
    out["scales"] = scale if case["scale"] == "f32" else scale.to(torch.float8_e8m0fnu)
    return out


def _plain_route(s):
    """The choice in 64 bits: two experts' values may differ by less than 32
    bits hold."""
    case = s["case"]
    x = s["logits"].double()
    T, E = x.shape
    K, G = case["K"], case["n_groups"]
    if case["scoring"] == "softmax":
        top = x.amax(1, keepdim=True).clamp(min=-1e300)
        score = torch.exp(x - top)
        score = score / score.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    value = score if s["bias"] is None else score + s["bias"].double()
    value = torch.where(x > -math.inf, value, -math.inf)
    # without a bias the order of the scores is that of the logits
    order = x if s["bias"] is None else value
    if case["top_groups"] < G:
        best = value.view(T, G, E // G).sort(dim=2, descending=True)[0][:, :, :case["group_top"]]
        best = torch.where(best > -math.inf, best, 0.0).sum(2) + torch.where(
            best[:, :, 0] > -math.inf, 0.0, -math.inf)
        rank = best.sort(dim=1, descending=True, stable=True)[1].argsort(1)
        keep = (rank < case["top_groups"]).repeat_interleave(E // G, 1)
        order = torch.where(keep, order, -math.inf)
    picked, ids = order.sort(dim=1, descending=True, stable=True)
    picked, ids = picked[:, :K], ids[:, :K]
    there = picked > -math.inf
    w = torch.where(there, score.gather(1, ids), 0.0)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return dict(weights=(w * case["scale"]).float(),
                ids=torch.where(there, ids, -1).to(torch.int32))


# ------------------------------------------------------------------ 64 bits


def exact(case, seed):
    """The operators' definitions in 64 bits, a block of tokens at a time."""
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    parts = [_exact_route(s, a, b) if case["op"] == "route" else _exact_norm(s, a, b)
             for a, b in _blocks(case)]
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _blocks(case):
    T = case["T"]
    step = max(1, (1 << 24) // max(1, case.get("H", 1) * case.get("K", 1), case.get("E", 1)))
    return [(a, min(T, a + step)) for a in range(0, T, step)]


def _exact_norm(s, a, b):
    case = s["case"]
    z = s["residual"][a:b].double()
    for n in range(case["N"]):
        z = z + s["partials"][n, a:b].double()
    if case["op"] == "combine":
        for k in range(case["K"]):
            r = s["rows"][a:b, k].long()
            term = s["experts"][r.clamp(min=0)].double() * s["weights"][a:b, k, None].double()
            z = z + torch.where(r[:, None] >= 0, term, 0.0)
    H = z.shape[1]
    rms = (torch.linalg.vector_norm(z, dim=1, keepdim=True) ** 2 / H + EPS).sqrt()
    y = z / rms * s["gamma"].double()
    if case["group"] < 0:
        return dict(out=y, residual=z)
    group = case["group"] or H
    amax = y.abs().reshape(b - a, H // group, group).max(2)[0]
    scale = amax / E4M3_MAX
    if case["scale"] == "e8m0":
        k = torch.log2(scale.clamp(min=SCALE_MIN)).floor()
        k = torch.where(torch.pow(2.0, k) < scale, k + 1, k)
        scale = torch.pow(2.0, k)
    scale = scale.clamp(min=SCALE_MIN)
    # the value before its rounding to 8 bits, as for a bf16 output
    return dict(out=y / scale.repeat_interleave(group, 1), residual=z, scales=scale)


def _exact_route(s, a, b):
    case = s["case"]
    x = s["logits"][a:b].double()
    masked = torch.isneginf(x)
    if case["scoring"] == "softmax":
        score = torch.where(masked, 0.0, torch.softmax(torch.where(masked, -1e30, x), 1))
    else:
        score = torch.where(masked, 0.0, torch.sigmoid(x))
    value = score + (0.0 if s["bias"] is None else s["bias"].double())
    value = torch.where(masked, -math.inf, value)
    order = torch.where(masked, -math.inf, x if s["bias"] is None else value)
    G = case["n_groups"]
    if case["top_groups"] < G:
        rest = value.reshape(b - a, G, -1).clone()
        total = torch.zeros_like(rest[:, :, 0])
        for i in range(case["group_top"]):
            m, at = rest.max(2)
            total = total + (m if i == 0 else torch.where(torch.isneginf(m), 0.0, m))
            rest.scatter_(2, at[:, :, None], -math.inf)
        keep = torch.zeros_like(total, dtype=torch.bool)
        for _ in range(case["top_groups"]):
            left = torch.where(keep, -math.inf, total)
            first = (left == left.max(1, keepdim=True)[0]) & ~keep
            first = first & (first.cumsum(1) == 1)
            keep = keep | first
        order = torch.where(keep.repeat_interleave(x.shape[1] // G, 1), order, -math.inf)
    weights, ids = [], []
    for _ in range(case["K"]):
        m = order.max(1, keepdim=True)[0]
        first = order == m
        first = first & (first.cumsum(1) == 1) & ~torch.isneginf(m)
        weights.append((score * first).sum(1))
        ids.append(torch.where(first.any(1), first.int().argmax(1), -1))
        order = torch.where(first, -math.inf, order)
    w, ids = torch.stack(weights, 1), torch.stack(ids, 1)
    if case["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, 1.0), 0.0)
    return dict(weights=w * case["scale"], ids=ids.to(torch.int32))


# ------------------------------------------------------------------ work


def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, K = case["E"], case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        return dict(bytes=T * E * size + (4 * E if case["bias"] else 0) + T * K * 8,
                    flops=T * E * 8 + T * K * 4)
    H, N = case["H"], case["N"]
    read, flops = (N + 1) * T * H * 2 + 2 * H, T * H * (N + 5)
    if case["op"] == "combine":
        # a dropped slot's row is not read; its index and weight are
        slots = T * case["K"]
        kept = slots * (1.0 - case["dropped"])
        read, flops = read + kept * H * 2 + slots * 8, flops + 2 * kept * H
    if case["group"] < 0:
        written = 2 * T * H * 2
    else:
        flops += 3 * T * H
        scales = T * (H // case["group"] if case["group"] else 1)
        written = T * H * 3 + scales * (4 if case["scale"] == "f32" else 1)
    return dict(bytes=read + written, flops=flops)
