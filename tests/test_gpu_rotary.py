"""Norm and rotation of q and k, and its gradients, against plain forms in 64
bits, on an MI355X.

Tolerances.  With u = 2^-24, a head's sum of squares adds at most 16 values in
a lane and then a tree of at most 6 levels: under 24 u, 12 u in its root; the
quotient, the weight, the turn's two products and sum add 8 u; the angle is off
by 4e-7 at most (the turn's fraction rounded to fp32, pi 2^-24 = 1.9e-7, and the
sine's own error), relative to the pair's length.  So y is off by under
(20 u + 4e-7) 1.5 < 4e-6 times the pair's length, and by half a step of its type
from the store.  A gradient has one more sum of that kind: 8e-6 times the
largest terms of the head, inv * max |t|, which bounds the pairs as well.  The
weights' gradients are sums over all rows in fp32, chains of at most 1,000 terms:
1,000 u = 6e-5 of the sum of magnitudes.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_token_amd import api
    api.load_library()


DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_step(x, dtype):
    fi = torch.finfo(dtype)
    return x.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def make(seed, T, H, HK, d, R, dtype, axes=1, weight="f32", far=100, lead=None):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    lead = lead or (T,)
    c = dict(q=n(*lead, H, d).to(DT[dtype]), k=None if HK == 0 else n(*lead, HK, d).to(DT[dtype]))
    c["positions"] = torch.randint(-far, far, ((axes,) if axes > 1 else ()) + lead, generator=g).to(torch.int32)
    c["inv_freq"] = torch.exp(-9.2 * torch.arange(R // 2) / max(1, R // 2)).float()
    c["axes"] = None if axes == 1 else (torch.arange(R // 2) % axes).to(torch.int32)
    c["q_weight"] = None if weight is None else (1 + 0.1 * n(d)).to(DT[weight])
    c["k_weight"] = None if weight is None or HK == 0 else (1 + 0.1 * n(d)).to(DT[weight])
    return c


def plain(x, weight, c, interleaved, norm, eps):
    """One of q and k in the tensors' own precision (64 bits here)."""
    pos, R = c["positions"].double(), 2 * c["inv_freq"].shape[0]
    if c["axes"] is None:
        angle = pos[..., None] * c["inv_freq"].double()
    else:
        angle = torch.stack([pos[int(a)] for a in c["axes"]], -1) * c["inv_freq"].double()
    cos, sin = torch.cos(angle)[..., None, :].to(x), torch.sin(angle)[..., None, :].to(x)
    h = x
    if norm:
        h = h / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if weight is not None:
        h = h * weight
    a, b = (h[..., 0:R:2], h[..., 1:R:2]) if interleaved else (h[..., : R // 2], h[..., R // 2: R])
    t0, t1 = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([t0, t1], -1).flatten(-2) if interleaved else torch.cat([t0, t1], -1)
    return torch.cat([turned, h[..., R:]], -1)


def pair_length(y, R, interleaved):
    out = y.abs().clone()
    if interleaved:
        p = torch.sqrt(y[..., 0:R:2] ** 2 + y[..., 1:R:2] ** 2)
        out[..., 0:R:2] = out[..., 1:R:2] = p
    else:
        p = torch.sqrt(y[..., : R // 2] ** 2 + y[..., R // 2: R] ** 2)
        out[..., : R // 2] = out[..., R // 2: R] = p
    return out


def dev(c):
    return {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in c.items()}


def call(c, interleaved=False, norm=True, eps=1e-6, **kw):
    from gated_delta_rule_token_amd import api
    r = api.qk_rotary(c["q"], c["k"], c["positions"], c["inv_freq"], axes=c["axes"], q_weight=c["q_weight"],
                      k_weight=c["k_weight"], eps=eps, interleaved=interleaved, norm=norm, **kw)
    torch.cuda.synchronize()
    return r


def double(t):
    return None if t is None else t.double()


def check(c, got, interleaved=False, norm=True, eps=1e-6):
    for name in ("q", "k"):
        x, y = c[name], getattr(got, name)
        if x is None:
            assert y is None
            continue
        ref = plain(double(x), double(c[name + "_weight"]), c, interleaved, norm, eps)
        assert y.shape == x.shape and y.dtype == x.dtype
        err = (y.cpu().double() - ref).abs()
        bound = 4e-6 * pair_length(ref, 2 * c["inv_freq"].shape[0], interleaved) + half_step(ref, x.dtype) * (1 + 1e-5)
        assert bool((err <= bound).all()), (name, float((err / bound).max()))


# T, H, HK, d, R, dtype, axes, weight, interleaved, norm
FORMS = [
    (1, 1, 1, 2, 2, "f32", 1, "f32", False, True), (3, 2, 2, 128, 128, "bf16", 1, "bf16", False, True),
    (77, 16, 16, 128, 128, "f16", 1, "f32", False, True), (300, 4, 1, 128, 64, "bf16", 3, "f32", False, True),
    (33, 5, 3, 64, 64, "f16", 2, "f16", True, True), (19, 3, 0, 256, 256, "bf16", 1, None, False, True),
    (40, 2, 7, 256, 64, "f32", 1, "f32", True, True), (25, 9, 3, 72, 40, "f32", 1, "f32", True, True),
    (25, 9, 3, 72, 40, "bf16", 4, "f32", False, True), (130, 1, 1, 63, 62, "f16", 1, "f32", False, True),
    (51, 3, 2, 255, 100, "bf16", 1, "bf16", True, True), (7, 70, 40, 16, 16, "bf16", 1, "f32", False, True),
    (12, 300, 1, 8, 4, "f32", 2, None, False, False), (65, 4, 4, 96, 32, "f16", 1, "f32", False, False),
    (1000, 2, 1, 40, 20, "bf16", 1, "f32", False, True), (18, 3, 3, 112, 112, "f16", 3, "f16", True, False),
]


@pytest.mark.parametrize("T,H,HK,d,R,dtype,axes,weight,inter,norm", FORMS, ids=["%d-%d-%d-%d-%d-%s" % f[:6] for f in FORMS])
def test_rotary(T, H, HK, d, R, dtype, axes, weight, inter, norm):
    c = make(T + d, T, H, HK, d, R, dtype, axes, weight)
    check(c, call(dev(c), inter, norm), inter, norm)


def test_far_positions_and_every_int32():
    """Angles to 2^31 turns of a radian: the product is not formed in 32 bits."""
    c = make(1, 64, 2, 2, 64, 64, "f32")
    c["positions"] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 1048575, 12345678] * 8, dtype=torch.int32)
    check(c, call(dev(c)))


def test_views_of_one_projection_rank_4_and_odd_offsets():
    B, L, H, HK, d = 3, 11, 4, 2, 64
    for dtype, pad in (("bf16", 64), ("f16", 3), ("f32", 1)):
        rows = torch.randn(B, L, (H + HK) * d + pad, generator=torch.Generator().manual_seed(3)).to(DT[dtype])
        c = make(4, 0, H, HK, d, 32, dtype, lead=(B, L), far=5000)
        for off in (0, pad):
            gpu = dev(c)
            wide = rows.cuda()
            gpu["q"] = wide[..., off: off + H * d].view(B, L, H, d)
            gpu["k"] = wide[..., off + H * d: off + (H + HK) * d].view(B, L, HK, d)
            c["q"], c["k"] = gpu["q"].cpu(), gpu["k"].cpu()
            fresh = call(gpu)
            check(c, fresh)
            # in place: the projection's other columns stay
            before = wide.clone()
            call(gpu, out=(gpu["q"], gpu["k"]))
            assert torch.equal(gpu["q"], fresh.q) and torch.equal(gpu["k"], fresh.k)
            assert torch.equal(wide[..., :off], before[..., :off])
            assert torch.equal(wide[..., off + (H + HK) * d:], before[..., off + (H + HK) * d:])


def test_rows_around_a_result_stay():
    c = make(6, 5, 2, 1, 64, 64, "bf16")
    wide = torch.full((7, 2 * 64 + 64 + 10), 3.0, dtype=torch.bfloat16, device="cuda")
    oq, ok = wide[1:6, 5:133].view(5, 2, 64), wide[1:6, 133:197].view(5, 1, 64)
    check(c, call(dev(c), out=(oq, ok)))
    rest = wide.clone()
    rest[1:6, 5:197] = 3.0
    assert bool((rest == 3.0).all())


def test_rows_past_32_bit_offsets():
    """Views whose last rows lie past 2^31 elements."""
    from gated_delta_rule_token_amd import api
    T, stride = 70000, 40000
    wide = torch.zeros(T, stride, dtype=torch.bfloat16, device="cuda")
    c = dev(make(5, 16, 2, 1, 64, 64, "bf16", far=4096))
    q, k = wide[:, 100:228].view(T, 2, 64), wide[:, 39900:39964].view(T, 1, 64)
    q[-16:], k[-16:] = c["q"], c["k"]
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[-16:] = c["positions"]
    want = call(c)
    kw = dict(q_weight=c["q_weight"], k_weight=c["k_weight"])
    got = api.qk_rotary(q, k, pos, c["inv_freq"], **kw)
    assert torch.equal(got.q[-16:], want.q) and torch.equal(got.k[-16:], want.k) and not bool(got.q[:-16].any())
    dq, dk = torch.zeros(T, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, 1, 64, dtype=torch.bfloat16, device="cuda")
    dq[-16:], dk[-16:] = want.q, want.k
    small = back(c, want.q, want.k)
    big = api.qk_rotary_backward(dq, dk, q, k, pos, c["inv_freq"], **kw)
    assert torch.equal(big.q[-16:], small.q) and torch.equal(big.k[-16:], small.k)
    api.qk_rotary(q, k, pos, c["inv_freq"], out=(q, k), **kw)  # in place
    assert torch.equal(q[-16:], want.q) and torch.equal(k[-16:], want.k) and not bool(wide[:-16].any())
    del wide, q, k
    torch.cuda.empty_cache()


def test_no_tokens_and_bad_axes():
    c = make(7, 0, 2, 1, 64, 64, "bf16")
    r = call(dev(c))
    assert r.q.shape == (0, 2, 64) and r.k.shape == (0, 1, 64)
    c = make(8, 9, 2, 1, 64, 64, "f32", axes=2)
    c["axes"] = torch.tensor([0, 1, -7, 99] * 8, dtype=torch.int32)
    got = call(dev(c))
    c["axes"] = torch.tensor([0, 1, 0, 1] * 8, dtype=torch.int32)
    check(c, got)


def test_infinities_and_nan_stay_in_their_heads():
    c = make(9, 6, 3, 2, 128, 128, "f32")
    clean = call(dev(c))
    c["q"][2, 1, 5] = float("nan")
    c["q"][4, 0, 70] = float("inf")
    c["k"][0, 1, 0] = 3e38  # its square is past fp32: inv = 0
    got = call(dev(c))
    keep = torch.ones(6, 3, dtype=torch.bool)
    keep[2, 1] = keep[4, 0] = False
    assert torch.equal(got.q.cpu()[keep], clean.q.cpu()[keep])
    assert bool(got.q[2, 1].isnan().all()) and bool(got.q[4, 0].isnan().any())
    assert bool((got.k[0, 1] == 0).all()) and torch.equal(got.k[1:], clean.k[1:])


def test_zero_heads():
    c = make(10, 4, 2, 2, 64, 64, "bf16")
    c["q"].zero_()
    got = call(dev(c))
    assert bool((got.q == 0).all())
    g = back(dev(c), torch.ones_like(c["q"]).cuda(), torch.ones_like(c["k"]).cuda())
    assert bool(g.q.isfinite().all())


# ------------------------------------------------------------------ gradients

def back(c, dq, dk, interleaved=False, norm=True, eps=1e-6, **kw):
    from gated_delta_rule_token_amd import api
    g = api.qk_rotary_backward(dq, dk, c["q"], c["k"], c["positions"], c["inv_freq"], axes=c["axes"],
                               q_weight=c["q_weight"], k_weight=c["k_weight"], eps=eps, interleaved=interleaved,
                               norm=norm, **kw)
    torch.cuda.synchronize()
    return g


def reference(c, name, d_out, interleaved, norm, eps=1e-6):
    """Gradients in 64 bits, of autograd through the plain form."""
    x = double(c[name]).requires_grad_()
    w = None if c[name + "_weight"] is None else double(c[name + "_weight"]).requires_grad_()
    y = plain(x, w, c, interleaved, norm, eps)
    grads = torch.autograd.grad(y, [x] if w is None else [x, w], d_out.double())
    return grads[0], None if w is None else grads[1]


def check_back(c, g, douts, interleaved=False, norm=True, eps=1e-6):
    for name, d_out in zip(("q", "k"), douts):
        if c[name] is None:
            assert getattr(g, name) is None
            continue
        x, w = double(c[name]), double(c[name + "_weight"])
        dx, dw = reference(c, name, d_out, interleaved, norm, eps)
        inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) if norm else torch.ones_like(x[..., :1])
        length = pair_length(d_out.double(), 2 * c["inv_freq"].shape[0], interleaved)
        most = inv * (length * (1 if w is None else w.abs())).amax(-1, keepdim=True)
        n = (x * inv).abs().amax(-1, keepdim=True).clamp(min=1)
        bound = 8e-6 * most * n * n + half_step(dx, c[name].dtype) * (1 + 1e-5)
        err = (getattr(g, name).cpu().double() - dx).abs()
        assert bool((err <= bound).all()), (name, float((err / bound).max()))
        got = getattr(g, name + "_weight")
        if w is None:
            assert got is None
            continue
        total = (length * (x * inv).abs()).flatten(0, -2).sum(0)
        err = (got.cpu().double() - dw).abs()
        assert got.dtype == torch.float32 and bool((err <= 6e-5 * total + 1e-30).all()), (name, float((err / total).max()))


def d_outs(c, seed=99):
    g = torch.Generator().manual_seed(seed)
    return [None if c[n] is None else (0.1 * torch.randn(c[n].shape, generator=g)).to(c[n].dtype) for n in ("q", "k")]


def cuda(ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("T,H,HK,d,R,dtype,axes,weight,inter,norm", FORMS, ids=["%d-%d-%d-%d-%d-%s" % f[:6] for f in FORMS])
def test_rotary_gradients(T, H, HK, d, R, dtype, axes, weight, inter, norm):
    c = make(T + d, T, H, HK, d, R, dtype, axes, weight)
    douts = d_outs(c)
    g = back(dev(c), *cuda(douts), inter, norm)
    check_back(c, g, douts, inter, norm)
    again = back(dev(c), *cuda(douts), inter, norm)
    for a, b in zip(g, again):
        assert (a is None and b is None) or torch.equal(a, b)  # a fixed order of sums


def test_gradients_over_many_workgroups():
    c = make(20, 5000, 8, 2, 128, 128, "bf16", far=100000)
    douts = d_outs(c)
    check_back(c, back(dev(c), *cuda(douts)), douts)


@pytest.mark.parametrize("T,H,HK,d,R,dtype", [(3597, 10, 10, 128, 64, "bf16"), (613, 4, 20, 256, 256, "f32"), (700, 16, 2, 128, 128, "f16"),
                                              (1013, 4, 1, 163, 146, "bf16"), (2600, 1, 9, 44, 12, "f16"), (9000, 1, 1, 13, 6, "f32")])
def test_gradients_with_turns_of_every_length(T, H, HK, d, R, dtype):
    c = make(T, T, H, HK, d, R, dtype, far=4096)
    douts = d_outs(c)
    check_back(c, back(dev(c), *cuda(douts)), douts)
    check(c, call(dev(c)))


def test_gradients_against_differences():
    """(f(x + h e) - f(x - h e)) / 2h of the calls themselves, in fp32 with
    h = 2^-6: the second-order term is h^2 times third derivatives of order 1
    (inv is 1 / (rms), its heads are of size 1), 2.4e-4 of the sum's scale, and
    the outputs' rounding u |f| / h = 4e-6 |f|."""
    c = make(21, 3, 2, 1, 64, 32, "f32", far=50)
    douts = d_outs(c)
    gpu, dd = dev(c), cuda(douts)
    g = back(gpu, *dd)
    f = lambda c: sum(float((r.double() * d.double()).sum()) for r, d in zip(call(c), dd))  # noqa: E731
    rng, h = np.random.default_rng(5), 2.0 ** -6
    for name in ("q", "k", "q_weight", "k_weight"):
        direction = torch.from_numpy(rng.choice([-1.0, 1.0], size=tuple(gpu[name].shape))).float().cuda()
        direction *= torch.from_numpy((rng.random(tuple(gpu[name].shape)) < 0.1)).cuda()
        up, down = dict(gpu), dict(gpu)
        up[name], down[name] = gpu[name] + h * direction, gpu[name] - h * direction
        slope = (f(up) - f(down)) / (2 * h)
        want = float((getattr(g, name).double() * direction.double()).sum())
        scale = float((getattr(g, name).double() * direction.double()).abs().sum())
        assert abs(slope - want) <= 5e-3 * scale + 1e-4, (name, slope, want, scale)


def test_gradients_into_views_of_one_buffer():
    T, H, HK, d = 37, 4, 2, 64
    c = make(22, T, H, HK, d, 64, "f16")
    douts = d_outs(c)
    wide = torch.full((T, (H + HK) * d + 6), 7.0, dtype=torch.float16, device="cuda")
    out = (wide[:, 2: 2 + H * d].view(T, H, d), wide[:, 2 + H * d: 2 + (H + HK) * d].view(T, HK, d))
    g = back(dev(c), *cuda(douts), out=out)
    check_back(c, g, douts)
    assert bool((wide[:, :2] == 7).all()) and bool((wide[:, 2 + (H + HK) * d:] == 7).all())


def test_gradients_without_tokens_are_zero():
    c = make(23, 0, 2, 1, 64, 64, "bf16")
    g = back(dev(c), *cuda(d_outs(c)))
    assert bool((g.q_weight == 0).all()) and bool((g.k_weight == 0).all())


def test_other_streams_and_captured_graphs():
    """Two captured calls of each, replayed several times between eager work:
    every replay gives the eager result."""
    from gated_delta_rule_token_amd import api
    c = make(24, 200, 4, 4, 128, 128, "bf16", far=9999)
    gpu, dd = dev(c), cuda(d_outs(c))
    want, wantg = call(gpu), back(gpu, *dd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(gpu)
    assert torch.equal(got.q, want.q) and torch.equal(got.k, want.k)
    outs, graphs = [], []
    for _ in range(2):
        o = (torch.empty_like(gpu["q"]), torch.empty_like(gpu["k"]))
        og = (torch.empty_like(gpu["q"]), torch.empty_like(gpu["k"]))
        ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        kw = dict(axes=None, q_weight=gpu["q_weight"], k_weight=gpu["k_weight"])
        with torch.cuda.graph(graph):
            api.qk_rotary(gpu["q"], gpu["k"], gpu["positions"], gpu["inv_freq"], out=o, **kw)
            g = api.qk_rotary_backward(*dd, gpu["q"], gpu["k"], gpu["positions"], gpu["inv_freq"], out=og, workspace=ws, **kw)
        outs.append((o, g))
        graphs.append(graph)
    for _ in range(3):
        for (o, g), graph in zip(outs, graphs):
            for t in (*o, *g):
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o[0], want.q) and torch.equal(o[1], want.k)
            assert all(torch.equal(a, b) for a, b in zip(g, wantg))
        call(gpu)


def test_refusals_on_the_gpu():
    from gated_delta_rule_token_amd import api
    c = dev(make(25, 6, 2, 1, 64, 32, "bf16", axes=2))
    args = lambda **o: [dict(c, **o)[n] for n in ("q", "k", "positions", "inv_freq")]  # noqa: E731
    kw = lambda **o: dict(dict(axes=c["axes"], q_weight=c["q_weight"], k_weight=c["k_weight"]), **o)  # noqa: E731
    bad = [
        ("strides", dict(q=c["q"].transpose(0, 1).contiguous().transpose(0, 1)), {}),
        ("strides", dict(q=torch.zeros(6, 2, 128, dtype=torch.bfloat16, device="cuda")[..., ::2]), {}),
        ("k must be", dict(k=c["k"].float()), {}),
        ("k has shape", dict(k=c["k"][:5]), {}),
        ("positions has shape", dict(positions=c["positions"][:, :5].contiguous()), {}),
        ("positions must be", dict(positions=c["positions"].long()), {}),
        ("axes has shape", {}, dict(axes=c["axes"][:5].contiguous())),
        ("need axes", {}, dict(axes=None)),
        ("inv_freq must be", dict(inv_freq=c["inv_freq"].double()), {}),
        ("rotary_dim", dict(inv_freq=torch.zeros(33, device="cuda")), dict(axes=torch.zeros(33, dtype=torch.int32, device="cuda"))),
        ("one dtype", {}, dict(k_weight=c["k_weight"].bfloat16())),
        ("q_weight has shape", {}, dict(q_weight=c["q_weight"][:60].contiguous())),
        ("k_weight given", dict(k=None), {}),
        ("overlaps", {}, dict(out=(c["q"], torch.as_strided(c["q"], (6, 1, 64), (128, 64, 1), 64)))),
        ("out of k must", {}, dict(out=(torch.empty_like(c["q"]), torch.empty_like(c["q"])))),
    ]
    for text, over, more in bad:
        with pytest.raises(api.GDRError, match=text):
            api.qk_rotary(*args(**over), **kw(**more))
    api.qk_rotary(*args(), **kw())
