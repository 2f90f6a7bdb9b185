"""Edges of the training operators and the norm on the GPU, against the fp64
oracle's: saturated gates, buffers of the caller's, values next to a rounding
border, calls of more rows than one launch holds."""
import numpy as np
import pytest

from gated_delta_rule_token_amd import workloads
from tests.gpu_helpers import say
from tests.test_gpu_training import FP32, HALF_STEP, check, draw_gradients, gpu_backward, host, oracle_backward

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_token_amd import api
    api.load_library()


@pytest.mark.parametrize("dtype", [np.float32, np.float16, "bf16"], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shared", [False, True], ids=["per_head", "shared"])
def test_rate_gradient_of_saturated_sigmoids(shared, dtype):
    """d_beta = d_rate r (1 - r), element by element: the gradient of the rate
    itself is good to FP32 of its largest value (the bar of every tensor), and
    the factor to 16 half steps of fp32 whatever the logit, so d_beta over the
    fp64 factor is held to the same bar.  With 1 - r formed from the rounded r
    the factor is off by 1e-2 at a logit of 12 and 0 from 17.4 on."""
    case = workloads.random_case(50, lengths=[90, 3, 40], H=2, HV=4, DK=32, DV=16, dtype=dtype, update_rule="gated_delta",
                                 beta_activation="sigmoid", qk_l2_norm=1)
    if shared:
        case["beta"] = np.ascontiguousarray(case["beta"][:, :1])
    logits = np.float32([8, -8, 12, -12, 17, 20, -20, 60, -60, 0.5])
    case["beta"] = case["beta"] * np.float32(0.1) + logits[np.arange(133) % 10][:, None]
    d_o, d_st = draw_gradients(case, True)
    got, want = host(gpu_backward(case, d_o, d_st).beta), oracle_backward(case, d_o, d_st)["beta"]
    t = np.exp(-np.abs(case["beta"].astype(np.float64)))
    factor = t / (1 + t) ** 2
    rate, bar = want / factor, (FP32 + 16 * 2.0 ** -24) * np.abs(want / factor).max()
    err = np.abs(got / factor - rate).max()
    say("  d_beta over r (1 - r): max err %.3e (bound %.1e)" % (err, bar))
    assert err <= bar


def test_caller_buffers_of_every_gradient():
    """A buffer given for the initial states' gradient is filled, with an
    initial state or without one; one for a tensor that the call does not have
    is refused, as nothing would be written to it."""
    from gated_delta_rule_token_amd import api
    none = dict.fromkeys(api.Gradients._fields)
    for with_initial in (True, False):
        case = workloads.random_case(51, lengths=[70, 0, 5], H=1, HV=2, DK=16, DV=24, update_rule="gated_delta",
                                     with_initial=with_initial)
        d_o, d_st = draw_gradients(case, False)
        want = gpu_backward(case, d_o, d_st, want_initial_state=True)
        buf = torch.full((3, 2, 24, 16), 7.0, device="cuda")
        got = gpu_backward(case, d_o, d_st, out=api.Gradients(**dict(none, initial_state=buf)))
        assert got.initial_state is buf and torch.equal(buf, want.initial_state)
        buf.fill_(7.0)
        left = gpu_backward(case, d_o, d_st, want_initial_state=False, out=api.Gradients(**dict(none, initial_state=buf)))
        assert left.initial_state is None and torch.all(buf == 7)
        for name in ("a_log", "dt_bias", "gate_scale"):
            with pytest.raises(api.GDRError, match=name):
                gpu_backward(case, d_o, d_st, out=api.Gradients(**dict(none, **{name: torch.zeros(2, device="cuda")})))
    case = workloads.random_case(52, lengths=[8], H=1, HV=2, DK=16, DV=16, update_rule="linear")
    d_o, d_st = draw_gradients(case, False)
    for name in ("gate", "beta"):
        with pytest.raises(api.GDRError, match=name):
            gpu_backward(case, d_o, d_st, out=api.Gradients(**dict(none, **{name: torch.zeros(8, 2, device="cuda")})))


def _quotient_codes(y, scale, group):
    """e4m3 of the fp32 quotient y / scale, nearest even, on the host."""
    width = y.shape[1]
    s = scale.cpu().repeat_interleave(group or width, 1)[:, :width]
    return (y.cpu() / s).clamp(-448, 448).to(torch.float8_e4m3fn).float()


@pytest.mark.parametrize("width,group", [(64, 0), (256, 32), (1001, 128), (4096, 0), (16400, 512)])
def test_norm_in_8_bits_rounds_the_quotient(width, group):
    """y8 is the fp32 quotient of the y and the scale that are returned,
    rounded to nearest even: bit for bit, also for values placed on the
    midpoints of two codes and on the floats beside them."""
    from gated_delta_rule_token_amd import api
    rng = np.random.Generator(np.random.PCG64(width))
    x = torch.from_numpy(rng.standard_normal((40, width)).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.standard_normal(width).astype(np.float32)).cuda()
    y = api.rms_norm(x, w).y
    got = api.rms_norm(x, w, out_dtype=torch.float8_e4m3fn, group=group)
    assert torch.equal(got.y.cpu().float(), _quotient_codes(y, got.scale, group))
    # rows of 2^-30 and eps = 1: inv is 1 and y is x
    g = group or width
    n = -(-width // g)
    top = (448 * 2.0 ** -30 * (1 + rng.random((40, n, 1)))).astype(np.float32)
    scale = top / np.float32(448)
    code = rng.integers(1, 126, (40, n, g))
    mag = np.where(code < 8, code * 2.0 ** -9, (8 + code % 8) * 2.0 ** (code // 8 - 10.0))
    step = np.where(code < 8, 2.0 ** -9, 2.0 ** (code // 8 - 10.0))
    v = ((mag + step / 2) * scale).astype(np.float32)
    v = (v.view(np.int32) + rng.integers(-2, 3, v.shape).astype(np.int32)).view(np.float32)
    v[..., :1] = top
    x = torch.from_numpy((v * rng.choice(np.float32([-1, 1]), v.shape)).reshape(40, n * g)[:, :width].copy()).cuda()
    got = api.rms_norm(x, eps=1.0, out_dtype=torch.float8_e4m3fn, group=group)
    assert torch.equal(api.rms_norm(x, eps=1.0).y, x)
    assert torch.equal(got.scale.cpu(), torch.from_numpy(scale[..., 0]))
    assert torch.equal(got.y.cpu().float(), _quotient_codes(x, got.scale, group))


@pytest.mark.parametrize("size", [1e-30, 1e-37, 1e-38, 1e-41, 1e-43, 1e-45])
@pytest.mark.parametrize("group", [0, 32])
def test_norm_in_8_bits_of_tiny_rows_has_their_scale(size, group):
    """Scales down to denormal ones: max / 448 in fp32, 1 only where that rounds
    to 0, and the codes of the quotients, so that the largest of a group lies
    at 448 but for the rounding of a denormal scale."""
    from gated_delta_rule_token_amd import api
    rng = np.random.Generator(np.random.PCG64(8))
    x = torch.from_numpy((rng.standard_normal((5, 200)) * size).astype(np.float32)).cuda()
    got = api.rms_norm(x, eps=1.0, out_dtype=torch.float8_e4m3fn, group=group)  # inv = 1: y = x
    for c, s in enumerate(got.scale.cpu().double().unbind(1)):
        part = x[:, c * group:(c + 1) * group] if group else x
        top = part.abs().amax(1).cpu().double() / 448
        zero = top <= 2.0 ** -150
        assert torch.all(s[zero] == 1)
        assert torch.all((s - top).abs()[~zero] <= 2.0 ** -24 * top[~zero] + 2.0 ** -150)
        full = (top > 2.0 ** -126) & ~zero
        q = got.y[:, c * group:(c + 1) * group] if group else got.y
        assert torch.all(q.cpu().float().abs().amax(1)[full] == 448)
    assert torch.equal(got.y.cpu().float(), _quotient_codes(x, got.scale, group))


# more rows than 2,048 workgroups of 16, 8, 4 or 1 rows take at once, and no multiple of that
MANY = [(33001, 128, 64), (16500, 250, 0), (9000, 512, 128), (8300, 2048, 0), (2500, 4096, 128), (2500, 4100, 0),
        (2100, 8200, 512), (2100, 16400, 256)]


@pytest.mark.parametrize("rows,width,group", MANY)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_norm_of_more_rows_than_one_launch_holds(rows, width, group, dtype):
    """A workgroup's further rows, with the next one on its way: in place, in
    8 bits and backwards, against fp64 (the bars of the small calls)."""
    from gated_delta_rule_token_amd import api
    dt, half = getattr(torch, dtype), HALF_STEP[dtype]
    gen = torch.Generator(device="cuda").manual_seed(rows + width)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    x, res, w, dy = draw(rows, width), draw(rows, width), draw(width), draw(rows, width)
    r = (x.float() + res.float()).to(dt)
    inv = torch.rsqrt(r.double().square().mean(-1, keepdim=True) + 1e-6)
    h = r.double() * inv
    y = h * w.double()
    kept = res.clone()
    got = api.rms_norm(x, w, residual=kept, residual_out=kept, want_inv_rms=True)
    assert torch.equal(kept, r)
    assert torch.all((got.inv_rms.double()[:, None] - inv).abs() <= 1e-5 * inv)
    assert torch.all((got.y.double() - y).abs() <= (half + 1e-5) * y.abs() + 2.0 ** -25)  # half of fp16's smallest value
    kept = res.clone()
    eight = api.rms_norm(x, w, residual=kept, residual_out=kept, out_dtype=torch.float8_e4m3fn, group=group)
    assert torch.equal(kept, r)
    g = group or width
    amax = torch.nn.functional.pad(y.abs(), (0, -width % g)).view(rows, -1, g).amax(-1)
    assert torch.all((eight.scale.double() - amax / 448).abs() <= 1e-5 * amax / 448)
    t = y / eight.scale.double().repeat_interleave(g, 1)[:, :width]
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    assert torch.all((eight.y.double() - t).abs() <= step / 2 + 2e-5 * t.abs())
    back = api.rms_norm_backward(dy, r, w, got.inv_rms)
    d = dy.double() * w.double()
    dx = inv * (d - h * (d * h).mean(-1, keepdim=True))
    assert (back.x.double() - dx).abs().max() <= (half + FP32) * dx.abs().max()
    dw = (dy.double() * h).sum(0)
    assert (back.weight.double() - dw).abs().max() <= FP32 * dw.abs().max()


def test_raw_gate_sums_over_many_chunks():
    """More chunks than the 256 threads that add up a head's sums."""
    rng = np.random.Generator(np.random.PCG64(9))
    check(workloads.random_case(53, lengths=rng.integers(0, 4, 700), H=1, HV=2, DK=16, DV=8, update_rule="gated_delta",
                                gate_activation="qwen", beta_activation="sigmoid", qk_l2_norm=1), what="700 requests")
    check(workloads.random_case(54, lengths=rng.integers(1, 3, 400), H=1, HV=3, DK=200, DV=8, update_rule="gated",
                                gate_activation="qwen", folded_scale=True), what="400 requests")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v", "d_o", "initial_state", "d_final_state"])
def test_backward_keeps_a_bad_value_in_its_request(where, bad):
    """A NaN or an infinity in one request: the rows and states of the others
    have the bits that they have without it."""
    case = workloads.random_case(55, lengths=[70, 100, 0, 65], H=1, HV=2, DK=32, DV=16, update_rule="gated_delta",
                                 gate_activation="qwen", beta_activation="sigmoid", qk_l2_norm=1)
    d_o, d_st = draw_gradients(case, True)
    good = gpu_backward(case, d_o, d_st)
    case = {name: x.copy() if isinstance(x, np.ndarray) else x for name, x in case.items()}
    d_o, d_st = d_o.copy(), d_st.copy()
    if where in ("initial_state", "d_final_state"):
        (case["initial_state"] if where == "initial_state" else d_st)[1, 0, 3, 5] = bad
    else:
        (d_o if where == "d_o" else case[where])[70 + 40, 0, 7] = bad
    got = gpu_backward(case, d_o, d_st)
    assert not torch.isfinite(got.q[70:170]).all() or not torch.isfinite(got.k[70:170]).all()
    for name in ("q", "k", "v", "gate", "beta"):
        for rows in (slice(0, 70), slice(170, 235)):
            assert torch.equal(getattr(got, name)[rows], getattr(good, name)[rows]), name
    for b in (0, 2, 3):
        assert torch.equal(got.initial_state[b], good.initial_state[b])
