"""Edges of the training operators and the norm on the GPU, against the fp64
oracle's: saturated gates, buffers of the caller's, values next to a rounding
border, calls of more rows than one launch holds."""
import numpy as np
import pytest

from gated_delta_rule_token_amd import workloads
from tests.gpu_helpers import say
from tests.test_gpu_training import FP32, draw_gradients, gpu_backward, host, oracle_backward

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
