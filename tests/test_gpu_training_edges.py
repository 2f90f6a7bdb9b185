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
