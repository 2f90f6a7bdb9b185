"""The backward pass, the gate's gradients and the norm on the GPU against the
fp64 oracle's.

Bars, as max |gpu - ref| / max |ref| of a tensor: fp32 results are sums of at
most n = dk + dv + 3 * 64 products and of the chunks' carries, rounded in
fp32: n 2^-24 < 4.2e-5 of the sum of their magnitudes, so 1e-4 (the bar of
the fp32 forward kernels).  A 16-bit result is rounded once more, by half a
step: 2^-11 (fp16), 2^-8 (bf16) of the element."""
import numpy as np
import pytest

from gated_delta_rule_token_amd import workloads
from oracle import gradients
from tests.gpu_helpers import assert_close, say, to_dev
from tests.test_oracle_gradients import covered

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FP32 = 1e-4
HALF_STEP = {"float32": 0.0, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
NAMES = ("gate", "beta", "a_log", "dt_bias", "cu_seqlens", "initial_state", "gate_scale", "seq_lens")
FLAGS = ("update_rule", "gate_activation", "beta_activation", "qk_l2_norm", "scale")
INPUTS = ("q", "k", "v", "gate", "beta", "initial_state", "a_log", "dt_bias", "gate_scale")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_token_amd import api
    api.load_library()


def tol(t):
    return FP32 + HALF_STEP[str(t.dtype).split(".")[1]]


def host(t):
    return t.double().cpu().numpy()


def draw_gradients(case, final, seed=11):
    """d_o in the activations' values (NaN on tokens that no request covers,
    which nothing may read) and the final states' gradient."""
    rng = np.random.Generator(np.random.PCG64(seed))
    dtype = np.float16 if case["act_dtype"] == "f16" else np.float32
    d_o = rng.standard_normal(case["v"].shape).astype(dtype)
    if case["act_dtype"] == "bf16":
        d_o = workloads.bf16_grid(d_o)
    d_o[~covered(case)] = np.nan
    B = (len(case["cu_seqlens"]) - 1 if case["cu_seqlens"] is not None else case["q"].shape[0] if case["q"].ndim == 4
         else len(case["initial_state"]) if case["initial_state"] is not None else 1)
    HV, dv, dk = case["v"].shape[-2], case["v"].shape[-1], case["q"].shape[-1]
    d_st = rng.standard_normal((B, HV, dv, dk)).astype(np.float32) if final else None
    return d_o, d_st


def gpu_backward(case, d_o, d_st, **over):
    from gated_delta_rule_token_amd import api
    d = to_dev(case)
    act = d["q"].dtype
    kw = {name: d[name] for name in NAMES}
    kw.update({name: case[name] for name in FLAGS})
    if d_st is not None:
        kw["d_final_state"] = torch.from_numpy(d_st).cuda()
    kw.update(over)
    return api.backward(d["q"], d["k"], d["v"], torch.from_numpy(d_o).cuda().to(act), **kw)


def oracle_backward(case, d_o, d_st):
    return gradients.backward(case["q"], case["k"], case["v"], np.nan_to_num(d_o.astype(np.float64)), d_final_state=d_st,
                              **{name: case[name] for name in NAMES + FLAGS})


def check(case, final=True, what="", bars=()):
    d_o, d_st = draw_gradients(case, final)
    got, want = gpu_backward(case, d_o, d_st), oracle_backward(case, d_o, d_st)
    torch.cuda.synchronize()
    for name in INPUTS:
        if case.get(name) is not None:
            t = getattr(got, name)
            assert t is not None and tuple(t.shape) == case[name].shape, name
            assert_close(host(t), want[name], dict(bars).get(name, tol(t)), "%s d_%s" % (what, name))
        else:
            assert getattr(got, name) is None, name
    return got


RAW = dict(gate_activation="qwen", beta_activation="sigmoid", qk_l2_norm=1)

SHAPES = {
    "one_token": dict(lengths=[1], H=1, HV=1, DK=16, DV=16),
    "odd": dict(lengths=[5, 0, 1, 70], H=1, HV=3, DK=12, DV=9),
    "boundaries": dict(lengths=[63, 64, 65, 128], H=2, HV=4, DK=32, DV=32),
    "uneven_dims": dict(lengths=[90, 40], H=2, HV=2, DK=72, DV=40),
    "d128": dict(lengths=[130, 1, 66], H=2, HV=4, DK=128, DV=128),
    "wide_keys": dict(lengths=[33, 70], H=1, HV=2, DK=200, DV=24),
    "wide_values": dict(lengths=[70], H=1, HV=1, DK=24, DV=200),
    "d256": dict(lengths=[31, 32, 65], H=1, HV=2, DK=256, DV=256),
}


@pytest.mark.parametrize("rule", ["linear", "gated", "delta", "gated_delta"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward_shapes(shape, rule):
    check(workloads.random_case(21, update_rule=rule, qk_l2_norm=int(rule == "gated"), **SHAPES[shape]), what=shape)


@pytest.mark.parametrize("rule", ["linear", "gated", "delta", "gated_delta"])
@pytest.mark.parametrize("lens,H,HV,DK,DV", [([1000], 1, 1, 32, 32), ([1700, 3, 0, 900], 1, 2, 128, 80), ([450], 1, 1, 200, 30),
                                             ([2100], 1, 1, 12, 9)])
def test_backward_of_long_chains(lens, H, HV, DK, DV, rule):
    """Few heads and long requests: the chains run in segments."""
    case = workloads.random_case(40, lengths=lens, H=H, HV=HV, DK=DK, DV=DV, update_rule=rule, qk_l2_norm=1)
    if case["gate"] is not None:
        case["gate"] *= 0.02  # states that reach over several segments
    check(case, what="long")


@pytest.mark.parametrize("dtype", [np.float32, np.float16, "bf16"], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", ["odd", "d128", "wide_keys"])
def test_backward_raw_gate_types(shape, dtype):
    check(workloads.random_case(22, dtype=dtype, update_rule="gated_delta", **RAW, **SHAPES[shape]), what=shape)
    check(workloads.random_case(23, dtype=dtype, update_rule="gated", gate_activation="qwen", folded_scale=True,
                                with_initial=False, **SHAPES[shape]), final=False, what=shape + " folded")


@pytest.mark.parametrize("seq_lens", [None, [70, 0, 1, 99]], ids=["full", "seq_lens"])
def test_backward_uniform_batches(seq_lens):
    case = workloads.random_case(24, rank4_batch=(4, 70), seq_lens=seq_lens, H=2, HV=4, DK=64, DV=48,
                                 update_rule="gated_delta", **RAW)
    got = check(case, what="uniform")
    if seq_lens is not None:
        for t in (got.q, got.k, got.v, got.gate, got.beta):
            assert torch.all(t[1] == 0) and torch.all(t[2, 1:] == 0), "rows of no request"


@pytest.mark.parametrize("dtype", [np.float32, "bf16"], ids=["f32", "bf16"])
def test_backward_shared_rate(dtype):
    case = workloads.random_case(25, lengths=[70, 3], H=2, HV=6, DK=32, DV=32, dtype=dtype, update_rule="delta",
                                 beta_activation="sigmoid", qk_l2_norm=1)
    case["beta"] = np.ascontiguousarray(case["beta"][:, :1])
    check(case, what="shared rate")


def test_backward_gate_in_the_activations_type():
    case = workloads.random_case(26, lengths=[100], H=1, HV=2, DK=32, DV=32, dtype=np.float16, update_rule="gated")
    case["gate"] = case["gate"].astype(np.float16)
    case["gate_activation"] = "qwen"
    case["gate_scale"], case["dt_bias"] = np.float32([-1, -0.5]), np.float32([0, 1])
    check(case, what="f16 gate")


def test_backward_resets_and_strong_decay():
    """A decay that wipes the state (-inf, -1000) and one so weak that it is 0:
    no NaN, and a decay that lets nothing through has a gradient of exactly zero."""
    case = workloads.random_case(27, lengths=[150], H=1, HV=2, DK=32, DV=16, update_rule="gated_delta")
    case["gate"][40] = -np.inf
    case["gate"][41] = -np.inf
    case["gate"][100] = -1000.0
    case["gate"][120:] = 0.0
    with np.errstate(invalid="ignore"):
        got = check(case, what="resets")
    assert torch.all(got.gate[40:42] == 0) and torch.all(got.gate[100] == 0)


def test_backward_zero_and_one_rates_and_zero_rows():
    case = workloads.random_case(28, lengths=[96], H=1, HV=2, DK=16, DV=16, update_rule="gated_delta", qk_l2_norm=1)
    case["beta"][10:20] = 0.0
    case["beta"][20:30] = 1.0
    case["q"][5], case["k"][6], case["v"][7] = 0, 0, 0
    # a zero row's gradient goes through 1 / sqrt(1e-12): 1e6 times any other, with the same relative rounding
    check(case, what="zeros")


def test_backward_scales_with_the_incoming_gradient():
    """Gradients of 1e-20 and 1e20 times the size give results of that size,
    to the same bits: products of powers of two round alike."""
    case = workloads.random_case(29, lengths=[80], H=1, HV=2, DK=32, DV=32, update_rule="gated_delta")
    d_o, d_st = draw_gradients(case, True)
    base = gpu_backward(case, d_o, d_st)
    for e in (-60, 60):
        f = np.float32(2.0 ** e)
        got = gpu_backward(case, d_o * f, d_st * f)
        for name in ("q", "k", "v", "gate", "beta", "initial_state"):
            assert torch.equal(getattr(got, name), getattr(base, name) * float(f)), name


def test_backward_many_requests_and_an_empty_call():
    rng = np.random.Generator(np.random.PCG64(3))
    lens = rng.integers(0, 4, 600)
    check(workloads.random_case(30, lengths=lens, H=1, HV=1, DK=8, DV=8, update_rule="gated_delta"), what="600 requests")
    case = workloads.random_case(31, lengths=[0, 0], H=1, HV=2, DK=8, DV=8, update_rule="gated_delta", **RAW)
    d_o, d_st = draw_gradients(case, True)
    got = gpu_backward(case, d_o, d_st)
    assert np.array_equal(host(got.initial_state), d_st.astype(np.float64)) and torch.all(got.a_log == 0)
    assert got.q.shape == (0, 1, 8)


@pytest.mark.parametrize("dtype", [np.float32, np.float16, "bf16"], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,H,HV,DK,DV", [([3, 0, 70, 1] * 35, 1, 1, 128, 16), ([1300], 2, 8, 100, 200),
                                             ([2, 0, 1] * 400, 1, 1, 8, 8)],
                         ids=["many_chains", "many_segments", "1200_requests"])
def test_backward_in_one_launch_and_in_two(lens, H, HV, DK, DV, dtype):
    """More chains than CUs: of keys of 128 in fp16 and fp32 the two chains are
    launched one after the other, whole and in segments; else side by side."""
    case = workloads.random_case(42, lengths=lens, H=H, HV=HV, DK=DK, DV=DV, dtype=dtype, update_rule="gated_delta", qk_l2_norm=1)
    case["gate"] = case["gate"] * np.float32(0.05)
    check(case, what="launches")


@pytest.mark.parametrize("cu", [[0, 50, 20, 90], [30, 10, 60, 999], [-5, 40, 40, 70]])
def test_backward_of_any_cu_seqlens(cu):
    """Entries out of order or out of range: the running maximum, clamped; rows
    that no request covers keep what a given gradient holds."""
    from gated_delta_rule_token_amd import api
    case = workloads.random_case(32, lengths=[90], H=1, HV=2, DK=16, DV=16, update_rule="gated_delta", with_initial=False)
    case["cu_seqlens"] = np.int32(cu)
    m = np.maximum.accumulate(np.clip(cu, 0, 90))
    d_o, _ = draw_gradients(case, False)
    d_o[:m[0]] = np.nan
    d_o[m[-1]:] = np.nan
    sevens = {name: torch.full(case[name].shape, 7.0, device="cuda") for name in ("q", "k", "v", "gate", "beta")}
    got = gpu_backward(case, d_o, None, out=api.Gradients(
        **sevens, initial_state=None, a_log=None, dt_bias=None, gate_scale=None))
    want = oracle_backward(case, d_o, None)
    inside = slice(int(m[0]), int(m[-1]))
    for name, t in sevens.items():
        assert getattr(got, name) is t
        assert_close(host(t)[inside], want[name][inside], FP32, "cu d_%s" % name)
        assert torch.all(t[:m[0]] == 7) and torch.all(t[m[-1]:] == 7), name


def test_backward_against_differences_of_the_forward_pass():
    """<gradient, step> against the fp64 forward pass at x +- 1e-4 step: the
    difference is off by 1e-8 / 6 of the third derivative, the GPU's gradient
    by FP32 of its norm."""
    from tests.test_oracle_gradients import _forward
    case = workloads.random_case(33, lengths=[70, 20], H=1, HV=2, DK=16, DV=16, update_rule="gated_delta", **RAW)
    d_o, d_st = draw_gradients(case, True)
    got = gpu_backward(case, d_o, d_st)
    rng = np.random.Generator(np.random.PCG64(5))

    def loss(name, x):
        o, st = _forward(case, **{name: x})
        return (o * d_o).sum() + (st * d_st).sum()

    for name in INPUTS:
        if case.get(name) is None:
            continue
        x, grad = np.asarray(case[name], np.float64), host(getattr(got, name))
        step = rng.standard_normal(x.shape)
        diff = (loss(name, x + 1e-4 * step) - loss(name, x - 1e-4 * step)) / 2e-4
        bound = FP32 * np.linalg.norm(grad) * np.linalg.norm(step)
        say("  d_%s: %.6g against %.6g (bound %.2g)" % (name, (grad * step).sum(), diff, bound))
        assert abs((grad * step).sum() - diff) <= bound, name


def _training_case():
    return workloads.random_case(34, lengths=[100, 0, 77], H=2, HV=4, DK=64, DV=64, dtype="bf16",
                                 update_rule="gated_delta", **RAW)


def test_backward_gives_equal_bits_on_another_stream():
    case = _training_case()
    d_o, d_st = draw_gradients(case, True)
    first = gpu_backward(case, d_o, d_st)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = gpu_backward(case, d_o, d_st)
    side.synchronize()
    for name in INPUTS:
        assert torch.equal(getattr(first, name), getattr(second, name)) if getattr(first, name) is not None else True, name


def test_backward_replays_in_a_graph():
    from gated_delta_rule_token_amd import api
    case = _training_case()
    d_o, d_st = draw_gradients(case, True)
    d = to_dev(case)
    kw = {name: d[name] for name in NAMES}
    kw.update({name: case[name] for name in FLAGS})
    d_o, d_st = torch.from_numpy(d_o).cuda().bfloat16(), torch.from_numpy(d_st).cuda()
    eager = api.backward(d["q"], d["k"], d["v"], d_o, d_final_state=d_st, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = api.backward(d["q"], d["k"], d["v"], d_o, d_final_state=d_st, **kw)
    for replay in range(4):
        if replay == 2:
            d_o.mul_(2.0)  # new values in the captured buffer
            d_st.mul_(2.0)
            eager = api.backward(d["q"], d["k"], d["v"], d_o, d_final_state=d_st, **kw)
        graph.replay()
        torch.cuda.synchronize()
        junk = torch.randn(1 << 20, device="cuda").sum()  # eager work between replays
        torch.cuda.synchronize()
        for name in INPUTS:
            if getattr(eager, name) is not None:
                assert torch.equal(getattr(captured, name), getattr(eager, name)), (replay, name)
    assert torch.isfinite(junk)


def test_backward_updates_the_state_gradient_in_place():
    """d_initial_state may be d_final_state's buffer: a chain of segments hands
    one buffer from call to call."""
    from gated_delta_rule_token_amd import api
    case = workloads.random_case(35, lengths=[70], H=1, HV=2, DK=32, DV=32, update_rule="gated_delta")
    d_o, d_st = draw_gradients(case, True)
    want = gpu_backward(case, d_o, d_st)
    buf = torch.from_numpy(d_st).cuda()
    none = dict.fromkeys(("q", "k", "v", "gate", "beta", "a_log", "dt_bias", "gate_scale"))
    got = gpu_backward(case, d_o, None, d_final_state=buf, out=api.Gradients(initial_state=buf, **none))
    assert got.initial_state is buf and torch.equal(buf, want.initial_state)


@pytest.fixture
def poisoned(monkeypatch):
    """Every tensor that the binding allocates starts as NaN (workspaces, too)."""
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: (lambda t: (t.view(-1).view(torch.uint8).fill_(255), t)[1]
                                                          if t.is_cuda and t.numel() else t)(real(*a, **kw)))


@pytest.mark.parametrize("rule,dtype,DK,DV", [("gated_delta", "bf16", 16, 16), ("gated_delta", np.float32, 12, 9),
                                              ("delta", np.float16, 5, 3), ("linear", np.float32, 130, 8)])
@pytest.mark.parametrize("cu", [[0, 90], [30, 10, 60, 70], [90, 90], [0, 0], [0], [95], [0, 1]])
def test_backward_zeroes_rows_of_no_request(poisoned, rule, dtype, DK, DV, cu):
    case = workloads.random_case(37, lengths=[90], H=1, HV=3, DK=DK, DV=DV, dtype=dtype, update_rule=rule, with_initial=False)
    case["cu_seqlens"] = np.int32(cu)
    if rule == "delta":
        case["beta"] = np.ascontiguousarray(case["beta"][:, :1])
    m = np.maximum.accumulate(np.clip(cu, 0, 90))
    d_o, _ = draw_gradients(dict(case, cu_seqlens=np.int32([0, 90])), False)
    d_o[:m[0]] = np.nan
    d_o[m[-1]:] = np.nan
    got = gpu_backward(case, d_o, None)
    want = oracle_backward(case, d_o, None) if len(cu) > 1 else None
    for name in ("q", "k", "v", "gate", "beta"):
        t = getattr(got, name)
        if t is not None:
            assert torch.all(t[:m[0]] == 0) and torch.all(t[m[-1]:] == 0), name
            if m[-1] > m[0]:
                assert_close(host(t)[m[0]:m[-1]], want[name][m[0]:m[-1]], tol(t), "rest d_%s" % name)


@pytest.mark.parametrize("seq_lens", [[70, 70, 70], [0, 0, 0], [1, 70, 33], [80, -3, 69]])
def test_backward_zeroes_the_padding(poisoned, seq_lens):
    case = workloads.random_case(38, rank4_batch=(3, 70), seq_lens=[70, 70, 70], H=1, HV=2, DK=16, DV=24, update_rule="gated_delta")
    case["seq_lens"] = np.int32(seq_lens)
    d_o, d_st = draw_gradients(dict(case, seq_lens=np.clip(seq_lens, 0, 70).astype(np.int32)), True)
    got = gpu_backward(case, d_o, d_st)
    case["seq_lens"] = np.clip(seq_lens, 0, 70).astype(np.int32)
    want = oracle_backward(case, d_o, d_st)
    for name in ("q", "k", "v", "gate", "beta"):
        t = getattr(got, name)
        assert_close(host(t), want[name], FP32, "padded d_%s" % name)
        for b, n in enumerate(case["seq_lens"]):
            assert torch.all(t[b, n:] == 0), name


def test_backward_in_segments_in_place_twice_at_once_and_replayed(poisoned):
    """A chain cut into segments: d_final_state's buffer taken for
    d_initial_state, two calls at once on two streams, and a captured call."""
    from gated_delta_rule_token_amd import api
    case = workloads.random_case(39, lengths=[3000, 0, 700], H=1, HV=2, DK=64, DV=64, dtype="bf16", update_rule="gated_delta", **RAW)
    d_o, d_st = draw_gradients(case, True)
    d = to_dev(case)
    kw = {name: d[name] for name in NAMES}
    kw.update({name: case[name] for name in FLAGS})
    d_o, d_st = torch.from_numpy(d_o).cuda().bfloat16(), torch.from_numpy(d_st).cuda()
    call = lambda **over: api.backward(d["q"], d["k"], d["v"], d_o, **{**dict(kw, d_final_state=d_st), **over})  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    same = lambda got: all(torch.equal(getattr(got, n), getattr(want, n)) for n in INPUTS  # noqa: E731
                           if getattr(want, n) is not None)
    buf = d_st.clone()
    none = dict.fromkeys(("q", "k", "v", "gate", "beta", "a_log", "dt_bias", "gate_scale"))
    assert same(call(d_final_state=buf, out=api.Gradients(initial_state=buf, **none)))
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    results = []
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            results += [call(), call()]
    for s in side:
        s.synchronize()
    assert all(map(same, results))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = call()
    for replay in range(3):
        for name in INPUTS:
            if getattr(captured, name) is not None:
                getattr(captured, name).zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(captured), replay
        assert same(call()), replay


def test_backward_refuses_wrong_tensors():
    from gated_delta_rule_token_amd import api
    case = workloads.random_case(36, lengths=[8], H=1, HV=2, DK=16, DV=16, update_rule="gated_delta")
    d_o, d_st = draw_gradients(case, True)
    good = torch.from_numpy(d_st).cuda()
    for over in (dict(d_final_state=good[:, :1]), dict(d_final_state=good.double()),
                 dict(d_final_state=good.transpose(2, 3)), dict(gate=None), dict(beta=torch.zeros(8, 3, device="cuda")),
                 dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")),
                 dict(update_rule="gated_delta_v2"), dict(initial_state=good.cpu())):
        with pytest.raises(api.GDRError):
            gpu_backward(case, d_o, d_st if "d_final_state" not in over else None, **over)


# ------------------------------------------------------------------ gate
@pytest.mark.parametrize("rows,heads", [(1, 1), (7, 3), (256, 32), (333, 40), (5, 2056), (3000, 8), (0, 4)])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_gate_backward(rows, heads, dtype):
    from gated_delta_rule_token_amd import api
    rng = np.random.Generator(np.random.PCG64(rows * 100 + heads))
    dt = getattr(torch, dtype)
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32) * 3).cuda()  # noqa: E731
    a, d, b, e = (draw(rows, heads).to(dt) for _ in range(4))
    bias, scale = draw(heads), -draw(heads).abs()
    got = api.gate_backward(a, bias, scale, d, b=b, d_beta=e)
    want = gradients.gate_backward(*(host(x) for x in (a, bias, scale, d, b, e)))
    for g, w, name in zip((got.a, got.b, got.dt_bias, got.decay_scale), want, ("a", "b", "dt_bias", "decay_scale")):
        if rows or name in ("dt_bias", "decay_scale"):
            # elementwise: the largest element's half step and 8 fp32 roundings; sums: 1e-5 of the largest
            assert_close(host(g), w, HALF_STEP[str(g.dtype).split(".")[1]] + 1e-5, "gate d_%s" % name)
    alone = api.gate_backward(a, bias, scale, d)
    assert alone.b is None and torch.equal(alone.a, got.a) and torch.equal(alone.dt_bias, got.dt_bias)


def test_gate_backward_far_arguments():
    from gated_delta_rule_token_amd import api
    a = torch.tensor([[-200.0, 200.0, 0.0, -20.0]], device="cuda")
    one = torch.ones(4, device="cuda")
    g = api.gate_backward(a, 0 * one, one, torch.ones_like(a), b=a, d_beta=torch.ones_like(a))
    want = gradients.gate_backward(*(host(x) for x in (a, 0 * one, one, torch.ones_like(a), a, torch.ones_like(a))))
    for got, w in zip((g.a, g.b, g.dt_bias, g.decay_scale), want):
        assert np.allclose(host(got), w, rtol=1e-5, atol=1e-38)


# ------------------------------------------------------------------ norm
WIDTHS = [1, 7, 8, 64, 100, 128, 129, 250, 512, 1001, 2048, 4096, 4100, 8200, 32768]


def _norm_inputs(rows, width, dtype, seed=0):
    rng = np.random.Generator(np.random.PCG64(width * 10 + seed))
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(dtype)  # noqa: E731
    return draw(rows, width), draw(rows, width), draw(width), draw(rows, width), draw(rows, width)


def check_dx(got, want, terms, what):
    """d_x = inv t - h mean(t h) inv: at a width of 1, h^2 = 1 - eps inv^2 and
    the two terms cancel but for 1e-6 of them.  Each is a product of four
    fp32 roundings (h twice, the mean, the product) of size |inv t|, so their
    difference is off by up to 8 * 2^-24 of max |inv t| whatever remains."""
    err = np.abs(host(got) - want).max()
    bound = (HALF_STEP[str(got.dtype).split(".")[1]] + FP32) * np.abs(want).max() + 2.0 ** -21 * np.abs(terms).max()
    say("  %-48s max err %.3e (bound %.1e)" % (what, err, bound))
    assert err <= bound, what


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_norm_and_its_gradients(width, dtype):
    from gated_delta_rule_token_amd import api
    dt = getattr(torch, dtype)
    for rows, wdt in ((1, torch.float32), (37, dt)):
        x, res, w, dy, dres = _norm_inputs(rows, width, dt)
        w = w.to(wdt)
        got = api.rms_norm(x, w, residual=res, want_inv_rms=True)
        r = (x.float() + res.float()).to(dt)
        assert torch.equal(got.residual, r) and got.scale is None
        y, inv = gradients.rms_norm(host(r), host(w))
        # a sum of `width` squares, one root, two products: far below 1e-5
        assert_close(host(got.inv_rms), inv, 1e-5, "inv_rms")
        assert_close(host(got.y), y, HALF_STEP[dtype] + 1e-5, "norm y %d" % width)
        back = api.rms_norm_backward(dy, got.residual, w, got.inv_rms, d_residual=dres)
        dx, dw = gradients.rms_norm_backward(host(dy), host(r), host(w), host(dres))
        check_dx(back.x, dx, host(dy) * host(w) * inv[:, None], "norm d_x %d" % width)
        assert back.weight.dtype == torch.float32
        assert_close(host(back.weight), dw, FP32, "norm d_weight %d" % width)
        plain = api.rms_norm_backward(dy, got.residual, None, got.inv_rms)
        assert plain.weight is None
        check_dx(plain.x, gradients.rms_norm_backward(host(dy), host(r))[0], host(dy) * inv[:, None],
                 "norm d_x, no weight %d" % width)


@pytest.mark.parametrize("rows", [2, 5000])
def test_norm_rows_and_views(rows):
    from gated_delta_rule_token_amd import api
    x, _, w, dy, _ = _norm_inputs(rows, 256, torch.bfloat16)
    got = api.rms_norm(x.view(rows, 2, 128), w[:128].contiguous(), want_inv_rms=True)
    y, inv = gradients.rms_norm(host(x).reshape(rows, 2, 128), host(w[:128]))
    assert got.y.shape == (rows, 2, 128) and got.inv_rms.shape == (rows, 2)
    assert_close(host(got.y), y, 2.0 ** -8 + 1e-5, "per head")
    back = api.rms_norm_backward(dy.view(rows, 2, 128), x.view(rows, 2, 128), w[:128].contiguous(), got.inv_rms)
    dx, dw = gradients.rms_norm_backward(host(dy).reshape(rows, 2, 128), host(x).reshape(rows, 2, 128), host(w[:128]))
    assert_close(host(back.x), dx, 2.0 ** -8 + FP32, "per head d_x")
    assert_close(host(back.weight), dw, FP32, "per head d_weight")


@pytest.mark.parametrize("width,group", [(1, 0), (64, 0), (64, 8), (100, 32), (128, 512), (130, 64), (1001, 128),
                                         (2048, 0), (4096, 128), (8200, 512), (32768, 256)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_norm_in_8_bits(width, group, dtype):
    """Each value is one of the two e4m3 neighbours of y / scale, the nearer
    one but for the fp32 rounding of y and of the quotient (1e-5 of it)."""
    from gated_delta_rule_token_amd import api
    x, res, w, _, _ = _norm_inputs(9, width, getattr(torch, dtype), seed=group)
    x[3] = 0
    res[3] = 0  # a row of zeros
    got = api.rms_norm(x, w, residual=res, out_dtype=torch.float8_e4m3fn, group=group)
    r = (x.float() + res.float()).to(x.dtype)
    assert torch.equal(got.residual, r)
    y, _ = gradients.rms_norm(host(r), host(w))
    g = group if group else width
    n = -(-width // g)
    assert got.scale.shape == (9, n)
    yp = np.zeros((9, n * g))
    yp[:, :width] = y
    amax = np.abs(yp.reshape(9, n, g)).max(-1)
    want = np.where(amax > 0, amax / 448, 1)
    assert np.allclose(host(got.scale), want, rtol=1e-5)
    assert torch.all(got.scale[3] == 1) and torch.all(got.y[3].float() == 0)
    t = y / np.repeat(host(got.scale), g, 1)[:, :width]
    table = gradients.e4m3_values()
    table = np.unique(table[np.isfinite(table)])
    codes = host(got.y.float())
    assert np.all(np.isin(codes, table))
    at = np.clip(np.searchsorted(table, t), 1, len(table) - 1)
    nearest = np.minimum(np.abs(t - table[at]), np.abs(t - table[at - 1]))
    assert np.all(np.abs(codes - t) <= nearest + 2e-5 * np.abs(t) + 1e-12)


def test_norm_of_infinities_nan_and_extremes():
    from gated_delta_rule_token_amd import api
    x = torch.randn(6, 64, device="cuda")
    x[0, 3], x[1, 5] = float("nan"), float("inf")
    x[2] = 1e-30
    x[3] = 1e18
    got = api.rms_norm(x)
    r = x.double()
    want = r / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-6)
    assert torch.isnan(got.y[0]).all() and torch.isnan(got.y[1, 5]) and torch.all(got.y[1, :5] == 0)
    assert torch.allclose(got.y[2:].double(), want[2:], rtol=1e-5)
    eight = api.rms_norm(x, out_dtype=torch.float8_e4m3fn)
    assert torch.isnan(eight.y[0].float()).all() and torch.isnan(eight.scale[0, 0])
    assert torch.isfinite(eight.y[2:].float()).all() and torch.isfinite(eight.scale[2:]).all()


@pytest.mark.parametrize("size", [1e-30, 1e-37, 1e-38, 1e-41, 1e-45])
@pytest.mark.parametrize("group", [0, 32])
def test_norm_in_8_bits_of_tiny_rows(size, group):
    """Scales down to denormal ones, whose reciprocal is infinite: zeros stay
    zero, and y8 is e4m3(y / scale) of the fp32 y and scale."""
    from gated_delta_rule_token_amd import api
    rng = np.random.Generator(np.random.PCG64(7))
    x = torch.from_numpy((rng.standard_normal((5, 200)) * size).astype(np.float32)).cuda()
    x[:, ::7] = 0.0
    y = api.rms_norm(x, eps=1.0).y  # inv = 1: y = x
    got = api.rms_norm(x, eps=1.0, out_dtype=torch.float8_e4m3fn, group=group)
    assert torch.equal(y, x)
    for c in range(0, 200, group or 200):
        part = slice(c, c + (group or 200))
        top = y[:, part].double().abs().amax(1, keepdim=True)
        scale = got.scale[:, c // (group or 200)][:, None].double()
        # m / 448 in fp32, by half a step of a normal or a denormal value, and 1 where that is 0
        assert torch.all(((scale - top / 448).abs() <= 2.0 ** -23 * top / 448 + 2.0 ** -149) | (scale == 1))
        q, want = got.y[:, part].double(), (y[:, part].double() / scale).clamp(-448, 448)
        assert torch.all(q[want == 0] == 0)
        # half a step of e4m3 (2^-4 of the value, 2^-10 below its normal range), and the product's roundings
        assert torch.all((q - want).abs() <= (2.0 ** -4 + 2.0 ** -20) * want.abs() + 2.0 ** -10 + 2.0 ** -30)


def test_norm_in_place_residual_empty_rows_and_refusals():
    from gated_delta_rule_token_amd import api
    x, res, w, _, _ = _norm_inputs(33, 200, torch.float16)
    want = api.rms_norm(x, w, residual=res)
    kept = res.clone()
    got = api.rms_norm(x, w, residual=kept, residual_out=kept)
    assert got.residual is kept and torch.equal(kept, want.residual) and torch.equal(got.y, want.y)
    empty = api.rms_norm(x[:0], w, residual=res[:0], out_dtype=torch.float8_e4m3fn)
    assert empty.y.shape == (0, 200) and empty.scale.shape == (0, 1)
    back = api.rms_norm_backward(x[:0], x[:0], w, torch.zeros(0, device="cuda"))
    assert back.x.shape == (0, 200) and torch.all(back.weight == 0)
    inv = torch.ones(33, device="cuda")
    for call in (lambda: api.rms_norm(x[:, :100], w[:100]), lambda: api.rms_norm(x, w[:100]),
                 lambda: api.rms_norm(x, w.double()), lambda: api.rms_norm(x, residual=res.float()),
                 lambda: api.rms_norm(x, residual_out=res), lambda: api.rms_norm(x, out_dtype=torch.int8),
                 lambda: api.rms_norm(x, group=64), lambda: api.rms_norm(x.double()),
                 lambda: api.rms_norm(x, out_dtype=torch.float8_e4m3fn, group=48),
                 lambda: api.rms_norm_backward(x, x, w, inv[:5]), lambda: api.rms_norm_backward(x, res[:1], w, inv)):
        with pytest.raises(api.GDRError):
            call()


def test_norm_replays_in_a_graph_and_gives_equal_bits():
    from gated_delta_rule_token_amd import api
    x, res, w, dy, dres = _norm_inputs(500, 384, torch.bfloat16)

    def step():
        y = api.rms_norm(x, w, residual=res, want_inv_rms=True)
        q = api.rms_norm(x, w, residual=res, out_dtype=torch.float8_e4m3fn, group=64)
        return y, q, api.rms_norm_backward(dy, y.residual, w, y.inv_rms, d_residual=dres)

    eager = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for replay in range(3):
        if replay == 1:
            x.mul_(-1.5)
            eager = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            for s, t in zip(a, b):
                if s is not None:
                    assert torch.equal(s.view(torch.uint8), t.view(torch.uint8)), replay


@pytest.mark.parametrize("rows,heads", [(256, 32), (1024, 8), (1025, 8), (1, 4096), (7, 1176)])
def test_gate_backward_in_one_slice_and_in_several(rows, heads):
    """Up to 8192 elements the sums need no second launch: the same results on
    both sides of that size, into memory that starts as NaN, on replays too."""
    from gated_delta_rule_token_amd import api
    rng = np.random.Generator(np.random.PCG64(rows + heads))
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    a, d, bias, scale = draw(rows, heads), draw(rows, heads), draw(heads), draw(heads)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    got = api.gate_backward(a, bias, scale, d, workspace=ws)
    x = a.double() + bias.double()
    d_a = d.double() * scale.double() * torch.sigmoid(x)
    sums = d_a.sum(0), (d.double() * torch.nn.functional.softplus(x)).sum(0)
    terms = d_a.abs().sum(0), (d.double() * torch.nn.functional.softplus(x)).abs().sum(0)
    for g, want, size in zip((got.dt_bias, got.decay_scale), sums, terms):
        # each term is good to 16 half steps (sigmoid, softplus and two products), and
        # a term is added at most 40 times on its way through a thread, a workgroup and the slices
        assert torch.all((g.double() - want).abs() <= 56 * 2.0 ** -24 * size)
    assert torch.all((got.a.double() - d_a).abs() <= 16 * 2.0 ** -24 * d_a.abs())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = api.gate_backward(a, bias, scale, d, workspace=ws)
    for _ in range(3):
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(captured, got) if s is not None)


# ------------------------------------------------------------------ as they are used together
def test_a_layer_forward_and_back():
    """norm -> projections -> gate -> recurrence -> norm per head -> projection,
    in fp32, and all the way back, against autograd of the same layer in fp64
    on the host (whose recurrence runs token by token)."""
    from gated_delta_rule_token_amd import api
    gen = torch.Generator().manual_seed(0)
    draw = lambda *s, std=1.0: (torch.randn(s, generator=gen) * std)  # noqa: E731
    lens, width, H, HV, d = [70, 0, 9], 48, 2, 4, 16
    T = sum(lens)
    params = {"x": draw(T, width), "res": draw(T, width), "w1": 1 + draw(width, std=0.1),
              "wq": draw(width, H * d, std=0.2), "wk": draw(width, H * d, std=0.2), "wv": draw(width, HV * d, std=0.2),
              "wa": draw(width, HV, std=0.2), "wb": draw(width, HV, std=0.2), "dt_bias": draw(HV),
              "scale": -draw(HV).exp(), "w2": 1 + draw(d, std=0.1), "wo": draw(HV * d, width, std=0.2)}
    d_out, d_res = draw(T, width), draw(T, width)

    # fp64, autograd
    p = {name: t.double().requires_grad_() for name, t in params.items()}
    rms = lambda x, w: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
    r = p["x"] + p["res"]
    n = rms(r, p["w1"])
    q, k, v = ((n @ p[w]).view(T, -1, d) for w in ("wq", "wk", "wv"))
    unit = lambda x: x / torch.sqrt(x.square().sum(-1, keepdim=True) + 1e-12)  # noqa: E731
    q, k = (unit(x).repeat_interleave(HV // H, 1) for x in (q, k))
    g = p["scale"] * torch.nn.functional.softplus(n @ p["wa"] + p["dt_bias"])
    b = torch.sigmoid(n @ p["wb"])
    o, at = [], 0
    for length in lens:
        S = torch.zeros(HV, d, d, dtype=torch.float64)
        for t in range(at, at + length):
            S = S * g[t].exp()[:, None, None]
            miss = v[t] - (S @ k[t][:, :, None])[..., 0]
            S = S + (b[t][:, None] * miss)[:, :, None] * k[t][:, None]
            o.append((S @ q[t][:, :, None])[..., 0] / d ** 0.5)
        at += length
    out = rms(torch.stack(o), p["w2"]).reshape(T, HV * d) @ p["wo"]
    ((out * d_out.double()).sum() + (r * d_res.double()).sum()).backward()

    # the framework's calls, projections by torch
    c = {name: t.cuda() for name, t in params.items()}
    n1 = api.rms_norm(c["x"], c["w1"], residual=c["res"], want_inv_rms=True)
    h = n1.y
    q, k, v = ((h @ c[w]).view(T, -1, d) for w in ("wq", "wk", "wv"))
    a, raw = h @ c["wa"], h @ c["wb"]
    decay, beta = api.gate(a, c["dt_bias"], c["scale"], b=raw, want_beta=True)
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    kw = dict(gate=decay, beta=beta, cu_seqlens=cu, qk_l2_norm=True)
    o, _ = api.forward(q, k, v, **kw)
    n2 = api.rms_norm(o, c["w2"], want_inv_rms=True)
    y = n2.y.view(T, HV * d) @ c["wo"]
    assert_close(host(y), out.detach().numpy(), FP32, "layer output")

    grads = {}
    dy = d_out.cuda()
    grads["wo"] = n2.y.view(T, HV * d).T @ dy
    b2 = api.rms_norm_backward((dy @ c["wo"].T).view(T, HV, d), o, c["w2"], n2.inv_rms)
    grads["w2"] = b2.weight
    br = api.backward(q, k, v, b2.x, **kw)
    bg = api.gate_backward(a, c["dt_bias"], c["scale"], br.gate, b=raw, d_beta=br.beta)
    grads["dt_bias"], grads["scale"] = bg.dt_bias, bg.decay_scale
    dh = torch.zeros_like(h)
    for w, dx in (("wq", br.q), ("wk", br.k), ("wv", br.v), ("wa", bg.a), ("wb", bg.b)):
        dx = dx.reshape(T, -1)
        grads[w] = h.T @ dx
        dh += dx @ c[w].T
    b1 = api.rms_norm_backward(dh, n1.residual, c["w1"], n1.inv_rms, d_residual=d_res.cuda())
    grads["w1"], grads["x"], grads["res"] = b1.weight, b1.x, b1.x
    for name, t in p.items():
        # two norms, the recurrence and up to four library products one after the other
        assert_close(host(grads[name]), t.grad.numpy(), 4 * FP32, "layer d_%s" % name)
