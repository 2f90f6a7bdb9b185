"""The state cache in 16 and 8 bits: writing, reading and steps on it, against
the formats' definitions and the fp64 oracle, on an MI355X.

Tolerances.  Writing and reading are exact: the codes are those of one rounding
to nearest even.  A step's new state differs from the 64-bit one by fp32
arithmetic before it is rounded: with dk <= 256 and rows of largest magnitude
m, a dot product with a unit key is off by at most dk 2^-24 sqrt(dk) m, 2.5e-4 m,
which enters the new row through a key's component (at most 1) and the update
rate (at most 1).  So a value may differ by half a step of its type and 2.5e-4 of
the larger of the row's old and new largest magnitude and |v|, and an output by
3e-4 of the same with the output's own rounding.
"""
import numpy as np
import pytest

import oracle
from gated_delta_rule_token_amd import workloads

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_token_amd import api
    api.load_library()


DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def write(states, dtype):
    """(data, scale bytes) of fp32 states, by the definition, on the CPU."""
    states = torch.as_tensor(states).float().cpu()
    if dtype != "e4m3":
        return states.to(DT[dtype]), None
    top = states.abs()
    top = torch.where(top.isnan(), torch.zeros_like(top), top).amax(-1).numpy()
    # the least e with top <= 448 2^e
    m, e = np.frexp(top)
    e = np.where(m > 0.875, e - 8, e - 9)
    e = np.where(np.isinf(top), 120, e)
    e = np.where(top == 0, -100, np.clip(e, -100, 120))
    codes = (states.double() * torch.from_numpy(2.0 ** -e.astype(np.float64))[..., None]).float().to(DT[dtype])
    return codes, torch.from_numpy((e + 127).astype(np.uint8))


def read(data, scale):
    """What a cache stands for, in 64 bits."""
    x = data.cpu().float().double()
    return x if scale is None else x * torch.exp2(scale.cpu().view(torch.uint8).double() - 127)[..., None]


def slab_of(states, dtype):
    """A GPU slab holding (num_slots, HV, dv, dk) states."""
    from gated_delta_rule_token_amd import api
    data, scale = write(states, dtype)
    return api.PackedSlab(data.cuda(), None if scale is None else scale.view(torch.float8_e8m0fnu).cuda())


def bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t.view(torch.int16)


def same(a, b):
    return torch.equal(bits(a.data), bits(b.data)) and (a.scale is None or torch.equal(bits(a.scale), bits(b.scale)))


def clone(s):
    from gated_delta_rule_token_amd import api
    return api.PackedSlab(s.data.clone(), None if s.scale is None else s.scale.clone())


def ids(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ writing and reading

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("HV,dv,dk", [(1, 1, 1), (2, 128, 128), (3, 40, 72), (2, 33, 9), (1, 256, 256), (5, 7, 130), (4, 64, 64),
                                      (1, 31, 255), (2, 130, 30), (3, 65, 33), (1, 128, 3), (2, 129, 5), (1, 3, 4)])
def test_pack_and_unpack(dtype, HV, dv, dk):
    from gated_delta_rule_token_amd import api
    g = torch.Generator().manual_seed(HV * dv + dk)
    states = torch.randn(3, HV, dv, dk, generator=g) * torch.exp(3 * torch.randn(3, HV, dv, 1, generator=g))
    states[1, 0, 0] = 0
    slab = slab_of(torch.randn(7, HV, dv, dk, generator=g), dtype)
    before = clone(slab)
    where = [5, 0, 3]
    api.state_pack(states.cuda(), slab, ids(*where))
    data, scale = write(states, dtype)
    assert torch.equal(bits(slab.data[where].cpu()), bits(data))
    if scale is not None:
        assert torch.equal(slab.scale.cpu().view(torch.uint8)[where], scale)
    rest = [1, 2, 4, 6]
    assert torch.equal(bits(slab.data[rest]), bits(before.data[rest]))
    out = api.state_unpack(slab, ids(*where))
    assert out.dtype == torch.float32 and torch.equal(out.double().cpu(), read(data, scale))
    # what was read, written again, reads the same
    api.state_pack(out, slab, ids(6, 1, 2))
    assert torch.equal(api.state_unpack(slab, ids(6, 1, 2)), out)


def test_every_code_and_every_scale():
    from gated_delta_rule_token_amd import api
    codes = torch.arange(256, dtype=torch.uint8).view(1, 1, 1, 256).expand(1, 1, 255, 256).contiguous().view(torch.float8_e4m3fn)
    scale = torch.arange(255, dtype=torch.uint8).view(1, 1, 255)
    out = api.state_unpack(api.PackedSlab(codes.cuda(), scale.view(torch.float8_e8m0fnu).cuda()), ids(0)).cpu()
    want = read(codes, scale).float()  # the product rounded to fp32 (denormals and overflow at the ends)
    normal = (want.abs() >= 2.0 ** -126) | (want == 0)
    assert torch.equal(out.isnan(), want.isnan())
    use = normal & ~want.isnan()
    assert torch.equal(out[use], want[use])
    tiny = ~normal & ~want.isnan()
    assert bool(((out[tiny] == want[tiny]) | (out[tiny] == 0)).all())


def test_borders_of_scales_and_halves():
    """Largest values around 448 2^e, values on the middle of two codes."""
    from gated_delta_rule_token_amd import api
    rows = []
    for e in (-100, -99, -20, 0, 7, 119):
        for top in (448.0, np.nextafter(np.float32(448), np.float32(449)), np.nextafter(np.float32(448), np.float32(0)), 224.5, 1.0):
            x = np.zeros(64, np.float32)
            x[0] = np.float32(top) * np.float32(2.0) ** e
            halves = np.array([17.0, 19.0, 1.0625, 0.0009765625, 0.0029296875, -18.0, -20.0], np.float32)
            x[1:8] = halves * np.float32(2.0) ** e
            rows.append(x)
    states = torch.from_numpy(np.stack(rows)).view(1, 1, len(rows), 64)
    for dtype in DT:
        slab = api.packed_slab(1, 1, len(rows), 64, DT[dtype])
        api.state_pack(states.cuda(), slab, ids(0))
        data, scale = write(states, dtype)
        assert torch.equal(bits(slab.data.cpu()), bits(data))
        assert scale is None or torch.equal(slab.scale.cpu().view(torch.uint8), scale)


def test_tiny_huge_and_non_finite_rows():
    from gated_delta_rule_token_amd import api
    x = torch.ones(1, 1, 6, 128)
    x[0, 0, 0] *= 2.0 ** -140
    x[0, 0, 1, 3] = 3.4e38
    x[0, 0, 2, 5], x[0, 0, 2, 6] = float("nan"), 2.0
    x[0, 0, 3, 7] = float("-inf")
    x[0, 0, 4] = float("nan")
    x[0, 0, 5] = -0.0
    for dtype in DT:
        slab = api.packed_slab(2, 1, 6, 128, DT[dtype])
        api.state_pack(x.cuda(), slab, ids(1))
        got = api.state_unpack(slab, ids(1)).cpu()[0, 0]
        assert bool((got[0].abs() <= 2.0 ** -139).all())
        assert bool(got[4].isnan().all()) and bool((got[5] == 0).all())
        assert int(got[2].isnan().sum()) == 1 and float(got[2, 6]) == 2.0 and float(got[2, 0]) == 1.0
        other = torch.arange(128) != 7
        if dtype == "e4m3":
            # 3.4e38 / 2^120 is 255.79; the nearest codes are 240 and 256, and 256 * 2^120 = 2^128 is
            # fp32's infinity: no code in between, whatever the row's power of two
            assert float(got[1, 3]) == float("inf") and float(slab.data[1, 0, 1, 3]) == 256.0
            assert bool(got[3, 7].isnan()) and bool(got[3, other].isfinite().all())
        else:
            assert float(got[3, 7]) == float("-inf") and bool((got[3, other] == 1).all())


@pytest.mark.parametrize("dtype", DT)
def test_slot_ids_out_of_range_and_unused_slots(dtype):
    from gated_delta_rule_token_amd import api
    slab = slab_of(torch.randn(4, 2, 8, 64, generator=torch.Generator().manual_seed(1)), dtype)
    before = clone(slab)
    bad = ids(-1, 4, 2 ** 31 - 1, -2 ** 31)
    api.state_pack(torch.ones(4, 2, 8, 64, device="cuda"), slab, bad)
    assert same(slab, before)
    out = torch.full((4, 2, 8, 64), 5.0, device="cuda")
    assert api.state_unpack(slab, bad, out=out) is out and bool((out == 0).all())
    api.state_pack(torch.empty(0, 2, 8, 64, device="cuda"), slab, ids())
    assert same(slab, before) and api.state_unpack(slab, ids()).shape == (0, 2, 8, 64)


# ------------------------------------------------------------------ steps

def gpu_tensors(case):
    from tests.gpu_helpers import to_dev
    d = to_dev(case)
    return d, dict(gate=d["gate"], beta=d["beta"], erase=d["erase"], a_log=d["a_log"], dt_bias=d["dt_bias"],
                   gate_scale=d["gate_scale"], cu_seqlens=d["cu_seqlens"], seq_lens=d["seq_lens"],
                   slot_ids=d["slot_ids"], update_rule=case["update_rule"], gate_activation=case["gate_activation"],
                   beta_activation=case["beta_activation"], qk_l2_norm=case["qk_l2_norm"], scale=case["scale"])


def oracle_step(case, states):
    return oracle.forward(case["q"], case["k"], case["v"], gate=case["gate"], beta=case["beta"], erase=case["erase"],
                          a_log=case["a_log"], dt_bias=case["dt_bias"], cu_seqlens=case["cu_seqlens"],
                          slot_ids=case["slot_ids"], slab=states, update_rule=case["update_rule"],
                          gate_activation=case["gate_activation"], beta_activation=case["beta_activation"],
                          qk_l2_norm=case["qk_l2_norm"], scale=case["scale"], gate_scale=case.get("gate_scale"),
                          seq_lens=case.get("seq_lens"))


HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
LEAST = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "e4m3": 2.0 ** -10}  # half a denormal step (e4m3: of the row's scale)


def step_and_check(case, dtype, tokens=1, **kw):
    from gated_delta_rule_token_amd import api
    d, args = gpu_tensors(case)
    start = case["slab"]
    slab = slab_of(start, dtype)
    before, states = clone(slab), read(slab.data, slab.scale).numpy()
    o = api.forward_packed(d["q"], d["k"], d["v"], slab=slab, **args, **kw)
    torch.cuda.synchronize()
    ro, rs = oracle_step(case, states)
    got = read(slab.data, slab.scale).numpy()
    used = [int(i) for i in case["slot_ids"] if 0 <= int(i) < start.shape[0]]
    lens = request_lengths(case)
    live = [int(i) for i, n in zip(case["slot_ids"], lens) if 0 <= int(i) < start.shape[0] and n > 0]
    idle = [i for i in range(start.shape[0]) if i not in live]
    assert torch.equal(bits(slab.data[idle]), bits(before.data[idle]))
    if dtype == "e4m3":
        assert torch.equal(bits(slab.scale[idle]), bits(before.scale[idle]))
    vmax = float(np.abs(case["v"]).max(initial=0.0))
    if live:
        top = np.maximum(np.abs(rs[live]).max(-1, keepdims=True), np.abs(states[live]).max(-1, keepdims=True))
        slack = 2.5e-4 * tokens * np.maximum(top, vmax)
        least = LEAST[dtype] * (1 if dtype != "e4m3" else np.exp2(slab.scale.cpu().view(torch.uint8).double().numpy()[live] - 127)[..., None])
        bound = HALF[dtype] * (np.abs(rs[live]) + slack) + least + slack
        err = np.abs(got[live] - rs[live])
        assert (err <= bound).all(), (dtype, float((err / bound).max()))
        if dtype == "e4m3":  # the least power of two, to within the arithmetic
            unit = np.exp2(slab.scale.cpu().view(torch.uint8).double().numpy()[live] - 127)
            m = np.abs(rs[live]).max(-1)
            s = slack[..., 0]
            assert (m <= 448 * unit + s).all() and ((m >= 224 * unit - s) | (unit == 2.0 ** -100)).all()
    out_eps = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}[str(o.dtype)[6:]]
    size = max(vmax, float(np.abs(states[used]).max(initial=0.0)), float(np.abs(rs[used]).max(initial=0.0)))
    qn = 1.0 if case["qk_l2_norm"] else float(np.sqrt((np.asarray(case["q"], np.float64) ** 2).sum(-1)).max(initial=0.0))
    scale = case["scale"] or 1 / np.sqrt(case["q"].shape[-1])
    mask = covered(case)
    err = np.abs(o.double().cpu().numpy() - ro)[mask]
    assert (err <= out_eps * np.abs(ro[mask]) + 3e-4 * tokens * size * max(1.0, qn) * scale * np.sqrt(case["q"].shape[-1]) + 2.0 ** -25).all()
    return slab, o


def request_lengths(case):
    T = int(np.prod(case["q"].shape[:-2]))
    if case["cu_seqlens"] is not None:
        cu = np.clip(case["cu_seqlens"].astype(np.int64), 0, T)
        return [max(0, int(b - a)) for a, b in zip(cu[:-1], cu[1:])]
    B = len(case["slot_ids"])
    L = T // B
    return [L] * B if case.get("seq_lens") is None else [min(max(int(n), 0), L) for n in case["seq_lens"]]


def covered(case):
    """Mask over o's leading axes of tokens that a request with a valid slot covers."""
    lead = case["q"].shape[:-2]
    T = int(np.prod(lead))
    m = np.zeros(T, bool)
    lens, slots = request_lengths(case), case["slab"].shape[0]
    for b, n in enumerate(lens):
        s = int(np.clip(case["cu_seqlens"][b], 0, T)) if case["cu_seqlens"] is not None else b * (T // len(lens))
        if 0 <= int(case["slot_ids"][b]) < slots:
            m[s: s + n] = True
    return m.reshape(lead)


RULES = [dict(update_rule="gated_delta", gate_activation="qwen", beta_activation="sigmoid"),
         dict(update_rule="gated_delta", per_key=True), dict(update_rule="delta", beta_activation="sigmoid"),
         dict(update_rule="gated"), dict(update_rule="gated", per_key=True), dict(update_rule="linear"),
         dict(update_rule="gated_delta_v2"), dict(update_rule="gated_delta_v2", per_key=True)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rule", range(len(RULES)))
def test_single_tokens_of_every_rule(dtype, rule):
    for act, dim in ((np.float16, 128), ("bf16", 64), (np.float32, 256), ("bf16", 72), (np.float32, 97)):
        case = workloads.random_case(50 + rule, rank4_batch=(3, 1), H=2, HV=4, DK=dim, DV=dim, dtype=act, slots=(7,), **RULES[rule])
        step_and_check(case, dtype)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("dk,dv,H,HV,L", [(128, 128, 1, 1, 1), (128, 72, 2, 6, 2), (64, 256, 3, 3, 4), (256, 1, 1, 2, 3),
                                          (256, 130, 1, 4, 8), (64, 33, 2, 2, 7), (128, 256, 1, 3, 5),
                                          (96, 96, 2, 4, 1), (17, 40, 1, 2, 3), (255, 9, 1, 1, 2), (33, 33, 2, 2, 1),
                                          (16, 16, 1, 4, 5), (130, 64, 1, 2, 8), (72, 40, 3, 9, 1),
                                          (15, 64, 2, 4, 1), (9, 12, 1, 2, 3), (1, 1, 1, 1, 4), (8, 256, 1, 1, 1)])
def test_dims_heads_and_several_tokens(dtype, dk, dv, H, HV, L):
    for act in (np.float16, np.float32):
        case = workloads.random_case(dk + dv + L, rank4_batch=(2, L), H=H, HV=HV, DK=dk, DV=dv, dtype=act, slots=(5,),
                                     qk_l2_norm=1, **RULES[0])
        step_and_check(case, dtype, tokens=L)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rule", [1, 6, 7])
def test_several_tokens_with_per_key_factors(dtype, rule):
    for act, dim, L in (("bf16", 128, 5), (np.float16, 40, 3), (np.float32, 256, 2), ("bf16", 11, 2), (np.float32, 128, 8),
                        (np.float16, 64, 8), ("bf16", 256, 7), (np.float16, 256, 4), (np.float32, 256, 8),
                         ("bf16", 17, 8), (np.float16, 73, 6), (np.float32, 120, 4), ("bf16", 250, 7)):
        case = workloads.random_case(60 + rule, rank4_batch=(2, L), H=2, HV=4, DK=dim, DV=dim, dtype=act, slots=(4,), **RULES[rule])
        step_and_check(case, dtype, tokens=L)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_tiny_and_huge_values_on_the_matrix_cores(dtype):
    """States and values in fp16's denormal range, and keys whose planes are
    scaled: products of small operands are not lost."""
    for act, size, keys in ((np.float16, 2.0 ** -13, 1.0), ("bf16", 2.0 ** -13, 1.0), ("bf16", 1.0, 2.0 ** 9),
                            ("bf16", 1.0, 2.0 ** -20), (np.float16, 1.0, 2.0 ** -6)):
        case = workloads.random_case(95, rank4_batch=(2, 3), H=2, HV=2, DK=128, DV=64, dtype=act, slots=(3,), qk_l2_norm=1, **RULES[0])
        to16 = (lambda x: x.astype(np.float16)) if act == np.float16 else (lambda x: x)
        case["v"] = to16(np.asarray(case["v"], np.float32) * np.float32(size))
        case["slab"] = case["slab"] * np.float32(size)
        for name in ("q", "k"):
            case[name] = to16(np.asarray(case[name], np.float32) * np.float32(keys))
        step_and_check(case, dtype, tokens=3)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("act", [np.float16, "bf16", np.float32])
@pytest.mark.parametrize("dk,rule", [(128, 0), (64, 0), (256, 0), (40, 0), (128, 1), (64, 6), (9, 7), (256, 7), (33, 6), (200, 1)])
def test_nan_and_infinities_reach_later_tokens_only(dtype, act, dk, rule):
    """What a token brings does not reach the outputs before it, other requests,
    or, through v, other rows; what its q holds reaches its own output alone."""
    from gated_delta_rule_token_amd import api
    case = workloads.random_case(97, rank4_batch=(2, 5), H=1, HV=2, DK=dk, DV=40, dtype=act, slots=(4,), **RULES[rule])
    d, args = gpu_tensors(case)
    one, other = (int(i) for i in case["slot_ids"])

    def run(name=None, where=None, value=0.0):
        a, x = dict(args), {n: d[n] for n in ("q", "k", "v")}
        if name is not None:
            bad = (x[name] if name in x else a[name]).clone()
            bad[where] = value
            (x if name in x else a)[name] = bad
        slab = slab_of(case["slab"], dtype)
        o = api.forward_packed(x["q"], x["k"], x["v"], slab=slab, **a)
        return o, bits(slab.data), None if slab.scale is None else bits(slab.scale)

    o, data, scale = run()
    for value in (float("nan"), float("inf")):
        for name in ("q", "k", "v", "gate", "beta", "erase"):
            if name not in ("q", "k", "v") and args[name] is None:
                continue
            oo, dd, ss = run(name, (0, 3, 0, 3) if name in ("q", "k", "v") else (0, 3, 0), value)
            assert torch.equal(bits(oo[0, :3]), bits(o[0, :3])) and torch.equal(bits(oo[1]), bits(o[1])), name
            assert torch.equal(dd[other], data[other]) and (scale is None or torch.equal(ss[other], scale[other])), name
            assert value == float("inf") or not bool(oo[0, 3:].isfinite().all()), name  # (an infinite gate forgets)
            if name == "v":
                rows = torch.arange(40) != 3
                assert torch.equal(bits(oo[0][..., rows]), bits(o[0][..., rows])) and torch.equal(dd[one][:, rows], data[one][:, rows])
                assert torch.equal(dd[one, 1], data[one, 1])
            if name == "q":
                assert torch.equal(dd, data) and torch.equal(bits(oo[0, 4]), bits(o[0, 4]))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("act,dk,rule", [("bf16", 128, 0), (np.float32, 64, 0), (np.float16, 64, 1), (np.float16, 72, 0), ("bf16", 5, 6)])
@pytest.mark.parametrize("algo", ["auto", "recurrent"])
def test_padding_is_neither_read_nor_written(dtype, act, dk, rule, algo):
    """Tokens past seq_lens, before the first and behind the last packed request."""
    from gated_delta_rule_token_amd import api
    case = workloads.random_case(98, rank4_batch=(3, 6), H=1, HV=2, DK=dk, DV=24, dtype=act, slots=(5,), **RULES[rule])
    d, args = gpu_tensors(case)
    names = ("q", "k", "v", "gate", "beta", "erase")

    def run(used, o, flat, **kw):
        x = {}
        for n in names:
            t = d[n] if n in d and d[n] is not None else None
            if t is not None:
                t = t.flatten(0, 1)
                t = torch.where(used.view(-1, *[1] * (t.dim() - 1)), t, torch.full_like(t, float("nan")))
                t = t.contiguous() if flat else t.unflatten(0, (3, 6)).contiguous()
            x[n] = t
        a = dict(args, algo=algo, out=o, **kw)
        a.update({n: x[n] for n in names[3:]})
        slab = slab_of(case["slab"], dtype)
        api.forward_packed(x["q"], x["k"], x["v"], slab=slab, **a)
        return o, slab

    at = torch.arange(18, device="cuda")
    used = at % 6 < torch.tensor([4, 0, 6], device="cuda")[at // 6]
    like = d["v"]
    runs = [run(used, torch.full_like(like, 7.0), False, seq_lens=ids(4, 0, 6))]
    gap = (at >= 2) & (at < 9)
    runs.append(run(gap, torch.full_like(like, 7.0).flatten(0, 1), True, cu_seqlens=ids(2, 2, 5, 9)))
    for (o, slab), u in zip(runs, (used, gap)):
        o = o.reshape(18, 2, 24)
        assert bool(o[u].isfinite().all()) and bool((o[~u] == 7).all())
        assert bool(read(slab.data, slab.scale).isfinite().all())


@pytest.mark.parametrize("seed", range(36))
def test_random_steps(seed):
    """Any dims, heads, lengths, rules, activations and packings of short requests."""
    rng = np.random.default_rng(1000 + seed)
    dk = int(rng.choice([64, 128, 256, rng.integers(1, 257)]))
    dv = int(rng.choice([64, 128, dk, rng.integers(1, 257)]))
    H = int(rng.integers(1, 4))
    B = int(rng.integers(1, 5))
    rule = dict(RULES[int(rng.integers(len(RULES)))])
    if rule["update_rule"] in ("gated", "gated_delta") and not rule.get("per_key") and rng.random() < 0.5:
        rule.update(gate_activation="qwen", folded_scale=bool(rng.random() < 0.5))
    packing = [dict(rank4_batch=(B, int(rng.integers(1, 9)))), dict(rank4_batch=(B, 1)),
               dict(lengths=[int(n) for n in rng.integers(0, 13, B)])][int(rng.integers(3))]
    if "lengths" in packing and sum(packing["lengths"]) > 8 * B:
        packing["lengths"][0] = 0
    act = [np.float16, "bf16", np.float32][int(rng.integers(3))]
    case = workloads.random_case(2000 + seed, H=H, HV=H * int(rng.choice([1, 2, 3])), DK=dk, DV=dv, dtype=act, slots=(B + 2,),
                                 qk_l2_norm=int(rng.random() < 0.5), **packing, **rule)
    if "lengths" in packing and sum(packing["lengths"]) > 8 * B:
        pytest.skip("a prompt")
    if case["beta"] is not None and rng.random() < 0.3:
        case["beta"] = np.ascontiguousarray(case["beta"][..., :1])  # one rate a token
    step_and_check(case, ["f16", "bf16", "e4m3"][seed % 3], tokens=max(1, max(request_lengths(case))))


@pytest.mark.parametrize("dtype", DT)
def test_spellings_and_kernels_agree(dtype):
    """Rank 3 with a token a request is rank 4 with one, to the bit; the other
    kernels' results on unpacked states differ by their arithmetic alone."""
    from gated_delta_rule_token_amd import api
    case = workloads.random_case(96, rank4_batch=(5, 1), H=2, HV=4, DK=128, DV=128, dtype=np.float16, slots=(8,), **RULES[0])
    d, args = gpu_tensors(case)
    a, b, c = (slab_of(case["slab"], dtype) for _ in range(3))
    oa = api.forward_packed(d["q"], d["k"], d["v"], slab=a, **args)
    flat = {n: t[:, 0].contiguous() if n in ("gate", "beta") and t is not None else t for n, t in args.items()}
    ob = api.forward_packed(d["q"][:, 0].contiguous(), d["k"][:, 0].contiguous(), d["v"][:, 0].contiguous(), slab=b, **flat)
    assert torch.equal(oa[:, 0], ob) and same(a, b)
    cu = torch.arange(6, dtype=torch.int32, device="cuda")
    for kw in (dict(algo="recurrent"), dict(algo="decode"), dict(cu_seqlens=cu)):
        rank4 = "cu_seqlens" not in kw
        c = slab_of(case["slab"], dtype)
        q, k, v = (d[n] if rank4 else d[n][:, 0].contiguous() for n in "qkv")
        oc = api.forward_packed(q, k, v, slab=c, **dict(args if rank4 else flat, **kw))
        assert float((oc.float().view(-1) - oa.float().view(-1)).abs().max()) <= 2e-3 * float(oa.float().abs().max())
        x, y = read(c.data, c.scale), read(a.data, a.scale)
        # a value may fall on the other side of a border between two codes
        assert bool(((x - y).abs() <= 2.1 * HALF[dtype] * y.abs() + 1e-4 * y.abs().amax(-1, keepdim=True) + 2 * LEAST[dtype]).all())


@pytest.mark.parametrize("dtype", DT)
def test_ragged_requests_empty_ones_and_ids_out_of_range(dtype):
    case = workloads.random_case(70, lengths=[1, 0, 3, 1, 2, 0, 1, 9], H=2, HV=4, DK=128, DV=128, dtype=np.float16, slots=(12,), **RULES[0])
    case["slot_ids"][3], case["slot_ids"][5] = -5, 12
    step_and_check(case, dtype, tokens=9)
    # padded rows, and lengths past the ends
    case = workloads.random_case(71, rank4_batch=(4, 3), H=2, HV=4, DK=128, DV=128, dtype="bf16", slots=(6,),
                                 seq_lens=[2, 0, 7, -1], **RULES[0])
    step_and_check(case, dtype, tokens=3)
    # rows that no request covers stay as they were
    from gated_delta_rule_token_amd import api
    d, args = gpu_tensors(case)
    out = torch.full((4, 3, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    api.forward_packed(d["q"], d["k"], d["v"], slab=slab_of(case["slab"], dtype), out=out, **args)
    keep = torch.from_numpy(covered(case)).cuda()
    assert bool((out[~keep] == 9).all()) and not bool((out[keep] == 9).all())


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("dk,dv,lengths,act", [(72, 40, [3, 0, 30, 1], np.float32), (128, 128, [200, 0, 150, 333], np.float16),
                                               (64, 64, [40, 17, 1, 0], "bf16"), (9, 12, [1, 1, 0, 1], np.float16)])
def test_prompts_run_the_forward_on_unpacked_states(dtype, dk, dv, lengths, act):
    """Bit for bit what unpack, forward and pack give; empty requests and ids
    out of range as ever."""
    from gated_delta_rule_token_amd import api
    case = workloads.random_case(80, lengths=lengths, H=2, HV=4, DK=dk, DV=dv, dtype=act, slots=(9,), qk_l2_norm=1, **RULES[0])
    case["slot_ids"][0] = 9
    d, args = gpu_tensors(case)
    slab = slab_of(case["slab"], dtype)
    want = clone(slab)
    out = torch.full(tuple(d["v"].shape), 3.0, dtype=d["q"].dtype, device="cuda")
    ref = out.clone()
    o = api.forward_packed(d["q"], d["k"], d["v"], slab=slab, out=out, **args)
    assert o is out
    states = api.state_unpack(want, d["slot_ids"])
    inner = torch.tensor([b if 0 <= int(i) < 9 else -1 for b, i in enumerate(case["slot_ids"])], dtype=torch.int32, device="cuda")
    api.forward(d["q"], d["k"], d["v"], state=states, out=ref, **dict(args, slot_ids=inner))
    live = [b for b, n in enumerate(lengths) if n > 0]
    api.state_pack(states[live].contiguous(), want, d["slot_ids"][live].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(o, ref) and same(slab, want)
    assert bool((o[: lengths[0]] == 3).all())


def test_no_requests_and_no_tokens():
    from gated_delta_rule_token_amd import api
    slab = slab_of(torch.ones(3, 2, 128, 128), "e4m3")
    before = clone(slab)
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    o = api.forward_packed(z(0, 1, 2, 128), z(0, 1, 2, 128), z(0, 1, 2, 128), slab=slab, slot_ids=ids(), update_rule="linear")
    assert o.shape == (0, 1, 2, 128)
    api.forward_packed(z(0, 2, 128), z(0, 2, 128), z(0, 2, 128), slab=slab, slot_ids=ids(1, 0), update_rule="linear",
                       cu_seqlens=ids(0, 0, 0))
    api.forward_packed(z(40, 2, 128), z(40, 2, 128), z(40, 2, 128), slab=slab, slot_ids=ids(1, 0), update_rule="linear",
                       cu_seqlens=ids(5, 5, 2))  # a decreasing entry is an empty request
    torch.cuda.synchronize()
    assert same(slab, before)


def test_resets_infinities_and_nan_stay_in_their_heads():
    from gated_delta_rule_token_amd import api
    case = workloads.random_case(90, rank4_batch=(3, 1), H=2, HV=2, DK=128, DV=128, dtype=np.float32, slots=(3,), update_rule="gated_delta")
    case["slot_ids"][:] = [0, 1, 2]
    case["gate"][0, 0, 1] = -np.inf  # a reset: the state is the token's own
    for dtype in DT:
        slab, _ = step_and_check(case, dtype)
        d, args = gpu_tensors(case)
        bad = slab_of(case["slab"], dtype)
        d["v"][1, 0, 0, 5] = float("nan")
        d["q"][2, 0, 1, 7] = float("inf")
        o = api.forward_packed(d["q"], d["k"], d["v"], slab=bad, **args)
        rows = torch.ones(3, 2, 128, dtype=torch.bool)
        rows[1, 0, 5] = False
        a, b = read(bad.data, bad.scale), read(slab.data, slab.scale)
        assert torch.equal(a[rows], b[rows]) and bool(a[1, 0, 5].isnan().all())
        assert bool(o[1, 0, 0, 5].isnan()) and bool(o[:2, 0, 1].isfinite().all()) and not bool(o[2, 0, 1].isfinite().any())


def test_slots_past_32_bit_offsets():
    """Offsets past 2^32 values: the last slots of a cache of 4.3e9 values."""
    from gated_delta_rule_token_amd import api
    slots = 2 ** 32 // (128 * 128) + 3
    case = workloads.random_case(91, rank4_batch=(2, 1), H=1, HV=1, DK=128, DV=128, dtype=np.float16, slots=(4,), **RULES[0])
    for dtype in ("e4m3", "bf16"):
        small = slab_of(case["slab"], dtype)
        d, args = gpu_tensors(case)
        data = torch.zeros(slots, 1, 128, 128, dtype=torch.uint8 if dtype == "e4m3" else torch.int16, device="cuda").view(DT[dtype])
        scale = None if dtype != "e4m3" else torch.full((slots, 1, 128), 27, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
        big = api.PackedSlab(data, scale)
        at = [slots - 1, slots - 2]
        for n, i in enumerate(case["slot_ids"]):
            bits(data)[at[n]] = bits(small.data)[int(i)]
            if scale is not None:
                bits(scale)[at[n]] = bits(small.scale)[int(i)]
        assert torch.equal(api.state_unpack(big, ids(*at)), api.state_unpack(small, d["slot_ids"]))
        o1 = api.forward_packed(d["q"], d["k"], d["v"], slab=big, **dict(args, slot_ids=ids(*at)))
        o2 = api.forward_packed(d["q"], d["k"], d["v"], slab=small, **args)
        got, want = api.state_unpack(big, ids(*at)), api.state_unpack(small, d["slot_ids"])
        assert torch.equal(o1, o2) and torch.equal(got, want)
        api.state_pack(want + 1, big, ids(*at))
        api.state_pack(want + 1, small, d["slot_ids"])
        assert torch.equal(api.state_unpack(big, ids(*at)), api.state_unpack(small, d["slot_ids"]))
        assert not bool(bits(data)[: slots - 2].any())
        del data, big
        torch.cuda.empty_cache()


def test_other_streams_and_captured_graphs():
    """A captured step of single tokens and one of a prompt, replayed in turn:
    every replay goes on with the cache as the eager calls do."""
    from gated_delta_rule_token_amd import api
    step = workloads.random_case(92, rank4_batch=(3, 1), H=2, HV=4, DK=128, DV=128, dtype=np.float16, slots=(6,), **RULES[0])
    long = workloads.random_case(93, lengths=[130, 260], H=2, HV=4, DK=128, DV=128, dtype=np.float16, slots=(6,), qk_l2_norm=1, **RULES[0])
    (d1, a1), (d2, a2) = gpu_tensors(step), gpu_tensors(long)
    p = api.build_problem(d2["q"], d2["k"], d2["v"], gate=d2["gate"], beta=d2["beta"], cu_seqlens=d2["cu_seqlens"],
                          slot_ids=d2["slot_ids"], state=torch.empty(6, 4, 128, 128), update_rule="gated_delta",
                          gate_activation="qwen", beta_activation="sigmoid")
    ws = torch.empty(api.packed_workspace_size(p), dtype=torch.uint8, device="cuda")
    for dtype in DT:
        eager, slab = slab_of(step["slab"], dtype), slab_of(step["slab"], dtype)
        o1, o2 = torch.empty_like(d1["v"]), torch.empty_like(d2["v"])
        g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g1):
            api.forward_packed(d1["q"], d1["k"], d1["v"], slab=slab, out=o1, **a1)
        with torch.cuda.graph(g2):
            api.forward_packed(d2["q"], d2["k"], d2["v"], slab=slab, out=o2, workspace=ws, **a2)
        for n in range(3):
            for g, d, a, o in ((g1, d1, a1, o1), (g2, d2, a2, o2), (g1, d1, a1, o1)):
                g.replay()
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    want = api.forward_packed(d["q"], d["k"], d["v"], slab=eager, **a)
                torch.cuda.current_stream().wait_stream(side)
                torch.cuda.synchronize()
                assert torch.equal(o, want) and same(slab, eager), (dtype, n)


def test_refusals_on_the_gpu():
    from gated_delta_rule_token_amd import api
    case = workloads.random_case(94, rank4_batch=(2, 1), H=2, HV=4, DK=128, DV=128, dtype=np.float16, slots=(4,), **RULES[0])
    d, args = gpu_tensors(case)
    slab = slab_of(case["slab"], "e4m3")
    qkv = (d["q"], d["k"], d["v"])
    for text, s in (("scales exactly", api.PackedSlab(slab.data)), ("scale has shape", api.PackedSlab(slab.data, slab.scale[:3])),
                    ("slab.data must be", api.PackedSlab(slab.data.float())), ("contiguous", api.PackedSlab(slab.data[:, :2], slab.scale[:, :2].contiguous())),
                    ("scale must be", api.PackedSlab(slab.data, slab.scale.view(torch.uint8))),
                    ("state has shape", api.PackedSlab(slab.data[:, :2].contiguous(), slab.scale[:, :2].contiguous()))):
        with pytest.raises(api.GDRError, match=text):
            api.forward_packed(*qkv, slab=s, **args)
    for text, over in (("slot_ids", dict(slot_ids=None)), ("slot_ids", dict(slot_ids=args["slot_ids"].long())),
                       ("beta", dict(beta=None)), ("gate", dict(gate=d["gate"][:1].contiguous())),
                       ("out", dict(out=torch.empty(2, 1, 4, 64, dtype=torch.float16, device="cuda"))),
                       ("overlaps", dict(out=d["v"]))):
        with pytest.raises(api.GDRError, match=text):
            api.forward_packed(*qkv, slab=slab, **dict(args, **over))
    for text, states in (("states has shape", torch.zeros(2, 4, 128, 64, device="cuda")), ("states must be", torch.zeros(2, 4, 128, 128, device="cuda").half())):
        with pytest.raises(api.GDRError, match=text):
            api.state_pack(states, slab, args["slot_ids"])
    with pytest.raises(api.GDRError, match="out has shape"):
        api.state_unpack(slab, args["slot_ids"], out=torch.zeros(1, 4, 128, 128, device="cuda"))
