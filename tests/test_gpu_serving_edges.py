"""Edges of the norm and rotation of q and k and of the state cache in fewer
bits, on an MI355X: values that are not finite, sizes at which a kernel changes
its course, and bounds that a lost plane of an operand exceeds."""
import numpy as np
import pytest

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


def ids(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


# ------------------------------------------------------------------ values that are not finite, in 8 bits

@pytest.mark.parametrize("dk", [2, 3, 4, 30, 64, 128, 150, 256])
def test_infinities_leave_the_rest_of_an_8_bit_row(dk):
    """A row's scale is that of its finite values: with an infinity in place of a
    zero every other code and the scale stay, and the infinity reads as NaN."""
    from gated_delta_rule_token_amd import api
    g = torch.Generator().manual_seed(dk)
    x = torch.randn(2, 2, 37, dk, generator=g) * torch.exp(4 * torch.randn(2, 2, 37, 1, generator=g))
    at = torch.randint(0, dk, (2, 2, 37, 1), generator=g)
    x.scatter_(-1, at, 0.0)
    bad = torch.tensor([float("inf"), -float("inf")]).repeat(74)[: 2 * 2 * 37].view(2, 2, 37, 1)
    y = x.scatter(-1, at, bad)
    y[1, 1, 5] = float("inf")  # nothing finite
    got = []
    for states in (x, y):
        slab = api.packed_slab(3, 2, 37, dk, torch.float8_e4m3fn)
        api.state_pack(states.cuda(), slab, ids(2, 0))
        got.append((bits(slab.data).cpu(), bits(slab.scale).cpu(), api.state_unpack(slab, ids(2, 0)).cpu()))
    (codes, scale, _), (codes_y, scale_y, read_y) = got
    hit = torch.zeros(3, 2, 37, dk, dtype=torch.bool)
    hit[[2, 0]] = torch.zeros(2, 2, 37, dk, dtype=torch.bool).scatter_(-1, at, True)
    hit[0, 1, 5] = True
    rows = torch.ones(3, 2, 37, dtype=torch.bool)
    rows[0, 1, 5] = False
    assert torch.equal(codes_y[~hit], codes[~hit]) and torch.equal(scale_y[rows], scale[rows])
    assert torch.equal(read_y.isnan(), hit[[2, 0]])


@pytest.mark.parametrize("act", [np.float16, "bf16", np.float32])
@pytest.mark.parametrize("L", [1, 3, 10])
@pytest.mark.parametrize("dk", [9, 64, 72, 128, 200, 256])
def test_an_infinite_key_leaves_the_rest_of_an_8_bit_row(dk, L, act):
    """Without retrieval a key channel's state is its own: an infinity there
    (column 3 of the last token's k) leaves the others' codes and the rows' scales as
    they are with a zero in its place."""
    from gated_delta_rule_token_amd import api
    packing = dict(lengths=[1, L]) if L > 8 else dict(rank4_batch=(2, L))
    case = workloads.random_case(dk + L, H=1, HV=2, DK=dk, DV=40, dtype=act, slots=(4,), update_rule="linear", **packing)
    cu = None if case["cu_seqlens"] is None else torch.from_numpy(case["cu_seqlens"]).cuda()
    dt = {"float16": torch.float16, "float32": torch.float32}.get(getattr(act, "__name__", ""), torch.bfloat16)
    q, k, v = (torch.from_numpy(np.asarray(case[n], np.float32)).to(dt).cuda() for n in "qkv")
    k[..., 3] = 0
    start = torch.from_numpy(np.asarray(case["slab"], np.float32))
    start[..., 3] = 0
    where = torch.from_numpy(case["slot_ids"]).cuda()
    got = []
    for value in (0.0, float("inf")):
        slab = api.packed_slab(4, 2, 40, dk, torch.float8_e4m3fn)
        api.state_pack(start.cuda(), slab, ids(0, 1, 2, 3))
        k.flatten(0, -3)[-1, :, 3] = value
        api.forward_packed(q, k, v, slab=slab, slot_ids=where, cu_seqlens=cu, update_rule="linear")
        got.append((bits(slab.data).cpu(), bits(slab.scale).cpu(), slab.data.float().cpu()))
    (codes, scale, _), (codes_y, scale_y, read_y) = got
    rest = torch.arange(dk) != 3
    assert torch.equal(codes_y[..., rest], codes[..., rest]) and torch.equal(scale_y, scale)
    assert bool(read_y[int(where[1]), ..., 3].isnan().all()) and not bool(read_y[int(where[0])].isnan().any())


# ------------------------------------------------------------------ the rotation

@pytest.mark.parametrize("d,R,dtype,weight,inter", [(128, 128, "bf16", "bf16", False), (72, 40, "f16", None, False),
                                                    (63, 30, "f32", "f32", True), (64, 64, "f32", None, False)])
def test_gradients_without_the_norm_do_not_depend_on_x(d, R, dtype, weight, inter):
    """d_x is weight * g then, whatever x holds; a weight's gradient sums x by column."""
    from tests.test_gpu_rotary import back, cuda, d_outs, dev, make
    c = make(31, 50, 3, 2, d, R, dtype, weight=weight)
    douts = cuda(d_outs(c))
    want = back(dev(c), *douts, inter, False)
    c["q"][7, 1, 5], c["q"][20, 0, d - 1], c["k"][3, 1, 2] = float("inf"), float("nan"), -float("inf")
    got = back(dev(c), *douts, inter, False)
    assert torch.equal(got.q, want.q) and torch.equal(got.k, want.k)
    if weight is not None:
        for g, w, columns in ((got.q_weight, want.q_weight, [5, d - 1]), (got.k_weight, want.k_weight, [2])):
            rest = torch.ones(d, dtype=torch.bool)
            rest[columns] = False
            assert torch.equal(g.cpu()[rest], w.cpu()[rest]) and not bool(g.cpu()[~rest].isfinite().any())


def test_sines_and_cosines_of_far_positions():
    """Pairs (1, 0) turn into (cos, sin).  With u = 2^-24: the rest of the turn, at
    most an eighth, is rounded by 2^-28, 2.4e-8 in the angle and 1.7e-8 in a sine of
    0.707; its series loses 1.2 u on the last product's factor (up to 6.28, rounded by
    2^-22 of at least 5.65), 0.3 u on its terms and u on the product, 2.5 u 0.707 =
    1.05e-7 if all err to one side, and the terms left out 2e-8 at the ends alone (3e-9 in
    the sine).  So each is within 1.3e-7 at most; a fraction of a whole turn rounded
    to fp32 exceeds that by itself with 9.4e-8 in the angle."""
    from gated_delta_rule_token_amd import api
    T, half = 16384, 64
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(-2000000, 2000000, (T,), generator=g).to(torch.int32)
    freq = torch.exp(-9.2 * torch.rand(half, generator=g))
    x = torch.cat([torch.ones(T, 1, half), torch.zeros(T, 1, half)], -1)
    y = api.qk_rotary(x.cuda(), None, pos.cuda(), freq.cuda(), norm=False).q.cpu().double()
    angle = pos.double()[:, None, None] * freq.double()
    err = (y - torch.cat([torch.cos(angle), torch.sin(angle)], -1)).abs()
    print("largest error %.3e" % float(err.max()))
    assert float(err.max()) <= 1.3e-7


def test_more_tokens_than_a_launch_has_workgroups():
    """2^24 and more workgroups of a token each: rows at the ends and around the
    2^24th against a call of those rows alone."""
    from gated_delta_rule_token_amd import api
    T, H = 2 ** 24 + 5, 128
    at = torch.cat([torch.arange(0, 3), torch.arange(2 ** 24 - 4, T)]).cuda()
    g = torch.Generator().manual_seed(6)
    rows = torch.randn(at.shape[0], H, 2, generator=g).half().cuda()
    p = torch.randint(-5000, 5000, (at.shape[0],), generator=g).to(torch.int32).cuda()
    freq = torch.tensor([0.3], device="cuda")
    q = torch.zeros(T, H, 2, dtype=torch.float16, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    q[at], pos[at] = rows, p
    api.qk_rotary(q, None, pos, freq, out=(q, None))
    assert torch.equal(q[at], api.qk_rotary(rows, None, p, freq).q)
    assert not bool(q[3: 2 ** 24 - 4].any())
    del q
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ steps of several tokens

FORMS = {"plain": dict(update_rule="delta"), "per_key": dict(update_rule="gated_delta", per_key=True),
         "erase": dict(update_rule="gated_delta_v2")}


@pytest.mark.parametrize("cache", DT)
@pytest.mark.parametrize("act", [np.float16, "bf16", np.float32])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dk,L", [(128, 1), (128, 3), (64, 8), (256, 5), (72, 4), (200, 7), (15, 3), (128, 12)])
def test_values_that_replace_far_larger_ones(cache, act, form, dk, L):
    """Each token has a key channel of its own, k = c there, and a rate (or an
    erase) of 1 / c^2: what stays of the old value S is v / c, up to 2^-14 times
    smaller, so the arithmetic's share of S shows: every product of the update
    takes part in 32 bits.  With u = 2^-24 and M = |S| + 2 |v|, which bounds
    every term: S k by planes 4 u, the difference from v and its factors 4 u, the
    planes of that and of k and their products 6 u, the sum with S u: 16 u M.  Two planes
    of 8 bits instead of three would add 64 u M."""
    from gated_delta_rule_token_amd import api
    from tests.test_gpu_packed import HALF, LEAST, gpu_tensors, oracle_step, read, slab_of
    from tests.test_gpu_packed import bits as code_bits
    far = {"f16": 2.0 ** 12, "bf16": 2.0 ** 15, "e4m3": 2.0 ** 18}[cache]
    if act == np.float16 and far > 2.0 ** 15:
        far = 2.0 ** 15  # (v times a power of two below)
    packing = dict(lengths=[1, L]) if L > 8 else dict(rank4_batch=(2, L))
    case = workloads.random_case(7 * dk + L, H=1, HV=2, DK=dk, DV=72, dtype=act, slots=(3,), **packing, **FORMS[form])
    rng = np.random.default_rng(dk + L)
    lead = case["q"].shape[:-2]
    T = int(np.prod(lead))
    narrow = {np.float16: lambda x: x.astype(np.float16), "bf16": lambda x: torch.from_numpy(x).bfloat16().float().numpy(),
              np.float32: lambda x: x}[act]
    column = np.concatenate([rng.permutation(dk)[:n] for n in ([1, L] if L > 8 else [L, L])])
    c = narrow(rng.uniform(0.5, 1.0, T).astype(np.float32))
    k, q = np.zeros((T, 1, dk), c.dtype), np.zeros((T, 1, dk), c.dtype)
    k[np.arange(T), 0, column] = c
    q[np.arange(T), 0, column] = narrow(rng.uniform(0.5, 1.0, T).astype(np.float32))
    case["k"], case["q"] = k.reshape(case["k"].shape), q.reshape(case["q"].shape)
    case["v"] = narrow((rng.uniform(0.5, 1.0, case["v"].shape) * rng.choice([-1, 1], case["v"].shape)).astype(np.float32))
    rate = (1 / c.astype(np.float64) ** 2).astype(np.float32)
    if case["gate"] is not None:
        case["gate"] = np.zeros_like(case["gate"])
    if case["beta"] is not None:
        case["beta"] = np.broadcast_to(rate.reshape(lead + (1,)), case["beta"].shape).astype(np.float32).copy()
    if case["erase"] is not None:
        case["erase"] = np.broadcast_to(rate.reshape(lead + (1, 1)), case["erase"].shape).astype(np.float32).copy()
    start = np.zeros_like(case["slab"])
    first = 0
    for b, n in enumerate([1, L] if L > 8 else [L, L]):
        mine = column[first: first + n]
        start[int(case["slot_ids"][b])][..., mine] = far * rng.uniform(0.5, 1.0, (2, 72, n)) * rng.choice([-1, 1], (2, 72, n))
        first += n
    case["slab"] = start
    slab = slab_of(start, cache)
    old = read(slab.data, slab.scale).numpy()
    d, args = gpu_tensors(case)
    o = api.forward_packed(d["q"], d["k"], d["v"], slab=slab, **args)
    ro, rs = oracle_step(case, old)
    got = read(slab.data, slab.scale).numpy()
    live = case["slot_ids"]
    M = np.abs(old[live]).max() + 2 * np.abs(np.asarray(case["v"], np.float64)).max()
    least = LEAST[cache] * (1 if cache != "e4m3" else np.exp2(code_bits(slab.scale).cpu().double().numpy()[live] - 127)[..., None])
    slack = 2.0 ** -20 * M
    bound = HALF[cache] * (np.abs(rs[live]) + slack) + least + slack
    err = np.abs(got[live] - rs[live])
    print("state: %.3f of the bound" % float((err / bound).max()))
    assert (err <= bound).all()
    out_half = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}[str(o.dtype)[6:]]
    err = np.abs(o.double().cpu().numpy() - ro)
    bound = out_half * np.abs(ro) + slack / np.sqrt(dk) * 1.01 + 2.0 ** -25
    print("outputs: %.3f of the bound" % float((err / bound).max()))
    assert (err <= bound).all()


@pytest.mark.parametrize("act", [np.float16, np.float32])
@pytest.mark.parametrize("dk", [72, 120, 150, 200, 250])
def test_a_growing_gate_stays_in_its_row(dk, act):
    """gate_scale = 300 and biases that take the softplus to 1e-20: decays of 1.  The
    lanes past a row's end, which have no bias, would see e^208."""
    from tests.test_gpu_packed import step_and_check
    case = workloads.random_case(dk, rank4_batch=(2, 3), H=1, HV=2, DK=dk, DV=24, dtype=act, slots=(3,), qk_l2_norm=1,
                                 update_rule="gated_delta", per_key=True, gate_activation="qwen", folded_scale=True)
    case["gate_scale"][:] = 300.0
    case["gate"][:] = 0
    case["dt_bias"][:] = -46.0
    for cache in DT:
        step_and_check(case, cache, tokens=3)


@pytest.mark.parametrize("cache", DT)
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("act", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk,dv,L", [(128, 128, 4), (64, 200, 7), (256, 130, 2), (96, 256, 3), (200, 120, 8)])
def test_many_states_give_what_few_do(cache, form, act, dk, dv, L):
    """64 requests of 32 heads fill the GPU with a wave for each state, which walks
    all its rows 16 at a time with the next ones on their way; four requests have up to 8
    waves a state, each with a part of its rows.  The same bits."""
    from gated_delta_rule_token_amd import api
    B, H, HV = 64, 16, 32
    g = torch.Generator("cuda").manual_seed(dk + dv)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = dict(q=n(B, L, H, dk).to(act), k=n(B, L, H, dk).to(act), v=n(B, L, HV, dv).to(act))
    rule = {"update_rule": FORMS[form]["update_rule"] if form != "plain" else "gated_delta"}
    if rule["update_rule"] != "delta":
        x["gate"] = -0.2 * n(B, L, HV, *((dk,) if form == "per_key" else ())).abs()
    if form == "erase":
        x["erase"] = torch.sigmoid(n(B, L, HV, dk))
    else:
        x["beta"] = torch.sigmoid(n(B, L, HV))
    states = n(B, HV, dv, dk) * torch.exp(2 * n(B, HV, dv, 1))
    where = torch.randperm(B, generator=g, device="cuda").to(torch.int32)
    start = api.packed_slab(B, HV, dv, dk, DT[cache])
    api.state_pack(states, start, where)
    big = api.PackedSlab(start.data.clone(), None if start.scale is None else start.scale.clone())

    def run(slab, rows):
        y = {name: t[rows].contiguous() for name, t in x.items()}
        return api.forward_packed(y.pop("q"), y.pop("k"), y.pop("v"), slab=slab, slot_ids=where[rows].contiguous(),
                                  qk_l2_norm=True, **y, **rule)

    o = run(big, slice(0, B))
    parts = torch.cat([run(start, slice(b, b + 4)) for b in range(0, B, 4)])
    assert torch.equal(o, parts) and bool(o.isfinite().all()) and torch.equal(bits(big.data), bits(start.data))
    assert start.scale is None or torch.equal(bits(big.scale), bits(start.scale))


@pytest.mark.parametrize("cache", DT)
@pytest.mark.parametrize("act", [torch.float16, torch.bfloat16])
def test_each_step_of_a_run_from_the_states_it_found(cache, act):
    """A prompt and six single tokens with positions; each call against 64 bits from
    what the cache held before it, so that no call's rounding hides the next one's work.
    With u = 2^-24, a dot of 128 products in fp32 is off by 128 u of its magnitudes and
    the norms, the rate and the decay add under 32 u: 160 u of sum |S| |k| and sum
    |S| |q|, and with the token's own part of |v|.  The prompt's states: the chunked form's
    bar, 2e-3 of the largest."""
    from gated_delta_rule_token_amd import api
    from tests.test_gpu_packed import HALF, LEAST, read
    from tests.test_gpu_serving import D, H, HV, inputs, recurrence, unit
    lens, steps, u = [150, 1, 70], 6, 2.0 ** -24
    c = inputs(lens, steps, act, 17)
    B, T0 = len(lens), sum(lens)
    slab = api.packed_slab(6, HV, D, D, DT[cache])
    slots = [4, 0, 5]
    dev = {n: t.cuda() for n, t in c.items()}
    d = {n: t.double() for n, t in c.items()}
    start = torch.tensor([0] + lens).cumsum(0)

    def call(rows, pos, **kw):
        n = rows.stop - rows.start
        wide = dev["qk"][rows]
        r = api.qk_rotary(wide[:, : H * D].view(n, H, D), wide[:, H * D:].view(n, H, D), pos.to(torch.int32).cuda(),
                          dev["freq"], q_weight=dev["qw"], k_weight=dev["kw"])
        v, a, b = (dev[name][rows].clone() for name in "vab")
        o = api.forward_packed(r.q, r.k, v, slab=slab, slot_ids=ids(*slots), gate=a, beta=b, gate_activation="qwen",
                               beta_activation="sigmoid", qk_l2_norm=True, a_log=dev["a_log"], dt_bias=dev["dt_bias"], **kw)
        q, k = (unit(t.cpu().double()).repeat_interleave(HV // H, 1) for t in r)
        g = -torch.exp(d["a_log"]) * torch.nn.functional.softplus(d["a"][rows] + d["dt_bias"])
        return o.cpu().double(), q, k, d["v"][rows], g, torch.sigmoid(d["b"][rows])

    def state():
        return read(slab.data, slab.scale)[slots]

    def check_states(want, slack):
        least = LEAST[cache] if cache != "e4m3" else \
            LEAST[cache] * torch.exp2(slab.scale.view(torch.uint8).cpu()[slots].double() - 127)[..., None]
        bound = HALF[cache] * (want.abs() + slack) + least + slack
        err = (state() - want).abs()
        assert bool((err <= bound).all()), float((err / bound).max())

    _, *x = call(slice(0, T0), torch.cat([torch.arange(n) for n in lens]), cu_seqlens=start.to(torch.int32).cuda())
    want = torch.stack([recurrence(*(t[start[b]: start[b + 1]] for t in x), torch.zeros(HV, D, D).double())[1] for b in range(B)])
    check_states(want, 2e-3 * float(want.abs().max()))
    for i in range(steps):
        before = state()
        o, q, k, v, g, beta = call(slice(T0 + i * B, T0 + (i + 1) * B), torch.tensor([n + i for n in lens]))
        S = before * torch.exp(g)[..., None, None]
        put = beta[..., None] * (v - (S * k[..., None, :]).sum(-1))
        new = S + put[..., None] * k[..., None, :]
        # magnitudes of the sums behind `put` (one a row) and behind an output
        around = beta[..., None] * (v.abs() + (S.abs() * k[..., None, :].abs()).sum(-1))
        check_states(new, 160 * u * (S.abs() + around[..., None] * k[..., None, :].abs()))
        ref = (new * q[..., None, :]).sum(-1) / D ** 0.5
        reach = ((S.abs() * q[..., None, :].abs()).sum(-1) + around * (q * k).abs().sum(-1)[..., None]) / D ** 0.5
        bound = torch.finfo(act).eps / 2 * ref.abs() + 2 * 160 * u * reach + 2.0 ** -25
        assert bool(((o - ref).abs() <= bound).all()), (i, float(((o - ref).abs() / bound).max()))
        assert float(ref.abs().max()) > 20 * float(bound.max())


@pytest.mark.parametrize("cache", DT)
@pytest.mark.parametrize("act", [np.float16, "bf16", np.float32])
@pytest.mark.parametrize("rule", [dict(update_rule="gated_delta"), dict(update_rule="gated_delta", per_key=True),
                                  dict(update_rule="gated_delta_v2", per_key=True)], ids=["plain", "per_key", "erase"])
@pytest.mark.parametrize("dk,L", [(128, 1), (128, 4), (64, 8), (256, 7), (72, 5), (200, 3), (13, 6)])
def test_several_tokens_within_their_arithmetic(cache, act, rule, dk, L):
    """Bounds that run along with the recurrence.  A holds the magnitudes that went
    into a state, E what it may be off by; with u = 2^-24 a dot of dk products in
    fp32 is off by dk u of its magnitudes, and planes, decays (up to 8 in a product, 3 u
    each), norms and rates by under 64 u: c = dk + 64.  So a new value is off by
    e = beta (c u sum A |k| + sum E |k|) + 4 u |put|, the state by E <- a E + e |k| +
    c u |put| |k| + 32 u A, an output by c u sum A |q| + sum E |q| and its rounding.  (That
    these bounds say something is asserted of the inputs: their median is under a
    hundredth of an output's.)"""
    from gated_delta_rule_token_amd import api
    from tests.test_gpu_packed import HALF, LEAST, gpu_tensors, read, slab_of
    case = workloads.random_case(3 * dk + L, rank4_batch=(2, L), H=2, HV=4, DK=dk, DV=40, dtype=act, slots=(3,), qk_l2_norm=1, **rule)
    slab = slab_of(case["slab"], cache)
    S = read(slab.data, slab.scale).numpy()[case["slot_ids"]]
    d, args = gpu_tensors(case)
    o = api.forward_packed(d["q"], d["k"], d["v"], slab=slab, **args)
    got, out = read(slab.data, slab.scale).numpy()[case["slot_ids"]], o.double().cpu().numpy()
    half_out = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}[str(o.dtype)[6:]]
    q, k, v = (np.asarray(case[n], np.float64) for n in "qkv")
    q, k = (np.repeat(x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-12), 2, 2) for x in (q, k))
    cu, u = (dk + 64) * 2.0 ** -24, 2.0 ** -24
    A, E = np.abs(S), np.zeros_like(S)
    for t in range(L):
        a = np.exp(case["gate"][:, t].astype(np.float64))
        a = a[..., None, :] if rule.get("per_key") else a[..., None, None]
        beta = np.ones((2, 4, 1)) if case["beta"] is None else case["beta"][:, t].astype(np.float64)[..., None]
        kr = k[:, t] if case["erase"] is None else k[:, t] * case["erase"][:, t].astype(np.float64)
        S, A, E = a * S, a * A, a * E
        dot = lambda M, x: (M * np.abs(x)[..., None, :]).sum(-1)  # noqa: E731
        put = beta * (v[:, t] - (S * kr[..., None, :]).sum(-1))
        most = beta * (np.abs(v[:, t]) + dot(A, kr))
        e = beta * (cu * dot(A, kr) + dot(E, kr)) + 4 * u * most
        outer = lambda x: x[..., None] * np.abs(k[:, t])[..., None, :]  # noqa: E731
        S = S + put[..., None] * k[:, t][..., None, :]
        E = E + outer(e) + cu * outer(most) + 32 * u * A
        A = A + outer(most)
        ref = (S * q[:, t][..., None, :]).sum(-1) / np.sqrt(dk)
        bound = half_out * np.abs(ref) + (cu * dot(A, q[:, t]) + dot(E, q[:, t])) / np.sqrt(dk) + 2.0 ** -25
        err = np.abs(out[:, t] - ref)
        assert (err <= bound).all(), (t, float((err / bound).max()))
        if act == np.float32:
            assert np.median(bound) < 1e-2 * np.median(np.abs(ref))
    least = LEAST[cache] * (1 if cache != "e4m3" else
                            np.exp2(slab.scale.view(torch.uint8).cpu().double().numpy()[case["slot_ids"]] - 127)[..., None])
    err, bound = np.abs(got - S), HALF[cache] * (np.abs(S) + E) + least + E
    assert (err <= bound).all(), float((err / bound).max())
