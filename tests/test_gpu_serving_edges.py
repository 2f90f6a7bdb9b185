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
