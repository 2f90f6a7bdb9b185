"""The operators of a layer with positions, run together as they are used: a
prompt and then single tokens on a packed state cache, and a training step,
against the whole sequence in 64 bits, on an MI355X."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_token_amd import api
    api.load_library()


H, HV, D = 2, 4, 128


def rotate(x, w, angle, eps=1e-6):
    h = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    a, b = h[..., : D // 2], h[..., D // 2:]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def unit(x):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-12)


def recurrence(q, k, v, g, beta, state):
    """One request, (L, heads, ...): outputs and the largest |S| |q| of a row at any step."""
    outs, reach = [], 0.0
    for t in range(q.shape[0]):
        state = state * torch.exp(g[t])[:, None, None]
        d = beta[t][:, None] * (v[t] - (state * k[t][:, None]).sum(-1))
        state = state + d[..., None] * k[t][:, None]
        outs.append((state * q[t][:, None]).sum(-1) / D ** 0.5)
        reach = max(reach, float((state.detach().abs() * q[t].detach().abs()[:, None]).sum(-1).max()) / D ** 0.5)
    return torch.stack(outs), state, reach


def inputs(lens, steps, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    T = sum(lens) + steps * len(lens)
    c = dict(qk=n(T, 2 * H * D).to(dtype), v=n(T, HV, D).to(dtype), a=n(T, HV).to(dtype), b=n(T, HV),
             a_log=-1 - torch.rand(HV, generator=g), dt_bias=torch.rand(HV, generator=g),
             qw=1 + 0.1 * n(D), kw=1 + 0.1 * n(D), freq=torch.exp(-9.0 * torch.arange(D // 2) / (D // 2)))
    return c


@pytest.mark.parametrize("cache,half", [(torch.float16, 2.0 ** -11), (torch.bfloat16, 2.0 ** -8), (torch.float8_e4m3fn, 2.0 ** -4)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_prompt_and_single_tokens_on_the_cache(cache, half, dtype):
    """Each call rounds the states it leaves once, by at most `half` of a value;
    the rule hands an error on without growing it (its transition is a decay of
    at most 1 times I - beta k k^T with a unit k), so after n calls an output is
    off by at most n half (|S| |q|) / sqrt(D), beside the calls' own arithmetic:
    the rotation's and the output's rounding to 16 bits and the prompt's chunked
    form, whose bars (4e-3 of the largest output) the forward pass's tests hold."""
    from gated_delta_rule_token_amd import api
    lens, steps = [150, 1, 70], 5
    c = inputs(lens, steps, dtype, 7)
    B, T0 = len(lens), sum(lens)
    slab = api.packed_slab(6, HV, D, D, cache)
    before = slab.data.clone()
    slots = torch.tensor([4, 0, 5], dtype=torch.int32, device="cuda")
    dev = {n: t.cuda() for n, t in c.items()}
    start = [0, lens[0], lens[0] + lens[1]]
    pos0 = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    gates = dict(update_rule="gated_delta", gate_activation="qwen", beta_activation="sigmoid", qk_l2_norm=True,
                 a_log=dev["a_log"], dt_bias=dev["dt_bias"])

    def run(rows, pos, **kw):
        wide = dev["qk"][rows]
        n = wide.shape[0]
        q, k = wide[:, : H * D].view(n, H, D), wide[:, H * D:].view(n, H, D)
        r = api.qk_rotary(q, k, pos.cuda(), dev["freq"], q_weight=dev["qw"], k_weight=dev["kw"])
        v, a, b = (dev[n][rows].clone() for n in "vab")  # 16-byte aligned
        return api.forward_packed(r.q, r.k, v, slab=slab, slot_ids=slots, gate=a, beta=b, **gates, **kw)

    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    got = [run(slice(0, T0), pos0, cu_seqlens=cu)]
    for i in range(steps):
        got.append(run(slice(T0 + i * B, T0 + (i + 1) * B), torch.tensor([n + i for n in lens], dtype=torch.int32)))
    torch.cuda.synchronize()
    for slot in (1, 2, 3):
        assert torch.equal(slab.data[slot].view(torch.uint8), before[slot].view(torch.uint8))

    d = {n: t.double() for n, t in c.items()}
    for r, n in enumerate(lens):
        rows = torch.cat([torch.arange(start[r], start[r] + n), T0 + r + B * torch.arange(steps)])
        angle = torch.arange(n + steps).double()[:, None] * d["freq"]
        q = unit(rotate(d["qk"][rows, : H * D].view(-1, H, D), d["qw"], angle)).repeat_interleave(HV // H, 1)
        k = unit(rotate(d["qk"][rows, H * D:].view(-1, H, D), d["kw"], angle)).repeat_interleave(HV // H, 1)
        g = -torch.exp(d["a_log"]) * torch.nn.functional.softplus(d["a"][rows] + d["dt_bias"])
        o, _, reach = recurrence(q, k, d["v"][rows], g, torch.sigmoid(d["b"][rows]), torch.zeros(HV, D, D).double())
        mine = torch.cat([got[0][start[r]: start[r] + n]] + [x[r: r + 1] for x in got[1:]]).cpu().double()
        own = 4e-3 * float(o.abs().max())
        err = (mine - o).abs()
        assert float(err[:n].max()) <= own, (r, float(err[:n].max()), own)
        for i in range(steps):
            bound = own + (i + 1) * half * reach
            assert float(err[n + i].max()) <= bound, (r, i, float(err[n + i].max()), bound)


def test_a_training_step_through_the_positions():
    """Gradients of a loss through rotation, gate fusion and recurrence, fp32
    activations, against autograd through the whole in 64 bits; the bar is the
    backward pass's (1e-4 of the largest gradient)."""
    from gated_delta_rule_token_amd import api
    lens = [70, 33]
    c = inputs(lens, 0, torch.float32, 9)
    T = sum(lens)
    dev = {n: t.cuda() for n, t in c.items()}
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    d_o = torch.randn(T, HV, D, generator=torch.Generator().manual_seed(3))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    q, k = dev["qk"][:, : H * D].view(T, H, D), dev["qk"][:, H * D:].view(T, H, D)
    rot = dict(q_weight=dev["qw"], k_weight=dev["kw"])
    r = api.qk_rotary(q, k, pos.cuda(), dev["freq"], **rot)
    decay, beta = api.gate(dev["a"], dev["dt_bias"], -torch.exp(dev["a_log"]), b=dev["b"], want_beta=True)
    o, _ = api.forward(r.q, r.k, dev["v"], gate=decay, beta=beta, cu_seqlens=cu, qk_l2_norm=True)
    g = api.backward(r.q, r.k, dev["v"], d_o.cuda(), gate=decay, beta=beta, cu_seqlens=cu, qk_l2_norm=True)
    d_qk = torch.empty_like(dev["qk"])
    gr = api.qk_rotary_backward(g.q, g.k, q, k, pos.cuda(), dev["freq"], **rot,
                                out=(d_qk[:, : H * D].view(T, H, D), d_qk[:, H * D:].view(T, H, D)))

    d = {n: t.double() for n, t in c.items()}
    leaves = {n: d[n].requires_grad_() for n in ("qk", "v", "qw", "kw")}
    outs, at = [], 0
    for n in lens:
        rows = slice(at, at + n)
        angle = torch.arange(n).double()[:, None] * d["freq"]
        qq = unit(rotate(leaves["qk"][rows, : H * D].view(-1, H, D), leaves["qw"], angle)).repeat_interleave(HV // H, 1)
        kk = unit(rotate(leaves["qk"][rows, H * D:].view(-1, H, D), leaves["kw"], angle)).repeat_interleave(HV // H, 1)
        gg = -torch.exp(d["a_log"]) * torch.nn.functional.softplus(d["a"][rows] + d["dt_bias"])
        outs.append(recurrence(qq, kk, leaves["v"][rows], gg, torch.sigmoid(d["b"][rows]), torch.zeros(HV, D, D).double())[0])
        at += n
    want = torch.cat(outs)
    plain = want.detach()
    assert float((o.cpu().double() - plain).abs().max()) <= 1e-4 * float(plain.abs().max())
    grads = torch.autograd.grad(want, list(leaves.values()), d_o.double())
    for name, ref, mine in zip(leaves, grads, (d_qk, g.v, gr.q_weight, gr.k_weight)):
        assert float((mine.cpu().double() - ref).abs().max()) <= 1e-4 * float(ref.abs().max()), name


def test_two_streams_at_once():
    """The same calls on two streams, each with its own tensors and workspace,
    give what they give alone."""
    from gated_delta_rule_token_amd import api
    sets = []
    for seed in (1, 2):
        c = {n: t.cuda() for n, t in inputs([300], 0, torch.bfloat16, seed).items()}
        q, k = c["qk"][:, : H * D].view(-1, H, D), c["qk"][:, H * D:].view(-1, H, D)
        pos = torch.arange(300, dtype=torch.int32, device="cuda")
        slot = torch.tensor([0], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
        sets.append((c, q, k, pos, slot, cu))
    torch.cuda.synchronize()

    def run(s):
        c, q, k, pos, slot, cu = s
        slab = api.packed_slab(1, HV, D, D, torch.float8_e4m3fn)
        r = api.qk_rotary(q, k, pos, c["freq"], q_weight=c["qw"], k_weight=c["kw"])
        o = api.forward_packed(r.q, r.k, c["v"], slab=slab, slot_ids=slot, gate=c["a"], beta=c["b"], cu_seqlens=cu,
                               a_log=c["a_log"], dt_bias=c["dt_bias"], gate_activation="qwen", beta_activation="sigmoid",
                               qk_l2_norm=True)
        g = api.qk_rotary_backward(r.q, r.k, q, k, pos, c["freq"], q_weight=c["qw"], k_weight=c["kw"])
        return o, slab.data.view(torch.uint8), api.state_unpack(slab, slot), *g

    alone = [run(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    together = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                together[i].append(run(sets[i]))
    torch.cuda.synchronize()
    for want, got in zip(alone, together):
        for one in got:
            assert all(torch.equal(a, b) for a, b in zip(want, one))
