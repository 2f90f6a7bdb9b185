"""The training operators and the norm, as they are measured: cases, inputs, plain forms and 64-bit results.

``own`` False computes each operator in its plain form (elementary torch
operations in 32 bits); True makes the framework's calls.

Operators (key ``op`` of a case):
  backward       gradients of the gated delta rule over ragged requests
  gate_backward  gradients of the gate fusion
  norm           root-mean-square norm, with the residual's addition, in 16/32 bits or in 8 bits with scales
  norm_backward  its gradients
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
CHUNK = 64
E4M3_MAX = 448.0

# the ragged batch the prefill workload draws (eight requests, 29,273 tokens)
RAGGED = "6945,2521,1351,2804,3690,6766,3978,1218"


def listed():
    back = dict(op="backward", rule="gated_delta", raw_gate=True, sigmoid=True, norm=True, init=False, final=False,
                per_token=False)
    return [
        # the smallest call: a unit test's or a first step's batch, where launches are all that counts
        dict(back, name="backward_tiny", lens="5,11", heads=2, heads_v=4, dk=32, dv=32, dtype="f32"),
        # fine-tuning on short replies: many requests shorter than a chunk, one of a single token
        dict(back, name="backward_short", dtype="bf16", heads=16, heads_v=32, dk=128, dv=128,
             lens="1,37,64,12,5,90,23,65,40,3,128,17,77,33,8,51,29,2,63,44,100,19,7,31"),
        # the ordinary training step: the ragged batch of the prefill workload, one layer
        dict(back, name="backward_ragged", dtype="bf16", heads=16, heads_v=32, dk=128, dv=128, lens=RAGGED,
             init=True, final=True),
        # training on one long document: decay and rate computed upstream, unit keys
        dict(back, name="backward_long", dtype="f16", heads=16, heads_v=16, dk=128, dv=128, lens="65536",
             raw_gate=False, sigmoid=False, norm=False),
        # odd sizes in fp32, an empty request, decay without retrieval
        dict(back, name="backward_odd", dtype="f32", heads=3, heads_v=9, dk=72, dv=40, lens="0,777,1,130",
             rule="gated", raw_gate=False, sigmoid=False, norm=False, init=True, final=True),
        # one optimizer step's gate gradients on a small batch
        dict(op="gate_backward", name="gate_backward_small", tokens=256, heads_v=32, dtype="f16", rate=False),
        # the same over a long batch, with the rate's gradient
        dict(op="gate_backward", name="gate_backward_large", tokens=65536, heads_v=32, dtype="bf16", rate=True),
        # serving: the decode batch's rows before an 8-bit projection
        dict(op="norm", name="norm_decode_8bit", rows=256, width=2048, dtype="bf16", weight="bf16", residual=True,
             eight=True, group=0),
        # prefill rows before an 8-bit projection, a scale for each 128 columns
        dict(op="norm", name="norm_prefill_8bit", rows=29273, width=4096, dtype="bf16", weight="bf16", residual=True,
             eight=True, group=128),
        # the norm of every head's output after the recurrence
        dict(op="norm", name="norm_heads", rows=29273 * 32, width=128, dtype="f16", weight="f32", residual=False,
             eight=False, group=0),
        # training: the gradients of the layer's input norm
        dict(op="norm_backward", name="norm_backward_train", rows=29273, width=2048, dtype="bf16", weight="bf16",
             residual=True),
        # an odd width in fp32
        dict(op="norm_backward", name="norm_backward_odd", rows=1217, width=1001, dtype="f32", weight="f32",
             residual=False),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["backward", "backward", "backward", "gate_backward", "norm", "norm", "norm_backward"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op == "gate_backward":
        return dict(op=op, tokens=_spread(rng, 1, 65536), heads_v=_spread(rng, 1, 64), dtype=dtype,
                    rate=rng.random() < 0.6)
    if op != "backward":
        width = _spread(rng, 32, 8192)
        if rng.random() < 0.5:
            width = max(32, width // 64 * 64)
        rows = _spread(rng, 1, min(400000, 29273 * 4096 // width))
        weight = rng.choice([dtype, "f32"])
        case = dict(op=op, rows=rows, width=width, dtype=dtype, weight=weight, residual=rng.random() < 0.6)
        if op == "norm":
            case["eight"] = rng.random() < 0.5
            case["group"] = rng.choice([0, 64, 128]) if case["eight"] else 0
        return case
    dk = rng.choice([64, 128, 128, 128, _spread(rng, 8, 256)])
    dv = dk if rng.random() < 0.6 else rng.choice([64, 128, _spread(rng, 8, 256)])
    heads = _spread(rng, 1, 16)
    heads_v = heads * rng.choice([1, 2, 4])
    most = min(32768, 65536 * 16 * 128 * 128 // (heads_v * max(dk, 64) * max(dv, 64)))
    total = _spread(rng, 1, max(1, most))
    batch = _spread(rng, 1, 48)
    cuts = sorted(rng.randint(0, total) for _ in range(batch - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    rule = rng.choice(["gated_delta", "gated_delta", "gated_delta", "delta", "gated", "linear"])
    decays, rate = rule in ("gated_delta", "gated"), rule in ("gated_delta", "delta")
    return dict(op=op, lens=",".join(map(str, lens)), heads=heads, heads_v=heads_v, dk=dk, dv=dv, dtype=dtype, rule=rule,
                raw_gate=decays and rng.random() < 0.5, sigmoid=rate and rng.random() < 0.5,
                norm=rate or rng.random() < 0.5, init=rng.random() < 0.5, final=rng.random() < 0.5,
                per_token=rate and heads_v > 1 and rng.random() < 0.3)


def _rules(case):
    return case["rule"] in ("gated_delta", "gated"), case["rule"] in ("gated_delta", "delta")


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo

    s = {"case": case}
    if case["op"] == "gate_backward":
        T, HV = case["tokens"], case["heads_v"]
        s.update(a=normal(T, HV, dtype=dtype), dt_bias=uniform(0, 1, HV), scale=-uniform(1, 16, HV),
                 d_decay=normal(T, HV, dtype=dtype), b=None, d_beta=None)
        if case["rate"]:
            s.update(b=normal(T, HV, dtype=dtype), d_beta=normal(T, HV, dtype=dtype))
        return s
    if case["op"] in ("norm", "norm_backward"):
        rows, width = case["rows"], case["width"]
        s.update(x=normal(rows, width, dtype=dtype), weight=(1 + normal(width, std=0.1)).to(DTYPES[case["weight"]]))
        if case["op"] == "norm":
            s["residual"] = normal(rows, width, std=2.0, dtype=dtype) if case["residual"] else None
        else:
            s["d_y"] = normal(rows, width, std=0.01, dtype=dtype)
            s["d_residual"] = normal(rows, width, std=0.01, dtype=dtype) if case["residual"] else None
            s["inv_rms"] = torch.rsqrt(s["x"].float().square().mean(-1) + 1e-6)  # as the forward pass left it
        return s
    lens = [int(n) for n in case["lens"].split(",")]
    T, B, H, HV, dk, dv = sum(lens), len(lens), case["heads"], case["heads_v"], case["dk"], case["dv"]
    decays, rate = _rules(case)
    silu = torch.nn.functional.silu  # q, k and v come out of a SiLU, and d_out has a part that all tokens share
    q, k, v = silu(normal(T, H, dk)), silu(normal(T, H, dk)), silu(normal(T, HV, dv))
    if not case["norm"]:
        k = k / k.norm(dim=-1, keepdim=True)
    s.update(lens=lens, q=q.to(dtype), k=k.to(dtype), v=v.to(dtype),
             d_out=(normal(T, HV, dv, std=0.1) + normal(1, HV, dv, std=0.1)).to(dtype),
             cu_seqlens=torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32),
             gate=None, a_log=None, dt_bias=None, beta=None, initial_state=None, d_final_state=None)
    if decays and case["raw_gate"]:
        s.update(gate=normal(T, HV, dtype=dtype), a_log=uniform(0, math.log(16.0), HV), dt_bias=uniform(0, 1, HV))
    elif decays:
        s["gate"] = -torch.nn.functional.softplus(normal(T, HV)) * uniform(1, 16, HV)
    if rate:
        b = normal(T, 1 if case["per_token"] else HV)
        s["beta"] = b if case["sigmoid"] else torch.sigmoid(b)
    if case["init"]:
        s["initial_state"] = normal(B, HV, dv, dk, std=0.05)
    if case["final"]:
        s["d_final_state"] = normal(B, HV, dv, dk, std=0.1)
    return s


# ------------------------------------------------------------------ plain forms

def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_gate_backward(s):
    x = s["a"].float() + s["dt_bias"]
    d = s["d_decay"].float()
    d_a = d * s["scale"] * torch.sigmoid(x)
    out = {"d_a": d_a.to(s["a"].dtype), "d_dt_bias": d_a.sum(0), "d_decay_scale": (d * _softplus(x)).sum(0)}
    if s["b"] is not None:
        r = torch.sigmoid(s["b"].float())
        out["d_b"] = (s["d_beta"].float() * r * (1 - r)).to(s["b"].dtype)
    return out


def _plain_norm(s):
    case, x = s["case"], s["x"]
    r = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    rf = r.float()
    y = rf * torch.rsqrt(rf.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
    out = {} if s["residual"] is None else {"residual": r}
    if not case["eight"]:
        return dict(out, y=y.to(x.dtype))
    width = y.shape[-1]
    group = case["group"] or width
    n = -(-width // group)
    yp = torch.nn.functional.pad(y, (0, n * group - width)).view(-1, n, group)
    amax = yp.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    q = (yp / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(-1, n * group)[:, :width]
    return dict(out, y=q.to(torch.float8_e4m3fn), scale=scale)


def _plain_norm_backward(s):
    x, dy, inv = s["x"].float(), s["d_y"].float(), s["inv_rms"][:, None]
    xh = x * inv
    wdy = dy * s["weight"].float()
    dx = inv * (wdy - xh * (wdy * xh).mean(-1, keepdim=True))
    if s["d_residual"] is not None:
        dx = dx + s["d_residual"].float()
    return {"d_x": dx.to(s["x"].dtype), "d_weight": (dy * xh).sum(0)}


def _unit_lower_inverse(n):
    """(I + n)^-1 for strictly lower triangular n of CHUNK rows: the product of I + (-n)^(2^i)."""
    eye = torch.eye(CHUNK, device=n.device)
    power, inv, reach = -n, eye - n, 2
    while reach < CHUNK:
        power = power @ power
        inv, reach = inv + inv @ power, 2 * reach
    return inv


def _plain_backward(s):
    """Chunked: everything of a chunk in batched products, one state handed from chunk to chunk."""
    case, lens, dtype = s["case"], s["lens"], s["q"].dtype
    decays, rate = _rules(case)
    H, HV, dk, dv, B = case["heads"], case["heads_v"], case["dk"], case["dv"], len(lens)
    T, R, dev = sum(lens), HV // H, s["q"].device
    scale = 1.0 / math.sqrt(dk)
    qf, kf = s["q"].float(), s["k"].float()
    one = torch.ones(T, H, 1, device=dev)
    rq = torch.rsqrt(qf.square().sum(-1, keepdim=True) + 1e-12) if case["norm"] else one
    rk = torch.rsqrt(kf.square().sum(-1, keepdim=True) + 1e-12) if case["norm"] else one
    qh, kh = qf * rq * scale, kf * rk
    g = torch.zeros(T, HV, device=dev)
    if decays and case["raw_gate"]:
        x, gs = s["gate"].float() + s["dt_bias"], -torch.exp(s["a_log"])
        g = gs * _softplus(x)
    elif decays:
        g = s["gate"].float()
    b = torch.ones(T, HV, device=dev)
    if rate:
        b = torch.sigmoid(s["beta"]) if case["sigmoid"] else s["beta"]
        b = b.expand(T, HV)

    # chunk table: token numbers (T stands for padding) and, for step i, each request's i-th chunk
    rows, at, starts = [], 0, []
    for n in lens:
        starts.append(len(rows))
        rows += [(at + c, min(CHUNK, n - c)) for c in range(0, n, CHUNK)]
        at += n
    counts = [-(-n // CHUNK) for n in lens]
    N = len(rows)
    first = torch.tensor([r[0] for r in rows], device=dev)[:, None]
    held = torch.tensor([r[1] for r in rows], device=dev)[:, None]
    pos = torch.arange(CHUNK, device=dev)[None]
    real = pos < held
    token = torch.where(real, first + pos, torch.full_like(pos, T))

    def chunks(x):  # (T, heads, ...) -> (N, HV, CHUNK, ...)
        x = torch.cat([x, x.new_zeros((1,) + x.shape[1:])])[token].transpose(1, 2)
        return x if x.shape[1] == HV else x.repeat_interleave(R, dim=1)

    q, k, v, do = chunks(qh), chunks(kh), chunks(s["v"].float()), chunks(s["d_out"].float())
    b, G = chunks(b[..., None]), chunks(g.double()).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=dev, dtype=torch.bool).tril()
    ex = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], torch.full((), -math.inf, device=dev,
                                                                                  dtype=torch.float64))).float()
    eG, eK = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    eC = torch.exp(G[..., -1]).float()[..., None, None]
    P = ex * (q @ k.transpose(-1, -2))
    L = (ex * (k @ k.transpose(-1, -2))).tril(-1) if rate else None
    if rate:
        inv = _unit_lower_inverse(b * L)
        U, W = inv @ (b * v), inv @ (b * eG * k)
    S, D = torch.empty(N, HV, dv, dk, device=dev), v.clone()
    state = torch.zeros(B, HV, dv, dk, device=dev) if s["initial_state"] is None else s["initial_state"].clone()
    steps = []
    for i in range(max(counts, default=0)):
        live = [r for r in range(B) if counts[r] > i]
        req = torch.tensor(live, device=dev)
        c = torch.tensor([starts[r] + i for r in live], device=dev)
        steps.append((req, c))
    for req, c in steps:
        S[c] = now = state[req]
        if rate:
            D[c] = U[c] - W[c] @ now.transpose(-1, -2)
        state[req] = eC[c] * now + (eK[c] * D[c]).transpose(-1, -2) @ k[c]
    dstate = torch.zeros_like(state) if s["d_final_state"] is None else s["d_final_state"].clone()
    dS, Y = torch.empty_like(S), P.transpose(-1, -2) @ do
    into = (eG * do).transpose(-1, -2) @ q
    for req, c in reversed(steps):
        dS[c] = now = dstate[req]
        Y[c] += eK[c] * (k[c] @ now.transpose(-1, -2))
        if rate:
            Y[c] = inv[c].transpose(-1, -2) @ Y[c]
        dstate[req] = eC[c] * now + into[c]
        if rate:
            dstate[req] -= (b[c] * eG[c] * Y[c]).transpose(-1, -2) @ k[c]
    F = (do @ D.transpose(-1, -2)).tril()
    dq0, dk0 = eG * (do @ S), eK * (D @ dS)
    u, w = (k * dk0).sum(-1), (q * dq0).sum(-1)
    M = F * P
    F = F * ex
    dq, dkk = dq0 + F @ k, dk0 + F.transpose(-1, -2) @ q
    out = {}
    if rate:
        X = (Y @ D.transpose(-1, -2)).tril(-1)
        row = -b * eG * (Y @ S)
        w = w + (k * row).sum(-1)
        M = M - X * L * b
        out["d_beta"] = (Y * (v - eG * (k @ S.transpose(-1, -2)))).sum(-1) - (X * L).sum(-1)
        X = X * ex * b
        dkk = dkk + row - (X + X.transpose(-1, -2)) @ k
        Y = b * Y

    def tokens(x):  # (N, HV, CHUNK, ...) -> (T, HV, ...)
        r = x.new_zeros((T,) + (HV,) + x.shape[3:])
        r[token[real]] = x.transpose(1, 2)[real]
        return r

    def unit(d, x, r):  # through the L2 norm, summed over the heads that share it
        d = tokens(d).view(T, H, R, dk).sum(2)
        return (r * (d - x * (x * d).sum(-1, keepdim=True) * r * r) if case["norm"] else d)

    out["d_q"], out["d_k"] = (scale * unit(dq, qf, rq)).to(dtype), unit(dkk, kf, rk).to(dtype)
    out["d_v"] = tokens(Y).to(dtype)
    if s["initial_state"] is not None:
        out["d_initial_state"] = dstate
    if decays:
        # rows t >= s of columns r < s
        across = (M.cumsum(-1) - M).flip(-2).cumsum(-2).flip(-2).diagonal(dim1=-2, dim2=-1)
        dg = tokens((eC[..., 0] * (dS * S).sum((-1, -2))[..., None]) + (u.cumsum(-1) - u)
                    + w.flip(-1).cumsum(-1).flip(-1) + across)
        if case["raw_gate"]:
            da = dg * gs * torch.sigmoid(x)
            out["d_gate"], out["d_dt_bias"], out["d_a_log"] = da.to(s["gate"].dtype), da.sum(0), (dg * g).sum(0)
        else:
            out["d_gate"] = dg
    if rate:
        db = tokens(out["d_beta"])
        db = db.sum(-1, keepdim=True) if case["per_token"] else db
        if case["sigmoid"]:
            r = torch.sigmoid(s["beta"])
            db = db * r * (1 - r)
        out["d_beta"] = db
    return out


# ------------------------------------------------------------------ the framework's calls

def _own_backward(s):
    from gated_delta_rule_token_amd import api
    case = s["case"]
    g = api.backward(s["q"], s["k"], s["v"], s["d_out"], gate=s["gate"], beta=s["beta"], a_log=s["a_log"],
                     dt_bias=s["dt_bias"], cu_seqlens=s["cu_seqlens"], initial_state=s["initial_state"],
                     d_final_state=s["d_final_state"], update_rule=case["rule"],
                     gate_activation="qwen" if case["raw_gate"] else "none",
                     beta_activation="sigmoid" if case["sigmoid"] else "none", qk_l2_norm=case["norm"])
    out = {"d_q": g.q, "d_k": g.k, "d_v": g.v, "d_gate": g.gate, "d_beta": g.beta, "d_a_log": g.a_log,
           "d_dt_bias": g.dt_bias, "d_initial_state": g.initial_state}
    return {name: t for name, t in out.items() if t is not None}


def _own_gate_backward(s):
    from gated_delta_rule_token_amd import api
    g = api.gate_backward(s["a"], s["dt_bias"], s["scale"], s["d_decay"], b=s["b"], d_beta=s["d_beta"])
    out = {"d_a": g.a, "d_b": g.b, "d_dt_bias": g.dt_bias, "d_decay_scale": g.decay_scale}
    return {name: t for name, t in out.items() if t is not None}


def _own_norm(s):
    from gated_delta_rule_token_amd import api
    case = s["case"]
    r = api.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=1e-6,
                     out_dtype=torch.float8_e4m3fn if case["eight"] else None, group=case["group"])
    out = {"y": r.y, "scale": r.scale, "residual": r.residual}
    return {name: t for name, t in out.items() if t is not None}


def _own_norm_backward(s):
    from gated_delta_rule_token_amd import api
    g = api.rms_norm_backward(s["d_y"], s["x"], s["weight"], s["inv_rms"], d_residual=s["d_residual"])
    return {"d_x": g.x, "d_weight": g.weight}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"backward": _own_backward, "gate_backward": _own_gate_backward, "norm": _own_norm,
                "norm_backward": _own_norm_backward}[op](state)
    return {"backward": _plain_backward, "gate_backward": _plain_gate_backward, "norm": _plain_norm,
            "norm_backward": _plain_norm_backward}[op](state)


# ------------------------------------------------------------------ work

def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "gate_backward":
        n = case["tokens"] * case["heads_v"]
        return {"bytes": n * e * (6 if case["rate"] else 3) + 16 * case["heads_v"],
                "flops": n * (16 if case["rate"] else 10)}
    if case["op"] in ("norm", "norm_backward"):
        n, w = case["rows"] * case["width"], case["width"] * SIZE[case["weight"]]
        if case["op"] == "norm_backward":
            return {"bytes": n * e * (4 if case["residual"] else 3) + 4 * case["rows"] + w + 4 * case["width"],
                    "flops": 10 * n}
        out = n * (1 if case["eight"] else e)
        if case["eight"]:
            out += 4 * case["rows"] * (-(-case["width"] // case["group"]) if case["group"] else 1)
        return {"bytes": n * e * (3 if case["residual"] else 1) + out + w, "flops": 6 * n}
    lens = [int(n) for n in case["lens"].split(",")]
    T, B, H, HV, dk, dv = sum(lens), len(lens), case["heads"], case["heads_v"], case["dk"], case["dv"]
    decays, rate = _rules(case)
    state = 4 * B * HV * dk * dv
    size = 4 * T * H * dk * e + 3 * T * HV * dv * e          # q, k and their gradients; v, d_out, d_v
    size += 2 * T * HV * (e if case["raw_gate"] else 4) if decays else 0
    size += 2 * T * (1 if case["per_token"] else HV) * 4 if rate else 0
    size += state * ((2 if case["init"] else 0) + (1 if case["final"] else 0))
    # per token and head, in units of dk * dv: the forward state again (write 2; decay 1; retrieve 2), the read-out's
    # gradient (2 into the state's, 2 into q's), the write's (2 into k's, 2 into the delta's), the retrieval's (2 + 2),
    # the decay's (1 on the state, 2 into the gate's)
    per = 10 + (6 if rate else 0) + (4 if decays else 0)
    return {"bytes": size, "flops": T * HV * dk * dv * per}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "backward":
        return _exact_backward(s) if max(int(n) for n in case["lens"].split(",")) <= 16384 else None
    f = {name: t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t for name, t in s.items()}
    if case["op"] == "gate_backward":
        x = f["a"] + f["dt_bias"]
        soft = torch.logaddexp(x, torch.zeros_like(x))
        d_a = f["d_decay"] * f["scale"] / (1 + torch.exp(-x))
        out = {"d_a": d_a, "d_dt_bias": d_a.sum(0), "d_decay_scale": (f["d_decay"] * soft).sum(0)}
        if f["b"] is not None:
            t = torch.exp(-f["b"].abs())
            out["d_b"] = f["d_beta"] * t / (1 + t) ** 2
        return out
    if case["op"] == "norm":
        out, r = {}, f["x"]
        if f["residual"] is not None:
            r = (r + f["residual"]).to(s["x"].dtype).double()
            out["residual"] = r
        y = r * f["weight"] / torch.sqrt((r * r).sum(-1, keepdim=True) / case["width"] + 1e-6)
        if not case["eight"]:
            return dict(out, y=y)
        group = case["group"] or case["width"]
        parts = y.split(group, dim=-1)
        scales = [p.abs().amax(-1, keepdim=True) / E4M3_MAX for p in parts]
        q = torch.cat([p / c for p, c in zip(parts, scales)], -1)
        return dict(out, y=q, scale=torch.cat(scales, -1))
    h = f["x"] * f["inv_rms"][:, None]
    t = f["d_y"] * f["weight"]
    dx = f["inv_rms"][:, None] * (t - h * ((t * h).sum(-1, keepdim=True) / case["width"]))
    return {"d_x": dx if f["d_residual"] is None else dx + f["d_residual"], "d_weight": (f["d_y"] * h).sum(0)}


def _exact_backward(s):
    """Token by token, every request side by side, states kept at every 64th token."""
    case, lens = s["case"], s["lens"]
    decays, rate = _rules(case)
    H, HV, dk, dv, B = case["heads"], case["heads_v"], case["dk"], case["dv"], len(lens)
    T, R, dev, top, keep = sum(lens), HV // H, s["q"].device, max(lens), 64
    qf, kf = s["q"].double(), s["k"].double()
    nq = torch.sqrt((qf * qf).sum(-1, keepdim=True) + 1e-12) if case["norm"] else torch.ones_like(qf[..., :1])
    nk = torch.sqrt((kf * kf).sum(-1, keepdim=True) + 1e-12) if case["norm"] else torch.ones_like(kf[..., :1])
    if decays and case["raw_gate"]:
        x = s["gate"].double() + s["dt_bias"].double()
        coef = -torch.exp(s["a_log"].double())
        g = coef * torch.logaddexp(x, torch.zeros_like(x))
    else:
        g = s["gate"].double() if decays else qf.new_zeros(T, HV)
    raw = s["beta"].double() if rate else qf.new_ones(T, 1)
    b = (1 / (1 + torch.exp(-raw)) if case["sigmoid"] else raw).expand(T, HV)
    ends = torch.tensor(lens, device=dev).cumsum(0)
    begin = (ends - torch.tensor(lens, device=dev))[:, None]
    when = torch.arange(top, device=dev)[None]
    inside = when < torch.tensor(lens, device=dev)[:, None]
    where = torch.where(inside, begin + when, torch.full_like(when, T))       # (B, top)

    def padded(x):
        x = x.repeat_interleave(HV // x.shape[1], 1) if x.shape[1] != HV else x
        return torch.cat([x, x.new_zeros((1,) + x.shape[1:])])[where.T]       # (top, B, HV, ...)

    q, k, v, do = padded(qf / nq / math.sqrt(dk)), padded(kf / nk), padded(s["v"].double()), padded(s["d_out"].double())
    a, b = torch.exp(padded(g))[..., None, None], padded(b)[..., None]
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(a[..., 0, 0]), torch.zeros_like(a[..., 0, 0])
    S = q.new_zeros(B, HV, dv, dk) if s["initial_state"] is None else s["initial_state"].double()

    def step(S, t):
        A = a[t] * S
        miss = v[t] - (A * k[t][..., None, :]).sum(-1) if rate else v[t]
        d = b[t] * miss if rate else v[t]
        return A, miss, d, A + d[..., :, None] * k[t][..., None, :]

    saved = []
    for t in range(top):
        if t % keep == 0:
            saved.append(S)
        S = step(S, t)[3]
    dS = torch.zeros_like(S) if s["d_final_state"] is None else s["d_final_state"].double()
    for block in range(len(saved) - 1, -1, -1):
        S, past = saved[block], []
        for t in range(block * keep, min(top, (block + 1) * keep)):
            past.append(step(S, t))
            S = past[-1][3]
        for t in range(min(top, (block + 1) * keep) - 1, block * keep - 1, -1):
            A, miss, d, S = past[t - block * keep]
            dS = dS + do[t][..., :, None] * q[t][..., None, :]
            dq[t] = (S * do[t][..., :, None]).sum(-2)
            dd = (dS * k[t][..., None, :]).sum(-1)
            dkk[t] = (dS * d[..., :, None]).sum(-2)
            if rate:
                db[t] = (dd * miss).sum(-1)
                dd = b[t] * dd
                dkk[t] -= (A * dd[..., :, None]).sum(-2)
                dS = dS - dd[..., :, None] * k[t][..., None, :]
            dvv[t] = dd
            dg[t] = (dS * A).sum((-1, -2))
            dS = a[t] * dS

    def flat(x):
        r = x.new_zeros((T,) + x.shape[2:])
        r[where[inside]] = x.transpose(0, 1)[inside]
        return r

    def heads(d, x, n):
        d = flat(d).view(T, H, R, dk).sum(2)
        return (d - x * (x * d).sum(-1, keepdim=True) / (n * n)) / n if case["norm"] else d

    dg, db = flat(dg), flat(db)
    out = {"d_q": heads(dq, qf, nq) / math.sqrt(dk), "d_k": heads(dkk, kf, nk), "d_v": flat(dvv)}
    if s["initial_state"] is not None:
        out["d_initial_state"] = dS
    if decays and case["raw_gate"]:
        da = dg * coef / (1 + torch.exp(-x))
        out.update(d_gate=da, d_dt_bias=da.sum(0), d_a_log=(dg * g).sum(0))
    elif decays:
        out["d_gate"] = dg
    if rate:
        db = db.sum(-1, keepdim=True) if case["per_token"] else db
        t = torch.exp(-raw.abs())
        out["d_beta"] = db * t / (1 + t) ** 2 if case["sigmoid"] else db
    return out
