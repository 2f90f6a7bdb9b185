"""What the training operators and the norm refuse, on the host: argument
checks run before any HIP call, so fake aligned pointers are enough."""
import ctypes
import os

import pytest
import torch

from gated_delta_rule_token_amd import api

_BASE = 0x7F0000000000


def _fake(i):
    return _BASE + i * (1 << 28)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(api.library_path()):
        from gated_delta_rule_token_amd import build
        build.build()
    return api.load_library()


def _good(problem=(), tensors=(), grads=()):
    p = api.Problem(total_tokens=16, batch=2, seq_len=0, num_heads_qk=2, num_heads_v=4, head_dim_k=32, head_dim_v=32,
                    act_dtype=api.F32, gate_dtype=api.F32, update_rule=api.RULES["gated_delta"],
                    gate_activation=api.GATES["qwen"], beta_activation=api.BETAS["sigmoid"], qk_l2_norm=1, chunk_size=64)
    t = api.Tensors(q=_fake(1), k=_fake(2), v=_fake(3), gate=_fake(4), beta=_fake(5), a_log=_fake(6), dt_bias=_fake(7),
                    cu_seqlens=_fake(8), initial_state=_fake(9))
    g = api.GradientPointers(d_o=_fake(20), d_final_state=_fake(21), d_q=_fake(22), d_k=_fake(23), d_v=_fake(24),
                             d_gate=_fake(25), d_beta=_fake(26), d_initial_state=_fake(27), d_a_log=_fake(28),
                             d_dt_bias=_fake(29))
    for s, over in ((p, problem), (t, tensors), (g, grads)):
        for name, value in dict(over).items():
            setattr(s, name, value)
    return p, t, g


def _call(lib, p, t, g, ws=_fake(40), size=1 << 27):
    return lib.gdr_backward(ctypes.byref(p), ctypes.byref(t) if t is not None else None,
                            ctypes.byref(g) if g is not None else None, ws, size, None)


BAD = [
    ("erase_gate", dict(update_rule=4, gate_activation=0, beta_activation=0), (), (), api.GDR_E_UNSUPPORTED),
    ("decay_per_key", dict(decay_per_key=1), (), (), api.GDR_E_UNSUPPORTED),
    ("slab", dict(num_slots=4), dict(slot_ids=_fake(10), initial_state=None), (), api.GDR_E_UNSUPPORTED),
    ("too_many_chunks", dict(total_tokens=2**31 - 1, num_heads_qk=64, num_heads_v=128), (), (), api.GDR_E_INVALID),
    ("hv_not_multiple", dict(num_heads_v=3), (), (), api.GDR_E_INVALID),
    ("q_missing", (), dict(q=None), (), api.GDR_E_INVALID),
    ("gate_missing", (), dict(gate=None), (), api.GDR_E_INVALID),
    ("d_o_missing", (), (), dict(d_o=None), api.GDR_E_INVALID),
    ("d_q_missing", (), (), dict(d_q=None), api.GDR_E_INVALID),
    ("d_gate_missing", (), (), dict(d_gate=None), api.GDR_E_INVALID),
    ("d_beta_missing", (), (), dict(d_beta=None), api.GDR_E_INVALID),
    ("d_a_log_missing", (), (), dict(d_a_log=None), api.GDR_E_INVALID),
    ("d_gate_scale_without_it", (), (), dict(d_gate_scale=_fake(30)), api.GDR_E_INVALID),
    ("d_beta_for_gated", dict(update_rule=1, beta_activation=0), dict(beta=None), (), api.GDR_E_INVALID),
    ("misaligned", (), (), dict(d_v=_fake(24) + 8), api.GDR_E_INVALID),
    ("d_q_over_q", (), (), dict(d_q=_fake(1)), api.GDR_E_ALIAS),
    ("d_q_over_d_k", (), (), dict(d_q=_fake(23) + 256), api.GDR_E_ALIAS),
    ("d_v_over_d_o", (), (), dict(d_v=_fake(20)), api.GDR_E_ALIAS),
    ("d_initial_over_initial", (), (), dict(d_initial_state=_fake(9)), api.GDR_E_ALIAS),
    ("d_initial_partly_over_d_final", (), (), dict(d_initial_state=_fake(21) + 256), api.GDR_E_ALIAS),
    ("zero_rest_of_2", (), (), dict(zero_rest=2), api.GDR_E_INVALID),
    ("rows_too_wide", dict(num_heads_qk=140000, num_heads_v=140000, head_dim_k=64, head_dim_v=64), (), (), api.GDR_E_INVALID),
    ("workspace_over_q", (), dict(q=_fake(40) + 4096), (), api.GDR_E_ALIAS),
]


@pytest.mark.parametrize("name,problem,tensors,grads,status", BAD, ids=[b[0] for b in BAD])
def test_backward_refuses(lib, name, problem, tensors, grads, status):
    p, t, g = _good(problem, tensors, grads)
    assert _call(lib, p, t, g) == status, lib.gdr_last_error()
    assert lib.gdr_last_error() != b""


def test_backward_refuses_a_small_workspace_and_null_structs(lib):
    p, t, g = _good()
    n = ctypes.c_size_t(0)
    assert lib.gdr_backward_workspace_size(ctypes.byref(p), ctypes.byref(n)) == api.GDR_OK and n.value > 0
    assert _call(lib, p, t, g, size=n.value - 1) == api.GDR_E_WORKSPACE
    assert _call(lib, p, t, g, ws=None) == api.GDR_E_WORKSPACE
    assert _call(lib, p, None, g) == api.GDR_E_INVALID
    assert _call(lib, p, t, None) == api.GDR_E_INVALID
    assert lib.gdr_backward_workspace_size(ctypes.byref(p), None) == api.GDR_E_INVALID


def test_backward_workspace_grows_with_the_call(lib):
    sizes = []
    for T, rule in ((16, "linear"), (16, "gated_delta"), (4096, "gated_delta"), (40960, "gated_delta")):
        p, _, _ = _good(dict(total_tokens=T, update_rule=api.RULES[rule], gate_activation=0, beta_activation=0))
        sizes.append(api.backward_workspace_size(p))
    assert sizes == sorted(set(sizes))
    p, _, _ = _good(dict(total_tokens=1 << 20, num_heads_qk=32, num_heads_v=32, head_dim_k=128, head_dim_v=128))
    assert api.backward_workspace_size(p) > 1 << 36  # counted in 64 bits


def _gate(lib, **over):
    kw = dict(count=64, heads=4, dtype=api.F32, a=_fake(1), dt_bias=_fake(2), scale=_fake(3), b=_fake(4), dd=_fake(5),
              de=_fake(6), da=_fake(7), db=_fake(8), dbias=_fake(9), dscale=_fake(10), ws=_fake(11), size=1 << 20)
    kw.update(over)
    return lib.gdr_gate_backward(kw["count"], kw["heads"], kw["dtype"], kw["a"], kw["dt_bias"], kw["scale"], kw["b"],
                                 kw["dd"], kw["de"], kw["da"], kw["db"], kw["dbias"], kw["dscale"], kw["ws"],
                                 kw["size"], None)


@pytest.mark.parametrize("over,status", [
    (dict(count=-1), api.GDR_E_INVALID), (dict(heads=0), api.GDR_E_INVALID), (dict(count=65), api.GDR_E_INVALID),
    (dict(dtype=3), api.GDR_E_INVALID), (dict(a=None), api.GDR_E_INVALID), (dict(dd=None), api.GDR_E_INVALID),
    (dict(da=None), api.GDR_E_INVALID), (dict(dbias=None), api.GDR_E_INVALID), (dict(b=None), api.GDR_E_INVALID),
    (dict(db=None), api.GDR_E_INVALID), (dict(de=None), api.GDR_E_INVALID), (dict(a=_fake(1) + 2), api.GDR_E_INVALID),
    (dict(ws=None), api.GDR_E_WORKSPACE), (dict(size=4), api.GDR_E_WORKSPACE), (dict(da=_fake(1)), api.GDR_E_ALIAS),
    (dict(dscale=_fake(9)), api.GDR_E_ALIAS), (dict(count=4 * 70000, heads=70000), api.GDR_E_INVALID),
])
def test_gate_backward_refuses(lib, over, status):
    assert _gate(lib, **over) == status, lib.gdr_last_error()


def _norm(lib, **over):
    kw = dict(rows=8, width=64, dtype=api.BF16, wdtype=api.BF16, out=api.E4M3, group=0, eps=1e-6, x=_fake(1),
              residual=_fake(2), weight=_fake(3), y=_fake(4), scale=_fake(5), rout=_fake(6), inv=_fake(7))
    kw.update(over)
    return lib.gdr_rms_norm(kw["rows"], kw["width"], kw["dtype"], kw["wdtype"], kw["out"], kw["group"], kw["eps"],
                            kw["x"], kw["residual"], kw["weight"], kw["y"], kw["scale"], kw["rout"], kw["inv"], None)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), api.GDR_E_INVALID), (dict(rows=1 << 31), api.GDR_E_INVALID), (dict(width=0), api.GDR_E_INVALID),
    (dict(width=32769), api.GDR_E_UNSUPPORTED), (dict(dtype=api.E4M3), api.GDR_E_INVALID),
    (dict(wdtype=api.F16), api.GDR_E_INVALID), (dict(out=api.F16), api.GDR_E_INVALID),
    (dict(group=4), api.GDR_E_INVALID), (dict(group=96), api.GDR_E_INVALID), (dict(group=1024), api.GDR_E_INVALID),
    (dict(group=64, out=api.BF16, scale=None), api.GDR_E_INVALID), (dict(eps=-1.0), api.GDR_E_INVALID),
    (dict(eps=float("nan")), api.GDR_E_INVALID), (dict(x=None), api.GDR_E_INVALID), (dict(y=None), api.GDR_E_INVALID),
    (dict(scale=None), api.GDR_E_INVALID), (dict(out=api.BF16), api.GDR_E_INVALID),
    (dict(residual=None), api.GDR_E_INVALID), (dict(rout=None), api.GDR_E_INVALID),
    (dict(x=_fake(1) + 2), api.GDR_E_INVALID), (dict(y=_fake(1)), api.GDR_E_ALIAS),
    (dict(rout=_fake(1)), api.GDR_E_ALIAS), (dict(rout=_fake(2) + 64), api.GDR_E_ALIAS),
    (dict(rout=_fake(4)), api.GDR_E_ALIAS),
])
def test_norm_refuses(lib, over, status):
    assert _norm(lib, **over) == status, lib.gdr_last_error()


def _norm_back(lib, **over):
    kw = dict(rows=8, width=64, dtype=api.F16, wdtype=api.F32, dy=_fake(1), x=_fake(2), weight=_fake(3), inv=_fake(4),
              dres=_fake(5), dx=_fake(6), dw=_fake(7), ws=_fake(8), size=1 << 20)
    kw.update(over)
    return lib.gdr_rms_norm_backward(kw["rows"], kw["width"], kw["dtype"], kw["wdtype"], kw["dy"], kw["x"], kw["weight"],
                                     kw["inv"], kw["dres"], kw["dx"], kw["dw"], kw["ws"], kw["size"], None)


@pytest.mark.parametrize("over,status", [
    (dict(width=0), api.GDR_E_INVALID), (dict(width=40000), api.GDR_E_UNSUPPORTED), (dict(dy=None), api.GDR_E_INVALID),
    (dict(inv=None), api.GDR_E_INVALID), (dict(dx=None), api.GDR_E_INVALID), (dict(dw=None), api.GDR_E_INVALID),
    (dict(weight=None), api.GDR_E_INVALID), (dict(ws=None), api.GDR_E_WORKSPACE), (dict(size=64), api.GDR_E_WORKSPACE),
    (dict(dx=_fake(1)), api.GDR_E_ALIAS), (dict(dx=_fake(5)), api.GDR_E_ALIAS), (dict(wdtype=api.BF16), api.GDR_E_INVALID),
    (dict(dx=_fake(6) + 8), api.GDR_E_INVALID),
])
def test_norm_backward_refuses(lib, over, status):
    assert _norm_back(lib, **over) == status, lib.gdr_last_error()


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 8)
    for call in (lambda: api.backward(x, x, x, x, update_rule="linear"),
                 lambda: api.gate_backward(x, x[0, 0], x[0, 0], x),
                 lambda: api.rms_norm(x),
                 lambda: api.rms_norm_backward(x, x, None, x[..., 0])):
        with pytest.raises(api.GDRError, match="GPU"):
            call()
