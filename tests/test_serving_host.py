"""What the norm and rotation of q and k and the packed state cache refuse, on
the host: argument checks run before any HIP call, so fake aligned pointers
(and, for the binding, tensors that are not on a GPU) are enough."""
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


def _rotary(**over):
    r = api.RotaryArguments(tokens=16, heads_q=4, heads_k=2, head_dim=32, rotary_dim=16, axes=1, interleaved=0, norm=1,
                            dtype=api.F32, weight_dtype=api.F32, eps=1e-6, q_stride=128, k_stride=64, q=_fake(1),
                            k=_fake(2), q_weight=_fake(3), k_weight=_fake(4), positions=_fake(5), inv_freq=_fake(6))
    for name, value in over.items():
        setattr(r, name, value)
    return r


BAD_ROTARY = [
    ("tokens", dict(tokens=-1), api.GDR_E_INVALID), ("tokens_past_32_bits", dict(tokens=2 ** 31), api.GDR_E_INVALID),
    ("tokens_past_a_launch", dict(tokens=2 ** 28), api.GDR_E_INVALID),
    ("no_heads", dict(heads_q=0), api.GDR_E_INVALID), ("many_heads", dict(heads_q=65537), api.GDR_E_INVALID),
    ("dim", dict(head_dim=257), api.GDR_E_INVALID), ("odd_rotary", dict(rotary_dim=15), api.GDR_E_INVALID),
    ("no_rotary", dict(rotary_dim=0), api.GDR_E_INVALID), ("rotary_past_dim", dict(rotary_dim=34), api.GDR_E_INVALID),
    ("axes", dict(axes=5), api.GDR_E_INVALID), ("no_axes", dict(axes=0), api.GDR_E_INVALID),
    ("interleaved", dict(interleaved=2), api.GDR_E_INVALID), ("norm", dict(norm=-1), api.GDR_E_INVALID),
    ("dtype", dict(dtype=api.E4M3), api.GDR_E_INVALID), ("weight_dtype", dict(weight_dtype=api.F16), api.GDR_E_INVALID),
    ("eps", dict(eps=float("nan")), api.GDR_E_INVALID), ("negative_eps", dict(eps=-1.0), api.GDR_E_INVALID),
    ("no_q", dict(q=None), api.GDR_E_INVALID), ("no_k", dict(k=None), api.GDR_E_INVALID),
    ("k_without_heads", dict(heads_k=0), api.GDR_E_INVALID), ("no_positions", dict(positions=None), api.GDR_E_INVALID),
    ("no_inv_freq", dict(inv_freq=None), api.GDR_E_INVALID), ("q_misaligned", dict(q=_fake(1) + 2), api.GDR_E_INVALID),
    ("positions_misaligned", dict(positions=_fake(5) + 2), api.GDR_E_INVALID),
    ("stride_below_a_row", dict(q_stride=127), api.GDR_E_INVALID), ("k_stride_below", dict(k_stride=63), api.GDR_E_INVALID),
    ("huge_stride", dict(q_stride=2 ** 62), api.GDR_E_INVALID),
]


@pytest.mark.parametrize("name,over,status", BAD_ROTARY, ids=[b[0] for b in BAD_ROTARY])
def test_rotary_refuses(lib, name, over, status):
    r = _rotary(**over)
    assert lib.gdr_qk_rotary(ctypes.byref(r), _fake(10), 128, _fake(11), 64, None) == status, lib.gdr_last_error()
    assert lib.gdr_last_error() != b""
    assert lib.gdr_qk_rotary_backward(ctypes.byref(r), _fake(12), _fake(13), _fake(10), 128, _fake(11), 64, _fake(14),
                                      _fake(15), _fake(16), 1 << 20, None) == status


# (q_out, stride, k_out, stride) against q at 1 (16 rows of 512 bytes), k at 2 (of 256)
ROTARY_OUTS = [
    ("q_out_over_k", (_fake(2), 128, _fake(11), 64), api.GDR_E_ALIAS),
    ("q_out_a_row_late", (_fake(1) + 512, 128, _fake(11), 64), api.GDR_E_ALIAS),
    ("q_out_other_stride", (_fake(1), 256, _fake(11), 64), api.GDR_E_ALIAS),
    ("results_overlap", (_fake(10), 128, _fake(10) + 256, 64), api.GDR_E_ALIAS),
    ("k_out_over_weight", (_fake(10), 128, _fake(3), 64), api.GDR_E_ALIAS),
    ("k_out_over_positions", (_fake(10), 128, _fake(5), 64), api.GDR_E_ALIAS),
    ("result_stride_below", (_fake(10), 127, _fake(11), 64), api.GDR_E_INVALID),
    ("q_out_missing", (None, 128, _fake(11), 64), api.GDR_E_INVALID),
    ("k_out_missing", (_fake(10), 128, None, 64), api.GDR_E_INVALID),
    ("results_in_one_buffer_overlap", (_fake(10), 192, _fake(10) + 4 * 127, 192), api.GDR_E_ALIAS),
    ("results_in_one_buffer_wrap", (_fake(10) + 4 * 70, 192, _fake(10) + 4 * 7, 192), api.GDR_E_ALIAS),
]


@pytest.mark.parametrize("name,outs,status", ROTARY_OUTS, ids=[b[0] for b in ROTARY_OUTS])
def test_rotary_refuses_results(lib, name, outs, status):
    r = _rotary()
    assert lib.gdr_qk_rotary(ctypes.byref(r), *outs, None) == status, lib.gdr_last_error()


def test_rotary_in_place_and_shared_buffers_pass_the_checks(lib):
    """A call without tokens is checked like any other and launches nothing."""
    r = _rotary(tokens=0)
    assert lib.gdr_qk_rotary(ctypes.byref(r), _fake(1), 128, _fake(2), 64, None) == api.GDR_OK, lib.gdr_last_error()
    assert lib.gdr_qk_rotary(None, _fake(1), 128, _fake(2), 64, None) == api.GDR_E_INVALID


def _back(lib, r, **over):
    kw = dict(dqo=_fake(12), dko=_fake(13), dq=_fake(10), sq=128, dk=_fake(11), sk=64, dqw=_fake(14), dkw=_fake(15),
              ws=_fake(16), size=1 << 20)
    kw.update(over)
    return lib.gdr_qk_rotary_backward(ctypes.byref(r), kw["dqo"], kw["dko"], kw["dq"], kw["sq"], kw["dk"], kw["sk"],
                                      kw["dqw"], kw["dkw"], kw["ws"], kw["size"], None)


@pytest.mark.parametrize("over,status", [
    (dict(dqo=None), api.GDR_E_INVALID), (dict(dko=None), api.GDR_E_INVALID), (dict(dqw=None), api.GDR_E_INVALID),
    (dict(dkw=None), api.GDR_E_INVALID), (dict(dqo=_fake(12) + 2), api.GDR_E_INVALID),
    (dict(ws=None), api.GDR_E_WORKSPACE), (dict(size=8), api.GDR_E_WORKSPACE), (dict(ws=_fake(16) + 4), api.GDR_E_INVALID),
    (dict(dq=_fake(1)), api.GDR_E_ALIAS), (dict(dq=_fake(12)), api.GDR_E_ALIAS), (dict(dqw=_fake(15)), api.GDR_E_ALIAS),
    (dict(dk=_fake(16)), api.GDR_E_ALIAS), (dict(ws=_fake(2)), api.GDR_E_ALIAS),
])
def test_rotary_backward_refuses(lib, over, status):
    assert _back(lib, _rotary(), **over) == status, lib.gdr_last_error()


def test_rotary_backward_workspace(lib):
    n = ctypes.c_size_t(1)
    size = lambda **over: (lib.gdr_qk_rotary_backward_workspace_size(ctypes.byref(_rotary(**over)), ctypes.byref(n)),  # noqa: E731
                           n.value)
    assert size() == (api.GDR_OK, 2 * 32 * 4)
    assert size(k_weight=None) == (api.GDR_OK, 32 * 4)
    assert size(q_weight=None, k_weight=None) == (api.GDR_OK, 0)
    assert size(tokens=1 << 20)[1] > 2 * 32 * 4
    assert size(head_dim=0)[0] == api.GDR_E_INVALID
    assert lib.gdr_qk_rotary_backward_workspace_size(ctypes.byref(_rotary()), None) == api.GDR_E_INVALID


def _slab(**over):
    s = api.SlabPointers(_fake(30), _fake(31), api.E4M3)
    for name, value in over.items():
        setattr(s, name, value)
    return s


def _pack(lib, slab, **over):
    kw = dict(batch=4, heads=2, dv=16, dk=32, slots=8, states=_fake(32), ids=_fake(33))
    kw.update(over)
    head = (kw["batch"], kw["heads"], kw["dv"], kw["dk"], kw["slots"])
    byref = None if slab is None else ctypes.byref(slab)
    a = lib.gdr_state_pack(*head, kw["states"], kw["ids"], byref, None)
    assert lib.gdr_state_unpack(*head, byref, kw["ids"], kw["states"], None) == a
    return a


@pytest.mark.parametrize("slab,over,status", [
    (dict(dtype=api.F32), {}, api.GDR_E_INVALID), (dict(dtype=7), {}, api.GDR_E_INVALID),
    (dict(data=None), {}, api.GDR_E_INVALID), (dict(scale=None), {}, api.GDR_E_INVALID),
    (dict(dtype=api.F16), {}, api.GDR_E_INVALID), (dict(data=_fake(30) + 8), {}, api.GDR_E_INVALID),
    ({}, dict(batch=-1), api.GDR_E_INVALID), ({}, dict(heads=0), api.GDR_E_INVALID), ({}, dict(dk=257), api.GDR_E_INVALID),
    ({}, dict(dv=0), api.GDR_E_INVALID), ({}, dict(slots=-1), api.GDR_E_INVALID),
    ({}, dict(batch=2 ** 30, heads=2 ** 20), api.GDR_E_INVALID),
    ({}, dict(batch=2 ** 19, heads=32), api.GDR_E_INVALID), ({}, dict(states=None), api.GDR_E_INVALID),
    ({}, dict(ids=None), api.GDR_E_INVALID), ({}, dict(states=_fake(32) + 4), api.GDR_E_INVALID),
    ({}, dict(states=_fake(30)), api.GDR_E_ALIAS), ({}, dict(states=_fake(31) - 4096), api.GDR_E_ALIAS),
    ({}, dict(batch=0), api.GDR_OK), ({}, dict(slots=0), api.GDR_OK),
])
def test_pack_and_unpack_refuse(lib, slab, over, status):
    assert _pack(lib, _slab(**slab), **over) == status, lib.gdr_last_error()
    assert _pack(lib, None) == api.GDR_E_INVALID


def test_slot_ids_may_not_lie_in_what_is_written(lib):
    s = _slab()
    assert lib.gdr_state_pack(4, 2, 16, 32, 8, _fake(32), _fake(30), ctypes.byref(s), None) == api.GDR_E_ALIAS
    assert lib.gdr_state_unpack(4, 2, 16, 32, 8, ctypes.byref(s), _fake(32) + 64, _fake(32), None) == api.GDR_E_ALIAS


def _step(problem=(), tensors=()):
    p = api.Problem(total_tokens=4, batch=4, seq_len=1, num_heads_qk=2, num_heads_v=4, head_dim_k=128, head_dim_v=128,
                    num_slots=8, act_dtype=api.F16, gate_dtype=api.F32, update_rule=api.RULES["gated_delta"],
                    chunk_size=64)
    t = api.Tensors(q=_fake(1), k=_fake(2), v=_fake(3), o=_fake(4), gate=_fake(5), beta=_fake(6), slot_ids=_fake(7))
    for s, over in ((p, problem), (t, tensors)):
        for name, value in dict(over).items():
            setattr(s, name, value)
    return p, t


@pytest.mark.parametrize("name,problem,tensors,slab,status", [
    ("no_slots", dict(num_slots=0), dict(slot_ids=None), {}, api.GDR_E_INVALID),
    ("no_ids", (), dict(slot_ids=None), {}, api.GDR_E_INVALID),
    ("final_state", (), dict(final_state=_fake(9)), {}, api.GDR_E_INVALID),
    ("initial_state", (), dict(initial_state=_fake(9)), {}, api.GDR_E_INVALID),
    ("no_gate", (), dict(gate=None), {}, api.GDR_E_INVALID),
    ("fp32_slab", (), (), dict(dtype=api.F32), api.GDR_E_INVALID),
    ("scales_missing", (), (), dict(scale=None), api.GDR_E_INVALID),
    ("scales_of_16_bits", (), (), dict(dtype=api.BF16), api.GDR_E_INVALID),
    ("data_misaligned", (), (), dict(data=_fake(30) + 8), api.GDR_E_INVALID),
    ("o_over_data", (), dict(o=_fake(30) + 8 * 4 * 128 * 128 - 256), {}, api.GDR_E_ALIAS),
    ("o_over_scales", (), dict(o=_fake(31)), {}, api.GDR_E_ALIAS),
    ("scales_over_q", (), (), dict(scale=_fake(1)), api.GDR_E_ALIAS),
    ("data_over_ids", (), dict(slot_ids=_fake(30)), {}, api.GDR_E_ALIAS),
    ("scales_over_data", (), (), dict(scale=_fake(30) + 64), api.GDR_E_ALIAS),
    ("decode_of_other_dims", dict(algo=2, head_dim_k=64), (), {}, api.GDR_E_UNSUPPORTED),
    ("more_than_a_launch", dict(batch=2 ** 20, total_tokens=2 ** 20), (), {}, api.GDR_E_INVALID),
    ("no_workspace", dict(seq_len=9, total_tokens=36), (), {}, api.GDR_E_WORKSPACE),
])
def test_forward_packed_refuses(lib, name, problem, tensors, slab, status):
    p, t = _step(problem, tensors)
    s = _slab(**slab)
    assert lib.gdr_forward_packed(ctypes.byref(p), ctypes.byref(t), ctypes.byref(s), None, 0, None) == status, \
        lib.gdr_last_error()
    assert lib.gdr_last_error() != b""


def test_forward_packed_workspace(lib):
    n = ctypes.c_size_t(1)

    def size(**problem):
        p, _ = _step(problem)
        assert lib.gdr_packed_workspace_size(ctypes.byref(p), ctypes.byref(n)) == api.GDR_OK
        return n.value

    state = 4 * 4 * 128 * 128 * 4
    assert size() == 0 and size(seq_len=8, total_tokens=32) == 0
    assert size(head_dim_k=64) == 0 and size(head_dim_k=256, head_dim_v=72) == 0  # one pass
    assert size(head_dim_k=72) == 0 and size(head_dim_k=1, head_dim_v=9) == 0
    assert size(batch=0, total_tokens=0, algo=1) == 0
    assert size(seq_len=9, total_tokens=36) >= state  # fp32 states in the workspace
    assert 0 < size(head_dim_k=9, seq_len=9, total_tokens=36) < state and size(algo=1) >= state
    long = size(seq_len=4096, total_tokens=4 * 4096)
    p, _ = _step(dict(seq_len=4096, total_tokens=4 * 4096, num_slots=4))
    assert long == api.workspace_size(p) + state + 256
    p, t = _step(dict(seq_len=4096, total_tokens=4 * 4096))
    call = lambda ws, size: lib.gdr_forward_packed(ctypes.byref(p), ctypes.byref(t), ctypes.byref(_slab()), ws, size, None)  # noqa: E731
    assert call(_fake(40), long - 1) == api.GDR_E_WORKSPACE
    assert call(_fake(40) + 8, long) == api.GDR_E_INVALID
    assert call(_fake(1), long) == api.GDR_E_ALIAS
    assert lib.gdr_forward_packed(ctypes.byref(p), None, ctypes.byref(_slab()), None, 0, None) == api.GDR_E_INVALID
    assert lib.gdr_forward_packed(ctypes.byref(p), ctypes.byref(t), None, None, 0, None) == api.GDR_E_INVALID


def test_binding_refuses_tensors_off_the_gpu():
    q, k = torch.zeros(4, 2, 8), torch.zeros(4, 1, 8)
    pos, freq = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(api.GDRError, match="GPU"):
        api.qk_rotary(q, k, pos, freq)
    with pytest.raises(api.GDRError, match="q must be"):
        api.qk_rotary(torch.zeros(4, 8), None, pos, freq)
    slab = api.packed_slab(3, 2, 4, 8, torch.float8_e4m3fn, device="cpu")
    assert float(slab.scale.float().max()) == 2.0 ** -100
    with pytest.raises(api.GDRError, match="GPU"):
        api.state_unpack(slab, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(api.GDRError, match="packed slab is"):
        api.packed_slab(3, 2, 4, 8, torch.float32, device="cpu")
    with pytest.raises(api.GDRError, match="GPU"):
        api.forward_packed(torch.zeros(1, 1, 8), torch.zeros(1, 1, 8), torch.zeros(1, 1, 8), slab=slab,
                           slot_ids=torch.zeros(1, dtype=torch.int32))
