"""Checks of the training operators' binding that come before any device
access, so that host tensors reach them."""
import os
import re

import pytest
import torch

from gated_delta_rule_token_amd import api


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not os.path.exists(api.library_path()):
        from gated_delta_rule_token_amd import build
        build.build()


@pytest.mark.parametrize("group", [2 ** 31, 2 ** 32 + 8, -2 ** 32 + 8, 2 ** 40 + 64])
def test_norm_refuses_a_group_past_32_bits(group):
    """ctypes would hand the library the low 32 bits: a group of 8 columns for
    scales that were allocated for one group a row."""
    with pytest.raises(api.GDRError, match="group"):
        api.rms_norm(torch.zeros(4, 64), out_dtype=torch.float8_e4m3fn, group=group)


@pytest.mark.parametrize("value,fits", [(0, True), (2 ** 31 - 1, True), (-2 ** 31, True), (2 ** 31, False),
                                        (2 ** 32, False), (-2 ** 31 - 1, False)])
def test_sizes_handed_to_the_library_fit_32_bits(value, fits):
    if fits:
        assert api._int32(value, "size") == value
    else:
        with pytest.raises(api.GDRError, match="size"):
            api._int32(value, "size")


def test_no_kernel_that_no_call_launches():
    """The chains have kernels of their own only where the launch rule can
    choose them (keys of 65 to 128 in fp16 and fp32), and the norm's forward
    pass one form of rows for each width.  By the kernels' names in the library."""
    with open(api.library_path(), "rb") as f:
        code = f.read()
    instances = lambda kernel: set(re.findall(kernel + rb"ILi(\d+)E(DF16b|DF16_|f)", code))  # noqa: E731
    everything = {(dk, t) for dk in (b"64", b"128", b"256") for t in (b"DF16b", b"DF16_", b"f")}
    assert instances(rb"k_back_chains") == everything and instances(rb"k_back_grad") == everything
    assert instances(rb"k_back_states") == instances(rb"k_back_chain") == {(b"128", b"DF16_"), (b"128", b"f")}
    forms = set(re.findall(rb"6k_normI(?:DF16b|DF16_|f)+Li(\d+)ELi(\d+)E", code))
    assert (b"64", b"4") in forms and (b"256", b"1") not in forms
