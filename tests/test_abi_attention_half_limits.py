"""Refusals of the attention half's operators and of the engine's mode for
8-bit activations that are answered on the host, before any CUDA call."""
import ctypes
import os
import re

import pytest

from inputs import CONFIGS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sf():
    import offloaded_fine_tuning_gb300 as sfp
    sfp.lib(build_if_needed=True)
    return sfp


@pytest.mark.parametrize("value", [3, -1, 2 ** 31 - 1, -2 ** 31])
def test_unknown_activation_mode_is_refused(sf, value):
    cfg = sf.make_config(CONFIGS["tiny"], offload_activations=value)
    h = ctypes.c_void_p()
    assert sf.lib().sf_init_model(ctypes.byref(cfg), ctypes.byref(h)) == sf.SF_EINVAL
    assert not h.value
    assert b"offload_activations" in sf.lib().sf_last_error(None)


A = 4096  # an aligned address that is never read: every call below is refused


@pytest.mark.parametrize("call,at,step", [
    ("op_attn_window_fwd", 2, 2), ("op_attn_window_bwd", 3, 2), ("op_attn_window_bwd", 4, 1),
    ("op_rmsnorm_fwd_save8", 3, 2), ("op_rmsnorm_fwd_load8", 4, 2), ("op_rmsnorm_bwd_load8", 3, 2),
    ("op_rmsnorm_bwd_load8", 8, 1)])
def test_arrays_between_their_elements_are_refused(sf, call, at, step):
    """lse, delta, rstd and dg start at a whole element of their type: between two
    of them the kernels' accesses would fault."""
    pointers, rest = {"op_attn_window_fwd": (3, (1, 16, 4, 2, 64, 8, 1)), "op_attn_window_bwd": (7, (1, 16, 4, 2, 64, 8, 1)),
                      "op_rmsnorm_fwd_save8": (6, (0, 4, 128, 1e-5)), "op_rmsnorm_fwd_load8": (6, (0, 4, 128, 1e-5)),
                      "op_rmsnorm_bwd_load8": (10, (0, 4, 128))}[call]
    p = [A] * pointers
    p[at] = A + step
    assert getattr(sf, call)(*p, *rest) == sf.SF_EINVAL


def test_header_lists_every_device_error():
    """Each code that a kernel can write is explained at sf_op_device_error, and a
    kernel that waited for nothing does not report a timeout."""
    src = lambda *p: open(os.path.join(ROOT, *p)).read()
    csrc = ("offloaded_fine_tuning_gb300", "csrc")
    codes = dict(re.findall(r"(kDev\w+) = (\d+)", src(*csrc, "sf_internal.h")))
    head = src("include", "sf.h")
    text = head[:head.index("int sf_op_device_error")].rsplit("/*", 1)[1]
    for value in codes.values():
        assert re.search(rf"\b{value}[,:]", text), value
    aligned = re.findall(r"if \(s0 & 1023u\) \{\s*if \(threadIdx.x == 0\) record_error\(err, (\w+)\)",
                         src(*csrc, "attention_tc.cu"))
    assert aligned == ["kDevSharedBase"] * 2
