"""Refusals of the attention half's operators and of the engine's mode for
8-bit activations that are answered on the host, before any CUDA call."""
import ctypes

import pytest

from inputs import CONFIGS


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
