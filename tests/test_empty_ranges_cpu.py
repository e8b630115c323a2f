"""Empty arrays share no byte with anything, wherever their pointers are: a
call with no rows is not refused for one inside another array.  (Without a
device such a call ends with a CUDA error, with one it does its work.)"""
import ctypes

import pytest

K = 1 << 24


@pytest.fixture(scope="module")
def lib():
    from bidirectional_mamba_ssm_b200 import build
    build.build()
    from bidirectional_mamba_ssm_b200 import _lib
    return _lib


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up pointers: only where nothing can be launched")


def test_a_prompt_call_without_rows(lib):
    d = lib.make_dims(2, 0, 2, 64, 128, 1)
    status = lib.library().bimamba_prompt_scan(
        ctypes.byref(d), 7 * K + 64, 7 * K + 128, 3 * K, 4 * K, 5 * K, None, 6 * K, 7 * K, 8 * K, 3, 9 * K, None,
        8 * K + 64, 11 * K, K, None)
    assert status not in (lib.BIMAMBA_ERR_INVALID, lib.BIMAMBA_ERR_WORKSPACE)


def test_a_norm_backward_without_rows(lib):
    status = lib.library().bimamba_layer_norm_backward(0, 64, 7 * K + 16, 7 * K + 32, 3 * K, 7 * K + 48, 7 * K + 64,
                                                       None, 8 * K + 16, 7 * K, 8 * K, 1, None, 0, None)
    assert status not in (lib.BIMAMBA_ERR_INVALID, lib.BIMAMBA_ERR_WORKSPACE)
