"""Argument checks of the prompt scan and the token step: found on the host,
before anything touches a device."""
import ctypes

import pytest
import torch

import causal_ref as ref


@pytest.fixture(scope="module")
def lib():
    from bidirectional_mamba_ssm_b200 import build
    build.build()
    from bidirectional_mamba_ssm_b200 import _lib
    return _lib


K = 1 << 24
BASE = dict(xbc=K, dt=2 * K, A=3 * K, D=4 * K, conv_w=5 * K, conv_b=None, cu=6 * K, state=7 * K, tail=8 * K, pool=3,
            slots=9 * K, resume=None, y=10 * K, ws=11 * K, wsz=K)


def _prompt(lib, dims, **over):
    a = dict(BASE, **over)
    return lib.library().bimamba_prompt_scan(
        ctypes.byref(dims), a["xbc"], a["dt"], a["A"], a["D"], a["conv_w"], a["conv_b"], a["cu"], a["state"],
        a["tail"], a["pool"], a["slots"], a["resume"], a["y"], a["ws"], a["wsz"], None)


def _step(lib, dims, **over):
    a = dict(BASE, **over)
    return lib.library().bimamba_token_step(
        ctypes.byref(dims), a["xbc"], a["dt"], a["A"], a["D"], a["conv_w"], a["conv_b"], a["state"], a["tail"],
        a["pool"], a["slots"], a["y"], a["ws"], a["wsz"], None)


@pytest.mark.parametrize("call,length", [(_prompt, 40), (_step, 1)])
def test_refusals(lib, call, length):
    bad, no = lib.BIMAMBA_ERR_INVALID, lib.BIMAMBA_ERR_UNSUPPORTED
    dims = lambda **o: lib.make_dims(**dict(dict(batch=2, seqlen=length, heads=2, headdim=64, d_state=128,  # noqa: E731
                                                 dtype=1), **o))
    for over, status in [(dict(batch=-1), bad), (dict(heads=0), bad), (dict(dtype=5), bad), (dict(headdim=60), no),
                         (dict(headdim=136), no), (dict(d_state=100), no), (dict(ngroups=2), no),
                         (dict(d_conv=3), no), (dict(batch=65536), no)]:
        assert call(lib, dims(**over)) == status, over
    d = dims()
    for k in ("xbc", "dt", "A", "D", "conv_w", "state", "tail", "slots", "y"):
        assert call(lib, d, **{k: None}) == bad, k
        if k != "slots":
            assert call(lib, d, **{k: BASE[k] + 8}) == bad, k
    assert call(lib, d, slots=9 * K + 2) == bad
    assert call(lib, d, pool=0) == bad
    assert call(lib, d, ws=None) == lib.BIMAMBA_ERR_WORKSPACE
    assert call(lib, d, wsz=0) == lib.BIMAMBA_ERR_WORKSPACE
    assert call(lib, d, ws=11 * K + 4) == lib.BIMAMBA_ERR_WORKSPACE
    assert call(lib, d, y=K) == bad                          # y over xbc
    assert call(lib, d, y=7 * K + 64) == bad                 # y inside the states
    assert call(lib, d, tail=7 * K) == bad                   # the pools overlap
    assert call(lib, d, ws=8 * K, wsz=K) == bad              # the workspace inside the tails
    assert call(lib, dims(batch=0)) == lib.BIMAMBA_OK


def test_prompt_only_refusals(lib):
    d = lib.make_dims(2, 40, 2, 64, 128, torch.bfloat16)
    assert _prompt(lib, d, cu=None) == lib.BIMAMBA_ERR_INVALID
    assert _prompt(lib, d, cu=6 * K + 1) == lib.BIMAMBA_ERR_INVALID
    assert _prompt(lib, d, resume=6 * K + 6) == lib.BIMAMBA_ERR_INVALID
    assert _step(lib, d) == lib.BIMAMBA_ERR_INVALID          # a step is one token a row


def test_workspace_sizes(lib):
    for dt in (torch.float32, torch.bfloat16):
        a = lib.bimamba_prompt_workspace_bytes(lib.make_dims(4, 1000, 2, 64, 128, dt))
        b = lib.bimamba_prompt_workspace_bytes(lib.make_dims(40, 100000, 2, 64, 128, dt))
        assert 0 < a <= b
        assert lib.bimamba_token_step_workspace_bytes(lib.make_dims(300, 1, 2, 64, 128, dt)) >= 1200
    assert lib.bimamba_prompt_workspace_bytes(lib.make_dims(4, 1000, 2, 60, 128, 1)) == 0


def test_the_binding_checks_its_tensors(lib):
    d = ref.draw(4, 2, 2, 64, 128, torch.float32, seed=0, pool=2)
    y, ws = torch.zeros(4, 128), torch.zeros(256, dtype=torch.uint8)
    kw = dict(heads=2, headdim=64, d_state=128)
    cu = torch.tensor([0, 2, 4], dtype=torch.int32)
    with pytest.raises(lib.BimambaError, match="CUDA tensor"):
        lib.bimamba_prompt_scan(d["xbc"], d["dt"], d["A"], d["D"], d["conv_w"], d["conv_b"], cu, d["state"],
                                d["tail"], d["slots"], None, y, ws, **kw)
    with pytest.raises(lib.BimambaError, match="CUDA tensor"):
        lib.bimamba_token_step(d["xbc"], d["dt"], d["A"], d["D"], d["conv_w"], d["conv_b"], d["state"], d["tail"],
                               d["slots"], y, ws, **kw)
