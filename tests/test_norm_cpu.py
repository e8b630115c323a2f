"""Argument checks of the layer norm entry points: found on the host, before
anything touches a device."""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from bidirectional_mamba_ssm_b200 import build
    build.build()
    from bidirectional_mamba_ssm_b200 import _lib
    return _lib


K = 1 << 20


def _forward(lib, rows=4, cols=64, eps=1e-5, dtype=1, **over):
    a = dict(x=K, residual=None, gamma=2 * K, beta=None, y=3 * K, sum_out=None, mean=4 * K, rstd=5 * K)
    a.update(over)
    return lib.library().bimamba_layer_norm(rows, cols, a["x"], a["residual"], a["gamma"], a["beta"], eps,
                                            a["y"], a["sum_out"], a["mean"], a["rstd"], dtype, None)


def test_forward_refusals(lib):
    bad, no = lib.BIMAMBA_ERR_INVALID, lib.BIMAMBA_ERR_UNSUPPORTED
    assert _forward(lib, rows=-1) == bad
    assert _forward(lib, cols=0) == bad
    assert _forward(lib, dtype=2) == bad
    assert _forward(lib, cols=60) == no
    assert _forward(lib, cols=8200) == no
    assert _forward(lib, rows=1 << 31) == no
    assert _forward(lib, eps=-1e-5) == bad
    assert _forward(lib, eps=float("nan")) == bad
    for k in ("x", "gamma", "y", "mean", "rstd"):
        assert _forward(lib, **{k: None}) == bad, k
    assert _forward(lib, residual=6 * K) == bad             # a residual needs sum_out
    assert _forward(lib, sum_out=6 * K) == bad              # and sum_out a residual
    assert _forward(lib, y=3 * K + 8) == bad                # misaligned
    assert _forward(lib, y=K) == bad                        # y over x
    assert _forward(lib, mean=3 * K + 16) == bad            # statistics inside y
    assert _forward(lib, residual=6 * K, sum_out=6 * K) == bad
    assert _forward(lib, rows=0) == lib.BIMAMBA_OK


def _backward(lib, rows=4, cols=64, dtype=1, ws=9 * K, wsz=K, **over):
    a = dict(dy=K, h=2 * K, gamma=3 * K, mean=4 * K, rstd=5 * K, dsum=None, dx=6 * K, dgamma=7 * K,
             dbeta=8 * K)
    a.update(over)
    return lib.library().bimamba_layer_norm_backward(
        rows, cols, a["dy"], a["h"], a["gamma"], a["mean"], a["rstd"], a["dsum"], a["dx"], a["dgamma"],
        a["dbeta"], dtype, ws, wsz, None)


def test_backward_refusals(lib):
    bad, no = lib.BIMAMBA_ERR_INVALID, lib.BIMAMBA_ERR_UNSUPPORTED
    assert _backward(lib, rows=-1) == bad
    assert _backward(lib, cols=12) == no
    assert _backward(lib, dtype=-1) == bad
    for k in ("dy", "h", "gamma", "mean", "rstd", "dx", "dgamma"):
        assert _backward(lib, **{k: None}) == bad, k
    assert _backward(lib, dx=2 * K) == bad                  # dx over h
    assert _backward(lib, dsum=6 * K) == bad                # dsum over dx
    assert _backward(lib, dbeta=7 * K) == bad
    assert _backward(lib, h=2 * K + 2) == bad
    need = lib.bimamba_layer_norm_backward_workspace_bytes(4, 64)
    assert need > 0
    assert _backward(lib, wsz=need - 1) == lib.BIMAMBA_ERR_WORKSPACE
    assert _backward(lib, ws=None, wsz=0) == lib.BIMAMBA_ERR_WORKSPACE
    assert _backward(lib, ws=6 * K, wsz=K) == bad           # workspace over dx
    assert lib.bimamba_layer_norm_backward_workspace_bytes(4, 60) == 0


def test_the_binding_checks_its_tensors(lib):
    x = torch.zeros(2, 8)
    v, r = torch.zeros(8), torch.zeros(2)
    with pytest.raises(lib.BimambaError, match="CUDA tensor"):
        lib.bimamba_layer_norm(x, v, None, x.clone(), r, r.clone())
