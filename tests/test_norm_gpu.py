"""GPU parity of the layer norm entry points (bimamba_layer_norm and
bimamba_layer_norm_backward) against the formulas in 64 bits.

Tolerances, fixed before the first run.  Every output is one rounding of an
fp32 value: bf16 outputs are off by at most 2^-8 of the value from that
rounding.  The fp32 value itself: with u = 2^-24, n columns and values of
order one, tree sums of at most 2^13 terms err by a few times log2(n) u of
their absolute sums, so 64 u of the largest magnitude of the row (column, for
dgamma and dbeta: times the number of rows for a sum in order) bounds every
element-wise step and sum here.
"""
import numpy as np
import pytest
import torch

from parity_util import to_np

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def lib():
    from bidirectional_mamba_ssm_b200 import _lib
    return _lib


def _draw(rows, cols, dtype, seed, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return {"x": (r(rows, cols) + offset * r(rows, 1)).to(dtype), "res": r(rows, cols).to(dtype),
            "gamma": 1.0 + 0.2 * r(cols), "beta": 0.1 * r(cols), "dy": r(rows, cols).to(dtype),
            "dsum": r(rows, cols).to(dtype)}


def _forward(d, residual, bias, eps=1e-5):
    h = to_np(d["x"]) + (to_np(d["res"]) if residual else 0.0)
    m = h.mean(1)
    s = 1.0 / np.sqrt(((h - m[:, None]) ** 2).mean(1) + eps)
    y = (h - m[:, None]) * s[:, None] * to_np(d["gamma"])
    return h, m, s, y + (to_np(d["beta"]) if bias else 0.0)


def _close(got, want, dtype, scale, what):
    """|got - want| <= one rounding of the value + 64 u of `scale`."""
    got, want = to_np(got), np.asarray(want)
    assert np.isfinite(got).all(), what
    tol = ROUND[dtype] * np.abs(want) * (1 + 2.0 ** -8) + 64 * U32 * scale
    bad = np.abs(got - want) - tol
    assert bad.max() <= 0, (what, bad.max(), float(np.abs(got - want).max()))


SHAPES = [(1, 8), (3, 64), (7, 256), (5, 520), (33, 1024), (2, 1032), (65, 2048), (9, 2056), (4, 4104),
          (3, 8192), (1501, 72)]


def _run_forward(lib, d, residual, bias, eps=1e-5):
    c = {k: v.cuda() for k, v in d.items()}
    y = torch.full_like(c["x"], float("nan"))
    s = torch.full_like(c["x"], float("nan")) if residual else None
    mean = torch.full((c["x"].shape[0],), float("nan"), device="cuda")
    rstd = torch.full_like(mean, float("nan"))
    lib.bimamba_layer_norm(c["x"], c["gamma"], c["beta"] if bias else None, y, mean, rstd,
                           residual=c["res"] if residual else None, sum_out=s, eps=eps)
    return y, s, mean, rstd


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(lib, rows, cols, dtype):
    for residual, bias in ((False, True), (True, False)):
        d = _draw(rows, cols, dtype, seed=rows + cols)
        h, m, s, y = _forward(d, residual, bias)
        gy, gs, gm, gr = _run_forward(lib, d, residual, bias)
        hmax = np.abs(h).max(1)
        _close(gm, m, torch.float32, hmax, "mean")
        _close(gr, s, torch.float32, s * (1 + hmax * s), "rstd")
        ymax = (np.abs(to_np(d["gamma"])).max() + 1) * (1 + hmax * s) ** 2
        _close(gy, y, dtype, ymax[:, None], "y")
        if residual:
            _close(gs, h, dtype, hmax[:, None], "sum")
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK


def test_forward_of_rows_far_from_zero(lib):
    """A mean 2^12 times the spread: one-pass sums of squares would lose every
    digit of the variance.  Values are exact in fp32."""
    g = torch.Generator().manual_seed(5)
    k = torch.randint(-64, 65, (6, 1024), generator=g).float() / 64
    d = {"x": k + 4096.0, "res": torch.zeros_like(k), "gamma": torch.ones(1024), "beta": torch.zeros(1024)}
    h, m, s, y = _forward(d, False, False)
    gy, _, gm, gr = _run_forward(lib, d, False, False)
    # the mean is off by at most a few half steps of 2^12 (2^-12 each), against a spread of ~0.6
    assert np.abs(to_np(gm) - m).max() <= 8 * 2.0 ** -12
    assert np.abs(to_np(gr) / s - 1).max() <= 1e-5      # (the shift enters squared)
    assert np.abs(to_np(gy) - y).max() <= 8 * 2.0 ** -12 * s.max() + 1e-4


def test_constant_rows_and_tiny_eps(lib):
    d = _draw(3, 256, torch.float32, seed=1)
    d["x"] = torch.full((3, 256), 2.5)
    gy, _, gm, gr = _run_forward(lib, d, False, True, eps=1e-5)
    assert torch.equal(gm.cpu(), torch.full((3,), 2.5))
    np.testing.assert_allclose(to_np(gr), 1e-5 ** -0.5, rtol=1e-6)
    np.testing.assert_array_equal(to_np(gy), np.broadcast_to(to_np(d["beta"]), (3, 256)))


def test_a_bad_row_stays_in_its_row(lib):
    d = _draw(9, 512, torch.bfloat16, seed=2)
    d["x"][4, 17] = float("nan")
    d["x"][6, 3] = float("inf")
    gy, _, _, _ = _run_forward(lib, d, False, True)
    fine = torch.isfinite(gy).all(1).cpu()
    assert fine.tolist() == [i not in (4, 6) for i in range(9)]


def _backward64(d, m, s, dsum, h=None):
    h = to_np(d["x"]) if h is None else h
    z = (h - m[:, None]) * s[:, None]
    dy = to_np(d["dy"])
    a = dy * to_np(d["gamma"])
    dx = s[:, None] * (a - a.mean(1, keepdims=True) - z * (a * z).mean(1, keepdims=True))
    return dx + (to_np(d["dsum"]) if dsum else 0.0), (dy * z).sum(0), dy.sum(0), z, a


def _run_backward(lib, d, mean, rstd, dsum, bias, stream=None):
    c = {k: v.cuda() for k, v in d.items()}
    dx = torch.full_like(c["x"], float("nan"))
    dg = torch.full((c["x"].shape[1],), float("nan"), device="cuda")
    db = torch.full_like(dg, float("nan")) if bias else None
    ws = lib.new_layer_norm_workspace(c["x"])
    lib.bimamba_layer_norm_backward(c["dy"], c["x"], c["gamma"], mean, rstd, dx, dg, db, ws,
                                    dsum=c["dsum"] if dsum else None)
    return dx, dg, db


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES + [(0, 64)])
def test_backward(lib, rows, cols, dtype):
    for dsum, bias in ((False, True), (True, False)):
        d = _draw(rows, cols, dtype, seed=rows + 3 * cols)
        _, m, s, _ = _forward(d, False, False)
        mean, rstd = (torch.from_numpy(v).float() for v in (m, s))
        dx, dg, db, z, a = _backward64(d, to_np(mean), to_np(rstd), dsum)
        gx, gg, gb = _run_backward(lib, d, mean.cuda(), rstd.cuda(), dsum, bias)
        if rows:
            scale = to_np(rstd) * (np.abs(a).max(1) + np.abs(z).max(1) * np.abs(a * z).mean(1)) + 1
            _close(gx, dx, dtype, scale[:, None], "dx")
        zmax, dmax = (np.abs(z).max(), np.abs(to_np(d["dy"])).max()) if rows else (0.0, 0.0)
        _close(gg, dg, torch.float32, rows * zmax * dmax / 8 + 1e-30, "dgamma")
        if bias:
            _close(gb, db, torch.float32, rows * dmax / 8 + 1e-30, "dbeta")
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK


def test_backward_matches_differences(lib):
    """d/de of sum(w y) + sum(v h) along random directions, from the forward
    entry point in fp32 (central differences)."""
    rows, cols, eps_fd = 6, 320, 2.0 ** -7
    d = _draw(rows, cols, torch.float32, seed=9)
    g = torch.Generator().manual_seed(10)

    def loss(x, gamma, beta):
        q = dict(d, x=x, gamma=gamma, beta=beta)
        y, s, _, _ = _run_forward(lib, q, True, True)
        return float((to_np(y) * to_np(d["dy"])).sum() + (to_np(s) * to_np(d["dsum"])).sum())

    y, s, mean, rstd = _run_forward(lib, d, True, True)
    gx, gg, gb = _run_backward(lib, dict(d, x=s.cpu()), mean, rstd, True, True)
    for name, grad in (("x", gx), ("gamma", gg), ("beta", gb)):
        v = torch.randn(d[name].shape, generator=g)
        v /= v.norm()
        args = {k: d[k] for k in ("x", "gamma", "beta")}
        up = loss(**dict(args, **{name: d[name] + eps_fd * v}))
        dn = loss(**dict(args, **{name: d[name] - eps_fd * v}))
        want = float((to_np(grad) * to_np(v)).sum())
        # truncation: third derivative times eps^2 / 6 (order one here, in a unit direction); rounding: the
        # loss sums 2 * 1920 products, each off by some u, over 2 eps
        tol = eps_fd ** 2 * (1 + abs(want)) + 64 * U32 * np.sqrt(2 * rows * cols) / (2 * eps_fd) * 4
        assert abs((up - dn) / (2 * eps_fd) - want) <= tol, (name, (up - dn) / (2 * eps_fd), want)


def test_backward_is_the_same_every_time(lib):
    d = _draw(2000, 256, torch.bfloat16, seed=3)
    _, m, s, _ = _forward(d, False, False)
    mean, rstd = (torch.from_numpy(v).float().cuda() for v in (m, s))
    one, two = (_run_backward(lib, d, mean, rstd, True, True) for _ in range(2))
    for p, q in zip(one, two):
        assert torch.equal(p, q)


def test_captured_and_on_another_stream(lib):
    """Forward and backward captured into one graph on a side stream, replayed
    on new inputs."""
    rows, cols = 130, 1024
    d = {k: v.cuda() for k, v in _draw(rows, cols, torch.bfloat16, seed=4).items()}
    y, s, dx = (torch.empty_like(d["x"]) for _ in range(3))
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
    dg, db = (torch.empty(cols, device="cuda") for _ in range(2))
    ws = lib.new_layer_norm_workspace(d["x"])

    def both(stream=None):
        lib.bimamba_layer_norm(d["x"], d["gamma"], d["beta"], y, mean, rstd, residual=d["res"], sum_out=s,
                               stream=stream)
        lib.bimamba_layer_norm_backward(d["dy"], s, d["gamma"], mean, rstd, dx, dg, db, ws, dsum=d["dsum"],
                                        stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    new = _draw(rows, cols, torch.bfloat16, seed=40)
    for k in d:
        d[k].copy_(new[k])
    graph.replay()
    got = [t.clone() for t in (y, s, mean, rstd, dx, dg, db)]
    both()
    for p, q in zip(got, (y, s, mean, rstd, dx, dg, db)):
        assert torch.equal(p, q)
    h, m, r, want = _forward(new, True, True)
    _close(got[0], want, torch.bfloat16, 8.0, "y")


def test_the_binding_refuses_missing_and_other_tensors(lib):
    x = torch.zeros((2, 8), device="cuda")
    v, r = torch.zeros(8, device="cuda"), torch.zeros(2, device="cuda")
    ws = lib.new_layer_norm_workspace(x)
    call = lambda dy, h=x: lib.bimamba_layer_norm_backward(dy, h, v, r, r, x.clone(), v.clone(), None, ws)  # noqa: E731
    for dy in (None, x[:, ::2], x.double(), x[:1], x.cpu()):
        with pytest.raises(lib.BimambaError):
            call(dy)
    with pytest.raises(lib.BimambaError):
        call(torch.zeros((), device="cuda"), torch.zeros((), device="cuda"))
