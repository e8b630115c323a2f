"""The layer norm's backward pass where a group of warps takes more rows than
its ring of copies holds (3 for bf16, 2 for fp32), and a number of them that is
no multiple of the groups, for every layout (8, 4 and 2 rows a CTA, one of 8
warps, one of 16): each ring stage used again, each row's statistics
prefetched, the columns' sums over many rows.  Against the formulas in 64
bits; tolerances as in test_norm_gpu."""
import numpy as np
import pytest
import torch

from parity_util import to_np
from test_norm_gpu import _backward64, _close, _draw, _forward, _run_backward

pytestmark = pytest.mark.gpu

SHAPES = [(10007, 72), (7500, 256), (5003, 1024), (2501, 2048), (1301, 4096), (700, 8192), (601, 4104)]


@pytest.fixture(scope="module")
def lib():
    from bidirectional_mamba_ssm_b200 import _lib
    return _lib


def _inputs(rows, cols, dtype):
    d = _draw(rows, cols, dtype, seed=rows + 5 * cols)
    _, m, s, _ = _forward(d, False, False)
    return d, *(torch.from_numpy(v).float() for v in (m, s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dsum,bias", [(True, True), (False, False)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_many_rows_a_group(lib, rows, cols, dsum, bias, dtype):
    d, mean, rstd = _inputs(rows, cols, dtype)
    dx, dg, db, z, a = _backward64(d, to_np(mean), to_np(rstd), dsum)
    gx, gg, gb = _run_backward(lib, d, mean.cuda(), rstd.cuda(), dsum, bias)
    scale = to_np(rstd) * (np.abs(a).max(1) + np.abs(z).max(1) * np.abs(a * z).mean(1)) + 1
    _close(gx, dx, dtype, scale[:, None], "dx")
    zmax, dmax = np.abs(z).max(), np.abs(to_np(d["dy"])).max()
    _close(gg, dg, torch.float32, rows * zmax * dmax / 8, "dgamma")
    if bias:
        _close(gb, db, torch.float32, rows * dmax / 8, "dbeta")
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(2501, 2048), (700, 8192)])
def test_the_same_every_time_and_captured(lib, rows, cols, dtype):
    """Equal bits from call to call, and from a captured call replayed on
    other inputs."""
    d, mean, rstd = _inputs(rows, cols, dtype)
    other = _draw(rows, cols, dtype, seed=1)
    c = {k: v.cuda() for k, v in other.items()}
    mean, rstd = mean.cuda(), rstd.cuda()
    dx, dg, db = torch.empty_like(c["x"]), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = lib.new_layer_norm_workspace(c["x"])

    def call():
        lib.bimamba_layer_norm_backward(c["dy"], c["x"], c["gamma"], mean, rstd, dx, dg, db, ws, dsum=c["dsum"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k, v in d.items():
        c[k].copy_(v)
    graph.replay()
    one, two = (_run_backward(lib, d, mean, rstd, True, True) for _ in range(2))
    for p, q, r in zip((dx, dg, db), one, two):
        assert torch.equal(p, q) and torch.equal(q, r)
