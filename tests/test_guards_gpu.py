"""Bytes around what a call may write: workspaces of exactly the size asked
for, outputs, and the pool's entries that no row names, between guard bytes."""
import pytest
import torch

import causal_ref as ref

pytestmark = pytest.mark.gpu
GUARD, EDGE = 0xA5, 4096


@pytest.fixture(scope="module")
def lib():
    from bidirectional_mamba_ssm_b200 import _lib
    return _lib


class Guarded:
    """Tensors inside buffers whose edges are checked at the end."""

    def __init__(self):
        self.all = []

    def like(self, t):
        raw = torch.full((2 * EDGE + t.numel() * t.element_size(),), GUARD, dtype=torch.uint8, device="cuda")
        self.all.append(raw)
        inner = raw[EDGE:EDGE + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        inner.copy_(t)
        return inner

    def check(self):
        for raw in self.all:
            assert (raw[:EDGE] == GUARD).all() and (raw[-EDGE:] == GUARD).all()


@pytest.mark.parametrize("dtype,shape", [(torch.bfloat16, (2, 64, 128)), (torch.bfloat16, (3, 32, 16)), (torch.float32, (2, 64, 128))])
@pytest.mark.parametrize("lens", [[1], [0, 0], [129, 0, 3], [2600, 5, 1, 700], [31] * 40])
def test_prompt_and_step(lib, lens, dtype, shape):
    H, P, N = shape
    kw = dict(heads=H, headdim=P, d_state=N)
    n, g = len(lens), Guarded()
    d = ref.draw(sum(lens), n, *shape, dtype, seed=50, pool=n + 2)
    c = {k: g.like(v) for k, v in d.items() if v.numel()}
    rows = sum(lens)
    x = c.get("xbc", d["xbc"].cuda())
    dt = c.get("dt", d["dt"].cuda())
    y = g.like(torch.zeros((max(rows, 1), H * P), dtype=dtype))[:rows]
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ws = g.like(torch.full((lib.bimamba_prompt_workspace_bytes(lib.make_dims(n, rows, H, P, N, dtype)),), 7, dtype=torch.uint8))
    lib.bimamba_prompt_scan(x, dt, c["A"], c["D"], c["conv_w"], c["conv_b"], cu, c["state"], c["tail"], c["slots"], None, y, ws, **kw)
    y1 = g.like(torch.zeros((n, H * P), dtype=dtype))
    one = ref.draw(n, n, *shape, dtype, seed=51, pool=n + 2)
    sws = g.like(torch.zeros(max(1, lib.bimamba_token_step_workspace_bytes(lib.make_dims(n, 1, H, P, N, dtype))), dtype=torch.uint8))
    lib.bimamba_token_step(g.like(one["xbc"]), g.like(one["dt"]), c["A"], c["D"], c["conv_w"], c["conv_b"], c["state"], c["tail"],
                           c["slots"], y1, sws, **kw)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    g.check()
    assert torch.isfinite(y).all() and torch.isfinite(y1).all()
    rest = sorted(set(range(n + 2)) - set(d["slots"].tolist()))
    assert torch.equal(c["state"][rest].cpu(), d["state"][rest]) and torch.equal(c["tail"][rest].cpu(), d["tail"][rest])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 8), (5, 520), (601, 4104), (333, 8192), (2501, 256)])
def test_layer_norm(lib, rows, cols, dtype):
    g = Guarded()
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, res, dy = (g.like(r(rows, cols).to(dtype)) for _ in range(3))
    gamma, beta = g.like(1 + r(cols)), g.like(r(cols))
    y, s, dx = (g.like(torch.zeros((rows, cols), dtype=dtype)) for _ in range(3))
    mean, rstd, dg, db = g.like(r(rows)), g.like(r(rows)), g.like(r(cols)), g.like(r(cols))
    ws = g.like(torch.full((lib.bimamba_layer_norm_backward_workspace_bytes(rows, cols),), 7, dtype=torch.uint8))
    lib.bimamba_layer_norm(x, gamma, beta, y, mean, rstd, residual=res, sum_out=s)
    lib.bimamba_layer_norm_backward(dy, s, gamma, mean, rstd, dx, dg, db, ws, dsum=res)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    g.check()
    for t in (y, s, mean, rstd, dx, dg, db):
        assert torch.isfinite(t).all()
