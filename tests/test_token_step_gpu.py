"""GPU parity of the single-token step (bimamba_token_step) against the
recurrence in 64 bits.  One step in fp32: a few roundings (u = 2^-24) per
value and one 2-ulp exponential; the 1e-6 bound on 2-norms is 17 u.  y sums N
products in fp32 and, for bf16, is rounded once (at most 2^-8)."""
import numpy as np
import pytest
import torch

import causal_ref as ref
from parity_util import to_np

pytestmark = pytest.mark.gpu

Y_TOL = {torch.float32: 1e-6, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def lib():
    from bidirectional_mamba_ssm_b200 import _lib
    return _lib


def _run(lib, d, shape, ws=None, stream=None):
    c = {k: None if v is None else v.cuda() for k, v in d.items()}
    rows = c["xbc"].shape[0]
    kw = dict(zip(("heads", "headdim", "d_state"), shape))
    y = torch.full((rows, shape[0] * shape[1]), float("nan"), dtype=c["xbc"].dtype, device="cuda")
    if ws is None:
        ws = lib.new_step_workspace(rows, dtype=c["xbc"].dtype, **kw)
    lib.bimamba_token_step(c["xbc"], c["dt"], c["A"], c["D"], c["conv_w"], c["conv_b"], c["state"], c["tail"],
                           c["slots"], y, ws, stream=stream, **kw)
    return y, c["state"], c["tail"]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(2, 64, 128), (4, 32, 16), (1, 8, 8), (3, 128, 256), (5, 40, 32), (2, 128, 64),
                                   (2, 72, 128)])
@pytest.mark.parametrize("rows", [1, 5, 300])
def test_rows(lib, shape, dtype, rows):
    d = ref.draw(rows, rows, *shape, dtype, seed=rows, pool=rows + 3, bias=rows != 5)
    y, s, t = _run(lib, d, shape)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    wy, ws, wt = ref.prompts(d, [1] * rows, [1] * rows, *shape)
    assert ref.far(y, wy) <= Y_TOL[dtype]
    assert ref.far(s, ws) <= 1e-6
    np.testing.assert_array_equal(to_np(t), wt)
    rest = sorted(set(range(rows + 3)) - set(d["slots"].tolist()))
    assert torch.equal(s[rest].cpu(), d["state"][rest])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_are_the_prompt(lib, dtype):
    """Token after token in one workspace (captured and replayed) gives the
    prompt's outputs, state and tail."""
    shape, n, rows = (2, 64, 128), 9, 3
    kw = dict(heads=2, headdim=64, d_state=128)
    d = ref.draw(rows * n, rows, *shape, dtype, seed=4, pool=4)
    wy, wst, wt = ref.prompts(d, [n] * rows, [1] * rows, *shape)
    c = {k: v.cuda() for k, v in d.items()}
    x, dt = torch.empty_like(c["xbc"][:rows]), torch.empty_like(c["dt"][:rows])
    y = torch.empty((rows, 128), dtype=dtype, device="cuda")
    ws = lib.new_step_workspace(rows, dtype=dtype, **kw)

    def call():
        lib.bimamba_token_step(x, dt, c["A"], c["D"], c["conv_w"], c["conv_b"], c["state"], c["tail"], c["slots"], y,
                               ws, **kw)
    keep = c["state"].clone(), c["tail"].clone()
    x.copy_(c["xbc"][:rows]), dt.copy_(c["dt"][:rows])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    c["state"].copy_(keep[0]), c["tail"].copy_(keep[1])
    got = torch.empty((rows, n, 128), dtype=dtype)
    at = torch.arange(rows, device="cuda") * n
    for i in range(n):
        x.copy_(c["xbc"][at + i]), dt.copy_(c["dt"][at + i])
        graph.replay()
        got[:, i] = y.cpu()
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    assert ref.far(got.reshape(rows * n, 128), wy) <= 2 * Y_TOL[dtype]
    assert ref.far(c["state"], wst) <= 1e-5
    np.testing.assert_array_equal(to_np(c["tail"]), wt)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bad_rows_are_skipped_and_reported(lib, dtype):
    shape, rows = (3, 64, 128), 5
    d = ref.draw(rows, rows, *shape, dtype, seed=2, pool=6)
    good = _run(lib, d, shape)
    base = d["slots"].tolist()
    kw = dict(heads=3, headdim=64, d_state=128)
    ws = lib.new_step_workspace(rows, dtype=dtype, **kw)     # kept through the refused rows
    for slots, skipped, status in [(base[:2] + [-1] + base[3:], {2}, lib.BIMAMBA_OK),
                                   (base[:2] + [6] + base[3:], {2}, lib.BIMAMBA_ERR_INVALID),
                                   (base[:2] + [base[0]] + base[3:], {0, 2}, lib.BIMAMBA_ERR_INVALID),
                                   (base, set(), lib.BIMAMBA_OK)]:
        y, s, t = _run(lib, dict(d, slots=torch.tensor(slots, dtype=torch.int32)), shape, ws=ws)
        assert lib.bimamba_get_error() == status
        for k in range(rows):
            if k in skipped:
                assert torch.isnan(y[k]).all()
                assert torch.equal(s[base[k]].cpu(), d["state"][base[k]])
                assert torch.equal(t[base[k]].cpu(), d["tail"][base[k]])
            else:
                assert torch.equal(y[k], good[0][k]) and torch.equal(s[base[k]], good[1][base[k]])
                assert torch.equal(t[base[k]], good[2][base[k]])


def test_a_large_pool(lib):
    """An entry past 2^32 bytes of the state pool (and 2^31 elements)."""
    H, P, N = 64, 64, 128
    free, _ = torch.cuda.mem_get_info()
    pool = 4200                                              # 8.8 GB of states
    if free < 12 << 30:
        pytest.skip("not enough free memory")
    d = ref.draw(2, 2, H, P, N, torch.bfloat16, seed=1, pool=2)
    want = _run(lib, dict(d, slots=torch.tensor([0, 1], dtype=torch.int32)), (H, P, N))
    state = torch.zeros((pool, H, P, N), device="cuda")
    tail = torch.zeros((pool, 4, H * P + 2 * N), dtype=torch.bfloat16, device="cuda")
    state[pool - 1], state[pool - 2] = d["state"][0].cuda(), d["state"][1].cuda()
    tail[pool - 1], tail[pool - 2] = d["tail"][0].cuda(), d["tail"][1].cuda()
    c = {k: v.cuda() for k, v in d.items() if k not in ("state", "tail", "slots")}
    y = torch.empty((2, H * P), dtype=torch.bfloat16, device="cuda")
    kw = dict(heads=H, headdim=P, d_state=N)
    lib.bimamba_token_step(c["xbc"], c["dt"], c["A"], c["D"], c["conv_w"], c["conv_b"], state, tail,
                           torch.tensor([pool - 1, pool - 2], dtype=torch.int32, device="cuda"), y,
                           lib.new_step_workspace(2, dtype=torch.bfloat16, **kw), **kw)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    assert torch.equal(y, want[0])
    assert torch.equal(state[pool - 1], want[1][0]) and torch.equal(state[pool - 2], want[1][1])
    assert torch.equal(tail[pool - 1], want[2][0])


def test_thousands_of_steps_of_a_slow_decay(lib):
    """4096 equal steps of decays near 1: two roundings a step (at most 2^-24
    each, independent) are sqrt(8192) 2^-24 / sqrt(3) = 3e-6 of the state; a
    decay rounded alike at every step would be some 4096 2^-25 / sqrt(3) =
    7e-5.  1e-5."""
    shape, n = (4, 64, 128), 4096
    d = ref.draw(n, 1, *shape, torch.float32, seed=11, pool=1, a_range=(1e-4, 1e-2))
    d["dt"].fill_(0.05)
    _, want, _ = ref.prompts(d, [n], [1], *shape)
    c = {k: v.cuda() for k, v in d.items()}
    kw = dict(heads=4, headdim=64, d_state=128)
    ws = lib.new_step_workspace(1, dtype=torch.float32, **kw)
    y = torch.empty((1, 256), device="cuda")
    for t in range(n):
        lib.bimamba_token_step(c["xbc"][t:t + 1], c["dt"][t:t + 1], c["A"], c["D"], c["conv_w"], c["conv_b"],
                               c["state"], c["tail"], c["slots"], y, ws, **kw)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    for h in range(4):
        assert ref.far(c["state"][0, h], want[0, h]) <= 1e-5, h
