"""GPU parity of the causal prompt scan (bimamba_prompt_scan) against the
recurrence in 64 bits (causal_ref): every row of y, the whole state pool and
the whole tail pool, entries that no prompt names included.

Tolerances, fixed before the first run (2-norms over a whole tensor).
  fp32 y, and the fp32 states of either path: every operand carries the
  rounding of at most a few fp32 operations (u = 2^-24) and of a decay whose
  exponent is a sum of up to a few hundred terms, so some tens of u; 1e-5
  (170 u) leaves room for the approximate exponentials (2 ulp).  The
  tensor-core path forms its states from operands split into two bf16 halves
  (what is left out is below 2^-17 of each product), which the same bound
  covers.
  bf16 y: the value is rounded once (at most 2^-8, on average about 2^-9 /
  sqrt(3) in the 2-norm) and, on the tensor cores, so are x, B, C, the masked
  product and the state that enter it: 5 roundings and the output's, each
  about 1.7e-3 in the 2-norm and independent, together 4e-3; 6e-3.
"""
import numpy as np
import pytest
import torch

import causal_ref as ref
from parity_util import to_np

pytestmark = pytest.mark.gpu

Y_TOL = {torch.float32: 1e-5, torch.bfloat16: 6e-3}
STATE_TOL = 1e-5


@pytest.fixture(scope="module")
def lib():
    from bidirectional_mamba_ssm_b200 import _lib
    return _lib


def _check(lib, d, lens, resume, shape, extra_rows=0, **kw):
    y, s, t = ref.run(lib, d, lens, resume, *shape, **kw)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    wy, ws, wt = ref.prompts(d, lens, resume if resume is not None else [0] * len(lens), *shape)
    total = sum(lens)
    assert ref.far(y[:total], wy[:total]) <= Y_TOL[d["xbc"].dtype], ref.far(y[:total], wy[:total])
    assert torch.isnan(y[total:]).all()                      # rows behind the last prompt: as they were
    for k in range(len(d["state"])):                         # entry by entry: a large one hides no other
        assert ref.far(s[k], ws[k]) <= STATE_TOL, (k, ref.far(s[k], ws[k]))
    np.testing.assert_array_equal(to_np(t), wt)
    return y, s, t


SHAPES = [(2, 64, 128), (4, 32, 16), (3, 64, 128), (1, 8, 8), (2, 128, 256), (5, 40, 32), (1, 128, 64), (2, 16, 256)]
LENS = [[1], [2, 3], [31, 0, 33], [127, 128, 129], [4, 1, 260, 0, 64]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_ragged_prompts(lib, shape, dtype):
    for i, lens in enumerate(LENS):
        n = len(lens)
        d = ref.draw(sum(lens) + 2, n, *shape, dtype, seed=i, pool=n + 2, bias=i % 2 == 0,
                     a_range=[(0.02, 16.0), (1e-3, 1e-2)][i % 2])
        resume = [(i + k) % 2 for k in range(n)]
        _check(lib, d, lens, resume, shape)
    _check(lib, d, lens, None, shape)


@pytest.mark.parametrize("lens", [[1300], [513, 2000, 7], [255, 256, 257, 383, 384, 385]])
@pytest.mark.parametrize("memory", [(1.0, 16.0), (1e-3, 1e-2)])
def test_longer_prompts(lib, lens, memory):
    """Walks of many chunks (and cut into segments), both ways a state decays."""
    shape = (4, 64, 128)
    d = ref.draw(sum(lens), len(lens), *shape, torch.bfloat16, seed=len(lens), pool=len(lens) + 1, a_range=memory)
    _check(lib, d, lens, [k % 2 for k in range(len(lens))], shape)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_prompt_in_pieces_is_the_prompt(lib, dtype):
    """Resuming: a prompt fed in pieces of any length leaves the state, tail
    and outputs of the prompt fed at once."""
    shape, pieces = (2, 64, 128), [1, 2, 130, 1, 3, 64]
    total = sum(pieces)
    d = ref.draw(total, 1, *shape, dtype, seed=3, pool=2)
    wy, ws, wt = ref.prompts(d, [total], [0], *shape)
    c = dict(d)
    got, at = [], 0
    for i, n in enumerate(pieces):
        part = dict(c, xbc=d["xbc"][at:at + n], dt=d["dt"][at:at + n])
        y, s, t = ref.run(lib, part, [n], [int(i > 0)], *shape)
        c.update(state=s.cpu(), tail=t.cpu())
        got.append(y)
        at += n
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    assert ref.far(torch.cat(got), wy) <= Y_TOL[dtype]
    assert ref.far(c["state"], ws) <= 2 * STATE_TOL
    np.testing.assert_array_equal(to_np(c["tail"]), wt)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_neighbours_do_not_mix(lib, dtype):
    """A prompt of infinities and NaNs leaves the prompts packed around it
    (inside the same 128-row tiles) exactly as they are without it."""
    shape, lens = (2, 64, 128), [70, 50, 90, 30]
    d = ref.draw(sum(lens), 4, *shape, dtype, seed=5, pool=5)
    y0, s0, t0 = ref.run(lib, d, lens, [1, 1, 0, 1], *shape)
    bad = dict(d, xbc=d["xbc"].clone(), dt=d["dt"].clone())
    bad["xbc"][70:120:2] = float("inf")
    bad["xbc"][71:120:3] = float("nan")
    bad["dt"][70:120] = float("nan")
    y1, s1, t1 = ref.run(lib, bad, lens, [1, 1, 0, 1], *shape)
    keep = [int(d["slots"][k]) for k in (0, 2, 3)] + [4 if 4 not in d["slots"] else int(d["slots"][0])]
    assert torch.equal(y0[:70], y1[:70]) and torch.equal(y0[120:], y1[120:])
    assert torch.equal(s0[keep], s1[keep]) and torch.equal(t0[keep], t1[keep])
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bad_entries_are_skipped_and_reported(lib, dtype):
    """A slot outside the pool, one named twice, ranges that are none: those
    prompts leave y and the pool as they were; a negative slot is silent."""
    shape, lens = (2, 64, 128), [40, 30, 20, 10, 50]
    d = ref.draw(sum(lens), 5, *shape, dtype, seed=6, pool=6)
    good = ref.run(lib, d, lens, [1] * 5, *shape)
    starts = np.cumsum([0] + lens)

    def expect(slots, skipped, status, cu=None):
        q = dict(d, slots=torch.tensor(slots, dtype=torch.int32))
        y, s, t = ref.run(lib, q, lens, [1] * 5, *shape, cu=cu)
        assert lib.bimamba_get_error() == status
        assert lib.bimamba_get_error() == lib.BIMAMBA_OK
        for k in range(5):
            rows, slot = slice(starts[k], starts[k + 1]), int(d["slots"][k])
            if k in skipped:
                assert torch.isnan(y[rows]).all()
                assert torch.equal(s[slot].cpu(), d["state"][slot]) and torch.equal(t[slot].cpu(), d["tail"][slot])
            else:
                assert torch.equal(y[rows], good[0][rows])
                assert torch.equal(s[slot], good[1][slot]) and torch.equal(t[slot], good[2][slot])

    base = d["slots"].tolist()
    put = lambda i, v: base[:i] + [v] + base[i + 1:]  # noqa: E731
    bad = lib.BIMAMBA_ERR_INVALID
    expect(put(2, -1), {2}, lib.BIMAMBA_OK)
    expect(put(2, 6), {2}, bad)
    expect(put(2, 1 << 30), {2}, bad)
    expect(put(2, base[4]), {2, 4}, bad)
    cu = starts.tolist()
    expect(base, {4}, bad, cu=cu[:5] + [cu[4] - 1])          # ends before it starts
    expect(base, {4}, bad, cu=cu[:5] + [cu[5] + 1])          # ends past the rows
    expect(base, {0}, bad, cu=[-1] + cu[1:])


def test_a_workspace_serves_other_calls(lib):
    """One zero-filled workspace through calls of other sizes, types and
    errors; each result is that of a fresh workspace."""
    shape = (2, 64, 128)
    ws = None
    for i, (lens, dtype) in enumerate([([300, 1, 129], torch.bfloat16), ([5], torch.float32), ([64] * 6, torch.bfloat16),
                                       ([700], torch.bfloat16), ([300, 1, 129], torch.float32)]):
        d = ref.draw(sum(lens), len(lens), *shape, dtype, seed=i, pool=8)
        if ws is None:
            ws = torch.zeros(max(lib.bimamba_prompt_workspace_bytes(lib.make_dims(8, 2000, *shape, t))
                                 for t in (torch.float32, torch.bfloat16)), dtype=torch.uint8, device="cuda")
        if i == 2:   # an entry that is refused leaves the workspace fit for use
            bad = dict(d, slots=torch.tensor([0, 1, 9, 1, 2, -1], dtype=torch.int32))
            ref.run(lib, bad, lens, None, *shape, ws=ws)
            assert lib.bimamba_get_error() == lib.BIMAMBA_ERR_INVALID
        one = ref.run(lib, d, lens, [1] * len(lens), *shape, ws=ws)
        two = ref.run(lib, d, lens, [1] * len(lens), *shape)
        for p, q in zip(one, two):
            assert torch.equal(p, q)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_captured_and_replayed_with_other_lengths(lib, dtype):
    """The lengths live on the device: one captured graph serves batches of
    other lengths (and padding entries)."""
    shape, rows, n = (2, 64, 128), 600, 4
    dev = lambda d: {k: None if v is None else v.cuda() for k, v in d.items()}  # noqa: E731
    d = ref.draw(rows, n, *shape, dtype, seed=1, pool=6)
    c = dev(d)
    cu = torch.tensor([0, 100, 200, 300, 400], dtype=torch.int32, device="cuda")
    resume = torch.ones(n, dtype=torch.int32, device="cuda")
    y = torch.zeros((rows, 128), dtype=dtype, device="cuda")
    kw = dict(heads=2, headdim=64, d_state=128)
    ws = lib.new_prompt_workspace(c["xbc"], batch=n, **kw)

    def call():
        lib.bimamba_prompt_scan(c["xbc"], c["dt"], c["A"], c["D"], c["conv_w"], c["conv_b"], cu, c["state"],
                                c["tail"], c["slots"], resume, y, ws, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i, lens in enumerate([[600, 0, 0, 0], [1, 2, 3, 400], [150, 150, 150, 150]]):
        d = ref.draw(rows, n, *shape, dtype, seed=10 + i, pool=6)
        for k, v in dev(d).items():
            c[k].copy_(v)
        cu.copy_(torch.tensor(np.cumsum([0] + lens), dtype=torch.int32))
        y.fill_(float("nan"))
        if i == 1:
            c["slots"][3] = -1
        graph.replay()
        got = (y.clone(), c["state"].clone(), c["tail"].clone())
        want = ref.run(lib, dict(d, slots=c["slots"].cpu()), lens, [1] * n, *shape)
        for p, q in zip(got, want):
            assert torch.equal(p.nan_to_num(7.0), q.nan_to_num(7.0))
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK


def test_two_calls_at_once(lib):
    """Two streams, each with its own workspace and pool."""
    shape, lens = (4, 64, 128), [500, 37, 700]
    kw = dict(heads=4, headdim=64, d_state=128)
    sets, want = [], []
    for i in range(2):
        d = ref.draw(sum(lens), 3, *shape, torch.bfloat16, seed=20 + i, pool=3)
        want.append(ref.run(lib, d, lens, [1, 0, 1], *shape))
        c = {k: v.cuda() for k, v in d.items()}
        c["y"] = torch.empty((sum(lens), 256), dtype=torch.bfloat16, device="cuda")
        c["ws"] = lib.new_prompt_workspace(c["xbc"], batch=3, **kw)
        sets.append(c)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    res = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for c in sets:
        lib.bimamba_prompt_scan(c["xbc"], c["dt"], c["A"], c["D"], c["conv_w"], c["conv_b"], cu, c["state"],
                                c["tail"], c["slots"], res, c["y"], c["ws"], stream=torch.cuda.Stream(), **kw)
    torch.cuda.synchronize()
    for c, (y, s, t) in zip(sets, want):
        assert torch.equal(c["y"], y) and torch.equal(c["state"], s) and torch.equal(c["tail"], t)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK


def test_the_pool_feeds_the_block_decode(lib):
    """A prompt, tokens one by one, then a block: the pool's entry is the
    prefix cache that the block decode continues from."""
    H, P, N = 2, 64, 128
    kw = dict(heads=H, headdim=P, d_state=N)
    lens, steps, blk = [200, 77], 3, 48
    per = [n + steps + blk for n in lens]
    d = ref.draw(sum(per), 2, H, P, N, torch.bfloat16, seed=8, pool=4)
    at = np.cumsum([0] + per)
    rows = [torch.arange(at[s], at[s + 1]) for s in range(2)]
    pick = lambda a, b: torch.cat([r[a[s]:b[s]] for s, r in enumerate(rows)])  # noqa: E731
    prompt = pick([0, 0], lens)
    y, st, tl = ref.run(lib, dict(d, xbc=d["xbc"][prompt], dt=d["dt"][prompt]), lens, None, H, P, N)
    slots = d["slots"].cuda()
    g = {k: v.cuda() for k, v in d.items()}
    ws = lib.new_step_workspace(2, dtype=torch.bfloat16, **kw)
    ys = torch.empty((2, H * P), dtype=torch.bfloat16, device="cuda")
    for i in range(steps):
        r = pick([n + i for n in lens], [n + i + 1 for n in lens]).cuda()
        lib.bimamba_token_step(g["xbc"][r], g["dt"][r], g["A"], g["D"], g["conv_w"], g["conv_b"], st, tl, slots,
                               ys, ws, **kw)
    b = torch.stack([rows[s][lens[s] + steps:] for s in range(2)]).cuda()
    yb = torch.empty((2, blk, H * P), dtype=torch.bfloat16, device="cuda")
    want_y, want_s, want_t = ref.prompts(dict(d), [n + steps for n in lens], [0, 0], H, P, N, cu=at[:2].tolist())
    for k in slots.tolist():
        assert ref.far(st[k], want_s[k]) <= STATE_TOL
        np.testing.assert_array_equal(to_np(tl[k]), want_t[k])
    lib.bimamba_block_decode_pool(g["xbc"][b], g["dt"][b], g["A"], g["D"], g["conv_w"], g["conv_b"], st, tl, slots,
                                  None, yb, lib.new_workspace(lib.make_dims(2, blk, H, P, N, torch.bfloat16)), **kw)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    _, end_s, end_t = ref.prompts(dict(d), per, [0, 0], H, P, N)
    for k in slots.tolist():
        assert ref.far(st[k], end_s[k]) <= 6e-3              # the block decode's state operands are bf16
        np.testing.assert_array_equal(to_np(tl[k]), end_t[k])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("where", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("at", [0, 5, 127, 130])
def test_a_bad_token_leaves_the_rows_before_it(lib, dtype, where, at):
    """An infinity or NaN enters the outputs at its own token, not before
    (although the tokens of a 128-row tile share their products), and in x
    only its own channel."""
    shape, n = (2, 64, 128), 200
    H, P, N = shape
    d = ref.draw(n, 1, *shape, dtype, seed=9, pool=1)
    y0, _, _ = ref.run(lib, d, [n], [1], *shape)
    for value in (float("nan"), float("inf")):
        bad = dict(d, xbc=d["xbc"].clone(), dt=d["dt"].clone())
        if where == "dt":
            bad["dt"][at, 1] = value
        else:
            bad["xbc"][at, {"x": 70, "B": H * P + 3, "C": H * P + N + 3}[where]] = value
        y1, s1, _ = ref.run(lib, bad, [n], [1], *shape)
        assert torch.equal(y0[:at], y1[:at])
        if where == "x":
            rest = [c for c in range(H * P) if c != 70]
            assert torch.equal(y0[:, rest], y1[:, rest])
            assert not torch.isfinite(y1[at:, 70]).any()
            assert not torch.isfinite(s1[0, 1, 6]).any() and torch.isfinite(s1[0, 1, 7]).all()
        elif where == "C":
            assert not torch.isfinite(y1[at]).any() and torch.isfinite(y1[at + 4:]).all()
        elif where == "dt":
            assert torch.equal(y0[:, :64], y1[:, :64])       # the other head
            assert not torch.isfinite(y1[at:, 64:]).any()
        else:
            assert not torch.isfinite(y1[at:]).any()
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_rows_at_all(lib, dtype):
    """A batch of empty prompts: entries that resume stay, the others are zeroed."""
    shape = (2, 64, 128)
    d = ref.draw(0, 3, *shape, dtype, seed=1, pool=4)
    _, s, t = ref.run(lib, d, [0, 0, 0], [1, 0, 1], *shape)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    k = int(d["slots"][1])
    keep = [i for i in range(4) if i != k]
    assert torch.equal(s[keep].cpu(), d["state"][keep]) and torch.equal(t[keep].cpu(), d["tail"][keep])
    assert not s[k].any() and not t[k].any()


@pytest.mark.parametrize("a_range", [(200.0, 400.0), (1e-6, 1e-5)])
def test_extreme_decays(lib, a_range):
    """Decays that leave nothing of a token two tokens on, and ones that lose
    nothing over a thousand."""
    shape, lens = (2, 64, 128), [300, 1000]
    d = ref.draw(sum(lens), 2, *shape, torch.bfloat16, seed=12, pool=2, a_range=a_range)
    _check(lib, d, lens, [1, 0], shape)


def test_many_prompts(lib):
    """More prompts than a plan pass takes at once, most of them empty or short."""
    shape, n = (2, 64, 128), 700
    lens = [(7 * i) % 5 if i % 9 else 130 for i in range(n)]
    d = ref.draw(sum(lens), n, *shape, torch.bfloat16, seed=13, pool=n + 1)
    _check(lib, d, lens, [i % 2 for i in range(n)], shape)


def test_larger_batch_of_the_model_shape(lib):
    """64 heads, a batch that fills the SMs more than once, against the fp32
    kernel on the same values (which the tests above hold against 64 bits)."""
    shape, lens = (64, 64, 128), [900, 17, 2500, 300, 1, 64, 1025, 777]
    d = ref.draw(sum(lens), len(lens), *shape, torch.bfloat16, seed=14, pool=len(lens))
    res = [i % 2 for i in range(len(lens))]
    y, s, t = ref.run(lib, d, lens, res, *shape)
    f = dict(d, xbc=d["xbc"].float(), dt=d["dt"].float(), tail=d["tail"].float())
    fy, fs, ft = ref.run(lib, f, lens, res, *shape)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    assert ref.far(y, to_np(fy)) <= Y_TOL[torch.bfloat16]
    for k in range(len(lens)):
        assert ref.far(s[k], to_np(fs[k])) <= 2 * STATE_TOL
    assert torch.equal(t.float(), ft)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ranges_of_the_same_rows(lib, dtype):
    """Prompts that all name the same 1280 rows (their ranges run backwards in
    between) are more than a call of that many rows can hold: reported, every
    entry of the pool finite, and the next call right."""
    shape, n, rows = (2, 64, 128), 64, 1280
    d = ref.draw(rows, n, *shape, dtype, seed=8, pool=n)
    y, s, t = ref.run(lib, d, [0] * n, [1] * n, *shape, cu=[0, rows] * (n // 2) + [0])
    assert lib.bimamba_get_error() == lib.BIMAMBA_ERR_INVALID
    assert torch.isfinite(s).all() and torch.isfinite(t).all()
    d = ref.draw(100, 1, *shape, dtype, seed=9, pool=2)
    _check(lib, d, [100], [1], shape)


def test_several_long_prompts(lib):
    """Prompts cut into segments of many chunks beside short and empty ones;
    then two of them naming one entry, which are skipped and reported."""
    shape, lens, resume = (2, 64, 128), [2600, 5, 9000, 0, 3000], [1, 0, 1, 1, 0]
    d = ref.draw(sum(lens), 5, *shape, torch.bfloat16, seed=21, pool=6, a_range=(1e-3, 1e-2))
    y, s, t = _check(lib, d, lens, resume, shape)
    slots = d["slots"].tolist()
    y2, s2, t2 = ref.run(lib, dict(d, slots=torch.tensor(slots[:4] + slots[:1], dtype=torch.int32)), lens, resume,
                         *shape)
    assert lib.bimamba_get_error() == lib.BIMAMBA_ERR_INVALID
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    assert torch.isnan(y2[:2600]).all() and torch.isnan(y2[-3000:]).all()
    assert torch.equal(y2[2600:-3000], y[2600:-3000])
    for k in (slots[0], slots[4]):
        assert torch.equal(s2[k].cpu(), d["state"][k]) and torch.equal(t2[k].cpu(), d["tail"][k])
    for k in slots[1:4]:
        assert torch.equal(s2[k], s[k]) and torch.equal(t2[k], t[k])
