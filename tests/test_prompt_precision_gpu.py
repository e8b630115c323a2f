"""How exact the bf16 prompt scan's rows are: against the recurrence in 64
bits, beside what rounding the exact values to bf16 once costs, and over the
range of values that bf16 inputs can have.

Tolerance of the first test, fixed before its first run.  With r the 2-norm
error of rounding exact values to bf16 once, a value that enters as fp16 (X,
M, C and the state of C S^T) adds at most r / 8, these four together
r sqrt(4) / 8; B and C enter G = C B^T as bf16, r each, but only through the
part of y that is neither D x nor the state that entered the chunk, s of y's
2-norm.  sqrt(1 + 4 / 64 + 2 s^2) r: with |D| >= 0.4 s is below 0.35 here, and
1.15 r bounds it."""
import numpy as np
import pytest
import torch

import causal_ref as ref
from parity_util import to_np

pytestmark = pytest.mark.gpu

# Of an element of the state, of the sum of its terms' magnitudes.  w x and B
# enter its products as two bf16 halves each: a half is off by at most 2^-9 of
# its value, so the pair by 2^-18, and the product of the two lower halves,
# 2^-18 at most, is left out: 3 2^-18 = 1.14e-5, and fp32 roundings of the
# decays, some 2^-20 each.
STATE_PART = 1.5e-5
# Of an element, where the terms of y may cancel: y is rounded once (2^-9 of
# it), and of the sum A of its terms' magnitudes each factor's rounding takes
# its part: B and C in G 2^-9 each; X and M, or C and the state, 2^-12 each.
# What is below fp32's smallest normal number, 2^-126, may be flushed.
Y_PART, A_PART = 2.0 ** -9 * 1.01, (2 * 2.0 ** -9 + 2 * 2.0 ** -12) * 1.01


def _terms(d, n, shape):
    """A, and that of the state: one resumed prompt of n tokens, every term by its magnitude."""
    H, P, N = shape
    f = lambda k: to_np(d[k])  # noqa: E731
    rows = np.concatenate([f("tail")[0][1:], f("xbc")[:n]])
    u = sum(rows[j:j + n] * f("conv_w")[:, j] for j in range(4)) + (0.0 if d["conv_b"] is None else f("conv_b"))
    u = np.abs(u / (1.0 + np.exp(np.minimum(-u, 700.0))))
    h, out = np.abs(f("state")[0]), np.zeros((n, H, P))
    dts, A, D = f("dt"), f("A"), np.abs(f("D"))
    for t in range(n):
        x, dt = u[t, :H * P].reshape(H, P), dts[t]
        h = h * np.exp(dt * A)[:, None, None] + (dt[:, None] * x)[..., None] * u[t, H * P:H * P + N]
        out[t] = h @ u[t, H * P + N:] + D[:, None] * x
    return out.reshape(n, H * P), h


@pytest.fixture(scope="module")
def lib():
    from bidirectional_mamba_ssm_b200 import _lib
    return _lib


@pytest.mark.parametrize("memory", [(1.0, 16.0), (0.02, 16.0), (1e-3, 1e-2)])
@pytest.mark.parametrize("lens,resume", [([37], [1]), ([1], [0]), ([700, 1, 1300, 129], [0, 1, 1, 0]), ([4500], [0])])
def test_rows_are_as_exact_as_one_rounding(lib, lens, resume, memory):
    shape = (4, 64, 128)
    d = ref.draw(sum(lens), len(lens), *shape, torch.bfloat16, seed=31, pool=len(lens), a_range=memory)
    d["D"] = torch.tensor([0.6, -0.4, 1.1, -1.6])
    y, s, _ = ref.run(lib, d, lens, resume, *shape)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    wy, ws, _ = ref.prompts(d, lens, resume, *shape)
    once = ref.far(torch.from_numpy(wy).to(torch.bfloat16), wy)
    assert ref.far(y, wy) <= 1.15 * once, (ref.far(y, wy), once)
    for k in range(len(d["state"])):
        assert ref.far(s[k], ws[k]) <= 1e-5


def _scaled(case, n, shape, seed=32):
    H, P, N = shape
    d = ref.draw(n, 1, *shape, torch.bfloat16, seed=seed, pool=1, a_range=(1e-2, 1.0), bias=case not in ("x tiny", "x of one head tiny", "x zero"))
    x, B, C = slice(0, H * P), slice(H * P, H * P + N), slice(H * P + N, None)

    def times(columns, f):
        d["xbc"][:, columns] = (d["xbc"][:, columns].float() * f).to(torch.bfloat16)
        d["tail"][..., columns] = (d["tail"][..., columns].float() * f).to(torch.bfloat16)
    {"x of one head tiny": lambda: times(slice(P, 2 * P), 1e-9), "x zero": lambda: times(x, 0.0), "x large": lambda: times(x, 1e4), "x tiny": lambda: times(x, 1e-9), "x of one channel huge": lambda: times(slice(70, 71), 1e30),
     "x of one token large": lambda: d["xbc"].__setitem__((130, x), (d["xbc"][130, x].float() * 3000).to(torch.bfloat16)),
     "B large": lambda: times(B, 1e6), "B tiny": lambda: times(B, 1e-6), "C large": lambda: times(C, 1e6),
     "C tiny": lambda: times(C, 1e-8), "a token's C large": lambda: d["xbc"].__setitem__((40, C), (d["xbc"][40, C].float() * 1e12).to(torch.bfloat16)),
     "D large": lambda: d.update(D=d["D"] * 1e5), "D zero": lambda: d.update(D=torch.zeros(H)),
     "dt tiny": lambda: d.update(dt=(d["dt"].float() * 1e-6).to(torch.bfloat16)),
     "state large": lambda: d.update(state=d["state"] * 1e15), "state tiny": lambda: d.update(state=d["state"] * 1e-15),
     "a state row large": lambda: d["state"][0, 1, 5].mul_(1e25), "a state row tiny": lambda: d["state"][0, 1, 5].mul_(1e-12)}[case]()
    return d


CASES = ["x of one head tiny", "x zero", "x large", "x tiny", "x of one channel huge", "x of one token large", "B large", "B tiny", "C large", "C tiny",
         "a token's C large", "D large", "D zero", "dt tiny", "state large", "state tiny", "a state row large",
         "a state row tiny"]


@pytest.mark.parametrize("case", CASES)
def test_values_of_any_size(lib, case):
    """Element by element: a large one hides no other."""
    shape, n = (2, 64, 128), 700
    d = _scaled(case, n, shape)
    y, s, _ = ref.run(lib, d, [n], [1], *shape)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    wy, ws, _ = ref.prompts(d, [n], [1], *shape)
    terms, state = _terms(d, n, shape)
    off = np.abs(to_np(y) - wy) - Y_PART * np.abs(wy) - A_PART * terms - 2.0 ** -126
    assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))
    off = np.abs(to_np(s)[0] - ws[0]) - STATE_PART * state - 2.0 ** -126
    assert off.max() <= 0, off.max()


def test_a_large_activation_leaves_the_other_channels_bits(lib):
    """Past fp16's range in one channel: that channel right, the others' bits
    as without it."""
    shape, n = (2, 64, 128), 300
    d = ref.draw(n, 1, *shape, torch.bfloat16, seed=33, pool=1)
    y0, s0, _ = ref.run(lib, d, [n], [1], *shape)
    big = dict(d, xbc=d["xbc"].clone())
    big["xbc"][140:150, 70] = 20000.0
    y1, s1, _ = ref.run(lib, big, [n], [1], *shape)
    wy, ws, _ = ref.prompts(big, [n], [1], *shape)
    rest = [c for c in range(128) if c != 70]
    assert torch.equal(y0[:, rest], y1[:, rest])
    assert torch.equal(y0[:128, 70], y1[:128, 70])
    off = np.abs(to_np(y1[:, 70]) - wy[:, 70]) - Y_PART * np.abs(wy[:, 70]) - A_PART * _terms(big, n, shape)[0][:, 70]
    assert off.max() <= 0
    assert ref.far(s1, ws) <= 1e-5
    assert torch.equal(s0[0, 0], s1[0, 0])
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK


def test_rows_of_many_growing_chunks(lib):
    """A state that grows for hundreds of chunks (no decay to speak of) and
    one that a jump in B enlarges a million times on the way: the bound that
    its operand is scaled by follows."""
    shape, n = (2, 64, 128), 40000
    d = ref.draw(n, 1, *shape, torch.bfloat16, seed=34, pool=1, a_range=(1e-6, 1e-5))
    H, P, N = shape
    d["xbc"][21000:, H * P:H * P + N] = (d["xbc"][21000:, H * P:H * P + N].float() * 1e6).to(torch.bfloat16)
    y, s, _ = ref.run(lib, d, [n], [0], *shape)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    wy, ws, _ = ref.prompts(d, [n], [0], *shape)
    # (2-norms over the rows before and after: of y, its rounding and those of B and C, 1.7e-3 each)
    for rows in (slice(0, 21000), slice(21000, n)):
        assert ref.far(y[rows], wy[rows]) <= 6e-3
    assert ref.far(s, ws) <= 1e-5


@pytest.mark.parametrize("memory", [(1e-3, 1e-2), (0.02, 16.0)])
def test_channels_far_smaller_than_their_head_s_others(lib, memory):
    """x of channels 1e-1 to 1e-6 times the others' all along (D = 0, so that y
    is their states' and the chunk's alone): as exact for their size."""
    shape, n = (2, 64, 128), 3000
    H, P, N = shape
    d = ref.draw(n, 1, *shape, torch.bfloat16, seed=35, pool=1, a_range=memory, bias=False)
    d["D"] = torch.zeros(H)
    for c in range(8, P):
        d["xbc"][:, c] = (d["xbc"][:, c].float() * 10.0 ** -(c // 8 - 1)).to(torch.bfloat16)
        d["state"][0, 0, c] *= 10.0 ** -(c // 8 - 1)
        d["tail"][..., c] = (d["tail"][..., c].float() * 10.0 ** -(c // 8 - 1)).to(torch.bfloat16)
    y, s, _ = ref.run(lib, d, [n], [1], *shape)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    wy, ws, _ = ref.prompts(d, [n], [1], *shape)
    terms, _ = _terms(d, n, shape)
    # (2-norms of channels: the roundings of B and C in G, 1.7e-3 each of terms that cancel in part; 6e-3)
    off = np.linalg.norm(to_np(y) - wy, axis=0) / np.linalg.norm(wy, axis=0)
    assert off.max() <= 6e-3, [float(v) for v in off[::8]]
    off = np.abs(to_np(y) - wy) - Y_PART * np.abs(wy) - A_PART * terms
    assert off.max() <= 0
    # (2-norm: where one token outweighs the others, its conv may cancel, which the
    # magnitudes of activations do not show)
    assert ref.far(s, ws) <= 1e-5


def test_a_sum_past_the_range_is_an_infinity(lib):
    """Raw values whose conv sum is past 2^120 (here above 2^128 / 16 in
    magnitude) act as infinities do: on their channel from their token on."""
    shape, n = (2, 64, 128), 300
    d = ref.draw(n, 1, *shape, torch.bfloat16, seed=36, pool=1)
    d["conv_w"][70] = torch.tensor([0.25, 0.5, 0.125, 0.25])
    outs = []
    for v in (3e38, float("inf")):
        big = dict(d, xbc=d["xbc"].clone())
        big["xbc"][140, 70] = v
        outs.append(ref.run(lib, big, [n], [1], *shape))
        assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    y0, s0, _ = ref.run(lib, d, [n], [1], *shape)
    for a, b in zip(outs[0][:2], outs[1][:2]):
        assert torch.equal(a.isnan(), b.isnan())
        assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
    y, s = outs[0][:2]
    rest = [c for c in range(128) if c != 70]
    assert torch.equal(y[:140], y0[:140])
    assert torch.equal(y[:, rest], y0[:, rest])
    assert not y[140:, 70].isfinite().any() and not s[0, 1, 6].isfinite().any()
    keep = [c for c in range(64) if c != 6]
    assert torch.equal(s[0, 0], s0[0, 0]) and torch.equal(s[0, 1, keep], s0[0, 1, keep])
