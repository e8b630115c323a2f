"""What the prompt scan's plan and workspace hold where ranges overlap."""
import pytest
import torch

import causal_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from bidirectional_mamba_ssm_b200 import _lib
    return _lib


def test_overlapping_long_ranges_take_no_more_than_the_rows(lib):
    """32 prompts that all name the same 2000 rows, long enough to be cut, with
    ranges that run backwards in between: the first is done, the others, more
    rows than there are, are reported and left alone."""
    shape, n, rows = (2, 64, 128), 64, 2000
    d = ref.draw(rows, n, *shape, torch.bfloat16, seed=41, pool=n, a_range=(1e-3, 1e-2))
    y, s, t = ref.run(lib, d, [0] * n, [1] * n, *shape, cu=[0, rows] * (n // 2) + [0])
    assert lib.bimamba_get_error() == lib.BIMAMBA_ERR_INVALID
    wy, ws, wt = ref.run(lib, dict(d, slots=d["slots"][:1]), [rows], [1], *shape)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    assert torch.equal(y, wy) and torch.equal(s, ws) and torch.equal(t, wt)


@pytest.mark.parametrize("heads,most,fewer", [(64, 15104, 14976), (48, 896, 768)])
def test_a_workspace_of_the_largest_call_serves_fewer_rows(lib, heads, most, fewer):
    """Row counts at which the rule cuts the smaller call into more pieces."""
    shape = (heads, 64, 128)
    d = ref.draw(fewer, 1, *shape, torch.bfloat16, seed=42, pool=1)
    ws = torch.empty(lib.bimamba_prompt_workspace_bytes(lib.make_dims(1, most, *shape, torch.bfloat16)),
                     dtype=torch.uint8, device="cuda")
    one = ref.run(lib, d, [fewer], [1], *shape, ws=ws)
    two = ref.run(lib, d, [fewer], [1], *shape)
    assert lib.bimamba_get_error() == lib.BIMAMBA_OK
    for p, q in zip(one, two):
        assert torch.equal(p, q)
