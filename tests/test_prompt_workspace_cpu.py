"""Sizes of the prompt scan's workspace: host queries only."""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from bidirectional_mamba_ssm_b200 import build
    build.build()
    from bidirectional_mamba_ssm_b200 import _lib
    return _lib


def _bytes(lib, heads, prompts, rows, dtype=torch.bfloat16):
    return lib.bimamba_prompt_workspace_bytes(lib.make_dims(prompts, rows, heads, 64, 128, dtype))


@pytest.mark.parametrize("heads,prompts,rows", [(48, 512, 768), (64, 256, 1024), (64, 256, 768), (64, 65535, 65535),
                                                (64, 1000, 2048), (2, 4000, 5000)])
def test_short_prompts_need_no_segments(lib, heads, prompts, rows):
    """A prompt, however short, has one chunk of operand rows (128 of 1024
    bytes and two bytes of exponents); states of segments only the few prompts
    that can be long: no more than all the rows in 16 pieces and a few cuts."""
    chunks = rows // 128 + min(prompts, rows)
    segments = 48 * (heads * 64 * 128 * 4 + 256)
    assert _bytes(lib, heads, prompts, rows) <= chunks * 128 * 1026 + 64 * (prompts + 48) + segments + 4096


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads", [2, 16, 48, 64, 96])
def test_a_larger_call_needs_no_less(lib, heads, dtype):
    """Rows and prompts each up: never fewer bytes (a workspace made for the
    largest call serves all)."""
    sizes = [[_bytes(lib, heads, prompts, rows, dtype) for rows in
              [*range(0, 40000, 331), 65536, 100000, 524288 + 127, 524288 + 128, 1 << 20, 3 << 20]]
             for prompts in (1, 2, 5, 8, 11, 64)]
    for row in sizes:
        assert all(a <= b for a, b in zip(row, row[1:]))
    for a, b in zip(sizes, sizes[1:]):
        assert all(p <= q for p, q in zip(a, b))
