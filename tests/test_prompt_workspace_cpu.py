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
