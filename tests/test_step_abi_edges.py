"""Sizes past one launch of the vocabulary loss, on the CPU: refused before anything is enqueued (the device
addresses below are never dereferenced)."""
import pytest

from tests.test_product_abi import E_SHAPE, call


@pytest.mark.parametrize("tokens", [1 << 28, (1 << 31) - 256])
def test_linear_cross_entropy_of_too_many_tokens(tokens):
    """16 tokens to a workgroup of 256 where the tiles are joined, and a launch counts its work-items in 32 bits: the tiles
    of a short vocabulary alone would still fit."""
    big = dict(x=1 << 44, w=1 << 46, targets=1 << 45, tokens=tokens, vocab=17, k=32, scale=1.0, workspace=1 << 47,
               workspace_bytes=1 << 46, loss=1 << 42, lse=1 << 43, stream=None)
    assert call("trace_linear_cross_entropy", big) == E_SHAPE
