"""The int8 expert block on tokens that stand in a wider buffer: what it gives for the same tokens by themselves."""
import pytest
import torch

from tests.test_gpu_int8_example import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden", [(1, 64), (37, 200)])
def test_tokens_at_a_pitch(tokens, hidden):
    block = make(tokens, 16, 4, 3, hidden, 72, 5)[0]
    wide = torch.randn(tokens, hidden + 24, device="cuda", dtype=torch.bfloat16)
    x = wide[:, :hidden]
    want, logits = block(x.contiguous()), block.logits.clone()
    y = block(x)
    assert torch.equal(block.logits, logits) and torch.equal(y, want)
