"""GPU: the scores of a beam selection over the longest rows."""
import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq


@pytest.mark.parametrize("vocab", [1 << 28, (1 << 28) - 12345])
@pytest.mark.parametrize("below", [0.357421875, 0.51171875])
def test_the_normalizer_of_a_long_row(vocab, below):
    """The first 2^17 logits are the largest, so that each lane has some, and all others `below` them:
    log sum exp is log(2^17 + (vocab - 2^17) exp(-below)).  A lane meets 65536 tokens; summed up in fp32 one after the other they are off by 2e-5.  The
    scores are off by an fp32 rounding of theirs, 2^-24 of some 19, and by 2^-18 of the sum: 32
    additions in fp32 before a wider one, and exponentials off by (1 + below) * 2^-23."""
    print("normalizer", vocab, below, file=sys.stderr, flush=True)
    logits = torch.full((1, 1, vocab), 1.0 - below, dtype=torch.float32, device="cuda")
    assert logits[0, 0, 0].item() == 1.0 - below
    top = 1 << 17
    logits[0, 0, :top] = 1.0
    score = torch.tensor([[-2.0]], device="cuda")
    out = torch.empty(1, 2, device="cuda")
    token, parent = (torch.empty(1, 2, dtype=torch.int32, device="cuda") for _ in range(2))
    ssq.ssq_beam_select(logits, score, out, token, parent)
    assert token.tolist() == [[0, 1]] and parent.tolist() == [[0, 0]]
    want = -2.0 - math.log(top + (vocab - top) * math.exp(-below))
    for got in out[0].tolist():
        assert abs(got - want) <= abs(want) * 2.0 ** -24 + 2.0 ** -18, got - want
