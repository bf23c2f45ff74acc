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


@pytest.mark.parametrize("dtype,bits,patterns", [(torch.bfloat16, torch.int16, (0x7F81, -0x7F, 0x7FC0, -1)), (torch.float16, torch.int16, (0x7C01, -0x3FF, 0x7E00, -1)),
                                                 (torch.float32, torch.int32, (0x7F800001, -0x7FFFFF, 0x7FC00000, -1))])
def test_every_kind_of_nan_is_no_candidate(dtype, bits, patterns):
    """Signalling and quiet ones, of either sign."""
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(2, 3, 20000, generator=gen).to(dtype)
    hit = torch.rand(x.shape, generator=gen)
    for i, p in enumerate(patterns):
        x.view(bits)[(hit > 0.2 * i) & (hit <= 0.2 * i + 0.2)] = p
    assert 0.7 < x.isnan().float().mean() < 0.9
    clean = torch.where(x.isnan(), -math.inf, x.float()).to(dtype)
    scores = -torch.rand(2, 3, generator=gen)
    outs = []
    for y in (x, clean):
        out = torch.empty(2, 6, device="cuda")
        token, parent = (torch.empty(2, 6, dtype=torch.int32, device="cuda") for _ in range(2))
        ssq.ssq_beam_select(y.cuda(), scores.cuda(), out, token, parent)
        outs.append((out, token, parent))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
