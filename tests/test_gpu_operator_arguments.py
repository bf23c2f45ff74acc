"""GPU: sizes and numbers past 32 bits are refused by linear attention and beam selection: taken
modulo 2^32 they would be other, valid ones."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq

WRAP = 1 << 32


def selection(vocab, dtype=torch.float32, **kw):
    x = torch.empty(1, 1, vocab, dtype=dtype, device="cuda")
    if vocab < 100:
        x.zero_()
    out = torch.empty(1, 2, device="cuda")
    token, parent = (torch.full((1, 2), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    ssq.ssq_beam_select(x, torch.zeros(1, 1, device="cuda"), out, token, parent, **kw)
    return token


def test_a_vocabulary_past_32_bits():
    with pytest.raises(ValueError, match="vocab"):
        selection(WRAP + 5, torch.bfloat16)  # 8.6 GB that nothing reads


@pytest.mark.parametrize("pad", [WRAP, WRAP + 3, -WRAP])
def test_a_pad_token_past_32_bits(pad):
    with pytest.raises(ValueError, match="pad_token"):
        selection(8, pad_token=pad)
    assert selection(8, pad_token=3).tolist() == [[0, 1]]


def test_linear_attention():
    st = ssq.ssq_alloc_state(ssq.make_desc(ssq.SSQ_MAMBA2, "fp32", 2, 2, 16))
    q, v = torch.zeros(2, 1, 128, device="cuda"), torch.zeros(2, 2, 16, device="cuda")
    for readout in (WRAP, WRAP + 1):
        with pytest.raises(ValueError, match="readout"):
            ssq.ssq_linattn_step(st, q, q, v, None, torch.empty_like(v), readout=readout)
    for nseq, tokens in ((WRAP + 1, 100), (1, (1 << 64) + 100), (-WRAP, 0)):
        with pytest.raises(ValueError):
            ssq.ssq_linattn_workspace(st, nseq, tokens)
    assert ssq.ssq_linattn_workspace(st, 1, 100) >= 0


class StreamElsewhere:
    """What a stream of a second device looks like to a call; its handle is this device's default stream."""
    cuda_stream = 0
    device = torch.device("cuda", 1)


def test_a_stream_of_another_device():
    """Its kernels would run there, on this device's memory, and a workspace would come from there."""
    there = StreamElsewhere()
    st = ssq.ssq_alloc_state(ssq.make_desc(ssq.SSQ_MAMBA2, "int8_sym", 2, 2, 16))
    q, v = torch.zeros(2, 1, 128, device="cuda"), torch.zeros(2, 2, 16, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    parents = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    for call in (lambda: ssq.ssq_linattn_prefill(st, q, q, v, None, torch.empty_like(v), cu, stream=there),
                 lambda: ssq.ssq_linattn_step(st, q, q, v, None, torch.empty_like(v), stream=there),
                 lambda: ssq.ssq_state_reorder(st, parents, stream=there), lambda: selection(8, stream=there)):
        with pytest.raises(ValueError, match="stream"):
            call()
    ssq.ssq_state_reorder(st, parents, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
