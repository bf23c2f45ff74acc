"""GPU: what stands beside a channel, a sequence or a slot that holds NaN comes out bit for bit as without it, every output and
every row of the states compared."""
import sys

import pytest
import torch

from tests import gated_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq
    from tests.test_gpu_gated import state_of, values_of

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("C,at,bad", [(72, (10, 100, 101, 330), 7), (40, (0, 700, 1500, 2600), 0), (2056, (3, 40, 41, 90), 2055)])
def test_neighbours_of_nan(dtype, C, at, bad):
    """Sequences 0, 1 (one token) and 2 in slots 2, 4 and 0 of 5; NaN in sequence 1, in channel `bad` of sequence 2, around the
    sequences, in the states of the slots that nobody names and of the fresh sequence 0."""
    print("neighbours", dtype, C, file=sys.stderr, flush=True)
    gen = torch.Generator().manual_seed(C)
    T = at[-1] + 70
    x, g = (t.cuda() for t in ref.inputs(gen, T, C, dtype, 1))
    do = torch.randn(T, C, generator=gen).to(dtype).cuda()
    start, dlast = torch.randn(5, C, generator=gen), torch.randn(3, C, generator=gen).cuda()
    cu, slots = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (at, (2, 4, 0)))
    fresh = torch.tensor([1, 0, 0], dtype=torch.uint8, device="cuda")
    runs = []
    for dirty in (False, True):
        st = state_of(start)
        if dirty:
            for t in (x, g, do):
                t[:at[0]] = t[at[3]:] = t[at[1]:at[2]] = torch.nan
                t[at[2] + 20, bad] = torch.nan
            st.regions()[0][1:4] = torch.nan
        o, dx, dg = (torch.zeros_like(x) for _ in range(3))
        ck = torch.full((ssq.ssq_gated_checkpoint_rows(3, T), C), torch.nan, device="cuda")
        dfirst = torch.zeros(3, C, device="cuda")
        ssq.ssq_gated_scan(st, x, g, o, cu, gate=1, input=2, slots=slots, fresh=fresh, checkpoints=ck)
        ssq.ssq_gated_scan_backward(ck, x, g, do, dx, dg, cu, gate=1, input=2, dlast=dlast, dfirst=dfirst, state=st, slots=slots)
        runs.append([t.cpu() for t in (o, dx, dg, dfirst)] + [values_of(st)])
    clean, dirty = runs
    other = torch.arange(C) != bad
    for a, b in zip(clean[:3], dirty[:3]):
        assert torch.equal(a[:at[1]], b[:at[1]])                              # around the first sequence and in it
        assert torch.equal(a[at[2]:at[3], other], b[at[2]:at[3], other])      # the last one's other channels
        assert torch.equal(a[at[3]:], b[at[3]:]) and (b[at[3]:] == 0).all()   # rows of no sequence stay
    assert torch.equal(clean[3][0], dirty[3][0]) and torch.equal(clean[3][2, other], dirty[3][2, other])  # dfirst
    assert torch.equal(clean[4][2], dirty[4][2]) and torch.equal(clean[4][0, other], dirty[4][0, other])  # states
    assert torch.equal(clean[4][[1, 3]], start[[1, 3]]) and dirty[4][[1, 3]].isnan().all()
