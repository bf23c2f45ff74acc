"""GPU: stochastic rounding of the states that prompts leave, code for code.

A call draws the uniforms of the state's next token for every row it rounds, and the row is the
state's, not the call's: the rows of the fp32 call's result, quantized by the oracle with those
uniforms, are the bytes that the quantized call leaves."""
import sys

import numpy as np
import pytest
import torch

import oracle
from tests import linattn_ref as ref
from tests.test_gpu_linattn import BF, F32, cu_of, state_of, values_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq
    from tests import parity as par


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,G,P", [(4, 2, 32), (60, 1, 16)])  # sequences in parts; whole ones
@pytest.mark.parametrize("fmt", ["int8_sym", "int8_asym", "int4_sym", "int4_asym"])
def test_codes_of_the_states_that_prompts_leave(fmt, H, G, P, dtype):
    say("stochastic prompts", fmt, H, G, P, dtype)
    gen = torch.Generator().manual_seed(H)
    lens, slots, fresh = [70, 0, 300, 0, 1, 9], [5, 0, 6, 2, -1, 3], [1, 0, 0, 1, 0, 1]
    B, rows, seed, step = 8, H * P, 987654321, 1 << 33
    start = torch.randn(B, H, P, 128, generator=gen)
    st = state_of(start, G, fmt)
    ssq.ssq_set_rounding(st, ssq.SSQ_ROUND_STOCHASTIC, seed, step)
    dslots = torch.tensor(slots, dtype=torch.int32, device="cuda")
    dfresh = torch.tensor(fresh, dtype=torch.uint8, device="cuda")
    for call in range(2):
        q, k, v, g = (x.cuda() for x in ref.inputs(gen, sum(lens), H, G, P, dtype))
        old = par.read_gpu_state(st, fmt)
        f32 = state_of(values_of(st), G)
        o, of = torch.zeros_like(v), torch.zeros_like(v)
        ssq.ssq_linattn_prefill(f32, q, k, v, g, of, cu_of(lens), slots=dslots, fresh=dfresh)
        ssq.ssq_linattn_prefill(st, q, k, v, g, o, cu_of(lens), slots=dslots, fresh=dfresh)
        assert torch.equal(o, of)
        assert ssq.ssq_get_rounding(st) == (ssq.SSQ_ROUND_STOCHASTIC, seed, step + call + 1)
        h, got = values_of(f32).reshape(B * rows, 128).numpy(), par.read_gpu_state(st, fmt)
        moved = {s for s, n, f in zip(slots, lens, fresh) if s >= 0 and (n or f)}
        for s in range(B):
            for r in range(s * rows, (s + 1) * rows):
                if s in moved:
                    U = oracle.sr_row_uniforms(seed, step + call, B * rows, r, 128)
                    code, scale, zero = oracle.quantize_row_sr(h[r], fmt, U)
                else:
                    code, scale, zero = (old[n][r] if old.get(n) is not None else 0 for n in ("code", "scale", "zero"))
                assert np.array_equal(got["code"][r], code), (call, s, r)
                assert got["scale"][r] == scale and (got.get("zero") is None or got["zero"][r] == zero), (call, s, r)
