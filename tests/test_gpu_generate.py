"""GPU: the linear-attention and beam-search calls together, as a program uses them: prompts into
the states of two layers, the first tokens chosen, the states copied to their beams, then token
after token: a step of each layer, logits, a selection, and the states follow their beams.

The reference is the same program in 64 bits on the CPU.  Choices are compared exactly: the test's
logits are integers times a step far above the differences of rounding, plus a part from the
layers' outputs that is scaled below that step, so that no near tie decides (the gap is checked).
A second run replays the loop's body from one captured graph."""
import math
import sys

import pytest
import torch

from tests import linattn_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq

LAYERS, REQUESTS, BEAMS, H, G, P, VOCAB, STEPS = 2, 3, 4, 4, 2, 32, 1000, 5


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def program(seed):
    """Inputs of every layer for the prompts and for each (step, beam), and a table of logits."""
    gen = torch.Generator().manual_seed(seed)
    lens = [37, 1, 90]
    prompts = [ref.inputs(gen, sum(lens), H, G, P, torch.float32) for _ in range(LAYERS)]
    tokens = [[ref.inputs(gen, REQUESTS * BEAMS, H, G, P, torch.float32) for _ in range(LAYERS)] for _ in range(STEPS)]
    table = torch.randn(STEPS + 1, REQUESTS * BEAMS, VOCAB, generator=gen) * 2
    out = torch.randn(H * P, 8, generator=gen) / 50
    return lens, prompts, tokens, table, out


def mix(table, o, out):
    """Logits of a step: the table's, the first 8 tokens moved by the layers' outputs."""
    x = table.clone()
    x[:, :8] += o.reshape(o.shape[0], -1) @ out.to(o)
    return x


def reference(lens, prompts, tokens, table, out):
    states = torch.zeros(LAYERS, REQUESTS * BEAMS, H, P, 128, dtype=torch.float64)
    last = torch.zeros(REQUESTS * BEAMS, H, P, dtype=torch.float64)
    at = 0
    for r, n in enumerate(lens):
        for layer, (q, k, v, g) in enumerate(prompts):
            span = slice(at, at + n)
            o, s, _, _ = ref.recurrence(q[span], k[span], v[span], g[span], torch.zeros(H, P, 128), 1.0)
            states[layer, r * BEAMS:(r + 1) * BEAMS] = s
            last[r * BEAMS:(r + 1) * BEAMS] += o[-1]
        at += n
    scores = torch.full((REQUESTS, BEAMS), -math.inf, dtype=torch.float64)
    scores[:, 0] = 0.0
    chosen, gap = [], math.inf
    for t in range(STEPS + 1):
        logp = torch.log_softmax(mix(table[t].double(), last, out), -1)
        cand = (scores.reshape(-1, 1) + logp).reshape(REQUESTS, -1)
        best = cand.topk(BEAMS + 1)
        gap = min(gap, (best.values[:, :-1] - best.values[:, 1:]).min().item())
        scores, flat = best.values[:, :BEAMS], best.indices[:, :BEAMS]
        parents = flat // VOCAB
        chosen.append((flat % VOCAB, parents))
        frm = (parents + torch.arange(0, REQUESTS * BEAMS, BEAMS)[:, None]).reshape(-1)
        states = states[:, frm]
        if t == STEPS:
            break
        last = torch.zeros_like(last)
        for layer, (q, k, v, g) in enumerate(tokens[t]):
            for b in range(REQUESTS * BEAMS):
                o, s, _, _ = ref.recurrence(q[b:b + 1], k[b:b + 1], v[b:b + 1], g[b:b + 1], states[layer, b], 1.0)
                states[layer, b], last[b] = s, last[b] + o[0]
    return chosen, scores, states, gap


@pytest.mark.parametrize("graph", [False, True])
def test_prompts_tokens_beams_and_their_states(graph):
    say("generate", "graph" if graph else "eager")
    lens, prompts, tokens, table, out = program(3)
    want, scores, states, gap = reference(lens, prompts, tokens, table, out)
    assert gap > 1e-4  # far above fp32's differences, so that choices can be compared
    dev = [[x.cuda() for x in p] for p in prompts]
    layers = [ssq.ssq_alloc_state(ssq.make_desc(ssq.SSQ_MAMBA2, "fp32", REQUESTS * BEAMS, H, P, 128, G)) for _ in range(LAYERS)]
    slots = torch.arange(0, REQUESTS * BEAMS, BEAMS, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    fresh = torch.ones(REQUESTS, dtype=torch.uint8, device="cuda")
    ends = (cu[1:] - 1).long()
    last = torch.zeros(REQUESTS, H, P, device="cuda")
    for st, (q, k, v, g) in zip(layers, dev):
        o = torch.empty_like(v)
        ssq.ssq_linattn_prefill(st, q, k, v, g, o, cu, slots=slots, fresh=fresh)
        last += o[ends]
    last = last.repeat_interleave(BEAMS, 0)
    score = torch.full((REQUESTS, BEAMS), -math.inf, device="cuda")
    score[:, 0] = 0.0
    new = torch.empty_like(score)
    token, parent = (torch.empty(REQUESTS, BEAMS, dtype=torch.int32, device="cuda") for _ in range(2))
    outw, step_table = out.cuda(), table[0].cuda()
    ins = [[torch.empty_like(x).cuda() for x in tokens[0][0]] for _ in range(LAYERS)]
    outs = [torch.empty(REQUESTS * BEAMS, H, P, device="cuda") for _ in range(LAYERS)]

    def choose():
        logits = mix(step_table, last, outw).view(REQUESTS, BEAMS, VOCAB)
        ssq.ssq_beam_select(logits, score, new, token, parent)
        score.copy_(new)
        ssq.ssq_state_reorder(layers, parent)

    def advance():
        last.zero_()
        for st, (q, k, v, g), o in zip(layers, ins, outs):
            ssq.ssq_linattn_step(st, q, k, v, g, o)
            last.add_(o)
        choose()

    choose()
    got = [(token.cpu().long(), parent.cpu().long())]
    captured = None
    for t in range(STEPS):
        step_table.copy_(table[t + 1])
        for to, frm in zip(ins, tokens[t]):
            for x, y in zip(to, frm):
                x.copy_(y)
        if graph and captured is None and t == 1:  # after an eager pass
            captured = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(captured):
                advance()
        if captured is not None:
            captured.replay()
        else:
            advance()
        got.append((token.cpu().long(), parent.cpu().long()))
    for t, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), t
    assert (score.cpu().double() - scores).abs().max() < 1e-4
    for st, w in zip(layers, states):
        x = torch.empty(REQUESTS * BEAMS, H, P, 128, device="cuda")
        ssq.ssq_dequant(st, x)
        assert torch.allclose(x.cpu().double(), w, rtol=0, atol=2e-5 * w.abs().max().item())
