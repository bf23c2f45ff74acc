"""GPU: linear attention, selection and reordering on states and tensors past 4 GiB.

A call that reaches past byte 2^32 is compared, byte for byte where the same kernel runs, with the
same call on a small state or tensor that holds copies of the sequences it names; what it does not
name stays as it was."""
import sys

import pytest
import torch

from tests import linattn_ref as ref
from tests.test_gpu_beam import reference
from tests.test_gpu_linattn import BF, F32, check_o, check_state, cu_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mamba_decode_amd as ssq

H, P, G = 128, 64, 1


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def new_state(fmt, batch):
    desc = ssq.make_desc(ssq.SSQ_MAMBA2, fmt, batch, H, P, 128, G)
    return ssq.ssq_alloc_state(desc, torch.zeros(ssq.ssq_state_bytes(desc), dtype=torch.uint8, device="cuda"))


def by_sequence(st):
    """Codes (or fp32 rows), scales and zero points as [batch][...]."""
    return [x.view(st.desc.batch, -1) for x in st.regions() if x is not None]


@pytest.mark.parametrize("fmt,batch", [("fp32", 1100), ("int8_asym", 4200)])
def test_linear_attention_on_a_large_state(fmt, batch):
    say("large state", fmt, batch)
    assert batch * H * P * (512 if fmt == "fp32" else 128) > 1 << 32
    named = [batch - 1, 0, batch - 2, batch // 2, 1]
    big, small = new_state(fmt, batch), new_state(fmt, len(named))
    slots = torch.tensor(named, dtype=torch.int32, device="cuda")
    lens = [40, 0, 130, 1, 65]
    gen = torch.Generator().manual_seed(batch)
    for turn in range(2):  # the second reads what the first has stored
        q, k, v, g = (x.cuda() for x in ref.inputs(gen, sum(lens), H, G, P, BF))
        o, o2 = torch.zeros_like(v), torch.zeros_like(v)
        ssq.ssq_linattn_prefill(big, q, k, v, g, o, cu_of(lens), slots=slots)
        ssq.ssq_linattn_prefill(small, q, k, v, g, o2, cu_of(lens))
        assert torch.equal(o, o2)
        n = len(named)
        ssq.ssq_linattn_step(big, q[:n], k[:n], v[:n], g[:n], o[:n], slots=slots)
        ssq.ssq_linattn_step(small, q[:n], k[:n], v[:n], g[:n], o2[:n])
        assert torch.equal(o, o2)
        for x, y in zip(by_sequence(big), by_sequence(small)):
            assert torch.equal(x[slots.long()], y) and y.any()
    for x in by_sequence(big):
        x[slots.long()] = 0
        assert not any(part.any() for part in x.split(64)), "sequences that no slot names"


@pytest.mark.parametrize("fmt", ["int8_sym", "fp32"])
def test_tokens_of_a_whole_large_state(fmt):
    """A call over every sequence, with outputs past 32-bit counts of bytes in the state."""
    batch = 4200 if fmt == "int8_sym" else 1100
    say("whole large state", fmt, batch)
    big = new_state(fmt, batch)
    gen = torch.Generator(device="cuda").manual_seed(1)
    d = dict(device="cuda", generator=gen)
    q, k = (torch.randn(batch, G, 128, **d).div_(11).to(BF) for _ in range(2))
    v, g = torch.randn(batch, H, P, **d).to(BF), -torch.rand(batch, H, **d)
    o = torch.zeros_like(v)
    for _ in range(2):
        ssq.ssq_linattn_step(big, q, k, v, g, o)
    for a in (0, batch // 2, batch - 3):
        span = slice(a, a + 3)
        small = new_state(fmt, 3)
        o2 = torch.zeros_like(v[span])
        for _ in range(2):
            ssq.ssq_linattn_step(small, q[span], k[span], v[span], g[span], o2)
        assert torch.equal(o[span], o2)
        for x, y in zip(by_sequence(big), by_sequence(small)):
            assert torch.equal(x[span], y) and y.any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompts_at_the_ends_of_large_tensors(dtype):
    """v and o of more than 4 GiB: a sequence at their start, one that is skipped, one at their end."""
    size = 2 if dtype == BF else 4
    T = (1 << 32) // (H * P * size) + 500
    say("large tensors", dtype, T)
    lens, heads = [50, T - 50 - 70 - 9, 70], H
    gen = torch.Generator().manual_seed(size)
    ends = [(0, 50), (T - 79, T - 9)]
    q, k = (torch.zeros(T, G, 128, dtype=dtype, device="cuda") for _ in range(2))
    v, o = torch.zeros(T, heads, P, dtype=dtype, device="cuda"), torch.zeros(T, heads, P, dtype=dtype, device="cuda")
    g = torch.zeros(T, heads, device="cuda")
    parts = [[x.cuda() for x in ref.inputs(gen, b - a, heads, G, P, dtype)] for a, b in ends]
    for (a, b), part in zip(ends, parts):
        for x, y in zip((q, k, v, g), part):
            x[a:b] = y
    big, small = new_state("fp32", 2), new_state("fp32", 2)
    slots = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")
    ssq.ssq_linattn_prefill(big, q, k, v, g, o, cu_of(lens), slots=slots)
    both = [torch.cat(x) for x in zip(*parts)]
    o2 = torch.zeros_like(both[2])
    ssq.ssq_linattn_prefill(small, *both, o2, cu_of([50, 70]), slots=torch.tensor([1, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(torch.cat([o[a:b] for a, b in ends]), o2) and o2.any()
    assert torch.equal(by_sequence(big)[0], by_sequence(small)[0])
    assert not any(part.any() for part in o[50:T - 79].split(4096)) and not o[T - 9:].any()


def test_selection_from_large_logits():
    """The scores of the first and the last requests of 4.3 GB of logits, against 64 bits: one rounding
    to fp32, and 2^-18 for the sum."""
    b, m, v, n = 2060, 4, 131071, 8
    assert b * m * v * 4 > 1 << 32
    say("large logits", b, m, v)
    gen = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.empty(b, m, v, device="cuda").normal_(0, 3, generator=gen)
    scores = -10 * torch.rand(b, m, device="cuda", generator=gen)
    out = torch.empty(b, n, device="cuda")
    token, parent = (torch.empty(b, n, dtype=torch.int32, device="cuda") for _ in range(2))
    ssq.ssq_beam_select(logits, scores, out, token, parent)
    for span in (slice(0, 3), slice(b - 3, b)):
        val, tok, par = reference(logits[span].cpu(), scores[span].cpu(), None, n, 0)
        off = (out[span].cpu().double() - val).abs()
        assert (off <= val.abs() * 2.0 ** -24 + 2.0 ** -18).all()
        assert (val[:, :-1] - val[:, 1:]).min() > 2.0 ** -17  # no near tie: choices can be compared
        assert torch.equal(token[span].cpu().long(), tok) and torch.equal(parent[span].cpu().long(), par)


@pytest.mark.parametrize("fmt,batch", [("int8_asym", 4200), ("fp32", 1104)])
def test_a_large_state_follows_its_beams(fmt, batch):
    say("large reorder", fmt, batch)
    beams = 4
    st = new_state(fmt, batch)
    gen = torch.Generator(device="cuda").manual_seed(4)
    st.storage.random_(0, 256, generator=gen)
    before = st.storage.clone()
    parents = torch.randint(0, beams, (batch // beams, beams), device="cuda", generator=gen).to(torch.int32)
    ssq.ssq_state_reorder(st, parents)
    old = ssq.State(None, st.desc, st.layout, before)
    frm = (parents.long() + torch.arange(0, batch, beams, device="cuda")[:, None]).view(-1)
    for x, y in zip(by_sequence(st), by_sequence(old)):
        x, y = x.view(torch.uint8).view(batch, -1), y.view(torch.uint8).view(batch, -1)
        for i in range(0, batch, 60):  # a slice's copies at a time
            assert torch.equal(x[i:i + 60], y[frm[i:i + 60]])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_prompt_of_millions_of_tokens(dtype):
    """Split into parts, tokens past byte 2^32 of q and v: what the state has forgotten (e^-150 over 300
    tokens is 0) does not count, so that any tokens can be checked from those shortly before them."""
    T = (1 << 25) + 77 if dtype == BF else (1 << 24) + 77
    say("one long prompt", dtype, T)
    gen = torch.Generator(device="cuda").manual_seed(5)
    d = dict(device="cuda", dtype=dtype, generator=gen)
    q, k = (torch.randn(T, 1, 128, **d).div_(11) for _ in range(2))
    v = torch.randn(T, 1, 64, **d)
    g = torch.rand(T, 1, device="cuda", generator=gen).mul_(-0.2).sub_(0.5)
    o = torch.zeros_like(v)
    assert v.numel() * v.element_size() > 1 << 32
    desc = ssq.make_desc(ssq.SSQ_MAMBA2, "fp32", 1, 1, 64, 128, 1)
    st = ssq.ssq_alloc_state(desc, torch.zeros(ssq.ssq_state_bytes(desc), dtype=torch.uint8, device="cuda"))
    ssq.ssq_linattn_prefill(st, q, k, v, g, o, cu_of([T]))
    for end in (600, T // 2 + 5, T):
        span = slice(end - 600, end)
        wo, ws, om, sm = ref.recurrence(*(x[span].cpu() for x in (q, k, v, g)), torch.zeros(1, 64, 128), 1.0)
        check_o(o[end - 300:end].cpu(), wo[300:], om[300:], 600, dtype, end)
        if end == T:
            check_state(by_sequence(st)[0].view(1, 64, 128).cpu(), ws, sm, 600, end)
