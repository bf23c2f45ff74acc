"""Cases for measuring the linear-attention, beam-search and state-reordering operators.

``run`` computes an operator either in its plain form (elementary torch operations, in 32 bits or
more, rounded once at the end) or, where ``own`` is true, through this repository's entry points.
Both update the caller's state in place, as a serving program does.
"""
import math
import random

import torch

own = False

N = 128  # entries of a state row: the key dimension
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
# -ln(decay) of a head: strongly, moderately and weakly decaying heads in turn
BANDS = (0.325, 0.0325, 0.00325)


def listed():
    return [
        # a chat turn of one request on a small model: a launch-bound call
        dict(name="prompt 77", op="prefill", dtype="bf16", heads=24, groups=1, p=64, nseq=1, mean=77, slots=4, tail=0, mix=1),
        # one document on a small model: few heads, so the sequence has to be split to fill the card
        dict(name="prompt 2048", op="prefill", dtype="bf16", heads=24, groups=1, p=64, nseq=1, mean=2048, slots=1, tail=0, mix=2),
        # a batch of prompts of unequal lengths, an empty and a one-token one among them, with padding rows behind them
        dict(name="ragged batch", op="prefill", dtype="bf16", heads=32, groups=1, p=64, nseq=24, mean=700, slots=32, tail=61, mix=3),
        # a long prompt on one layer of a large model, keys shared by 16 heads
        dict(name="prompt 8192, 128 heads", op="prefill", dtype="bf16", heads=128, groups=8, p=64, nseq=1, mean=8192, slots=1, tail=0, mix=4),
        # heads of 128 values with keys of their own, as matrix-state layers have them
        dict(name="heads of 128", op="prefill", dtype="bf16", heads=32, groups=32, p=128, nseq=3, mean=1500, slots=8, tail=0, mix=5),
        # a checking run in full precision
        dict(name="ragged fp32", op="prefill", dtype="fp32", heads=24, groups=1, p=64, nseq=5, mean=611, slots=8, tail=3, mix=6),
        # one request's next token
        dict(name="token, 1 request", op="step", dtype="bf16", format="fp32", heads=24, groups=1, p=64, nseq=1, slots=16),
        # the next token of a full batch on a large model's layer
        dict(name="token, 240 of 256", op="step", dtype="bf16", format="fp32", heads=128, groups=8, p=64, nseq=240, slots=256),
        # the next token on an 8-bit state, which is read back as the values it stands for
        dict(name="token, 8-bit state", op="step", dtype="bf16", format="int8_asym", heads=32, groups=1, p=64, nseq=61, slots=64),
        # one request's beams
        dict(name="4 beams of 50280", op="select", dtype="bf16", batch=1, beams=4, vocab=50280, nselect=4),
        # a batch of searches over a large vocabulary, twice the beams kept so that finished ones can be taken out
        dict(name="32x8 beams of 131071", op="select", dtype="fp32", batch=32, beams=8, vocab=131071, nselect=16),
        # the states of all layers of a model follow their beams
        dict(name="48 layers follow 8x4 beams", op="reorder", format="int4_asym", layers=48, heads=32, p=64, batch=32, beams=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prefill", "step", "select", "reorder"))
    if op == "prefill":
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        groups = rng.choice((1, 1, 2, 5, 8))
        heads = groups * rng.choice((1, 2, 3, 4, 8, 16))
        p = 16 * rng.choice((1, 2, 3, 4, 4, 5, 8, 8))
        nseq = _log_int(rng, 1, 24)
        most = 8192 * 128 * 64 // (2 if dtype == "bf16" else 8) // (heads * p)
        mean = _log_int(rng, 1, max(1, min(16000, most) // nseq))
        return dict(op=op, dtype=dtype, heads=heads, groups=groups, p=p, nseq=nseq, mean=mean,
                    slots=nseq + rng.randrange(4), tail=rng.choice((0, 0, 1, 37)), mix=rng.randrange(1 << 20))
    if op == "step":
        groups = rng.choice((1, 1, 3, 8))
        heads = groups * rng.choice((1, 4, 8, 16))
        p = 16 * rng.choice((1, 3, 4, 4, 8))
        slots = _log_int(rng, 1, max(1, min(256, 240 * 128 * 64 // (heads * p))))
        return dict(op=op, dtype=rng.choice(("bf16", "fp16", "fp32")), format=rng.choice(("fp32", "fp32", "int8_asym")),
                    heads=heads, groups=groups, p=p, nseq=rng.randint(max(1, slots // 2), slots), slots=slots)
    if op == "select":
        beams = rng.choice((1, 2, 3, 4, 5, 8, 16))
        vocab = _log_int(rng, 500, 150000)
        batch = _log_int(rng, 1, max(1, min(64, 32 * 8 * 131071 // (beams * vocab))))
        return dict(op=op, dtype=rng.choice(("bf16", "fp16", "fp32")), batch=batch, beams=beams, vocab=vocab,
                    nselect=rng.choice((beams, 2 * beams)))
    beams = rng.choice((2, 3, 4, 5, 8, 16))
    heads = rng.choice((8, 24, 32, 48))
    p = 16 * rng.choice((2, 4, 4, 8))
    fmt = rng.choice(("int4_asym", "int4_sym", "int8_asym", "int8_sym", "fp32"))
    group = heads * p * ROW_BYTES[fmt] * beams
    layers = max(1, min(rng.choice((1, 6, 24, 48)), (200 << 20) // group))
    most = (200 << 20) // (layers * group)
    return dict(op=op, format=fmt, layers=layers, heads=heads, p=p, batch=beams * _log_int(rng, 1, max(1, min(64, most))), beams=beams)


# ----------------------------------------------------------------------------- a state's bytes

ROW_BYTES = {"fp32": 512, "int8_sym": 128, "int8_asym": 128, "int4_sym": 64, "int4_asym": 64}


def _regions(fmt, rows):
    """Byte ranges of a state's codes, scales and zero points in its storage, and the storage's size."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    end = up(rows * ROW_BYTES[fmt])
    spans = [(0, rows * ROW_BYTES[fmt])]
    if fmt != "fp32":
        for _ in range(2 if fmt.endswith("asym") else 1):
            spans.append((end, 4 * rows))
            end = up(end + 4 * rows)
        end = up(end + 8)
    return spans, end


def _region(storage, span, dtype, *shape):
    return storage[span[0]: span[0] + span[1]].view(dtype).view(*shape)


def _storage(fmt, batch, heads, p, gen):
    """A state of `batch` sequences as it stands in the middle of generation."""
    rows = batch * heads * p
    spans, size = _regions(fmt, rows)
    s = torch.zeros(size, dtype=torch.uint8, device="cuda")
    if fmt == "fp32":
        _region(s, spans[0], torch.float32, rows, N).normal_(generator=gen)
        return s
    _region(s, spans[0], torch.uint8, -1).random_(0, 256, generator=gen)
    if fmt == "int8_sym":  # the code -128 is not on the grid
        c = _region(s, spans[0], torch.int8, -1)
        c.clamp_(min=-127)
    if fmt == "int4_sym":
        c = _region(s, spans[0], torch.uint8, -1)
        c.sub_((c & 15 == 8).to(torch.uint8)).sub_((c >> 4 == 8).to(torch.uint8) * 16)
    _region(s, spans[1], torch.float32, rows).uniform_(0.01, 0.03, generator=gen)
    if fmt.endswith("asym"):
        mid = 128 if fmt == "int8_asym" else 8
        _region(s, spans[2], torch.float32, rows).normal_(mid, mid / 16, generator=gen).round_()
    return s


def _handle(case, storage, heads, p, groups, batch):
    """The framework's handle of a state over `storage`, which it keeps as it is."""
    import mamba_decode_amd as ssq
    filled = storage.clone()
    state = ssq.ssq_alloc_state(ssq.make_desc(ssq.SSQ_MAMBA2, case["format"], batch, heads, p, N, groups), storage)
    storage.copy_(filled)
    return state


# ----------------------------------------------------------------------------- inputs


def _lengths(case):
    """Lengths of the prompts: the mean's for one, else unequal, with an empty and a one-token one among many."""
    n, mean = case["nseq"], case["mean"]
    if n == 1:
        return [mean]
    r = random.Random(case["mix"])
    lens = [max(1, int(mean * r.uniform(0.3, 1.5))) for _ in range(n)]
    if n >= 4:
        lens[r.randrange(n - 1)], lens[n - 1] = 0, 1
    return lens


def _qkvg(tokens, heads, groups, p, dtype, gen):
    d = dict(device="cuda", generator=gen)
    q, k = (torch.randn(tokens, groups, N, **d).div_(math.sqrt(N)).to(dtype) for _ in range(2))
    v = torch.randn(tokens, heads, p, **d).to(dtype)
    band = torch.tensor(BANDS, device="cuda").repeat(heads // 3 + 1)[:heads]
    g = -(torch.randn(tokens, heads, **d) * 0.7).exp() * band
    return q, k, v, g


def prepare(case, seed):
    op = case["op"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if op == "prefill":
        case = dict(case, format="fp32")
        lens = _lengths(case)
        tokens = sum(lens) + case["tail"]
        dtype = DTYPES[case["dtype"]]
        q, k, v, g = _qkvg(tokens, case["heads"], case["groups"], case["p"], dtype, gen)
        host = random.Random(seed)
        s = dict(case=case, q=q, k=k, v=v, g=g, o=torch.zeros_like(v), longest=max(lens),
                 cu=torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32),
                 slots=torch.tensor(host.sample(range(case["slots"]), case["nseq"]), dtype=torch.int32, device="cuda"),
                 fresh=torch.tensor([i % 3 != 2 for i in range(case["nseq"])], dtype=torch.uint8, device="cuda"))
        s["storage"] = _storage("fp32", case["slots"], case["heads"], case["p"], gen)
    elif op == "step":
        q, k, v, g = _qkvg(case["nseq"], case["heads"], case["groups"], case["p"], DTYPES[case["dtype"]], gen)
        host = random.Random(seed)
        s = dict(case=case, q=q, k=k, v=v, g=g, o=torch.zeros_like(v),
                 slots=torch.tensor(host.sample(range(case["slots"]), case["nseq"]), dtype=torch.int32, device="cuda"))
        s["storage"] = _storage(case["format"], case["slots"], case["heads"], case["p"], gen)
        if case["format"] != "fp32":
            s["values"] = torch.zeros(case["slots"], case["heads"], case["p"], N, device="cuda")
    elif op == "select":
        b, m, v = case["batch"], case["beams"], case["vocab"]
        logits = torch.randn(b, m, v, device="cuda", generator=gen).mul_(3.0)
        # tokens that the search may not take: -inf, or the type's lowest value, as a mask in the model writes it
        logits.masked_fill_(torch.rand(v, device="cuda", generator=gen) < 0.05, -math.inf)
        logits = logits.to(DTYPES[case["dtype"]])
        logits.masked_fill_(torch.rand(v, device="cuda", generator=gen) < 0.05, torch.finfo(logits.dtype).min)
        scores = -20 * torch.rand(b, m, device="cuda", generator=gen)
        finished = torch.rand(b, m, device="cuda", generator=gen) < 0.15
        first = torch.arange(b, device="cuda") % 4 == 3  # searches at their first token: one beam is alive
        scores[first, 1:] = -math.inf
        finished[first] = False
        s = dict(case=case, logits=logits, scores=scores, finished=finished.to(torch.uint8),
                 out_scores=torch.empty(b, case["nselect"], device="cuda"),
                 out_tokens=torch.empty(b, case["nselect"], dtype=torch.int32, device="cuda"),
                 out_parents=torch.empty(b, case["nselect"], dtype=torch.int32, device="cuda"))
        return s
    else:
        b, m = case["batch"], case["beams"]
        s = dict(case=case, parents=torch.randint(0, m, (b // m, m), device="cuda", generator=gen).to(torch.int32),
                 storages=[_storage(case["format"], b, case["heads"], case["p"], gen) for _ in range(case["layers"])])
        if own:
            s["states"] = [_handle(case, x, case["heads"], case["p"], 1, b) for x in s["storages"]]
        return s
    if own:
        s["state"] = _handle(case, s["storage"], case["heads"], case["p"], case["groups"], case["slots"])
    return s


# ----------------------------------------------------------------------------- plain forms


def _plain_prefill(s, C=64):
    """Chunks of C tokens: products inside a chunk, the states between chunks by their decays."""
    c, cu = s["case"], s["cu"].long()
    B, H, G, P = c["nseq"], c["heads"], c["groups"], c["p"]
    nc = max(1, -(-s["longest"] // C))
    at = cu[:-1, None] + torch.arange(nc * C, device="cuda")
    valid = at < cu[1:, None]
    at = at.clamp(max=s["q"].shape[0] - 1)
    pad = lambda x: torch.where(valid[..., None, None], x[at].float(), 0.0).view(B, nc, C, x.shape[1], -1).permute(0, 3, 1, 2, 4)  # noqa: E731
    q, k, v = pad(s["q"]), pad(s["k"]), pad(s["v"])  # [B][heads or groups][chunks][C][...]
    cum = pad(s["g"][..., None])[..., 0].double().cumsum(-1)  # [B][H][nc][C]
    total = cum[..., -1]
    share = lambda x: x.repeat_interleave(H // G, 1)  # noqa: E731
    low = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    inner = (cum[..., :, None] - cum[..., None, :]).masked_fill(~low, -math.inf).float().exp()
    att = share(q @ k.transpose(-1, -2).contiguous()).mul_(inner)
    o = att @ v
    del inner, att
    grown = (v * (total[..., None] - cum).float().exp()[..., None]).transpose(-1, -2).contiguous() @ share(k)  # [B][H][nc][P][N]
    # state before chunk i: decays over the chunks between, of the state at hand and of each chunk's own part
    ends = torch.cat([torch.zeros_like(total[..., :1]), total.cumsum(-1)], -1)
    earlier = torch.ones(nc + 1, nc, dtype=torch.bool, device="cuda").tril(-1)
    between = (ends[..., :, None] - ends[..., None, 1:]).masked_fill(~earlier, -math.inf).float().exp()
    slots = s["slots"].long()
    state = _region(s["storage"], _regions("fp32", c["slots"] * H * P)[0][0], torch.float32, c["slots"], H, P, N)
    start = torch.where(s["fresh"].bool()[:, None, None, None], 0.0, state[slots])
    before = (between @ grown.view(B, H, nc, P * N)).view(B, H, nc + 1, P, N)
    before += ends.float().exp()[..., None, None] * start[:, :, None]
    o += cum.float().exp()[..., None] * (share(q) @ before[:, :, :nc].transpose(-1, -2).contiguous())
    o = (o / math.sqrt(N)).permute(0, 2, 3, 1, 4).reshape(B, nc * C, H, P)
    s["o"][at[valid]] = o[valid].to(s["o"].dtype)
    state[slots] = before[:, :, nc]
    return {"o": s["o"], "state": state}


def _plain_step(s):
    c = s["case"]
    H, G, P, slots = c["heads"], c["groups"], c["p"], s["slots"].long()
    spans = _regions(c["format"], c["slots"] * H * P)[0]
    share = lambda x: x.float().repeat_interleave(H // G, 1)[:, :, None]  # noqa: E731
    lam = s["g"].double().exp().float()[..., None, None]
    write = s["v"].float()[..., None] * share(s["k"])  # one rounding of each product
    if c["format"] == "fp32":
        state = _region(s["storage"], spans[0], torch.float32, c["slots"], H, P, N)
        new = lam * state[slots] + write
        state[slots] = new
        o = ((new * share(s["q"])).sum(-1) / math.sqrt(N)).to(s["o"].dtype)
        s["o"].copy_(o)
        return {"o": s["o"], "state": state}
    codes = _region(s["storage"], spans[0], torch.uint8, c["slots"], H, P, N)
    scale, zero = (_region(s["storage"], x, torch.float32, c["slots"], H, P, 1) for x in spans[1:])
    old = scale[slots] * (codes[slots].float() - zero[slots])
    new = (lam.double() * old.double() + write.double()).float()  # one rounding
    lo, hi = new.amin(-1, keepdim=True), new.amax(-1, keepdim=True)
    step = ((hi - lo).double() / 255).float()  # values next to a border between two codes: in 64 bits
    inv = (1.0 / step.double()).float()
    z = -(lo.double() * inv.double()).round() + 0.0
    code = (new.double() * inv.double() + z).round().clamp(0, 255)
    codes[slots], scale[slots], zero[slots] = code.to(torch.uint8), step, z.float()
    read = step * (code - z).float()
    s["o"].copy_((read * share(s["q"])).sum(-1) / math.sqrt(N))
    torch.mul(codes.float().sub_(zero), scale, out=s["values"])
    return {"o": s["o"], "values": s["values"]}


def _plain_select(s):
    c = s["case"]
    b, m, v, n = c["batch"], c["beams"], c["vocab"], c["nselect"]
    x = s["logits"].double()  # sums over a long row, and scores next to each other
    top = x.amax(-1, keepdim=True)
    logp = (x - top) - (x - top).exp().sum(-1, keepdim=True).log()
    done = s["finished"].bool()[..., None]
    pad = torch.arange(v, device="cuda") == 0
    logp = torch.where(done, torch.where(pad, 0.0, -math.inf), logp)
    score = (s["scores"].double()[..., None] + logp).view(b, m * v)
    score, at = score.sort(dim=-1, descending=True, stable=True)  # the lowest index of equal scores first
    score, at = score[:, :n], at[:, :n]
    none = score == -math.inf
    s["out_scores"].copy_(score)
    s["out_tokens"].copy_(torch.where(none, -1, at % v))
    s["out_parents"].copy_(torch.where(none, torch.arange(n, device="cuda") % m, at // v))
    return {"scores": s["out_scores"], "tokens": s["out_tokens"], "parents": s["out_parents"]}


def _plain_reorder(s):
    c = s["case"]
    b, m = c["batch"], c["beams"]
    frm = (s["parents"].long() + torch.arange(0, b, m, device="cuda")[:, None]).view(-1)
    spans = _regions(c["format"], b * c["heads"] * c["p"])[0]
    parts = [_region(x, span, torch.uint8, b, -1) for x in s["storages"] for span in spans]
    [x.copy_(x[frm]) for x in parts]
    return {"layer %d" % i: x for i, x in enumerate(s["storages"])}


def run(state):
    s, c = state, state["case"]
    if own:
        import mamba_decode_amd as ssq
        if c["op"] == "prefill":
            ssq.ssq_linattn_prefill(s["state"], s["q"], s["k"], s["v"], s["g"], s["o"], s["cu"], slots=s["slots"],
                                    fresh=s["fresh"], scale=1 / math.sqrt(N))
            return {"o": s["o"], "state": s["storage"][: 4 * N * c["slots"] * c["heads"] * c["p"]].view(torch.float32).view(c["slots"], c["heads"], c["p"], N)}
        if c["op"] == "step":
            ssq.ssq_linattn_step(s["state"], s["q"], s["k"], s["v"], s["g"], s["o"], slots=s["slots"], scale=1 / math.sqrt(N))
            if c["format"] == "fp32":
                return {"o": s["o"], "state": s["storage"][: 4 * N * c["slots"] * c["heads"] * c["p"]].view(torch.float32).view(c["slots"], c["heads"], c["p"], N)}
            ssq.ssq_dequant(s["state"], s["values"])
            return {"o": s["o"], "values": s["values"]}
        if c["op"] == "select":
            ssq.ssq_beam_select(s["logits"], s["scores"], s["out_scores"], s["out_tokens"], s["out_parents"],
                                finished=s["finished"], pad_token=0)
            return {"scores": s["out_scores"], "tokens": s["out_tokens"], "parents": s["out_parents"]}
        ssq.ssq_state_reorder(s["states"], s["parents"])
        return {"layer %d" % i: x for i, x in enumerate(s["storages"])}
    return {"prefill": _plain_prefill, "step": _plain_step, "select": _plain_select, "reorder": _plain_reorder}[c["op"]](s)


# ----------------------------------------------------------------------------- what a pass has to move and compute


def work(case):
    op = case["op"]
    if op in ("prefill", "step"):
        size = 4 if case["dtype"] == "fp32" else 2
        H, G, P = case["heads"], case["groups"], case["p"]
        lens = _lengths(case) if op == "prefill" else [1] * case["nseq"]
        T = sum(lens)
        io = T * (2 * G * N * size + 2 * H * P * size + 4 * H)
        if op == "step":
            fmt = case["format"]
            row = ROW_BYTES[fmt] + (0 if fmt == "fp32" else 8)
            back = 0 if fmt == "fp32" else case["slots"] * H * P * (row + 4 * N)
            return {"bytes": io + 2 * T * H * P * row + back, "flops": T * H * P * N * 5}
        read = sum(i % 3 == 2 for i in range(len(lens)))  # sequences that go on from their state
        # the products with the state, and the ones among a chunk's own tokens, of 64
        return {"bytes": io + 4 * N * H * P * (len(lens) + read), "flops": T * H * (4 * N * P + 64 * (N + P))}
    if op == "select":
        n = case["batch"] * case["beams"] * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "fp32" else 2) + case["batch"] * (5 * case["beams"] + 12 * case["nselect"]), "flops": 4 * n}
    fmt, m = case["format"], case["beams"]
    row = ROW_BYTES[fmt] + (0 if fmt == "fp32" else 8 if fmt.endswith("asym") else 4)
    one = case["layers"] * case["heads"] * case["p"] * row
    # of parents drawn evenly: beams whose parent is another one, and beams that another one comes from
    moved, read = m - 1, m * (1 - (1 - 1 / m) ** (m - 1))
    return {"bytes": case["batch"] // m * one * (moved + read), "flops": 0}


# ----------------------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    op = case["op"]
    if op == "reorder":
        return None  # bytes that move are no computed numbers
    s = prepare(case, seed)
    if op == "select":
        x = s["logits"].double()
        rows = s["scores"].double()[..., None] + torch.log_softmax(x, -1)
        alive = s["finished"] == 0
        rows = torch.where(alive[..., None], rows, -math.inf)
        rows[..., 0] = torch.where(alive, rows[..., 0], s["scores"].double())
        best = rows.flatten(1).topk(case["nselect"]).values
        return {"scores": best, "tokens": None, "parents": None}
    H, G, P = case["heads"], case["groups"], case["p"]
    q, k, v, g = (s[n].double() for n in "qkvg")
    q, k = q.repeat_interleave(H // G, 1), k.repeat_interleave(H // G, 1)
    slots = s["slots"].long()
    if op == "step":
        spans = _regions(case["format"], case["slots"] * H * P)[0]
        if case["format"] == "fp32":
            S = _region(s["storage"], spans[0], torch.float32, case["slots"], H, P, N).double()
            S[slots] = S[slots] * g.exp()[..., None, None] + v[..., None] * k[:, :, None]
            return {"o": (S[slots] * q[:, :, None]).sum(-1) / math.sqrt(N), "state": S}
        return None  # the grid is defined by roundings to 32 bits: the plain form takes them one by one
    cu = s["cu"].tolist()
    lens = torch.tensor([b - a for a, b in zip(cu, cu[1:])], device="cuda")
    begin = s["cu"].long()[:-1]
    S = _region(s["storage"], (0, 4 * N * case["slots"] * H * P), torch.float32, case["slots"], H, P, N).double()
    h = torch.where(s["fresh"].bool()[:, None, None, None], 0.0, S[slots])
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    order = lens.argsort(descending=True)  # the longest first, so that the live ones are the first ones
    h, begin, sorted_lens = h[order], begin[order], lens[order].tolist()
    live = len(sorted_lens)
    for t in range(s["longest"]):  # one token after the other
        while sorted_lens[live - 1] <= t:
            live -= 1
        at = begin[:live] + t
        h[:live] *= g[at].exp()[..., None, None]
        h[:live].addcmul_(v[at][..., None], k[at][:, :, None])
        o[at] = (h[:live] * q[at][:, :, None]).sum(-1) / math.sqrt(N)
    S[slots[order]] = h
    return {"o": o, "state": S}
