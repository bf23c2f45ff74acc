"""Cases for measuring the gated recurrence, the group norm with an activation and the moves of states.

``run`` computes an operator either in its plain form (elementary torch operations, in 32 bits,
rounded once at the end) or, where ``own`` is true, through this repository's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
# -ln(decay) of a channel: strongly, moderately and weakly decaying channels in turn
BANDS = (0.325, 0.0325, 0.00325)
MOST = 8192 * 8192  # tokens x channels of the largest case in a half type
EPS = 1e-5


def listed():
    return [
        # a chat turn of one request on a small model: a launch-bound call
        dict(name="scan 77", op="scan", dtype="fp16", gate="log", input="plain", channels=1536, nseq=1, mean=77, slots=4, tail=0, mix=1),
        # a batch of prompts of unequal lengths, an empty and a one-token one among them, padding behind them
        dict(name="scan ragged", op="scan", dtype="bf16", gate="log", input="norm", channels=2048, nseq=24, mean=700, slots=32, tail=61, mix=2),
        # a long document on one layer of a large model
        dict(name="scan 8192", op="scan", dtype="bf16", gate="sigmoid", input="complement", channels=8192, nseq=1, mean=8192, slots=2, tail=0, mix=3),
        # a training step on packed documents that go on from their last piece's state
        dict(name="train packed", op="train", dtype="bf16", gate="log", input="norm", channels=4096, nseq=8, mean=2048, slots=8, tail=0, mix=4),
        # a checking run in full precision
        dict(name="train fp32", op="train", dtype="fp32", gate="sigmoid", input="complement", channels=1544, nseq=5, mean=611, slots=5, tail=3, mix=5),
        # one request's next token
        dict(name="step, 1 request", op="step", dtype="bf16", gate="log", input="norm", channels=2048, nseq=1, slots=16),
        # the next token of a full batch on a large model's layer
        dict(name="step, 240 of 256", op="step", dtype="bf16", gate="sigmoid", input="complement", channels=8192, nseq=240, slots=256),
        # heads normalised and gated after a token of a batch
        dict(name="norm of heads, 61 tokens", op="norm", dtype="bf16", act="gate_output", center=True, groups=32, width=64, tokens=61),
        # a training step of the norm before an output product, 8 groups, gated first, on a long sequence
        dict(name="norm train 8192", op="normtrain", dtype="bf16", act="gate_input", center=False, groups=8, width=1024, tokens=8192),
        # one group over all channels in full precision
        dict(name="norm train fp32", op="normtrain", dtype="fp32", act="silu", center=True, groups=1, width=4104, tokens=1999),
        # a request starts from a cached prefix: its states come from the pool of prefixes
        dict(name="prefix to 1 request", op="move", format="fp32", layers=24, heads=24, p=64, batch=16, pool=8, moves=1, kind="fetch", mix=6),
        # prompts forked to 7 continuations each, the rest of the pool freed, in all layers
        dict(name="48 layers forked", op="move", format="int4_asym", layers=48, heads=32, p=64, batch=64, pool=0, moves=56, kind="fork", mix=7),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("scan", "train", "step", "norm", "normtrain", "move"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    gates = dict(gate=rng.choice(("log", "sigmoid")), input=rng.choice(("plain", "complement", "norm")))
    most = MOST // (2 if dtype == "fp32" else 1)
    if op in ("scan", "train"):
        channels = 8 * _log_int(rng, 16, 1024)
        nseq = _log_int(rng, 1, 24)
        mean = _log_int(rng, 1, max(1, min(24000, most // channels) // nseq))
        return dict(op=op, dtype=dtype, **gates, channels=channels, nseq=nseq, mean=mean, slots=nseq + rng.randrange(4),
                    tail=rng.choice((0, 0, 1, 37)), mix=rng.randrange(1 << 20))
    if op == "step":
        slots = _log_int(rng, 1, 256)
        return dict(op=op, dtype=dtype, **gates, channels=8 * _log_int(rng, 16, 1024), nseq=rng.randint(max(1, slots // 2), slots), slots=slots)
    if op in ("norm", "normtrain"):
        width = 8 * _log_int(rng, 2, 1024)
        groups = _log_int(rng, 1, max(1, min(128, 8192 // width)))
        return dict(op=op, dtype=dtype, act=rng.choice(("silu", "gate_output", "gate_input")), center=rng.random() < 0.5, groups=groups,
                    width=width, tokens=_log_int(rng, 1, min(16384, most // (groups * width))))
    kind = rng.choice(("fetch", "fork", "compact"))
    heads, p = rng.choice((8, 24, 32, 48)), 16 * rng.choice((2, 4, 4, 8))
    fmt = rng.choice(("int4_asym", "int4_sym", "int8_asym", "int8_sym", "fp32"))
    one = heads * p * ROW_BYTES[fmt]
    batch = _log_int(rng, 2, max(2, min(256, (200 << 20) // one)))
    layers = max(1, min(rng.choice((1, 6, 24, 48)), (200 << 20) // (one * batch)))
    pool = _log_int(rng, 1, batch) if kind == "fetch" else 0
    return dict(op=op, format=fmt, layers=layers, heads=heads, p=p, batch=batch, pool=pool, moves=rng.randint(1, batch - 1),
                kind=kind, mix=rng.randrange(1 << 20))


# ----------------------------------------------------------------------------- a state's bytes

ROW_BYTES = {"fp32": 512, "int8_sym": 128, "int8_asym": 128, "int4_sym": 64, "int4_asym": 64}


def _arrays(fmt):
    return 0 if fmt == "fp32" else 2 if fmt.endswith("asym") else 1


def _regions(fmt, rows):
    """Byte ranges of a state's codes, scales and zero points in its storage, and the storage's size."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    end = up(rows * ROW_BYTES[fmt])
    spans = [(0, rows * ROW_BYTES[fmt])]
    for _ in range(_arrays(fmt)):
        spans.append((end, 4 * rows))
        end = up(end + 4 * rows)
    return spans, up(end + 8) if _arrays(fmt) else end


def _pool(case, batch, gen):
    """The states of all layers for `batch` requests, in the middle of generation."""
    out = []
    for _ in range(case["layers"]):
        rows = batch * case["heads"] * case["p"]
        spans, size = _regions(case["format"], rows)
        s = torch.zeros(size, dtype=torch.uint8, device="cuda")
        if case["format"] == "fp32":
            s[: spans[0][1]].view(torch.float32).normal_(generator=gen)
        else:
            s[: spans[0][1]].random_(0, 256, generator=gen)
            s[spans[1][0]: spans[1][0] + spans[1][1]].view(torch.float32).uniform_(0.01, 0.03, generator=gen)
            if len(spans) > 2:
                s[spans[2][0]: spans[2][0] + spans[2][1]].view(torch.float32).normal_(8, 1, generator=gen).round_()
        out.append(s)
    return out


def _handles(case, storages, batch):
    import mamba_decode_amd as ssq
    return [_handle(ssq.make_desc(ssq.SSQ_MAMBA2, case["format"], batch, case["heads"], case["p"]), s) for s in storages]


def _handle(desc, storage):
    """The framework's handle of a state over `storage`, which it keeps as it is."""
    import mamba_decode_amd as ssq
    filled = storage.clone()
    state = ssq.ssq_alloc_state(desc, storage)
    storage.copy_(filled)
    return state


def _moves(case):
    """(to, from) of each move; from -1 frees."""
    r = random.Random(case["mix"])
    b, n = case["batch"], case["moves"]
    if case["kind"] == "fetch":  # prefixes of the other pool into requests of this one
        n = min(n, b)
        return r.sample(range(b), n), [r.randrange(case["pool"]) for _ in range(n)]
    if case["kind"] == "fork":  # some requests to many others, every ninth of which is freed instead
        order = r.sample(range(b), b)
        to = order[: n]
        heads = order[n: n + max(1, min(b - n, (n + 6) // 7))]
        return to, [-1 if i % 9 == 8 else heads[i * len(heads) // n] for i in range(n)]
    live = sorted(r.sample(range(b), n))  # compaction that keeps the order, what is behind is freed
    return list(range(b)), live + [-1] * (b - n)


# ----------------------------------------------------------------------------- inputs


def _lengths(case):
    """Lengths of the sequences: the mean's for one, else unequal, with an empty and a one-token one among many."""
    n, mean = case["nseq"], case["mean"]
    if n == 1:
        return [mean]
    r = random.Random(case["mix"])
    lens = [max(1, int(mean * r.uniform(0.5, 1.5))) for _ in range(n)]
    scale = n * mean / max(n * mean, sum(lens))
    lens = [max(1, int(x * scale)) for x in lens]
    if n >= 4:
        lens[r.randrange(n - 1)], lens[n - 1] = 0, 1
    return lens


def _gates(case, tokens, gen):
    d = dict(device="cuda", generator=gen)
    c = case["channels"]
    if case["gate"] == "log":
        g = (torch.randn(tokens, c, **d) * 0.7).exp_().mul_(torch.tensor(BANDS, device="cuda").repeat(c // 3 + 1)[:c].neg_())
    else:
        g = torch.randn(tokens, c, **d).mul_(1.5).add_(torch.linspace(0.0, 6.0, c, device="cuda"))
    g.masked_fill_(torch.rand(tokens, 1, **d) < 0.0005, -math.inf)  # a new document inside a sequence
    return g.to(DTYPES[case["dtype"]])


def prepare(case, seed):
    op = case["op"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)
    if op == "move":
        to, frm = _moves(case)
        s = dict(case=case, storages=_pool(case, case["batch"], gen), sources=_pool(case, case["pool"], gen) if case["pool"] else None,
                 to=torch.tensor(to, dtype=torch.int32, device="cuda"), frm=torch.tensor(frm, dtype=torch.int32, device="cuda"))
        if own:
            s["states"] = _handles(case, s["storages"], case["batch"])
            s["from_states"] = _handles(case, s["sources"], case["pool"]) if case["pool"] else None
        return s
    dtype = DTYPES[case["dtype"]]
    d = dict(device="cuda", generator=gen)
    if op in ("norm", "normtrain"):
        shape = (case["tokens"], case["groups"], case["width"])
        s = dict(case=case, x=torch.randn(shape, **d).mul_(1.5).add_(torch.randn(shape[1:], **d)).to(dtype),
                 z=None if case["act"] == "silu" else torch.randn(shape, **d).to(dtype),
                 weight=torch.randn(shape[1:], **d).mul_(0.2).add_(1.0), bias=torch.randn(shape[1:], **d).mul_(0.1))
        s["y"] = torch.empty_like(s["x"])
        if op == "normtrain":
            s["dy"] = torch.randn(shape, **d).to(dtype)
            s["dx"], s["dz"] = torch.empty_like(s["x"]), None if s["z"] is None else torch.empty_like(s["z"])
            s["dweight"], s["dbias"] = torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
        return s
    c = case["channels"]
    lens = _lengths(case) if op != "step" else [1] * case["nseq"]
    tokens = sum(lens) + case.get("tail", 0)
    s = dict(case=case, x=torch.randn(tokens, c, **d).to(dtype), g=_gates(case, tokens, gen),
             slots=torch.tensor(host.sample(range(case["slots"]), case["nseq"]), dtype=torch.int32, device="cuda"),
             h=torch.randn(case["slots"], c, **d))
    s["o"] = torch.zeros_like(s["x"])
    if op != "step":
        s["longest"] = max(lens)
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        s["fresh"] = torch.tensor([i % 3 == 1 for i in range(case["nseq"])], dtype=torch.uint8, device="cuda")
    if op == "train":
        s["do"] = torch.randn(tokens, c, **d).to(dtype)
        s["dlast"] = torch.randn(case["nseq"], c, **d)
        s["dx"], s["dg"], s["dfirst"] = torch.zeros_like(s["x"]), torch.zeros_like(s["g"]), torch.zeros_like(s["dlast"])
    if own:
        import mamba_decode_amd as ssq
        desc = ssq.make_desc(ssq.SSQ_GATED, "fp32", case["slots"], 1, 1, c)
        s["storage"] = torch.zeros(ssq.ssq_state_bytes(desc), dtype=torch.uint8, device="cuda")
        s["state"] = ssq.ssq_alloc_state(desc, s["storage"], s["h"])
        s["h"] = s["state"].regions()[0]  # the state itself
        if op == "train":
            s["checkpoints"] = torch.empty(ssq.ssq_gated_checkpoint_rows(case["nseq"], tokens), c, device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms


def _gate(case, g, x, slopes=False):
    """a, s, s x of fp32 gates, and the slopes of a and s along the gate."""
    if case["gate"] == "log":
        a, left, da = g.exp(), -g.expm1(), g.exp()
        both = -(2 * g).expm1()  # 1 - a^2
    else:
        a, left = 1 / (1 + (-g).exp()), 1 / (1 + g.exp())
        da, both = a * left, left * (1 + a)
    s = {"plain": torch.ones_like(a), "complement": left, "norm": both.clamp(min=0).sqrt()}[case["input"]]
    if not slopes:
        return a, s * x
    ds = {"plain": torch.zeros_like(a), "complement": -da,
          "norm": torch.where(s > 0, -a * da / torch.where(s > 0, s, 1.0), 0.0)}[case["input"]]
    return a, s, da, ds


def _recur(a, b, step=16):
    """h_t = a_t h_(t-1) + b_t from zero along dim 1 of [B][T][C], `step` tokens one after the other and the steps by doubling."""
    B, T, C = b.shape
    n = max(1, -(-T // step))
    a = torch.nn.functional.pad(a, (0, 0, 0, n * step - T), value=1.0).view(B, n, step, C)
    b = torch.nn.functional.pad(b, (0, 0, 0, n * step - T)).view(B, n, step, C).clone()
    through = a.clone()
    for j in range(1, step):
        b[:, :, j] += a[:, :, j] * b[:, :, j - 1]
        through[:, :, j] *= through[:, :, j - 1]
    end, by = b[:, :, -1].clone(), through[:, :, -1].clone()
    d = 1
    while d < n:
        end[:, d:] = end[:, d:] + by[:, d:] * end[:, :-d]
        by[:, d:] = by[:, d:] * by[:, :-d]
        d *= 2
    b[:, 1:] += through[:, 1:] * end[:, :-1, None]
    return b.view(B, n * step, C)[:, :T]


def _padded(s):
    """Rows of every sequence's tokens as [B][longest], and which of them are there."""
    cu = s["cu"].long()
    at = cu[:-1, None] + torch.arange(max(1, s["longest"]), device="cuda")
    valid = at < cu[1:, None]
    return at.clamp(max=max(0, s["x"].shape[0] - 1)), valid


def _plain_scan(s):
    case, slots = s["case"], s["slots"].long()
    at, valid = _padded(s)
    a, b = _gate(case, s["g"][at].float(), s["x"][at].float())
    a, b = torch.where(valid[..., None], a, 1.0), torch.where(valid[..., None], b, 0.0)
    start = torch.where(s["fresh"].bool()[:, None], 0.0, s["h"][slots])
    b[:, 0] += a[:, 0] * start
    h = _recur(torch.cat([torch.zeros_like(a[:, :1]), a[:, 1:]], 1), b)
    s["o"][at[valid]] = h[valid].to(s["o"].dtype)
    s["h"][slots] = h[:, -1]
    return {"o": s["o"], "state": s["h"]}, at, valid, a, start, h


def _plain_train(s):
    case = s["case"]
    out, at, valid, a, start, h = _plain_scan(s)
    x = s["x"][at].float()
    _, scale, da, ds = _gate(case, s["g"][at].float(), x, slopes=True)
    before = torch.cat([start[:, None], h[:, :-1]], 1)
    dh = torch.where(valid[..., None], s["do"][at].float(), 0.0)
    dh[:, -1] += s["dlast"]  # tokens behind a sequence's end decay by 1
    back = torch.cat([torch.zeros_like(a[:, :1]), a[:, 1:].flip(1)], 1)
    dh = _recur(back, dh.flip(1)).flip(1)
    s["dx"][at[valid]] = (scale * dh)[valid].to(s["dx"].dtype)
    s["dg"][at[valid]] = (dh * (da * before + ds * x))[valid].to(s["dg"].dtype)
    s["dfirst"].copy_(a[:, 0] * dh[:, 0])
    return dict(out, dx=s["dx"], dg=s["dg"], dfirst=s["dfirst"])


def _plain_step(s):
    slots = s["slots"].long()
    a, b = _gate(s["case"], s["g"].float(), s["x"].float())
    h = a * s["h"][slots] + b
    s["h"][slots] = h
    s["o"].copy_(h)
    return {"o": s["o"], "state": s["h"]}


def _norm(s):
    case = s["case"]
    x = s["x"].float()
    z = None if s["z"] is None else s["z"].float()
    sig = None if z is None else 1 / (1 + (-z).exp())
    u = x * z * sig if case["act"] == "gate_input" else x
    c = u - u.mean(-1, keepdim=True) if case["center"] else u
    r = 1 / ((c * c).mean(-1, keepdim=True) + EPS).sqrt()
    m = c * r
    n = m * s["weight"] + s["bias"]
    if case["act"] == "silu":
        sig = 1 / (1 + (-n).exp())
        y = n * sig
    else:
        y = n * z * sig if case["act"] == "gate_output" else n
    s["y"].copy_(y)
    return x, z, sig, r, m, n


def _plain_normtrain(s):
    case = s["case"]
    x, z, sig, r, m, n = _norm(s)
    dn = s["dy"].float()
    if case["act"] == "silu":
        dn = dn * sig * (1 + n * (1 - sig))
    elif case["act"] == "gate_output":
        s["dz"].copy_(dn * n * sig * (1 + z * (1 - sig)))
        dn = dn * z * sig
    s["dweight"].copy_((dn * m).sum(0))
    s["dbias"].copy_(dn.sum(0))
    dm = dn * s["weight"]
    du = dm - m * (dm * m).mean(-1, keepdim=True)
    if case["center"]:
        du = du - dm.mean(-1, keepdim=True)
    du = du * r
    if case["act"] == "gate_input":
        s["dz"].copy_(du * x * sig * (1 + z * (1 - sig)))
        du = du * z * sig
    s["dx"].copy_(du)
    return _norm_outputs(s)


def _norm_outputs(s):
    out = {"y": s["y"], "dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    return out if s["dz"] is None else dict(out, dz=s["dz"])


def _plain_move(s):
    c, to, frm = s["case"], s["to"].long(), s["frm"].long()
    for i, dst in enumerate(s["storages"]):
        src = s["sources"][i] if s["sources"] else dst
        there = [src[a: a + n].view(c["pool"] or c["batch"], -1) for a, n in _regions(c["format"], (c["pool"] or c["batch"]) * c["heads"] * c["p"])[0]]
        here = [dst[a: a + n].view(c["batch"], -1) for a, n in _regions(c["format"], c["batch"] * c["heads"] * c["p"])[0]]
        for x, y in zip(here, there):
            x[to] = torch.where(frm[:, None] >= 0, y[frm.clamp(min=0)], 0)
    return {"layer %d" % i: x for i, x in enumerate(s["storages"])}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "norm":
            _norm(s)
            return {"y": s["y"]}
        if op == "scan":
            return _plain_scan(s)[0]
        return {"train": _plain_train, "step": _plain_step, "normtrain": _plain_normtrain, "move": _plain_move}[op](s)
    import mamba_decode_amd as ssq
    if op == "move":
        ssq.ssq_state_move(s["states"], s["to"], s["frm"], sources=s["from_states"])
        return {"layer %d" % i: x for i, x in enumerate(s["storages"])}
    if op in ("norm", "normtrain"):
        how = dict(act={"silu": ssq.SSQ_ACT_SILU, "gate_output": ssq.SSQ_ACT_GATE_OUTPUT, "gate_input": ssq.SSQ_ACT_GATE_INPUT}[c["act"]],
                   center=c["center"], eps=EPS, weight=s["weight"], bias=s["bias"], z=s["z"])
        ssq.ssq_group_norm(s["x"], s["y"], **how)
        if op == "norm":
            return {"y": s["y"]}
        ssq.ssq_group_norm_backward(s["dy"], s["x"], s["dx"], dz=s["dz"], dweight=s["dweight"], dbias=s["dbias"], **how)
        return _norm_outputs(s)
    how = dict(gate={"log": ssq.SSQ_GATE_LOG, "sigmoid": ssq.SSQ_GATE_SIGMOID}[c["gate"]],
               input={"plain": ssq.SSQ_INPUT_PLAIN, "complement": ssq.SSQ_INPUT_COMPLEMENT, "norm": ssq.SSQ_INPUT_NORM}[c["input"]])
    if op == "step":
        ssq.ssq_gated_step(s["state"], s["x"], s["g"], s["o"], slots=s["slots"], **how)
        return {"o": s["o"], "state": s["h"]}
    ssq.ssq_gated_scan(s["state"], s["x"], s["g"], s["o"], s["cu"], slots=s["slots"], fresh=s["fresh"],
                       checkpoints=s.get("checkpoints"), **how)
    out = {"o": s["o"], "state": s["h"]}
    if op == "train":
        ssq.ssq_gated_scan_backward(s["checkpoints"], s["x"], s["g"], s["do"], s["dx"], s["dg"], s["cu"], dlast=s["dlast"],
                                    dfirst=s["dfirst"], **how)
        out.update(dx=s["dx"], dg=s["dg"], dfirst=s["dfirst"])
    return out


# ----------------------------------------------------------------------------- what a pass has to move and compute


def work(case):
    op = case["op"]
    if op == "move":
        to, frm = _moves(case)
        row = ROW_BYTES[case["format"]] + 4 * _arrays(case["format"])
        one = case["layers"] * case["heads"] * case["p"] * row
        moved = [(t, f) for t, f in zip(to, frm) if case["pool"] or t != f]
        return {"bytes": one * (len(moved) + len({f for _, f in moved if f >= 0})), "flops": 0}
    size = 4 if case["dtype"] == "fp32" else 2
    if op in ("norm", "normtrain"):
        n = case["tokens"] * case["groups"] * case["width"]
        par = 4 * case["groups"] * case["width"]
        one = 1 if case["act"] == "silu" else 2  # x, and z
        if op == "norm":
            return {"bytes": n * size * (one + 1) + 2 * par, "flops": 12 * n}
        return {"bytes": n * size * (one + 1 + 2 * one + 1) + 6 * par, "flops": 40 * n}
    c = case["channels"]
    lens = [1] * case["nseq"] if op == "step" else _lengths(case)
    n = sum(lens) * c
    read = len(lens) if op == "step" else sum(i % 3 != 1 for i in range(len(lens)))  # sequences that go on from their state
    fwd = {"bytes": 3 * n * size + 4 * c * (len(lens) + read), "flops": 8 * n}
    if op != "train":
        return fwd
    return {"bytes": fwd["bytes"] + 5 * n * size + 8 * c * len(lens), "flops": 28 * n}


# ----------------------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    op = case["op"]
    if op == "move":
        return None  # bytes that move are no computed numbers
    if op in ("scan", "train") and max(_lengths(case)) > 50000:
        return None  # one token after the other would take too long
    s = prepare(case, seed)
    if op in ("norm", "normtrain"):
        return _exact_norm(s)
    H = s["h"].double()
    x, g = s["x"].double(), s["g"].double()
    if case["gate"] == "log":
        a = torch.exp(g)
        keep = {"plain": None, "complement": -torch.expm1(g), "norm": torch.sqrt(-torch.expm1(2 * g))}[case["input"]]
    else:
        a = torch.sigmoid(g)
        keep = {"plain": None, "complement": torch.sigmoid(-g), "norm": torch.sqrt(torch.sigmoid(-g) * (1 + a))}[case["input"]]
    slots = s["slots"].long()
    b = x if keep is None else keep * x
    if op == "step":
        H[slots] = a * H[slots] + b
        return {"o": H[slots], "state": H}
    cu = s["cu"].tolist()
    lens = torch.tensor([q - p for p, q in zip(cu, cu[1:])], device="cuda")
    order = lens.argsort(descending=True)  # the longest first, so that the live ones are the first ones
    begin, sizes = s["cu"].long()[:-1][order], lens[order].tolist()
    h = torch.where(s["fresh"].bool()[:, None], 0.0, H[slots])[order]
    o = torch.zeros_like(x)
    previous = torch.zeros_like(x) if op == "train" else None
    live = [sum(n > t for n in sizes) for t in range(max(sizes))]
    for t, m in enumerate(live):
        at = begin[:m] + t
        if op == "train":
            previous[at] = h[:m]
        h[:m] = a[at] * h[:m] + b[at]
        o[at] = h[:m]
    H[slots[order]] = h
    if op == "scan":
        return {"o": o, "state": H}
    dh, dx, dg = s["dlast"].double()[order], torch.zeros_like(x), torch.zeros_like(x)
    grad = s["do"].double()
    for t in reversed(range(len(live))):  # dh: of the state behind token t
        at = begin[: live[t]] + t
        m = live[t]
        total = grad[at] + dh[:m]
        dx[at] = total
        dh[:m] = a[at] * total
    dfirst = torch.empty_like(dh)
    dfirst[order] = dh
    slope = a if case["gate"] == "log" else a * torch.sigmoid(-g)
    dg = dx * slope * previous
    if keep is not None:
        bend = -slope if case["input"] == "complement" else torch.where(keep > 0, -a * slope / keep, 0.0)
        dg = dg + dx * torch.where(keep > 0, bend, 0.0) * x
        dx = dx * keep
    rows = torch.zeros(x.shape[0], 1, dtype=torch.bool, device="cuda")
    rows[: cu[-1]] = True
    return {"o": o, "state": H, "dx": torch.where(rows, dx, 0.0), "dg": torch.where(rows, dg, 0.0), "dfirst": dfirst}


def _exact_norm(s):
    """The norm in 64 bits, its gradients by torch's differentiation of the definition."""
    case = s["case"]
    x, w, b = (s[k].double().requires_grad_() for k in ("x", "weight", "bias"))
    z = None if s["z"] is None else s["z"].double().requires_grad_()
    swish = lambda v: v * torch.sigmoid(v)  # noqa: E731
    u = x * swish(z) if case["act"] == "gate_input" else x
    var = u.var(-1, unbiased=False, keepdim=True) if case["center"] else u.square().mean(-1, keepdim=True)
    n = (u - u.mean(-1, keepdim=True) if case["center"] else u) * torch.rsqrt(var + EPS) * w + b
    y = swish(n) if case["act"] == "silu" else n * swish(z) if case["act"] == "gate_output" else n
    if case["op"] == "norm":
        return {"y": y.detach()}
    grads = torch.autograd.grad(y, [x, w, b] + ([] if z is None else [z]), s["dy"].double())
    return {"y": y.detach(), **dict(zip(("dx", "dweight", "dbias", "dz"), grads))}
