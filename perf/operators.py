"""The operators that stand beside the recurrent language model's own path, as a program calls them.

Three operators belong together: a population of language models that share their weights and differ
by a low-rank term each (antithetic pairs of probes, or the adapters of several requests) is
  * projected  (adapters: y = x W^T + b + s (x D_a^T) U_a^T, adapter a and scale s by row),
  * run over its tokens by a state space recurrence with its short causal convolution (scan: whole
    prompts, or one token for each of many sequences), and
  * scored against a teacher's top logits (distill: the loss by row and its mean by model, or the loss
    and its gradient).

With `own` False `run` computes them from elementary torch operations in 32 bits (the scan's running
sums of log-decays in 64); with `own` True it calls the library.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


# --- the cases ---------------------------------------------------------------------------------


def listed():
    return [
        # One sequence is being generated: one token through one layer of 16 heads of 64 (width 1024).
        _scan("scan step, one row", "step", 1, 1, 16, 64, 1, 128, 4, "bf16", gate=True, carry=True),
        # A serving batch, width 4096; seven of its 256 rows are padding. The largest state traffic.
        _scan("scan step, 256 rows", "step", 256, 256, 64, 64, 1, 128, 4, "bf16", gate=True, carry=True, pad=7),
        # One long prompt, width 4096: few rows, so the time axis has to be split.
        _scan("scan prompt, 1 x 8192", "prompt", 1, 8192, 64, 64, 1, 128, 4, "bf16", gate=True, carry=True),
        # A ragged batch of prompts and continued prompts in float32, two groups, odd head width.
        _scan("scan prompt, ragged f32", "ragged", 33, 9001, 14, 40, 2, 100, 3, "f32", gate=False, carry=True),
        # The character language model's batch: 1,024 sequences of 10 tokens, no state kept.
        _scan("scan prompt, 1024 x 10", "prompt", 1024, 10240, 16, 64, 1, 64, 4, "bf16", gate=True, carry=False),
        # One token's gate projection, 1024 -> 4096, with one request's adapter: latency.
        _adapters("adapters, one row", 1, 1024, 4096, 1, 16, "bf16", "single", bias=True),
        # A decode step of 48 requests over 40 adapters at the 1.1B model's width.
        _adapters("adapters, 48 requests", 48, 5888, 5888, 40, 16, "bf16", "mixed", bias=False),
        # A chunk of 4 antithetic pairs, 1,024 sequences each, at width 4096: rows of one model lie together.
        _adapters("adapters, 4 pairs x 1024", 8192, 4096, 4096, 4, 8, "bf16", "pairs", bias=False),
        # The transduction tasks' sizes (64 sequences of 20 tokens), one off in every width; ragged ranks.
        _adapters("adapters, f32 odd widths", 1279, 129, 515, 23, 12, "f32", "runs", bias=True),
        # 64 perturbed character models' losses over 160 positions each.
        _distill("distill losses, V 50", "losses", 10240, 50, 8, 64, "f32", 1.0),
        # A training step over a word-piece vocabulary: the loss and its gradient.
        _distill("distill grad, V 32768", "grad", 4096, 32768, 64, 1, "bf16", 2.0),
        # Few rows, an odd vocabulary and stride, float32.
        _distill("distill grad, odd f32", "grad", 301, 30011, 20, 7, "f32", 1.5),
    ]


def _scan(name, form, seqs, tokens, heads, head_dim, groups, state, width, dtype, gate, carry, pad=0):
    return {"name": name, "op": "scan", "form": form, "seqs": seqs, "tokens": tokens, "heads": heads, "head_dim": head_dim,
            "groups": groups, "state": state, "width": width, "dtype": dtype, "gate": gate, "carry": carry, "pad": pad}


def _adapters(name, rows, k, o, adapters, rank, dtype, order, bias):
    return {"name": name, "op": "adapters", "rows": rows, "k": k, "o": o, "adapters": adapters, "rank": rank, "dtype": dtype,
            "order": order, "bias": bias}


def _distill(name, form, rows, vocab, top, models, dtype, temperature):
    return {"name": name, "op": "distill", "form": form, "rows": rows, "vocab": vocab, "top": top, "models": models, "dtype": dtype,
            "temperature": temperature}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "adapters", "distill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "scan":
        form = rng.choice(["step", "prompt", "ragged"])
        head_dim, groups = rng.choice([16, 32, 40, 64, 64, 96, 128]), rng.choice([1, 1, 2, 4])
        heads = groups * _log(rng, 1, 16)
        state, width = rng.choice([16, 32, 64, 100, 128, 128, 256]), rng.choice([2, 3, 4, 4])
        # a state of all sequences of at most 1/2 of the largest listed one
        most = max(1, (1 << 26) // (heads * head_dim * state))
        if form == "step":
            seqs = tokens = min(_log(rng, 1, 300), most)
            pad = rng.randrange(0, max(1, seqs // 8))
        else:
            seqs = min(_log(rng, 1, 256 if form == "prompt" else 64), most)
            # as many inputs as the longest listed prompt has; a ragged batch is wider than its tokens when it is padded
            room = (1 << (25 if form == "prompt" else 23)) // (heads * head_dim + 2 * groups * state) // seqs
            tokens = seqs * _log(rng, 1, max(1, min(5000, room)))
            tokens += rng.randrange(0, seqs) if form == "ragged" else 0
            pad = 0
        case = _scan("", form, seqs, tokens, heads, head_dim, groups, state, width, dtype,
                     rng.random() < 0.6, form == "step" or rng.random() < 0.7, pad)
    elif op == "adapters":
        k, o = _log(rng, 64, 4200), _log(rng, 48, 5000)
        if rng.random() < 0.6:
            k, o = -(-k // 64) * 64, -(-o // 64) * 64
        order = rng.choice(["mixed", "runs", "pairs"])
        rows = _log(rng, 1, 5000)
        case = _adapters("", rows, k, o, min(_log(rng, 1, 64), rows), rng.choice([1, 4, 8, 13, 16, 32, 64]), dtype, order,
                         rng.random() < 0.5)
    else:
        vocab = _log(rng, 10, 60000)
        rows = min(_log(rng, 1, 8192), (1 << 26) // vocab)
        case = _distill("", rng.choice(["losses", "grad"]), rows, vocab, min(rng.choice([1, 5, 8, 20, 64, 100]), vocab),
                        math.gcd(rows, rng.choice([1, 2, 4, 8, 16])), dtype, rng.choice([1.0, 1.0, 2.0, 0.7]))
    del case["name"]
    return case


# --- the inputs ----------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return {"scan": _prepare_scan, "adapters": _prepare_adapters, "distill": _prepare_distill}[case["op"]](case, g)


def _normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _uniform(g, shape, lo, hi):
    return torch.rand(shape, generator=g, device=DEV, dtype=torch.float32) * (hi - lo) + lo


def _prepare_scan(c, g):
    t, H, P, G, N, W, n = TYPES[c["dtype"]], c["heads"], c["head_dim"], c["groups"], c["state"], c["width"], c["seqs"]
    d, C, tokens = H * P, H * P + 2 * G * N, c["tokens"]
    # one input projection's output: the gate, the convolution's channels and the steps lie side by side
    wide = _normal(g, (tokens, (d if c["gate"] else 0) + C + H), t)
    at = d if c["gate"] else 0
    s = {"case": c, "z": wide[:, :d] if c["gate"] else None, "xbc": wide[:, at:at + C], "dt": wide[:, at + C:],
         "conv_weight": _uniform(g, (C, W), -0.5, 0.5).to(t), "conv_bias": _uniform(g, (C,), -0.2, 0.2).to(t),
         "decay": -_uniform(g, (H,), 1.0, 16.0), "skip": _normal(g, (H,), scale=0.3) + 1.0}
    step = torch.exp(_uniform(g, (H,), math.log(1e-3), math.log(1e-1)))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus of it is the step
    s["y"] = torch.zeros((tokens, d), device=DEV, dtype=t)
    if c["form"] == "ragged":
        cuts = torch.sort(torch.randint(0, tokens + 1, (n - 1,), generator=g, device=DEV))[0]
        ends = torch.tensor([tokens], device=DEV)
        s["offsets"] = torch.cat([torch.zeros_like(ends), cuts, ends]).to(torch.int32)
        s["longest"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    else:
        s["offsets"], s["longest"] = None, tokens // n
    s["slots"] = s["positions"] = s["conv_in"] = s["conv_out"] = s["ssm_in"] = s["ssm_out"] = None
    if c["carry"]:
        # each sequence has a slot of the cache; half of the prompts continue an earlier one
        s["slots"] = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
        back = torch.randint(1, 5000, (n,), generator=g, device=DEV, dtype=torch.int32)
        if c["form"] != "step":
            back = torch.where(torch.rand(n, generator=g, device=DEV) < 0.5, back, torch.zeros_like(back))
        s["positions"] = back
        if c["pad"]:
            s["slots"][n - c["pad"]:] = -1
        s["conv_in"], s["ssm_in"] = _normal(g, (n, W, C), t), _normal(g, (n, H, P, N), scale=0.3)
        s["conv_out"], s["ssm_out"] = torch.zeros_like(s["conv_in"]), torch.zeros_like(s["ssm_in"])
    if own:
        from zero_order_recurrent_amd import binding as b
        cfg = b.make_scan_config(H, P, G, N, W, c["dtype"])
        s["layer"] = b.ScanLayer(cfg, s["conv_weight"], s["conv_bias"], s["decay"], s["skip"], s["dt_bias"])
    return s


def _prepare_adapters(c, g):
    t, rows, K, O, A, R = TYPES[c["dtype"]], c["rows"], c["k"], c["o"], c["adapters"], c["rank"]
    s = {"case": c, "x": _normal(g, (rows, K), t), "weight": _normal(g, (O, K), t, K ** -0.5),
         "bias": _normal(g, (O,), t) if c["bias"] else None,
         "down": _normal(g, (A, R, K), t, K ** -0.5), "up": _normal(g, (A, O, R), t, R ** -0.5), "row_scale": None, "ranks": None}
    if c["order"] == "pairs":  # model 2i has probe i at +, model 2i + 1 at -
        model = torch.arange(rows, device=DEV) * (2 * A) // rows
        s["row_adapter"] = (model // 2).to(torch.int32)
        s["row_scale"] = (1.0 - 2.0 * (model % 2)) * 0.01
    elif c["order"] == "runs":  # requests of several tokens, some without an adapter, ragged ranks
        s["row_adapter"] = (torch.sort(torch.randint(0, A + 1, (rows,), generator=g, device=DEV))[0] - 1).to(torch.int32)
        s["ranks"] = torch.randint(0, R + 1, (A,), generator=g, device=DEV, dtype=torch.int32)
    elif c["order"] == "mixed":  # one token of each request, in any order
        s["row_adapter"] = (torch.randint(0, A + 1, (rows,), generator=g, device=DEV) - 1).to(torch.int32)
        s["row_scale"] = _uniform(g, (rows,), 0.5, 2.0)
    else:
        s["row_adapter"] = torch.zeros(rows, device=DEV, dtype=torch.int32)
    s["y"] = torch.empty((rows, O), device=DEV, dtype=t)
    if own:
        from zero_order_recurrent_amd import binding as b
        cfg = b.make_adapter_config(K, O, A, R, c["dtype"])
        s["layer"] = b.AdapterProjection(cfg, s["weight"], s["bias"], s["down"], s["up"], s["ranks"])
    return s


def _prepare_distill(c, g):
    t, rows, V, k = TYPES[c["dtype"]], c["rows"], c["vocab"], c["top"]
    logits = _normal(g, (rows, V), t, 2.0)
    # the teacher agrees in part with the student; its k largest, in falling order
    sure, ids = torch.topk(logits.float() * 0.5 + _normal(g, (rows, V), scale=2.0), k, dim=1)
    ids = ids.to(torch.int32)
    # one row in 16 is not scored (no teacher entry), others have fewer than k entries
    have = torch.randint(1, k + 1, (rows,), generator=g, device=DEV)
    have = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.5, have, torch.full_like(have, k))
    have = torch.where(torch.rand(rows, generator=g, device=DEV) < 1 / 16, torch.zeros_like(have), have)
    ids = torch.where(torch.arange(k, device=DEV)[None] < have[:, None], ids, torch.full_like(ids, -1))
    s = {"case": c, "logits": logits, "ids": ids, "teacher": sure.contiguous(),
         "row_losses": torch.empty(rows, device=DEV), "losses": torch.empty(c["models"], device=DEV)}
    if c["form"] == "grad":
        s["row_grad"] = torch.full((rows,), 1.0 / rows, device=DEV)
        s["dlogits"] = torch.empty_like(logits)
    if own:
        from zero_order_recurrent_amd import binding as b
        s["loss"] = b.DistillLoss(b.make_distill_config(V, k, c["models"], c["temperature"], c["dtype"]))
    return s


# --- one pass ----------------------------------------------------------------------------------


def run(s):
    c = s["case"]
    if c["op"] == "scan":
        if not own:
            y, conv, ssm = _plain_step(s) if c["form"] == "step" else _plain_prompt(s)
            return [y] if conv is None else [y, conv, ssm]
        if c["form"] == "step":
            s["layer"].step(s["xbc"], s["dt"], s["y"], s["positions"], s["conv_in"], s["ssm_in"], z=s["z"], slots=s["slots"],
                            conv_out=s["conv_out"], ssm_out=s["ssm_out"])
        else:
            s["layer"].prompt(s["xbc"], s["dt"], s["y"], c["seqs"], z=s["z"], offsets=s["offsets"], slots=s["slots"],
                              positions=s["positions"], conv_state=s["conv_in"], ssm_state=s["ssm_in"],
                              conv_out=s["conv_out"], ssm_out=s["ssm_out"])
        return [s["y"], s["conv_out"], s["ssm_out"]] if c["carry"] else [s["y"]]
    if c["op"] == "adapters":
        if not own:
            return [_plain_adapters(s)]
        s["layer"].project(s["x"], s["row_adapter"], s["y"], row_scale=s["row_scale"])
        return [s["y"]]
    if not own:
        return _plain_distill(s)
    if c["form"] == "losses":
        s["loss"].losses(s["logits"], s["ids"], s["teacher"], s["row_losses"], s["losses"])
        return [s["row_losses"], s["losses"]]
    s["loss"].grad(s["logits"], s["ids"], s["teacher"], s["row_grad"], s["row_losses"], s["losses"], s["dlogits"])
    return [s["row_losses"], s["losses"], s["dlogits"]]


# --- plain forms: the scan -------------------------------------------------------------------------


def _silu(x):
    return x * torch.sigmoid(x)


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _ring_after(s, rows, q, mine, last, fresh):
    """The convolution's ring of each sequence after its tokens: entry e holds the newest token whose place is e modulo
    the width. rows: [n, R, C] inputs at the places q [n, R]; last [n]: the number of tokens then; fresh: those of this call."""
    c, W = s["case"], s["case"]["width"]
    e = torch.arange(W, device=DEV)[None]
    newest = (last - 1)[:, None] - torch.remainder((last - 1)[:, None] - e, W)  # [n, W]
    i = newest - q[:, :1]
    take = fresh(newest)
    new = torch.gather(rows, 1, i.clamp(0, rows.shape[1] - 1).long()[:, :, None].expand(-1, -1, rows.shape[2]))
    out = torch.where(take[:, :, None], new, s["conv_in"][s["slots"].clamp(min=0).long()].float())
    return s["conv_out"].index_copy(0, s["slots"][mine].long(), out[mine].to(TYPES[c["dtype"]]))


def _plain_step(s):
    c = s["case"]
    t, H, P, G, N, W, n = TYPES[c["dtype"]], c["heads"], c["head_dim"], c["groups"], c["state"], c["width"], c["seqs"]
    d, pos, slots = H * P, s["positions"].long(), s["slots"].clamp(min=0).long()
    mine = torch.arange(n - c["pad"], device=DEV)  # rows that are not padding
    x = s["xbc"].float()
    q = pos[:, None] - (W - 1) + torch.arange(W - 1, device=DEV)[None]
    old = torch.gather(s["conv_in"][slots].float(), 1, torch.remainder(q, W)[:, :, None].expand(-1, -1, x.shape[1]))
    taps = torch.cat([torch.where(q[:, :, None] >= 0, old, torch.zeros_like(old)), x[:, None]], 1)  # [n, W, C]
    u = _silu((taps * s["conv_weight"].float().t()[None]).sum(1) + s["conv_bias"].float())
    X, B, Cc = u[:, :d].view(n, H, P), u[:, d:d + G * N].view(n, G, N), u[:, d + G * N:].view(n, G, N)
    B, Cc = B.repeat_interleave(H // G, 1), Cc.repeat_interleave(H // G, 1)
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    h = s["ssm_in"][slots] * torch.exp(dt * s["decay"])[:, :, None, None] * (pos > 0)[:, None, None, None]
    h = h + (dt[:, :, None] * X)[:, :, :, None] * B[:, :, None, :]
    y = (h * Cc[:, :, None, :]).sum(3) + s["skip"][None, :, None] * X
    y = y.reshape(n, d)
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    y = s["y"].index_copy(0, mine, y[mine].to(t))
    conv = _ring_after(s, x[:, None], pos[:, None], mine, pos + 1, lambda newest: newest >= pos[:, None])
    return y, conv, s["ssm_out"].index_copy(0, slots[mine], h[mine])


def _plain_prompt(s, Q=64):
    """The recurrence over blocks of Q tokens: inside a block by its matrix of decays, between the blocks by theirs."""
    c = s["case"]
    t, H, P, G, N, W, n = TYPES[c["dtype"]], c["heads"], c["head_dim"], c["groups"], c["state"], c["width"], c["seqs"]
    d, tokens, wide = H * P, c["tokens"], -(-max(1, s["longest"]) // Q) * Q
    if s["offsets"] is None:
        first = torch.arange(n, device=DEV) * (tokens // n)
        length = torch.full_like(first, tokens // n)
    else:
        first, length = s["offsets"][:-1].long(), (s["offsets"][1:] - s["offsets"][:-1]).long()
    pos = s["positions"].long() if c["carry"] else torch.zeros_like(first)
    place = torch.arange(wide, device=DEV)[None]
    real = place < length[:, None]
    index = torch.where(real, first[:, None] + place, torch.zeros_like(place))
    x = s["xbc"][index].float() * real[:, :, None]
    q = pos[:, None] - (W - 1) + torch.arange(W - 1, device=DEV)[None]
    if c["carry"]:
        slots = s["slots"].long()
        old = torch.gather(s["conv_in"][slots].float(), 1, torch.remainder(q, W)[:, :, None].expand(-1, -1, x.shape[2]))
        old = torch.where(q[:, :, None] >= 0, old, torch.zeros_like(old))
    else:
        old = torch.zeros((n, W - 1, x.shape[2]), device=DEV)
    full = torch.cat([old, x], 1)
    u = _silu((full.unfold(1, W, 1) * s["conv_weight"].float()).sum(-1) + s["conv_bias"].float()) * real[:, :, None]
    blocks = wide // Q
    X = u[:, :, :d].reshape(n, blocks, Q, H, P).transpose(2, 3)  # [n, blocks, H, Q, P]
    B = u[:, :, d:d + G * N].reshape(n, blocks, Q, G, N).transpose(2, 3)
    Cc = u[:, :, d + G * N:].reshape(n, blocks, Q, G, N).transpose(2, 3)
    dt = _softplus(s["dt"][index].float() + s["dt_bias"]) * real[:, :, None]
    dt = dt.reshape(n, blocks, Q, H).transpose(2, 3)  # [n, blocks, H, Q]
    a = torch.cumsum(dt.double() * s["decay"].double()[None, None, :, None], 3)
    fall = torch.exp((a[:, :, :, :, None] - a[:, :, :, None, :]).float()) * dt[:, :, :, None, :]
    tri = torch.ones((Q, Q), device=DEV, dtype=torch.bool).tril()
    cb = torch.matmul(Cc, B.transpose(3, 4).contiguous()).repeat_interleave(H // G, 2)
    y = torch.matmul(torch.where(tri, cb * fall, torch.zeros_like(cb)), X)
    # each block's own state at its end, then the state before each block
    Bh, Ch = B.repeat_interleave(H // G, 2), Cc.repeat_interleave(H // G, 2)
    left = torch.exp((a[:, :, :, -1:] - a).float()) * dt
    state = torch.matmul((X * left[..., None]).transpose(3, 4).contiguous(), Bh)  # [n, blocks, H, P, N]
    start = (s["ssm_in"][slots] * (pos > 0)[:, None, None, None] if c["carry"] else torch.zeros_like(state[:, 0]))[:, None]
    state = torch.cat([start, state], 1)  # contributions 0 .. blocks
    total = torch.cumsum(torch.cat([torch.zeros_like(a[:, :1, :, -1]), a[:, :, :, -1]], 1), 1).transpose(1, 2)  # [n, H, blocks + 1]
    far = torch.exp((total[:, :, :, None] - total[:, :, None, :]).float())
    tri = torch.ones((blocks + 1, blocks + 1), device=DEV, dtype=torch.bool).tril()
    state = torch.matmul(torch.where(tri, far, torch.zeros_like(far)), state.transpose(1, 2).reshape(n, H, blocks + 1, P * N))
    state = state.view(n, H, blocks + 1, P, N).transpose(1, 2)
    y = y + torch.matmul(Ch, state[:, :-1].transpose(3, 4).contiguous()) * torch.exp(a.float())[..., None]
    y = (y + s["skip"][None, None, :, None, None] * X).transpose(2, 3).reshape(n, wide, d)
    out = y[real]
    if s["z"] is not None:
        out = out * _silu(s["z"].float())
    out = out.to(t)
    if not c["carry"]:
        return out, None, None
    conv = _ring_after(s, x, pos[:, None] + place, torch.arange(n, device=DEV), pos + length, lambda newest: newest >= pos[:, None])
    return out, conv, s["ssm_out"].index_copy(0, slots, state[:, -1])


# --- plain forms: adapters and the loss ----------------------------------------------------------


def _plain_adapters(s):
    c = s["case"]
    x, a = s["x"].float(), s["row_adapter"].long()
    y = torch.matmul(x, s["weight"].float().t())
    if s["bias"] is not None:
        y = y + s["bias"].float()
    A, R, K = s["down"].shape
    down = s["down"].float()
    if s["ranks"] is not None:
        down = torch.where((torch.arange(R, device=DEV)[None] < s["ranks"][:, None])[:, :, None], down, torch.zeros_like(down))
    # every adapter for every row, and then only the row's own: [rows, A R] in the place of a gather of weights by row
    v = torch.matmul(x, down.view(A * R, K).t()).view(-1, A, R)
    v = torch.where((a[:, None] == torch.arange(A, device=DEV)[None])[:, :, None], v, torch.zeros_like(v))
    if s["row_scale"] is not None:
        v = v * s["row_scale"][:, None, None]
    y = y + torch.matmul(v.view(-1, A * R), s["up"].float().transpose(1, 2).reshape(A * R, -1))
    return y.to(TYPES[c["dtype"]])


def _plain_distill(s):
    c = s["case"]
    tau, z = c["temperature"], s["logits"].float() / c["temperature"]
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    here = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    w = torch.where(here, s["teacher"] / tau, torch.full_like(s["teacher"], -torch.inf))
    scored = here.any(1)
    most = torch.where(scored, w.amax(1), torch.zeros_like(w[:, 0]))[:, None]
    p = torch.exp(w - most)
    mass = p.sum(1, keepdim=True)
    p = p / torch.where(scored[:, None], mass, torch.ones_like(mass))
    logp = torch.where(here, w - most - torch.log(torch.where(scored[:, None], mass, torch.ones_like(mass))), torch.zeros_like(w))
    row = tau * tau * (p * (logp - torch.gather(z, 1, ids) + lse)).sum(1)
    each = row.view(c["models"], -1)
    losses = each.sum(1) / scored.view(c["models"], -1).sum(1)
    if c["form"] == "losses":
        return [row, losses]
    up = torch.where(scored, s["row_grad"] * tau, torch.zeros_like(row))[:, None]
    grad = (e / total * up).scatter_add(1, ids, -p * up)
    return [row, losses, grad.to(TYPES[c["dtype"]])]


# --- what a pass cannot do without -----------------------------------------------------------------


def work(case):
    c = case
    w = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "scan":
        H, P, G, N = c["heads"], c["head_dim"], c["groups"], c["state"]
        rows = c["tokens"] - c["pad"]
        seqs = c["seqs"] - c["pad"]
        C = H * P + 2 * G * N
        nbytes = rows * (C + H + H * P * (2 if c["gate"] else 1)) * w + C * (c["width"] + 1) * w + 12 * H
        if c["carry"]:
            started = 1.0 if c["form"] == "step" else 0.5
            nbytes += seqs * (1 + started) * (4 * H * P * N + C * (c["width"] - 1) * w)
        return {"bytes": nbytes, "flops": rows * (5.0 * H * P * N + 2.0 * c["width"] * C)}
    if c["op"] == "adapters":
        rows, K, O, R = c["rows"], c["k"], c["o"], c["rank"]
        used = min(c["adapters"], rows)
        return {"bytes": w * (rows * (K + O) + K * O + used * R * (K + O)) + 4 * rows, "flops": 2.0 * rows * (K * O + R * (K + O))}
    rows, V, k = c["rows"], c["vocab"], c["top"]
    return {"bytes": rows * (V * w * (2 if c["form"] == "grad" else 1) + 8 * k + 8), "flops": 4.0 * rows * V}


# --- the definitions in 64 bits --------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"scan": _exact_scan, "adapters": _exact_adapters, "distill": _exact_distill}[case["op"]](case, s)


def _exact_scan(c, s):
    """Token by token: h = exp(dt A) h + dt x B^T, y = h C + D x, on the sequences that still have a token."""
    f = torch.float64
    H, P, G, N, W, n = c["heads"], c["head_dim"], c["groups"], c["state"], c["width"], c["seqs"]
    if c["form"] == "ragged":
        first = s["offsets"][:-1].tolist()
        lengths = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
    else:
        lengths = [c["tokens"] // n] * n
        first = [i * (c["tokens"] // n) for i in range(n)]
    order = sorted(range(n), key=lambda i: -lengths[i])  # longest first: those still running are a front part
    idx = torch.tensor(order, device=DEV)
    begin = torch.tensor(first, device=DEV)[idx]
    cw, cb = s["conv_weight"].to(f), s["conv_bias"].to(f)
    hist = torch.zeros((n, W - 1, cw.shape[0]), device=DEV, dtype=f)
    h = torch.zeros((n, H, P, N), device=DEV, dtype=f)
    pos = [0] * n
    if c["carry"]:
        pos = [s["positions"].tolist()[i] for i in order]
        slot = [s["slots"].tolist()[i] for i in order]
        for j in range(n):
            if pos[j] > 0 and slot[j] >= 0:
                h[j] = s["ssm_in"][slot[j]].to(f)
                for back in range(1, W):
                    if pos[j] - back >= 0:
                        hist[j, W - 1 - back] = s["conv_in"][slot[j], (pos[j] - back) % W].to(f)
    y = torch.zeros(s["y"].shape, device=DEV, dtype=f)
    d = H * P
    for step in range(max(lengths)):
        m = sum(lengths[i] > step for i in order)
        if c["form"] == "step":
            m = n - c["pad"]
        at = begin[:m] + step
        x = s["xbc"][at].to(f)
        conv = cb + (hist[:m] * cw.t()[None, :W - 1]).sum(1) + x * cw[:, W - 1]
        hist[:m] = torch.cat([hist[:m, 1:], x[:, None]], 1)
        u = conv / (1 + torch.exp(-conv))
        dt = torch.logaddexp(s["dt"][at].to(f) + s["dt_bias"].to(f), torch.zeros((), device=DEV, dtype=f))
        X = u[:, :d].view(m, G, H // G, P)
        Bm, Cm = u[:, d:d + G * N].view(m, G, 1, N), u[:, d + G * N:].view(m, G, 1, N)
        hv = h[:m].view(m, G, H // G, P, N)
        hv.mul_(torch.exp(dt * s["decay"].to(f)).view(m, G, H // G, 1, 1))
        hv.add_((dt.view(m, G, H // G, 1) * X)[..., None] * Bm[:, :, :, None, :])
        out = torch.matmul(hv.reshape(m * G, (H // G) * P, N), Cm.reshape(m * G, N, 1)).view(m, H, P)
        out = (out + s["skip"].to(f)[None, :, None] * X.reshape(m, H, P)).reshape(m, d)
        if s["z"] is not None:
            zz = s["z"][at].to(f)
            out = out * zz / (1 + torch.exp(-zz))
        y[at] = out
    if not c["carry"]:
        return [y]
    conv_out, ssm_out = s["conv_out"].to(f), s["ssm_out"].to(f)
    for j, i in enumerate(order):
        if slot[j] < 0:
            continue
        ssm_out[slot[j]] = h[j]
        ring = s["conv_in"][slot[j]].to(f).clone()
        for k in range(max(0, lengths[i] - W), lengths[i]):
            ring[(pos[j] + k) % W] = s["xbc"][first[i] + k].to(f)
        conv_out[slot[j]] = ring
    return [y, conv_out, ssm_out]


def _exact_adapters(c, s):
    f = torch.float64
    x = s["x"].to(f)
    y = x @ s["weight"].to(f).t()
    if s["bias"] is not None:
        y += s["bias"].to(f)
    for a in range(c["adapters"]):
        rows = torch.nonzero(s["row_adapter"] == a).view(-1)
        r = c["rank"] if s["ranks"] is None else int(s["ranks"][a])
        if len(rows) and r:
            low = x[rows] @ s["down"][a, :r].to(f).t() @ s["up"][a, :, :r].to(f).t()
            if s["row_scale"] is not None:
                low = low * s["row_scale"][rows].to(f)[:, None]
            y[rows] += low
    return [y]


def _exact_distill(c, s):
    f, tau = torch.float64, c["temperature"]
    rows, V = c["rows"], c["vocab"]
    row = torch.zeros(rows, device=DEV, dtype=f)
    grad = torch.zeros((rows, V), device=DEV, dtype=f) if c["form"] == "grad" else None
    scored = (s["ids"] >= 0).any(1)
    for at in range(0, rows, 1024):
        z = s["logits"][at:at + 1024].to(f) / tau
        logq = torch.log_softmax(z, 1)
        ids = s["ids"][at:at + 1024].long()
        t = (s["teacher"][at:at + 1024].to(f) / tau).masked_fill(ids < 0, -1e300)
        p = torch.softmax(t, 1).masked_fill(ids < 0, 0.0)
        entropy = torch.special.entr(p).sum(1)
        cross = -(p * torch.gather(logq, 1, ids.clamp(min=0))).sum(1)
        row[at:at + 1024] = torch.where(scored[at:at + 1024], tau * tau * (cross - entropy), torch.zeros_like(cross))
        if grad is not None:
            target = torch.zeros_like(z).scatter_add_(1, ids.clamp(min=0), p)
            scale = (s["row_grad"][at:at + 1024].to(f) * tau * scored[at:at + 1024])[:, None]
            grad[at:at + 1024] = scale * (torch.exp(logq) - target)
    m = c["models"]
    losses = row.view(m, -1).sum(1) / scored.view(m, -1).sum(1)
    return [row, losses] if grad is None else [row, losses, grad]
