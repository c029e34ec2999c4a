"""Three further operators of a population of language models, as a program calls them.

They stand beside the low-rank adapters, the selective scan and the distillation loss, and belong together in the same
way: a model that is evaluated by forward passes alone is
  * projected by weights that are stored in four bits (mx: microscaled 4-bit floating point, blocks of 32 along the
    reduction with a power of two each; quantisation, and the product with rows that are quantised on the way in),
  * run over its tokens by a recurrence whose state forgets by the gated delta rule (delta: whole prompts, or one token
    for each of many sequences), and
  * scored (scores: log probabilities of given tokens, the entropy, the top alternatives, which are what the
    distillation loss takes from a teacher; or the gradient of log probability and entropy).

With `own` False `run` computes them from elementary torch operations in 32 bits (running sums of log-decays in 64); with
`own` True it calls the library.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"
NORM_EPS = 1e-6


# --- the cases ---------------------------------------------------------------------------------


def listed():
    return [
        # One sequence is being generated: one token through one layer of 8 heads of 128 x 128 (width 1024).
        _delta("delta step, one row", "step", 1, 1, 8, 4, 128, 128, "bf16", carry=True),
        # A serving batch, width 4096, two value heads to a key head; seven of its 256 rows are padding.
        _delta("delta step, 256 rows", "step", 256, 256, 32, 16, 128, 128, "bf16", carry=True, pad=7),
        # One long prompt, width 4096: few rows, a long chain of states.
        _delta("delta prompt, 1 x 8192", "prompt", 1, 8192, 32, 16, 128, 128, "bf16", carry=True),
        # A ragged batch of prompts and continued prompts in float32, two key heads, odd widths.
        _delta("delta prompt, ragged f32", "ragged", 33, 9001, 14, 2, 100, 40, "f32", carry=True),
        # 64 perturbed character models' positions, 160 each, with five alternatives.
        _scores("scores, V 50", "scores", 10240, 50, 5, "f32", 1.0),
        # A decode step of 48 requests over a word-piece vocabulary: latency.
        _scores("scores, 48 requests", "scores", 48, 32768, 20, "bf16", 0.7),
        # A teacher's positions, scored, with the 64 alternatives that a distillation loss takes.
        _scores("scores, V 32768", "scores", 4096, 32768, 64, "bf16", 1.0),
        # The gradient of log probability and entropy; few rows, an odd vocabulary and stride, float32.
        _scores("scores grad, odd f32", "grad", 301, 30011, 0, "f32", 1.5),
        # One token's projection, 1024 -> 4096, from weights in four bits: latency.
        _mx("mx project, one row", "project", 1, 1024, 4096, "bf16", bias=True),
        # A decode step of 48 requests at the 1.1B model's width.
        _mx("mx project, 48 requests", "project", 48, 5888, 5888, "bf16", bias=False),
        # A chunk of 4 antithetic pairs, 1,024 sequences each, at width 4096.
        _mx("mx project, 4 pairs x 1024", "project", 8192, 4096, 4096, "bf16", bias=False),
        # A weight matrix is stored in four bits and read back; odd sizes, float32.
        _mx("mx quantize, odd f32", "quantize", 5887, 4099, 1, "f32", bias=False),
    ]


def _delta(name, form, seqs, tokens, heads, groups, key_dim, value_dim, dtype, carry, pad=0):
    return {"name": name, "op": "delta", "form": form, "seqs": seqs, "tokens": tokens, "heads": heads, "groups": groups,
            "key_dim": key_dim, "value_dim": value_dim, "dtype": dtype, "carry": carry, "pad": pad}


def _scores(name, form, rows, vocab, top, dtype, temperature):
    return {"name": name, "op": "scores", "form": form, "rows": rows, "vocab": vocab, "top": top, "dtype": dtype,
            "temperature": temperature}


def _mx(name, form, rows, k, o, dtype, bias):
    return {"name": name, "op": "mx", "form": form, "rows": rows, "k": k, "o": o, "dtype": dtype, "bias": bias}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "scores", "mx"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "delta":
        form = rng.choice(["step", "prompt", "ragged"])
        groups = rng.choice([1, 2, 4, 8])
        heads = groups * rng.choice([1, 1, 2, 3, 4])
        key_dim, value_dim = rng.choice([16, 32, 64, 100, 128, 128, 192, 256]), rng.choice([16, 32, 40, 64, 128, 128, 256])
        # a state of all sequences of at most 1/2 of the largest listed one
        most = max(1, (1 << 26) // (heads * key_dim * value_dim))
        if form == "step":
            seqs = tokens = min(_log(rng, 1, 300), most)
            pad = rng.randrange(0, max(1, seqs // 8))
        else:
            seqs = min(_log(rng, 1, 256 if form == "prompt" else 64), most)
            # fewer inputs than the longest listed prompt has; a ragged batch is wider than its tokens when it is padded
            room = (1 << (25 if form == "prompt" else 23)) // (heads * (key_dim + value_dim)) // seqs
            tokens = seqs * _log(rng, 1, max(1, min(5000, room)))
            tokens += rng.randrange(0, seqs) if form == "ragged" else 0
            pad = 0
        case = _delta("", form, seqs, tokens, heads, groups, key_dim, value_dim, dtype, form == "step" or rng.random() < 0.7, pad)
    elif op == "scores":
        vocab = _log(rng, 10, 60000)
        rows = min(_log(rng, 1, 8192), (1 << 26) // vocab)
        form = rng.choice(["scores", "scores", "grad"])
        top = 0 if form == "grad" else min(rng.choice([0, 1, 5, 8, 20, 64, 100, 300]), vocab // 4)
        case = _scores("", form, rows, vocab, top, dtype, rng.choice([1.0, 1.0, 2.0, 0.7]))
    else:
        k, o, rows = _log(rng, 64, 4200), _log(rng, 48, 5000), _log(rng, 1, 5000)
        if rng.random() < 0.6:
            k, o = -(-k // 64) * 64, -(-o // 64) * 64
        form = rng.choice(["project", "project", "quantize"])
        case = _mx("", form, rows, k, 1 if form == "quantize" else o, dtype, form == "project" and rng.random() < 0.5)
    del case["name"]
    return case


# --- the inputs ----------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return {"delta": _prepare_delta, "scores": _prepare_scores, "mx": _prepare_mx}[case["op"]](case, g)


def _normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _uniform(g, shape, lo, hi):
    return torch.rand(shape, generator=g, device=DEV, dtype=torch.float32) * (hi - lo) + lo


def _prepare_delta(c, g):
    t, H, G, K, V, n = TYPES[c["dtype"]], c["heads"], c["groups"], c["key_dim"], c["value_dim"], c["seqs"]
    tokens = c["tokens"]
    # one input projection's output: queries, keys, values, and the raw steps and strengths lie side by side
    wide = _normal(g, (tokens, 2 * G * K + H * V + 2 * H), t)
    at = [0, G * K, 2 * G * K, 2 * G * K + H * V, 2 * G * K + H * V + H, 2 * G * K + H * V + 2 * H]
    q, k, v, dt, beta = (wide[:, a:b] for a, b in zip(at, at[1:]))
    s = {"case": c, "q": q, "k": k, "v": v, "dt": dt, "beta": beta, "decay": -_uniform(g, (H,), 1.0, 16.0)}
    step = torch.exp(_uniform(g, (H,), math.log(1e-3), math.log(1e-1)))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus of it is the step
    s["y"] = torch.zeros((tokens, H * V), device=DEV, dtype=t)
    if c["form"] == "ragged":
        cuts = torch.sort(torch.randint(0, tokens + 1, (n - 1,), generator=g, device=DEV))[0]
        ends = torch.tensor([tokens], device=DEV)
        s["offsets"] = torch.cat([torch.zeros_like(ends), cuts, ends]).to(torch.int32)
        s["longest"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    else:
        s["offsets"], s["longest"] = None, tokens // n
    s["slots"] = s["positions"] = s["state_in"] = s["state_out"] = None
    if c["carry"]:
        # each sequence has a slot of the cache; half of the prompts continue an earlier one
        s["slots"] = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
        back = torch.randint(1, 5000, (n,), generator=g, device=DEV, dtype=torch.int32)
        if c["form"] != "step":
            back = torch.where(torch.rand(n, generator=g, device=DEV) < 0.5, back, torch.zeros_like(back))
        s["positions"] = back
        if c["pad"]:
            s["slots"][n - c["pad"]:] = -1
        s["state_in"] = _normal(g, (n, H, V, K), scale=0.3)
        s["state_out"] = torch.zeros_like(s["state_in"])
    if own:
        from zero_order_recurrent_amd import binding as b
        s["layer"] = b.DeltaLayer(b.make_delta_config(H, G, K, V, c["dtype"], norm_eps=NORM_EPS), s["decay"], s["dt_bias"])
    return s


def _prepare_scores(c, g):
    t, rows, V = TYPES[c["dtype"]], c["rows"], c["vocab"]
    wide = V + (5 if V % 2 else 0)  # an odd vocabulary's rows lie apart
    logits = _normal(g, (rows, wide), t, 2.5)[:, :V]
    # a few tokens are likely ones, as a trained model has them; one row in eight may not say half of the vocabulary
    logits.scatter_add_(1, torch.randint(0, V, (rows, 3), generator=g, device=DEV), _uniform(g, (rows, 3), 0.0, 12.0).to(t))
    barred = (torch.rand(rows, generator=g, device=DEV) < 0.125)[:, None] & (torch.arange(V, device=DEV) % 2 == 1)[None]
    logits.masked_fill_(barred, -math.inf)
    tokens = torch.randint(0, (V + 1) // 2, (rows,), generator=g, device=DEV) * 2
    # half of the given tokens are the model's own choice, one in sixteen is padding
    likely = logits.float().argmax(1)
    tokens = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.5, likely, tokens)
    tokens = torch.where(torch.rand(rows, generator=g, device=DEV) < 1 / 16, torch.full_like(tokens, -1), tokens).to(torch.int32)
    s = {"case": c, "logits": logits, "tokens": tokens}
    if c["form"] == "grad":
        s["up_logprob"] = _normal(g, (rows,), scale=1.0 / rows)
        s["up_entropy"] = _normal(g, (rows,), scale=0.1 / rows)
        s["dlogits"] = torch.empty((rows, wide), device=DEV, dtype=t)[:, :V]
    else:
        s["logprobs"], s["entropy"] = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        s["top_ids"] = torch.empty((rows, c["top"]), device=DEV, dtype=torch.int32) if c["top"] else None
        s["top_logprobs"] = torch.empty((rows, c["top"]), device=DEV) if c["top"] else None
    if own:
        from zero_order_recurrent_amd import binding as b
        s["scores"] = b.TokenScores(b.make_score_config(V, c["top"], c["temperature"], c["dtype"]))
    return s


def _prepare_mx(c, g):
    t, rows, K, O = TYPES[c["dtype"]], c["rows"], c["k"], c["o"]
    if c["form"] == "quantize":
        s = {"case": c, "x": _normal(g, (rows, K), t, K ** -0.5), "values": torch.empty((rows, K), device=DEV, dtype=t)}
        if own:
            from zero_order_recurrent_amd import binding as b
            s["format"] = b.MxFormat(b.make_mx_config(K, O, c["dtype"]))
            s["codes"], s["scales"] = s["format"].empty(rows)
        return s
    # activations of uneven columns, as they come out of a normalisation with its weights
    x = _normal(g, (rows, K)) * torch.exp(_normal(g, (K,)) * 0.5)
    weight = _normal(g, (O, K), torch.float32, K ** -0.5)
    s = {"case": c, "x": x.to(t), "bias": _normal(g, (O,), t) if c["bias"] else None,
         "y": torch.empty((rows, O), device=DEV, dtype=t)}
    # the weights were stored in four bits before: a code of 4 bits for each value, a scale for each 32
    s["w_codes"], s["w_scales"] = _mx_codes(weight)
    if own:
        from zero_order_recurrent_amd import binding as b
        s["layer"] = b.MxProjection(b.make_mx_config(K, O, c["dtype"]), s["w_codes"], s["w_scales"], s["bias"])
    return s


# --- one pass ----------------------------------------------------------------------------------


def run(s):
    c = s["case"]
    if c["op"] == "delta":
        if not own:
            y, state = _plain_delta_step(s) if c["form"] == "step" else _plain_delta_prompt(s)
            return [y] if state is None else [y, state]
        if c["form"] == "step":
            s["layer"].step(s["q"], s["k"], s["v"], s["dt"], s["beta"], s["y"], s["positions"], s["state_in"], slots=s["slots"],
                            state_out=s["state_out"])
        else:
            s["layer"].prompt(s["q"], s["k"], s["v"], s["dt"], s["beta"], s["y"], c["seqs"], offsets=s["offsets"], slots=s["slots"],
                              positions=s["positions"], state=s["state_in"], state_out=s["state_out"])
        return [s["y"], s["state_out"]] if c["carry"] else [s["y"]]
    if c["op"] == "scores":
        if not own:
            return _plain_scores(s)
        if c["form"] == "grad":
            s["scores"].grad(s["logits"], s["tokens"], s["up_logprob"], s["up_entropy"], s["dlogits"])
            return [s["dlogits"]]
        s["scores"].scores(s["logits"], s["tokens"], s["logprobs"], s["entropy"], s["top_ids"], s["top_logprobs"])
        return [s["logprobs"], s["entropy"]] + ([s["top_ids"], s["top_logprobs"]] if c["top"] else [])
    if c["form"] == "quantize":
        if not own:
            return [_mx_values(*_mx_codes(s["x"].float()), c["k"]).to(TYPES[c["dtype"]])]
        s["format"].quantize(s["x"], s["codes"], s["scales"])
        s["format"].dequantize(s["codes"], s["scales"], s["values"])
        return [s["values"]]
    if not own:
        return [_plain_project(s)]
    s["layer"].project(s["x"], s["y"])
    return [s["y"]]


# --- plain forms: the delta rule -------------------------------------------------------------------


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _units(x, heads, width, repeat):
    """Rows of heads at length one, in 32 bits, shared by `repeat` value heads each."""
    x = x.float().reshape(*x.shape[:-1], heads, width)
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) + NORM_EPS)
    return x.repeat_interleave(repeat, -2)


def _plain_delta_step(s):
    c = s["case"]
    t, H, G, K, V, n = TYPES[c["dtype"]], c["heads"], c["groups"], c["key_dim"], c["value_dim"], c["seqs"]
    pos, slots = s["positions"].long(), s["slots"].clamp(min=0).long()
    mine = torch.arange(n - c["pad"], device=DEV)  # rows that are not padding
    q, k = _units(s["q"], G, K, H // G) * K ** -0.5, _units(s["k"], G, K, H // G)
    v = s["v"].float().reshape(n, H, V)
    fade = torch.exp(_softplus(s["dt"].float() + s["dt_bias"]) * s["decay"])
    b = torch.sigmoid(s["beta"].float())
    S = s["state_in"][slots] * (fade * (pos > 0)[:, None])[:, :, None, None]
    S = S + ((v - (S * k[:, :, None, :]).sum(3)) * b[:, :, None])[:, :, :, None] * k[:, :, None, :]
    y = (S * q[:, :, None, :]).sum(3).reshape(n, H * V)
    return s["y"].index_copy(0, mine, y[mine].to(t)), s["state_out"].index_copy(0, slots[mine], S[mine])


def _plain_delta_prompt(s, Q=64):
    """Blocks of Q tokens: what a block's tokens correct of each other is a triangular system, solved for all blocks at
    once; then the state goes from block to block."""
    c = s["case"]
    t, H, G, K, V, n = TYPES[c["dtype"]], c["heads"], c["groups"], c["key_dim"], c["value_dim"], c["seqs"]
    tokens, wide = c["tokens"], -(-max(1, s["longest"]) // Q) * Q
    if s["offsets"] is None:
        first = torch.arange(n, device=DEV) * (tokens // n)
        length = torch.full_like(first, tokens // n)
    else:
        first, length = s["offsets"][:-1].long(), (s["offsets"][1:] - s["offsets"][:-1]).long()
    place = torch.arange(wide, device=DEV)[None]
    real = place < length[:, None]
    index = torch.where(real, first[:, None] + place, torch.zeros_like(place))
    blocks = wide // Q

    def cut(x):  # [n, wide, H, w] -> [n, blocks, H, Q, w]
        return (x * real[:, :, None, None]).reshape(n, blocks, Q, H, -1).transpose(2, 3).contiguous()

    q, k = cut(_units(s["q"][index], G, K, H // G) * K ** -0.5), cut(_units(s["k"][index], G, K, H // G))
    v = cut(s["v"][index].float().reshape(n, wide, H, V))
    g = cut((_softplus(s["dt"][index].float() + s["dt_bias"]) * s["decay"])[..., None])[..., 0]
    b = cut(torch.sigmoid(s["beta"][index].float())[..., None])
    a = torch.cumsum(g.double(), 3)
    fall = torch.exp((a[..., :, None] - a[..., None, :]).clamp(max=0).float())
    low = torch.ones((Q, Q), device=DEV, dtype=torch.bool).tril()
    kt = k.transpose(3, 4).contiguous()
    L = torch.where(low.tril(-1), torch.matmul(k, kt) * fall * b, torch.zeros_like(fall))
    T = torch.eye(Q, device=DEV).expand_as(L).contiguous()  # (1 + L)^-1, row by row
    for i in range(1, Q):
        T[..., i, :i] = -torch.matmul(L[..., i:i + 1, :i], T[..., :i, :i].contiguous())[..., 0, :]
    grown = torch.exp(a.float())[..., None]
    U, Wk = torch.matmul(T, b * v), torch.matmul(T, b * grown * k)
    P = torch.where(low, torch.matmul(q, kt) * fall, torch.zeros_like(fall))
    qg, left = q * grown, (k * torch.exp((a[..., -1:] - a).float())[..., None]).transpose(3, 4).contiguous()
    total = torch.exp(a[..., -1].float())[..., None, None]
    S = torch.zeros((n, H, K, V), device=DEV)  # the state on its side
    if c["carry"]:
        slots = s["slots"].long()
        S = (s["state_in"][slots] * (s["positions"] > 0)[:, None, None, None]).transpose(2, 3).contiguous()
    y = torch.empty((n, blocks, Q, H, V), device=DEV)
    for i in range(blocks):
        new = U[:, i] - torch.matmul(Wk[:, i], S)
        y[:, i] = (torch.matmul(qg[:, i], S) + torch.matmul(P[:, i], new)).transpose(1, 2)
        S = S * total[:, i] + torch.matmul(left[:, i], new)
    out = y.reshape(n, wide, H * V)[real].to(t)
    if not c["carry"]:
        return out, None
    return out, s["state_out"].index_copy(0, slots, S.transpose(2, 3))


# --- plain forms: scores and four bits --------------------------------------------------------------


def _plain_scores(s):
    c = s["case"]
    tau, x = c["temperature"], s["logits"].float()
    z = (x - x.amax(1, keepdim=True)) / tau
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    logp = z - torch.log(total)
    given = s["tokens"] >= 0
    at = s["tokens"].clamp(min=0).long()[:, None]
    # what a token of no probability adds to the entropy is its limit, zero
    p = e / total
    plogp = torch.where(e > 0, p * logp, torch.zeros_like(p))
    entropy = -plogp.sum(1)
    if c["form"] == "grad":
        up = torch.where(given, s["up_logprob"], torch.zeros_like(s["up_logprob"]))[:, None]
        grad = -up * p - s["up_entropy"][:, None] * (plogp + p * entropy[:, None])
        return [(grad.scatter_add(1, at, up) / tau).to(TYPES[c["dtype"]])]
    out = [torch.where(given, torch.gather(logp, 1, at)[:, 0], torch.zeros_like(entropy)), entropy]
    if c["top"]:
        # largest first, equal ones by their place: a whole number of both
        bits = (x + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
        key = order * (1 << 26) - torch.arange(c["vocab"], device=DEV)[None]
        ids = -(torch.topk(key, c["top"], dim=1)[0] % -(1 << 26))
        out += [ids.to(torch.int32), torch.gather(logp, 1, ids)]
    return out


def _mx_codes(x):
    """[rows, K] float32 -> codes [rows, 16 * blocks], two to a byte, the first in its low half, and scales [rows, blocks].
    A scale is a power of two, 2^(byte - 127), that brings the block's largest magnitude into [4, 8)."""
    rows, K = x.shape
    blocks = -(-K // 32)
    if K % 32:
        x = torch.cat([x, x.new_zeros((rows, blocks * 32 - K))], 1)
    x = x.reshape(rows, blocks, 32)
    most = x.abs().amax(2)
    power = (torch.frexp(most)[1] - 3).clamp(-127, 127)
    power = torch.where(most > 0, power, torch.full_like(power, -127))
    # two factors, either of them a normal number
    half = power // 2
    m = (x * torch.exp2(-half.float())[:, :, None] * torch.exp2((half - power).float())[:, :, None]).abs()
    # steps of 1/2 below 2, of 1 below 4, of 2 up to 6; torch.round takes ties to the even code
    m = torch.where(m < 2, torch.round(m * 2), torch.where(m < 4, torch.round(m) + 2, torch.round(m / 2) + 4)).clamp(max=7)
    code = (m.to(torch.uint8) | ((x < 0).to(torch.uint8) << 3)).reshape(rows, blocks * 16, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), (power + 127).to(torch.uint8)


def _mx_values(codes, scales, K):
    rows, blocks = scales.shape
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    code = torch.stack([codes & 15, codes >> 4], 2).reshape(rows, blocks, 32)
    power = scales.int() - 127
    half = power // 2
    v = table[code.int()] * torch.exp2(half.float())[:, :, None] * torch.exp2((power - half).float())[:, :, None]
    return v.reshape(rows, blocks * 32)[:, :K]


def _plain_project(s):
    c = s["case"]
    x = _mx_values(*_mx_codes(s["x"].float()), c["k"])
    y = torch.matmul(x, _mx_values(s["w_codes"], s["w_scales"], c["k"]).t().contiguous())
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(TYPES[c["dtype"]])


# --- what a pass cannot do without -----------------------------------------------------------------


def work(case):
    c = case
    w = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "delta":
        H, G, K, V = c["heads"], c["groups"], c["key_dim"], c["value_dim"]
        rows, seqs = c["tokens"] - c["pad"], c["seqs"] - c["pad"]
        nbytes = rows * (2 * G * K + 2 * H * V + 2 * H) * w + 8 * H
        if c["carry"]:
            nbytes += seqs * (2.0 if c["form"] == "step" else 1.5) * 4 * H * K * V
        return {"bytes": nbytes, "flops": 7.0 * rows * H * K * V}
    if c["op"] == "scores":
        rows, V = c["rows"], c["vocab"]
        if c["form"] == "grad":
            return {"bytes": rows * (2 * V * w + 12), "flops": 6.0 * rows * V}
        return {"bytes": rows * (V * w + 12 + 8 * c["top"]), "flops": 4.0 * rows * V}
    rows, K, O = c["rows"], c["k"], c["o"]
    if c["form"] == "quantize":  # values, codes and scales are written and the latter read again
        return {"bytes": rows * (2 * K * w + 2 * 17 * -(-K // 32)), "flops": 4.0 * rows * K}
    return {"bytes": rows * (K + O) * w + O * 17 * -(-K // 32), "flops": 2.0 * rows * K * O}


# --- the definitions in 64 bits --------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "scores": _exact_scores, "mx": _exact_mx}[case["op"]](case, s)


def _exact_delta(c, s):
    """Token by token: S = a S, then S += b (v - S k) k^T, y = S q, on the sequences that still have a token."""
    f = torch.float64
    H, G, K, V, n = c["heads"], c["groups"], c["key_dim"], c["value_dim"], c["seqs"]
    if c["form"] == "ragged":
        first = s["offsets"][:-1].tolist()
        lengths = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
    else:
        lengths = [c["tokens"] // n] * n
        first = [i * (c["tokens"] // n) for i in range(n)]
    if max(lengths) * n * H * K * V > 1.2e13:
        return None
    order = sorted(range(n), key=lambda i: -lengths[i])  # longest first: those still running are a front part
    begin = torch.tensor(first, device=DEV)[torch.tensor(order, device=DEV)]
    S = torch.zeros((n, H, V, K), device=DEV, dtype=f)
    if c["carry"]:
        pos = [s["positions"].tolist()[i] for i in order]
        slot = [s["slots"].tolist()[i] for i in order]
        for j in range(n):
            if pos[j] > 0 and slot[j] >= 0:
                S[j] = s["state_in"][slot[j]].to(f)
    zero = torch.zeros((), device=DEV, dtype=f)
    fade = torch.exp(torch.logaddexp(s["dt"].to(f) + s["dt_bias"].to(f), zero) * s["decay"].to(f))
    strength = 1 / (1 + torch.exp(-s["beta"].to(f)))

    def unit(x):
        x = x.to(f).reshape(-1, G, 1, K)
        return (x * torch.rsqrt(torch.square(x).sum(-1, keepdim=True) + NORM_EPS)).expand(-1, G, H // G, K).reshape(-1, H, K, 1)

    q, k, v = unit(s["q"]) / math.sqrt(K), unit(s["k"]), s["v"].to(f).reshape(-1, H, V, 1)
    y = torch.zeros(s["y"].shape, device=DEV, dtype=f)
    for step in range(max(lengths)):
        m = n - c["pad"] if c["form"] == "step" else sum(lengths[i] > step for i in order)
        at = begin[:m] + step
        now = S[:m]
        now.mul_(fade[at][:, :, None, None])
        now.add_((v[at] - torch.matmul(now, k[at])) * strength[at][:, :, None, None] * k[at].transpose(2, 3))
        y[at] = torch.matmul(now, q[at]).reshape(m, H * V)
    if not c["carry"]:
        return [y]
    out = s["state_out"].to(f)
    for j in range(n):
        if slot[j] >= 0:
            out[slot[j]] = S[j]
    return [y, out]


def _exact_scores(c, s):
    f, tau = torch.float64, c["temperature"]
    rows = c["rows"]
    parts = []
    for at in range(0, rows, 512):
        raw = s["logits"][at:at + 512].to(f)
        logq = torch.log_softmax(raw / tau, 1)
        prob = torch.exp(logq)
        entropy = torch.special.entr(prob).sum(1)
        token = s["tokens"][at:at + 512].long()
        here = (token >= 0).to(f)
        pick = token.clamp(min=0)[:, None]
        if c["form"] == "grad":
            one = torch.zeros_like(prob).scatter_(1, pick, 1.0)
            d_log = (one - prob) * here[:, None] * s["up_logprob"][at:at + 512].to(f)[:, None]
            d_ent = (torch.special.entr(prob) - prob * entropy[:, None]) * s["up_entropy"][at:at + 512].to(f)[:, None]
            parts.append([(d_log + d_ent) / tau])
            continue
        lp = torch.gather(logq, 1, pick)[:, 0]
        part = [torch.where(here > 0, lp, torch.zeros_like(lp)), entropy]
        if c["top"]:
            ids = torch.sort(raw, dim=1, descending=True, stable=True)[1][:, :c["top"]]
            part += [ids.to(torch.int32), torch.gather(logq, 1, ids)]
        parts.append(part)
    return [torch.cat(p) for p in zip(*parts)]


def _exact_values(x):
    """The values that a matrix's four-bit form stands for: the nearest of the format's, ties to the even code."""
    f = torch.float64
    rows, K = x.shape
    pad = -K % 32
    x = torch.nn.functional.pad(x.to(f), (0, pad)).reshape(rows, -1, 32)
    top = x.abs().amax(2, keepdim=True)
    scale = torch.exp2((torch.floor(torch.log2(top.clamp(min=2.0 ** -160))) - 2).clamp(min=-127))
    # a logarithm may be off by a rounding next to a power of two
    scale = torch.where(top >= scale * 8, scale * 2, torch.where((top < scale * 4) & (scale > 2.0 ** -127), scale / 2, scale))
    r = x.abs() / scale
    out = torch.zeros_like(r)
    # a border belongs to the code below it where that one is even
    for border, below, value in [(0.25, True, 0.5), (0.75, False, 1), (1.25, True, 1.5), (1.75, False, 2), (2.5, True, 3),
                                 (3.5, False, 4), (5.0, True, 6)]:
        out = torch.where((r > border) if below else (r >= border), torch.full_like(r, value), out)
    return (out * scale * torch.sign(x)).reshape(rows, K + pad)[:, :K]


def _exact_mx(c, s):
    f = torch.float64
    if c["form"] == "quantize":
        return [_exact_values(s["x"])]
    codes, scales = s["w_codes"], s["w_scales"].to(f)
    blocks = scales.shape[1]
    nibble = torch.stack([codes & 15, codes >> 4], 2).reshape(c["o"], blocks, 32)
    small, exponent, mantissa = (nibble & 6) == 0, ((nibble >> 1) & 3).to(f), (nibble & 1).to(f)
    size = torch.where(small, mantissa / 2, torch.exp2(exponent - 1) * (1 + mantissa / 2))
    w = torch.where(nibble >= 8, -size, size) * torch.exp2(scales - 127)[:, :, None]
    y = _exact_values(s["x"]) @ w.reshape(c["o"], -1)[:, :c["k"]].t()
    return [y if s["bias"] is None else y + s["bias"].to(f)]
