"""Timing cases of the operators between a model's logits and the draw: penalties for repeated tokens, additive biases,
grammar masks, the per-request state that they read, and the draw from the constrained logits.

Each case is one step of an LLM server's sampling loop. ``run`` computes it in plain torch operations, or, with ``own``
set, by the calls that a user of the framework makes.
"""
import math

import torch

own = False

PROMPT_BIT = -(1 << 31)  # bit 31 of a history word: the token is in the prompt
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
MOST = 256 * 151936  # elements of the largest batch


def listed():
    return [
        # Admission of requests: their state rows are cleared and refilled with the prompt, any output generated so far
        # (a resumed request) and the request's bias list.
        # a short chat turn admitted alone
        dict(name="admit-1", op="admit", rows=1, slots=8, vocab=32768, prompt=700, output=0, biases=0),
        # one long document
        dict(name="admit-long", op="admit", rows=1, slots=4, vocab=151936, prompt=131072, output=2048, biases=16),
        # a full batch after a restart, ragged prompts and outputs, long bias lists
        dict(name="admit-batch", op="admit", rows=64, slots=96, vocab=151936, prompt=8192, output=1024, biases=300),
        # The processed logits themselves, for a caller that goes on with another sampler.
        # one interactive request
        dict(name="process-1", op="process", rows=1, vocab=32768, dtype="f32", out="f32", pitch=0, history=512, biases=16,
             mask="mixed", inplace=False),
        # a serving batch, everything in use, binary32 results from bf16 logits
        dict(name="process-256", op="process", rows=256, vocab=151936, dtype="bf16", out="f32", pitch=0, history=4096,
             biases=32, mask="mixed", inplace=False),
        # an odd vocabulary inside a padded buffer, results in the logits' type
        dict(name="process-odd", op="process", rows=96, vocab=100003, dtype="f16", out="f16", pitch=5, history=2048,
             biases=8, mask="mixed", inplace=False),
        # a structured-output batch whose grammar mask is applied to the model's buffer
        dict(name="mask-inplace", op="process", rows=256, vocab=151936, dtype="bf16", out="bf16", pitch=0, history=0,
             biases=0, mask="sparse", inplace=True),
        # The draw from the constrained logits, one decode step.
        # one interactive request
        dict(name="draw-1", op="draw", rows=1, vocab=32768, dtype="f32", pitch=0, history=512, biases=16, mask="mixed",
             greedy=0.0),
        # a small batch, penalties and biases only
        dict(name="draw-8", op="draw", rows=8, vocab=151936, dtype="f32", pitch=0, history=4096, biases=32, mask="none",
             greedy=0.25),
        # a serving batch, everything in use
        dict(name="draw-256", op="draw", rows=256, vocab=151936, dtype="bf16", pitch=0, history=4096, biases=32,
             mask="mixed", greedy=0.1),
        # a structured-output batch: the grammar leaves a few tokens in every row
        dict(name="draw-grammar", op="draw", rows=256, vocab=151936, dtype="bf16", pitch=0, history=1024, biases=0,
             mask="sparse", greedy=0.25),
        # an odd vocabulary inside a padded buffer
        dict(name="draw-odd", op="draw", rows=96, vocab=100003, dtype="f16", pitch=5, history=2048, biases=8, mask="mixed",
             greedy=0.25),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["admit", "process", "process", "draw", "draw"])
    vocab = _spread(rng, 257, 262144)
    if op == "admit":
        rows = _spread(rng, 1, 64)
        if rows * vocab > 64 * 151936:
            rows = 64 * 151936 // vocab
        prompt = _spread(rng, 1, 131072)
        prompt = max(1, min(prompt, 64 * 8192 // rows))
        return dict(op=op, rows=rows, slots=rows + rng.randrange(0, 33), vocab=vocab, prompt=prompt,
                    output=rng.choice([0, _spread(rng, 1, 1024)]), biases=rng.choice([0, min(vocab // 4, _spread(rng, 1, 300))]))
    dtype = rng.choice(["f32", "bf16", "f16"])
    out = rng.choice([dtype, "f32"])
    most = MOST * 5 // (SIZES[dtype] + SIZES[out]) if op == "process" else MOST * 2 // SIZES[dtype]
    rows = max(1, min(_spread(rng, 1, 256), min(most, MOST) // vocab))
    case = dict(op=op, rows=rows, vocab=vocab, dtype=dtype, pitch=rng.choice([0, 0, -vocab % 64, rng.randrange(1, 9)]),
                history=rng.choice([0, _spread(rng, 1, 4096)]), biases=rng.choice([0, min(vocab // 4, _spread(rng, 1, 300))]),
                mask=rng.choice(["none", "mixed", "sparse"]))
    if op == "process":
        case.update(out=out, inplace=False)
    else:
        case.update(greedy=rng.choice([0.0, 0.25]))
    return case


# ----------------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator("cuda").manual_seed(int(seed) * 7919 + 11)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _tokens(g, n, vocab):
    """Token ids spread evenly over the logarithm of the id, as frequent tokens have low ids."""
    return (torch.exp(torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * math.log(vocab)).long() - 1).clamp_(0, vocab - 1)


def _ragged(g, rows, longest, vocab):
    """Lists of up to `longest` tokens, the first of them that long: the tokens of all rows and the rows' offsets."""
    lengths = (_uniform(g, rows) * (longest + 1)).long().clamp_(max=longest)
    lengths[0] = longest
    offsets = torch.zeros(rows + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = lengths.cumsum(0)
    return _tokens(g, int(offsets[-1]), vocab), offsets


def _biases(g, rows, count, vocab):
    """`count` different token ids a row and their biases; one in ten bans its token."""
    start = (_uniform(g, rows, 1) * vocab).long()
    step = 1 + (_uniform(g, rows, 1) * (vocab // max(count, 1) - 1)).long()
    ids = (start + step * torch.arange(count, device="cuda")) % vocab
    values = (_uniform(g, rows, count) * 2 - 1) * 8
    values = torch.where(_uniform(g, rows, count) < 0.1, torch.full_like(values, -100.0), values)
    return ids.reshape(-1), values.reshape(-1), torch.arange(rows + 1, device="cuda") * count


def _row_of(offsets, n):
    return torch.searchsorted(offsets, torch.arange(n, device="cuda"), right=True) - 1


def _pack(bits):
    """Truth values [n, 32 * w] as int32 words [n, w], the lowest bit first."""
    b = bits.reshape(bits.shape[0], -1, 32).long()
    return (b << torch.arange(32, device="cuda")).sum(2).to(torch.int32)


def _filled(state, rows, prompt, prompt_offsets, output, output_offsets, bias_ids, bias_values, bias_offsets):
    """The plain form of an admission: state rows `rows` hold exactly these lists afterwards."""
    history, bias, touched = state
    n, ld = rows.numel(), history.shape[1]
    seen = torch.zeros(n, ld, dtype=torch.bool, device="cuda")
    count = torch.zeros(n, ld, dtype=torch.int32, device="cuda")
    mark = torch.zeros(n, ld, dtype=torch.bool, device="cuda")
    value = torch.zeros(n, ld, device="cuda")
    true = torch.ones((), dtype=torch.bool, device="cuda")
    at = _row_of(prompt_offsets, prompt.numel())
    seen.index_put_((at, prompt), true)
    at = _row_of(output_offsets, output.numel())
    count.index_put_((at, output), torch.ones((), dtype=torch.int32, device="cuda"), accumulate=True)
    at = _row_of(bias_offsets, bias_ids.numel())
    value.index_put_((at, bias_ids), bias_values)
    mark.index_put_((at, bias_ids), true)
    rows = rows.long()
    history[rows] = torch.where(seen, count + PROMPT_BIT, count)
    bias[rows] = value
    touched[rows] = _pack(seen | (count > 0) | mark)


def _new_state(slots, vocab):
    ld = (vocab + 31) // 32 * 32
    return (torch.zeros(slots, ld, dtype=torch.int32, device="cuda"), torch.zeros(slots, ld, device="cuda"),
            torch.zeros(slots, ld // 32, dtype=torch.int32, device="cuda"))


def _mask(g, rows, vocab, kind):
    """Grammar masks, one bit a token (set: allowed), and the mask row of each batch row (-1: no grammar). Rows inside a
    string allow nearly everything; rows at a structural place allow from none to a few hundred tokens."""
    words = (vocab + 31) // 32
    most = max(2, min(300, vocab // 8))
    free = _uniform(g, rows, words * 32) < 0.97
    few = torch.zeros(rows, words * 32, dtype=torch.bool, device="cuda")
    size = (torch.exp(_uniform(g, rows) * math.log(most + 1)) - 0.5).long()
    ids = (_uniform(g, rows, most) * vocab).long()
    few.scatter_(1, ids, torch.arange(most, device="cuda")[None, :] < size[:, None])
    place = torch.arange(rows, device="cuda") % 4
    bits = torch.where((place == 3)[:, None], few, free) if kind == "mixed" else few
    which = torch.arange(rows, device="cuda", dtype=torch.int32)
    if kind == "mixed":
        which = torch.where(place == 2, -1, which).to(torch.int32)
    return _pack(bits), which


def prepare(case, seed):
    g = _generator(seed)
    rows, vocab = case["rows"], case["vocab"]
    s = {"op": case["op"], "vocab": vocab}
    if case["op"] == "admit":
        slots = case["slots"]
        s["rows"] = torch.argsort(_uniform(g, slots))[:rows].to(torch.int32)
        s["state"] = _new_state(slots, vocab)
        # what earlier requests left in the rows
        old = _ragged(g, slots, max(1, case["prompt"] // 2), vocab) + _ragged(g, slots, 64, vocab) + _biases(g, slots, 0, vocab)
        _filled(s["state"], torch.arange(slots, device="cuda"), *old)
        s["lists"] = _ragged(g, rows, case["prompt"], vocab) + _ragged(g, rows, case["output"], vocab) + _biases(g, rows, case["biases"], vocab)
        return s
    x = torch.randn(rows, vocab, generator=g, device="cuda") * 4
    x = x + 6 * (_uniform(g, rows, vocab) < 32 / vocab)
    x = torch.where(_uniform(g, rows, vocab) < 0.002, torch.full_like(x, -math.inf), x)
    buffer = torch.zeros(rows, vocab + case["pitch"], dtype=TYPES[case["dtype"]], device="cuda")
    s["logits"] = buffer[:, :vocab]
    s["logits"].copy_(x)
    s["state"] = s["slots"] = s["repetition"] = s["frequency"] = s["presence"] = None
    if case["history"] or case["biases"]:
        slots = rows + 3
        s["state"] = _new_state(slots, vocab)
        s["slots"] = torch.argsort(_uniform(g, slots))[:rows].to(torch.int32)
        lists = _ragged(g, rows, case["history"], vocab) + _ragged(g, rows, case["history"] // 4, vocab) + _biases(g, rows, case["biases"], vocab)
        _filled(s["state"], s["slots"], *lists)
        s["repetition"] = 1 + 0.5 * _uniform(g, rows)
        s["frequency"] = _uniform(g, rows) - 0.2
        s["presence"] = _uniform(g, rows) - 0.2
    s["mask"], s["mask_rows"] = _mask(g, rows, vocab, case["mask"]) if case["mask"] != "none" else (None, None)
    if case["op"] == "process":
        s["inplace"], s["out"] = case["inplace"], TYPES[case["out"]]
        return s
    t = 0.3 + 1.2 * _uniform(g, rows)
    s["temperature"] = torch.where(_uniform(g, rows) < case["greedy"], torch.zeros_like(t), t)
    s["seed"] = torch.randint(-(1 << 62), 1 << 62, (rows,), generator=g, device="cuda")
    s["offset"] = torch.randint(0, 1 << 40, (rows,), generator=g, device="cuda")
    return s


# ----------------------------------------------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------------------------------------------
def _processed(s):
    """The constrained logits in binary32."""
    x = s["logits"].float()
    vocab = s["vocab"]
    if s["state"] is not None:
        history, bias, _ = s["state"]
        slots = s["slots"].long()
        h = history[slots, :vocab]
        y = x + bias[slots, :vocab]
        rep = s["repetition"][:, None]
        y = torch.where(h != 0, torch.where(y > 0, y / rep, y * rep), y)
        c = h & 0x7FFFFFFF
        y = torch.where(c > 0, y - s["frequency"][:, None] * c - s["presence"][:, None], y)
        x = torch.where(x == -math.inf, x, y)
    if s["mask"] is not None:
        which = s["mask_rows"].long()
        words = s["mask"][which.clamp(min=0)]
        allowed = ((words[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).reshape(len(which), -1)[:, :vocab]
        x = torch.where((allowed == 1) | (which < 0)[:, None], x, torch.full_like(x, -math.inf))
    return x


def _high_low(multiplier, x):
    """The high and low halves of the 64-bit product of two 32-bit words held in int64."""
    p = x * multiplier
    return (p >> 32) & 0xFFFFFFFF, p & 0xFFFFFFFF


def _philox_words(rows, vocab, seed, offset):
    """Philox4x32-10 (Salmon et al., SC'11): word i & 3 of block i >> 2 for every element i, counter (i >> 2, row, offset)."""
    groups = (vocab + 3) // 4
    low = lambda v: v & 0xFFFFFFFF  # noqa: E731
    c0 = torch.arange(groups, device="cuda")[None, :].expand(rows, groups)
    c1 = torch.arange(rows, device="cuda")[:, None]
    c2, c3 = low(offset)[:, None], low(offset >> 32)[:, None]
    k0, k1 = low(seed)[:, None], low(seed >> 32)[:, None]
    for _ in range(10):
        h0, l0 = _high_low(0xD2511F53, c0)
        h1, l1 = _high_low(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = low(k0 + 0x9E3779B9), low(k1 + 0xBB67AE85)
    shape = (rows, groups)
    words = torch.stack([c.expand(shape) for c in (c0, c1, c2, c3)], dim=2)
    return words.reshape(rows, -1)[:, :vocab]


def _drawn(s):
    """argmax of x / T + g, or of x where T is not above 0; the lowest index on ties, -1 where nothing is left."""
    x, t = _processed(s), s["temperature"][:, None]
    u = ((_philox_words(*x.shape, s["seed"], s["offset"]) >> 9).float() + 0.5) * 2.0 ** -23
    noisy = x / t - torch.log(-torch.log(u))
    score = torch.where(t > 0, noisy, x)
    score = torch.where(torch.isnan(score), torch.full_like(score, -math.inf), score)
    best = score.amax(1, keepdim=True)
    index = torch.arange(x.shape[1], device="cuda")
    first = torch.where(score == best, index, x.shape[1]).amin(1)
    return torch.where(best[:, 0] == -math.inf, -1, first)


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "admit":
        _filled(s["state"], s["rows"], *s["lists"])
        return dict(zip(("history", "bias", "touched"), s["state"]))
    if s["op"] == "draw":
        return _drawn(s)
    y = _processed(s).to(s["out"])
    return s["logits"].copy_(y) if s["inplace"] else y


def _run_own(s):
    import token_sampling_logits_gb300 as gs

    if "handle" not in s:  # kept by a server for the life of its slots
        s["handle"] = gs.LogitState(*s["state"], vocab=s["vocab"]) if s["state"] is not None else None
        if s["op"] == "draw":
            s["workspace"] = gs.new_workspace(s["logits"].shape[0], s["logits"].device)
    state = s["handle"]
    if s["op"] == "admit":
        prompt, prompt_offsets, output, output_offsets, ids, values, bias_offsets = s["lists"]
        gs.state_reset(state, slots=s["rows"])
        gs.history_append(state, prompt, slots=s["rows"], offsets=prompt_offsets, prompt=True)
        if output.numel():
            gs.history_append(state, output, slots=s["rows"], offsets=output_offsets)
        if ids.numel():
            gs.bias_set(state, ids, values, slots=s["rows"], offsets=bias_offsets)
        return {"history": state.history, "bias": state.bias, "touched": state.touched}
    constraints = dict(state=state, slots=s["slots"], repetition=s["repetition"], frequency=s["frequency"],
                       presence=s["presence"], mask=s["mask"], mask_rows=s["mask_rows"])
    if s["op"] == "draw":
        return gs.constrained_gumbel_argmax(s["logits"], s["temperature"], s["seed"], s["offset"],
                                            workspace=s["workspace"], **constraints)
    if s["inplace"]:
        return gs.process_logits(s["logits"], out=s["logits"], **constraints)
    return gs.process_logits(s["logits"], out_dtype=s["out"], **constraints)


# ----------------------------------------------------------------------------------------------------------------------
# work and exact values
# ----------------------------------------------------------------------------------------------------------------------
def _different(tokens, vocab):
    """About how many different ids `tokens` draws of _tokens hold."""
    scale = tokens / math.log(vocab)
    return min(vocab, tokens, scale * (1 + math.log(max(1.0, vocab / max(1.0, scale)))))


def work(case):
    rows, vocab = case["rows"], case["vocab"]
    if case["op"] == "admit":
        # half of the longest list on average; tokens in, the words and bits that change out, the bits of the rows
        lists = case["prompt"] * (1 if rows == 1 else 0.5), case["output"] * (1 if rows == 1 else 0.5)
        words = sum(_different(n, vocab) for n in lists) + case["biases"]
        return {"bytes": rows * (8 * sum(lists) + 12 * case["biases"] + 4 * words + vocab / 8), "flops": rows * sum(lists)}
    left = {"none": 1.0, "mixed": 0.75, "sparse": 0.0}[case["mask"]]  # the share of elements that masks leave
    few = {"none": 0, "mixed": 0.25, "sparse": 1.0}[case["mask"]] * 53  # tokens at a structural place
    elements = rows * (left * vocab + few)
    touched = _different(0.625 * case["history"], vocab) + case["biases"] if case["history"] or case["biases"] else 0
    size = SIZES[case["dtype"]]
    bits = rows * vocab / 8 * ((case["mask"] != "none") * (0.75 if case["mask"] == "mixed" else 1) + (touched > 0))
    read = elements * size + bits + rows * touched * max(left, 0.001) * 8
    if case["op"] == "draw":
        return {"bytes": read + rows * 28, "flops": 4 * elements}
    if case["inplace"]:
        return {"bytes": bits + (rows * vocab - elements) * size, "flops": rows * vocab}
    return {"bytes": read + rows * vocab * SIZES[case["out"]], "flops": rows * vocab}


def exact(case, seed):
    """The processed logits in 64 bits, row by row from the definition; the state's words counted on the host."""
    if case["op"] == "draw":
        return None
    s = prepare(case, seed)
    if case["op"] == "admit":
        history, bias, touched = (t.cpu().clone() for t in s["state"])
        prompt, p_at, output, o_at, ids, values, b_at = (t.cpu() for t in s["lists"])
        for i, r in enumerate(s["rows"].tolist()):
            p, o = prompt[p_at[i]:p_at[i + 1]], output[o_at[i]:o_at[i + 1]]
            e = slice(int(b_at[i]), int(b_at[i + 1]))
            history[r] = torch.bincount(o, minlength=history.shape[1]).int()
            history[r, p.unique()] += PROMPT_BIT
            bias[r] = 0
            bias[r, ids[e]] = values[e]
            bits = history[r] != 0
            bits[ids[e]] = True
            weights = torch.ones(32, dtype=torch.int64).cumsum(0).sub(1)
            touched[r] = torch.bitwise_left_shift(bits.view(-1, 32).long(), weights).sum(1).to(torch.int32)
        return {"history": history, "bias": bias.double(), "touched": touched}
    out = s["logits"].double()
    for b in range(case["rows"]):
        x = out[b]
        if s["state"] is not None:
            r = int(s["slots"][b])
            h, bias = s["state"][0][r, :case["vocab"]].long(), s["state"][1][r, :case["vocab"]].double()
            y = x.clone()
            some = bias.nonzero()[:, 0]
            y[some] += bias[some]
            some = h.nonzero()[:, 0]
            rep = float(s["repetition"][b])
            y[some] = y[some] * torch.where(y[some] > 0, 1 / rep, rep)
            count = h % (1 << 31)
            some = count.nonzero()[:, 0]
            y[some] -= float(s["frequency"][b]) * count[some].double() + float(s["presence"][b])
            x.copy_(torch.where(x > -math.inf, y, x))
        m = -1 if s["mask"] is None else int(s["mask_rows"][b])
        if m >= 0:
            words = s["mask"][m].long() & 0xFFFFFFFF
            place = torch.arange(case["vocab"], device="cuda")
            x[(words[place // 32] // (1 << (place % 32))) % 2 == 0] = -math.inf
    return out
