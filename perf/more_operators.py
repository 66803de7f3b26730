"""Timing cases of the operators of one decode step that stays on the GPU: the draw from a row's top-k / top-p / min-p set
with the caller's random numbers, the verification of speculative drafts against the target's logits, and the block tables
and slot maps of a paged cache.

``run`` computes each in plain torch operations, or, with ``own`` set, by the calls that a user of the framework makes.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
MOST = 256 * 151936  # elements of the largest batch


def listed():
    return [
        # The draw, with its log-probability. "mixed": every row has its own request's settings, some greedy.
        # one interactive request
        dict(name="draw-1", op="draw", rows=1, vocab=32768, dtype="f32", pitch=0, filters="mixed", heat=1.0),
        # a small batch
        dict(name="draw-8", op="draw", rows=8, vocab=151936, dtype="f32", pitch=0, filters="mixed", heat=1.0),
        # a serving batch
        dict(name="draw-256", op="draw", rows=256, vocab=151936, dtype="bf16", pitch=0, filters="mixed", heat=1.0),
        # reinforcement-learning rollouts: the whole distribution at temperature one
        dict(name="draw-rollout", op="draw", rows=256, vocab=151936, dtype="bf16", pitch=0, filters="none", heat=1.0),
        # creative writing at high temperatures: nuclei of tens of thousands of tokens
        dict(name="draw-hot", op="draw", rows=64, vocab=151936, dtype="bf16", pitch=0, filters="nucleus", heat=3.0),
        # an odd vocabulary inside a padded buffer
        dict(name="draw-odd", op="draw", rows=96, vocab=100003, dtype="f16", pitch=5, filters="mixed", heat=1.0),
        # Verification of drafts.
        # one interactive request, drafts looked up in its prompt (no draft probabilities)
        dict(name="verify-1", op="verify", requests=1, drafts=3, vocab=32768, dtype="f32", pitch=0, filters="mixed", probs=False),
        # a serving batch with a draft model
        dict(name="verify-64", op="verify", requests=64, drafts=4, vocab=151936, dtype="bf16", pitch=0, filters="mixed", probs=True),
        # an odd vocabulary, long looked-up drafts of any length
        dict(name="verify-odd", op="verify", requests=24, drafts=9, vocab=100003, dtype="f16", pitch=5, filters="mixed", probs=False),
        # Pages: slots are extended, their slot map and the batch's block table are built, and the step is taken back.
        # a decode step of a large batch with long contexts: one token each
        dict(name="pages-decode", op="pages", requests=256, slots=320, page=16, context=32768, grow=1, batch_table=True),
        # the verification step of that batch: up to eight tokens each
        dict(name="pages-verify", op="pages", requests=256, slots=256, page=16, context=32768, grow=8, batch_table=True),
        # prompts admitted to be scored, and released
        dict(name="pages-admit", op="pages", requests=64, slots=96, page=64, context=0, grow=8192, batch_table=False),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["draw", "draw", "verify", "pages"])
    if op == "pages":
        requests = _spread(rng, 1, 512)
        grow = rng.choice([1, rng.randrange(2, 10), _spread(rng, 10, 8192)])
        grow = max(1, min(grow, 64 * 8192 // requests))
        context = 0 if grow > 9 and rng.random() < 0.5 else _spread(rng, 1, 32768)
        context = min(context, 256 * 32768 // requests)
        return dict(op=op, requests=requests, slots=requests + rng.randrange(0, 65), page=rng.choice([1, 8, 16, 16, 32, 48, 64, 128, 256]),
                    context=context, grow=grow, batch_table=rng.random() < 0.6)
    vocab = _spread(rng, 257, 262144)
    dtype = rng.choice(["f32", "bf16", "f16"])
    most = MOST * 2 // SIZES[dtype]
    case = dict(op=op, vocab=vocab, dtype=dtype, pitch=rng.choice([0, 0, -vocab % 64, rng.randrange(1, 9)]))
    if op == "draw":
        case.update(rows=max(1, min(_spread(rng, 1, 256), most // vocab)), filters=rng.choice(["mixed", "mixed", "nucleus", "none"]),
                    heat=rng.choice([1.0, 1.0, 2.0]))
        return case
    drafts = rng.randrange(1, 10)
    probs = rng.random() < 0.5
    limit = (most // 4 if probs else most) // (vocab * (drafts + 1))
    case.update(requests=max(1, min(_spread(rng, 1, 64), limit)), drafts=drafts, filters=rng.choice(["mixed", "mixed", "none"]), probs=probs)
    return case


# ----------------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator("cuda").manual_seed(int(seed) * 6367 + 5)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _head(g, rows, vocab):
    """Logits as a language model gives them: a wide bulk, a few dozen likely tokens that fall off with their rank, and some
    tokens that were masked upstream. Binary32."""
    x = torch.randn(rows, vocab, generator=g, device="cuda") * 2.5
    likely = min(64, max(1, vocab // 8))
    ids = (_uniform(g, rows, likely) * vocab).long()
    rank = torch.arange(1, likely + 1, device="cuda").float().log()
    top = 20 - rank * (0.5 + 2.5 * _uniform(g, rows, 1)) + 0.5 * torch.randn(rows, likely, generator=g, device="cuda")
    x.scatter_reduce_(1, ids, top, "amax")
    return x.masked_fill_(_uniform(g, rows, vocab) < 0.002, -math.inf)


def _padded(x, case):
    buffer = torch.zeros(x.shape[0], x.shape[1] + case["pitch"], dtype=TYPES[case["dtype"]], device="cuda")
    return buffer[:, :x.shape[1]].copy_(x)


def _settings(g, n, filters, heat):
    """temperature, top_k, top_p and min_p of n requests (None: no such filter in the batch)."""
    t = (0.5 + 0.7 * _uniform(g, n)) * heat
    if filters == "none":
        return torch.ones(n, device="cuda") * heat, None, None, None
    p = 0.8 + 0.19 * _uniform(g, n)
    if filters == "nucleus":
        return t, None, p, None
    t = torch.where(_uniform(g, n) < 0.1, torch.zeros_like(t), t)
    k = torch.where(_uniform(g, n) < 0.5, (_uniform(g, n) * 100 + 1).int(), 0).int()
    p = torch.where(_uniform(g, n) < 0.3, torch.ones_like(p), p)
    m = torch.where(_uniform(g, n) < 0.5, 0.02 + 0.1 * _uniform(g, n), torch.zeros_like(p))
    return t, k, p, m


def _lengths(g, n, most):
    """n list lengths spread evenly over 1 to `most`, that one among them, in any order; the same ones from any seed."""
    return (most - torch.arange(n, device="cuda") * most // n)[torch.argsort(_uniform(g, n))]


def _offsets(lengths):
    o = torch.zeros(lengths.numel() + 1, dtype=torch.int64, device="cuda")
    o[1:] = lengths.cumsum(0)
    return o


def prepare(case, seed):
    g = _generator(seed)
    s = {"op": case["op"]}
    if case["op"] == "pages":
        return _prepare_pages(case, g, s)
    if case["op"] == "draw":
        s["logits"] = _padded(_head(g, case["rows"], case["vocab"]), case)
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = _settings(g, case["rows"], case["filters"], case["heat"])
        s["uniform"] = _uniform(g, case["rows"])
        return s
    n, most = case["requests"], case["drafts"]
    lengths = _lengths(g, n, most + 1)
    if case["probs"]:
        lengths.fill_(most + 1)  # a draft model proposes as many tokens for every request
    s["offsets"] = _offsets(lengths)
    rows = int(s["offsets"][-1])
    x = _head(g, rows, case["vocab"])
    s["logits"] = _padded(x, case)
    s["temperature"], s["top_k"], s["top_p"], s["min_p"] = _settings(g, n, case["filters"], 1.0)
    s["uniform"], s["uniform_draw"] = _uniform(g, rows), _uniform(g, n)
    x = x.add_(torch.randn(x.shape, generator=g, device="cuda") * 0.5)  # the draft model's logits
    if case["probs"]:
        s["probs"] = torch.softmax(x, 1)
        s["draft"] = (torch.cumsum(s["probs"], 1) <= _uniform(g, rows, 1)).sum(1).clamp_(max=case["vocab"] - 1)
    else:
        s["probs"] = None
        s["draft"] = x.argmax(1)
    return s


def _prepare_pages(case, g, s):
    n, slots, page = case["requests"], case["slots"], case["page"]
    most = -(-(case["context"] + case["grow"]) // page)
    used = _lengths(g, slots, case["context"]).int()
    held = (used + page - 1) // page
    first = _offsets(held)
    pages = int(first[-1]) + n * (-(-case["grow"] // page) + 1)
    ids = torch.randperm(pages, generator=g, device="cuda").int()
    column = torch.arange(most, device="cuda")
    at = (first[:-1, None] + column).clamp_(max=pages - 1)
    table = torch.where(column < held[:, None], ids[at], -1)
    left = pages - int(first[-1])
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:left] = ids[int(first[-1]):]
    s.update(table=table.contiguous(), length=used, free=free, free_count=torch.tensor([left], dtype=torch.int32, device="cuda"), page=page)
    s["slots"] = torch.argsort(_uniform(g, slots))[:n].int()
    grow = _lengths(g, n, case["grow"])
    s["offsets"] = _offsets(grow) if case["grow"] > 1 else None
    s["total"] = int(grow.sum())
    # a scheduler on the host, as the plain form needs one, counts the pages that it hands out
    old = used[s["slots"].long()].long()
    s["total_pages"] = int(((old + grow + page - 1) // page - (old + page - 1) // page).sum())
    s["columns"] = most if case["batch_table"] else 0
    return s


# ----------------------------------------------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------------------------------------------
def _kept(x, t, k, p, m):
    """The weights exp((x - max) / t) of every row's top-k / top-p / min-p set, zero outside, in 64 bits; one-hot where t is
    not above zero. t, k, p and m have one entry a row."""
    x = x.double()
    top, first = x.max(1, keepdim=True)
    z = (x - top) / t[:, None].double()
    e = torch.exp(z)
    if k is not None or p is not None:
        order = torch.sort(x, dim=1, descending=True, stable=True)[1]
        ranked = e.gather(1, order)
        keep = torch.ones_like(ranked, dtype=torch.bool)
        if k is not None:
            keep &= (torch.arange(x.shape[1], device="cuda") < k[:, None]) | (k < 1)[:, None]
        if p is not None:
            before = ranked.cumsum(1) - ranked
            keep &= (before < p[:, None].double() * ranked.sum(1, keepdim=True)) | (p >= 1)[:, None]
        keep[:, 0] = True
        e = e * torch.empty_like(keep).scatter_(1, order, keep)
    if m is not None:
        e = torch.where((z >= m[:, None].double().log()) | (m <= 0)[:, None], e, 0)
    greedy = torch.zeros_like(e).scatter_(1, (x == top).int().argmax(1, keepdim=True), 1)
    return torch.where((t > 0)[:, None], e, greedy)


def _pick(w, u):
    """The smallest index whose running sum of weights passes u times their sum."""
    c = w.cumsum(1)
    return (c <= u[:, None].double() * c[:, -1:]).sum(1)


def _drawn(s):
    w = _kept(s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    i = _pick(w, s["uniform"])
    return i, torch.log(w.gather(1, i[:, None])[:, 0] / w.sum(1)).float()


def _rows(v, request):
    return None if v is None else v[request]


def _verified(s):
    offsets, draft = s["offsets"], s["draft"]
    n, rows = offsets.numel() - 1, draft.numel()
    row = torch.arange(rows, device="cuda")
    request = torch.searchsorted(offsets, row, right=True) - 1
    w = _kept(s["logits"], *(_rows(s[name], request) for name in ("temperature", "top_k", "top_p", "min_p")))
    w = w / w.sum(1, keepdim=True)
    q = s["probs"]
    at = draft[:, None]
    chance = q.gather(1, at)[:, 0].double() if q is not None else 1.0
    last = row == offsets[request + 1] - 1
    accepted = (s["uniform"].double() * chance < w.gather(1, at)[:, 0]) & ~last
    stop = torch.full((n,), rows, device="cuda").scatter_reduce(0, request, torch.where(accepted, rows, row), "amin")
    left = w[stop]
    if q is None:
        rest = left.scatter(1, at[stop], 0)
    else:
        rest = (left - q[stop].double()).clamp_(min=0)
    use = ~last[stop] & (rest.sum(1) > 0)
    token = _pick(torch.where(use[:, None], rest, left), s["uniform_draw"])
    out = torch.where(row < stop[request], draft, torch.where(row == stop[request], token[request], -1))
    return out, (stop - offsets[:-1] + 1).int()


def _extended_and_trimmed(s):
    """Extension in order while pages last, then the step taken back: the pages go back where they were taken from."""
    page, table, length, free = s["page"], s["table"], s["length"], s["free"]
    slots = s["slots"].long()
    n, most = slots.numel(), table.shape[1]
    offsets = torch.arange(n + 1, device="cuda") if s["offsets"] is None else s["offsets"]
    count = offsets.diff()
    old = length[slots].long()
    held = (old + page - 1) // page
    need = (old + count + page - 1) // page - held
    fits = (old + count <= most * page) & (torch.bincount(slots, minlength=table.shape[0])[slots] == 1)
    need = torch.where(fits, need, 0)
    end = need.cumsum(0)
    fits &= (need == 0) | (end <= s["free_count"])
    need = torch.where(fits, need, 0)
    first = need.cumsum(0) - need
    # the j-th new page of request i is entry first[i] + j from the top
    r = torch.repeat_interleave(torch.arange(n, device="cuda"), need, output_size=s["total_pages"])
    j = torch.arange(r.numel(), device="cuda") - first[r]
    entry = (s["free_count"].long() - 1 - first[r] - j).long()
    ids = free[entry]
    table[slots[r], held[r] + j] = ids
    start = torch.where(fits, old, -1).int()
    r2 = torch.repeat_interleave(torch.arange(n, device="cuda"), count, output_size=s["total"])
    position = old[r2] + torch.arange(s["total"], device="cuda") - offsets[r2]
    slot_map = torch.where(fits[r2], table[slots[r2], (position // page).clamp(max=most - 1)].long() * page + position % page, -1)
    out = {"start": start, "slot_map": slot_map}
    out["lengths"] = torch.where(fits, old + count, 0).int()
    if s["columns"]:
        column = torch.arange(s["columns"], device="cuda")
        now = torch.where(fits, held + need, 0)
        out["batch_table"] = torch.where(column < now[:, None], table[slots][:, :s["columns"]], -1)
    # taken back
    length[slots] = old.int()
    free[entry] = ids
    table[slots[r], held[r] + j] = -1
    out.update(table=table, length=length, free=free, free_count=s["free_count"])
    return out


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "draw":
        return _drawn(s)
    if s["op"] == "verify":
        return _verified(s)
    return _extended_and_trimmed(s)


def _run_own(s):
    import token_sampling_logits_gb300 as gs

    if s["op"] == "draw":
        return gs.filtered_categorical(s["logits"], s["temperature"], s["uniform"], top_k=s["top_k"], top_p=s["top_p"],
                                       min_p=s["min_p"], logprob=True)
    if s["op"] == "verify":
        if "workspace" not in s:
            s["workspace"] = gs.new_verify_workspace(s["logits"].shape[0], s["logits"].device)
        return gs.verify_drafts(s["logits"], s["draft"], s["offsets"], s["temperature"], s["uniform"], s["uniform_draw"],
                                probs=s["probs"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], workspace=s["workspace"])
    if "state" not in s:  # kept by a server for the life of its cache
        s["state"] = gs.PageState(s["table"], s["length"], s["free"], s["free_count"], page_size=s["page"])
    state, n = s["state"], s["slots"].numel()
    out = {"lengths": torch.empty(n, dtype=torch.int32, device="cuda")}
    if s["columns"]:
        out["batch_table"] = torch.empty(n, s["columns"], dtype=torch.int32, device="cuda")
    out["start"], out["slot_map"] = gs.pages_extend(state, s["total"], slots=s["slots"], offsets=s["offsets"],
                                                    lengths=out["lengths"], table=out.get("batch_table"))
    gs.pages_trim(state, slots=s["slots"], start=out["start"])
    out.update(table=state.table, length=state.length, free=state.free, free_count=state.free_count)
    return {name: out[name] for name in ("start", "slot_map", "lengths", "batch_table", "table", "length", "free", "free_count")
            if name in out}


# ----------------------------------------------------------------------------------------------------------------------
# work and exact values
# ----------------------------------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "draw":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * SIZES[case["dtype"]] + case["rows"] * 32, "flops": 4 * n}
    if case["op"] == "verify":
        n = case["requests"]
        rows = n * (case["drafts"] + 1 if case["probs"] or n == 1 else case["drafts"] / 2 + 1)
        # the target's rows; the draft's probabilities of the row that a draft was refused in, for two requests in three
        read = rows * case["vocab"] * SIZES[case["dtype"]] + (2 / 3 * n * case["vocab"] * 4 if case["probs"] else 0)
        return {"bytes": read + rows * 32, "flops": 4 * rows * case["vocab"]}
    n = case["requests"]
    total = n * (case["grow"] + 1) / 2
    new = n * case["grow"] / 2 / case["page"]
    columns = -(-(case["context"] + case["grow"]) // case["page"]) if case["batch_table"] else 0
    # lists, lengths, the slot map; new pages taken and given back; the batch's table: half of it read, all of it written
    return {"bytes": n * 32 + total * 8 + new * 24 + n * columns * 6, "flops": total + 4 * n}


def exact(case, seed):
    """Row by row on the host, from the definitions; pages by a plain scheduler's loop."""
    s = prepare(case, seed)
    if case["op"] == "pages":
        return _exact_pages(s)
    import numpy as np

    def host(v):
        return None if v is None else v.double().cpu().numpy() if v.dtype.is_floating_point else v.cpu().numpy()

    t, k, p, m = (host(s[name]) for name in ("temperature", "top_k", "top_p", "min_p"))

    def weights(r, request):
        x = host(s["logits"][r])
        w = np.zeros(len(x))
        if not t[request] > 0:
            w[np.argmax(x)] = 1
            return w
        ids = np.argsort(-x, kind="stable")
        ids = ids[x[ids] > -np.inf]
        e = np.exp((x[ids] - x[ids[0]]) / t[request])
        many = len(ids)
        if k is not None and k[request] >= 1:
            many = min(many, k[request])
        if p is not None and p[request] < 1:
            many = min(many, 1 + int(np.searchsorted(np.cumsum(e), p[request] * np.sum(e), "left")))
        if m is not None and m[request] > 0:
            many = min(many, int(np.count_nonzero((x[ids] - x[ids[0]]) / t[request] >= np.log(m[request]))))
        w[ids[:many]] = e[:many]
        return w

    def pick(w, u):
        return int(np.searchsorted(np.cumsum(w), u * np.cumsum(w)[-1], "right"))

    u = host(s["uniform"])
    if case["op"] == "draw":
        index, logprob = [], []
        for r in range(case["rows"]):
            w = weights(r, r)
            index.append(pick(w, u[r]))
            logprob.append(math.log(w[index[-1]]) - math.log(w.sum()))
        return torch.tensor(index), torch.tensor(logprob, dtype=torch.float64)
    offsets, draft, v = host(s["offsets"]), host(s["draft"]), host(s["uniform_draw"])
    out, counts = np.full(len(draft), -1), []
    for i in range(len(offsets) - 1):
        for r in range(offsets[i], offsets[i + 1]):
            w = weights(r, i)
            w /= w.sum()
            if r == offsets[i + 1] - 1:
                out[r] = pick(w, v[i])
                break
            q = np.zeros(len(w)) if s["probs"] is None else host(s["probs"][r])
            if s["probs"] is None:
                q[draft[r]] = 1
            if u[r] * q[draft[r]] < w[draft[r]]:
                out[r] = draft[r]
                continue
            rest = np.maximum(w - q, 0)
            out[r] = pick(rest if rest.sum() > 0 else w, v[i])
            break
        counts.append(r + 1 - offsets[i])
    return torch.from_numpy(out), torch.tensor(counts, dtype=torch.int32)


def _exact_pages(s):
    table, length, free = (s[name].tolist() for name in ("table", "length", "free"))
    page, slots, top = s["page"], s["slots"].tolist(), int(s["free_count"])
    offsets = range(len(slots) + 1) if s["offsets"] is None else s["offsets"].tolist()
    start, slot_map, lengths, rows = [], [], [], []
    for i, slot in enumerate(slots):
        start.append(length[slot])
        held = [b for b in table[slot] if b >= 0]
        for position in range(length[slot], length[slot] + offsets[i + 1] - offsets[i]):
            if position // page == len(held):
                top -= 1
                held.append(free[top])
            slot_map.append(held[position // page] * page + position % page)
        lengths.append(length[slot] + offsets[i + 1] - offsets[i])
        rows.append(held + [-1] * (s["columns"] - len(held)))
    out = {"start": torch.tensor(start, dtype=torch.int32), "slot_map": torch.tensor(slot_map),
           "lengths": torch.tensor(lengths, dtype=torch.int32)}
    if s["columns"]:
        out["batch_table"] = torch.tensor(rows, dtype=torch.int32)
    # the step was taken back: the state is as it was
    out.update(table=s["table"], length=s["length"], free=s["free"], free_count=s["free_count"])
    return out
