"""The serving operators around the paged KV cache, as cases to be measured.

  tables     tables_ragged_paged: the row offsets, the page table's new entries and
             the slot map of one step, from the sequences' lengths and a stack of
             free pages
  attention  attention_ragged_paged: attention of each sequence's new tokens (one
             token, a few, or a chunk of a prompt) over its pages, bf16 or e4m3

listed() names the cases, draw() gives others of the same ranges, prepare() makes
what a serving program holds before the call, run() is one call (the plain form in
elementary torch operations, or the library's kernels where `own` is true), exact()
the same answer in 64 bits, and work() the bytes and operations of one call.

A case's lengths follow from its own numbers (so that work() knows them); page ids
and values follow from the seed.
"""
import math
import random

import torch

own = False

# the projections' workload: hidden rows of 4096 = 32 heads of 128, 8 key/value
# heads, pages of 128 slots, eight prompts of 1 to 1024 tokens
BASE = {"hq": 32, "hkv": 8, "d": 128, "page": 128, "layers": 1, "cache": "bf16", "gran": 0, "causal": True,
        "window": 0}


def _attention(name, batch, new, history, **over):
    """new, history: "n" = that many for every sequence, "a-b" = uniform in a .. b."""
    return {"name": name, "op": "attention", "batch": batch, "new": str(new), "history": str(history), "lens": 5,
            **BASE, **over}


def _tables(name, batch, new, history, page, slack=64):
    return {"name": name, "op": "tables", "batch": batch, "new": str(new), "history": str(history), "lens": 5,
            "page": page, "slack": slack}


def listed():
    return [
        # one decode step of a small batch: nothing but latency
        _tables("tables step 32", 32, 1, "1-4096", 128),
        # a step that schedules chunks for two thousand sequences, small pages
        _tables("tables chunks 2048", 2048, "0-512", "0-8192", 16, slack=5000),
        # one user, one token: the smallest attention call
        _attention("one token 512", 1, 1, 511, layers=2),
        # decode steps of a full batch, both kinds of cache
        _attention("decode 64 bf16", 64, 1, "1-8191"),
        _attention("decode 64 e4m3", 64, 1, "1-8191", cache="e4m3", gran=128),
        # few sequences with a long history: the work is split over the length
        _attention("decode 4 long e4m3", 4, 1, "30000-131000", cache="e4m3", gran=64),
        # several drafted tokens per sequence, odd heads, an odd page, the finest scales
        _attention("draft 24 odd e4m3", 24, "1-6", "1-4000", hq=12, hkv=4, d=64, page=48, cache="e4m3", gran=32),
        # eight prompts from their first token (the projections' lengths)
        _attention("prompts 8 bf16", 8, "1-1024", 0, layers=2),
        # chunks of prompts that have a history, quantized cache
        _attention("chunks 8 e4m3", 8, "1-1024", "0-4096", cache="e4m3", gran=128),
        # one long prompt in one call: the largest product
        _attention("prompt 8192 bf16", 1, 8192, 0),
        # one chunk of a very long prompt
        _attention("chunk 1000 of 33000", 1, 1000, 32000),
        # a sliding window, wide heads, more query heads per key head
        _attention("window 1024 wide", 6, "100-2000", "0-6000", hq=16, hkv=2, d=256, page=64, window=1024),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    most = max(_cost(c) for c in listed() if c["op"] == "attention")
    while True:
        lens = rng.randrange(1 << 20)
        if rng.random() < 0.25:
            new = "1" if rng.random() < 0.4 else "%d-%d" % (rng.randrange(2), _spread(rng, 2, 512))
            return {"op": "tables", "batch": _spread(rng, 1, 2048), "new": new,
                    "history": "%d-%d" % (rng.randrange(2), _spread(rng, 1, 8192)), "lens": lens,
                    "page": rng.choice([1, 16, 32, 48, 64, 100, 128, 256]), "slack": rng.randrange(5000)}
        kind = rng.random()
        batch = _spread(rng, 1, 96) if kind < 0.6 else _spread(rng, 1, 12)
        new = "1" if kind < 0.4 else "%d-%d" % (rng.randrange(2), _spread(rng, 2, 8) if kind < 0.6 else _spread(rng, 16, 8192))
        top = _spread(rng, 1, 131000) if kind < 0.75 else 0
        cache = rng.choice(["bf16", "e4m3"])
        gran = rng.choice([32, 64, 128]) if cache == "e4m3" else 0
        d = rng.choice([64, 128, 128, 128, 256, 80, 96, 72]) if cache == "bf16" else gran * rng.choice([1, 2, 2, 3, 4])
        hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
        case = {"op": "attention", "batch": batch, "new": new, "history": "%d-%d" % (top // rng.choice([1, 2, 8, 1000]), top),
                "lens": lens, "hq": hkv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16]), "hkv": hkv, "d": d,
                "page": rng.choice([8, 16, 32, 48, 64, 100, 128, 128, 256]), "layers": rng.choice([1, 2]),
                "cache": cache, "gran": gran, "causal": rng.random() < 0.85, "window": 0}
        if case["causal"] and rng.random() < 0.25:
            case["window"] = _spread(rng, 1, 4096)
        if d <= 256 and case["hq"] <= 128 and sum(_lengths(case)[0]) > 0 and _cost(case) <= most:
            return case


def _lengths(case):
    """New tokens and history of each sequence."""
    r = random.Random(case["lens"])

    def one(text):
        lo, _, hi = text.partition("-")
        return r.randint(int(lo), int(hi or lo))
    new = [one(case["new"]) for _ in range(case["batch"])]
    return new, [one(case["history"]) for _ in range(case["batch"])]


def _cost(case):
    """Elements of the padded score matrix and of the padded cache rows: what a plain
    pass holds, which bounds what is drawn."""
    new, hist = _lengths(case)
    longest = max(n + h for n, h in zip(new, hist))
    rows = case["batch"] * case["hq"] * max(new) * longest
    return max(rows, 2 * case["batch"] * longest * case["hkv"] * case["d"])


def _visible(case, new, hist):
    """Pairs of a token and a position it sees, and positions that some token sees."""
    pairs = seen = 0
    w = case["window"]
    for n, h in zip(new, hist):
        if not case["causal"]:
            pairs += n * (n + h)
        elif w:
            pairs += sum(min(w, h + j + 1) for j in range(n))
        else:
            pairs += n * h + n * (n + 1) // 2
        seen += 0 if n == 0 else n + (min(h, w - 1) if w else h)
    return pairs, seen


def work(case):
    new, hist = _lengths(case)
    batch, total, page = case["batch"], sum(new), case["page"]
    if case["op"] == "tables":
        fresh = sum(-(-(n + h) // page) - -(-h // page) for n, h in zip(new, hist))
        touched = sum(-(-(n + h) // page) - h // page for n, h in zip(new, hist) if n)
        # both lengths, the ids taken, the old entries that tokens land in; offsets, entries, slots, result
        return {"bytes": 4 * (2 * batch + fresh + (touched - fresh) + batch + 1 + fresh + total + 2),
                "flops": 4 * total + 8 * batch}
    pairs, seen = _visible(case, new, hist)
    row = case["hkv"] * case["d"]
    cache = 2 * seen * (row * 2 if case["cache"] == "bf16" else row + 4 * row // case["gran"])
    return {"bytes": 2 * 2 * total * case["hq"] * case["d"] + cache + 4 * (2 * batch + 1) + 4 * seen // page,
            "flops": 4 * pairs * case["hq"] * case["d"]}


def _tables_state(case, g, new, hist):
    """Page ids are distinct: each sequence's own pages first, then the free stack."""
    page, batch = case["page"], case["batch"]
    held = [-(-h // page) for h in hist]
    need = [-(-(n + h) // page) for n, h in zip(new, hist)]
    fresh = sum(need) - sum(held)
    wide = max(need) + 1
    ids = torch.randperm(sum(held) + fresh + case["slack"], generator=g, device="cuda").to(torch.int32)
    table = torch.full((batch, wide), -1, dtype=torch.int32, device="cuda")
    filled = torch.arange(wide, device="cuda")[None] < torch.tensor(held, device="cuda")[:, None]
    table[filled] = ids[:sum(held)]
    free = ids[sum(held):].clone()
    return {"case": case, "total": sum(new), "table": table, "free": free,
            "free_count": torch.tensor([free.numel()], dtype=torch.int32, device="cuda"),
            "cache_lengths": torch.tensor(hist, dtype=torch.int32, device="cuda"),
            "new_lengths": torch.tensor(new, dtype=torch.int32, device="cuda"),
            "offsets": torch.zeros(batch + 1, dtype=torch.int32, device="cuda"),
            "slots": torch.zeros(sum(new), dtype=torch.int32, device="cuda"),
            "result": torch.zeros(2, dtype=torch.int32, device="cuda")}


def _attention_state(case, g, new, hist):
    page, batch, hkv, d = case["page"], case["batch"], case["hkv"], case["d"]
    need = [-(-(n + h) // page) for n, h in zip(new, hist)]
    pages, wide = sum(need) + 3, max(need) + 1
    shape = (case["layers"], 2, pages, page, hkv, d)
    table = torch.zeros((batch, wide), dtype=torch.int32, device="cuda")
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    filled = torch.arange(wide, device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    table[filled] = ids[:sum(need)]
    stale = ids[sum(need):].long()
    # what a projection writes is near a normal distribution; pages that nobody holds
    # carry whatever was there (NaN here)
    layer = case["layers"] - 1
    if case["cache"] == "bf16":
        blocks = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        blocks[layer] = torch.randn(shape[1:], generator=g, device="cuda", dtype=torch.bfloat16)
        blocks[layer][:, stale] = float("nan")
        scales = None
    else:
        runs = torch.randn((*shape[1:5], d // case["gran"], case["gran"]), generator=g, device="cuda")
        s = runs.abs().amax(-1) / 448
        codes = (runs / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(shape[1:])
        codes[:, stale] = 0x7F
        blocks = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        blocks[layer] = codes
        scales = torch.zeros((*shape[:5], d // case["gran"]), device="cuda")
        scales[layer] = s
        blocks = blocks.view(torch.float8_e4m3fn)
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    state = {"case": case, "blocks": blocks, "scales": scales, "table": table, "layer": layer,
             "q": torch.randn((offsets[-1], case["hq"], d), generator=g, device="cuda", dtype=torch.bfloat16),
             "offsets": torch.tensor(offsets, dtype=torch.int32, device="cuda"),
             "cache_lengths": torch.tensor(hist, dtype=torch.int32, device="cuda"),
             "new_most": max(new), "len_most": max(n + h for n, h in zip(new, hist)),
             "scale": d ** -0.5}
    state["out"] = torch.zeros_like(state["q"])
    if own:   # a serving program allocates the workspace once, for all its layers and steps
        import grouped_gemm_qgemm_amd as lib
        n = lib.attention_ragged_paged_workspace(offsets[-1], batch, case["hq"], hkv, d)
        state["workspace"] = torch.empty(n, device="cuda")
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new, hist = _lengths(case)
    return (_tables_state if case["op"] == "tables" else _attention_state)(case, g, new, hist)


def _plain_tables(s):
    page, total = s["case"]["page"], s["total"]
    hist, new = s["cache_lengths"].long(), s["new_lengths"].long()
    offsets = torch.cat([new.new_zeros(1), new.cumsum(0)])
    held, need = (hist + page - 1) // page, (hist + new + page - 1) // page
    first = (need - held).cumsum(0) - (need - held)          # each sequence's first new page
    taken = (need - held).sum()
    cols = torch.arange(s["table"].shape[1], device="cuda")[None]
    nth = first[:, None] + cols - held[:, None]
    fresh = (cols >= held[:, None]) & (cols < need[:, None])
    pick = (s["free_count"].long() - 1 - nth).clamp(0, s["free"].numel() - 1) if s["free"].numel() else nth * 0
    ids = s["free"][pick] if s["free"].numel() else torch.zeros_like(s["table"])
    table = torch.where(fresh, ids, s["table"])
    rows = torch.arange(total, device="cuda")
    seq = torch.searchsorted(offsets[1:], rows, right=True)
    pos = hist[seq] + rows - offsets[seq]
    slots = table[seq, pos // page] * page + pos % page
    result = torch.stack([s["free_count"][0].long() - taken, taken * 0])
    return {"offsets": offsets.int(), "table": table, "slots": slots.int(), "result": result.int()}


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    group, batch, most, span = hq // hkv, case["batch"], s["new_most"], s["len_most"]
    offsets, hist = s["offsets"].long(), s["cache_lengths"].long()
    new = offsets[1:] - offsets[:-1]
    # keys and values of every position, zeros past a sequence's end
    pos = torch.arange(span, device="cuda")
    there = pos[None] < (hist + new)[:, None]
    at = s["table"][:, pos // page].long() * page + pos % page
    at = torch.where(there, at, 0)
    rows = s["blocks"][s["layer"]].reshape(2, -1, hkv, d)
    if s["scales"] is None:
        kv = rows[:, at].float()
    else:
        sc = s["scales"][s["layer"]].reshape(2, -1, hkv, d // case["gran"], 1)
        kv = (rows.view(torch.uint8)[:, at].view(torch.float8_e4m3fn).float().unflatten(-1, (d // case["gran"], -1)) * sc[:, at]).flatten(-2)
    kv = torch.where(there[None, :, :, None, None], kv, 0.0)                    # [2, batch, span, hkv, d]
    # queries, padded to the longest chunk: [batch, hkv, group * most, d]
    j = torch.arange(most, device="cuda")
    src = (offsets[:-1, None] + j[None]).clamp(max=s["q"].shape[0] - 1)
    qp = s["q"][src].float().view(batch, most, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, group * most, d)
    scores = torch.matmul(qp, kv[0].permute(0, 2, 3, 1).contiguous()).view(batch, hkv, group, most, span) * s["scale"]
    token = hist[:, None] + j[None]                                              # positions of the new tokens
    see = there[:, None, :].expand(batch, most, span)
    if case["causal"]:
        see = see & (pos[None, None] <= token[..., None])
    if case["window"]:
        see = see & (pos[None, None] > token[..., None] - case["window"])
    scores = torch.where(see[:, None, None], scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == float("-inf"), 0.0, top))
    del scores
    o = torch.matmul(e.view(batch, hkv, group * most, span), kv[1].permute(0, 2, 1, 3).contiguous())
    total = e.sum(-1).view(batch, hkv, group * most, 1)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.view(batch, hkv, group, most, d).permute(0, 3, 1, 2, 4)               # [batch, most, hkv, group, d]
    r = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(offsets[1:], r, right=True)
    return o[seq, r - offsets[seq]].reshape(-1, hq, d).to(torch.bfloat16)


def run(s):
    if not own:
        return _plain_tables(s) if s["case"]["op"] == "tables" else _plain_attention(s)
    import grouped_gemm_qgemm_amd as lib
    case = s["case"]
    if case["op"] == "tables":
        lib.tables_ragged_paged(s["offsets"], s["slots"], s["table"], s["result"], s["cache_lengths"], s["new_lengths"],
                                s["free"], s["free_count"], case["page"])
        return {"offsets": s["offsets"], "table": s["table"], "slots": s["slots"], "result": s["result"]}
    lib.attention_ragged_paged(s["out"], s["q"], s["offsets"], s["blocks"], s["cache_lengths"], s["table"], s["layer"],
                               s["scale"], s["workspace"], causal=case["causal"], window=case["window"],
                               kv_scales=s["scales"], quantization_granularity=case["gran"])
    return s["out"]


def exact(case, seed):
    """Attention by its definition, sequence by sequence and head by head, in 64 bits.
    The tables hold whole numbers, which need no such value."""
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    new, hist = _lengths(case)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b in range(case["batch"]):
        n, length = new[b], new[b] + hist[b]
        if n == 0:
            continue
        ids = s["table"][b, :-(-length // page)].long()
        kv = []
        for plane in (0, 1):
            x = s["blocks"].view(torch.uint8 if s["scales"] is not None else torch.bfloat16)[s["layer"], plane][ids]
            x = (x.view(torch.float8_e4m3fn) if s["scales"] is not None else x).double()
            if s["scales"] is not None:
                x = x * s["scales"][s["layer"], plane][ids].double().repeat_interleave(case["gran"], -1)
            kv.append(x.flatten(0, 1)[:length])
        p = torch.arange(length, device="cuda")[None]
        t = torch.arange(hist[b], length, device="cuda")[:, None]
        hide = torch.zeros((n, length), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hide |= p > t
        if case["window"]:
            hide |= p <= t - case["window"]
        for h in range(hq):
            k, v = (x[:, h // (hq // hkv)] for x in kv)
            z = (s["q"][row:row + n, h].double() @ k.t()) * s["scale"]
            z.masked_fill_(hide, float("-inf"))
            out[row:row + n, h] = torch.softmax(z, -1) @ v
        row += n
    return out
