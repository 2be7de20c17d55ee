"""The operators of speculative decoding over the paged KV cache, as cases to be measured.

  rope     rope_ragged_paged: rotary positions on the new tokens' queries and keys; keys
           and values written into their pages, bf16 or quantized to e4m3
  tree     attention_tree_ragged_paged: attention of each sequence's tree of drafted
           tokens over its history and the tokens' own ancestors
  keep     kv_keep_ragged_paged: the rows of the accepted path moved together, in every
           layer of the cache
  release  release_ragged_paged: pages that a sequence no longer needs, back on the stack
  read     kv_read_ragged_paged: ranges of the cache read back as dense rows

listed() names the cases, draw() gives others of the same ranges, prepare() makes
what a serving program holds before the call, run() is one call (the plain form in
elementary torch operations, or the library's kernels where `own` is true), exact()
the same answer in 64 bits, and work() the bytes and operations of one call.

A case's lengths and trees follow from its own numbers (so that work() knows them);
page ids and values follow from the seed.
"""
import math
import random

import torch

own = False

# the projections' workload: hidden rows of 4096 = 32 heads of 128, 8 key/value
# heads, pages of 128 slots
BASE = {"hq": 32, "hkv": 8, "d": 128, "page": 128, "layers": 1, "cache": "bf16", "gran": 0}


def _case(name, op, batch, new, history, **over):
    """new, history: "n" = that many for every sequence, "a-b" = uniform in a .. b."""
    return {"name": name, "op": op, "batch": batch, "new": str(new), "history": str(history), "lens": 5, **BASE, **over}


def listed():
    return [
        # one decode step of a full batch into a quantized cache: latency. Queries, keys
        # and values are parts of one row, as a fused projection leaves them
        _case("rope decode 64 e4m3", "rope", 64, 1, "1-8191", cache="e4m3", gran=128, rot=128, interleaved=False, fused=True),
        # eight prompts (the projections' lengths), half of the head turned, pairs side by side
        _case("rope prompts 8 bf16", "rope", 8, "1-1024", 0, layers=2, rot=64, interleaved=True, fused=False),
        # chunks of prompts far into long contexts, the finest scales, an odd page
        _case("rope chunks 16 e4m3", "rope", 16, "1000-3000", "0-1000000", page=48, cache="e4m3", gran=32, rot=128,
              interleaved=False, fused=True),
        # one user, a tree of 13 tokens: the smallest attention call
        _case("tree of 13", "tree", 1, 13, 500, layers=2, window=0),
        # a full batch with trees of 64 tokens
        _case("trees 32 of 64 bf16", "tree", 32, 64, "1-8191", window=0),
        # few sequences with a long history, quantized, trees of odd sizes, an odd page
        _case("trees 6 long e4m3", "tree", 6, "20-120", "8000-40000", page=48, cache="e4m3", gran=64, window=0),
        # five of eight tokens kept for one user, 32 layers
        _case("keep 1", "keep", 1, 8, 1000, layers=32, page=16),
        # a full batch, up to 9 tokens of trees of 64 kept, quantized cache
        _case("keep 64 e4m3", "keep", 64, 64, "1-8191", layers=32, cache="e4m3", gran=128),
        # the pages of 32 sequences' rejected tokens
        _case("release 32", "release", 32, 64, "1-4096", page=16),
        # a large batch, small pages, some sequences given up whole
        _case("release 4096", "release", 4096, "0-256", "0-2000", page=16),
        # the rows just written, in 16 bits, to work on them again
        _case("read 64 bf16", "read", 64, "1-64", "1-4096", out="bf16"),
        # long contexts out of a quantized cache
        _case("read 4 long e4m3", "read", 4, "30000-131000", "0-100", page=64, cache="e4m3", gran=64, out="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        op = rng.choice(["rope", "rope", "rope", "tree", "tree", "tree", "keep", "release", "read", "read"])
        cache = rng.choice(["bf16", "e4m3"])
        gran = rng.choice([32, 64, 128]) if cache == "e4m3" else 0
        d = rng.choice([64, 128, 128, 128, 256, 80, 96, 72]) if cache == "bf16" else gran * rng.choice([1, 2, 2, 3, 4])
        hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
        case = {"op": op, "lens": rng.randrange(1 << 20), "hq": hkv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16]), "hkv": hkv,
                "d": d, "page": rng.choice([8, 16, 32, 48, 64, 100, 128, 128, 256]), "layers": rng.choice([1, 2]),
                "cache": cache, "gran": gran}

        def upto(least, largest):
            """Between 0 or 1 and a size out of the range; or that size for all."""
            n = _spread(rng, least, largest)
            return str(n) if rng.random() < 0.3 else "%d-%d" % (rng.randrange(2), n)

        if op == "rope":
            case |= {"batch": _spread(rng, 1, 256), "new": upto(1, 4096), "history": upto(1, 1000000),
                     "rot": rng.choice([d, d, d, d // 2, d // 4, 2 * rng.randint(0, d // 2)]) // 2 * 2,
                     "interleaved": rng.random() < 0.5, "fused": rng.random() < 0.5}
        elif op == "tree":
            case |= {"batch": _spread(rng, 1, 64), "new": upto(1, 256), "history": upto(1, 40000),
                     "window": _spread(rng, 1, 4096) if rng.random() < 0.2 else 0}
        elif op == "keep":
            case |= {"batch": _spread(rng, 1, 256), "new": upto(1, 128), "history": upto(1, 8192), "layers": _spread(rng, 1, 64)}
        elif op == "release":
            case |= {"batch": _spread(rng, 1, 4096), "new": upto(1, 256), "history": upto(1, 8192)}
        else:
            case |= {"batch": _spread(rng, 1, 128), "new": upto(1, 131000), "history": upto(1, 4096),
                     "out": rng.choice(["bf16", "f32"])}
        if d <= 256 and case["hq"] <= 128 and sum(_lengths(case)[0]) > 0 and _cost(case) <= most[op]:
            return case


def _lengths(case):
    """New tokens (drafted ones, rows read back) and history of each sequence."""
    r = random.Random(case["lens"])

    def one(text):
        lo, _, hi = text.partition("-")
        return r.randint(int(lo), int(hi or lo))
    new = [one(case["new"]) for _ in range(case["batch"])]
    return new, [one(case["history"]) for _ in range(case["batch"])]


def _parents(case, new):
    """Each drafted token's parent among its sequence's, or -1: wide trees whose tokens come
    level by level, as a drafter adds them."""
    r = random.Random(case["lens"] + 1)
    return [[-1 if j == 0 else max(r.randrange(j), r.randrange(j)) if r.random() < 0.8 else j - 1 for j in range(n)] for n in new]


def _accepted(case, new):
    """The tokens of one path from the root of each sequence's tree."""
    r = random.Random(case["lens"] + 2)
    paths = []
    for parents in _parents(case, new):
        at = r.randrange(len(parents)) if parents else -1
        path = []
        while at >= 0:
            path.append(at)
            at = parents[at]
        paths.append(path[::-1][:9])
    return paths


def _kept(case, new, hist):
    """Lengths after the step: part of the drafted tokens stays; one sequence in 16 ends."""
    r = random.Random(case["lens"] + 3)
    return [0 if r.random() < 1 / 16 else h + r.randint(0, n) for n, h in zip(new, hist)]


def _row_bytes(case):
    """A position's keys (or values) in the cache, with their scales."""
    row = case["hkv"] * case["d"]
    return row * 2 if case["cache"] == "bf16" else row + 4 * row // case["gran"]


def _cost(case):
    """Elements that a plain pass holds or moves, which bounds what is drawn."""
    new, hist = _lengths(case)
    row = case["hkv"] * case["d"]
    if case["op"] == "rope":
        return sum(new) * (case["hq"] + 2 * case["hkv"]) * case["d"]
    if case["op"] == "tree":
        longest = max(n + h for n, h in zip(new, hist))
        return max(case["batch"] * case["hq"] * max(new) * longest, 2 * case["batch"] * longest * row)
    if case["op"] == "keep":
        return sum(map(len, _accepted(case, new))) * case["layers"] * row
    if case["op"] == "release":
        return case["batch"] * (max(n + h for n, h in zip(new, hist)) // case["page"] + 2)
    return sum(new) * row * (2 if case["out"] == "f32" else 1)


def work(case):
    new, hist = _lengths(case)
    batch, total, page, d = case["batch"], sum(new), case["page"], case["d"]
    if case["op"] == "rope":
        turned = total * (case["hq"] + case["hkv"]) * case["rot"]
        kept = 2 * total * case["hkv"] * d
        return {"bytes": 2 * total * (2 * case["hq"] + 2 * case["hkv"]) * d + 2 * total * _row_bytes(case)
                + 4 * (2 * batch + 1) + 4 * total // page + 2 * case["rot"],
                "flops": 3 * turned + (2 * kept if case["gran"] else 0) + 20 * total * case["rot"]}
    if case["op"] == "tree":
        pairs = seen = 0
        w = case["window"]
        for n, h, parents in zip(new, hist, _parents(case, new)):
            depth = []
            for p in parents:
                depth.append(1 if p < 0 else depth[p] + 1)
            pairs += sum(k + (min(h, max(w - k, 0)) if w else h) for k in depth)
            seen += 0 if n == 0 else n + (min(h, max(w - 1, 0)) if w else h)
        words = -(-max(max(new), 1) // 32)
        return {"bytes": 2 * 2 * total * case["hq"] * d + 2 * seen * _row_bytes(case) + 4 * total * words
                + 4 * (2 * batch + 1) + 4 * seen // page,
                "flops": 4 * pairs * case["hq"] * d}
    if case["op"] == "keep":
        paths = _accepted(case, new)
        moved = sum(at != i for path in paths for i, at in enumerate(path))
        return {"bytes": 2 * 2 * moved * case["layers"] * _row_bytes(case) + 4 * (sum(map(len, paths)) + 2 * batch + 2 * moved),
                "flops": 0}
    if case["op"] == "release":
        back = sum(max(0, -(-(n + h) // page) - -(-k // page)) for n, h, k in zip(new, hist, _kept(case, new, hist)))
        return {"bytes": 4 * (2 * batch + 2 * back + 3), "flops": 4 * batch}
    wide = 2 if case["out"] == "bf16" else 4
    return {"bytes": 2 * total * (_row_bytes(case) + case["hkv"] * d * wide) + 4 * (2 * batch + 1) + 4 * total // page,
            "flops": 2 * total * case["hkv"] * d if case["gran"] else 0}


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(new):
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    return _ints(offsets)


def _table(g, first, need, spare):
    """Page table [B, W] with distinct ids for each sequence's entries first .. need - 1, and
    the number of pages. Entries that the call has no use for hold a page of somebody else's."""
    held = [max(0, n - f) for f, n in zip(first, need)]
    pages, wide = sum(held) + spare, max(need) + 1
    table = torch.zeros((len(need), wide), dtype=torch.int32, device="cuda")
    cols = torch.arange(wide, device="cuda")[None]
    filled = (cols >= _ints(first)[:, None]) & (cols < _ints(need)[:, None])
    ids = (torch.randperm(pages - 1, generator=g, device="cuda") + 1).to(torch.int32)
    table[filled] = ids[:sum(held)]
    return table, pages


def _cache(case, g, pages, filled):
    """One cache: zeros, or what a projection writes (near a normal distribution) in the layers
    that are used."""
    shape = (case["layers"], 2, pages, case["page"], case["hkv"], case["d"])
    layers = range(case["layers"]) if case["op"] == "keep" else [case["layers"] - 1]
    gran = case["gran"]
    if not gran:
        blocks = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        for layer in layers if filled else []:
            blocks[layer] = torch.randn(shape[1:], generator=g, device="cuda", dtype=torch.bfloat16)
        return blocks, None
    blocks = torch.zeros(shape, dtype=torch.uint8, device="cuda")
    scales = torch.zeros((*shape[:5], case["d"] // gran), device="cuda")
    for layer in layers if filled else []:
        runs = torch.randn((*shape[1:5], case["d"] // gran, gran), generator=g, device="cuda")
        s = runs.abs().amax(-1) / 448
        blocks[layer] = (runs / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(shape[1:])
        scales[layer] = s
    return blocks.view(torch.float8_e4m3fn), scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new, hist = _lengths(case)
    op, page, hq, hkv, d = case["op"], case["page"], case["hq"], case["hkv"], case["d"]
    need = [-(-(n + h) // page) for n, h in zip(new, hist)]
    total = sum(new)
    s = {"case": case, "layer": case["layers"] - 1, "offsets": _offsets(new), "cache_lengths": _ints(hist)}
    if op == "release":
        kept = _kept(case, new, hist)
        s["table"], pages = _table(g, [0] * len(new), need, 1)
        s["held"], s["kept"] = _ints([n + h for n, h in zip(new, hist)]), _ints(kept)
        count = 50
        s["free"] = torch.zeros(count + pages, dtype=torch.int32, device="cuda")
        s["free"][:count] = pages + torch.randperm(count, generator=g, device="cuda").to(torch.int32)
        s["free_count"], s["result"] = _ints([count]), _ints([0, 0])
        return s
    # only pages that the call touches are there: history matters to attention alone
    first = [0] * len(new) if op == "tree" else [h // page for h in hist]
    s["table"], pages = _table(g, first, need, 3)
    s["blocks"], s["scales"] = _cache(case, g, pages, op != "rope")
    if op == "rope":
        shape = (total, hq + 2 * hkv, d)
        if case["fused"]:
            s["qkv"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        else:
            s["q"], s["k"], s["v"] = (torch.randn((total, n, d), generator=g, device="cuda", dtype=torch.bfloat16)
                                      for n in (hq, hkv, hkv))
        s["q_out"] = torch.zeros((total, hq, d), dtype=torch.bfloat16, device="cuda")
        # frequencies of base 10000, slowed for long contexts (each by its own factor), and the
        # amplitude that goes with that
        half = case["rot"] // 2
        i = torch.arange(half, device="cuda", dtype=torch.float64)
        slow = 1 + 7 * torch.rand(half, generator=g, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-i / max(half, 1)) / slow).float()
        s["amplitude"] = 1.2079
    elif op == "tree":
        words = -(-max(max(new), 1) // 32)
        rows = []
        for parents in _parents(case, new):
            seen = []
            for j, p in enumerate(parents):
                seen.append(1 << j | (seen[p] if p >= 0 else 0))
                rows.append([(seen[j] >> 32 * w & 0xFFFFFFFF) for w in range(words)])
        s["mask"] = torch.tensor(rows, dtype=torch.int64, device="cuda").to(torch.int32)
        s["q"] = torch.randn((total, hq, d), generator=g, device="cuda", dtype=torch.bfloat16)
        s["out"] = torch.zeros_like(s["q"])
        s["scale"] = d ** -0.5
        s["new_most"], s["len_most"] = max(new), max(n + h for n, h in zip(new, hist))
        if own:   # a serving program allocates the workspace once, for all its layers and steps
            import grouped_gemm_qgemm_amd as lib
            s["workspace"] = torch.empty(lib.attention_ragged_paged_workspace(total, case["batch"], hq, hkv, d), device="cuda")
    elif op == "keep":
        paths = _accepted(case, new)
        wide = max(1, max(map(len, paths)))
        s["path"] = _ints([path + [0] * (wide - len(path)) for path in paths])
        s["kept"] = _ints([len(path) for path in paths])
    else:
        kind = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        s["k_out"], s["v_out"] = (torch.zeros((total, hkv, d), dtype=kind, device="cuda") for _ in range(2))
    return s


def _rows_of(s):
    """Sequence of each row, its place among the sequence's rows, and its slot in a plane."""
    page = s["case"]["page"]
    offsets, hist = s["offsets"].long(), s["cache_lengths"].long()
    total = (s["q_out"] if "q_out" in s else s["k_out"]).shape[0]
    rows = torch.arange(total, device="cuda")
    seq = torch.searchsorted(offsets[1:], rows, right=True)
    pos = hist[seq] + rows - offsets[seq]
    return pos, s["table"][seq, pos // page].long() * page + pos % page


def _turned(x, cos, sin, half, interleaved):
    """x [T, H, D] with its first 2 * half dims turned by the angles of cos and sin [T, 1, half]."""
    r = 2 * half
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :half], x[..., half:r])
    c, z = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([c, z], -1).flatten(-2) if interleaved else torch.cat([c, z], -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_rope(s):
    case = s["case"]
    hq, hkv, d, gran = case["hq"], case["hkv"], case["d"], case["gran"]
    q, k, v = (t.float() for t in (s["qkv"].split([hq, hkv, hkv], 1) if case["fused"] else (s["q"], s["k"], s["v"])))
    pos, at = _rows_of(s)
    angle = pos.double()[:, None, None] * s["inv_freq"].double()
    cos, sin = ((f(angle) * s["amplitude"]).float() for f in (torch.cos, torch.sin))
    half = case["rot"] // 2
    s["q_out"].copy_(_turned(q, cos, sin, half, case["interleaved"]).to(torch.bfloat16))
    kv = torch.stack([_turned(k, cos, sin, half, case["interleaved"]), v])
    if not gran:
        s["blocks"][s["layer"]].view(2, -1, hkv, d)[:, at] = kv.to(torch.bfloat16)
        return {"q": s["q_out"], "blocks": s["blocks"]}
    runs = kv.unflatten(-1, (d // gran, gran))
    size = runs.abs().amax(-1) / 448
    codes = torch.where(size[..., None] > 0, runs / size[..., None], 0.0).to(torch.float8_e4m3fn).view(torch.uint8)
    s["blocks"].view(torch.uint8)[s["layer"]].view(2, -1, hkv, d)[:, at] = codes.flatten(-2)
    s["scales"][s["layer"]].view(2, -1, hkv, d // gran)[:, at] = size
    return {"q": s["q_out"], "blocks": s["blocks"], "scales": s["scales"]}


def _values(s, at):
    """Keys and values [2, *at.shape, Hkv, D] of slots `at`, in 32 bits."""
    case = s["case"]
    hkv, d, gran = case["hkv"], case["d"], case["gran"]
    if not gran:
        return s["blocks"][s["layer"]].view(2, -1, hkv, d)[:, at].float()
    codes = s["blocks"].view(torch.uint8)[s["layer"]].view(2, -1, hkv, d)[:, at].view(torch.float8_e4m3fn).float()
    return (codes.unflatten(-1, (d // gran, gran)) * s["scales"][s["layer"]].view(2, -1, hkv, d // gran, 1)[:, at]).flatten(-2)


def _plain_tree(s):
    case = s["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    group, batch, most, span = hq // hkv, case["batch"], s["new_most"], s["len_most"]
    offsets, hist = s["offsets"].long(), s["cache_lengths"].long()
    new = offsets[1:] - offsets[:-1]
    # keys and values of every position, zeros past a sequence's end
    pos = torch.arange(span, device="cuda")
    there = pos[None] < (hist + new)[:, None]
    at = torch.where(there, s["table"][:, pos // page].long() * page + pos % page, 0)
    kv = torch.where(there[None, :, :, None, None], _values(s, at), 0.0)             # [2, batch, span, hkv, d]
    # queries, padded to the largest tree: [batch, hkv, group * most, d]
    j = torch.arange(most, device="cuda")
    src = (offsets[:-1, None] + j[None]).clamp(max=s["q"].shape[0] - 1)
    qp = s["q"][src].float().view(batch, most, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, group * most, d)
    scores = torch.matmul(qp, kv[0].permute(0, 2, 3, 1).contiguous()).view(batch, hkv, group, most, span) * s["scale"]
    # drafted tokens that a token sees, [batch, most, most]; of the history all, or what the window leaves
    drafted = (s["mask"][src].long()[..., j // 32] >> (j % 32) & 1).bool() & (j[None, None] < new[:, None, None])
    low = torch.zeros_like(src)
    if case["window"]:
        low = (hist[:, None] - (case["window"] - drafted.sum(-1)).clamp(min=0)).clamp(min=0)
    i = pos[None] - hist[:, None]                                                    # [batch, span]
    own_tree = torch.gather(drafted, 2, i.clamp(0, most - 1)[:, None].expand(batch, most, span))
    see = torch.where(i[:, None] < 0, pos[None, None] >= low[..., None], own_tree & (i < most)[:, None])
    scores = torch.where(see[:, None, None], scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == float("-inf"), 0.0, top))
    del scores
    o = torch.matmul(e.view(batch, hkv, group * most, span), kv[1].permute(0, 2, 1, 3).contiguous())
    total = e.sum(-1).view(batch, hkv, group * most, 1)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.view(batch, hkv, group, most, d).permute(0, 3, 1, 2, 4)                   # [batch, most, hkv, group, d]
    r = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(offsets[1:], r, right=True)
    return o[seq, r - offsets[seq]].reshape(-1, hq, d).to(torch.bfloat16)


def _plain_keep(s):
    case = s["case"]
    page = case["page"]
    i = torch.arange(s["path"].shape[1], device="cuda")[None]
    hist = s["cache_lengths"].long()[:, None]
    there = i < s["kept"][:, None]
    # what is not kept moves from slot to slot of itself
    to = hist + torch.where(there, i, 0)
    of = hist + torch.where(there, s["path"].long(), 0)
    slot = [torch.gather(s["table"], 1, p // page).long() * page + p % page for p in (to, of)]
    slot = [torch.where(there, x, 0).flatten() for x in slot]
    for t in (s["blocks"].view(torch.uint8) if case["gran"] else s["blocks"], s["scales"]):
        if t is not None:
            flat = t.view(case["layers"], 2, -1, case["hkv"], t.shape[-1])
            flat[:, :, slot[0]] = flat[:, :, slot[1]]
    return {"blocks": s["blocks"]} if s["scales"] is None else {"blocks": s["blocks"], "scales": s["scales"]}


def _plain_release(s):
    page = s["case"]["page"]
    held, kept = ((x.long() + page - 1) // page for x in (s["held"], s["kept"]))
    back = (held - kept).clamp(min=0)
    first, total = back.cumsum(0) - back, back.sum()
    cols = torch.arange(s["table"].shape[1], device="cuda")[None]
    goes = (cols >= kept[:, None]) & (cols < held[:, None])
    # the last page of the last sequence lies deepest; what does not go lands behind the stack's end
    place = s["free_count"].long() + total - 1 - (first[:, None] + cols - kept[:, None])
    wide = torch.cat([s["free"], s["free"][:1]])
    wide[torch.where(goes, place, s["free"].numel())] = s["table"]
    s["free"].copy_(wide[:-1])
    s["result"].copy_(torch.stack([s["free_count"][0].long() + total, total * 0]))
    return {"free": s["free"], "result": s["result"]}


def _plain_read(s):
    kv = _values(s, _rows_of(s)[1])
    s["k_out"].copy_(kv[0].to(s["k_out"].dtype))
    s["v_out"].copy_(kv[1].to(s["v_out"].dtype))
    return {"k": s["k_out"], "v": s["v_out"]}


def run(s):
    case = s["case"]
    if not own:
        return {"rope": _plain_rope, "tree": _plain_tree, "keep": _plain_keep, "release": _plain_release,
                "read": _plain_read}[case["op"]](s)
    import grouped_gemm_qgemm_amd as lib
    if case["op"] == "rope":
        hq, hkv = case["hq"], case["hkv"]
        q, k, v = s["qkv"].split([hq, hkv, hkv], 1) if case["fused"] else (s["q"], s["k"], s["v"])
        lib.rope_ragged_paged(s["q_out"], q, k, v, s["offsets"], s["blocks"], s["cache_lengths"], s["table"], s["layer"],
                              s["inv_freq"], interleaved=case["interleaved"], amplitude=s["amplitude"],
                              kv_scales=s["scales"], quantization_granularity=case["gran"])
        out = {"q": s["q_out"], "blocks": s["blocks"]}
        return out if s["scales"] is None else out | {"scales": s["scales"]}
    if case["op"] == "tree":
        lib.attention_tree_ragged_paged(s["out"], s["q"], s["offsets"], s["mask"], s["blocks"], s["cache_lengths"], s["table"],
                                        s["layer"], s["scale"], s["workspace"], window=case["window"],
                                        kv_scales=s["scales"], quantization_granularity=case["gran"])
        return s["out"]
    if case["op"] == "keep":
        lib.kv_keep_ragged_paged(s["path"], s["kept"], s["blocks"], s["cache_lengths"], s["table"], kv_scales=s["scales"],
                                 quantization_granularity=case["gran"])
        return {"blocks": s["blocks"]} if s["scales"] is None else {"blocks": s["blocks"], "scales": s["scales"]}
    if case["op"] == "release":
        lib.release_ragged_paged(s["free"], s["result"], s["table"], s["held"], s["kept"], s["free_count"], case["page"])
        return {"free": s["free"], "result": s["result"]}
    lib.kv_read_ragged_paged(s["k_out"], s["v_out"], s["offsets"], s["cache_lengths"], s["blocks"], s["table"], s["layer"],
                             kv_scales=s["scales"], quantization_granularity=case["gran"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _exact_slots(s, b, first, count):
    page = s["case"]["page"]
    p = torch.arange(first, first + count, device="cuda")
    return s["table"][b].long()[p // page], p % page


def _exact_values(s, plane, where):
    """Rows of one plane in 64 bits, at (pages, slots)."""
    gran = s["case"]["gran"]
    if not gran:
        return s["blocks"][s["layer"], plane][where].double()
    codes = s["blocks"].view(torch.uint8)[s["layer"], plane][where].view(torch.float8_e4m3fn).double()
    return codes * s["scales"][s["layer"], plane][where].double().repeat_interleave(gran, -1)


def exact(case, seed):
    """Each operator by its definition, sequence by sequence, in 64 bits. Whole numbers (the
    stack of pages) need no such value. Codes are given before their rounding."""
    if case["op"] == "release":
        return None
    s = prepare(case, seed)
    new, hist = _lengths(case)
    hq, hkv, d, gran = case["hq"], case["hkv"], case["d"], case["gran"]
    starts = [sum(new[:b]) for b in range(case["batch"])]
    if case["op"] == "rope":
        half = case["rot"] // 2
        q_out = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda")
        blocks = torch.zeros(s["blocks"].shape, dtype=torch.float64, device="cuda")
        scales = None if not gran else torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
        for b, (n, h, r) in enumerate(zip(new, hist, starts)):
            if n == 0:
                continue
            rows = slice(r, r + n)
            q, k, v = ((s["qkv"][rows, :hq], s["qkv"][rows, hq:hq + hkv], s["qkv"][rows, hq + hkv:]) if case["fused"]
                       else (s["q"][rows], s["k"][rows], s["v"][rows]))
            angle = torch.arange(h, h + n, device="cuda", dtype=torch.float64)[:, None] * s["inv_freq"].double()[None]
            turn = torch.polar(torch.full_like(angle, s["amplitude"]), angle)[:, None]       # as complex numbers
            turned = []
            for x in (q.double(), k.double()):
                y = x.clone()
                if case["interleaved"]:
                    z = torch.view_as_complex(x[..., :2 * half].reshape(n, -1, half, 2)) * turn
                    y[..., :2 * half] = torch.view_as_real(z).flatten(-2)
                else:
                    z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
                    y[..., :half], y[..., half:2 * half] = z.real, z.imag
                turned.append(y)
            q_out[rows] = turned[0]
            where = _exact_slots(s, b, h, n)
            for plane, x in enumerate((turned[1], v.double())):
                if gran:
                    size = x.reshape(n, hkv, d // gran, gran).abs().amax(-1) / 448
                    scales[s["layer"], plane][where] = size
                    x = x / size.repeat_interleave(gran, -1)
                blocks[s["layer"], plane][where] = x
        return {"q": q_out, "blocks": blocks} if not gran else {"q": q_out, "blocks": blocks, "scales": scales}
    if case["op"] == "read":
        out = [torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
        for b, (n, h, r) in enumerate(zip(new, hist, starts)):
            for plane in (0, 1):
                out[plane][r:r + n] = _exact_values(s, plane, _exact_slots(s, b, h, n))
        return {"k": out[0], "v": out[1]}
    if case["op"] == "keep":
        blocks = s["blocks"].view(torch.uint8) if gran else s["blocks"]
        paths = _accepted(case, new)
        for t in (blocks, s["scales"]):
            for b, (h, path) in enumerate(zip(hist, paths)):
                if t is not None and path:
                    pages, slots = _exact_slots(s, b, h, max(path) + 1)
                    rows = t[:, :, pages[path], slots[path]].clone()
                    t[:, :, pages[:len(path)], slots[:len(path)]] = rows
        blocks = (blocks.view(torch.float8_e4m3fn) if gran else blocks).double()
        return {"blocks": blocks} if not gran else {"blocks": blocks, "scales": s["scales"].double()}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (n, h, r, parents) in enumerate(zip(new, hist, starts, _parents(case, new))):
        if n == 0:
            continue
        sees = torch.zeros((n, n), dtype=torch.bool)
        for j, p in enumerate(parents):
            if p >= 0:
                sees[j] = sees[p]
            sees[j, j] = True
        hide = torch.zeros((n, h + n), dtype=torch.bool, device="cuda")
        hide[:, h:] = ~sees.cuda()
        if case["window"]:
            left = (case["window"] - sees.sum(1)).clamp(min=0).cuda()
            hide[:, :h] = torch.arange(h, device="cuda")[None] < h - left[:, None]
        where = _exact_slots(s, b, 0, h + n)
        k, v = (_exact_values(s, plane, where) for plane in (0, 1))
        for head in range(hq):
            z = (s["q"][r:r + n, head].double() @ k[:, head // (hq // hkv)].t()) * s["scale"]
            z.masked_fill_(hide, float("-inf"))
            out[r:r + n, head] = torch.softmax(z, -1) @ v[:, head // (hq // hkv)]
    return out
