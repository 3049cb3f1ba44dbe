"""Measured cases of the operators that keep a long paged KV cache small.

Three operators over the paged, position-free pool, five calls:

  prefill_window, decode_window   attention in which a key at position n is visible to a query at position m iff n <= m and
                                  (m - n < window or n < sinks)
  prefill_mass, decode_mass       the attention weight that every cached token has received, per KV head, added to what it had
                                  (decode_mass: one decode step, its output and the weights together)
  evict                           each KV head keeps its first `sinks` tokens, its last `recent` ones and those of the rest with
                                  the most weight, `budget` in all, copied into pages of their own

Tables are ragged: a request is a few documents, each in consecutive pages of its own with a partial last page, then its own
(writable) segment. Decode calls also append the step's token, so a pass starts by putting the table back to what it was.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
THETA = 5.0e5


# ------------------------------------------------------------------------------------------------ cases

def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="bf16", hq=32, hkv=8, d=128, requests=1, docs=4, doc_min=256, doc_max=256, tail=64,
             rows_min=0, rows=0, window=0, sinks=0, budget=0, recent=0, decay=1.0, lengths=1)
    c.update(kw)
    return c


def listed():
    return [
        # one layer of an 8B-shaped model: 16 requests of 8 documents, the query segments' prefill under a short window
        _case("prefill window, 8B", "prefill_window", requests=16, docs=8, tail=64, rows_min=64, rows=64, window=512, sinks=4),
        # a long prompt prefilled from nothing: every token is a query row
        _case("prefill window, prompt", "prefill_window", docs=0, tail=8192, rows_min=8192, rows=8192, window=1024, sinks=16),
        # long contexts of ragged documents, a window wider than most of them, query segments of odd lengths
        _case("prefill window, long", "prefill_window", requests=8, docs=20, doc_min=700, doc_max=1024, tail=128, rows_min=33,
              rows=128, window=8192, sinks=64, lengths=2),
        # one user's next token: latency
        _case("decode window, one", "decode_window", requests=1, docs=15, tail=100, window=1024, sinks=4),
        # a serving batch of long contexts (20 documents of up to 512 tokens)
        _case("decode window, batch", "decode_window", requests=128, docs=20, doc_min=400, doc_max=512, tail=40, window=4096,
              sinks=4, lengths=3),
        # the fp32 pool of the parity configurations
        _case("decode window, fp32", "decode_window", dtype="f32", hq=4, hkv=2, d=64, requests=4, docs=6, doc_min=30, doc_max=250,
              tail=33, window=300, sinks=5, lengths=4),
        # observation of a step for one user: latency
        _case("decode mass, one", "decode_mass", requests=1, docs=8, tail=70),
        # a serving batch of a 70B-shaped layer, weights that fade
        _case("decode mass, batch", "decode_mass", hq=64, requests=64, docs=16, doc_min=300, doc_max=512, tail=50, decay=0.9,
              lengths=5),
        # the last 64 prompt tokens observe the cache before it is cut down (8B-shaped layer)
        _case("prefill mass, 8B", "prefill_mass", requests=16, docs=8, tail=64, rows_min=64, rows=64, decay=0.0),
        # long contexts, query segments of odd lengths observe
        _case("prefill mass, long", "prefill_mass", requests=8, docs=20, doc_min=700, doc_max=1024, tail=128, rows_min=100, rows=128,
              lengths=6),
        # one user's cache cut to a quarter
        _case("evict, one", "evict", requests=1, docs=8, tail=70, budget=512, sinks=4, recent=128),
        # a serving batch cut to 2048 tokens a request
        _case("evict, batch", "evict", requests=32, docs=20, doc_min=400, doc_max=512, tail=100, budget=2048, sinks=16, recent=512,
              lengths=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill_window", "decode_window", "prefill_mass", "decode_mass", "evict"])
    hq, hkv = rng.choice([(32, 8), (64, 8), (16, 8), (8, 8)])
    docs, doc_max = _log(rng, 1, 20), _log(rng, 17, 1024)
    tokens = docs * doc_max
    c = _case("", op, hq=hq, hkv=hkv, docs=docs, doc_max=doc_max, doc_min=max(1, int(doc_max * rng.uniform(0.3, 1.0))),
              lengths=rng.randrange(1 << 20))
    c.pop("name")
    if op.startswith("prefill"):
        c["rows"] = _log(rng, 1, 128)
        c["rows_min"] = max(1, int(c["rows"] * rng.uniform(0.3, 1.0)))
        c["tail"] = c["rows"] + rng.randrange(20)
        most = min(16, int(5e8 / (c["rows"] * hq * (tokens + 200))))
    else:
        c["tail"] = _log(rng, 1, 300)
        most = min(64, int(6e5 / (tokens + 300)))
    c["requests"] = _log(rng, 1, max(1, most))
    if op.endswith("window"):
        c["window"], c["sinks"] = _log(rng, 1, 8192), rng.choice([0, 1, 4, rng.randrange(100)])
    elif op.endswith("mass"):
        c["decay"] = rng.choice([0.0, 1.0, rng.uniform(0.5, 1.0)])
    else:
        c["sinks"], c["recent"] = rng.randrange(20), rng.randrange(64)
        c["budget"] = max(c["sinks"] + c["recent"], 1, int((tokens + 16) * rng.uniform(0.1, 0.9)))
    return c


def _lengths(case):
    """Per request: its documents' lengths, its own segment's, its query rows (from the case alone)."""
    rng = random.Random(case["lengths"])
    got = []
    for _ in range(case["requests"]):
        rows = rng.randint(case["rows_min"], case["rows"])
        got.append(([rng.randint(case["doc_min"], case["doc_max"]) for _ in range(case["docs"])], case["tail"], rows))
    return got


def _pages(n):
    return -(-n // PAGE)


def _visible(case, n, m):
    """How many of the positions 0..n-1 a query at m sees."""
    n = min(n, m + 1)
    if not case["window"]:
        return n
    lo = max(0, m - case["window"] + 1)
    return max(0, n - lo) + min(case["sinks"], lo, n)


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    size = 4 if case["dtype"] == "f32" else 2
    decode = case["op"].startswith("decode")
    by = fl = 0
    for docs, tail, rows in _lengths(case):
        n = sum(docs) + tail
        if case["op"] == "evict":   # the weights once; the kept rows read and written, K and V
            kept = min(n, case["budget"])
            by += n * hkv * 4 + kept * hkv * (4 * d * size + 4)
            continue
        n += decode
        rows = 1 if decode else rows
        by += (hq * d * size) * rows + (2 * hkv * d * size if decode else 0)   # q, the step's k and v
        mass = case["op"].endswith("mass")
        if rows and mass:
            live = n
        elif rows:   # keys that some row sees
            lo = max(0, n - rows - case["window"] + 1)
            live = n - lo + min(case["sinks"], lo)
        else:
            live = 0
        if case["op"] != "prefill_mass":
            by += live * hkv * 2 * d * size + rows * hq * d * size             # K, V, the output
        else:
            by += live * hkv * d * size                                        # K
        if mass:
            by += n * hkv * 4 * (2 if case["decay"] else 1)                    # weights read and written
        pairs = sum(_visible(case, n, m) for m in range(n - rows, n))
        fl += pairs * hq * d * (2 if case["op"] == "prefill_mass" else 4)
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------------------------------------ inputs

def _table(case):
    """The requests' segments: (first page, start, tokens, pages, writable) each, and the pages used. Documents lie in
    consecutive pages; the order of the documents in the pool is not the requests'."""
    lengths = _lengths(case)
    spans = []
    for r, (docs, tail, _) in enumerate(lengths):
        at = 0
        for n in docs:
            spans.append([r, at, n, _pages(n), False])
            at += n
        spans.append([r, at, tail, _pages(tail) + (1 if case["op"].startswith("decode") else 0), True])
    order = list(range(len(spans)))
    random.Random(case["lengths"] + 1).shuffle(order)
    first, used = [0] * len(spans), 0
    for i in order:
        first[i] = used
        used += spans[i][3]
    table = [[] for _ in lengths]
    for f, (r, at, n, pages, w) in zip(first, spans):
        table[r].append((f, at, n, pages, w))
    return table, used


def _entries(table):
    """The packed 64-bit entries of all requests and the requests' offsets."""
    words, offsets = [], [0]
    for segments in table:
        for first, at, n, pages, w in segments:
            j = np.arange(pages, dtype=np.int64)
            words.append((first + j) | ((at + PAGE * j) << 32) | (np.clip(n - PAGE * j, 0, PAGE) << 58) | (np.int64(-1 << 63) if w else np.int64(0)))
        offsets.append(offsets[-1] + sum(s[3] for s in segments))
    return np.concatenate(words), np.array(offsets, np.int32)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    op, hq, hkv, d, R = case["op"], case["hq"], case["hkv"], case["d"], case["requests"]
    t = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    table, used = _table(case)
    words, offsets = _entries(table)
    lengths = _lengths(case)
    tokens = [sum(docs) + tail for docs, tail, _ in lengths]
    positions = max(tokens) + 2
    kept_pages = _pages(case["budget"])
    num_pages = used + R * kept_pages
    s = {"case": case, "used": used}

    if own:   # the handle that a program keeps: the pool with its position table, the batch with its table
        import position_agnostic_kv_lazyattn_gb300 as L
        pool = L.DevicePool(num_pages, hq, hkv, d, case["dtype"], THETA, positions, device=dev)
        rows = [x[2] for x in lengths]
        batch = L.Batch([[L.Segment(range(f, f + p), at, n, writable=w) for f, at, n, p, w in segments] for segments in table],
                        rows if case["rows"] else (), [n - x for n, x in zip(tokens, rows)], device=dev)
        s.update(L=L, pool=pool, batch=batch, k=pool.k_pool, v=pool.v_pool, entries=batch.entries)
        if op.endswith("window"):
            kind = L.LAZYATTN_OP_PREFILL if op.startswith("prefill") else L.LAZYATTN_OP_DECODE
            size = L.lazyattn_window_workspace_size(pool.handle, kind, batch.c, case["window"], case["sinks"])
        elif op.endswith("mass"):
            kind = L.LAZYATTN_OP_PREFILL_MASS if op.startswith("prefill") else L.LAZYATTN_OP_DECODE_MASS
            size = L.lazyattn_workspace_size(pool.handle, kind, batch.c)
        else:
            size = 0
        s.update(ws=torch.zeros(max(size, 256), dtype=torch.uint8, device=dev), ws_bytes=size)
    else:
        s.update(k=torch.zeros(num_pages, hkv, PAGE, d, dtype=t, device=dev), v=torch.zeros(num_pages, hkv, PAGE, d, dtype=t, device=dev))

    # documents' keys and values; slots without a token hold zeros, as everywhere in a pool
    filled = np.zeros((used, PAGE), bool)
    for segments in table:
        for first, at, n, pages, w in segments:
            filled[first:first + pages] = np.arange(pages * PAGE).reshape(pages, PAGE) < n
    mask = torch.from_numpy(filled).to(dev)[:, None, :, None]
    for x in (s["k"], s["v"]):
        x[:used].normal_(generator=gen)
        x[:used].mul_(mask)

    s["entries0"] = torch.from_numpy(words).to(dev)
    # the table as one row of entries per request, for the plain forms: -1 where a request has fewer
    E = int(np.diff(offsets).max())
    at = np.full((R, E), -1, np.int64)
    for r in range(R):
        at[r, : offsets[r + 1] - offsets[r]] = np.arange(offsets[r], offsets[r + 1])
    s["entry"] = torch.from_numpy(at).to(dev)
    s["offsets"] = offsets
    angle = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * (
        THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device=dev) / d))
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(t)

    def weights():   # a few tokens hold most of the weight; some were never seen at all
        w = 0.02 * torch.exp(2.0 * torch.randn(len(words), hkv, PAGE, generator=gen, device=dev))
        return w * (torch.rand(w.shape, generator=gen, device=dev) > 0.2)

    if op.startswith("decode"):
        s.update(q=normal(R, hq, d, scale=2.0), k_new=normal(R, hkv, d), v_new=normal(R, hkv, d))
        s["out"] = torch.empty(R, hq, d, dtype=t, device=dev)
        # where the step's token goes, for the plain forms: the first free slot of the request's own segment
        spot = [(int(offsets[r + 1]) - table[r][-1][3] + case["tail"] // PAGE, case["tail"] % PAGE) for r in range(R)]
        s["spot"] = torch.tensor(spot, device=dev)
        s["m"] = torch.tensor(tokens, device=dev)
    elif op.startswith("prefill"):
        rows = [x[2] for x in lengths]
        s.update(q=normal(sum(rows), hq, d, scale=2.0), out=torch.empty(sum(rows), hq, d, dtype=t, device=dev))
        j = np.arange(max(rows))[None, :]
        start = np.cumsum([0] + rows)[:-1, None]
        s["row"] = torch.from_numpy(np.where(j < np.array(rows)[:, None], start + j, -1)).to(dev)
        s["m"] = torch.from_numpy((np.array(tokens) - np.array(rows))[:, None] + j).to(dev)
        s["rows"] = rows
    if op.endswith("mass"):
        s["mass"] = weights() if case["decay"] else None
        s["mass_out"] = torch.zeros(len(words), hkv, PAGE, device=dev)
    if op == "evict":
        s["mass"] = weights()
        page = used + torch.arange(R * kept_pages, device=dev)
        s["dst0"] = page | (-1 << 63)                                # writable pages of each request's own
        s["dst"] = s["dst0"].clone()
        s["dst_offsets"] = (kept_pages * torch.arange(R + 1, device=dev)).to(torch.int32)
        s["kept"] = torch.empty(R, hkv, case["budget"], dtype=torch.int32, device=dev)
        s["dst_mass"] = torch.zeros(R * kept_pages, hkv, PAGE, device=dev)
        s["tokens"] = tokens
    return s


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    if op == "evict":
        return _plain_evict(s)
    return _plain_attention(s)


def _own(s):
    c, L, pool, batch = s["case"], s["L"], s["pool"], s["batch"]
    op = c["op"]
    if op == "prefill_window":
        L.lazyattn_prefill_window(pool.handle, batch.c, s["q"], s["out"], c["window"], c["sinks"], s["ws"], s["ws_bytes"])
        return s["out"]
    if op == "prefill_mass":
        L.lazyattn_prefill_mass(pool.handle, batch.c, s["q"], s["mass"], s["mass_out"], c["decay"], s["ws"], s["ws_bytes"])
        return s["mass_out"]
    if op == "evict":
        L.lazyattn_evict(pool.handle, batch.c, s["mass"], c["budget"], c["sinks"], c["recent"], s["dst"], s["dst_offsets"],
                         s["kept"], s["dst_mass"])
        return {"kept": s["kept"], "entries": s["dst"], "mass": s["dst_mass"], "k": s["k"][s["used"]:], "v": s["v"][s["used"]:]}
    s["entries"].copy_(s["entries0"])   # the step appends to the table
    if op == "decode_window":
        L.lazyattn_decode_window(pool.handle, batch.c, s["q"], s["k_new"], s["v_new"], s["out"], c["window"], c["sinks"],
                                 s["ws"], s["ws_bytes"])
        return {"out": s["out"], "entries": s["entries"]}
    L.lazyattn_decode_mass(pool.handle, batch.c, s["q"], s["k_new"], s["v_new"], s["out"], s["mass"], s["mass_out"], c["decay"],
                           s["ws"], s["ws_bytes"])
    return {"out": s["out"], "entries": s["entries"], "mass": s["mass_out"]}


def _slots(entries, entry):
    """Of each request's table slots: page [R, E], position and whether a token is there [R, E * 16]."""
    e = torch.where(entry >= 0, entries[entry.clamp(min=0)], 0)
    j = torch.arange(PAGE, device=e.device)
    position = ((e >> 32) & ((1 << 26) - 1))[:, :, None] + j
    there = j < ((e >> 58) & 31)[:, :, None]
    return e & 0xFFFFFFFF, position.flatten(1), there.flatten(1)


def _rotate(x, position, s):
    """Rotary encoding of x [R, N, heads, D] at position [R, N], dims paired half with half."""
    position = position.clamp(0, s["cos"].shape[0] - 1)
    cos, sin = s["cos"][position][:, :, None], s["sin"][position][:, :, None]
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_attention(s):
    c, entries = s["case"], s["entries0"]
    hq, hkv, d, R = c["hq"], c["hkv"], c["d"], c["requests"]
    decode = c["op"].startswith("decode")
    if decode:   # append the step's token
        at, slot = s["spot"].T
        page = entries[at] & 0xFFFFFFFF
        s["k"][page, :, slot] = s["k_new"]
        s["v"][page, :, slot] = s["v_new"]
        entries = entries.clone()
        entries[at] += 1 << 58
        q, m = s["q"].float()[:, None], s["m"][:, None]
    else:
        q, m = torch.where((s["row"] >= 0)[:, :, None, None], s["q"].float()[s["row"].clamp(min=0)], 0.0), s["m"]
    page, position, there = _slots(entries, s["entry"])
    rows = q.shape[1]

    k = s["k"][page].float().transpose(2, 3).flatten(1, 2)                      # [R, slots, Hkv, D]
    k = _rotate(k, position, s).transpose(1, 2)
    q = _rotate(q, m, s).unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [R, Hkv, rows * g, D]
    seen = there[:, None] & (position[:, None] <= m[:, :, None])                # [R, rows, slots]
    if c["window"]:
        seen &= (m[:, :, None] - position[:, None] < c["window"]) | (position[:, None] < c["sinks"])
    if not decode:
        seen &= (s["row"] >= 0)[:, :, None]
    seen = seen.repeat_interleave(hq // hkv, 1)[:, None]
    score = (q @ k.transpose(2, 3) / math.sqrt(d)).masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)

    out = {}
    if c["op"] != "prefill_mass":
        o = p @ s["v"][page].float().transpose(2, 3).flatten(1, 2).transpose(1, 2)
        o = o.unflatten(2, (rows, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3).to(s["q"].dtype)
        out["out"] = o[:, 0] if decode else o[s["row"] >= 0]
    if decode:
        out["entries"] = entries
    if c["op"].endswith("mass"):
        w = p.sum(2).unflatten(2, (-1, PAGE)).transpose(1, 2)[s["entry"] >= 0]  # [entries, Hkv, 16]
        held = there.unflatten(1, (-1, PAGE))[s["entry"] >= 0][:, None]
        out["mass"] = w if s["mass"] is None else torch.where(held, w + c["decay"] * s["mass"], 0.0)
    return out if decode else out.popitem()[1]


def _plain_evict(s):
    c = s["case"]
    R, hkv, budget = c["requests"], c["hkv"], c["budget"]
    page, position, there = _slots(s["entries0"], s["entry"])
    order = there.cumsum(1) - 1                                                 # the token's number in its request
    count = there.sum(1)
    w = s["mass"][s["entry"].clamp(min=0)].transpose(1, 2).flatten(2)           # [R, Hkv, slots]
    first = there & ((order < c["sinks"]) | (order >= (count - c["recent"])[:, None]))
    w = torch.where(first[:, None], math.inf, w).masked_fill(~there[:, None], -math.inf)
    best = w.sort(dim=2, descending=True, stable=True).indices[:, :, :budget]       # of equal ones the first
    kept = count.clamp(max=budget)
    held = torch.arange(min(budget, best.shape[2]), device=w.device) < kept[:, None]
    best = torch.where(held[:, None], best, w.shape[2]).sort(dim=2).values          # in the table's order
    best = torch.nn.functional.pad(best, (0, _pages(budget) * PAGE - best.shape[2]), value=w.shape[2])
    held = (best < w.shape[2]).transpose(1, 2)                                  # [R, kept slots, Hkv]
    slot = torch.where(held, best.transpose(1, 2), 0)
    r, h = torch.arange(R, device=w.device)[:, None, None], torch.arange(hkv, device=w.device)
    src = page[r, slot // PAGE]

    def pages(x):                                                               # [R * pages, Hkv, 16, ...]
        return x.unflatten(1, (-1, PAGE)).transpose(2, 3).flatten(0, 1)

    k, v = (pages(torch.where(held[..., None], x[src, h, slot % PAGE], 0)) for x in (s["k"], s["v"]))
    s["k"][s["used"]:], s["v"][s["used"]:] = k, v
    j = torch.arange(_pages(budget), device=w.device)
    entries = s["dst0"].unflatten(0, (R, -1)) | (j * PAGE << 32) | ((kept[:, None] - PAGE * j).clamp(0, PAGE) << 58)
    return {"kept": torch.where(held, position[r, slot], -1).transpose(1, 2)[:, :, :budget].to(torch.int32).contiguous(), "entries": entries.flatten(),
            "mass": pages(torch.where(held, s["mass"][s["entry"][r, slot // PAGE].clamp(min=0), h, slot % PAGE], 0.0)),
            "k": s["k"][s["used"]:], "v": s["v"][s["used"]:]}


# ------------------------------------------------------------------------------------------------ in 64 bits

def _rope64(x, position):
    """x [N, heads, D] in 64 bits as complex pairs (i, i + D/2), turned by position * theta^(-2i/D)."""
    half = x.shape[-1] // 2
    turn = torch.pow(torch.tensor(THETA, dtype=torch.float64, device=x.device), -torch.arange(half, dtype=torch.float64, device=x.device) / half)
    z = torch.complex(x[..., :half], x[..., half:]) * torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                                                                  position.double()[:, None] * turn)[:, None]
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g, decode = hq // hkv, case["op"].startswith("decode")
    table, _ = _table(case)
    dev = s["k"].device
    outs, mass = [], torch.zeros(len(s["entries0"]), hkv, PAGE, dtype=torch.float64, device=dev)
    row0 = 0
    for r, segments in enumerate(table):
        # the request's tokens in order: their pages, slots and entries
        place, e = [], int(s["offsets"][r])
        for first, at, n, pages, w in segments:
            place += [(first + j // PAGE, j % PAGE, e + j // PAGE) for j in range(n + (decode and w))]
            e += pages
        page, slot, entry = torch.tensor(place, device=dev).T
        k, v = s["k"][page, :, slot].double(), s["v"][page, :, slot].double()   # [N, Hkv, D]
        n = len(place)
        if decode:
            k[-1], v[-1] = s["k_new"][r].double(), s["v_new"][r].double()
            q = s["q"][r:r + 1].double()
        else:
            q = s["q"][row0:row0 + s["rows"][r]].double()
            row0 += len(q)
        where = torch.arange(n, device=dev)
        m = where[n - len(q):]
        k, q = _rope64(k, where), _rope64(q, m)
        hidden = where[None] > m[:, None]
        if case["window"]:
            hidden |= (where[None] <= m[:, None] - case["window"]) & (where[None] >= case["sinks"])
        o = torch.empty(len(q), hq, d, dtype=torch.float64, device=dev)
        for h in range(hq):
            a = torch.softmax((q[:, h] @ k[:, h // g].T / d ** 0.5).masked_fill(hidden, float("-inf")), -1)
            o[:, h] = a @ v[:, h // g]
            mass[entry, h // g, slot] += a.sum(0)
        if case["op"].endswith("mass") and s["mass"] is not None:
            mass[entry, :, slot] += case["decay"] * s["mass"][entry, :, slot].double()
        outs.append(o)
    out = torch.cat(outs)
    if case["op"] == "prefill_mass":
        return mass
    if not decode:
        return out
    got = {"out": out, "entries": None}
    if case["op"] == "decode_mass":
        got["mass"] = mass
    return got


def _exact_evict(s):
    """The kept tokens by sorting (weight, then place) on the host."""
    c = s["case"]
    table, _ = _table(c)
    R, hkv, budget, per = c["requests"], c["hkv"], c["budget"], _pages(c["budget"])
    kept = np.full((R, hkv, budget), -1, np.int32)
    w_all = s["mass"].double().cpu().numpy()
    shape = (R * per, hkv, PAGE)
    mass = np.zeros(shape)
    src = np.full(shape, -1, np.int64)                                          # page * 16 + slot of what goes there
    for r, segments in enumerate(table):
        place, e = [], int(s["offsets"][r])
        for first, at, n, pages, w in segments:
            place += [(first + j // PAGE, j % PAGE, e + j // PAGE, at + j) for j in range(n)]
            e += pages
        place = np.array(place)
        n = len(place)
        for h in range(hkv):
            w = w_all[place[:, 2], h, place[:, 1]]
            free = np.arange(n)[c["sinks"]:max(c["sinks"], n - c["recent"])]
            most = max(0, min(n, budget) - (n - len(free)))
            free = free[np.lexsort((free, -w[free]))][:most]
            ids = np.sort(np.concatenate([np.arange(min(n, c["sinks"])), free, np.arange(max(min(n, c["sinks"]), n - c["recent"]), n)]))
            kept[r, h, :len(ids)] = place[ids, 3]
            j = np.arange(len(ids))
            mass[r * per + j // PAGE, h, j % PAGE] = w[ids]
            src[r * per + j // PAGE, h, j % PAGE] = place[ids, 0] * PAGE + place[ids, 1]
    dev = s["k"].device
    at = torch.from_numpy(src).to(dev)
    h = torch.arange(hkv, device=dev)[:, None]
    k, v = (torch.where((at >= 0)[..., None], x[at.clamp(min=0) // PAGE, h, at.clamp(min=0) % PAGE].double(), 0.0) for x in (s["k"], s["v"]))
    return {"kept": torch.from_numpy(kept), "entries": None, "mass": torch.from_numpy(mass), "k": k, "v": v}
