"""Cases, plain forms and 64-bit definitions of the operators that serve a model around the block,
for timing and comparison:

* ``prompt``  causal attention of packed prompts of different lengths, with grouped heads
* ``tree``    attention of new tokens (one, or a tree of drafted ones) over a paged cache
* ``fork``    sequences of a cache forked, extended by a token each and written
* ``verify``  drafted tokens appended to sequences of a cache, the accepted ones kept

``run`` computes them by elementary torch operations in 32 bits, or with ``own`` through the
library's binding.
"""

import math

import torch

own = False


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one short prompt through the smallest block: 4 heads of 64, its window of 32
        dict(name="prompt tiny", op="prompt", lengths="128", pad=0, q_heads=4, kv_heads=4,
             head_dim=64, window=32, packed=True),
        # four equal prompts, the hidden-2048 block's heads and window
        dict(name="prompt 4x2048 window", op="prompt", lengths="2048,2048,2048,2048", pad=0,
             q_heads=16, kv_heads=16, head_dim=128, window=512, packed=True),
        # a serving batch of ragged prompts in a buffer with room left, shared key heads
        dict(name="prompt ragged 8192", op="prompt",
             lengths="1,517,64,2049,0,130,33,1111,7,1500,260,129,900,1000,395", pad=96, q_heads=32,
             kv_heads=8, head_dim=128, window=0, packed=True),
        # one long document, full causal
        dict(name="prompt 16384", op="prompt", lengths="16384", pad=0, q_heads=32, kv_heads=8,
             head_dim=128, window=0, packed=False),
        # one sequence of a small model, one token: latency
        dict(name="decode 1x500", op="tree", batch=1, length=500, ragged=False, drafts=1, q_heads=4,
             kv_heads=4, head_dim=64, page=16, window=0),
        # a decoding step of a batch of 64 sequences with shared key heads
        dict(name="decode 64x8192", op="tree", batch=64, length=8192, ragged=True, drafts=1,
             q_heads=32, kv_heads=8, head_dim=128, page=64, window=0),
        # one very long sequence
        dict(name="decode 1x131072", op="tree", batch=1, length=131072, ragged=False, drafts=1,
             q_heads=32, kv_heads=8, head_dim=128, page=64, window=0),
        # verification of a tree of 16 drafted tokens for eight sequences
        dict(name="tree 8x16 over 16384", op="tree", batch=8, length=16384, ragged=True, drafts=16,
             q_heads=32, kv_heads=8, head_dim=128, page=64, window=0),
        # odd everything: small trees, a window, pages that end inside tiles
        dict(name="tree odd 3x7", op="tree", batch=3, length=1777, ragged=True, drafts=7, q_heads=20,
             kv_heads=5, head_dim=64, page=24, window=700),
        # one sequence of a one-layer cache: 7 drafts, some kept
        dict(name="verify 1x7", op="verify", batch=1, length=500, drafts=7, layers=1, kv_heads=5,
             head_dim=64, page=24),
        # eight layers, 64 sequences, 16 drafts each
        dict(name="verify 64x16", op="verify", batch=64, length=1024, drafts=16, layers=8,
             kv_heads=8, head_dim=128, page=64),
        # eight prompts of a cache of eight layers, each continued by eight samples
        dict(name="fork 8 to 64", op="fork", batch=8, length=4096, copies=8, layers=8, kv_heads=8,
             head_dim=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "tree", "tree", "tree", "verify", "fork"])
    dh = rng.choice([64, 128, 128])
    kv = _log(rng, 1, 16)
    if op == "prompt":
        group = rng.choice([1, 1, 2, 3, 4, 5, 8])
        window = rng.choice([0, 0, _log(rng, 1, 8192)])
        tokens = _log(rng, 8, 32768)
        # scores of all heads, 16384 x 16384 / 2 x 32 at most
        heads = kv * group
        while heads * tokens * min(tokens, 2 * window or tokens) > 32 * 16384 ** 2:
            tokens = tokens * 2 // 3
        lengths, left = [], tokens
        most = rng.choice([tokens, max(1, tokens // 3), max(1, tokens // 20)])
        while left > 0 and len(lengths) < 100:
            n = min(left, _log(rng, max(1, most // 12), most))
            lengths.append(n)
            left -= n
            if rng.random() < 0.05:
                lengths.append(0)
        return dict(op=op, lengths=",".join(map(str, lengths)), pad=rng.choice([0, 0, 1, 77]),
                    q_heads=heads, kv_heads=kv, head_dim=dh, window=window,
                    packed=rng.random() < 0.5)
    if op == "tree":
        group = rng.choice([1, 2, 4, 4, 5, 8])
        drafts = rng.choice([1, 1, 1, rng.randint(2, 8), rng.randint(9, 32)])
        batch = _log(rng, 1, 128)
        row = batch * kv * dh  # values of one position: 1.1 GB of k and v at most
        length = _log(rng, 16, max(17, min(131072, 268_000_000 // row)))
        return dict(op=op, batch=batch, length=length, ragged=rng.random() < 0.7, drafts=drafts,
                    q_heads=kv * group, kv_heads=kv, head_dim=dh,
                    page=rng.choice([16, 32, 64, 128, rng.randint(1, 100)]),
                    window=rng.choice([0, 0, _log(rng, 1, length)]))
    page, layers, batch = rng.choice([16, 64, rng.randint(8, 100)]), rng.randint(1, 8), _log(rng, 1, 64)
    row = batch * layers * kv * dh  # a pool of 0.5 GB at most
    length = _log(rng, 16, max(17, min(8192, 130_000_000 // row - page - 64)))
    if op == "verify":
        return dict(op=op, batch=batch, length=length, drafts=rng.randint(1, 32), layers=layers,
                    kv_heads=kv, head_dim=dh, page=page)
    return dict(op=op, batch=max(1, batch // 8), length=length, copies=rng.randint(1, 8),
                layers=layers, kv_heads=kv, head_dim=dh, page=page)


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


def _counts(case):
    """New tokens of every sequence of a tree or verify case: up to `drafts`."""
    d = case["drafts"]
    return [d if i % 4 == 0 else max(1, d - i % 3) for i in range(case["batch"])]


def _before(case):
    """Cached tokens of every sequence before the new ones."""
    n = case["length"]
    if not case.get("ragged", True):
        return [n] * case["batch"]
    return [max(0, n - (i * 7919 % 16) * n // 17) for i in range(case["batch"])]


def _pairs(n, window):
    """(query, key) pairs of a causal sequence of n tokens."""
    w = min(window or n, n)
    return w * (w + 1) // 2 + (n - w) * w


def work(case):
    d, kv = case["head_dim"], case["kv_heads"]
    if case["op"] == "prompt":
        ns, h = _lengths(case), case["q_heads"]
        return dict(bytes=2 * d * sum(ns) * (2 * h + 2 * kv) + 4 * (len(ns) + 1),
                    flops=4 * d * h * sum(_pairs(n, case["window"]) for n in ns))
    if case["op"] == "tree":
        cs, bs, h, w = _counts(case), _before(case), case["q_heads"], case["window"]
        seen = [min(b, w - 1) if w else b for b in bs]
        keys = sum(s + c for s, c in zip(seen, cs))
        pages = sum(-(-(b + c) // case["page"]) for b, c in zip(bs, cs))
        return dict(bytes=4 * d * kv * keys + 4 * d * h * sum(cs) + 4 * pages + 4 * sum(cs),
                    flops=4 * d * h * sum(c * (s + (c + 1) // 2) for s, c in zip(seen, cs)))
    token = 2 * 2 * d * kv * case["layers"]  # k and v of one token
    if case["op"] == "verify":
        n = sum(_counts(case))  # written from k and v; about half of them moved
        return dict(bytes=2 * token * n + token * n, flops=n)
    n = case["batch"] * case["copies"]  # a partly filled page copied, one token written, for each
    pages = n * (-(-case["length"] // case["page"]))
    part = sum(b % case["page"] for b in _before(case)) * case["copies"]
    return dict(bytes=2 * token * (part + n) + 4 * 3 * pages, flops=pages)


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return at


def _pool(st, g, lengths, slots, spare, layers, slot_pages):
    """A cache whose first sequences hold `lengths` tokens, their pages in any order."""
    case = st["case"]
    page, kv, d = case["page"], case["kv_heads"], case["head_dim"]
    used = [-(-n // page) for n in lengths]
    pages = sum(used) + spare
    st["k"] = torch.empty(layers, pages, kv, page, d, dtype=torch.bfloat16, device="cuda")
    st["v"] = torch.empty_like(st["k"])
    for t in (st["k"], st["v"]):
        for layer in t:
            layer.copy_(torch.randn(layer.shape, generator=g, device="cuda"))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    st["table"] = torch.full((slots, slot_pages), -1, dtype=torch.int32, device="cuda")
    st["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(used):
        st["table"][i, :n] = order[at:at + n]
        at += n
    st["refs"][order[:at].long()] = 1
    st["lengths"] = _ints(list(lengths) + [0] * (slots - len(lengths)))


def _tokens(st, counts):
    """The new tokens of a call: which listed sequence each belongs to, its index there."""
    st["counts"] = counts
    st["starts"] = _ints(_starts(counts))
    n = torch.tensor(counts, device="cuda")
    st["seq"] = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), n)
    st["index"] = torch.arange(sum(counts), device="cuda") - st["starts"].long()[st["seq"]]


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    d, kv = case["head_dim"], case["kv_heads"]
    if case["op"] == "prompt":
        ns, h = _lengths(case), case["q_heads"]
        t = sum(ns) + case["pad"]
        if case["packed"]:  # columns of one [q | k | v] buffer
            buf = _randn(g, (t, h + 2 * kv, d))
            st["q"], st["k"], st["v"] = buf[:, :h], buf[:, h:h + kv], buf[:, h + kv:]
        else:
            st["q"], st["k"], st["v"] = (_randn(g, (t, n, d)) for n in (h, kv, kv))
        st["out"] = _randn(g, (t, h, d))  # rows behind the last sequence stay as they are
        st["starts"] = _ints(_starts(ns))
        return st
    if case["op"] == "tree":
        counts, before = _counts(case), _before(case)
        lengths = [b + c for b, c in zip(before, counts)]
        most = max(-(-n // case["page"]) for n in lengths)
        _pool(st, g, lengths, case["batch"], 3, 1, most + 2)
        _tokens(st, counts)
        st["slots"] = torch.randperm(case["batch"], generator=g, device="cuda").to(torch.int32)
        # slot order: the listed sequence i is slot slots[i]
        for name in ("table", "lengths"):
            t = st[name].clone()
            t[st["slots"].long()] = st[name]
            st[name] = t
        st["q"] = _randn(g, (sum(counts), case["q_heads"], d))
        # node i hangs below one of the nodes before it, or below the last cached token (-1)
        u = torch.rand(sum(counts), generator=g, device="cuda")
        st["parents"] = (torch.floor(u * (st["index"] + 1)).to(torch.int32) - 1).clamp(max=63) \
            if case["drafts"] > 1 else None
        return st
    page, layers = case["page"], case["layers"]
    before = _before(case)
    if case["op"] == "verify":
        counts = _counts(case)
        slots, spare = case["batch"], sum(-(-c // page) + 1 for c in counts)
        listed_slots = list(range(slots))
        most = max(-(-(b + c) // page) for b, c in zip(before, counts))
    else:
        n = case["batch"] * case["copies"]
        counts, slots, spare = [1] * n, case["batch"] + n, 2 * n + 5
        listed_slots = list(range(case["batch"], slots))
        most = max(-(-(b + 1) // page) for b in before)
        st["from"] = _ints([i // case["copies"] for i in range(n)])
    _pool(st, g, before, slots, spare, layers, most + 1)
    _tokens(st, counts)
    st["slots"] = _ints(listed_slots)
    st["new_k"], st["new_v"] = (_randn(g, (layers, sum(counts), kv, d)) for _ in range(2))
    if case["op"] == "verify":
        st["base"] = _ints(before)
        # each draft is accepted or not; the accepted ones, ascending, lead the list
        yes = torch.rand(sum(counts), generator=g, device="cuda") < 0.5
        key = st["seq"] * 4096 + torch.where(yes, 0, 2048) + st["index"]
        st["path"] = (torch.sort(key).values % 2048).to(torch.int32)
        st["kept"] = torch.zeros(len(counts), dtype=torch.int32, device="cuda").index_add_(
            0, st["seq"], yes.to(torch.int32))
    else:
        st["empty"] = _ints([0] * len(counts))
    return st


# ------------------------------------------------------------------------- plain forms

def _attend(q, k, v, mask):
    """q [heads of k, rows, d], k and v [heads of k, keys, d], mask [rows, keys]."""
    s = torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(q.shape[-1]))
    s = s.masked_fill(~mask, -math.inf)
    e = torch.exp(s - s.amax(-1, keepdim=True))
    return torch.matmul(e, v) / e.sum(-1, keepdim=True)


def _prompt_plain(st):
    case = st["case"]
    kv, d = case["kv_heads"], case["head_dim"]
    group = case["q_heads"] // kv
    at = 0
    for n in _lengths(case):
        w = min(case["window"] or n, n)
        for c in range(0, n, 1024):
            e = min(n, c + 1024)
            lo = max(0, c - w + 1)
            q = st["q"][at + c:at + e].float().view(e - c, kv, group, d).permute(1, 2, 0, 3)
            k, v = (st[x][at + lo:at + e].float().transpose(0, 1) for x in ("k", "v"))
            gap = torch.arange(c, e, device="cuda").view(-1, 1) - torch.arange(
                lo, e, device="cuda")
            mask = ((gap >= 0) & (gap < w)).repeat(group, 1)
            o = _attend(q.reshape(kv, group * (e - c), d), k, v, mask)
            o = o.view(kv, group, e - c, d).permute(2, 0, 1, 3).reshape(e - c, kv * group, d)
            st["out"][at + c:at + e] = o.to(torch.bfloat16)
        at += n
    return st["out"]


def _ancestors(st):
    """[sequences, most, most]: node j is node i or above it; rows behind the last are empty."""
    n, most = len(st["counts"]), max(st["counts"])
    above = torch.zeros(n, most, most, device="cuda")
    if st["parents"] is not None:
        p = st["parents"].long()
        above[st["seq"], st["index"], p.clamp(min=0)] = (p >= 0).float()
    above[st["seq"], st["index"], st["index"]] = 1.0
    steps = 1
    while steps < most:  # paths of up to 2 x steps edges
        above = (torch.matmul(above, above) > 0).float()
        steps *= 2
    return above


def _tree_plain(st):
    case = st["case"]
    kv, d, page = case["kv_heads"], case["head_dim"], case["page"]
    group = case["q_heads"] // kv
    above = _ancestors(st)
    depth = above.sum(-1) - 1
    outs, first = [], 0
    for i, (b, c) in enumerate(zip(_before(case), st["counts"])):
        n = b + c
        row = st["table"].index_select(0, st["slots"][i:i + 1])[0, :-(-n // page)].long()
        k, v = (st[x][0].index_select(0, row).transpose(0, 1).reshape(kv, -1, d)[:, :n].float()
                for x in ("k", "v"))
        at = b + depth[i, :c].view(-1, 1)  # position of every new token
        where = torch.cat([torch.arange(b, device="cuda").float(), b + depth[i, :c]])
        mask = torch.cat([torch.ones(c, b, device="cuda"), above[i, :c, :c]], 1) > 0
        if case["window"]:
            mask = mask & (at - where < case["window"])
        q = st["q"][first:first + c].float().view(c, kv, group, d).permute(1, 2, 0, 3)
        o = _attend(q.reshape(kv, group * c, d), k, v, mask.repeat(group, 1))
        outs.append(o.view(kv, group, c, d).permute(2, 0, 1, 3).reshape(c, kv * group, d))
        first += c
    return torch.cat(outs).to(torch.bfloat16)


def _release(st, slots, old, new):
    """Pages of the listed sequences behind their new lengths lose a user."""
    page = st["case"]["page"]
    col = torch.arange(st["table"].shape[1], device="cuda")
    drop = (col >= -(-new // page).view(-1, 1)) & (col < -(-old // page).view(-1, 1))
    pages = st["table"][slots].long().clamp(min=0)
    st["refs"].scatter_add_(0, pages.view(-1), -drop.view(-1).to(torch.int32))


def _truncate(st, slots, to):
    old = st["lengths"][slots]
    new = torch.minimum(old, to)
    _release(st, slots, old, new)
    st["lengths"][slots] = new


def _fork(st, src, dst):
    page = st["case"]["page"]
    rows, old, n = st["table"][src], st["lengths"][dst], st["lengths"][src]
    used = torch.arange(rows.shape[1], device="cuda") < -(-n // page).view(-1, 1)
    st["refs"].scatter_add_(0, rows.long().clamp(min=0).view(-1), used.view(-1).to(torch.int32))
    _release(st, dst, old, torch.zeros_like(old))
    st["table"][dst] = torch.where(used, rows, st["table"][dst])
    st["lengths"][dst] = n


def _extend(st, slots):
    page = st["case"]["page"]
    n = st["lengths"][slots].long()
    cnt = torch.tensor(st["counts"], device="cuda")
    have, want = -(-n // page), -(-(n + cnt) // page)
    rows = st["table"][slots].long()
    last = (n // page).view(-1, 1)
    old = rows.gather(1, last)
    copy = (n % page != 0) & (cnt > 0) & (st["refs"][old.clamp(min=0)].view(-1) > 1)
    need = want - have + copy
    first = (torch.cumsum(need, 0) - need).view(-1, 1)
    free = torch.argsort((st["refs"] != 0).to(torch.int32), stable=True)
    col = torch.arange(rows.shape[1], device="cuda").view(1, -1)
    fresh = (col >= have.view(-1, 1)) & (col < want.view(-1, 1))
    moved = copy.view(-1, 1) & (col == last)
    rank = torch.where(moved, first, first + copy.view(-1, 1) + col - have.view(-1, 1))
    take = free[rank.clamp(0, free.numel() - 1)]
    new = fresh | moved
    st["table"][slots] = torch.where(new, take, rows).to(torch.int32)
    st["refs"].scatter_add_(0, take.view(-1), new.view(-1).to(torch.int32))
    st["refs"].scatter_add_(0, old.clamp(min=0).view(-1), -copy.to(torch.int32))
    src = old.clamp(min=0).view(-1)
    dst = torch.where(copy, st["table"][slots].gather(1, last).view(-1).long(), src)
    live = torch.arange(page, device="cuda") < (n % page).view(-1, 1)
    for pool in (st["k"], st["v"]):
        for layer in pool:
            layer[dst] = torch.where(live.view(-1, 1, page, 1), layer[src], layer[dst])
    st["lengths"][slots] = (n + cnt).to(torch.int32)


def _places(st, slots, pos):
    page = st["case"]["page"]
    return st["table"][slots[st["seq"]], pos // page].long(), pos % page


def _write(st, slots):
    cnt = torch.tensor(st["counts"], device="cuda")
    pos = (st["lengths"][slots].long() - cnt)[st["seq"]] + st["index"]
    at, row = _places(st, slots, pos)
    for pool, new in ((st["k"], st["new_k"]), (st["v"], st["new_v"])):
        for layer, x in zip(pool, new):
            layer[at, :, row] = x


def _keep(st, slots):
    cnt = torch.tensor(st["counts"], device="cuda")
    old = st["lengths"][slots]
    base = old - cnt
    go = st["index"] < st["kept"][st["seq"]]
    frm = torch.where(go, st["path"].long(), st["index"]) + base[st["seq"]]
    src, src_row = _places(st, slots, frm)
    dst, dst_row = _places(st, slots, base[st["seq"]] + st["index"])
    for pool in (st["k"], st["v"]):
        for layer in pool:
            layer[dst, :, dst_row] = layer[src, :, src_row]
    new = (base + st["kept"]).to(torch.int32)
    _release(st, slots, old, new)
    st["lengths"][slots] = new


def _cache_out(st):
    return {n: st[n] for n in ("k", "v", "table", "lengths", "refs")}


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    if case["op"] == "prompt":
        return _prompt_plain(st)
    if case["op"] == "tree":
        return _tree_plain(st)
    slots = st["slots"].long()
    if case["op"] == "verify":
        _truncate(st, slots, st["base"])  # the last pass's tokens are dropped
        _extend(st, slots)
        _write(st, slots)
        _keep(st, slots)
    else:
        _truncate(st, slots, st["empty"])  # the last pass's samples are freed
        _fork(st, st["from"].long(), slots)
        _extend(st, slots)
        _write(st, slots)
    return _cache_out(st)


# ------------------------------------------------------------------- the library's calls

def _run_own(st):
    from transformer_block_gb300 import pb
    case = st["case"]
    if case["op"] == "prompt":
        if "scratch" not in st:
            st["scratch"] = torch.empty(
                pb.prompt_attention_scratch_bytes(st["q"].shape[0], st["starts"].numel() - 1),
                dtype=torch.uint8, device="cuda")
        return pb.prompt_attention(st["q"], st["k"], st["v"], st["starts"],
                                   window=case["window"] or None, out=st["out"],
                                   scratch=st["scratch"])
    if "cache" not in st:
        st["cache"] = pb.Cache(st["k"], st["v"], st["table"], st["lengths"], st["refs"])
    cache = st["cache"]
    if case["op"] == "tree":
        return cache.attention(st["q"], st["slots"], st["starts"], parents=st["parents"], layer=0,
                               window=case["window"] or None)
    if case["op"] == "verify":
        cache.truncate(st["slots"], st["base"])
        cache.extend(st["slots"], st["starts"])
        cache.write(st["new_k"], st["new_v"], st["slots"], st["starts"])
        cache.keep(st["slots"], st["starts"], st["path"], st["kept"])
    else:
        cache.truncate(st["slots"], st["empty"])
        cache.fork(st["from"], st["slots"])
        cache.extend(st["slots"], st["starts"])
        cache.write(st["new_k"], st["new_v"], st["slots"], st["starts"])
    return _cache_out(st)


# ----------------------------------------------------------------- the definition in 64 bits

def _softmax_mean(q, keys, values, visible):
    """Row r of q [rows, d]: the mean of values [n, d] weighted by exp of its scores."""
    score = torch.einsum("rd,nd->rn", q, keys) * q.shape[-1] ** -0.5
    score = torch.where(visible, score, torch.full_like(score, -math.inf))
    return torch.einsum("rn,nd->rd", torch.exp(
        score - torch.logsumexp(score, 1, keepdim=True)), values)


def exact(case, seed):
    if case["op"] in ("verify", "fork"):
        return None  # whole numbers and copies
    st = prepare(case, seed)
    group = case["q_heads"] // case["kv_heads"]
    if case["op"] == "prompt":
        out = st["out"].double()
        first = 0
        for n in _lengths(case):
            if n == 0:
                continue
            reach = case["window"] or n
            for h in range(case["q_heads"]):
                key = st["k"][first:first + n, h // group].double()
                val = st["v"][first:first + n, h // group].double()
                for top in range(0, n, 2048):
                    end = min(n, top + 2048)
                    low = max(0, top + 1 - reach)
                    i = torch.arange(top, end, device="cuda").unsqueeze(1)
                    j = torch.arange(low, end, device="cuda").unsqueeze(0)
                    out[first + top:first + end, h] = _softmax_mean(
                        st["q"][first + top:first + end, h].double(), key[low:end], val[low:end],
                        (j <= i) & (j > i - reach))
            first += n
        return out
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lengths, table = st["lengths"].tolist(), st["table"].cpu()
    starts = st["starts"].tolist()
    for i, slot in enumerate(st["slots"].tolist()):
        a, z = starts[i], starts[i + 1]
        n = lengths[slot]
        base = n - (z - a)
        parent = [-1] * (z - a) if st["parents"] is None else st["parents"][a:z].tolist()
        pos = torch.arange(n)
        place = (table[slot][pos // case["page"]].long().cuda(), (pos % case["page"]).cuda())
        rows = []
        for node in range(z - a):  # walk to the root
            path, at = [], node
            while at >= 0:
                path.append(at)
                at = parent[at]
            here = base + len(path) - 1
            reach = case["window"] or here + 1
            row = torch.zeros(n, dtype=torch.bool)
            row[max(0, here + 1 - reach):base] = True
            for up, at in enumerate(path):
                row[base + at] = up < reach
            rows.append(row)
        seen = torch.stack(rows).cuda()
        for h in range(case["q_heads"]):
            key, val = (st[x][0][place[0], h // group, place[1]].double() for x in ("k", "v"))
            out[a:z, h] = _softmax_mean(st["q"][a:z, h].double(), key, val, seen)
    return out
