"""The operators of a verify round over trees of drafted tokens, and their measured cases.

A sequence's new rows are a tree in depth-first order, row 0 the last committed
token: end[j] is one past the last row of row j's subtree (both count from the
sequence's first new row), so that row i descends from row j iff j <= i < end[j].
A chain has end = the number of rows everywhere. `start[s] .. start[s + 1] - 1` are
the new rows of sequence s, which are also the last rows of its paged cache.

* attention: a row sees its sequence's older rows (causal, window and prefix mask
  over positions, a tanh cap, a distance bias) and of the new ones itself and
  those it descends from.
* sample: one token of each row's logits, with temperature, top-k, top-p and
  min-p of the row's own, from a given uniform number.
* accept: the walk from row 0 through the children whose token is the one sampled
  at their parent; the emitted tokens, the kept rows, and the cache's new length.
* commit: K, V, position and weight of the kept rows move to the front of the
  tree's rows, in the caches of all layers.
"""

import math
import random

import torch

own = False

_MUSE = {"nq": 32, "nkv": 8, "hd": 128}
_DSPARK = {"nq": 16, "nkv": 8, "hd": 128}
_TINY = {"nq": 4, "nkv": 2, "hd": 16}


def _case(op, **kw):
    base = {"op": op, "dtype": "bf16", "mix": 0}
    if op == "sample":
        base |= {"rows": 1, "vocab": 1, "kind": "mixed"}
    else:
        base |= {"seqs": 1, "nodes": 1}
    if op == "attention":
        base |= {**_MUSE, "len": 1, "page": 64, "window": 0, "softcap": 0.0, "bias": False, "prefix": 0}
    elif op == "accept":
        base |= {"width": 8}
    elif op == "commit":
        base |= {**_MUSE, "len": 1, "page": 64, "layers": 1, "width": 8}
    assert not set(kw) - set(base) - {"name"}, kw
    return {**base, **kw}


def listed():
    return [
        # the tree of one request in a sliding-window layer: the smallest call, where latency counts
        _case("attention", name="tree_block16_window", nodes=16, len=2064, window=2048),
        # the trees of a batch of requests, lengths and sizes of all kinds
        _case("attention", name="tree_batch", seqs=24, nodes=64, len=12345, mix=1),
        # a large tree after a long prompt
        _case("attention", name="tree_long", nodes=64, len=32768, page=128),
        # trees in full precision, pages of 16 rows
        _case("attention", **_DSPARK, name="tree_blocks_f32", seqs=8, nodes=20, len=4099, dtype="f32", page=16, mix=2),
        # one token of one request, with the usual filters
        _case("sample", name="sample_one", rows=1, vocab=202048, kind="top_k"),
        # every node of one request's tree, nucleus sampling
        _case("sample", name="sample_tree16", rows=16, vocab=202048, kind="top_p"),
        # every node of a batch of trees, each request with parameters of its own
        _case("sample", name="sample_batch", rows=256, vocab=202048, kind="mixed", mix=3),
        # logits in full precision over a vocabulary of an odd size
        _case("sample", name="sample_odd_f32", rows=48, vocab=65537, dtype="f32", kind="mixed", mix=4),
        # the walk of one request
        _case("accept", name="accept_tree16", nodes=16),
        # the walks of a batch
        _case("accept", name="accept_batch", seqs=256, nodes=64, width=16, mix=5),
        # the accepted rows of one request, the layers of a small model
        _case("commit", name="commit_tree16", nodes=16, len=2064, layers=6, mix=4),
        # of a batch, the layers of a larger one
        _case("commit", name="commit_batch", seqs=48, nodes=64, len=300, layers=24, width=16, mix=6),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))


def draw(rng):
    """Trees of 1 to 128 rows, batches of 1 to 48 sequences, lengths of 1 to 32768, vocabularies of 100 to 262144, head layouts
    of this repository's configurations and others; at most as much work as the largest listed case of the operator."""
    op = rng.choice(["attention", "attention", "sample", "sample", "accept", "commit"])
    works = [work(c) for c in listed() if c["op"] == op]
    top_bytes, top_flops = max(w["bytes"] for w in works), max(w["flops"] for w in works)
    while True:
        dtype = "f32" if rng.random() < 0.3 else "bf16"
        nkv = rng.choice([1, 2, 4, 8])
        heads = rng.choice([_MUSE, _DSPARK, _TINY, {"nq": nkv * rng.choice([1, 2, 3, 5, 7, 8]), "nkv": nkv, "hd": rng.choice([64, 80, 96, 128, 256])}])
        c = {"mix": rng.randrange(1000), "dtype": dtype}
        if op == "sample":
            c |= {"rows": _log_int(rng, 1, 512), "vocab": _log_int(rng, 100, 262144), "kind": rng.choice(["top_k", "top_p", "mixed", "mixed"])}
        else:
            c |= {"seqs": rng.choice([1, _log_int(rng, 1, 48)]), "nodes": _log_int(rng, 1, 128)}
        if op == "attention":
            c |= {**heads, "page": rng.choice([16, 32, 64, 128, 256]), "softcap": rng.choice([0.0, 0.0, 0.0, 20.0]), "bias": rng.random() < 0.2}
            c["len"] = max(c["nodes"], _log_int(rng, 1, 32768))
            c |= {"window": rng.choice([0, 0, _log_int(rng, 8, 8192)]), "prefix": rng.choice([0, 0, rng.randint(0, min(512, c["len"]))])}
        elif op == "accept":
            c |= {"seqs": _log_int(rng, 1, 512), "width": rng.choice([4, 8, 16, 32])}
        elif op == "commit":
            c |= {**heads, "page": rng.choice([16, 32, 64, 128, 256]), "layers": _log_int(rng, 1, 32), "width": rng.choice([4, 8, 16, 32])}
            c["len"] = max(c["nodes"], _log_int(rng, 16, 1024))
            if c["seqs"] * c["len"] * c["layers"] * c["nkv"] * c["hd"] > 48 * 300 * 24 * 8 * 128:  # what the caches hold
                continue
        c = _case(op, **c)
        w = work(c)
        if w["bytes"] <= top_bytes and w["flops"] <= top_flops and (dtype == "bf16" or c.get("hd", 0) <= 128 or w["flops"] < 2e10):
            return c


def _trees(case):
    """Of each sequence: (cached rows, tree as a list of ends, depths). The first has the case's own sizes, the others smaller ones
    of all kinds, some without new rows."""
    r = random.Random(case["mix"])
    out = []
    for s in range(case["seqs"]):
        n = case["nodes"] if s == 0 else r.choice([0, 1, r.randint(1, case["nodes"]), case["nodes"], case["nodes"]])
        depth, open_rows, end = [], [], [n] * n
        for i in range(n):
            # a drafted token continues its branch or opens another, more often near the root
            d = 0 if i == 0 else len(open_rows) if r.random() < 0.4 else min(r.randint(1, len(open_rows)) for _ in range(2))
            d = min(d, 16)
            while len(open_rows) > d:
                end[open_rows.pop()] = i
            open_rows.append(i)
            depth.append(d)
        length = case.get("len", n)
        out.append((length if s == 0 else r.randint(max(n, length // 8, 1), max(n, length, 1)), end, depth))
    return out


def _parents(end):
    up = [-1] * len(end)
    for j in range(len(end)):
        for i in range(j + 1, end[j]):
            up[i] = j
    return up


def _paths(case):
    """Accepted rows of each sequence's tree, as a walk of random length gives them, at most `width`."""
    r = random.Random(case["mix"] + 1)
    out = []
    for _, end, _ in _trees(case):
        path, cur = [0] if end else [], 0
        while path and len(path) < case["width"]:
            kids, j = [], cur + 1
            while j < end[cur]:
                kids.append(j)
                j = end[j]
            if not kids or r.random() < 0.1:
                break
            cur = r.choices(kids, [end[j] - j for j in kids])[0]  # what a drafter expands, it believes in
            path.append(cur)
        out.append(path)
    return out


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sample":
        # each logit read once; a comparison and an exponential's worth of arithmetic
        return {"bytes": case["rows"] * (case["vocab"] * es + 28), "flops": case["rows"] * case["vocab"] * 4}
    trees = _trees(case)
    t = sum(len(end) for _, end, _ in trees)
    if case["op"] == "accept":
        return {"bytes": t * 12 + case["seqs"] * (12 + 8 * case["width"]), "flops": t}
    nkv, hd = case["nkv"], case["hd"]
    if case["op"] == "commit":
        moved = sum(r != i for p in _paths(case) for i, r in enumerate(p))
        return {"bytes": 2 * moved * case["layers"] * nkv * (2 * hd * es + 8) + 4 * sum(len(p) for p in _paths(case)), "flops": moved}
    pairs = keys = 0
    for length, end, depth in trees:
        if not end:
            continue
        old = length - len(end)
        first = max(0, old - case["window"]) if case["window"] else 0
        keys += length - first + min(first, case["prefix"])
        for i, d in enumerate(depth):
            lo = max(0, old + d - case["window"]) if case["window"] else 0
            pairs += max(0, old - lo) + min(min(lo, old), case["prefix"]) + min(d, case["window"] or d) + 1
    return {"bytes": keys * nkv * (2 * hd * es + 4) + t * case["nq"] * (2 * hd * es + 4), "flops": pairs * case["nq"] * (4 * hd + 4)}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    st = {"case": case}
    if case["op"] == "sample":
        r, v = case["rows"], case["vocab"]
        x = torch.randn(r, v, generator=g, device=dev) * 3
        # half of the rows know what comes next: a few tokens far above the others
        sure = torch.rand(r, 1, generator=g, device=dev) < 0.5
        likely = torch.randint(0, v, (r, 8), generator=g, device=dev)
        x.scatter_add_(1, likely, torch.rand(r, 8, generator=g, device=dev) * 14 * sure)
        kind = torch.randint(0, 6, (r,), generator=g, device=dev) if case["kind"] == "mixed" else None
        if kind is not None:  # a grammar hides most tokens of some rows
            hidden = (torch.rand(r, v, generator=g, device=dev) < 0.9) & (kind == 5)[:, None]
            hidden[:, :2] = False
            x.masked_fill_(hidden, -math.inf)
        st |= {"logits": x.to(dt), "uniform": torch.rand(r, generator=g, device=dev),
               "token": torch.zeros(r, dtype=torch.int32, device=dev), "prob": torch.zeros(r, device=dev),
               "temperature": None, "top_k": None, "top_p": None, "min_p": None}
        if case["kind"] == "top_k":
            st |= {"temperature": torch.full((r,), 0.8, device=dev), "top_k": torch.full((r,), 64, dtype=torch.int32, device=dev),
                   "top_p": torch.full((r,), 0.95, device=dev)}
        elif case["kind"] == "top_p":
            st |= {"temperature": torch.ones(r, device=dev), "top_p": torch.full((r,), 0.95, device=dev)}
        else:  # greedy, plain, top-k, top-p, min-p and all together
            st |= {"temperature": torch.where(kind == 0, 0.0, 0.6 + 0.8 * torch.rand(r, generator=g, device=dev)),
                   "top_k": torch.where((kind == 2) | (kind == 5), torch.randint(1, 300, (r,), generator=g, device=dev), 0).to(torch.int32),
                   "top_p": torch.where((kind == 3) | (kind == 5), 0.7 + 0.29 * torch.rand(r, generator=g, device=dev), 1.0),
                   "min_p": torch.where((kind == 4) | (kind == 5), 0.02 + 0.1 * torch.rand(r, generator=g, device=dev), 0.0)}
        return st
    trees = _trees(case)
    s = len(trees)
    starts = [0]
    for _, end, _ in trees:
        starts.append(starts[-1] + len(end))
    t = starts[-1]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    st |= {"start": ints(starts), "length": ints([n for n, _, _ in trees]), "end": ints([e for _, end, _ in trees for e in end]).reshape(t)}
    if case["op"] == "accept":
        # siblings have different tokens; most nodes' sample is one of their children's
        up = [starts[i] + p if p >= 0 else -1 for i, (_, end, _) in enumerate(trees) for p in _parents(end)]
        draft = torch.randint(0, 1 << 14, (t,), generator=g, device=dev) * 256 + torch.arange(t, device=dev) % 256
        parent = torch.tensor(up, dtype=torch.long, device=dev).reshape(t)
        chance = torch.rand(t, generator=g, device=dev)
        sampled = torch.randint(0, 1 << 22, (t,), generator=g, device=dev)
        child = torch.nonzero((parent >= 0) & (chance < 0.8)).flatten()
        best = torch.full((t,), -1.0, device=dev).scatter_reduce_(0, parent[child], chance[child], "amax")
        win = child[best[parent[child]] == chance[child]]
        sampled[parent[win]] = draft[win]
        return st | {"draft": draft.to(torch.int32), "sampled": sampled.to(torch.int32), "n_max": max(len(e) for _, e, _ in trees),
                     "tokens": torch.zeros(s, case["width"], dtype=torch.int32, device=dev), "path": torch.zeros(s, case["width"], dtype=torch.int32, device=dev),
                     "count": torch.zeros(s, dtype=torch.int32, device=dev), "length_out": torch.zeros(s, dtype=torch.int32, device=dev)}
    nq, nkv, hd, ps = case["nq"], case["nkv"], case["hd"], case["page"]
    width = -(-max(n for n, _, _ in trees) // ps)
    n_pages = s * width + 3
    st["table"] = torch.randperm(n_pages, generator=g, device=dev)[: s * width].reshape(s, width).to(torch.int32)
    # a row's position: its place in the text, which in a tree is its depth after the committed rows
    place = torch.arange(width * ps, device=dev).repeat(s, 1)
    for i, (n, end, depth) in enumerate(trees):
        if end:
            place[i, n - len(end):n] = torch.tensor(depth, device=dev) + (n - len(end))
    pos = torch.zeros(n_pages, nkv, ps, dtype=torch.int32, device=dev)
    pos[st["table"].long()] = place.to(torch.int32).reshape(s, width, 1, ps).expand(-1, -1, nkv, -1)

    def pages(*layers):
        return torch.randn(*layers, n_pages, nkv, ps, hd, generator=g, device=dev, dtype=dt)

    if case["op"] == "commit":
        layers, paths = case["layers"], _paths(case)
        path = [p + [-1] * (case["width"] - len(p)) for p in paths]
        st["length"] = ints([n - len(end) + len(p) for (n, end, _), p in zip(trees, paths)])  # as the walk leaves it
        return st | {"k": pages(layers), "v": pages(layers), "pos": pos.repeat(layers, 1, 1, 1), "path": ints(path), "count": ints([len(p) for p in paths]),
                     "weight": torch.rand(layers, *pos.shape, generator=g, device=dev)}
    st |= {"k": pages(), "v": pages(), "pos": pos, "width": width, "n_max": max(len(e) for _, e, _ in trees),
           "q": (torch.randn(t, nq, hd, generator=g, device=dev) * 1.5).to(dt),
           "q_pos": ints([n - len(end) + d for n, end, depth in trees for d in depth]).reshape(t),
           "out": torch.zeros(t, nq, hd, dtype=dt, device=dev), "lse": torch.zeros(t, nq, device=dev), "scale": hd ** -0.5,
           "slopes": torch.exp2(-8.0 * torch.arange(1, nq + 1, device=dev) / nq) if case["bias"] else None,
           "prefix": torch.full((s,), case["prefix"], dtype=torch.int32, device=dev) if case["prefix"] else None}
    return st


def _dense(pages, table):
    """[s, kv_heads, rows, ...] of paged rows."""
    x = pages[table.long()].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, *x.shape[4:])


def _padded(st, x):
    """[s, n_max, ...] of values of the new rows; what lies behind a sequence's rows is anything."""
    start = st["start"].long()
    return x[(start[:-1, None] + torch.arange(st["n_max"], device=start.device)).clamp(max=x.shape[0] - 1)]


def _plain_attention(st):
    case, start, length = st["case"], st["start"].long(), st["length"].long()
    nkv, group, n_max, dev = case["nkv"], case["nq"] // case["nkv"], st["n_max"], start.device
    n = start[1:] - start[:-1]
    k, pos = _dense(st["k"], st["table"]).float(), _dense(st["pos"], st["table"])
    q = _padded(st, st["q"]).float().unflatten(2, (nkv, group)).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (group, n_max))  # [s, nkv, group, n, rows]
    x *= st["scale"]
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    far = _padded(st, st["q_pos"])[:, None, :, None] - pos[:, :, None, :]
    if st["slopes"] is not None:
        x -= st["slopes"].view(nkv, group, 1, 1) * far.abs().float()[:, :, None]
    seen = far >= 0
    if case["window"] > 0:
        seen &= far.abs() <= case["window"]
    if st["prefix"] is not None:
        seen |= (pos < st["prefix"][:, None, None])[:, :, None]
    slot, row = torch.arange(pos.shape[-1], device=dev), torch.arange(n_max, device=dev)
    node = slot - (length - n)[:, None]  # which of the new rows a cached one is; negative: an older one
    end = torch.gather(_padded(st, st["end"]).long(), 1, node.clamp(0, n_max - 1))
    tree = (node[:, None] < 0) | ((node[:, None] <= row[:, None]) & (row[:, None] < end[:, None]))
    tree &= (slot < length[:, None])[:, None] & (row < n[:, None])[..., None]
    seen &= tree[:, None]
    x.masked_fill_(~seen[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _dense(st["v"], st["table"]).float()
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, p.shape[2:4]) / torch.where(total > 0, total, torch.ones_like(total))
    token = torch.arange(st["q"].shape[0], device=dev)
    seq = torch.searchsorted(start[1:], token, right=True)
    out = o.permute(0, 3, 1, 2, 4)[seq, token - start[seq]].flatten(1, 2).to(st["q"].dtype)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2)[seq, token - start[seq]].flatten(1, 2)
    return out, lse


def _plain_sample(st):
    x, u = st["logits"].double(), st["uniform"].double()[:, None]
    x = torch.where(x.isnan(), -math.inf, x)
    rank = torch.arange(x.shape[1], device=x.device)
    order = x.sort(dim=1, descending=True, stable=True).indices
    top = x.gather(1, order[:, :1])
    t = torch.ones_like(top) if st["temperature"] is None else st["temperature"].double()[:, None]
    w = torch.where(x > -math.inf, ((x - top) / torch.where(t > 0, t, 1.0)).exp(), 0.0)  # (values next to a border: 64 bits)
    ranked = w.gather(1, order)
    keep = torch.ones_like(ranked, dtype=torch.bool)
    if st["top_k"] is not None:
        k = st["top_k"][:, None]
        keep &= (rank < k) | (k <= 0)
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        run = (ranked * keep).cumsum(1)
        before = torch.cat([torch.zeros_like(top), run[:, :-1]], 1)
        keep &= (before < p * run[:, -1:]) | (p >= 1)
    if st["min_p"] is not None:
        keep &= ranked >= st["min_p"].double()[:, None].clamp(max=1.0)
    keep &= (t > 0) | (rank == 0)
    keep[:, 0] = True
    kept = torch.zeros_like(w).scatter_(1, order, ranked * keep)
    run = kept.cumsum(1)
    token = torch.searchsorted(run, u * run[:, -1:], right=True).clamp(max=x.shape[1] - 1)
    st["token"].copy_(token[:, 0])
    st["prob"].copy_((kept.gather(1, token) / run[:, -1:])[:, 0])
    return st["token"], st["prob"]


def _plain_accept(st):
    case, start = st["case"], st["start"].long()
    n, n_max, width, dev = start[1:] - start[:-1], st["n_max"], case["width"], start.device
    row = torch.arange(n_max, device=dev)
    end, draft, sampled = _padded(st, st["end"]).long(), _padded(st, st["draft"]), _padded(st, st["sampled"])
    above = (row[:, None] > row) & (row[:, None] < end[:, None])  # [s, i, j]: i descends from j
    parent = torch.where(above, row, -1).amax(2)
    cur, alive = torch.zeros_like(n), n > 0
    count = torch.zeros_like(n)
    st["path"].fill_(-1)
    st["tokens"].fill_(-1)
    for i in range(width):
        said = sampled.gather(1, cur[:, None])
        st["path"][:, i] = torch.where(alive, cur, -1)
        st["tokens"][:, i] = torch.where(alive, said[:, 0], -1)
        count += alive
        match = (parent == cur[:, None]) & (draft == said) & (row < n[:, None])
        alive = alive & match.any(1)
        cur = torch.where(alive, match.byte().argmax(1), cur)
    st["count"].copy_(count)
    st["length_out"].copy_(st["length"].long() - n + count)
    return st["tokens"], st["path"], st["count"], st["length_out"]


def _plain_commit(st):
    case, table, count = st["case"], st["table"].long(), st["count"].long()
    i = torch.arange(case["width"], device=table.device)
    s, i = torch.nonzero(i < count[:, None], as_tuple=True)
    to = (st["length"].long() - count)[s] + i
    of = to - i + st["path"].long()[s, i]
    ps = case["page"]
    to, of = (table[s, to // ps], to % ps), (table[s, of // ps], of % ps)
    for name in ("k", "v", "pos", "weight"):
        x = st[name]
        x[:, to[0], :, to[1]] = x[:, of[0], :, of[1]]
    return {"k": st["k"], "v": st["v"], "pos": st["pos"], "weight": st["weight"]}


def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        return {"attention": _plain_attention, "sample": _plain_sample, "accept": _plain_accept, "commit": _plain_commit}[op](st)
    from block_speculative_decoding_dflash_gb300 import binding
    if op == "sample":
        binding.sample(st["logits"], st["uniform"], st["token"], prob=st["prob"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                       min_p=st["min_p"])
        return st["token"], st["prob"]
    if op == "accept":
        binding.tree_accept(st["end"], st["start"], st["draft"], st["sampled"], st["tokens"], st["path"], st["count"], length=st["length"],
                            length_out=st["length_out"])
        return st["tokens"], st["path"], st["count"], st["length_out"]
    if op == "commit":
        if "caches" not in st:  # the program's cache objects, made on the first call
            st["caches"] = [binding.PagedCache(k, v, pos, st["table"], st["length"], weight=w)
                            for k, v, pos, w in zip(st["k"], st["v"], st["pos"], st["weight"])]
        binding.paged_tree_commit(st["caches"], st["path"], st["count"])
        return {"k": st["k"], "v": st["v"], "pos": st["pos"], "weight": st["weight"]}
    if "cache" not in st:
        st["cache"] = binding.PagedCache(st["k"], st["v"], st["pos"], st["table"], st["length"])
    st["cache"].tree_attention(st["q"], st["q_pos"], st["start"], st["end"], st["out"], lse=st["lse"], scale=st["scale"], window=case["window"],
                               softcap=case["softcap"], slopes=st["slopes"], prefix=st["prefix"], max_len=case["len"])
    return st["out"], st["lse"]


def exact(case, seed):
    if case["op"] == "accept":
        return None  # whole numbers
    st = prepare(case, seed)
    if case["op"] == "sample":
        prob = []
        for r in range(case["rows"]):
            x = st["logits"][r].double()
            x[x.isnan()] = -math.inf
            t, k, p, m = (None if st[n] is None else st[n][r].item() for n in ("temperature", "top_k", "top_p", "min_p"))
            if t is not None and not t > 0:
                prob.append(1.0)
                continue
            share = torch.softmax(x / (1.0 if t is None else t), 0)
            order = torch.argsort(x, descending=True, stable=True)
            if k is not None and 0 < k < len(order):
                order = order[:k]
            if p is not None and p < 1:
                mass = share[order].cumsum(0)
                order = order[: int((mass < p * mass[-1]).sum()) + 1]
            if m is not None and m > 0:
                order = order[: max(1, int((share[order] >= min(m, 1.0) * share[order[0]]).sum()))]
            order = order.sort().values
            mass = share[order].cumsum(0)
            at = int((mass <= st["uniform"][r].item() * mass[-1]).sum())
            prob.append(float(share[order[min(at, len(order) - 1)]] / mass[-1]))
        return None, torch.tensor(prob, dtype=torch.float64, device=st["prob"].device)
    ps, nkv = case["page"], case["nkv"]

    def where(s, rows):
        """(page, row in it) of rows of sequence s."""
        r = torch.as_tensor(rows, dtype=torch.long, device=st["table"].device)
        return st["table"][s].long()[r // ps], r % ps

    if case["op"] == "commit":
        lengths, counts, paths = st["length"].tolist(), st["count"].tolist(), st["path"].tolist()
        got = {name: st[name].double() for name in ("k", "v", "weight")}
        for name, y in got.items():
            for s, (n, c) in enumerate(zip(lengths, counts)):
                for i, j in enumerate(paths[s][:c]):
                    (tp, tr), (fp, fr) = where(s, [n - c + i]), where(s, [n - c + j])
                    y[:, tp, :, tr] = st[name][:, fp, :, fr].double()
        return {"k": got["k"], "v": got["v"], "pos": None, "weight": got["weight"]}
    group = case["nq"] // nkv
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device=st["q"].device)
    first = 0
    for s, (length, end, _) in enumerate(_trees(case)):
        n, up = len(end), _parents(end)
        if not n:
            continue
        new, old = slice(first, first + n), length - n
        first += n
        related = torch.zeros(n, n, dtype=torch.bool)
        for i in range(n):
            j = i
            while j >= 0:
                related[i, j] = True
                j = up[j]
        page, r = where(s, list(range(length)))
        for h in range(nkv):
            far = st["q_pos"][new].long()[:, None] - st["pos"][page, h, r].long()[None]
            hidden = far < 0
            if case["window"] > 0:
                hidden |= far > case["window"]
            if case["prefix"]:
                hidden &= st["pos"][page, h, r][None] >= case["prefix"]
            hidden[:, old:] |= ~related.to(hidden.device)
            k, v = st["k"][page, h, r].double(), st["v"][page, h, r].double()
            for i in range(h * group, (h + 1) * group):
                x = (st["q"][new, i].double() @ k.T) * st["scale"]
                if case["softcap"]:
                    x = torch.tanh(x / case["softcap"]) * case["softcap"]
                if st["slopes"] is not None:
                    x = x - st["slopes"][i].double() * far.abs()
                x[hidden] = -math.inf
                lse[new, i] = torch.logsumexp(x, -1)
                out[new, i] = torch.softmax(x, -1) @ v
    return out, lse
