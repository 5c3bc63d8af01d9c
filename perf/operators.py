"""The paged-cache operators and their measured cases.

A paged KV cache holds K and V as [n_pages][kv_heads][page_rows][head_dim];
row r of sequence s sits in page table[s][r // page_rows]. Four operators work
on it, for a batch of sequences with `start[s] .. start[s + 1] - 1` the new
rows of sequence s and length[s] its cached rows, the new ones included:

* append: per-head RMSNorm of q and k, rotation by one or several position
  axes, K and V into the pages.
* attention: the new rows against their sequence's cached rows, with a causal,
  window and prefix mask over the rows' positions, a tanh cap and a distance
  bias.
* key_weight: how much attention each cached row received, per kv head.
* evict: the heaviest `budget` rows of each sequence and kv head are kept.
"""

import math
import random

import torch

own = False

_MUSE = {"nq": 32, "nkv": 8, "hd": 128}
_DSPARK = {"nq": 16, "nkv": 8, "hd": 128}
_TINY = {"nq": 4, "nkv": 2, "hd": 16}
_EPS = 1e-6
_THETA = 1e6


def _case(op, heads, **kw):
    base = {"op": op, "seqs": 1, "rows": 1, "len": 1, "page": 64, "dtype": "bf16", "mix": 0, **heads}
    if op == "append":
        base |= {"axes": 1, "neox": True, "norm": True, "far": 0}
    elif op == "evict":
        base |= {"budget": 1, "recent": 0}
    else:
        base |= {"causal": True, "window": 0, "softcap": 0.0, "bias": False, "prefix": 0, "kept": False}
    assert not set(kw) - set(base) - {"name"}, kw
    return {**base, **kw}


def listed():
    return [
        # one speculative round's verify block of a single request
        _case("append", _MUSE, name="append_block16", rows=16, len=2064),
        # a prompt with images and video: three position axes, adjacent pairs, far into a document
        _case("append", _MUSE, name="append_video_prompt", rows=16384, len=16384, page=128, axes=3, neox=False, far=900000),
        # a batch of verify blocks in full precision
        _case("append", _DSPARK, name="append_batch_f32", seqs=48, rows=9, len=1500, dtype="f32", page=16, mix=3),
        # the verify block of one request in a sliding-window layer: the smallest call, where latency counts
        _case("attention", _MUSE, name="attend_block4_window", rows=4, len=2052, window=2048),
        # a batch of requests that decode one token each, lengths of all kinds, after evictions
        _case("attention", _MUSE, name="attend_decode_batch", seqs=48, rows=1, len=12345, mix=1, kept=True),
        # a chunk of a long prompt
        _case("attention", _MUSE, name="attend_prefill_32k", rows=2048, len=32768, page=128),
        # prompts and verify blocks together: capped scores, distance bias, an always visible prefix, pages of 16 rows
        _case("attention", {"nq": 28, "nkv": 4, "hd": 64}, name="attend_mixed_capped", seqs=9, rows=777, len=5001, page=16, window=1024,
              softcap=20.0, bias=True, prefix=100, mix=5),
        # verify blocks in full precision
        _case("attention", _DSPARK, name="attend_blocks_f32", seqs=8, rows=10, len=4099, dtype="f32", mix=2),
        # the weight that a verify block gives to each cached row
        _case("key_weight", _MUSE, name="weigh_block16", rows=16, len=6000),
        # the last 512 rows of a long prompt, before the first eviction
        _case("key_weight", _MUSE, name="weigh_prompt_32k", rows=512, len=32768, page=128),
        # after each round a few rows go
        _case("evict", _MUSE, name="evict_round", len=2304, budget=2048, recent=128),
        # a batch of prompts brought down to half
        _case("evict", _MUSE, name="evict_prompts", seqs=12, len=32768, budget=16000, recent=1000, page=128, mix=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))


def _ceiling(op):
    works = [work(c) for c in listed() if c["op"] == op]
    return max(w["bytes"] for w in works), max(w["flops"] for w in works)


def draw(rng):
    """Head layouts of this repository's configurations and others, pages of 16 to 256 rows, batches of 1 to 64 sequences
    and lengths of 1 to 32768, at most as much work as the largest listed case of the operator. float32 calls are the batches
    and blocks of requests that the listed ones are."""
    op = rng.choice(["append", "attention", "attention", "key_weight", "evict"])
    top_bytes, top_flops = _ceiling(op)
    while True:
        nkv = rng.choice([1, 2, 4, 8])
        heads = rng.choice([_MUSE, _DSPARK, _TINY, {"nq": nkv * rng.choice([1, 2, 3, 5, 7, 8]), "nkv": nkv, "hd": rng.choice([64, 80, 96, 128])}])
        dtype = "f32" if heads is _TINY or rng.random() < 0.2 else "bf16"
        c = {"seqs": rng.choice([1, 1, _log_int(rng, 2, 64)]), "len": _log_int(rng, 1, 32768), "page": rng.choice([16, 32, 64, 128, 256]),
             "dtype": dtype, "mix": rng.randrange(1000)}
        c["rows"] = min(c["len"], _log_int(rng, 1, 4096 if dtype == "bf16" else 32) if rng.random() < 0.7 else 1)
        if op == "append":
            c |= {"axes": rng.choice([1, 2, 3]), "neox": rng.random() < 0.5, "norm": rng.random() < 0.7, "far": rng.choice([0, _log_int(rng, 1, 1 << 20)])}
            c["rows"] = min(c["len"], c["rows"] * rng.choice([1, 4]))
        elif op == "evict":
            c |= {"budget": rng.randint(max(1, c["len"] // 8), c["len"] + 1), "rows": 1}
            c["recent"] = rng.choice([0, rng.randint(0, c["budget"])])
        else:
            c["kept"] = rng.random() < 0.3
            if not c["kept"]:
                c |= {"causal": rng.random() < 0.8, "window": rng.choice([0, 0, _log_int(rng, 8, 8192)]), "prefix": rng.choice([0, 0, rng.randint(0, min(512, c["len"]))])}
            c |= {"softcap": rng.choice([0.0, 0.0, 20.0, 50.0]), "bias": rng.random() < 0.25}
        c = _case(op, heads, **c)
        w = work(c)
        if w["bytes"] <= top_bytes and w["flops"] <= top_flops and (dtype == "bf16" or w["flops"] < 5e10):
            return c


def _lengths(case):
    """(new rows, cached rows) of each sequence: the case's own for the first, shorter ones of all kinds for the others."""
    r = random.Random(case["mix"])
    got = [(case["rows"], case["len"])]
    for _ in range(case["seqs"] - 1):
        n = case["rows"] if case["rows"] == 1 else r.choice([0, 1, r.randint(1, case["rows"]), r.randint(1, case["rows"])])
        got.append((n, r.randint(max(n, case["len"] // 8, 1), case["len"])))
    return got


def _pairs(case):
    """(visible (query, key) pairs, keys that some query sees), summed over the sequences, for one head."""
    pairs, keys = 0, 0
    w, pre = case["window"], case["prefix"]
    for n, length in _lengths(case):
        if not n:
            continue
        if case["kept"]:
            pairs += n * (length - n) + n * (n + 1) // 2
            keys += length
            continue
        first = length - n
        lo = 0 if w <= 0 else max(0, first - w)
        seen = length if case["causal"] or w <= 0 else min(length, length + w)
        keys += seen - lo + min(lo, pre)
        for i in range(n):
            p = first + i
            a = 0 if w <= 0 else max(0, p - w)
            b = p + 1 if case["causal"] else length if w <= 0 else min(length, p + w + 1)
            pairs += b - a + max(0, min(a, pre)) + max(0, min(length, pre) - b)
    return pairs, keys


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    t = sum(n for n, _ in _lengths(case))
    if case["op"] == "append":
        return {"bytes": t * (2 * (nq + 2 * nkv) * hd * es + nkv * 8 + 4 * (case["axes"] + 1)), "flops": t * (nq + nkv) * hd * 7}
    if case["op"] == "evict":
        moved = read = 0
        for _, n in _lengths(case):
            read += n * nkv * 8 + min(n, case["budget"]) * nkv * 8
            if n > case["budget"]:  # rows beyond the budget are kept as often as others, but for the recent ones, which all are
                late = min(case["recent"], n - case["budget"])
                moved += nkv * (late + (n - case["budget"] - late) * max(0, case["budget"] - case["recent"]) // max(1, n - case["recent"]))
        return {"bytes": read + moved * hd * es * 4, "flops": read}
    pairs, keys = _pairs(case)
    if case["op"] == "attention":
        return {"bytes": keys * nkv * (2 * hd * es + 4) + t * nq * (2 * hd * es + 4), "flops": pairs * nq * (4 * hd + 4)}
    return {"bytes": keys * nkv * (hd * es + 4) + sum(n for _, n in _lengths(case)) * nkv * 8 + t * nq * (hd * es + 4),
            "flops": pairs * nq * (2 * hd + 4)}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    nq, nkv, hd, ps = case["nq"], case["nkv"], case["hd"], case["page"]
    lengths = _lengths(case)
    s, n_max, l_max = len(lengths), max(n for n, _ in lengths), max(l for _, l in lengths)
    t = sum(n for n, _ in lengths)
    width = -(-l_max // ps)
    n_pages = s * width + 3

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dt)

    starts = [0]
    for n, _ in lengths:
        starts.append(starts[-1] + n)
    st = {"op": case["op"], "case": case, "n_max": n_max, "width": width,
          "start": torch.tensor(starts, dtype=torch.int32, device=dev),
          "length": torch.tensor([l for _, l in lengths], dtype=torch.int32, device=dev),
          "table": torch.randperm(n_pages, generator=g, device=dev)[: s * width].reshape(s, width).to(torch.int32),
          "k": normal(n_pages, nkv, ps, hd), "v": normal(n_pages, nkv, ps, hd),
          "weight": torch.zeros(n_pages, nkv, ps, device=dev), "pos": torch.zeros(n_pages, nkv, ps, dtype=torch.int32, device=dev)}
    start, length, table = st["start"].long(), st["length"].long(), st["table"].long()
    token = torch.arange(t, device=dev)
    seq = torch.searchsorted(start[1:], token, right=True)
    slot = length[seq] - (start[seq + 1] - start[seq]) + token - start[seq]
    if case["op"] == "append":
        qkv = normal(t, nq + 2 * nkv, hd)  # one projection's output: q, k and v are slices of its rows
        st |= {"q": qkv[:, :nq], "k_new": qkv[:, nq:nq + nkv], "v_new": qkv[:, nq + nkv:], "row_pos": slot.to(torch.int32),
               "q_out": torch.zeros(t, nq, hd, dtype=dt, device=dev)}
        grid = [slot + case["far"]] if case["axes"] == 1 else [case["far"] + slot // 300, slot % 300 // 20, slot % 20][: case["axes"]]
        st["rope_pos"] = torch.stack(grid).to(torch.int32).contiguous()
        third = max(1, hd // 2 // case["axes"])
        st["pair_axis"] = bytes(min(i // third, case["axes"] - 1) for i in range(hd // 2))
        st["q_norm"], st["k_norm"] = (((1 + 0.1 * torch.randn(hd, generator=g, device=dev)).to(dt), (1 + 0.1 * torch.randn(hd, generator=g, device=dev)).to(dt))
                                      if case["norm"] else (None, None))
        return st
    row = torch.arange(width * ps, device=dev)
    if case["op"] == "evict":
        # weights with a heavy tail, as attention leaves them; some rows got none at all
        w = torch.rand(s, nkv, width * ps, generator=g, device=dev).pow(-1.2) - 1
        w *= torch.rand(s, nkv, width * ps, generator=g, device=dev) > 0.05
        st["next_pos"] = (2 * length).to(torch.int32)
        pos = 2 * row.expand(s, nkv, -1) + torch.randint(0, 2, (s, nkv, width * ps), generator=g, device=dev)
        st |= {"weight_out": torch.zeros_like(st["weight"]), "pos_out": torch.zeros_like(st["pos"]), "length_out": torch.zeros_like(st["length"])}
    else:
        w = torch.rand(s, nkv, width * ps, generator=g, device=dev)
        pos, first = row.expand(s, nkv, -1), 0
        if case["kept"]:  # an evicted cache: gaps, and rows that were moved
            n = (start[1:] - start[:-1])[:, None, None]
            pos = 2 * row + torch.randint(0, 2, (s, nkv, width * ps), generator=g, device=dev)
            moved = (row + 60 * torch.rand(s, nkv, width * ps, generator=g, device=dev)).argsort(-1)
            old = row < length[:, None, None] - n
            moved = torch.where(old, moved.minimum(length[:, None, None] - n - 1), row)
            pos = torch.where(old, pos.gather(-1, moved), row + length[:, None, None])
            first = length[seq]
        st["q_pos"] = (slot + first).to(torch.int32)
        st["q"] = normal(t, nq, hd, scale=1.5)
        st["scale"] = hd ** -0.5
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, nq + 1, device=dev) / nq) if case["bias"] else None
        st["prefix"] = torch.full((s,), case["prefix"], dtype=torch.int32, device=dev) if case["prefix"] else None
        if case["op"] == "attention":
            st |= {"out": torch.zeros(t, nq, hd, dtype=dt, device=dev), "lse": torch.zeros(t, nq, device=dev)}
        else:
            st["weight_out"] = torch.zeros_like(st["weight"])
    st["pos"][table] = pos.to(torch.int32).reshape(s, nkv, width, ps).transpose(1, 2)
    st["weight"][table] = w.reshape(s, nkv, width, ps).transpose(1, 2)
    if case["op"] == "key_weight":
        st["lse"] = _plain_attention(st)[1]
    return st


def _dense(pages, table):
    """[s, kv_heads, rows, ...] of paged rows."""
    x = pages[table.long()].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, *x.shape[4:])


def _owners(st):
    """(sequence, row within its new rows) of each new row."""
    token = torch.arange(st["q"].shape[0], device=st["q"].device)
    start = st["start"].long()
    seq = torch.searchsorted(start[1:], token, right=True)
    return seq, token - start[seq]


def _scores(st):
    """Masked scores [s, kv_heads, group, new rows, cached rows] in fp32; -inf where a row is not seen."""
    case, start, length = st["case"], st["start"].long(), st["length"].long()
    nkv, group, n_max = case["nkv"], case["nq"] // case["nkv"], st["n_max"]
    at = (start[:-1, None] + torch.arange(n_max, device=start.device)).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][at].float().unflatten(2, (nkv, group)).permute(0, 2, 3, 1, 4)  # [s, nkv, group, n, hd]
    k, pos = _dense(st["k"], st["table"]).float(), _dense(st["pos"], st["table"])
    x = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (group, n_max))
    x *= st["scale"]
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    far = st["q_pos"][at][:, None, :, None] - pos[:, :, None, :]  # [s, nkv, n, rows]
    if st["slopes"] is not None:
        x -= st["slopes"].view(nkv, group, 1, 1) * far.abs().float()[:, :, None]
    seen = torch.ones_like(far, dtype=torch.bool)
    if case["causal"]:
        seen &= far >= 0
    if case["window"] > 0:
        seen &= far.abs() <= case["window"]
    if st["prefix"] is not None:
        seen |= (pos < st["prefix"][:, None, None])[:, :, None]
    seen &= (torch.arange(pos.shape[-1], device=pos.device) < length[:, None])[:, None, None]
    seen &= (torch.arange(n_max, device=pos.device) < (start[1:] - start[:-1])[:, None])[:, None, :, None]
    return x.masked_fill_(~seen[:, :, None], -math.inf)


def _plain_attention(st):
    x = _scores(st)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _dense(st["v"], st["table"]).float()
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, p.shape[2:4]) / torch.where(total > 0, total, torch.ones_like(total))
    seq, row = _owners(st)
    out = o.permute(0, 3, 1, 2, 4)[seq, row].flatten(1, 2).to(st["q"].dtype)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2)[seq, row].flatten(1, 2)
    return out, lse


def _plain_append(st):
    case, start, length, table = st["case"], st["start"].long(), st["length"].long(), st["table"].long()
    half = case["hd"] // 2
    axis = torch.tensor(list(st["pair_axis"]), device=table.device)
    freq = _THETA ** (-torch.arange(half, dtype=torch.float64, device=table.device) / half)
    angle = st["rope_pos"][axis].double().T * freq  # [t, half]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, gain):
        x = x.float()
        if gain is not None:
            x = x * (x.square().mean(-1, keepdim=True) + _EPS).rsqrt() * gain.float()
        if case["neox"]:
            a, b = x[..., :half], x[..., half:]
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)

    st["q_out"].copy_(turned(st["q"], st["q_norm"]))
    seq, row = _owners(st)
    slot = length[seq] - (start[seq + 1] - start[seq]) + row
    page, r = table[seq, slot // case["page"]], slot % case["page"]
    st["k"][page, :, r] = turned(st["k_new"], st["k_norm"]).to(st["k"].dtype)
    st["v"][page, :, r] = st["v_new"]
    st["pos"][page, :, r] = st["row_pos"][:, None]
    st["weight"][page, :, r] = 0.0
    return {"q": st["q_out"], "k": st["k"], "v": st["v"], "pos": st["pos"], "weight": st["weight"]}


def _put(pages, table, rows):
    pages[table.long()] = rows.reshape(rows.shape[0], rows.shape[1], table.shape[1], pages.shape[2], *rows.shape[3:]).transpose(1, 2)


def _plain_key_weight(st):
    x = _scores(st)
    start = st["start"].long()
    at = (start[:-1, None] + torch.arange(st["n_max"], device=start.device)).clamp(max=st["q"].shape[0] - 1)
    lse = st["lse"][at].unflatten(2, (x.shape[1], x.shape[2])).permute(0, 2, 3, 1)[..., None]
    got = x.sub_(lse).exp_().sum((2, 3))
    held = torch.arange(got.shape[-1], device=got.device) < st["length"].long()[:, None, None]
    rows = torch.where(held, 0.9 * _dense(st["weight"], st["table"]) + got, _dense(st["weight_out"], st["table"]))
    _put(st["weight_out"], st["table"], rows)
    return st["weight_out"]


def _plain_evict(st):
    case, table, length = st["case"], st["table"], st["length"].long()[:, None, None]
    w, pos = _dense(st["weight"], table), _dense(st["pos"], table)
    row = torch.arange(w.shape[-1], device=w.device).expand_as(w)
    key = torch.where(pos >= st["next_pos"][:, None, None] - case["recent"], torch.full_like(w, math.inf), w)
    key = torch.where(row < length, key, torch.full_like(w, -math.inf))
    order = key.sort(stable=True, dim=-1, descending=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, row)
    kept = (rank < case["budget"]) & (row < length)
    hole = ~kept & (row < length.clamp(max=case["budget"]))
    late = kept & (row >= case["budget"])
    to, of = (~hole).byte().sort(stable=True, dim=-1).indices, (~late).byte().sort(stable=True, dim=-1).indices
    source = row.scatter(-1, to, torch.where(row < hole.sum(-1, keepdim=True), of, to))
    _put(st["k"], table, _dense(st["k"], table).gather(2, source[..., None].expand(-1, -1, -1, case["hd"])))
    _put(st["v"], table, _dense(st["v"], table).gather(2, source[..., None].expand(-1, -1, -1, case["hd"])))
    left = row < length.clamp(max=case["budget"])
    _put(st["weight_out"], table, torch.where(left, w.gather(-1, source), _dense(st["weight_out"], table)))
    _put(st["pos_out"], table, torch.where(left, pos.gather(-1, source), _dense(st["pos_out"], table)))
    st["length_out"].copy_(st["length"].clamp(max=case["budget"]))
    return {"k": st["k"], "v": st["v"], "weight": st["weight_out"], "pos": st["pos_out"], "length": st["length_out"]}


def _cache(st):
    """The program's cache object over the state's tensors, made on the first call."""
    if "cache" not in st:
        from block_speculative_decoding_dflash_gb300 import binding
        st["cache"] = binding.PagedCache(st["k"], st["v"], st["pos"], st["table"], st["length"], weight=st["weight"])
    return st["cache"]


def run(st):
    case, op = st["case"], st["op"]
    if not own:
        if op == "append":
            return _plain_append(st)
        if op == "attention":
            return _plain_attention(st)
        return _plain_key_weight(st) if op == "key_weight" else _plain_evict(st)
    cache = _cache(st)
    if op == "append":
        cache.append(st["q"], st["k_new"], st["v_new"], st["row_pos"], st["start"], st["q_out"], rope_pos=st["rope_pos"], pair_axis=st["pair_axis"],
                     theta=_THETA, neox=case["neox"], q_norm=st["q_norm"], k_norm=st["k_norm"], eps=_EPS)
        return {"q": st["q_out"], "k": st["k"], "v": st["v"], "pos": st["pos"], "weight": st["weight"]}
    if op == "evict":
        cache.evict(case["budget"], case["recent"], st["next_pos"], weight_out=st["weight_out"], pos_out=st["pos_out"], length_out=st["length_out"])
        return {"k": st["k"], "v": st["v"], "weight": st["weight_out"], "pos": st["pos_out"], "length": st["length_out"]}
    mask = {"scale": st["scale"], "causal": case["causal"], "window": case["window"], "softcap": case["softcap"], "slopes": st["slopes"], "prefix": st["prefix"]}
    if op == "attention":
        cache.attention(st["q"], st["q_pos"], st["start"], st["out"], lse=st["lse"], **mask)
        return st["out"], st["lse"]
    cache.key_weight(st["q"], st["q_pos"], st["start"], st["lse"], weight_out=st["weight_out"], decay=0.9, **mask)
    return st["weight_out"]


def exact(case, seed):
    st = prepare(case, seed)
    starts, lengths = st["start"].tolist(), st["length"].tolist()
    ps, nkv, group = case["page"], case["nkv"], case["nq"] // case["nkv"]

    def where(s, rows):
        """(page, row in it) of rows of sequence s."""
        r = torch.as_tensor(rows, device=st["table"].device)
        return st["table"][s].long()[r // ps], r % ps

    if case["op"] == "append":
        half = case["hd"] // 2
        freq = torch.tensor([_THETA ** (-i / half) for i in range(half)], dtype=torch.float64, device=st["k"].device)
        turn = torch.stack([st["rope_pos"][a].double() * freq[i] for i, a in enumerate(st["pair_axis"])], 1)
        turn = torch.polar(torch.ones_like(turn), turn)[:, None]

        def moved(x, gain):
            x = x.double()
            if gain is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS) * gain.double()
            pairs = x.unflatten(-1, (2, half)).transpose(-1, -2) if case["neox"] else x.unflatten(-1, (half, 2))
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            return (z.transpose(-1, -2) if case["neox"] else z).flatten(-2)

        k, v, w, kk = st["k"].double(), st["v"].double(), st["weight"].double(), moved(st["k_new"], st["k_norm"])
        for s, length in enumerate(lengths):
            n = starts[s + 1] - starts[s]
            if n:
                at = where(s, list(range(length - n, length)))
                new = slice(starts[s], starts[s + 1])
                k[at[0], :, at[1]], v[at[0], :, at[1]], w[at[0], :, at[1]] = kk[new], st["v_new"][new].double(), 0.0
        return {"q": moved(st["q"], st["q_norm"]), "k": k, "v": v, "pos": None, "weight": w}
    if case["op"] == "evict":
        k, v, w_out = st["k"].double(), st["v"].double(), st["weight_out"].double()
        budget = case["budget"]
        for s, length in enumerate(lengths):
            page, r = where(s, list(range(length)))
            nxt = int(st["next_pos"][s])
            for h in range(nkv):
                w, pos = st["weight"][page, h, r].tolist(), st["pos"][page, h, r].tolist()
                weigh = [math.inf if p >= nxt - case["recent"] else x for x, p in zip(w, pos)]
                first = sorted(range(length), key=lambda i: (-weigh[i], i))[:budget]
                keep = set(first)
                holes = [i for i in range(min(budget, length)) if i not in keep]
                late = sorted(i for i in first if i >= budget)
                left = min(budget, length)
                w_out[page[:left], h, r[:left]] = torch.tensor(w[:left], dtype=torch.float64, device=page.device)
                if holes:
                    to, of = torch.tensor(holes, device=page.device), torch.tensor(late, device=page.device)
                    for x, y in ((k, st["k"]), (v, st["v"]), (w_out, st["weight"])):
                        x[page[to], h, r[to]] = y[page[of], h, r[of]].double()
        return {"k": k, "v": v, "weight": w_out, "pos": None, "length": None}
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device=st["q"].device)
    w_out = st["weight_out"].double() if case["op"] == "key_weight" else None
    for s, length in enumerate(lengths):
        new = slice(starts[s], starts[s + 1])
        page, r = where(s, list(range(length)))
        for h in range(nkv):
            k, pos, seen = st["k"][page, h, r].double(), st["pos"][page, h, r].long(), None
            mass = torch.zeros(length, dtype=torch.float64, device=page.device)
            if new.stop > new.start:
                far = st["q_pos"][new].long()[:, None] - pos[None]
                hidden = torch.zeros_like(far, dtype=torch.bool)
                if case["causal"]:
                    hidden |= far < 0
                if case["window"] > 0:
                    hidden |= far.abs() > case["window"]
                if case["prefix"]:
                    hidden &= pos[None] >= case["prefix"]
            for j in range(group if new.stop > new.start else 0):
                i = h * group + j
                x = (st["q"][new, i].double() @ k.T) * st["scale"]
                if case["softcap"]:
                    x = torch.tanh(x / case["softcap"]) * case["softcap"]
                if st["slopes"] is not None:
                    x = x - st["slopes"][i].double() * far.abs()
                x[hidden] = -math.inf
                if w_out is None:
                    lse[new, i] = torch.logsumexp(x, -1)
                    p = torch.exp(x - lse[new, i, None])
                    p[hidden] = 0.0
                    out[new, i] = p @ st["v"][page, h, r].double()
                else:
                    mass += torch.exp(x - st["lse"][new, i, None].double()).nan_to_num(0.0).sum(0)
            if w_out is not None:
                w_out[page, h, r] = 0.9 * st["weight"][page, h, r].double() + mass
    return w_out if w_out is not None else (out, lse)
