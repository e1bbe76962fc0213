"""The serving operators around the indexer, as workloads: what is measured and what they compute.

append     cache_append: a step's keys and values rotated and written into the paged cache, its queries rotated
attention  attention: every query over all tokens of its sequence in the paged cache; a prefix that sequences
           share is given once; optionally scores capped by a tanh and a bias that falls with the distance
selected   attention_selected: every query over the tokens that an indexer selected for it

Layout of every case: S sequences with the same number of new tokens (queries) each, at the end of ragged lengths.
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a batch of 16 with two draft tokens each: launch latency
        _case("append_decode_16x3", "append", seqs=16, queries=3, length=2048, q_heads=64, kv_heads=8, dim=128, page=64),
        # the indexer's own keys of a step: one head, no values, no queries, contiguous pages of one token
        _case("append_index_keys_8x1", "append", seqs=8, queries=1, length=4096, q_heads=0, kv_heads=1, dim=128, page=16,
              values=False),
        # a prompt of 32768 tokens in one call: bandwidth
        _case("append_prefill_32768", "append", seqs=1, queries=32768, length=32768, q_heads=32, kv_heads=8, dim=128, page=64),
        # several prompts, small heads, half of each head rotated in neighbouring pairs, pages of an odd size
        _case("append_prefill_7x1001_d64", "append", seqs=7, queries=1001, length=1500, q_heads=24, kv_heads=24, dim=64,
              page=33, half=True, rotated=32, interleaved=True, heads_first=True),
        # one short sequence, one token: launch latency
        _case("decode_1x1000", "attention", seqs=1, queries=1, length=1000, q_heads=16, kv_heads=2, dim=128, page=16, half=True),
        # the decode batch of 16 sequences of 32768 tokens with two draft tokens each
        _case("decode_16x32768", "attention", seqs=16, queries=3, length=32768, q_heads=32, kv_heads=8, dim=128, page=64),
        # 64 conversations over one long document
        _case("shared_64x32768", "attention", seqs=64, queries=1, length=1500, shared=32768, groups=1, q_heads=64, kv_heads=8,
              dim=128, page=64, cap=30.0),
        # a chunk of a prompt behind a long cached part, scores with a distance bias
        _case("chunk_2x1000_of_16384", "attention", seqs=2, queries=1000, length=16384, q_heads=32, kv_heads=4, dim=128, page=128,
              bias=True),
        # the hierarchical decode batch: 8 sequences of 131072 tokens, 2048 selected
        _case("selected_8x131072", "selected", seqs=8, queries=1, length=131072, q_heads=32, kv_heads=2, dim=128, page=64, select=2048),
        # one sequence of 4096 tokens, 64 query positions at its end, 256 selected
        _case("selected_1x64_of_4096", "selected", seqs=1, queries=64, length=4096, q_heads=16, kv_heads=4, dim=64, page=16,
              select=256, half=True, cap=20.0),
        # part of a long prompt, all heads on one key head
        _case("selected_prefill_3000", "selected", seqs=1, queries=3000, length=32768, q_heads=64, kv_heads=1, dim=128, page=64,
              select=2048),
    ]


def _case(name, op, **kw):
    c = dict(op=op, seqs=1, queries=1, length=1, shared=0, groups=0, q_heads=8, kv_heads=1, dim=128, page=64, half=False,
             rotated=-1, interleaved=False, values=True, heads_first=False, cap=0.0, bias=False, select=0)
    c.update(kw)
    if name:
        c["name"] = name
    if c["rotated"] < 0:
        c["rotated"] = c["dim"]
    return c


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "selected"])
    dim, half, page = rng.choice([64, 128, 128]), rng.random() < 0.4, rng.choice([1, 16, 16, 33, 64, 64, 100, 128, 256])
    kv = rng.choice([1, 1, 2, 4, 8])
    q_heads = kv * rng.choice([1, 2, 3, 4, 7, 8, 16])
    more = dict(dim=dim, half=half, page=page, kv_heads=kv, q_heads=q_heads, heads_first=rng.random() < 0.3)
    if op == "append":
        seqs = _log_int(rng, 1, 128)
        if rng.random() < 0.2:
            more.update(q_heads=0, values=False)
        queries = _log_int(rng, 1, max(1, 1500000 // (more["q_heads"] + 2 * kv) // seqs))
        queries = min(queries, 32768 // seqs)
        rotated = rng.choice([0, dim // 2, dim, dim])
        return _case("", op, seqs=seqs, queries=queries, length=queries + _log_int(rng, 1, max(1, 65536 // seqs)) - 1,
                     rotated=rotated, interleaved=rng.random() < 0.5, **more)
    cap, bias = rng.choice([0.0, 0.0, 20.0, 50.0]), rng.random() < 0.3
    if op == "selected":
        seqs = _log_int(rng, 1, 16)
        queries = rng.choice([1, 1, 3, _log_int(rng, 1, max(1, 2048 // seqs))])
        length = max(queries, _log_int(rng, 1, 262144 // seqs))
        select = _log_int(rng, 1, 2048)
        if seqs * queries * select * kv > 3000 * 2048:
            select = max(1, 3000 * 2048 // (seqs * queries * kv))
        return _case("", op, seqs=seqs, queries=queries, length=length, select=select, cap=cap, bias=bias, **more)
    kind = rng.choice(["decode", "decode", "shared", "chunk"])
    if kind == "chunk":
        seqs = rng.choice([1, 1, 2, 3])
        queries = _log_int(rng, 5, 900 // seqs)
        more["q_heads"] = kv * max(1, min(q_heads // kv, 32 // kv))
        return _case("", op, seqs=seqs, queries=queries, length=queries + _log_int(rng, 1, 12000) - 1, cap=cap, bias=bias, **more)
    queries = rng.choice([1, 1, 2, 3])
    if kind == "shared":
        groups = rng.choice([1, 1, 2, 3])
        seqs = groups * _log_int(rng, 1, 64 // groups)
        return _case("", op, seqs=seqs, queries=queries, length=queries + _log_int(rng, 1, 1500) - 1, groups=groups,
                     shared=_log_int(rng, 1, 24000), cap=cap, bias=bias, **more)
    seqs = _log_int(rng, 1, 64)
    return _case("", op, seqs=seqs, queries=queries, length=queries + _log_int(rng, 1, 360000 // seqs) - 1, cap=cap, bias=bias, **more)


# ---------------------------------------------------------------- shapes that follow from a case
def _lengths(case):
    """Tokens of each sequence behind its shared prefix (new tokens included): ragged, between half and all of `length`."""
    n, top = case["queries"], case["length"]
    return [max(n, top - (s * 7919 + 13 * s * s) % (top // 2 + 1)) for s in range(case["seqs"])]


def _prefixes(case):
    """Shared tokens of each group: the later groups share a little less."""
    return [max(1, case["shared"] - g * (case["shared"] // 5)) for g in range(case["groups"])]


def _prefix_of_seq(case):
    if not case["groups"]:
        return [0] * case["seqs"]
    each, p = case["seqs"] // case["groups"], _prefixes(case)
    return [p[s // each] for s in range(case["seqs"])]


def work(case):
    e, d, hq, hk = 2, case["dim"], case["q_heads"], case["kv_heads"]
    n = case["queries"]
    t = case["seqs"] * n
    if case["op"] == "append":
        rows = hq + hk * (2 if case["values"] else 1)
        turned = (hq + hk) * case["rotated"]
        return {"bytes": t * (2 * rows * d * e + 4 * min(case["rotated"], d)) + 4 * t, "flops": 3 * t * turned}
    io = 2 * t * hq * d * e + 4 * t * hq
    row = 2 * hk * d * e
    if case["op"] == "selected":
        pairs = rows = 0
        for length in _lengths(case):
            seen = [min(case["select"], length - n + i + 1) for i in range(n)]
            pairs += sum(seen)
            rows += min(sum(seen), length)
        return {"bytes": io + rows * row + 4 * t * case["select"], "flops": 4 * hq * d * pairs}
    pairs = 0
    for length, p in zip(_lengths(case), _prefix_of_seq(case)):
        pairs += n * p + sum(length - n + i + 1 for i in range(n))
    return {"bytes": io + (sum(_lengths(case)) + sum(_prefixes(case))) * row, "flops": 4 * hq * d * pairs}


# ---------------------------------------------------------------- inputs
def _inputs(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 17)
    dt = torch.float16 if case["half"] else torch.bfloat16
    n, seqs, d, page = case["queries"], case["seqs"], case["dim"], case["page"]
    t = seqs * n

    def normal(*shape, mean=0.0, out=dt):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) + mean).to(out)

    prefix = _prefix_of_seq(case)
    lens = [a + b for a, b in zip(_lengths(case), prefix)]
    pages_of = [-(-x // page) for x in lens]
    s = {"case": case, "lens_list": lens}
    # the page table: pages in no order; the whole pages of a shared prefix are the same for its group
    each = seqs // case["groups"] if case["groups"] else 1
    count, rows = 0, []
    for i in range(seqs):
        lead = i // each * each
        same = prefix[i] // page if case["groups"] and i != lead else 0
        rows.append([*(rows[lead][:same] if same else []), *range(count, count + pages_of[i] - same)])
        count += pages_of[i] - same
    order = torch.randperm(count, generator=g, device=dev).to(torch.int32)
    wide = max(pages_of)
    table = torch.zeros(seqs, wide, dtype=torch.int64)
    for i, r in enumerate(rows):
        table[i, :len(r)] = torch.tensor(r)
    s["table"] = order[table.to(dev)].contiguous()
    shape = (count, case["kv_heads"], page, d) if case["heads_first"] else (count, page, case["kv_heads"], d)
    view = (lambda x: x.transpose(1, 2)) if case["heads_first"] else (lambda x: x)
    s["k"] = view(normal(*shape))
    s["v"] = view(normal(*shape, mean=0.25)) if case["values"] else None
    s["lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
    s["pos"] = (s["lens"][:, None] - n + torch.arange(n, device=dev, dtype=torch.int32)[None]).reshape(-1).contiguous()
    if any(p % page for p in prefix):
        # a prefix that ends inside a page: each sequence keeps a copy of that page's shared tokens
        cut = torch.tensor(prefix, device=dev)
        first = torch.arange(seqs, device=dev) // each * each
        at = torch.arange(page, device=dev)
        here = at[None] < (cut % page)[:, None]
        src, dst = s["table"][first, cut // page].long(), s["table"][torch.arange(seqs, device=dev), cut // page].long()
        for c in (s["k"], s["v"]):
            c[dst] = torch.where(here[:, :, None, None], c[src], c[dst])
    if case["op"] == "append":
        rows = case["q_heads"] + case["kv_heads"] * (2 if case["values"] else 1)
        qkv = normal(t, rows, d)  # the fused projection's output: queries, keys and values side by side
        hq, hk = case["q_heads"], case["kv_heads"]
        s["q"] = qkv[:, :hq] if hq else None
        s["new_k"] = qkv[:, hq:hq + hk]
        s["new_v"] = qkv[:, hq + hk:] if case["values"] else None
        s["q_out"] = torch.zeros(t, hq, d, device=dev, dtype=dt) if hq else None
        s["rope"] = None
        if case["rotated"]:
            r = case["rotated"]
            freq = 10000.0 ** (-torch.arange(0, r, 2, device=dev, dtype=torch.float64) / r)
            angle = torch.arange(max(lens), device=dev, dtype=torch.float64)[:, None] * freq
            s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        return s
    hq = case["q_heads"]
    s["q"] = normal(t, hq, d)
    s["slopes"] = None
    if case["bias"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (i + 1) / hq) for i in range(hq)], device=dev)
    if case["op"] == "selected":
        # distinct tokens spread over the prefix, in no order; a prefix shorter than the selection is taken whole, padded with -1
        k = case["select"]
        j = torch.arange(k, device=dev, dtype=torch.int64)[None]
        seen = (s["pos"].long() + 1)[:, None]
        lo, hi = j * seen // k, (j + 1) * seen // k
        u = torch.rand(t, k, generator=g, device=dev)
        some = lo + (u * (hi - lo)).long().clamp(max=torch.clamp(hi - lo - 1, min=0))
        idx = torch.where(seen > k, some, torch.where(j < seen, j.expand(t, k), torch.full_like(some, -1)))
        s["idx"] = idx[:, torch.randperm(k, generator=g, device=dev)].to(torch.int32).contiguous()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import long_context_sparse_misa_b200 as misa
        n, seqs, hq = case["queries"], case["seqs"], case["q_heads"]
        s["prob"] = misa.Problem(s["lens_list"], [i * n for i in range(seqs + 1)], s["pos"].cpu().numpy(), num_heads=1, block=64)
        s["cache"] = misa.KVCache(s["k"], s["v"], s["table"])
        s["share"] = None
        if case["op"] != "append":
            if case["groups"]:
                each = seqs // case["groups"]
                s["share"] = misa.SharedPrefix([i * each for i in range(case["groups"] + 1)], _prefixes(case))
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:2], device="cuda", dtype=torch.float32)
            size = misa.attention_workspace_size(s["prob"], s["cache"], hq, k=case["select"], share=s["share"])
            s["ws"] = torch.empty(size, device="cuda", dtype=torch.uint8)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attention": _own_attention, "selected": _own_selected}[op](state)
    return {"append": _append, "attention": _attention, "selected": _selected}[op](state)


# ---------------------------------------------------------------- the framework's operators
def _own_append(s):
    import long_context_sparse_misa_b200 as misa
    misa.cache_append(s["prob"], s["cache"], s["new_k"], s["new_v"], q=s["q"], q_out=s["q_out"], rope=s["rope"],
                      interleaved=s["case"]["interleaved"])
    return [x for x in (s["k"], s["v"], s["q_out"]) if x is not None]


def _own_attention(s):
    import long_context_sparse_misa_b200 as misa
    misa.attention(s["prob"], s["cache"], s["q"], s["out"], s["ws"], lse=s["lse"], softcap=s["case"]["cap"], slopes=s["slopes"],
                   share=s["share"])
    return s["out"], s["lse"]


def _own_selected(s):
    import long_context_sparse_misa_b200 as misa
    misa.attention_selected(s["prob"], s["cache"], s["q"], s["idx"], s["out"], s["ws"], lse=s["lse"], softcap=s["case"]["cap"],
                            slopes=s["slopes"])
    return s["out"], s["lse"]


# ---------------------------------------------------------------- plain forms
def _turn(x, rope, pos, interleaved):
    if rope is None:
        return x
    r = rope.shape[1]
    row = rope[pos.long()][:, None]
    c, sn = row[..., :r // 2], row[..., r // 2:]
    f = x[..., :r].float()
    if interleaved:
        a, b = f[..., 0::2], f[..., 1::2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = f[..., :r // 2], f[..., r // 2:]
        y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([y.to(x.dtype), x[..., r:]], -1)


def _append(s):
    case, page = s["case"], s["case"]["page"]
    pos = s["pos"].long()
    seq = torch.arange(case["seqs"], device=pos.device).repeat_interleave(case["queries"])
    at, off = s["table"][seq, pos // page].long(), pos % page
    s["k"][at, off] = _turn(s["new_k"], s["rope"], pos, case["interleaved"])
    if s["v"] is not None:
        s["v"][at, off] = s["new_v"]
    if s["q"] is not None:
        s["q_out"].copy_(_turn(s["q"], s["rope"], pos, case["interleaved"]))
    return [x for x in (s["k"], s["v"], s["q_out"]) if x is not None]


def _changed(x, far, s):
    """Scaled products [seqs or queries, kv heads, rows, keys] with the cap and the bias; far: distances that broadcast to x."""
    x = x * (1.0 / math.sqrt(s["case"]["dim"]))
    if s["case"]["cap"]:
        x = s["case"]["cap"] * torch.tanh(x / s["case"]["cap"])
    if s["slopes"] is not None:
        hk = s["case"]["kv_heads"]
        x = x - s["slopes"].view(1, hk, 1, -1, 1) * far
    return x


def _pick(cache, table, at):
    """Rows of positions at [b, l] by the table's rows [b] as [b, kv heads, l, dim] in 32 bits; positions past a sequence are clamped."""
    page = cache.shape[1]
    return cache[table.gather(1, (at // page).clamp(max=table.shape[1] - 1)).long(), at % page].transpose(1, 2).float()


def _attention(s):
    case, dev = s["case"], s["q"].device
    seqs, n, hk, d = case["seqs"], case["queries"], case["kv_heads"], case["dim"]
    grp = case["q_heads"] // hk
    groups, each = max(1, case["groups"]), seqs // max(1, case["groups"])
    q = s["q"].view(seqs, n, hk, grp, d).permute(0, 2, 1, 3, 4).float()
    start = torch.tensor(_prefix_of_seq(case), device=dev)
    pos = s["pos"].view(seqs, 1, n, 1, 1).long()
    lanes = max(_lengths(case))
    at = start[:, None] + torch.arange(lanes, device=dev)
    k, v = _pick(s["k"], s["table"], at), _pick(s["v"], s["table"], at)
    where = at.view(seqs, 1, 1, 1, lanes)
    x = torch.matmul(q.reshape(seqs, hk, n * grp, d), k.transpose(2, 3)).view(seqs, hk, n, grp, lanes)
    x = _changed(x, (pos - where).float(), s).masked_fill(where > pos, -math.inf)
    if case["groups"]:
        lead, most = torch.arange(groups, device=dev) * each, max(_prefixes(case))
        there = torch.arange(most, device=dev)[None].expand(groups, most)
        kp, vp = _pick(s["k"], s["table"][lead], there), _pick(s["v"], s["table"][lead], there)
        qp = q.view(groups, each, hk, n * grp, d).transpose(1, 2).reshape(groups, hk, each * n * grp, d)
        y = torch.matmul(qp, kp.transpose(2, 3)).view(groups, hk, each, n, grp, most).transpose(1, 2).reshape(seqs, hk, n, grp, most)
        w = torch.arange(most, device=dev)
        y = _changed(y, (pos - w).float(), s).masked_fill(w >= start.view(seqs, 1, 1, 1, 1), -math.inf)
        x = torch.cat([y, x], -1)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p[..., p.shape[-1] - lanes:].reshape(seqs, hk, n * grp, lanes), v)
    if case["groups"]:
        pp = p[..., :most].reshape(groups, each, hk, n * grp, most).transpose(1, 2).reshape(groups, hk, each * n * grp, most)
        o = o + torch.matmul(pp, vp).view(groups, hk, each, n * grp, d).transpose(1, 2).reshape(seqs, hk, n * grp, d)
    o = o.view(seqs, hk, n, grp, d) / total
    lse = (top + torch.log(total))[..., 0]
    return (o.permute(0, 2, 1, 3, 4).reshape(seqs * n, hk * grp, d).to(s["q"].dtype), lse.permute(0, 2, 1, 3).reshape(seqs * n, hk * grp))


def _selected(s):
    case = s["case"]
    hk, d, t = case["kv_heads"], case["dim"], s["q"].shape[0]
    grp = case["q_heads"] // hk
    idx = s["idx"].long()
    table = s["table"].repeat_interleave(case["queries"], 0)
    k, v = _pick(s["k"], table, idx.clamp(min=0)), _pick(s["v"], table, idx.clamp(min=0))
    x = torch.matmul(s["q"].view(t, hk, grp, d).float(), k.transpose(2, 3))[:, :, None]
    far = (s["pos"].long()[:, None] - idx).float().view(t, 1, 1, 1, -1)
    x = _changed(x, far, s)[:, :, 0].masked_fill((idx < 0)[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / total
    return o.reshape(t, hk * grp, d).to(s["q"].dtype), (top + torch.log(total)).reshape(t, hk * grp)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "selected": _exact_selected}[case["op"]](s)


def _exact_append(s):
    case, n, page = s["case"], s["case"]["queries"], s["case"]["page"]
    length = torch.tensor(s["lens_list"], device="cuda")
    p = (length[:, None] - n + torch.arange(n, device="cuda")).reshape(-1)
    row = torch.arange(case["seqs"], device="cuda")[:, None].expand(-1, n).reshape(-1)
    slot = s["table"].long()[row, torch.div(p, page, rounding_mode="floor")] * page + p % page

    def turned(x):
        x = x.double().clone()
        r = case["rotated"]
        if not r:
            return x
        c, sn = s["rope"].double()[p, None, :r // 2], s["rope"].double()[p, None, r // 2:]
        first = slice(0, r, 2) if case["interleaved"] else slice(0, r // 2)
        second = slice(1, r, 2) if case["interleaved"] else slice(r // 2, r)
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(c, sn)
        x[..., first], x[..., second] = z.real, z.imag
        return x

    def written(cache, new):
        flat = cache.double().reshape(-1, case["kv_heads"], case["dim"])
        flat[slot] = new
        return flat.view(cache.shape)

    out = [written(s["k"], turned(s["new_k"]))]
    if s["v"] is not None:
        out.append(written(s["v"], s["new_v"].double()))
    if s["q"] is not None:
        out.append(turned(s["q"]))
    return out


def _exact_rows(s, q, k, v, far, visible):
    """softmax attention of q [r, grp, d] of one kv head over k, v [r or 1, l, d]; far and visible [r, l]; slopes of these heads."""
    cap = s["case"]["cap"]
    x = torch.einsum("rgd,rld->rgl", q, k.expand(q.shape[0], -1, -1)) if k.shape[0] > 1 else torch.einsum("rgd,ld->rgl", q, k[0])
    x = x / math.sqrt(s["case"]["dim"])
    if cap:
        x = torch.tanh(x / cap) * cap
    if s["slope"] is not None:
        x = x - s["slope"].double()[None, :, None] * far[:, None].double()
    x = torch.where(visible[:, None], x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    o = torch.einsum("rgl,rld->rgd", p, v) if v.shape[0] > 1 else torch.einsum("rgl,ld->rgd", p, v[0])
    return o, lse


def _exact_attention(s):
    case, n, page = s["case"], s["case"]["queries"], s["case"]["page"]
    hk, grp = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["lens_list"]):
        # a sequence's own table names its shared pages too, and its copy of the page in which the prefix ends
        where = torch.arange(length, device="cuda")
        at, off = s["table"][i].long()[where // page], where % page
        rows, here = slice(i * n, i * n + n), s["pos"][i * n:i * n + n].long()
        for h in range(hk):
            k, v = s["k"][at, off, h].double()[None], s["v"][at, off, h].double()[None]
            heads = slice(h * grp, h * grp + grp)
            s["slope"] = s["slopes"][heads] if s["slopes"] is not None else None
            for a in range(0, n, 64):
                b = slice(rows.start + a, min(rows.stop, rows.start + a + 64))
                far = here[a:a + 64, None] - where
                out[b, heads], lse[b, heads] = _exact_rows(s, s["q"][b, heads].double(), k, v, far, far >= 0)
    return out, lse


def _exact_selected(s):
    case, n, page = s["case"], s["case"]["queries"], s["case"]["page"]
    hk, grp, t = case["kv_heads"], case["q_heads"] // case["kv_heads"], s["q"].shape[0]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for a in range(0, t, 128):
        b = slice(a, min(t, a + 128))
        idx = s["idx"][b].long()
        row = torch.arange(b.start, b.stop, device="cuda") // n
        there = idx.clamp(min=0)
        at, off = s["table"].long()[row[:, None], there // page], there % page
        for h in range(hk):
            heads = slice(h * grp, h * grp + grp)
            s["slope"] = s["slopes"][heads] if s["slopes"] is not None else None
            k, v = s["k"][at, off, h].double(), s["v"][at, off, h].double()
            out[b, heads], lse[b, heads] = _exact_rows(s, s["q"][b, heads].double(), k, v, s["pos"][b].long()[:, None] - idx, idx >= 0)
    return out, lse
