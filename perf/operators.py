"""The paged-cache operators as they are measured: cases, inputs, plain forms, exact values.

A paged cache keeps the keys and values of many streams in pages of a few tokens, out of one
pool per layer, K and V each [n_pages, kv_heads, page_tokens, 128] bf16. Row s of `page_table`
names the pages of stream s in logical order, kv_len[s] is its number of cached tokens (the
chunk's own included) and rows [q_start[s], q_start[s + 1]) of the chunk tensors are its new
tokens, the last of the cached ones. The operators:

* write:  a chunk's K and V into the pages;
* attend: softmax(q K^T / sqrt(128)) V of the chunk's rows over the pages (causal by token, or
          the whole chunk visible), with the rows' log-sum-exp where `lse` is set;
* weigh:  attend that also adds to weight[s, h, j] the attention weight that key j of KV head h
          received from the call's rows (keys of the chunk itself start at zero);
* evict:  keep the first `sinks` and last `recent` tokens of every (stream, KV head) and the
          heaviest of the others, `keep` in all, moved to the front in their order.
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)


def _case(name, op, seqs, q_heads, kv_heads, page, q, kv, ragged=True, causal=True, lse=False, keep=0, sinks=0,
          recent=0):
    c = dict(op=op, seqs=seqs, q_heads=q_heads, kv_heads=kv_heads, page=page, q=q, kv=kv, ragged=ragged,
             causal=causal, lse=lse, keep=keep, sinks=sinks, recent=recent)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of each of 64 streams goes into the cache: a decode step's smallest launch
        _case("write-tokens", "write", 64, 8, 8, 16, 1, 2048),
        # a 480P video chunk (3 frames of 1560 tokens, 40 heads): the clean write-back
        _case("write-chunk", "write", 1, 40, 40, 64, 4680, 28080, ragged=False),
        # one stream, one token, a few thousand cached: latency
        _case("attend-token", "attend", 1, 32, 8, 16, 1, 4097, ragged=False, lse=True),
        # a serving batch: one token each of streams from a few to 16 thousand tokens
        _case("attend-tokens", "attend", 48, 32, 8, 16, 1, 16384),
        # one token against a very long cache: all of the card on one stream
        _case("attend-token-long", "attend", 1, 64, 8, 64, 1, 131071, ragged=False),
        # a few drafted tokens per stream checked at once
        _case("attend-draft", "attend", 16, 32, 4, 32, 7, 8192),
        # a video chunk over its window (3 frames of 880 tokens, 24 heads, 21 frames cached), frames see each other
        _case("attend-frames", "attend", 1, 24, 24, 16, 2640, 18480, ragged=False, causal=False),
        # a chunk of a long prompt on top of what is cached already, causal
        _case("attend-chunk", "attend", 1, 32, 8, 128, 2048, 32768, ragged=False),
        # decode steps of a cache that evicts by weight
        _case("weigh-tokens", "weigh", 24, 32, 8, 16, 1, 8192),
        # prompt chunks of a cache that evicts by weight
        _case("weigh-chunk", "weigh", 4, 32, 8, 32, 512, 8192, lse=True),
        # many streams trimmed to half
        _case("evict-batch", "evict", 16, 8, 8, 16, 0, 8192, keep=4096, sinks=4, recent=256),
        # one long stream trimmed to a quarter
        _case("evict-long", "evict", 1, 8, 8, 64, 0, 65536, ragged=False, keep=16384, sinks=64, recent=2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "attend", "attend", "attend", "weigh", "weigh", "evict"])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 24, 40])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16]) if kv_heads <= 8 else 1
    q_heads = kv_heads * group
    seqs = _log_int(rng, 1, 64)
    ragged = seqs > 1 or rng.random() < 0.5
    if op == "write":
        q = _log_int(rng, 1, max(1, 200000 // (seqs * kv_heads)))
        kv = q + _log_int(rng, 1, 1024)
        return _case(None, op, seqs, q_heads, kv_heads, page, q, kv, ragged)
    if op == "evict":
        kv = _log_int(rng, 64, max(64, min(65536, 1000000 // (seqs * kv_heads))))
        keep = max(16, int(kv * rng.uniform(0.1, 0.95)))
        sinks = rng.randint(0, keep // 4)
        return _case(None, op, seqs, q_heads, kv_heads, page, 0, kv, ragged, keep=keep, sinks=sinks,
                     recent=rng.randint(0, keep // 2))
    # tokens, drafts or chunks; the pairs of row and key stay under the largest listed case's
    q = rng.choice([1, 1, _log_int(rng, 2, 16), _log_int(rng, 17, 2048)])
    kv = _log_int(rng, 16, max(17, min(131072, 4000000 // (seqs * kv_heads), 1000000000 // (seqs * q_heads * q))))
    q = min(q, kv)
    return _case(None, op, seqs, q_heads, kv_heads, page, q, kv, ragged, causal=rng.random() < 0.7,
                 lse=rng.random() < 0.3)


def _lengths(c):
    """Cached tokens and chunk rows of every stream; ragged cases from the longest down to almost nothing."""
    n, kv, q = c["seqs"], c["kv"], c["q"]
    if not c["ragged"]:
        return [kv] * n, [q] * n
    kvs = [max(1, int(kv * (((i * 7) % n + 1) / n) ** 1.5)) for i in range(n)]
    qs = [min(k, max(1 if q else 0, int(q * ((i * 5) % n + 1) / n))) for i, k in enumerate(kvs)]
    return kvs, qs


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, hk, hq, page = c["seqs"], c["kv_heads"], c["q_heads"], c["page"]
    kvs, qs = _lengths(c)
    counts = [-(-k // page) for k in kvs]
    width, total = max(counts), sum(counts)
    rows = sum(qs)
    pages = total + 3  # a few pages of nobody

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    # pages in no order, as a cache that has served for a while hands them out
    ids = torch.randperm(pages, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.zeros((n, width), dtype=torch.int32, device="cuda")
    col = torch.arange(width, device="cuda")
    used = col[None] < torch.tensor(counts, device="cuda")[:, None]
    table[used] = ids
    st = dict(case=dict(c))
    st["k_pages"] = torch.randn((pages, hk, page, D), generator=g, device="cuda", dtype=torch.bfloat16)
    st["v_pages"] = torch.randn((pages, hk, page, D), generator=g, device="cuda", dtype=torch.bfloat16)
    st["table"] = table
    st["kv_len"] = torch.tensor(kvs, dtype=torch.int32, device="cuda")
    starts = [0]
    for x in qs:
        starts.append(starts[-1] + x)
    st["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    st["max_q"], st["max_kv"] = max(qs), max(kvs)
    if c["op"] == "write":
        st["k"] = normal(rows, hk, D).to(torch.bfloat16)
        st["v"] = normal(rows, hk, D).to(torch.bfloat16)
    if c["op"] in ("attend", "weigh"):
        # heads look in directions of their own, and a stream's first tokens lie in them: sinks
        look = normal(hk, D)
        first = st["k_pages"][table[:, 0].long(), :, :4].float() + 0.35 * look[None, :, None]
        st["k_pages"][table[:, 0].long(), :, :4] = first.to(torch.bfloat16)
        q = normal(rows, hq, D) + 0.35 * look.repeat_interleave(hq // hk, 0)[None]
        st["q"] = q.to(torch.bfloat16)
        st["out"] = torch.empty_like(st["q"])
        if c["lse"]:
            st["lse"] = torch.empty((rows, hq), dtype=torch.float32, device="cuda")
    if c["op"] in ("weigh", "evict"):
        # a few tokens gather most of the weight; many of the others exactly none
        u = torch.rand((n, hk, st["max_kv"]), generator=g, device="cuda")
        st["weight"] = torch.where(u < 0.1, torch.zeros_like(u), (-torch.log1p(-u)) ** 3)
    if c["op"] == "evict":
        st["kept"] = torch.empty((n, hk, c["keep"]), dtype=torch.int32, device="cuda")
        st["kv_len_out"] = torch.empty_like(st["kv_len"])
    if own:
        # what a serving program keeps: the layer's pool, the step's batch, a workspace
        import rolling_kv_chunked_b200 as rkv
        st["pool"] = rkv.PagePool(st["k_pages"], st["v_pages"])
        st["batch"] = rkv.PagedBatch(st["table"], st["kv_len"], st["q_start"], st["max_q"], st["max_kv"])
        if c["op"] in ("attend", "weigh"):
            size = rkv.paged_workspace_bytes(st["pool"], st["batch"], rows, hq, weight=c["op"] == "weigh")
            st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return st


def run(state):
    st = state
    c = st["case"]
    if own:
        import rolling_kv_chunked_b200 as rkv
        if c["op"] == "write":
            rkv.paged_write(st["pool"], st["batch"], st["k"], st["v"])
            return [st["k_pages"], st["v_pages"]]
        if c["op"] == "evict":
            rkv.paged_evict(st["pool"], st["batch"], st["weight"], c["keep"], c["sinks"], c["recent"], st["kept"],
                            st["kv_len_out"])
            return [st["k_pages"], st["v_pages"], st["weight"], st["kept"], st["kv_len_out"]]
        rkv.paged_attention(st["pool"], st["batch"], st["q"], st["out"], causal=c["causal"], lse=st.get("lse"),
                            weight=st.get("weight"), workspace=st["workspace"])
        return [st["out"], st.get("lse"), st.get("weight")]
    if c["op"] == "write":
        return _plain_write(st)
    if c["op"] == "evict":
        return _plain_evict(st)
    return _plain_attend(st)


def _rows_of(st):
    """Stream, place in the chunk, cached tokens and chunk length of every chunk row."""
    start, length = st["q_start"].long(), st["kv_len"].long()
    rows = st["k"].shape[0] if "k" in st else st["q"].shape[0]
    i = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(start, i, right=True) - 1
    return seq, i - start[seq], length[seq], (start[1:] - start[:-1])[seq]


def _plain_write(st):
    page = st["case"]["page"]
    seq, i, length, n_q = _rows_of(st)
    pos = length - n_q + i
    ids = st["table"].long()[seq, pos // page]
    st["k_pages"][ids, :, pos % page] = st["k"]
    st["v_pages"][ids, :, pos % page] = st["v"]
    return [st["k_pages"], st["v_pages"]]


def _plain_attend(st):
    c = st["case"]
    n, hk, hq = c["seqs"], c["kv_heads"], c["q_heads"]
    grp, m, t = hq // hk, st["max_q"], st["max_kv"]
    length = st["kv_len"].long()
    n_q = (st["q_start"][1:] - st["q_start"][:-1]).long()

    def cached(pages):  # [n, hk, t, D]
        x = pages[st["table"].long()]
        return x.permute(0, 2, 1, 3, 4).reshape(n, hk, -1, D)[:, :, :t].float()

    seq, i, _, _ = _rows_of(st)
    q = torch.zeros((n, m, hq, D), device="cuda")
    q[seq, i] = st["q"].float()
    q = q.reshape(n, m, hk, grp, D).permute(0, 2, 3, 1, 4).reshape(n, hk, grp * m, D)
    s = (q @ cached(st["k_pages"]).transpose(-1, -2)).mul_(SCALE).reshape(n, hk, grp, m, t)
    j = torch.arange(t, device="cuda")
    r = torch.arange(m, device="cuda")
    last = length[:, None] - 1 + ((r[None] - n_q[:, None] + 1) if c["causal"] else 0 * r[None])  # [n, m]
    seen = (j[None, None] <= last[:, :, None]) & (r[None] < n_q[:, None])[:, :, None]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    s.div_(torch.where(total > 0, total, torch.ones_like(total)))
    o = s.reshape(n, hk, grp * m, t) @ cached(st["v_pages"])
    o = o.reshape(n, hk, grp, m, D).permute(0, 3, 1, 2, 4).reshape(n, m, hq, D)
    st["out"].copy_(o[seq, i])
    if c["lse"]:
        z = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(n, m, hq)
        st["lse"].copy_(z[seq, i])
    if c["op"] == "weigh":
        got = s.sum((2, 3))
        old = (j[None] < (length - n_q)[:, None])[:, None]
        live = ((j[None] < length[:, None]) & (n_q > 0)[:, None])[:, None]
        w = torch.where(old, st["weight"], torch.zeros_like(got)) + got
        st["weight"].copy_(torch.where(live, w, st["weight"]))
    return [st["out"], st.get("lse"), st.get("weight")]


def _plain_evict(st):
    c = st["case"]
    keep, page, w = c["keep"], c["page"], st["weight"]
    t = w.shape[-1]
    length = st["kv_len"].long()
    j = torch.arange(max(t, keep), device="cuda")
    w = torch.nn.functional.pad(w, (0, max(t, keep) - t))
    fixed = (j[None] < c["sinks"]) | (j[None] >= (length - c["recent"])[:, None])
    order = torch.where(fixed[:, None], math.inf, w.double())
    order = torch.where((j[None] < length[:, None])[:, None], order, -math.inf)
    kept = torch.sort(order, dim=-1, descending=True, stable=True)[1][..., :keep].sort(-1)[0]
    there = torch.arange(keep, device="cuda")[None] < length[:, None].clamp(max=keep)  # [n, keep]
    new = torch.where(there[:, None], kept, -1)
    s, h, i = torch.nonzero(new >= 0, as_tuple=True)
    src = kept[s, h, i]
    table = st["table"].long()
    to = (table[s, i // page], h, i % page)
    at = (table[s, src // page], h, src % page)
    for pages in (st["k_pages"], st["v_pages"]):
        pages[to] = pages[at]
    st["weight"][s, h, i] = st["weight"][s, h, src]
    st["kept"].copy_(new)
    st["kv_len_out"].copy_(length.clamp(max=keep))
    return [st["k_pages"], st["v_pages"], st["weight"], st["kept"], st["kv_len_out"]]


def work(case):
    c = case
    hk, hq = c["kv_heads"], c["q_heads"]
    kvs, qs = _lengths(c)
    rows, keys = sum(qs), sum(kvs)
    if c["op"] == "write":
        return {"bytes": rows * hk * D * 2 * 2 * 2, "flops": 0}
    if c["op"] == "evict":
        # of the kept tokens the sinks never move; the weights are read once
        moved = sum(max(0, min(k, c["keep"]) - c["sinks"]) for k in kvs if k > c["keep"])
        return {"bytes": hk * (moved * (D * 2 * 2 * 2 + 4) + keys * 4 + len(kvs) * c["keep"] * 4), "flops": 0}
    pairs = sum(q * k - (q * (q - 1) // 2 if c["causal"] else 0) for q, k in zip(qs, kvs))
    used = sum(k for q, k in zip(qs, kvs) if q > 0)
    b = used * hk * D * 2 * 2 + rows * hq * D * 2 * 2 + (rows * hq * 4 if c["lse"] else 0)
    if c["op"] == "weigh":
        b += used * hk * 4 * 2
    return {"bytes": b, "flops": 4 * D * pairs * hq}


def exact(case, seed):
    """The same outputs from the definitions in 64 bits, stream by stream."""
    st = prepare(case, seed)
    c = st["case"]
    hk, grp, page = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["page"]
    kvs, qs = _lengths(c)
    starts = st["q_start"].tolist()
    if c["op"] == "write":
        kp, vp = st["k_pages"].clone(), st["v_pages"].clone()
        for s, (n, m) in enumerate(zip(kvs, qs)):
            for src, dst in ((st["k"], kp), (st["v"], vp)):
                ids = st["table"][s, :-(-n // page)].long()
                flat = dst[ids].transpose(0, 1).flatten(1, 2)
                flat[:, n - m:n] = src[starts[s]:starts[s + 1]].transpose(0, 1)
                dst[ids] = flat.unflatten(1, (-1, page)).transpose(0, 1)
        return [kp.double(), vp.double()]
    if c["op"] == "evict":
        kp, vp, w = st["k_pages"].clone(), st["v_pages"].clone(), st["weight"].clone()
        kept = torch.full_like(st["kept"], -1)
        for s, n in enumerate(kvs):
            ids = st["table"][s, :-(-n // page)].long()
            fk, fv = kp[ids].transpose(0, 1).flatten(1, 2), vp[ids].transpose(0, 1).flatten(1, 2)
            nk, nv = fk.clone(), fv.clone()
            a, b = min(c["sinks"], n), max(min(c["sinks"], n), n - c["recent"])
            for h in range(hk):
                if n <= c["keep"]:
                    pick = torch.arange(n, device="cuda")
                else:
                    best = torch.argsort(-st["weight"][s, h, a:b].double(), stable=True)[:c["keep"] - a - (n - b)]
                    ends = [torch.arange(a, device="cuda"), torch.arange(b, n, device="cuda")]
                    pick = torch.cat([ends[0], best.sort()[0] + a, ends[1]])
                kept[s, h, :len(pick)] = pick.int()
                nk[h, :len(pick)], nv[h, :len(pick)] = fk[h, pick], fv[h, pick]
                w[s, h, :len(pick)] = st["weight"][s, h, pick]
            kp[ids] = nk.unflatten(1, (-1, page)).transpose(0, 1)
            vp[ids] = nv.unflatten(1, (-1, page)).transpose(0, 1)
        return [kp.double(), vp.double(), w.double(), kept, st["kv_len"].clamp(max=c["keep"])]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    weight = st["weight"].double() if c["op"] == "weigh" else None
    for s, (n, m) in enumerate(zip(kvs, qs)):
        if m == 0:
            continue
        ids = st["table"][s, :-(-n // page)].long()
        kd = st["k_pages"][ids].transpose(0, 1).flatten(1, 2)[:, :n].double()
        vd = st["v_pages"][ids].transpose(0, 1).flatten(1, 2)[:, :n].double()
        if weight is not None:
            weight[s, :, n - m:n] = 0
        hidden = torch.ones((m, n), dtype=torch.bool, device="cuda").triu(n - m + 1) if c["causal"] else None
        for h in range(hk * grp):
            x = st["q"][starts[s]:starts[s + 1], h].double() @ kd[h // grp].T / math.sqrt(D)
            if hidden is not None:
                x = x.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - z[:, None])
            out[starts[s]:starts[s + 1], h] = p @ vd[h // grp]
            lse[starts[s]:starts[s + 1], h] = z
            if weight is not None:
                weight[s, h // grp, :n] += p.sum(0)
    return [out, lse if c["lse"] else None, weight]
