"""Cases of the paged key/value cache of a verify forward: attention of a batch of streams over their pages with
a shared prefix, taking a block in (reserve, append, roll back), forking streams, and compacting the pool.

A cache holds, for every stream, `length` stored tokens in the pages `table[s, :held[s]]`; `refcount[p]` says how
many table entries hold page p (0 = free).  The pools are [layers, 2 (K, V), pages, kv heads, page tokens, head
dim].  The plain forms below are elementary torch operations on those tensors.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # one user's verify block behind a chat of a few thousand tokens: the latency of a single stream
        dict(name="attend one stream", op="attend", S=1, B=8, Hq=56, Hkv=8, D=128, page=64, prefix=0, lo=4093, hi=4093,
             dtype="bf16", ragged=False, tree=False),
        # plain decoding (one position a stream) of a batch without a shared prefix: bound by reading the keys
        dict(name="attend decode batch", op="attend", S=96, B=1, Hq=32, Hkv=8, D=128, page=128, prefix=0, lo=700,
             hi=6000, dtype="bf16", ragged=False, tree=False),
        # a verify batch behind a common system prompt and some turns of each user's own
        dict(name="attend shared prompt", op="attend", S=32, B=8, Hq=56, Hkv=8, D=128, page=64, prefix=8192, lo=150,
             hi=1500, dtype="bf16", ragged=False, tree=False),
        # many users asking about one long document: most of the work is the shared part
        dict(name="attend long document", op="attend", S=64, B=8, Hq=64, Hkv=8, D=128, page=64, prefix=32768, lo=60,
             hi=2000, dtype="bf16", ragged=False, tree=False),
        # narrow heads, small pages, drafts of different lengths that form a tree
        dict(name="attend draft trees", op="attend", S=24, B=11, Hq=32, Hkv=4, D=64, page=16, prefix=2000, lo=1, hi=900,
             dtype="fp16", ragged=True, tree=True),
        # taking a block in: one stream and one layer (the smallest call), ...
        dict(name="advance one stream", op="advance", L=1, S=1, B=8, Hkv=8, D=128, page=64, lo=1000, hi=1000, dtype="bf16"),
        # ... a verify batch over a stack of eight layers, ...
        dict(name="advance verify batch", op="advance", L=8, S=32, B=8, Hkv=8, D=128, page=64, lo=1, hi=2000, dtype="bf16"),
        # ... and the prompts of new streams, written in one long block, with an odd length
        dict(name="advance prompts", op="advance", L=4, S=24, B=1999, Hkv=4, D=64, page=16, lo=0, hi=40, dtype="fp16"),
        # candidates of a few streams are dropped and drawn anew from their parents; the next block follows
        dict(name="fork few", op="fork", L=8, parents=2, kids=3, B=8, Hkv=8, D=128, page=64, lo=700, hi=1500, dtype="bf16"),
        # many candidates of each parent, over deep caches with large pages
        dict(name="fork many", op="fork", L=16, parents=16, kids=7, B=8, Hkv=8, D=128, page=128, lo=500, hi=6000, dtype="bf16"),
        # the pool of a small server after some streams have left
        dict(name="compact small", op="compact", L=2, S=13, Hkv=8, D=128, page=16, lo=1, hi=600, gone=0.4, dtype="bf16"),
        # the pool of a long-running batch, a third of whose streams have left
        dict(name="compact large", op="compact", L=8, S=96, Hkv=8, D=128, page=64, lo=100, hi=3000, gone=0.35, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "advance", "fork", "compact"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "attend":
        S, B = _log(rng, 1, 64), _log(rng, 1, 16)
        prefix = page * (_log(rng, 1, 16000) // page) if rng.random() < 0.6 else 0
        lo = _log(rng, 1, 500)
        return dict(op=op, S=S, B=B, Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv=Hkv, D=D, page=page, prefix=prefix, lo=lo,
                    hi=lo + _log(rng, 1, 3000), dtype=dtype, ragged=rng.random() < 0.5, tree=rng.random() < 0.3)
    if op == "advance":
        lo = _log(rng, 1, 300) - 1
        return dict(op=op, L=rng.randint(1, 8), S=_log(rng, 1, 64), B=_log(rng, 1, 500), Hkv=Hkv, D=D, page=page, lo=lo,
                    hi=lo + _log(rng, 1, 1500), dtype=dtype)
    if op == "fork":
        lo = _log(rng, 1, 500)
        return dict(op=op, L=rng.randint(1, 8), parents=_log(rng, 1, 16), kids=rng.randint(1, 7), B=_log(rng, 1, 40), Hkv=Hkv,
                    D=D, page=page, lo=lo, hi=lo + _log(rng, 1, 3000), dtype=dtype)
    lo = _log(rng, 1, 300)
    return dict(op=op, L=rng.randint(1, 8), S=_log(rng, 2, 96), Hkv=Hkv, D=D, page=page, lo=lo, hi=lo + _log(rng, 1, 2500),
                gone=round(rng.uniform(0.1, 0.7), 2), dtype=dtype)


# ------------------------------------------------------------------------------------------------ inputs


def _ceil(a, b):
    return -(-a // b)


def _lengths(case, n, g):
    """Evenly spread over the case's range, in an order of the seed's: every seed fills as many pages."""
    spread = torch.linspace(case["lo"], case["hi"], n + 2)[1:-1].round().int()
    return spread[torch.randperm(n, generator=g)].tolist()


class _Pages:
    """Page tables as a server makes them: streams take pages from a shuffled list, in turn."""

    def __init__(self, S, MP, P, page, g):
        self.page, self.free = page, torch.randperm(P, generator=g).tolist()
        self.length, self.held = [0] * S, [0] * S
        self.table, self.refcount = [[-1] * MP for _ in range(S)], [0] * P

    def grow(self, s, tokens):
        while self.held[s] < _ceil(tokens, self.page):
            p = self.free.pop()
            self.table[s][self.held[s]] = p
            self.refcount[p] += 1
            self.held[s] += 1
        self.length[s] = tokens

    def share(self, s, src, pages):
        for i in range(pages):
            self.table[s][i] = self.table[src][i]
            self.refcount[self.table[src][i]] += 1
        self.held[s] = pages
        self.length[s] = pages * self.page

    def drop(self, s):
        for i in range(self.held[s]):
            self.refcount[self.table[s][i]] -= 1
            self.table[s][i] = -1
        self.held[s] = self.length[s] = 0

    def tensors(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(length=torch.tensor(self.length, **i32), held=torch.tensor(self.held, **i32),
                    table=torch.tensor(self.table, **i32), refcount=torch.tensor(self.refcount, **i32))


def _pool(case, L, P, seed):
    """Keys with a few strong channels, values with a mean of their own, as projections give them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (L, 2, P, case["Hkv"], case["page"], case["D"])
    x = torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[case["dtype"]])
    x[:, 1] += torch.randn((1, 1, case["Hkv"], 1, case["D"]), generator=g, device="cuda").to(x.dtype)
    x[:, 0, ..., ::17] *= 1.5
    return x


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed + 1)
    op, page = case["op"], case["page"]
    st = dict(op=op, page=page, case=dict(case))
    if op == "attend":
        S, B = case["S"], case["B"]
        own_len, pre = _lengths(case, S, g), case["prefix"]
        npre = pre // page
        MP = npre + _ceil(case["hi"] + B, page)
        P = npre + sum(_ceil(n + B, page) for n in own_len) + 3
        pages = _Pages(S + 1, MP, P, page, g)      # the last stream slot holds the shared prefix alone
        pages.grow(S, pre)
        for s in range(S):
            pages.share(s, S, npre)
            pages.grow(s, pre + own_len[s] + B)     # the block's keys are stored, and not yet committed
            pages.length[s] = pre + own_len[s]
        st["pool"] = _pool(case, 1, P, seed + 2)
        st.update(pages.tensors())
        st["q"] = torch.randn((S, B, case["Hq"], case["D"]), generator=gd, device="cuda", dtype=DTYPES[case["dtype"]]) * 1.3
        st["lengths"] = torch.randint(0 if S > 1 else 1, B + 1, (S,), generator=g).int().cuda() if case["ragged"] else None
        st["mask"] = None
        if case["tree"]:                            # position b sees itself and its ancestors
            rows = []
            for _ in range(S):
                seen = []
                for b in range(B):
                    up = int(torch.randint(-1, b, (1,), generator=g)) if b else -1
                    seen.append((seen[up] if up >= 0 else 0) | (1 << b))
                rows.append(seen)
            st["mask"] = torch.tensor(rows, dtype=torch.int64, device="cuda")
        st["scale"] = 1.0 / math.sqrt(case["D"])
        st["out"] = torch.zeros((S, B, case["Hq"], case["D"]), dtype=st["q"].dtype, device="cuda")
        st["lse"] = torch.zeros((S, B, case["Hq"]), dtype=torch.float32, device="cuda")
    elif op == "advance":
        S, B, L = case["S"], case["B"], case["L"]
        lens = _lengths(case, S, g)
        MP = _ceil(case["hi"] + B, page)
        P = sum(_ceil(n + B, page) for n in lens) + 2
        pages = _Pages(S, MP, P, page, g)
        for s in range(S):
            pages.grow(s, lens[s])
        st["pool"] = _pool(case, L, P, seed + 2)
        st.update(pages.tensors())
        st["new"] = torch.randn((L, 2, S, B, case["Hkv"], case["D"]), generator=gd, device="cuda", dtype=DTYPES[case["dtype"]])
        st["base"] = st["length"].clone()           # the pass starts from these lengths ...
        keep = torch.randint(1, B + 1, (S,), generator=g).int().cuda()
        st["final"] = st["base"] + keep             # ... and keeps so much of the block
    elif op == "fork":
        n, kids, L, B = case["parents"], case["kids"], case["L"], case["B"]
        lens = _lengths(case, n, g)
        S = n * (kids + 1)
        MP = _ceil(case["hi"] + B, page)
        P = sum((kids + 1) * (1 + _ceil(B, page)) + _ceil(m + B, page) for m in lens) + 2
        pages = _Pages(S, MP, P, page, g)
        for s in range(n):
            pages.grow(s, lens[s])
        st["pool"] = _pool(case, L, P, seed + 2)
        st.update(pages.tensors())
        i32 = dict(dtype=torch.int32, device="cuda")
        st["src"] = torch.arange(n, **i32).repeat_interleave(kids)
        st["dst"] = torch.arange(n, S, **i32)[torch.randperm(S - n, generator=g).cuda()]
        st["drop"] = torch.cat([st["length"][:n], torch.zeros(S - n, **i32)])
        st["B"] = B
    else:
        S, L = case["S"], case["L"]
        lens = _lengths(case, S, g)
        MP = _ceil(case["hi"], page)
        P = sum(_ceil(n, page) for n in lens) + 1
        pages = _Pages(S, MP, P, page, g)
        for s in range(S):
            pages.grow(s, lens[s])
        for s in torch.randperm(S, generator=g).tolist()[:max(1, int(S * case["gone"]))]:
            pages.drop(s)
        st["pool"] = _pool(case, L, P, seed + 2)
        st.update(pages.tensors())
        st["was"] = (st["table"].clone(), st["refcount"].clone())
    if own:     # the handle over the same pool, and a state that holds the same tables
        import mxfp4_moe_expert_gb300 as pkg
        c = pkg.KvCache(layers=[(kv[0], kv[1]) for kv in st["pool"]], num_streams=st["table"].shape[0],
                        max_pages=st["table"].shape[1])
        for name, view in (("length", c.length), ("held", c.held), ("table", c.page_table), ("refcount", c.refcount)):
            view.copy_(st[name])
            st[name] = view
        st["cache"] = c
    return st


# ------------------------------------------------------------------------------------------------ plain forms


def _attend(st):
    case, page = st["case"], st["page"]
    S, B, Hq, Hkv, D = (case[n] for n in ("S", "B", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    table = st["table"][:S].long().clamp(min=0)
    kv = st["pool"][0][:, table].float().transpose(3, 2)              # [2, S, Hkv, MP, page, D]
    k, v = kv.reshape(2, S, Hkv, -1, D)
    q = st["q"].float().view(S, B, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, B * G, D)
    s = (q @ k.transpose(-1, -2)).view(S, Hkv, B, G, -1) * st["scale"]
    j = torch.arange(k.shape[2], device="cuda")
    rel = j[None, None, :] - st["length"][:S, None, None]             # key's position in the block
    b = torch.arange(B, device="cuda")
    if st["mask"] is None:
        seen = rel <= b[None, :, None]
    else:
        seen = (rel < 0) | ((rel < B) & ((st["mask"][:, :, None] >> rel.clamp(0, 63)) & 1 > 0))
    s = s.masked_fill(~seen[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    o = (p.view(S, Hkv, B * G, -1) @ v).view(S, Hkv, B, G, D) / torch.where(z == 0, 1.0, z)
    lse = (m + torch.log(z)).squeeze(-1)
    o = o.permute(0, 2, 1, 3, 4).reshape(S, B, Hq, D).to(st["q"].dtype)
    lse = lse.permute(0, 2, 1, 3).reshape(S, B, Hq)
    if st["lengths"] is not None:                                     # unused positions keep what was there
        used = b[None, :] < st["lengths"][:, None]
        o = torch.where(used[:, :, None, None], o, st["out"])
        lse = torch.where(used[:, :, None], lse, st["lse"])
    return o, lse


def _truncate(st, new):
    """Pages behind the new length are given back."""
    table, page = st["table"], st["page"]
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    keep = (new + page - 1) // page
    gone = (j >= keep[:, None]) & (j < st["held"][:, None])
    st["refcount"].scatter_add_(0, table.clamp(min=0).long().view(-1), -gone.int().view(-1))
    table.masked_fill_(gone, -1)
    st["held"].copy_(torch.minimum(st["held"], keep))
    st["length"].copy_(new)


def _reserve(st, n):
    """Room for n more tokens in every stream, lowest free pages first; the tokens of a partly filled page that others
    hold too are copied to a page of the stream's own, unless its writers alone hold it and this is the first of them."""
    table, page, length, held, ref = (st[k] for k in ("table", "page", "length", "held", "refcount"))
    S, MP = table.shape
    j = torch.arange(MP, device="cuda")[None, :]
    s = torch.arange(S, device="cuda")
    last = length // page
    partial = (length % page != 0) & (last < held)
    at = table.gather(1, last.clamp(max=MP - 1).long()[:, None])[:, 0]
    at = torch.where(partial, at, -1 - s.int())
    same = at[:, None] == at[None, :]
    first = same.int().argmax(1) == s
    count = ref[at.clamp(min=0).long()]
    copy = partial & (count > 1) & ~(first & (count == same.sum(1)))
    need = (length + n + page - 1) // page
    fresh = ((j >= held[:, None]) & (j < need[:, None])) | (copy[:, None] & (j == last[:, None]))
    free = torch.argsort((ref > 0).int(), stable=True)
    rank = (fresh.view(-1).cumsum(0) - 1).clamp(0, ref.numel() - 1)
    ids = free[rank].view(S, MP).int()
    src = at[copy].long()
    ref.scatter_add_(0, src, torch.full_like(src, -1).int())
    table.copy_(torch.where(fresh, ids, table))
    ref.scatter_add_(0, table.clamp(min=0).long().view(-1), fresh.int().view(-1))
    held.copy_(torch.maximum(held, need))
    dst = table.gather(1, last.clamp(max=MP - 1).long()[:, None])[:, 0][copy].long()
    filled = torch.arange(page, device="cuda")[None, :] < (length % page)[copy][:, None]
    st["pool"][:, :, dst] = torch.where(filled[:, None, :, None], st["pool"][:, :, src], st["pool"][:, :, dst])


def _append(st):
    new, page = st["new"], st["page"]
    S, B = new.shape[2:4]
    pos = st["length"][:, None] + torch.arange(B, device="cuda")
    at = st["table"].gather(1, (pos // page).long()).long()
    st["pool"][:, :, at, :, (pos % page).long()] = new.permute(2, 3, 0, 1, 4, 5)


def _fork(st):
    src, dst = st["src"].long(), st["dst"].long()
    pages = (st["length"][src] + st["page"] - 1) // st["page"]
    taken = torch.arange(st["table"].shape[1], device="cuda")[None, :] < pages[:, None]
    rows = torch.where(taken, st["table"][src], -1)
    st["table"][dst] = rows
    st["held"][dst] = pages
    st["length"][dst] = st["length"][src]
    st["refcount"].scatter_add_(0, rows.clamp(min=0).long().view(-1), taken.int().view(-1))


def _compact(st):
    ref, table = st["refcount"], st["table"]
    live = ref > 0
    i = torch.arange(ref.numel(), device="cuda")
    n = live.sum()
    src = (live & (i >= n)).nonzero()[:, 0]
    dst = (~live & (i < n)).nonzero()[:, 0]
    st["pool"][:, :, dst] = st["pool"][:, :, src]
    i[src] = dst
    table.copy_(torch.where(table >= 0, i[table.clamp(min=0).long()].int(), table))
    ref[dst] = ref[src]
    ref[src] = 0


def _state(st):
    return [st[n] for n in ("length", "held", "table", "refcount", "pool")]


def run(st):
    op, c = st["op"], st.get("cache")
    if op == "attend":
        if own:
            pre = st["case"]["prefix"]
            return c.attend(0, st["q"], lengths=st["lengths"], mask=st["mask"], shared_stream=st["case"]["S"],
                            shared_tokens=pre, scale=st["scale"], out=st["out"], lse=st["lse"])
        return _attend(st)
    if op == "advance":
        st["length"].copy_(st["base"])
        B = st["new"].shape[3]
        if own:
            c.reserve(B)
            for layer, (k, v) in enumerate(st["new"]):
                c.append(layer, k, v)
            c.truncate(st["final"])
        else:
            _reserve(st, B)
            _append(st)
            _truncate(st, st["final"])
        return _state(st)
    if op == "fork":
        if own:
            c.truncate(st["drop"])
            c.fork(st["src"], st["dst"])
            c.reserve(st["B"])
        else:
            _truncate(st, st["drop"])
            _fork(st)
            _reserve(st, st["B"])
        return _state(st)
    st["table"].copy_(st["was"][0])
    st["refcount"].copy_(st["was"][1])
    if own:
        c.compact()
    else:
        _compact(st)
    return _state(st)


# ------------------------------------------------------------------------------------------------ work, exact


def _size(case):
    return case["Hkv"] * case["D"] * 2 * 2          # bytes of a token's keys and values in one layer


def work(case):
    """By the mean of the lengths that prepare() draws."""
    mean, page = (case["lo"] + case["hi"]) / 2, case["page"]
    if case["op"] == "attend":
        S, B, rows = case["S"], case["B"], case["S"] * case["B"] * case["Hq"]
        if case["ragged"]:
            rows *= 0.5
        keys = case["prefix"] + S * (mean + B)
        io = rows * (4 * case["D"] + 4)
        return {"bytes": keys * _size(case) + io, "flops": 4.0 * case["D"] * rows * (case["prefix"] + mean + B / 2)}
    if case["op"] == "advance":
        return {"bytes": 2.0 * case["L"] * case["S"] * case["B"] * _size(case) + 64.0 * case["S"], "flops": 0.0}
    if case["op"] == "fork":    # each candidate copies the filled part of its parent's last page, half a page on average
        half = min(mean, page / 2)
        meta = case["parents"] * case["kids"] * _ceil(mean, page) * 12
        return {"bytes": 2.0 * case["L"] * case["parents"] * case["kids"] * half * _size(case) + meta, "flops": 0.0}
    gone = max(1, int(case["S"] * case["gone"])) / case["S"]
    total = case["S"] * (mean / page + 0.5)
    moved = total * gone * (1 - gone)               # live pages that lie above the number of live pages
    return {"bytes": 2.0 * case["L"] * moved * page * _size(case) + 8.0 * total, "flops": 0.0}


def _exact_attend(st):
    case, page = st["case"], st["page"]
    S, B, Hq, Hkv = (case[n] for n in ("S", "B", "Hq", "Hkv"))
    out, lse = st["out"].double(), st["lse"].double()
    length, table = st["length"].tolist(), st["table"].tolist()
    used = [B] * S if st["lengths"] is None else st["lengths"].tolist()
    mask = None if st["mask"] is None else st["mask"].tolist()
    for s in range(S):
        n = used[s]
        if n == 0:
            continue
        total = length[s] + n
        ids = torch.tensor(table[s][:_ceil(total, page)], device="cuda")
        k, v = (st["pool"][0, i][ids].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :total] for i in (0, 1))
        hide = torch.zeros((n, total), dtype=torch.bool)
        for b in range(n):
            for i in range(n):
                hide[b, length[s] + i] = i > b if mask is None else not (mask[s][b] >> i) & 1
        q = st["q"][s, :n].double().transpose(0, 1)                     # [Hq, n, D]
        k, v = (x.repeat_interleave(Hq // Hkv, 0) for x in (k, v))
        a = torch.matmul(q, k.transpose(1, 2)) * st["scale"]
        a[:, hide.cuda()] = -math.inf
        z = torch.logsumexp(a, -1)
        out[s, :n] = torch.matmul(torch.softmax(a, -1), v).transpose(0, 1)
        lse[s, :n] = z.transpose(0, 1)
    return out, lse


class _Book:
    """The cache's books kept one entry at a time, from the definitions."""

    def __init__(self, st):
        self.length, self.held, self.table, self.ref = (st[n].tolist() for n in ("length", "held", "table", "refcount"))
        self.page, self.pool = st["page"], st["pool"]

    def truncate(self, new):
        for s, n in enumerate(new):
            while self.held[s] > _ceil(n, self.page):
                self.held[s] -= 1
                self.ref[self.table[s][self.held[s]]] -= 1
                self.table[s][self.held[s]] = -1
            self.length[s] = n

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            self.held[b], self.length[b] = _ceil(self.length[a], self.page), self.length[a]
            for i in range(self.held[b]):
                self.table[b][i] = self.table[a][i]
                self.ref[self.table[a][i]] += 1

    def reserve(self, n):
        free = [p for p, r in enumerate(self.ref) if r == 0][::-1]
        writers = {}
        for s, m in enumerate(self.length):
            if m % self.page and m // self.page < self.held[s]:
                writers.setdefault(self.table[s][m // self.page], []).append(s)
        held_by = {p: self.ref[p] for p in writers}
        for s, m in enumerate(self.length):
            i = m // self.page
            if m % self.page and i < self.held[s]:
                p = self.table[s][i]
                w = writers[p]
                if held_by[p] > 1 and not (held_by[p] == len(w) and w[0] == s):
                    to = free.pop()
                    self.pool[:, :, to, :, :m % self.page] = self.pool[:, :, p, :, :m % self.page]
                    self.ref[p] -= 1
                    self.ref[to] += 1
                    self.table[s][i] = to
            while self.held[s] < _ceil(m + n, self.page):
                self.table[s][self.held[s]] = free.pop()
                self.ref[self.table[s][self.held[s]]] += 1
                self.held[s] += 1

    def append(self, new):
        for s, m in enumerate(self.length):
            b = 0
            while b < new.shape[3]:
                i, off = divmod(m + b, self.page)
                n = min(self.page - off, new.shape[3] - b)
                self.pool[:, :, self.table[s][i], :, off:off + n] = new[:, :, s, b:b + n].transpose(2, 3)
                b += n

    def compact(self):
        live = [p for p, r in enumerate(self.ref) if r]
        low = [p for p in range(len(live)) if not self.ref[p]]
        to = {}
        for p in live:
            if p >= len(live):
                to[p] = low.pop(0)
                self.pool[:, :, to[p]] = self.pool[:, :, p]
                self.ref[to[p]], self.ref[p] = self.ref[p], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]

    def all(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        return [torch.tensor(x, **i32) for x in (self.length, self.held, self.table, self.ref)] + [self.pool]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(st)
    book = _Book(st)
    if case["op"] == "advance":
        book.reserve(case["B"])
        book.append(st["new"])
        book.truncate(st["final"].tolist())
    elif case["op"] == "fork":
        book.truncate(st["drop"].tolist())
        book.fork(st["src"].tolist(), st["dst"].tolist())
        book.reserve(case["B"])
    else:
        book.compact()
    return book.all()
