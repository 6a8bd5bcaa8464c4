"""Cases of what a verify forward does around its attention and its acceptance: norms of queries and keys with the
position rotation, the same on the way into the paged cache, penalties, biases and grammar masks on the logits, alone
and with the acceptance of drafted chains and trees, and the accepted path of a tree kept in the cache.

Rotation: pair i of a head turns by position * f_i.  Edits: with c the count of a token in a stream's generated tokens
and in the block positions that a position sees, z -> z / r (z r below zero) where the token was seen or prompted,
- f c - p [c > 0], + bias, and -inf where the grammar does not allow it.  Trees: bit i of mask[s, b] says that block
position b sees position i, its ancestors and itself.  The plain forms below are elementary torch operations.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # the queries and keys of one user's verify block, far into a long chat: the latency of one small call
        dict(name="rotate one block", op="rotate", N=8, Hq=56, Hkv=8, D=128, R=128, inter=False, norm=True, scale="parts",
             far=130000, dtype="bf16"),
        # a long prompt of odd length, normed heads
        dict(name="rotate prompt", op="rotate", N=16381, Hq=56, Hkv=8, D=128, R=128, inter=False, norm=True, scale="none",
             far=16381, dtype="bf16"),
        # many prompts at once, narrow heads of which half turn, pairs side by side
        dict(name="rotate half of narrow heads", op="rotate", N=47976, Hq=32, Hkv=4, D=64, R=32, inter=True, norm=False,
             scale="linear", far=60000, dtype="fp16"),
        # taking a block in: one stream and one layer, ...
        dict(name="take in one stream", op="take", L=1, S=1, B=8, Hq=56, Hkv=8, D=128, page=64, lo=4093, hi=4093, R=128,
             inter=False, norm=True, scale="parts", tree=False, dtype="bf16"),
        # ... a verify batch over a stack of eight layers, ...
        dict(name="take in verify batch", op="take", L=8, S=32, B=8, Hq=56, Hkv=8, D=128, page=64, lo=1, hi=2000, R=128,
             inter=False, norm=True, scale="none", tree=False, dtype="bf16"),
        # ... and the prompts of new streams, in one long block of odd length
        dict(name="take in prompts", op="take", L=2, S=24, B=1999, Hq=32, Hkv=4, D=64, page=16, lo=0, hi=40, R=32,
             inter=True, norm=False, scale="ntk", tree=False, dtype="fp16"),
        # one step of a sampler: penalties, biases and a strict grammar on the next token of every stream
        dict(name="edit next tokens", op="edit", S=96, B=1, V=32000, lo=40, hi=6000, bias=50, grammar=0.03, tree=False,
             dtype="fp32"),
        # the logits of a verify batch, penalties and biases without a grammar
        dict(name="edit verify batch", op="edit", S=32, B=8, V=151936, lo=100, hi=3000, bias=20, grammar=0.0, tree=False,
             dtype="fp32"),
        # acceptance of one user's block: the latency of a single stream
        dict(name="accept one stream", op="accept", S=1, B=8, V=151936, lo=4093, hi=4093, bias=10, grammar=0.0, tree=False,
             dtype="fp32"),
        # trees of drafts under a loose grammar (free text inside a template), logits as the projection gives them
        dict(name="accept draft trees", op="accept", S=48, B=11, V=151936, lo=100, hi=4000, bias=0, grammar=0.5, tree=True,
             dtype="bf16"),
        # the accepted path of one tree, kept in eight layers, ...
        dict(name="keep one path", op="keep", L=8, S=1, B=8, Hq=56, Hkv=8, D=128, page=64, lo=1000, hi=1000, R=128,
             inter=False, norm=True, scale="none", tree=True, dtype="bf16"),
        # ... and those of a batch with wide trees
        dict(name="keep paths of a batch", op="keep", L=8, S=64, B=40, Hq=32, Hkv=8, D=128, page=64, lo=100, hi=3000, R=128,
             inter=False, norm=False, scale="none", tree=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "take", "edit", "accept", "keep"])
    if op in ("edit", "accept"):
        B = _log(rng, 1, 32)
        V = rng.choice([_log(rng, 500, 160000), 4 * _log(rng, 125, 40000)])
        S = _log(rng, 1, max(1, min(128, 38000000 // (B * V))))
        lo = _log(rng, 1, 1000)
        return dict(op=op, S=S, B=B, V=V, lo=lo, hi=lo + _log(rng, 1, 5000), bias=rng.choice([0, 1, 30, 300]),
                    grammar=rng.choice([0.0, 0.03, 0.5, 0.97]), tree=rng.random() < 0.5,
                    dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]))
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 8])
    Hq = Hkv * rng.choice([1, 2, 5, 8])
    c = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, R=rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)]),
             inter=rng.random() < 0.5, norm=rng.random() < 0.5, scale=rng.choice(["none", "linear", "ntk", "parts"]),
             dtype=rng.choice(["bf16", "fp16"]))
    if op == "rotate":
        c.update(N=_log(rng, 1, 100000000 // (D * (Hq + Hkv))), far=_log(rng, 10, 2000000))
        return c
    c.update(L=rng.randint(1, 8), S=_log(rng, 1, 64), page=rng.choice([16, 32, 64, 128]), tree=rng.random() < 0.4)
    if op == "keep":
        c.update(B=_log(rng, 2, 48), tree=True)
    else:
        most = 100000000 // (D * (Hq + 2 * Hkv) * c["L"] * c["S"])
        c.update(B=_log(rng, 1, max(1, min(64 if c["tree"] else 2000, most))))
    lo = _log(rng, 1, 300) - 1
    c.update(lo=lo, hi=lo + _log(rng, 1, 2000))
    return c


# ------------------------------------------------------------------------------------------------ inputs


BASE, EPS, FACTOR, ORIGINAL, LOW, HIGH = 10000.0, 1e-6, 8.0, 8192, 1.0, 32.0


def _ceil(a, b):
    return -(-a // b)


def _lengths(case, n, g):
    """Evenly spread over the case's range, in an order of the seed's: every seed has as many tokens."""
    spread = torch.linspace(case["lo"], case["hi"], n + 2)[1:-1].round().int()
    return spread[torch.randperm(n, generator=g)]


def _gain(case):
    return 0.1 * math.log(FACTOR) + 1.0 if case["scale"] == "parts" else 1.0


def _frequencies(case):
    R, base = case["R"], BASE
    if case["scale"] == "ntk" and R > 2:
        base = BASE * FACTOR ** (R / (R - 2))
    f = torch.tensor([base ** (-2 * i / R) for i in range(R // 2)], dtype=torch.float64)
    if case["scale"] == "linear":
        f = f / FACTOR
    elif case["scale"] == "parts":      # pairs that turn often in the original length stay, slow ones are stretched
        keep = ((ORIGINAL * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / FACTOR
    return f


def _trees(S, B, g):
    """Random trees: position b sees its ancestors and itself.  Returns mask [S][B] and parents [S][B]."""
    masks, parents = [], []
    for _ in range(S):
        seen, up = [1], [-1]
        for b in range(1, B):
            p = max(int(torch.randint(0, b, (1,), generator=g)), int(torch.randint(0, b, (1,), generator=g)))
            up.append(p)
            seen.append(seen[p] | (1 << b))
        masks.append(seen)
        parents.append(up)
    return masks, parents


def _mask_tensor(masks):
    return torch.tensor([[m - (1 << 64) if m >> 63 else m for m in row] for row in masks], dtype=torch.int64, device="cuda")


def _projection(case, shape, gd):
    """Projections' outputs: some channels stronger than others, values with a mean of their own."""
    x = torch.randn(shape, generator=gd, device="cuda", dtype=DTYPES[case["dtype"]])
    x[..., ::17] *= 2.5
    return x


def _rotary(st, case, gd):
    D = case["D"]
    st["freq"] = _frequencies(case).cuda()
    st["q_w"] = st["k_w"] = None
    if case["norm"]:
        st["q_w"], st["k_w"] = (1 + 0.2 * torch.randn((2, D), generator=gd, device="cuda")).to(DTYPES[case["dtype"]])
    if own:
        import mxfp4_moe_expert_gb300 as pkg
        scaling = None if case["scale"] == "none" else dict(kind=case["scale"], factor=FACTOR)
        if case["scale"] == "parts":
            scaling.update(original=ORIGINAL, low=LOW, high=HIGH)
        st["rotary"] = pkg.Rotary(head_dim=D, rotary_dim=case["R"], base=BASE, scaling=scaling, interleaved=case["inter"],
                                  gain=_gain(case), q_norm=st["q_w"], k_norm=st["k_w"], eps=EPS,
                                  dtype=DTYPES[case["dtype"]], device="cuda")


def _prepare_rotate(st, case, g, gd):
    N, D = case["N"], case["D"]
    st["qk"] = _projection(case, (N, case["Hq"] + case["Hkv"], D), gd)
    first = torch.randint(0, max(1, case["far"] - N), (1,), generator=g).item()
    st["pos"] = (torch.arange(N) + first).int().cuda()
    _rotary(st, case, gd)


def _prepare_cache(st, case, g, gd):
    S, B, L, D, page = case["S"], case["B"], case["L"], case["D"], case["page"]
    Hq, Hkv = case["Hq"], case["Hkv"]
    lens = _lengths(case, S, g).tolist()
    MP = _ceil(case["hi"] + B, page)
    held = [_ceil(n + B, page) for n in lens]           # the block is reserved
    P = sum(held) + 3
    free = torch.randperm(P, generator=g).tolist()
    table, ref = [[-1] * MP for _ in range(S)], [0] * P
    for i in range(MP):                                 # streams take pages in turn, as they grow
        for s in range(S):
            if i < held[s]:
                table[s][i] = free.pop()
                ref[table[s][i]] = 1
    i32 = dict(dtype=torch.int32, device="cuda")
    st["was"] = torch.cat([torch.tensor(x, **i32).view(-1) for x in (lens, held, table, ref)])
    st["pool"] = torch.randn((L, 2, P, Hkv, page, D), generator=gd, device="cuda", dtype=DTYPES[case["dtype"]])
    st["qkv"] = _projection(case, (L, S, B, Hq + 2 * Hkv, D), gd)
    st["q_out"] = torch.empty((L, S, B, Hq, D), device="cuda", dtype=DTYPES[case["dtype"]])
    st["mask"] = None
    if case["tree"]:
        masks, parents = _trees(S, B, g)
        st["mask"] = _mask_tensor(masks)
        paths, accepted = torch.full((S, B), -1), []
        for s in range(S):                              # from a node up to the root
            n, at = int(torch.randint(0, B, (1,), generator=g)), []
            while n >= 0:
                at.append(n)
                n = parents[s][n]
            paths[s, :len(at)] = torch.tensor(at[::-1])
            accepted.append(len(at))
        st["path"], st["accepted"] = paths.int().cuda(), torch.tensor(accepted, **i32)
    if case["op"] == "keep":
        st["tokens"] = torch.randint(0, 50000, (S, B), generator=g).int().cuda()
        st["history"] = torch.randint(0, 50000, (S, case["hi"] + B), generator=g).int().cuda()
    _rotary(st, case, gd)
    books = None
    if own:     # the handle over the same pool, and a state that holds the same tables
        import mxfp4_moe_expert_gb300 as pkg
        c = st["cache"] = pkg.KvCache(layers=[(kv[0], kv[1]) for kv in st["pool"]], num_streams=S, max_pages=MP)
        books = c.state[16:16 + st["was"].numel()]
        books.copy_(st["was"])
    st["books"] = books = st["was"].clone() if books is None else books
    st["length"], st["held"], st["table"], st["ref"] = books.split([S, S, S * MP, P])
    st["table"] = st["table"].view(S, MP)


def _prepare_logits(st, case, g, gd):
    """Logits with a clear winner at most positions, which is often a drafted token; token histories whose common
    tokens come back often; streams with and without penalties."""
    S, B, V = case["S"], case["B"], case["V"]
    common = lambda n: (V ** torch.rand(n, generator=g, dtype=torch.float64) - 1).long().clamp(0, V - 1)   # noqa: E731
    x = 2 * torch.randn((S, B, V), generator=gd, device="cuda")
    tokens = torch.randint(0, V, (S, B), generator=g)
    st["mask"], parents = None, [[b - 1 for b in range(B)] for _ in range(S)]
    if case["tree"]:
        masks, parents = _trees(S, B, g)
        st["mask"] = _mask_tensor(masks)
    best = common((S, B))
    for s in range(S):
        for b in range(1, B):
            if torch.rand(1, generator=g) < 0.8:
                best[s, parents[s][b]] = tokens[s, b]
    x.scatter_add_(2, best.cuda()[:, :, None], 9 + 4 * torch.rand((S, B, 1), generator=gd, device="cuda"))
    st["logits"], st["tokens"] = x.to(DTYPES[case["dtype"]]), tokens.int().cuda()
    lens = _lengths(case, S, g)
    st["history"] = common((S, case["hi"])).int().cuda()
    st["history_lengths"] = lens.cuda()
    st["prompt_lengths"] = (lens * torch.rand(S, generator=g)).int().cuda()
    f32 = dict(dtype=torch.float32, device="cuda")
    on = (torch.rand((3, S), generator=g) < 0.8).float()
    st["repetition"] = (1 + 0.3 * on[0] * torch.rand(S, generator=g)).to(**f32)
    st["frequency"] = (0.4 * on[1] * torch.rand(S, generator=g)).to(**f32)
    st["presence"] = (0.6 * on[2] * torch.rand(S, generator=g)).to(**f32)
    st["bias"] = None
    if case["bias"]:
        n = min(case["bias"], V)
        ids = torch.stack([torch.randperm(V, generator=g)[:n] for _ in range(S)])
        st["bias"] = (torch.arange(0, S * n + 1, n).int().cuda(), ids.view(-1).int().cuda(),
                      (4 * torch.randn(S * n, generator=g)).to(**f32))
    st["allowed"] = None
    if case["grammar"]:
        words = _ceil(V, 32)
        p = case["grammar"]
        bits = torch.rand((S, B, words, 32), generator=gd, device="cuda", dtype=torch.float16) < p
        st["allowed"] = (bits.int() << torch.arange(32, device="cuda", dtype=torch.int32)).sum(-1, dtype=torch.int32)
        at = best.cuda()                                 # the likeliest token fits the grammar as a rule
        word = st["allowed"].gather(2, (at >> 5)[:, :, None])
        bit = (1 << (at & 31)).int()[:, :, None] * (torch.rand((S, B, 1), generator=gd, device="cuda") < 0.9)
        st["allowed"].scatter_(2, (at >> 5)[:, :, None], word | bit.int())
    st["out"] = torch.empty_like(st["logits"]) if case["op"] == "edit" else None


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed + 1)
    st = dict(op=case["op"], case=dict(case))
    if case["op"] == "rotate":
        _prepare_rotate(st, case, g, gd)
    elif case["op"] in ("take", "keep"):
        _prepare_cache(st, case, g, gd)
    else:
        _prepare_logits(st, case, g, gd)
    return st


# ------------------------------------------------------------------------------------------------ plain forms


def _turn(st, x, weight, pos):
    """x [N, H, D] at positions pos [N]: normed and turned, in fp32, rounded once."""
    case, kind = st["case"], x.dtype
    angle = pos.double()[:, None] * st["freq"]
    cos, sin = ((f(angle) * _gain(case)).float()[:, None] for f in (torch.cos, torch.sin))
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    R = case["R"]
    y = x.clone()
    if case["inter"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2], y[..., R // 2:R] = a * cos - b * sin, a * sin + b * cos
    return y.to(kind)


def _depth(st):
    """Position of each block position behind its stream's length: the earlier ones it sees."""
    case = st["case"]
    b = torch.arange(case["B"], device="cuda")
    if st["mask"] is None:
        return b.expand(case["S"], -1)
    seen = (st["mask"][:, :, None] >> b) & 1
    return (seen * (b[None, :] < b[:, None])).sum(-1)


def _take(st):
    case, page = st["case"], st["case"]["page"]
    L, S, B, Hq, Hkv, D = (case[n] for n in ("L", "S", "B", "Hq", "Hkv", "D"))
    pos = (st["length"][:, None] + _depth(st)).view(-1)
    slot = st["length"][:, None] + torch.arange(B, device="cuda")
    at = st["table"].gather(1, (slot // page).long()).long()
    for layer in range(L):
        q, k, v = st["qkv"][layer].view(S * B, -1, D).split([Hq, Hkv, Hkv], 1)
        st["q_out"][layer] = _turn(st, q, st["q_w"], pos).view(S, B, Hq, D)
        st["pool"][layer, 0][at, :, (slot % page).long()] = _turn(st, k, st["k_w"], pos).view(S, B, Hkv, D)
        st["pool"][layer, 1][at, :, (slot % page).long()] = v.reshape(S, B, Hkv, D)


def _keep(st):
    case, page = st["case"], st["case"]["page"]
    S, B = case["S"], case["B"]
    path, n = st["path"].long().clamp(min=0), st["accepted"]
    i = torch.arange(B, device="cuda")[None, :]
    use = i < n[:, None]
    src = st["length"][:, None].long() + path
    dst = (st["length"][:, None] + i).long()
    s = torch.arange(S, device="cuda")[:, None].expand(S, B)[use]
    a, b = src[use], dst[use]
    moved = st["pool"][:, :, st["table"][s, a // page].long(), :, a % page]
    st["pool"][:, :, st["table"][s, b // page].long(), :, b % page] = moved
    st["history"][s, b] = st["tokens"].gather(1, path)[use]
    new = st["length"] + n
    keep = (new + page - 1) // page
    j = torch.arange(st["table"].shape[1], device="cuda")[None, :]
    gone = (j >= keep[:, None]) & (j < st["held"][:, None])
    st["ref"].scatter_add_(0, st["table"].clamp(min=0).long().view(-1), -gone.int().view(-1))
    st["table"].masked_fill_(gone, -1)
    st["held"].copy_(torch.minimum(st["held"], keep))
    st["length"].copy_(new)


def _edited(st):
    """The edited logits in fp32 [S, B, V], and where a token is allowed."""
    case = st["case"]
    S, B, V = case["S"], case["B"], case["V"]
    z = st["logits"].float()
    j = torch.arange(st["history"].shape[1], device="cuda")[None, :]
    prompt = j < st["prompt_lengths"][:, None]
    made = (j < st["history_lengths"][:, None]) & ~prompt
    h = st["history"].long()
    prompted = torch.zeros((S, V), device="cuda").scatter_add_(1, h, prompt.float()) > 0
    count = torch.zeros((S, V), device="cuda").scatter_add_(1, h, made.float())[:, None].repeat(1, B, 1)
    b = torch.arange(B, device="cuda")
    if st["mask"] is None:
        sees = (b[None, :] <= b[:, None]).expand(S, B, B)
    else:
        sees = (((st["mask"][:, :, None] >> b) & 1 > 0) & (b[None, :] < b[:, None])) | (b[None, :] == b[:, None])
    count.scatter_add_(2, st["tokens"].long()[:, None].expand(S, B, B), sees.float())
    r, f, p = (st[n][:, None, None] for n in ("repetition", "frequency", "presence"))
    seen = (count > 0) | prompted[:, None]
    z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
    z = z - f * count - p * (count > 0)
    if st["bias"] is not None:
        begin, ids, values = st["bias"]
        s = torch.repeat_interleave(torch.arange(S, device="cuda"), (begin[1:] - begin[:-1]).long(), output_size=ids.numel())
        z = z + torch.zeros((S, V), device="cuda").index_put((s, ids.long()), values)[:, None]
    if st["allowed"] is None:
        return z, None
    ok = ((st["allowed"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).view(S, B, -1)[..., :V] > 0
    return z, ok


def _accept(st):
    case = st["case"]
    S, B, V = case["S"], case["B"], case["V"]
    z, ok = _edited(st)
    if ok is not None:
        z = torch.where(ok, z, -math.inf)
    top = z.amax(-1, keepdim=True)
    v = torch.arange(V, device="cuda")
    target = torch.where(z == top if ok is None else (z == top) & ok, v, V).amin(-1)
    target = torch.where(target == V, -1, target).int()
    tokens = st["tokens"]
    b = torch.arange(B, device="cuda")
    if st["mask"] is None:
        parent = (b - 1).expand(S, B)
    else:
        seen = ((st["mask"][:, :, None] >> b) & 1 > 0) & (b[None, :] < b[:, None])
        parent = torch.where(seen, b, -1).amax(-1)
    s = torch.arange(S, device="cuda")
    at, alive = torch.zeros(S, dtype=torch.long, device="cuda"), torch.ones(S, dtype=torch.bool, device="cuda")
    path = torch.full((S, B), -1, dtype=torch.int32, device="cuda")
    accepted = torch.zeros(S, dtype=torch.int32, device="cuda")
    for i in range(B):
        path[:, i] = torch.where(alive, at, -1)
        accepted += alive
        fits = (parent == at[:, None]) & (tokens == target[s, at][:, None]) & (b > 0)
        child = torch.where(fits, b, B).amin(-1)
        alive = alive & (child < B)
        at = torch.where(alive, child, at)
    return target, accepted, target[s, at], path


def run(st):
    op, case = st["op"], st["case"]
    if op == "rotate":
        q, k = st["qk"].split([case["Hq"], case["Hkv"]], 1)
        if own:
            return st["rotary"].rotate(q, k, st["pos"])
        return _turn(st, q, st["q_w"], st["pos"]), _turn(st, k, st["k_w"], st["pos"])
    if op == "take" or op == "keep":
        if op == "keep":                                # the books as they were before the block was accepted
            st["books"].copy_(st["was"])
        if own:
            c = st["cache"]
            for layer in range(case["L"]):
                q, k, v = st["qkv"][layer].split([case["Hq"], case["Hkv"], case["Hkv"]], 2)
                c.append_rotated(layer, q, k, v, st["rotary"], mask=st["mask"], out=st["q_out"][layer])
            if op == "keep":
                c.commit(st["accepted"], path=st["path"], tokens=st["tokens"], history=st["history"])
        else:
            _take(st)
            if op == "keep":
                _keep(st)
        out = [st["q_out"], st["pool"]]
        return out + [st[n] for n in ("length", "held", "table", "ref", "history")] if op == "keep" else out
    if own:
        import mxfp4_moe_expert_gb300 as pkg
        edits = {n: st[n] for n in ("mask", "history", "history_lengths", "prompt_lengths", "repetition", "frequency",
                                    "presence", "bias", "allowed")}
        if op == "edit":
            return pkg.edit_logits(st["logits"], st["tokens"], out=st["out"], **edits)
        return pkg.accept_edited(st["logits"], st["tokens"], **edits)
    if op == "accept":
        return _accept(st)
    z, ok = _edited(st)
    if ok is not None:
        z = torch.where(ok, z, -math.inf)
    st["out"].copy_(z)
    return st["out"]


# ------------------------------------------------------------------------------------------------ work, exact


def work(case):
    """By the mean of the lengths that prepare() draws."""
    op = case["op"]
    if op == "rotate":
        n = case["N"] * (case["Hq"] + case["Hkv"]) * case["D"]
        return {"bytes": 4.0 * n + 4.0 * case["N"], "flops": (3.0 * case["R"] / case["D"] + 4.0 * case["norm"]) * n}
    if op in ("edit", "accept"):
        rows, V, size = case["S"] * case["B"], case["V"], 4 if case["dtype"] == "fp32" else 2
        total = rows * V * size * (2 if op == "edit" else 1) + case["S"] * 4 * (case["lo"] + case["hi"]) / 2
        total += case["S"] * 8 * case["bias"] + (rows * V / 8 if case["grammar"] else 0) + rows * 12
        return {"bytes": float(total), "flops": 1.0 * rows * V}
    L, tokens, Hq, Hkv, D = case["L"], case["S"] * case["B"], case["Hq"], case["Hkv"], case["D"]
    n = L * tokens * (Hq + 2 * Hkv) * D
    moved = 0.0
    if op == "keep":                                    # about half of an accepted path lies elsewhere
        moved = 0.5 * L * case["S"] * min(case["B"], 2 * math.log(case["B"] + 1)) * 2 * Hkv * D * 4
    return {"bytes": 4.0 * n + moved, "flops": (3.0 * case["R"] / D + 4.0 * case["norm"]) * L * tokens * (Hq + Hkv) * D}


def _exact_turn(st, x, weight, pos):
    """Pairs as complex numbers, times e^(i angle)."""
    case = st["case"]
    R = case["R"]
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["D"] + EPS) * weight.double()
    head, rest = x[..., :R], x[..., R:]
    pairs = head.unflatten(-1, (R // 2, 2)) if case["inter"] else head.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    f = _frequencies(case).cuda()
    spin = torch.polar(torch.full((), _gain(case), dtype=torch.float64, device="cuda"), torch.outer(pos.double(), f))
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * spin[:, None])
    turned = turned.flatten(-2) if case["inter"] else turned.transpose(-1, -2).flatten(-2)
    return torch.cat([turned, rest], -1)


def _exact_cache(st):
    case, page = st["case"], st["case"]["page"]
    L, S, B, Hq, Hkv, D = (case[n] for n in ("L", "S", "B", "Hq", "Hkv", "D"))
    length, table = st["length"].tolist(), st["table"].tolist()
    masks = st["mask"].tolist() if st["mask"] is not None else [[(1 << (b + 1)) - 1 for b in range(B)]] * S
    pool, q_out = st["pool"].double(), torch.empty((L, S, B, Hq, D), dtype=torch.float64, device="cuda")
    pos = [length[s] + bin(masks[s][b] & ((1 << b) - 1)).count("1") for s in range(S) for b in range(B)]
    x = st["qkv"].view(L, S * B, -1, D)
    pos = torch.tensor(pos, device="cuda")
    for layer in range(L):
        q_out[layer] = _exact_turn(st, x[layer, :, :Hq], st["q_w"], pos).view(S, B, Hq, D)
        k = _exact_turn(st, x[layer, :, Hq:Hq + Hkv], st["k_w"], pos)
        v = x[layer, :, Hq + Hkv:].double()
        for s in range(S):
            t = length[s]
            while t < length[s] + B:                    # run by run of a page
                n = min(page - t % page, length[s] + B - t)
                rows = slice(s * B + t - length[s], s * B + t - length[s] + n)
                for which, new in ((0, k), (1, v)):
                    pool[layer, which, table[s][t // page], :, t % page:t % page + n] = new[rows].transpose(0, 1)
                t += n
    if case["op"] == "take":
        return [q_out, pool]
    path, accepted, held, ref = st["path"].tolist(), st["accepted"].tolist(), st["held"].tolist(), st["ref"].tolist()
    history, tokens = st["history"].tolist(), st["tokens"].tolist()
    for s in range(S):
        for i in range(accepted[s]):
            a, b = length[s] + path[s][i], length[s] + i
            pool[:, :, table[s][b // page], :, b % page] = pool[:, :, table[s][a // page], :, a % page]
            history[s][b] = tokens[s][path[s][i]]
        length[s] += accepted[s]
        while held[s] > _ceil(length[s], page):
            held[s] -= 1
            ref[table[s][held[s]]] -= 1
            table[s][held[s]] = -1
    i32 = dict(dtype=torch.int32, device="cuda")
    return [q_out, pool] + [torch.tensor(x, **i32) for x in (length, held, table, ref, history)]


def _exact_logits(st):
    """One position at a time."""
    case = st["case"]
    S, B, V = case["S"], case["B"], case["V"]
    tokens, n_all, n_prompt = st["tokens"].tolist(), st["history_lengths"].tolist(), st["prompt_lengths"].tolist()
    masks = st["mask"].tolist() if st["mask"] is not None else [[(1 << (b + 1)) - 1 for b in range(B)]] * S
    out = torch.empty((S, B, V), dtype=torch.float64, device="cuda") if case["op"] == "edit" else None
    target = [[-1] * B for _ in range(S)]
    shift = torch.arange(32, device="cuda")
    for s in range(S):
        h = st["history"][s].long()
        told = torch.bincount(h[:n_prompt[s]], minlength=V) > 0
        made = torch.bincount(h[n_prompt[s]:n_all[s]], minlength=V)
        r, f, p = (float(st[n][s]) for n in ("repetition", "frequency", "presence"))
        bias = torch.zeros(V, dtype=torch.float64, device="cuda")
        if st["bias"] is not None:
            lo, hi = st["bias"][0][s:s + 2].tolist()
            bias[st["bias"][1][lo:hi].long()] = st["bias"][2][lo:hi].double()
        for b in range(B):
            c = made.clone()
            for j in range(b + 1):
                if j == b or (masks[s][b] >> j) & 1:
                    c[tokens[s][j]] += 1
            z = st["logits"][s, b].double()
            hit = told | (c > 0)
            z[hit & (z > 0)] /= r
            z[hit & (st["logits"][s, b] <= 0)] *= r
            z = z - f * c.double() + bias
            z[c > 0] -= p
            if st["allowed"] is not None:
                word = st["allowed"][s, b].long()
                z[((word[:, None] >> shift) & 1).view(-1)[:V] == 0] = -math.inf
            if out is not None:
                out[s, b] = z
            elif z.max() > -math.inf:
                target[s][b] = int((z == z.max()).nonzero()[0, 0])
    if out is not None:
        return out
    path, accepted, last = [[-1] * B for _ in range(S)], [], []
    for s in range(S):
        at, n = 0, 0
        while at is not None:
            path[s][n] = at
            n += 1
            here, at = at, None
            for c in range(here + 1, B):
                below = masks[s][c] & ((1 << c) - 1)
                if below.bit_length() - 1 == here and tokens[s][c] == target[s][here]:
                    at = c
                    break
        accepted.append(n)
        last.append(target[s][here])
    i32 = dict(dtype=torch.int32, device="cuda")
    return tuple(torch.tensor(x, **i32) for x in (target, accepted, last, path))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotate":
        q, k = st["qk"][:, :case["Hq"]], st["qk"][:, case["Hq"]:]
        return _exact_turn(st, q, st["q_w"], st["pos"]), _exact_turn(st, k, st["k_w"], st["pos"])
    if case["op"] in ("take", "keep"):
        return _exact_cache(st)
    return _exact_logits(st)
