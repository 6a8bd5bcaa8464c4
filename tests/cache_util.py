"""Plain definitions of the paged cache for its tests: books kept one entry at a time, and the attention of a block in
64 bits with the error that its arithmetic allows."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step of the type, relative


def ceil_div(a, b):
    return -(-a // b)


class Books:
    """length, held, table and refcount of a cache, and (optionally) pools [L, 2, P, Hkv, page, D] on the CPU."""

    def __init__(self, S, M, P, page, pool=None):
        self.S, self.M, self.P, self.page, self.pool = S, M, P, page, pool
        self.length, self.held = [0] * S, [0] * S
        self.table, self.ref = [[-1] * M for _ in range(S)], [0] * P

    def reserve(self, add):
        """False (and nothing done) when there are too few pages or a stream would pass its table."""
        if any(n > 0 and self.length[s] + n > self.M * self.page for s, n in enumerate(add)):
            return False
        writers = {}
        for s, n in enumerate(add):
            if n > 0 and self.length[s] % self.page:
                writers.setdefault(self.table[s][self.length[s] // self.page], []).append(s)
        copies = {s for p, w in writers.items() for s in w
                  if self.ref[p] > 1 and not (self.ref[p] == len(w) and s == w[0])}
        free = [p for p in range(self.P) if self.ref[p] == 0]
        need = [max(self.held[s], ceil_div(self.length[s] + n, self.page)) if n > 0 else self.held[s]
                for s, n in enumerate(add)]
        if len(copies) + sum(need) - sum(self.held) > len(free):
            return False
        for s in range(self.S):
            if s in copies:
                i, used = divmod(self.length[s], self.page)
                old, new = self.table[s][i], free.pop(0)
                if self.pool is not None:
                    self.pool[:, :, new, :, :used] = self.pool[:, :, old, :, :used]
                self.ref[old] -= 1
                self.ref[new] = 1
                self.table[s][i] = new
            for i in range(self.held[s], need[s]):
                self.table[s][i] = free.pop(0)
                self.ref[self.table[s][i]] = 1
            self.held[s] = need[s]
        return True

    def append(self, k, v, layer, used):
        for s, n in enumerate(used):
            for b in range(n):
                i, off = divmod(self.length[s] + b, self.page)
                self.pool[layer, 0, self.table[s][i], :, off] = k[s, b]
                self.pool[layer, 1, self.table[s][i], :, off] = v[s, b]

    def truncate(self, new):
        for s, n in enumerate(new):
            if n < 0 or n > self.held[s] * self.page:
                continue
            for i in range(ceil_div(n, self.page), self.held[s]):
                self.ref[self.table[s][i]] -= 1
                self.table[s][i] = -1
            self.held[s] = min(self.held[s], ceil_div(n, self.page))
            self.length[s] = n

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            self.length[b], self.held[b] = self.length[a], ceil_div(self.length[a], self.page)
            for i in range(self.held[b]):
                self.table[b][i] = self.table[a][i]
                self.ref[self.table[a][i]] += 1

    def compact(self):
        used = [p for p in range(self.P) if self.ref[p]]
        holes = [p for p in range(len(used)) if not self.ref[p]]
        to = dict(zip([p for p in used if p >= len(used)], holes))
        for a, b in to.items():
            if self.pool is not None:
                self.pool[:, :, b] = self.pool[:, :, a]
            self.ref[b], self.ref[a] = self.ref[a], 0
        for s in range(self.S):
            for i in range(self.held[s]):
                self.table[s][i] = to.get(self.table[s][i], self.table[s][i])

    def consistent(self):
        counts = [0] * self.P
        for s in range(self.S):
            assert self.held[s] * self.page >= self.length[s]
            for i in range(self.held[s]):
                counts[self.table[s][i]] += 1
        assert counts == self.ref


def write_books(cache, books):
    for view, rows in ((cache.length, books.length), (cache.held, books.held), (cache.page_table, books.table),
                       (cache.refcount, books.ref)):
        view.copy_(torch.tensor(rows, dtype=torch.int32))


def assert_books(cache, books):
    assert cache.length.tolist() == books.length
    assert cache.held.tolist() == books.held
    assert cache.refcount.tolist() == books.ref
    table = cache.page_table.tolist()
    for s in range(books.S):
        assert table[s][:books.held[s]] == books.table[s][:books.held[s]], s
    # marks of the library are at rest: the next call starts from there
    assert not cache.state[2 + 2:16].any()


def attend_reference(q, k, v, ctx, used, scale, mask=None):
    """One stream.  q [B, Hq, D]; k, v [Hkv, >= ctx + used, D], all fp64.  Returns out [used, Hq, D], lse [used, Hq] and
    the errors they may have: (per unit of the type's half step, and absolute, of out; absolute of lse)."""
    B, Hq, D = q.shape
    n = ctx + used
    G = Hq // k.shape[0]
    seen = torch.zeros((used, n), dtype=torch.bool, device=q.device)
    seen[:, :ctx] = True
    for b in range(used):
        for i in range(used):
            seen[b, ctx + i] = i <= b if mask is None else bool((mask[b] >> i) & 1)
    outs, lses, per_u, abs_o, abs_l = [], [], [], [], []
    for h in range(Hq):
        kk, vv = k[h // G, :n], v[h // G, :n]
        s = torch.where(seen, scale * (q[:used, h] @ torch.where(seen.any(0)[:, None], kk, 0).T), -math.inf)
        m = s.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0, m)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        w = p / torch.where(z == 0, 1, z)
        hidden = torch.where(seen.any(0)[:, None], vv, 0)
        o = torch.stack([w[b][seen[b]] @ hidden[seen[b]] for b in range(used)])
        a = torch.stack([w[b][seen[b]] @ hidden[seen[b]].abs() for b in range(used)])
        # scores: D products summed in fp32 (a step of 2^-22 for each covers a sum that truncates), then the scaling
        # and the subtraction of the maximum, 2^-22 of the largest score each
        mag = abs(scale) * (q[:used, h].abs() @ torch.where(seen.any(0)[:, None], kk, 0).abs().T)
        mag = torch.where(seen, mag, 0).amax(-1, keepdim=True) if n else torch.zeros_like(z)
        ds = (D + 8) * 2.0 ** -22 * mag + 2.0 ** -21
        outs.append(o); lses.append((m + torch.log(z)).squeeze(-1))
        per_u.append(o.abs() + a)           # the output's rounding, and that of the softmax's terms
        # scores' error in terms and sum; fp32 sums (2^-20); terms below the smallest normal fp16 (steps of 2^-24)
        abs_o.append((2 * ds + 2.0 ** -20) * a + n * 2.0 ** -25 * hidden.abs().amax() * 2.0 ** -1)
        abs_l.append((ds + 2.0 ** -20 + 2.0 ** -22 * lses[-1].abs()[:, None]).squeeze(-1))
    cat = lambda x: torch.stack(x, 1)  # noqa: E731
    return cat(outs), cat(lses), cat(per_u), cat(abs_o), cat(abs_l)


def gather(pool, table, held, page):
    """The keys or values of a stream: [Hkv, held * page, D] from pool [P, Hkv, page, D]."""
    ids = torch.as_tensor(table[:held], dtype=torch.long, device=pool.device)
    return pool[ids].permute(1, 0, 2, 3).reshape(pool.shape[1], held * page, pool.shape[3])


def assert_attention(out, lse, q, pool_k, pool_v, books, used, scale, mask=None, streams=None):
    """Every row of streams with used[s] > 0 against the reference, within what the arithmetic allows."""
    u = U[q.dtype]
    for s in streams if streams is not None else range(q.shape[0]):
        if used[s] == 0:
            continue
        k = gather(pool_k, books.table[s], books.held[s], books.page).double()
        v = gather(pool_v, books.table[s], books.held[s], books.page).double()
        o, z, pu, ao, al = attend_reference(q[s].double(), k, v, books.length[s], used[s], scale,
                                            None if mask is None else mask[s])
        err = (out[s, :used[s]].double() - o).abs()
        tol = 1.01 * u * pu + ao
        assert (err <= tol).all(), (s, float((err / tol).max()), float(err.max()))
        got = lse[s, :used[s]].double()
        empty = z == -math.inf
        assert torch.equal(got == -math.inf, empty), s
        lerr = torch.where(empty, 0.0, (got - z).abs())
        assert (lerr <= torch.where(empty, 1.0, al)).all(), (s, float(lerr.max()))
