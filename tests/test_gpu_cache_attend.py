"""GPU tests of the verify block's attention over the paged cache, against the definition in 64 bits; the tolerance is
what the stated arithmetic allows, element by element (tests/cache_util.py)."""
import math
import os
import random

import pytest
import torch

import mxfp4_moe_expert_gb300 as pkg
from cache_util import Books, assert_attention, ceil_div, gather, write_books
from mxfp4_moe_expert_gb300.synth import Workload
from mxfp4_moe_expert_gb300.workload import device_layers

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(pkg.LIB_PATH):
        from mxfp4_moe_expert_gb300 import build
        build.build()
    pkg.load_library()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Streams with given contexts behind a shared prefix (held by the last stream slot), their block stored."""

    def __init__(self, ctx, B, Hq, Hkv, D=128, page=64, prefix=0, dtype=torch.bfloat16, alone=(), seed=0, interleaved=False,
                 fill=None):
        S = len(ctx)
        self.S, self.B, self.Hq, self.Hkv, self.D, self.page, self.prefix = S, B, Hq, Hkv, D, page, prefix
        rng = random.Random(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        assert prefix % page == 0
        npre = prefix // page
        M = max(ceil_div(max(list(ctx) + [0]) + B, page), npre, 1) + 1
        P = npre + sum(ceil_div(n + B, page) for n in ctx) + 5
        free = list(range(P))
        rng.shuffle(free)
        b = self.books = Books(S + 1, M, P, page)
        b.table[S][:npre] = [free.pop() for _ in range(npre)]
        b.held[S], b.length[S] = npre, prefix
        for p in b.table[S][:npre]:
            b.ref[p] += 1
        for s, n in enumerate(ctx):
            held = ceil_div(n + B, page)
            for i in range(held):
                shared = s not in alone and n >= prefix and i < npre
                b.table[s][i] = b.table[S][i] if shared else free.pop()
                b.ref[b.table[s][i]] += 1
            b.held[s], b.length[s] = held, n
        shape = (P, 2, Hkv, page, D) if interleaved else (2, P, Hkv, page, D)
        mem = torch.randn(shape, generator=g, device="cuda").to(dtype)
        self.k, self.v = (mem[:, 0], mem[:, 1]) if interleaved else (mem[0], mem[1])
        self.v += torch.randn((1, Hkv, 1, D), generator=g, device="cuda").to(dtype)
        if fill is not None:                       # what no stream has stored holds `fill`
            used = torch.zeros((P, page), dtype=torch.bool)
            for s in range(S + 1):
                stored = b.length[s] + (B if s < S else 0)
                for i in range(b.held[s]):
                    used[b.table[s][i], :max(0, min(page, stored - i * page))] = True
            hole = (~used).cuda()[:, None, :, None]
            self.k.masked_fill_(hole, fill)
            self.v.masked_fill_(hole, fill)
        self.q = (1.3 * torch.randn((S, B, Hq, D), generator=g, device="cuda")).to(dtype)
        self.cache = pkg.KvCache(layers=[(self.k, self.v)], num_streams=S + 1, max_pages=M)
        write_books(self.cache, b)

    def attend(self, **kw):
        if self.prefix and "shared_tokens" not in kw:
            kw.update(shared_stream=self.S, shared_tokens=self.prefix)
        out, lse = self.cache.attend(0, self.q, **kw)
        torch.cuda.synchronize()
        self.cache.check()
        return out, lse

    def check(self, out, lse, used=None, mask=None, scale=None, streams=None):
        assert_attention(out, lse, self.q, self.k, self.v, self.books, used or [self.B] * self.S,
                         self.D ** -0.5 if scale is None else scale, mask, streams)


@pytest.mark.parametrize("B,Hq,Hkv", [(1, 1, 1), (8, 56, 8), (3, 7, 1), (5, 6, 2), (64, 16, 2), (1, 16, 2), (8, 32, 2), (17, 4, 4)])
@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.float16)])
def test_heads_and_blocks(B, Hq, Hkv, D, dtype):
    c = Case([0, 1, 63, 64, 127, 128, 129, 300], B, Hq, Hkv, D=D, dtype=dtype, seed=B)
    c.check(*c.attend())


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D,dtype,interleaved", [(128, torch.float16, True), (64, torch.bfloat16, False)])
def test_pages_and_a_shared_prefix(page, D, dtype, interleaved):
    """Contexts that end inside, at and behind tiles and pages; a stream of its own pages, one shorter than the prefix."""
    prefix = 384
    ctx = [prefix, prefix + 1, prefix + page - 1, prefix + page, prefix + 700, 5, 0, prefix + 40]
    c = Case(ctx, 8, 8, 2, D=D, page=page, prefix=prefix, dtype=dtype, alone=(7,), seed=page, interleaved=interleaved)
    out, lse = c.attend()
    c.check(out, lse)
    out2, lse2 = c.attend(shared_tokens=0)            # the same without sharing
    c.check(out2, lse2)
    if page <= 64:
        c.check(*c.attend(shared_stream=c.S, shared_tokens=page * 2))   # a part of what is shared


@pytest.mark.parametrize("S,prefix,lo,hi", [(1, 0, 20000, 20000), (2, 4096, 4096, 4100), (40, 2048, 2048, 2500), (130, 256, 256, 400)])
def test_long_and_many(S, prefix, lo, hi):
    rng = random.Random(S)
    c = Case([rng.randint(lo, hi) for _ in range(S)], 8, 14, 2, prefix=prefix, seed=S)
    out, lse = c.attend()
    c.check(out, lse, streams=sorted({0, S - 1, S // 2, S // 3}))


@pytest.mark.parametrize("S,Hq,D,prefix,hi", [(32, 56, 128, 8192, 1500), (24, 64, 64, 12288, 3000),
                                                (64, 64, 128, 12288, 100), (24, 64, 64, 6000, 900)])
def test_many_tiles_for_every_cta(S, Hq, D, prefix, hi):
    """Enough tiles of the shared prefix and of the streams' own keys that every ring goes round many times, and
    passes from one kind of work to the other; every row of some streams, and all rows twice."""
    rng = random.Random(S)
    c = Case([prefix + rng.randint(1, hi) for _ in range(S)], 8, Hq, 8, D=D, page=16 if D == 64 else 64, prefix=prefix, seed=S)
    out, lse = c.attend()
    c.check(out, lse, streams=sorted(rng.sample(range(S), 4)))
    alone, alse = c.attend(shared_tokens=0)
    assert (lse - alse).abs().max() <= 2e-5
    again, again_lse = c.attend()
    assert torch.equal(again, out) and torch.equal(again_lse, lse)


@pytest.mark.parametrize("prefix,B,Hq,Hkv", [(0, 3, 4, 2), (48, 3, 4, 2), (48, 20, 16, 1)])
def test_more_units_than_one_pass_of_the_schedule(prefix, B, Hq, Hkv):
    """900 streams, narrow and wide units, some of them without rows; streams of the first, the second and the third
    pass, and all rows twice."""
    S = 900
    c = Case([prefix + (53 * s) % 200 for s in range(S)], B, Hq, Hkv, D=64, page=16, prefix=prefix, alone=(7, 500), seed=25)
    used = [(s * 7) % (B + 1) for s in range(S)]
    out, lse = c.attend(lengths=i32(used))
    c.check(out, lse, used=used, streams=[0, 7, 8, 383, 384, 385, 500, 767, 768, 769, 898, 899])
    again, again_lse = c.attend(lengths=i32(used))
    assert torch.equal(again, out) and torch.equal(again_lse, lse)
    alone, alse = c.attend(lengths=i32(used), shared_tokens=0)
    seen = lse.isfinite()
    assert torch.equal(seen, alse.isfinite()) and (lse[seen] - alse[seen]).abs().max() <= 2e-5


def test_as_many_kv_heads_as_there_may_be():
    c = Case([0, 65, 300], 2, 512, 256, D=64, page=16, seed=26)
    c.check(*c.attend())


@pytest.mark.parametrize("B,Hq,Hkv,prefix", [(1, 256, 1, 0), (3, 255, 1, 256), (2, 512, 2, 128), (1, 129, 1, 64)])
def test_many_heads_on_one(B, Hq, Hkv, prefix):
    c = Case([prefix + n for n in (0, 1, 130, 500)], B, Hq, Hkv, prefix=prefix, seed=Hq)
    c.check(*c.attend())


def test_the_shared_stream_may_be_one_of_the_batch():
    """Streams forked from stream 0, which goes on itself; stream 2 was cut back into the prefix and has new pages."""
    S, page, D, Hkv = 5, 32, 64, 2
    mem = torch.randn((2, 120, Hkv, page, D), device="cuda").bfloat16()
    cache = pkg.KvCache(layers=[(mem[0], mem[1])], num_streams=S, max_pages=20)
    books = Books(S, 20, 120, page)
    for c in (cache, books):
        arg = (lambda x: x) if c is books else i32
        c.reserve(arg([330, 0, 0, 0, 0]))
        c.truncate(arg([330, -1, -1, -1, -1]))
        c.fork(arg([0, 0, 0]), arg([1, 2, 4]))
        c.truncate(arg([-1, -1, 70, -1, -1]))
        c.reserve(arg([0, 0, 300, 0, 0]))
        c.truncate(arg([-1, -1, 360, -1, -1]))
        c.reserve(arg([6, 6, 6, 6, 6]))
    cache.check()
    q = torch.randn((S, 6, 12, D), device="cuda").bfloat16()
    out, lse = cache.attend(0, q, shared_stream=0, shared_tokens=320)
    cache.check()
    assert_attention(out, lse, q, mem[0], mem[1], books, [6] * S, D ** -0.5)


def test_padded_positions_are_left_alone():
    used = [0, 5, 8, 1, 0, 7]
    c = Case([100, 640, 641, 0, 3000, 700], 8, 8, 2, prefix=640, seed=3)
    out = torch.full_like(c.q, 7.0)
    lse = torch.full((c.S, c.B, c.Hq), 7.0, device="cuda")
    lengths = i32(used)
    c.attend(lengths=lengths, out=out, lse=lse)
    c.check(out, lse, used=used)
    for s in range(c.S):
        assert (out[s, used[s]:] == 7).all() and (lse[s, used[s]:] == 7).all()
    out, lse = c.attend(lengths=i32([0] * c.S))
    assert not out.any() and not lse.any()
    c.attend(lengths=i32([9, 100, 8, -1, -5, 8]))      # more than the block: all of it; less than none: none


@pytest.mark.parametrize("B,prefix", [(11, 0), (64, 128), (1, 0)])
def test_tree_masks_and_empty_rows(B, prefix):
    """Masks of random bits, rows that see no block position, and, in streams without a context, nothing at all."""
    rng = random.Random(B)
    ctx = [prefix, 0, prefix + 77, 0, prefix + 200]
    c = Case(ctx, B, 4, 2, D=64, page=16, prefix=prefix, dtype=torch.float16, seed=B)
    rows = [[rng.getrandbits(B) for _ in range(B)] for _ in ctx]
    rows[1][0] = 0
    rows[0][B - 1] = 0
    rows[3] = [0] * B
    as_i64 = torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in rows], dtype=torch.int64, device="cuda")
    out, lse = c.attend(mask=as_i64)
    c.check(out, lse, mask=rows)
    assert not out[3].any() and (lse[3] == -math.inf).all()
    used = [B, max(1, B - 3), B, B // 2, 1]
    out, lse = c.attend(mask=as_i64, lengths=i32(used))
    c.check(out, lse, used=used, mask=rows)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("page,D", [(16, 64), (128, 128)])
def test_what_is_not_stored_has_no_part(fill, page, D):
    c = Case([0, 5, 130, 256, 391], 3, 8, 4, D=D, page=page, prefix=0, seed=5, fill=fill)
    c.check(*c.attend())
    c = Case([256, 261, 300, 511], 3, 8, 4, D=D, page=page, prefix=256, seed=6, fill=fill)
    c.check(*c.attend())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_keys_that_a_row_does_not_see_have_no_part(bad):
    """Non-finite keys and values at a block position: earlier positions are as without them, and later ones get what
    the sums give."""
    ctx, B = [0, 61, 126, 200], 6
    c = Case(ctx, B, 4, 2, prefix=0, seed=9)
    want, wlse = c.attend()
    for s in range(c.S):
        i, off = divmod(ctx[s] + 3, c.page)
        c.v[c.books.table[s][i], :, off, 5] = bad
    out, lse = c.attend()
    assert torch.equal(out[:, :3], want[:, :3]) and torch.equal(lse, wlse)
    keep = [d for d in range(c.D) if d != 5]
    assert torch.equal(out[..., keep], want[..., keep])
    assert torch.equal(out[:, 3:, :, 5].isnan(), torch.full_like(out[:, 3:, :, 5], math.isnan(bad), dtype=torch.bool))
    assert not out[:, 3:, :, 5].isfinite().any()
    for s in range(c.S):
        i, off = divmod(ctx[s] + 3, c.page)
        c.k[c.books.table[s][i], :, off, 7] = float("nan")
    out, lse = c.attend()
    assert torch.equal(out[:, :3], want[:, :3]) and torch.equal(lse[:, :3], wlse[:, :3])
    assert out[:, 3:].isnan().all() and lse[:, 3:].isnan().all()


@pytest.mark.parametrize("D,prefix", [(128, 0), (64, 128)])
def test_bad_values_in_blocks_of_many_rows(D, prefix):
    """Blocks whose rows fill both halves of a CTA, and several CTAs."""
    B, used = 90, [90, 33, 0, 77]
    c = Case([prefix, prefix + 100, prefix + 3, prefix + 259], B, 8, 2, D=D, page=32, prefix=prefix, seed=D)
    lengths = i32(used)
    want, wlse = c.attend(lengths=lengths)
    c.check(want, wlse, used=used)
    for s in range(c.S):
        for pos, col in ((20, 3), (76, 7), (89, 11)):
            i, off = divmod(c.books.length[s] + pos, c.page)
            c.v[c.books.table[s][i], :, off, col] = float("nan")
            c.k[c.books.table[s][i], :, off, col] = float("inf") if pos == 89 else 0.5
    base = c.v.clone()
    clean = torch.where(base.isnan(), torch.zeros_like(base), base)
    c.v.copy_(clean)
    want, wlse = c.attend(lengths=lengths)
    c.v.copy_(base)
    out, lse = c.attend(lengths=lengths)
    for s, n in enumerate(used):
        assert torch.equal(lse[s, :min(n, 89)], wlse[s, :min(n, 89)])
        for b in range(min(n, 89)):
            bad = [col for pos, col in ((20, 3), (76, 7)) if pos <= b]
            keep = [d for d in range(D) if d not in bad]
            assert torch.equal(out[s, b][:, keep], want[s, b][:, keep]), (s, b)
            assert out[s, b][:, bad].isnan().all(), (s, b)


def test_bad_values_in_many_short_blocks_that_follow_one_another():
    """Several units of more than 128 rows for every CTA, each a tile long, with a bad value in its block: each
    unit's rows get their own, in both halves, every time."""
    S, B, D, Hkv = 300, 20, 64, 2
    c = Case([(37 * s) % 90 for s in range(S)], B, 16, Hkv, D=D, page=32, seed=20)
    want, wlse = c.attend()
    at = torch.tensor([(7 * s) % B for s in range(S)], device="cuda")
    col = torch.tensor([(11 * s) % D for s in range(S)], device="cuda")
    for s in range(S):
        i, off = divmod(c.books.length[s] + int(at[s]), c.page)
        c.v[c.books.table[s][i], :, off, int(col[s])] = float("inf") if s % 3 else float("nan")
    sees = torch.arange(B, device="cuda")[None, :] >= at[:, None]
    bad = sees[:, :, None, None] & (torch.arange(D, device="cuda") == col[:, None])[:, None, None, :]
    for _ in range(20):
        out, lse = c.attend()
        assert torch.equal(lse, wlse)
        assert torch.equal(~out.isfinite(), bad.expand_as(out))
        assert torch.equal(torch.where(bad, 0, out), torch.where(bad, 0, want))


def bad_prompt(B, Hkv, D=128, every=64):
    """A prompt of B positions with a NaN at every 64th, whose rows are slow to write out; what its rows should be."""
    c = Case([0], B, Hkv, Hkv, D=D, page=128, seed=21)
    want, wlse = c.attend()
    ids = torch.tensor(c.books.table[0][:c.books.held[0]], device="cuda")
    for at in range(every // 2, B, every):
        c.v[ids[at // c.page], :, at % c.page, at // every % D] = float("nan")
    b = torch.arange(B, device="cuda")[:, None]
    last = (b + every // 2) // every - 1                     # number of the last bad value that the row sees
    bad = torch.arange(D, device="cuda")[None, :] <= last
    return c, want, wlse, bad[None, :, None, :]


def assert_bad_prompt(out, lse, want, wlse, bad):
    assert torch.equal(lse, wlse)
    assert torch.equal(out.isnan(), bad.expand_as(out))
    assert torch.equal(torch.where(bad, 0, out), torch.where(bad, 0, want))


def test_bad_values_of_a_long_prompt_are_no_reason_to_give_up():
    """Writing out rows with bad values is quick enough for the waits of the other warps, at 16384 positions too."""
    c, want, wlse, bad = bad_prompt(16384, 8)
    out, lse = c.attend()
    assert_bad_prompt(out, lse, want, wlse, bad)


@pytest.mark.parametrize("D,dtype", [(128, torch.float16), (64, torch.bfloat16)])
def test_infinities_of_both_signs_and_nan(D, dtype):
    """Every kind of bad value at random block positions and columns, under random masks: a column is what the sum of
    the bad values that the row sees is."""
    rng = random.Random(D)
    B, Hkv = 40, 2
    c = Case([0, 3, 100, 250], B, 8, Hkv, D=D, dtype=dtype, page=16, seed=22)
    rows = [[rng.getrandbits(B) | 1 << b for b in range(B)] for _ in range(c.S)]
    mask = torch.tensor(rows, dtype=torch.int64, device="cuda")
    want, wlse = c.attend(mask=mask)
    kinds = [float("inf"), -float("inf"), float("nan")]
    seen = [[[[] for _ in range(D)] for _ in range(Hkv)] for _ in range(c.S)]
    for s in range(c.S):
        for _ in range(25):
            pos, h, col, x = rng.randrange(B), rng.randrange(Hkv), rng.randrange(D), kinds[rng.choice([0, 0, 1, 1, 2])]
            i, off = divmod(c.books.length[s] + pos, c.page)
            if c.v[c.books.table[s][i], h, off, col].isfinite():
                c.v[c.books.table[s][i], h, off, col] = x
                seen[s][h][col].append((pos, x))
    out, lse = c.attend(mask=mask)
    assert torch.equal(lse, wlse)
    ref = want.cpu().clone()
    for s in range(c.S):
        for h in range(Hkv):
            for col in range(D):
                for b in range(B):
                    xs = [x for pos, x in seen[s][h][col] if rows[s][b] >> pos & 1]
                    if xs:
                        ref[s, b, 4 * h:4 * h + 4, col] = sum(xs)
    assert torch.equal(out.cpu().nan_to_num(nan=12345.0), ref.nan_to_num(nan=12345.0))


def test_a_wait_that_runs_out_is_an_error_that_the_host_reads():
    """A limit of 1 us is below what a warp waits for rows with bad values to be written out: the call ends, check()
    says why, and the next call, on a handle with the usual limit, is right."""
    c, want, wlse, bad = bad_prompt(2048, 64)
    hasty = pkg.KvCache(layers=[(c.k, c.v)], num_streams=2, max_pages=c.books.M, timeout_us=1)
    write_books(hasty, c.books)
    for _ in range(3):
        hasty.attend(0, c.q)
        with pytest.raises(pkg.MoeError) as e:
            hasty.check()
        assert e.value.status == pkg.MOE_ERR_TIMEOUT
        hasty.check()
        out, lse = c.attend()
        assert_bad_prompt(out, lse, want, wlse, bad)


def test_masks_of_one_row_leave_the_others_alone():
    """The same with a mask: a bad value is seen by the rows whose bit is set, and by no other."""
    B = 5
    c = Case([40, 125], B, 4, 2, seed=10)
    rows = [[0b00001, 0b10010, 0b00101, 0b01000, 0b10000], [0b11111, 0b00000, 0b00100, 0b01011, 0b00010]]
    mask = torch.tensor(rows, dtype=torch.int64, device="cuda")
    want, _ = c.attend(mask=mask)
    for s, n in enumerate([40, 125]):
        i, off = divmod(n + 2, c.page)
        c.v[c.books.table[s][i], :, off] = float("nan")
    out, _ = c.attend(mask=mask)
    for s in range(2):
        for b in range(B):
            if rows[s][b] >> 2 & 1:
                assert out[s, b].isnan().all()
            else:
                assert torch.equal(out[s, b], want[s, b])


def test_extreme_scores():
    """Scores far apart (the running maximum climbs tile by tile), large equal ones, and a scale of zero."""
    c = Case([700, 1029], 4, 4, 2, seed=11)
    ramp = torch.linspace(-3, 3, 1100, device="cuda")
    for s in range(c.S):
        for i in range(c.books.held[s]):
            n = i * c.page
            c.k[c.books.table[s][i]] = (ramp[n % 1000:n % 1000 + c.page, None] * torch.ones(c.D, device="cuda")).to(c.k.dtype)
    c.q.fill_(1.0)
    c.check(*c.attend())
    c.check(*c.attend(scale=0.0), scale=0.0)
    c.q.fill_(-2.0)
    c.check(*c.attend(scale=1.0), scale=1.0)


@pytest.mark.parametrize("together", [False, True])
@pytest.mark.parametrize("k0,bits", [(-2.875, 16), (-4.59375, 26), (-5.0, 28)])
def test_long_tails_of_small_terms(k0, bits, together):
    """fp16: one key at the top and 65535 whose terms are 2^-16 .. 2^-28 of its own, in parts of some hundred tiles; the
    values of all but the first are one, so that the output is the tail's weight.  Terms and output are rounded to the
    type (2^-11 relative each); a term has no more than 2^-37 of the largest as its own last half step."""
    S, n, Hkv, D, page = 40, 65536, 8, 64, 128
    mem = torch.zeros((2, n // page + S, Hkv, page, D), dtype=torch.float16, device="cuda")
    cache = pkg.KvCache(layers=[(mem[0], mem[1])], num_streams=S, max_pages=n // page + 1)
    b = Books(S, n // page + 1, n // page + S, page)
    for s in range(S):                               # all hold the same pages, and one more for the block
        b.table[s] = list(range(n // page)) + [n // page + s]
        b.held[s], b.length[s] = n // page + 1, n - 1
    write_books(cache, b)
    mem[0, :, :, :, 0] = k0
    mem[0, 0, :, 0] = 0
    mem[1] = 1
    mem[1, 0, :, 0] = 0
    q = torch.zeros((S, 4, Hkv, D), dtype=torch.float16, device="cuda")
    q[..., 0] = 4
    out, lse = cache.attend(0, q, shared_stream=0, shared_tokens=(n - page) if together else 0, scale=1.0)
    cache.check()
    term = math.exp(4 * k0)
    assert 2 ** -(bits + 1) < term < 2 ** -bits
    for i in range(4):
        tail = (n - 1 + i) * term
        want, u = tail / (1 + tail), 2.0 ** -11
        tol = 2.02 * u * want + (n + 3) * 2.0 ** -37 + 2.0 ** -25
        assert (out[:, i].double() - want).abs().max() <= tol, (want, float(out[:, i].min()), float(out[:, i].max()))
        # a sum in 32 bits of up to 512 tiles, each addition off by half a step of the sum: 512 * 2^-24; and the rest
        assert (lse[:, i].double() - math.log1p(tail)).abs().max() <= 2.0 ** -15 + 2.0 ** -20


@pytest.mark.parametrize("size", [1024, 1400, 2048, 4096, 8192])
def test_fp16_scores_in_the_millions(size):
    """Equal scores of 2^20 to 2^26, and their negatives: all terms are equal, and finite, however coarse the steps of
    the exponents are."""
    c = Case([500, 0, 129], 3, 4, 2, D=64, dtype=torch.float16, seed=24)
    c.k.fill_(0)
    c.k[..., 0] = size * 1.28125
    c.q.fill_(0)
    c.q[..., 0] = size
    c.q[2] *= -1
    out, lse = c.attend(scale=1.0)
    assert out.isfinite().all()
    x = size * c.k[0, 0, 0, 0].double() * torch.tensor([1.0, 1.0, -1.0], device="cuda")
    assert ((lse - x[:, None, None]).abs() <= x[0] * 2.0 ** -20 + 8).all()
    for s in range(3):
        n = c.books.length[s] + 3
        v = gather(c.v, c.books.table[s], c.books.held[s], c.page).double()[:, :n]
        # Weights of parts that are merged carry the steps of their lse, of half and more here, so a row is held to its
        # values' range; a row of one part has equal weights.  Its terms are rounded alike (2^-11), and the output (2^-11).
        slack = 2.0 ** -9 * v.abs().max()
        got = out[s, 2].double().view(2, 2, c.D)
        assert (got <= v.amax(1)[:, None] + slack).all() and (got >= v.amin(1)[:, None] - slack).all()
        if n <= 128:
            assert (got - v.mean(1)[:, None]).abs().max() <= slack


@pytest.mark.parametrize("scale", [0.0, 1e-40, -1e-38, 1e-36])
def test_tiny_scales_of_huge_scores(scale):
    c = Case([700, 129, 0], 4, 4, 2, seed=23)
    c.q *= 2.0 ** 54
    c.k *= 2.0 ** 54
    c.check(*c.attend(scale=scale), scale=scale)


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.float16)])
def test_the_maximum_climbs_along_a_shared_prefix(D, dtype):
    """Scores that grow by some tens along the prefix for half of the rows and fall for the others, in units that fill
    both halves of a CTA: the accumulators are rescaled many times."""
    S, prefix = 24, 12288
    c = Case([prefix + n for n in range(1, 25)], 8, 64, 8, D=D, dtype=dtype, page=64, prefix=prefix, seed=18)
    ids = torch.tensor(c.books.table[S][:prefix // c.page], device="cuda")
    ramp = torch.linspace(-20, 20, len(ids), device="cuda")[:, None, None, None]
    c.k[ids] = (c.k[ids].float() * 0.5 + ramp).to(dtype)
    out, lse = c.attend()
    c.check(out, lse, streams=[0, 11, 23])
    again, _ = c.attend()
    assert torch.equal(again, out)


def test_rows_of_a_fused_projection_and_bad_tables():
    c = Case([100, 259], 4, 4, 2, seed=12)
    want, wlse = c.attend()
    fused = torch.zeros((2, 4, 12, c.D), dtype=c.q.dtype, device="cuda")
    fused[:, :, 3:7] = c.q
    out, lse = c.cache.attend(0, fused[:, :, 3:7])
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    # entries outside the pool and fewer pages than the length says: read as if absent, no fault, others unharmed
    c.cache.page_table[0, 0] = 1 << 30
    c.cache.page_table[0, 1] = -5
    out, _ = c.cache.attend(0, c.q)
    assert torch.equal(out[1], want[1])
    c.cache.held[0] = 0
    c.cache.length[0] = 1 << 20
    out, _ = c.cache.attend(0, c.q)
    torch.cuda.synchronize()
    assert torch.equal(out[1], want[1])
    pkg.moe_mxfp4_cache_check(c.cache.handle, c.cache.state.data_ptr(), torch.cuda.current_stream().cuda_stream)


def test_prompt_blocks():
    """Long blocks (a prompt behind a shared one): causal over many row tiles, ragged."""
    used = [500, 0, 333]
    c = Case([256, 256, 300], 500, 8, 2, prefix=256, seed=13)
    out, lse = c.attend(lengths=i32(used))
    c.check(out, lse, used=used)


def test_offsets_beyond_32_bits():
    P, Hkv, page, D = 16500, 8, 128, 128
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    mem = torch.empty((2, P, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    b = Books(1, 8, P, page)
    ids = [P - 1, 0, P - 2, 16400, 3]
    mem[:, ids] = torch.randn((2, len(ids), Hkv, page, D), device="cuda").bfloat16()
    b.table[0][:5], b.held[0], b.length[0] = ids, 5, 600
    for p in ids:
        b.ref[p] = 1
    cache = pkg.KvCache(layers=[(mem[0], mem[1])], num_streams=1, max_pages=8)
    write_books(cache, b)
    q = torch.randn((1, 4, 16, D), device="cuda").bfloat16()
    out, lse = cache.attend(0, q)
    cache.check()
    assert_attention(out, lse, q, mem[0], mem[1], b, [4], D ** -0.5)


def test_graph_replay_follows_the_books_and_repeats_bit_for_bit():
    c = Case([256, 700, 300], 8, 8, 2, prefix=256, seed=14)
    out, lse = c.attend()
    out2, lse2 = c.attend()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        gout, glse = c.cache.attend(0, c.q, shared_stream=c.S, shared_tokens=256)
    with torch.cuda.stream(side):
        g.replay()
    side.synchronize()
    assert torch.equal(gout, out) and torch.equal(glse, lse)
    c.cache.truncate(i32([256, 440, 299, 256]))        # shorter streams (with other pages), the same graph
    c.books.truncate([256, 440, 299, 256])
    c.cache.reserve(i32([8, 8, 8, 0]))
    c.books.reserve([8, 8, 8, 0])
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    c.check(gout, glse)


def test_calls_that_overlap_on_two_streams():
    c = Case([700, 3000, 1200, 90], 8, 16, 2, prefix=64, seed=16)
    c2 = Case([500, 64, 2000], 5, 8, 4, prefix=64, seed=17)
    want = [x.clone() for case in (c, c2) for x in case.attend()]
    streams = [torch.cuda.Stream() for _ in range(2)]
    q2 = c.q.flip(0).contiguous()
    flipped = [x.clone() for x in c.cache.attend(0, q2, shared_stream=c.S, shared_tokens=64)]
    ws = [torch.empty(c.cache.attend_bytes(c.S, c.B, c.Hq), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for k, q in ((0, c.q), (1, q2)):
            with torch.cuda.stream(streams[k]):
                got.append((k, c.cache.attend(0, q, shared_stream=c.S, shared_tokens=64, workspace=ws[k])))
        with torch.cuda.stream(streams[1]):
            got.append((2, c2.cache.attend(0, c2.q, shared_stream=c2.S, shared_tokens=64)))
    torch.cuda.synchronize()
    for k, (out, lse) in got:
        ref = (want[0], want[1]) if k == 0 else tuple(flipped) if k == 1 else (want[2], want[3])
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1]), k


def test_outputs_belong_to_the_stream_of_the_call():
    """attend(stream=...) while torch's current stream is busy: the fills of the outputs do not wait for that one, and
    no later fill reaches them."""
    c = Case([700, 90, 0, 300], 8, 16, 2, prefix=64, seed=19)
    used = i32([8, 3, 0, 8])
    want, wlse = c.attend(lengths=used)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)              # some 10 ms on the current stream
        got = [c.cache.attend(0, c.q, lengths=used, shared_stream=c.S, shared_tokens=64, stream=side.cuda_stream),
               c.cache.attend(0, c.q, lengths=used, shared_stream=c.S, shared_tokens=64, stream=side.cuda_stream)]
        side.synchronize()
        early = [(out.cpu(), lse.cpu()) for out, lse in got]
        torch.cuda.synchronize()
        for (out, lse), (e, el) in zip(got, early):
            assert torch.equal(out, want) and torch.equal(lse, wlse)
            assert torch.equal(e, want.cpu()) and torch.equal(el, wlse.cpu())
    out, lse = c.cache.attend(0, c.q, lengths=used, shared_stream=c.S, shared_tokens=64, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_a_verify_forward_from_reserve_to_commit():
    """The calls as a user makes them: streams fork from a prompt, and blocks are reserved, appended, attended, judged
    by accept() and committed; the attention then equals that over contiguous keys."""
    torch.manual_seed(0)
    S, B, Hq, Hkv, D, page, V = 5, 4, 8, 2, 64, 16, 50
    mem = torch.zeros((2, 2, 60, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    c = pkg.KvCache(layers=[(mem[i, 0], mem[i, 1]) for i in range(2)], num_streams=S + 1, max_pages=12)
    prompt = 37
    c.reserve(i32([0] * S + [prompt]))
    pk, pv = torch.randn((2, 1, prompt, Hkv, D), device="cuda").bfloat16()
    allk, allv = [pk[0].clone() for _ in range(S)], [pv[0].clone() for _ in range(S)]
    slot = torch.zeros((S + 1, prompt, Hkv, D), dtype=torch.bfloat16, device="cuda")
    slot[S] = pk[0]
    slotv = torch.zeros_like(slot)
    slotv[S] = pv[0]
    for layer in range(2):
        c.append(layer, slot, slotv, lengths=i32([0] * S + [prompt]))
    c.commit(i32([0] * S + [prompt]))
    c.fork(i32([S] * S), i32(list(range(S))))
    shared = prompt // page * page
    for step in range(9):
        c.reserve(i32([B] * S + [0]))
        k, v = torch.randn((2, S, B, Hkv, D), device="cuda").bfloat16()
        q = torch.randn((S, B, Hq, D), device="cuda").bfloat16()
        for layer in range(2):
            c.append(layer, k, v)
            out, lse = c.attend(layer, q, shared_stream=S, shared_tokens=shared)
        logits = torch.randn((S, B, V), device="cuda")
        target = logits.argmax(-1).int()
        tokens = torch.zeros((S, B), dtype=torch.int32, device="cuda")
        tokens[:, 1:] = target[:, :-1]
        tokens[step % S, 1 + step % (B - 1):] = -1     # one stream's drafts fail early
        _, acc, _ = pkg.accept(logits, tokens)
        for s in range(S):
            kk, vv = torch.cat([allk[s], k[s]]), torch.cat([allv[s], v[s]])
            flat = Books(1, 1, 1, kk.shape[0])
            flat.table, flat.held, flat.length = [[0]], [1], [allk[s].shape[0]]
            assert_attention(out[s:s + 1], lse[s:s + 1], q[s:s + 1], kk.transpose(0, 1)[None], vv.transpose(0, 1)[None],
                             flat, [B], D ** -0.5)
            n = int(acc[s])
            allk[s], allv[s] = torch.cat([allk[s], k[s, :n]]), torch.cat([allv[s], v[s, :n]])
        c.commit(torch.cat([acc, torch.zeros(1, dtype=torch.int32, device="cuda")]))
        if step == 4:
            c.compact()
        c.check()
    for s in range(S):
        n = allk[s].shape[0]
        assert c.length[s].item() == n
        assert torch.equal(gather(mem[1, 0], c.page_table[s].tolist(), c.held[s].item(), page)[:, :n], allk[s].transpose(0, 1))


def test_the_loop_around_a_moe_layer_eager_and_captured():
    """A whole step (reserve, append, attend, the MoE layer, accept, commit) with one slot for each stream of the batch,
    whose prefix the first one holds: three steps one by one, and as replays of one graph, with the same bits."""
    torch.manual_seed(3)
    S, B, Hq, Hkv, D, page, V = 4, 4, 8, 2, 64, 16, 64
    wl = Workload("loop", T=S * B, H=512, I=512, E=8, k=2, seed=0x5EED0400)
    _, layers = device_layers(wl)
    moe = pkg.MoeLayers(hidden=wl.H, inter=wl.I, num_experts=wl.E, top_k=wl.k, max_tokens=wl.T, layers=layers)
    wq, wk, wv = (0.1 * torch.randn((wl.H, n * D), device="cuda").bfloat16() for n in (Hq, Hkv, Hkv))
    wo, head = 0.1 * torch.randn((Hq * D, wl.H), device="cuda").bfloat16(), torch.randn((wl.H, V), device="cuda")
    prompt = torch.randn((1, 40, wl.H), device="cuda").bfloat16()
    xs = torch.randn((3, S, B, wl.H), device="cuda").bfloat16()
    tokens = torch.randint(0, 3, (3, S, B), device="cuda").int()       # (few drafts are right)

    def begin():
        mem = torch.zeros((1, 2, 60, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
        c = pkg.KvCache(layers=[(mem[0, 0], mem[0, 1])], num_streams=S, max_pages=12)
        c.reserve(i32([40] + [0] * (S - 1)))
        c.append(0, (prompt @ wk).view(1, 40, Hkv, D), (prompt @ wv).view(1, 40, Hkv, D))
        c.commit(i32([40] + [0] * (S - 1)))
        c.fork(i32([0] * (S - 1)), i32(list(range(1, S))))
        return mem, c

    def step(c, x, drafts):
        c.reserve(B)
        c.append(0, (x @ wk).view(S, B, Hkv, D), (x @ wv).view(S, B, Hkv, D))
        out, lse = c.attend(0, (x @ wq).view(S, B, Hq, D), shared_stream=0, shared_tokens=32)
        h = x + (out.view(S, B, Hq * D) @ wo)
        logits = (h.float() + moe.forward(h.view(S * B, wl.H)).view(S, B, wl.H)) @ head
        target, accepted, next_token = pkg.accept(logits, drafts)
        c.commit(accepted)
        return out, lse, logits, target, accepted

    mem, c = begin()
    want = [[t.clone() for t in step(c, x, d)] + [c.length.clone()] for x, d in zip(xs, tokens)]
    c.check()
    assert c.length.tolist() == [40 + sum(int(w[4][s]) for w in want) for s in range(S)]
    mem2, c2 = begin()
    x, d, side, g = xs[0].clone(), tokens[0].clone(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    step(begin()[1], x, d)                            # workspaces and libraries are set up outside the capture
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        got = step(c2, x, d)
    for i in range(3):
        x.copy_(xs[i])
        d.copy_(tokens[i])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([*got, c2.length], want[i])), i
    c2.check()
    assert torch.equal(mem, mem2)


def test_refusals():
    c = Case([10, 20], 4, 4, 2, seed=15)
    q, cache = c.q, c.cache
    for call in (lambda: cache.attend(0, q.half()), lambda: cache.attend(0, q[..., :64]), lambda: cache.attend(0, q[0]),
                 lambda: cache.attend(0, q, out=q[:1]), lambda: cache.attend(0, q, lse=torch.zeros(3, device="cuda")),
                 lambda: cache.attend(0, q, mask=torch.zeros((2, 4), dtype=torch.int32, device="cuda")),
                 lambda: cache.attend(0, q, lengths=i32([1])), lambda: cache.attend(0, q.transpose(1, 2))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: cache.attend(1, q), lambda: cache.attend(0, q[:, :, :3]),
                 lambda: cache.attend(0, q, shared_tokens=65), lambda: cache.attend(0, q, shared_tokens=-64),
                 lambda: cache.attend(0, q, shared_tokens=64, shared_stream=3),
                 lambda: cache.attend(0, q, shared_tokens=64 * 1000), lambda: cache.attend(0, q, scale=float("nan")),
                 lambda: cache.attend(0, torch.zeros((2, 65, 4, 128), dtype=q.dtype, device="cuda"),
                                      mask=torch.zeros((2, 65), dtype=torch.int64, device="cuda")),
                 lambda: cache.attend(0, torch.zeros((4, 1, 4, 128), dtype=q.dtype, device="cuda"))):
        with pytest.raises(pkg.MoeError) as e:
            call()
        assert e.value.status == pkg.MOE_ERR_INVALID_ARG
    with pytest.raises(pkg.MoeError) as e:
        cache.attend(0, q, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.status == pkg.MOE_ERR_WORKSPACE
    out, lse = cache.attend(0, q[:0])
    assert out.numel() == 0 and lse.numel() == 0
