"""GPU tests of the edits of logits and of the acceptance of chains and trees with them, against 64 bits."""
import math
import os
import random

import pytest
import torch

import mxfp4_moe_expert_gb300 as pkg
from forward_util import TINY, U, edit_reference, pack_allowed, random_trees, targets_of, to_mask, walk

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


def f32(x):
    return torch.tensor(x, dtype=torch.float32, device="cuda")


class Case:
    """A batch with everything that edits it, on the GPU and in the plain form."""

    def __init__(self, S, B, V, dtype=torch.float32, seed=0, tree=False, ragged=False, what="hpbgt", hist=40, bias=6, extra=0, margin=True):
        rng, g = random.Random(seed), torch.Generator().manual_seed(seed)
        self.S, self.B, self.V = S, B, V
        x = 3 * torch.randn((S, B, V), generator=g)
        token = lambda: min(V - 1, int(V ** rng.random()) - 1 + rng.randrange(2))   # noqa: E731
        self.masks = random_trees(S, B, rng) if tree else None
        self.lengths = [rng.choice([0, B, rng.randint(0, B)]) for _ in range(S)] if ragged else None
        tokens = [[token() for _ in range(B)] for _ in range(S)]
        if margin:                       # a winner that no rounding decides on, often the next drafted token
            for s in range(S):
                for b in range(B):
                    x[s, b, token()] += 30 + rng.random()
                for b in range(1, B):
                    up = (self.masks[s][b] & ((1 << b) - 1)).bit_length() - 1 if tree else b - 1
                    if rng.random() < 0.7:
                        x[s, up, tokens[s][b]] += 60 + 20 * rng.random()
        self.logits = x.to(dtype)
        on = dict(tokens=i32(tokens))
        plain = dict(tokens=tokens, masks=self.masks, lengths=self.lengths)
        if tree:
            on["mask"] = to_mask(self.masks).cuda()
        if ragged:
            on["lengths"] = i32(self.lengths)
        if "h" in what:
            n = [rng.choice([0, 1, hist, rng.randint(0, hist)]) for _ in range(S)]
            history = [[rng.choice([token(), token(), -1, V, V + 7]) for _ in range(hist)] for _ in range(S)]
            on.update(history=i32(history).view(S, hist), history_lengths=i32(n))
            plain["history"] = [h[:k] for h, k in zip(history, n)]
            if "p" in what:
                plain["prompt"] = [rng.randint(0, k) for k in n]
                on["prompt_lengths"] = i32(plain["prompt"])
            for name, value in (("repetition", lambda: 1 + rng.random()), ("frequency", rng.random), ("presence", lambda: rng.random() - 0.5)):
                plain[name] = torch.tensor([value() for _ in range(S)]).tolist()
                on[name] = f32(plain[name])
        if "b" in what:
            lists = [[(rng.choice([token(), token(), -3, V]), round(rng.uniform(-4, 4), 3)) for _ in range(rng.choice([0, 1, bias]))] for _ in range(S)]
            plain["bias"] = [[(t, float(torch.tensor(v))) for t, v in x] for x in lists]
            begin = [0]
            for x in lists:
                begin.append(begin[-1] + len(x))
            flat = [e for x in lists for e in x]
            on["bias"] = (i32(begin), i32([t for t, _ in flat]), f32([v for _, v in flat]))
        self.allowed = None
        if "g" in what:
            kinds = [None, set(), {token()}, {token() for _ in range(20)}, set(range(V)) - {token()},
                     {t for t in range(V) if rng.random() < 0.5}, {t for t in range(V) if rng.random() < 0.9}]
            self.allowed = [[rng.choice(kinds) for _ in range(B)] for _ in range(S)]
            on["allowed"] = pack_allowed(self.allowed, S, B, V, extra).cuda()
            plain["allowed"] = self.allowed
        self.on, self.plain = on, plain
        self.z, self.err = edit_reference(self.logits, **plain)

    def used(self, s):
        return self.B if self.lengths is None else max(0, min(self.B, self.lengths[s]))

    def check_edit(self, out, unused=0.0):
        got, z, u = out.cpu().double(), self.z, U[self.logits.dtype]
        for s in range(self.S):
            n = self.used(s)
            assert (out[s, n:] == unused).all()
            a, b = got[s, :n], z[s, :n]
            assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a == -math.inf, b == -math.inf)
            assert torch.equal(a == math.inf, b == math.inf)
            fine = torch.isfinite(b)
            tol = 1.01 * u * b[fine].abs() + 1.01 * self.err[s, :n][fine] + TINY[self.logits.dtype]
            assert ((a[fine] - b[fine]).abs() <= tol).all(), s

    def check_accept(self, got):
        target = targets_of(self.z, self.allowed, self.lengths)
        accepted, nxt, paths = walk(target, self.plain["tokens"], self.masks, self.lengths)
        assert [t.tolist() for t in got] == [target, accepted, nxt, paths]


CASES = [dict(S=3, B=5, V=77), dict(S=2, B=4, V=5000, tree=True), dict(S=4, B=1, V=4096), dict(S=2, B=3, V=4097, ragged=True),
         dict(S=1, B=8, V=9001, tree=True), dict(S=5, B=2, V=1), dict(S=3, B=6, V=33, tree=True, ragged=True), dict(S=1, B=64, V=300, tree=True),
         dict(S=2, B=130, V=100), dict(S=2, B=3, V=12288, hist=700, bias=300), dict(S=40, B=2, V=600, extra=3), dict(S=2, B=2, V=8192, bias=3000),
         dict(S=1, B=1, V=20000, hist=9000), dict(S=3, B=4, V=16384 + 8), dict(S=2, B=5, V=6000, what="hb"), dict(S=2, B=3, V=5001, what="g"),
         dict(S=3, B=3, V=4444, what="b"), dict(S=2, B=9, V=1000, what="t"), dict(S=2, B=4, V=7000, what="h", ragged=True)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kw", CASES)
def test_edits_and_acceptance(kw, dtype):
    c = Case(**kw, dtype=dtype, seed=kw["V"])
    x = c.logits.cuda()
    out = pkg.edit_logits(x, **c.on)
    c.check_edit(out)
    assert torch.equal(x.cpu(), c.logits)
    c.check_accept(pkg.accept_edited(x, **c.on))
    assert pkg.edit_logits(x, out=x, **c.on) is x                              # in place
    for s in range(c.S):
        n = c.used(s)
        assert torch.equal(x[s, :n], out[s, :n]) or torch.equal(torch.isnan(x[s, :n]), torch.isnan(out[s, :n]))
        assert torch.equal(x[s, n:].cpu(), c.logits[s, n:])
    if c.lengths is not None:                                                  # rows behind are left as they were
        y = torch.full_like(out, 7.0)
        c.check_edit(pkg.edit_logits(c.logits.cuda(), out=y, **c.on), unused=7.0)


@pytest.mark.parametrize("dtype,kw", [
    (torch.bfloat16, dict(S=100, B=17, V=9000)), (torch.float32, dict(S=100, B=17, V=9001, what="hpbt")),
    (torch.float16, dict(S=60, B=40, V=8192 + 40, ragged=True, tree=True)), (torch.bfloat16, dict(S=60, B=40, V=8192, ragged=True, what="hpt")),
    (torch.float32, dict(S=150, B=64, V=4104, tree=True, what="hpbt")), (torch.bfloat16, dict(S=30, B=300, V=4099, what="hpt"))])
def test_many_positions_of_a_stream_at_once(kw, dtype):
    """Batches whose CTAs take several positions: groups that end with the block, tokens that only some of them see."""
    c = Case(**kw, dtype=dtype, seed=kw["S"])
    x = c.logits.cuda()
    c.check_edit(pkg.edit_logits(x, **c.on))
    c.check_accept(pkg.accept_edited(x, **c.on))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,room,skip", [(1000, 1000, 0), (1000, 1024, 0), (999, 1003, 0), (4100, 4120, 1), (4096, 4097, 3), (515, 520, 5)])
def test_rows_of_any_stride_and_alignment(V, room, skip, dtype):
    c = Case(S=3, B=4, V=V, dtype=dtype, seed=V, extra=1)
    mem = torch.full((12 * room + skip,), 5.0, dtype=dtype, device="cuda")
    x = mem[skip:].view(3, 4, room)[..., :V]
    x.copy_(c.logits)
    c.check_accept(pkg.accept_edited(x, **c.on))
    c.check_edit(pkg.edit_logits(x, **c.on))
    other = torch.full((12 * (room + 3) + 1,), 6.0, dtype=dtype, device="cuda")
    y = other[1:].view(3, 4, room + 3)[..., :V]
    c.check_edit(pkg.edit_logits(x, out=y, **c.on))
    pkg.edit_logits(x, out=x, **c.on)
    c.check_edit(x)
    assert (mem[:skip] == 5).all() and (mem[skip:].view(3, 4, room)[..., V:] == 5).all()
    assert other[0] == 6 and (other[1:].view(3, 4, room + 3)[..., V:] == 6).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_values_that_are_not_finite_ties_and_zeros(dtype):
    V = 6000
    x = torch.zeros((1, 9, V), dtype=dtype)
    x[0, 0, 70] = math.nan                                # NaN ranks as -inf: the first of the zeros wins
    x[0, 1] = -math.inf                                   # all equal: the lowest
    x[0, 2, 5000], x[0, 2, 4999] = 3, 3                   # ties across and within runs
    x[0, 3, 10], x[0, 3, 4096] = math.inf, math.inf
    x[0, 4] = -0.0
    x[0, 4, 77] = 0.0                                     # -0 and +0 are equal: the lowest
    x[0, 5] = math.nan
    x[0, 6] = -5.0                                        # a NaN that is allowed, and not the only one
    x[0, 6, 3] = math.nan
    x[0, 7] = torch.finfo(dtype).min                      # the lowest value is a value
    x[0, 7, 12] = -math.inf
    allowed = [[None] * 9]
    allowed[0][6] = {3, 8}
    allowed[0][7] = {12, 4500}
    allowed[0][8] = set()
    on = dict(allowed=pack_allowed(allowed, 1, 9, V).cuda())
    tokens = torch.zeros((1, 9), dtype=torch.int32, device="cuda")
    target = pkg.accept_edited(x.cuda(), tokens, **on)[0]
    assert target.tolist() == [[0, 0, 4999, 10, 0, 0, 8, 4500, -1]]
    z, _ = edit_reference(x, allowed=allowed)
    got = pkg.edit_logits(x.cuda(), **on).cpu().double()
    assert torch.equal(torch.nan_to_num(got, nan=99.0), torch.nan_to_num(z, nan=99.0))


def test_without_edits_it_is_the_plain_acceptance():
    S, B, V = 7, 6, 10007
    x = torch.randn((S, B, V), device="cuda")
    tokens = torch.randint(0, V, (S, B), dtype=torch.int32, device="cuda")
    want = pkg.accept(x, tokens)
    tokens[:, 1:] = torch.where(torch.rand((S, B - 1), device="cuda") < 0.8, want[0][:, :-1], tokens[:, 1:])
    want = pkg.accept(x, tokens)
    got = pkg.accept_edited(x, tokens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    i = torch.arange(B, device="cuda")
    assert torch.equal(got[3], torch.where(i < got[1][:, None], i, -1).int())


def test_what_is_accepted_is_the_largest_edited_logit():
    """Both entry points round alike: the target is where the edited logits, as fp32 writes them, are largest."""
    for seed in range(3):
        c = Case(S=6, B=5, V=50000, seed=seed, tree=True, margin=False)
        x = c.logits.cuda()
        z = pkg.edit_logits(x, **c.on)
        target = pkg.accept_edited(x, **c.on)[0]
        v = torch.arange(c.V, device="cuda")
        want = torch.where((z == z.amax(-1, keepdim=True)) & (z > -math.inf), v, c.V).amin(-1)
        assert torch.equal(target, torch.where(want == c.V, -1, want).int())


def test_many_repeats_of_one_token_and_long_histories():
    V, n = 5000, 70000
    x = torch.randn((2, 1, V), device="cuda")
    history = torch.full((2, n), 4321, dtype=torch.int32, device="cuda")
    history[1, ::2] = 4999
    tokens = i32([[4321], [7]])
    got = pkg.edit_logits(x, tokens, history=history, history_lengths=i32([n, n + 5]), prompt_lengths=i32([0, 100]),
                          frequency=f32([2.0 ** -10, 2.0 ** -10]), presence=f32([0.0, 0.5]))
    want = x.clone().double()
    want[0, 0, 4321] -= (n + 1) * 2.0 ** -10
    for t in (4321, 4999):
        want[1, 0, t] -= (n // 2 - 50) * 2.0 ** -10 + 0.5
    want[1, 0, 7] -= 2.0 ** -10 + 0.5
    assert ((got.double() - want).abs() <= 3 * 2.0 ** -24 * (want.abs() + 70)).all()


def test_lengths_beyond_the_history_and_the_biases_are_cut():
    """A view of a wider history is read as far as it goes; so are the entries of the biases."""
    V = 50
    x = torch.zeros((2, 1, V), device="cuda")
    wide = i32([[1, 2, 3, 4, 5, 6], [7, 8, 9, 10, 11, 12]])
    got = pkg.edit_logits(x, history=wide[:, 2:4], history_lengths=i32([6, 100]), presence=f32([1.0, 1.0]),
                          bias=(i32([-3, 1, 9]), i32([20, 21]), f32([4.0, 5.0])))
    want = torch.zeros((2, 1, V))
    want[0, 0, 3] = want[0, 0, 4] = want[1, 0, 9] = want[1, 0, 10] = -1
    want[0, 0, 20], want[1, 0, 21] = 4, 5
    assert torch.equal(got.cpu(), want)


def test_offsets_beyond_32_bits():
    """Positions whose elements, and bytes, lie beyond 2^31 of the tensor's start."""
    S, B, V, stride = 2, 5, 5003, (1 << 28) + 3
    c = Case(S=S, B=B, V=V, dtype=torch.bfloat16, seed=11, tree=True)
    x = torch.empty((S * B - 1) * stride + V, dtype=torch.bfloat16, device="cuda").as_strided((S, B, V), (B * stride, stride, 1))
    x.copy_(c.logits)
    c.check_accept(pkg.accept_edited(x, **c.on))
    c.check_edit(pkg.edit_logits(x, **c.on))
    pkg.edit_logits(x, out=x, **c.on)
    c.check_edit(x)


def test_on_another_stream_in_a_graph_and_with_a_workspace():
    c = Case(S=4, B=6, V=30000, seed=3, tree=True)
    x = c.logits.cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = pkg.edit_logits(x, stream=side.cuda_stream, **c.on)
    got = pkg.accept_edited(x, stream=side.cuda_stream, **c.on)
    side.synchronize()
    c.check_edit(out)
    c.check_accept(got)
    st, n = pkg.moe_mxfp4_accept_edited_bytes(c.S, c.B, c.V)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    c.check_accept(pkg.accept_edited(x, workspace=ws, **c.on))
    with pytest.raises(pkg.MoeError):
        pkg.accept_edited(x, workspace=ws[:-1], **c.on)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pkg.accept_edited(x, **c.on)
        out = pkg.edit_logits(x, **c.on)
    for _ in range(3):
        for t in got:
            t.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        c.check_accept(got)
        c.check_edit(out)


def test_two_calls_at_once():
    cases = [Case(S=8, B=6, V=20000, seed=s, tree=s % 2 == 0) for s in range(2)]
    xs = [c.logits.cuda() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(5):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(pkg.accept_edited(xs[i], **c.on))
    torch.cuda.synchronize()
    for c, g in zip(cases, got):
        for x in g:
            c.check_accept(x)


def test_two_captured_graphs_and_a_given_workspace():
    """Graphs whose calls make their workspaces do not share them; one that is given serves calls one after the other."""
    cases = [Case(S=5, B=6, V=9000, seed=s, tree=s == 1) for s in range(2)]
    xs = [c.logits.cuda() for c in cases]
    ws = torch.empty(max(pkg.moe_mxfp4_accept_edited_bytes(5, 6, 9000)[1], 8), dtype=torch.uint8, device="cuda")
    for given in (None, ws):
        graphs, got = [], []
        for c, x in zip(cases, xs):
            pkg.accept_edited(x, workspace=given, **c.on)
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                got.append(pkg.accept_edited(x, workspace=given, **c.on))
        for i in (0, 1, 1, 0):
            graphs[i].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for c, g in zip(cases, got):
            c.check_accept(g)


def test_empty_batches():
    x = torch.zeros((0, 3, 50), device="cuda")
    tokens = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    assert pkg.edit_logits(x, tokens).shape == (0, 3, 50)
    assert [t.shape[0] for t in pkg.accept_edited(x, tokens)] == [0] * 4


def test_the_binding_refuses_wrong_tensors():
    x, t = torch.zeros((2, 3, 50), device="cuda"), torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    one = torch.zeros(2, dtype=torch.int32, device="cuda")
    h = torch.zeros((2, 9), dtype=torch.int32, device="cuda")
    bad = [dict(mask=torch.zeros((3, 2), dtype=torch.int64, device="cuda")), dict(allowed=torch.zeros((3, 2, 2), dtype=torch.int32, device="cuda")),
           dict(mask=t), dict(mask=torch.zeros((2, 3), dtype=torch.int64)), dict(lengths=one.long()), dict(lengths=one[:1]), dict(history=h),
           dict(history_lengths=one), dict(prompt_lengths=one), dict(history=h.long(), history_lengths=one),
           dict(history=h[:1], history_lengths=one), dict(history=h.T, history_lengths=one), dict(repetition=one),
           dict(history=h[:1].expand(2, 9), history_lengths=one), dict(frequency=torch.zeros(3, device="cuda")),
           dict(bias=(one, one, torch.zeros(2, device="cuda"))), dict(allowed=torch.zeros((2, 3, 1), dtype=torch.int32, device="cuda")),
           dict(allowed=torch.zeros((2, 3, 2), dtype=torch.int64, device="cuda"))]
    for kw in bad:
        with pytest.raises(ValueError):
            pkg.edit_logits(x, t, **kw)
        with pytest.raises(ValueError):
            pkg.accept_edited(x, t, **kw)
    for out in (torch.zeros((2, 3, 49), device="cuda"), x.half(), x.cpu()):
        with pytest.raises(ValueError):
            pkg.edit_logits(x, t, out=out)
    for tokens in (t[:1], t.T.contiguous(), t.view(6)):
        with pytest.raises(ValueError):
            pkg.edit_logits(x, tokens)
    with pytest.raises(ValueError):
        pkg.edit_logits(x.long(), t)
    with pytest.raises(ValueError):
        pkg.accept_edited(x, t, workspace=torch.zeros(1000, dtype=torch.uint8))
