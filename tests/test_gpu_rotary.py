"""GPU tests of the norms and the rotation of queries and keys, on their own and on the way into the cache, against 64 bits."""
import os
import random

import pytest
import torch

import mxfp4_moe_expert_gb300 as pkg
from cache_util import Books, assert_attention, assert_books, write_books
from forward_util import assert_rounded, depth, frequencies, random_trees, rotate_reference, to_mask

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


def weights(D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2)]


SCALINGS = [None, dict(kind="linear", factor=8.0), dict(kind="ntk", factor=4.0),
            dict(kind="parts", factor=16.0, original=4096.0, low=1.0, high=32.0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,R", [(64, 64), (128, 128), (128, 64), (64, 16), (128, 32), (128, 96), (64, 48), (64, 0), (64, 2),
                                 (128, 20), (64, 30), (128, 126), (64, 62), (128, 8), (64, 24)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [0, 1, 2, 3])                 # none, weights, ones, weights of the queries alone
def test_every_layout(dtype, D, R, inter, norm):
    g = torch.Generator().manual_seed(D + R)
    N, Hq, Hkv = 7, 5, 3
    w = weights(D, dtype)
    q_w, k_w = (w if norm == 1 else (w[0], None) if norm == 3 else (None, None))
    r = pkg.Rotary(head_dim=D, rotary_dim=R, interleaved=inter, gain=1.0 if norm else 1.25, q_norm=q_w, k_norm=k_w,
                   norm=norm > 0, eps=1e-5, dtype=dtype, device="cuda")
    q, k = ((3 * torch.randn((N, H, D), generator=g)).to(dtype).cuda() for H in (Hq, Hkv))
    q[2, 1] = 0                                                # a head of zeros stays zero
    pos = i32([0, 1, 5, 131071, -3, 2 ** 31 - 1, -2 ** 31])
    got = r.rotate(q, k, pos)
    for x, y, weight in ((q, got[0], q_w), (k, got[1], k_w)):
        want, err = rotate_reference(x, pos, frequencies(R), inter, 1.0 if norm else 1.25, norm > 0, weight, 1e-5)
        assert_rounded(y, want, err)
    assert not got[0][2, 1].any()


@pytest.mark.parametrize("scaling", SCALINGS)
def test_scaled_frequencies_at_far_positions(scaling):
    D, N = 128, 33
    r = pkg.Rotary(head_dim=D, base=500000.0, scaling=scaling, dtype=torch.float16, device="cuda")
    q = torch.randn((N, 2, D), dtype=torch.float16, device="cuda")
    pos = i32([2 ** 20 + 1717 * i for i in range(N)])
    want, err = rotate_reference(q, pos, frequencies(D, 500000.0, scaling))
    assert_rounded(r.rotate(q, None, pos)[0], want, err)


def test_given_frequencies():
    f = [0.0, 1.0, -0.5, 3.0, 1e-9] + [0.25] * 27
    r = pkg.Rotary(head_dim=64, frequencies=f, interleaved=True, dtype=torch.float16, device="cuda")
    q = torch.randn((9, 3, 64), dtype=torch.float16, device="cuda")
    pos = i32(list(range(9)))
    want, err = rotate_reference(q, pos, f, True)
    assert_rounded(r.rotate(q, None, pos)[0], want, err)


@pytest.mark.parametrize("N,Hq,Hkv", [(1, 1, 0), (1, 0, 1), (1, 56, 8), (3, 7, 1), (2000, 2, 1), (701, 33, 5), (40000, 1, 1), (5, 300, 17), (70001, 1, 0),
                                      (9999, 3, 1), (30001, 5, 2)])
@pytest.mark.parametrize("D,R", [(128, 128), (64, 32), (64, 34), (128, 90)])
def test_sizes(N, Hq, Hkv, D, R):
    """Few and many tokens, few and many heads; tokens of a wider tensor; two leading dimensions."""
    dtype = torch.bfloat16
    x = torch.randn((N, Hq + Hkv + 2, D), dtype=dtype, device="cuda")
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    w = weights(D, dtype, 3)
    pos = torch.randint(0, 100000, (N,), dtype=torch.int32, device="cuda")
    r = pkg.Rotary(head_dim=D, rotary_dim=R, q_norm=w[0], k_norm=w[1], dtype=dtype, device="cuda")
    out = r.rotate(q, k, pos)
    pick = torch.tensor(sorted({0, N - 1, N // 2, N // 3}))
    for t, y, weight in ((q, out[0], w[0]), (k, out[1], w[1])):
        want, err = rotate_reference(t[pick.cuda()], pos[pick.cuda()], frequencies(R), norm=True, w=weight)
        assert_rounded(y[pick.cuda()], want, err)
    again = x.clone()
    r.rotate(again[:, :Hq], again[:, Hq:Hq + Hkv], pos, again[:, :Hq], again[:, Hq:Hq + Hkv])      # in place
    assert torch.equal(again[:, :Hq], out[0]) and torch.equal(again[:, Hq:Hq + Hkv], out[1])
    assert torch.equal(again[:, Hq + Hkv:], x[:, Hq + Hkv:])
    if N % 5 == 0:
        two = r.rotate(q.unflatten(0, (5, N // 5)), k.unflatten(0, (5, N // 5)), pos.view(5, N // 5))
        assert two[0].shape == (5, N // 5, Hq, D) and torch.equal(two[0].flatten(0, 1), out[0]) and torch.equal(two[1].flatten(0, 1), out[1])


def test_nothing_to_rotate():
    r = pkg.Rotary(head_dim=64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((0, 3, 64), dtype=torch.bfloat16, device="cuda")
    assert r.rotate(q, q, i32([]))[0].shape == (0, 3, 64)
    q = torch.zeros((4, 0, 64), dtype=torch.bfloat16, device="cuda")
    assert r.rotate(q, None, i32([0, 1, 2, 3]))[0].shape == (4, 0, 64)


def test_values_that_are_not_finite_stay_in_their_head():
    r = pkg.Rotary(head_dim=64, norm=True, dtype=torch.bfloat16, device="cuda")
    q = torch.randn((4, 6, 64), dtype=torch.bfloat16, device="cuda")
    pos = i32([1, 2, 3, 4])
    clean = r.rotate(q, None, pos)[0]
    q[1, 2, 5], q[2, 3, 60], q[3, 0, 0] = float("nan"), float("inf"), -float("inf")
    got = r.rotate(q, None, pos)[0]
    for t, h in ((1, 2), (2, 3), (3, 0)):
        assert got[t, h].isnan().any()
        got[t, h] = clean[t, h]
    assert torch.equal(got, clean)


def test_offsets_beyond_32_bits():
    """Rows whose elements, and bytes, lie beyond 2^31 of the tensor's start."""
    D, H, N, stride = 64, 2, 9, 1 << 28
    x = torch.empty((N - 1) * stride + H * D, dtype=torch.float16, device="cuda").as_strided((N, H, D), (stride, D, 1))
    for t in range(N):
        x[t] = torch.randn((H, D), device="cuda").half()
    r = pkg.Rotary(head_dim=D, dtype=torch.float16, device="cuda")
    pos = i32(list(range(100, 100 + N)))
    want = r.rotate(x.contiguous(), None, pos)[0]
    assert torch.equal(r.rotate(x, None, pos)[0], want)
    r.rotate(x, None, pos, x)
    assert torch.equal(x.contiguous(), want)


def test_on_another_stream_and_in_a_graph():
    r = pkg.Rotary(head_dim=128, norm=True, dtype=torch.bfloat16, device="cuda")
    q, k = torch.randn((50, 8, 128), device="cuda").bfloat16(), torch.randn((50, 2, 128), device="cuda").bfloat16()
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    want = r.rotate(q, k, pos)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = r.rotate(q, k, pos, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = [torch.zeros_like(t) for t in (q, k)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.rotate(q, k, pos, *out)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        pos += 7
        want = r.rotate(q, k, pos)
        torch.cuda.synchronize()


def test_two_calls_at_once():
    r = pkg.Rotary(head_dim=128, norm=True, dtype=torch.bfloat16, device="cuda")
    xs = [torch.randn((3000, 9, 128), device="cuda").bfloat16() for _ in range(2)]
    pos = [torch.arange(3000, dtype=torch.int32, device="cuda") + 1000 * i for i in range(2)]
    want = [r.rotate(x, None, p)[0] for x, p in zip(xs, pos)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[r.rotate(x, None, p, stream=s.cuda_stream)[0] for _ in range(4)] for x, p, s in zip(xs, pos, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(t, w) for t in g)


def test_the_binding_refuses_wrong_tensors():
    r = pkg.Rotary(head_dim=64, dtype=torch.bfloat16, device="cuda")
    q, pos = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda"), i32([0, 1, 2, 3])
    for a in ((q.half(), None, pos), (q.cpu(), None, pos), (q, q[:3], pos), (q, None, pos[:3]), (q, None, pos.long()),
              (q, None, pos.cpu()), (q, None, i32(list(range(8)))[::2]), (q, None, pos, q[:3]), (q, None, pos, torch.zeros_like(q).half())):
        with pytest.raises(ValueError):
            r.rotate(*a)


# ------------------------------------------------------------------------------------------- into the cache


def make(L=2, S=5, M=6, P=30, Hkv=2, page=16, D=64, dtype=torch.bfloat16, seed=0, room=8):
    """A cache that holds some tokens, with room for `room` more in every stream, and its plain twin."""
    g = torch.Generator().manual_seed(seed)
    host = torch.randn((L, 2, P, Hkv, page, D), generator=g).to(dtype)
    mem = host.cuda()
    c = pkg.KvCache(layers=[(mem[i, 0], mem[i, 1]) for i in range(L)], num_streams=S, max_pages=M)
    b = Books(S, M, P, page, host)
    rng = random.Random(seed)
    assert b.reserve([min(M * page - room, rng.choice([0, 1, page - 1, page, 3 * page + 5])) for _ in range(S)])
    most = M * page - room
    b.length = [min(most, rng.randint(b.held[s] * page - page + 1, b.held[s] * page)) if b.held[s] else 0 for s in range(S)]
    write_books(c, b)
    return c, mem, b


def status(c):
    return pkg.moe_mxfp4_cache_check(c.handle, c.state.data_ptr(), torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("kw,B,Hq,R,inter,norm,tree,ragged", [
    (dict(), 8, 4, 64, False, True, False, False), (dict(dtype=torch.float16, page=32, Hkv=1), 3, 8, 32, True, False, False, True),
    (dict(D=128, Hkv=3, page=64, M=4), 11, 6, 128, False, True, True, False), (dict(D=128, Hkv=8, dtype=torch.float16), 1, 56, 64, True, True, False, False),
    (dict(S=3, page=128, M=3, Hkv=5), 64, 5, 20, False, False, True, True), (dict(S=2, M=40, P=90), 300, 2, 64, True, True, False, True),
    (dict(S=1, D=128, Hkv=2), 1, 0, 128, False, True, False, False), (dict(S=5, M=20, P=110, Hkv=1), 64, 2, 64, False, True, True, True),
    (dict(S=4, D=128, M=20, P=90, Hkv=1), 100, 0, 20, False, False, False, True), (dict(S=2, M=20, P=50, Hkv=1), 200, 0, 64, True, True, False, False),
    (dict(S=3, M=20, P=70, Hkv=1, dtype=torch.float16), 90, 1, 64, False, True, False, True), (dict(S=5, Hkv=33, M=4), 7, 33, 50, True, True, True, True)])
def test_a_block_on_its_way_into_the_cache(kw, B, Hq, R, inter, norm, tree, ragged):
    c, mem, b = make(**kw, seed=B, room=B)
    S, D, Hkv, dtype, L = b.S, c.head_dim, c.kv_heads, c.dtype, c.num_layers
    rng = random.Random(B)
    used = [rng.choice([0, B, rng.randint(0, B)]) for _ in range(S)] if ragged else [B] * S
    masks = random_trees(S, B, rng) if tree else None
    w = weights(D, dtype, 1) if norm else [None, None]
    r = pkg.Rotary(head_dim=D, rotary_dim=R, interleaved=inter, q_norm=w[0], k_norm=w[1], dtype=dtype, device="cuda")
    assert b.reserve(used)
    c.reserve(i32(used))
    before = mem.clone()
    for layer in range(L):
        x = torch.randn((S, B, Hq + 2 * Hkv, D), device="cuda").to(dtype)
        q, k, v = x.split([Hq, Hkv, Hkv], 2)
        out = c.append_rotated(layer, q if Hq else None, k, v, r, mask=None if masks is None else to_mask(masks).cuda(),
                               lengths=i32(used) if ragged else None)
        assert status(c) == pkg.MOE_OK and (out is None) == (Hq == 0)
        for s in range(S):
            n = used[s]
            if out is not None:
                assert not out[s, n:].any()
            pos = torch.tensor([b.length[s] + (depth(masks[s][i], i) if tree else i) for i in range(n)], dtype=torch.int32)
            if n == 0:
                continue
            if Hq:
                assert_rounded(out[s, :n], *rotate_reference(q[s, :n], pos, frequencies(R), inter, 1.0, norm, w[0]))
            want, err = rotate_reference(k[s, :n], pos, frequencies(R), inter, 1.0, norm, w[1])
            for i in range(n):
                at, off = divmod(b.length[s] + i, b.page)
                p = b.table[s][at]
                assert_rounded(mem[layer, 0, p, :, off], want[i], err[i])
                assert torch.equal(mem[layer, 1, p, :, off], v[s, i])
                before[layer, :, p, :, off] = mem[layer, :, p, :, off]
    assert torch.equal(mem.view(torch.int16), before.view(torch.int16))    # nothing else was touched
    b.pool = None
    assert_books(c, b)
    c.close()


def test_alone_and_into_the_cache_give_the_same_bits():
    c, mem, b = make(D=128, Hkv=4)
    S, B, Hq = b.S, 6, 8
    c.reserve(B); b.reserve([B] * S)
    w = weights(128, c.dtype)
    r = pkg.Rotary(head_dim=128, q_norm=w[0], k_norm=w[1], dtype=c.dtype, device="cuda")
    q, k, v = (torch.randn((S, B, H, 128), device="cuda").to(c.dtype) for H in (Hq, 4, 4))
    out = c.append_rotated(0, q, k, v, r)
    pos = (c.length[:, None] + torch.arange(B, device="cuda", dtype=torch.int32)).int().contiguous()
    rq, rk = r.rotate(q, k, pos)
    assert torch.equal(out, rq)
    c.append(1, rk, v)
    used = [b.table[s][(b.length[s] + i) // b.page] for s in range(S) for i in range(B)]
    assert torch.equal(mem[0, 0, used][..., :0], mem[1, 0, used][..., :0])
    for s in range(S):
        for i in range(B):
            at, off = divmod(b.length[s] + i, b.page)
            assert torch.equal(mem[0, :, b.table[s][at], :, off], mem[1, :, b.table[s][at], :, off])
    q2 = q.clone()
    assert c.append_rotated(0, q2, k, v, r, out=q2) is q2 and torch.equal(q2, out)      # in place
    c.close()


def test_pages_beyond_32_bits():
    """Pages whose elements lie beyond 2^31 of the pool's start: appending into them, and moving a path there."""
    S, M, P, Hkv, page, D, B = 2, 3, 10, 2, 16, 64, 12
    stride = (1 << 28) + 8
    pools = [torch.empty((P - 1) * stride + Hkv * page * D, dtype=torch.bfloat16, device="cuda").as_strided(
        (P, Hkv, page, D), (stride, page * D, D, 1)) for _ in range(2)]
    c = pkg.KvCache(layers=[tuple(pools)], num_streams=S, max_pages=M)
    b = Books(S, M, P, page)
    b.length, b.held = [13, 30], [2, 3]
    b.table, b.ref = [[9, 8, -1], [1, 7, 6]], [0, 1, 0, 0, 0, 0, 1, 1, 1, 1]
    write_books(c, b)
    r = pkg.Rotary(head_dim=D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.randn((S, B, Hkv, D), device="cuda").bfloat16() for _ in range(2))
    c.append_rotated(0, None, k, v, r)
    path = [[0, 2, 3, 5, 11], [1, 2, 4, 8, 9]]
    pos = (c.length[:, None] + torch.arange(B, device="cuda", dtype=torch.int32)).int().contiguous()
    rk = r.rotate(k, None, pos)[0]
    c.commit(i32([5, 5]), path=i32([p + [-1] * (B - 5) for p in path]))
    assert status(c) == pkg.MOE_OK and c.length.tolist() == [18, 35]
    for s in range(S):
        for i, x in enumerate(path[s]):
            at, off = divmod(b.length[s] + i, page)
            assert torch.equal(pools[0][b.table[s][at], :, off], rk[s, x]) and torch.equal(pools[1][b.table[s][at], :, off], v[s, x])
    c.close()


def test_positions_that_are_not_reserved_or_shared_are_skipped():
    """The queries are rotated all the same; the first error is kept."""
    c, mem, b = make(S=4, P=30, M=4)
    b = Books(4, 4, 30, 16)
    b.reserve([40, 20, 16, 0])
    b.length = [40, 20, 16, 0]
    b.ref[b.table[1][1]] = 2                       # stream 1's last page is shared
    write_books(c, b)
    r = pkg.Rotary(head_dim=64, dtype=c.dtype, device="cuda")
    B = 4
    q, k, v = (torch.randn((4, B, H, 64), device="cuda").to(c.dtype) for H in (4, 2, 2))
    before = mem.clone()
    out = c.append_rotated(0, q, k, v, r)
    assert status(c) == pkg.MOE_ERR_CACHE_STATE and status(c) == pkg.MOE_OK
    pos = (c.length[:, None] + torch.arange(B, device="cuda", dtype=torch.int32)).int().contiguous()
    assert torch.equal(out, r.rotate(q, None, pos)[0])
    for i in range(B):                             # stream 0 has room in its last page (48 tokens held)
        at, off = divmod(40 + i, 16)
        before[0, :, b.table[0][at], :, off] = mem[0, :, b.table[0][at], :, off]
        assert torch.equal(mem[0, 1, b.table[0][at], :, off], v[0, i])
    assert torch.equal(mem, before)
    c.table_was = c.page_table.clone()
    c.page_table[0, 2] = 10 ** 6                   # an entry outside the pool
    c.append_rotated(0, q[:1], k[:1], v[:1], r)
    assert status(c) == pkg.MOE_ERR_CACHE_STATE
    assert torch.equal(mem, before)
    c.close()


def test_append_rotated_refuses():
    c, mem, b = make(S=4)
    q, k, v = (torch.zeros((4, 3, H, 64), dtype=c.dtype, device="cuda") for H in (4, 2, 2))
    r = pkg.Rotary(head_dim=64, dtype=c.dtype, device="cuda")
    for other in (pkg.Rotary(head_dim=128, dtype=c.dtype, device="cuda"), pkg.Rotary(head_dim=64, dtype=torch.float16, device="cuda")):
        with pytest.raises(pkg.MoeError):
            c.append_rotated(0, q, k, v, other)
    with pytest.raises(pkg.MoeError):
        c.append_rotated(2, q, k, v, r)
    with pytest.raises(ValueError):
        c.append_rotated(0, q, k, v, pkg.Rotary(head_dim=64, dtype=c.dtype, device="cpu"))
    with pytest.raises(ValueError):
        c.append_rotated(0, q[:3], k, v, r)
    with pytest.raises(ValueError):
        c.append_rotated(0, q, k, v, r, out=q[..., :32])
    with pytest.raises(ValueError):
        c.append_rotated(0, None, k, v, r, out=q)
    with pytest.raises(ValueError):
        c.append_rotated(0, q, k, v, r, mask=torch.zeros((4, 2), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        c.append_rotated(0, q, k, v, r, lengths=i32([1, 1, 1]))
    long = [torch.zeros((1, 65, H, 64), dtype=c.dtype, device="cuda") for H in (4, 2, 2)]
    with pytest.raises(pkg.MoeError):
        c.append_rotated(0, *long, r, mask=torch.zeros((1, 65), dtype=torch.int64, device="cuda"))
    assert status(c) == pkg.MOE_OK
    c.close()


# ------------------------------------------------------------------------------------------- accepted paths


def paths_of(masks, rng):
    """A random path from the root of each tree."""
    out = []
    for row in masks:
        node = rng.randrange(len(row))
        out.append([i for i in range(len(row)) if (row[node] >> i) & 1])
    return out


@pytest.mark.parametrize("kw,B,streams", [(dict(), 8, 5), (dict(D=128, Hkv=8, page=32, L=3), 40, 4), (dict(Hkv=1, dtype=torch.float16), 2, 5),
                                          (dict(Hkv=5, page=128, M=3, L=1), 64, 3), (dict(L=130, Hkv=1, P=20, M=4), 9, 5),
                                          (dict(S=300, M=5, P=1500, L=1, Hkv=1), 5, 297)])
@pytest.mark.parametrize("history", [False, True])
def test_accepted_paths_are_moved_together(kw, B, streams, history):
    c, mem, b = make(**kw, seed=B, room=B)
    S, page = b.S, b.page
    rng = random.Random(B)
    assert b.reserve([B] * S)
    c.reserve(B)
    masks = random_trees(streams, B, rng)
    paths = paths_of(masks, rng)
    accepted = [len(p) for p in paths] + [rng.choice([0, 1, -1]) for _ in range(S - streams)]
    accepted[0] = 0                                      # a whole block is dropped, ...
    if streams > 2:
        accepted[1] = -1                                 # ... a stream left alone
    table = torch.tensor([p + [-1] * (B - len(p)) for p in paths])
    tokens = torch.randint(0, 1000, (streams, B), dtype=torch.int32)
    room = max(b.length) + B
    said = torch.randint(0, 1000, (streams, room), dtype=torch.int32)
    dev = said.cuda()
    c.commit(i32(accepted), path=table.int().cuda(), tokens=tokens.cuda() if history else None, history=dev if history else None)
    assert status(c) == pkg.MOE_OK
    for s in range(streams):
        for i in range(max(0, accepted[s])):
            (a, x), (d, y) = divmod(b.length[s] + paths[s][i], page), divmod(b.length[s] + i, page)
            b.pool[:, :, b.table[s][d], :, y] = b.pool[:, :, b.table[s][a], :, x]
            said[s, b.length[s] + i] = tokens[s, paths[s][i]]
    b.truncate([b.length[s] + n if n >= 0 else -1 for s, n in enumerate(accepted)])
    assert_books(c, b)
    assert torch.equal(mem.cpu().view(torch.int16), b.pool.view(torch.int16))
    if history:
        assert torch.equal(dev.cpu(), said)
    c.close()


@pytest.mark.parametrize("D,Hkv,page", [(64, 3, 16), (128, 2, 32)])
def test_long_paths_move_by_any_distance(D, Hkv, page):
    """Paths of more positions than are looked up at once, over many pages, whose moves overlap: each node goes to where
    another one came from."""
    B = 64
    paths = [[0] + list(range(2, B)), list(range(5, B)), list(range(B)), [B - 1], list(range(0, B, 2)), list(range(1, B)),
             [0, 1, 2] + list(range(31, B)), list(range(32)) + list(range(33, B))]
    c, mem, b = make(L=2, S=len(paths), M=10, P=90, Hkv=Hkv, page=page, D=D, room=B)
    assert b.reserve([B] * b.S)
    c.reserve(B)
    c.commit(i32([len(p) for p in paths]), path=i32([p + [-1] * (B - len(p)) for p in paths]))
    assert status(c) == pkg.MOE_OK
    for s, path in enumerate(paths):
        for i, x in enumerate(path):
            (a, x), (d, y) = divmod(b.length[s] + x, page), divmod(b.length[s] + i, page)
            b.pool[:, :, b.table[s][d], :, y] = b.pool[:, :, b.table[s][a], :, x]
    b.truncate([b.length[s] + len(p) for s, p in enumerate(paths)])
    assert_books(c, b)
    assert torch.equal(mem.cpu().view(torch.int16), b.pool.view(torch.int16))
    c.close()


def test_a_history_without_a_path():
    c, mem, b = make()
    b.reserve([4] * b.S)
    c.reserve(4)
    tokens, said = torch.randint(0, 9, (3, 4), dtype=torch.int32), torch.zeros((3, 200), dtype=torch.int32)
    dev = said.cuda()
    acc = [2, 4, 0, 1, 3]
    c.commit(i32(acc), tokens=tokens.cuda(), history=dev)
    for s in range(3):
        said[s, b.length[s]:b.length[s] + acc[s]] = tokens[s, :acc[s]]
    b.truncate([b.length[s] + n for s, n in enumerate(acc)])
    assert status(c) == pkg.MOE_OK
    assert_books(c, b)
    assert torch.equal(dev.cpu(), said) and torch.equal(mem.cpu(), b.pool)
    c.close()


@pytest.mark.parametrize("wrong", ["order", "twice", "negative", "beyond", "long", "unreserved", "shared", "history", "outside"])
def test_paths_that_are_refused_leave_their_stream_alone(wrong):
    c, mem, b = make(S=3, M=6)
    S, B, page = 3, 6, b.page
    b = Books(3, 6, 30, page, mem.cpu())
    b.reserve([20, 30, 9])
    b.length = [20, 30, 9]
    b.reserve([B] * S)
    path, accepted, room = [[0, 2, 3, -1, -1, -1] for _ in range(S)], [3, 3, 3], 64
    t = 1                                                # the stream that is at fault
    if wrong == "order":
        path[t] = [0, 3, 2, -1, -1, -1]
    elif wrong == "twice":
        path[t] = [0, 2, 2, -1, -1, -1]
    elif wrong == "negative":
        path[t] = [0, 2, -1, 3, 4, 5]
    elif wrong == "beyond":
        path[t] = [0, 2, 6, -1, -1, -1]
    elif wrong == "long":
        accepted[t] = 7
    elif wrong == "unreserved":
        path[t], b.length[t] = [0, 2, 5, -1, -1, -1], b.held[t] * page - 5
    elif wrong == "shared":
        b.ref[b.table[t][b.length[t] // page]] = 2
    elif wrong == "history":
        room = 32
    write_books(c, b)
    if wrong == "outside":
        c.page_table[t, b.length[t] // page] = -5
    tokens, said = torch.randint(0, 9, (S, B), dtype=torch.int32), torch.full((S, room), -7, dtype=torch.int32)
    dev = said.cuda()
    c.commit(i32(accepted), path=i32(path), tokens=tokens.cuda(), history=dev)
    state = torch.zeros(2, dtype=torch.int32)
    state.copy_(c.state[:2])
    assert state.tolist() == [pkg.MOE_ERR_CACHE_STATE, t]
    assert status(c) == pkg.MOE_ERR_CACHE_STATE
    if wrong == "outside":
        c.page_table[t, b.length[t] // page] = b.table[t][b.length[t] // page]
    for s in (0, 2):
        for i in range(3):
            (a, x), (d, y) = divmod(b.length[s] + path[s][i], page), divmod(b.length[s] + i, page)
            b.pool[:, :, b.table[s][d], :, y] = b.pool[:, :, b.table[s][a], :, x]
            said[s, b.length[s] + i] = tokens[s, path[s][i]]
    b.truncate([b.length[0] + 3, -1, b.length[2] + 3])
    assert_books(c, b)
    assert torch.equal(mem.cpu(), b.pool) and torch.equal(dev.cpu(), said)
    c.close()


@pytest.mark.parametrize("first", [[-5, -3, 2], [-2, -1, 0], [-20, -19, -18], [-1, 0, 1], [-1 << 31, -1 << 30, 0]])
def test_paths_that_begin_below_the_block_are_refused(first):
    """Ascending all the same.  The other streams' paths are kept."""
    c, mem, b = make(S=3, M=6)
    S, B, page = 3, 6, b.page
    b = Books(3, 6, 30, page, mem.cpu())
    b.reserve([20, 30, 9])
    b.length = [20, 30, 9]
    b.reserve([B] * S)
    write_books(c, b)
    path = [[0, 2, 3, -1, -1, -1], first + [-1] * 3, [0, 2, 3, -1, -1, -1]]
    c.commit(i32([3, 3, 3]), path=i32(path))
    assert c.state[:2].tolist() == [pkg.MOE_ERR_CACHE_STATE, 1]
    assert status(c) == pkg.MOE_ERR_CACHE_STATE
    for s in (0, 2):
        for i in range(3):
            (a, x), (d, y) = divmod(b.length[s] + path[s][i], page), divmod(b.length[s] + i, page)
            b.pool[:, :, b.table[s][d], :, y] = b.pool[:, :, b.table[s][a], :, x]
    b.truncate([b.length[0] + 3, -1, b.length[2] + 3])
    assert_books(c, b)
    assert torch.equal(mem.cpu(), b.pool)
    c.close()


def test_commit_refuses_wrong_tensors():
    c, mem, b = make()
    path = i32([[0, 1]] * 5)
    acc = i32([0] * 5)
    for kw in (dict(path=path.long()), dict(path=path[:, :1].expand(5, 2)), dict(path=i32([[0]] * 6)), dict(tokens=path),
               dict(history=path), dict(path=path, history=path), dict(path=path, tokens=path[:4], history=path),
               dict(path=path, tokens=path, history=path[:4]), dict(path=path, tokens=path, history=path.long()),
               dict(path=path.cpu()), dict(path=path, tokens=path)):
        with pytest.raises(ValueError):
            c.commit(acc, **kw)
    c.close()


# ------------------------------------------------------------------------------------------- together


@pytest.mark.parametrize("captured", [False, True])
def test_a_verify_loop_with_trees(captured):
    """Blocks of drafted trees through rotation, cache, attention, acceptance and the accepted path, eagerly and as one
    captured graph: what the cache holds afterwards is what the accepted tokens would have stored one after the other."""
    g = torch.Generator().manual_seed(5)
    S, B, Hq, Hkv, D, page, V, M = 3, 7, 4, 2, 64, 16, 40, 12
    dtype = torch.bfloat16
    pools = torch.zeros((2, S * M + 2, Hkv, page, D), dtype=dtype, device="cuda")
    c = pkg.KvCache(layers=[(pools[0], pools[1])], num_streams=S, max_pages=M)
    w = weights(D, dtype)
    r = pkg.Rotary(head_dim=D, rotary_dim=32, q_norm=w[0], k_norm=w[1], dtype=dtype, device="cuda")
    embed = torch.randn((V, (Hq + 2 * Hkv) * D), generator=g).to(dtype).cuda()
    head = torch.randn((Hq * D, V), generator=g).cuda()
    history = torch.full((S, M * page), -1, dtype=torch.int32, device="cuda")
    penalty = [torch.full((S,), x, device="cuda") for x in (1.2, 0.3, 0.4)]
    tokens, mask = torch.zeros((S, B), dtype=torch.int32, device="cuda"), torch.zeros((S, B), dtype=torch.int64, device="cuda")
    out = {}

    def step():
        c.reserve(B)
        x = embed[tokens.long()].view(S, B, -1, D)
        q, k, v = x.split([Hq, Hkv, Hkv], 2)
        rq = c.append_rotated(0, q, k, v, r, mask=mask)
        o, lse = c.attend(0, rq, mask=mask)
        logits = (o.float().view(S, B, -1) @ head).contiguous()
        target, accepted, nxt, path = pkg.accept_edited(logits, tokens, mask=mask, history=history, history_lengths=c.length,
                                                        repetition=penalty[0], frequency=penalty[1], presence=penalty[2])
        c.commit(accepted, path=path, tokens=tokens, history=history)
        out.update(rq=rq, o=o, lse=lse, logits=logits, target=target, accepted=accepted, next=nxt, path=path)

    rng = random.Random(7)
    said = [[] for _ in range(S)]
    last = [3, 5, 8]
    graph = None
    for turn in range(8):
        masks = random_trees(S, B, rng)
        toks = [[last[s]] + [rng.randrange(4) for _ in range(B - 1)] for s in range(S)]
        tokens.copy_(i32(toks))
        mask.copy_(to_mask(masks).cuda())
        if captured and turn == 1:
            keep = [t.clone() for t in (c.state, pools, history)]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for t, was in zip((c.state, pools, history), keep):
                assert torch.equal(t, was)
        if graph is not None:
            graph.replay()
        else:
            step()
        assert status(c) == pkg.MOE_OK
        for s in range(S):
            n, path = int(out["accepted"][s]), out["path"][s].tolist()
            assert n >= 1 and path[0] == 0 and path[n:] == [-1] * (B - n)
            for a, p in zip(path, path[1:n]):
                assert masks[s][p] & ((1 << p) - 1) == masks[s][a] and toks[s][p] == int(out["target"][s, a])
            said[s] += [toks[s][p] for p in path[:n]]
            last[s] = int(out["next"][s])
            assert last[s] == int(out["target"][s, path[n - 1]])
            assert history[s, :len(said[s])].tolist() == said[s]
        assert c.length.tolist() == [len(x) for x in said]
    for s in range(S):
        ids = torch.tensor(said[s], device="cuda")
        k = embed[ids].view(len(ids), -1, D)[:, Hq:Hq + Hkv]
        v = embed[ids].view(len(ids), -1, D)[:, Hq + Hkv:]
        want, err = rotate_reference(k, torch.arange(len(ids), dtype=torch.int32), frequencies(32), norm=True, w=w[1])
        for t in range(len(ids)):
            p = int(c.page_table[s, t // page])
            assert_rounded(pools[0, p, :, t % page], want[t], err[t])
            assert torch.equal(pools[1, p, :, t % page], v[t])
    c.close()
