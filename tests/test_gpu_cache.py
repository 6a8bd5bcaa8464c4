"""GPU tests of the paged cache's books and pages, against the plain definitions: integers and moved bytes are equal."""
import os
import random

import pytest
import torch

import mxfp4_moe_expert_gb300 as pkg
from cache_util import Books, assert_books, ceil_div, write_books

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(pkg.LIB_PATH):
        from mxfp4_moe_expert_gb300 import build
        build.build()
    pkg.load_library()


def make(L=2, S=6, M=7, P=24, Hkv=2, page=16, D=64, dtype=torch.bfloat16, interleaved=True, seed=0):
    """A cache over pools [L, 2, P, ...] (interleaved: K and V pages alternate in memory), and its plain twin."""
    g = torch.Generator().manual_seed(seed)
    host = torch.randn((L, 2, P, Hkv, page, D), generator=g).to(dtype)
    if interleaved:
        mem = torch.empty((L, P, 2, Hkv, page, D), dtype=dtype, device="cuda").transpose(1, 2)
    else:
        mem = torch.empty((L, 2, P, Hkv, page, D), dtype=dtype, device="cuda")
    mem.copy_(host)
    c = pkg.KvCache(layers=[(mem[i, 0], mem[i, 1]) for i in range(L)], num_streams=S, max_pages=M)
    return c, mem, Books(S, M, P, page, host)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status(c):
    return pkg.moe_mxfp4_cache_check(c.handle, c.state.data_ptr(), torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("kw,seed", [
    (dict(), 1), (dict(page=32, D=128, Hkv=3, interleaved=False), 2), (dict(page=64, S=1, P=9, L=1), 3),
    (dict(page=128, D=128, dtype=torch.float16, Hkv=1, L=3), 4), (dict(S=70, P=300, M=9, page=16, L=1), 5)])
def test_any_sequence_of_calls_keeps_the_books(kw, seed):
    c, mem, b = make(**kw, seed=seed)
    rng = random.Random(seed)
    S, L = b.S, mem.shape[0]
    for step in range(60):
        op = rng.choice(["block", "block", "truncate", "fork", "compact"])
        if op == "block":
            B = rng.choice([1, 3, b.page, b.page + 5])
            add = [rng.choice([0, B, B, rng.randint(0, B)]) for _ in range(S)]
            ok = b.reserve(add)
            if rng.random() < 0.3 and len(set(add)) == 1:
                c.reserve(add[0])
            else:
                c.reserve(i32(add))
            assert status(c) == (pkg.MOE_OK if ok else status_of_refusal(b, add))
            if ok:
                k, v = (torch.randn((S, B, mem.shape[3], mem.shape[5])).to(mem.dtype) for _ in range(2))
                for layer in range(L):
                    c.append(layer, k.cuda(), v.cuda(), lengths=i32(add))
                    b.append(k, v, layer, add)
                acc = [rng.randint(0, n) for n in add]
                c.commit(i32(acc))
                b.truncate([b.length[s] + acc[s] for s in range(S)])
        elif op == "truncate":
            new = [rng.choice([-1, 0, b.length[s] // 2, b.length[s]]) for s in range(S)]
            c.truncate(i32(new))
            b.truncate(new)
        elif op == "fork":
            empty = [s for s in range(S) if not b.held[s]]
            full = [s for s in range(S) if b.held[s]]
            if empty and full:
                dst = rng.sample(empty, rng.randint(1, len(empty)))
                src = [rng.choice(full) for _ in dst]
                c.fork(i32(src), i32(dst))
                b.fork(src, dst)
        else:
            c.compact()
            b.compact()
        assert status(c) == pkg.MOE_OK
        b.consistent()
        assert_books(c, b)
        assert torch.equal(mem.cpu().view(torch.int16), b.pool.view(torch.int16)), (step, op)
    c.close()


@pytest.mark.parametrize("S,P,seed", [(1100, 5000, 1), (2100, 9000, 2)])
def test_books_of_more_streams_and_pages_than_one_pass(S, P, seed):
    """More streams than a planning CTA has threads, and more pages than it looks at in one pass; copies included."""
    c, mem, b = make(L=1, S=S, M=6, P=P, Hkv=1, page=16, D=64, seed=seed)
    rng = random.Random(seed)
    for step in range(14):
        add = [rng.choice([0, 0, 3, 16, 40]) for _ in range(S)]
        ok = b.reserve(add)
        c.reserve(i32(add))
        assert status(c) == (pkg.MOE_OK if ok else status_of_refusal(b, add)), step
        if ok:
            acc = [rng.randint(0, n) for n in add]
            c.commit(i32(acc))
            b.truncate([b.length[s] + acc[s] for s in range(S)])
        new = [rng.choice([-1, -1, 0, b.length[s] // 2, b.length[s]]) for s in range(S)]
        c.truncate(i32(new))
        b.truncate(new)
        empty = [s for s in range(S) if not b.held[s]]
        full = [s for s in range(S) if b.held[s]]
        if full and empty:
            dst = rng.sample(empty, rng.randint(1, len(empty)))
            src = [rng.choice(full[:20]) for _ in dst]       # many holders of a page, many writers of it next
            c.fork(i32(src), i32(dst))
            b.fork(src, dst)
        if step % 4 == 3:
            c.compact()
            b.compact()
        assert status(c) == pkg.MOE_OK
        b.consistent()
        assert_books(c, b)
    assert torch.equal(mem.cpu().view(torch.int16), b.pool.view(torch.int16))


def status_of_refusal(b, add):
    over = any(n > 0 and b.length[s] + n > b.M * b.page for s, n in enumerate(add))
    return pkg.MOE_ERR_CACHE_STATE if over else pkg.MOE_ERR_CACHE_FULL


def test_reserve_is_all_or_nothing():
    c, mem, b = make(S=4, M=8, P=10, page=16, L=1)
    c.reserve(32)
    assert b.reserve([32] * 4)
    c.commit(i32([32] * 4))
    b.truncate([32] * 4)
    c.reserve(16)                                  # 4 pages wanted, 2 free
    assert not b.reserve([16] * 4)
    assert c.state[1].item() == 4 and status(c) == pkg.MOE_ERR_CACHE_FULL and status(c) == pkg.MOE_OK
    assert_books(c, b)
    c.reserve(i32([0, 8 * 16, 0, 1]))              # stream 1 would pass its table
    assert c.state[1].item() == 1
    with pytest.raises(pkg.MoeError) as e:
        c.check()
    assert e.value.status == pkg.MOE_ERR_CACHE_STATE
    assert_books(c, b)
    c.reserve(i32([0, 16, 16, 0]))                 # exactly what is left
    assert b.reserve([0, 16, 16, 0]) and status(c) == pkg.MOE_OK
    assert_books(c, b)
    c.reserve(i32([-5, 0, 0, 0]))
    c.reserve(0)
    assert status(c) == pkg.MOE_OK
    assert_books(c, b)


def test_copy_on_write_keeps_the_page_for_its_last_writers_first():
    c, mem, b = make(S=5, M=4, P=12, page=16, L=1)
    c.reserve(i32([20, 0, 0, 0, 0])); b.reserve([20, 0, 0, 0, 0])
    c.truncate(i32([20, -1, -1, -1, -1])); b.truncate([20, -1, -1, -1, -1])
    c.fork(i32([0, 0, 0]), i32([3, 1, 2])); b.fork([0, 0, 0], [3, 1, 2])
    c.reserve(i32([0, 1, 0, 1, 0])); b.reserve([0, 1, 0, 1, 0])       # two of four holders write: both copy
    assert_books(c, b)
    c.reserve(i32([1, 0, 1, 0, 0])); b.reserve([1, 0, 1, 0, 0])       # the other two: the first keeps the page
    assert_books(c, b)
    assert b.table[0][1] != b.table[2][1] and b.ref[b.table[0][1]] == 1
    assert torch.equal(mem.cpu(), b.pool) and status(c) == pkg.MOE_OK


def test_append_refuses_what_is_not_its_own():
    c, mem, b = make(S=4, M=3, P=8, page=16, L=1)
    c.reserve(i32([16, 16, 0, 0])); b.reserve([16, 16, 0, 0])
    c.truncate(i32([8, 16, -1, -1])); b.truncate([8, 16, -1, -1])
    c.fork(i32([0]), i32([2])); b.fork([0], [2])
    k, v = torch.randn((2, 4, 16, 2, 64)).bfloat16().cuda()
    c.append(0, k, v, lengths=i32([4, 0, 0, 0]))   # shared with stream 2: skipped
    assert c.state[:2].tolist() == [pkg.MOE_ERR_CACHE_STATE, 0] and status(c) == pkg.MOE_ERR_CACHE_STATE
    c.append(0, k, v, lengths=i32([0, 1, 0, 0]))   # not reserved
    assert c.state[:2].tolist() == [pkg.MOE_ERR_CACHE_STATE, 1] and status(c) == pkg.MOE_ERR_CACHE_STATE
    c.page_table[1, 0] = 8                          # a page outside the pool
    c.length[1] = 3
    c.append(0, k, v, lengths=i32([0, 1, 0, 0]))
    assert status(c) == pkg.MOE_ERR_CACHE_STATE
    c.page_table[1, 0] = -7
    c.append(0, k, v, lengths=i32([0, 1, 0, 0]))
    c.reserve(i32([0, 1, 0, 0]))
    assert status(c) == pkg.MOE_ERR_CACHE_STATE
    c.append(0, k, v, lengths=i32([-3, 0, 0, 0]))
    c.append(0, k[:0], v[:0])
    c.append(0, k[:, :0], v[:, :0])
    assert status(c) == pkg.MOE_OK
    torch.cuda.synchronize()
    assert torch.equal(mem.cpu(), b.pool)


@pytest.mark.parametrize("src,dst,detail", [([0], [1], 0), ([0, 0], [2, 2], None), ([2], [2], 0), ([0, 2], [2, 3], 1),
                                            ([9], [2], 0), ([0, 0], [2, 4], 1), ([-1], [2], 0)])
def test_fork_refusals_change_nothing(src, dst, detail):
    c, mem, b = make(S=4, M=3, P=8, L=1)
    for x in (c, b):
        args = [17, 5, 0, 0]
        x.reserve(args if x is b else i32(args))
        x.truncate(args if x is b else i32(args))
    c.fork(i32(src), i32(dst))
    if detail is not None:
        assert c.state[1].item() == detail
    assert status(c) == pkg.MOE_ERR_CACHE_STATE
    assert_books(c, b)
    c.fork(i32([0]), i32([3])); b.fork([0], [3])    # and the next call works
    assert status(c) == pkg.MOE_OK
    assert_books(c, b)


def test_truncate_refuses_what_is_not_held():
    c, mem, b = make(S=3, M=3, P=8, L=1)
    c.reserve(20); b.reserve([20] * 3)
    new = [33, 32, -2]
    c.truncate(i32(new)); b.truncate(new)
    assert c.state[:2].tolist() == [pkg.MOE_ERR_CACHE_STATE, 0] and status(c) == pkg.MOE_ERR_CACHE_STATE
    assert_books(c, b)
    c.commit(i32([2 ** 31 - 1, 1, 1]))
    assert status(c) == pkg.MOE_ERR_CACHE_STATE
    b.truncate([-1, -1, 1])
    assert_books(c, b)


def test_compact_of_an_empty_a_full_and_a_packed_pool():
    c, mem, b = make(S=2, M=6, P=6, L=1)
    c.compact(); b.compact()
    assert_books(c, b)
    c.reserve(48); b.reserve([48, 48])
    c.truncate(i32([48, 48])); b.truncate([48, 48])
    c.compact(); b.compact()
    assert_books(c, b)
    c.truncate(i32([0, 48])); b.truncate([0, 48])
    c.compact(); b.compact()
    assert_books(c, b)
    c.compact(); b.compact()
    assert_books(c, b)
    assert torch.equal(mem.cpu(), b.pool) and status(c) == pkg.MOE_OK


def test_a_pool_of_one_page():
    c, mem, b = make(L=1, S=2, M=1, P=1, page=16)
    for call in (lambda x, a: x.reserve(a([0, 16])), lambda x, a: x.truncate(a([-1, 7])), lambda x, a: x.compact(),
                 lambda x, a: x.fork(a([1]), a([0])), lambda x, a: x.truncate(a([-1, 0])), lambda x, a: x.reserve(a([9, 0])),
                 lambda x, a: x.compact(), lambda x, a: x.truncate(a([0, 0])), lambda x, a: x.compact()):
        call(c, i32)
        call(b, lambda x: x)
        assert status(c) == pkg.MOE_OK
        assert_books(c, b)
    c.reserve(1)                                   # two pages wanted, one there
    assert status(c) == pkg.MOE_ERR_CACHE_FULL
    assert_books(c, b)
    assert torch.equal(mem.cpu(), b.pool)


def test_more_pools_than_one_launch_copies():
    """130 layers: the copies go out in two launches."""
    c, mem, b = make(L=130, S=3, M=2, P=5, page=16, Hkv=1, D=64)
    c.reserve(i32([0, 0, 9])); b.reserve([0, 0, 9])
    c.truncate(i32([0, 0, 9])); b.truncate([0, 0, 9])
    c.fork(i32([2]), i32([0])); b.fork([2], [0])
    c.reserve(i32([1, 0, 0])); b.reserve([1, 0, 0])
    assert torch.equal(mem.cpu(), b.pool)
    c.truncate(i32([-1, -1, 0])); b.truncate([-1, -1, 0])
    c.compact(); b.compact()
    assert torch.equal(mem.cpu(), b.pool)
    assert_books(c, b)


def test_rows_of_a_fused_projection_and_one_stream():
    """k and v as slices of one tensor's rows; a batch of one, and of one position."""
    for S, B in ((3, 5), (1, 4), (4, 1), (1, 1)):
        c, mem, b = make(S=4, M=3, P=12, L=1, seed=S)
        used = [B] * S + [0] * (4 - S)
        c.reserve(i32(used)); b.reserve(used)
        fused = torch.randn((S, B, 10, 64)).bfloat16().cuda()
        c.append(0, fused[:, :, 5:7], fused[:, :, 7:9])
        b.append(fused[:, :, 5:7].cpu(), fused[:, :, 7:9].cpu(), 0, used[:S])
        assert torch.equal(mem.cpu(), b.pool) and status(c) == pkg.MOE_OK


def test_pages_beyond_32_bit_offsets():
    """A pool of more than 2^31 elements: append, copy on write and compact at its end."""
    P, Hkv, page, D = 16500, 8, 128, 128
    free = torch.cuda.mem_get_info()[0]
    if free < 20 << 30:
        pytest.skip("needs 20 GB")
    mem = torch.empty((2, P, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    c = pkg.KvCache(layers=[(mem[0], mem[1])], num_streams=3, max_pages=4)
    b = Books(3, 4, P, page)
    b.ref = [1] * (P - 6) + [0] * 6               # all but the last pages are in use
    write_books(c, b)
    add = [100, 0, 0]
    c.reserve(i32(add)); b.reserve(add)
    k, v = torch.randn((2, 1, 100, Hkv, D), device="cuda").bfloat16()
    c.append(0, k, v)
    c.truncate(i32([100, -1, -1])); b.truncate([100, -1, -1])
    c.fork(i32([0]), i32([2])); b.fork([0], [2])
    c.reserve(i32([0, 0, 1])); b.reserve([0, 0, 1])
    assert b.table[2][0] == P - 5
    assert torch.equal(mem[0, P - 6, :, :100], k[0].transpose(0, 1))
    assert torch.equal(mem[1, P - 5, :, :100], v[0].transpose(0, 1))
    c.refcount[7] = 0; b.ref[7] = 0               # a hole near the front
    c.compact(); b.compact()
    assert b.table[2][0] == 7 or b.table[0][0] == 7
    s = 2 if b.table[2][0] == 7 else 0
    assert torch.equal(mem[1, 7, :, :100], v[0].transpose(0, 1))
    assert c.page_table[s, 0].item() == 7 and status(c) == pkg.MOE_OK
    assert_books(c, b)


def test_two_streams_a_graph_and_its_replay():
    """The books' calls captured once and replayed on another stream: the second pass continues from the first."""
    c, mem, b = make(S=3, M=6, P=20, L=2)
    k, v = torch.randn((2, 3, 7, 2, 64), device="cuda").bfloat16()
    acc = i32([7, 3, 0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            c.reserve(7)
            for layer in range(2):
                c.append(layer, k, v)
            c.commit(acc)
        for _ in range(4):
            g.replay()
    side.synchronize()
    for _ in range(4):
        b.reserve([7] * 3)
        for layer in range(2):
            b.append(k.cpu(), v.cpu(), layer, [7] * 3)
        b.truncate([b.length[s] + n for s, n in enumerate([7, 3, 0])])
    assert_books(c, b)
    assert torch.equal(mem.cpu(), b.pool) and status(c) == pkg.MOE_OK


def test_every_call_on_a_stream_of_its_own():
    """stream= of each call, while another stream is current (and busy)."""
    c, mem, b = make(S=4, M=6, P=24, L=2, seed=3)
    k, v = torch.randn((2, 4, 20, 2, 64)).bfloat16()
    gk, gv, side = k.cuda(), v.cuda(), torch.cuda.Stream()
    n, dst, src, acc, cut = i32([20, 20, 20, 0]), i32([3]), i32([1]), i32([20, 9, 0, 0]), i32([-1, -1, -1, 4])
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    on = dict(stream=side.cuda_stream)
    c.reserve(n, **on)
    for layer in range(2):
        c.append(layer, gk, gv, lengths=n, **on)
    c.commit(acc, **on)
    c.fork(src, dst, **on)
    c.truncate(cut, **on)
    c.reserve(1, **on)
    c.compact(**on)
    c.check(**on)
    b.reserve([20, 20, 20, 0])
    for layer in range(2):
        b.append(k, v, layer, [20, 20, 20, 0])
    b.truncate([20, 9, 0, -1])
    b.fork([1], [3])
    b.truncate([-1, -1, -1, 4])
    b.reserve([1] * 4)
    b.compact()
    torch.cuda.synchronize()
    assert_books(c, b)
    assert torch.equal(mem.cpu(), b.pool)


def test_argument_checks_of_the_binding():
    c, mem, b = make()
    k = torch.zeros((6, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: c.append(0, k.float(), k), lambda: c.append(0, k, k[:, :1]), lambda: c.append(0, k.cpu(), k.cpu()),
                 lambda: c.append(0, k.transpose(0, 1), k.transpose(0, 1)), lambda: c.append(0, k[..., :32], k[..., :32]),
                 lambda: c.reserve(torch.zeros(5, dtype=torch.int32, device="cuda")), lambda: c.reserve(1 << 40),
                 lambda: c.commit(torch.zeros(6, dtype=torch.int64, device="cuda")), lambda: c.fork(i32([0, 1]), i32([2])),
                 lambda: c.truncate(torch.zeros(6, dtype=torch.int32)),
                 lambda: pkg.KvCache(layers=[], num_streams=1, max_pages=1),
                 lambda: pkg.KvCache(layers=[(k, k.half())], num_streams=1, max_pages=1),
                 lambda: pkg.KvCache(layers=[(k.float(), k.float())], num_streams=1, max_pages=1)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: c.append(2, k, k), lambda: c.append(-1, k, k),
                 lambda: c.fork(i32(list(range(7))), i32(list(range(7)))),
                 lambda: pkg.KvCache(layers=[(mem[0, 0], mem[0, 1])], num_streams=0, max_pages=1),
                 lambda: pkg.KvCache(layers=[(mem[0, 0], mem[0, 1])], num_streams=1, max_pages=0)):
        with pytest.raises(pkg.MoeError) as e:
            call()
        assert e.value.status == pkg.MOE_ERR_INVALID_ARG
    assert ceil_div(5, 2) == 3
