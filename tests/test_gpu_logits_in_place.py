"""GPU tests of edits in place, to the bit, and of captured graphs that run at the same time."""
import os

import pytest
import torch

import mxfp4_moe_expert_gb300 as pkg
from test_gpu_logits import CASES, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(pkg.LIB_PATH):
        from mxfp4_moe_expert_gb300 import build
        build.build()
    pkg.load_library()


def bits(t):
    return t.view(torch.int32 if t.dtype is torch.float32 else torch.int16)


# lists of more tokens than a warp has lanes, and than it asks for at once, at any part of a run
LONG = [dict(S=2, B=3, V=12288, hist=5000, bias=2000), dict(S=3, B=4, V=4097, hist=4000, bias=900, tree=True),
        dict(S=2, B=17, V=9001, hist=3000, bias=500, ragged=True), dict(S=1, B=1, V=40000, hist=30000), dict(S=20, B=8, V=8192 + 24, hist=900, bias=90)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kw", CASES + LONG)
def test_in_place_writes_what_another_output_gets(kw, dtype):
    """A warp stores words that it masked and then reads the listed tokens behind its first 32 from the same row."""
    c = Case(**kw, dtype=dtype, seed=kw["V"] + 1)
    x = c.logits.cuda()
    out = pkg.edit_logits(x, **c.on)
    c.check_edit(out)
    assert pkg.edit_logits(x, out=x, **c.on) is x
    for s in range(c.S):
        n = c.used(s)
        assert torch.equal(bits(x[s, :n]), bits(out[s, :n])), s
        assert torch.equal(bits(x[s, n:].cpu()), bits(c.logits[s, n:])), s


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V,room,skip", [(9001, 9001, 0), (9001, 9011, 3), (8192, 8193, 1), (12289, 12296, 5)])
def test_in_place_in_rows_that_do_not_begin_on_16_bytes(V, room, skip, dtype):
    c = Case(S=3, B=5, V=V, dtype=dtype, seed=V, hist=4000, bias=700)
    mem = torch.full((15 * room + skip,), 5.0, dtype=dtype, device="cuda")
    x = mem[skip:].view(3, 5, room)[..., :V]
    x.copy_(c.logits)
    out = pkg.edit_logits(x, **c.on)
    c.check_edit(out)
    pkg.edit_logits(x, out=x, **c.on)
    assert torch.equal(bits(x.contiguous()), bits(out))
    assert (mem[:skip] == 5).all() and (mem[skip:].view(3, 5, room)[..., V:] == 5).all()


def test_graphs_that_make_their_workspaces_run_at_the_same_time():
    """Two captured graphs, replayed over and over on a stream each: neither writes what the other reads."""
    cases = [Case(S=5, B=6, V=9000, seed=s, tree=s == 1) for s in range(2)]
    xs = [c.logits.cuda() for c in cases]
    graphs, got, streams = [], [], [torch.cuda.Stream() for _ in cases]
    for c, x in zip(cases, xs):
        pkg.accept_edited(x, **c.on)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):            # several calls each, so that the two have time to meet
            got.append([pkg.accept_edited(x, **c.on) for _ in range(8)])
    torch.cuda.synchronize()
    for _ in range(20):
        for g in got:
            for call in g:
                for t in call:
                    t.fill_(-9)
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    graph.replay()
        torch.cuda.synchronize()
        for c, g in zip(cases, got):
            for call in g:
                c.check_accept(call)
