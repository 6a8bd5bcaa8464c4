"""The paged cache without a GPU: refusals that come before any device call, and the plain definitions that the GPU
tests compare with."""
import os
import random

import pytest

import mxfp4_moe_expert_gb300 as pkg
from cache_util import Books


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(pkg.LIB_PATH):
        from mxfp4_moe_expert_gb300 import build
        build.build()
    pkg.load_library()


GOOD = dict(num_layers=1, num_streams=4, max_pages=8, num_pages=16, page_tokens=64, kv_heads=8, head_dim=128,
            dtype=pkg.MOE_DTYPE_BF16, page_stride=0, timeout_us=0)


@pytest.mark.parametrize("bad", [
    dict(num_layers=0), dict(num_layers=1025), dict(num_streams=0), dict(num_streams=65537), dict(max_pages=0),
    dict(max_pages=1 << 24), dict(num_pages=0), dict(num_pages=(1 << 24) + 1), dict(page_tokens=8), dict(page_tokens=48),
    dict(page_tokens=256), dict(kv_heads=0), dict(kv_heads=257), dict(head_dim=96), dict(head_dim=256), dict(dtype=2),
    dict(page_stride=64 * 8 * 128 - 8), dict(page_stride=64 * 8 * 128 + 4), dict(timeout_us=-1)])
def test_create_refuses_bad_sizes(bad):
    cfg = pkg.moe_mxfp4_cache_config(**{**GOOD, **bad})
    layers = [pkg.moe_mxfp4_cache_layer(256, 512)] * max(1, min(cfg.num_layers, 1024))
    st, h = pkg.moe_mxfp4_cache_create(cfg, layers)
    assert st == pkg.MOE_ERR_INVALID_ARG and not h


def test_create_refuses_missing_and_misaligned_pools():
    for k, v in ((None, 512), (256, None), (264, 512), (256, 520)):
        st, h = pkg.moe_mxfp4_cache_create(pkg.moe_mxfp4_cache_config(**GOOD), [pkg.moe_mxfp4_cache_layer(k, v)])
        assert st == pkg.MOE_ERR_INVALID_ARG and not h


def test_every_call_refuses_a_null_handle():
    bad = pkg.MOE_ERR_INVALID_ARG
    assert pkg.moe_mxfp4_cache_state_bytes(None)[0] == bad
    assert pkg.moe_mxfp4_cache_reserve(None, None, None, 1, None) == bad
    assert pkg.moe_mxfp4_cache_append(None, None, 0, None, None, 0, 1, 1, None, None) == bad
    assert pkg.moe_mxfp4_cache_truncate(None, None, None, None) == bad
    assert pkg.moe_mxfp4_cache_commit(None, None, None, None) == bad
    assert pkg.moe_mxfp4_cache_fork(None, None, None, None, 1, None) == bad
    assert pkg.moe_mxfp4_cache_compact(None, None, None) == bad
    assert pkg.moe_mxfp4_cache_attend_bytes(None, 1, 1, 8)[0] == bad
    assert pkg.moe_mxfp4_cache_attend(None, None, 0, pkg.moe_mxfp4_attend_args(), None, 0, None) == bad
    assert pkg.moe_mxfp4_cache_check(None, None, None) == bad
    pkg.moe_mxfp4_cache_destroy(None)


def test_status_strings_of_the_cache():
    assert "pages" in pkg.moe_mxfp4_status_string(pkg.MOE_ERR_CACHE_FULL)
    assert "books" in pkg.moe_mxfp4_status_string(pkg.MOE_ERR_CACHE_STATE)


@pytest.mark.parametrize("seed", range(4))
def test_plain_books_stay_consistent(seed):
    """The definitions that the GPU is held to: counts equal the table entries after any calls, and a page that a
    stream writes to is its own."""
    rng = random.Random(seed)
    b = Books(S=9, M=12, P=40, page=16)
    for _ in range(300):
        op = rng.choice(["reserve", "reserve", "truncate", "fork", "compact"])
        if op == "reserve":
            add = [rng.choice([0, 1, 5, 16, 33]) for _ in range(b.S)]
            if b.reserve(add):
                for s, n in enumerate(add):
                    if n and b.length[s] % b.page:
                        assert b.ref[b.table[s][b.length[s] // b.page]] == 1
                b.truncate([b.length[s] + rng.randint(0, n) for s, n in enumerate(add)])
        elif op == "truncate":
            b.truncate([rng.choice([-1, 0, b.length[s] // 2, b.length[s]]) for s in range(b.S)])
        elif op == "fork":
            empty = [s for s in range(b.S) if not b.held[s]]
            full = [s for s in range(b.S) if b.held[s]]
            if empty and full:
                dst = rng.sample(empty, rng.randint(1, len(empty)))
                b.fork([rng.choice(full) for _ in dst], dst)
        else:
            before = [[b.table[s][i] for i in range(b.held[s])] for s in range(b.S)]
            b.compact()
            live = sum(r > 0 for r in b.ref)
            assert all(b.ref[p] for p in range(live)) and [len(x) for x in before] == b.held
        b.consistent()
