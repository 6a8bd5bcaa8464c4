"""The rotation without a GPU: frequencies as fractions of a turn, refusals that come before any device call, and how the
binding lays rows out."""
import ctypes
import math
import os
from fractions import Fraction

import pytest
import torch

import mxfp4_moe_expert_gb300 as pkg
from forward_util import frequencies

BAD, OK = pkg.MOE_ERR_INVALID_ARG, pkg.MOE_OK
TWO_PI = 2 * (Fraction(math.pi) + Fraction(1.2246467991473532e-16))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(pkg.LIB_PATH):
        from mxfp4_moe_expert_gb300 import build
        build.build()
    pkg.load_library()


def turns(R, base=10000.0, scaling=None):
    out = (ctypes.c_uint64 * max(1, R // 2))()
    if scaling is not None:
        scaling = pkg.moe_mxfp4_rotary_scaling(*scaling)
    return pkg.moe_mxfp4_rotary_turns(R, base, scaling, out), list(out[:R // 2])


@pytest.mark.parametrize("f", [0.0, 1.0, -1.0, 0.5, 1e-4, 1e-12, 3.1, 2 * math.pi, -2 * math.pi, 10000 ** (-2 / 128)])
def test_a_frequency_as_a_fraction_of_a_turn(f):
    out = (ctypes.c_uint64 * 1)()
    assert pkg.moe_mxfp4_rotary_from((ctypes.c_double * 1)(f), 1, out) == OK
    want = Fraction(f) / TWO_PI * 2 ** 64
    off = (out[0] - want) % 2 ** 64
    assert min(off, 2 ** 64 - off) <= 2        # half a unit, and what two doubles leave of 1 / 2 pi (2^-107 of 2^62)


@pytest.mark.parametrize("R", [2, 20, 64, 128])
@pytest.mark.parametrize("scaling", [None, dict(kind="linear", factor=8.0), dict(kind="ntk", factor=4.0),
                                     dict(kind="parts", factor=16.0, original=4096.0, low=1.0, high=32.0)])
def test_frequencies_of_the_scalings(R, scaling):
    kinds = {"linear": 1, "ntk": 2, "parts": 3}
    c = None if scaling is None else [kinds[scaling["kind"]]] + [scaling.get(n, 0.0) for n in ("factor", "original", "low", "high")]
    st, got = turns(R, scaling=c)
    assert st == OK
    for x, f in zip(got, frequencies(R, scaling=scaling)):
        assert abs(x - Fraction(f) / TWO_PI * 2 ** 64) <= f / 6.28 * 2 ** 64 * 2.0 ** -49 + 1   # some roundings of doubles


def test_turns_refuse():
    assert turns(3)[0] == BAD and turns(-2)[0] == BAD and turns(8, base=0.0)[0] == BAD and turns(8, base=math.nan)[0] == BAD
    assert turns(8, base=math.inf)[0] == BAD and turns(8, scaling=[4, 2.0])[0] == BAD and turns(8, scaling=[1, 0.0])[0] == BAD
    assert turns(8, scaling=[3, 2.0, 0.0, 1.0, 2.0])[0] == BAD and turns(8, scaling=[3, 2.0, 100.0, 2.0, 2.0])[0] == BAD
    assert turns(0)[0] == OK and turns(2, scaling=[2, 8.0])[0] == OK
    assert pkg.moe_mxfp4_rotary_turns(8, 10000.0, None, None) == BAD
    assert pkg.moe_mxfp4_rotary_from(None, 1, None) == BAD and pkg.moe_mxfp4_rotary_from(None, 0, None) == OK
    one = (ctypes.c_uint64 * 1)()
    for f in (7.0, -7.0, math.inf, math.nan):
        assert pkg.moe_mxfp4_rotary_from((ctypes.c_double * 1)(f), 1, one) == BAD


def rotary(**kw):
    c = dict(turns_dev=256, q_norm_dev=None, k_norm_dev=None, head_dim=64, rotary_dim=64, dtype=0, flags=0, eps=1e-6, gain=1.0)
    return pkg.moe_mxfp4_rotary(*{**c, **kw}.values())


def rotate_args(**kw):
    c = dict(q_dev=512, k_dev=512, q_out_dev=1024, k_out_dev=1024, positions_dev=256, q_stride=0, k_stride=0, q_out_stride=0,
             k_out_stride=0, tokens=1, q_heads=2, kv_heads=1)
    return pkg.moe_mxfp4_rotate_args(*{**c, **kw}.values())


@pytest.mark.parametrize("bad", [
    dict(head_dim=96), dict(head_dim=0), dict(rotary_dim=66), dict(rotary_dim=63), dict(rotary_dim=-2), dict(dtype=2), dict(flags=4),
    dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(gain=math.nan), dict(turns_dev=None), dict(turns_dev=260),
    dict(q_norm_dev=264), dict(k_norm_dev=8)])
def test_rotate_refuses_a_bad_rotary(bad):
    assert pkg.moe_mxfp4_rotate(rotary(**bad), rotate_args(), None) == BAD


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(q_heads=-1), dict(kv_heads=65537), dict(q_stride=120), dict(k_stride=68), dict(q_out_stride=64),
    dict(k_out_stride=65), dict(q_dev=None), dict(k_dev=None), dict(q_out_dev=None), dict(k_out_dev=None), dict(q_dev=520),
    dict(k_out_dev=8), dict(positions_dev=None), dict(positions_dev=258)])
def test_rotate_refuses_bad_rows(bad):
    assert pkg.moe_mxfp4_rotate(rotary(), rotate_args(**bad), None) == BAD


def test_rotate_of_nothing():
    assert pkg.moe_mxfp4_rotate(rotary(), rotate_args(tokens=0, q_dev=None, k_dev=None, positions_dev=None), None) == OK
    assert pkg.moe_mxfp4_rotate(rotary(), rotate_args(q_heads=0, kv_heads=0, q_dev=None, k_dev=None), None) == OK


def test_calls_of_the_cache_refuse_a_null_handle():
    assert pkg.moe_mxfp4_cache_append_rotated(None, None, 0, rotary(), pkg.moe_mxfp4_append_args(), None) == BAD
    assert pkg.moe_mxfp4_cache_commit_path(None, None, pkg.moe_mxfp4_commit_args(), None) == BAD


def bare(D=64):
    r = pkg.Rotary.__new__(pkg.Rotary)
    r.device, r.dtype, r.head_dim, r._layouts, r._index = torch.device("cpu"), torch.bfloat16, D, {}, -1
    return r


def test_rows_of_the_binding():
    r = bare()
    x = torch.zeros((3, 5, 12, 64), dtype=torch.bfloat16)
    assert r._rows("q", x) == (15, 12, 768) and r._rows("q", x[..., 2:6, :]) == (15, 4, 768) and r._rows("q", x[0, 0]) == (1, 12, 768)
    assert r._rows("q", x[1]) == (5, 12, 768) and r._rows("q", x[:, 2]) == (3, 12, 3840) and r._rows("q", x[:, :1]) == (3, 12, 3840)
    assert r._rows("q", x[:0])[0] == 0
    for t in (x[:, ::2], x[..., ::2, :], x.transpose(0, 1), x.expand(3, 5, 12, 64).transpose(2, 3)):
        with pytest.raises(ValueError):
            r._rows("q", t)
    with pytest.raises(ValueError, match="share memory"):
        r._rows("q", x[:1, :1].expand(3, 5, 12, 64))
    with pytest.raises(ValueError):
        r._rows("q", x.float())
    with pytest.raises(ValueError):
        r._rows("q", torch.zeros((4, 2, 32), dtype=torch.bfloat16))


def test_the_rotary_refuses():
    for kw in (dict(head_dim=96), dict(rotary_dim=7), dict(rotary_dim=66), dict(dtype=torch.float32), dict(eps=-1.0),
               dict(gain=math.inf), dict(scaling=dict(kind="other", factor=2.0)), dict(scaling=dict(kind="linear")),
               dict(scaling=dict(kind="parts", factor=2.0)), dict(scaling=dict(kind="linear", factor=2.0, low=1.0)),
               dict(frequencies=[0.1]), dict(q_norm=torch.ones(64)), dict(q_norm=torch.ones(32, dtype=torch.bfloat16)),
               dict(q_norm=torch.ones(64, dtype=torch.bfloat16), norm=False)):
        with pytest.raises(ValueError):
            pkg.Rotary(**{**dict(head_dim=64, device="cpu"), **kw})
    with pytest.raises(pkg.MoeError):
        pkg.Rotary(head_dim=64, base=-1.0, device="cpu")
    r = pkg.Rotary(head_dim=64, device="cpu")
    with pytest.raises(ValueError, match="cpu"):
        r.rotate(torch.zeros((1, 2, 64), dtype=torch.bfloat16), None, torch.zeros(1, dtype=torch.int32))
    r = pkg.Rotary(head_dim=64, rotary_dim=0, device="cpu")
    assert r.turns.numel() == 0 and r.desc.flags == 0
