"""Edits and acceptance without a GPU: refusals that come before any device call, and the definitions that the GPU tests
compare with."""
import os
import random

import pytest
import torch

import mxfp4_moe_expert_gb300 as pkg
from forward_util import edit_reference, pack_allowed, targets_of, walk
from oracle import moe_oracle as O

BAD, OK = pkg.MOE_ERR_INVALID_ARG, pkg.MOE_OK


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(pkg.LIB_PATH):
        from mxfp4_moe_expert_gb300 import build
        build.build()
    pkg.load_library()


def args(**kw):
    a = pkg.moe_mxfp4_edit_args()
    for name, value in {**dict(logits_dev=256, dtype=2, streams=1, block=2, vocab=100, tokens_dev=256), **kw}.items():
        setattr(a, name, value)
    return a


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=-1), dict(streams=-1), dict(block=0), dict(block=1025), dict(block=65, mask_dev=256), dict(vocab=0),
    dict(vocab=1 << 31), dict(row_stride=99), dict(allowed_stride=3), dict(streams=1 << 30), dict(logits_dev=None), dict(logits_dev=258),
    dict(logits_dev=257, dtype=0), dict(history_dev=256), dict(history_dev=256, history_lengths_dev=256, history_room=-1),
    dict(history_dev=256, history_lengths_dev=256, history_room=9, history_stride=8), dict(bias_begin_dev=256, bias_entries=1),
    dict(bias_begin_dev=256, bias_ids_dev=256, bias_entries=1), dict(bias_begin_dev=256, bias_entries=-1), dict(mask_dev=260), dict(tokens_dev=258),
    dict(lengths_dev=2), dict(allowed_dev=257), dict(repetition_dev=258), dict(presence_dev=1), dict(frequency_dev=2)])
def test_both_entry_points_refuse(bad):
    assert pkg.moe_mxfp4_edit_logits(args(**bad), 256, 0, None) == BAD
    assert pkg.moe_mxfp4_accept_edited(args(**bad), 256, 256, 256, 256, 256, 1 << 20, None) == BAD


def test_outputs_and_workspaces_that_are_refused():
    assert pkg.moe_mxfp4_edit_logits(args(), None, 0, None) == BAD and pkg.moe_mxfp4_edit_logits(args(), 258, 0, None) == BAD
    assert pkg.moe_mxfp4_edit_logits(args(), 512, 99, None) == BAD
    assert pkg.moe_mxfp4_edit_logits(args(row_stride=128), 256, 100, None) == BAD      # in place with another stride
    accept = lambda a, *p: pkg.moe_mxfp4_accept_edited(a, *p, None)   # noqa: E731
    assert accept(args(tokens_dev=None), 256, 256, None, None, 256, 1 << 20) == BAD
    assert accept(args(), None, 256, None, None, 256, 1 << 20) == BAD and accept(args(), 256, None, None, None, 256, 1 << 20) == BAD
    assert accept(args(), 256, 256, 257, None, 256, 1 << 20) == BAD and accept(args(), 256, 256, None, 258, 256, 1 << 20) == BAD
    st, n = pkg.moe_mxfp4_accept_edited_bytes(1, 2, 100)
    assert st == OK and n > 0
    assert accept(args(), 256, 256, None, None, None, n) == pkg.MOE_ERR_WORKSPACE
    assert accept(args(), 256, 256, None, None, 260, n) == pkg.MOE_ERR_WORKSPACE
    assert accept(args(), 256, 256, None, None, 256, n - 1) == pkg.MOE_ERR_WORKSPACE
    for bad in ((-1, 2, 100), (1, 0, 100), (1, 1025, 100), (1, 2, 0), (1, 2, 1 << 31)):
        assert pkg.moe_mxfp4_accept_edited_bytes(*bad)[0] == BAD


def test_nothing_to_do():
    assert pkg.moe_mxfp4_edit_logits(args(streams=0, logits_dev=None), None, 0, None) == OK
    assert pkg.moe_mxfp4_accept_edited(args(streams=0, logits_dev=None), None, None, None, None, None, 0, None) == OK


def test_the_binding_refuses_tensors_on_the_cpu():
    with pytest.raises(ValueError, match="logits"):
        pkg.edit_logits(torch.zeros((1, 2, 8)))
    with pytest.raises(ValueError, match="logits"):
        pkg.accept_edited(torch.zeros((1, 2, 8)), torch.zeros((1, 2), dtype=torch.int32))


def test_rows_of_logits():
    x = torch.zeros((3, 4, 10))
    assert pkg._logit_rows("x", x) == 10 and pkg._logit_rows("x", x[..., :7]) == 10 and pkg._logit_rows("x", x[:, :1, :7]) == 40
    assert pkg._logit_rows("x", x[:, :1]) == 40 and pkg._logit_rows("x", x[:0]) == 10
    for t in (x[:, :3], x[..., ::2], x.transpose(0, 1)):
        with pytest.raises(ValueError):
            pkg._logit_rows("x", t)
    with pytest.raises(ValueError, match="share"):
        pkg._logit_rows("x", x[:1, :1].expand(3, 4, 10))


@pytest.mark.parametrize("seed", range(5))
def test_a_chain_is_what_the_plain_acceptance_accepts(seed):
    rng = random.Random(seed)
    S, B, V = 6, 5, 4
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((S, B, V), generator=g)
    tokens = torch.tensor([[rng.randrange(V) for _ in range(B)] for _ in range(S)])
    ref = O.accept_block(z.double().numpy(), tokens.numpy())
    target = targets_of(z.double(), None)
    accepted, nxt, paths = walk(target, tokens.tolist())
    assert target == ref["target"].tolist() and accepted == ref["accepted"].tolist() and nxt == ref["next_token"].tolist()
    assert all(p == list(range(n)) + [-1] * (B - n) for p, n in zip(paths, accepted))
    masks = [[(1 << (b + 1)) - 1 for b in range(B)]] * S
    assert walk(target, tokens.tolist(), masks) == (accepted, nxt, paths)


def test_a_tree_by_hand():
    #   0 -> 1 (token 7), 2 (token 8); 1 -> 3 (token 5); 2 -> 4 (token 6)
    masks = [[0b1, 0b11, 0b101, 0b1011, 0b10101]]
    tokens = [[9, 7, 8, 5, 6]]
    assert walk([[8, 5, 6, 1, 2]], tokens, masks) == ([3], [2], [[0, 2, 4, -1, -1]])
    assert walk([[7, 6, 6, 1, 2]], tokens, masks) == ([2], [6], [[0, 1, -1, -1, -1]])
    assert walk([[8, 5, 6, 1, 2]], tokens, masks, [4]) == ([2], [6], [[0, 2, -1, -1, -1]])
    assert walk([[-1, 5, 6, 1, 2]], [[9, -1, -1, 5, 6]], masks) == ([1], [-1], [[0, -1, -1, -1, -1]])


def test_edits_by_hand():
    z = torch.tensor([[[2.0, -2.0, 1.0, 4.0, 0.5]]])
    got, _ = edit_reference(z, [[3]], history=[[0, 1, 1]], prompt=[1], repetition=[2.0], frequency=[0.25], presence=[0.5],
                            bias=[[(4, 1.0), (4, 2.0)]], allowed=[[{0, 1, 3, 4}]])
    assert got[0, 0].tolist() == [1.0, -4.0 - 0.5 - 0.5, float("-inf"), 2.0 - 0.25 - 0.5, 2.5]
    assert pack_allowed([[{0, 1, 3, 4}]], 1, 1, 5)[0, 0].tolist() == [(0b11011 | ~0x1F)]
