"""GPU tests of the repetition penalty over all of its range: one operation, rounded once, so equal to the bit."""
import os

import numpy as np
import pytest
import torch

import mxfp4_moe_expert_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(pkg.LIB_PATH):
        from mxfp4_moe_expert_gb300 import build
        build.build()
    pkg.load_library()


# the smallest above 0, subnormal ones, the ends of the normal range, and common ones
REPETITION = [2.0 ** -149, 2.0 ** -130, 2.0 ** -128, 2.0 ** -127, 1.1e-38, 2.0 ** -126, 3e-20, 0.5, 1.0, 1.05, 1.2, 1.3, 1.998309, 3.0, 2.0 ** 100,
              2.0 ** 126, 1.7e38, 3.4028234663852886e38]


def logits_of(dtype, S, V, seed):
    """Values of every size that the type has, zeros of both signs and infinities among them."""
    g = torch.Generator().manual_seed(seed)
    info = torch.finfo(dtype)
    low, high = np.log2(info.smallest_normal) - 6, np.log2(info.max) - 3
    x = torch.randn((S, 1, V), generator=g, dtype=torch.float64)
    x = x * torch.where(torch.rand((S, 1, V), generator=g) < 0.5, 1.0, 2.0 ** (low + (high - low) * torch.rand((S, 1, V), generator=g).double()))
    x[:, :, 5], x[:, :, 6], x[:, :, 7], x[:, :, 8] = 0.0, -0.0, float("inf"), -float("inf")
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [4096, 9001])
def test_logits_are_divided_by_the_penalty_and_not_multiplied_by_a_reciprocal(dtype, V):
    S = len(REPETITION)
    x = logits_of(dtype, S, V, V)
    rng = np.random.default_rng(V)
    told = rng.integers(0, V, (S, 700), dtype=np.int32)
    told[:, :4] = [5, 6, 7, 8]
    seen = np.zeros((S, 1, V), dtype=bool)
    for s in range(S):
        seen[s, 0, told[s]] = True
    r = torch.tensor(REPETITION, dtype=torch.float32)
    z, by = x.float().numpy(), r.numpy()[:, None, None]
    with np.errstate(all="ignore"):
        z = np.where(seen, np.where(z > 0, z / by, z * by), z).astype(np.float32)
    on = dict(history=torch.from_numpy(told).cuda(), history_lengths=torch.full((S,), 700, dtype=torch.int32, device="cuda"),
              prompt_lengths=torch.full((S,), 350, dtype=torch.int32, device="cuda"), repetition=r.cuda())
    got = pkg.edit_logits(x.cuda(), **on).cpu()
    want = torch.from_numpy(z).to(dtype)
    bits = torch.int32 if dtype is torch.float32 else torch.int16
    for s in range(S):
        same = (got[s].view(bits) == want[s].view(bits)) | (torch.isnan(got[s]) & torch.isnan(want[s]))
        assert same.all(), (REPETITION[s], x[s][~same][:5], got[s][~same][:5], want[s][~same][:5])
    x[:, :, 7] = 1.0                                      # (without an infinity: the largest of the quotients)
    with np.errstate(all="ignore"):
        z[:, 0, 7] = np.float32(1) / r.numpy()
    z = np.where(np.isnan(z), -np.inf, z)
    target = pkg.accept_edited(x.cuda(), torch.full((S, 1), -1, dtype=torch.int32, device="cuda"), **on)[0]
    assert target[:, 0].tolist() == [int(np.flatnonzero(z[s, 0] == z[s, 0].max())[0]) for s in range(S)]


def test_a_small_penalty_keeps_the_order_of_what_it_divides():
    """Two logits that are said, over 2^-130: finite quotients, of which the second is the larger."""
    x = torch.full((1, 1, 600), -4.0, device="cuda")
    x[0, 0, 40], x[0, 0, 300] = 2.0 ** -20, 1.5 * 2.0 ** -20
    history = torch.tensor([[40, 300]], dtype=torch.int32, device="cuda")
    n = torch.tensor([2], dtype=torch.int32, device="cuda")
    on = dict(history=history, history_lengths=n, repetition=torch.tensor([2.0 ** -130], device="cuda"))
    out = pkg.edit_logits(x, **on)
    assert out[0, 0, 40] == 2.0 ** 110 and out[0, 0, 300] == 1.5 * 2.0 ** 110
    assert pkg.accept_edited(x, torch.tensor([[7]], dtype=torch.int32, device="cuda"), **on)[0].tolist() == [[300]]
