"""Attention of few queries over long keys, whose keys the CTAs of a cluster share (2, 4 or 8 of
them): against the formulas, with windows, and with values that are not finite in one part."""
import math

import pytest

from test_gpu_prompt import check, gsk, i32, inputs, sums  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

# queries and keys of each sequence, heads, key heads, columns, window, CTAs of a cluster
CASES = [([1], [2500], 8, 1, 128, None, 8), ([1], [5003], 2, 2, 64, None, 8), ([130], [2300], 8, 1, 64, None, 8),
         ([130], [2300], 5, 1, 96, None, 8), ([300], [2300], 8, 1, 128, None, 4), ([5, 3], [4000, 3000], 16, 2, 128, 2500, 8),
         ([200], [3000], 16, 2, 64, 1500, 4), ([260], [3000], 16, 2, 64, None, 2), ([250], [1500], 8, 1, 128, 1100, 4), ([1, 1, 1, 1], [9000, 10, 0, 1], 8, 1, 128, None, 8)]


def shared_by(nq, nk, H, KV, window):
    """How many CTAs share an item's keys: as many as leave each two blocks, up to 128 CTAs in all."""
    tp = 128 // (H // KV)
    items = lambda tiles: (sum(nq) // (tiles * tp) + len(nq)) * KV  # noqa: E731
    keys, split = sum(nk) // len(nq), 1
    if window:
        keys = min(keys, window + tp)
    while items(2) <= 152 and split < 8 and items(1) * split * 2 <= 128 and keys >= split * 2 * 256:
        split *= 2
    return split


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("nq,nk,H,KV,D,window,ctas", CASES)
def test_formulas(gsk, nq, nk, H, KV, D, window, ctas, dtype):  # noqa: F811
    assert shared_by(nq, nk, H, KV, window) == ctas
    q, k, v = inputs(nq, nk, H, KV, D, dtype, sum(nk) + D)
    check(gsk, q, k, v, sums(nq), sums(nk), D ** -0.5, window=window, dtype=dtype, glse=True)


@pytest.mark.parametrize("name,bad", [("v", math.inf), ("v", math.nan), ("k", math.nan)])
@pytest.mark.parametrize("window", [None, 2100])
def test_values_that_are_not_finite_in_one_part(gsk, name, bad, window):  # noqa: F811
    """They reach the queries that see them, in their column, and no other."""
    nq, nk, H, KV, D = [40, 30], [2500, 2300], 8, 1, 128
    assert shared_by(nq, nk, H, KV, window) == 8
    cu, ck = i32(sums(nq)), i32(sums(nk))
    t = torch.arange(70, device="cuda")
    place = torch.where(t < 40, 2500 - 40 + t, 2500 + 2300 - 30 + t - 40)     # of each query's own key
    for at in (0, 100, 380, 385, 700, 1300, 2100, 2470, 2499, 2500, 3000, 4700, 4798):
        q, k, v = inputs(nq, nk, H, KV, D, "bf16", at)
        want, wlse = gsk.csa_prompt_attend(q, k, v, cu, 0.1, cu_k=ck, window=window)
        (k if name == "k" else v)[at, 0, 5] = bad
        out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.1, cu_k=ck, window=window)
        sees = (place >= at) & (place - at < (window or 1 << 20)) & ((t < 40) == (at < 2500))
        assert torch.equal(out[~sees], want[~sees]) and torch.equal(lse[~sees], wlse[~sees])
        if name == "k":
            assert torch.isnan(out[sees]).all() and torch.isnan(lse[sees]).all()
        else:
            assert not torch.isfinite(out[sees][..., 5]).any() and torch.equal(lse, wlse)
            keep = [c for c in range(D) if c != 5]
            assert torch.equal(out[..., keep], want[..., keep])
