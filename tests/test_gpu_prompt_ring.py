"""The warp that cleans operands, in attention over packed sequences: items whose tiles are
many and mostly seen in full, so that it has little to do between two tiles that it cleans, over many
launches. Only hidden places hold NaN, so a tile that missed its cleaning shows."""
import math

import pytest

from test_gpu_prompt import gsk, i32, inputs, make, sums  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nq,nk,H,KV,D,window", [
    ([4000, 7], None, 4, 1, 128, None),           # tiles of 32 tokens behind up to 31 blocks, most of them seen in full
    ([4000, 700], None, 2, 2, 64, 1500),          # windows: cleaned, seen in full, cleaned
    ([1, 3], [9000, 5000], 16, 2, 128, None),     # alternate blocks of two groups, clusters
    ([300] * 4, [4300] * 4, 8, 1, 64, None)])     # chunks
def test_tiles_seen_in_full_between_cleaned_ones(gsk, nq, nk, H, KV, D, window):  # noqa: F811
    nk = nk or nq
    q, k, v = inputs(nq, nk, H, KV, D, "bf16", 5, spare=130)
    cu, ck = i32(sums(nq)), i32(sums(nk))
    g = make(q.shape, "bf16", 6)
    want = None
    for _ in range(30):
        out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.1, cu_k=ck, window=window)
        got = (out, lse, *gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, 0.1, cu_k=ck, window=window))
        if want is None:                          # from finite rows; then the rows behind the last sequence hold NaN
            want = got
            for t, n in ((q, sum(nq)), (k, sum(nk)), (v, sum(nk)), (g, sum(nq))):
                t[n:] = math.nan
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.isfinite(t[: sum(nq)]).all() for t in want[:3])
