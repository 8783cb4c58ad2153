"""csa_cache_attend gives the same bits from call to call, where parts of a
tile are handled apart: rows that only some queries see, rows that are not
there, references that lie far apart. Tolerances in cache_ref.attend_tolerance."""
import numpy as np
import pytest

from test_gpu_cache_attend import Setup, gsk, i32  # noqa: F401 (gsk is a fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("D,shared,group", [(64, True, 2), (128, False, 4), (128, True, 2), (256, False, 2), (512, True, 4),
                                            (512, False, 2)])
@pytest.mark.parametrize("n", [128, 125, 99, 380])
def test_nan_and_missing_rows_at_a_tiles_end(gsk, D, shared, group, n):  # noqa: F811
    """Every key of the last tile's second half holds NaN in some column, each is
    seen by some queries and not by others, and the tile may end before its 128th."""
    queries = 50
    s = Setup([n], [queries], group, 1, D, shared, 32, 16, seed=D + n)
    first = (n - 1) // 128 * 128 + 64
    for j in range(first, n):
        s.bytes[s.table[0, j // 32], :, j % 32, (7 * j) % D] = 0x7F
    s.visible = [min(n, first - 3 + i * (n - first + 6) // queries) for i in range(queries)]
    out, lse = s.check(gsk)
    assert torch.isnan(out).any() and torch.isfinite(out[0]).all()
    for _ in range(20):
        again = s.run(gsk)
        assert same(again[0], out) and same(again[1], lse)


@pytest.mark.parametrize("far", [0, 1])
@pytest.mark.parametrize("D,shared", [(64, False), (128, False), (128, True), (256, True), (512, True), (512, False)])
def test_one_half_of_a_tile_sees_only_zeros(gsk, D, shared, far):  # noqa: F811
    """A tile is two tokens of 32 heads. One token sees nothing but a block of
    zeros, which the writer gives the scale 2^-120: its two references are 120
    powers of two apart. The other sees ordinary rows too, and its bits are those
    that it has beside a token that sees them as well."""
    lens = [700, 130, 2000]
    s = Setup(lens, [2] * 3, 32, 1, D, shared, 64, 16, seed=D)
    for t in s.table:
        s.bytes[t[0], :, :16] = 0
        s.scales[t[0], :, 0] = 2.0 ** -120
    near = [2 * i + 1 - far for i in range(3)]
    s.visible = [n for n in lens for _ in range(2)]
    want = s.check(gsk)
    for i in range(3):
        s.visible[2 * i + far] = 11 + i
    out, lse = s.check(gsk)
    assert (out[[2 * i + far for i in range(3)]] == 0).all()
    assert same(out[near], want[0][near]) and same(lse[near], want[1][near])
    args, visible = s.args(), i32(s.visible)
    for _ in range(50):
        again = gsk.csa_cache_attend(s.q, *args, shared=shared, visible=visible)
        assert same(again[0], out) and same(again[1], lse)
