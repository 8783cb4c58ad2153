"""csa_cache_attend beside scales that a query must not notice. Tolerances in
cache_ref.attend_tolerance, which counts 2^-12 of the 2^-11 that half a step of
fp16 is at most: the other 2^-12 is added."""
import math

import numpy as np
import pytest

import cache_ref
from test_gpu_cache_attend import Setup, gsk  # noqa: F401 (gsk is a fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,shared,group,queries", [(64, False, 2, 4), (128, True, 8, 2), (512, True, 4, 3), (512, False, 2, 8),
                                                    (64, True, 32, 2), (128, False, 8, 20), (256, True, 16, 8),
                                                    (512, True, 64, 2), (512, False, 64, 2)])
@pytest.mark.parametrize("bad", [math.inf, math.nan, -math.inf, -1.0, 3e38])
def test_scales_of_rows_that_a_query_does_not_see(gsk, D, shared, group, queries, bad):  # noqa: F811
    """A block whose scale is no number, seen by each sequence's last query alone:
    the others get what they get beside an ordinary block, within the tolerance."""
    lens = [100, 200, 47]
    s = Setup(lens, [queries] * 3, group, 1, D, shared, 32, 16, seed=D + group)
    s.visible = []
    for n in lens:
        s.visible += [(n - 1) // 16 * 16 - i for i in range(queries - 1)] + [n]
    others = [i * queries + k for i in range(3) for k in range(queries - 1)]
    s.check(gsk)
    scales = s.scales.copy()
    want = cache_ref.attend(s.q.double().cpu().numpy(), s.bytes, scales.astype(np.float64), s.table, lens, s.cu, 1,
                            s.scale, shared, s.visible)
    tol_o, tol_l = cache_ref.attend_tolerance(*want, D, max(lens), 2.0 ** -7)
    tol_o = tol_o + (1 + 2.0 ** -7) * 2.0 ** -12 * want[2]
    for i, n in enumerate(lens):
        s.scales[s.table[i, (n - 1) // 32], :, (n - 1) % 32 // 16] = bad
    out, lse = s.run(gsk)
    o, l = out.double().cpu().numpy()[others], lse.double().cpu().numpy()[others]
    assert (np.abs(o - want[0][others]) <= tol_o[others]).all()
    assert (np.abs(l - want[1][others]) <= tol_l[others]).all()
