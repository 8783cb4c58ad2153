"""csa_cache_attend with scales that are no powers of two.

A scale s that is no power of two enters a weight as 2^(z + log2 s), or as
2^z 2^(log2 s). With L the largest |log2 s| of a sequence, beside what
cache_ref.attend_tolerance counts:
  - log2 in the fast form: 2^-22 absolute near 1, else 2 units in the last
    place, at most 2 * 2^-23 L;
  - roundings of sums that log2 s takes part in (z + log2 s, the difference to
    the reference, that reference itself, the final factor's exponent): at
    most 8, each half a unit, 2^-24, of at most 2 (|z| + L) in units of log2,
    of which the parts with z are in e_z;
  - one more exponential, 2^-22 relative (2 units of ex2 in the fast form).
An error e of an exponent is e ln 2 of the weight: ln 2 (2^-22 + 2^-22 L +
2^-20 L) + 2^-22 <= 2^-21 (1 + 2 L). What fp16 drops of a weight is at most
half its smallest step, 2^-25, where the largest weight is at least 2^7:
2^-32 of the largest p s a row, times values of at most 448. The keys'
products with s round once more each, 2^-24 of dz, which e_z has room for
(D + 8 units of 2^-23, of which D + 4 are used). A weight's rounding to fp16 is
half a step, eps / 2 = 2^-11 of it at most, of which attend_tolerance counts
2^-12: the other 2^-12 is added here.
"""
import numpy as np
import pytest

import cache_ref
from test_gpu_cache_attend import Setup, gsk  # noqa: F401 (gsk is a fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def weights_top(s):
    """[T, H]: the largest p_j s_j of each query and head, in 64 bits."""
    n = int(s.cu[-1])
    q = s.q[:n].double().cpu().numpy()
    page = s.bytes.shape[2]
    block = page // s.scales.shape[2]
    group = q.shape[1] // s.kv
    top = np.zeros(q.shape[:2])
    for i, length in enumerate(s.lens):
        for t in range(s.cu[i], s.cu[i + 1]):
            m = length if s.visible is None else max(0, min(length, s.visible[t]))
            if m == 0:
                continue
            pg, slot = s.table[i, np.arange(m) // page], np.arange(m) % page
            for h in range(s.kv):
                ks, vs = (s.scales[pg, x, slot // block].astype(np.float64) for x in (h, h if s.shared else s.kv + h))
                z = q[t, h * group:(h + 1) * group] @ (cache_ref.TABLE[s.bytes[pg, h, slot]] * ks[:, None]).T * s.scale
                p = np.exp(z - z.max(-1, keepdims=True))
                top[t, h * group:(h + 1) * group] = (p / p.sum(-1, keepdims=True) * vs).max(-1)
    return top


def check(gsk, s):  # noqa: F811
    out, lse = s.run(gsk)
    n = int(s.cu[-1])
    want = cache_ref.attend(s.q[:n].double().cpu().numpy(), s.bytes, s.scales.astype(np.float64), s.table, s.lens, s.cu,
                            s.kv, s.scale, s.shared, s.visible)
    eps = torch.finfo(out.dtype).eps
    tol_o, tol_l = cache_ref.attend_tolerance(*want, s.D, max(s.lens), eps)
    used = s.scales[s.scales > 0]
    L = float(np.abs(np.log2(used)).max())
    tol_o = tol_o + (1 + eps) * ((2.0 ** -12 + 2.0 ** -21 * (1 + 2 * L)) * want[2] + max(s.lens) * 448 * 2.0 ** -32 * weights_top(s)[..., None])
    o, l = out[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()
    bad = ~(np.abs(o - want[0]) <= tol_o)
    assert not bad.any(), (np.argwhere(bad)[:4], o[bad][:4], want[0][bad][:4], tol_o[bad][:4], bad.sum())
    fine = np.isfinite(want[1])
    assert (np.isfinite(l) == fine).all()
    assert (np.abs(l[fine] - want[1][fine]) <= tol_l[fine]).all()


SHAPES = [(64, False, 2, 3, 1), (128, False, 2, 8, 1), (128, True, 1, 4, 2), (512, True, 1, 16, 1),   # few rows
          (64, True, 1, 64, 1), (128, False, 1, 16, 9), (256, False, 1, 64, 1), (512, True, 1, 64, 1)]  # many


@pytest.mark.parametrize("D,shared,kv,group,queries", SHAPES)
@pytest.mark.parametrize("spread", [0, 6, 20, 34])
def test_scales_that_are_no_powers_of_two(gsk, D, shared, kv, group, queries, spread):  # noqa: F811
    """Uniform in [1, 2) times powers of two up to `spread` apart, half the pages'
    as amax / 448 of normal values; past 30 the weights take an exponential of
    their own."""
    lens = [300, 17, 129]
    s = Setup(lens, [queries] * 3, kv * group, kv, D, shared, 32, 16, "fp16" if spread == 6 else "bf16", seed=D + spread)
    r = np.random.default_rng(D + spread)
    shape = s.scales.shape
    power = 2.0 ** r.integers(-7 - spread, -6, shape)
    amax = np.abs(r.standard_normal((*shape, 16))).max(-1) / 448
    s.scales = np.where((np.arange(shape[0]) % 2 == 0)[:, None, None], r.uniform(1, 2, shape) * power, amax).astype(np.float32)
    check(gsk, s)
    # values that stand far above 1, past the two factors' range
    if not shared and spread == 34:
        s.scales[:, kv:] *= np.float32(1.3e12)
        check(gsk, s)
