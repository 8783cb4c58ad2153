"""csa_cache_append against the list implementation: every byte and every scale."""
import numpy as np
import pytest

import cache_ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def gsk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_softmax_kv_gb300 as g
    g.build()
    return g


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


class Setup:
    """A cache of random bytes and scales, sequences with shuffled pages."""

    def __init__(self, held, new, heads, D, page, block, dtype, seed=0, width=None):
        r = np.random.default_rng(seed)
        ends = [a + b for a, b in zip(held, new)]
        pages = sum(-(-e // page) for e in ends) + 3
        order = r.permutation(pages)
        width = width or max(1, max(-(-e // page) for e in ends))
        self.table = np.full((len(held), width), -1)
        at = 0
        for s, e in enumerate(ends):
            k = min(width, -(-e // page))
            self.table[s, :k] = order[at:at + k]
            at += k
        self.bytes = r.integers(0, 256, (pages, heads, page, D)).astype(np.uint8)
        self.scales = 2.0 ** r.integers(-6, 2, (pages, heads, page // block)).astype(np.float32)
        self.cu = np.concatenate([[0], np.cumsum(new)])
        self.held = held
        n = int(self.cu[-1])
        x = r.standard_normal((n, heads, D)) * 2.0 ** r.integers(-8, 8, (n, heads, 1))
        self.rows = torch.from_numpy(x).to(DTYPES[dtype]).cuda()

    def check(self, gsk, rows=None, stream=None):
        rows = self.rows if rows is None else rows
        cache = torch.from_numpy(self.bytes.copy()).cuda().view(torch.float8_e4m3fn)
        scales = torch.from_numpy(self.scales.copy()).cuda()
        table, held, cu = i32(self.table), i32(self.held), i32(self.cu)
        torch.cuda.synchronize()                            # inputs are there for any stream
        gsk.csa_cache_append(rows, cache, scales, table, held, cu, stream=stream)
        torch.cuda.synchronize()
        want_c, want_s = self.bytes.copy(), self.scales.copy().astype(np.float64)
        cache_ref.append(want_c, want_s, self.table, self.held, rows.double().cpu().numpy(), self.cu)
        np.testing.assert_array_equal(scales.double().cpu().numpy(), want_s)
        got = cache.view(torch.uint8).cpu().numpy()
        nan = (want_c & 0x7F) == 0x7F                       # the sign of a NaN is not kept
        np.testing.assert_array_equal(got[~nan], want_c[~nan])
        assert ((got[nan] & 0x7F) == 0x7F).all()
        return cache, scales


CASES = [  # held, new, heads, D, page, block
    ([0], [1], 1, 64, 16, 16), ([5], [1], 1, 512, 64, 16), ([63], [2], 2, 128, 64, 64), ([0, 3, 16], [0, 0, 1], 1, 64, 16, 1),
    ([0, 17, 64, 100, 7], [33, 1, 64, 0, 200], 1, 512, 64, 64), ([1, 2, 3], [15, 14, 13], 3, 256, 16, 8),
    ([255, 256, 0], [1, 1, 513], 2, 64, 256, 256), ([9] * 40, [1] * 40, 1, 128, 32, 32), ([0, 0], [70, 300], 8, 128, 128, 2)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("held,new,heads,D,page,block", CASES)
def test_bytes_and_scales(gsk, held, new, heads, D, page, block, dtype):
    Setup(held, new, heads, D, page, block, dtype, seed=len(held) + D).check(gsk)


def test_values_at_the_edges(gsk):
    """Zeros, the largest values of the type, subnormals, infinities, NaN; a block that is all of one kind."""
    s = Setup([0, 3], [64, 40], 1, 64, 16, 4, "fp32", seed=2)
    x = s.rows
    x[0:4] = 0.0
    x[4:8] = torch.finfo(torch.float32).max
    x[8:12] = 1e-45
    x[12:16] = float("nan")
    x[16:20] = float("-inf")
    x[20, 0, 5], x[21, 0, 6], x[22, 0, 7] = float("inf"), float("nan"), 3.0
    x[24:28] = 448.0
    x[28:32] = 448.00003
    x[32:36] = 2.0 ** -111
    x[36:40] = torch.linspace(-1, 1, 4 * 64).view(4, 1, 64).cuda()
    s.check(gsk)


def test_strided_rows_and_a_stream(gsk):
    s = Setup([3, 0], [20, 9], 2, 128, 32, 8, "bf16", seed=4)
    n = s.rows.shape[0]
    hold = torch.zeros((2, n, 136 + 8), dtype=torch.bfloat16, device="cuda")
    v = hold[:, :, 8:136].transpose(0, 1)
    v.copy_(s.rows)
    s.check(gsk, v)
    s.check(gsk, s.rows[:1].expand(n, 2, 128))              # one row for all
    s.check(gsk, s.rows, stream=torch.cuda.Stream())
    with pytest.raises(gsk.CsaError):
        s.check(gsk, torch.zeros((n, 2, 132), dtype=torch.bfloat16, device="cuda")[:, :, 4:])


def test_row_by_row_equals_at_once(gsk):
    """Normal values keep their bits when a block's scale grows (here every value
    is above 2^-6 of the final scale, so none is rounded twice)."""
    r = np.random.default_rng(7)
    n, D, page, block = 37, 64, 16, 16
    x = torch.from_numpy((1 + r.random((n, 1, D))) * 2.0 ** r.integers(0, 4, (n, 1, 1))).to(torch.bfloat16).cuda()
    table = i32([[2, 0, 1]])

    def empty():
        return (torch.zeros((3, 1, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                torch.zeros((3, 1, 1), device="cuda"))

    a, sa = empty()
    gsk.csa_cache_append(x, a, sa, table, i32([0]), i32([0, n]))
    b, sb = empty()
    for i in range(n):
        gsk.csa_cache_append(x[i:i + 1], b, sb, table, i32([i]), i32([0, 1]))
    assert torch.equal(sa, sb) and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_bad_tables_stay_inside(gsk):
    """Pages outside the pool, missing pages, rows behind the table, lengths and
    offsets that make no sense: skipped, everything else written."""
    s = Setup([0, 0, 0, 0], [16, 16, 16, 40], 1, 64, 16, 16, "bf16", seed=9, width=2)
    s.table[0, 0], s.table[1, 0] = -1, 10 ** 6
    cache = torch.from_numpy(s.bytes.copy()).cuda().view(torch.float8_e4m3fn)
    scales = torch.from_numpy(s.scales.copy()).cuda()
    gsk.csa_cache_append(s.rows, cache, scales, i32(s.table), i32([0] * 4), i32(s.cu))
    got = cache.view(torch.uint8).cpu().numpy()
    want_c, want_s = s.bytes.copy(), s.scales.astype(np.float64)
    rows = s.rows.double().cpu().numpy()
    cache_ref.append(want_c, want_s, s.table[2:], [0, 0], rows, np.array([32, 48, 48 + 32]))
    np.testing.assert_array_equal(got, want_c)
    for lens, cu in (([-5] * 4, s.cu), ([0] * 4, [0, -3, 5, 4, 2 ** 30]), ([2 ** 31 - 1] * 4, s.cu)):
        gsk.csa_cache_append(s.rows, cache, scales, i32(s.table), i32(lens), i32(cu))
    torch.cuda.synchronize()


def test_refusals(gsk):
    s = Setup([0], [4], 2, 64, 16, 16, "bf16")
    cache = torch.from_numpy(s.bytes).cuda().view(torch.float8_e4m3fn)
    scales = torch.from_numpy(s.scales).cuda()
    t, h, cu = i32(s.table), i32([0]), i32(s.cu)
    for bad in (s.rows[:, :1], s.rows[..., :32], s.rows[0]):
        with pytest.raises(ValueError):
            gsk.csa_cache_append(bad, cache, scales, t, h, cu)
    with pytest.raises(ValueError):
        gsk.csa_cache_append(s.rows, cache, scales, t, h, cu[:1])
    with pytest.raises(ValueError):
        gsk.csa_cache_append(s.rows, cache, scales[:, :1], t, h, cu)
    with pytest.raises(TypeError):
        gsk.csa_cache_append(s.rows.double(), cache, scales, t, h, cu)
    with pytest.raises(TypeError):
        gsk.csa_cache_append(s.rows, cache, scales, t.long(), h, cu)
    gsk.csa_cache_append(s.rows[:0], cache, scales, t, h, i32([0, 0]))   # nothing to do


def test_past_32_bits(gsk):
    """A pool of more than 2^32 bytes: the last page's bytes."""
    pages, page, D = 2 ** 32 // (256 * 512) + 2, 256, 512
    cache = torch.zeros((pages, 1, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros((pages, 1, 1), device="cuda")
    x = torch.randn((300, 1, D), device="cuda").to(torch.bfloat16)
    gsk.csa_cache_append(x, cache, scales, i32([[pages - 1, 0]]), i32([0]), i32([0, 300]))
    got = cache.view(torch.uint8)[[pages - 1, 0]].cpu().numpy()
    want, ws = np.zeros((2, 1, page, D), np.uint8), np.zeros((2, 1, 1))
    cache_ref.append(want, ws, [[0, 1]], [0], x.double().cpu().numpy(), [0, 300])
    np.testing.assert_array_equal(got, want)
    assert int(cache.view(torch.uint8)[1:pages - 1].max()) == 0
