"""csa_cache_attend against the 64-bit attention; tolerances in
cache_ref.attend_tolerance."""
import math

import numpy as np
import pytest

import cache_ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


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
    def __init__(self, lens, queries, heads, kv, D, shared, page=64, block=16, dtype="bf16", seed=0, extra=0,
                 spread=3):
        r = np.random.default_rng(seed)
        self.lens, self.kv, self.shared, self.D = list(lens), kv, shared, D
        H = kv * (1 if shared else 2)
        pages = sum(-(-n // page) for n in lens) + 2
        order = r.permutation(pages)
        width = max(1, max(-(-n // page) for n in lens))
        self.table = np.full((len(lens), width), -1)
        at = 0
        for s, n in enumerate(lens):
            k = -(-n // page)
            self.table[s, :k] = order[at:at + k]
            at += k
        x = r.standard_normal((pages, H, page, D))
        x = np.clip(x * 100, -448, 448)
        self.scales = (2.0 ** r.integers(-7 - spread, -6, (pages, H, page // block))).astype(np.float32)
        self.bytes = cache_ref.quantise(x)
        # everything behind a sequence's last row, and the pages of nobody, is NaN
        mask = np.ones((pages, page), bool)
        for s, n in enumerate(lens):
            for j in range(n):
                mask[self.table[s, j // page], j % page] = False
        self.bytes[np.broadcast_to(mask[:, None, :, None], self.bytes.shape)] = 0x7F
        self.cu = np.concatenate([[0], np.cumsum(queries)])
        self.T = int(self.cu[-1]) + extra
        self.q = torch.from_numpy(r.standard_normal((self.T, heads, D))).to(DTYPES[dtype]).cuda()
        self.scale = D ** -0.5
        self.visible = None

    def args(self):
        return (torch.from_numpy(self.bytes).cuda().view(torch.float8_e4m3fn),
                torch.from_numpy(self.scales).cuda(), i32(self.table), i32(self.lens), i32(self.cu), self.kv,
                self.scale)

    def run(self, gsk, q=None, **kw):
        args = self.args()
        visible = None if self.visible is None else i32(self.visible)
        torch.cuda.synchronize()                            # inputs are there for any stream
        return gsk.csa_cache_attend(self.q if q is None else q, *args, shared=self.shared, visible=visible, **kw)

    def check(self, gsk, q=None, **kw):
        q = self.q if q is None else q
        out, lse = self.run(gsk, q, **kw)
        torch.cuda.synchronize()
        n = int(self.cu[-1])
        want = cache_ref.attend(q[:n].double().cpu().numpy(), self.bytes, self.scales.astype(np.float64), self.table,
                                self.lens, self.cu, self.kv, self.scale, self.shared, self.visible)
        tol_o, tol_l = cache_ref.attend_tolerance(*want, self.D, max(self.lens + [1]),
                                                  torch.finfo(out.dtype).eps)
        o, l = out[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()
        np.testing.assert_array_equal(np.isnan(o), np.isnan(want[0]))
        np.testing.assert_array_equal(np.isinf(l), np.isinf(want[1]))
        fine = ~np.isnan(want[0])
        bad = fine & ~(np.abs(o - want[0]) <= tol_o)
        assert not bad.any(), (np.argwhere(bad)[:4], o[bad][:4], want[0][bad][:4], tol_o[bad][:4], bad.sum())
        fine = np.isfinite(want[1])
        bad = fine & ~(np.abs(np.where(fine, l - np.where(fine, want[1], 0), 0)) <= tol_l)
        assert not bad.any(), (np.argwhere(bad)[:4], l[bad][:4], want[1][bad][:4], bad.sum())
        return out, lse


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 130, 300]


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("kv,group", [(1, 1), (2, 3), (1, 16), (2, 8), (1, 20), (1, 64)])
def test_single_tokens(gsk, D, shared, kv, group):
    Setup(LENS, [1] * len(LENS), kv * group, kv, D, shared, seed=D + group).check(gsk)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page,block", [(16, 1), (16, 16), (32, 8), (128, 128), (256, 32), (64, 2)])
def test_pages_and_blocks(gsk, page, block, dtype):
    for D, shared, kv, group in ((128, False, 2, 4), (512, True, 1, 8), (512, True, 1, 64), (64, True, 3, 1)):
        Setup([300, 33, 0, 257], [1, 1, 1, 1], kv * group, kv, D, shared, page, block, dtype, seed=page).check(gsk)


@pytest.mark.parametrize("D,shared,kv,group", [(64, False, 2, 1), (128, False, 2, 4), (128, True, 1, 16), (256, False, 1, 2),
                                               (512, True, 1, 8), (512, True, 1, 64), (512, False, 1, 3), (64, True, 1, 40)])
def test_chunks_of_queries_with_their_past(gsk, D, shared, kv, group):
    """Each query sees the rows before it; the first ones see none; NaN in rows
    that only some of a tile's queries see stays with those."""
    lens, queries = [70, 5, 0, 129, 40], [30, 21, 3, 17, 0]
    s = Setup(lens, queries, kv * group, kv, D, shared, 32, 16, "bf16", seed=D, extra=3)
    vis = []
    for n, k in zip(lens, queries):
        vis += [max(0, n - k // 2 + i) for i in range(k)] if n else [7] * k
    vis[0], vis[1], vis[2] = 0, -4, 1
    s.visible = vis + [5] * 3
    out, lse = s.check(gsk)
    # NaN in a row that the later queries see: they get NaN, the earlier ones their old bits
    j = 60
    s.bytes[s.table[0, j // 32], :, j % 32, 3] = 0x7F
    out2, lse2 = s.check(gsk)
    sees = np.array(s.visible[:30]) > j
    assert sees.any() and not sees.all()
    assert torch.equal(out2[:30][~sees], out[:30][~sees]) and torch.equal(lse2[:30][~sees], lse[:30][~sees])


def test_rows_behind_the_last_sequence_stay(gsk):
    for D, group in ((128, 4), (512, 64)):
        s = Setup([40, 9], [2, 3], group, 1, D, True, seed=1, extra=5)
        out = torch.full((s.T, group, D), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((s.T, group), 4.0, device="cuda")
        got = s.check(gsk, out=out, lse=lse)
        assert got[0] is out and (out[5:] == 3).all() and (lse[5:] == 4).all()


@pytest.mark.parametrize("D,group", [(64, 2), (128, 8), (512, 4), (512, 64)])
def test_ranges_of_values(gsk, D, group):
    """Far apart scales, large logits, a scale that outweighs the attended block's, infinities and NaN in q."""
    s = Setup([200, 64, 30, 100], [1] * 4, group, 1, D, True, 16, 16, "bf16", seed=5, spread=20)
    s.check(gsk)
    s.scale = 3.0                                           # one row takes nearly everything
    s.check(gsk)
    s.scale = -0.2
    s.check(gsk)
    s.scale = 0.0                                           # the mean
    s.check(gsk)
    s.scale = D ** -0.5
    # a block of huge values that no weight falls on, beside ordinary ones
    far = Setup([40], [1], 2 * group, 2, D, False, 16, 16, "bf16", seed=6)
    far.bytes[far.table[0, 0], :2, :, 0] = 0xF8             # keys of block 0: far below
    far.q[..., 0] = 30.0
    far.scale = 1.0
    far.scales[far.table[0, 0], 2:] = 2.0 ** 60
    far.bytes[far.table[0, 1], :2, :, 0] = 0x38
    far.check(gsk)
    s.q[0, 0, 3], s.q[1, group - 1, 5] = math.inf, math.nan
    out, lse = s.run(gsk)
    assert torch.isnan(out[0, 0]).all() and torch.isnan(out[1, group - 1]).all()
    assert torch.isfinite(out[2:]).all() and torch.isfinite(out[0, 1:]).all()
    t = Setup([33, 20], [1, 1], group, 1, D, True, 16, 16, "fp16", seed=8)
    t.q.clamp_(-3, 3).mul_(20000.0)                         # near fp16's largest value
    t.scale = 1e-4
    t.check(gsk)
    t.q.mul_(1e-9)                                          # fp16 subnormals
    t.scale = 1.0
    t.check(gsk)
    u = Setup([33, 20], [1, 1], group, 1, D, True, 16, 16, "bf16", seed=8)
    u.q.mul_(2.0 ** 100)
    u.scale = 2.0 ** -104
    u.check(gsk)
    u.q.mul_(2.0 ** -126).mul_(2.0 ** -60)
    u.scale = 2.0 ** 80
    u.check(gsk)


def test_nan_and_infinite_rows(gsk):
    for D, group in ((128, 3), (512, 64)):
        s = Setup([50, 50], [1, 1], group, 1, D, True, 16, 16, seed=3)
        s.bytes[s.table[0, 1], 0, 4, 7] = 0xFF
        out, lse = s.check(gsk)
        assert torch.isnan(lse[0]).all() and torch.isfinite(out[1]).all()
        t = Setup([50, 50], [1, 1], group, 1, D, False, 16, 16, seed=3)
        t.bytes[t.table[0, 1], 1, 4, 7] = 0x7F               # a value: its column alone
        out, lse = t.run(gsk)
        bad = torch.isnan(out[0])
        assert bad[:, 7].all() and int(bad.sum()) == group and torch.isfinite(lse).all()


def test_zero_scales(gsk):
    """Blocks that stand for zeros: their keys have logit 0, their values add nothing."""
    for D, group in ((128, 3), (512, 64)):
        s = Setup([50, 20], [1, 1], group, 1, D, True, 16, 16, seed=3)
        s.scales[s.table[0, 1]] = 0.0
        s.scales[s.table[1, :2]] = 0.0
        out, lse = s.check(gsk)
        assert (out[1] == 0).all()


def test_missing_pages_are_not_seen(gsk):
    for D, group in ((128, 3), (512, 64)):
        s = Setup([100, 64, 20], [1, 2, 1], group, 1, D, True, 16, 8, seed=4)
        s.table[0, 2], s.table[1, 0], s.table[2, :2] = -1, 10 ** 7, -7
        out, lse = s.check(gsk)
        assert (out[3] == 0).all() and (lse[3] == -math.inf).all()
        s.lens = [10 ** 9, 64, 20]                           # more rows than the table holds: cut
        long = s.run(gsk)
        s.lens = [s.table.shape[1] * 16, 64, 20]
        cut = s.run(gsk)
        # the last page's tail is NaN in this set-up, so both are, alike
        assert torch.equal(long[0].view(torch.int16), cut[0].view(torch.int16))


def test_strides_streams_and_repeats(gsk):
    s = Setup([200, 33, 90], [1, 2, 1], 8, 2, 128, False, seed=11)
    base = torch.zeros((8, 4, 160), dtype=torch.bfloat16, device="cuda")
    q = base[:, :, 16:144].transpose(0, 1)
    q.copy_(s.q)
    a = s.check(gsk, q)
    b = s.check(gsk)
    assert torch.equal(a[0], b[0])
    one = s.q[:1, :1].expand(4, 8, 128)
    s.check(gsk, one)
    side = torch.cuda.Stream()
    c = s.run(gsk, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(c[0], b[0]) and torch.equal(c[1], b[1])


@pytest.mark.parametrize("D,shared,kv,group,n", [(128, False, 2, 8, 5000), (512, True, 1, 16, 3000), (512, True, 1, 64, 4000),
                                                 (64, True, 1, 1, 9000), (512, True, 1, 128, 2000), (128, True, 1, 128, 6000),
                                                 (64, True, 2, 128, 4000), (64, False, 1, 80, 5000)])
def test_long_sequences_are_split_and_joined(gsk, D, shared, kv, group, n):
    """One long sequence next to short ones, against a 64-bit product on the GPU."""
    lens = [n, 3, 0, 700]
    g = torch.Generator(device="cuda").manual_seed(n)
    page, pages = 64, sum(-(-x // 64) for x in lens)
    H = kv * (1 if shared else 2)
    bits = (torch.randn((pages, H, page, D), generator=g, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = torch.exp2(torch.randint(-8, -5, (pages, H, 4), generator=g, device="cuda").float())
    order = torch.randperm(pages, generator=g, device="cuda").tolist()
    width, at = -(-n // 64), 0
    table = np.full((4, width), -1)
    for i, x in enumerate(lens):
        k = -(-x // 64)
        table[i, :k] = order[at:at + k]
        at += k
    q = torch.randn((4, kv * group, D), generator=g, device="cuda").to(torch.bfloat16)

    def call():
        return gsk.csa_cache_attend(q, bits, scales, i32(table), i32(lens), i32([0, 1, 2, 3, 4]), kv, D ** -0.5,
                                    shared=shared)

    out, lse = call()
    for _ in range(3):
        again = call()
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    x = bits.double() * scales.double().repeat_interleave(16, -1)[..., None]
    for i, m in enumerate(lens):
        if m == 0:
            assert (out[i] == 0).all() and (lse[i] == -math.inf).all()
            continue
        rows = x[torch.tensor(table[i, :-(-m // 64)], device="cuda")].transpose(0, 1).reshape(H, -1, D)[:, :m]
        for h in range(kv):
            k, v = rows[h], rows[h if shared else kv + h]
            qq = q[i, h * group:(h + 1) * group].double()
            z = (qq @ k.T) * D ** -0.5
            p = torch.softmax(z, -1)
            want, mass = p @ v, p @ v.abs()
            dz = (qq.abs() @ k.abs().T).amax(-1) * D ** -0.5
            l = torch.logsumexp(z, -1)
            to, tl = cache_ref.attend_tolerance(want.cpu().numpy(), l.cpu().numpy(), mass.cpu().numpy(), dz.cpu().numpy(), D, m,
                                                2.0 ** -7)
            hs = slice(h * group, (h + 1) * group)
            assert ((out[i, hs].double() - want).abs().cpu().numpy() <= to).all()
            assert ((lse[i, hs].double() - l).abs().cpu().numpy() <= tl).all()


def test_many_sequences(gsk):
    """More sequences than there are thread blocks, most of them short or empty."""
    r = np.random.default_rng(5)
    lens = r.integers(0, 40, 700).tolist()
    for D, shared, kv, group in ((64, False, 1, 2), (512, True, 1, 32)):
        s = Setup(lens, [1] * 700, kv * group, kv, D, shared, 16, 16, seed=6)
        s.check(gsk)


def test_graphs_replay_on_new_lengths(gsk):
    """Two captured graphs, replayed in turn with lengths that changed since."""
    sets = []
    for D, group in ((128, 8), (512, 64)):
        s = Setup([400, 100, 7], [1, 1, 1], group, 1, D, True, seed=D)
        args = s.args()
        out, lse = s.run(gsk)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gsk.csa_cache_attend(s.q, *args, shared=True, out=out, lse=lse)
        sets.append((s, args, graph, out, lse))
    for lens in ([400, 100, 7], [1, 0, 5], [390, 64, 0]):
        for s, args, graph, out, lse in sets:
            args[3].copy_(i32(lens))
        for s, args, graph, out, lse in sets:
            graph.replay()
        torch.cuda.synchronize()
        for s, args, graph, out, lse in sets:
            s.lens = lens
            want = s.run(gsk)
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_refusals(gsk):
    s = Setup([20], [2], 4, 2, 64, False)
    a = s.args()
    for q in (s.q[:, :, :32], s.q[0], s.q.transpose(1, 2)):
        with pytest.raises(ValueError):
            gsk.csa_cache_attend(q, *a)
    with pytest.raises(TypeError):
        gsk.csa_cache_attend(s.q.float(), *a)
    with pytest.raises(ValueError):
        gsk.csa_cache_attend(s.q, *a, visible=i32([1]))
    with pytest.raises(ValueError):
        gsk.csa_cache_attend(s.q, *a, out=s.q)
    with pytest.raises(ValueError):
        gsk.csa_cache_attend(s.q, *a, lse=torch.zeros(2, 3, device="cuda"))
    for kv in (0, 3, 4):
        with pytest.raises(gsk.CsaError):
            gsk.csa_cache_attend(s.q, *a[:5], kv, 1.0)
    with pytest.raises(gsk.CsaError):                       # rows that are not 16-byte aligned
        gsk.csa_cache_attend(torch.zeros(2, 4, 68, dtype=torch.bfloat16, device="cuda")[:, :, 4:], *a)
    out, lse = gsk.csa_cache_attend(s.q[:0], *a[:4], i32([0, 0]), *a[5:])
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_a_pool_past_32_bits(gsk):
    pages, page, D = 2 ** 32 // (256 * 512) + 2, 256, 512
    cache = torch.zeros((pages, 1, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros((pages, 1, 1), device="cuda")
    s = Setup([300], [1], 64, 1, D, True, 256, 256, seed=1)
    t = [pages - 1, pages - 2]
    cache.view(torch.uint8)[t] = torch.from_numpy(s.bytes[s.table[0, :2]]).cuda()
    scales[t] = torch.from_numpy(s.scales[s.table[0, :2]]).cuda()
    for h in (64, 4):
        got = gsk.csa_cache_attend(s.q[:, :h].contiguous(), cache, scales, i32([t]), i32([300]), i32([0, 1]), 1, s.scale, shared=True)
        small = gsk.csa_cache_attend(s.q[:, :h].contiguous(), *s.args(), shared=True)
        assert torch.equal(got[0], small[0])


@pytest.mark.parametrize("D,shared,kv,group,queries", [(64, True, 1, 2, 1), (64, False, 2, 3, 5), (128, False, 2, 8, 1),
                                                       (256, True, 1, 4, 3), (512, False, 1, 5, 1), (512, True, 1, 64, 1),
                                                       (128, False, 1, 8, 20), (256, False, 1, 64, 1), (64, True, 1, 64, 2),
                                                       (64, False, 2, 70, 1)])
def test_short_and_wide_tables(gsk, D, shared, kv, group, queries):
    """Items are cut or not by the width of the table: the same sequences under a
    table just wide enough, and under ones that have room for far more rows."""
    lens = [250, 1, 0, 97, 256, 16, 130]
    s = Setup(lens, [queries] * len(lens), kv * group, kv, D, shared, 64, 16, seed=D + group)
    narrow, table = s.check(gsk), s.table
    for width in (16, 17, 40, 4000):
        s.table = np.full((len(lens), width), -1)
        s.table[:, :table.shape[1]] = table
        out, lse = s.check(gsk)
        seen = np.repeat(np.array(lens) > 0, queries)
        # each is within its tolerance of the same value; fewer than two rows need no sum
        one = np.repeat(np.array(lens) < 2, queries)
        assert torch.equal(out[one], narrow[0][one]) and torch.equal(lse[one], narrow[1][one])
        assert (out[~seen] == 0).all()


@pytest.mark.parametrize("D,group,tokens", [(64, 2, 8), (512, 4, 6), (128, 16, 40), (512, 64, 7)])
def test_queries_that_are_not_there(gsk, D, group, tokens):
    """Offsets that promise more queries than the call has give those of the call;
    decreasing and negative ones give none, and the other sequences theirs."""
    s = Setup([200], [tokens], group, 1, D, True, seed=D)
    want = s.check(gsk)
    a = list(s.args())
    for cu in ([0, 2 ** 30], [0, 2 ** 31 - 1]):
        a[4] = i32(cu)
        out, lse = gsk.csa_cache_attend(s.q, *a, shared=True)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    a[2], a[3] = i32(np.repeat(s.table, 3, 0)), i32([200] * 3)
    for cu, first in (([9, 2, 0, tokens], 0), ([-2 ** 31, -5, 2, tokens], 2), ([2 ** 31 - 1, -2 ** 31, 2, 1], None)):
        a[4] = i32(cu)
        out, lse = torch.full_like(want[0], 3.0), torch.full_like(want[1], 3.0)
        gsk.csa_cache_attend(s.q, *a, shared=True, out=out, lse=lse)
        if first is not None:
            # the same logits, summed from another split: 200 2^-24 for the sum, 2^-22 a
            # term and 128 2^-24 for its exponent, |lse| 2^-23 < 2^-16: below 2^-14 together
            assert ((lse[first:] - want[1][first:]).abs() <= 2.0 ** -14).all(), cu
            assert (lse[:first] == 3).all() and (out[:first] == 3).all()
        else:
            assert (out == 3).all() and (lse == 3).all()


def test_two_streams_at_once(gsk):
    """Calls of both kernels on two streams, each with its own workspace."""
    sets = []
    for D, group in ((128, 8), (512, 64)):
        s = Setup([3000, 900, 7], [1, 1, 1], group, 1, D, True, seed=D)
        sets.append((s, s.args(), s.check(gsk), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k, (s, args, want, stream) in enumerate(sets):
            got[k].append(gsk.csa_cache_attend(s.q, *args, shared=True, stream=stream))
    torch.cuda.synchronize()
    for k, (s, args, want, stream) in enumerate(sets):
        for out, lse in got[k]:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
