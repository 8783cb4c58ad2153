"""The operators as they are used together: compress, turn, cache, attend, fork
and go on; eagerly and replayed from a graph."""
import numpy as np
import pytest

import cache_ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gsk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_softmax_kv_gb300 as g
    g.build()
    return g


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_prompt_then_branches(gsk):
    """A prompt of three sequences is compressed, turned, cached and read; then
    two branches of the longest one each get a row of their own and are read."""
    D, ratio, coff, H, page, block = 128, 4, 2, 16, 16, 8
    lens = [37, 131, 3]
    rows = [n // ratio for n in lens]
    g = torch.Generator(device="cuda").manual_seed(0)
    T = sum(lens)
    kv = torch.randn((T, coff * D), generator=g, device="cuda").to(torch.bfloat16)
    score = torch.randn((T, coff * D), generator=g, device="cuda").to(torch.bfloat16)
    ape = torch.randn((ratio, coff * D), generator=g, device="cuda")
    cu = i32([0] + np.cumsum(lens).tolist())
    cuc = i32([0] + np.cumsum(rows).tolist())
    capacity = sum(rows) + 5
    comp = gsk.csa_compress_fwd(kv, score, ape, cu, cuc, capacity, ratio, coff, D)
    f, a = gsk.csa_rope_freqs(64, scaling="yarn", factor=4.0)
    turned = gsk.csa_rope(comp, f, cu_seqlens_comp=cuc, ratio=ratio, offset=64, amplitude=a)
    pages, seqs, width = 12, 5, 4
    cache = torch.zeros((pages, 1, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros((pages, 1, page // block), device="cuda")
    table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
    held = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    status = i32([0])
    new = i32(rows + [0, 0])
    gsk.csa_cache_reserve(cache, scales, table, held, refs, i32([0, 1, 2]), new[:3], status)
    cu_rows = torch.cat([cuc, cuc[-1:], cuc[-1:]])
    gsk.csa_cache_append(turned[:, None], cache, scales, table, held, cu_rows)
    held += new
    # queries of the last tokens, each sees the rows that end before or at it
    n_q = [37, 20, 3, 0, 0]
    q = torch.randn((sum(n_q), H, D), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.cat([torch.arange(n - k, n, device="cuda") for n, k in zip(lens, n_q)])
    q = gsk.csa_rope(q, f, pos, offset=64, amplitude=a)
    cu_q = [0] + np.cumsum(n_q).tolist()
    visible = ((pos + 1) // ratio).to(torch.int32)

    def check(q, cu_q, visible):
        out, lse = gsk.csa_cache_attend(q, cache, scales, table, held, i32(cu_q), 1, D ** -0.5, shared=True, visible=visible)
        want = cache_ref.attend(q.double().cpu().numpy(), cache.view(torch.uint8).cpu().numpy(),
                                scales.double().cpu().numpy(), table.tolist(), held.tolist(), cu_q, 1, D ** -0.5, True,
                                None if visible is None else visible.tolist())
        to, tl = cache_ref.attend_tolerance(*want, D, 64, 2.0 ** -7)
        assert (np.abs(out.double().cpu().numpy() - want[0]) <= to).all()
        fine = np.isfinite(want[1])
        l = lse.double().cpu().numpy()
        assert (np.isfinite(l) == fine).all() and (np.abs(l - want[1])[fine] <= tl[fine]).all()
        return out

    out = check(q, cu_q, visible)
    assert (out[:3] == 0).all()                             # the first tokens of a prompt see no row
    # what the cache stands for is the turned rows, to e4m3's half step (2^-4 relative, or half of
    # the smallest step, 2^-10 of a scale that is below amax / 224)
    x = cache_ref.TABLE[cache.view(torch.uint8).cpu().numpy()] * scales.double().cpu().numpy().repeat(block, -1)[..., None]
    t1 = x[table[1, :3].tolist()].reshape(-1, D)[:rows[1]]
    w1 = turned[rows[0]: rows[0] + rows[1]].double().cpu().numpy()
    assert (np.abs(t1 - w1) <= np.maximum(np.abs(w1) * 2.0 ** -4, np.abs(w1).max() / 224 * 2.0 ** -10)).all()
    # two branches of sequence 1
    assert rows[1] == 32
    gsk.csa_cache_fork(table, held, refs, i32([1, 1]), i32([3, 4]), page, status)
    grown = i32([1, 3, 4])
    for i in range(2):                                      # the second row comes next to the first
        gsk.csa_cache_reserve(cache, scales, table, held, refs, grown, i32([1, 1, 1]), status)
        own = torch.randn((3, 1, D), generator=g, device="cuda").to(torch.bfloat16) * 4 ** i
        gsk.csa_cache_append(own, cache, scales, table, held, i32([0, 0, 1, 1, 2, 3]))
        held[grown.long()] += 1
    assert status.item() == 0 and len({table[s, 2].item() for s in (1, 3, 4)}) == 3
    q1 = torch.randn((5, H, D), generator=g, device="cuda").to(torch.bfloat16)
    before = check(q1, [0, 1, 2, 3, 4, 5], None)
    gsk.csa_cache_free(table, held, refs, i32([0, 1]))
    live = i32([0])
    gsk.csa_cache_compact(cache, scales, table, refs, live)
    assert live.item() == int((refs > 0).sum())
    after = check(q1, [0, 1, 2, 3, 4, 5], None)
    assert (after[:2] == 0).all()
    tol = 2 * 2.0 ** -8 * before[2:].float().abs() + 1e-3 * before[2:].float().abs().amax()
    assert ((after[2:].float() - before[2:].float()).abs() <= tol).all()


def test_a_decoding_step_as_a_graph(gsk):
    """reserve, turn, append, lengths, attend in one captured graph, replayed ten
    times, against the same steps made eagerly."""
    D, H, page, block, seqs, width, pages = 512, 64, 16, 16, 6, 3, 30
    g = torch.Generator(device="cuda").manual_seed(1)
    f, _ = gsk.csa_rope_freqs(64)
    x = torch.randn((seqs, 1, D), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((seqs, H, D), generator=g, device="cuda").to(torch.bfloat16)
    all_seqs, ones, cu = i32(list(range(seqs))), i32([1] * seqs), i32(list(range(seqs + 1)))

    def world():
        return dict(cache=torch.zeros((pages, 1, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                    scales=torch.zeros((pages, 1, page // block), device="cuda"),
                    table=torch.full((seqs, width), -1, dtype=torch.int32, device="cuda"), held=i32([0] * seqs),
                    refs=i32([0] * pages), status=i32([0]), x=x.clone(), q=q.clone())

    def step(w):
        gsk.csa_cache_reserve(w["cache"], w["scales"], w["table"], w["held"], w["refs"], all_seqs, ones, w["status"])
        row = gsk.csa_rope(w["x"], f, w["held"], offset=448)
        gsk.csa_cache_append(row, w["cache"], w["scales"], w["table"], w["held"], cu)
        w["held"].add_(1)
        return gsk.csa_cache_attend(gsk.csa_rope(w["q"], f, w["held"], offset=448), w["cache"], w["scales"], w["table"],
                                    w["held"], cu, 1, D ** -0.5, shared=True)

    a, b = world(), world()
    b["held"].copy_(i32([0, 3, 15, 16, 17, 1]))
    a["held"].copy_(b["held"])
    for w in (a, b):                                        # rows that are there already: pages for them
        lens = w["held"].clone()
        w["held"].zero_()
        gsk.csa_cache_reserve(w["cache"], w["scales"], w["table"], w["held"], w["refs"], all_seqs, lens, w["status"])
        w["held"].copy_(lens)
        w["scales"].fill_(1.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    saved = {k: v.clone() for k, v in b.items()}
    with torch.cuda.stream(s):
        step(b)
    torch.cuda.current_stream().wait_stream(s)
    for k, v in saved.items():
        b[k].copy_(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(b)
    for i in range(10):
        for w in (a, b):
            w["x"].copy_(x * (i + 1))
            w["q"].copy_(q.roll(i, 0))
        eager = step(a)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager[0], out) and torch.equal(eager[1], lse)
        for k in ("table", "held", "refs", "scales", "status"):
            assert torch.equal(a[k], b[k]), k
        assert torch.equal(a["cache"].view(torch.uint8), b["cache"].view(torch.uint8))
    assert a["status"].item() == 0
