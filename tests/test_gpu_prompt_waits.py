"""Waits inside the kernels of attention over packed sequences: work that lasts as long as its
sequence is long, with many query heads over one key head (a tile is a token or two)."""
import ctypes

import pytest

from test_gpu_prompt import gsk, i32, inputs, make, sums  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture
def polls(gsk):  # noqa: F811
    """The limit of a wait, put back after the test."""
    from gated_softmax_kv_gb300.binding import load
    limit = ctypes.c_int32.in_dll(load(), "csa_prompt_polls")
    usual = limit.value
    assert usual == 1 << 20
    yield limit
    limit.value = usual


def test_an_item_may_outlast_the_limit_of_a_wait(gsk, polls):  # noqa: F811
    """6000 tokens of 128 heads over one: a block of keys meets up to 6000 tiles, of a microsecond or
    more each; 1024 polls are 1.4 ms."""
    q, k, v = inputs([6000], [6000], 128, 1, 64, "bf16", 1)
    g, cu = make(q.shape, "bf16", 2), i32([0, 6000])

    def run():
        out, lse = gsk.csa_prompt_attend(q, k, v, cu, 0.125)
        return (out, lse, *gsk.csa_prompt_attend_bwd(q, k, v, out, lse, g, cu, 0.125))

    want = run()
    polls.value = 1024
    got = run()
    torch.cuda.synchronize()
    assert all(torch.isfinite(t).all() for t in want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


CALLS = [([700, 300, 1], None, 8, 2, 128, None), ([900, 40], None, 6, 2, 64, None), ([1200], None, 8, 1, 64, 100),
         ([130, 64], [2000, 900], 4, 2, 128, None), ([1], [9000], 8, 1, 128, None), ([1, 2], [5000, 5000], 16, 2, 128, 3000),
         ([2500, 9], None, 128, 1, 64, None)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("limit", [0, 2, 16])
def test_what_was_given_up_is_nan(gsk, polls, limit, dtype):  # noqa: F811
    """Waits of so few polls run out here and there (one is 1.4 us, a copy takes about as long). Each row
    of a result is NaN then, or right; nothing keeps what its memory held, and the next call is right."""
    from gated_softmax_kv_gb300 import prompt
    from gated_softmax_kv_gb300.binding import load
    lost = 0
    for nq, nk, H, KV, D, window in CALLS:
        q, k, v = inputs(nq, nk or nq, H, KV, D, dtype, 5)
        cu, ck = i32(sums(nq)), i32(sums(nk or nq))
        g, scale = make(q.shape, dtype, 6), 0.1
        how, _ = prompt._describe(q, k, v, cu, ck, scale, window)

        def forward():
            out, rest, lse = torch.full_like(q, 7.0), torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
            gsk.csa_prompt_attend(q, k, v, cu, scale, cu_k=ck, window=window, out=out, rest=rest, lse=lse)
            return out, rest, lse

        def backward(out, rest, lse):
            dq, dk, dv = (torch.full_like(t, 7.0) for t in (q, k, v))
            assert load().csa_prompt_attend_bwd(how, out.data_ptr(), rest.data_ptr(), lse.data_ptr(), g.data_ptr(), H * D, D, None,
                                                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                                torch.cuda.current_stream().cuda_stream) == 0
            return dq, dk, dv

        polls.value = 1 << 20
        want = forward()
        want += backward(*want)
        for _ in range(3):
            polls.value = limit
            got = forward()
            got += backward(*want[:3])
            polls.value = 1 << 20
            after = forward()
            after += backward(*after)
            torch.cuda.synchronize()
            for a, b, c in zip(got, want, after):
                assert torch.equal(c, b)
                nan = torch.isnan(a)
                if a.dim() == 3:
                    assert (nan.all(-1) == nan.any(-1)).all()
                assert torch.equal(torch.where(nan, b, a), b)
                lost += int(nan.sum())
            assert (torch.isnan(got[0]).all(-1) == torch.isnan(got[2])).all()
    assert lost > 0 or limit > 0
