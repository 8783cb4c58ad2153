"""Waits inside the kernels of attention over packed sequences: work that lasts as long as its
sequence is long, with many query heads over one key head (a tile is a token or two)."""
import ctypes

import pytest

from test_gpu_prompt import gsk, i32, inputs, make  # noqa: F401

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
