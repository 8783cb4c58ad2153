"""autograd.prompt_attend where no gradient is wanted: the plain call, with nothing kept."""
import pytest

from test_gpu_prompt import gsk, i32, inputs  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["no_grad", "inference_mode", "leaves"])
def test_nothing_is_kept_where_no_gradient_is_wanted(gsk, how):  # noqa: F811
    from gated_softmax_kv_gb300 import autograd
    q, k, v = (t.requires_grad_(how != "leaves") for t in inputs([2000], [2000], 8, 2, 128, "bf16", 1))
    cu = i32([0, 2000])
    want = gsk.csa_prompt_attend(q.detach(), k.detach(), v.detach(), cu, 0.1, window=300)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with torch.no_grad() if how == "no_grad" else torch.inference_mode(how == "inference_mode"):
        out, lse = autograd.prompt_attend(q, k, v, cu, 0.1, window=300)
    made = out.numel() * 2 + lse.numel() * 4
    # torch's allocator counts whole blocks: it leaves a cached block unsplit when less than 2^20 bytes would remain (out, of
    # 4096000 bytes, comes from its pool of large blocks), and rounds lse's 64000 up to 512. A further tensor of out's
    # size would add 4096000.
    assert torch.cuda.max_memory_allocated() - before < made + 2 ** 20 + 512
    assert not out.requires_grad and not lse.requires_grad
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_a_gradient_of_one_input_keeps_what_it_needs(gsk):  # noqa: F811
    from gated_softmax_kv_gb300 import autograd
    q, k, v = inputs([200], [200], 4, 2, 64, "bf16", 1)
    cu, g = i32([0, 200]), torch.randn((200, 4, 64), device="cuda").bfloat16()
    want = None
    for name in ("all", "q", "k", "v"):
        t = {"q": q.clone(), "k": k.clone(), "v": v.clone()}
        need = [n for n in t if name in ("all", n)]
        for n in need:
            t[n].requires_grad_()
        out, lse = autograd.prompt_attend(t["q"], t["k"], t["v"], cu, 0.1)
        got = dict(zip(need, torch.autograd.grad(out, [t[n] for n in need], g)))
        want = want or got
        assert all(torch.equal(got[n], want[n]) for n in need)
