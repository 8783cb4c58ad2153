"""Outputs that the caller gives, x itself among them, are known to autograd as
changed: a graph that had saved their old values refuses its backward pass."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gsk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_softmax_kv_gb300 as g
    g.build()
    return g


def test_rope_in_place_on_a_saved_tensor(gsk):
    f, _ = gsk.csa_rope_freqs(64)
    pos = torch.arange(4, device="cuda")
    for whole in (True, False):                             # the tensor itself, a view of it, apart
        x = torch.randn(4, 2, 64, device="cuda")
        w = torch.ones(4, 2, 64, device="cuda", requires_grad=True)
        y = (w * x).sum()
        view = x if whole else x[1:3]
        gsk.csa_rope(view, f, pos if whole else pos[1:3], out=view)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    x, out = torch.randn(4, 2, 64, device="cuda"), torch.zeros(4, 2, 64, device="cuda")
    y = (w * out).sum() + (w * x).sum()
    gsk.csa_rope(x, f, pos, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_rope_leaves_its_input_alone(gsk):
    f, _ = gsk.csa_rope_freqs(64)
    pos = torch.arange(4, device="cuda")
    x = torch.randn(4, 2, 64, device="cuda")
    w = torch.ones(4, 2, 64, device="cuda", requires_grad=True)
    y = (w * x).sum()
    gsk.csa_rope(x, f, pos)
    gsk.csa_rope(x, f, pos, out=torch.empty_like(x))
    y.backward()
    assert torch.equal(w.grad, x)
    with torch.inference_mode():                            # such tensors keep no count of changes
        z = torch.randn(4, 2, 64, device="cuda")
        want = gsk.csa_rope(z, f, pos)
        assert torch.equal(gsk.csa_rope(z, f, pos, out=z), want)


def test_attention_into_a_saved_tensor(gsk):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = torch.zeros(2, 2, 16, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.ones(2, 2, 1, device="cuda")
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    args = (cache, scales, i32([[0]]), i32([5]), i32([0, 2]), 1, 0.125)
    for which in ("out", "lse"):
        hold = {"out": torch.zeros_like(q), "lse": torch.zeros(2, 4, device="cuda")}
        w = torch.ones_like(hold[which], requires_grad=True)
        y = (w * hold[which]).sum()
        gsk.csa_cache_attend(q, *args, **hold)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    with torch.inference_mode():
        hold = torch.zeros_like(q)
        gsk.csa_cache_attend(q, *args, out=hold)


def test_attention_carries_no_gradient(gsk):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = torch.zeros(2, 2, 16, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    q = torch.randn(2, 4, 64, device="cuda").bfloat16().requires_grad_()
    out, lse = gsk.csa_cache_attend(q, cache, torch.ones(2, 2, 1, device="cuda"), i32([[0]]), i32([5]), i32([0, 2]), 1, 0.125)
    assert not out.requires_grad and not lse.requires_grad
    assert "Not recorded by autograd" in gsk.csa_cache_attend.__doc__
