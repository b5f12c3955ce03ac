"""What the device finds wrong in an autograd call reaches the caller who gives `errors`: documents longer than the
table, a malformed cu_seqlens, in forward and backward, through a graph; a good call leaves it alone, and the results
are those without it."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HEADS, KV, HD, N = 4, 2, 64, 300
C = (HEADS + 2 * KV) * HD


def _cu(*at):
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _call(layer, dtype, cu, table, errors):
    """(leaves, o) of qkv_attention, or of the layer with the convolution before it."""
    from dynamic_short_convolutions_b200 import ops

    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype).requires_grad_()
    if not layer:
        leaves = [rnd(N, C)]
        return leaves, ops.qkv_attention(*leaves, HEADS, KV, HD, table, cu_seqlens=cu, errors=errors)
    leaves = [rnd(N, C), rnd(N, 64), rnd(64, 16), rnd(16, 3 * C)]
    return leaves, ops.dynamic_conv_attention(*leaves, 3, HEADS, KV, HD, table, cu_seqlens=cu, errors=errors)


def _status(errors):
    from dynamic_short_convolutions_b200 import _lib as L

    return L.dynconv_device_status(errors), L.dynconv_last_error()


@pytest.mark.parametrize("layer", [False, True], ids=["attention", "layer"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_a_good_call(dtype, layer):
    from dynamic_short_convolutions_b200 import ops

    table, errors = ops.rope_table(N, HD), torch.zeros(256, dtype=torch.uint8, device="cuda")
    runs = []
    for e in (None, errors):
        leaves, o = _call(layer, dtype, _cu(0, 100, N), table, e)
        runs.append([o, *torch.autograd.grad(o, leaves, torch.ones_like(o))])
    for a, b in list(zip(*runs))[:2]:                # o, and what the attention hands back
        assert torch.equal(a, b)
    assert not errors.any() and _status(errors)[0] == 0


@pytest.mark.parametrize("layer", [False, True], ids=["attention", "layer"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_a_document_longer_than_the_table(dtype, layer):
    from dynamic_short_convolutions_b200 import ops

    table, errors = ops.rope_table(150, HD), torch.zeros(256, dtype=torch.uint8, device="cuda")
    leaves, o = _call(layer, dtype, _cu(0, 100, N), table, errors)
    code, text = _status(errors)
    assert code == 5 and "longer" in text and not errors.any()
    torch.autograd.grad(o, leaves, torch.ones_like(o))           # the backward rotates back
    code, text = _status(errors)
    assert code == 5 and "longer" in text


@pytest.mark.parametrize("layer", [False, True], ids=["attention", "layer"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("at", [(0, 200, 100, N), (0, 100), (5, N)], ids=str)
def test_malformed_documents(at, dtype, layer):
    errors = torch.zeros(300, dtype=torch.uint8, device="cuda")
    leaves, o = _call(layer, dtype, _cu(*at), None, errors)
    code, text = _status(errors)
    assert code == 5 and "cu_seqlens" in text
    if not layer:
        torch.autograd.grad(o, leaves, torch.ones_like(o))
        code, text = _status(errors)
        assert code == 5 and "cu_seqlens" in text
    leaves, o = _call(layer, dtype, _cu(0, 100, N), None, errors)
    torch.autograd.grad(o, leaves, torch.ones_like(o))
    assert _status(errors)[0] == 0


def test_errors_of_the_backward():
    """The bit of a wait that ran out, set on the host in the workspaces that the backward reads its errors from."""
    from dynamic_short_convolutions_b200 import ops

    errors = torch.zeros(256, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16().requires_grad_()
    u, h, A, B = rnd(N, C), rnd(N, 64), rnd(64, 16), rnd(16, 3 * C)
    y = ops.dynamic_short_conv(u, h, A, B, 3, errors=errors)
    o = ops.qkv_attention(y, HEADS, KV, HD, errors=errors)
    for out, to in ((y, u), (o, y)):
        assert _status(errors)[0] == 0
        out.grad_fn.plan.ws[0] = 2
        torch.autograd.grad(out, to, torch.ones_like(out), retain_graph=True)
        code, text = _status(errors)
        assert code == 5 and "timed out" in text


def test_through_a_graph():
    from dynamic_short_convolutions_b200 import ops

    table, errors, cu = ops.rope_table(150, HD), torch.zeros(256, dtype=torch.uint8, device="cuda"), _cu(0, 151, N)
    g = torch.Generator(device="cuda").manual_seed(2)
    qkv = torch.randn((N, C), generator=g, device="cuda").bfloat16()
    run = lambda: ops.qkv_attention(qkv, HEADS, KV, HD, table, cu_seqlens=cu, errors=errors)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    errors.zero_()
    graph.replay()
    assert _status(errors)[0] == 5
    cu.copy_(_cu(0, 150, N))
    graph.replay()
    torch.cuda.synchronize()
    graph.replay()
    assert _status(errors)[0] == 0


def test_what_cannot_hold_errors_is_refused():
    qkv_errors = [torch.zeros(255, dtype=torch.uint8, device="cuda"), torch.zeros(256, device="cuda"),
                  torch.zeros(512, dtype=torch.uint8, device="cuda")[::2], torch.zeros(257, dtype=torch.uint8, device="cuda")[1:],
                  torch.zeros(256, dtype=torch.uint8)]
    for layer in (False, True):
        for e in qkv_errors:
            with pytest.raises(ValueError, match="errors"):
                _call(layer, torch.float32, None, None, e)
