"""What qkv_attention's backward reads again must be as the forward saw it: a table or a cu_seqlens that was written to
in between is refused, as autograd refuses any saved tensor, and does not give gradients of another rotation."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["table", "cu", "none"])
def test_saved_tensors_written_to(which):
    from dynamic_short_convolutions_b200 import ops

    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((64, 4 * 64), generator=g, device="cuda").bfloat16().requires_grad_()
    table, cu = ops.rope_table(64, 64), torch.tensor([0, 20, 64], dtype=torch.int32, device="cuda")
    o = ops.qkv_attention(qkv, 2, 1, 64, table, cu_seqlens=cu)
    if which == "table":
        table.mul_(0.5)
    elif which == "cu":
        cu.copy_(torch.tensor([0, 30, 64], dtype=torch.int32))
    else:
        assert torch.isfinite(torch.autograd.grad(o, qkv, torch.ones_like(o))[0]).all()
        return
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(o, qkv, torch.ones_like(o))
