"""qkv_attention where columns, rows or gradients start off a 16-byte boundary: one token with heads of odd widths, whose
column slices torch calls contiguous; rows out of the middle of a larger buffer; gradients that arrive as views of one."""
import pytest

from attn_reference import attention, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rows(n, heads, kv, hd, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda w: torch.randn((n, w * hd), generator=g, device="cuda").to(DT[dtype])
    return rnd(heads + 2 * kv), rnd(heads)


def _layer(qkv, go, heads, kv, hd, table, batch=1, cu=None):
    from dynamic_short_convolutions_b200 import ops

    leaf = qkv.detach().requires_grad_()
    o = ops.qkv_attention(leaf, heads, kv, hd, table, batch, cu)
    return o.detach(), torch.autograd.grad(o, leaf, go)[0]


@pytest.mark.parametrize("packed", [False, True], ids=["dense", "packed"])
@pytest.mark.parametrize("rot", [0, 4])
@pytest.mark.parametrize("heads,kv,hd", [(2, 1, 37), (3, 1, 5), (3, 3, 20), (1, 1, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_token_of_odd_heads(dtype, heads, kv, hd, rot, packed):
    """The first of two sequences of one token, alone and beside the other, bit by bit; unrotated against the formula."""
    two, go = _rows(2, heads, kv, hd, dtype, 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    table = torch.randn((1, rot), generator=g, device="cuda") if rot else None
    want = _layer(two, go, heads, kv, hd, table, 2)
    cu = torch.tensor([0, 0, 1, 1], dtype=torch.int32, device="cuda") if packed else None
    got = _layer(two[:1], go[:1], heads, kv, hd, table, 1, cu)
    assert torch.equal(got[0], want[0][:1]) and torch.equal(got[1], want[1][:1])
    if not rot:
        wq, wk = heads * hd, kv * hd
        q, k, v = two[:1, :wq], two[:1, wq:wq + wk], two[:1, wq + wk:]
        ref = attention(q, k, v, [0, 1], heads, kv, hd, go[:1], 0.0, 2.0 ** -7 if dtype == "bf16" else 0.0)
        d = got[1]
        for name, t in (("o", got[0]), ("dq", d[:, :wq]), ("dk", d[:, wq:wq + wk]), ("dv", d[:, wq + wk:])):
            check(name, t, ref[name])


@pytest.mark.parametrize("heads,kv,hd,rot", [(1, 1, 37, 0), (1, 1, 37, 4), (3, 1, 5, 2), (2, 1, 64, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_that_are_views(dtype, heads, kv, hd, rot):
    """Outputs joined by cat along the tokens and along the channels: autograd hands back views of the joined gradient."""
    from dynamic_short_convolutions_b200 import ops

    table = ops.rope_table(3, rot) if rot else None
    a, ga = _rows(3, heads, kv, hd, dtype, 3)
    b, gb = _rows(3, heads, kv, hd, dtype, 4)
    want = [_layer(x, g, heads, kv, hd, table)[1] for x, g in ((a, ga), (b, gb))]
    a.requires_grad_()
    b.requires_grad_()
    outs = [ops.qkv_attention(x, heads, kv, hd, table) for x in (a, b)]
    got = torch.autograd.grad(torch.cat(outs), (a, b), torch.cat((ga, gb)))
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    outs = [ops.qkv_attention(x[:1], heads, kv, hd, table) for x in (a, b)]
    odd = ga.new_ones((1, 1))
    got = torch.autograd.grad(torch.cat((odd, *outs), 1), (a, b), torch.cat((odd, ga[:1], gb[:1]), 1))
    for x, g, d in ((a, ga, got[0]), (b, gb, got[1])):
        assert torch.equal(d[:1], _layer(x[:1], g[:1], heads, kv, hd, table)[1]) and not d[1:].any()


@pytest.mark.parametrize("heads,kv,hd,rot", [(1, 1, 37, 0), (3, 1, 5, 2), (2, 1, 64, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_a_larger_buffer(dtype, heads, kv, hd, rot):
    """qkv that starts at an odd row, or at an odd column, of a buffer."""
    from dynamic_short_convolutions_b200 import ops

    table = ops.rope_table(4, rot) if rot else None
    rows, go = _rows(4, heads, kv, hd, dtype, 5)
    want = _layer(rows, go, heads, kv, hd, table)
    flat = torch.empty(rows.numel() + 1, dtype=rows.dtype, device="cuda")
    wide = torch.empty((4, rows.shape[1] + 3), dtype=rows.dtype, device="cuda")
    for view in (flat[1:].view(rows.shape), wide[:, 3:]):
        view.copy_(rows)
        assert view.data_ptr() % 16
        got = _layer(view, go, heads, kv, hd, table)
        # 64 channels: strided rows run on other kernels than dense ones, and the copy on those of dense ones
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
