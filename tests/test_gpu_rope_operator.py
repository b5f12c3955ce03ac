"""The rotary operator (dynconv_rope) against a 64-bit restatement: both pair layouts, a part of the
head, strided rows, in place, forward and inverse, positions by place, by document and given."""
import pytest

from attn_reference import check, rope

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = {"bf16": 2.0 ** -7, "f32": 0.0}


def _table(max_pos, rot, **kw):
    from dynamic_short_convolutions_b200 import ops

    return ops.rope_table(max_pos, rot, device="cuda", **kw)


SHAPES = [  # batch, seqlen, heads, head_dim, rot_dim, extra columns
    (1, 1, 1, 2, 2, 0),
    (3, 7, 5, 64, 64, 0),
    (2, 33, 3, 128, 64, 24),
    (1, 130, 20, 128, 128, 256),
    (2, 5, 2, 20, 6, 0),            # runs that are no multiple of 16 bytes: the narrow kernel
    (1, 9, 7, 80, 40, 3),
    (4, 3, 3, 33, 10, 1),
]


@pytest.mark.parametrize("inverse", [False, True], ids=["forward", "inverse"])
@pytest.mark.parametrize("half", [False, True], ids=["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_rotation(shape, dtype, half, inverse):
    from dynamic_short_convolutions_b200 import _lib as L, ops

    batch, seqlen, heads, hd, rot, extra = shape
    N, width = batch * seqlen, heads * hd
    g = torch.Generator(device="cuda").manual_seed(1)
    buf = torch.randn((N, width + extra), generator=g, device="cuda").to(DT[dtype])
    x = buf[:, :width]
    table = _table(seqlen + 3, rot, scaling="yarn", factor=4.0, original_max_pos=64)
    plan = ops.RopePlan(DT[dtype], batch, seqlen, heads, hd, table, L.ROPE_HALF if half else L.ROPE_INTERLEAVED,
                        x_row_stride=width + extra)
    pos = torch.arange(N, device="cuda") % seqlen
    check("y", plan.apply(x, inverse=inverse), rope(x, table, pos, heads, hd, half, inverse, EPS[dtype]))
    assert L.dynconv_device_status(plan.ws) == 0


@pytest.mark.parametrize("half", [False, True], ids=["interleaved", "half"])
def test_documents_and_given_positions(half):
    from dynamic_short_convolutions_b200 import _lib as L, ops

    N, heads, hd = 41, 3, 64
    layout = L.ROPE_HALF if half else L.ROPE_INTERLEAVED
    x = torch.randn((N, heads * hd), device="cuda").bfloat16()
    table = _table(70000, 32)
    plan = ops.RopePlan(torch.bfloat16, 1, N, heads, hd, table, layout)
    cu = torch.tensor([0, 1, 1, 18, 41], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n) for n in (1, 17, 23)]).cuda()
    check("packed", plan.apply(x, cu_seqlens=cu), rope(x, table, pos, heads, hd, half, eps=2.0 ** -7))
    pos = torch.randint(0, 70000, (N,), dtype=torch.int32, device="cuda")
    check("given", plan.apply(x, positions=pos), rope(x, table, pos, heads, hd, half, eps=2.0 ** -7))
    assert L.dynconv_device_status(plan.ws) == 0


@pytest.mark.parametrize("half", [False, True], ids=["interleaved", "half"])
def test_in_place_leaves_the_other_columns(half):
    from dynamic_short_convolutions_b200 import _lib as L, ops

    N, heads, hd = 50, 4, 64
    buf = torch.randn((N, heads * hd + 64), device="cuda").bfloat16()
    before = buf.clone()
    table = _table(N, 32)
    plan = ops.RopePlan(torch.bfloat16, 1, N, heads, hd, table, L.ROPE_HALF if half else L.ROPE_INTERLEAVED,
                        x_row_stride=buf.shape[1], y_row_stride=buf.shape[1])
    x = buf[:, :heads * hd]
    out = plan.apply(x, y=x)
    assert out.data_ptr() == buf.data_ptr()
    pos = torch.arange(N, device="cuda")
    check("in place", x, rope(before[:, :heads * hd], table, pos, heads, hd, half, eps=2.0 ** -7))
    assert torch.equal(buf[:, heads * hd:], before[:, heads * hd:])


def test_positions_outside_the_table_raise_the_device_check():
    from dynamic_short_convolutions_b200 import _lib as L, ops

    table = _table(16, 64)
    plan = ops.RopePlan(torch.float32, 1, 4, 1, 64, table)
    x = torch.randn((4, 64), device="cuda")
    for bad in (-1, 16, 2 ** 31 - 1):
        pos = torch.tensor([0, 3, bad, 15], dtype=torch.int32, device="cuda")
        y = plan.apply(x, positions=pos)
        assert L.dynconv_device_status(plan.ws) == 5 and "position" in L.dynconv_last_error()
        good = torch.tensor([0, 1, 3], device="cuda")
        check("rows in range", y[good], rope(x[good], table, pos[good], 1, 64, False))
    plan.apply(x)
    assert L.dynconv_device_status(plan.ws) == 0
    long = ops.RopePlan(torch.float32, 1, 40, 1, 64, table)
    cu = torch.tensor([0, 17, 40], dtype=torch.int32, device="cuda")           # a document of 17 and one of 23
    long.apply(torch.randn((40, 64), device="cuda"), cu_seqlens=cu)
    assert L.dynconv_device_status(long.ws) == 5


def test_refusals():
    from dynamic_short_convolutions_b200 import _lib as L, ops

    table = _table(64, 64)
    x = torch.randn((8, 128), device="cuda")
    plan = ops.RopePlan(torch.float32, 1, 8, 2, 64, table)
    with pytest.raises(TypeError):
        plan.apply(x.bfloat16())
    with pytest.raises(ValueError):
        plan.apply(x[:, :64])
    with pytest.raises(ValueError):
        plan.apply(x.t().contiguous().t())
    with pytest.raises(ValueError):
        plan.apply(x, positions=torch.zeros(8, dtype=torch.int64, device="cuda"))
    with pytest.raises(L.DynConvError) as e:
        plan.apply(x, positions=torch.zeros(8, dtype=torch.int32, device="cuda"),
                   cu_seqlens=torch.tensor([0, 8], dtype=torch.int32, device="cuda"))
    assert e.value.status == 1
    with pytest.raises(L.DynConvError) as e:
        ops.RopePlan(torch.float32, 1, 65, 1, 64, table).apply(torch.randn((65, 64), device="cuda"))
    assert e.value.status == 1 and "max_pos" in str(e.value)
    with pytest.raises(L.DynConvError):                       # a rotated part larger than the head
        ops.RopePlan(torch.float32, 1, 8, 4, 32, table).apply(x)
    empty = ops.RopePlan(torch.float32, 0, 8, 2, 64, table).apply(torch.empty((0, 128), device="cuda"))
    assert empty.shape == (0, 128)
