"""Causal attention (dynconv_attn_fwd / _bwd) against the 64-bit reference, element by element within
bounds that count the kernels' roundings: dense batches and packed documents, grouped heads, both
storage types, both kernel families, lengths around the tile sizes, strided rows, masked places that
hold infinities and NaN, graphs and streams."""
import numpy as np
import pytest

from attn_reference import attention, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = {"bf16": 2.0 ** -7, "f32": 0.0}


def _inputs(N, heads, kv, hd, dtype, seed=0, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda n, s=1.0: (s * torch.randn((N, n * hd), generator=g, device="cuda")).to(DT[dtype])
    return rnd(heads, gain), rnd(kv), rnd(kv), rnd(heads)


def _run(q, k, v, do, batch, seqlen, heads, kv, hd, cu=None, algo=0, scale=0.0):
    from dynamic_short_convolutions_b200 import _lib as L, ops

    plan = ops.AttnPlan(q.dtype, batch, seqlen, heads, kv, hd, scale, algo=algo)
    cu_t = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    nan = lambda n: torch.full((q.shape[0], n * hd), float("nan"), dtype=q.dtype, device="cuda")
    o, lse = plan.forward(q, k, v, cu_t, o=nan(heads), want_lse=True)
    out = plan.backward(do, q, k, v, o, lse, cu_t, out={"dq": nan(heads), "dk": nan(kv), "dv": nan(kv)})
    assert L.dynconv_device_status(plan.ws) == 0, L.dynconv_last_error()
    return dict(o=o, lse=lse, **out)


def _check(got, q, k, v, do, cu, heads, kv, hd, scale=0.0):
    eps = EPS["bf16" if q.dtype == torch.bfloat16 else "f32"]
    ref = attention(q, k, v, cu, heads, kv, hd, do, scale, eps)
    for n in ("o", "lse", "dq", "dk", "dv"):
        check(n, got[n], ref[n])
    if eps == 0.0:
        # The library's fp32 bar, rel-L2 1e-5, plus what scores of size |s| cost beyond it: the score, the
        # row's lse and their difference are each rounded by at most 2^-24 |s|, which the exponential turns
        # into a relative error of a probability of at most 3 * 2^-24 |s|.
        group, w = heads // kv, lambda t: t.double().view(t.shape[0], -1, hd).transpose(0, 1)
        s = (w(q) @ w(k).repeat_interleave(group, 0).transpose(-1, -2)).abs().max() * (scale or hd ** -0.5)
        bar = 1e-5 + 3 * 2.0 ** -24 * float(s)
        for n in ("o", "dq", "dk", "dv"):
            off = float((got[n].double() - ref[n][0]).norm() / ref[n][0].norm().clamp_min(1e-30))
            assert off <= bar or ref[n][0].abs().max() < 1e-6, f"{n}: rel-L2 {off:.3g}"


DENSE = [  # batch, seqlen, heads, kv_heads, head_dim
    (1, 1, 1, 1, 64),
    (3, 1, 4, 2, 128),
    (2, 2, 2, 1, 8),
    (1, 63, 3, 3, 64),
    (1, 128, 2, 2, 128),
    (2, 129, 4, 1, 64),
    (1, 255, 2, 1, 80),
    (1, 257, 8, 2, 128),
    (3, 200, 5, 5, 96),
    (1, 641, 2, 2, 64),
    (2, 520, 4, 2, 40),
]
ODD = [  # head widths and strides the tensor-core kernels do not take
    (2, 70, 2, 1, 4),
    (1, 65, 3, 1, 100),
    (1, 33, 2, 2, 1),
    (1, 70, 8, 8, 37),
]


@pytest.mark.parametrize("algo", [0, 1], ids=["auto", "simt"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", DENSE + ODD, ids=lambda c: "-".join(map(str, c)))
def test_dense(case, dtype, algo):
    batch, seqlen, heads, kv, hd = case
    q, k, v, do = _inputs(batch * seqlen, heads, kv, hd, dtype)
    got = _run(q, k, v, do, batch, seqlen, heads, kv, hd, algo=algo)
    _check(got, q, k, v, do, np.arange(0, batch * seqlen + 1, seqlen), heads, kv, hd)


PACKED = [
    [1] * 40,
    [1, 127, 1, 128, 0, 129, 3],
    [700],
    [64, 64, 64, 64, 64],
    [0, 0, 5, 0],
    [300, 1, 2, 510, 37],
    [383, 2, 385],
]


@pytest.mark.parametrize("shape", [(4, 2, 128), (3, 3, 64), (2, 1, 37)], ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", PACKED, ids=lambda x: "docs%d-%d" % (len(x), sum(x)))
def test_packed(lens, dtype, shape):
    heads, kv, hd = shape
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v, do = _inputs(int(cu[-1]), heads, kv, hd, dtype, seed=2)
    got = _run(q, k, v, do, 1, int(cu[-1]), heads, kv, hd, cu=cu)
    _check(got, q, k, v, do, cu, heads, kv, hd)


@pytest.mark.parametrize("heads,kv", [(8, 1), (5, 1), (6, 2), (12, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_groups(dtype, heads, kv):
    """Group sizes that are and are not powers of two: the sums of dk and dv over the heads of a group."""
    lens = [1, 200, 77, 150]
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v, do = _inputs(428, heads, kv, 64, dtype, seed=11)
    _check(_run(q, k, v, do, 1, 428, heads, kv, 64, cu=cu), q, k, v, do, cu, heads, kv, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_documents(dtype):
    """Enough key tiles to fill the GPU without sharing out a group's heads."""
    lens = [61 + 37 * i % 90 for i in range(180)]
    cu = np.concatenate([[0], np.cumsum(lens)])
    N, heads, kv = int(cu[-1]), 8, 4
    q, k, v, do = _inputs(N, heads, kv, 64, dtype, seed=12)
    _check(_run(q, k, v, do, 1, N, heads, kv, 64, cu=cu), q, k, v, do, cu, heads, kv, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores_and_a_given_scale(dtype):
    """Rows that one key dominates, scores up to some hundreds: the running maximum moves a lot."""
    q, k, v, do = _inputs(400, 2, 1, 64, dtype, seed=3, gain=6.0)
    k[-100:] *= 3
    got = _run(q, k, v, do, 1, 400, 2, 1, 64, scale=0.5)
    _check(got, q, k, v, do, [0, 400], 2, 1, 64, scale=0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_scores(dtype):
    q, k, v, do = _inputs(300, 2, 2, 64, dtype, seed=4)
    q.zero_()
    got = _run(q, k, v, do, 1, 300, 2, 2, 64)
    _check(got, q, k, v, do, [0, 300], 2, 2, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_places_may_hold_anything(dtype):
    """NaN and infinities in a later token of a document, and in a whole other document, reach no row
    that does not see them: those rows' o, and the clean documents' gradients, stay within their bounds."""
    heads, kv, hd = 4, 2, 64
    lens = [150, 90, 200]
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v, do = _inputs(int(cu[-1]), heads, kv, hd, dtype, seed=5)
    clean = [t.clone() for t in (q, k, v, do)]
    for t, x in ((k, float("nan")), (v, float("inf")), (q, float("-inf")), (do, float("nan"))):
        t[170:240] = x                                       # most of the second document
    got = _run(q, k, v, do, 1, int(cu[-1]), heads, kv, hd, cu=cu)
    eps = EPS[dtype]
    ref = attention(*clean[:3], cu, heads, kv, hd, clean[3], eps=eps)
    keep = torch.cat([torch.arange(0, 170), torch.arange(240, 440)]).cuda()
    check("o", got["o"][keep], [t[keep] for t in ref["o"]])
    keep = torch.cat([torch.arange(0, 150), torch.arange(240, 440)]).cuda()
    for n in ("dq", "dk", "dv"):
        check(n, got[n][keep], [t[keep] for t in ref[n]])
    q, k, v, do = (t.clone() for t in clean)                  # one token of the third document, v alone
    v[300, 5] = float("nan")
    got = _run(q, k, v, do, 1, int(cu[-1]), heads, kv, hd, cu=cu)
    keep = torch.arange(0, 300).cuda()
    check("o", got["o"][keep], [t[keep] for t in ref["o"]])
    assert torch.isnan(got["o"][300:, 5]).all() and torch.isnan(got["o"][300:, hd + 5]).all()
    assert torch.isfinite(got["o"][:, 6]).all()


def test_lowest_values():
    """Keys and queries of the type's lowest value: equal (infinite) logits do not poison other documents."""
    low = torch.finfo(torch.bfloat16).min
    q, k, v, do = _inputs(200, 1, 1, 64, "bf16", seed=6)
    ref = attention(q, k, v, [0, 130, 200], 1, 1, 64, do, eps=EPS["bf16"])
    k[130:] = low
    got = _run(q, k, v, do, 1, 200, 1, 1, 64, cu=[0, 130, 200])
    for n in ("o", "dq", "dk", "dv"):
        check(n, got[n][:130], [t[:130] for t in ref[n]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_fused_buffer_slices_and_gradient_slices(dtype):
    """q, k, v as column slices of one buffer, gradients written into one buffer of padded rows:
    bitwise what dense tensors give, the columns behind them left as they were."""
    from dynamic_short_convolutions_b200 import ops

    N, heads, kv, hd = 190, 4, 2, 64
    wq, wk = heads * hd, kv * hd
    q, k, v, do = _inputs(N, heads, kv, hd, dtype, seed=7)
    want = _run(q, k, v, do, 2, 95, heads, kv, hd)
    C = wq + 2 * wk + 16
    buf = torch.cat((q, k, v, torch.randn((N, 16), device="cuda").to(q.dtype)), 1).contiguous()
    d = torch.full((N, C), 7.0, dtype=q.dtype, device="cuda")
    plan = ops.AttnPlan(q.dtype, 2, 95, heads, kv, hd, 0.0, C, C, C, C, C, C)
    qs, ks, vs = buf[:, :wq], buf[:, wq:wq + wk], buf[:, wq + wk:wq + 2 * wk]
    o, lse = plan.forward(qs, ks, vs, want_lse=True)
    plan.backward(do, qs, ks, vs, o, lse, out={"dq": d[:, :wq], "dk": d[:, wq:wq + wk], "dv": d[:, wq + wk:wq + 2 * wk]})
    assert torch.equal(o, want["o"]) and torch.equal(lse, want["lse"])
    assert torch.equal(d[:, :wq], want["dq"]) and torch.equal(d[:, wq:wq + wk], want["dk"])
    assert torch.equal(d[:, wq + wk:wq + 2 * wk], want["dv"]) and (d[:, wq + 2 * wk:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_bitwise_and_on_another_stream(dtype):
    q, k, v, do = _inputs(700, 4, 2, 128, dtype, seed=8)
    a = _run(q, k, v, do, 1, 700, 4, 2, 128, cu=[0, 333, 700])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = _run(q, k, v, do, 1, 700, 4, 2, 128, cu=[0, 333, 700])
    side.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_into_a_graph(dtype):
    from dynamic_short_convolutions_b200 import ops

    N, heads, kv, hd = 260, 2, 1, 64
    q, k, v, do = _inputs(N, heads, kv, hd, dtype, seed=9)
    cu = torch.tensor([0, 100, 260], dtype=torch.int32, device="cuda")
    plan = ops.AttnPlan(q.dtype, 1, N, heads, kv, hd)
    plan.forward(q, k, v, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = plan.forward(q, k, v, cu, want_lse=True)
        grads = plan.backward(do, q, k, v, o, lse, cu)
    fresh = _inputs(N, heads, kv, hd, dtype, seed=10)
    for t, x in zip((q, k, v, do), fresh):
        t.copy_(x)
    cu.copy_(torch.tensor([0, 37, 260], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    want = _run(*fresh, 1, N, heads, kv, hd, cu=[0, 37, 260])
    assert torch.equal(o, want["o"])
    for n in ("dq", "dk", "dv"):
        assert torch.equal(grads[n], want[n]), n


def test_bad_cu_seqlens_raise_the_device_check():
    from dynamic_short_convolutions_b200 import _lib as L, ops

    q, k, v, do = _inputs(300, 2, 1, 64, "bf16")
    for bad in ([0, 200], [1, 300], [0, 250, 100, 300], [0, -5, 300], [0, 2 ** 31 - 1, 300]):
        for algo in (0, 1):
            plan = ops.AttnPlan(torch.bfloat16, 1, 300, 2, 1, 64, algo=algo)
            cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
            o, lse = plan.forward(q, k, v, cu, want_lse=True)
            assert L.dynconv_device_status(plan.ws) == 5 and "cu_seqlens" in L.dynconv_last_error()
            plan.backward(do, q, k, v, o, lse, cu)
            assert L.dynconv_device_status(plan.ws) == 5


def test_refusals_with_tensors():
    from dynamic_short_convolutions_b200 import _lib as L, ops

    q, k, v, do = _inputs(10, 2, 1, 64, "bf16")
    plan = ops.AttnPlan(torch.bfloat16, 1, 10, 2, 1, 64)
    with pytest.raises(TypeError):
        plan.forward(q.float(), k, v)
    with pytest.raises(ValueError):
        plan.forward(q, q, v)
    with pytest.raises(ValueError):
        plan.forward(q[:9], k, v)
    with pytest.raises(ValueError):
        plan.forward(q, k, v, cu_seqlens=torch.tensor([0, 10], device="cuda"))       # int64
    wide = torch.zeros((10, 136), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        plan.forward(wide[:, :128], k, v)                                            # another stride
    strided = ops.AttnPlan(torch.bfloat16, 1, 10, 2, 1, 64, q_row_stride=136)
    with pytest.raises(L.DynConvError) as e:
        strided.forward(wide[:, 4:132], k, v)                                        # misaligned base
    assert e.value.status == 1 and "aligned" in str(e.value)
    with pytest.raises(L.DynConvError) as e:
        L.dynconv_attn_fwd(plan.desc, None, q.cpu(), k, v, torch.empty_like(q), None, plan.ws)
    assert e.value.status == 1 and "device pointer" in str(e.value)
    with pytest.raises(L.DynConvError) as e:
        L.dynconv_attn_fwd(plan.desc, None, q, k, v, torch.empty_like(q), None, plan.ws[:16])
    assert e.value.status == 3
    dense = ops.AttnPlan(torch.bfloat16, 2, 5, 2, 1, 64)
    with pytest.raises(L.DynConvError) as e:
        dense.forward(q, k, v, cu_seqlens=torch.tensor([0, 10], dtype=torch.int32, device="cuda"))
    assert e.value.status == 1
    none = ops.AttnPlan(torch.bfloat16, 0, 5, 2, 1, 64)
    assert none.forward(q[:0], k[:0], v[:0]).shape == (0, 128)
