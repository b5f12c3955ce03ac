"""Attention at the edges of what its callers may ask: several tiles per block, caches and rows whose offsets pass
32 bits, no tokens, heads of odd widths in a fused buffer, two plans at once on two streams, two captured graphs
that share a workspace, a captured backward pass through autograd."""
import math

import pytest

from attn_reference import attention, check
from test_gpu_attention import _check, _run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _qkv(N, heads, kv, hd, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda n: torch.randn((N, n * hd), generator=g, device="cuda").to(DT[dtype])
    return rnd(heads), rnd(kv), rnd(kv), rnd(heads)


@pytest.mark.parametrize("hd", [128, 72, 64])
@pytest.mark.parametrize("lens", [[700] * 3, [1, 900, 0, 130, 127, 129, 400, 128, 256]], ids=["dense", "packed"])
def test_many_tiles(lens, hd):
    """More (head, tile) pairs than the GPU has multiprocessors."""
    heads, kv, N = 24, 4, sum(lens)
    q, k, v, do = _qkv(N, heads, kv, hd, "bf16", 1)
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    dense = len(set(lens)) == 1
    got = _run(q, k, v, do, len(lens) if dense else 1, lens[0] if dense else N, heads, kv, hd, None if dense else cu)
    _check(got, q, k, v, do, cu, heads, kv, hd)


@pytest.mark.parametrize("hd", [128, 64])
def test_many_tiles_some_with_infinities(hd):
    """Documents whose neighbours hold infinities and NaN: their tiles, and only theirs, take the slow way."""
    heads, kv, lens = 16, 2, [300, 200, 700, 500, 900]
    N, bad = sum(lens), [1, 3]
    q, k, v, do = _qkv(N, heads, kv, hd, "bf16", 2)
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    clean = _run(q, k, v, do, 1, N, heads, kv, hd, cu)
    for d, x in zip(bad, (float("inf"), float("nan"))):
        for t in (q, k, v, do):
            t[cu[d]:cu[d + 1]] = x
    got = _run(q, k, v, do, 1, N, heads, kv, hd, cu)
    ok = torch.ones(N, dtype=torch.bool, device="cuda")
    for d in bad:
        ok[cu[d]:cu[d + 1]] = False
    pick = lambda r: {n: (t[:, ok] if n == "lse" else t[ok]) for n, t in r.items()}
    rows = [t[ok] for t in (q, k, v, do)]
    cu_ok = [0, 300, 1000, 1900]
    _check(pick(got), *rows, cu_ok, heads, kv, hd)
    _check(pick(clean), *rows, cu_ok, heads, kv, hd)


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_rows_beyond_32_bits(dtype, hd):
    N, heads, kv, row = 4200, 2, 1, 1 << 20
    from dynamic_short_convolutions_b200 import _lib as L, ops

    q, k, v, do = _qkv(N, heads, kv, hd, dtype, 3)
    x = torch.empty((N, row), dtype=DT[dtype], device="cuda")
    d = torch.empty((N, row), dtype=DT[dtype], device="cuda")
    wq, wk = heads * hd, kv * hd
    cols = lambda t: (t[:, :wq], t[:, wq:wq + wk], t[:, row - wk:])
    for to, t in zip(cols(x), (q, k, v)):
        to.copy_(t)
    plan = ops.AttnPlan(DT[dtype], 1, N, heads, kv, hd, 0.0, *[row] * 6)
    o, lse = plan.forward(*cols(x), want_lse=True)
    plan.backward(do, *cols(x), o, lse, out=dict(zip(("dq", "dk", "dv"), cols(d))))
    assert L.dynconv_device_status(plan.ws) == 0
    _check(dict(o=o, lse=lse, **{n: t.contiguous() for n, t in zip(("dq", "dk", "dv"), cols(d))}), q, k, v, do, [0, N],
           heads, kv, hd)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,heads", [(1, 2), (12, 4), (40, 2)])
def test_cache_beyond_32_bits(tokens, heads, dtype):
    """All rows zero but the last `special` cached ones, each four times a query of the step, which it draws to itself.

    A zero row adds 1 to a row's sum and nothing to its output.  The bound: rounding of P, and of o (half steps);
    a dot product, the sum of the special rows and an exponential in fp32, as in the reference; and the sum of the
    n0 zero rows, at most n0 2^-24 of it, times its share of the whole."""
    from dynamic_short_convolutions_b200 import _lib as L, ops

    batch, kv, hd, max_len = 3, 2, 128, 3 << 21
    group, lens = heads // kv, [200, max_len - tokens - 5, 700]
    special = tokens * group
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])
    q, k, v = rnd(batch * tokens, heads * hd), rnd(batch * tokens, kv * hd), rnd(batch * tokens, kv * hd)
    caches = [torch.zeros((batch, kv, max_len, hd), dtype=DT[dtype], device="cuda") for _ in range(2)]
    assert caches[0].numel() > 1 << 32
    qg = q.view(batch, tokens, kv, group, hd).permute(0, 2, 1, 3, 4).reshape(batch, kv, special, hd)
    vs = rnd(batch, kv, special, hd)
    for b, n in enumerate(lens):
        caches[0][b, :, n - special:n] = 4 * qg[b]
        caches[1][b, :, n - special:n] = vs[b]
    dec = ops.AttnDecoder(DT[dtype], batch, heads, kv, hd, max_len, tokens, k_cache=caches[0], v_cache=caches[1],
                          lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    o = dec.step(q, k, v)
    assert L.dynconv_device_status(dec.ws) == 0, L.dynconv_last_error()
    h = 2.0 ** -8 if dtype == "bf16" else 0.0
    new = lambda t: t.view(batch, tokens, kv, hd).transpose(1, 2).double()
    keys = torch.cat((4 * qg.double(), new(k)), 2)
    vals = torch.cat((vs.double(), new(v)), 2)
    n0 = torch.tensor([n - special for n in lens], dtype=torch.float64, device="cuda").view(-1, 1, 1, 1)
    s = qg.double() @ keys.transpose(-1, -2) / math.sqrt(hd)
    m = torch.arange(special, device="cuda").view(-1, 1) // group                    # a row's token
    late = torch.arange(tokens, device="cuda") > m
    s = torch.cat((s[..., :special], s[..., special:].masked_fill(late, -math.inf)), -1)
    e = s.exp()
    total = e.sum(-1, keepdim=True) + n0
    p = e / total
    want, size = p @ vals, p @ vals.abs()
    big = float((qg.double().abs() @ keys.abs().transpose(-1, -2)).max()) / math.sqrt(hd)
    r = (hd + special + tokens + 32) * 2.0 ** -24 * (2 + big) + n0 / total * n0 * 2.0 ** -24
    back = lambda t: t.view(batch, kv, tokens, group, hd).permute(0, 2, 1, 3, 4).reshape(batch * tokens, heads * hd)
    check("o", o, (back(want), back(h * (want.abs() + size) + r * size)))
    for b, n in enumerate(lens):
        assert torch.equal(caches[0][b, :, n:n + tokens].double(), new(k)[b])
        assert torch.equal(caches[1][b, :, n:n + tokens].double(), new(v)[b])
        assert not caches[0][b, :, n + tokens:].any() and not caches[0][b, :, :n - special].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens(dtype):
    from dynamic_short_convolutions_b200 import ops

    qkv = torch.zeros((0, 512), dtype=DT[dtype], device="cuda", requires_grad=True)
    table = ops.rope_table(16, 64)
    o = ops.qkv_attention(qkv, 4, 2, 64, table)
    d, = torch.autograd.grad(o, qkv, torch.zeros_like(o))
    assert o.shape == (0, 256) and d.shape == qkv.shape


@pytest.mark.parametrize("packed", [False, True], ids=["dense", "packed"])
@pytest.mark.parametrize("heads,kv,hd", [(2, 1, 37), (3, 1, 5), (3, 3, 20), (1, 1, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_fused_rows_of_odd_heads(dtype, heads, kv, hd, packed):
    from dynamic_short_convolutions_b200 import ops

    lens = [50, 1, 69] if packed else [60, 60]
    N, cu = 120, [sum(lens[:i]) for i in range(len(lens) + 1)]
    q, k, v, do = _qkv(N, heads, kv, hd, dtype, 5)
    qkv = torch.cat((q, k, v), 1).requires_grad_()
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda") if packed else None
    o = ops.qkv_attention(qkv, heads, kv, hd, batch=1 if packed else 2, cu_seqlens=cu_t)
    d, = torch.autograd.grad(o, qkv, do)
    wq, wk = heads * hd, kv * hd
    eps = 2.0 ** -7 if dtype == "bf16" else 0.0
    ref = attention(q, k, v, cu, heads, kv, hd, do, 0.0, eps)
    for name, t in (("o", o), ("dq", d[:, :wq]), ("dk", d[:, wq:wq + wk]), ("dv", d[:, wq + wk:])):
        check(name, t.detach(), ref[name])
    with torch.no_grad():
        assert torch.equal(o, ops.qkv_attention(qkv, heads, kv, hd, batch=1 if packed else 2, cu_seqlens=cu_t))
    o = ops.qkv_attention(qkv, heads, kv, hd, batch=1 if packed else 2, cu_seqlens=cu_t)
    d, = torch.autograd.grad(o, qkv, do, create_graph=True)
    with pytest.raises(RuntimeError):                          # no second derivatives
        torch.autograd.grad(d.sum(), qkv)


def test_two_plans_at_once():
    from dynamic_short_convolutions_b200 import ops

    heads, kv, hd, N = 8, 2, 128, 2048
    sets = [_qkv(N, heads, kv, hd, "bf16", s) for s in (6, 7)]
    plans = [ops.AttnPlan(torch.bfloat16, 1, N, heads, kv, hd) for _ in sets]
    run = lambda p, t: (lambda f: [*f, *p.backward(t[3], *t[:3], *f).values()])(p.forward(*t[:3], want_lse=True))
    want = [run(p, t) for p, t in zip(plans, sets)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(plans[i], sets[i]))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, r))


def test_graphs_that_share_a_workspace():
    """A plan's forward and backward, and a decoder's steps, captured apart and replayed in turn."""
    from dynamic_short_convolutions_b200 import ops

    heads, kv, hd, N = 4, 2, 64, 600
    q, k, v, do = _qkv(N, heads, kv, hd, "bf16", 8)
    cu = torch.tensor([0, 100, 350, 600], dtype=torch.int32, device="cuda")
    plan = ops.AttnPlan(torch.bfloat16, 1, N, heads, kv, hd)
    dec = ops.AttnDecoder(torch.bfloat16, 2, heads, kv, hd, 700, 3)
    dec.k_cache.normal_()
    dec.v_cache.normal_()
    dec.lens.fill_(650)
    rows = [t[:6].contiguous() for t in (q, k, v)]
    o, lse = plan.forward(q, k, v, cu, want_lse=True)
    want = [o, *plan.backward(do, q, k, v, o, lse, cu).values(), dec.step(*rows)]
    want = [t.clone() for t in want]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for call in (lambda: [plan.forward(q, k, v, cu)], lambda: list(plan.backward(do, q, k, v, o, lse, cu).values()),
                 lambda: [dec.step(*rows)], lambda: [dec.step(*rows)]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for _ in range(3):
        for t in sum(outs, []):
            t.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want + want[-1:], sum(outs, [])):
            assert torch.equal(a, b)


def test_captured_training_step():
    """Forward and backward of a leaf through autograd, captured; no eager graph of the leaf is alive."""
    from dynamic_short_convolutions_b200 import ops

    heads, kv, hd, N = 4, 2, 64, 384
    q, k, v, do = _qkv(N, heads, kv, hd, "bf16", 9)
    leaf = torch.cat((q, k, v), 1).requires_grad_()
    cu = torch.tensor([0, 100, 384], dtype=torch.int32, device="cuda")
    table = ops.rope_table(N, hd)

    def step():
        o = ops.qkv_attention(leaf, heads, kv, hd, table, cu_seqlens=cu)
        return o.detach(), torch.autograd.grad(o, leaf, do)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(2):
        for t in got:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
