"""Rows all of whose visible scores are minus infinity: their softmax has no value (0 / 0), and NaN is what they get,
in every kernel; rows that see a finite score too, rows that see nothing and idle slots keep theirs."""
import pytest

from attn_reference import attention, check, decode

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = {"bf16": 2.0 ** -7, "f32": 0.0}


@pytest.mark.parametrize("hd,algo", [(64, 0), (128, 0), (40, 0), (128, 1), (64, 1), (37, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_causal_rows(dtype, hd, algo):
    """A document that begins with `lost` keys of score minus infinity, between two others."""
    from dynamic_short_convolutions_b200 import _lib as L, ops

    heads, kv, cu, lost = 4, 2, [0, 70, 400, 431], 150
    N = cu[-1]
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda n: torch.randn((N, n * hd), generator=g, device="cuda").to(DT[dtype])
    q, k, v = rnd(heads), rnd(kv), rnd(kv)
    q.view(N, heads, hd)[:, :, 0].abs_().add_(0.5)
    clean = k.clone()
    k.view(N, kv, hd)[cu[1]:cu[1] + lost, :, 0] = -float("inf")
    plan = ops.AttnPlan(DT[dtype], 1, N, heads, kv, hd, algo=algo)
    o, lse = plan.forward(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), want_lse=True)
    assert L.dynconv_device_status(plan.ws) == 0
    gone = slice(cu[1], cu[1] + lost)
    assert torch.isnan(o[gone]).all() and (lse[:, gone] == -float("inf")).all()
    # the rest: the document from its first finite key on, which is all that has weight there
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[gone] = False
    short = [0, 70, 400 - lost, 431 - lost]
    ref = attention(q[keep], clean[keep], v[keep], short, heads, kv, hd, None, 0.0, EPS[dtype])
    check("o", o[keep], ref["o"])
    check("lse", lse[:, keep], ref["lse"])


@pytest.mark.parametrize("hd,algo", [(64, 0), (128, 0), (128, 1), (37, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_other_documents(dtype, hd, algo):
    """Tiles that hold the end of a document of such rows and the beginning of another: the other's gradients."""
    from dynamic_short_convolutions_b200 import _lib as L, ops

    heads, kv, cu = 4, 2, [0, 70, 300, 431]
    N = cu[-1]
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda n: torch.randn((N, n * hd), generator=g, device="cuda").to(DT[dtype])
    q, k, v, do = rnd(heads), rnd(kv), rnd(kv), rnd(heads)
    q.view(N, heads, hd)[:, :, 0].abs_().add_(0.5)
    ref = attention(q, k, v, cu, heads, kv, hd, do, 0.0, EPS[dtype])
    k.view(N, kv, hd)[cu[1]:cu[2], :, 0] = -float("inf")
    plan = ops.AttnPlan(DT[dtype], 1, N, heads, kv, hd, algo=algo)
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, lse = plan.forward(q, k, v, cu_t, want_lse=True)
    d = plan.backward(do, q, k, v, o, lse, cu_t)
    assert L.dynconv_device_status(plan.ws) == 0
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[cu[1]:cu[2]] = False
    for name, t in dict(o=o, **d).items():
        check(name, t[keep], [x[keep] for x in ref[name]])
    assert torch.isnan(o[~keep]).all()


# lens of the sequences: all cached scores lost, half of them, none cached, idle; tokens, heads, kv_heads
STEPS = [(1, 4, 2), (2, 8, 2), (4, 8, 2), (7, 8, 2), (24, 8, 2)]


@pytest.mark.parametrize("hd", [64, 128, 24])
@pytest.mark.parametrize("tokens,heads,kv", STEPS)
@pytest.mark.parametrize("long", [False, True], ids=["one-run", "runs"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps(dtype, long, tokens, heads, kv, hd):
    from dynamic_short_convolutions_b200 import _lib as L, ops

    lens, max_len = ([1800, 1800, 0, -1], 2000) if long else ([40, 40, 0, -1], 100)
    b, n = len(lens), lens[0]
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])
    q, k, v = rnd(b * tokens, heads * hd), rnd(b * tokens, kv * hd), rnd(b * tokens, kv * hd)
    q.view(-1, heads, hd)[:, :, 0].abs_().add_(0.5)
    caches = [rnd(b, kv, max_len, hd) for _ in range(2)]
    caches[0][0, :, :, 0] = -float("inf")
    caches[0][1, :, :n // 2, 0] = -float("inf")
    rows = k.view(b, tokens, kv, hd)
    rows[0, :, :, 0] = -float("inf")
    # sequence 2: its first token sees nothing, the others (if any) themselves
    trees = [[1 << m for m in range(tokens)] for _ in lens]
    trees[2][0] = 0
    signed = [[x - (1 << 64) if x >> 63 else x for x in t] for t in trees]
    dec = ops.AttnDecoder(DT[dtype], b, heads, kv, hd, max_len, tokens, k_cache=caches[0], v_cache=caches[1],
                          lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    o = dec.step(q, k, v, torch.tensor(signed, dtype=torch.int64, device="cuda")).view(b, tokens, -1)
    assert L.dynconv_device_status(dec.ws) == 0
    assert torch.isnan(o[0]).all()
    assert not o[2, 0].any() and not o[3].any()
    # sequence 1 from its first finite row on
    k1, v1 = (t[1:2, :, n // 2:] for t in (dec.k_cache, dec.v_cache))
    ref = decode(q.view(b, tokens, -1)[1:2].reshape(tokens, -1), k1, v1, [n - n // 2], trees[1:2], heads, kv,
                 hd, tokens, eps=EPS[dtype])
    check("o", o[1], ref)
    ref = decode(q.view(b, tokens, -1)[2:3].reshape(tokens, -1), dec.k_cache[2:3], dec.v_cache[2:3], [0], trees[2:3], heads, kv,
                 hd, tokens, eps=EPS[dtype])
    check("o", o[2], ref)
