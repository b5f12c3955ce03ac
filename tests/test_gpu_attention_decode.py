"""Attention of new or drafted tokens over a cache (dynconv_attn_decode) against the 64-bit reference:
single tokens, chains and trees, caches from empty to full, grouped heads, both storage types, rotations,
idle slots, masked and stale rows that hold NaN, graphs; and the prompt's attention continued token by token."""
import random

import pytest

from attn_reference import attention, check, decode, rope

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = {"bf16": 2.0 ** -7, "f32": 0.0}
# rotated q is held in bf16 as a value and a remainder: two roundings, 2^-8 x 2^-8 in all
Q_ERR = {"bf16": 2.0 ** -16, "f32": 0.0}


def _trees(batch, tokens, seed):
    r = random.Random(seed)
    out = []
    for _ in range(batch):
        masks = []
        for m in range(tokens):
            parent = r.randint(-1, m - 1)
            masks.append((masks[parent] if parent >= 0 else 0) | (1 << m))
        out.append(masks)
    return out


def _signed(x):
    return x - (1 << 64) if x >> 63 else x


def _tensor(trees):
    return torch.tensor([[_signed(x) for x in row] for row in trees], dtype=torch.int64, device="cuda")


def _setup(dtype, lens, tokens, heads, kv, hd, max_len, rot=0, half=False, seed=0, gain=1.0):
    from dynamic_short_convolutions_b200 import _lib as L, ops

    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])
    b = len(lens)
    q, k, v = gain * rnd(b * tokens, heads * hd), rnd(b * tokens, kv * hd), rnd(b * tokens, kv * hd)
    table = ops.rope_table(max_len + 3, rot, device="cuda") if rot else None
    dec = ops.AttnDecoder(DT[dtype], b, heads, kv, hd, max_len, tokens, rope_table=table,
                          rope_layout=L.ROPE_HALF if half else L.ROPE_INTERLEAVED, k_cache=rnd(b, kv, max_len, hd),
                          v_cache=rnd(b, kv, max_len, hd), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    return dec, q, k, v, table


def _step_and_check(dtype, dec, q, k, v, table, lens, trees, heads, kv, hd, half, ancestors=True):
    from dynamic_short_convolutions_b200 import _lib as L

    tokens, eps = dec.tokens, EPS[dtype]
    before = dec.k_cache.clone(), dec.v_cache.clone()
    o = torch.full_like(q, float("nan"))
    dec.step(q, k, v, _tensor(trees) if ancestors else None, o=o)
    assert L.dynconv_device_status(dec.ws) == 0, L.dynconv_last_error()
    pos = torch.tensor([max(n, 0) + bin(t & ~(1 << m)).count("1") for n, row in zip(lens, trees)
                        for m, t in enumerate(row)], device="cuda")
    qr = rope(q, table, pos, heads, hd, half)[0] if table is not None else q.double()
    kr = rope(k, table, pos, kv, hd, half, eps=eps) if table is not None else (k.double(), torch.zeros_like(k).double())
    for b, n in enumerate(lens):
        rows = slice(b * tokens, (b + 1) * tokens)
        if n < 0:
            assert torch.equal(dec.k_cache[b], before[0][b]) and torch.equal(dec.v_cache[b], before[1][b])
            assert (o[rows] == 0).all()
            continue
        new = lambda t: t[rows].reshape(tokens, kv, hd).transpose(0, 1)
        check("k_cache", dec.k_cache[b, :, n:n + tokens], [new(t) for t in kr])
        assert torch.equal(dec.v_cache[b, :, n:n + tokens], new(v))
        for now, old in ((dec.k_cache, before[0]), (dec.v_cache, before[1])):
            assert torch.equal(now[b, :, :n], old[b, :, :n]) and torch.equal(now[b, :, n + tokens:], old[b, :, n + tokens:])
    check("o", o, decode(qr, dec.k_cache, dec.v_cache, lens, trees, heads, kv, hd, tokens, eps=eps, q_err=Q_ERR[dtype]))
    return o


CASES = [  # lens, tokens, heads, kv_heads, head_dim, max_len, rotated
    ([0], 1, 1, 1, 64, 1, 0),
    ([5], 1, 12, 12, 64, 2048, 64),
    ([63, 64, 65, 0, 1], 1, 8, 2, 128, 200, 128),
    ([199, 127, 128, 129], 1, 16, 4, 128, 200, 64),
    ([1000, 3, 517], 1, 4, 4, 80, 1500, 40),
    ([40, 0, 197], 3, 8, 2, 64, 200, 64),
    ([100, 64, 0, 333], 24, 16, 4, 128, 400, 128),
    ([500, 10], 64, 8, 1, 64, 600, 64),
    ([31, 32, 33], 17, 3, 3, 96, 64, 6),
    ([2000, 1999], 5, 5, 1, 128, 2048, 128),
    ([700], 33, 2, 2, 8, 800, 0),
    ([128, 256, 255, 129, 0], 12, 16, 4, 64, 300, 32),
    ([3000, 2049], 60, 16, 2, 128, 3100, 128),
    ([1500, 1499, 1281] * 13, 9, 16, 4, 64, 1600, 64),          # a run of many tiles, then the drafted one
]


@pytest.mark.parametrize("half", [False, True], ids=["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%d-m%d-h%d-%d-d%d-l%d-r%d" % (len(c[0]), *c[1:]))
def test_trees(case, dtype, half):
    lens, tokens, heads, kv, hd, max_len, rot = case
    dec, q, k, v, table = _setup(dtype, lens, tokens, heads, kv, hd, max_len, rot, half, seed=1)
    _step_and_check(dtype, dec, q, k, v, table, lens, _trees(len(lens), tokens, 3), heads, kv, hd, half)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 4, 64])
def test_a_chain_is_the_default(tokens, dtype):
    lens = [70, 0, 129]
    chain = [[(2 << m) - 1 for m in range(tokens)]] * 3
    dec, q, k, v, table = _setup(dtype, lens, tokens, 4, 2, 64, 256, 64, seed=2)
    a = _step_and_check(dtype, dec, q, k, v, table, lens, chain, 4, 2, 64, False, ancestors=False)
    b = _step_and_check(dtype, dec, q, k, v, table, lens, chain, 4, 2, 64, False)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_idle_slots_and_rows_that_see_nothing(dtype):
    lens = [-1, 10, -5, 0]
    trees = [[1, 2], [0, 3], [1, 3], [0, 2]]                     # token 0 sees no drafted token
    dec, q, k, v, table = _setup(dtype, lens, 2, 4, 2, 64, 64, 32, seed=3)
    o = _step_and_check(dtype, dec, q, k, v, table, lens, trees, 4, 2, 64, False)
    assert (o[6] == 0).all()                                     # no cached row either


@pytest.mark.parametrize("heads", [2, 8, 16])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_stale_and_masked_rows_may_hold_anything(dtype, heads):
    lens, tokens, kv, hd = [100, 7], 8, 2, 128
    trees = [[1 << m for m in range(8)], [1, 3, 7, 9, 16, 48, 64, 193]]
    dec, q, k, v, table = _setup(dtype, lens, tokens, heads, kv, hd, 300, 128, True, seed=4)
    for b, n in enumerate(lens):
        dec.k_cache[b, :, n:] = float("nan")
        dec.v_cache[b, :, n:] = float("inf")
    a = dec.step(q, k, v, _tensor(trees))
    k[3] = float("nan")                                          # one drafted token of the first sequence
    v[3, 1::2] = float("nan")
    v[3, ::2] = float("inf")
    b = dec.step(q, k, v, _tensor(trees))
    keep = [i for i in range(16) if i != 3]
    pos = torch.tensor([n + bin(t & ~(1 << m)).count("1") for n, row in zip(lens, trees) for m, t in enumerate(row)],
                       device="cuda")
    clean_k, clean_v = dec.k_cache.clone(), dec.v_cache.clone()
    clean_k[0, :, 103], clean_v[0, :, 103] = 0, 0
    ref = decode(rope(q, table, pos, heads, hd, True)[0], clean_k, clean_v, lens, trees, heads, kv, hd, tokens,
                 eps=EPS[dtype], q_err=Q_ERR[dtype])
    for o in (a, b):
        check("o", o[keep], [t[keep] for t in ref])
    assert not torch.isfinite(b[3]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_continue_a_prompt(dtype):
    """Token by token over the cache gives what causal attention gives over the whole prompt."""
    from dynamic_short_convolutions_b200 import ops

    n, heads, kv, hd = 70, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda w: torch.randn((2 * n, w * hd), generator=g, device="cuda").to(DT[dtype])
    q, k, v = rnd(heads), rnd(kv), rnd(kv)
    table = ops.rope_table(n, hd, device="cuda")
    dec = ops.AttnDecoder(DT[dtype], 2, heads, kv, hd, n, rope_table=table)
    got = torch.empty_like(q)
    for t in range(n):
        rows = torch.tensor([t, n + t], device="cuda")
        got[rows] = dec.step(q[rows], k[rows], v[rows])
        dec.advance()
    pos = torch.arange(2 * n, device="cuda") % n
    cached = lambda c: c.transpose(1, 2).reshape(2 * n, kv * hd)
    check("k_cache", cached(dec.k_cache), rope(k, table, pos, kv, hd, False, eps=EPS[dtype]))
    check("o", got, attention(rope(q, table, pos, heads, hd, False)[0], cached(dec.k_cache), cached(dec.v_cache),
                              [0, n, 2 * n], heads, kv, hd, eps=EPS[dtype], q_err=Q_ERR[dtype])["o"])
    assert dec.lens.tolist() == [n, n]
    dec.reset()
    assert dec.lens.tolist() == [0, 0]


def test_repeats_bitwise_streams_and_a_graph():
    lens = [1500, 3, 900]
    dec, q, k, v, table = _setup("bf16", lens, 2, 16, 4, 128, 2000, 128, seed=6)
    a = dec.step(q, k, v)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = dec.step(q, k, v)
    side.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = dec.step(q, k, v)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, c)
    dec.lens.copy_(torch.tensor([7, 3, -1], dtype=torch.int32))        # the graph reads lens anew
    graph.replay()
    torch.cuda.synchronize()
    d = dec.step(q, k, v)
    assert torch.equal(c, d) and (c[4:] == 0).all()


def test_overflowing_lengths_and_positions_raise_the_device_check():
    from dynamic_short_convolutions_b200 import _lib as L, ops

    for dtype in ("bf16", "f32"):
        lens = [10, 63, 2 ** 31 - 1, 5]
        dec, q, k, v, _ = _setup(dtype, lens, 2, 4, 2, 64, 64, seed=7)
        before = dec.k_cache.clone()
        o = dec.step(q, k, v)
        assert L.dynconv_device_status(dec.ws) == 5 and "cache" in L.dynconv_last_error()
        assert (o[2:6] == 0).all() and torch.equal(dec.k_cache[1:3], before[1:3])
        check("others", o, decode(q, dec.k_cache, dec.v_cache, [10, -1, -1, 5], [[1, 3]] * 4, 4, 2, 64, 2, eps=EPS[dtype]))
        table = ops.rope_table(20, 64, device="cuda")
        short = ops.AttnDecoder(DT[dtype], 2, 4, 2, 64, 64, 2, rope_table=table,
                                lens=torch.tensor([18, 19], dtype=torch.int32, device="cuda"))
        o = short.step(q[:4], k[:4], v[:4])
        assert L.dynconv_device_status(short.ws) == 5 and "position" in L.dynconv_last_error()
        assert (o[2:] == 0).all() and (o[:2] != 0).any() and (short.k_cache[1] == 0).all()


def test_fused_rows():
    """q, k, v as column slices of one row buffer: bitwise what dense rows give."""
    from dynamic_short_convolutions_b200 import ops

    dec, q, k, v, _ = _setup("bf16", [30, 40], 3, 4, 2, 64, 64, seed=8)
    want = dec.step(q, k, v)
    buf = torch.cat((q, k, v), 1).contiguous()
    C = buf.shape[1]
    two = ops.AttnDecoder(torch.bfloat16, 2, 4, 2, 64, 64, 3, q_row_stride=C, k_row_stride=C, v_row_stride=C,
                          k_cache=dec.k_cache, v_cache=dec.v_cache, lens=dec.lens)
    assert torch.equal(two.step(buf[:, :256], buf[:, 256:384], buf[:, 384:]), want)


def test_refusals():
    from dynamic_short_convolutions_b200 import _lib as L, ops

    dec, q, k, v, _ = _setup("bf16", [3], 1, 4, 2, 64, 64)
    with pytest.raises(TypeError):
        dec.step(q.float(), k, v)
    with pytest.raises(ValueError):
        dec.step(q, q, v)
    with pytest.raises(ValueError):
        dec.step(q, k, v, ancestors=torch.ones((1, 2), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        ops.AttnDecoder(torch.bfloat16, 1, 4, 2, 64, 64, k_cache=dec.k_cache[:, :, :32])
    for kw in (dict(tokens=65), dict(tokens=0), dict(head_dim=60), dict(head_dim=136), dict(max_len=0), dict(heads=3),
               dict(scale=-1.0), dict(q_row_stride=260), dict(tokens=9, max_len=8), dict(batch=-1)):
        full = dict(dict(dtype=torch.bfloat16, batch=1, heads=4, kv_heads=2, head_dim=64, max_len=64), **kw)
        with pytest.raises(L.DynConvError):
            ops.AttnDecoder(**full)
    none = ops.AttnDecoder(torch.bfloat16, 0, 4, 2, 64, 64)
    assert none.step(q[:0], k[:0], v[:0]).shape == (0, 256)
