"""The QKV placement as a layer runs it: dynamic short convolution of the fused QKV rows, rotary positions,
causal attention (ops.dynamic_conv_attention), forward and backward over packed documents and dense batches,
against a 64-bit restatement with autograd; and the same layer served token by token: the decode step of the
convolution, then the attention step over the cache."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _plain(u, h, A, B, K, heads, kv, hd, table, half, cu):
    """64-bit layer on [N, C] rows, written from the formulas."""
    C, wq, wk = u.shape[1], heads * hd, kv * hd
    w = (h @ A @ B).view(-1, C, K) if A is not None else (h @ B).view(len(h), -1, K)
    if A is None:
        w = w.repeat_interleave(C // w.shape[1], 1)
    outs = []
    for a, b in zip(cu[:-1], cu[1:]):
        x, f, n = u[a:b], w[a:b], b - a
        y = x + sum(f[:, :, j] * torch.cat((x.new_zeros(min(j, n), C), x[:max(n - j, 0)])) for j in range(K))
        rot = table.shape[1]
        cos, sin = table[:n, None, 0::2].double(), table[:n, None, 1::2].double()
        z = y[:, :wq + wk].reshape(n, heads + kv, hd)
        p, rest = z[..., :rot], z[..., rot:]
        e, o = (p[..., :rot // 2], p[..., rot // 2:]) if half else (p[..., 0::2], p[..., 1::2])
        r = (e * cos - o * sin, e * sin + o * cos)
        z = torch.cat((torch.cat(r, -1) if half else torch.stack(r, -1).flatten(-2), rest), -1)
        q, k = z[:, :heads].transpose(0, 1), z[:, heads:].transpose(0, 1).repeat_interleave(heads // kv, 0)
        v = y[:, wq + wk:].reshape(n, kv, hd).transpose(0, 1).repeat_interleave(heads // kv, 0)
        s = (q @ k.transpose(-1, -2) / math.sqrt(hd)).masked_fill(
            torch.ones(n, n, dtype=torch.bool, device=u.device).triu(1), -math.inf)
        outs.append((torch.softmax(s, -1) @ v).transpose(0, 1).reshape(n, wq))
    return torch.cat(outs)


def _layer(dtype, N, heads, kv, hd, K, rank, filter_hd, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    C, d = (heads + 2 * kv) * hd, 128
    rnd = lambda *s, std=1.0: (std * torch.randn(s, generator=g, device="cuda")).to(dtype)
    u, h = rnd(N, C), rnd(N, d)
    if rank:
        return u, h, rnd(d, rank, std=d ** -0.5), rnd(rank, C * K, std=rank ** -0.5), rnd(N, heads * hd)
    return u, h, None, rnd(d, C // filter_hd * K, std=d ** -0.5), rnd(N, heads * hd)


@pytest.mark.parametrize("dtype,limit", [(torch.float32, 2e-5), (torch.bfloat16, 2e-2)], ids=["f32", "bf16"])
@pytest.mark.parametrize("half", [False, True], ids=["interleaved", "half"])
@pytest.mark.parametrize("packed", [False, True], ids=["dense", "packed"])
@pytest.mark.parametrize("rank", [16, 0], ids=["lowrank", "headwise"])
def test_layer_and_its_gradients(rank, packed, half, dtype, limit):
    """rel-L2 of the output and of every gradient.  fp32: the library's 1e-5 for each of the two stages.
    bf16: the library's 2e-2 for a call, here for three calls whose roundings (2^-8 each at most, of y, the
    rotated rows, P, dS, o and the gradients, some 1.7e-3 rms each) add up to well below it."""
    from dynamic_short_convolutions_b200 import _lib as L, ops

    N, heads, kv, hd, K = 256, 4, 2, 64, 3
    u, h, A, B, go = _layer(dtype, N, heads, kv, hd, K, rank, 64, seed=1)
    table = ops.rope_table(N, 32, device="cuda")
    cu = [0, 1, 90, 256] if packed else [0, 128, 256]
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda") if packed else None
    leaves = [t.clone().requires_grad_() if t is not None else None for t in (u, h, A, B)]
    o = ops.dynamic_conv_attention(*leaves, K, heads, kv, hd, table, 0 if rank else 64, 1 if packed else 2, cu_t,
                                   layout=L.ROPE_HALF if half else L.ROPE_INTERLEAVED)
    used = [t for t in leaves if t is not None]
    got = [o] + list(torch.autograd.grad(o, used, go))
    ref_leaves = [t.double().requires_grad_() if t is not None else None for t in (u, h, A, B)]
    ref = _plain(*ref_leaves, K, heads, kv, hd, table, half, cu)
    want = [ref] + list(torch.autograd.grad(ref, [t for t in ref_leaves if t is not None], go.double()))
    for name, a, b in zip(["o", "du", "dh"] + (["dA"] if rank else []) + ["dB"], got, want):
        off = float((a.detach().double() - b.detach()).norm() / b.detach().norm())
        assert off <= limit, f"{name}: rel-L2 {off:.3g}"


@pytest.mark.parametrize("dtype,limit", [(torch.float32, 2e-5), (torch.bfloat16, 2e-2)], ids=["f32", "bf16"])
def test_layer_served_token_by_token(dtype, limit):
    """The convolution's decode step, then the attention step, against the 64-bit layer over the prompt."""
    from dynamic_short_convolutions_b200 import _lib as L, ops

    batch, n, heads, kv, hd, K, rank = 3, 20, 4, 2, 64, 3, 16
    C, wq, wk = (heads + 2 * kv) * hd, heads * hd, kv * hd
    u, h, A, B, _ = _layer(dtype, batch * n, heads, kv, hd, K, rank, 64, seed=2)
    table = ops.rope_table(n, hd, device="cuda")
    conv = ops.DynConvDecoder(L.LOWRANK, dtype, batch, 128, C, K, rank)
    attn = ops.AttnDecoder(dtype, batch, heads, kv, hd, n, rope_table=table, rope_layout=L.ROPE_HALF, q_row_stride=C,
                           k_row_stride=C, v_row_stride=C)
    ref = _plain(*(t.double() for t in (u, h, A, B)), K, heads, kv, hd, table, True, list(range(0, batch * n + 1, n)))
    got = torch.empty((batch * n, wq), dtype=dtype, device="cuda")
    for t in range(n):
        rows = torch.arange(batch, device="cuda") * n + t
        y = conv.step(u[rows], h[rows], A, B)
        got[rows] = attn.step(y[:, :wq], y[:, wq:wq + wk], y[:, wq + wk:])
        attn.advance()
    assert L.dynconv_device_status(attn.ws) == 0
    off = float((got.double() - ref).norm() / ref.norm())
    assert off <= limit, f"rel-L2 {off:.3g}"


def test_layer_refuses_what_does_not_fit():
    from dynamic_short_convolutions_b200 import ops

    qkv = torch.zeros((8, 512), device="cuda")
    with pytest.raises(ValueError):
        ops.qkv_attention(qkv, 4, 1, 64)                          # 512 channels are no 4 + 2 heads of 64
    with pytest.raises(ValueError):
        ops.qkv_attention(qkv, 4, 2, 64, batch=3)
