"""64-bit reference of the rotary and attention operators, with element-wise error bounds.

The bounds count the roundings a kernel may make.  One rounding to the storage type moves a value by
at most half a step, relatively eps / 2 (bf16: 2^-8).  For bf16 storage the kernels may round the
probabilities (for o and dv), ds (for dq and dk), the output o that D = d_o . o is taken from, and each
output:
  o:   eps/2 (|o| + sum p |v|)                 dv:  eps/2 (|dv| + sum p |d_o|)
  dq:  eps/2 (|dq| + scale sum_j (|ds| + p Dabs_i) |k_j|),  Dabs_i = sum_c |d_o| |o|
  dk:  eps/2 (|dk| + scale sum_i (|ds| + p Dabs_i) |q_i|)
fp32 arithmetic adds, relative to the sums of absolute values, `r32` = (hd + L + 32) 2^-24 (2 + max |s|):
a dot product of hd terms, a sum of L terms and an exponential of an argument of size |s| (an error of
2^-24 |s| there is a relative error of the result), each rounded term by term.

`TINY`: a probability below the smallest normal fp32 number, 2^-126, may be held as 0.  Each such term is
off by less than 2^-126 times factors (values, gradients, queries, scale) of less than 2^12 here, and at
most 2^13 of them are summed: 2^(-126 + 12 + 13) < 2^-100.
"""
import math

import torch

TINY = 2.0 ** -100


def doc_ranges(cu):
    return [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:]) if b > a]


def attention(q, k, v, cu, heads, kv_heads, hd, d_o=None, scale=0.0, eps=0.0, q_err=0.0):
    """values and bounds ({name: (value, bound)}) of o, lse and, with d_o, dq, dk, dv.
    q, k, v, d_o: [N, heads * hd] tensors of any float type on any device; q_err: relative error of q as
    the kernel holds it."""
    dev = q.device
    N, G = q.shape[0], heads // kv_heads
    scale = scale or 1.0 / math.sqrt(hd)
    h = eps / 2
    q, k, v = (t.double().reshape(N, n, hd) for t, n in ((q, heads), (k, kv_heads), (v, kv_heads)))
    z = lambda n: torch.zeros((N, n, hd), dtype=torch.float64, device=dev)
    val = {"o": z(heads), "dq": z(heads), "dk": z(kv_heads), "dv": z(kv_heads)}
    bnd = {n: torch.zeros_like(t) for n, t in val.items()}
    lse = torch.zeros((heads, N), dtype=torch.float64, device=dev)
    lse_bound = torch.zeros_like(lse)
    do = d_o.double().reshape(N, heads, hd) if d_o is not None else None
    for a, b in doc_ranges(cu):
        n = b - a
        qd = q[a:b].permute(1, 0, 2).reshape(kv_heads, G, n, hd)
        kd, vd = (t[a:b].permute(1, 0, 2)[:, None] for t in (k, v))            # [kv, 1, n, hd]
        s = scale * qd @ kd.transpose(-1, -2)
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=dev).triu(1), -math.inf)
        ls = torch.logsumexp(s, -1, keepdim=True)
        p = (s - ls).exp()
        # the largest score as the exponent's argument sees it, and the size of its terms
        big = scale * float((qd.abs() @ kd.abs().transpose(-1, -2)).max())
        r = (hd + n + 32) * 2.0 ** -24 * (2 + big) + 2 * q_err * big
        back = lambda t: t.reshape(-1, n, hd).permute(1, 0, 2)
        o = p @ vd
        size = p @ vd.abs()
        val["o"][a:b], bnd["o"][a:b] = back(o), back(h * (o.abs() + size) + r * size)
        lse[:, a:b] = ls.reshape(heads, n)
        lse_bound[:, a:b] = r * (1 + ls.reshape(heads, n).abs())
        if do is None:
            continue
        dd = do[a:b].permute(1, 0, 2).reshape(kv_heads, G, n, hd)
        dv = (p.transpose(-1, -2) @ dd).sum(1)
        size = (p.transpose(-1, -2) @ dd.abs()).sum(1)
        val["dv"][a:b], bnd["dv"][a:b] = back(dv), back(h * (dv.abs() + size) + r * G * size)
        dp = dd @ vd.transpose(-1, -2)
        D = (dd * o).sum(-1, keepdim=True)
        Dabs = (dd.abs() * o.abs()).sum(-1, keepdim=True)
        ds = p * (dp - D)
        err = h * (ds.abs() + p * Dabs) + r * p * (dd.abs() @ vd.abs().transpose(-1, -2) + Dabs)
        dq = scale * ds @ kd
        dk = scale * (ds.transpose(-1, -2) @ qd).sum(1)
        val["dq"][a:b] = back(dq)
        bnd["dq"][a:b] = back(h * dq.abs() + scale * err @ kd.abs() + r * dq.abs())
        val["dk"][a:b] = back(dk)
        bnd["dk"][a:b] = back(h * dk.abs() + scale * (err.transpose(-1, -2) @ qd.abs()).sum(1)
                              + r * G * scale * (ds.abs().transpose(-1, -2) @ qd.abs()).sum(1))
    flat = lambda t: t.reshape(N, -1)
    out = {n: (flat(val[n]), flat(bnd[n])) for n in (val if d_o is not None else ("o",))}
    out["lse"] = (lse, lse_bound)
    return out


def decode(q, k_cache, v_cache, lens, trees, heads, kv_heads, hd, tokens, scale=0.0, eps=0.0, q_err=0.0):
    """(value, bound) of o for rotated q [batch * tokens, heads * hd] (64 bits) over caches that already hold
    the new rows; trees[b][m]: bitmask of the drafted tokens that token m sees; lens < 0: zero rows.
    q_err: relative error of q as the kernel holds it."""
    scale = scale or 1.0 / math.sqrt(hd)
    G = heads // kv_heads
    q = q.double().reshape(len(lens), tokens, kv_heads, G, hd)
    val, bnd = torch.zeros_like(q), torch.zeros_like(q)
    for b, n in enumerate(lens):
        if n < 0:
            continue
        k, v = (t[b, :, :n + tokens].double() for t in (k_cache, v_cache))     # [kv, rows, hd]
        for m in range(tokens):
            at = list(range(n)) + [n + j for j in range(tokens) if trees[b][m] >> j & 1]
            if not at:
                continue
            ks, vs = k[:, at], v[:, at]
            s = scale * torch.einsum("kgd,kjd->kgj", q[b, m], ks)
            p = torch.softmax(s, -1)
            size = torch.einsum("kgj,kjd->kgd", p, vs.abs())
            big = scale * float(torch.einsum("kgd,kjd->kgj", q[b, m].abs(), ks.abs()).max())
            r = (hd + len(at) + 32) * 2.0 ** -24 * (2 + big) + 2 * q_err * big
            o = torch.einsum("kgj,kjd->kgd", p, vs)
            val[b, m], bnd[b, m] = o, eps / 2 * (o.abs() + size) + r * size
    return val.reshape(-1, heads * hd), bnd.reshape(-1, heads * hd)


def rope(x, table, pos, heads, hd, half, inverse=False, eps=0.0):
    """(value, bound) of the rotation of x [N, heads * hd] at positions pos [N]."""
    N, rot = x.shape[0], table.shape[1]
    x = x.double().reshape(N, heads, hd)
    f = table.double()[pos.long()]
    c, s = f[:, None, 0::2], f[:, None, 1::2]
    s = -s if inverse else s
    ia = torch.arange(rot // 2, device=x.device)
    ia, ib = (ia, ia + rot // 2) if half else (2 * ia, 2 * ia + 1)
    a, b = x[..., ia], x[..., ib]
    y, size = x.clone(), torch.zeros_like(x)
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia], size[..., ib] = (a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()
    bound = eps / 2 * y.abs() + 3 * 2.0 ** -24 * size
    bound[..., rot:] = -TINY                                 # copied as they are
    return y.reshape(N, -1), bound.reshape(N, -1)


def check(name, got, ref):
    """got within its bound of ref = (value, bound), element by element, and finite."""
    value, bound = ref
    got = got.double()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - value).abs() - (bound + TINY)
    i = int(over.argmax())
    assert over.max() <= 0, (f"{name}: element {i} is {float(got.flatten()[i]):.6g}, {float(value.flatten()[i]):.6g} expected, "
                             f"off by more than {float(bound.flatten()[i]):.3g}")
