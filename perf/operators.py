"""Cases for the attention-side operators that follow the QKV convolution: rotary positions, causal
attention over packed prompts (forward and backward) and attention of new or drafted tokens over a
key/value cache.

``run`` computes them in plain torch (32-bit arithmetic, rounded once) where ``own`` is false and
through ``dynamic_short_convolutions_b200.ops`` where it is true; ``exact`` restates them in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # A serving step's new tokens (one per sequence) at far positions of a long, scaled context.
        dict(name="rope_serve", op="rope", dtype="bf16", batch=64, seqlen=1, heads=20, head_dim=128, rot_dim=128,
             half=True, scaled="yarn", positions=True, inverse=False),
        # Q and K of a 2B-scale GQA layer (16 + 4 heads of 128) over a training batch of 4 x 4096.
        dict(name="rope_train", op="rope", dtype="bf16", batch=4, seqlen=4096, heads=20, head_dim=128, rot_dim=128,
             half=False, scaled="none", positions=False, inverse=False),
        # The backward rotation in fp32, half layout, a part of the head rotated, an odd length.
        dict(name="rope_backward_partial", op="rope", dtype="f32", batch=8, seqlen=1999, heads=12, head_dim=64,
             rot_dim=32, half=True, scaled="linear", positions=False, inverse=True),
        # A short prompt on its own: latency.
        dict(name="prompt_short", op="prompt", dtype="bf16", train=False, docs=1, mean=77, spread=0.0, lens_seed=0,
             heads=12, kv_heads=12, head_dim=64),
        # A 2B-scale GQA layer's prompts of one length: 4 x 4096, 16 query and 4 key/value heads of 128.
        dict(name="prompt_2b", op="prompt", dtype="bf16", train=False, docs=4, mean=4096, spread=0.0, lens_seed=0,
             heads=16, kv_heads=4, head_dim=128),
        # Training step of the 150M-scale layer's attention: 8 x 2048, 12 heads of 64.
        dict(name="train_150m", op="prompt", dtype="bf16", train=True, docs=8, mean=2048, spread=0.0, lens_seed=0,
             heads=12, kv_heads=12, head_dim=64),
        # Training step over packed documents of very different lengths, 2B-scale heads.
        dict(name="train_2b_packed", op="prompt", dtype="bf16", train=True, docs=9, mean=1500, spread=1.0,
             lens_seed=3, heads=16, kv_heads=4, head_dim=128),
        # Training step in fp32 (parity runs), packed, odd lengths.
        dict(name="train_f32", op="prompt", dtype="f32", train=True, docs=5, mean=400, spread=0.7, lens_seed=5,
             heads=8, kv_heads=2, head_dim=64),
        # One sequence's next token: latency.
        dict(name="decode_one", op="decode", dtype="bf16", batch=1, tokens=1, max_len=2048, fill=0.6, lens_seed=1,
             heads=12, kv_heads=12, head_dim=64, half=False),
        # A serving batch's next tokens over long caches, 2B-scale heads.
        dict(name="decode_batch", op="decode", dtype="bf16", batch=64, tokens=1, max_len=4096, fill=0.9, lens_seed=2,
             heads=16, kv_heads=4, head_dim=128, half=True),
        # Checking a tree of drafted tokens for a small batch.
        dict(name="decode_tree", op="decode", dtype="bf16", batch=8, tokens=24, max_len=4096, fill=0.8, lens_seed=4,
             heads=16, kv_heads=4, head_dim=128, half=True),
        # fp32 cache, a short chain of drafted tokens, odd lengths.
        dict(name="decode_f32", op="decode", dtype="f32", batch=13, tokens=3, max_len=1031, fill=0.7, lens_seed=6,
             heads=8, kv_heads=2, head_dim=64, half=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "prompt", "decode", "decode"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    head_dim = rng.choice([32, 64, 64, 80, 96, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
    if op == "rope":
        batch = _log(rng, 1, 16)
        seqlen = max(1, min(_log(rng, 1, 4096), 40_000_000 // (batch * heads * head_dim)))
        return dict(op=op, dtype=dtype, batch=batch, seqlen=seqlen, heads=heads, head_dim=head_dim,
                    rot_dim=rng.choice([head_dim, head_dim // 2]), half=rng.random() < 0.5,
                    scaled=rng.choice(["none", "linear", "yarn"]), positions=rng.random() < 0.4,
                    inverse=rng.random() < 0.4)
    if op == "prompt":
        train = rng.random() < 0.6
        docs = _log(rng, 1, 24)
        mean = _log(rng, 1, 4096)
        # cost: score entries of all heads, at most those of the largest listed cases
        most = (1.2e9 if train else 4e9) * (64 / max(64, head_dim)) * (0.05 if dtype == "f32" else 1.0) / 4
        mean = max(1, min(mean, int(math.sqrt(most / (docs * heads)))))
        return dict(op=op, dtype=dtype, train=train, docs=docs, mean=mean, spread=rng.choice([0.0, 0.5, 1.0]),
                    lens_seed=rng.randrange(1000), heads=heads, kv_heads=kv_heads, head_dim=head_dim)
    batch = _log(rng, 1, 64)
    tokens = rng.choice([1, 1, 1, 2, 5, 16, 33, 60])
    max_len = _log(rng, 70, 8192)
    max_len = max(tokens + 1, min(max_len, 120_000_000 // (batch * kv_heads * head_dim),
                                  200_000_000 // (batch * heads * tokens)))
    return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, max_len=max_len, fill=rng.choice([0.1, 0.5, 0.9]),
                lens_seed=rng.randrange(1000), heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                half=rng.random() < 0.5)


def _doc_lens(c):
    """Document lengths of a packed batch: equal (spread 0), or spread about the mean on a log scale."""
    r = random.Random(c["lens_seed"])
    return [max(1, int(round(c["mean"] * math.exp(r.uniform(-1.5, 1.0) * c["spread"])))) for _ in range(c["docs"])]


def _cache_lens(c):
    """Tokens each sequence already has in the cache, with room for the new ones; one is empty in a batch."""
    r = random.Random(c["lens_seed"])
    room = c["max_len"] - c["tokens"]
    lens = [min(room, max(0, int(room * c["fill"] * r.uniform(0.5, 1.1)))) for _ in range(c["batch"])]
    if c["batch"] > 4:
        lens[c["batch"] // 2] = 0
    return lens


def _tree(c):
    """Ancestor bitmasks [batch][tokens], each token's own bit among them: random trees (a chain for few tokens)."""
    r = random.Random(c["lens_seed"] + 77)
    rows = []
    for _ in range(c["batch"]):
        masks = []
        for m in range(c["tokens"]):
            parent = m - 1 if c["tokens"] < 4 else r.randint(max(-1, m - 6), m - 1)
            masks.append((masks[parent] if parent >= 0 else 0) | (1 << m))
        rows.append(masks)
    return rows


# ------------------------------------------------------------------------------------------- inputs
def _table(max_pos, rot_dim, scaled):
    """fp32 [max_pos, rot_dim]: cos and sin of each pair's angle side by side, from 64-bit angles.
    linear: positions divided by 4.  yarn: pairs that turn less than once over the original 4096
    positions slowed by 16, those that turn 32 times or more left, a ramp between, and cos and sin
    times 0.1 ln 16 + 1."""
    p = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None]
    f = 10000.0 ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device="cuda") / rot_dim)
    gain = 1.0
    if scaled == "linear":
        f = f / 4.0
    elif scaled == "yarn":
        dim = [rot_dim * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0)) for turns in (32.0, 1.0)]
        low, high = max(math.floor(dim[0]), 0), min(math.ceil(dim[1]), rot_dim - 1)
        at = torch.arange(rot_dim // 2, dtype=torch.float64, device="cuda")
        slow = ((at - low) / max(high - low, 1e-3)).clamp(0, 1)
        f = f * (1 - slow) + f / 16.0 * slow
        gain = 0.1 * math.log(16.0) + 1.0
    a = p * f
    return (gain * torch.stack((a.cos(), a.sin()), -1)).reshape(max_pos, rot_dim).float().contiguous()


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(DTYPES[dtype])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, hd = c["dtype"], c["head_dim"]
    s = {"case": c}
    if c["op"] == "rope":
        n = c["batch"] * c["seqlen"]
        max_pos = 65536 if c["positions"] else c["seqlen"]
        s["x"] = _normal(g, (n, c["heads"] * hd), dt)
        s["table"] = _table(max_pos, c["rot_dim"], c["scaled"])
        s["pos"] = torch.arange(n, device="cuda", dtype=torch.int32) % c["seqlen"]
        if c["positions"]:
            s["pos"] = torch.randint(0, max_pos, (n,), generator=g, device="cuda", dtype=torch.int32)
        if own:
            from dynamic_short_convolutions_b200 import _lib as L, ops

            s["plan"] = ops.RopePlan(DTYPES[dt], c["batch"], c["seqlen"], c["heads"], hd, s["table"],
                                     layout=L.ROPE_HALF if c["half"] else L.ROPE_INTERLEAVED)
    elif c["op"] == "prompt":
        lens = _doc_lens(c)
        n, top = sum(lens), max(lens)
        s["q"] = _normal(g, (n, c["heads"] * hd), dt)
        s["k"] = _normal(g, (n, c["kv_heads"] * hd), dt)
        s["v"] = _normal(g, (n, c["kv_heads"] * hd), dt)
        s["do"] = _normal(g, (n, c["heads"] * hd), dt) if c["train"] else None
        start = torch.tensor([0] + lens, device="cuda").cumsum(0)
        s["cu"] = start.int() if c["spread"] else None        # one length: a dense batch
        # packed row of each place of a [docs, longest] batch (the plain form pads), and the places that are real
        at = torch.arange(top, device="cuda")
        s["held"] = at[None] < torch.tensor(lens, device="cuda")[:, None]
        s["rows"] = torch.where(s["held"], start[:-1, None] + at[None], 0)
        s["real"] = s["held"].reshape(-1).nonzero()[:, 0]
        if own:
            from dynamic_short_convolutions_b200 import ops

            s["plan"] = ops.AttnPlan(DTYPES[dt], *((1, n) if c["spread"] else (c["docs"], c["mean"])), c["heads"],
                                     c["kv_heads"], hd)
    else:
        b, m, kv = c["batch"], c["tokens"], c["kv_heads"]
        s["q"] = _normal(g, (b * m, c["heads"] * hd), dt)
        s["k"] = _normal(g, (b * m, kv * hd), dt)
        s["v"] = _normal(g, (b * m, kv * hd), dt)
        s["k_cache"] = _normal(g, (b, kv, c["max_len"], hd), dt)
        s["v_cache"] = _normal(g, (b, kv, c["max_len"], hd), dt)
        s["lens"] = torch.tensor(_cache_lens(c), dtype=torch.int32, device="cuda")
        s["tree"] = torch.tensor(_tree(c), dtype=torch.int64, device="cuda")
        s["table"] = _table(c["max_len"], hd, "none")
        if own:
            from dynamic_short_convolutions_b200 import _lib as L, ops

            s["plan"] = ops.AttnDecoder(DTYPES[dt], b, c["heads"], kv, hd, c["max_len"], tokens=m,
                                        rope_table=s["table"],
                                        rope_layout=L.ROPE_HALF if c["half"] else L.ROPE_INTERLEAVED,
                                        k_cache=s["k_cache"], v_cache=s["v_cache"], lens=s["lens"])
    return s


# ------------------------------------------------------------------------------------------- plain forms
def _rotate(x, rows, half, inverse):
    """x [..., heads, head_dim] turned by the table rows [..., rot_dim] of its positions."""
    rot = rows.shape[-1]
    cos, sin = rows[..., None, 0::2], rows[..., None, 1::2]
    sin = -sin if inverse else sin
    part, rest = x[..., :rot], x[..., rot:]
    if half:
        a, b = part[..., : rot // 2], part[..., rot // 2:]
        part = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return torch.cat((part, rest), -1)


def _prompt(s):
    c = s["case"]
    h, kv, hd = c["heads"], c["kv_heads"], c["head_dim"]
    dt, scale = DTYPES[c["dtype"]], hd ** -0.5
    docs, top = s["rows"].shape

    def padded(x, heads):      # [docs, kv, heads / kv, longest, hd]
        return x.float().view(-1, heads, hd)[s["rows"]].view(docs, top, kv, heads // kv, hd).permute(0, 2, 3, 1, 4)

    def packed(x, heads):
        return x.permute(0, 3, 1, 2, 4).reshape(docs * top, heads * hd)[s["real"]].to(dt)

    q, k, v = padded(s["q"], h), padded(s["k"], kv), padded(s["v"], kv)
    later = torch.ones(top, top, dtype=torch.bool, device="cuda").triu(1)
    p = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(later, float("-inf"))
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True))
    o = packed(p @ v, h)
    if not c["train"]:
        return o
    do = padded(s["do"], h)
    do = do.masked_fill_(~s["held"][:, None, None, :, None], 0.0)      # places behind a document's end
    dv = (p.transpose(-1, -2) @ do).sum(2, keepdim=True)
    ds = do @ v.transpose(-1, -2)
    ds = ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = ds @ k
    dk = (ds.transpose(-1, -2) @ q).sum(2, keepdim=True)
    return {"o": o, "dq": packed(dq, h), "dk": packed(dk, kv), "dv": packed(dv, kv)}


def _bits(tree, tokens):
    return (tree[..., None] >> torch.arange(tokens, device="cuda")) & 1      # [batch, tokens, tokens]


def _decode(s):
    c = s["case"]
    b, m, h, kv, hd, top = c["batch"], c["tokens"], c["heads"], c["kv_heads"], c["head_dim"], c["max_len"]
    lens = s["lens"].long()
    bits = _bits(s["tree"], m)
    rows = s["table"][lens[:, None] + bits.sum(-1) - 1]                        # [batch, tokens, hd]
    q = _rotate(s["q"].float().view(b, m, h, hd), rows, c["half"], False)
    k = _rotate(s["k"].float().view(b, m, kv, hd), rows, c["half"], False)
    at = (lens[:, None] + torch.arange(m, device="cuda")).view(b, 1, m, 1).expand(b, kv, m, hd)
    s["k_cache"].scatter_(2, at, k.transpose(1, 2).to(s["k_cache"].dtype))
    s["v_cache"].scatter_(2, at, s["v"].view(b, m, kv, hd).transpose(1, 2))
    q = q.view(b, m, kv, h // kv, hd).permute(0, 2, 1, 3, 4).reshape(b, kv, m * (h // kv), hd)
    p = (q @ s["k_cache"].float().transpose(-1, -2)).mul_(hd ** -0.5).view(b, kv, m, h // kv, top)
    place = torch.arange(top, device="cuda") - lens[:, None]                   # [batch, top]
    seen = torch.gather(bits, 2, place.clamp(0, m - 1)[:, None].expand(b, m, top)) > 0
    seen = (place < 0)[:, None] | (seen & ((place >= 0) & (place < m))[:, None])
    p = p.masked_fill_(~seen[:, None, :, None], float("-inf"))
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True)).view(b, kv, m * (h // kv), top)
    o = (p @ s["v_cache"].float()).view(b, kv, m, h // kv, hd).permute(0, 2, 1, 3, 4).reshape(b * m, h * hd)
    return {"o": o.to(DTYPES[c["dtype"]]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    s, c = state, state["case"]
    if c["op"] == "rope":
        if own:
            return s["plan"].apply(s["x"], positions=s["pos"] if c["positions"] else None, inverse=c["inverse"])
        x = s["x"].float().view(-1, c["heads"], c["head_dim"])
        y = _rotate(x, s["table"][s["pos"].long()], c["half"], c["inverse"])
        return y.reshape(s["x"].shape).to(s["x"].dtype)
    if c["op"] == "prompt":
        if not own:
            return _prompt(s)
        if not c["train"]:
            return s["plan"].forward(s["q"], s["k"], s["v"], cu_seqlens=s["cu"])
        o, lse = s["plan"].forward(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], want_lse=True)
        grads = s["plan"].backward(s["do"], s["q"], s["k"], s["v"], o, lse, cu_seqlens=s["cu"])
        return {"o": o, "dq": grads["dq"], "dk": grads["dk"], "dv": grads["dv"]}
    if own:
        o = s["plan"].step(s["q"], s["k"], s["v"], ancestors=s["tree"])
        return {"o": o, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return _decode(s)


# ------------------------------------------------------------------------------------------- floors
def work(case):
    c = case
    e, hd = BYTES[c["dtype"]], c["head_dim"]
    if c["op"] == "rope":
        n = c["batch"] * c["seqlen"]
        rows = min(n, 65536) if c["positions"] else c["seqlen"]
        return {"bytes": 2 * n * c["heads"] * hd * e + rows * c["rot_dim"] * 4,
                "flops": 3 * n * c["heads"] * c["rot_dim"]}
    h, kv = c["heads"], c["kv_heads"]
    if c["op"] == "prompt":
        lens = _doc_lens(c)
        n, pairs = sum(lens), sum(x * (x + 1) // 2 for x in lens)
        wide = 2 * h + 2 * kv + ((2 * h + 2 * kv) if c["train"] else 0)
        return {"bytes": n * wide * hd * e, "flops": (14 if c["train"] else 4) * hd * h * pairs}
    lens, m = _cache_lens(c), c["tokens"]
    seen = sum(lens)
    return {"bytes": 2 * seen * kv * hd * e + c["batch"] * m * (2 * h + 4 * kv) * hd * e,
            "flops": 4 * hd * h * m * (seen + sum(bin(x).count("1") for x in sum(_tree(c), [])) // max(1, m))}


# ------------------------------------------------------------------------------------------- 64 bits
def _turn(x, table, pos, half, inverse):
    """Pair i of the first rot channels as a complex number times cos + i sin (its conjugate for the inverse)."""
    rot = table.shape[1]
    z = torch.view_as_complex(table.double().view(-1, rot // 2, 2)[pos.long()])
    z = (z.conj() if inverse else z)[:, None]
    first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if half else (slice(0, rot, 2), slice(1, rot, 2))
    y = x.clone()
    w = torch.complex(x[..., first], x[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    hd = c["head_dim"]
    if c["op"] == "rope":
        x = s["x"].double().view(-1, c["heads"], hd)
        return _turn(x, s["table"], s["pos"], c["half"], c["inverse"]).reshape(s["x"].shape)
    h, kv = c["heads"], c["kv_heads"]
    group = h // kv
    if c["op"] == "prompt":
        q, k, v = (s[n].double().view(-1, w, hd) for n, w in (("q", h), ("k", kv), ("v", kv)))
        o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        do = s["do"].double().view(-1, h, hd) if c["train"] else None
        start = 0
        for n in _doc_lens(c):
            at = slice(start, start + n)
            start += n
            for i in range(h):
                j = i // group
                logits = torch.einsum("id,jd->ij", q[at, i], k[at, j]) / math.sqrt(hd)
                allowed = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
                logits = torch.where(allowed, logits, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
                p = torch.softmax(logits, -1)
                o[at, i] = p @ v[at, j]
                if c["train"]:
                    dv[at, j] += p.T @ do[at, i]
                    dp = do[at, i] @ v[at, j].T
                    ds = p * (dp - (do[at, i] * o[at, i]).sum(-1, keepdim=True)) / math.sqrt(hd)
                    dq[at, i] = ds @ k[at, j]
                    dk[at, j] += ds.T @ q[at, i]
        o = o.reshape(-1, h * hd)
        if not c["train"]:
            return o
        return {"o": o, "dq": dq.reshape(-1, h * hd), "dk": dk.reshape(-1, kv * hd), "dv": dv.reshape(-1, kv * hd)}
    m, lens, tree = c["tokens"], _cache_lens(c), _tree(c)
    pos = torch.tensor([[n + bin(x).count("1") - 1 for x in row] for n, row in zip(lens, tree)], device="cuda").view(-1)
    q = _turn(s["q"].double().view(-1, h, hd), s["table"], pos, c["half"], False).view(-1, m, h, hd)
    k = _turn(s["k"].double().view(-1, kv, hd), s["table"], pos, c["half"], False).view(-1, m, kv, hd)
    o = torch.zeros_like(q)
    for i, n in enumerate(lens):
        s["k_cache"][i, :, n:n + m] = k[i].transpose(0, 1).to(s["k_cache"].dtype)
        s["v_cache"][i, :, n:n + m] = s["v"].view(-1, m, kv, hd)[i].transpose(0, 1)
        keys = s["k_cache"][i, :, :n + m].double().repeat_interleave(group, 0)
        vals = s["v_cache"][i, :, :n + m].double().repeat_interleave(group, 0)
        logits = torch.einsum("mhd,hjd->hmj", q[i], keys) / math.sqrt(hd)
        allowed = torch.tensor([[True] * n + [bool(x >> j & 1) for j in range(m)] for x in tree[i]], device="cuda")
        p = torch.softmax(logits.masked_fill(~allowed, -math.inf), -1)
        o[i] = torch.einsum("hmj,hjd->mhd", p, vals)
    # the caches are held in the storage type: rounding the new keys is the operator's own last step
    return {"o": o.reshape(-1, h * hd), "k_cache": None, "v_cache": None}
