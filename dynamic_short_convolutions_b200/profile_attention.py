"""One of the operators that follow the Q/K/V convolution, for profiling a kernel under ncu.

    python -m dynamic_short_convolutions_b200.profile_attention --op train --batch 8 --seqlen 2048 \\
        --heads 12 --kv-heads 12 --head-dim 64 [--dtype f32] [--repeats 2]

runs rotary positions of Q and K (``rope``), causal attention (``prompt``; with gradients ``train``) or a
step of ``--tokens`` tokens per sequence over caches of ``--seqlen`` rows (``step``) `repeats` times on
seeded inputs, checks the device status and prints the problem.  Meant for captures such as
``ncu --set full --clock-control none -k regex:attn_fwd_kernel -s 1 -c 1 python -m ...``.
"""
from __future__ import annotations

import argparse
import sys


def build_parser() -> argparse.ArgumentParser:
    ap = argparse.ArgumentParser()
    ap.add_argument("--op", default="prompt", choices=["rope", "prompt", "train", "step"])
    ap.add_argument("--dtype", default="bf16", choices=["bf16", "f32"])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--seqlen", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv-heads", type=int, default=4)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--tokens", type=int, default=1)
    ap.add_argument("--repeats", type=int, default=2)
    return ap


def main(argv=None) -> int:
    a = build_parser().parse_args(argv)
    import torch

    from . import _lib as L, ops

    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(0)

    def rnd(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    step = a.op == "step"
    N = a.batch * (a.tokens if step else a.seqlen)
    q, k, v = (rnd(N, n * a.head_dim) for n in (a.heads, a.kv_heads, a.kv_heads))
    if a.op == "rope":
        plan = ops.RopePlan(dtype, a.batch, a.seqlen, a.heads + a.kv_heads, a.head_dim,
                            ops.rope_table(a.seqlen, a.head_dim))
        qk = torch.cat((q, k), 1)
        run = lambda: plan.apply(qk)
    elif step:
        rows = (a.batch, a.kv_heads, a.seqlen + a.tokens, a.head_dim)
        plan = ops.AttnDecoder(dtype, a.batch, a.heads, a.kv_heads, a.head_dim, rows[2], a.tokens,
                               rope_table=ops.rope_table(rows[2], a.head_dim), k_cache=rnd(*rows), v_cache=rnd(*rows))
        plan.lens.fill_(a.seqlen)
        run = lambda: plan.step(q, k, v)
    else:
        plan = ops.AttnPlan(dtype, a.batch, a.seqlen, a.heads, a.kv_heads, a.head_dim)
        do = rnd(N, a.heads * a.head_dim)

        def run():
            o, lse = plan.forward(q, k, v, want_lse=True)
            if a.op == "train":
                plan.backward(do, q, k, v, o, lse)

    for _ in range(a.repeats):
        run()
    torch.cuda.synchronize()
    st = L.dynconv_device_status(plan.ws)
    if st != 0:
        print("device status", st, L.dynconv_last_error(), file=sys.stderr)
        return 1
    print(f"{a.op}: {a.batch} x {a.seqlen}, heads {a.heads} over {a.kv_heads} of {a.head_dim}, {a.dtype}, "
          f"tokens {a.tokens if step else '-'}, repeats {a.repeats}")
    return 0


if __name__ == "__main__":
    sys.exit(main())
