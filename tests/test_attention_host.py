"""Rotary and attention operators without a GPU: descriptor validation, kernel-family query,
descriptor layouts against the header, the scaled tables, and the 64-bit reference's gradients
against differences."""
import ctypes
import math
import os

import pytest

torch = pytest.importorskip("torch")

from attn_reference import attention, rope  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _desc(dtype=1, batch=2, seqlen=64, heads=4, kv=2, hd=64, **kw):
    from dynamic_short_convolutions_b200 import _lib as L

    return L.make_attn_desc(dtype, batch, seqlen, heads, kv, hd, **kw)


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(batch=-1), dict(seqlen=-3), dict(heads=0), dict(heads=3), dict(kv=0),
                                dict(hd=0), dict(hd=129), dict(algo=3), dict(scale=-1.0), dict(scale=float("inf")),
                                dict(scale=float("nan")), dict(q_row_stride=255), dict(dv_row_stride=-8),
                                dict(batch=1 << 20, seqlen=1 << 20), dict(batch=1 << 62, seqlen=4),
                                dict(seqlen=1 << 31, batch=0), dict(heads=1 << 40, kv=1), dict(k_row_stride=1 << 62),
                                dict(batch=1, seqlen=(1 << 31) - 1, heads=4, kv=4, algo=0, dq_row_stride=1 << 40)],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_attention_descriptors_refused(kw):
    from dynamic_short_convolutions_b200 import _lib as L

    assert L.dynconv_attn_workspace_bytes(_desc(**kw)) == 0
    assert L.dynconv_last_error()
    with pytest.raises(L.DynConvError) as e:
        L.dynconv_attn_query_family(_desc(**kw))
    assert e.value.status in (1, 2)


def test_attention_families():
    from dynamic_short_convolutions_b200 import _lib as L

    f, b, why = L.dynconv_attn_query_family(_desc(dtype=0))
    assert (f, b) == ("cuda_core", "cuda_core") and why
    f, b, why = L.dynconv_attn_query_family(_desc(algo=L.ALGO_SIMT))
    assert (f, b) == ("cuda_core", "cuda_core") and "CUDA-core" in why
    for kw in (dict(dtype=0), dict(hd=36), dict(q_row_stride=257)):
        f, b, why = L.dynconv_attn_query_family(_desc(**kw))
        assert (f, b) == ("cuda_core", "cuda_core") and why
        with pytest.raises(L.DynConvError) as e:
            L.dynconv_attn_query_family(_desc(algo=L.ALGO_TC, **kw))
        assert e.value.status == 2
    assert L.dynconv_attn_workspace_bytes(_desc()) >= 256 + 4 * 128 * 4


def test_host_pointers_are_refused():
    from dynamic_short_convolutions_b200 import _lib as L

    t = torch.zeros((128, 256), dtype=torch.bfloat16)
    lib = L.load()
    p = ctypes.c_void_p(t.data_ptr())
    d = _desc()
    assert lib.dynconv_attn_fwd(ctypes.byref(d), None, 0, p, p, p, p, None, p, 1 << 20, None) == 1
    assert lib.dynconv_attn_bwd(ctypes.byref(d), None, 0, p, p, p, p, p, p, p, p, p, p, 1 << 20, None) == 1
    assert lib.dynconv_attn_fwd(None, None, 0, p, p, p, p, None, p, 1 << 20, None) == 1
    r = L.make_rope_desc(1, 0, 2, 64, 4, 64, torch.zeros((64, 64)))
    assert lib.dynconv_rope(ctypes.byref(r), None, 0, None, p, p, p, 256, None) == 1
    assert lib.dynconv_rope(None, None, 0, None, p, p, p, 256, None) == 1


def test_descriptor_layouts_match_the_header(tmp_path):
    import shutil
    import subprocess

    from dynamic_short_convolutions_b200 import _lib as L

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {n: getattr(L, n) for n in ("dynconv_rope_desc", "dynconv_attn_desc", "dynconv_attn_decode_desc")
               if hasattr(L, n)}
    body = "".join(f'    printf("{n} %zu\\n", sizeof({n}));\n' + "".join(
        f'    printf("{n}.{f[0]} %zu\\n", offsetof({n}, {f[0]}));\n' for f in s._fields_) for n, s in structs.items())
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dynconv_attn.h"\nint main(void) {\n'
                   f"{body}    return 0;\n}}\n")
    exe = tmp_path / "probe"
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    out = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for n, s in structs.items():
        assert int(out[n]) == ctypes.sizeof(s)
        for f in s._fields_:
            assert int(out[f"{n}.{f[0]}"]) == getattr(s, f[0]).offset, f"{n}.{f[0]}"


def test_scaled_tables():
    from dynamic_short_convolutions_b200 import ops

    def angles(**kw):
        t = ops.rope_table(3, 64, device="cpu", **kw).double()
        return torch.atan2(t[1, 1::2], t[1, 0::2]), t[1, 0::2].hypot(t[1, 1::2])

    plain, one = angles()
    assert torch.allclose(plain, 10000.0 ** (-torch.arange(0, 64, 2).double() / 64), atol=1e-7)
    assert torch.allclose(one, torch.ones(32, dtype=torch.float64), atol=1e-6)
    assert torch.allclose(angles(scaling="linear", factor=4.0)[0], plain / 4, atol=1e-7)
    ntk = angles(scaling="ntk", factor=8.0)[0]
    assert math.isclose(float(ntk[0]), 1.0, rel_tol=1e-6) and math.isclose(float(ntk[-1]), float(plain[-1]) / 8, rel_tol=1e-4)
    yarn, gain = angles(scaling="yarn", factor=16.0, original_max_pos=4096)
    assert torch.allclose(gain, torch.full((32,), 0.1 * math.log(16.0) + 1, dtype=torch.float64), atol=1e-6)
    turns = 4096 * plain / (2 * math.pi)
    assert torch.allclose(yarn[turns > 40], plain[turns > 40], rtol=1e-5)
    assert torch.allclose(yarn[turns < 0.7], plain[turns < 0.7] / 16, rtol=1e-3, atol=1e-8)
    assert ((yarn <= plain * (1 + 1e-6)) & (yarn >= plain / 16 * (1 - 1e-3))).all()
    assert torch.equal(angles(scaling="yarn", factor=16.0, gain=1.0)[0] > 0, yarn > 0)
    far = ops.rope_table(70000, 8, device="cpu")[69999].double()
    want = 69999 * 10000.0 ** (-torch.arange(0, 8, 2).double() / 8)
    assert torch.allclose(far[0::2], want.cos(), atol=1e-7) and torch.allclose(far[1::2], want.sin(), atol=1e-7)
    for bad in (dict(head_dim=7), dict(head_dim=8, scaling="other"), dict(head_dim=8, scaling="linear", factor=0.5)):
        with pytest.raises(ValueError):
            ops.rope_table(4, device="cpu", **bad)


def test_reference_gradients_against_differences():
    torch.manual_seed(0)
    N, heads, kv, hd, cu = 9, 4, 2, 3, [0, 1, 6, 9]
    x = {n: torch.randn((N, w * hd), dtype=torch.float64) for n, w in (("q", heads), ("k", kv), ("v", kv))}
    do = torch.randn((N, heads * hd), dtype=torch.float64)
    ref = attention(x["q"], x["k"], x["v"], cu, heads, kv, hd, do)
    e = 1e-5
    for n, g in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        for i in range(0, x[n].numel(), 5):
            f = []
            for step in (e, -e):
                y = {a: t.clone() for a, t in x.items()}
                y[n].view(-1)[i] += step
                f.append(float((attention(y["q"], y["k"], y["v"], cu, heads, kv, hd)["o"][0] * do).sum()))
            assert math.isclose((f[0] - f[1]) / (2 * e), float(ref[g][0].view(-1)[i]), rel_tol=1e-6, abs_tol=1e-8)


def test_reference_rotation_is_orthogonal_and_its_inverse_undoes_it():
    from dynamic_short_convolutions_b200 import ops

    torch.manual_seed(1)
    x = torch.randn((5, 24), dtype=torch.float64)
    table, pos = ops.rope_table(50, 8, device="cpu"), torch.tensor([0, 3, 49, 7, 7])
    for half in (False, True):
        y = rope(x, table, pos, 2, 12, half)[0]
        assert torch.allclose(y.norm(dim=1), x.norm(dim=1), rtol=1e-6)
        assert torch.allclose(rope(y, table, pos, 2, 12, half, inverse=True)[0], x, atol=1e-6)
        assert torch.equal(y[0], x[0]) and torch.equal(y.view(5, 2, 12)[..., 8:], x.view(5, 2, 12)[..., 8:])


def test_token_limit():
    """The last tile of the longest run still has 31-bit indices."""
    from dynamic_short_convolutions_b200 import _lib as L

    most = (1 << 31) - 256
    assert L.dynconv_attn_workspace_bytes(_desc(batch=1, seqlen=most, heads=1, kv=1, hd=8)) > 0
    assert L.dynconv_attn_workspace_bytes(_desc(batch=1, seqlen=most + 1, heads=1, kv=1, hd=8)) == 0
    assert "2^31 - 256" in L.dynconv_last_error()


def test_sequences_have_to_share_the_tokens():
    from dynamic_short_convolutions_b200 import ops

    for batch in (0, -1, 3):
        with pytest.raises(ValueError):
            ops.qkv_attention(torch.zeros((8, 512)), 4, 2, 64, batch=batch)
