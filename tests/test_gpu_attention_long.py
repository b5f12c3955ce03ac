"""Long packed inputs: more query and key tiles than attention's preparation has bins to sort them into (1024), and
documents of some thousand tokens, against the 64-bit reference."""
import pytest

from attn_reference import attention, check
from test_gpu_attention import EPS, _inputs, _run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,hd,tile", [("bf16", 8, 128), ("bf16", 72, 128), ("f32", 8, 64)])
def test_more_tiles_than_bins(dtype, hd, tile):
    lens = [8000, 1, 0, 5003, 127, 129] + [400 + 739 * i % 4000 for i in range(58)]
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    N, heads, kv = cu[-1], 2, 1
    assert N > 1024 * tile and max(lens) <= 1 << 13
    q, k, v, do = _inputs(N, heads, kv, hd, dtype, seed=21)
    got = _run(q, k, v, do, 1, N, heads, kv, hd, cu=cu)
    ref = attention(q, k, v, cu, heads, kv, hd, do, 0.0, EPS[dtype])
    for name in ("o", "lse", "dq", "dk", "dv"):
        check(name, got[name], ref[name])
