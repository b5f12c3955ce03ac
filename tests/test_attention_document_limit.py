"""How many documents attention takes: its kernels search cu_seqlens with 32-bit sums of two indices and walk it in
steps of a block, so the count stays at 2^30 (empty documents count, so it may pass the number of tokens)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

MOST = 1 << 30


def test_indices_of_the_search_and_the_walk_stay_in_32_bits():
    """What seg_bounds32 and attn_prep_kernel compute at the limit, and what one past the search's range would."""
    top = (1 << 31) - 1
    assert (MOST - 1) + MOST <= top                            # lo + hi, lo < hi <= documents
    assert MOST - 1 + 1024 <= top                              # the walk's last step, 1024 threads
    assert (MOST + 1) + (MOST + 2) > top


@pytest.mark.parametrize("docs", [MOST + 1, (1 << 31) - 2])
def test_more_documents_are_refused(docs):
    from dynamic_short_convolutions_b200 import _lib as L

    lib, d = L.load(), L.make_attn_desc(1, 1, 64, 4, 2, 64)
    t = torch.zeros((64, 256), dtype=torch.bfloat16)           # never read: the count is refused before any pointer is
    p = ctypes.c_void_p(t.data_ptr())
    assert lib.dynconv_attn_fwd(ctypes.byref(d), p, docs, p, p, p, p, None, p, 1 << 20, None) == 2
    assert "documents" in L.dynconv_last_error()
    assert lib.dynconv_attn_bwd(ctypes.byref(d), p, docs, p, p, p, p, p, p, p, p, p, p, 1 << 20, None) == 2
    assert "documents" in L.dynconv_last_error()


def test_the_limit_itself_gets_past_the_count():
    from dynamic_short_convolutions_b200 import _lib as L

    lib, d = L.load(), L.make_attn_desc(1, 1, 64, 4, 2, 64)
    t = torch.zeros((64, 256), dtype=torch.bfloat16)
    p = ctypes.c_void_p(t.data_ptr())
    # a host pointer: what is refused next
    assert lib.dynconv_attn_fwd(ctypes.byref(d), p, MOST, p, p, p, p, None, p, 1 << 20, None) == 1
    assert "documents" not in L.dynconv_last_error()
