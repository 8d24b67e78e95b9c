"""Host-side checks of the cache calls: what the library and the binding refuse
before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import mixture_experts_layer_fwd_gb300 as m


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    from mixture_experts_layer_fwd_gb300 import _lib
    return _lib.load()


P = ctypes.c_void_p
A = P(4096)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def norm(lib, T=4, Hq=8, Hkv=2, D=128, qs=1024, ks=256, vs=256, rot=128, top=9, page=64, pages=4, q=A, cs=A, pool=A,
         k_out=None, v=A, slots=A):
    return lib.moe_qk_norm_rope(q, qs, A, ks, v, vs, T, Hq, Hkv, D, A, A, 1e-6, cs, top, rot, 0, A, A, k_out, pool, pages,
                                page, A, A, slots, None)


def test_norm_rope_host_checks(lib):
    assert norm(lib, T=0) == 0
    assert norm(lib, T=-1) == INVALID
    assert norm(lib, D=96) == UNSUPPORTED
    assert norm(lib, rot=24) == UNSUPPORTED
    assert norm(lib, rot=144) == UNSUPPORTED
    assert norm(lib, page=48) == UNSUPPORTED
    assert norm(lib, T=1 << 24) == UNSUPPORTED
    assert norm(lib, q=None) == INVALID
    assert norm(lib, q=P(4104)) == INVALID
    assert norm(lib, qs=1020) == INVALID     # not a multiple of 8
    assert norm(lib, qs=1016) == INVALID     # tokens overlap
    assert norm(lib, cs=None) == INVALID
    assert norm(lib, top=0) == INVALID
    assert norm(lib, pool=None) == INVALID   # keys would go nowhere
    assert norm(lib, v=None) == INVALID
    assert norm(lib, slots=None) == INVALID
    assert norm(lib, pages=0) == INVALID


def attn(lib, T=4, Hq=8, Hkv=2, D=128, qs=1024, page=64, B=2, M=3, causal=1, window=0, q=A, ws=A, nbytes=1 << 40, pages=4):
    return lib.moe_kv4_attention(q, qs, T, Hq, A, pages, page, Hkv, D, A, A, A, A, A, B, M, 0.1, causal, window, A, None, ws,
                                 nbytes, None)


def test_attention_host_checks(lib):
    assert attn(lib, T=0) == 0
    assert attn(lib, B=0) == 0
    assert attn(lib, T=-1) == INVALID
    assert attn(lib, D=256) == UNSUPPORTED
    assert attn(lib, page=16) == UNSUPPORTED
    assert attn(lib, Hkv=3) == UNSUPPORTED
    assert attn(lib, window=5, causal=0) == INVALID
    assert attn(lib, window=-1) == INVALID
    assert attn(lib, q=None) == INVALID
    assert attn(lib, qs=1000) == INVALID
    assert attn(lib, M=0) == INVALID
    assert attn(lib, M=1 << 25) == UNSUPPORTED
    assert attn(lib, ws=P(4100)) == INVALID
    assert attn(lib, pages=0) == INVALID


def test_workspace_sizes(lib):
    f = lib.moe_kv4_attention_workspace_size
    assert f(0, 1, 8, 2, 128) == 0 and f(4, 1, 8, 3, 128) == 0 and f(4, 1, 8, 2, 96) == 0
    assert f(4, 4, 8, 2, 128) > 0
    assert f(4096, 1, 8, 2, 128) > f(4, 4, 8, 2, 128)
    g = lib.moe_kv_pages_workspace_size
    assert g(0, 4) == 0 and g(1000, 4) >= 2 * 4 * 1000


def pages_call(lib, name, S=4, M=2, N=8, page=64, n=2, table=A, refs=A, ws=A, nbytes=1 << 30, layers=1, stride=64, rec=16):
    if name == "extend":
        return lib.moe_kv_extend(A, n, table, A, refs, S, M, N, page, A, A, refs, A, A, ws, nbytes, None)
    if name == "fork":
        return lib.moe_kv_fork(A, A, n, table, A, refs, S, M, N, page, A, A, refs, A, layers, stride, rec, ws, nbytes, None)
    if name == "free":
        return lib.moe_kv_free(A, n, table, A, refs, S, M, N, page, A, A, refs, None)
    return lib.moe_kv_compact(table, refs, S, M, N, A, refs, A, A, layers, stride, rec, ws, nbytes, None)


@pytest.mark.parametrize("name", ["extend", "fork", "free", "compact"])
def test_page_operations_host_checks(lib, name):
    assert pages_call(lib, name, S=-1) == INVALID
    assert pages_call(lib, name, M=0) == INVALID
    assert pages_call(lib, name, N=0) == INVALID
    assert pages_call(lib, name, table=None) == INVALID
    assert pages_call(lib, name, refs=P(4100)) == INVALID
    if name != "compact":
        assert pages_call(lib, name, page=16) == UNSUPPORTED
        assert pages_call(lib, name, n=-1) == INVALID
        assert pages_call(lib, name, S=0) == 0
    if name != "free":
        assert pages_call(lib, name, ws=None) == INVALID
        assert pages_call(lib, name, nbytes=16) == WORKSPACE
    if name in ("fork", "compact"):
        assert pages_call(lib, name, rec=24) == INVALID
        assert pages_call(lib, name, layers=-1) == INVALID
    assert lib.moe_kv_copy_pages(A, 1, 64, 16, 4, None, None, 0, None) == 0
    assert lib.moe_kv_copy_pages(A, 1, 64, 16, 4, None, A, 2, None) == INVALID
    assert lib.moe_kv_copy_pages(P(4104), 1, 64, 16, 4, A, A, 2, None) == INVALID


def test_lengths_of_a_step_are_an_array_of_their_own(lib):
    f = lambda lens_out, kv: lib.moe_kv_extend_ex(A, 2, A, A, A, 4, 2, 8, 64, A, lens_out, A, A, A, kv, A, 1 << 30, None)  # noqa: E731
    assert f(P(8192), P(8192)) == INVALID and f(P(8192), A) == INVALID and f(A, P(4098)) == INVALID


@pytest.mark.parametrize("name", ["extend", "fork", "free", "compact"])
def test_page_operations_check_refs_of_a_table_without_rows(lib, name):
    """They are read 16 bytes at a time with no rows too."""
    assert pages_call(lib, name, S=0, refs=P(4100)) == INVALID
    assert pages_call(lib, name, S=0, refs=None) == INVALID


def test_status_of_missing_pages_has_a_name(lib):
    assert lib.moe_status_string(6) == b"MOE_ERR_PAGES"


def test_binding_rejects_host_tensors():
    bf, i = torch.bfloat16, lambda *s: torch.zeros(*s, dtype=torch.int32)
    q, k = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(2, 2, 64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_qk_norm_rope(q, k)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_kv4_attention(q, torch.zeros(1, 2, 4608, dtype=torch.uint8), torch.ones(2), torch.ones(2), i(2), i(1), i(1, 1))
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_kv_extend(i(3), 2, i(2, 2), i(2), i(4), 64)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_kv_fork(i(1), i(1), i(2, 2), i(2), i(4))
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_kv_free(i(1), i(2, 2), i(2), i(4))
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_kv_compact(i(2, 2), i(4))
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_kv_copy_pages(torch.zeros(1, 2, 4, dtype=torch.uint8), i(1), i(1))
