"""Paged cache on the CPU: batches with nothing to do and tables past what the
kernels' 32-bit slot numbers hold.  No GPU call is made."""
import pytest


@pytest.fixture(scope="module")
def vc():
    from lossless_draft_verify_gb300 import build, vc
    build.build()
    vc.load()
    return vc


A = 1 << 20
BIG = 1 << 50


def _cache(vc, **kw):
    f = dict(k_pages=A, v_pages=A, block_table=A, status=A, B=2, Hkv=2, d=128, page=64, n_pages=10, max_blocks=4, dt=0)
    f.update(kw)
    return vc.PagedCacheC(*[f[n] for n, _ in vc.PagedCacheC._fields_])


def test_a_batch_without_rows_needs_no_row_arrays(vc):
    """An empty tensor's address is null: with T = 0 the calls take it."""
    L = vc.load()
    c = _cache(vc)
    rope = vc.vc_rope_init(64, 1e4)
    assert L.vc_paged_append(None, None, None, 1e-6, rope, None, A, A, 0, 4, c, None, None) == 0
    ws = L.vc_paged_attn_h2o_workspace_bytes(c, 0, 4)
    assert 0 < ws <= 1 << 20
    assert L.vc_paged_attn(None, c, A, A, 0, 4, 1.0, None, A, ws, None) == 0
    assert L.vc_paged_attn_h2o(None, c, A, A, 0, 4, 1.0, None, A, 256, A, ws, None) == 0
    # what is not empty is still checked
    assert L.vc_paged_append(None, None, None, 1e-6, rope, None, A, A, 1, 4, c, A, None) == 1
    assert L.vc_paged_append(A, None, None, 1e-6, rope, None, A, A, 1, 4, c, None, None) == 1
    assert L.vc_paged_append(None, None, None, 1e-6, rope, None, None, A, 0, 4, c, None, None) == 1
    assert L.vc_paged_append(None, None, None, 1e-6, rope, None, A, A, 0, 3, c, None, None) == 1
    for i, want in ((0, 1), (7, 1)):
        a = [A, c, A, A, 1, 4, 1.0, A + 4096, A, BIG, None]
        a[i] = None
        assert L.vc_paged_attn(*a) == want
    assert L.vc_paged_attn(None, c, None, A, 0, 4, 1.0, None, A, ws, None) == 1
    assert L.vc_paged_attn(None, c, A, A, 0, 4, -1.0, None, A, ws, None) == 1
    assert L.vc_paged_attn_h2o(None, c, A, A, 0, 4, 1.0, None, None, 256, A, ws, None) == 1
