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


def test_tables_past_two_to_the_30_slots_are_refused(vc):
    """Slots are 32-bit numbers that the kernels add tiles and strides to: the
    eviction's last warp ran past 2^31 where a sequence came near it."""
    L = vc.load()
    rope = vc.vc_rope_init(64, 1e4)
    for page, blocks in ((256, (1 << 23) - 1), (256, (1 << 22) + 1), (16, (1 << 26) + 1)):
        c = _cache(vc, page=page, max_blocks=blocks)
        assert L.vc_paged_append(A, None, None, 1e-6, rope, None, A, A, 0, 4, c, A + 4096, None) == 2
        assert L.vc_paged_attn(A, c, A, A, 0, 4, 1.0, A + 4096, A, BIG, None) == 2
        assert L.vc_paged_attn_h2o(A, c, A, A, 0, 4, 1.0, A + 4096, A, (1 << 31) - 1, A, BIG, None) == 2
        assert L.vc_paged_attn_workspace_bytes(c, 4, 4) == 0 == L.vc_paged_attn_h2o_workspace_bytes(c, 4, 4)
        for s, t in ((c, _cache(vc)), (_cache(vc), c)):
            assert L.vc_paged_evict(A, (1 << 31) - 1, s, A, vc.DropCfg(4, 4), t, A + 64, A, 1 << 30, None, 0, None) == 2
    c = _cache(vc, page=256, max_blocks=1 << 22)
    assert L.vc_paged_attn(A, c, A, A, 0, 4, 1.0, A + 4096, A, BIG, None) == 0
    assert L.vc_paged_attn_workspace_bytes(c, 4, 4) > 0


def test_the_mass_workspace_is_bounded(vc):
    """Stored scores are sized by the table, which may be much wider than the
    batch: past 1 GiB of them the call does without."""
    L = vc.load()
    for B, n, slots, stored in ((256, 1, 32768, 1 << 30), (256, 1, 131072, 0), (256, 4, 131072, 0), (1, 1, 1 << 23, 1 << 30),
                                (1, 1, 1 << 24, 0), (16, 1, 32768, 1 << 26)):
        c = _cache(vc, B=B, Hkv=8, max_blocks=slots // 64)
        plain = L.vc_paged_attn_workspace_bytes(c, B * n, 32)
        extra = L.vc_paged_attn_h2o_workspace_bytes(c, B * n, 32) - plain
        assert stored <= extra <= stored + 4 * B * n * 32 + 512, (B, n, slots)
