"""Paged-cache operators on the GPU at the edges of what they accept: scores far
outside the usual range, tables much wider than their sequences, batches of
more sequences than a warp keeps."""
import pytest
import torch

import paged_ref
from helpers import lib
from paged_ref import U_F32, Batch, close, half_step

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _call(vc, bt, q, scale, scores=None):
    cache = vc.PagedCache(bt.k, bt.v, bt.block_table)
    out = torch.full_like(q, 7.0)
    T, Hq, _ = q.shape
    if scores is None:
        ws = vc.Workspace(vc.vc_paged_attn_workspace_bytes(cache, T, Hq))
        vc.vc_paged_attn(q, cache, bt.q_start, bt.ctx, scale, out, ws)
    else:
        ws = vc.Workspace(vc.vc_paged_attn_h2o_workspace_bytes(cache, T, Hq))
        vc.vc_paged_attn_h2o(q, cache, bt.q_start, bt.ctx, scale, out, scores, ws)
    assert vc.vc_poll_status(ws) == 0 and int(cache.status) == 0
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("power,scale", [(41, 1e8), (0, 1e8), (20, 1.0)])
@pytest.mark.parametrize("ns,cs", [([1, 1, 1], [30, 200, 9000]), ([3, 40, 2], [60, 9000, 170])])
def test_scores_of_any_size(dtype, sign, power, scale, ns, cs):
    """Products up to 1e25 at a scale of 1e8, all of one sign, in whole units
    (short contexts) and cut ones (9000 tokens): equal largest scores share the
    weight, all others are too far below to count.  One channel of q and k is
    set, so every product is exact, and equal products give equal scores.  The
    weights are then exactly one before the division; what is left is the sum
    over the values (at most twice (L + 16) half steps of fp32) and the output's
    rounding."""
    vc = lib()
    page, d, G = 16, 64, 2
    bt = Batch(ns, cs, 1, d, page, dtype, seed=1)
    key = torch.where(torch.isnan(bt.k), bt.k, torch.zeros_like(bt.k))
    for b in range(bt.B):
        for s in range(bt.lens[b]):
            key[bt.table[b][s // page], 0, s % page, 0] = (1.375 if s % 3 == 0 else 1.625) * 2.0 ** power
    bt.k = key
    q = torch.zeros(bt.T, G, d, dtype=dtype, device="cuda")
    q[:, :, 0] = sign * 1.6875 * 2.0 ** power
    slots = bt.width * page
    scores = torch.zeros(bt.B, 1, slots, device="cuda")
    outs = [_call(vc, bt, q, scale), _call(vc, bt, q, scale, scores)]
    assert torch.equal(*outs)
    for b in range(bt.B):
        k, v = bt.rows(bt.k, b, 0)[:, 0] * sign, bt.rows(bt.v, b, 0)
        best = torch.zeros(slots, dtype=torch.bool)
        for i in range(ns[b]):
            n = cs[b] + i + 1
            tie = k[:n] == k[:n].max()
            want = v[:n][tie].mean(0).expand(G, d)
            tol = 2 * (n + 16) * U_F32 * v[:n][tie].abs().mean(0) + half_step(dtype) * want.abs() * 1.01
            close(outs[0][bt.start[b] + i], want, tol, f"row {i} of sequence {b}")
            best[:n] |= tie
        got = scores[b, 0].cpu()
        assert torch.isfinite(got).all() and (got[~best] == 0).all() and (got[best] > 0).all()
        assert got.max() <= ns[b] * G * (1 + (ns[b] * G + 16) * U_F32)


@pytest.mark.parametrize("top,recent,slots", [(20, 10, 128), (0, 60, 128), (500, 30, 128), (20, 70, 17000)])
def test_evicted_scores_have_no_negative_zero(top, recent, slots):
    """Zeros of both signs among the chosen and among the newest slots: the
    scores that come out are zeros without sign."""
    vc = lib()
    page, lens = 16, [100, 7]
    bt = Batch([0, 0], lens, 2, 64, page, BF, seed=3, width=-(-slots // page))
    src = vc.PagedCache(bt.k, bt.v, bt.block_table)
    scores = torch.zeros(2, 2, src.slots, device="cuda")
    scores[..., ::2] = -0.0
    n = min(top + recent, src.slots)
    blocks = -(-n // page)
    k2 = torch.zeros(2 * blocks, 2, page, 64, dtype=BF, device="cuda")
    dst = vc.PagedCache(k2, k2.clone(), torch.arange(2 * blocks, dtype=torch.int32, device="cuda").view(2, blocks))
    i32 = dict(dtype=torch.int32, device="cuda")
    n2, kept = torch.zeros(2, **i32), torch.zeros(2, 2, n, **i32)
    out = torch.full((2, 2, n), 5.0, device="cuda")
    vc.vc_paged_evict(scores, src, torch.tensor(lens, **i32), top, recent, dst, n2, kept, scores_out=out)
    torch.cuda.synchronize()
    for b in range(2):
        m = int(n2[b])
        assert m == min(top, max(lens[b] - recent, 0)) + min(recent, lens[b])
        for h in range(2):
            assert kept[b, h, :m].tolist() == paged_ref.evict(scores[b, h].tolist(), lens[b], top, recent)
        assert (out[b, :, :m].view(torch.int32) == 0).all() and (out[b, :, m:] == 5.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_an_empty_batch(dtype):
    """Tensors of no rows: every call returns without touching anything."""
    vc = lib()
    bt = Batch([0, 0], [30, 7], 2, 64, 16, dtype, seed=4)
    cache = vc.PagedCache(bt.k, bt.v, bt.block_table)
    k0 = bt.k.clone()
    q = torch.empty(0, 4, 64, dtype=dtype, device="cuda")
    scores = torch.rand(2, 2, cache.slots, device="cuda")
    before = scores.clone()
    ws = vc.Workspace(vc.vc_paged_attn_h2o_workspace_bytes(cache, 0, 4))
    vc.vc_paged_append(torch.empty(0, 8 * 64, dtype=dtype, device="cuda"), cache, bt.q_start, bt.ctx,
                       torch.empty_like(q), vc.vc_rope_init(64, 1e4))
    vc.vc_paged_attn(q, cache, bt.q_start, bt.ctx, 0.1, torch.empty_like(q), ws)
    vc.vc_paged_attn_h2o(q, cache, bt.q_start, bt.ctx, 0.1, torch.empty_like(q), scores, ws)
    torch.cuda.synchronize()
    assert torch.equal(scores, before) and int(cache.status) == 0 and vc.vc_poll_status(ws) == 0
    assert torch.equal(torch.nan_to_num(bt.k.float(), nan=3.0), torch.nan_to_num(k0.float(), nan=3.0))


def test_an_eviction_that_keeps_nothing():
    """keep_top = keep_recent = 0 with outputs of no entries: the lengths become
    zero and no page is written."""
    vc = lib()
    bt = Batch([0, 0], [30, 7], 2, 64, 16, BF, seed=4)
    src = vc.PagedCache(bt.k, bt.v, bt.block_table)
    k2 = torch.full((2, 2, 16, 64), 7.0, dtype=BF, device="cuda")
    dst = vc.PagedCache(k2, k2.clone(), torch.tensor([[0], [1]], dtype=torch.int32, device="cuda"))
    i32 = dict(dtype=torch.int32, device="cuda")
    n = torch.full((2,), -5, **i32)
    vc.vc_paged_evict(torch.rand(2, 2, src.slots, device="cuda"), src, torch.tensor(bt.lens, **i32), 0, 0, dst, n,
                      torch.empty(2, 2, 0, **i32), scores_out=torch.empty(2, 2, 0, device="cuda"))
    torch.cuda.synchronize()
    assert n.tolist() == [0, 0] and int(src.status) == int(dst.status) == 0
    assert (dst.k == 7.0).all() and (dst.v == 7.0).all()


def test_mass_under_a_table_too_wide_for_stored_scores():
    """A decode step whose scores, one per table slot, would take 2 GiB."""
    vc = lib()
    lens = [(173 * i) % 700 for i in range(16)]
    bt = Batch([1] * 16, lens, 2, 64, 256, BF, seed=5, width=1 << 12)
    cache = vc.PagedCache(bt.k, bt.v, bt.block_table)
    assert vc.vc_paged_attn_h2o_workspace_bytes(cache, 16, 32) < 1 << 30
    q = bt.randn(16, 32, 64, scale=1.5)
    scores = torch.zeros(16, 2, bt.width * 256, device="cuda")
    out = _call(vc, bt, q, 0.125, scores)
    want, tol, mass, mtol = paged_ref.attn(bt, q, 0.125)
    close(out, want, tol, "out")
    close(scores, mass, mtol, "scores")
    for b in range(16):
        assert (scores[b, :, bt.lens[b]:] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ns,cs", [([1] * 5, [3000, 7, 0, 513, 90]), ([4, 0, 30, 150], [2000, 9, 600, 0])])
def test_scores_change_no_bit_of_the_output(dtype, d, ns, cs):
    """vc_paged_attn_h2o's output is vc_paged_attn's, with the scores stored (few
    rows per sequence) and without."""
    vc = lib()
    bt = Batch(ns, cs, 2, d, 32, dtype, seed=9)
    q = bt.randn(bt.T, 8, d, scale=2.0)
    scores = torch.zeros(bt.B, 2, bt.width * 32, device="cuda")
    assert torch.equal(_call(vc, bt, q, 0.1), _call(vc, bt, q, 0.1, scores))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [3, 40])
def test_more_sequences_than_the_search_keeps(dtype, rows):
    """2100 sequences: the search for a CTA's piece keeps the totals of the
    first 1024 and goes on from there.  Runs of sequences without rows, and long
    ones, around its 32- and 1024-sequence marks; few rows per sequence, whose
    scores are stored, and many."""
    vc = lib()
    B = 2100
    empty = set(range(28, 34)) | set(range(1000, 1030)) | set(range(1500, 1600)) | set(range(2090, 2100))
    ns = [0 if i in empty else i % rows for i in range(B)]
    cs = [(37 * i) % 150 for i in range(B)]
    for b in (27, 34, 64, 999, 1031, 1057, 1700):
        ns[b], cs[b] = 1 + b % 5, 1500 + b
    bt = Batch(ns, cs, 1, 64, 32, dtype, seed=6, head_rows=1, tail_rows=2)
    q = bt.randn(bt.T, 2, 64, scale=1.5)
    scores = torch.zeros(B, 1, bt.width * 32, device="cuda")
    out = _call(vc, bt, q, 0.125, scores)
    assert torch.equal(out, _call(vc, bt, q, 0.125))
    want, tol, mass, mtol = paged_ref.attn(bt, q, 0.125)
    close(out[1:-2], want[1:-2], tol[1:-2], "out")
    assert (out[0] == 7.0).all() and (out[-2:] == 7.0).all()
    close(scores, mass, mtol, "scores")
    for b in range(B):
        assert (scores[b, :, bt.lens[b] if ns[b] else 0:] == 0).all()


@pytest.mark.parametrize("ctx", [2300, 4000, 6000, 9000])
def test_mass_of_many_key_tiles_at_heads_of_128(ctx):
    """Groups of one, two, three and four key tiles of 128 channels."""
    vc = lib()
    bt = Batch([20], [ctx], 8, 128, 64, BF, seed=7)
    q = bt.randn(bt.T, 32, 128, scale=1.5)
    scores = torch.zeros(1, 8, bt.width * 64, device="cuda")
    out = _call(vc, bt, q, 128 ** -0.5, scores)
    want, tol, mass, mtol = paged_ref.attn(bt, q, 128 ** -0.5)
    close(out, want, tol, "out")
    close(scores, mass, mtol, "scores")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ns,cs", [([1] * 6, [300, 0, 2000, 64, 5, 0]), ([30, 0, 7, 600], [100, 50, 900, 3])])
def test_a_table_much_wider_than_its_sequences(dtype, ns, cs):
    """Under a table for 131072 tokens every operator gives what it gives under one
    of the sequences' own width, bit for bit."""
    vc = lib()
    page, d, Hq, Hkv = 32, 64, 4, 2
    rope = vc.vc_rope_init(d, 1e4)
    got = []
    for width in (0, 131072 // page):
        bt = Batch(ns, cs, Hkv, d, page, dtype, seed=8, width=width)
        cache = vc.PagedCache(bt.k, bt.v, bt.block_table)
        qkv = bt.randn(bt.T, (Hq + 2 * Hkv) * d)
        q = torch.empty(bt.T, Hq, d, dtype=dtype, device="cuda")
        vc.vc_paged_append(qkv, cache, bt.q_start, bt.ctx, q, rope)
        scores = torch.zeros(bt.B, Hkv, cache.slots, device="cuda")
        plain = _call(vc, bt, q, 0.125)
        out = _call(vc, bt, q, 0.125, scores)
        assert torch.equal(plain, out)
        want, tol, mass, mtol = paged_ref.attn(bt, q, 0.125)
        close(out, want, tol, "out")
        close(scores, mass, mtol, "scores")
        i32 = dict(dtype=torch.int32, device="cuda")
        n2, kept = torch.zeros(bt.B, **i32), torch.full((bt.B, Hkv, 90), -1, **i32)
        k2 = torch.zeros(3 * bt.B, Hkv, page, d, dtype=dtype, device="cuda")
        dst = vc.PagedCache(k2, k2.clone(), torch.arange(3 * bt.B, **i32).view(bt.B, 3))
        vc.vc_paged_evict(scores, cache, torch.tensor(bt.lens, **i32), 70, 20, dst, n2, kept)
        torch.cuda.synchronize()
        assert int(cache.status) == int(dst.status) == 0
        w = max(bt.lens)
        got.append((q, plain, out, scores[..., :w].clone(), n2, kept, dst.k, dst.v))
        for b in range(bt.B):
            for h in range(Hkv):
                keep = paged_ref.evict(scores[b, h].tolist(), bt.lens[b], 70, 20)
                assert kept[b, h, :len(keep)].tolist() == keep
    for a, b in zip(*got):
        assert torch.equal(a, b)
