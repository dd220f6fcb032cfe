"""Paged-cache operators on the GPU against their fp64 forms (paged_ref.py,
where the tolerances are derived)."""
import math

import pytest
import torch

import paged_ref
from helpers import lib
from paged_ref import Batch, close

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _cache(vc, bt):
    return vc.PagedCache(bt.k, bt.v, bt.block_table)


def _attn(vc, bt, q, scale, mass=False, scores=None, cache=None, ws=None, out=None):
    cache = cache or _cache(vc, bt)
    out = torch.full_like(q, 7.0) if out is None else out
    T, Hq, _ = q.shape
    if mass:
        ws = ws or vc.Workspace(vc.vc_paged_attn_h2o_workspace_bytes(cache, T, Hq))
        vc.vc_paged_attn_h2o(q, cache, bt.q_start, bt.ctx, scale, out, scores, ws)
    else:
        ws = ws or vc.Workspace(vc.vc_paged_attn_workspace_bytes(cache, T, Hq))
        vc.vc_paged_attn(q, cache, bt.q_start, bt.ctx, scale, out, ws)
    assert vc.vc_poll_status(ws) == 0 and int(cache.status) == 0
    return out


def _compare(bt, q, out, scale, what=""):
    want, tol, mass, mtol = paged_ref.attn(bt, q, scale)
    rows = torch.zeros(q.shape[0], dtype=torch.bool)
    for b in range(bt.B):
        rows[bt.start[b]:bt.start[b + 1]] = True
    close(out.cpu()[rows], want[rows], tol[rows], what + " out")
    assert (out.cpu()[~rows] == 7.0).all(), what + ": a row of no sequence was written"
    return mass, mtol


# (chunks, contexts, query heads, kv heads, d, page)
CASES = [
    ([1], [0], 1, 1, 128, 16),                              # one token that sees itself
    ([1], [200], 8, 8, 64, 16),
    ([1, 1, 1], [0, 1, 15], 4, 4, 128, 16),                 # around a page's end
    ([1, 1, 1], [127, 128, 129], 4, 1, 128, 32),            # around a key tile's end
    ([1] * 5, [700, 3, 1500, 64, 2222], 8, 2, 128, 64),     # decode, several parts per unit
    ([5, 0, 1, 17, 0], [300, 50, 0, 129, 7], 8, 2, 128, 16),     # empty chunks
    ([33, 33], [640, 1000], 8, 2, 128, 128),                # 132 rows: just past one tile
    ([64, 63, 65], [0, 100, 255], 4, 2, 128, 64),           # 128, 126, 130 rows
    ([128, 2], [256, 700], 8, 4, 64, 256),                  # 256 rows
    ([129, 300], [1, 0], 2, 1, 128, 32),                    # prompts from the start
    ([70, 9], [333, 411], 14, 2, 128, 16),                  # 7 query heads per kv head
    ([43, 1], [90, 513], 9, 3, 64, 64),                     # 3 per kv head
    ([3, 260], [2000, 1], 40, 1, 64, 32),                   # 40 per kv head
    ([600], [900], 4, 2, 128, 64),                          # a long chunk over many tiles
    ([2], [9000], 16, 2, 128, 64),                          # few rows, a long context
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, dtype):
    vc = lib()
    ns, cs, Hq, Hkv, d, page = CASES[case]
    bt = Batch(ns, cs, Hkv, d, page, dtype, seed=case, head_rows=case % 3, tail_rows=case % 4, width=case % 5)
    q = bt.randn(bt.T, Hq, d, scale=1.5)
    out = _attn(vc, bt, q, d ** -0.5)
    _compare(bt, q, out, d ** -0.5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_mass(case, dtype):
    vc = lib()
    ns, cs, Hq, Hkv, d, page = CASES[case]
    bt = Batch(ns, cs, Hkv, d, page, dtype, seed=100 + case, head_rows=case % 2, tail_rows=case % 3)
    q = bt.randn(bt.T, Hq, d, scale=1.5)
    S = bt.width * page + case % 4                          # an odd stride is fine
    before = torch.rand(bt.B, Hkv, S, device="cuda")
    scores = before.clone()
    out = _attn(vc, bt, q, d ** -0.5, True, scores)
    mass, mtol = _compare(bt, q, out, d ** -0.5)
    w = bt.width * page
    want = before.cpu().double()[..., :w] + mass
    close(scores[..., :w], want, mtol + paged_ref.U_F32 * want, "scores")
    for b in range(bt.B):
        untouched = bt.lens[b] if bt.ns[b] else 0
        assert torch.equal(scores[b, :, untouched:], before[b, :, untouched:])


# row tiles of a batch in groups of one, two, three and four key tiles; more
# sequences than a warp has lanes
MASS = [([20], [c], 32, 8) for c in (2300, 4000, 6000, 9000)] + [
    ([20 + i % 7 for i in range(40)], [(37 * i) % 500 for i in range(40)], 4, 2),
    ([30 * (i % 3) for i in range(70)], [(53 * i) % 300 for i in range(70)], 8, 8)]


@pytest.mark.parametrize("case", range(len(MASS)))
def test_mass_of_many_key_tiles_and_sequences(case):
    vc = lib()
    ns, cs, Hq, Hkv = MASS[case]
    bt = Batch(ns, cs, Hkv, 64, 64, BF, seed=200 + case)
    q = bt.randn(bt.T, Hq, 64, scale=1.5)
    scores = torch.zeros(bt.B, Hkv, bt.width * 64, device="cuda")
    out = _attn(vc, bt, q, 0.125, True, scores)
    mass, mtol = _compare(bt, q, out, 0.125)
    close(scores, mass, mtol, "scores")
    for b in range(bt.B):
        assert (scores[b, :, bt.lens[b] if bt.ns[b] else 0:] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale,peak", [(0.0, 1.0), (0.3, 6.0), (1.0, 4.0)])
def test_attention_scales(dtype, scale, peak):
    """A scale of zero (the mean of what is visible) and peaked weights: the
    running maximum moves by far more than a few powers of two, up and down
    the context."""
    vc = lib()
    bt = Batch([3, 40], [1500, 700], 2, 128, 64, dtype, seed=9)
    q = bt.randn(bt.T, 8, 128, scale=peak)
    ramp = torch.linspace(0.1, 3, bt.n_pages, device="cuda").view(-1, 1, 1, 1)
    bt.k = (bt.k * ramp).to(dtype)
    out = _attn(vc, bt, q, scale)
    _compare(bt, q, out, scale)


def test_attention_repeats_and_rides_in_a_graph():
    """Two calls give the same bits; so do a captured call replayed twice over
    new lengths and queries, on a side stream with the eager call's workspace."""
    vc = lib()
    bt = Batch([5, 1, 90], [1300, 40, 200], 2, 128, 32, BF, seed=3)
    cache = _cache(vc, bt)
    q = bt.randn(bt.T, 8, 128)
    n = vc.vc_paged_attn_h2o_workspace_bytes(cache, bt.T, 8)
    ws = vc.Workspace(n)
    sc = [torch.zeros(bt.B, 2, cache.slots, device="cuda") for _ in range(2)]
    a = _attn(vc, bt, q, 0.1, True, sc[0], cache, ws)
    b = _attn(vc, bt, q, 0.1, True, sc[1], cache, ws)
    assert torch.equal(a, b) and torch.equal(*sc)
    out, scores = torch.zeros_like(q), torch.zeros_like(sc[0])
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side, capture_error_mode="thread_local"):
        vc.vc_paged_attn_h2o(q, cache, bt.q_start, bt.ctx, 0.1, out, scores, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a) and torch.equal(scores, sc[0])
    q.copy_(bt.randn(*q.shape))
    bt.q_start.copy_(torch.tensor([0, 3, 3, 80], dtype=torch.int32))
    bt.ctx.copy_(torch.tensor([1000, 41, 199], dtype=torch.int32))
    scores.zero_(), out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    bt.start, bt.ns, bt.cs = [0, 3, 3, 80], [3, 0, 77], [1000, 41, 199]
    bt.lens = [1003, 41, 276]
    mass, mtol = _compare(bt, q, out, 0.1, "replayed")
    close(scores, mass, mtol, "replayed scores")
    assert vc.vc_poll_status(ws) == 0


def test_two_graphs_share_a_workspace():
    """Nothing of a call stays in the workspace: two captured batches of other
    shapes replay in turn on one."""
    vc = lib()
    jobs, need = [], 0
    for ns, cs, Hq in (([1, 1, 1], [3000, 77, 900], 8), ([60, 200], [500, 40], 4)):
        bt = Batch(ns, cs, 2, 128, 32, BF, seed=len(jobs))
        cache = _cache(vc, bt)
        q = bt.randn(bt.T, Hq, 128)
        need = max(need, vc.vc_paged_attn_h2o_workspace_bytes(cache, bt.T, Hq))
        jobs.append((bt, cache, q, torch.empty_like(q), torch.zeros(bt.B, 2, cache.slots, device="cuda")))
    ws = vc.Workspace(need)
    graphs = []
    for bt, cache, q, out, scores in jobs:
        _attn(vc, bt, q, 0.1, True, scores.clone(), cache, ws)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], capture_error_mode="thread_local"):
            vc.vc_paged_attn_h2o(q, cache, bt.q_start, bt.ctx, 0.1, out, scores, ws)
    for _ in range(2):
        for (bt, cache, q, out, scores), g in zip(jobs, graphs):
            out.fill_(7.0), scores.zero_()
            g.replay()
    torch.cuda.synchronize()
    for bt, cache, q, out, scores in jobs:
        mass, mtol = _compare(bt, q, out, 0.1)
        close(scores, mass, mtol, "scores")
    assert vc.vc_poll_status(ws) == 0


def test_sixteen_byte_alignment_is_enough():
    vc = lib()
    bt = Batch([9, 2], [300, 77], 2, 64, 16, BF, seed=6)

    def shifted(t):
        x = torch.zeros(t.numel() + 8, dtype=t.dtype, device="cuda")[8:].view(t.shape)
        return x.copy_(t)
    q = shifted(bt.randn(bt.T, 4, 64))
    bt.k, bt.v = shifted(bt.k), shifted(bt.v)
    scores = torch.zeros(bt.B, 2, bt.width * 16, device="cuda")
    out = _attn(vc, bt, q, 0.2, True, scores, out=shifted(torch.full_like(q, 7.0)))
    mass, mtol = _compare(bt, q, out, 0.2)
    close(scores, mass, mtol, "scores")
    bt = Batch([9, 2], [300, 77], 2, 64, 16, BF, seed=6)
    qkv, qo = shifted(bt.randn(bt.T, 8 * 64)), shifted(torch.zeros(bt.T, 4, 64, dtype=BF, device="cuda"))
    vc.vc_paged_append(qkv, _cache(vc, bt), bt.q_start, bt.ctx, qo, vc.vc_rope_init(64, 1e4))
    y, _, tol = paged_ref.append(bt, qkv, 4, [1e4 ** (-j / 32) for j in range(32)],
                                 [c + i for n, c in zip(bt.ns, bt.cs) for i in range(n)], None, None, 0.0)
    close(qo, y[:, :4], tol[:, :4], "q")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pools_past_two_to_the_31_elements(dtype):
    """Pages whose elements lie past 2^31: every operator gives what it gives
    on a small pool, bit for bit."""
    vc = lib()
    Hkv, page, d = 8, 256, 128
    small = Batch([3, 1], [600, 255], Hkv, d, page, dtype, seed=7, width=4)
    n_big = 2 ** 31 // (Hkv * page * d) + 20
    shift = n_big - small.n_pages
    big_k = torch.empty(n_big, Hkv, page, d, dtype=dtype, device="cuda")
    big_v = torch.empty_like(big_k)
    big_k[shift:], big_v[shift:] = small.k, small.v
    table = torch.where(small.block_table >= 0, small.block_table + shift, small.block_table)
    q = small.randn(small.T, 16, d)
    qkv = small.randn(small.T, (16 + 2 * Hkv) * d)
    rope = vc.vc_rope_init(d, 1e4)
    got = []
    for k, v, tab in ((small.k, small.v, small.block_table), (big_k, big_v, table)):
        cache = vc.PagedCache(k, v, tab)
        ws = vc.Workspace(vc.vc_paged_attn_h2o_workspace_bytes(cache, small.T, 16))
        out, qo = torch.empty_like(q), torch.empty_like(q)
        scores = torch.zeros(2, Hkv, cache.slots, device="cuda")
        vc.vc_paged_append(qkv, cache, small.q_start, small.ctx, qo, rope)
        vc.vc_paged_attn_h2o(q, cache, small.q_start, small.ctx, 0.1, out, scores, ws)
        # eviction into two pages that no table names
        spare = [p for p in range(small.n_pages) if not (small.block_table == p).any()][:2]
        off = 0 if k is small.k else shift
        dst = vc.PagedCache(k, v, torch.tensor([[spare[0] + off], [spare[1] + off]], dtype=torch.int32, device="cuda"))
        n, kept = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, Hkv, 90, dtype=torch.int32,
                                                                                device="cuda")
        vc.vc_paged_evict(scores, cache, (small.ctx + torch.tensor([3, 1], device="cuda")).int(), 70, 20, dst, n, kept)
        torch.cuda.synchronize()
        assert int(cache.status) == int(dst.status) == 0 and vc.vc_poll_status(ws) == 0
        rows = k[dst.block_table[:, 0].long(), :, :90]
        got.append((out, qo, scores, n, kept, rows.clone(), v[dst.block_table[:, 0].long(), :, :90].clone()))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_two_calls_at_once_on_two_streams():
    vc = lib()
    jobs = []
    for i in range(2):
        bt = Batch([7, 1], [900 + i, 2000], 2, 128, 64, BF, seed=20 + i)
        cache = _cache(vc, bt)
        q = bt.randn(bt.T, 8, 128)
        ws = vc.Workspace(vc.vc_paged_attn_workspace_bytes(cache, bt.T, 8))
        jobs.append((bt, cache, q, torch.full_like(q, 7.0), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for bt, cache, q, out, ws, st in jobs:
            vc.vc_paged_attn(q, cache, bt.q_start, bt.ctx, 0.1, out, ws, stream=st)
    torch.cuda.synchronize()
    for bt, cache, q, out, ws, st in jobs:
        _compare(bt, q, out, 0.1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_does_not_fit_is_reported_and_left_alone(dtype):
    """Bad page numbers and lengths: the status word says so, nothing outside
    the pool is touched and the other sequences' results stand."""
    vc = lib()
    for mass in (False, True):
        bt = Batch([4, 6, 2, 3], [100, 333, 40, 64], 2, 128, 32, dtype, seed=5)
        q = bt.randn(bt.T, 4, 128)
        cache = _cache(vc, bt)
        ws = vc.Workspace(vc.vc_paged_attn_h2o_workspace_bytes(cache, bt.T, 4))
        scores = torch.zeros(bt.B, 2, cache.slots, device="cuda")
        bt.block_table[1, 3], bt.block_table[1, 5] = bt.n_pages, -7
        bt.ctx[2] = cache.slots                              # more than the table holds
        out = torch.full_like(q, 7.0)

        def call():
            if mass:
                vc.vc_paged_attn_h2o(q, cache, bt.q_start, bt.ctx, 0.1, out, scores, ws)
            else:
                vc.vc_paged_attn(q, cache, bt.q_start, bt.ctx, 0.1, out, ws)
            torch.cuda.synchronize()
        call()
        assert int(cache.status) == vc.VC_PAGED_BAD_PAGE | vc.VC_PAGED_BAD_LENGTH and vc.vc_poll_status(ws) == 0
        want, tol, m, mt = paged_ref.attn(bt, q, 0.1)
        for b in (0, 3):
            r = slice(bt.start[b], bt.start[b + 1])
            close(out[r], want[r], tol[r], f"sequence {b}")
            if mass:
                close(scores[b], m[b], mt[b], f"scores {b}")
        assert (out[bt.start[2]:bt.start[3]] == 7.0).all() and (scores[2] == 0).all()
        bt.q_start[4] = bt.T + 1                             # the last sequence leaves the packed rows
        cache.status.zero_()
        out.fill_(7.0)
        call()
        assert int(cache.status) & vc.VC_PAGED_BAD_LENGTH and (out[bt.start[3]:] == 7.0).all()
        close(out[:4], want[:4], tol[:4], "sequence 0")


APPEND = [
    ([1], [0], 1, 1, 64, 16, 64, False), ([1] * 16, [500] * 16, 32, 8, 128, 64, 128, True),
    ([3, 0, 40, 1], [15, 9, 200, 0], 6, 2, 128, 16, 64, True), ([700, 1, 33], [3, 0, 31], 4, 4, 64, 32, 32, False),
    ([2, 5], [255, 256], 7, 1, 128, 256, 16, True), ([1] * 70, list(range(70)), 3, 3, 64, 128, 64, True),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case, dtype):
    vc = lib()
    ns, cs, Hq, Hkv, d, page, rot, norm = APPEND[case]
    bt = Batch(ns, cs, Hkv, d, page, dtype, seed=case, head_rows=case % 2, tail_rows=case % 3)
    T = bt.T
    qkv = bt.randn(T, (Hq + 2 * Hkv) * d, scale=2.0)
    gains = [bt.randn(d, scale=0.3) + 1 for _ in range(2)] if norm else [None, None]
    k0, v0 = bt.k.clone(), bt.v.clone()
    cache = _cache(vc, bt)
    q_out = torch.full((T, Hq, d), 7.0, dtype=dtype, device="cuda")
    pos = None
    if case % 2:
        pos = torch.randint(-50000, 1 << 20, (T,), generator=bt.g).int().cuda()
        if case == 3:
            pos[0], pos[1] = 2 ** 31 - 1, -2 ** 31
    inv = [1e4 ** (-2.0 * j / rot) for j in range(rot // 2)]
    vc.vc_paged_append(qkv, cache, bt.q_start, bt.ctx, q_out, vc.vc_rope_init(rot, 1e4), pos, *gains, eps=1e-5)
    torch.cuda.synchronize()
    assert int(cache.status) == 0
    place = [-1] * T                                        # (b, slot) of every row
    for b in range(bt.B):
        for i in range(ns[b]):
            place[bt.start[b] + i] = (b, cs[b] + i)
    position = pos.cpu().tolist() if pos is not None else [p[1] if p != -1 else 0 for p in place]
    y, v, tol = paged_ref.append(bt, qkv, Hq, inv, position, *gains, 1e-5)
    rows = torch.tensor([p != -1 for p in place])
    close(q_out.cpu()[rows], y[rows, :Hq], tol[rows, :Hq], "q")
    assert (q_out.cpu()[~rows] == 7.0).all()
    k, vv = bt.k.cpu().double(), bt.v.cpu().double()
    touched = torch.zeros(bt.n_pages, page, dtype=torch.bool)
    for r, p in enumerate(place):
        if p == -1:
            continue
        pg, o = bt.table[p[0]][p[1] // page], p[1] % page
        touched[pg, o] = True
        close(k[pg, :, o], y[r, Hq:], tol[r, Hq:], f"k of row {r}")
        assert torch.equal(vv[pg, :, o], v[r])
    for new, old in ((bt.k, k0), (bt.v, v0)):
        keep = ~touched.cuda()[:, None, :, None].expand_as(old)
        assert torch.equal(torch.nan_to_num(new[keep].float(), nan=5.0), torch.nan_to_num(old[keep].float(), nan=5.0))


def test_append_reports_what_does_not_fit():
    vc = lib()
    bt = Batch([2, 2, 2], [10, 20, 30], 1, 64, 16, BF, seed=1)
    k0 = bt.k.clone()
    cache = _cache(vc, bt)
    qkv = bt.randn(6, 3 * 64)
    q = torch.zeros(6, 1, 64, dtype=BF, device="cuda")
    bt.block_table[0, 0] = bt.n_pages + 3
    bt.ctx[1] = cache.slots - 1
    vc.vc_paged_append(qkv, cache, bt.q_start, bt.ctx, q, vc.vc_rope_init(64, 1e4))
    torch.cuda.synchronize()
    assert int(cache.status) == vc.VC_PAGED_BAD_PAGE | vc.VC_PAGED_BAD_LENGTH
    assert (q[2:4] == 0).all() and (q[4:] != 0).any()
    changed = [p for p in range(bt.n_pages)
               if not torch.equal(torch.nan_to_num(bt.k[p].float(), nan=3.0), torch.nan_to_num(k0[p].float(), nan=3.0))]
    assert set(changed) <= {bt.table[2][1], bt.table[2][2] if bt.width > 2 else -1}


def _evict(vc, bt, scores, top, recent, page2, with_scores=True, lens=None, pool=None):
    lens = lens or bt.lens
    cap = min(top + recent, bt.width * bt.page)
    n = [min(top, max(L - recent, 0)) + min(recent, L) for L in lens]
    blocks = [-(-m // page2) for m in n]
    width = max(-(-cap // page2), 1)
    n2 = sum(blocks) + 1
    g = torch.Generator().manual_seed(8)
    order = torch.randperm(n2, generator=g).tolist()
    table = torch.full((bt.B, width), -1, dtype=torch.int32)
    for b in range(bt.B):
        for i in range(blocks[b]):
            table[b, i] = order.pop()
    k2 = torch.full((n2, bt.Hkv, page2, bt.d), 7.0, dtype=bt.dtype, device="cuda")
    v2 = k2.clone()
    src, dst = _cache(vc, bt), vc.PagedCache(k2, v2, table.cuda())
    out_len = torch.full((bt.B,), -5, dtype=torch.int32, device="cuda")
    kept = torch.full((bt.B, bt.Hkv, max(cap, 1)), -5, dtype=torch.int32, device="cuda")
    sc2 = torch.full((bt.B, bt.Hkv, max(cap, 1)), -5.0, device="cuda") if with_scores else None
    vc.vc_paged_evict(scores, src, torch.tensor(lens, dtype=torch.int32, device="cuda"), top, recent, dst, out_len,
                      kept, scores_out=sc2)
    torch.cuda.synchronize()
    assert int(src.status) == 0 and int(dst.status) == 0
    assert out_len.tolist() == n
    want_k, want_v = torch.full_like(k2, 7.0), torch.full_like(k2, 7.0)
    host = scores.cpu()
    kc, sc = kept.cpu(), sc2.cpu() if with_scores else None
    for b in range(bt.B):
        for h in range(bt.Hkv):
            keep = paged_ref.evict(host[b, h].tolist(), lens[b], top, recent)
            assert kc[b, h, :n[b]].tolist() == keep, (b, h)
            assert (kc[b, h, n[b]:] == -5).all()
            if with_scores:
                a = sc[b, h, :n[b]]
                e = host[b, h, keep] if keep else a
                assert torch.equal(torch.nan_to_num(a, nan=99.0), torch.nan_to_num(e, nan=99.0))
                assert (sc[b, h, n[b]:] == -5).all()
            idx = torch.tensor(keep, dtype=torch.long)
            pg = torch.tensor(bt.table[b])[idx // bt.page].cuda() if keep else None
            for i0 in range(0, n[b], page2):
                i1 = min(n[b], i0 + page2)
                p = int(table[b, i0 // page2])
                o = (idx[i0:i1] % bt.page).cuda()
                want_k[p, h, :i1 - i0] = bt.k[pg[i0:i1].long(), h, o]
                want_v[p, h, :i1 - i0] = bt.v[pg[i0:i1].long(), h, o]
    assert torch.equal(k2, want_k) and torch.equal(v2, want_v)
    return kept, out_len, dst, sc2


EVICT = [
    ([1], 1, 1, 16, 64, 16), ([5, 0, 17], 3, 2, 16, 64, 16), ([40, 700, 3], 20, 10, 32, 128, 16),
    ([700, 699], 0, 64, 16, 128, 64), ([700, 30], 100, 0, 64, 64, 32), ([64, 9], 500, 500, 16, 64, 16),
    ([5000, 4097, 4096], 900, 65, 64, 64, 64), ([9000], 8990, 5, 256, 128, 128), ([300], 0, 0, 16, 64, 16),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(EVICT)))
def test_evict(case, dtype):
    vc = lib()
    lens, top, recent, page, d, page2 = EVICT[case]
    bt = Batch([0] * len(lens), lens, 2, d, page, dtype, seed=case, width=case % 3)
    g = torch.Generator().manual_seed(case)
    S = bt.width * page + case % 2
    sc = torch.randn(bt.B, 2, S, generator=g)
    if case % 3 == 1:                                       # ties everywhere, signed zeros among them
        sc = (sc * 2).round() / 2 * torch.where(torch.rand(sc.shape, generator=g) < 0.5, 1.0, -1.0)
    if case % 3 == 2:
        r = torch.rand(sc.shape, generator=g)
        sc[r < 0.2], sc[(r > 0.2) & (r < 0.3)], sc[r > 0.9] = math.nan, -math.inf, math.inf
        sc[(r > 0.3) & (r < 0.35)], sc[(r > 0.35) & (r < 0.4)] = -0.0, 1e-42
    _evict(vc, bt, sc.cuda(), top, recent, page2, with_scores=case != 4)


def test_evict_all_equal_scores():
    vc = lib()
    bt = Batch([0, 0], [3000, 77], 2, 64, 16, BF, seed=2)
    _evict(vc, bt, torch.zeros(2, 2, bt.width * 16, device="cuda"), 100, 20, 16)
    _evict(vc, bt, torch.full((2, 2, bt.width * 16), math.nan, device="cuda"), 100, 20, 32)


@pytest.mark.parametrize("lens,top,recent,slots", [
    ([16384, 16000], 700, 65, 16384), ([16385, 5], 700, 65, 16400), ([700, 0, 64], 20, 10, 16400),
    ([5000, 4097, 4096], 900, 65, 40000), ([140000, 3], 5000, 100, 140000), ([20000], 19990, 5, 20000)])
def test_evict_where_the_selection_changes_form(lens, top, recent, slots):
    """One CTA per unit up to 16384 slots of the table, a cluster beyond, which
    keeps up to 131072 scores on chip: ties, signed zeros and NaN on each side."""
    vc = lib()
    page = 16
    bt = Batch([0] * len(lens), lens, 2, 64, page, BF, seed=slots % 97, width=-(-slots // page))
    assert slots <= bt.width * page < slots + page
    g = torch.Generator().manual_seed(slots % 89)
    sc = (torch.randn(bt.B, 2, bt.width * page, generator=g) * 4).round() / 4
    sc = sc * torch.where(torch.rand(sc.shape, generator=g) < 0.5, 1.0, -1.0)
    sc[torch.rand(sc.shape, generator=g) < 0.02] = math.nan
    _evict(vc, bt, sc.cuda(), top, recent, 32)


def test_evict_reports_what_does_not_fit():
    vc = lib()
    bt = Batch([0] * 3, [100, 60, 50], 2, 64, 16, BF, seed=4)
    src = _cache(vc, bt)
    k2 = torch.zeros(9, 2, 16, 64, dtype=BF, device="cuda")
    dst = vc.PagedCache(k2, k2.clone(), torch.tensor([[0, 1], [99, -1], [2, 3]], dtype=torch.int32, device="cuda"))
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    kept = torch.zeros(3, 2, 20, dtype=torch.int32, device="cuda")
    scores = torch.rand(3, 2, src.slots, device="cuda")
    scores[0, :, 32:36] = 2.0                               # kept, on the page whose number is bad
    bt.block_table[0, 2] = -9
    vc.vc_paged_evict(scores, src, torch.tensor([100, 60, src.slots + 1], dtype=torch.int32, device="cuda"), 15, 5,
                      dst, n, kept)
    torch.cuda.synchronize()
    assert int(src.status) == vc.VC_PAGED_BAD_PAGE | vc.VC_PAGED_BAD_LENGTH and int(dst.status) == vc.VC_PAGED_BAD_PAGE
    assert n.tolist() == [20, 20, 0] and (k2[2:] == 0).all()


def test_a_server_run():
    """The operators together, as a server calls them: prompts read in chunks
    (append, attention with scores), an eviction into fresh pages of the same
    pool, then decoding on the shortened cache at the old positions.  Against
    the fp64 forms at every step."""
    vc = lib()
    B, Hq, Hkv, d, page, n_pages = 2, 8, 2, 128, 16, 64
    g = torch.Generator().manual_seed(0)
    k = torch.full((n_pages, Hkv, page, d), float("nan"), dtype=BF, device="cuda")
    v = k.clone()
    free = torch.randperm(n_pages, generator=g).tolist()
    rope = vc.vc_rope_init(d, 1e4)
    inv = [1e4 ** (-2.0 * j / d) for j in range(d // 2)]
    gains = [(torch.randn(d, generator=g) * 0.2 + 1).to(BF).cuda() for _ in range(2)]
    width, lens, seen = 12, [0, 0], [0, 0]
    table = torch.full((B, width), -1, dtype=torch.int32)
    scores = torch.zeros(B, Hkv, width * page, device="cuda")
    scale = d ** -0.5

    def step(ns):
        bt = Batch.__new__(Batch)
        bt.ns, bt.cs, bt.lens, bt.B = ns, list(lens), [a + b for a, b in zip(lens, ns)], B
        for b in range(B):
            for i in range(-(-bt.lens[b] // page)):
                if int(table[b, i]) < 0:
                    table[b, i] = free.pop()
        bt.Hkv, bt.d, bt.page, bt.width, bt.dtype, bt.k, bt.v = Hkv, d, page, width, BF, k, v
        bt.table, bt.block_table = table.tolist(), table.cuda()
        bt.start = [0, ns[0], sum(ns)]
        T = sum(ns)
        i32 = dict(dtype=torch.int32, device="cuda")
        q_start, ctx = torch.tensor(bt.start, **i32), torch.tensor(bt.cs, **i32)
        pos = [seen[b] + i for b in range(B) for i in range(ns[b])]
        qkv = torch.randn(T, (Hq + 2 * Hkv) * d, generator=g).to(BF).cuda()
        cache = vc.PagedCache(k, v, bt.block_table)
        q, out = torch.empty(T, Hq, d, dtype=BF, device="cuda"), torch.empty(T, Hq, d, dtype=BF, device="cuda")
        ws = vc.Workspace(vc.vc_paged_attn_h2o_workspace_bytes(cache, T, Hq))
        vc.vc_paged_append(qkv, cache, q_start, ctx, q, rope, torch.tensor(pos, **i32), *gains)
        before = scores.clone()
        vc.vc_paged_attn_h2o(q, cache, q_start, ctx, scale, out, scores, ws)
        torch.cuda.synchronize()
        assert vc.vc_poll_status(ws) == 0 and int(cache.status) == 0
        y, vals, tol = paged_ref.append(bt, qkv, Hq, inv, pos, *gains, 1e-6)
        close(q, y[:, :Hq], tol[:, :Hq], "q")
        for b in range(B):
            r = slice(bt.start[b], bt.start[b + 1])
            for h in range(Hkv):
                close(bt.rows(k, b, h)[lens[b]:], y[r, Hq + h], tol[r, Hq + h], "k")
                assert torch.equal(bt.rows(v, b, h)[lens[b]:], vals[r, h])
        want, tol, mass, mtol = paged_ref.attn(bt, q, scale)
        close(out, want, tol, "out")
        total = before.cpu().double() + mass
        close(scores, total, mtol + paged_ref.U_F32 * total, "scores")
        for b in range(B):
            lens[b] += ns[b]
            seen[b] += ns[b]
        return bt

    step([40, 90])
    step([30, 1])
    bt = step([1, 1])
    # evict to 20 + 8 tokens, into pages of the same pool
    new = torch.full((B, width), -1, dtype=torch.int32)
    for b in range(B):
        for i in range(2):
            new[b, i] = free.pop()
    src, dst = vc.PagedCache(k, v, bt.block_table), vc.PagedCache(k, v, new.cuda())
    i32 = dict(dtype=torch.int32, device="cuda")
    n, kept = torch.zeros(B, **i32), torch.zeros(B, Hkv, 28, **i32)
    scores2 = torch.zeros_like(scores)
    old = [[(bt.rows(k, b, h), bt.rows(v, b, h)) for h in range(Hkv)] for b in range(B)]
    vc.vc_paged_evict(scores, src, torch.tensor(lens, **i32), 20, 8, dst, n, kept, scores_out=scores2)
    torch.cuda.synchronize()
    assert n.tolist() == [28, 28] and int(src.status) == int(dst.status) == 0
    for b in range(B):
        for h in range(Hkv):
            assert kept[b, h].tolist() == paged_ref.evict(scores[b, h].tolist(), lens[b], 20, 8)
    free.extend(p for p in table.flatten().tolist() if p >= 0)
    table, lens[:] = new, [28, 28]
    scores.copy_(scores2)
    bt.table, bt.lens = table.tolist(), [28, 28]
    for b in range(B):
        for h in range(Hkv):
            idx = kept[b, h].long().cpu()
            assert torch.equal(bt.rows(k, b, h), old[b][h][0][idx]) and torch.equal(bt.rows(v, b, h), old[b][h][1][idx])
    step([1, 1])
    step([5, 33])
