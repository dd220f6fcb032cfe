"""Attention over shared prefixes on the GPU against the plain form of each
sequence by itself (paged_ref.py, where the tolerances are derived)."""
import pytest
import torch

import paged_ref
from helpers import lib
from paged8_ref import Batch8
from paged_ref import close

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


class Shared:
    """A batch whose groups (first sequences, prefix lengths) share the whole
    pages of their prefix; `apart`: the other sequences' table entries for those
    blocks name no page."""

    def __init__(self, bt, first, prefix, bits, apart=False):
        self.bt, self.bits = bt, bits
        self.first, self.prefix = list(first) + [bt.B], list(prefix)
        i32 = dict(dtype=torch.int32, device=bt.device)
        table = [list(r) for r in bt.table]
        for g, n in enumerate(self.prefix):
            for b in range(self.first[g] + 1, self.first[g + 1]):
                m = n // bt.page
                bt.table[b][:m] = bt.table[self.first[g]][:m]
                table[b][:m] = [-1] * m if apart else bt.table[b][:m]
        self.block_table = torch.tensor(table, **i32)
        self.seq_start, self.len = torch.tensor(self.first, **i32), torch.tensor(self.prefix, **i32)

    def cache(self, vc):
        bt = self.bt
        return bt.cache8(vc, self.block_table) if self.bits == 8 else vc.PagedCache(bt.k, bt.v, self.block_table)


def _call(vc, sh, q, scale, cache=None, ws=None, out=None, stream=None):
    bt = sh.bt
    cache = cache or sh.cache(vc)
    out = torch.full_like(q, 7.0) if out is None else out
    T, Hq, _ = q.shape
    call, size = ((vc.vc_paged8_attn_shared, vc.vc_paged8_attn_shared_workspace_bytes) if sh.bits == 8 else
                  (vc.vc_paged_attn_shared, vc.vc_paged_attn_shared_workspace_bytes))
    ws = ws or vc.Workspace(size(cache, len(sh.prefix), T, Hq))
    call(q, cache, sh.seq_start, sh.len, bt.q_start, bt.ctx, scale, out, ws, stream=stream)
    return out, cache, ws


def _compare(bt, q, out, scale):
    """The tolerance of paged_ref.attn; the join of the halves adds some ten
    roundings of fp32 and two logarithms' and exponentials' errors to a weight, the
    (L + 16) u of its sums covers them from L = 16 on."""
    want, tol, _, _ = paged_ref.attn(bt, q, scale)
    tol = tol + 32 * paged_ref.U_F32 * torch.nan_to_num(want).abs().amax()
    rows = torch.zeros(q.shape[0], dtype=torch.bool)
    for b in range(bt.B):
        rows[bt.start[b]:bt.start[b + 1]] = True
    close(out.cpu()[rows], want[rows], tol[rows], "out")
    assert (out.cpu()[~rows] == 7.0).all(), "a row of no sequence was written"


CASES = [  # chunks, own contexts, groups' first sequences, prefixes, Hq, Hkv, d, page
    ([1, 1], [0, 5], [0], [16], 1, 1, 128, 16),              # one page, nothing after it
    ([1] * 4, [40, 0, 17, 3], [0], [600], 8, 8, 64, 16),     # 600 = 37 pages and 8 tokens
    ([1] * 8, [7 * i for i in range(8)], [0], [1000], 16, 2, 128, 64),
    ([3, 0, 20, 1, 5], [1, 9, 70, 0, 300], [0, 2], [130, 700], 8, 2, 128, 32),    # an empty chunk, two groups
    ([2, 1, 1, 4], [300, 2, 2, 9], [1], [200], 4, 1, 64, 64),      # a sequence before the groups
    ([17] * 6, [50 * i for i in range(6)], [0, 3, 4], [900, 400, 300], 14, 2, 128, 16),   # a group of one
    ([1] * 40, [3 * i for i in range(40)], list(range(0, 40, 2)), [100 + 8 * i for i in range(20)], 4, 2, 64, 32),
    ([1] * 5, [10] * 5, [0], [15], 4, 2, 128, 16),           # a prefix of less than a page
    ([100, 140], [3, 90], [0], [512], 4, 2, 128, 256),
    ([300, 1], [0, 0], [0], [256], 2, 1, 64, 128),
    ([1] * 64, [i % 5 for i in range(64)], [0], [3000], 8, 1, 128, 64),           # 512 rows in the prefix
    ([1, 1, 1], [20, 30, 40], [], [], 4, 2, 128, 64)]        # no groups


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_shared_prefix(case, dtype, bits):
    vc = lib()
    ns, own, first, prefix, Hq, Hkv, d, page = CASES[case]
    cs = list(own)
    for g, n in enumerate(prefix):
        for b in range(first[g], (first + [len(ns)])[g + 1]):
            cs[b] += n
    bt = Batch8(ns, cs, Hkv, d, page, dtype, seed=case, head_rows=case % 3, tail_rows=case % 2)
    sh = Shared(bt, first, prefix, bits, apart=case % 2 == 1)
    q = bt.randn(bt.T, Hq, d, scale=1.5)
    out, cache, ws = _call(vc, sh, q, d ** -0.5)
    assert vc.vc_poll_status(ws) == 0 and int(cache.status) == 0
    _compare(bt, q, out, d ** -0.5)


def _case(ns, own, first, prefix, Hq, Hkv, d, page, dtype, bits, seed=0, **kw):
    cs = list(own)
    for g, n in enumerate(prefix):
        for b in range(first[g], (first + [len(ns)])[g + 1]):
            cs[b] += n
    bt = Batch8(ns, cs, Hkv, d, page, dtype, seed=seed, **kw)
    return bt, Shared(bt, first, prefix, bits), bt.randn(bt.T, Hq, d, scale=1.5)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ns,own,first,prefix,Hq,Hkv,d,page", [
    ([1] * 3, [5, 0, 90], [0], [9000], 8, 2, 128, 64),       # 12 rows, many parts of each
    ([1, 2, 2], [0, 300, 7], [0], [5000], 12, 2, 64, 16),    # 30 rows
    ([1] * 20, [11 * i for i in range(20)], [0, 10, 12, 14, 16], [1100, 40, 700, 16, 300], 8, 2, 128, 32),    # one group of 40
    ([1] * 20, [3000] + [2] * 19, [0], [2000], 8, 2, 128, 64),     # 80 rows; an own context of many parts
    ([1] * 5, [700, 1, 2, 3, 4], [], [], 8, 2, 64, 32)])     # no group
def test_groups_of_few_rows(ns, own, first, prefix, Hq, Hkv, d, page, dtype, bits):
    vc = lib()
    bt, sh, q = _case(ns, own, first, prefix, Hq, Hkv, d, page, dtype, bits, seed=7)
    out, cache, ws = _call(vc, sh, q, d ** -0.5)
    assert vc.vc_poll_status(ws) == 0 and int(cache.status) == 0
    _compare(bt, q, out, d ** -0.5)
    assert torch.equal(out, _call(vc, sh, q, d ** -0.5, cache, ws)[0])


FORMS = [(dt, bits, ns) for dt in (BF, F32) for bits in (16, 8) for ns in ([1] * 6, [17, 3, 30, 9, 1, 20])]


@pytest.mark.parametrize("dtype,bits,ns", FORMS)
def test_repeats_and_rides_in_a_graph(dtype, bits, ns):
    """The same bits twice and replayed; a replay over other lengths, groups and
    queries gives those results."""
    vc = lib()
    bt, sh, q = _case(ns, [5, 0, 70, 200, 9, 31], [0, 3], [700, 260], 8, 2, 128, 32, dtype, bits)
    a, cache, ws = _call(vc, sh, q, 0.1)
    _compare(bt, q, a, 0.1)
    assert torch.equal(a, _call(vc, sh, q, 0.1, cache, ws)[0])
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream(), capture_error_mode="thread_local"):
        _call(vc, sh, q, 0.1, cache, ws, out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a)
    q.copy_(bt.randn(*q.shape))
    sh.seq_start.copy_(torch.tensor([0, 4, 6], dtype=torch.int32))      # sequence 3's own table from now on
    sh.len.copy_(torch.tensor([200, 250], dtype=torch.int32))
    bt.ctx.copy_(torch.tensor([650, 690, 702, 300, 255, 256], dtype=torch.int32))
    bt.cs = bt.ctx.tolist()
    bt.lens = [c + n for c, n in zip(bt.cs, ns)]
    # (the first 192 slots of sequence 3 are to be those of sequence 0: six pages)
    bt.table[3][:6] = bt.table[0][:6]
    sh.block_table[3, :6] = sh.block_table[0, :6]
    out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    _compare(bt, q, out, 0.1)
    assert vc.vc_poll_status(ws) == 0 and int(cache.status) == 0


def test_graphs_share_a_workspace_and_calls_run_at_once():
    vc = lib()
    jobs = []
    for i, (dt, bits, ns) in enumerate(FORMS):
        bt, sh, q = _case(ns, [5, 0, 70, 200, 9, 31], [0, 3], [500 + 10 * i, 260], 8, 2, 64, 16, dt, bits, seed=i)
        out, cache, ws = _call(vc, sh, q, 0.1)
        jobs.append([bt, sh, q, out, cache, ws])
    one = vc.Workspace(max(j[5].nbytes for j in jobs))
    graphs = []
    for bt, sh, q, out, cache, ws in jobs:
        _call(vc, sh, q, 0.1, cache, one)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], capture_error_mode="thread_local"):
            _call(vc, sh, q, 0.1, cache, one, out)
    for _ in range(2):
        for j, g in zip(jobs, graphs):
            j[3].fill_(7.0)
            g.replay()
    torch.cuda.synchronize()
    for bt, sh, q, out, cache, ws in jobs:
        _compare(bt, q, out, 0.1)
        out.fill_(7.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(4):
        for (bt, sh, q, out, cache, ws), st in zip(jobs, streams):
            _call(vc, sh, q, 0.1, cache, ws, out, stream=st)
    torch.cuda.synchronize()
    for bt, sh, q, out, cache, ws in jobs:
        _compare(bt, q, out, 0.1)
        assert vc.vc_poll_status(ws) == 0 and int(cache.status) == 0


@pytest.mark.parametrize("dtype,bits,ns", FORMS)
def test_what_does_not_fit_is_reported(dtype, bits, ns):
    """Groups and lengths that do not fit: sequences attend on their own, one whose
    context does not hold the prefix is left alone, others' results stand."""
    vc = lib()
    bt, sh, q = _case(ns, [5, 0, 70, 200, 9, 31], [0, 3], [300, 260], 4, 2, 64, 16, dtype, bits)
    out, cache, ws = _call(vc, sh, q, 0.2)
    bad = vc.VC_PAGED_BAD_LENGTH

    def call():
        cache.status.zero_()
        out.fill_(7.0)
        _call(vc, sh, q, 0.2, cache, ws, out)
        torch.cuda.synchronize()
        assert vc.vc_poll_status(ws) == 0
        return int(cache.status)
    first, lens, ctx = sh.seq_start.clone(), sh.len.clone(), bt.ctx.clone()
    for f, n in (([-1, 3, 6], [300, 260]), ([0, 3, 7], [300, 260]), ([0, 3, 6], [-1, 260]), ([0, 3, 6], [300, 1 << 30]),
                 ([6, 3, 2], [300, 260])):
        sh.seq_start.copy_(torch.tensor(f, dtype=torch.int32))
        sh.len.copy_(torch.tensor(n, dtype=torch.int32))
        assert call() == bad
        _compare(bt, q, out, 0.2)
    sh.seq_start.copy_(first), sh.len.copy_(lens)
    bt.ctx[1] = 255                                          # less than the 288 slots that its group shares
    assert call() == bad
    want, tol, _, _ = paged_ref.attn(bt, q, 0.2)
    tol = tol + 32 * paged_ref.U_F32 * torch.nan_to_num(want).abs().amax()
    for b in (0, 2, 3, 4, 5):
        r = slice(bt.start[b], bt.start[b + 1])
        close(out[r], want[r], tol[r], f"sequence {b}")
    assert (out[bt.start[1]:bt.start[2]] == 7.0).all()
    bt.ctx.copy_(ctx)
    # rows out of order: nothing is read or written outside the buffers, the other group's results stand
    starts = bt.q_start.clone()
    bt.q_start.copy_(torch.tensor([bt.start[1], bt.start[2], 0, bt.start[3], bt.start[4], bt.start[5], bt.start[6]],
                                  dtype=torch.int32))
    assert call() & bad
    for b in (3, 4, 5):
        r = slice(bt.start[b], bt.start[b + 1])
        close(out[r], want[r], tol[r], f"sequence {b}")
    bt.q_start.copy_(starts)
    # a bad page of the prefix: reported, the other group's results stand
    sh.block_table[0, 2] = bt.n_pages
    assert call() == vc.VC_PAGED_BAD_PAGE
    for b in (3, 4, 5):
        r = slice(bt.start[b], bt.start[b + 1])
        close(out[r], want[r], tol[r], f"sequence {b}")


@pytest.mark.parametrize("dtype,bits,ns", FORMS)
def test_scores_of_any_size(dtype, bits, ns):
    """Weights far apart on both sides of the join: the prefix's scores all far
    above, or below, those of the sequences' own slots."""
    vc = lib()
    for sign in (1.0, -1.0):
        bt, sh, q = _case(ns, [5, 1, 70, 200, 9, 31], [0, 3], [304, 256], 4, 2, 64, 16, dtype, bits, seed=4)
        # one channel decides: keys of the prefix at +-8 times the others'
        q[..., 0] = 4.0
        for pages in (bt.k, bt.k8):
            x = pages.view(torch.uint8) if pages is bt.k8 else pages
            for g, f in ((0, 19), (3, 16)):
                for i in range(f):
                    p = bt.table[g][i]
                    if pages is bt.k8:
                        x[p, :, :, 0] = 0x7e if sign > 0 else 0xfe       # +-448
                    else:
                        x[p, :, :, 0] = sign * 448 * torch.exp2(bt.ks[p].view(torch.uint8).float() - 127).to(dtype)
        out, cache, ws = _call(vc, sh, q, 40.0)
        assert vc.vc_poll_status(ws) == 0 and int(cache.status) == 0
        _compare(bt, q, out, 40.0)


def test_heads_and_rows_at_the_edges():
    """One kv head of many query heads, many groups of two, wide tables."""
    vc = lib()
    for Hq, Hkv, n_seq in ((128, 1, 4), (5, 5, 70)):
        first = list(range(0, n_seq, 2))
        bt, sh, q = _case([1] * n_seq, [3 * i % 40 for i in range(n_seq)], first, [64 + i for i in range(len(first))], Hq,
                          Hkv, 64, 16, BF, 16, seed=2, width=600)
        out, cache, ws = _call(vc, sh, q, 0.1)
        _compare(bt, q, out, 0.1)
        assert int(cache.status) == 0


def test_a_server_run():
    """The operators together, as a server calls them: a document is read into
    8-bit pages, conversations about it share those pages, append their own words,
    attend, and one of them is read back.  Against the fp64 forms at every step."""
    import paged8_ref
    vc = lib()
    B, Hq, Hkv, d, page, n_pages, doc = 3, 8, 2, 128, 16, 80, 150
    g = torch.Generator().manual_seed(0)
    i32 = dict(dtype=torch.int32, device="cuda")
    k8 = torch.full((n_pages, Hkv, page, d), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v8 = k8.clone()
    ks = torch.full((n_pages, Hkv, page), 255, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    vs = ks.clone()
    free = torch.randperm(n_pages, generator=g).tolist()
    rope, width, lens = vc.vc_rope_init(d, 1e4), 20, [0] * B
    table = torch.full((B, width), -1, dtype=torch.int32)

    def step(ns, groups):
        for b in range(B):
            for i in range(-(-(lens[b] + ns[b]) // page)):
                if int(table[b, i]) < 0:
                    table[b, i] = free.pop()
        start = [0]
        for n in ns:
            start.append(start[-1] + n)
        T = start[-1]
        cache = vc.Paged8Cache(k8, v8, ks, vs, table.cuda())
        q_start, ctx = torch.tensor(start, **i32), torch.tensor(lens, **i32)
        qkv = torch.randn(T, (Hq + 2 * Hkv) * d, generator=g).to(BF).cuda()
        q, out = torch.empty(T, Hq, d, dtype=BF, device="cuda"), torch.empty(T, Hq, d, dtype=BF, device="cuda")
        vc.vc_paged8_append(qkv, cache, q_start, ctx, q, rope)
        if groups:
            first, pre = torch.tensor([0, B], **i32), torch.tensor([doc], **i32)
            ws = vc.Workspace(vc.vc_paged8_attn_shared_workspace_bytes(cache, 1, T, Hq))
            vc.vc_paged8_attn_shared(q, cache, first, pre, q_start, ctx, d ** -0.5, out, ws)
        else:
            ws = vc.Workspace(vc.vc_paged8_attn_workspace_bytes(cache, T, Hq))
            vc.vc_paged8_attn(q, cache, q_start, ctx, d ** -0.5, out, ws)
        k, v = (torch.empty(T, Hkv, d, dtype=BF, device="cuda") for _ in "kv")
        vc.vc_paged8_read(cache, q_start, ctx, k, v)
        torch.cuda.synchronize()
        assert vc.vc_poll_status(ws) == 0 and int(cache.status) == 0
        bt = Batch8.__new__(Batch8)
        bt.ns, bt.cs, bt.B, bt.Hkv, bt.d, bt.page, bt.width, bt.dtype = ns, list(lens), B, Hkv, d, page, width, BF
        bt.lens, bt.start, bt.table = [a + b for a, b in zip(lens, ns)], start, table.tolist()
        bt.k = torch.nan_to_num(paged8_ref.values(k8, ks.view(torch.uint8)), posinf=0, neginf=0).to(BF).cuda()
        bt.v = torch.nan_to_num(paged8_ref.values(v8, vs.view(torch.uint8)), posinf=0, neginf=0).to(BF).cuda()
        want, tol, _, _ = paged_ref.attn(bt, q, d ** -0.5)
        close(out, want, tol + 32 * paged_ref.U_F32 * want.abs().amax(), "out")
        raw = qkv.cpu().double().view(T, -1, d)[:, Hq + Hkv:]
        code, byte = paged8_ref.quantise(raw)
        assert torch.equal(v.cpu().double(), code * paged8_ref._two(byte - 127)[..., None])
        for b in range(B):
            assert torch.equal(k[start[b]:start[b + 1], 1].cpu().double(), bt.rows(bt.k, b, 1)[lens[b]:])
            lens[b] += ns[b]

    step([doc, 0, 0], False)                                 # the document
    for b in (1, 2):                                         # whose whole pages the others share, the rest copied
        m = doc // page
        table[b, :m] = table[0, :m]
        table[b, m] = free.pop()
        for x in (k8, v8, ks, vs):
            x.view(torch.uint8)[int(table[b, m])] = x.view(torch.uint8)[int(table[0, m])]
        lens[b] = doc
    step([5, 9, 1], True)
    step([1, 1, 1], True)
    step([30, 1, 17], True)


def test_programmatic_launch_changes_no_result():
    """VC_PDL=0 (a process of its own) gives the same bits: no kernel of the chain
    starts on something that an earlier one has not finished."""
    import hashlib
    import os
    import subprocess
    import sys
    code = """
import sys, hashlib, torch
sys.path[:0] = [%r, %r]
import test_gpu_paged_shared as t
from helpers import lib
vc, h = lib(), hashlib.sha256()
for i, (dt, bits, ns) in enumerate(t.FORMS):
    bt, sh, q = t._case(ns, [5, 0, 70, 200, 9, 31], [0, 3], [900, 260], 8, 2, 64, 16, dt, bits, seed=i)
    cache = sh.cache(vc)
    ws = None
    for _ in range(20):
        out, cache, ws = t._call(vc, sh, q, 0.1, cache, ws)
    h.update(out.cpu().view(torch.uint8).numpy().tobytes())
print(h.hexdigest())
"""
    here = os.path.dirname(os.path.abspath(__file__))
    code = code % (os.path.dirname(here), here)
    got = []
    for pdl in ("1", "0"):
        r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, VC_PDL=pdl), capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        got.append(r.stdout.strip().splitlines()[-1])
    assert got[0] == got[1] and len(got[0]) == hashlib.sha256().digest_size * 2


@pytest.mark.parametrize("graph", [False, True])
def test_calls_in_a_row_on_one_workspace_do_not_meet(graph):
    """Batches of other lengths, groups, types and kernels follow one another without a
    pause on one workspace: a kernel that began too early would read the plan, the
    parts or the places of the call before.  The bits of each call alone."""
    vc = lib()
    jobs = []
    for i, (dt, bits, ns) in enumerate(FORMS * 2):
        far = i >= len(FORMS)
        own, prefix = ([900, 3, 40, 0, 2000, 5], [260, 1300]) if far else ([5, 0, 70, 200, 9, 31], [900, 260])
        bt, sh, q = _case(ns[::-1] if far else ns, own, [0, 2] if far else [0, 3], prefix, 8, 2, 64, 16, dt, bits, seed=i)
        want, cache, ws = _call(vc, sh, q, 0.1)
        torch.cuda.synchronize()
        _compare(bt, q, want, 0.1)
        jobs.append((sh, q, cache, want, ws.nbytes))
    one = vc.Workspace(max(j[4] for j in jobs))
    order = [(7 * i) % len(jobs) for i in range(6 * len(jobs))]      # every batch after another kind of one
    outs = [torch.full_like(jobs[i][1], 7.0) for i in order]

    def run():
        for i, out in zip(order, outs):
            sh, q, cache, _, _ = jobs[i]
            _call(vc, sh, q, 0.1, cache, one, out)
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            run()
        g.replay()
        g.replay()
    else:
        run()
    torch.cuda.synchronize()
    assert vc.vc_poll_status(one) == 0
    for i, out in zip(order, outs):
        assert torch.equal(out, jobs[i][3]), i
