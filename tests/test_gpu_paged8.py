"""The 8-bit paged cache on the GPU against its plain forms (paged8_ref.py,
paged_ref.py, where the tolerances are derived)."""
import math

import pytest
import torch

import paged8_ref
import paged_ref
from helpers import lib
from paged8_ref import Batch8
from paged_ref import close

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _attn(vc, bt, q, scale, cache=None, ws=None, out=None):
    cache = cache or bt.cache8(vc)
    out = torch.full_like(q, 7.0) if out is None else out
    ws = ws or vc.Workspace(vc.vc_paged8_attn_workspace_bytes(cache, q.shape[0], q.shape[1]))
    vc.vc_paged8_attn(q, cache, bt.q_start, bt.ctx, scale, out, ws)
    assert vc.vc_poll_status(ws) == 0 and int(cache.status) == 0
    return out


def _compare(bt, q, out, scale, what=""):
    want, tol, _, _ = paged_ref.attn(bt, q, scale)
    rows = torch.zeros(q.shape[0], dtype=torch.bool)
    for b in range(bt.B):
        rows[bt.start[b]:bt.start[b + 1]] = True
    close(out.cpu()[rows], want[rows], tol[rows], what + " out")
    assert (out.cpu()[~rows] == 7.0).all(), what + ": a row of no sequence was written"


# ------------------------------------------------------------------- append --
APPEND = [  # chunks, contexts, Hq, Hkv, d, page, rotary, norm
    ([1], [0], 1, 1, 128, 16, 128, True),
    ([1] * 16, list(range(16)), 32, 8, 128, 64, 128, True),
    ([3, 0, 40], [15, 3, 60], 8, 2, 64, 16, 64, False),
    ([17, 5], [250, 0], 7, 1, 128, 32, 64, True),
    ([700, 33], [100, 255], 4, 2, 64, 256, 16, True),
    ([611], [7], 28, 4, 128, 128, 128, False)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case, dtype):
    """q within half a step of its type, v the nearest codes exactly, k within half
    a step of the rotated row, whose own error is paged_ref.append's."""
    vc = lib()
    ns, cs, Hq, Hkv, d, page, rotary, norm = APPEND[case]
    bt = Batch8(ns, cs, Hkv, d, page, dtype, seed=case, head_rows=case % 3, tail_rows=case % 2)
    T = bt.T
    qkv = bt.randn(T, (Hq + 2 * Hkv) * d, scale=2.0)
    qg, kg = (bt.randn(d), bt.randn(d)) if norm else (None, None)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (T,), generator=bt.g).int()
    if case == 2:
        qkv[0] = 0                                           # a row of zeros
    inv_freq = [1e4 ** (-2 * j / rotary) for j in range(rotary // 2)]
    rope = vc.vc_rope_init(rotary, 1e4)
    cache = bt.cache8(vc)
    k0, v0, ks0, vs0 = (t.view(torch.uint8).clone() for t in (bt.k8, bt.v8, bt.ks, bt.vs))
    q = torch.full((T, Hq, d), 7.0, dtype=dtype, device="cuda")
    vc.vc_paged8_append(qkv, cache, bt.q_start, bt.ctx, q, rope, positions=pos.cuda(), q_gain=qg, k_gain=kg, eps=1e-5)
    assert int(cache.status) == 0
    # the position's angle reduced exactly, as the library does
    turns = torch.tensor([[(int(p) * int(rope.turn[j])) % 2 ** 64 / 2.0 ** 64 for j in range(rotary // 2)] for p in pos])
    y, v, tol = _append_ref(bt, qkv, Hq, turns, qg, kg)
    rows = torch.zeros(T, dtype=torch.bool)
    for b in range(bt.B):
        rows[bt.start[b]:bt.start[b + 1]] = True
    close(q.cpu()[rows], y[rows, :Hq], (tol + paged_ref.half_step(dtype) * y.abs())[rows, :Hq], "q")
    assert (q.cpu()[~rows] == 7.0).all()
    written = torch.zeros(k0.shape[:3], dtype=torch.bool)
    for b in range(bt.B):
        for i in range(ns[b]):
            row, slot = bt.start[b] + i, cs[b] + i
            p, r = bt.table[b][slot // page], slot % page
            written[p, :, r] = True
            code, byte = paged8_ref.quantise(v[row])
            assert torch.equal(bt.vs[p, :, r].view(torch.uint8).cpu().long(), byte)
            assert torch.equal(paged8_ref.decode(bt.v8[p, :, r].view(torch.uint8).cpu()), code)
            want, err = y[row, Hq:], tol[row, Hq:]
            kb = bt.ks[p, :, r].view(torch.uint8).cpu().long()
            top = want.abs().amax(-1)
            assert (kb >= paged8_ref.scale_byte((top - err.amax(-1)).clamp(min=0))).all()
            assert (kb <= paged8_ref.scale_byte(top + err.amax(-1))).all()
            got = paged8_ref.values(bt.k8[p, :, r], bt.ks[p, :, r].view(torch.uint8))
            step = torch.maximum(paged8_ref.U_E4M3 * (want.abs() + err), 2.0 ** -10 * paged8_ref._two(kb - 127)[:, None])
            close(got, want, err + step, f"k of row {row}")
    for new, old in ((bt.k8, k0), (bt.v8, v0), (bt.ks, ks0), (bt.vs, vs0)):
        assert torch.equal(new.view(torch.uint8).cpu()[~written], old.cpu()[~written])


def _append_ref(bt, qkv, Hq, turns, qg, kg):
    """paged_ref.append with angles given in turns."""
    d, Hkv, T = bt.d, bt.Hkv, qkv.shape[0]
    x = qkv.detach().cpu().double().view(T, Hq + 2 * Hkv, d)
    y = x[:, :Hq + Hkv].clone()
    if qg is not None:
        gain = torch.cat([qg.cpu().double().expand(Hq, d), kg.cpu().double().expand(Hkv, d)])
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-5) * gain
    r2 = turns.shape[1]
    amp = y.abs().clone()
    a, b = y[..., :r2].clone(), y[..., r2:2 * r2].clone()
    c, s = torch.cos(2 * math.pi * turns)[:, None], torch.sin(2 * math.pi * turns)[:, None]
    y[..., :r2], y[..., r2:2 * r2] = a * c - b * s, b * c + a * s
    amp[..., :r2] = amp[..., r2:2 * r2] = torch.sqrt(a * a + b * b)
    return y, x[:, Hq + Hkv:], (d + 40) * paged_ref.U_F32 * amp * 1.01


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_rounds_every_value_as_e4m3_does(dtype):
    """Rows of every size (zeros, subnormal scales, saturation), values at and
    next to the borders between codes: the nearest code, ties to even."""
    vc = lib()
    d, T = 128, 4096
    g = torch.Generator().manual_seed(1)
    table = paged8_ref.decode(torch.arange(127, dtype=torch.uint8))
    mid = (table[:-1] + table[1:]) / 2
    near = torch.cat([table, mid, mid * (1 + 2.0 ** -7), mid * (1 - 2.0 ** -8)])
    x = near[torch.randint(0, len(near), (T, d), generator=g)] * torch.where(torch.rand(T, d, generator=g) < 0.5, -1, 1)
    x[:, 0] = torch.tensor([448.0, 225.0, 300.0, 250.0])[torch.arange(T) % 4]
    e = torch.linspace(-140, 118, T).round().long()
    x = x * paged8_ref._two(e)[:, None]
    x[5] = 0
    x[6] = 3.3e38
    x = x.to(dtype).double()
    kv = torch.stack([torch.zeros_like(x), torch.zeros_like(x), x], 1).to(dtype).reshape(T, 3 * d).cuda()
    bt = Batch8([T], [0], 1, d, 64, dtype)
    q = torch.empty(T, 1, d, dtype=dtype, device="cuda")
    vc.vc_paged8_append(kv, bt.cache8(vc), bt.q_start, bt.ctx, q, vc.vc_rope_init(128, 1e4))
    code, byte = paged8_ref.quantise(x)
    at = torch.tensor(bt.table[0]).long()
    got_b = bt.vs.view(torch.uint8).cpu()[at, 0].reshape(-1)[:T].long()
    got = paged8_ref.decode(bt.v8.view(torch.uint8).cpu()[at, 0].reshape(-1, d)[:T])
    assert torch.equal(got_b, byte) and torch.equal(got, code)
    assert (bt.ks.view(torch.uint8).cpu()[at, 0].reshape(-1)[:T] == 10).all()       # rows of zeros


# --------------------------------------------------------------------- read --
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(5))
def test_read(case, dtype):
    vc = lib()
    ns, cs, Hkv, d, page = [([1], [0], 1, 64, 16), ([5, 0, 33], [11, 4, 0], 2, 128, 16), ([200, 1], [0, 300], 8, 64, 256),
                            ([16] * 40, [3 * i for i in range(40)], 4, 128, 32), ([1000], [37], 3, 128, 64)][case]
    bt = Batch8(ns, cs, Hkv, d, page, dtype, seed=case, head_rows=case % 3, tail_rows=case % 4, spread=True)
    k, v = (torch.full((bt.T, Hkv, d), 7.0, dtype=dtype, device="cuda") for _ in "kv")
    cache = bt.cache8(vc)
    vc.vc_paged8_read(cache, bt.q_start, bt.ctx, k, v)
    assert int(cache.status) == 0
    rows = torch.zeros(bt.T, dtype=torch.bool)
    for b in range(bt.B):
        lo, hi = bt.start[b], bt.start[b + 1]
        rows[lo:hi] = True
        for h in range(Hkv):
            assert torch.equal(k[lo:hi, h].cpu().double(), bt.rows(bt.k, b, h)[cs[b]:])
            assert torch.equal(v[lo:hi, h].cpu().double(), bt.rows(bt.v, b, h)[cs[b]:])
    assert (k.cpu()[~rows] == 7).all() and (v.cpu()[~rows] == 7).all()


def test_read_gives_every_code_and_scale():
    """All codes but NaN under all scales 10 .. 246, in both types."""
    vc = lib()
    codes = torch.tensor([c for c in range(256) if c & 127 != 127] + [0, 0], dtype=torch.uint8)
    byte = torch.arange(10, 247, dtype=torch.uint8)
    T, page = 237, 256
    k8 = codes.view(2, 128)[None, :, None, :].expand(1, 2, page, 128).contiguous().cuda()
    ks = torch.full((1, 2, page), 10, dtype=torch.uint8)
    ks[:, :, :T] = byte
    ks = ks.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    for dtype in (BF, F32):
        cache = vc.Paged8Cache(k8, k8.clone(), ks, ks.clone(), torch.zeros(1, 1, **i32), dtype)
        k, v = torch.empty(T, 2, 128, dtype=dtype, device="cuda"), torch.empty(T, 2, 128, dtype=dtype, device="cuda")
        vc.vc_paged8_read(cache, torch.tensor([0, T], **i32), torch.zeros(1, **i32), k, v)
        want = paged8_ref.values(codes.view(1, 2, 128).expand(T, 2, 128), byte[:, None].expand(T, 2))
        fits = want.abs() < 3.3895e38
        assert torch.equal(k.cpu().double()[fits], want[fits]) and torch.equal(v.cpu().double()[fits], want[fits])


# ---------------------------------------------------------------- attention --
CASES = [  # (chunks, contexts, query heads, kv heads, d, page)
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
    ([1] * 40, [37 * i % 700 for i in range(40)], 8, 2, 128, 16),     # more sequences than a warp has lanes
    ([1, 2, 1], [3000, 5000, 17], 16, 1, 64, 32)]           # 16 and 32 rows per kv head


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, dtype):
    vc = lib()
    ns, cs, Hq, Hkv, d, page = CASES[case]
    bt = Batch8(ns, cs, Hkv, d, page, dtype, seed=case, head_rows=case % 3, tail_rows=case % 4, width=case % 5)
    q = bt.randn(bt.T, Hq, d, scale=1.5)
    out = _attn(vc, bt, q, d ** -0.5)
    _compare(bt, q, out, d ** -0.5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_rows_of_very_different_sizes(d, dtype):
    """Scales from 2^-18 to 2^9 of the ordinary one, rows of zeros."""
    vc = lib()
    bt = Batch8([1, 40, 3], [500, 333, 1000], 2, d, 16, dtype, seed=9, spread=True)
    q = bt.randn(bt.T, 8, d)
    out = _attn(vc, bt, q, d ** -0.5)
    _compare(bt, q, out, d ** -0.5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ns,cs", [([1, 1], [1500, 700]), ([3, 40], [1500, 700]), ([200], [900])])
@pytest.mark.parametrize("scale,peak", [(0.0, 1.0), (0.3, 6.0), (1.0, 4.0)])
def test_attention_scales(ns, cs, scale, peak, dtype):
    """A scale of zero (the mean of what is visible) and peaked weights: the
    running maximum moves by far more than a few powers of two."""
    vc = lib()
    bt = Batch8(ns, cs, 2, 128, 64, dtype, seed=9, spread=scale == 0.3)
    q = bt.randn(bt.T, 8, 128, scale=peak)
    out = _attn(vc, bt, q, scale)
    _compare(bt, q, out, scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_values_far_apart_in_size(d, dtype):
    """The first keys carry values of 2^40 under weights of about 2^-60, the last
    ones ordinary values under ordinary weights, and the other way round: what is
    small beside the largest product is lost, nothing else."""
    vc = lib()
    for flip in (False, True):
        bt = Batch8([1, 2], [300, 1000], 1, d, 16, dtype, seed=3)
        q = bt.randn(bt.T, 4, d)
        q[..., 0] = 8.0
        for b in range(2):
            L = bt.lens[b]
            for i in range(L):
                p, r = bt.table[b][i // 16], i % 16
                old = (i < L // 2) != flip
                bt.ks[p, :, r] = torch.tensor(120, dtype=torch.uint8).view(torch.float8_e8m0fnu)
                bt.k8.view(torch.uint8)[p, :, r, 0] = 0xf0 if old else 0x00          # -128 and 0
                bt.vs.view(torch.uint8)[p, :, r] = 127 + 40 if old else 122
        # the values the bytes stand for
        bt.k = paged8_ref.values(bt.k8, bt.ks.view(torch.uint8)).to(dtype).cuda()
        bt.v = paged8_ref.values(bt.v8, bt.vs.view(torch.uint8)).to(dtype).cuda()
        out = _attn(vc, bt, q, 5.0)
        _compare(bt, q, out, 5.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ns,Hq", [([1, 2], 4), ([2, 1], 10), ([30, 9], 4)])
@pytest.mark.parametrize("size", [112, 60, -60, -108])
def test_large_keys_under_small_queries(size, ns, Hq, dtype):
    """Keys of 2^size under queries of 2^-size, products of ordinary size; one query
    row in three is 2^-40 of the others."""
    vc = lib()
    bt = Batch8(ns, [300, 77], 1, 128, 16, dtype, seed=4)
    byte = bt.ks.view(torch.uint8)
    byte[byte < 255] += torch.tensor(size, dtype=torch.int8, device="cuda").view(torch.uint8)
    assert int(byte.min()) >= 10
    bt.k = paged8_ref.values(bt.k8, byte).to(dtype).cuda()
    q = bt.randn(bt.T, Hq, 128) * 2.0 ** -size
    q[:, ::3] *= 2.0 ** -40 if size < 100 else 1.0
    out = _attn(vc, bt, q, 0.1)
    _compare(bt, q, out, 0.1)


def test_attention_gives_the_bits_of_bf16_pages():
    """Where both take the tensor-core kernel (more than 16 rows per kv head) the
    expansion is exact: the same bits as pages that hold the values."""
    vc = lib()
    bt = Batch8([90, 33], [1300, 200], 2, 128, 32, BF, seed=3, spread=True)
    q = bt.randn(bt.T, 8, 128)
    a = _attn(vc, bt, q, 0.1)
    cache = vc.PagedCache(bt.k, bt.v, bt.block_table)
    ws = vc.Workspace(vc.vc_paged_attn_workspace_bytes(cache, bt.T, 8))
    b = torch.full_like(q, 7.0)
    vc.vc_paged_attn(q, cache, bt.q_start, bt.ctx, 0.1, b, ws)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ns,cs,Hq", [([1] * 3, [1300, 40, 200], 8), ([5, 1, 90], [1300, 40, 200], 8)])
def test_attention_repeats_and_rides_in_a_graph(ns, cs, Hq, dtype):
    """Two calls give the same bits; so does a captured call, on a side stream
    with the eager call's workspace, also over new lengths and queries."""
    vc = lib()
    bt = Batch8(ns, cs, 2, 128, 32, dtype, seed=3)
    cache = bt.cache8(vc)
    q = bt.randn(bt.T, Hq, 128)
    ws = vc.Workspace(vc.vc_paged8_attn_workspace_bytes(cache, bt.T, Hq))
    a = _attn(vc, bt, q, 0.1, cache, ws)
    assert torch.equal(a, _attn(vc, bt, q, 0.1, cache, ws))
    out, k, v = torch.zeros_like(q), *(torch.zeros(bt.T, 2, 128, dtype=dtype, device="cuda") for _ in "kv")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream(), capture_error_mode="thread_local"):
        vc.vc_paged8_attn(q, cache, bt.q_start, bt.ctx, 0.1, out, ws)
        vc.vc_paged8_read(cache, bt.q_start, bt.ctx, k, v)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a)
    q.copy_(bt.randn(*q.shape))
    n2 = [max(n - 2, 0) for n in ns]
    bt.start = [0, n2[0], n2[0] + n2[1], sum(n2)]
    bt.q_start.copy_(torch.tensor(bt.start, dtype=torch.int32))
    bt.ctx.copy_(torch.tensor([1000, 41, 199], dtype=torch.int32))
    out.fill_(7.0), k.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    bt.ns, bt.cs = n2, [1000, 41, 199]
    bt.lens = [c + n for c, n in zip(bt.cs, n2)]
    _compare(bt, q, out, 0.1, "replayed")
    for b in range(3):
        for h in range(2):
            assert torch.equal(k[bt.start[b]:bt.start[b + 1], h].cpu().double(), bt.rows(bt.k, b, h)[bt.cs[b]:])
    assert (k[sum(n2):] == 7).all() and vc.vc_poll_status(ws) == 0


def test_two_graphs_share_a_workspace():
    """Nothing of a call stays in the workspace: captured batches of other shapes
    and kernels replay in turn on one."""
    vc = lib()
    jobs, need = [], 0
    for ns, cs, Hq, dt in (([1, 1, 1], [3000, 77, 900], 8, BF), ([60, 200], [500, 40], 4, BF), ([7, 1], [600, 50], 4, F32)):
        bt = Batch8(ns, cs, 2, 128, 32, dt, seed=len(jobs))
        cache = bt.cache8(vc)
        q = bt.randn(bt.T, Hq, 128)
        need = max(need, vc.vc_paged8_attn_workspace_bytes(cache, bt.T, Hq))
        jobs.append((bt, cache, q, torch.full_like(q, 7.0)))
    ws = vc.Workspace(need)
    graphs = []
    for bt, cache, q, out in jobs:
        _attn(vc, bt, q, 0.1, cache, ws)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], capture_error_mode="thread_local"):
            vc.vc_paged8_attn(q, cache, bt.q_start, bt.ctx, 0.1, out, ws)
    for _ in range(2):
        for (bt, cache, q, out), g in zip(jobs, graphs):
            out.fill_(7.0)
            g.replay()
    torch.cuda.synchronize()
    for bt, cache, q, out in jobs:
        _compare(bt, q, out, 0.1)
    assert vc.vc_poll_status(ws) == 0


def test_two_calls_at_once_on_two_streams():
    vc = lib()
    jobs = []
    for i in range(4):
        bt = Batch8([1, 1] if i < 2 else [30, 1], [900 + i, 2000], 2, 128, 64, BF, seed=20 + i)
        cache = bt.cache8(vc)
        q = bt.randn(bt.T, 8, 128)
        ws = vc.Workspace(vc.vc_paged8_attn_workspace_bytes(cache, bt.T, 8))
        jobs.append((bt, cache, q, torch.full_like(q, 7.0), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for bt, cache, q, out, ws, st in jobs:
            vc.vc_paged8_attn(q, cache, bt.q_start, bt.ctx, 0.1, out, ws, stream=st)
    torch.cuda.synchronize()
    for bt, cache, q, out, ws, st in jobs:
        _compare(bt, q, out, 0.1)


@pytest.mark.parametrize("ns", [[9, 2], [2, 1]])
def test_sixteen_byte_alignment_is_enough(ns):
    vc = lib()
    bt = Batch8(ns, [300, 77], 2, 64, 16, BF, seed=6)

    def shifted(t):
        n = 16 // t.element_size()
        x = torch.zeros(t.numel() + n, dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device="cuda")[n:]
        return x.view(t.dtype).view(t.shape).copy_(t)
    q = shifted(bt.randn(bt.T, 16, 64))
    bt.k8, bt.v8, bt.ks, bt.vs = (shifted(t.view(torch.uint8)) for t in (bt.k8, bt.v8, bt.ks, bt.vs))
    out = _attn(vc, bt, q, 0.2, out=shifted(torch.full_like(q, 7.0)))
    _compare(bt, q, out, 0.2)
    k, v = (shifted(torch.zeros(bt.T, 2, 64, dtype=BF, device="cuda")) for _ in "kv")
    vc.vc_paged8_read(bt.cache8(vc), bt.q_start, bt.ctx, k, v)
    assert torch.equal(v[:ns[0], 1].cpu().double(), bt.rows(bt.v, 0, 1)[300:])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pools_past_two_to_the_31_elements(dtype):
    """Pages whose codes lie past 2^31 bytes: every operator gives what it gives
    on a small pool, bit for bit."""
    vc = lib()
    Hkv, page, d = 4, 256, 128
    for ns in ([1, 1], [40, 3]):
        small = Batch8(ns, [600, 255], Hkv, d, page, dtype, seed=7, width=4)
        n_big = 2 ** 31 // (Hkv * page * d) + 20
        shift = n_big - small.n_pages
        table = torch.where(small.block_table >= 0, small.block_table + shift, small.block_table)
        big = [torch.zeros((n_big,) + t.shape[1:], dtype=torch.uint8, device="cuda") for t in (small.k8, small.v8, small.ks, small.vs)]
        for x, t in zip(big, (small.k8, small.v8, small.ks, small.vs)):
            x[shift:] = t.view(torch.uint8)
        q = small.randn(small.T, 16, d)
        qkv = small.randn(small.T, (16 + 2 * Hkv) * d)
        got = []
        for cache in (small.cache8(vc), vc.Paged8Cache(*big, table, dtype)):
            ws = vc.Workspace(vc.vc_paged8_attn_workspace_bytes(cache, small.T, 16))
            out, qo = torch.empty_like(q), torch.empty_like(q)
            k, v = (torch.empty(small.T, Hkv, d, dtype=dtype, device="cuda") for _ in "kv")
            vc.vc_paged8_append(qkv, cache, small.q_start, small.ctx, qo, vc.vc_rope_init(d, 1e4))
            vc.vc_paged8_attn(q, cache, small.q_start, small.ctx, 0.1, out, ws)
            vc.vc_paged8_read(cache, small.q_start, small.ctx, k, v)
            torch.cuda.synchronize()
            assert int(cache.status) == 0 and vc.vc_poll_status(ws) == 0
            got.append((out, qo, k, v))
        for a, b in zip(*got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ns", [[4, 6, 2, 3], [1, 1, 1, 1], [40, 60, 20, 30]])
def test_what_does_not_fit_is_reported_and_left_alone(ns, dtype):
    """Bad page numbers and lengths: the status word says so, nothing outside the
    pool is touched and the other sequences' results stand."""
    vc = lib()
    bt = Batch8(ns, [100, 333, 40, 64], 2, 128, 32, dtype, seed=5)
    q = bt.randn(bt.T, 4, 128)
    cache = bt.cache8(vc)
    ws = vc.Workspace(vc.vc_paged8_attn_workspace_bytes(cache, bt.T, 4))
    bt.block_table[1, 3], bt.block_table[1, 5] = bt.n_pages, -7
    bt.ctx[2] = cache.slots                                  # more than the table holds
    out = torch.full_like(q, 7.0)
    k, v = (torch.full((bt.T, 2, 128), 7.0, dtype=dtype, device="cuda") for _ in "kv")

    def call():
        cache.status.zero_()
        out.fill_(7.0)
        vc.vc_paged8_attn(q, cache, bt.q_start, bt.ctx, 0.1, out, ws)
        torch.cuda.synchronize()
        assert vc.vc_poll_status(ws) == 0
        return int(cache.status)
    assert call() == vc.VC_PAGED_BAD_PAGE | vc.VC_PAGED_BAD_LENGTH
    want, tol, _, _ = paged_ref.attn(bt, q, 0.1)
    for b in (0, 3):
        r = slice(bt.start[b], bt.start[b + 1])
        close(out[r], want[r], tol[r], f"sequence {b}")
    assert (out[bt.start[2]:bt.start[3]] == 7.0).all()
    cache.status.zero_()
    bt.block_table[0, 3] = bt.n_pages + 5                    # slots 96 on: the chunk's first page
    vc.vc_paged8_read(cache, bt.q_start, bt.ctx, k, v)
    torch.cuda.synchronize()
    assert int(cache.status) == vc.VC_PAGED_BAD_PAGE | vc.VC_PAGED_BAD_LENGTH
    assert (k[0] == 7).all() and (v[0] == 7).all() and (k[bt.start[2]:bt.start[3]] == 7).all()
    assert torch.equal(k[bt.start[3]:, 1].cpu().double(), bt.rows(bt.k, 3, 1)[64:])
    kept = bt.k8.view(torch.uint8).clone()
    cache.status.zero_()
    vc.vc_paged8_append(bt.randn(bt.T, 8 * 128), cache, bt.q_start, bt.ctx, torch.empty_like(q), vc.vc_rope_init(128, 1e4))
    torch.cuda.synchronize()
    assert int(cache.status) == vc.VC_PAGED_BAD_PAGE | vc.VC_PAGED_BAD_LENGTH
    mine = {bt.table[b][s // 32] for b in (0, 1, 3) for s in range(bt.cs[b], bt.lens[b])} - {bt.table[0][3]}
    for p in set(range(bt.n_pages)) - mine:
        assert torch.equal(bt.k8.view(torch.uint8)[p], kept[p])
    bt.q_start[4] = bt.T + 1                                 # the last sequence leaves the packed rows
    assert call() & vc.VC_PAGED_BAD_LENGTH and (out[bt.start[3]:] == 7.0).all()


def test_empty_batches():
    vc = lib()
    bt = Batch8([0, 0], [30, 0], 2, 64, 16, BF)
    cache = bt.cache8(vc)
    q, k = torch.zeros(0, 4, 64, dtype=BF, device="cuda"), torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    ws = vc.Workspace(vc.vc_paged8_attn_workspace_bytes(cache, 0, 4))
    vc.vc_paged8_attn(q, cache, bt.q_start, bt.ctx, 0.1, q.clone(), ws)
    vc.vc_paged8_read(cache, bt.q_start, bt.ctx, k, k.clone())
    vc.vc_paged8_append(torch.zeros(0, 8 * 64, dtype=BF, device="cuda"), cache, bt.q_start, bt.ctx, q, vc.vc_rope_init(64, 1e4))
    bt = Batch8([0, 0], [30, 0], 2, 64, 16, BF, tail_rows=3)  # rows of no sequence only
    q = bt.randn(3, 4, 64)
    out = _attn(vc, bt, q, 0.1)
    assert (out == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_table_much_wider_than_its_sequences_and_many_sequences(dtype):
    """Few rows, 700 sequences, a table of 5000 pages: the results of a narrow one."""
    vc = lib()
    bt = Batch8([1] * 700, [(13 * i) % 90 for i in range(700)], 1, 64, 16, dtype, seed=1)
    q = bt.randn(bt.T, 4, 64)
    out = _attn(vc, bt, q, 0.125)
    _compare(bt, q, out, 0.125)
    wide = torch.full((700, 5000), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.width] = bt.block_table
    assert torch.equal(out, _attn(vc, bt, q, 0.125, bt.cache8(vc, wide)))


@pytest.mark.parametrize("ns,cs,Hq,Hkv,d,page", [([1100], [300], 8, 2, 128, 16), ([1030], [0], 8, 2, 64, 256),
                                                 ([1500, 600], [77, 1], 8, 2, 64, 32)])
def test_attention_of_many_rows(ns, cs, Hq, Hkv, d, page):
    """From 4096 rows per sequence and kv head on the pages are expanded first:
    the bits of bf16 pages, bad pages and padded rows as everywhere."""
    vc = lib()
    bt = Batch8(ns, cs, Hkv, d, page, BF, seed=5, spread=True, head_rows=1, tail_rows=2, width=2)
    q = bt.randn(bt.T, Hq, d)
    cache = bt.cache8(vc)
    ws = vc.Workspace(vc.vc_paged8_attn_workspace_bytes(cache, bt.T, Hq))
    assert ws.nbytes >= 4 * bt.B * cache.slots * Hkv * d
    out = _attn(vc, bt, q, 0.1, cache, ws)
    _compare(bt, q, out, 0.1)
    full = vc.PagedCache(bt.k, bt.v, bt.block_table)
    other = torch.full_like(q, 7.0)
    vc.vc_paged_attn(q, full, bt.q_start, bt.ctx, 0.1, other,
                     vc.Workspace(vc.vc_paged_attn_workspace_bytes(full, bt.T, Hq)))
    assert torch.equal(out, other)
    bt.block_table[0, 2] = bt.n_pages
    vc.vc_paged8_attn(q, cache, bt.q_start, bt.ctx, 0.1, out, ws)
    torch.cuda.synchronize()
    assert int(cache.status) == vc.VC_PAGED_BAD_PAGE and vc.vc_poll_status(ws) == 0
    if len(ns) > 1:
        assert torch.equal(out[bt.start[1]:], other[bt.start[1]:])
