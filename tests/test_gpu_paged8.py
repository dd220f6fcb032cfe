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
    """q as vc_paged_append writes it; v the nearest codes exactly; k within half
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
    plain = paged_ref.Batch(ns, cs, Hkv, d, page, dtype, seed=case, head_rows=case % 3, tail_rows=case % 2)
    q2 = torch.full_like(q, 7.0)
    vc.vc_paged_append(qkv, vc.PagedCache(plain.k, plain.v, plain.block_table), bt.q_start, bt.ctx, q2, rope,
                       positions=pos.cuda(), q_gain=qg, k_gain=kg, eps=1e-5)
    assert torch.equal(q, q2)
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
