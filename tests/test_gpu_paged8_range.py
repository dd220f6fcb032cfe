"""Attention over 8-bit pages where values are far apart in size, or far from
one: a weight that is zero stays so beside any value, and one that is not is kept
wherever its row's values lie.  Against the fp64 form (paged_ref.py, where the
tolerances are derived; the joins of shared prefixes are covered by the (L + 16) u
of their sums, as every row but those that must be exact sees 100 keys or more)."""
import math

import pytest
import torch

import paged8_ref
import paged_ref
from helpers import lib
from paged8_ref import Batch8
from paged_ref import close
from test_gpu_paged_shared import Shared

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _scale_values(bt, slots, byte, zero=False):
    """The values of sequence b's slots, for b, slots of a dict, under scales of
    this byte, or all zeros."""
    for b, ii in slots.items():
        for i in ii:
            p, r = bt.table[b][i // bt.page], i % bt.page
            bt.vs.view(torch.uint8)[p, :, r] = byte
            if zero:
                bt.v8.view(torch.uint8)[p, :, r] = 0
    bt.v = paged8_ref.values(bt.v8, bt.vs).to(bt.dtype).cuda()


def _run(vc, bt, q, scale, sh=None):
    out = torch.full_like(q, 7.0)
    T, Hq, _ = q.shape
    if sh is None:
        cache = bt.cache8(vc)
        ws = vc.Workspace(vc.vc_paged8_attn_workspace_bytes(cache, T, Hq))
        vc.vc_paged8_attn(q, cache, bt.q_start, bt.ctx, scale, out, ws)
    else:
        cache = sh.cache(vc)
        size, call = ((vc.vc_paged8_attn_shared_workspace_bytes, vc.vc_paged8_attn_shared) if sh.bits == 8 else
                      (vc.vc_paged_attn_shared_workspace_bytes, vc.vc_paged_attn_shared))
        ws = vc.Workspace(size(cache, len(sh.prefix), T, Hq))
        call(q, cache, sh.seq_start, sh.len, bt.q_start, bt.ctx, scale, out, ws)
    assert vc.vc_poll_status(ws) == 0 and int(cache.status) == 0
    return out


def _compare(bt, q, out, scale, lost=0.0):
    want, tol, _, _ = paged_ref.attn(bt, q, scale)
    close(out, want, tol + lost, "out")


# chunks, contexts, Hq, Hkv, d: contexts that end at a key tile (32 keys of 128
# channels, 64 of 64), so that a chunk's first rows see nothing of its last tile
LATE = [([2], [1023], 32, 8, 128), ([2] * 4, [2047] * 4, 32, 8, 128), ([4], [511], 32, 8, 128), ([2], [1023], 8, 8, 64),
        ([3, 1, 2], [1022, 300, 639], 8, 2, 64), ([100], [1000], 2, 2, 128)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("byte", [129, 132, 159, 200])
@pytest.mark.parametrize("case", range(len(LATE)))
def test_large_values_that_earlier_rows_do_not_see(case, byte, dtype):
    """The values of every token but a chunk's first are 1000, 10^4, 2^40 and 2^80:
    nothing of them reaches the rows before."""
    vc = lib()
    ns, cs, Hq, Hkv, d = LATE[case]
    bt = Batch8(ns, cs, Hkv, d, 64, dtype, seed=case)
    _scale_values(bt, {b: range(cs[b] + 1, cs[b] + ns[b]) for b in range(bt.B)}, byte)
    q = bt.randn(bt.T, Hq, d)
    _compare(bt, q, _run(vc, bt, q, d ** -0.5), d ** -0.5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("byte", [132, 140, 200])
@pytest.mark.parametrize("ns,cs", [([2], [0]), ([5, 2], [0, 40]), ([3, 1], [64, 0]), ([40], [31])])
def test_rows_that_have_seen_only_zeros(ns, cs, byte, dtype):
    """Zeros up to a chunk's first token, large values after it: the first rows are
    exactly zero."""
    vc = lib()
    for d in (64, 128):
        bt = Batch8(ns, cs, 2, d, 16, dtype, seed=5)
        _scale_values(bt, {b: range(cs[b] + 1) for b in range(bt.B)}, 10, zero=True)
        _scale_values(bt, {b: range(cs[b] + 1, cs[b] + ns[b]) for b in range(bt.B)}, byte)
        q = bt.randn(bt.T, 8, d)
        out = _run(vc, bt, q, 0.1)
        _compare(bt, q, out, 0.1)
        for b in range(bt.B):
            assert (out[bt.start[b]] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("byte", [140, 200])
@pytest.mark.parametrize("ns,cs", [([1, 1], [300, 20]), ([2, 3], [0, 31]), ([40], [77])])
def test_a_value_of_zero_under_the_only_weight(ns, cs, byte, dtype):
    """Key 0 has all the weight and a value of zero; the others' weights, 2^-230,
    are no fp32 numbers and may be lost whatever their values: 2^-126 of each."""
    vc = lib()
    bt = Batch8(ns, cs, 1, 128, 16, dtype, seed=6)
    bt.ks.view(torch.uint8)[bt.ks.view(torch.uint8) < 255] = 120
    bt.k8.view(torch.uint8)[..., 0] = 0xf0                   # -128 * 2^-7
    for b in range(bt.B):
        bt.k8.view(torch.uint8)[bt.table[b][0], :, 0, 0] = 0
    bt.k = paged8_ref.values(bt.k8, bt.ks).to(dtype).cuda()
    _scale_values(bt, {b: range(1, bt.lens[b]) for b in range(bt.B)}, byte)
    _scale_values(bt, {b: [0] for b in range(bt.B)}, 10, zero=True)
    q = torch.zeros(bt.T, 4, 128, dtype=dtype, device="cuda")
    q[..., 0] = 8.0
    _compare(bt, q, _run(vc, bt, q, 20.0), 20.0, lost=max(bt.lens) * 2.0 ** -126 * 2.0 ** (byte - 127 + 9))


# chunks, contexts after the prefix, groups' first sequences, prefixes, Hq, Hkv, d, page
SHARED = [([2, 4, 2], [15, 47, 31], [0], [1040], 8, 2, 128, 16),      # a small group
          ([2] * 6, [31, 63, 0, 1, 95, 31], [0], [512], 16, 2, 128, 64),      # own slots only through the kernel of few rows
          ([2, 1, 3, 4], [63, 100, 190, 126], [0, 2], [320, 128], 8, 2, 64, 64),
          ([50, 9], [30, 60], [0], [256], 2, 2, 128, 32)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("byte", [129, 140, 200])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_large_values_after_a_shared_prefix(case, byte, dtype):
    vc = lib()
    ns, own, first, prefix, Hq, Hkv, d, page = SHARED[case]
    cs = [c + prefix[max(g for g, f in enumerate(first) if f <= b)] for b, c in enumerate(own)]
    bt = Batch8(ns, cs, Hkv, d, page, dtype, seed=case)
    sh = Shared(bt, first, prefix, 8)
    _scale_values(bt, {b: range(cs[b] + 1, cs[b] + ns[b]) for b in range(bt.B)}, byte)
    q = bt.randn(bt.T, Hq, d)
    _compare(bt, q, _run(vc, bt, q, d ** -0.5, sh), d ** -0.5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("less", [0, 23, 60, 100])
@pytest.mark.parametrize("scale", [0.0, 1e-30, 2.0 ** -20])
@pytest.mark.parametrize("ns,cs", [([1, 1], [300, 1000]), ([2, 3], [1023, 95]), ([40], [200])])
def test_small_values_under_small_scales(ns, cs, scale, less, dtype):
    """Values of 2^-less under weights that are nearly or exactly the same: their
    mean, however small."""
    vc = lib()
    bt = Batch8(ns, cs, 2, 128, 16, dtype, seed=8)
    byte = bt.vs.view(torch.uint8)
    byte[byte < 255] -= less
    assert int(byte.min()) >= 10
    bt.v = paged8_ref.values(bt.v8, bt.vs).to(dtype).cuda()
    q = bt.randn(bt.T, 8, 128)
    _compare(bt, q, _run(vc, bt, q, scale), scale)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_small_values_of_a_shared_prefix_under_a_scale_of_zero(case, dtype, bits):
    vc = lib()
    ns, own, first, prefix, Hq, Hkv, d, page = SHARED[case]
    cs = [c + prefix[max(g for g, f in enumerate(first) if f <= b)] for b, c in enumerate(own)]
    bt = Batch8(ns, cs, Hkv, d, page, dtype, seed=case)
    sh = Shared(bt, first, prefix, bits)
    byte = bt.vs.view(torch.uint8)
    byte[byte < 255] -= 40
    bt.v = paged8_ref.values(bt.v8, bt.vs).to(dtype).cuda()
    q = bt.randn(bt.T, Hq, d)
    _compare(bt, q, _run(vc, bt, q, 0.0, sh), 0.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ns,cs,Hq", [([1, 1], [300, 77], 4), ([3, 2], [95, 640], 4), ([30], [200], 4)])
@pytest.mark.parametrize("size,scale", [(120, 1e6), (126, 1e8), (100, 1e8)])
def test_large_queries_under_large_scales(size, scale, ns, cs, Hq, dtype):
    """Queries of 2^size meet keys of 2^-117 times 0 to 15 under a large scale:
    every score is finite, and the row's output is the value of its largest key."""
    vc = lib()
    bt = Batch8(ns, cs, 2, 128, 16, dtype, seed=12)
    bt.ks.view(torch.uint8)[bt.ks.view(torch.uint8) < 255] = 10
    code = torch.tensor([0x08 * (i % 16) for i in range(max(bt.lens))], dtype=torch.uint8)      # 0, 2^-6 .. 2^8
    for b in range(bt.B):
        turn = torch.randperm(bt.lens[b], generator=bt.g)
        for i in range(bt.lens[b]):
            p, r = bt.table[b][i // 16], i % 16
            bt.k8.view(torch.uint8)[p, :, r] = 0
            bt.k8.view(torch.uint8)[p, :, r, 0] = code[int(turn[i]) % 15]
        bt.k8.view(torch.uint8)[bt.table[b][0], :, 3, 0] = 0x7e      # the largest: slot 3
    q = torch.zeros(bt.T, Hq, 128, dtype=dtype, device="cuda")
    q[..., 0] = 2.0 ** size
    q[..., 1] = -2.0 ** size                                 # meets zeros
    out = _run(vc, bt, q, scale)
    for b in range(bt.B):
        for h in range(2):
            want = bt.rows(bt.v, b, h)[3].expand(ns[b], Hq // 2, 128)
            assert torch.equal(out[bt.start[b]:bt.start[b + 1], h * Hq // 2:(h + 1) * Hq // 2].cpu().double(), want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_scale_of_the_largest_size_is_forgotten(dtype):
    """Keys whose values are zeros under scales of 2^127, then keys of 2^112 times
    their weights with ordinary values: those are the result.  (Two query heads, so
    that one's maximum moves while the other's weights lie above one; as many units as
    leave a warp with some of them whole.)"""
    vc = lib()
    B, L = 240, 160
    bt = Batch8([1] * B, [L - 1] * B, 8, 128, 32, dtype, seed=3)
    k8, ks, v8, vs = (t.view(torch.uint8) for t in (bt.k8, bt.ks, bt.v8, bt.vs))
    k8.zero_(), ks.fill_(127)
    at = [torch.tensor([bt.table[b][i] for b in range(B)]).long().cuda() for i in range(5)]
    v8[at[0]] = 0
    v8[at[1]] = 0
    vs[at[0]] = 254
    vs[at[1]] = 254
    for i, code in ((1, 0x4e), (2, 0x6e), (3, 0x6e), (4, 0x6e)):     # scores 0, 7 and 112
        k8[at[i], :, :, 0] = code
        if i > 1:
            vs[at[i]] = 139
    bt.k = paged8_ref.values(bt.k8, bt.ks).to(dtype).cuda()
    bt.v = paged8_ref.values(bt.v8, bt.vs).to(dtype).cuda()
    q = torch.zeros(B, 16, 128, dtype=dtype, device="cuda")
    q[:, 0::2, 0], q[:, 1::2, 0] = 1.0, 4.0
    scale = 0.6931472
    _compare(bt, q, _run(vc, bt, q, scale), scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("byte", [30, 100, 140, 200])
@pytest.mark.parametrize("gap", [40, 100, 122])
@pytest.mark.parametrize("ns,cs", [([1, 1], [300, 20]), ([2, 3], [9, 95]), ([40], [77])])
def test_tiny_weights_of_values_beside_zeros(ns, cs, gap, byte, dtype):
    """Key 0 has nearly all the weight and a value of zero; the result is the others',
    2^-gap of their values."""
    vc = lib()
    bt = Batch8(ns, cs, 1, 128, 16, dtype, seed=6)
    bt.ks.view(torch.uint8)[bt.ks.view(torch.uint8) < 255] = 120
    bt.k8.view(torch.uint8)[..., 0] = 0xf0                   # -128 * 2^-7
    for b in range(bt.B):
        bt.k8.view(torch.uint8)[bt.table[b][0], :, 0, 0] = 0
    bt.k = paged8_ref.values(bt.k8, bt.ks).to(dtype).cuda()
    _scale_values(bt, {b: range(1, bt.lens[b]) for b in range(bt.B)}, byte)
    _scale_values(bt, {b: [0] for b in range(bt.B)}, 10, zero=True)
    q = torch.zeros(bt.T, 4, 128, dtype=dtype, device="cuda")
    q[..., 0] = 8.0
    scale = gap * math.log(2) / 8
    # A row's place is 2^115 at most, a weight there is rounded to 2^-24 at the finest, off
    # by half of it, and meets codes of 448 at most: 2^-25 * 2^-115 * 448 < 2^-131 per key.
    # A bf16 result is rounded to 2^-133.
    lost = max(bt.lens) * 2.0 ** -131 + (2.0 ** -134 if dtype == BF else 2.0 ** -150)
    _compare(bt, q, _run(vc, bt, q, scale), scale, lost=lost)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("zero,byte", [(127, 80), (200, 119), (254, 100), (40, 20)])
@pytest.mark.parametrize("ns,cs", [([1, 1], [300, 1000]), ([2, 3], [1023, 95]), ([40], [200])])
def test_rows_of_zeros_under_any_scale(ns, cs, zero, byte, dtype):
    """Two keys in three have values of zero under a larger scale than the others (of
    another quantizer, say): they take their weight, and nothing else."""
    vc = lib()
    for d in (64, 128):
        bt = Batch8(ns, cs, 2, d, 16, dtype, seed=8)
        _scale_values(bt, {b: [i for i in range(L) if i % 3] for b, L in enumerate(bt.lens)}, zero, zero=True)
        _scale_values(bt, {b: range(0, L, 3) for b, L in enumerate(bt.lens)}, byte)
        q = bt.randn(bt.T, 8, d)
        _compare(bt, q, _run(vc, bt, q, 0.1), 0.1)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_rows_of_zeros_after_a_shared_prefix(case, dtype):
    vc = lib()
    ns, own, first, prefix, Hq, Hkv, d, page = SHARED[case]
    cs = [c + prefix[max(g for g, f in enumerate(first) if f <= b)] for b, c in enumerate(own)]
    bt = Batch8(ns, cs, Hkv, d, page, dtype, seed=case)
    sh = Shared(bt, first, prefix, 8)
    _scale_values(bt, {b: [i for i in range(L) if i % 3 == 1] for b, L in enumerate(bt.lens)}, 170, zero=True)
    q = bt.randn(bt.T, Hq, d)
    _compare(bt, q, _run(vc, bt, q, d ** -0.5, sh), d ** -0.5)
