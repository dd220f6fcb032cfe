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
        if first and isinstance(first[-1], tuple):
            raise ValueError
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
