"""Plain fp64 forms of the paged-cache operators, and ragged batches over
randomly placed pages for their tests (CPU or GPU)."""
import math

import torch

U_BF16, U_F32 = 2.0 ** -8, 2.0 ** -24        # half a step, relative


def half_step(dtype):
    return U_BF16 if dtype == torch.bfloat16 else U_F32


class Batch:
    """B sequences with chunk lengths ns over contexts cs, Hkv kv heads; the
    pool's pages are handed out in random order.  Slots past a sequence's end
    and unused pages hold NaN; table entries past the last page are -1."""

    def __init__(self, ns, cs, Hkv, d, page, dtype, seed=0, device="cuda", head_rows=0, tail_rows=0, width=0):
        g = torch.Generator().manual_seed(seed)
        self.ns, self.cs, self.Hkv, self.d, self.page, self.dtype = list(ns), list(cs), Hkv, d, page, dtype
        self.B, self.lens, self.device = len(ns), [a + b for a, b in zip(ns, cs)], device
        self.g = g
        blocks = [-(-L // page) for L in self.lens]
        self.n_pages = sum(blocks) + 2
        self.width = max(max(blocks), 1, width)
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = [[-1] * self.width for _ in range(self.B)]
        for b, m in enumerate(blocks):
            for i in range(m):
                self.table[b][i] = order.pop()
        self.k = torch.full((self.n_pages, Hkv, page, d), float("nan"))
        self.v = self.k.clone()
        for b, L in enumerate(self.lens):
            for i in range(blocks[b]):
                m = min(page, L - i * page)
                self.k[self.table[b][i], :, :m] = torch.randn(Hkv, m, d, generator=g)
                self.v[self.table[b][i], :, :m] = torch.randn(Hkv, m, d, generator=g)
        self.k, self.v = self.k.to(dtype).to(device), self.v.to(dtype).to(device)
        start = [head_rows]
        for n in ns:
            start.append(start[-1] + n)
        self.start, self.T = start, start[-1] + tail_rows
        i32 = dict(dtype=torch.int32, device=device)
        self.q_start, self.ctx = torch.tensor(start, **i32), torch.tensor(self.cs, **i32)
        self.block_table = torch.tensor(self.table, **i32)

    def randn(self, *shape, scale=1.0):
        return (torch.randn(*shape, generator=self.g) * scale).to(self.dtype).to(self.device)

    def rows(self, pages, b, h):
        """fp64 [L_b][d], on the CPU"""
        L = self.lens[b]
        if L == 0:
            return torch.zeros(0, self.d, dtype=torch.float64)
        used = self.table[b][:-(-L // self.page)]
        return torch.cat([pages[p, h].cpu() for p in used])[:L].double()


def attn(bt: Batch, q, scale):
    """out, mass [B][Hkv][slots] and the tolerances of both.

    A score s = scale q.k summed in fp32 is off by at most
    ds = (d + 4) u S, S = scale sum |q_c k_c|, u = 2^-24, twice that for a
    matrix unit that truncates; its weight by a factor e^+-2ds (numerator and
    sum), the exponential and the sum of L weights add (L + 16) u.  A weight
    rounded to bf16 is off by half a step of bf16, and the output by half a
    step of its type."""
    q = q.detach().cpu().double()
    T, Hq, d = q.shape
    G = Hq // bt.Hkv
    out = torch.full((T, Hq, d), float("nan"), dtype=torch.float64)
    tol = torch.zeros_like(out)
    S = bt.width * bt.page
    mass = torch.zeros(bt.B, bt.Hkv, S, dtype=torch.float64)
    mtol = torch.zeros_like(mass)
    for b in range(bt.B):
        n, c, r0, L = bt.ns[b], bt.cs[b], bt.start[b], bt.lens[b]
        if n == 0:
            continue
        sees = torch.arange(L)[None] <= c + torch.arange(n)[:, None]
        for h in range(bt.Hkv):
            k, v = bt.rows(bt.k, b, h), bt.rows(bt.v, b, h)
            for hq in range(h * G, (h + 1) * G):
                x = q[r0:r0 + n, hq]
                s = torch.where(sees, x @ k.T * scale, -math.inf)
                p = torch.softmax(s, -1)
                ds = 2 * (d + 4) * U_F32 * float((x.abs() @ k.abs().T).max()) * scale
                rel = 2 * ds + (L + 16) * U_F32
                o = p @ v
                w = p @ v.abs()
                out[r0:r0 + n, hq] = o
                bf = U_BF16 if bt.dtype == torch.bfloat16 else 0.0
                tol[r0:r0 + n, hq] = half_step(bt.dtype) * o.abs() + (rel + bf * (1 + rel)) * w * 1.01
                mass[b, h, :L] += p.sum(0)
                mtol[b, h, :L] += p.sum(0) * (rel + (n * G + 16) * U_F32) + 1e-30
    return out, tol, mass, mtol


def append(bt: Batch, qkv, Hq, inv_freq, positions, q_gain, k_gain, eps):
    """q [T][Hq][d], rotated k and v [T][Hkv][d] and the tolerance of q | k.

    The norm's factor is off by (d + 8) u, sine and cosine by 2 pi u (the
    angle's rounding) + 4 u, a rotation adds two roundings: all below
    (d + 40) u of the pair's size; then half a step of the type."""
    T = qkv.shape[0]
    d, Hkv = bt.d, bt.Hkv
    x = qkv.detach().cpu().double().view(T, Hq + 2 * Hkv, d)
    y = x[:, :Hq + Hkv].clone()
    if q_gain is not None:
        gain = torch.cat([q_gain.cpu().double().expand(Hq, d), k_gain.cpu().double().expand(Hkv, d)])
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * gain
    r2 = len(inv_freq)
    amp = y.abs().clone()
    a, b = y[..., :r2].clone(), y[..., r2:2 * r2].clone()
    ang = torch.tensor(positions, dtype=torch.float64)[:, None] * torch.tensor(inv_freq, dtype=torch.float64)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    y[..., :r2], y[..., r2:2 * r2] = a * c - b * s, b * c + a * s
    size = torch.sqrt(a * a + b * b)
    amp[..., :r2], amp[..., r2:2 * r2] = size, size
    tol = half_step(bt.dtype) * y.abs() + (d + 40) * U_F32 * amp * 1.01
    return y, x[:, Hq + Hkv:], tol


def evict(scores, L, top, recent):
    """Kept slots of one (sequence, head), ascending (a list)."""
    old = max(L - recent, 0)

    def key(i):
        s = float(scores[i])
        return (1, 0.0, i) if math.isnan(s) else (0, -s, i)
    best = sorted(range(old), key=key)[:top]
    return sorted(best) + list(range(old, L))


def close(got, want, tol, what):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - want).abs() > tol
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i]:.6g} for "
                             f"{want[i]:.6g} (tolerance {tol[i]:.2g})")
