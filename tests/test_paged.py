"""Paged cache on the CPU: refusals of every entry point (no GPU call is
made), the rotation table, the device checks and the division of ragged work
over CTAs, compiled for the host."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import paged_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def vc():
    from lossless_draft_verify_gb300 import build, vc
    build.build()
    vc.load()
    return vc


def _cache(vc, **kw):
    a = 1 << 20
    f = dict(k_pages=a, v_pages=a, block_table=a, status=a, B=2, Hkv=2, d=128, page=64, n_pages=10, max_blocks=4, dt=0)
    f.update(kw)
    return vc.PagedCacheC(*[f[n] for n, _ in vc.PagedCacheC._fields_])


A = 1 << 20
BIG = 1 << 34

BAD_CACHES = [(dict(k_pages=None), 1), (dict(v_pages=A + 8), 1), (dict(block_table=None), 1), (dict(status=None), 1),
              (dict(B=0), 1), (dict(Hkv=-1), 1), (dict(n_pages=0), 1), (dict(max_blocks=0), 1), (dict(dt=7), 1),
              (dict(page=0), 1), (dict(page=24), 2), (dict(page=8), 2), (dict(page=512), 2), (dict(d=96), 2),
              (dict(n_pages=1 << 30), 2), (dict(max_blocks=1 << 30), 2), (dict(B=1 << 28), 2)]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches_are_refused(vc, kw, want):
    L = vc.load()
    c = _cache(vc, **kw)
    rope = vc.vc_rope_init(64, 1e4)
    assert L.vc_paged_append(A, None, None, 1e-6, rope, None, A, A, 4, 4, c, A + 64, None) == want
    assert L.vc_paged_attn(A, c, A, A, 4, 4, 1.0, A + 64, A, BIG, None) == want
    assert L.vc_paged_attn_h2o(A, c, A, A, 4, 4, 1.0, A + 64, A, 1 << 30, A, BIG, None) == want
    assert L.vc_paged_attn_workspace_bytes(c, 4, 4) == 0 == L.vc_paged_attn_h2o_workspace_bytes(c, 4, 4)
    good = _cache(vc, **{k: v for k, v in kw.items() if k in ("B", "Hkv", "d", "dt")})
    for s, t in ((c, good), (good, c)):
        assert L.vc_paged_evict(A, 1 << 30, s, A, vc.DropCfg(4, 4), t, A + 64, A, 1 << 30, None, 0, None) in (1, 2)


def test_bad_arguments_are_refused(vc):
    L = vc.load()
    c = _cache(vc)
    rope = vc.vc_rope_init(128, 1e4)
    app = [A, None, None, 1e-6, rope, None, A, A, 4, 4, c, A + 4096, None]
    for i, x, want in [(0, None, 1), (0, A + 2, 1), (1, A, 1), (2, A, 1), (3, -1.0, 1), (3, math.nan, 1), (6, None, 1),
                       (7, None, 1), (8, -1, 1), (9, 0, 1), (9, 3, 1), (11, None, 1), (11, A, 1), (3, math.inf, 1),
                       (8, 1 << 29, 2)]:
        a = list(app)
        a[i] = x
        assert L.vc_paged_append(*a) == want, (i, x)
    assert L.vc_paged_append(*app[:4], None, *app[5:]) == 1
    assert L.vc_paged_append(*app[:4], rope, *app[5:10], _cache(vc, d=64), *app[11:]) == 1   # rotates past the head
    assert L.vc_paged_append(*app[:4], vc.Rope(), *app[5:]) == 1                              # not initialised
    need = L.vc_paged_attn_workspace_bytes(c, 4, 4)
    need2 = L.vc_paged_attn_h2o_workspace_bytes(c, 4, 4)
    assert 0 < need < need2
    at = [A, c, A, A, 4, 4, 1.0, A + 4096, A, need, None]
    for i, x, want in [(0, None, 1), (0, A + 8, 1), (2, None, 1), (3, None, 1), (4, -1, 1), (5, 0, 1), (5, 5, 1),
                       (6, -1.0, 1), (6, math.nan, 1), (6, math.inf, 1), (7, None, 1), (7, A + 4, 1), (8, None, 1),
                       (8, A + 16, 1), (9, need - 1, 1), (4, 1 << 29, 2), (5, 258, 2), (7, A, 1)]:
        a = list(at)
        a[i] = x
        assert L.vc_paged_attn(*a) == want, (i, x)
    assert L.vc_paged_attn_h2o(A, c, A, A, 4, 4, 1.0, A + 64, None, 256, A, need2, None) == 1
    assert L.vc_paged_attn_h2o(A, c, A, A, 4, 4, 1.0, A + 64, A, 255, A, need2, None) == 1      # fewer scores than slots
    assert L.vc_paged_attn_h2o(A, c, A, A, 4, 4, 1.0, A + 64, A, 256, A, need2 - 1, None) == 1
    # no rows: nothing to do, nothing enqueued
    assert L.vc_paged_attn(A, c, A, A, 0, 4, 1.0, A + 64, A, BIG, None) == 0
    assert L.vc_paged_append(*app[:8], 0, *app[9:]) == 0
    ev = [A, 256, c, A, vc.DropCfg(20, 10), c, A + 64, A, 30, A + 128, 30, None]
    for i, x in [(0, None), (1, 255), (3, None), (4, vc.DropCfg(-1, 0)), (4, vc.DropCfg(0, -1)), (6, None), (6, A),
                 (7, None), (8, 29), (9, A), (10, 29), (5, _cache(vc, d=64)), (5, _cache(vc, B=3)),
                 (5, _cache(vc, Hkv=1)), (5, _cache(vc, dt=1)), (5, _cache(vc, max_blocks=1, page=16))]:
        a = list(ev)
        a[i] = x
        assert L.vc_paged_evict(*a) == 1, (i, x)


def test_rope_tables(vc):
    L = vc.load()
    r = vc.Rope()
    for dim, theta in [(8, 1e4), (24, 1e4), (144, 1e4), (64, 0.0), (64, -1.0), (64, math.nan), (64, math.inf)]:
        assert L.vc_rope_init(r, dim, theta) == 1
    assert L.vc_rope_init(None, 64, 1e4) == 1
    bad = (ctypes.c_double * 8)(*([1.0] * 7 + [math.inf]))
    assert L.vc_rope_init_freqs(r, 16, bad) == 1 and L.vc_rope_init_freqs(r, 16, None) == 1
    got = vc.vc_rope_init(128, 5e5)
    for j in range(64):
        turns = 5e5 ** (-2.0 * j / 128) / (2 * math.pi)
        # fp64 of the frequency, and the step of the 64-bit fraction
        assert abs(got.turn[j] / 2.0 ** 64 - turns) <= 2.0 ** -52 * turns + 2.0 ** -64
    # whole turns drop out, negative frequencies wrap
    got = vc.vc_rope_init_freqs([2 * math.pi, -math.pi / 2] + [0.0] * 6)
    assert got.turn[0] == 0 and got.turn[1] == 3 << 62 and got.rotary_dim == 16


def test_a_scale_past_the_range_is_refused(vc):
    L = vc.load()
    c = _cache(vc)
    for scale, want in ((1.01e8, 2), (3e38, 2)):
        assert L.vc_paged_attn(A, c, A, A, 4, 4, scale, A + 4096, A, BIG, None) == want
        assert L.vc_paged_attn_h2o(A, c, A, A, 4, 4, scale, A + 4096, A, 256, A, BIG, None) == want
    assert L.vc_paged_attn(A, c, A, A, 0, 4, 1e8, A + 4096, A, BIG, None) == 0


def test_the_binding_refuses(vc):
    k = torch.zeros(4, 2, 16, 64)
    tab = torch.zeros(1, 2, dtype=torch.int32)
    c = vc.PagedCache(k, k.clone(), tab)
    assert c.slots == 32 and c.c.page == 16
    with pytest.raises(AssertionError):
        vc.PagedCache(k, k[:2], tab)
    with pytest.raises(AssertionError):
        vc.PagedCache(k, k.clone(), tab.long())
    i32 = dict(dtype=torch.int32)
    st, ctx = torch.tensor([0, 3], **i32), torch.tensor([5], **i32)
    ws = vc.Workspace(256, device="cpu")
    q = torch.zeros(3, 4, 64)
    with pytest.raises(ValueError):
        vc.vc_paged_attn(q, c, st, torch.zeros(2, **i32), 1.0, q.clone(), ws)
    with pytest.raises(TypeError):
        vc.vc_paged_attn(q, c, st.long(), ctx, 1.0, q.clone(), ws)
    with pytest.raises(TypeError):
        vc.vc_paged_attn(q.bfloat16(), c, st, ctx, 1.0, q.clone(), ws)
    with pytest.raises(ValueError):
        vc.vc_paged_attn(q.transpose(0, 1), c, st, ctx, 1.0, q.clone().transpose(0, 1), ws)
    with pytest.raises(ValueError):
        vc.vc_paged_attn_h2o(q, c, st, ctx, 1.0, q.clone(), torch.zeros(1, 1, 32), ws)
    with pytest.raises(ValueError):
        vc.vc_paged_append(torch.zeros(3, 7 * 64), c, st, ctx, q, vc.vc_rope_init(64, 1e4))
    with pytest.raises(TypeError):
        vc.vc_paged_append(torch.zeros(3, 8 * 64), c, st, ctx, q, vc.vc_rope_init(64, 1e4),
                           positions=torch.zeros(3))
    with pytest.raises(ValueError, match="not on a GPU"):
        vc.vc_paged_attn(q, c, st, ctx, 1.0, q.clone(), ws)
    with pytest.raises(ValueError):
        vc.vc_paged_evict(torch.zeros(1, 2, 32), c, ctx, 1, 1, c, torch.zeros(2, **i32), torch.zeros(1, 2, 2, **i32))


HOST = r"""
#include <array>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>
#include "paged.cuh"
using namespace vc::paged;
#define NEED(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } } while (0)

// every key tile of every unit falls to one CTA; a shared unit's parts sit in
// consecutive CTAs, the first in slot 1, the others in slot 0, no slot twice;
// small units are not shared
template <int BM, int BN> void division(std::mt19937 &r)
{
    const int B = 1 + r() % 12, G = 1 + r() % 9, Hkv = 1 + r() % 5, n_cta = r() % 2 ? 152 : 304, mode = r() % 4;
    std::vector<int32_t> qs(B + 1), cl(B);
    int T = 0;
    for (int b = 0; b < B; ++b) {
        qs[b] = T;
        const int n = r() % 5 == 0 ? 0 : mode == 0 ? 1 : mode == 1 ? r() % 3 : r() % 600;
        cl[b] = mode == 3 ? r() % 30000 : r() % 700;
        T += n;
    }
    qs[B] = T;
    int32_t status = 0;
    Pool P{};
    P.status = &status, P.B = B, P.Hkv = Hkv, P.page_log2 = 4, P.n_pages = 1, P.max_blocks = 1 << 20;
    WorkDim W{qs.data(), cl.data(), T, G};
    using U = Units<BM, BN>;
    auto seq = [&](int b) { return load_seq(P, W.q_start, W.ctx_len, T, b); };
    long total = 0;
    for (int b = 0; b < B; ++b) total += U::head_cost(seq(b), G) * Hkv;
    const long per = piece_len(total, n_cta, U::kMinPiece);
    std::map<std::tuple<int, int, int>, std::vector<std::array<int, 5>>> got;
    for (int c = 0; c < n_cta; ++c) {
        Piece p{};
        const long lo = per * c, hi = lmin(total, lo + per);
        if (lo < hi) {
            long before = 0;
            for (int b = 0; b < B; ++b) {
                const Seq s = seq(b);
                const long hc = U::head_cost(s, G);
                if (hc > 0 && before <= lo && lo < before + hc * Hkv) {
                    U::place(s, G, hc, lo - before, p);
                    p.b = b, p.len = hi - lo, p.per = per;
                }
                before += hc * Hkv;
            }
            NEED(p.len > 0);
        }
        Walk<BM, BN> w;
        w.start(P, W, p);
        Item it;
        int used[2] = {0, 0};
        while (w.next(P, W, it)) {
            const int slot = it.whole ? -1 : it.head ? 1 : 0;
            if (slot >= 0) NEED(used[slot]++ == 0);
            NEED(it.rows > 0 && it.rows <= BM);
            got[std::make_tuple(it.b, it.h, it.mt)].push_back(std::array<int, 5>{it.t_lo, it.t_hi, c, slot, it.parts});
        }
    }
    long units = 0;
    for (int b = 0; b < B; ++b)
        for (int h = 0; h < Hkv; ++h)
            for (int m = 0; m < U::mtiles(seq(b), G); ++m) {
                ++units;
                auto &v = got[std::make_tuple(b, h, m)];
                int at = 0;
                for (size_t i = 0; i < v.size(); ++i) {
                    NEED(v[i][0] == at);
                    at = v[i][1];
                    if (v.size() == 1) NEED(v[i][3] == -1);
                    if (v.size() > 1) NEED(v[i][3] == (i == 0) && v[i][2] == v[0][2] + (int)i);
                }
                if (v.size() > 1) NEED(v[0][4] == (int)v.size());
                if (U::cost(seq(b), G, m) <= U::kWhole) NEED(v.size() == 1);
                NEED(at == U::tiles(seq(b), G, m));
            }
    NEED(units == (long)got.size() && status == 0);
}

int main()
{
    std::mt19937 r(1);
    for (int i = 0; i < 400; ++i) {
        division<64, 32>(r);
        division<16, 64>(r);
        division<256, 128>(r);
    }
    // lengths that do not fit make the sequence empty and are reported
    const int32_t table[6] = {0, 2, 3, -1, 1, 1 << 30};
    int32_t status = 0;
    Pool P{};
    P.table = table, P.status = &status, P.B = 2, P.Hkv = 3, P.page_log2 = 4, P.n_pages = 3, P.max_blocks = 3;
    auto fits = [&](int a, int e, int ctx, int T) {
        const int32_t qs[2] = {a, e};
        status = 0;
        const Seq s = load_seq(P, qs, &ctx, T, 0);
        if (status) NEED(status == VC_PAGED_BAD_LENGTH && s.n == 0 && s.ctx == 0 && s.tok0 == 0);
        return status == 0;
    };
    NEED(fits(0, 0, 0, 0) && fits(0, 5, 43, 5) && fits(2, 2, 48, 5) && fits(0, 48, 0, 48));
    NEED(!fits(0, 5, 44, 5) && !fits(-1, 3, 0, 5) && !fits(3, 2, 0, 5) && !fits(0, 6, 0, 5) && !fits(0, 1, -1, 5));
    NEED(!fits(0, 1, 0x7fffffff, 5) && !fits(0x7fffffff, 0, 0, 5));
    // page numbers outside the pool are never used
    status = 0;
    NEED(P.page_of(0, 0) == 0 && P.page_of(0, 1) == 2 && P.page_of(1, 1) == 1 && status == 0);
    NEED(P.page_of(0, 2) == -1 && status == VC_PAGED_BAD_PAGE);
    status = 0;
    NEED(P.page_of(1, 0) == -1 && status == VC_PAGED_BAD_PAGE && P.page_of(1, 2) == -1);
    // rows past 2^31 elements
    NEED(P.row(1 << 26, 2, 15) == ((((size_t)1 << 26) * 3 + 2) << 4) + 15);
    std::printf("ok\n");
}
"""


def test_checks_and_division_on_the_host(tmp_path):
    from lossless_draft_verify_gb300 import build
    src = tmp_path / "paged_host.cu"
    src.write_text(HOST)
    exe = tmp_path / "paged_host"
    subprocess.run([build.nvcc(), "-std=c++17", "--expt-relaxed-constexpr", "-I", build.INCLUDE, "-I", build.CSRC,
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


def test_reference_against_itself():
    """The fp64 forms: attention weights sum to one per row, eviction keeps
    what sorting by hand keeps."""
    bt = paged_ref.Batch([3, 0, 1], [5, 2, 0], 2, 64, 16, torch.float32, device="cpu")
    q = bt.randn(4, 4, 64)
    out, tol, mass, _ = paged_ref.attn(bt, q, 0.125)
    assert torch.allclose(mass.sum(-1), torch.tensor([[6.0, 6.0], [0.0, 0.0], [2.0, 2.0]], dtype=torch.float64))
    assert torch.equal(out[3, 0], bt.rows(bt.v, 2, 0)[0])
    s = [1.0, math.nan, -0.0, 0.0, math.inf, -math.inf, 2.0, 9.0]
    assert paged_ref.evict(s, 8, 3, 1) == [0, 4, 6, 7]
    assert paged_ref.evict(s, 8, 4, 1) == [0, 2, 4, 6, 7]
    assert paged_ref.evict(s, 8, 6, 1) == [0, 2, 3, 4, 5, 6, 7]
    assert paged_ref.evict(s, 3, 9, 9) == [0, 1, 2] and paged_ref.evict(s, 8, 0, 0) == []
