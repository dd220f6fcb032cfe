"""The 8-bit paged cache and shared prefixes on the CPU: refusals of every entry
point (no GPU call is made), the plain forms against torch's types, and the
division of planned and few-row batches over CTAs, compiled for the host."""
import math
import subprocess

import pytest
import torch

import paged8_ref



@pytest.fixture(scope="module")
def vc():
    from lossless_draft_verify_gb300 import build, vc
    build.build()
    vc.load()
    return vc


A = 1 << 20
BIG = 1 << 34


def _cache8(vc, **kw):
    f = dict(k_pages=A, v_pages=A, k_scale=A, v_scale=A, block_table=A, status=A, B=2, Hkv=2, d=128, page=64, n_pages=10,
             max_blocks=4, dt=0)
    f.update(kw)
    return vc.Paged8CacheC(*[f[n] for n, _ in vc.Paged8CacheC._fields_])


def _cache(vc, **kw):
    f = dict(k_pages=A, v_pages=A, block_table=A, status=A, B=2, Hkv=2, d=128, page=64, n_pages=10, max_blocks=4, dt=0)
    f.update(kw)
    return vc.PagedCacheC(*[f[n] for n, _ in vc.PagedCacheC._fields_])


BAD = [(dict(k_pages=None), 1), (dict(v_pages=A + 8), 1), (dict(block_table=None), 1), (dict(status=None), 1),
       (dict(B=0), 1), (dict(Hkv=-1), 1), (dict(n_pages=0), 1), (dict(max_blocks=0), 1), (dict(dt=7), 1),
       (dict(page=0), 1), (dict(page=24), 2), (dict(page=8), 2), (dict(page=512), 2), (dict(d=96), 2),
       (dict(n_pages=1 << 30), 2), (dict(max_blocks=1 << 30), 2), (dict(B=1 << 28), 2)]
BAD8 = BAD + [(dict(k_scale=None), 1), (dict(v_scale=None), 1), (dict(k_scale=A + 8), 1), (dict(v_scale=A + 1), 1)]


@pytest.mark.parametrize("kw,want", BAD8)
def test_bad_8_bit_caches_are_refused(vc, kw, want):
    L = vc.load()
    c, g = _cache8(vc, **kw), vc.SharedPrefixC(A, A, 1)
    rope = vc.vc_rope_init(64, 1e4)
    assert L.vc_paged8_append(A, None, None, 1e-6, rope, None, A, A, 4, 4, c, A + 64, None) == want
    assert L.vc_paged8_read(c, A, A, 4, A, A + 64, None) == want
    assert L.vc_paged8_attn(A, c, A, A, 4, 4, 1.0, A + 64, A, BIG, None) == want
    assert L.vc_paged8_attn_shared(A, c, g, A, A, 4, 4, 1.0, A + 64, A, BIG, None) == want
    assert L.vc_paged8_attn_workspace_bytes(c, 4, 4) == 0 == L.vc_paged8_attn_shared_workspace_bytes(c, 1, 4, 4)


@pytest.mark.parametrize("kw,want", BAD)
def test_bad_caches_of_a_shared_prefix_are_refused(vc, kw, want):
    L = vc.load()
    c, g = _cache(vc, **kw), vc.SharedPrefixC(A, A, 1)
    assert L.vc_paged_attn_shared(A, c, g, A, A, 4, 4, 1.0, A + 64, A, BIG, None) == want
    assert L.vc_paged_attn_shared_workspace_bytes(c, 1, 4, 4) == 0


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq", [(1, 2), (3, 14), (16, 8), (2, 256)])
def test_a_workspace_is_enough_for_fewer_rows(vc, B, Hq, d, dt):
    L = vc.load()
    c, c8 = _cache(vc, B=B, d=d, dt=dt), _cache8(vc, B=B, d=d, dt=dt)
    for size in (lambda T: L.vc_paged8_attn_workspace_bytes(c8, T, Hq),
                 lambda T: L.vc_paged8_attn_shared_workspace_bytes(c8, 3, T, Hq),
                 lambda T: L.vc_paged_attn_shared_workspace_bytes(c, 3, T, Hq)):
        need = [size(T) for T in [*range(1, 200), 1000, 4000, 20000]]
        assert need[0] > 0 and need == sorted(need)


def test_bad_arguments_are_refused(vc):
    L = vc.load()
    c, c8, rope = _cache(vc), _cache8(vc), vc.vc_rope_init(128, 1e4)
    assert L.vc_paged8_append(A, None, None, 1e-6, rope, None, A, A, 4, 4, None, A + 64, None) == 1
    assert L.vc_paged8_attn(A, None, A, A, 4, 4, 1.0, A + 64, A, BIG, None) == 1
    app = [A, None, None, 1e-6, rope, None, A, A, 4, 4, c8, A + 4096, None]
    for i, x, want in [(0, None, 1), (0, A + 2, 1), (1, A, 1), (2, A, 1), (3, -1.0, 1), (3, math.nan, 1), (4, None, 1),
                       (6, None, 1), (7, None, 1), (8, -1, 1), (9, 0, 1), (9, 3, 1), (11, None, 1), (11, A, 1),
                       (8, 1 << 29, 2)]:
        a = list(app)
        a[i] = x
        assert L.vc_paged8_append(*a) == want, (i, x)
    assert L.vc_paged8_append(*app[:8], 0, *app[9:]) == 0                    # no rows: nothing to do
    assert L.vc_paged8_append(*app[:10], _cache8(vc, d=64), *app[11:]) == 1     # rotates past the head
    read = [c8, A, A, 4, A, A + 4096, None]
    for i, x, want in [(0, None, 1), (1, None, 1), (2, None, 1), (3, -1, 1), (4, None, 1), (5, None, 1), (4, A + 8, 1),
                       (5, A, 1), (5, A + 4, 1), (3, (1 << 29) + 1, 2)]:
        a = list(read)
        a[i] = x
        assert L.vc_paged8_read(*a) == want, (i, x)
    assert L.vc_paged8_read(_cache8(vc, Hkv=1 << 20, B=1, n_pages=1), A, A, 1, A, A + 64, None) == 2
    assert L.vc_paged8_read(c8, A, A, 0, None, None, None) == 0
    for call, size, cache in ((L.vc_paged8_attn, L.vc_paged8_attn_workspace_bytes, c8),
                              (L.vc_paged8_attn_shared, L.vc_paged8_attn_shared_workspace_bytes, c8),
                              (L.vc_paged_attn_shared, L.vc_paged_attn_shared_workspace_bytes, c)):
        shared = call is not L.vc_paged8_attn
        need = size(cache, 1, 4, 4) if shared else size(cache, 4, 4)
        assert need > 0
        at = [A, cache, A, A, 4, 4, 1.0, A + 4096, A, need, None]

        def run(a, g=vc.SharedPrefixC(A, A, 1)):
            return call(*a[:2], g, *a[2:]) if shared else call(*a)
        for i, x, want in [(0, None, 1), (0, A + 8, 1), (2, None, 1), (3, None, 1), (4, -1, 1), (5, 0, 1), (5, 5, 1),
                           (6, -1.0, 1), (6, math.nan, 1), (6, math.inf, 1), (6, 1.01e8, 2), (7, None, 1), (7, A + 4, 1),
                           (7, A, 1), (8, None, 1), (8, A + 16, 1), (9, need - 1, 1), (4, 1 << 29, 2), (5, 258, 2)]:
            a = list(at)
            a[i] = x
            assert run(a) == want, (call, i, x)
        none = list(at)
        none[4] = 0
        assert run(none) == 0
        if shared:
            for g, want in [(vc.SharedPrefixC(None, A, 1), 1), (vc.SharedPrefixC(A, None, 1), 1),
                            (vc.SharedPrefixC(A + 2, A, 1), 1), (vc.SharedPrefixC(A, A, -1), 1),
                            (vc.SharedPrefixC(A, A, 1 << 30), 2)]:
                assert run(at, g) == want
            assert run(none, vc.SharedPrefixC(None, None, 0)) == 0
            assert call(*at[:2], None, *at[2:]) == 1
            big = list(at)
            big[4:6], big[9] = [(1 << 29) // 4 + 1, 4], 1 << 60
            assert run(big) == 2
            assert size(cache, -1, 4, 4) == 0 == size(None, 1, 4, 4)


def test_the_binding_refuses(vc):
    u8 = dict(dtype=torch.uint8)
    k, s = torch.zeros(4, 2, 16, 64, **u8), torch.full((4, 2, 16), 127, **u8)
    tab = torch.zeros(2, 2, dtype=torch.int32)
    c = vc.Paged8Cache(k, k.clone(), s, s.clone(), tab)
    assert c.slots == 32 and c.c.page == 16 and c.dtype == torch.bfloat16
    vc.Paged8Cache(k.view(torch.float8_e4m3fn), k.clone(), s.view(torch.float8_e8m0fnu), s, tab, torch.float32)
    for bad in ((k.float(), k, s, s, tab), (k, k[:2], s, s, tab), (k, k, s[:2], s, tab), (k, k, s.int(), s, tab),
                (k, k, s, s, tab.long()), (k.transpose(2, 3), k.transpose(2, 3), s, s, tab)):
        with pytest.raises(AssertionError):
            vc.Paged8Cache(*bad)
    with pytest.raises(TypeError):
        vc.Paged8Cache(k, k, s, s, tab, torch.float16)
    i32 = dict(dtype=torch.int32)
    st, ctx, ws = torch.tensor([0, 3, 3], **i32), torch.tensor([5, 0], **i32), vc.Workspace(256, device="cpu")
    first, pre = torch.tensor([0, 2], **i32), torch.tensor([5], **i32)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    full = vc.PagedCache(k.bfloat16(), k.bfloat16(), tab)
    for call, cache in ((vc.vc_paged_attn, c), (vc.vc_paged8_attn, full)):
        with pytest.raises(TypeError):
            call(q, cache, st, ctx, 1.0, q.clone(), ws)
    for call, cache in ((vc.vc_paged_attn_shared, c), (vc.vc_paged8_attn_shared, full)):
        with pytest.raises(TypeError):
            call(q, cache, first, pre, st, ctx, 1.0, q.clone(), ws)
    with pytest.raises(TypeError):
        vc.vc_paged_append(torch.zeros(3, 8 * 64, dtype=torch.bfloat16), c, st, ctx, q, vc.vc_rope_init(64, 1e4))
    with pytest.raises(TypeError):
        vc.vc_paged8_attn_workspace_bytes(full, 3, 4)
    for call, cache in ((vc.vc_paged_attn_shared, full), (vc.vc_paged8_attn_shared, c)):
        with pytest.raises(TypeError):
            call(q, cache, first.long(), pre, st, ctx, 1.0, q.clone(), ws)
        with pytest.raises(ValueError):
            call(q, cache, first, torch.zeros(2, **i32), st, ctx, 1.0, q.clone(), ws)
        with pytest.raises(ValueError, match="not on a GPU"):
            call(q, cache, first, pre, st, ctx, 1.0, q.clone(), ws)
    with pytest.raises(ValueError):
        vc.vc_paged8_attn(q, c, st, ctx[:1], 1.0, q.clone(), ws)
    with pytest.raises(TypeError):
        vc.vc_paged8_attn(q.float(), c, st, ctx, 1.0, q.clone(), ws)
    r = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        vc.vc_paged8_read(full, st, ctx, r, r.clone())
    with pytest.raises(ValueError):
        vc.vc_paged8_read(c, st, ctx, r, r[:2])
    with pytest.raises(TypeError):
        vc.vc_paged8_read(c, st, ctx, r.float(), r.float())
    with pytest.raises(ValueError, match="not on a GPU"):
        vc.vc_paged8_read(c, st, ctx, r, r.clone())


def test_the_plain_forms_are_those_of_the_types():
    """Every code stands for what torch's e4m3 says, values round as torch rounds
    them, and scales are the least that fit."""
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double()
    got = paged8_ref.decode(codes)
    assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(want, nan=1e9))
    g = torch.Generator().manual_seed(0)
    x = torch.randn(100000, generator=g) * torch.exp2(torch.randint(-12, 8, (100000,), generator=g).float())
    x = torch.cat([x.clamp(-448, 448), (want[:126] + want[1:127]).float() / 2, torch.tensor([448.0, 0.0, 2.0 ** -10])])
    assert torch.equal(paged8_ref.round_e4m3(x), x.to(torch.float8_e4m3fn).double())
    finite = want[~want.isnan()]
    assert torch.equal(paged8_ref.decode(paged8_ref.codes_of(finite)), finite)
    for amax, byte in ((448.0, 127), (448.1, 128), (224.0, 126), (1.0, 119), (0.0, 10), (1e-38, 10), (3.3e38, 246)):
        assert int(paged8_ref.scale_byte(torch.tensor(amax))) == byte
    big = torch.rand(1000, generator=g).double() * torch.exp2(torch.linspace(-100, 100, 1000).round().double())
    s = 2.0 ** (paged8_ref.scale_byte(big).double() - 127)
    assert (big <= 448 * s).all() and (big > 224 * s).all()


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

// Entries of a plan, the cost model C: every key tile of every unit falls to one
// CTA, a shared unit's parts sit in consecutive ones, no slot twice.
template <int BM, int BN, typename C> void division(std::mt19937 &r)
{
    const int n = 1 + r() % 12, G = 1 + r() % 9, Hkv = 1 + r() % 4, n_cta = r() % 2 ? 152 : 1824, mode = r() % 4;
    std::vector<VSeq> plan(n);
    int T = 0;
    for (int i = 0; i < n; ++i) {
        const int rows = r() % 5 == 0 ? 0 : mode == 0 ? 1 : mode == 1 ? r() % 3 : r() % 700, step = r() % 3 != 0;
        plan[i] = VSeq{T, rows, rows ? (int)(mode == 3 ? r() % 30000 : r() % 700) : 0, step, 0, i, T, 0};
        T += rows;
    }
    int32_t status = 0;
    Pool P{};
    P.status = &status, P.B = n, P.Hkv = Hkv, P.page_log2 = 4, P.n_pages = 1, P.max_blocks = 1 << 20;
    WorkDim W{nullptr, nullptr, T, G, plan.data(), n};
    using U = Units<BM, BN, C>;
    long total = 0;
    for (const VSeq &s : plan) {
        long c = 0;
        for (int m = 0; m < U::mtiles(s, G); ++m) c += U::cost(s, G, m);
        NEED(c == U::head_cost(s, G));
        total += c * Hkv;
        // the place of every cost unit near a boundary
        long x = 0;
        for (int m = 0; m < U::mtiles(s, G); ++m) {
            for (long o : {0l, (long)U::cost(s, G, m) / 2, (long)U::cost(s, G, m) - 1}) {
                Piece p{};
                U::place(s, G, c, x + o, p);
                NEED(p.h == 0 && p.mt == m && p.off == o);
            }
            x += U::cost(s, G, m);
        }
    }
    const long per = piece_len(total, n_cta, U::kMinPiece);
    std::map<std::tuple<int, int, int>, std::vector<std::array<int, 5>>> got;
    for (int c = 0; c < n_cta; ++c) {
        Piece p{};
        const long lo = per * c, hi = lmin(total, lo + per);
        if (lo < hi) {
            long before = 0;
            for (int b = 0; b < n; ++b) {
                const long hc = U::head_cost(plan[b], G);
                if (hc > 0 && before <= lo && lo < before + hc * Hkv) {
                    U::place(plan[b], G, hc, lo - before, p);
                    p.b = b, p.len = hi - lo, p.per = per;
                }
                before += hc * Hkv;
            }
            NEED(p.len > 0);
        }
        Walk<BM, BN, VSeq, C> w;
        w.start(P, W, p);
        ItemOf<VSeq> it;
        int used[2] = {0, 0};
        while (w.next(P, W, it)) {
            const int slot = it.whole ? -1 : it.head ? 1 : 0;
            if (slot >= 0) NEED(used[slot]++ == 0);
            NEED(it.rows > 0 && it.rows <= BM && it.out_tok0() == plan[it.b].tok0);
            NEED(c + it.parts <= n_cta && it.parts < 65536);
            const Place at = Place::in_parts(c, it.parts, BM - 1);
            NEED(at.cta() == c && at.parts() == it.parts && at.r == BM - 1);
            got[std::make_tuple(it.b, it.h, it.mt)].push_back(std::array<int, 5>{it.t_lo, it.t_hi, c, slot, it.parts});
        }
    }
    long units = 0;
    for (int b = 0; b < n; ++b)
        for (int h = 0; h < Hkv; ++h)
            for (int m = 0; m < U::mtiles(plan[b], G); ++m) {
                ++units;
                auto &v = got[std::make_tuple(b, h, m)];
                int at = 0;
                NEED(!v.empty());
                for (size_t i = 0; i < v.size(); ++i) {
                    NEED(v[i][0] == at);
                    at = v[i][1];
                    if (v.size() == 1) NEED(v[i][3] == -1);
                    if (v.size() > 1) NEED(v[i][3] == (i == 0) && v[i][2] == v[0][2] + (int)i);
                }
                if (v.size() > 1) NEED(v[0][4] == (int)v.size());
                if (U::cost(plan[b], G, m) <= U::kWhole) NEED(v.size() == 1);
                NEED(at == U::tiles(plan[b], G, m));
            }
    NEED(units == (long)got.size() && status == 0 && Place::in_output().parts() == 0);
}

int main()
{
    std::mt19937 r(1);
    for (int i = 0; i < 300; ++i) {
        division<8, 32, CostFew>(r);
        division<16, 32, CostFew>(r);
        division<8, 64, CostFew>(r);
        division<16, 16, CostFew>(r);
        division<8, 32, CostFewCut>(r);
        division<16, 64, CostFewCut>(r);
        division<256, 128, Cost<256>>(r);
        division<64, 32, Cost<64>>(r);
    }
    std::printf("ok\n");
}
"""


def test_division_on_the_host(tmp_path):
    from lossless_draft_verify_gb300 import build
    src = tmp_path / "paged8_host.cu"
    src.write_text(HOST)
    exe = tmp_path / "paged8_host"
    subprocess.run([build.nvcc(), "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-I", build.INCLUDE, "-I", build.CSRC,
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


PLACES = r"""
#include <cstdio>
#include <cstdlib>
#include "paged.cuh"
using namespace vc::paged;
#define NEED(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } } while (0)
int main()
{
    const Parts p{nullptr, nullptr, nullptr, 16, 1824};
    NEED(!Place::in_output().fits(p));
    NEED(Place::in_parts(0, 2, 0).fits(p) && Place::in_parts(1822, 2, 15).fits(p) && Place::in_parts(0, 1824, 3).fits(p));
    NEED(!Place::in_parts(1823, 2, 0).fits(p) && !Place::in_parts(0, 1825, 0).fits(p) && !Place::in_parts(5, 2, 16).fits(p));
    for (uint32_t x : {0x7f800000u, 0x7fc00000u, 0xffffffffu, 0x3f800000u, 0x00010720u, 0x40000001u})
        for (uint32_t r : {0u, 15u, 16u, 0xffffffffu, 0x80000000u}) {
            const Place at{x, r};
            NEED(!at.fits(p) || (at.cta() + at.parts() <= 1824 && at.parts() > 0 && r < 16));
        }
    std::printf("ok\n");
}
"""


def test_a_place_that_was_never_written_names_nothing_outside_the_parts(tmp_path):
    """After a wait that ran out the join finds whatever the workspace held."""
    from lossless_draft_verify_gb300 import build
    src, exe = tmp_path / "places.cu", tmp_path / "places"
    src.write_text(PLACES)
    subprocess.run([build.nvcc(), "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-I", build.INCLUDE, "-I", build.CSRC,
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
