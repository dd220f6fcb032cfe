// paged_attn_tc.cu -- causal attention of ragged chunks over a paged bf16
// cache on the tensor cores (TMA, tcgen05, tensor memory).
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j), j <= ctx + i
//
// A unit (paged.cuh) is up to 256 (query, head) rows of one kv head against
// tiles of 128 keys.  A persistent CTA per SM walks its share of the batch:
//   warps 0-3, 4-7  softmax of stream 0 and 1, one thread per row;
//   warps 8, 10     producers: one TMA box per (page, 64 channels), into a ring
//                   of 128-key K and V tiles.  They share a tile's boxes, a
//                   lane each: one warp issues the 32 boxes of a K and V tile of
//                   16-slot pages too slowly (a decode step of 16 x 32768
//                   tokens 415 against 319 us, pages of 64 the same);
//   warp 9          issues the MMAs: S = Q K^T and O += P V, accumulators and
//                   P (bf16, over S's columns) in tensor memory.
// The two streams keep the tensor cores busy in turn: while stream 0 takes the
// exponentials of its S, stream 1's products run.  With more than 128 rows the
// streams are the unit's two row tiles, sharing every K/V tile; with fewer they
// take the key tiles alternately for the same rows and are merged at the end,
// so that a short unit, which HBM bounds, has both softmax groups on it.
// Measured, 32/8 heads of 128: a decode step of 16 x 32768 tokens 318 us = 6.75
// TB/s; 2048 tokens over 30000 785 to 805 us = 1.31 PFLOP/s at the power limit
// (735 in a short run below it), bound by a stream's chain S, softmax, P V.  Heads
// of 64: 204 us (5.3 TB/s) and 648.
//
// The running maximum is raised only when it grows by more than 2^8 (P and the
// sum then stay within fp32 and bf16 range), so O is rarely rescaled; the sum
// is taken over the unrounded exponentials, in fp32.  P is rounded to bf16 for
// the second product (half a step of bf16 per weight, the type the matrix unit
// takes), out once.
//
// With STORE the products q . k are written out too (fp32), for the attention
// mass of a batch of few rows: G scores of 4 bytes per key and kv head
// beside 4 d bytes of K and V, instead of a second read of K.
//
// V rows past the sequence's end may hold any bits and 0 * NaN is not 0: those
// that share the last page with tokens are cleared in shared memory, further
// pages are not read (their boxes lie outside the map and fill with zeros).
#include <type_traits>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace vc {
namespace paged {
namespace {

constexpr int BN = 128;
constexpr int kRowsTile = 128;
constexpr int kThreads = 352;
constexpr int kProducer = 8, kIssuer = 9, kProducer2 = 10;     // warps
constexpr int kSoftmax = 256;
constexpr int kSharedBytes = 3 << 10;                          // barriers, the roles' walks
constexpr float kLazy = 8.f;                                   // log2 domain

template <int D>
struct Geom {
    static constexpr int HALVES = D / 64;
    static constexpr int TILE = BN * D * 2;                  // bytes of a K or V tile (and of a Q row tile)
    static constexpr int STAGES = 5 * (128 / D);
    static constexpr int SM_Q = 0;
    static constexpr int SM_KV = 2 * TILE;
    static constexpr int SM_BAR = SM_KV + STAGES * TILE;
    static constexpr int SMEM = SM_BAR + kSharedBytes;
    static constexpr uint32_t COL_O = 256;                   // S0 | S1 | O0 | O1
};

struct Shared {
    uint64_t full[10], empty[10];
    uint64_t q_ready, s_full[2], p_ready[2], o_full[2], meet;
    uint32_t tmem;
    Piece piece;
    struct {
        Walk<256, BN> walk;
        Item it;
        bool more;
    } role[11];        // each warp's walk through the piece: in registers it would make the softmax threads spill
};

struct Params {
    Pool P;
    WorkDim W;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    float *lse_out;
    Parts parts;
    int32_t *status;
    float *s_out;                  // STORE: products of row r of q at s_out + r * s_stride
    long s_stride;
    int Hq, box_rows, n_rows;      // n_rows: rows of the pool's tensor map
    float sl2;
};

// The warp's next part; false at the end of the piece.  (Of a part, the ring
// holds K_0 (K_1), then V_i, K_{i + ahead}: the order in which the products
// need them.)
__device__ __forceinline__ bool step(Shared *S, int warp, const Params &A)
{
    auto &x = S->role[warp];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) x.more = x.walk.next(A.P, A.W, x.it);
    __syncwarp();
    return x.more;
}

template <int D, bool STORE>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, Params A)
{
    using G = Geom<D>;
    constexpr int NST = G::STAGES;
    extern __shared__ __align__(1024) uint8_t sm[];
    Shared *S = reinterpret_cast<Shared *>(sm + G::SM_BAR);
    static_assert(sizeof(Shared) <= kSharedBytes, "shared block");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    if (smem_u32(sm) & 1023u) {                              // never expected: the swizzled tiles need it
        if (threadIdx.x == 0) {
            report_timeout(A.status, 90);
            A.parts.desc[blockIdx.x].parts = 0;              // the merge reads it
        }
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&S->full[i], 1);
            mbar_init(&S->empty[i], 1);
        }
        mbar_init(&S->q_ready, kSoftmax);
        mbar_init(&S->meet, kSoftmax);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&S->s_full[t], 1);
            mbar_init(&S->p_ready[t], 128);
            mbar_init(&S->o_full[t], 1);
        }
        fence_mbar_init();
    }
    if (warp == kIssuer) {
        tc::tmem_alloc(&S->tmem, 512);
        tc::tmem_relinquish();
    }
    if (warp == kProducer) find_piece<256, BN>(A.P, A.W, blockIdx.x, gridDim.x, &S->piece);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    pdl_trigger();
    const uint32_t tmem = S->tmem;
    if (lane == 0) S->role[warp].walk.start(A.P, A.W, S->piece);

    if (warp == kProducer || warp == kProducer2) {
        // ------------------------------------------------------- producer --
        const Item &it = S->role[warp].it;
        if (lane == 0) {
            tc::prefetch_tmap(&tmK);
            tc::prefetch_tmap(&tmV);
        }
        // the two warps share a tile's boxes (at most 16), one to a lane
        const int boxes = BN / A.box_rows * G::HALVES, mine = (boxes + 1) / 2;
        const int box = (warp == kProducer2 ? mine : 0) + lane, bp = box / G::HALVES, half = box % G::HALVES;
        const bool on = lane < mine && box < boxes;
        Ring<NST> ring;
        bool ok = true, filled = false;                      // filled: the ring has been round once
        auto load = [&](const CUtensorMap *map, int row) {
            const int s = ring.slot;
            if (filled) {
                if (lane == 0) ok = wait_bar(&S->empty[s], ring.phase ^ 1, A.status, 91);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) return;
            }
            uint8_t *dst = sm + G::SM_KV + s * G::TILE;
            // (the other warp's boxes may land first: the phase ends with this arrival and all bytes)
            if (lane == 0 && warp == kProducer) mbar_arrive_expect_tx(&S->full[s], G::TILE);
            __syncwarp();
            if (on)
                tc::tma_load_3d(dst + half * (BN * 128) + bp * A.box_rows * 128, map, half * 64, row, 0, &S->full[s]);
            ring.next();
            filled = filled || ring.slot == 0;
        };
        while (ok && step(S, warp, A)) {
            const int n = it.t_hi - it.t_lo, len = it.ctx + it.n;
            const int ahead = it.rows > kRowsTile ? 1 : 2;
            // the lane's box of key tile i: its table entry is read some tiles
            // before it is looked at
            auto entry = [&](int i) {
                const int slot = (it.t_lo + i) * BN + bp * A.box_rows;
                return on && i < n && slot < len
                           ? A.P.table[(size_t)it.b * A.P.max_blocks + (slot >> A.P.page_log2)] : 0;
            };
            // past the sequence's end or through a bad page number: a row
            // outside the map, which fills with zeros
            auto row = [&](int i, int page) {
                const int slot = (it.t_lo + i) * BN + bp * A.box_rows;
                if (!on || slot >= len) return A.n_rows;
                if ((unsigned)page < (unsigned)A.P.n_pages)
                    return (int)A.P.row(page, it.h, slot & (A.P.page() - 1));
                set_flag(A.P.status, VC_PAGED_BAD_PAGE);
                return A.n_rows;
            };
            int e0 = entry(0), e1 = entry(1), e2 = entry(2);
            load(&tmK, row(0, e0));
            if (ok && ahead == 2 && n > 1) load(&tmK, row(1, e1));
            for (int i = 0; i < n && ok; ++i) {
                const int e3 = entry(i + 3);
                load(&tmV, row(i, e0));
                if (ok && i + ahead < n) load(&tmK, row(i + ahead, ahead == 1 ? e1 : e2));
                e0 = e1, e1 = e2, e2 = e3;
            }
        }
        if (!ok && lane == 0)                                // copies in flight end before the CTA does
            for (int i = 0; i < NST; ++i) {
                if (filled || i < ring.slot) mbar_wait(&S->full[i], i < ring.slot ? ring.phase : ring.phase ^ 1);
            }
    } else if (warp == kIssuer) {
        // -------------------------------------------------------- issuer --
        // The warp runs as one and an elected thread issues: operands that are
        // the same for the whole warp then stay in uniform registers.  All
        // tensor memory is this CTA's, so its addresses are constants.
        const Item &it = S->role[warp].it;
        constexpr uint32_t idS = tc::idesc_bf16(kRowsTile, BN, false, false);
        constexpr uint32_t idO = tc::idesc_bf16(kRowsTile, D, false, true);
        constexpr uint32_t hi = tc::desc_hi(1024, tc::kSwizzle128B), HALF = BN * 128 >> 4;
        const uint32_t kv_lo = tc::desc_lo(smem_u32(sm + G::SM_KV), BN * 128), q_lo = tc::desc_lo(smem_u32(sm), 16);
        Ring<NST> ring;
        uint32_t units = 0, ready[2] = {0, 0};               // q_ready, p_ready phases
        bool ok = tmem == 0;
        if (!ok) report_timeout(A.status, 89);               // never expected
        auto arrived = [&](const Ring<NST> &x) { return wait_warp(&S->full[x.slot], x.phase, A.status, 92); };
        auto release = [&]() {                               // once the products issued so far are done
            if (tc::elect()) tc::commit(&S->empty[ring.slot]);
            ring.next();
        };
        // S of stream T: row tile QT against a K tile
        auto issue_S = [&](auto T, auto QT, int slot) {
            const uint32_t a = q_lo + QT * (G::TILE >> 4), k = kv_lo + slot * (G::TILE >> 4);
            if (tc::elect()) {
                tc::mma_ss2<false>(T * BN, a, hi, k, hi, idS);
#pragma unroll
                for (int kk = 1; kk < D / 16; ++kk)
                    tc::mma_ss2<true>(T * BN, a + (kk >> 2) * HALF + (kk & 3) * 2, hi, k + (kk >> 2) * HALF + (kk & 3) * 2,
                                      hi, idS);
                tc::commit(&S->s_full[T]);
            }
        };
        auto issue_PV = [&](auto T, int slot, bool first, bool last) {
            constexpr uint32_t d = G::COL_O + T * D, p = T * BN;
            const uint32_t v = kv_lo + slot * (G::TILE >> 4);
            if (tc::elect()) {
                tc::mma_ts2(d, p, v, hi, idO, first ? 0u : 1u);
#pragma unroll
                for (int kk = 1; kk < BN / 16; ++kk) tc::mma_ts2(d, p + kk * 8, v + kk * (2048 >> 4), hi, idO, 1u);
                if (last) tc::commit(&S->o_full[T]);
            }
        };
        using C0 = std::integral_constant<int, 0>;
        using C1 = std::integral_constant<int, 1>;
        auto p_wait = [&](auto T) {
            const bool r = wait_warp(&S->p_ready[T], ready[T] & 1, A.status, 93);
            ++ready[T];
            tc::fence_after();
            return r;
        };
        while (ok && step(S, warp, A)) {
            const int n = it.t_hi - it.t_lo;
            ok = wait_warp(&S->q_ready, units & 1, A.status, 94);
            ++units;
            tc::fence_after();
            ok = ok && arrived(ring);
            if (!ok) break;
            if (it.rows > kRowsTile) {
                // the streams are two row tiles on the same keys
                issue_S(C0{}, C0{}, ring.slot);
                issue_S(C1{}, C1{}, ring.slot);
                release();
                for (int j = 0; j < n; ++j) {
                    const bool more = j + 1 < n;
                    const Ring<NST> k = ring.after();        // K_{j+1}, after V_j
                    ok = arrived(ring) && (!more || arrived(k)) && p_wait(C0{});
                    if (!ok) break;
                    issue_PV(C0{}, ring.slot, j == 0, !more);
                    if (more) issue_S(C0{}, C0{}, k.slot);
                    ok = p_wait(C1{});
                    if (!ok) break;
                    issue_PV(C1{}, ring.slot, j == 0, !more);
                    release();
                    if (more) {
                        issue_S(C1{}, C1{}, ring.slot);
                        release();
                    }
                }
            } else {
                // the streams take the key tiles of one row tile in turn
                issue_S(C0{}, C0{}, ring.slot);
                release();
                if (n > 1) {
                    ok = arrived(ring);
                    if (!ok) break;
                    issue_S(C1{}, C0{}, ring.slot);
                    release();
                }
                auto one = [&](auto T, int j) {
                    ok = arrived(ring) && p_wait(T);
                    if (!ok) return;
                    issue_PV(T, ring.slot, j < 2, j + 2 >= n);
                    release();
                    if (j + 2 < n) {
                        ok = arrived(ring);
                        if (!ok) return;
                        issue_S(T, C0{}, ring.slot);
                        release();
                    }
                };
                for (int j = 0; j < n && ok; j += 2) {
                    one(C0{}, j);
                    if (ok && j + 1 < n) one(C1{}, j + 1);
                }
            }
        }
    } else {
        // ------------------------------------------------------- softmax --
        const Item &it = S->role[warp].it;
        const int t = warp >> 2;                             // stream
        const int r = threadIdx.x & 127;                     // row of the stream's tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + t * BN;
        uint32_t steps = 0, units[2] = {0, 0}, met = 0;      // s_full, o_full and meet phases
        uint32_t item = 0;                                   // ring items of the parts before this one
        bool ok = true;
        auto meet = [&](int where) {                         // both softmax groups
            mbar_arrive(&S->meet);
            const bool r = wait_warp(&S->meet, met & 1, A.status, where);
            ++met;
            return r;
        };
        // the streams' (m, l) where the second row tile's Q would be
        float2 *ml_x = reinterpret_cast<float2 *>(sm + G::SM_Q + G::TILE);
        if (threadIdx.x == 0) A.parts.desc[blockIdx.x].parts = 0;
        while (ok && step(S, warp, A)) {
            const int n = it.t_hi - it.t_lo, len = it.ctx + it.n;
            const bool big = it.rows > kRowsTile;
            const int row0 = it.mt * 256;
            auto out_row = [&](int rr) {                     // row of q, out and lse_out
                const int R = row0 + rr;
                return (size_t)(it.tok0 + R / A.W.G) * A.Hq + it.h * A.W.G + R % A.W.G;
            };
            {
                // Q: big, the stream's tile; else each group half of the one tile
                constexpr int CH = D / 8, RP = 128 / CH;     // 16-byte chunks per row, rows per pass
                const int c = r % CH, q0 = r / CH;
                uint8_t *sQ = sm + G::SM_Q + (big ? t * G::TILE : 0);
                const int lo = big ? 0 : t * 64, cnt = big ? 128 : 64, base = big ? t * 128 : 0;
#pragma unroll 1
                for (int i0 = q0; i0 < cnt; i0 += 8 * RP) {
                    uint4 x[8];                              // eight loads in flight
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int rr = lo + i0 + e * RP;
                        x[e] = make_uint4(0, 0, 0, 0);
                        if (i0 + e * RP < cnt && base + rr < it.rows)
                            x[e] = *reinterpret_cast<const uint4 *>(A.q + out_row(base + rr) * D + c * 8);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int rr = lo + i0 + e * RP;
                        if (i0 + e * RP < cnt)
                            *reinterpret_cast<uint4 *>(sQ + (c >> 3) * (BN * 128) + rr * 128 +
                                                       (((c & 7) ^ (rr & 7)) << 4)) = x[e];
                    }
                }
                fence_async_smem();
                tc::fence_before();
                mbar_arrive(&S->q_ready);
                __syncwarp();
            }
            const int R = (big ? t * 128 : 0) + r;           // row within the unit
            const bool valid = R < it.rows;
            const int kmax = valid ? it.ctx + (row0 + R) / A.W.G : -1;
            // keys every row of the tile sees
            const int kall = it.ctx + (row0 + (big ? t * 128 : 0)) / A.W.G;
            float *s_row = STORE && valid ? A.s_out + (long)out_row(R) * A.s_stride : nullptr;
            float m = kLowestProduct, l = 0.f;               // m: of the products
            const int mine = big ? n : (n + 1 - t) / 2;      // this stream's steps
            // V rows of the last page past the sequence's end, before the product
            // with key tile i (big: stream 0's comes first)
            auto zero_tail = [&](int i) {
                const int key0 = (it.t_lo + i) * BN;
                if (i != n - 1 || key0 + BN <= len || (big && t == 1)) return;
                const uint32_t vi = item + 2u * n - 1;       // the part's last ring item
                ok = wait_warp(&S->full[vi % NST], (vi / NST) & 1, A.status, 96);
                uint8_t *sV = sm + G::SM_KV + (vi % NST) * G::TILE;
                const int page = A.P.page();
                const int z0 = len - key0, z1 = ok ? min(BN, (len + page - 1) / page * page - key0) : 0;
                for (int x = r; x < (z1 - z0) * (D / 8); x += 128) {
                    const int row = z0 + x / (D / 8), c = x % (D / 8);
                    *reinterpret_cast<uint4 *>(sV + (c >> 3) * (BN * 128) + row * 128 + (c & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
            };
            // a warp without a row of the unit (most, where a token decodes)
            // keeps the barriers' count; the P it leaves makes rows of O that
            // nobody reads
            const bool live = __any_sync(0xffffffffu, valid);
            for (int j = 0; j < mine && !live; ++j) {
                ok = wait_warp(&S->s_full[t], steps & 1, A.status, 95);
                ++steps;
                if (!ok) break;
                zero_tail(big ? j : 2 * j + t);
                mbar_arrive(&S->p_ready[t]);
            }
            for (int j = 0; j < mine && live; ++j) {
                const int i = big ? j : 2 * j + t;           // key tile of the part
                const int key0 = (it.t_lo + i) * BN;
                ok = wait_warp(&S->s_full[t], steps & 1, A.status, 95);
                ++steps;
                if (!ok) break;
                tc::fence_after();
                const bool cut = key0 + BN - 1 > kall;       // some row does not see all keys
                // a score chunk: 32 keys of the row, those it does not see at -inf
                auto chunk = [&](int h, uint32_t (&u)[32]) {
                    if (!cut) return;
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (key0 + h * 32 + c > kmax) u[c] = 0xff800000u;
                };
                // Exponentials against the running maximum as it stands, the
                // tile's maximum in the same pass.  Where it has grown by more
                // than 2^8 (a first tile, and rarely after it) O is rescaled
                // and the pass repeated; P is stored once it holds.
                uint32_t pk[64];
                float2 sum[2];
                for (;;) {
                    const float2 sc = make_float2(A.sl2, A.sl2), nm = make_float2(-m, -m);
                    sum[0] = sum[1] = make_float2(0.f, 0.f);
                    float top[2] = {kLowestProduct, kLowestProduct};
                    uint32_t u[2][32];
                    tc::ld32(tS, u[0]);
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        tc::ld_wait();
                        if (h < 3) tc::ld32(tS + (h + 1) * 32, u[(h + 1) & 1]);
                        uint32_t (&v)[32] = u[h & 1];
                        if constexpr (STORE) {
                            if (valid) {
                                float *dst = s_row + key0 + h * 32;
#pragma unroll
                                for (int c = 0; c < 32; c += 4)
                                    *reinterpret_cast<uint4 *>(dst + c) = make_uint4(v[c], v[c + 1], v[c + 2], v[c + 3]);
                            }
                            __syncwarp();
                        }
                        chunk(h, v);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 s = make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                            top[e & 1] = fmaxf(top[e & 1], fmaxf(s.x, s.y));
                            // the difference first: zero at the maximum however large the
                            // scores, where an fma would leave the rounding of m * scale (and
                            // take 1 to 2% less on prompts; the fma in warps without large
                            // scores only takes 10% more)
                            const float2 x = mul2(add2(s, nm), sc);
                            const float2 p = make_float2(ex2(x.x), ex2(x.y));
                            sum[e & 1] = add2(sum[e & 1], p);
                            const __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
                            pk[16 * h + e] = *reinterpret_cast<const uint32_t *>(&b);
                        }
                    }
                    const float mx = fmaxf(top[0], top[1]);
                    const bool grown = (mx - m) * A.sl2 > kLazy;
                    if (!__any_sync(0xffffffffu, grown)) break;
                    float alpha = 1.f;
                    if (grown) {
                        alpha = ex2((m - mx) * A.sl2);
                        m = mx;
                    }
                    l *= alpha;
                    // the stream's previous O += P V came before this S in the
                    // issue order, so it is complete
                    if (j > 0) {
#pragma unroll 1
                        for (int h = 0; h < D; h += 32) {
                            uint32_t o[32];
                            const uint32_t tO = tmem + lanes + G::COL_O + t * D + h;
                            tc::ld32(tO, o);
                            tc::ld_wait();
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                            tc::st32(tO, o);
                        }
                    }
                }
                tc::st32(tS, reinterpret_cast<uint32_t (&)[32]>(pk[0]));
                tc::st32(tS + 32, reinterpret_cast<uint32_t (&)[32]>(pk[32]));
                const float2 s2 = add2(sum[0], sum[1]);
                l += s2.x + s2.y;
                zero_tail(i);
                if (!ok) break;
                tc::st_wait();
                tc::fence_before();
                mbar_arrive(&S->p_ready[t]);
            }
            if (!ok) break;
            // ------------------------------------------------ output of the part --
            const size_t pr = A.parts.row(blockIdx.x, it.head ? 1 : 0, R);
            auto finish = [&](float M, float L, float w0, float w1, int c0, int c1) {
                // channels [c0, c1): w0 O_t (+ w1 O_1 of the merged streams)
                const float inv = it.whole ? 1.f / L : 1.f;
                const size_t row = valid ? out_row(R) : 0;
#pragma unroll 1
                for (int c = c0; c < c1 && live; c += 32) {
                    uint32_t o[32], o1[32];
                    __syncwarp();
                    tc::ld32(tmem + lanes + G::COL_O + (big ? t * D : 0) + c, o);
                    if (!big && n > 1) tc::ld32(tmem + lanes + G::COL_O + D + c, o1);
                    tc::ld_wait();
                    float x[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        x[e] = __uint_as_float(o[e]) * w0;
                        if (!big && n > 1) x[e] = fmaf(__uint_as_float(o1[e]), w1, x[e]);
                    }
                    if (valid && it.whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const __nv_bfloat162 b = __floats2bfloat162_rn(x[e + 2 * k] * inv, x[e + 2 * k + 1] * inv);
                                w[k] = *reinterpret_cast<const uint32_t *>(&b);
                            }
                            *reinterpret_cast<uint4 *>(A.out + row * D + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else if (valid) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(A.parts.o + pr * D + c + e) =
                                make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                    }
                }
                if (valid && c0 == 0) {
                    if (!it.whole) A.parts.ml[pr] = make_float2(M, L);
                    else if (A.lse_out) A.lse_out[row] = M + log2f(L);
                }
            };
            if (big) {
                ok = wait_warp(&S->o_full[t], units[t] & 1, A.status, 97);
                ++units[0], ++units[1];
                if (!ok) break;
                tc::fence_after();
                finish(m * A.sl2, l, 1.f, 0.f, 0, D);
            } else {
                ml_x[t * kRowsTile + r] = make_float2(m * A.sl2, l);
                ok = wait_warp(&S->o_full[0], units[0] & 1, A.status, 98) &&
                     (n == 1 || wait_warp(&S->o_full[1], units[1] & 1, A.status, 99));
                ++units[0];
                if (n > 1) ++units[1];
                ok = ok && meet(100);
                if (!ok) break;
                tc::fence_after();
                const float2 a = ml_x[r], b = ml_x[kRowsTile + r];
                const float M = fmaxf(a.x, b.x), w0 = ex2(a.x - M), w1 = ex2(b.x - M);
                finish(M, fmaf(a.y, w0, b.y * w1), w0, w1, t * (D / 2), (t + 1) * (D / 2));
                tc::fence_before();
                ok = meet(101);                              // O and the (m, l) are free again
                if (!ok) break;
                tc::fence_after();
            }
            if (!it.whole && it.head && threadIdx.x == 0) {
                PartDesc &d = A.parts.desc[blockIdx.x];
                d.parts = it.parts;
                d.tok0 = it.tok0;
                d.h = it.h;
                d.row0 = row0;
                d.rows = it.rows;
            }
            item += 2u * n;
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == kIssuer) {
        __syncwarp();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int D, bool STORE>
cudaError_t launch(const Pool &P, const WorkDim &W, const void *q, int Hq, float sl2, void *out, float *lse,
                   float *s_out, long s_stride, const Parts &parts, int32_t *status, cudaStream_t st)
{
    Params A;
    A.P = P;
    A.W = W;
    A.q = (const __nv_bfloat16 *)q;
    A.out = (__nv_bfloat16 *)out;
    A.lse_out = lse;
    A.parts = parts;
    A.status = status;
    A.s_out = s_out;
    A.s_stride = s_stride;
    A.Hq = Hq;
    A.box_rows = std::min(1 << P.page_log2, BN);
    A.n_rows = (P.n_pages * P.Hkv) << P.page_log2;
    A.sl2 = std::max(sl2, 1e-38f);     // a masked product is -inf; times zero it would be NaN
    CUtensorMap mk, mv;
    const uint64_t bytes = (uint64_t)D * 2;
    if (!tma_map_bf16_3d(&mk, P.k, D, A.n_rows, 1, bytes, bytes * A.n_rows, 64, A.box_rows, 1) ||
        !tma_map_bf16_3d(&mv, P.v, D, A.n_rows, 1, bytes, bytes * A.n_rows, 64, A.box_rows, 1))
        return cudaErrorInvalidValue;
    auto kern = attn_tc_kernel<D, STORE>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Geom<D>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(tc_ctas()), dim3(kThreads), Geom<D>::SMEM, st, mk, mv, A);
}

}  // namespace

int tc_ctas() { return device_sm_count(); }

cudaError_t attn_tc(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, void *out, float *lse,
                    float *s_out, long s_stride, const Parts &parts, int32_t *status, cudaStream_t st)
{
    if (s_out)
        return d == 128 ? launch<128, true>(P, W, q, Hq, sl2, out, lse, s_out, s_stride, parts, status, st)
                        : launch<64, true>(P, W, q, Hq, sl2, out, lse, s_out, s_stride, parts, status, st);
    return d == 128 ? launch<128, false>(P, W, q, Hq, sl2, out, lse, nullptr, 0, parts, status, st)
                    : launch<64, false>(P, W, q, Hq, sl2, out, lse, nullptr, 0, parts, status, st);
}

}  // namespace paged
}  // namespace vc
