// paged_mass_tc.cu -- the attention weight every slot of a paged bf16 cache
// receives from a ragged batch of chunks, on the tensor cores:
//
//   scores[b][h][j] += sum over the rows r = (i, g) that see slot j of
//       2^(scale' q_r . k_j - lse_r),   j <= ctx + i, lse from the attention.
//
// One fma gives the exponent where no |lse| of a row tile is above 2^20 (it is
// then off by 2^-5, lse's rounding, at most).  Above, the scaled score is rounded
// first, as it was for the row's maximum, so that no weight exceeds one whatever
// the scores' size (in every tile 3% more for the two chunks below).
//
// The product is taken transposed, S^T = K Q^T: a key is a row of the
// accumulator, so one thread holds all of a key's weights for 128 query rows
// and sums them without any exchange; every slot is owned by one thread and
// its sum has a fixed order.  A group of up to four key tiles of 128 stays in
// shared memory while the sequence's row tiles pass (a row tile is floor(128 / G)
// queries of the G heads, one TMA box), so K is read from HBM once and a row tile
// from L2 once per group.  With one row tile (decoding) this is a stream of K,
// bound by HBM; with many by the sums' arithmetic and waits: 156 us after the 230
// of the attention for two 512-token chunks over 16000 tokens, 32/8 heads, the
// tensor cores busy a third of it.
// A batch's groups all have one size, chosen by an estimate (find_share).  With
// the attention, in single calls, as chosen and with groups of 1, 2, 3, 4: two
// chunks of 512 over 16000 387 us and 521, 406, 382, 384; 512 over 8000 131 and
// 174, 144, 152, 131; 2048 over 8000 498 and 648, 534, 485, 532; four of 300 over
// 4000, 7 query heads to each of 8, 247 and 350, 275, 265, 244; a fresh prompt of
// 1500, 8/1 heads, 169 and 163, 181, 211, 254.  The last has 12 key tiles: work is
// not divided over rows, so most SMs are idle there.
//   warps 0-15      sums, four warps to a key tile of the group and to one of
//                   four accumulators;
//   warp 16         producer; warp 17 issues the MMAs.
#include "paged.cuh"
#include "tcgen05.cuh"

namespace vc {
namespace paged {
namespace {

constexpr int BN = 128;          // keys per tile
constexpr int kGroup = 4;        // key tiles of a group
constexpr int kThreads = 576;
constexpr int kProducer = 16, kIssuer = 17;     // warps
constexpr int kQStages = 2;

template <int D>
struct Geom {
    static constexpr int HALVES = D / 64;
    static constexpr int TILE = BN * D * 2;
    static constexpr int STAGES = kGroup * (128 / D);
    static constexpr int SM_Q = 0;
    static constexpr int SM_K = kQStages * TILE;
    static constexpr int SM_X = SM_K + STAGES * TILE;
    static constexpr int SMEM = SM_X + 16 * 512 + 1024;
};

// A CTA's share: groups of up to `size` key tiles, in the order sequence, head,
// group, each with the cost 4 row tiles + 1; a group belongs to the CTA in whose
// part of the total it begins.
struct MassWalk {
    int b, h, g;                 // next group
    int nt, mt, rt;              // of the sequence: key tiles, row tiles, rows per row tile
    int size;
    Seq s;
    long at, end;                // cost at the next group's beginning, end of the share

    static __device__ __forceinline__ long cost(int mt) { return 4l * mt + 1; }
    __device__ __forceinline__ int groups(int k) const { return (nt + k - 1) / k; }
    __device__ __forceinline__ void shape(const Pool &P, const WorkDim &W, int b_)
    {
        b = b_;
        s = load_seq(P, W.q_start, W.ctx_len, W.T, b);
        rt = BN / W.G * W.G;
        mt = (s.n * W.G + rt - 1) / rt;
        nt = mt > 0 ? (s.ctx + s.n + BN - 1) / BN : 0;
    }
};

struct MassItem {
    int b, h, key0, tiles;       // key tiles of the group
    int tok0, ctx, len, mt0, mt; // row tiles mt0 .. mt - 1 see the group
    int rows;
};

struct Shared {
    uint64_t k_full[2 * kGroup], k_empty[2 * kGroup], q_full[kQStages], q_empty[kQStages], s_full[4], s_free[4];
    uint32_t tmem;
    MassWalk start;
};

struct Params {
    Pool P;
    WorkDim W;
    const float *lse;
    float *scores;
    int32_t *status;
    int Hq, scores_stride, box_rows, n_rows, q_box;   // q_box: queries per row tile box
    float sl2;
};

// One warp finds where the CTA's share begins.  First the size of the groups, by
// an estimate: a round of a group of k tiles (a row tile's products and sums)
// takes about 0.7 + 0.4 k us, every group has the batch's average rounds (rows
// that see none of a group's keys counted too), and the CTA with the most groups
// is the last one.
__device__ __forceinline__ void find_share(const Params &A, int cta, int n_cta, MassWalk *out)
{
    const int lane = threadIdx.x & 31;
    MassWalk w;
    auto take = [&](int b0) {                          // the lane's sequence of 32
        if (b0 == 0 || b0 + lane >= A.P.B) w.nt = 0;
        if (b0 + lane < A.P.B) w.shape(A.P, A.W, b0 + lane);
    };
    float n[kGroup] = {}, c[kGroup] = {};              // groups, rounds
    for (int b0 = 0; b0 < A.P.B; b0 += 32) {
        take(b0);
        if (w.nt == 0) continue;
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
            const float x = (float)w.groups(k + 1) * A.P.Hkv;
            n[k] += x;
            c[k] += x * w.mt;
        }
    }
    int size = 1;
    float best = 0.f;
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            n[k] += __shfl_xor_sync(0xffffffffu, n[k], o);
            c[k] += __shfl_xor_sync(0xffffffffu, c[k], o);
        }
        const float t = n[k] > 0.f ? ceilf(n[k] / n_cta) * (c[k] / n[k]) * (7 + 4 * (k + 1)) : 0.f;
        if (k == 0 || t <= best) {
            best = t;
            size = k + 1;
        }
    }
    const bool few = A.P.B <= 32;                      // the lanes still hold them
    auto of = [&] { return w.nt > 0 ? (long)w.groups(size) * A.P.Hkv * MassWalk::cost(w.mt) : 0l; };
    long total = 0;
    for (int b0 = 0; b0 < A.P.B; b0 += 32) {
        if (!few) take(b0);
        long x = of();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        total += x;
    }
    const long per = (total + n_cta - 1) / n_cta, lo = per * cta, hi = lmin(total, lo + per);
    if (lane == 0) out->at = out->end = 0;
    __syncwarp();
    if (lo >= hi) return;
    long before = 0;
    for (int b0 = 0; b0 < A.P.B; b0 += 32) {
        if (!few) take(b0);
        const long x = of();
        long incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const long start = before + incl - x;
        if (x > 0 && start <= lo && lo < start + x) {
            // the first group that begins at lo or later (it may be the next sequence's first)
            const long cg = MassWalk::cost(w.mt), i = (lo - start + cg - 1) / cg;
            w.h = (int)(i / w.groups(size));
            w.g = (int)(i % w.groups(size));
            w.at = start + i * cg;
            w.end = hi;
            w.size = size;
            *out = w;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
}

__device__ __forceinline__ bool next_group(MassWalk &w, const Params &A, MassItem &it)
{
    while (w.at < w.end) {
        if (w.g * w.size >= w.nt) {
            w.g = 0;
            ++w.h;
        }
        if (w.nt == 0 || w.h >= A.P.Hkv) {
            if (w.b + 1 >= A.P.B) return false;
            w.shape(A.P, A.W, w.b + 1);
            w.h = w.g = 0;
            continue;
        }
        it.b = w.b;
        it.h = w.h;
        it.key0 = w.g * w.size * BN;
        it.tok0 = w.s.tok0;
        it.ctx = w.s.ctx;
        it.len = w.s.ctx + w.s.n;
        it.tiles = min(w.size, w.nt - w.g * w.size);
        it.rows = w.s.n * A.W.G;
        it.mt0 = (int)(lmax(it.key0 - w.s.ctx, 0) * A.W.G / w.rt);
        it.mt = w.mt;
        w.at += MassWalk::cost(w.mt);
        ++w.g;
        return true;
    }
    return false;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
mass_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ, Params A)
{
    using G = Geom<D>;
    constexpr int NST = G::STAGES;
    extern __shared__ __align__(1024) uint8_t sm[];
    float *s_lse = reinterpret_cast<float *>(sm + G::SM_X);  // [16 warps][128]: -lse
    Shared *S = reinterpret_cast<Shared *>(sm + G::SM_X + 16 * 512);
    static_assert(sizeof(Shared) <= 1024, "shared block");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    if (smem_u32(sm) & 1023u) {                              // never expected: the swizzled tiles need it
        if (threadIdx.x == 0) report_timeout(A.status, 110);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&S->k_full[i], 1);
            mbar_init(&S->k_empty[i], 1);
        }
        for (int i = 0; i < kQStages; ++i) {
            mbar_init(&S->q_full[i], 1);
            mbar_init(&S->q_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&S->s_full[i], 1);
            mbar_init(&S->s_free[i], 4);                     // the warps of a group of sums
        }
        fence_mbar_init();
    }
    if (warp == kIssuer) {
        tc::tmem_alloc(&S->tmem, 512);
        tc::tmem_relinquish();
    }
    if (warp == kProducer) find_share(A, blockIdx.x, gridDim.x, &S->start);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    pdl_trigger();
    const uint32_t tmem = S->tmem;
    const int rt = BN / A.W.G * A.W.G;                       // rows of a row tile
    MassWalk walk = S->start;
    MassItem it;

    if (warp == kProducer) {
        // ------------------------------------------------------- producer --
        const int boxes = BN / A.box_rows * G::HALVES;
        const int bp = lane / G::HALVES, half = lane % G::HALVES;
        const uint32_t q_bytes = (uint32_t)A.q_box * A.W.G * D * 2;
        Ring<NST> kr;
        Ring<kQStages> qr;
        bool ok = true, k_round = false, q_round = false;
        auto load_q = [&](int mt) {
            if (q_round) {
                if (lane == 0) ok = wait_bar(&S->q_empty[qr.slot], qr.phase ^ 1, A.status, 111);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) return;
            }
            if (lane == 0) {
                uint8_t *dst = sm + G::SM_Q + qr.slot * G::TILE;
                mbar_arrive_expect_tx(&S->q_full[qr.slot], q_bytes);
#pragma unroll
                for (int x = 0; x < G::HALVES; ++x)
                    tc::tma_load_3d(dst + x * (BN * 128), &tmQ, x * 64, it.h * A.W.G, it.tok0 + mt * (BN / A.W.G),
                                    &S->q_full[qr.slot]);
            }
            qr.next();
            q_round = q_round || qr.slot == 0;
        };
        while (ok && next_group(walk, A, it)) {
            load_q(it.mt0);
            for (int k = 0; k < it.tiles && ok; ++k) {
                const int slot = it.key0 + k * BN + bp * A.box_rows;
                int row = A.n_rows;                          // outside the map: zeros
                if (lane < boxes && slot < it.len) {
                    const int pg = A.P.page_of(it.b, slot >> A.P.page_log2);
                    if (pg >= 0) row = (int)A.P.row(pg, it.h, slot & (A.P.page() - 1));
                }
                if (k_round) {
                    if (lane == 0) ok = wait_bar(&S->k_empty[kr.slot], kr.phase ^ 1, A.status, 112);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&S->k_full[kr.slot], G::TILE);
                __syncwarp();
                if (lane < boxes)
                    tc::tma_load_3d(sm + G::SM_K + kr.slot * G::TILE + half * (BN * 128) + bp * A.box_rows * 128, &tmK,
                                    half * 64, row, 0, &S->k_full[kr.slot]);
                kr.next();
                k_round = k_round || kr.slot == 0;
            }
            for (int q = it.mt0 + 1; q < it.mt && ok; ++q) load_q(q);
        }
        if (!ok && lane == 0) {                              // copies in flight end before the CTA does
            for (int i = 0; i < NST; ++i)
                if (k_round || i < kr.slot) mbar_wait(&S->k_full[i], i < kr.slot ? kr.phase : kr.phase ^ 1);
            for (int i = 0; i < kQStages; ++i)
                if (q_round || i < qr.slot) mbar_wait(&S->q_full[i], i < qr.slot ? qr.phase : qr.phase ^ 1);
        }
    } else if (warp == kIssuer) {
        // -------------------------------------------------------- issuer --
        // The warp runs as one and an elected thread issues: operands that are
        // the same for the whole warp then stay in uniform registers.  All
        // tensor memory is this CTA's, so its addresses are constants.
        constexpr uint32_t hi = tc::desc_hi(1024, tc::kSwizzle128B), HALF = BN * 128 >> 4;
        const uint32_t k_lo = tc::desc_lo(smem_u32(sm + G::SM_K), 16), q_lo = tc::desc_lo(smem_u32(sm + G::SM_Q), 16);
        Ring<NST> k0;                                        // the group's first key tile
        Ring<kQStages> qr;
        uint32_t used[kGroup] = {};                          // rounds of each key tile's accumulator
        bool ok = tmem == 0;
        if (!ok) report_timeout(A.status, 109);              // never expected
        while (ok && next_group(walk, A, it)) {
            Ring<NST> kr = k0;
            for (int q = it.mt0; q < it.mt && ok; ++q) {
                ok = wait_warp(&S->q_full[qr.slot], qr.phase, A.status, 113);
                if (!ok) break;
                const int cols = min(rt, it.rows - q * rt);
                const uint32_t id = tc::idesc_bf16(BN, (cols + 15) / 16 * 16, false, false);
                const uint32_t bq = q_lo + qr.slot * (G::TILE >> 4);
                kr = k0;
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    if (k >= it.tiles) break;
                    ok = wait_warp(&S->k_full[kr.slot], kr.phase, A.status, 114) &&
                         (used[k] == 0 || wait_warp(&S->s_free[k], (used[k] - 1) & 1, A.status, 115));
                    if (!ok) break;
                    tc::fence_after();
                    const uint32_t ak = k_lo + kr.slot * (G::TILE >> 4), d = k * BN;
                    if (tc::elect()) {
                        tc::mma_ss2<false>(d, ak, hi, bq, hi, id);
#pragma unroll
                        for (int kk = 1; kk < D / 16; ++kk)
                            tc::mma_ss2<true>(d, ak + (kk >> 2) * HALF + (kk & 3) * 2, hi,
                                              bq + (kk >> 2) * HALF + (kk & 3) * 2, hi, id);
                        tc::commit(&S->s_full[k]);
                        if (q == it.mt - 1) tc::commit(&S->k_empty[kr.slot]);
                    }
                    ++used[k];
                    kr.next();
                }
                if (ok && tc::elect()) tc::commit(&S->q_empty[qr.slot]);
                qr.next();
            }
            k0 = kr;
        }
    } else {
        // ---------------------------------------------------------- sums --
        const int k = warp >> 2, wq = warp & 3;              // the warp's key tile of the group
        const uint32_t lanes = (uint32_t)(wq * 32) << 16;
        float *my_lse = s_lse + warp * BN;
        uint32_t used = 0;
        bool ok = true;
        int off[4];                                          // lse of the lane's rows in a row tile
#pragma unroll
        for (int x = 0; x < 4; ++x) off[x] = (lane + 32 * x) / A.W.G * A.Hq + (lane + 32 * x) % A.W.G;
        while (ok && next_group(walk, A, it)) {
            if (k >= it.tiles) continue;
            const int tile0 = it.key0 + k * BN, key = tile0 + wq * 32 + lane;
            float sum = 0.f;
            // lse of a row tile, four rows per lane, on its way a tile ahead
            float next[4];
            const float *lse = A.lse + (size_t)it.tok0 * A.Hq + it.h * A.W.G;
            auto fetch = [&](int q) {
                const float *p = lse + (size_t)q * (rt / A.W.G) * A.Hq;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int c = lane + 32 * x;
                    next[x] = c < rt && q * rt + c < it.rows ? p[off[x]] : 0.f;
                }
            };
            fetch(it.mt0);
            for (int q = it.mt0; q < it.mt && ok; ++q) {
                const int cols = min(rt, it.rows - q * rt);
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 4; ++x) my_lse[lane + 32 * x] = -next[x];
                const bool large = __any_sync(0xffffffffu, fmaxf(fmaxf(fabsf(next[0]), fabsf(next[1])),
                                                                 fmaxf(fabsf(next[2]), fabsf(next[3]))) > 0x1p20f);
                __syncwarp();
                if (q + 1 < it.mt) fetch(q + 1);
                ok = wait_warp(&S->s_full[k], used & 1, A.status, 116);
                ++used;
                if (!ok) break;
                tc::fence_after();
                // columns [lo, cols) see the key; [lo_all, cols) every key of the tile
                const int lo = min(max(max(key - it.ctx, 0) * A.W.G - q * rt, 0), BN);
                const int lo_all = min(max(max(tile0 + BN - 1 - it.ctx, 0) * A.W.G - q * rt, 0), BN);
                float2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
                const float2 sc = make_float2(A.sl2, A.sl2);
                const uint32_t tS = tmem + lanes + k * BN;
#pragma unroll 1
                for (int c0 = 0; c0 < cols; c0 += 32) {
                    uint32_t v[32];
                    tc::ld32(tS + c0, v);
                    tc::ld_wait();
                    if (c0 >= lo_all && c0 + 32 <= cols && !large) {
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 e = *reinterpret_cast<const float4 *>(my_lse + c0 + c);
                            const float2 x = fma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sc,
                                                  make_float2(e.x, e.y));
                            const float2 y = fma2(make_float2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])),
                                                  sc, make_float2(e.z, e.w));
                            acc[0] = add2(acc[0], make_float2(ex2(x.x), ex2(x.y)));
                            acc[1] = add2(acc[1], make_float2(ex2(y.x), ex2(y.y)));
                        }
                    } else {
                        // columns past the rows hold whatever was there: chosen, not multiplied away
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float p = ex2(__fadd_rn(__fmul_rn(__uint_as_float(v[c]), A.sl2), my_lse[c0 + c]));
                            if (c0 + c >= lo && c0 + c < cols) acc[0].x += p;
                        }
                        __syncwarp();
                    }
                }
                sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S->s_free[k]);
            }
            if (!ok) break;
            if (key < it.len) A.scores[((size_t)it.b * A.P.Hkv + it.h) * A.scores_stride + key] += sum;
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

template <int D>
cudaError_t launch(const Pool &P, const WorkDim &W, const void *q, int Hq, float sl2, const float *lse, float *scores,
                   int scores_stride, int32_t *status, cudaStream_t st)
{
    Params A;
    A.P = P;
    A.W = W;
    A.lse = lse;
    A.scores = scores;
    A.status = status;
    A.Hq = Hq;
    A.scores_stride = scores_stride;
    A.box_rows = std::min(1 << P.page_log2, BN);
    A.n_rows = (P.n_pages * P.Hkv) << P.page_log2;
    A.q_box = std::min(BN / W.G, W.T);
    A.sl2 = sl2;
    CUtensorMap mk, mq;
    const uint64_t bytes = (uint64_t)D * 2;
    if (!tma_map_bf16_3d(&mk, P.k, D, A.n_rows, 1, bytes, bytes * A.n_rows, 64, A.box_rows, 1) ||
        !tma_map_bf16_3d(&mq, q, D, Hq, W.T, bytes, bytes * Hq, 64, W.G, A.q_box))
        return cudaErrorInvalidValue;
    auto kern = mass_tc_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Geom<D>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(device_sm_count()), dim3(kThreads), Geom<D>::SMEM, st, mk, mq, A);
}

}  // namespace

cudaError_t mass_tc(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, const float *lse,
                    float *scores, int scores_stride, int32_t *status, cudaStream_t st)
{
    return d == 128 ? launch<128>(P, W, q, Hq, sl2, lse, scores, scores_stride, status, st)
                    : launch<64>(P, W, q, Hq, sl2, lse, scores, scores_stride, status, st);
}

}  // namespace paged
}  // namespace vc
