// paged_attn8_few.cu -- causal attention over 8-bit pages for batches of few rows
// (decoding, drafting): up to 16 (query, head) rows per kv head.
//
//   out_i = sum_j p_ij 2^f_j v_j / sum_j p_ij,  p_ij = exp(scale 2^e_j q_i . k_j)
//
// with k_j, v_j the codes of key j and e_j, f_j its scales' exponents.  HBM bounds
// it, if the codes can be fed to the matrix units at that pace: 24 of them per SM
// and clock.  e4m3 numbers are f16 numbers and one instruction expands two; with the
// keys in the place of an MMA's 16 rows (S^T = K Q^T, O^T = V^T P^T) they go straight
// from the tile as it lies in memory to the operands, and a unit's 8 rows are the
// MMA's 8 columns:
//   K  a thread's four bytes of a row are two pairs of neighbouring channels; which
//      channels an MMA's k slots stand for is free, if Q has them alike;
//   V  operand pairs are two keys at one channel: byte permutes of two rows;
//   P  an 8 x 8 transpose between its place as result and as operand.
// The scales meet the products and the weights, not the codes.  The tensor-core kernel
// (paged_attn_tc.cuh) writes bf16 tiles to shared memory instead, which costs more
// than it saves where rows are few (a decode step of 16 x 32768 tokens, 32/8 heads:
// 392 us there).
//
// A warp is alone with its piece of the batch: it requests 16-key tiles by TMA some
// stages ahead, past a unit's end too, and needs no barrier but those of the copies.
//
// Ranges.  q is scaled to f16 by its row's largest exponent (an element is off by
// 2^-25 of the row's largest, at most).  The running maximum is raised when it has
// grown by more than 2^8, as in the tensor-core kernel.  The weights p 2^f, which
// become f16, are scaled by a power of two per row such that the largest so far lies
// at 2^6: what is lost below f16's smallest number is 2^-31 of it per key.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "paged8.cuh"
#include "tcgen05.cuh"

namespace vc {
namespace paged {
namespace {

constexpr int BN = kFewKeys;
constexpr int kWarps = kFewWarps, kStages = 4;
constexpr float kLazy = 8.f, kGrown = 512.f;                   // log2 domain; a weight above 2^kLazy beyond doubt
constexpr float kTop = 64.f, kMost = 32768.f;                  // where weights are put, and how far they may grow

template <int D>
struct Geom {
    static constexpr int TILE = BN * D;                        // bytes of a K or V tile
    static constexpr int STAGE = 2 * TILE;
    static constexpr int SM_WARP = kStages * STAGE;
};

template <int BM>
struct Warp {
    uint64_t full[kStages];
    alignas(16) uint8_t scale[kStages][2][BN];
    Piece piece;
    struct {
        Walk<BM, BN> walk;
        Item it;
        bool more;
    } ask, use;                        // the walk of the requests, and that of the arithmetic
};

struct Params {
    Pool P;
    WorkDim W;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    Parts parts;
    int32_t *status;
    int Hq, n_rows;
    float sl2;
};

__device__ __forceinline__ uint32_t half2_of(uint32_t codes)   // the low 16 bits
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// The 16-byte chunk `c` of row r of a tile, as the TMA's swizzle places it.
template <int D>
__device__ __forceinline__ uint4 chunk(const uint8_t *tile, int r, int c)
{
    const int s = D == 128 ? r & 7 : r >> 1 & 3;
    return *reinterpret_cast<const uint4 *>(tile + r * D + ((c ^ s) << 4));
}

// NB: blocks of 8 rows.  Lane 4 g + q holds, of S^T, keys g and g + 8 of rows 2 q
// and 2 q + 1 (of each block), of O^T channels D/8 g .. + D/8 - 1 of the same rows.
template <int D, int NB>
__global__ void __launch_bounds__(32 * kWarps, 1)
attn8_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, Params A)
{
    constexpr int BM = 8 * NB, KS = D / 16, MT = D / 16, KC = D / 64;    // k steps, m tiles, chunks of a K row per lane
    using G = Geom<D>;
    extern __shared__ __align__(1024) uint8_t sm[];
    __shared__ Warp<BM> warps[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
    Warp<BM> &S = warps[warp];
    uint8_t *tiles = sm + warp * G::SM_WARP;
    // neighbouring pieces on different SMs
    const int n_piece = gridDim.x * kWarps, me = warp * gridDim.x + blockIdx.x;
    pdl_wait();
    if (lane == 0) {
        A.parts.desc[me].parts = 0;
        for (int i = 0; i < kStages; ++i) mbar_init(&S.full[i], 1);
        fence_mbar_init();
    }
    find_piece<BM, BN>(A.P, A.W, me, n_piece, &S.piece);
    pdl_trigger();
    if (smem_u32(sm) & 1023u) {                              // never expected: the swizzled tiles need it
        if (lane == 0) report_timeout(A.status, 110);
        return;
    }
    if (S.piece.len <= 0) return;
    if (lane == 0) {
        S.ask.walk.start(A.P, A.W, S.piece);
        S.use.walk.start(A.P, A.W, S.piece);
        tc::prefetch_tmap(&tmK);
        tc::prefetch_tmap(&tmV);
    }
    auto step = [&](auto &x) {                               // the next part; false at the piece's end
        __syncwarp();
        if (lane == 0) x.more = x.walk.next(A.P, A.W, x.it);
        __syncwarp();
        return x.more;
    };

    // ---- requests: a tile's rows lie in one page, side by side ----
    Ring<kStages> ask;
    bool asking = true;
    int aj = 0, an = 0, page = 0, page_next = 0;             // of the part: tile, tiles; a lane's page numbers of 32 tiles
    auto request = [&]() {
        if (!asking) return;
        const Item &it = S.ask.it;
        auto entry = [&](int j) {
            return j < an ? A.P.table[(size_t)it.b * A.P.max_blocks + ((it.t_lo + j) * BN >> A.P.page_log2)] : 0;
        };
        if (aj == an) {
            asking = step(S.ask);
            if (!asking) return;
            aj = 0;
            an = it.t_hi - it.t_lo;
            page_next = entry(lane);
        }
        if ((aj & 31) == 0) {
            page = page_next;
            page_next = entry(aj + 32 + lane);
        }
        const int p = __shfl_sync(0xffffffffu, page, aj & 31);
        const bool ok = (unsigned)p < (unsigned)A.P.n_pages;
        const int row = ok ? (int)A.P.row(p, it.h, (it.t_lo + aj) * BN & (A.P.page() - 1)) : A.n_rows;   // outside: zeros
        uint64_t *bar = &S.full[ask.slot];
        uint8_t *dst = tiles + ask.slot * G::STAGE;
        if (lane == 0) {
            if (!ok) set_flag(A.P.status, VC_PAGED_BAD_PAGE);
            mbar_arrive_expect_tx(bar, G::STAGE + (ok ? 2 * BN : 0));
        }
        __syncwarp();
        if (lane == 0) tc::tma_load_3d(dst, &tmK, 0, row, 0, bar);
        if (lane == 1) tc::tma_load_3d(dst + G::TILE, &tmV, 0, row, 0, bar);
        if (lane == 2 && ok) bulk_g2s(S.scale[ask.slot][0], A.P.k_scale + row, BN, bar);
        if (lane == 3 && ok) bulk_g2s(S.scale[ask.slot][1], A.P.v_scale + row, BN, bar);
        ask.next();
        ++aj;
    };
    for (int i = 0; i < kStages; ++i) request();

    Ring<kStages> ring;
    bool fine = true;
    while (fine && step(S.use)) {
        const Item &it = S.use.it;
        const int n = it.t_hi - it.t_lo, len = it.len(), row0 = it.mt * BM;
        auto head_row = [&](int r) {                         // row of q and out
            const int R = row0 + r;
            return (size_t)(it.tok0 + R / A.W.G) * A.Hq + it.h * A.W.G + R % A.W.G;
        };
        // ---- Q: row g of each block, scaled to [1, 2) at its largest ----
        uint32_t b[NB][KS][2];
        float qs[NB][2];
        int kmax[NB][2];
#pragma unroll
        for (int x = 0; x < NB; ++x) {
            const bool on = 8 * x + g < it.rows;
            uint4 w[2 * KC] = {};
            const __nv_bfloat16 *src = A.q + (on ? head_row(8 * x + g) * D : 0);
#pragma unroll
            for (int i = 0; i < 2 * KC; ++i)
                if (on) w[i] = *reinterpret_cast<const uint4 *>(src + (i / 2) * 64 + q4 * 16 + (i % 2) * 8);
            uint32_t top = 0;                                // the largest magnitude's bits
#pragma unroll
            for (int i = 0; i < 2 * KC; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) top = max(top, max(u[e] & 0x7fffu, u[e] >> 16 & 0x7fffu));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t ex = min(max(top >> 7, 1u), 253u);
            const float inv = scale_of(254u - ex), back = scale_of(ex);
#pragma unroll
            for (int i = 0; i < 2 * KC; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)                  // chunk i holds k steps 2 i, 2 i + 1
                    b[x][2 * i + e / 2][e % 2] = pack_half2(bf16_lo(u[e]) * inv, bf16_hi(u[e]) * inv);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                qs[x][r] = __shfl_sync(0xffffffffu, back, 8 * q4 + 4 * r);
                const int R = 8 * x + 2 * q4 + r;
                kmax[x][r] = R < it.rows ? it.last((row0 + R) / A.W.G) : -1;
            }
        }
        const int kall = it.last(row0 / A.W.G);              // keys every row sees
        float o[NB][MT][4], m[NB][2], l[NB][2], put[NB][2], level[NB][2];
#pragma unroll
        for (int x = 0; x < NB; ++x) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x][t][e] = 0.f;
#pragma unroll
            for (int r = 0; r < 2; ++r) m[x][r] = kLowestProduct, l[x][r] = 0.f, put[x][r] = 1.f, level[x][r] = 0.f;
        }
        for (int i = 0; i < n; ++i) {
            const int key0 = (it.t_lo + i) * BN, live = len - key0;
            fine = wait_warp(&S.full[ring.slot], ring.phase, A.status, 111);
            if (!fine) break;
            const uint8_t *tK = tiles + ring.slot * G::STAGE, *tV = tK + G::TILE;
            const uint8_t *sc = S.scale[ring.slot][0];
            const float ks[2] = {scale_of(sc[g]), scale_of(sc[g + 8])};
            const float vs[2] = {g < live ? scale_of(sc[BN + g]) : 0.f, g + 8 < live ? scale_of(sc[BN + g + 8]) : 0.f};
            // ---- S^T = K Q^T ----
            float s[NB][4];
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[x][e] = 0.f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const uint4 lo = chunk<D>(tK, g, 4 * c + q4), hi = chunk<D>(tK, g + 8, 4 * c + q4);
                const uint32_t u[4] = {lo.x, lo.y, lo.z, lo.w}, v[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t a[4] = {half2_of(u[e]), half2_of(v[e]), half2_of(u[e] >> 16), half2_of(v[e] >> 16)};
#pragma unroll
                    for (int x = 0; x < NB; ++x) mma(s[x], a, b[x][4 * c + e][0], b[x][4 * c + e][1]);
                }
            }
            // ---- weights ----
            const bool cut = key0 + BN - 1 > kall;
            float p[NB][4];
            uint32_t w[NB][2];
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[x][e] *= ks[e >> 1] * qs[x][e & 1];
                    if (cut && key0 + g + 8 * (e >> 1) > kmax[x][e & 1]) s[x][e] = __uint_as_float(0xff800000u);
                }
            for (int moves = 0;; ++moves) {
                bool far = false;
#pragma unroll
                for (int x = 0; x < NB; ++x) {
                    float u[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[x][e] = ex2((s[x][e] - m[x][e & 1]) * A.sl2);
                        u[e] = p[x][e] * vs[e >> 1] * put[x][e & 1];
                        far = far || p[x][e] > kGrown || u[e] > kMost;
                    }
                    w[x][0] = pack_half2(u[0], u[1]);
                    w[x][1] = pack_half2(u[2], u[3]);
                }
                if (!__any_sync(0xffffffffu, far) || moves == 2) break;   // (one move is enough, for finite rows)
                // rarely: the maximum, or the place of the weights, moves
#pragma unroll
                for (int x = 0; x < NB; ++x)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        auto over_keys = [&](float v) {
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                            return v;
                        };
                        const float top = over_keys(fmaxf(s[x][r], s[x][2 + r]));
                        const float mn = (top - m[x][r]) * A.sl2 > kLazy ? top : m[x][r];
                        const float alpha = ex2((m[x][r] - mn) * A.sl2);
                        const float big = over_keys(fmaxf(ex2((s[x][r] - mn) * A.sl2) * vs[0],
                                                          ex2((s[x][2 + r] - mn) * A.sl2) * vs[1]));
                        const float lv = fmaxf(level[x][r] * alpha, big);
                        // kTop over the level's power of two; the exponent within fp32's range
                        const uint32_t ex = min(max(__float_as_uint(lv) >> 23, 7u), 253u);
                        const float to = scale_of(254u - ex) * kTop, from = 1.f / put[x][r];
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            o[x][t][r] = o[x][t][r] * from * (alpha * to);
                            o[x][t][2 + r] = o[x][t][2 + r] * from * (alpha * to);
                        }
                        m[x][r] = mn;
                        l[x][r] *= alpha;
                        level[x][r] = lv;
                        put[x][r] = to;
                    }
            }
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                l[x][0] += p[x][0] + p[x][2];
                l[x][1] += p[x][1] + p[x][3];
                w[x][0] = transpose8(w[x][0]);
                w[x][1] = transpose8(w[x][1]);
            }
            // ---- O^T += V^T P^T: rows 2 q, 2 q + 1, 2 q + 8, 2 q + 9 at this lane's channels ----
            uint32_t v[4][D / 32];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = 2 * q4 + (k & 1) + 8 * (k >> 1);
                if constexpr (D == 128) {
                    const uint4 x = chunk<D>(tV, r, g);
                    v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(tV + r * D + (((g >> 1) ^ (r >> 1 & 3)) << 4) + (g & 1) * 8);
                    v[k][0] = x.x, v[k][1] = x.y;
                }
            }
            if (live < BN) {                                 // rows past the end may hold any bits
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (2 * q4 + (k & 1) + 8 * (k >> 1) >= live)
#pragma unroll
                        for (int e = 0; e < D / 32; ++e) v[k][e] = 0;
            }
            fence_async_smem();                              // the stage has been read
            __syncwarp();
            request();
            ring.next();
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const uint32_t sel = t & 1 ? 0x7362 : 0x5140;
                const uint32_t y = __byte_perm(v[0][t / 2], v[1][t / 2], sel), z = __byte_perm(v[2][t / 2], v[3][t / 2], sel);
                const uint32_t a[4] = {half2_of(y), half2_of(y >> 16), half2_of(z), half2_of(z >> 16)};
#pragma unroll
                for (int x = 0; x < NB; ++x) mma(o[x][t], a, w[x][0], w[x][1]);
            }
        }
        if (!fine) break;
        // ---- output of the part ----
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[x][r];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const int R = 8 * x + 2 * q4 + r;
                if (R >= it.rows) continue;
                const float f = it.whole ? 1.f / put[x][r] / sum : 1.f / put[x][r];
                float y[2 * MT];
#pragma unroll
                for (int t = 0; t < MT; ++t) y[2 * t] = o[x][t][r] * f, y[2 * t + 1] = o[x][t][2 + r] * f;
                if (it.whole) {
                    __nv_bfloat16 *dst = A.out + head_row(R) * D + 2 * MT * g;
#pragma unroll
                    for (int e = 0; e < 2 * MT; e += 8) {
                        uint32_t z[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(y[e + 2 * k], y[e + 2 * k + 1]);
                            z[k] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                        *reinterpret_cast<uint4 *>(dst + e) = make_uint4(z[0], z[1], z[2], z[3]);
                    }
                } else {
                    const size_t pr = A.parts.row(me, it.head ? 1 : 0, R);
                    float *dst = A.parts.o + pr * D + 2 * MT * g;
#pragma unroll
                    for (int e = 0; e < 2 * MT; e += 4)
                        *reinterpret_cast<float4 *>(dst + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                    if (g == 0) A.parts.ml[pr] = make_float2(m[x][r] * A.sl2, sum);
                }
            }
        if (!it.whole && it.head && lane == 0) {
            PartDesc &d = A.parts.desc[me];
            d.parts = it.parts;
            d.tok0 = it.tok0;
            d.h = it.h;
            d.row0 = row0;
            d.rows = it.rows;
        }
    }
    if (!fine) {                                             // copies in flight end before the CTA does
        for (int i = 0; i < kStages; ++i)
            if (lane == 0) mbar_wait(&S.full[i], i < ask.slot ? ask.phase : ask.phase ^ 1);
        __syncwarp();
    }
}

template <int D, int NB>
cudaError_t launch(const Pool &P, const WorkDim &W, const void *q, int Hq, float sl2, void *out, const Parts &parts,
                   int32_t *status, cudaStream_t st)
{
    Params A;
    A.P = P;
    A.W = W;
    A.q = (const __nv_bfloat16 *)q;
    A.out = (__nv_bfloat16 *)out;
    A.parts = parts;
    A.status = status;
    A.Hq = Hq;
    A.n_rows = (P.n_pages * P.Hkv) << P.page_log2;
    A.sl2 = std::max(sl2, 1e-38f);     // a masked product is -inf; times zero it would be NaN
    CUtensorMap mk, mv;
    if (!tma_map_u8_2d(&mk, P.k, D, A.n_rows, BN, true) || !tma_map_u8_2d(&mv, P.v, D, A.n_rows, BN, true))
        return cudaErrorInvalidValue;
    auto kern = attn8_few_kernel<D, NB>;
    constexpr int smem = kWarps * Geom<D>::SM_WARP;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(few_pieces() / kWarps), dim3(32 * kWarps), smem, st, mk, mv, A);
}

}  // namespace

int few_pieces() { return device_sm_count() * kWarps; }

cudaError_t attn8_few(const Pool &P, const WorkDim &W, int d, int rows, const void *q, int Hq, float sl2, void *out,
                      const Parts &parts, int32_t *status, cudaStream_t st)
{
    if (rows == 8)
        return d == 128 ? launch<128, 1>(P, W, q, Hq, sl2, out, parts, status, st)
                        : launch<64, 1>(P, W, q, Hq, sl2, out, parts, status, st);
    return d == 128 ? launch<128, 2>(P, W, q, Hq, sl2, out, parts, status, st)
                    : launch<64, 2>(P, W, q, Hq, sl2, out, parts, status, st);
}

}  // namespace paged
}  // namespace vc
