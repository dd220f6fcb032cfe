// paged_attn_few.cuh -- causal attention over 8-bit pages, and over bf16 pages in
// planned batches, for batches of few rows (decoding, drafting): up to 16 (query,
// head) rows per kv head, on the batch's average; and of fp32 rows over 8-bit pages in
// all batches.
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
// than it saves where rows are few (a decode step of 16 x 32768 tokens, 32/8 heads of
// 128, 1.08 GB: 176 us here, 90% of the copy rate, 392 there; four tokens of 16 over
// 8192, 16 rows, 69 and 122; from 24 rows on there is nothing between them).
//
// A warp is alone with its piece of the batch: it requests the K and V rows of 4 KB
// tiles by TMA ahead of its arithmetic, past a unit's end too, and needs no barrier but
// those of the copies.
//
// bf16 pages (KV8 false) take the same products of bf16 operands: K through ldmatrix,
// V through its transposing form, and nothing is scaled; the weights are rounded to bf16,
// as in the tensor-core kernel.  They serve the own slots of
// sequences that share a prefix, a few hundred tokens each, for which the tensor-core
// kernel's 8 us per unit are too many, and the prefixes of small groups.
//
// fp32 rows over 8-bit pages take the same products: the codes are exact operands, and
// q and the weights are two f16 terms each, 22 bits, for twice the products.  The unit
// does not round its running sums to nearest, so each product of 16 is added to them
// outside it.  Four chunks of 300 over 2000, 16/4 heads of 128, take 233 us
// (583 on the CUDA cores), a token of 8 sequences over 4000, 32/8 heads, 27 (169).
//
// Ranges.  q is scaled by its row's largest exponent to 2^14 (beside the roundings to
// 11 or 22 bits, an element is off by at most 2^-39 of the row's largest; rows below
// 2^-112 are taken as of that size).  The running maximum is raised when it has grown by
// more than 2^8, as in the tensor-core kernel, and with a row's first key.  The weights
// p 2^f, which become f16, are scaled by a power of two per row, its place, such that the
// largest so far lies at 2^6: what is lost below f16's smallest number is 2^-31 of it per
// key.  They may grow to 2^15 before the place moves.
#pragma once

#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "paged8.cuh"
#include "tcgen05.cuh"

namespace vc {
namespace paged {
namespace {

constexpr int kBlock = 16;                                     // rows of a request: they lie in one page
constexpr float kLazy = 8.f, kGrown = 4096.f;                  // log2 domain; a lane's sum with a weight above 2^kLazy
constexpr float kLeast = -3e38f;                               // a row that has seen no key
// The least scale of scores (log2 domain).  A product of -inf times zero would be NaN;
// a row's first key lies 30 above kLeast at least, so that its maximum and the place of
// its weights move there; products of 1e30 change a weight by 1e-7.
constexpr float kLeastScore = 1e-37f;
constexpr float kQTop = 16384.f;                               // q rows lie in [kQTop, 2 kQTop) at their largest
constexpr int kBack = 48;                                      // log2: by how much products may be scaled up
constexpr float kTop = 64.f, kMost = 32768.f;                  // where weights are put, and how far they may grow

// Warps of a CTA (their accumulators are what limits them) and tiles, of K and V, of
// a warp's ring: 192 KB in all.
template <int D, int NB, bool KV8, typename E>
struct Geom {
    static constexpr int ROW = KV8 ? D : 2 * D;                // bytes
    static constexpr int BN = few_keys(D, KV8), BLOCKS = BN / kBlock, TILE = BN * ROW, STAGE = 2 * TILE;
    static constexpr int WARPS = NB == 1 ? 12 : 8, STAGES = 24 / WARPS;
    static constexpr int SMEM = WARPS * STAGES * STAGE;
    static constexpr int BOXES = KV8 || D == 64 ? 1 : 2;       // of a block: rows of 128 bytes at most
};

template <int BM, int BN, int STAGES, typename SEQ, typename C>
struct Warp {
    uint64_t full[STAGES];
    alignas(16) uint8_t scale[STAGES][2][BN];
    PieceOf<SEQ> piece;
    Walk<BM, BN, SEQ, C> walk;
    ItemOf<SEQ> part[4];               // the parts asked for last; the arithmetic is STAGES tiles behind
    bool more;
    static_assert(STAGES < 4, "parts");
};

struct Params {
    Pool P;
    WorkDim W;
    const void *q;
    void *out;
    Halves H;                          // instead, where the batch is planned
    Parts parts;
    int32_t *status;
    int Hq, n_rows;
    bool first;                        // planned: the kernel launched before is the plan's
    float sl2;
};

__device__ __forceinline__ uint32_t half2_of(uint32_t codes)   // the low 16 bits
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// the pair's nearest f16 numbers; leaves what they lack
__device__ __forceinline__ uint32_t take_half2(float &a, float &b)
{
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    a -= f.x;
    b -= f.y;
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// four 8 x 8 blocks, a row's address per lane
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const uint8_t *p)
{
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_u32(p)) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_u32(p)) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
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
// and 2 q + 1 (of each block), of O^T channels D/8 g .. + D/8 - 1 (KV8) or g + 8 i of
// the same rows.
template <int D, int NB, typename SEQ, bool KV8, typename E>
__global__ void __launch_bounds__(32 * Geom<D, NB, KV8, E>::WARPS, 1)
attn_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, Params A)
{
    constexpr int BM = 8 * NB, KS = D / 16, MT = D / 16, KC = D / 64;    // k steps, m tiles, chunks of a K row per lane
    constexpr bool F32 = std::is_same_v<E, float>;
    constexpr int TERMS = F32 ? 2 : 1;                       // f16 terms of q and of the weights
    static_assert(KV8 || !F32, "fp32 rows: 8-bit pages");
    using G = Geom<D, NB, KV8, E>;
    using It = ItemOf<SEQ>;
    constexpr bool PLANNED = std::is_same_v<SEQ, VSeq>;
    using C = std::conditional_t<F32 || PLANNED, CostFewCut, CostFew>;
    constexpr int BN = G::BN, kBlocks = G::BLOCKS, TILE = G::TILE, kStages = G::STAGES, kWarps = G::WARPS;
    extern __shared__ __align__(1024) uint8_t sm[];
    __shared__ Warp<BM, BN, kStages, SEQ, C> warps[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
    Warp<BM, BN, kStages, SEQ, C> &S = warps[warp];
    uint8_t *tiles = sm + warp * kStages * G::STAGE;
    // neighbouring pieces on different SMs
    const int n_piece = gridDim.x * kWarps, me = warp * gridDim.x + blockIdx.x;
    // A planned batch's entries come from the kernel before the one before this, which
    // has waited for it; that one runs beside this kernel (see the end).
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&tmK);
        tc::prefetch_tmap(&tmV);
    }
    if (!PLANNED || A.first) pdl_wait();
    if (lane == 0) {
        A.parts.desc[me].parts = 0;
        for (int i = 0; i < kStages; ++i) mbar_init(&S.full[i], 1);
        fence_mbar_init();
    }
    find_piece<BM, BN, SEQ, C>(A.P, A.W, me, n_piece, &S.piece);
    if (!PLANNED) pdl_trigger();
    const bool placed = (smem_u32(sm) & 1023u) == 0;         // the swizzled tiles need it
    if (!placed && lane == 0) report_timeout(A.status, 110); // never expected
    if (!PLANNED && (!placed || S.piece.len <= 0)) return;
    if (lane == 0) {
        S.walk.start(A.W, S.piece);
    }

    // One loop over the piece's tiles: requests first, then the arithmetic of the tile
    // that has arrived.  (Code that stands there twice is paid for in instruction
    // fetches: a call of one token over 200 takes 23 us with a walk and a request for
    // each use.)
    Ring<kStages> ask, ring;
    bool asking = placed && S.piece.len > 0, fine = true;
    int pending = 0, asked = -1, used = 0;                   // tiles on their way; parts asked for, and in use
    int left = 0, at = 0, page = 0, page_next = 0;           // tiles to ask for; a lane's page numbers of 32 blocks
    const int what = lane & 3, block = lane >> 2 & (kBlocks - 1);      // K, V, K's scales, V's (or second boxes); of lanes that request
    uint32_t b[NB][KS][TERMS][2];
    float qs[NB][2], back[NB][2];                            // log2 e times the scale; back: what products are scaled with first
    float o[NB][MT][4], m[NB][2], l[NB][2], put[NB][2], level[NB][2];
    int kmax[NB][2], kall = 0, key0 = -1;
    for (;;) {
        while (asking && pending < kStages) {
            if (left == 0) {
                __syncwarp();
                ++asked;
                if (lane == 0) S.more = S.walk.next(A.P, A.W, S.part[asked & 3]);
                __syncwarp();
                asking = S.more;
                if (!asking) break;
            }
            const It &it = S.part[asked & 3];
            auto entry = [&](int slot) {                     // -1: nothing to read there
                return slot < min(it.len(), it.t_hi * BN)
                           ? A.P.table[(size_t)it.b * A.P.max_blocks + ((it.first_slot() + slot) >> A.P.page_log2)] : -1;
            };
            if (left == 0) {
                left = it.t_hi - it.t_lo;
                at = 0;
                page_next = entry(it.t_lo * BN + lane * kBlock);
            }
            // a lane per 16-key block of K, V and their scales, whose rows lie in one
            // page, side by side
            const int slot = (it.t_hi - left) * BN, mine = slot + block * kBlock;
            if (at == 0) {
                page = page_next;
                page_next = entry(slot + (32 + lane) * kBlock);
            }
            const int p = __shfl_sync(0xffffffffu, page, (at + block) & 31);
            at = (at + kBlocks) & 31;
            --left;
            const bool wanted = lane < 4 * kBlocks && mine < it.len();
            const bool ok = wanted && (unsigned)p < (unsigned)A.P.n_pages;
            const int row = ok ? (int)A.P.row(p, it.h, mine & (A.P.page() - 1)) : A.n_rows;      // outside: zeros
            if (wanted && !ok) set_flag(A.P.status, VC_PAGED_BAD_PAGE);
            const unsigned scales = KV8 ? __popc(__ballot_sync(0xffffffffu, ok && what >= 2)) : 0;
            uint64_t *bar = &S.full[ask.slot];
            if (lane == 0) mbar_arrive_expect_tx(bar, G::STAGE + scales * kBlock);
            __syncwarp();
            // (bf16 rows of 128 channels: a box per half, the second by the lane of the scales)
            uint8_t *dst = tiles + ask.slot * G::STAGE + (what & 1) * TILE + block * kBlock * G::ROW + (what >> 1) * kBlock * 128;
            if (lane < 4 * kBlocks && (what < 2 || KV8 || G::BOXES == 2)) {
                const int c = KV8 ? 0 : (what >> 1) * 64;
                if (what == 0 || (!KV8 && what == 2)) tc::tma_load_3d(dst, &tmK, c, row, 0, bar);
                else if (what == 1 || (!KV8 && what == 3)) tc::tma_load_3d(dst, &tmV, c, row, 0, bar);
                else if (KV8 && ok) bulk_g2s(&S.scale[ask.slot][what - 2][block * kBlock],
                                      (what == 2 ? A.P.k_scale : A.P.v_scale) + row, kBlock, bar);
            }
            ask.next();
            ++pending;
        }
        if (pending == 0) break;
        const It &it = S.part[used & 3];
        const int len = it.len(), row0 = it.mt * BM;
        auto row_of = [&](int tok0, int r) {
            const int R = row0 + r;
            return (size_t)(tok0 + R / A.W.G) * A.Hq + it.h * A.W.G + R % A.W.G;
        };
        auto head_row = [&](int r) { return row_of(it.out_tok0(), r); };      // of out and lse_out
        if (key0 < 0) {
            // ---- a part begins; Q: row g of each block (8-bit pages: its largest in [kQTop, 2 kQTop)) ----
            key0 = it.t_lo * BN;
            kall = it.last(row0 / A.W.G);                    // keys every row sees
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                const bool on = 8 * x + g < it.rows;
                uint32_t ex = 127 + 14;                      // of the row's scale, 2^(ex - 141)
                if constexpr (KV8) {
                    float w[KC][16];                         // this lane's channels of the row
                    const E *src = (const E *)A.q + (on ? row_of(it.tok0, 8 * x + g) * D : 0) + q4 * 16;
                    float top = 0.f;
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        constexpr int PER = 16 / sizeof(E);
#pragma unroll
                        for (int i = 0; i < 16; i += PER) {
                            uint4 z = make_uint4(0, 0, 0, 0);
                            if (on) z = *reinterpret_cast<const uint4 *>(src + c * 64 + i);
                            const uint32_t u[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if constexpr (F32) w[c][i + k] = __uint_as_float(u[k]);
                                else w[c][i + 2 * k] = bf16_lo(u[k]), w[c][i + 2 * k + 1] = bf16_hi(u[k]);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(w[c][i]));
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    ex = min(max(__float_as_uint(top) >> 23, 15u), 253u);
                    const float inv = scale_of(254u - ex) * kQTop;
#pragma unroll
                    for (int c = 0; c < KC; ++c)
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {    // four channels are a k step's
                            float lo = w[c][i] * inv, hi = w[c][i + 1] * inv;
#pragma unroll
                            for (int k = 0; k < TERMS; ++k) b[x][4 * c + i / 4][k][i / 2 % 2] = take_half2(lo, hi);
                        }
                } else {
                    const uint32_t *src = reinterpret_cast<const uint32_t *>((const E *)A.q + (on ? row_of(it.tok0, 8 * x + g) * D : 0));
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        b[x][i][0][0] = on ? src[8 * i + q4] : 0;
                        b[x][i][0][1] = on ? src[8 * i + 4 + q4] : 0;
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    // a row's scale meets the products (below 2^32) before the keys' scales do,
                    // what is above kBack with the scale of the scores: nothing overflows that
                    // the product or the score itself does not
                    const int of = KV8 ? (int)__shfl_sync(0xffffffffu, ex, 8 * q4 + 4 * r) - 14 : 127;
                    back[x][r] = scale_of(min(of, 127 + kBack));
                    qs[x][r] = fmaxf(A.sl2 * scale_of(127 + max(of - 127 - kBack, 0)), kLeastScore);
                    const int R = 8 * x + 2 * q4 + r;
                    kmax[x][r] = R < it.rows ? it.last((row0 + R) / A.W.G) : -1;
                }
            }
#pragma unroll
            for (int x = 0; x < NB; ++x) {
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[x][t][e] = 0.f;
#pragma unroll
                for (int r = 0; r < 2; ++r) m[x][r] = kLeast, l[x][r] = 0.f, put[x][r] = 1.f, level[x][r] = 0.f;
            }
        }
        {
            const int live = len - key0;
            fine = wait_warp(&S.full[ring.slot], ring.phase, A.status, 111);
            if (!fine) break;
            const uint8_t *tK = tiles + ring.slot * G::STAGE, *tV = tK + TILE;
            const uint8_t *sc = &S.scale[ring.slot][0][g];
            // bf16: the 16-byte chunk c (8 channels) of key r of block y
            auto half_chunk = [&](const uint8_t *tile, int y, int r, int c) {
                return tile + y * kBlock * G::ROW + (c >> 3) * kBlock * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
            };
            float ks[2 * kBlocks], vs[2 * kBlocks];          // of keys g + 8 j
#pragma unroll
            for (int j = 0; j < 2 * kBlocks; ++j) {
                ks[j] = KV8 ? scale_of(sc[8 * j]) : 1.f;
                vs[j] = !KV8 ? 1.f : g + 8 * j < live ? scale_of(sc[BN + 8 * j]) : 0.f;
            }
            // ---- S^T = K Q^T; s[x][j][r]: key g + 8 j, row 2 q + r, less what q's scale has above 2^kBack ----
            // (a chain of products per block and chunk: one chain would wait for itself)
            float s[NB][2 * kBlocks][2], acc[NB][kBlocks][KC][4];
            if constexpr (!KV8) {
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int y = 0; y < kBlocks; ++y) {
                            uint32_t a[4];                   // keys 0 and 8, channels 0 and 8 on of the step
                            ldmatrix4<false>(a, half_chunk(tK, y, lane & 15, 8 * c + 2 * e + (lane >> 4)));
#pragma unroll
                            for (int x = 0; x < NB; ++x) {
                                if (e == 0) acc[x][y][c][0] = acc[x][y][c][1] = acc[x][y][c][2] = acc[x][y][c][3] = 0.f;
                                mma_bf16(acc[x][y][c], a, b[x][4 * c + e][0][0], b[x][4 * c + e][0][1]);
                            }
                        }
            } else {
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    uint32_t u[kBlocks][2][4];
#pragma unroll
                    for (int y = 0; y < kBlocks; ++y)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint4 k = chunk<D>(tK + y * kBlock * D, g + 8 * z, 4 * c + q4);
                            u[y][z][0] = k.x, u[y][z][1] = k.y, u[y][z][2] = k.z, u[y][z][3] = k.w;
                        }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int y = 0; y < kBlocks; ++y) {
                            const uint32_t a[4] = {half2_of(u[y][0][e]), half2_of(u[y][1][e]), half2_of(u[y][0][e] >> 16),
                                                   half2_of(u[y][1][e] >> 16)};
#pragma unroll
                            for (int x = 0; x < NB; ++x) {
                                if (e == 0) acc[x][y][c][0] = acc[x][y][c][1] = acc[x][y][c][2] = acc[x][y][c][3] = 0.f;
                                if constexpr (F32) {
                                    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                    for (int k = TERMS - 1; k >= 0; --k)
                                        mma(part, a, b[x][4 * c + e][k][0], b[x][4 * c + e][k][1]);
#pragma unroll
                                    for (int i = 0; i < 4; ++i) acc[x][y][c][i] += part[i];
                                } else {
                                    mma(acc[x][y][c], a, b[x][4 * c + e][0][0], b[x][4 * c + e][0][1]);
                                }
                            }
                        }
                }
            }
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
                for (int y = 0; y < kBlocks; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = acc[x][y][0][e];
#pragma unroll
                        for (int c = 1; c < KC; ++c) v += acc[x][y][c][e];
                        s[x][2 * y + (e >> 1)][e & 1] = KV8 ? v * back[x][e & 1] * ks[2 * y + (e >> 1)] : v;
                    }
            if (key0 + BN - 1 > kall) {                      // some row does not see all keys
#pragma unroll
                for (int x = 0; x < NB; ++x)
#pragma unroll
                    for (int j = 0; j < 2 * kBlocks; ++j)
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            if (key0 + g + 8 * j > kmax[x][r]) s[x][j][r] = __uint_as_float(0xff800000u);
            }
            // ---- weights ----
            uint32_t w[NB][2 * kBlocks][TERMS];
            float sum[NB][2];
            for (int moves = 0;; ++moves) {
                bool far = false;
#pragma unroll
                for (int x = 0; x < NB; ++x) {
                    sum[x][0] = sum[x][1] = 0.f;
                    __half2 most = __float2half2_rn(0.f);
#pragma unroll
                    for (int j = 0; j < 2 * kBlocks; ++j) {
                        float u[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float p = ex2((s[x][j][r] - m[x][r]) * qs[x][r]);
                            sum[x][r] += p;
                            // (in this order: vs * put may be infinite where p is zero or tiny, and p * vs
                            // vanish; p * put is finite once the row has its place, and what it loses below
                            // 2^-149 is below 2^-28 of the largest weight under any scale)
                            u[r] = KV8 ? p * put[x][r] * vs[j] : p;
                        }
                        if constexpr (KV8) {
#pragma unroll
                            for (int k = 0; k < TERMS; ++k) w[x][j][k] = take_half2(u[0], u[1]);
                            most = __hmax2(most, *reinterpret_cast<const __half2 *>(&w[x][j][0]));
                        } else {
                            w[x][j][0] = pack_bf16(u[0], u[1]);
                        }
                    }
                    far = far || fmaxf(sum[x][0], sum[x][1]) > kGrown ||
                          (KV8 && fmaxf(__low2float(most), __high2float(most)) > kMost);
                }
                if (!__any_sync(0xffffffffu, far) || moves == 2) break;   // (one move is enough, for finite rows)
                // rarely: the maximum, or the place of the weights, moves
                if constexpr (KV8) {
                    // a value row of zeros has no size, whatever its scale says (a quarter
                    // of a row per lane)
#pragma unroll
                    for (int j = 0; j < 2 * kBlocks; ++j) {
                        const uint4 *row = reinterpret_cast<const uint4 *>(tV + (g + 8 * j) * D + q4 * (D / 4));
                        uint32_t any = 0;
#pragma unroll
                        for (int i = 0; i < D / 64; ++i) any |= row[i].x | row[i].y | row[i].z | row[i].w;
                        any |= __shfl_xor_sync(0xffffffffu, any, 1);
                        any |= __shfl_xor_sync(0xffffffffu, any, 2);
                        if ((any & 0x7f7f7f7fu) == 0) vs[j] = 0.f;
                    }
                }
#pragma unroll
                for (int x = 0; x < NB; ++x)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        auto over_keys = [&](auto value) {
                            float v = value(0);
#pragma unroll
                            for (int j = 1; j < 2 * kBlocks; ++j) v = fmaxf(v, value(j));
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                            return v;
                        };
                        const float top = over_keys([&](int j) { return s[x][j][r]; });
                        const float mn = (top - m[x][r]) * qs[x][r] > kLazy ? top : m[x][r];
                        const float alpha = ex2((m[x][r] - mn) * qs[x][r]);
                        float to = 1.f, from = 1.f;
                        if constexpr (KV8) {
                            const float big = over_keys([&](int j) { return ex2((s[x][j][r] - mn) * qs[x][r]) * vs[j]; });
                            const float lv = fminf(fmaxf(level[x][r] * alpha, big), 3e38f);      // (infinite, it would stay so)
                            // kTop over the level's power of two, 2^115 at most (a row that has seen no
                            // value: any that comes fits there or moves it), so that weights of up to
                            // kGrown stay finite beside a scale that was set to zero above
                            const uint32_t ex = min(max(__float_as_uint(lv) >> 23, 18u), 253u);
                            to = scale_of(254u - ex) * kTop;
                            from = 1.f / put[x][r];
                            level[x][r] = lv;
                        }
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            o[x][t][r] = o[x][t][r] * from * (alpha * to);
                            o[x][t][2 + r] = o[x][t][2 + r] * from * (alpha * to);
                        }
                        m[x][r] = mn;
                        l[x][r] *= alpha;
                        put[x][r] = to;
                    }
            }
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                l[x][0] += sum[x][0];
                l[x][1] += sum[x][1];
#pragma unroll
                for (int j = 0; j < 2 * kBlocks; ++j)
#pragma unroll
                    for (int k = 0; k < TERMS; ++k) w[x][j][k] = transpose8(w[x][j][k]);
            }
            // ---- O^T += V^T P^T: of each block, rows 2 q, 2 q + 1, 2 q + 8, 2 q + 9 at this lane's channels ----
            if constexpr (!KV8) {
#pragma unroll
                for (int y = 0; y < kBlocks; ++y)
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        uint32_t a[4];                       // keys 0 (channels 0 and 8 on), keys 8
                        ldmatrix4<true>(a, half_chunk(tV, y, (lane & 7) + (lane >> 4) * 8, 2 * t + (lane >> 3 & 1)));
                        if (live < 16 * (y + 1)) {           // rows past the end may hold any bits
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int key = 16 * y + 2 * q4 + 8 * (e >> 1);
                                if (key >= live) a[e] = 0;
                                else if (key + 1 >= live) a[e] &= 0xffffu;
                            }
                        }
#pragma unroll
                        for (int x = 0; x < NB; ++x) mma_bf16(o[x][t], a, w[x][2 * y][0], w[x][2 * y + 1][0]);
                    }
            } else {
#pragma unroll
                for (int y = 0; y < kBlocks; ++y) {
                    uint32_t v[4][D / 32];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = 2 * q4 + (k & 1) + 8 * (k >> 1);
                        if constexpr (D == 128) {
                            const uint4 z = chunk<D>(tV + y * 16 * D, r, g);
                            v[k][0] = z.x, v[k][1] = z.y, v[k][2] = z.z, v[k][3] = z.w;
                        } else {
                            const uint2 z = *reinterpret_cast<const uint2 *>(tV + y * 16 * D + r * D +
                                                                             (((g >> 1) ^ (r >> 1 & 3)) << 4) + (g & 1) * 8);
                            v[k][0] = z.x, v[k][1] = z.y;
                        }
                    }
                    if (live < 16 * (y + 1)) {                   // rows past the end may hold any bits
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (16 * y + 2 * q4 + (k & 1) + 8 * (k >> 1) >= live)
#pragma unroll
                                for (int e = 0; e < D / 32; ++e) v[k][e] = 0;
                    }
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const uint32_t sel = t & 1 ? 0x7362 : 0x5140;
                        const uint32_t c = __byte_perm(v[0][t / 2], v[1][t / 2], sel), z = __byte_perm(v[2][t / 2], v[3][t / 2], sel);
                        const uint32_t a[4] = {half2_of(c), half2_of(c >> 16), half2_of(z), half2_of(z >> 16)};
#pragma unroll
                        for (int x = 0; x < NB; ++x)
                            if constexpr (F32) {
                                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                for (int k = TERMS - 1; k >= 0; --k) mma(part, a, w[x][2 * y][k], w[x][2 * y + 1][k]);
#pragma unroll
                                for (int i = 0; i < 4; ++i) o[x][t][i] += part[i];
                            } else {
                                mma(o[x][t], a, w[x][2 * y][0], w[x][2 * y + 1][0]);
                            }
                    }
                }
            }
        }
        fence_async_smem();                                  // the stage has been read
        __syncwarp();
        ring.next();
        --pending;
        key0 += BN;
        if (key0 < it.t_hi * BN) continue;
        key0 = -1;
        ++used;
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
                const float top = sum > 0.f ? m[x][r] * qs[x][r] : kLowest;
                float y[2 * MT];
#pragma unroll
                for (int t = 0; t < MT; ++t) y[2 * t] = o[x][t][r] * f, y[2 * t + 1] = o[x][t][2 + r] * f;
                const size_t row = it.whole ? head_row(R) : A.parts.row(me, it.head ? 1 : 0, R);
                if (it.whole && !PLANNED && !F32) {
                    __nv_bfloat16 *dst = (__nv_bfloat16 *)A.out + row * D + 2 * MT * g;
                    static_assert(KV8 || PLANNED, "a lane's channels are side by side");
#pragma unroll
                    for (int e = 0; e < 2 * MT; e += 8)
                        *reinterpret_cast<uint4 *>(dst + e) = make_uint4(pack_bf16(y[e], y[e + 1]), pack_bf16(y[e + 2], y[e + 3]),
                                                                         pack_bf16(y[e + 4], y[e + 5]), pack_bf16(y[e + 6], y[e + 7]));
                } else {
                    float *dst = (!it.whole ? A.parts.o : PLANNED ? A.H.o : (float *)A.out) + row * D;
                    if constexpr (KV8) {
#pragma unroll
                        for (int e = 0; e < 2 * MT; e += 4)
                            *reinterpret_cast<float4 *>(dst + 2 * MT * g + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 2 * MT; ++e) dst[8 * e + g] = y[e];
                    }
                    if (g == 0) {
                        if (PLANNED && it.head)
                            A.H.place[head_row(R)] = it.whole ? Place::in_output() : Place::in_parts(me, it.parts, R);
                        if (!it.whole) A.parts.ml[row] = make_float2(top, sum);
                        else if (PLANNED) A.H.lse[row] = top + log2f(sum);
                    }
                }
            }
        if (!it.whole && it.head && lane == 0) {
            PartDesc &d = A.parts.desc[me];
            d.parts = it.parts;
            d.tok0 = it.out_tok0();
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
    // A planned batch: the kernel before this one has written the other half.  Its end
    // is waited for here, so that what follows this kernel follows both.
    if (PLANNED) {
        pdl_wait();
        pdl_trigger();
    }
}

template <int D, int NB, typename SEQ, bool KV8, typename E>
cudaError_t launch_few(const Pool &P, const WorkDim &W, const void *q, int Hq, float sl2, void *out, const Halves &H,
                       bool first, const Parts &parts, int32_t *status, cudaStream_t st)
{
    using G = Geom<D, NB, KV8, E>;
    Params A;
    A.P = P;
    A.W = W;
    A.q = q;
    A.out = out;
    A.first = first;
    A.H = H;
    A.parts = parts;
    A.status = status;
    A.Hq = Hq;
    A.n_rows = (P.n_pages * P.Hkv) << P.page_log2;
    A.sl2 = sl2;
    CUtensorMap mk, mv;
    if constexpr (KV8) {
        if (!tma_map_u8_2d(&mk, P.k, D, A.n_rows, kBlock, true) || !tma_map_u8_2d(&mv, P.v, D, A.n_rows, kBlock, true))
            return cudaErrorInvalidValue;
    } else {
        const uint64_t bytes = (uint64_t)D * 2;
        if (!tma_map_bf16_3d(&mk, P.k, D, A.n_rows, 1, bytes, bytes * A.n_rows, 64, kBlock, 1) ||
            !tma_map_bf16_3d(&mv, P.v, D, A.n_rows, 1, bytes, bytes * A.n_rows, 64, kBlock, 1))
            return cudaErrorInvalidValue;
    }
    auto kern = attn_few_kernel<D, NB, SEQ, KV8, E>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(device_sm_count()), dim3(32 * G::WARPS), G::SMEM, st, mk, mv, A);
}

template <typename SEQ, bool KV8, typename E>
cudaError_t few_form(const Pool &P, const WorkDim &W, int d, int rows, const void *q, int Hq, float sl2, void *out,
                     const Halves &H, bool first, const Parts &parts, int32_t *status, cudaStream_t st)
{
    if (rows == 8)
        return d == 128 ? launch_few<128, 1, SEQ, KV8, E>(P, W, q, Hq, sl2, out, H, first, parts, status, st)
                        : launch_few<64, 1, SEQ, KV8, E>(P, W, q, Hq, sl2, out, H, first, parts, status, st);
    return d == 128 ? launch_few<128, 2, SEQ, KV8, E>(P, W, q, Hq, sl2, out, H, first, parts, status, st)
                    : launch_few<64, 2, SEQ, KV8, E>(P, W, q, Hq, sl2, out, H, first, parts, status, st);
}

}  // namespace
}  // namespace paged
}  // namespace vc
