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
// A warp is alone with its piece of the batch: it requests the K and V rows of 4 KB
// tiles by TMA ahead of its arithmetic, past a unit's end too, and needs no barrier but
// those of the copies.
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

constexpr int kBlock = 16;                                     // rows of a request: they lie in one page
constexpr float kLazy = 8.f, kGrown = 4096.f;                  // log2 domain; a lane's sum with a weight above 2^kLazy
constexpr float kLeast = -3e38f;                               // a row that has seen no key
constexpr float kTop = 64.f, kMost = 32768.f;                  // where weights are put, and how far they may grow

// Warps of a CTA (their accumulators are what limits them) and tiles, of K and V, of
// a warp's ring: 192 KB in all.
template <int D, int NB>
struct Geom {
    static constexpr int BN = few_keys(D), BLOCKS = BN / kBlock, TILE = BN * D, STAGE = 2 * TILE;
    static constexpr int WARPS = NB == 1 ? 12 : 8, STAGES = 24 / WARPS;
    static constexpr int SMEM = WARPS * STAGES * STAGE;
};

template <int BM, int BN, int STAGES>
struct Warp {
    uint64_t full[STAGES];
    alignas(16) uint8_t scale[STAGES][2][BN];
    Piece piece;
    Walk<BM, BN, Seq, CostFew> walk;
    Item part[4];                      // the parts asked for last; the arithmetic is STAGES tiles behind
    bool more;
    static_assert(STAGES < 4, "parts");
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
// and 2 q + 1 (of each block), of O^T channels D/8 g .. + D/8 - 1 of the same rows.
template <int D, int NB>
__global__ void __launch_bounds__(32 * Geom<D, NB>::WARPS, 1)
attn8_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, Params A)
{
    constexpr int BM = 8 * NB, KS = D / 16, MT = D / 16, KC = D / 64;    // k steps, m tiles, chunks of a K row per lane
    using G = Geom<D, NB>;
    constexpr int BN = G::BN, kBlocks = G::BLOCKS, TILE = G::TILE, kStages = G::STAGES, kWarps = G::WARPS;
    extern __shared__ __align__(1024) uint8_t sm[];
    __shared__ Warp<BM, BN, kStages> warps[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
    Warp<BM, BN, kStages> &S = warps[warp];
    uint8_t *tiles = sm + warp * kStages * G::STAGE;
    // neighbouring pieces on different SMs
    const int n_piece = gridDim.x * kWarps, me = warp * gridDim.x + blockIdx.x;
    pdl_wait();
    if (lane == 0) {
        A.parts.desc[me].parts = 0;
        for (int i = 0; i < kStages; ++i) mbar_init(&S.full[i], 1);
        fence_mbar_init();
    }
    find_piece<BM, BN, Seq, CostFew>(A.P, A.W, me, n_piece, &S.piece);
    pdl_trigger();
    if (smem_u32(sm) & 1023u) {                              // never expected: the swizzled tiles need it
        if (lane == 0) report_timeout(A.status, 110);
        return;
    }
    if (S.piece.len <= 0) return;
    if (lane == 0) {
        S.walk.start(A.P, A.W, S.piece);
        tc::prefetch_tmap(&tmK);
        tc::prefetch_tmap(&tmV);
    }

    // One loop over the piece's tiles: requests first, then the arithmetic of the tile
    // that has arrived.  (Code that stands there twice is paid for in instruction
    // fetches: a call of one token over 200 takes 23 us with a walk and a request for
    // each use.)
    Ring<kStages> ask, ring;
    bool asking = true, fine = true;
    int pending = 0, asked = -1, used = 0;                   // tiles on their way; parts asked for, and in use
    int left = 0, at = 0, page = 0, page_next = 0;           // tiles to ask for; a lane's page numbers of 32 blocks
    const int what = lane & 3, block = lane >> 2;            // K, V, K's scales, V's; of lanes that request
    uint32_t b[NB][KS][2];
    float qs[NB][2];                                         // log2 e times the scale, the row's own with it
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
            const Item &it = S.part[asked & 3];
            auto entry = [&](int slot) {                     // -1: nothing to read there
                return slot < min(it.len(), it.t_hi * BN)
                           ? A.P.table[(size_t)it.b * A.P.max_blocks + (slot >> A.P.page_log2)] : -1;
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
            const unsigned scales = __popc(__ballot_sync(0xffffffffu, ok && what >= 2));
            uint64_t *bar = &S.full[ask.slot];
            if (lane == 0) mbar_arrive_expect_tx(bar, G::STAGE + scales * kBlock);
            __syncwarp();
            uint8_t *dst = tiles + ask.slot * G::STAGE + what * TILE + block * kBlock * D;
            if (lane < 4 * kBlocks) {
                if (what == 0) tc::tma_load_3d(dst, &tmK, 0, row, 0, bar);
                else if (what == 1) tc::tma_load_3d(dst, &tmV, 0, row, 0, bar);
                else if (ok) bulk_g2s(&S.scale[ask.slot][what - 2][block * kBlock],
                                      (what == 2 ? A.P.k_scale : A.P.v_scale) + row, kBlock, bar);
            }
            ask.next();
            ++pending;
        }
        if (pending == 0) break;
        const Item &it = S.part[used & 3];
        const int len = it.len(), row0 = it.mt * BM;
        auto head_row = [&](int r) {                         // row of q and out
            const int R = row0 + r;
            return (size_t)(it.tok0 + R / A.W.G) * A.Hq + it.h * A.W.G + R % A.W.G;
        };
        if (key0 < 0) {
            // ---- a part begins; Q: row g of each block, scaled to [1, 2) at its largest ----
            key0 = it.t_lo * BN;
            kall = it.last(row0 / A.W.G);                    // keys every row sees
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
                const uint32_t ex = min(max(top >> 7, 27u), 253u);
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
                    qs[x][r] = fmaxf(A.sl2 * __shfl_sync(0xffffffffu, back, 8 * q4 + 4 * r), 1e-38f);   // -inf * 0: NaN
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
            float ks[2 * kBlocks], vs[2 * kBlocks];          // of keys g + 8 j
#pragma unroll
            for (int j = 0; j < 2 * kBlocks; ++j) {
                ks[j] = scale_of(sc[8 * j]);
                vs[j] = g + 8 * j < live ? scale_of(sc[BN + 8 * j]) : 0.f;
            }
            // ---- S^T = K Q^T; s[x][j][r]: key g + 8 j, row 2 q + r, less the scale of q ----
            // (a chain of products per block and chunk: one chain would wait for itself)
            float s[NB][2 * kBlocks][2], acc[NB][kBlocks][KC][4];
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
                            mma(acc[x][y][c], a, b[x][4 * c + e][0], b[x][4 * c + e][1]);
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
                        s[x][2 * y + (e >> 1)][e & 1] = v * ks[2 * y + (e >> 1)];
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
            uint32_t w[NB][2 * kBlocks];
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
                            u[r] = p * (vs[j] * put[x][r]);
                        }
                        w[x][j] = pack_half2(u[0], u[1]);
                        most = __hmax2(most, *reinterpret_cast<const __half2 *>(&w[x][j]));
                    }
                    far = far || fmaxf(sum[x][0], sum[x][1]) > kGrown ||
                          fmaxf(__low2float(most), __high2float(most)) > kMost;
                }
                if (!__any_sync(0xffffffffu, far) || moves == 2) break;   // (one move is enough, for finite rows)
                // rarely: the maximum, or the place of the weights, moves
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
                        const float big = over_keys([&](int j) { return ex2((s[x][j][r] - mn) * qs[x][r]) * vs[j]; });
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
                l[x][0] += sum[x][0];
                l[x][1] += sum[x][1];
#pragma unroll
                for (int j = 0; j < 2 * kBlocks; ++j) w[x][j] = transpose8(w[x][j]);
            }
            // ---- O^T += V^T P^T: of each block, rows 2 q, 2 q + 1, 2 q + 8, 2 q + 9 at this lane's channels ----
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
                    for (int x = 0; x < NB; ++x) mma(o[x][t], a, w[x][2 * y], w[x][2 * y + 1]);
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
                    if (g == 0) A.parts.ml[pr] = make_float2(sum > 0.f ? m[x][r] * qs[x][r] : kLowest, sum);
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
    A.sl2 = sl2;
    CUtensorMap mk, mv;
    if (!tma_map_u8_2d(&mk, P.k, D, A.n_rows, kBlock, true) || !tma_map_u8_2d(&mv, P.v, D, A.n_rows, kBlock, true))
        return cudaErrorInvalidValue;
    auto kern = attn8_few_kernel<D, NB>;
    using G = Geom<D, NB>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(device_sm_count()), dim3(32 * G::WARPS), G::SMEM, st, mk, mv, A);
}

}  // namespace

int few_pieces(int rows) { return device_sm_count() * (rows == 8 ? Geom<128, 1>::WARPS : Geom<128, 2>::WARPS); }

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
