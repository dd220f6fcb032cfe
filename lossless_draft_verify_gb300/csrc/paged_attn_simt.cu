// paged_attn_simt.cu -- causal attention of ragged chunks over a paged cache
// and its attention mass on the CUDA cores, fp32 throughout: the path of fp32
// caches, whose products may not be rounded to the tensor cores' input types.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j),
//   j <= ctx + i, in one pass over the keys with a running maximum and sum;
//   mass_j = sum_i p_ij / sum_j' p_ij' in a second one, with the final ones.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace cg = cooperative_groups;

namespace vc {
namespace paged {
namespace {

constexpr int kThreads = 256;

// rows [0, n_rows) of a tile into shared memory (pitch floats apart); row r at
// src(r), null: zeros
template <int D, typename F>
__device__ __forceinline__ void load_rows(float *dst, int pitch, int n_rows, F src)
{
    for (int i = threadIdx.x; i < n_rows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        const float *p = src(r);
        *reinterpret_cast<float4 *>(dst + r * pitch + c) =
            p ? *reinterpret_cast<const float4 *>(p + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

template <int D, int BM, int BN>
struct Geom {
    static constexpr int PQ = D + 4, PP = BN + 4;      // pitches: rows 4 banks apart
    static constexpr int STAGE = BN * PQ + BN * D;     // a key tile's K and V
    static constexpr int SMEM = (BM * PQ + 2 * STAGE + BM * PP) * 4;
};

// 16 bytes to shared memory, zeros where !on (src is then not read)
__device__ __forceinline__ void copy16(float *dst, const float *src, bool on)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(float *dst, const float *src, bool on)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                 :: "r"(smem_u32(dst)), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// One CTA per piece of the batch's work (paged.cuh).  256 threads as 16 x 16:
// thread (ty, tx) holds rows ty * RT .. + RT - 1 against keys tx + 16 j, and
// the same rows' outputs at channels 4 tx + 64 j.  Products are taken two
// channels at a time (half the instructions).  Bound by shared memory's reads and
// the instructions around them: four chunks of 300 over 2000 tokens, 16/4 heads
// of 128, 572 us, 37 TFLOP/s (larger tiles leave room for fewer warps); a token of
// 8 sequences over 4000, 32/8 heads, 157 us, 1.7 TB/s.
template <int D, int BM, int BN>
__global__ void __launch_bounds__(kThreads)
attn_simt_kernel(Pool P, WorkDim W, const float *__restrict__ q, int Hq, float scale_log2, float *__restrict__ out,
                 float *__restrict__ lse_out, Parts parts)
{
    constexpr int RT = BM / 16, KT = BN / 16, CT = D / 64;
    using G = Geom<D, BM, BN>;
    extern __shared__ __align__(16) float smf[];
    float *sQ = smf, *sKV = sQ + BM * G::PQ, *sP = sKV + 2 * G::STAGE;
    __shared__ Piece piece;
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x < 32) find_piece<BM, BN>(P, W, blockIdx.x, gridDim.x, &piece);
    __syncthreads();
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const float *pk = (const float *)P.k, *pv = (const float *)P.v;
    Walk<BM, BN> walk;
    walk.start(P, W, piece);
    if (threadIdx.x == 0) parts.desc[blockIdx.x].parts = 0;
    Item it;
    while (walk.next(P, W, it)) {
        const int row0 = it.mt * BM, len = it.ctx + it.n;
        auto token_row = [&](int r) {                  // row of q / out of tile row r
            const int R = row0 + r;
            return ((size_t)(it.tok0 + R / W.G) * Hq + it.h * W.G + R % W.G) * D;
        };
        __syncthreads();
        load_rows<D>(sQ, G::PQ, BM, [&](int r) { return r < it.rows ? q + token_row(r) : nullptr; });
        float m[RT], l[RT];
        float2 acc[RT][CT][2];
        int kmax[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            m[i] = kLowest;
            l[i] = 0.f;
            const int r = ty * RT + i;
            kmax[i] = r < it.rows ? it.ctx + (row0 + r) / W.G : -1;
#pragma unroll
            for (int j = 0; j < CT; ++j) acc[i][j][0] = acc[i][j][1] = make_float2(0.f, 0.f);
        }
        // Key tiles pass through two stages: a tile is on its way while the one
        // before it is computed with, its page numbers are read a tile earlier.
        constexpr int CH = D / 4, RP = kThreads / CH, NR = BN / RP;
        const int c4 = (int)threadIdx.x % CH * 4, r0 = threadIdx.x / CH;
        int pages[NR];
        auto look_up = [&](int t) {
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                const int slot = t * BN + r0 + x * RP;
                pages[x] = t < it.t_hi && slot < len ? P.page_of(it.b, slot >> P.page_log2) : -1;
            }
        };
        auto fetch = [&](int t) {
            float *k = sKV + (t & 1) * G::STAGE, *v = k + BN * G::PQ;
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                const int r = r0 + x * RP, slot = t * BN + r;
                const bool on = pages[x] >= 0;
                const size_t at = on ? P.row(pages[x], it.h, slot & (P.page() - 1)) * D + c4 : 0;
                copy16(k + r * G::PQ + c4, pk + at, on);
                copy16(v + r * D + c4, pv + at, on);
            }
            copy_commit();
        };
        look_up(it.t_lo);
        fetch(it.t_lo);
        look_up(it.t_lo + 1);
        for (int t = it.t_lo; t < it.t_hi; ++t) {
            const int key0 = t * BN;
            const float *sK = sKV + (t & 1) * G::STAGE, *sV = sK + BN * G::PQ;
            copy_wait();
            __syncthreads();
            if (t + 1 < it.t_hi) {
                fetch(t + 1);
                look_up(t + 2);
            }
            float2 s2[RT][KT];                         // even and odd channels
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < KT; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                float4 a[RT], b[KT];
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    a[i] = *reinterpret_cast<const float4 *>(sQ + (ty * RT + i) * G::PQ + c);
#pragma unroll
                for (int j = 0; j < KT; ++j) b[j] = *reinterpret_cast<const float4 *>(sK + (tx + 16 * j) * G::PQ + c);
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < KT; ++j) {
                        s2[i][j] = fma2(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), s2[i][j]);
                        s2[i][j] = fma2(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), s2[i][j]);
                    }
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                float s[KT], mx = kLowest;
#pragma unroll
                for (int j = 0; j < KT; ++j) {
                    s[j] = key0 + tx + 16 * j <= kmax[i] ? (s2[i][j].x + s2[i][j].y) * scale_log2 : -INFINITY;
                    mx = fmaxf(mx, s[j]);
                }
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mn = fmaxf(m[i], mx), alpha = exp2f(m[i] - mn);
                m[i] = mn;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < KT; ++j) {
                    const float p = exp2f(s[j] - mn);
                    sum += p;
                    sP[(ty * RT + i) * G::PP + tx + 16 * j] = p;
                }
                l[i] = l[i] * alpha + sum;             // this thread's keys only
#pragma unroll
                for (int j = 0; j < CT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) acc[i][j][e] = mul2(acc[i][j][e], make_float2(alpha, alpha));
            }
            __syncwarp();                              // a row's 16 threads are in one warp
#pragma unroll 2
            for (int key = 0; key < BN; key += 4) {
                float4 p[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    p[i] = *reinterpret_cast<const float4 *>(sP + (ty * RT + i) * G::PP + key);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int j = 0; j < CT; ++j) {
                        const float4 v = *reinterpret_cast<const float4 *>(sV + (key + kk) * D + 4 * tx + 64 * j);
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                            acc[i][j][0] = fma2(make_float2(w, w), make_float2(v.x, v.y), acc[i][j][0]);
                            acc[i][j][1] = fma2(make_float2(w, w), make_float2(v.z, v.w), acc[i][j][1]);
                        }
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
            const int r = ty * RT + i;
            if (r >= it.rows) continue;
            if (it.whole) {
                float *o = out + token_row(r);
                const float inv = 1.f / l[i];
#pragma unroll
                for (int j = 0; j < CT; ++j)
                    *reinterpret_cast<float4 *>(o + 4 * tx + 64 * j) = make_float4(
                        acc[i][j][0].x * inv, acc[i][j][0].y * inv, acc[i][j][1].x * inv, acc[i][j][1].y * inv);
                if (lse_out && tx == 0) lse_out[token_row(r) / D] = m[i] + log2f(l[i]);
            } else {
                const size_t pr = parts.row(blockIdx.x, it.head ? 1 : 0, r);
#pragma unroll
                for (int j = 0; j < CT; ++j)
                    *reinterpret_cast<float4 *>(parts.o + pr * D + 4 * tx + 64 * j) =
                        make_float4(acc[i][j][0].x, acc[i][j][0].y, acc[i][j][1].x, acc[i][j][1].y);
                if (tx == 0) parts.ml[pr] = make_float2(m[i], l[i]);
            }
        }
        if (!it.whole && it.head && threadIdx.x == 0) {
            PartDesc &d = parts.desc[blockIdx.x];
            d.parts = it.parts;
            d.tok0 = it.tok0;
            d.h = it.h;
            d.row0 = row0;
            d.rows = it.rows;
        }
    }
}

// Where the key tiles that the block table can hold are fewer than three per SM
// and the sequences have this many rows on average, a cluster shares a tile's
// rows.  16/4 heads of 128, with the attention, rows shared and one CTA per tile:
// one prompt of 900 194 and 439 us, 8 prompts of 600 (320 tiles) 643 and 643, 4
// chunks of 300 over 2000 tokens (576 tiles) 1039 and 883.
constexpr long kSplitRows = 1024;

// ----- attention mass ---------------------------------------------------------------
// scores[b][h][slot] += sum over the rows that see the slot of p, with every
// row's final maximum and sum, as lse = maximum + log2(sum).  A cluster of Z CTAs
// per (b, h, 64-key tile) takes the sequence's rows in tiles of 64 in turn and
// adds its sums in the order of its ranks; every slot is written by one thread,
// in an order that the lengths fix.
template <int D, int Z>
__global__ void __cluster_dims__(1, 1, Z) __launch_bounds__(kThreads)
mass_simt_kernel(Pool P, WorkDim W, const float *__restrict__ q, int Hq, float scale_log2,
                 const float *__restrict__ lse, float *__restrict__ scores, int scores_stride)
{
    constexpr int BM = 64, BN = 64, PQ = D + 4;
    extern __shared__ __align__(16) float smf[];
    float *sQs = smf, *sK = sQs + 2 * BM * PQ, *sSum = sK + BN * PQ;      // sSum [16][BN]
    __shared__ float s_lse[2][BM], s_tot[BN];
    __shared__ int s_page[BN / 16];
    pdl_wait();
    pdl_trigger();
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15, G = W.G;
    const float *pk = (const float *)P.k;
    for (long u = blockIdx.x; u < (long)P.B * P.Hkv; u += gridDim.x) {
        const int b = (int)(u / P.Hkv), h = (int)(u % P.Hkv);
        const Seq s = load_seq(P, W.q_start, W.ctx_len, W.T, b);
        const int len = s.ctx + s.n;
        if (s.n == 0) continue;
        for (int key0 = blockIdx.y * BN; key0 < len; key0 += gridDim.y * BN) {
            __syncthreads();
            if (threadIdx.x < BN / 16) {
                const int slot = key0 + threadIdx.x * 16;
                s_page[threadIdx.x] = slot < len ? P.page_of(b, slot >> P.page_log2) : -1;
            }
            __syncthreads();
            load_rows<D>(sK, PQ, BN, [&](int r) -> const float * {
                const int pg = s_page[r >> 4], slot = key0 + r;
                return pg >= 0 && slot < len ? pk + P.row(pg, h, slot & (P.page() - 1)) * D : nullptr;
            });
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            const int rows = s.n * G;
            // rows before the first one that sees the tile's first key contribute nothing
            const int first = max(key0 - s.ctx, 0) * G / BM * BM;
            // Row tiles pass through two stages, as the attention's key tiles do.
            constexpr int CH = D / 4, RP = kThreads / CH;
            const int c4 = (int)threadIdx.x % CH * 4, tr = threadIdx.x / CH;
            const int di = RP / G, dg = RP - di * G;
            auto fetch = [&](int r0, int stage) {
                int i = (r0 + tr) / G, g = r0 + tr - i * G;
#pragma unroll
                for (int x = 0; x < BM / RP; ++x) {
                    const int r = tr + x * RP;
                    const bool on = r0 + r < rows;
                    const size_t at = on ? ((size_t)(s.tok0 + i) * Hq + h * G + g) * D + c4 : 0;
                    copy16(sQs + (stage * BM + r) * PQ + c4, q + at, on);
                    i += di, g += dg;
                    if (g >= G) g -= G, ++i;
                }
                if (threadIdx.x < BM) {
                    const int R = r0 + threadIdx.x, t = R / G;
                    const bool on = R < rows;
                    copy4(&s_lse[stage][threadIdx.x],
                          lse + (on ? (size_t)(s.tok0 + t) * Hq + h * G + (R - t * G) : 0), on);
                }
                copy_commit();
            };
            int stage = 0, r0 = first + (int)blockIdx.z * BM;
            if (r0 < rows) fetch(r0, 0);
            for (; r0 < rows; r0 += Z * BM, stage ^= 1) {
                copy_wait();
                __syncthreads();
                if (r0 + Z * BM < rows) fetch(r0 + Z * BM, stage ^ 1);
                const float *sQ = sQs + stage * BM * PQ;
                float2 a4[4][4];                       // even and odd channels
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) a4[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
                for (int c = 0; c < D; c += 4) {
                    float4 a[4], k4[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(sQ + (ty * 4 + i) * PQ + c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const float4 *>(sK + (tx + 16 * j) * PQ + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            a4[i][j] = fma2(make_float2(a[i].x, a[i].y), make_float2(k4[j].x, k4[j].y), a4[i][j]);
                            a4[i][j] = fma2(make_float2(a[i].z, a[i].w), make_float2(k4[j].z, k4[j].w), a4[i][j]);
                        }
                }
                int tok = (r0 + ty * 4) / G, g = r0 + ty * 4 - tok * G;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int kmax = r0 + ty * 4 + i < rows ? s.ctx + tok : -1;
                    const float e = s_lse[stage][ty * 4 + i];
                    if (++g == G) g = 0, ++tok;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (key0 + tx + 16 * j <= kmax)        // the score rounded as for the row's maximum
                            sum[j] += exp2f(__fsub_rn(__fmul_rn(a4[i][j].x + a4[i][j].y, scale_log2), e));
                }
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) sSum[ty * BN + tx + 16 * j] = sum[j];
            __syncthreads();
            if (threadIdx.x < BN && key0 + threadIdx.x < len) {
                float tot = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) tot += sSum[i * BN + threadIdx.x];
                float *dst = scores + (size_t)u * scores_stride + key0 + threadIdx.x;
                if constexpr (Z == 1) *dst += tot;
                else s_tot[threadIdx.x] = tot;
            }
            if constexpr (Z > 1) {
                cg::cluster_group cluster = cg::this_cluster();
                cluster.sync();
                if (blockIdx.z == 0 && threadIdx.x < BN && key0 + threadIdx.x < len) {
                    float tot = 0.f;
                    for (int z = 0; z < Z; ++z) tot += *cluster.map_shared_rank(&s_tot[threadIdx.x], z);
                    scores[(size_t)u * scores_stride + key0 + threadIdx.x] += tot;
                }
                cluster.sync();                        // the sums have been read
            }
        }
    }
}

template <int D, int BM, int BN>
cudaError_t launch_attn(const Pool &P, const WorkDim &W, const void *q, int Hq, float sl2, void *out, float *lse,
                        const Parts &parts, int n_cta, cudaStream_t st)
{
    auto kern = attn_simt_kernel<D, BM, BN>;
    constexpr int smem = Geom<D, BM, BN>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(n_cta), dim3(kThreads), smem, st, P, W, (const float *)q, Hq, sl2, (float *)out, lse, parts);
}

template <int D, int Z>
cudaError_t launch_mass(const Pool &P, const WorkDim &W, const void *q, int Hq, float sl2, const float *lse,
                        float *scores, int scores_stride, cudaStream_t st)
{
    auto kern = mass_simt_kernel<D, Z>;
    constexpr int smem = (3 * 64 * (D + 4) + 16 * 64) * 4;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // about six CTAs per SM over the units; a cluster strides over its unit's key tiles
    const int units = (int)std::min<long>((long)P.B * P.Hkv, 1 << 20);
    const int per_unit = (int)std::max<long>(1, std::min<long>(6l * device_sm_count() / ((long)units * Z), 65535));
    return launch_pdl(kern, dim3(units, per_unit, Z), dim3(kThreads), smem, st, P, W, (const float *)q, Hq, sl2, lse,
                      scores, scores_stride);
}

template <int D>
cudaError_t mass_rows(const Pool &P, const WorkDim &W, const void *q, int Hq, float sl2, const float *lse,
                      float *scores, int scores_stride, cudaStream_t st)
{
    const long tiles = (long)P.B * P.Hkv * ((P.capacity() + 63) / 64);
    if ((long)W.T * W.G >= kSplitRows * P.B && tiles <= 3l * device_sm_count())
        return launch_mass<D, 8>(P, W, q, Hq, sl2, lse, scores, scores_stride, st);
    return launch_mass<D, 1>(P, W, q, Hq, sl2, lse, scores, scores_stride, st);
}

}  // namespace

// rows a CTA holds: 16 where the batch has no more per sequence on average
// (decoding), else 64
int simt_rows(int T, int G, int B) { return (long)T * G <= 16l * B ? 16 : 64; }
int simt_ctas() { return 2 * device_sm_count(); }

cudaError_t attn_simt(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, void *out, float *lse,
                      const Parts &parts, cudaStream_t st)
{
    const int n = simt_ctas();
    if (simt_rows(W.T, W.G, P.B) == 16)
        return d == 128 ? launch_attn<128, 16, 32>(P, W, q, Hq, sl2, out, lse, parts, n, st)
                        : launch_attn<64, 16, 64>(P, W, q, Hq, sl2, out, lse, parts, n, st);
    return d == 128 ? launch_attn<128, 64, 32>(P, W, q, Hq, sl2, out, lse, parts, n, st)
                    : launch_attn<64, 64, 32>(P, W, q, Hq, sl2, out, lse, parts, n, st);
}

cudaError_t mass_simt(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, const float *lse,
                      float *scores, int scores_stride, cudaStream_t st)
{
    return d == 128 ? mass_rows<128>(P, W, q, Hq, sl2, lse, scores, scores_stride, st)
                    : mass_rows<64>(P, W, q, Hq, sl2, lse, scores, scores_stride, st);
}

}  // namespace paged
}  // namespace vc
