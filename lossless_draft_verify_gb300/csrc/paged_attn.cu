// paged_attn.cu -- causal attention of ragged chunks over a paged cache.
#include <type_traits>

#include "paged.cuh"

namespace vc {
namespace paged {
namespace {

// Merge the parts of the units that several CTAs share.  blockIdx.x: the CTA
// that holds the unit's first part; a warp per row, lane l at channels
// 4 l (+ 128).  With maxima m_i and sums l_i: o = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
constexpr int kMergeWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps)
merge_kernel(Parts parts, int G, int Hq, T *__restrict__ out, float *__restrict__ lse_out)
{
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x, lane = threadIdx.x & 31;
    const PartDesc d = parts.desc[c];
    if (d.parts == 0) return;
    for (int r = blockIdx.y * kMergeWarps + (threadIdx.x >> 5); r < d.rows; r += gridDim.y * kMergeWarps) {
        float M = kLowest;
        for (int p = lane; p < d.parts; p += 32) M = fmaxf(M, parts.ml[parts.row(c + p, p == 0 ? 1 : 0, r)].x);
        M = warp_max(M);
        constexpr int V = D / 32;
        float acc[V], L = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll 4
        for (int p = 0; p < d.parts; ++p) {
            const size_t pr = parts.row(c + p, p == 0 ? 1 : 0, r);
            const float2 ml = parts.ml[pr];
            const float w = exp2f(ml.x - M);
            L = fmaf(w, ml.y, L);
            if constexpr (V == 4) {
                const float4 o = *reinterpret_cast<const float4 *>(parts.o + pr * D + 4 * lane);
                acc[0] = fmaf(w, o.x, acc[0]);
                acc[1] = fmaf(w, o.y, acc[1]);
                acc[2] = fmaf(w, o.z, acc[2]);
                acc[3] = fmaf(w, o.w, acc[3]);
            } else {
                const float2 o = *reinterpret_cast<const float2 *>(parts.o + pr * D + 2 * lane);
                acc[0] = fmaf(w, o.x, acc[0]);
                acc[1] = fmaf(w, o.y, acc[1]);
            }
        }
        const int R = d.row0 + r;
        const size_t row = (size_t)(d.tok0 + R / G) * Hq + d.h * G + R % G;
        const float inv = 1.f / L;
        T *o = out + row * D + V * lane;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = Elem<T>::from_f(acc[e] * inv);
        if (lse_out && lane == 0) lse_out[row] = M + log2f(L);
    }
}

// scores[b][h][j] += sum over the sequence's rows that see slot j of 2^(s - lse),
// from stored products: four slots per thread, the rows one after another.  A
// score is rounded before lse is subtracted, as for the row's maximum, so that no
// weight exceeds one.  Bound
// by HBM: 4 bytes per row and slot read, 8 per slot for the sums.
constexpr int kSumThreads = 256, kSumSlots = 4 * kSumThreads;

__global__ void __launch_bounds__(kSumThreads)
sum_kernel(Pool P, WorkDim W, const float *__restrict__ s_in, long s_stride, float sl2, const float *__restrict__ lse,
           int Hq, float *__restrict__ scores, int scores_stride, int chunks)
{
    pdl_wait();
    pdl_trigger();
    const int u = blockIdx.x / chunks, b = u / P.Hkv, h = u % P.Hkv;
    const Seq s = load_seq(P, W.q_start, W.ctx_len, W.T, b);
    const int j = blockIdx.x % chunks * kSumSlots + 4 * threadIdx.x, len = s.ctx + s.n;
    if (s.n == 0 || j >= len) return;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    // rows before the first that sees slot j contribute nothing
    int i = max(j - s.ctx, 0), g = 0;
    size_t row = (size_t)(s.tok0 + i) * Hq + h * W.G;
    const int left = (s.n - i) * W.G;
#pragma unroll 4
    for (int r = 0; r < left; ++r) {
        const float4 x = *reinterpret_cast<const float4 *>(s_in + row * s_stride + j);
        const float e = lse[row];
        auto weight = [&](float s) { return ex2(__fsub_rn(__fmul_rn(s, sl2), e)); };
        const int last = s.ctx + i - j;                    // slots up to j + last are seen
        sum[0] += weight(x.x);
        if (last >= 1) sum[1] += weight(x.y);
        if (last >= 2) sum[2] += weight(x.z);
        if (last >= 3) sum[3] += weight(x.w);
        ++row;
        if (++g == W.G) {
            g = 0;
            ++i;
            row += Hq - W.G;
        }
    }
    float *dst = scores + (size_t)u * scores_stride + j;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (j + e < len) dst[e] += sum[e];
}

struct WsLayout {
    size_t desc, ml, o, rows, stored, bytes;
    int rows_cap, n_cta;
    long s_stride;             // stored products of a row; 0: not stored
};

// [status | desc | partial (m, l) | partial o | lse of every row | stored scores]
// The scores of a bf16 batch are stored, for the mass, where it has 16 rows per
// sequence and kv head at most on average.  Stored and with a second pass over
// K, 32/8 heads: one token of 16 sequences over 32768 372 and 507 us, four over
// 8000 133 and 153, eight (twice the rows) 166 and 153.
// They are sized by the table, which is as wide as the longest sequence a server
// allows: past kStoredMost bytes (a decode step of 256 sequences, 32 heads, 32768
// table slots) the memory is saved at the price of the second pass: full tables at
// the bound 5.39 ms, just past it 7.34 ms.
constexpr size_t kStoredMost = size_t(1) << 30;

WsLayout layout(vc_dtype dt, int d, int T, int G, int Hq, int B, long cap, bool with_rows)
{
    WsLayout w;
    w.n_cta = dt == VC_BF16 ? tc_ctas() : simt_ctas();
    const long unit = dt == VC_BF16 ? kTcRows : simt_rows(T, G, B);
    w.rows_cap = (int)std::min<long>(unit, (long)T * G);
    const size_t n = (size_t)w.n_cta * 2 * w.rows_cap;
    w.desc = kStatusBytes;
    w.ml = w.desc + align256((size_t)w.n_cta * sizeof(PartDesc));
    w.o = w.ml + align256(n * sizeof(float2));
    w.rows = w.o + align256(n * d * sizeof(float));
    w.stored = w.rows + (with_rows ? align256((size_t)T * Hq * sizeof(float)) : 0);
    w.s_stride = (cap + kTcKeys - 1) / kTcKeys * kTcKeys;
    if (!with_rows || dt != VC_BF16 || (long)T * G > 16l * B || (size_t)T * Hq * w.s_stride * sizeof(float) > kStoredMost)
        w.s_stride = 0;
    w.bytes = w.stored + align256((size_t)T * Hq * w.s_stride * sizeof(float));
    return w;
}

template <typename T>
cudaError_t merge(const Parts &parts, int n_cta, int rows, int d, int G, int Hq, void *out, float *lse,
                  cudaStream_t st)
{
    const dim3 grid(n_cta, cdiv(rows, kMergeWarps));
    return d == 128 ? launch_pdl(merge_kernel<T, 128>, grid, dim3(32 * kMergeWarps), 0, st, parts, G, Hq, (T *)out, lse)
                    : launch_pdl(merge_kernel<T, 64>, grid, dim3(32 * kMergeWarps), 0, st, parts, G, Hq, (T *)out, lse);
}

template <typename T>
cudaError_t run(const Pool &P, const WorkDim &W, vc_dtype dt, int d, const void *q, int Hq, float sl2, void *out,
                float *scores, int scores_stride, uint8_t *ws, cudaStream_t st)
{
    const long cap = P.capacity();
    const WsLayout w = layout(dt, d, W.T, W.G, Hq, P.B, cap, scores != nullptr);
    Parts parts = {(PartDesc *)(ws + w.desc), (float2 *)(ws + w.ml), (float *)(ws + w.o), w.rows_cap};
    float *lse = scores ? (float *)(ws + w.rows) : nullptr;
    float *stored = w.s_stride ? (float *)(ws + w.stored) : nullptr;
    cudaError_t e;
    if constexpr (std::is_same_v<T, float>) e = attn_simt(P, W, d, q, Hq, sl2, out, lse, parts, st);
    else e = attn_tc(P, W, d, q, Hq, sl2, out, lse, stored, w.s_stride, parts, (int32_t *)ws, st);
    // no unit is cut where the block table cannot hold a sequence long enough
    constexpr int tile = std::is_same_v<T, float> ? kSimtKeys : kTcKeys, weight = std::is_same_v<T, float> ? 1 : 2;
    using C = Cost<std::is_same_v<T, float> ? 64 : kTcRows>;
    if (e == cudaSuccess && (cap + tile - 1) / tile * weight + C::kUnitCost > C::kWhole)
        e = merge<T>(parts, w.n_cta, w.rows_cap, d, W.G, Hq, out, lse, st);
    if (e != cudaSuccess || !scores) return e;
    if constexpr (std::is_same_v<T, float>) {
        return mass_simt(P, W, d, q, Hq, sl2, lse, scores, scores_stride, st);
    } else {
        if (!stored) return mass_tc(P, W, d, q, Hq, sl2, lse, scores, scores_stride, (int32_t *)ws, st);
        const int chunks = cdiv(cap, kSumSlots);
        return launch_pdl(sum_kernel, dim3((unsigned)(P.B * P.Hkv) * chunks), dim3(kSumThreads), 0, st, P, W,
                          (const float *)stored, w.s_stride, sl2, (const float *)lse, Hq, scores, scores_stride, chunks);
    }
}

}  // namespace

size_t attn_ws_bytes(vc_dtype dt, int d, int T, int Hq, int Hkv, int B, long cap, bool mass)
{
    return layout(dt, d, T, Hq / Hkv, Hq, B, cap, mass).bytes;
}

cudaError_t attn(const Pool &P, vc_dtype dt, int d, const void *q, const int32_t *q_start, const int32_t *ctx_len,
                 int T, int Hq, float sm_scale, void *out, float *scores, int scores_stride, void *ws, cudaStream_t st)
{
    WorkDim W;
    W.q_start = q_start;
    W.ctx_len = ctx_len;
    W.T = T;
    W.G = Hq / P.Hkv;
    const float sl2 = sm_scale * kLog2e;
    return dt == VC_BF16 ? run<__nv_bfloat16>(P, W, dt, d, q, Hq, sl2, out, scores, scores_stride, (uint8_t *)ws, st)
                         : run<float>(P, W, dt, d, q, Hq, sl2, out, scores, scores_stride, (uint8_t *)ws, st);
}

}  // namespace paged
}  // namespace vc
