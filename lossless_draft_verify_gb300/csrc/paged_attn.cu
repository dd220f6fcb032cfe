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

// The same where pieces are many and small (a warp's each).  A CTA looks at the
// descriptions of eight pieces (sixteen: fp32 chunks up to 17 over 2000 18.8 against 16.6
// us, four tokens of 16 over 8192 72 against 69, else the same).  Units of few parts: a warp per row.  Others: the
// warps share the rows and, where those are fewer, their parts.  What it takes are
// round trips to L2, so a warp asks for eight parts at once and rescales its running
// sum by their maximum.  Of a decode step (16 sequences of 32768 tokens, 32/8 heads)
// with a warp per row 180 us in all, with shared parts 173.
constexpr int kManyWarps = 16, kPieces = 8, kFewParts = 4, kAtOnce = 8;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kManyWarps)
merge_many_kernel(Parts parts, int n_piece, int G, int Hq, T *__restrict__ out)
{
    constexpr int V = D / 32;
    __shared__ PartDesc s_desc[kPieces];
    __shared__ float s_acc[kManyWarps][D];
    __shared__ float2 s_ml[kManyWarps];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c0 = blockIdx.x * kPieces;
    if (lane == 0 && warp < kPieces) {
        if (c0 + warp < n_piece) s_desc[warp] = parts.desc[c0 + warp];
        else s_desc[warp].parts = 0;
    }
    __syncthreads();
    float acc[V], M, L;
    auto join = [&](float m, float l, const float (&x)[V]) {
        const float top = fmaxf(M, m), a = ex2(M - top), b = ex2(m - top);
        M = top;
        L = fmaf(b, l, L * a);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(b, x[e], acc[e] * a);
    };
    // parts p0, p0 + step .. of row r of the unit that begins in piece c0 + i
    auto add = [&](int i, int n, int r, int p0, int step) {
        M = kLowest, L = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.f;
        for (int p = p0; p < n; p += kAtOnce * step) {
            float2 ml[kAtOnce];
            float x[kAtOnce][V];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int pk = p + k * step;
                ml[k] = make_float2(kLowest, 0.f);
#pragma unroll
                for (int e = 0; e < V; ++e) x[k][e] = 0.f;
                if (pk >= n) continue;
                const size_t at = parts.row(c0 + i + pk, pk == 0 ? 1 : 0, r);
                ml[k] = parts.ml[at];
                const float *o = parts.o + at * D + V * lane;
                if constexpr (V == 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(o);
                    x[k][0] = y.x, x[k][1] = y.y, x[k][2] = y.z, x[k][3] = y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2 *>(o);
                    x[k][0] = y.x, x[k][1] = y.y;
                }
            }
            float top = M;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, ml[k].x);
            const float a = ex2(M - top);
            M = top;
            L *= a;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] *= a;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const float w = ex2(ml[k].x - top);
                L = fmaf(w, ml[k].y, L);
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = fmaf(w, x[k][e], acc[e]);
            }
        }
    };
    auto store = [&](const PartDesc &d, int r) {
        const int R = d.row0 + r;
        const float inv = 1.f / L;
        const size_t row = (size_t)(d.tok0 + R / G) * Hq + d.h * G + R % G;
        T *o = out + row * D + V * lane;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = Elem<T>::from_f(acc[e] * inv);
    };
    // units of few parts, and of many
    const int n_parts = s_desc[lane % kPieces].parts;
    unsigned few = __ballot_sync(0xffffffffu, lane < kPieces && n_parts > 0 && n_parts <= kFewParts);
    unsigned many = __ballot_sync(0xffffffffu, lane < kPieces && n_parts > kFewParts);
    int turn = 0;
    for (; few; few &= few - 1) {
        const int i = __ffs(few) - 1;
        const PartDesc d = s_desc[i];
        for (int r = 0; r < d.rows; ++r) {
            if (turn++ % kManyWarps != warp) continue;
            add(i, d.parts, r, 0, 1);
            store(d, r);
        }
    }
    for (; many; many &= many - 1) {
        const int i = __ffs(many) - 1;
        const PartDesc d = s_desc[i];
        int share = kManyWarps;                              // warps per row
        while (share > 1 && d.rows * share > kManyWarps) share /= 2;
        const int sub = warp % share;
        for (int r0 = 0; r0 < d.rows; r0 += kManyWarps / share) {
            const int r = r0 + warp / share;
            add(i, r < d.rows ? d.parts : 0, r, sub, share);
#pragma unroll
            for (int e = 0; e < V; ++e) s_acc[warp][V * lane + e] = acc[e];
            if (lane == 0) s_ml[warp] = make_float2(M, L);
            __syncthreads();
            if (sub == 0 && r < d.rows) {
                for (int k = 1; k < share; ++k) {
                    float x[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) x[e] = s_acc[warp + k][V * lane + e];
                    join(s_ml[warp + k].x, s_ml[warp + k].y, x);
                }
                store(d, r);
            }
            __syncthreads();
        }
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
    size_t desc, ml, o, rows, stored, k, v, table, bytes;
    bool expand;               // 8-bit pages: taken as bf16 pages at k, v
    int rows_cap, n_cta;
    long s_stride;             // stored products of a row; 0: not stored
};

// [status | desc | partial (m, l) | partial o | lse of every row | stored scores |
//  expanded K | V | table]
// The scores of a bf16 batch are stored, for the mass, where it has 16 rows per
// sequence and kv head at most on average.  Stored and with a second pass over
// K, 32/8 heads: one token of 16 sequences over 32768 372 and 507 us, four over
// 8000 133 and 153, eight (twice the rows) 166 and 153.
// They are sized by the table, which is as wide as the longest sequence a server
// allows: past kStoredMost bytes (a decode step of 256 sequences, 32 heads, 32768
// table slots) the memory is saved at the price of the second pass: full tables at
// the bound 5.39 ms, just past it 7.34 ms.
constexpr size_t kStoredMost = size_t(1) << 30;
// 8-bit pages that many row tiles read (rows per sequence and kv head, on average)
// are expanded to bf16 pages once instead of by each tile, where those, again by the
// table, take no more memory than that.  Chunks over 30000 tokens, 32/8 heads, by each
// tile and once: heads of 128, 512 tokens (2048 rows) 243 and 242 us, 1024 467 and 418,
// 2048 915 and 766; heads of 64, 188 and 199, 362 and 357, 704 and 674.
constexpr long kExpandRows = 4096;
constexpr size_t kExpandMost = size_t(1) << 30;

// A batch over 8-bit pages whose rows are few, or fp32, takes a kernel of its own.
// The rows of its units, 8 or 16; 0: the batch does not.
int few_unit(vc_dtype dt, int T, int G, int B, bool kv8)
{
    const int rows = kv8 ? few_rows(T, G, B) : 0;
    return rows || !kv8 || dt == VC_BF16 ? rows : 16;
}

WsLayout layout(vc_dtype dt, int d, int T, int G, int Hq, int B, long cap, bool with_rows, bool kv8, bool planned = false,
                int few = 0)
{
    WsLayout w;
    if (!planned && !few) few = few_unit(dt, T, G, B, kv8);
    w.n_cta = few ? few_pieces(few) : dt == VC_BF16 ? tc_ctas() : simt_ctas();
    const long unit = few ? few : dt == VC_BF16 ? kTcRows : simt_rows(T, G, B, planned);
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
    w.k = w.stored + align256((size_t)T * Hq * w.s_stride * sizeof(float));
    const size_t pages = (size_t)B * cap * (Hq / G) * d * 2;             // bytes of K or V
    w.expand = kv8 && !planned && !few && (long)T * G >= kExpandRows * B && 2 * pages <= kExpandMost && Hq / G <= 65535;
    w.v = w.k + (w.expand ? align256(pages) : 0);
    w.table = w.v + (w.expand ? align256(pages) : 0);
    w.bytes = w.table + (w.expand ? align256((size_t)B * (cap / 16) * sizeof(int32_t)) : 0);      // pages of 16 at least
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

template <typename E>
cudaError_t merge_many(const Parts &parts, int n_piece, int d, int G, int Hq, void *out, cudaStream_t st)
{
    const dim3 grid(cdiv(n_piece, kPieces)), block(32 * kManyWarps);
    return d == 128 ? launch_pdl(merge_many_kernel<E, 128>, grid, block, 0, st, parts, n_piece, G, Hq, (E *)out)
                    : launch_pdl(merge_many_kernel<E, 64>, grid, block, 0, st, parts, n_piece, G, Hq, (E *)out);
}

// whether a unit can be cut: not where the block table cannot hold a sequence
// long enough
bool may_cut_few(long cap, int d, bool kv8)
{
    return (cap + few_keys(d, kv8) - 1) / few_keys(d, kv8) + CostFew::kUnitCost > CostFew::kWhole;
}

template <typename T>
bool may_cut(long cap)
{
    constexpr int tile = std::is_same_v<T, float> ? kSimtKeys : kTcKeys, weight = std::is_same_v<T, float> ? 1 : 2;
    using C = Cost<std::is_same_v<T, float> ? 64 : kTcRows>;
    return (cap + tile - 1) / tile * weight + C::kUnitCost > C::kWhole;
}

template <typename T>
cudaError_t run(const Pool &P, const WorkDim &W, vc_dtype dt, int d, const void *q, int Hq, float sl2, void *out,
                float *scores, int scores_stride, uint8_t *ws, cudaStream_t st)
{
    const long cap = P.capacity();
    const WsLayout w = layout(dt, d, W.T, W.G, Hq, P.B, cap, scores != nullptr, P.k_scale);
    Parts parts = {(PartDesc *)(ws + w.desc), (float2 *)(ws + w.ml), (float *)(ws + w.o), w.rows_cap, w.n_cta};
    float *lse = scores ? (float *)(ws + w.rows) : nullptr;
    float *stored = w.s_stride ? (float *)(ws + w.stored) : nullptr;
    cudaError_t e;
    const int few = few_unit(dt, W.T, W.G, P.B, P.k_scale);
    if (few) e = attn8_few(P, W, dt, d, few, q, Hq, sl2, out, parts, (int32_t *)ws, st);
    else if constexpr (std::is_same_v<T, float>) e = attn_simt(P, W, d, q, Hq, sl2, out, lse, parts, st);
    else if (w.expand) {
        Pool X = P;
        X.k = ws + w.k;
        X.v = ws + w.v;
        X.k_scale = X.v_scale = nullptr;
        X.table = (const int32_t *)(ws + w.table);
        X.n_pages = P.B * P.max_blocks;
        e = expand8(P, d, W.q_start, W.ctx_len, W.T, X.k, X.v, (int32_t *)(ws + w.table), st);
        if (e == cudaSuccess) e = attn_tc(X, W, d, q, Hq, sl2, out, nullptr, nullptr, 0, parts, (int32_t *)ws, st);
    } else if (P.k_scale) e = attn8_tc(P, W, d, q, Hq, sl2, out, parts, (int32_t *)ws, st);
    else e = attn_tc(P, W, d, q, Hq, sl2, out, lse, stored, w.s_stride, parts, (int32_t *)ws, st);
    if (e == cudaSuccess && (few ? may_cut_few(cap, d, true) : may_cut<T>(cap)))
        e = few ? merge_many<T>(parts, w.n_cta, d, W.G, Hq, out, st)
                : merge<T>(parts, w.n_cta, w.rows_cap, d, W.G, Hq, out, lse, st);
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

// [the attention's | that of the kernel of few rows, where it has a part | plan |
// places, lse and o of both halves]
struct SharedLayout {
    WsLayout attn, own;
    int few;                   // rows of a unit of the kernel of few rows; 0: it has no part
    bool all;                  // it takes all, else the sequences' own slots
    size_t own_at, plan, place, lse, o, bytes;
};

// Where groups have at most this many rows per kv head, on average (their ranges lie on the
// device), the kernel of few rows
// takes the prefixes too: a launch and units of 8 us less, a pass over the prefix more for
// each 16 rows.  Through the tensor-core kernel and so, contexts of up to 300 after the
// prefix, 32/8 heads of 128, bf16 and 8-bit pages: 4 sequences (16 rows) over 512 28, 22
// and 14, 17 us, over 8192 34, 33 and 21, 20, over 32768 48, 50 and 40, 31; 8 over 512
// 29, 30 and 16, 17, over 8192 34, 40 and 26, 23, over 32768 48, 49 and 57, 45; 16 over
// 512 29, 31 and 17, 19, over 8192 35, 41 and 38, 34, over 32768 51, 52 and 99, 75.
// One group of 32 over 8000 beside 15 of two over 100: 64 and 52 us (without sharing 156
// and 87).
constexpr long kGroupRows = 32;

SharedLayout shared_layout(vc_dtype dt, int d, int T, int G, int Hq, int B, long cap, int n_groups, bool kv8)
{
    SharedLayout w;
    const size_t rows = (size_t)2 * T * Hq;
    w.attn = layout(dt, d, T, G, Hq, B, cap, false, false, true);
    w.few = dt == VC_BF16 ? few_rows(T, G, B) : kv8 ? 16 : 0;
    w.all = w.few && (dt == VC_F32 || n_groups == 0 || (long)T * G <= kGroupRows * n_groups);
    if (w.all && dt == VC_BF16 && n_groups) w.few = (long)T * G <= 8l * n_groups ? 8 : 16;
    w.own_at = w.attn.bytes;
    w.own.bytes = 0;
    if (w.few) w.own = layout(dt, d, T, G, Hq, B, cap, false, true, false, w.few);
    w.plan = w.own_at + w.own.bytes;
    w.place = w.plan + align256(((size_t)B + n_groups) * sizeof(VSeq));
    w.lse = w.place + align256(rows * sizeof(Place));
    w.o = w.lse + align256(rows * sizeof(float));
    w.bytes = w.o + rows * d * sizeof(float);
    return w;
}

template <typename T>
cudaError_t run_shared(const Pool &P, WorkDim W, vc_dtype dt, int d, const void *q, int Hq, float sl2, const Groups &G,
                       void *out, uint8_t *ws, cudaStream_t st)
{
    const SharedLayout w = shared_layout(dt, d, W.T, W.G, Hq, P.B, P.capacity(), G.n, P.k_scale);
    auto parts_at = [&](const WsLayout &x, uint8_t *at) {
        return Parts{(PartDesc *)(at + x.desc), (float2 *)(at + x.ml), (float *)(at + x.o), x.rows_cap, x.n_cta};
    };
    const Parts parts = parts_at(w.attn, ws), own = w.few ? parts_at(w.own, ws + w.own_at) : parts;
    const Halves H = {(float *)(ws + w.o), (float *)(ws + w.lse), (Place *)(ws + w.place)};
    VSeq *plan = (VSeq *)(ws + w.plan);
    int32_t *status = (int32_t *)ws;
    cudaError_t e = plan_shared(P, W.q_start, W.ctx_len, W.T, G, plan, st);
    if (e != cudaSuccess) return e;
    W.plan = plan;
    W.n_plan = w.few && !w.all ? G.n : P.B + G.n;
    auto few = [&] {
        return P.k_scale ? attn8_few_planned(P, W, dt, d, w.few, q, Hq, sl2, H, w.all, own, status, st)
                         : attn_few_planned(P, W, d, w.few, q, Hq, sl2, H, w.all, own, status, st);
    };
    if (w.all) e = few();
    else if constexpr (std::is_same_v<T, float>) e = attn_simt(P, W, d, q, Hq, sl2, H.o, H.lse, parts, st, H.place);
    else if (P.k_scale) e = attn8_tc_planned(P, W, d, q, Hq, sl2, H, parts, status, st);
    else e = attn_tc_planned(P, W, d, q, Hq, sl2, H, parts, status, st);
    if (e == cudaSuccess && w.few && !w.all) {
        // The kernel before took the prefixes; the sequences' own slots follow beside its end.
        W.plan = plan + G.n;
        W.n_plan = P.B;
        e = few();
    }
    if (e != cudaSuccess) return e;
    return join_shared(P, dt, d, W.q_start, W.T, Hq, plan + G.n, H, w.all ? own : parts, own, out, st);
}

}  // namespace

// The kernels of few rows need more than those of a few more: what a batch of T rows
// is asked for is enough for one of fewer rows, too.  (Of as many as take one kernel
// the largest batch needs most.)
template <typename F>
size_t most_up_to(int T, int G, int B, int n_groups, F bytes)
{
    auto at = [&](long rows) { return bytes((int)std::min<long>(T, rows / G)); };
    return std::max({bytes(T), at(8l * B), at(16l * B), at(8l * n_groups), at(kGroupRows * n_groups)});
}

size_t attn_ws_bytes(vc_dtype dt, int d, int T, int Hq, int Hkv, int B, long cap, bool mass, bool kv8)
{
    auto bytes = [&](int t) { return layout(dt, d, t, Hq / Hkv, Hq, B, cap, mass, kv8).bytes; };
    return kv8 ? most_up_to(T, Hq / Hkv, B, 0, bytes) : bytes(T);
}

size_t attn_shared_ws_bytes(vc_dtype dt, int d, int T, int Hq, int Hkv, int B, long cap, int n_groups, bool kv8)
{
    return most_up_to(T, Hq / Hkv, B, n_groups,
                      [&](int t) { return shared_layout(dt, d, t, Hq / Hkv, Hq, B, cap, n_groups, kv8).bytes; });
}

cudaError_t attn(const Pool &P, vc_dtype dt, int d, const void *q, const int32_t *q_start, const int32_t *ctx_len,
                 int T, int Hq, float sm_scale, void *out, float *scores, int scores_stride, void *ws, cudaStream_t st)
{
    const WorkDim W = {q_start, ctx_len, T, Hq / P.Hkv, nullptr, 0};
    const float sl2 = sm_scale * kLog2e;
    return dt == VC_BF16 ? run<__nv_bfloat16>(P, W, dt, d, q, Hq, sl2, out, scores, scores_stride, (uint8_t *)ws, st)
                         : run<float>(P, W, dt, d, q, Hq, sl2, out, scores, scores_stride, (uint8_t *)ws, st);
}

cudaError_t attn_shared(const Pool &P, vc_dtype dt, int d, const void *q, const Groups &G, const int32_t *q_start,
                        const int32_t *ctx_len, int T, int Hq, float sm_scale, void *out, void *ws, cudaStream_t st)
{
    const WorkDim W = {q_start, ctx_len, T, Hq / P.Hkv, nullptr, 0};
    const float sl2 = sm_scale * kLog2e;
    return dt == VC_BF16 ? run_shared<__nv_bfloat16>(P, W, dt, d, q, Hq, sl2, G, out, (uint8_t *)ws, st)
                         : run_shared<float>(P, W, dt, d, q, Hq, sl2, G, out, (uint8_t *)ws, st);
}

}  // namespace paged
}  // namespace vc
