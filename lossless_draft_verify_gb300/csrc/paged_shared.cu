// paged_shared.cu -- attention of groups of sequences that share the pages of a
// prefix: the plan of such a batch, and the join of its two halves.
//
// A row's keys are its group's prefix and its sequence's own slots.  The plan has
// an entry per group, in which all rows of the group's sequences meet the prefix's
// keys (one pass over them, no mask), and one per sequence for its own slots.  The
// attention kernels take an entry as they take a sequence, and leave what they found
// of a row in fp32, in one piece or in several, with its place: o_i, sums l_i and
// maxima m_i, of which
//
//   o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,  M = max m_i.
//
// Both kernels here wait for round trips to L2, 3 and 5 us.  In a graph, with them, and
// without sharing (vc_paged_attn; most of its reads of a prefix hit L2), 32/8 heads of
// 128: one token of 32 sequences, a prefix of 32768 and up to 700 tokens of their own
// 59 and 428 us; 32 in two groups of up to 32000 over 8-bit pages 79 and 189; 24 chunks
// up to 17 in three groups, 28/4 heads, 81 and 105; four over 600 tokens 11.5 and 18,
// over 8192 and up to 300 of their own 21 and 30.
#include "paged.cuh"

namespace vc {
namespace paged {
namespace {

constexpr int kPlanThreads = 128;

// A group: its rows, and the slots that its sequences share: whole pages; none where
// it has one sequence only, or a length or range that does not fit.
struct Group {
    int row0, row1, slots;
};
__device__ __forceinline__ Group load_group(const Pool &P, const Groups &G, const int32_t *__restrict__ q_start, int T, int g)
{
    const int s0 = G.first[g], s1 = G.first[g + 1], n = G.prefix[g];
    if (s0 >= 0 && s1 >= s0 && s1 <= P.B && n >= 0 && n <= P.capacity()) {
        const int a = q_start[s0], e = q_start[s1];
        if (a >= 0 && e >= a && e <= T) return Group{a, e, s1 - s0 < 2 ? 0 : n & -P.page()};
    }
    set_flag(P.status, VC_PAGED_BAD_LENGTH);
    return Group{0, 0, 0};
}

__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(Pool P, const int32_t *__restrict__ q_start, const int32_t *__restrict__ ctx_len, int T, Groups G,
            VSeq *__restrict__ plan)
{
    pdl_wait();
    pdl_trigger();
    const int v = blockIdx.x * kPlanThreads + threadIdx.x;
    if (v >= G.n + P.B) return;
    VSeq s = {0, 0, 0, 1, 0, 0, 0, 0};
    if (v < G.n) {
        const Group g = load_group(P, G, q_start, T, v);
        if (g.slots > 0) s = VSeq{g.row0, g.row1 - g.row0, g.slots - 1, 0, 0, G.first[v], g.row0, 0};
    } else {
        const int b = v - G.n;
        const Seq q = load_seq(P, q_start, ctx_len, T, b);
        // the last group that begins at or before b
        int lo = 0, hi = G.n;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (G.first[mid] <= b) lo = mid + 1;
            else hi = mid;
        }
        int base = 0;
        if (lo > 0 && b < G.first[lo]) {
            const Group g = load_group(P, G, q_start, T, lo - 1);
            // (rows out of order: the group's do not hold these)
            if (g.row0 <= q.tok0 && q.tok0 + q.n <= g.row1) base = g.slots;
        }
        s = VSeq{q.tok0, q.n, q.ctx - base, 1, base, b, T + q.tok0, 0};
        if (q.n > 0 && q.ctx < base) {                       // a context that does not hold the prefix
            set_flag(P.status, VC_PAGED_BAD_LENGTH);
            s.n = 0;
        }
        if (s.n == 0) s.ctx = s.base = 0;
    }
    plan[v] = s;
}

// A row's parts by one warp, lane l at channels 4 l (2 l), or, where rows are few, by
// all warps of a CTA.  What it takes are round trips to L2: a warp asks for
// eight parts at once, and its running sum is rescaled by their maximum.
// Four sequences over a prefix of 32768 in 8-bit pages, 230 parts of a row (128 rows): 44
// us by a warp, 30 by eight; a decode step of 32 (1024 rows, 20 parts) 59 and 61.
constexpr int kAtOnce = 8;
constexpr long kSharedRows = 2;                              // per SM, at most: a CTA per row

template <bool SHARED>
constexpr int kJoinWarps = SHARED ? 8 : 4;

template <typename E, int D, bool SHARED>
__global__ void __launch_bounds__(32 * kJoinWarps<SHARED>)
join_kernel(int B, const int32_t *__restrict__ q_start, int T, int Hq, int heads, const VSeq *__restrict__ seqs, Halves H,
            Parts pre, Parts own, E *__restrict__ out)
{
    constexpr int V = D / 32, W = kJoinWarps<SHARED>, STEP = SHARED ? W : 1;
    __shared__ float s_acc[W][D];
    __shared__ float2 s_ml[W];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tok = SHARED ? blockIdx.x : blockIdx.x * W + warp;
    if (tok >= T) return;
    const size_t half = (size_t)T * Hq;
    auto place_of = [&](int x, int h) { return H.place[x * half + (size_t)tok * Hq + h]; };
    // (asked for before it is known whether they were written)
    Place at[2] = {place_of(0, blockIdx.y * heads), place_of(1, blockIdx.y * heads)};
    const int b = find_seq(q_start, B, tok);
    if (b < 0) return;
    const VSeq s = seqs[b];
    if (tok < s.tok0 || tok >= s.tok0 + s.n) return;
    for (int h = blockIdx.y * heads; h < min(Hq, (int)(blockIdx.y + 1) * heads); ++h) {
        const size_t row = (size_t)tok * Hq + h;
        if (h > (int)blockIdx.y * heads) at[0] = place_of(0, h), at[1] = place_of(1, h);
        if (!at[0].fits(pre)) at[0] = Place::in_output();
        if (!at[1].fits(own)) at[1] = Place::in_output();
        float M = kLowest, L = 0.f, acc[V];
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.f;
        // (a loop per half: with one over both a pass costs more than it saves, the
        // decode step below 67 us)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (x == 0 && s.base == 0) continue;
            const Parts &parts = x == 0 ? pre : own;
            const size_t here = x * half + row;
            const int n = at[x].parts();
            // a row in the output is one part with a sum of one
            for (int p0 = SHARED ? warp : 0; p0 < max(n, 1); p0 += kAtOnce * STEP) {
                float2 ml[kAtOnce];
                float y[kAtOnce][V];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const int p = p0 + k * STEP;
                    ml[k] = make_float2(kLowest, 0.f);
#pragma unroll
                    for (int e = 0; e < V; ++e) y[k][e] = 0.f;
                    if (p >= max(n, 1)) continue;
                    const size_t pr = n ? parts.row(at[x].cta() + p, p == 0 ? 1 : 0, at[x].r) : here;
                    ml[k] = n ? parts.ml[pr] : make_float2(H.lse[here], 1.f);
                    const float *o = (n ? parts.o : H.o) + pr * D + V * lane;
                    if constexpr (V == 4) {
                        const float4 z = *reinterpret_cast<const float4 *>(o);
                        y[k][0] = z.x, y[k][1] = z.y, y[k][2] = z.z, y[k][3] = z.w;
                    } else {
                        const float2 z = *reinterpret_cast<const float2 *>(o);
                        y[k][0] = z.x, y[k][1] = z.y;
                    }
                }
                float top = M;
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, ml[k].x);
                const float a = exp2f(M - top);
                M = top;
                L *= a;
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] *= a;
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const float w = exp2f(ml[k].x - top);
                    L = fmaf(w, ml[k].y, L);
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = fmaf(w, y[k][e], acc[e]);
                }
            }
        }
        if constexpr (SHARED) {
#pragma unroll
            for (int e = 0; e < V; ++e) s_acc[warp][V * lane + e] = acc[e];
            if (lane == 0) s_ml[warp] = make_float2(M, L);
            __syncthreads();
            if (threadIdx.x < D) {
                float x = 0.f;
                M = kLowest, L = 0.f;
                for (int k = 0; k < W; ++k) M = fmaxf(M, s_ml[k].x);
                for (int k = 0; k < W; ++k) {
                    const float w = exp2f(s_ml[k].x - M);
                    L = fmaf(w, s_ml[k].y, L);
                    x = fmaf(w, s_acc[k][threadIdx.x], x);
                }
                out[row * D + threadIdx.x] = Elem<E>::from_f(x / L);
            }
            __syncthreads();
        } else {
            const float inv = 1.f / L;
            E *dst = out + row * D + V * lane;
#pragma unroll
            for (int e = 0; e < V; ++e) dst[e] = Elem<E>::from_f(acc[e] * inv);
        }
    }
}

template <typename E, int D>
cudaError_t launch_join(int B, const int32_t *q_start, int T, int Hq, const VSeq *seqs, const Halves &H,
                        const Parts &pre, const Parts &own, void *out, cudaStream_t st)
{
    const long rows = (long)T * Hq;
    if (rows <= kSharedRows * device_sm_count())
        return launch_pdl(join_kernel<E, D, true>, dim3(T, Hq), dim3(32 * kJoinWarps<true>), 0, st, B, q_start, T, Hq, 1, seqs, H, pre, own, (E *)out);
    // a warp per head while there are warps to spare, else it looks up its token once
    const int heads = rows <= 64l * device_sm_count() ? 1 : std::max(4, cdiv(Hq, 65535));
    return launch_pdl(join_kernel<E, D, false>, dim3(cdiv(T, kJoinWarps<false>), cdiv(Hq, heads)),
                      dim3(32 * kJoinWarps<false>), 0, st, B, q_start, T, Hq, heads, seqs, H, pre, own, (E *)out);
}

}  // namespace

cudaError_t plan_shared(const Pool &P, const int32_t *q_start, const int32_t *ctx_len, int T, const Groups &G,
                        VSeq *plan, cudaStream_t st)
{
    return launch_pdl(plan_kernel, dim3(cdiv((long)G.n + P.B, kPlanThreads)), dim3(kPlanThreads), 0, st, P, q_start,
                      ctx_len, T, G, plan);
}

cudaError_t join_shared(const Pool &P, vc_dtype dt, int d, const int32_t *q_start, int T, int Hq, const VSeq *seqs,
                        const Halves &H, const Parts &pre, const Parts &own, void *out, cudaStream_t st)
{
    auto form = [&](auto elem) {
        using E = decltype(elem);
        return d == 128 ? launch_join<E, 128>(P.B, q_start, T, Hq, seqs, H, pre, own, out, st)
                        : launch_join<E, 64>(P.B, q_start, T, Hq, seqs, H, pre, own, out, st);
    };
    return dt == VC_BF16 ? form(__nv_bfloat16{}) : form(0.f);
}

}  // namespace paged
}  // namespace vc
