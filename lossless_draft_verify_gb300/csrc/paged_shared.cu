// paged_shared.cu -- attention of groups of sequences that share the pages of a
// prefix: the plan of such a batch, and the join of its two halves.
//
// A row's keys are its group's prefix and its sequence's own slots.  The plan has
// an entry per group, in which all rows of the group's sequences meet the prefix's
// keys (one pass over them, no mask), and one per sequence for its own slots.  The
// attention kernels take an entry as they take a sequence; each half of a row
// leaves o_i (normalised) and lse_i = log2 sum 2^s in fp32, and
//
//   o = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M),  M = max lse_i.
#include "paged.cuh"

namespace vc {
namespace paged {
namespace {

constexpr int kPlanThreads = 128;

// Slots of group g that its sequences share: whole pages; none where it has one
// sequence only, or a length or range that does not fit.
__device__ __forceinline__ int shared_slots(const Pool &P, const Groups &G, int g)
{
    const int s0 = G.first[g], s1 = G.first[g + 1], n = G.prefix[g];
    if (s0 < 0 || s1 < s0 || s1 > P.B || n < 0 || n > P.capacity()) {
        set_flag(P.status, VC_PAGED_BAD_LENGTH);
        return 0;
    }
    return s1 - s0 < 2 ? 0 : n & -P.page();
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
        const int n = shared_slots(P, G, v);
        if (n > 0) {
            const int a = q_start[G.first[v]], e = q_start[G.first[v + 1]];
            if (a >= 0 && e >= a && e <= T) s = VSeq{a, e - a, n - 1, 0, 0, G.first[v], a, 0};
        }
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
        if (lo > 0 && b < G.first[lo]) base = shared_slots(P, G, lo - 1);
        s = VSeq{q.tok0, q.n, q.ctx - base, 1, base, b, T + q.tok0, 0};
        if (q.n > 0 && q.ctx < base) {                       // a context that does not hold the prefix
            set_flag(P.status, VC_PAGED_BAD_LENGTH);
            s.n = 0;
        }
        if (s.n == 0) s.ctx = s.base = 0;
    }
    plan[v] = s;
}

// A warp per (row, four heads), lane l at channels 4 l (2 l) of each.
constexpr int kJoinWarps = 4, kJoinHeads = 4;

template <typename E, int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
join_kernel(int B, const int32_t *__restrict__ q_start, int T, int Hq, const VSeq *__restrict__ seqs,
            const float *__restrict__ o, const float *__restrict__ lse, E *__restrict__ out)
{
    pdl_wait();
    pdl_trigger();
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31, tok = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    if (tok >= T) return;
    const int b = find_seq(q_start, B, tok);
    if (b < 0) return;
    const VSeq s = seqs[b];
    if (tok < s.tok0 || tok >= s.tok0 + s.n) return;
    const size_t half = (size_t)T * Hq;
#pragma unroll
    for (int i = 0; i < kJoinHeads; ++i) {
        const int h = blockIdx.y * kJoinHeads + i;
        if (h >= Hq) return;
        const size_t row = (size_t)tok * Hq + h;
        float x[V];
        const float *own = o + (half + row) * D + V * lane, *pre = o + row * D + V * lane;
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = own[e];
        if (s.base > 0) {
            const float a = lse[row], c = lse[half + row], M = fmaxf(a, c);
            float wa = exp2f(a - M), wc = exp2f(c - M);
            const float inv = 1.f / (wa + wc);
            wa *= inv, wc *= inv;
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = fmaf(wa, pre[e], wc * x[e]);
        }
        E *dst = out + row * D + V * lane;
#pragma unroll
        for (int e = 0; e < V; ++e) dst[e] = Elem<E>::from_f(x[e]);
    }
}

template <typename E>
cudaError_t launch_join(int B, const int32_t *q_start, int T, int Hq, int d, const VSeq *seqs, const float *o,
                        const float *lse, void *out, cudaStream_t st)
{
    const dim3 grid(cdiv(T, kJoinWarps), cdiv(Hq, kJoinHeads)), block(32 * kJoinWarps);
    return d == 128 ? launch_pdl(join_kernel<E, 128>, grid, block, 0, st, B, q_start, T, Hq, seqs, o, lse, (E *)out)
                    : launch_pdl(join_kernel<E, 64>, grid, block, 0, st, B, q_start, T, Hq, seqs, o, lse, (E *)out);
}

}  // namespace

cudaError_t plan_shared(const Pool &P, const int32_t *q_start, const int32_t *ctx_len, int T, const Groups &G,
                        VSeq *plan, cudaStream_t st)
{
    return launch_pdl(plan_kernel, dim3(cdiv((long)G.n + P.B, kPlanThreads)), dim3(kPlanThreads), 0, st, P, q_start,
                      ctx_len, T, G, plan);
}

cudaError_t join_shared(const Pool &P, vc_dtype dt, int d, const int32_t *q_start, int T, int Hq, const VSeq *seqs,
                        const float *o, const float *lse, void *out, cudaStream_t st)
{
    return dt == VC_BF16 ? launch_join<__nv_bfloat16>(P.B, q_start, T, Hq, d, seqs, o, lse, out, st)
                         : launch_join<float>(P.B, q_start, T, Hq, d, seqs, o, lse, out, st);
}

}  // namespace paged
}  // namespace vc
