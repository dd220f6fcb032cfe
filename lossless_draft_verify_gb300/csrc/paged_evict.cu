// paged_evict.cu -- eviction from a paged cache by accumulated attention
// weight: per (sequence, kv head) the `recent` newest slots and the `top`
// best-scored older ones move, in ascending order, to other pages.
//
// Selection is exact: the kept set is the largest by (score descending, slot
// ascending).  One CTA, or a cluster of eight, takes one (sequence, head): an
// MSB-first radix select (11 + 11 + 10 bits of an order-preserving integer
// image of the scores) with one histogram per CTA in shared memory finds the
// threshold; in a cluster each CTA adds up an eighth of the digits through
// distributed shared memory, and the one that holds the searched digit tells
// the others.
// Every warp owns a run of consecutive slots; its counts above and at the
// threshold, prefixed over warps and CTAs, give the place of its first kept
// slot, and ballots order the rest.  The scores are read from memory once, 16
// loads in flight per thread, and kept in shared memory for the further passes
// (read again where a CTA has more than 16384).  A second kernel moves the
// rows: one read and one write of every kept row, which is what bounds the
// call.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace cg = cooperative_groups;

namespace vc {
namespace paged {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kCache = 16384;                          // scores a CTA keeps: 64 KB, two CTAs per SM

// One pattern per score: -0 as +0, every NaN as the all-ones one.
__device__ __forceinline__ uint32_t score_bits(float s)
{
    const uint32_t u = s == 0.f ? 0u : __float_as_uint(s);
    return s != s ? 0xffffffffu : u;
}
// larger score -> larger key; NaN, the lowest, is 0
__device__ __forceinline__ uint32_t score_key(uint32_t bits)
{
    return bits ^ ((uint32_t)((int32_t)bits >> 31) | 0x80000000u);
}

struct EvictParams {
    const float *scores;
    const int32_t *src_len;
    int32_t *dst_len, *kept_idx;
    float *scores_out;
    int scores_stride, kept_stride, out_stride, cache;
    long top, recent;
};

// tokens of sequence b; 0 (and the status bit) when they do not fit the table
__device__ __forceinline__ int src_tokens(const Pool &S, const int32_t *src_len, int b)
{
    const int L = src_len[b];
    if (L >= 0 && L <= S.capacity()) return L;
    atomicOr(S.status, VC_PAGED_BAD_LENGTH);
    return 0;
}

constexpr int kWarps = kThreads / 32;
// f(slot, bits, in range) for the slots of [lo, hi) that fall to the caller,
// `at` and every `stride`th from there on; all lanes of a warp run alike.  16
// loads are in flight per thread.
template <typename L, typename F>
__device__ __forceinline__ void for_scores(int lo, int hi, int at, int stride, L load, F f)
{
    constexpr int N = 16;
    int i = lo + at;
    for (; i - at + stride * N <= hi; i += stride * N) {
        uint32_t x[N];
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = load(i + e * stride);
#pragma unroll
        for (int e = 0; e < N; ++e) f(i + e * stride, x[e], true);
    }
    for (; i - at < hi; i += stride * 4) {
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = i + e * stride < hi ? load(i + e * stride) : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) f(i + e * stride, x[e], i + e * stride < hi);
    }
}

template <int Z>
__global__ void __cluster_dims__(Z, 1, 1) __launch_bounds__(kThreads)
select_kernel(Pool S, EvictParams E)
{
    __shared__ __align__(16) int hist[kBins];
    __shared__ int warp_sums[kWarps];
    __shared__ int s_slice[Z];                         // the CTAs' totals of their digits, of this pass
    __shared__ int s_digit, s_above;
    extern __shared__ uint32_t cache[];
    __shared__ int2 s_count[kWarps + 1];               // slots above / at the threshold: by warp, of the CTA
    cg::cluster_group cluster = cg::this_cluster();
    auto sync_all = [&] {
        if constexpr (Z == 1) __syncthreads();
        else cluster.sync();
    };
    pdl_wait();
    pdl_trigger();
    const int unit = blockIdx.x / Z, rank = (int)(blockIdx.x % Z);
    const int b = unit / S.Hkv;
    const int L = src_tokens(S, E.src_len, b);
    const int recent = (int)min(E.recent, (long)L), cand = L - recent;
    const int top = (int)min(E.top, (long)cand), keep = top + recent;
    const float *sc = E.scores + (size_t)unit * E.scores_stride;
    int32_t *kept = E.kept_idx + (size_t)unit * E.kept_stride;
    float *sc_out = E.scores_out ? E.scores_out + (size_t)unit * E.out_stride : nullptr;
    if (unit % S.Hkv == 0 && rank == 0 && threadIdx.x == 0) E.dst_len[b] = keep;
    // the CTA's candidates [lo, hi), in runs of `run` slots per warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int run = cdiv(cdiv(cand, Z * kWarps), 32) * 32;
    const int lo = (int)min((long)cand, (long)rank * run * kWarps), hi = (int)min((long)cand, lo + (long)run * kWarps);

    uint32_t prefix = 0;
    int remaining = top;                               // still to be taken among keys that match the prefix
    auto from_memory = [&](int i) { return score_bits(sc[i]); };
    auto from_cache = [&](int i) { return cache[i - lo]; };
    bool cached = false;
    if (top > 0 && top < cand) {
        const bool fits = hi - lo <= E.cache;
        int shift = 32;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int width = pass == 2 ? 10 : 11, bins = 1 << width, part = bins / Z;
            shift -= width;
            for (int i = threadIdx.x; i < bins; i += kThreads) hist[i] = 0;
            __syncthreads();
            auto add = [&](int, uint32_t bits, bool on) {
                const uint32_t key = score_key(bits);
                if (on && (key >> (shift + width)) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1);
            };
            if (pass == 0)
                for_scores(lo, hi, threadIdx.x, kThreads, from_memory, [&](int i, uint32_t bits, bool on) {
                    if (on && fits) cache[i - lo] = bits;
                    if (on) atomicAdd(&hist[score_key(bits) >> 21], 1);
                });
            else if (cached) for_scores(lo, hi, threadIdx.x, kThreads, from_cache, add);
            else for_scores(lo, hi, threadIdx.x, kThreads, from_memory, add);
            cached = fits;
            sync_all();
            if constexpr (Z == 1) {
                // four digits per thread, from the highest down
                const int dgt = bins - 4 - 4 * (int)threadIdx.x;
                int4 cnt = make_int4(0, 0, 0, 0);
                if (dgt >= 0) cnt = *reinterpret_cast<const int4 *>(&hist[dgt]);
                const int all4 = cnt.x + cnt.y + cnt.z + cnt.w;
                int incl = all4;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += up;
                }
                if (lane == 31) warp_sums[warp] = incl;
                __syncthreads();
                for (int w = 0; w < warp; ++w) incl += warp_sums[w];
                int before = incl - all4;
                if (before < remaining && remaining <= incl) {
                    const int by[4] = {cnt.w, cnt.z, cnt.y, cnt.x};
                    int e = 0;
                    while (e < 3 && remaining > before + by[e]) before += by[e++];
                    s_digit = dgt + 3 - e;
                    s_above = before;
                }
                __syncthreads();
            } else {
                // This CTA's digits, from the highest down: rank 0 has the highest
                // part of them.  Two threads per digit, four histograms each.
                const int dgt = bins - 1 - (rank * part + (int)threadIdx.x / 2);
                int cnt = 0;
                if ((int)threadIdx.x < 2 * part) {
#pragma unroll
                    for (int r = 0; r < Z / 2; ++r)
                        cnt += *cluster.map_shared_rank(&hist[dgt], (threadIdx.x & 1) * (Z / 2) + r);
                }
                cnt += __shfl_xor_sync(0xffffffffu, cnt, 1);
                int incl = threadIdx.x & 1 ? 0 : cnt;      // inclusive over the digits from the highest
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += up;
                }
                if (lane == 31) warp_sums[warp] = incl;
                __syncthreads();
                for (int w = 0; w < warp; ++w) incl += warp_sums[w];
                if (threadIdx.x == kThreads - 1)
                    for (int r = 0; r < Z; ++r) *cluster.map_shared_rank(&s_slice[rank], r) = incl;
                cluster.sync();
                int above = 0;                             // keys with digits of lower ranks
                for (int r = 0; r < rank; ++r) above += s_slice[r];
                const int before = above + incl - cnt;
                if (!(threadIdx.x & 1) && (int)threadIdx.x < 2 * part && before < remaining && remaining <= before + cnt)
                    for (int r = 0; r < Z; ++r) {
                        *cluster.map_shared_rank(&s_digit, r) = dgt;
                        *cluster.map_shared_rank(&s_above, r) = before;
                    }
                cluster.sync();                            // the digit has arrived, the histograms have been read
            }
            prefix = (prefix << width) | (uint32_t)s_digit;
            remaining -= s_above;
        }
    }
    // prefix is now the threshold key; of the slots that hold it the first
    // `remaining` are kept.  top = 0 keeps none, top = cand all.
    const bool none = top == 0, all = top == cand;
    const int wlo = min(hi, lo + warp * run), whi = min(hi, wlo + run);
    int2 mine = make_int2(0, 0);                       // kept for sure, tied
    auto tally = [&](int, uint32_t bits, bool on) {
        const uint32_t key = score_key(bits);
        mine.x += __popc(__ballot_sync(0xffffffffu, on && (all || key > prefix)));
        mine.y += __popc(__ballot_sync(0xffffffffu, on && !all && key == prefix));
    };
    if (cached) for_scores(wlo, whi, lane, 32, from_cache, tally);
    else if (!none) for_scores(wlo, whi, lane, 32, from_memory, tally);
    if (lane == 0) s_count[warp] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        int2 sum = make_int2(0, 0);
        for (int w = 0; w < kWarps; ++w) sum.x += s_count[w].x, sum.y += s_count[w].y;
        s_count[kWarps] = sum;
    }
    sync_all();
    int2 before = make_int2(0, 0);
    for (int r = 0; r < rank; ++r) {
        const int2 c = *cluster.map_shared_rank(&s_count[kWarps], r);
        before.x += c.x, before.y += c.y;
    }
    for (int w = 0; w < warp; ++w) before.x += s_count[w].x, before.y += s_count[w].y;
    if (mine.x + mine.y > 0) {
        // a tied slot is kept while fewer than `remaining` ties precede it
        auto write = [&](int i, uint32_t bits, bool on) {
            const uint32_t key = score_key(bits), below = (1u << lane) - 1;
            const bool gt = on && (all || key > prefix), eq = on && !all && key == prefix;
            const unsigned m_gt = __ballot_sync(0xffffffffu, gt), m_eq = __ballot_sync(0xffffffffu, eq);
            const int ties = before.y + __popc(m_eq & below);
            if (gt || (eq && ties < remaining)) {
                const int j = before.x + __popc(m_gt & below) + min(ties, remaining);
                kept[j] = i;
                if (sc_out) sc_out[j] = __uint_as_float(bits);
            }
            before.x += __popc(m_gt);
            before.y += __popc(m_eq);
        };
        if (cached) for_scores(wlo, whi, lane, 32, from_cache, write);
        else for_scores(wlo, whi, lane, 32, from_memory, write);
    }
    for (int i = rank * kThreads + threadIdx.x; i < recent; i += Z * kThreads) {
        kept[top + i] = cand + i;
        if (sc_out) sc_out[top + i] = __uint_as_float(score_bits(sc[cand + i]));
    }
    sync_all();                                        // no CTA leaves while its counts may be read
}

// Rows of kept slots from the source pages to the destination's.  16 bytes per
// lane; kRows rows of K and V are in flight per thread.
constexpr int kMoveThreads = 256, kRows = 4;

__global__ void __launch_bounds__(kMoveThreads)
move_kernel(Pool S, Pool Dp, EvictParams E, int row_bytes, int blocks_per_unit)
{
    pdl_wait();
    pdl_trigger();
    const int unit = blockIdx.x / blocks_per_unit, part = blockIdx.x % blocks_per_unit;
    const int b = unit / S.Hkv, h = unit % S.Hkv;
    const int L = src_tokens(S, E.src_len, b);
    const int recent = (int)min(E.recent, (long)L);
    const int keep = (int)min(E.top, (long)(L - recent)) + recent;
    const int32_t *kept = E.kept_idx + (size_t)unit * E.kept_stride;
    const int lanes = row_bytes / 16, per = kMoveThreads / lanes;
    const int lane = threadIdx.x % lanes, g = threadIdx.x / lanes;
    for (int j0 = part * per * kRows; j0 < keep; j0 += blocks_per_unit * per * kRows) {
        uint4 kx[kRows], vx[kRows];
        size_t dst[kRows];
        bool on[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int j = j0 + i * per + g;
            on[i] = j < keep;
            if (!on[i]) continue;
            const int slot = kept[j];
            const int ps = S.page_of(b, slot >> S.page_log2), pd = Dp.page_of(b, j >> Dp.page_log2);
            on[i] = ps >= 0 && pd >= 0;
            if (!on[i]) continue;
            const size_t src = S.row(ps, h, slot & (S.page() - 1)) * row_bytes + lane * 16;
            dst[i] = Dp.row(pd, h, j & (Dp.page() - 1)) * row_bytes + lane * 16;
            kx[i] = ldg_stream((const uint8_t *)S.k + src);
            vx[i] = ldg_stream((const uint8_t *)S.v + src);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (on[i]) {
                *reinterpret_cast<uint4 *>((uint8_t *)Dp.k + dst[i]) = kx[i];
                *reinterpret_cast<uint4 *>((uint8_t *)Dp.v + dst[i]) = vx[i];
            }
    }
}

template <int Z>
cudaError_t select(const Pool &S, EvictParams E, int units, long cap, cudaStream_t st)
{
    auto kern = select_kernel<Z>;
    const long runs = cdiv(cap, Z * kWarps * 32) * 32l * kWarps;       // a CTA's share of the largest sequence
    E.cache = (int)std::min<long>(kCache, runs);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kCache * 4);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)units * Z), dim3(kThreads), E.cache * 4, st, S, E);
}

}  // namespace

cudaError_t evict(const Pool &S, const Pool &Dp, int row_bytes, const float *scores, int scores_stride,
                  const int32_t *src_len, long top, long recent, int32_t *dst_len, int32_t *kept_idx, int kept_stride,
                  float *scores_out, int out_stride, cudaStream_t st)
{
    EvictParams E;
    E.scores = scores;
    E.src_len = src_len;
    E.dst_len = dst_len;
    E.kept_idx = kept_idx;
    E.scores_out = scores_out;
    E.scores_stride = scores_stride;
    E.kept_stride = kept_stride;
    E.out_stride = out_stride;
    E.top = top;
    E.recent = recent;
    const int units = S.B * S.Hkv;
    const long cap = (long)S.max_blocks << S.page_log2;
    // A table that one CTA's shared memory covers needs no cluster.  With the moves,
    // in single calls, one CTA and a cluster: 256 (sequence, head) units of 1000
    // tokens 46 and 132 us, 128 units of 16000 33 and 70, 8 units of 16000 25 and 23,
    // of 2000 17 and 23.  A wider table takes the cluster whatever its sequences hold.
    cudaError_t e = cap <= kCache ? select<1>(S, E, units, cap, st) : select<kCluster>(S, E, units, cap, st);
    if (e != cudaSuccess) return e;
    // about 12 CTAs per SM, none without a row to move
    const long most = std::min<long>(cap, top + recent);
    const int per = kMoveThreads / (row_bytes / 16) * kRows;
    const int bpu = (int)std::max<long>(1, std::min<long>(cdiv(most, per), cdiv(12l * device_sm_count(), units)));
    return launch_pdl(move_kernel, dim3((unsigned)units * bpu), dim3(kMoveThreads), 0, st, S, Dp, E, row_bytes, bpu);
}

}  // namespace paged
}  // namespace vc
