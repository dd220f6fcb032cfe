// paged_append.cu -- the new tokens of a ragged batch on their way into a
// paged cache: per head RMS norm of queries and keys, position rotation, the
// queries to q_out, keys and values into the pages.
//
//   x' = x / sqrt(mean(x^2) + eps) * gain                  (optional)
//   (x'_j, x'_{j + r/2}) turned by pos * w_j, j < r/2       (r = rotary_dim)
//
// Every value is read once and written once, about ten operations each: its
// floor is HBM's, what bounds it is latency (see launch).  A head's row is held by D/16 lanes, two 8-channel chunks
// per lane chosen so that both halves of a rotated pair meet in one lane (no
// exchange but the D/16-lane sum of squares).  Angles: w_j / 2 pi is kept as a
// 64-bit fraction of a turn, so pos * w_j modulo one turn is an integer
// product that is exact at any position; sine and cosine are computed once per
// (token, pair) and shared by the token's heads.
#include "paged.cuh"

namespace vc {
namespace paged {
namespace {

constexpr int kThreads = 256;

template <typename T> struct Row8;      // 8 consecutive channels: as read, and in pairs
template <> struct Row8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = ldg_stream(p);
        b = ldg_stream(p + 4);
    }
    __device__ __forceinline__ void get(float2 (&x)[4]) const
    {
        x[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
        x[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
        x[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
        x[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
    }
    static __device__ __forceinline__ void store(float *p, const float2 (&x)[4])
    {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
    }
};
template <> struct Row8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = ldg_stream(p); }
    __device__ __forceinline__ void get(float2 (&x)[4]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float2 (&x)[4])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// 8 floats of shared memory, in pairs
__device__ __forceinline__ void lds8(const float *p, float2 (&x)[4])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = make_float2(a.x, a.y);
    x[1] = make_float2(a.z, a.w);
    x[2] = make_float2(b.x, b.y);
    x[3] = make_float2(b.z, b.w);
}

struct AppendParams {
    Pool P;
    const int32_t *positions, *q_start, *ctx_len;
    const void *qkv, *q_gain, *k_gain;
    void *q_out;
    int T, Hq;
    float eps;
};

// TPB tokens per CTA; blockIdx.y takes its share of the heads.  A lane group
// keeps its next head in flight, as read: the first one while the tokens'
// sequences, pages and angles are looked up, each other one under the arithmetic
// of the one before (in a graph 19.5 us at 4670 tokens, 22.9 when it is read after
// it, 20.2 and 21.5 with two and three in flight).
template <typename E, int D, int TPB>
__global__ void __launch_bounds__(kThreads, 4)
append_kernel(AppendParams A, const __grid_constant__ vc_rope rope)
{
    constexpr int LANES = D / 16, GROUPS = kThreads / LANES;
    // 8 values per 12 words: the lanes' 16-byte reads fall on different banks
    __shared__ __align__(16) float s_cos[TPB][8 * 12], s_sin[TPB][8 * 12], s_gain[2][D / 8 * 12];
    __shared__ int s_pos[TPB], s_page[TPB], s_slot[TPB];      // page -1: no cache row, -2: row of no sequence
    pdl_wait();
    pdl_trigger();
    const int t0 = blockIdx.x * TPB;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = A.Hq + 2 * A.P.Hkv, items = min(TPB, A.T - t0) * heads;
    const int half = rope.rotary_dim / 2;
    const int g = threadIdx.x / LANES, l = threadIdx.x % LANES;
    const int rl = half / 8;                               // lanes that hold rotated pairs
    const bool rot = l < rl;
    const int c0 = 8 * (rot ? l : 2 * rl + 2 * (l - rl)), c1 = rot ? c0 + half : c0 + 8;
    const E *qkv = (const E *)A.qkv + (size_t)t0 * heads * D;
    const int stride = gridDim.y * GROUPS;
    Row8<E> r0 = {}, r1 = {};
    int i0 = blockIdx.y * GROUPS;
    auto load = [&](int i) {
        if (i < items) {
            r0.load(qkv + (size_t)i * D + c0);
            r1.load(qkv + (size_t)i * D + c1);
        }
    };
    load(i0 + g);
    if (A.q_gain)
        for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
            const int c = i % D;
            s_gain[i / D][c / 8 * 12 + c % 8] = Elem<E>::to_f(((const E *)(i < D ? A.q_gain : A.k_gain))[c]);
        }
    // One warp per token finds its sequence, the last one that starts at or
    // before it (32 probes a step).  Lengths that do not fit are reported by
    // the first CTA for all sequences, and give a token no row.
    for (int t = warp; t < TPB; t += kThreads / 32) {
        const int tok = t0 + t;
        if (lane == 0) s_page[t] = -2;
        __syncwarp();
        if (tok >= A.T) continue;
        int lo = 0, hi = A.P.B;
        for (;;) {
            const int step = (hi - lo + 31) / 32, b = lo + lane * step;
            const unsigned le = __ballot_sync(0xffffffffu, b < hi && A.q_start[b] <= tok);
            if (le == 0) {
                hi = lo;
                break;
            }
            lo += (31 - __clz(le)) * step;
            hi = min(hi, lo + step);
            if (step == 1) break;
        }
        if (lane == 0 && lo < hi) {
            const Seq s = load_seq(A.P, A.q_start, A.ctx_len, A.T, lo);
            const int i = tok - s.tok0;
            if (i >= 0 && i < s.n) {
                const int slot = s.ctx + i;
                s_page[t] = A.P.page_of(lo, slot >> A.P.page_log2);
                s_slot[t] = slot & (A.P.page() - 1);
                s_pos[t] = A.positions ? A.positions[tok] : slot;
            }
        }
    }
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int b = threadIdx.x; b < A.P.B; b += kThreads) load_seq(A.P, A.q_start, A.ctx_len, A.T, b);
    __syncthreads();
    for (int i = threadIdx.x; i < TPB * half; i += kThreads) {
        const int t = i / half, j = i % half;
        if (s_page[t] == -2) continue;
        // the angle in turns, as a signed 64-bit fraction
        const int64_t f = (int64_t)((uint64_t)(int64_t)s_pos[t] * rope.turn[j]);
        float sn, cs;
        sincospif((float)f * 0x1p-63f, &sn, &cs);
        s_cos[t][j / 8 * 12 + j % 8] = cs;
        s_sin[t][j / 8 * 12 + j % 8] = sn;
    }
    __syncthreads();
    const int p0 = c0 / 8 * 12, p1 = c1 / 8 * 12;
    int t = (i0 + g) / heads, hh = (i0 + g) % heads;       // the lane group's token and head
    for (; i0 < items; i0 += stride) {
        float2 x0[4], x1[4];
        r0.get(x0);
        r1.get(x1);
        load(i0 + stride + g);
        const bool on = t < TPB && i0 + g < items && s_page[t] != -2;
        const bool is_v = hh >= A.Hq + A.P.Hkv;
        if (A.q_gain) {
            float2 ss = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) ss = fma2(x0[e], x0[e], fma2(x1[e], x1[e], ss));
            float sum = ss.x + ss.y;                   // unread rows sum garbage, which nobody uses
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (on && !is_v) {
                const float inv = rsqrtf(sum * (1.f / D) + A.eps);
                const float *gain = s_gain[hh < A.Hq ? 0 : 1];
                const float2 inv2 = make_float2(inv, inv);
                float2 g0[4], g1[4];
                lds8(gain + p0, g0);
                lds8(gain + p1, g1);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x0[e] = mul2(mul2(x0[e], inv2), g0[e]);
                    x1[e] = mul2(mul2(x1[e], inv2), g1[e]);
                }
            }
        }
        if (on && rot && !is_v) {
            float2 c[4], s[4];
            lds8(s_cos[t] + p0, c);
            lds8(s_sin[t] + p0, s);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 a = x0[e], b = x1[e];
                x0[e] = sub2(mul2(a, c[e]), mul2(b, s[e]));
                x1[e] = fma2(a, s[e], mul2(b, c[e]));
            }
        }
        if (on && (hh < A.Hq || s_page[t] >= 0)) {     // a page outside the pool: nothing is written
            E *dst;
            if (hh < A.Hq) {
                dst = (E *)A.q_out + ((size_t)(t0 + t) * A.Hq + hh) * D;
            } else {
                const int h = is_v ? hh - A.Hq - A.P.Hkv : hh - A.Hq;
                dst = (E *)(is_v ? A.P.v : A.P.k) + A.P.row(s_page[t], h, s_slot[t]) * D;
            }
            Row8<E>::store(dst + c0, x0);
            Row8<E>::store(dst + c1, x1);
        }
        for (hh += stride; hh >= heads; hh -= heads) ++t;
    }
}

template <typename E, int D>
cudaError_t launch(const AppendParams &A, const vc_rope &rope, cudaStream_t st)
{
    const int heads = A.Hq + 2 * A.P.Hkv, groups = kThreads / (D / 16);
    // Few tokens: one per CTA, its heads over several CTAs, one head per lane
    // group; many: four per CTA, which share the look-ups and the sines.  32/8
    // heads of 128 in bf16, in a graph, one and four per CTA: 16 tokens 3.9 and 6.4
    // us, 600 7.0 and 6.7, 1200 11.3 and 7.8, 2400 20.5 and 11.2, 4670 37.3 and 19.5.
    // The last moves 115 MB, which about fills L2 from one replay to the next; with
    // inputs that are not there the call takes 24.1 us, 70% of the measured copy
    // rate: sequence, page and angles of four tokens are looked up before a CTA's
    // first store, in two waves of CTAs.
    if (A.T <= 4 * device_sm_count())
        return launch_pdl(append_kernel<E, D, 1>, dim3(A.T, cdiv(heads, groups)), dim3(kThreads), 0, st, A, rope);
    return launch_pdl(append_kernel<E, D, 4>, dim3(cdiv(A.T, 4)), dim3(kThreads), 0, st, A, rope);
}

}  // namespace

cudaError_t append(const Pool &P, vc_dtype dt, int d, const void *qkv, const void *q_gain, const void *k_gain,
                   float eps, const vc_rope &rope, const int32_t *positions, const int32_t *q_start,
                   const int32_t *ctx_len, int T, int Hq, void *q_out, cudaStream_t st)
{
    AppendParams A;
    A.P = P;
    A.positions = positions;
    A.q_start = q_start;
    A.ctx_len = ctx_len;
    A.qkv = qkv;
    A.q_gain = q_gain;
    A.k_gain = k_gain;
    A.q_out = q_out;
    A.T = T;
    A.Hq = Hq;
    A.eps = eps;
    if (dt == VC_BF16) return d == 128 ? launch<__nv_bfloat16, 128>(A, rope, st) : launch<__nv_bfloat16, 64>(A, rope, st);
    return d == 128 ? launch<float, 128>(A, rope, st) : launch<float, 64>(A, rope, st);
}

}  // namespace paged
}  // namespace vc
