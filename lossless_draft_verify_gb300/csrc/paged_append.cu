// paged_append.cu -- the new tokens of a ragged batch on their way into a
// paged cache: per head RMS norm of queries and keys, position rotation, the
// queries to q_out, keys and values into the pages.
//
//   x' = x / sqrt(mean(x^2) + eps) * gain                  (optional)
//   (x'_j, x'_{j + r/2}) turned by pos * w_j, j < r/2       (r = rotary_dim)
//
// Bound by HBM: every value is read once and written once, about ten
// operations each.  A head's row is held by D/16 lanes, two 8-channel chunks
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

template <typename T> struct Row8;      // 8 consecutive channels
template <> struct Row8<float> {
    static __device__ __forceinline__ void load(const float *p, float (&x)[8])
    {
        const uint4 a = ldg_stream(p), b = ldg_stream(p + 4);
        x[0] = __uint_as_float(a.x), x[1] = __uint_as_float(a.y), x[2] = __uint_as_float(a.z);
        x[3] = __uint_as_float(a.w), x[4] = __uint_as_float(b.x), x[5] = __uint_as_float(b.y);
        x[6] = __uint_as_float(b.z), x[7] = __uint_as_float(b.w);
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[8])
    {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <> struct Row8<__nv_bfloat16> {
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&x)[8])
    {
        const uint4 a = ldg_stream(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&x)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

struct AppendParams {
    Pool P;
    const int32_t *positions, *q_start, *ctx_len;
    const void *qkv, *q_gain, *k_gain;
    void *q_out;
    int T, Hq;
    float eps;
};

// TPB tokens per CTA; blockIdx.y takes its share of the heads.
template <typename E, int D, int TPB>
__global__ void __launch_bounds__(kThreads)
append_kernel(AppendParams A, const __grid_constant__ vc_rope rope)
{
    constexpr int LANES = D / 16, GROUPS = kThreads / LANES;
    __shared__ float2 s_cs[TPB][64];
    __shared__ int s_pos[TPB], s_page[TPB], s_slot[TPB];      // page -1: no cache row, -2: row of no sequence
    pdl_wait();
    pdl_trigger();
    const int t0 = blockIdx.x * TPB;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    const int half = rope.rotary_dim / 2;
    for (int i = threadIdx.x; i < TPB * half; i += kThreads) {
        const int t = i / half, j = i % half;
        if (s_page[t] == -2) continue;
        // the angle in turns, as a signed 64-bit fraction
        const int64_t f = (int64_t)((uint64_t)(int64_t)s_pos[t] * rope.turn[j]);
        float sn, cs;
        sincospif((float)f * 0x1p-63f, &sn, &cs);
        s_cs[t][j] = make_float2(cs, sn);
    }
    __syncthreads();
    const int heads = A.Hq + 2 * A.P.Hkv;
    const int g = threadIdx.x / LANES, l = threadIdx.x % LANES;
    const int rl = half / 8;                               // lanes that hold rotated pairs
    const bool rot = l < rl;
    const int c0 = 8 * (rot ? l : 2 * rl + 2 * (l - rl)), c1 = rot ? c0 + half : c0 + 8;
    for (int i0 = blockIdx.y * GROUPS; i0 < TPB * heads; i0 += gridDim.y * GROUPS) {
        const int i = i0 + g;
        const bool on = i < TPB * heads && s_page[i / heads] != -2;
        const int t = on ? i / heads : 0, hh = on ? i % heads : 0;
        const size_t tok = (size_t)t0 + t;
        float x0[8], x1[8];
        if (on) {
            const E *src = (const E *)A.qkv + (tok * heads + hh) * D;
            Row8<E>::load(src + c0, x0);
            Row8<E>::load(src + c1, x1);
        }
        const bool is_v = hh >= A.Hq + A.P.Hkv;
        if (A.q_gain) {
            float ss = 0.f;
            if (on) {
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
            }
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (on && !is_v) {
                const float inv = 1.f / sqrtf(ss * (1.f / D) + A.eps);
                const E *gain = (const E *)(hh < A.Hq ? A.q_gain : A.k_gain);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x0[e] *= inv * Elem<E>::to_f(gain[c0 + e]);
                    x1[e] *= inv * Elem<E>::to_f(gain[c1 + e]);
                }
            }
        }
        if (!on) continue;
        if (rot && !is_v) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 cs = s_cs[t][c0 + e];
                const float a = x0[e], b = x1[e];
                x0[e] = a * cs.x - b * cs.y;
                x1[e] = b * cs.x + a * cs.y;
            }
        }
        E *dst;
        if (hh < A.Hq) {
            dst = (E *)A.q_out + (tok * A.Hq + hh) * D;
        } else {
            if (s_page[t] < 0) continue;                   // a page outside the pool: nothing is written
            const int h = is_v ? hh - A.Hq - A.P.Hkv : hh - A.Hq;
            dst = (E *)(is_v ? A.P.v : A.P.k) + A.P.row(s_page[t], h, s_slot[t]) * D;
        }
        Row8<E>::store(dst + c0, x0);
        Row8<E>::store(dst + c1, x1);
    }
}

template <typename E, int D>
cudaError_t launch(const AppendParams &A, const vc_rope &rope, cudaStream_t st)
{
    const int heads = A.Hq + 2 * A.P.Hkv, groups = kThreads / (D / 16);
    // few tokens: one per CTA, its heads over several CTAs, one head per lane
    // group; many: four per CTA, which share the sines
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
