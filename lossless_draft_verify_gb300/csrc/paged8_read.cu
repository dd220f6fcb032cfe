// paged8_read.cu -- cached tokens back from 8-bit pages: row i of a sequence's
// chunk is its slot ctx + i, as packed rows of bf16 or fp32 values.
//
//   x = code * 2^(byte - 127)
//
// Bound by HBM: every code is read once, every value written once.  A lane takes
// as many codes as make one 16-byte store, so that a warp's loads and stores are
// both whole lines; the tokens of a CTA lie side by side in their page, so a head's
// rows are one run of it.  Four sequences of 32768 tokens, 8 heads of 128, to bf16
// 122.5 us for 807 MB, 97% of the copy rate.
#include <type_traits>

#include "paged.cuh"
#include "paged8.cuh"

namespace vc {
namespace paged {
namespace {

constexpr int kThreads = 256, kTokens = 16;

template <typename E, int D>
__global__ void __launch_bounds__(kThreads)
read8_kernel(Pool P, const int32_t *__restrict__ q_start, const int32_t *__restrict__ ctx_len, int T,
             E *__restrict__ k_out, E *__restrict__ v_out)
{
    constexpr int W = 16 / sizeof(E), CH = D / W;           // codes per lane, lanes per row
    __shared__ long s_row[kTokens];                          // row of head 0 in the pool, or -1
    pdl_wait();
    pdl_trigger();
    const int t0 = blockIdx.x * kTokens, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int t = warp; t < kTokens; t += kThreads / 32) {
        const int tok = t0 + t;
        const int b = tok < T ? find_seq(q_start, P.B, tok) : -1;
        if (lane) continue;
        long row = -1;
        if (b >= 0) {
            const Seq s = load_seq(P, q_start, ctx_len, T, b);
            const int i = tok - s.tok0, slot = s.ctx + i;
            if (i >= 0 && i < s.n) {
                const int page = P.page_of(b, slot >> P.page_log2);
                if (page >= 0) row = (long)P.row(page, 0, slot & (P.page() - 1));
            }
        }
        s_row[t] = row;
    }
    if (blockIdx.x == 0)                                     // lengths that do not fit are reported for all sequences
        for (int b = threadIdx.x; b < P.B; b += kThreads) load_seq(P, q_start, ctx_len, T, b);
    __syncthreads();
    const int items = 2 * P.Hkv * kTokens * CH;              // (k or v, head, token, lane of the row)
    constexpr int U = 4;
    for (int i0 = threadIdx.x; i0 < items; i0 += U * kThreads) {
        uint32_t w[U][W / 4];
        uint32_t byte[U];
        long to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kThreads;
            to[u] = -1;
            if (i >= items) continue;
            const int c = i % CH, t = i / CH % kTokens, kh = i / (CH * kTokens);
            const int h = kh < P.Hkv ? kh : kh - P.Hkv;
            if (s_row[t] < 0) continue;
            const size_t row = (size_t)s_row[t] + ((size_t)h << P.page_log2);
            const uint8_t *src = (const uint8_t *)(kh < P.Hkv ? P.k : P.v) + row * D + c * W;
            byte[u] = (kh < P.Hkv ? P.k_scale : P.v_scale)[row];
            if constexpr (W == 8) {
                const uint2 x = *reinterpret_cast<const uint2 *>(src);
                w[u][0] = x.x, w[u][W / 4 - 1] = x.y;
            } else {
                w[u][0] = *reinterpret_cast<const uint32_t *>(src);
            }
            to[u] = ((long)(t0 + t) * P.Hkv + h) * D + c * W;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (to[u] < 0) continue;
            const int kh = (i0 + u * kThreads) / (CH * kTokens);
            E *dst = (kh < P.Hkv ? k_out : v_out) + to[u];
            const float scale = scale_of(byte[u]);
            float x[W];
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
                const float2 f = decode2(w[u][j / 2] >> (j % 2 * 16));
                x[2 * j] = f.x * scale;
                x[2 * j + 1] = f.y * scale;
            }
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (W == 8) {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                    o[j] = *reinterpret_cast<const uint32_t *>(&p);
                } else {
                    o[j] = __float_as_uint(x[j]);
                }
            }
            *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// The pages of a batch as bf16 pages of their own, in the order of its table, and
// the table that names them (a bad page number stays one).  A head's rows of a page are
// one run of codes, and of values; blockIdx.y: the head.  Every thread looks its
// pages up itself: no barrier, so that one page's look-ups pass under another's copy.
// 32048 tokens, 8 heads of 128 (197 MB): some 30 us of the call that they are for.
__global__ void __launch_bounds__(kThreads)
expand8_kernel(Pool P, const int32_t *__restrict__ q_start, const int32_t *__restrict__ ctx_len, int T, int d_log2,
               uint4 *__restrict__ k_out, uint4 *__restrict__ v_out, int32_t *__restrict__ table_out)
{
    pdl_wait();
    pdl_trigger();
    const int blocks = P.B * P.max_blocks, chunks = (P.page() << d_log2) / 8, h = blockIdx.y;      // of 8 codes
    for (int i = blockIdx.x; i < blocks; i += gridDim.x) {
        const int b = i / P.max_blocks, blk = i % P.max_blocks;
        const int len = load_seq(P, q_start, ctx_len, T, b).len();
        const int page = ((long)blk << P.page_log2) < len ? P.page_of(b, blk) : -1;
        if (h == 0 && threadIdx.x == 0) table_out[i] = page >= 0 ? i : -1;
        if (page < 0) continue;
        const size_t row0 = P.row(page, h, 0), to = ((size_t)i * P.Hkv + h) * chunks;
#pragma unroll 4
        for (int c = threadIdx.x; c < chunks; c += kThreads) {
            const size_t row = row0 + (c * 8 >> d_log2), at = (row0 << d_log2) + (size_t)c * 8;
            auto expand = [&](const void *codes, const uint8_t *scales) {
                const uint2 w = *reinterpret_cast<const uint2 *>((const uint8_t *)codes + at);
                const float s = scale_of(scales[row]);
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = decode2((j < 2 ? w.x : w.y) >> (j % 2 * 16));
                    const __nv_bfloat162 p = __floats2bfloat162_rn(f.x * s, f.y * s);
                    o[j] = *reinterpret_cast<const uint32_t *>(&p);
                }
                return make_uint4(o[0], o[1], o[2], o[3]);
            };
            k_out[to + c] = expand(P.k, P.k_scale);
            v_out[to + c] = expand(P.v, P.v_scale);
        }
    }
}

template <typename E>
cudaError_t launch(const Pool &P, int d, const int32_t *q_start, const int32_t *ctx_len, int T, void *k, void *v,
                   cudaStream_t st)
{
    const dim3 grid(cdiv(T, kTokens));
    return d == 128 ? launch_pdl(read8_kernel<E, 128>, grid, dim3(kThreads), 0, st, P, q_start, ctx_len, T, (E *)k, (E *)v)
                    : launch_pdl(read8_kernel<E, 64>, grid, dim3(kThreads), 0, st, P, q_start, ctx_len, T, (E *)k, (E *)v);
}

}  // namespace

cudaError_t expand8(const Pool &P, int d, const int32_t *q_start, const int32_t *ctx_len, int T, void *k_out,
                    void *v_out, int32_t *table_out, cudaStream_t st)
{
    // eight CTAs per SM over the heads (at most 2^30 / 64 / 512 heads of a workspace's pages)
    const int each = std::max(1, std::min(P.B * P.max_blocks, 8 * device_sm_count() / P.Hkv));
    return launch_pdl(expand8_kernel, dim3(each, P.Hkv), dim3(kThreads), 0, st, P, q_start, ctx_len, T,
                      d == 128 ? 7 : 6, (uint4 *)k_out, (uint4 *)v_out, table_out);
}

cudaError_t read8(const Pool &P, vc_dtype dt, int d, const int32_t *q_start, const int32_t *ctx_len, int T, void *k_out,
                  void *v_out, cudaStream_t st)
{
    return dt == VC_BF16 ? launch<__nv_bfloat16>(P, d, q_start, ctx_len, T, k_out, v_out, st)
                         : launch<float>(P, d, q_start, ctx_len, T, k_out, v_out, st);
}

}  // namespace paged
}  // namespace vc
