// paged_attn_tc.cu -- the tensor-core attention over pages of bf16 rows
// (paged_attn_tc.cuh): plain batches, those whose products are stored, and
// planned ones.
#include "paged_attn_tc.cuh"

namespace vc {
namespace paged {

int tc_ctas() { return device_sm_count(); }

cudaError_t attn_tc(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, void *out, float *lse,
                    float *s_out, long s_stride, const Parts &parts, int32_t *status, cudaStream_t st)
{
    if (s_out)
        return d == 128 ? launch<128, true, Seq, false>(P, W, q, Hq, sl2, out, lse, s_out, s_stride, parts, status, st)
                        : launch<64, true, Seq, false>(P, W, q, Hq, sl2, out, lse, s_out, s_stride, parts, status, st);
    return d == 128 ? launch<128, false, Seq, false>(P, W, q, Hq, sl2, out, lse, nullptr, 0, parts, status, st)
                    : launch<64, false, Seq, false>(P, W, q, Hq, sl2, out, lse, nullptr, 0, parts, status, st);
}

cudaError_t attn_tc_planned(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, const Halves &H,
                            const Parts &parts, int32_t *status, cudaStream_t st)
{
    return d == 128 ? launch<128, false, VSeq, false>(P, W, q, Hq, sl2, H.o, H.lse, nullptr, 0, parts, status, st, H.place)
                    : launch<64, false, VSeq, false>(P, W, q, Hq, sl2, H.o, H.lse, nullptr, 0, parts, status, st, H.place);
}

}  // namespace paged
}  // namespace vc
