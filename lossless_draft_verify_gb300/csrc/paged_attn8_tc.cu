// paged_attn8_tc.cu -- the tensor-core attention over pages of 8-bit rows
// (paged_attn_tc.cuh): plain and planned batches.
#include "paged_attn_tc.cuh"

namespace vc {
namespace paged {

cudaError_t attn8_tc(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, void *out, float *lse,
                     const Parts &parts, int32_t *status, cudaStream_t st)
{
    if (W.plan)
        return d == 128 ? launch<128, false, VSeq, true>(P, W, q, Hq, sl2, out, lse, nullptr, 0, parts, status, st)
                        : launch<64, false, VSeq, true>(P, W, q, Hq, sl2, out, lse, nullptr, 0, parts, status, st);
    return d == 128 ? launch<128, false, Seq, true>(P, W, q, Hq, sl2, out, lse, nullptr, 0, parts, status, st)
                    : launch<64, false, Seq, true>(P, W, q, Hq, sl2, out, lse, nullptr, 0, parts, status, st);
}

}  // namespace paged
}  // namespace vc
