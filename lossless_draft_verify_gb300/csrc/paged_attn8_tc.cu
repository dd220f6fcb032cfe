// paged_attn8_tc.cu -- the tensor-core attention over pages of 8-bit rows
// (paged_attn_tc.cuh): plain and planned batches.
#include "paged_attn_tc.cuh"

namespace vc {
namespace paged {

cudaError_t attn8_tc(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, void *out,
                     const Parts &parts, int32_t *status, cudaStream_t st)
{
    return d == 128 ? launch<128, false, Seq, true>(P, W, q, Hq, sl2, out, nullptr, nullptr, 0, parts, status, st)
                    : launch<64, false, Seq, true>(P, W, q, Hq, sl2, out, nullptr, nullptr, 0, parts, status, st);
}

cudaError_t attn8_tc_planned(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, const Halves &H,
                             const Parts &parts, int32_t *status, cudaStream_t st)
{
    return d == 128 ? launch<128, false, VSeq, true>(P, W, q, Hq, sl2, H.o, H.lse, nullptr, 0, parts, status, st, H.place)
                    : launch<64, false, VSeq, true>(P, W, q, Hq, sl2, H.o, H.lse, nullptr, 0, parts, status, st, H.place);
}

}  // namespace paged
}  // namespace vc
