// paged_attn_few.cu -- attention of few rows (paged_attn_few.cuh) over bf16 pages, of
// planned batches.
#include "paged_attn_few.cuh"

namespace vc {
namespace paged {

cudaError_t attn_few_planned(const Pool &P, const WorkDim &W, int d, int rows, const void *q, int Hq, float sl2,
                             const Halves &H, bool first, const Parts &parts, int32_t *status, cudaStream_t st)
{
    return few_form<VSeq, false, __nv_bfloat16>(P, W, d, rows, q, Hq, sl2, nullptr, H, first, parts, status, st);
}

}  // namespace paged
}  // namespace vc
