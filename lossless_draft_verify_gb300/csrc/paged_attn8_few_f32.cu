// paged_attn8_few_f32.cu -- attention over 8-bit pages (paged_attn_few.cuh), fp32 rows.
#include "paged_attn_few.cuh"

namespace vc {
namespace paged {

cudaError_t attn8_few_f32(const Pool &P, const WorkDim &W, int d, int rows, const void *q, int Hq, float sl2, void *out,
                          const Halves &H, bool first, const Parts &parts, int32_t *status, cudaStream_t st)
{
    return W.plan ? few_form<VSeq, true, float>(P, W, d, rows, q, Hq, sl2, out, H, first, parts, status, st)
                  : few_form<Seq, true, float>(P, W, d, rows, q, Hq, sl2, out, H, first, parts, status, st);
}

}  // namespace paged
}  // namespace vc
