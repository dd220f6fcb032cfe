// paged_attn8_few.cu -- attention of few rows (paged_attn_few.cuh) over 8-bit pages.
#include "paged_attn_few.cuh"

namespace vc {
namespace paged {

int few_pieces(int rows) { return device_sm_count() * (rows == 8 ? Geom<128, 1, true>::WARPS : Geom<128, 2, true>::WARPS); }

cudaError_t attn8_few(const Pool &P, const WorkDim &W, int d, int rows, const void *q, int Hq, float sl2, void *out,
                      const Parts &parts, int32_t *status, cudaStream_t st)
{
    return few_form<Seq, true>(P, W, d, rows, q, Hq, sl2, out, Halves{}, parts, status, st);
}

cudaError_t attn8_few_planned(const Pool &P, const WorkDim &W, int d, int rows, const void *q, int Hq, float sl2,
                              const Halves &H, const Parts &parts, int32_t *status, cudaStream_t st)
{
    return few_form<VSeq, true>(P, W, d, rows, q, Hq, sl2, nullptr, H, parts, status, st);
}

}  // namespace paged
}  // namespace vc
