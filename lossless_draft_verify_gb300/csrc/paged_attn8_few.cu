// paged_attn8_few.cu -- attention of few rows (paged_attn_few.cuh) over 8-bit pages,
// bf16 rows.
#include "paged_attn_few.cuh"

namespace vc {
namespace paged {

cudaError_t attn8_few_f32(const Pool &P, const WorkDim &W, int d, int rows, const void *q, int Hq, float sl2, void *out,
                          const Halves &H, bool first, const Parts &parts, int32_t *status, cudaStream_t st);

int few_pieces(int rows)
{
    return device_sm_count() * (rows == 8 ? Geom<128, 1, true, float>::WARPS : Geom<128, 2, true, float>::WARPS);
}

cudaError_t attn8_few(const Pool &P, const WorkDim &W, vc_dtype dt, int d, int rows, const void *q, int Hq, float sl2,
                      void *out, const Parts &parts, int32_t *status, cudaStream_t st)
{
    if (dt == VC_F32) return attn8_few_f32(P, W, d, rows, q, Hq, sl2, out, Halves{}, false, parts, status, st);
    return few_form<Seq, true, __nv_bfloat16>(P, W, d, rows, q, Hq, sl2, out, Halves{}, false, parts, status, st);
}

cudaError_t attn8_few_planned(const Pool &P, const WorkDim &W, vc_dtype dt, int d, int rows, const void *q, int Hq,
                              float sl2, const Halves &H, bool first, const Parts &parts, int32_t *status,
                              cudaStream_t st)
{
    if (dt == VC_F32) return attn8_few_f32(P, W, d, rows, q, Hq, sl2, nullptr, H, first, parts, status, st);
    return few_form<VSeq, true, __nv_bfloat16>(P, W, d, rows, q, Hq, sl2, nullptr, H, first, parts, status, st);
}

}  // namespace paged
}  // namespace vc
