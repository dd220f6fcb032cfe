// paged.cuh -- what the paged-cache kernels share: the device view of a page
// pool, the checks of lengths and page numbers that live on the device, and
// the division of ragged attention work over a fixed number of CTAs.
#pragma once

#include <algorithm>

#include "vc_common.cuh"
#include "vc_internal.h"

namespace vc {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
// Below every score in the log2 domain (products within 1e30, times a scale of
// at most 1e8 and log2 e: 1.44e38), and its distance to the largest is finite.
// A row that has seen no key has it as its maximum.
constexpr float kLowest = -1.5e38f;
// the same for products not yet scaled
constexpr float kLowestProduct = -1.0e30f;

__host__ __device__ inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// The checks and the division of work below also compile for the host, where
// tests run them over many batches.
#ifdef __CUDA_ARCH__
__device__ __forceinline__ void set_flag(int32_t *status, int bit) { atomicOr(status, bit); }
#else
inline void set_flag(int32_t *status, int bit) { *status |= bit; }
#endif
__host__ __device__ inline long lmin(long a, long b) { return a < b ? a : b; }
__host__ __device__ inline long lmax(long a, long b) { return a > b ? a : b; }

// The pool as the kernels see it.  Pages hold 2^page_log2 slots.
struct Pool {
    void *k, *v;               // [n_pages][Hkv][page][d]
    const int32_t *table;      // [B][max_blocks]
    int32_t *status;
    int32_t B, Hkv, page_log2, n_pages, max_blocks;

    __host__ __device__ __forceinline__ int page() const { return 1 << page_log2; }
    __host__ __device__ __forceinline__ long capacity() const { return (long)max_blocks << page_log2; }
    // page number of block `blk` of sequence b; -1 (and the status bit) when
    // the table's entry lies outside the pool
    __host__ __device__ __forceinline__ int page_of(int b, int blk) const
    {
        const int p = table[(size_t)b * max_blocks + blk];
        if ((unsigned)p < (unsigned)n_pages) return p;
        set_flag(status, VC_PAGED_BAD_PAGE);
        return -1;
    }
    // first row (of d elements) of head h in page p: 64 bits, a pool may hold
    // more than 2^31 elements
    __host__ __device__ __forceinline__ size_t row(int p, int h, int slot_in_page) const
    {
        return (((size_t)p * Hkv + h) << page_log2) + slot_in_page;
    }
};

// One sequence of a ragged batch: its rows [tok0, tok0 + n) of the packed
// tokens and its cached tokens.  Lengths that do not fit (rows outside the
// packed range, a negative context, more slots than the table has) make the
// sequence empty and set the status bit.
struct Seq {
    int tok0, n, ctx;
};

struct RawSeq {
    int start, end, ctx;
};

__host__ __device__ __forceinline__ RawSeq raw_seq(const int32_t *__restrict__ q_start,
                                                   const int32_t *__restrict__ ctx_len, int b)
{
    return RawSeq{q_start[b], q_start[b + 1], ctx_len[b]};
}

__host__ __device__ __forceinline__ Seq check_seq(const Pool &P, const RawSeq &r, int T)
{
    const bool ok = r.start >= 0 && r.end >= r.start && r.end <= T && r.ctx >= 0 &&
                    (long)r.ctx + (r.end - r.start) <= P.capacity();
    if (!ok) {
        set_flag(P.status, VC_PAGED_BAD_LENGTH);
        return Seq{0, 0, 0};
    }
    return Seq{r.start, r.end - r.start, r.ctx};
}

__host__ __device__ __forceinline__ Seq load_seq(const Pool &P, const int32_t *__restrict__ q_start,
                                                 const int32_t *__restrict__ ctx_len, int T, int b)
{
    return check_seq(P, raw_seq(q_start, ctx_len, b), T);
}

// ----- division of the attention work ----------------------------------------
// A unit is (sequence b, kv head h, row tile mt): BM consecutive rows of the
// n * G (query, head of the group) rows that share a kv head, row = i * G + g.
// It takes the key tiles (BN keys) its last query can see.  The units of a
// batch, laid end to end by cost (a tile's, twice as much where more than half
// of a 256-row tile's rows are there, and kUnitCost for loading Q and writing
// the output), are cut into equal pieces, one per CTA: a piece may begin and
// end inside a unit, whose partial results are then merged.  One long sequence
// and many short ones thus fill the GPU alike, and the division depends on the
// lengths only.
struct WorkDim {
    const int32_t *q_start, *ctx_len;
    int T, G;
};

// A unit of at most kWhole is never cut: merging its parts would take longer
// than it does.  It belongs to the CTA in whose piece its middle lies.  A piece
// costs at least kMinPiece.
// Single calls, inputs not in L2, at a kUnitCost of 2, 9, 16 and 24 for row tiles
// of 256 (heads of 128): nine sequences (chunks of 1 to 700 over up to 20000
// tokens, 28/4 heads, pages of 16) 682, 523, 494 and 493 us; a decode step of 16
// x 32768 tokens 336, 334, 336 and 343, of 256 x 300 tokens 142, 142, 150 and 148;
// 16 x 33 over 32768 400, 399, 400 and 410.  The CUDA-core kernels' tiles take
// longer and their units less: at 1, 2, 4 and 8 a token of 8 sequences over 4000
// takes 163, 162, 169 and 175 us, four chunks of 300 over 2000 578, 582, 585 and
// 590, four chunks up to 17 over 2000 at most 27, 27, 27 and 25.
template <int BM>
struct Cost {
    static constexpr int kUnitCost = BM == 256 ? 16 : 1;
    static constexpr int kMinPiece = BM == 256 ? 10 : 2;
    static constexpr int kWhole = BM == 256 ? 20 : 3;
};

// What one CTA has to do: from unit (b, h, mt), cost offset `off` within it,
// `len` cost units on.  Written to shared memory by one warp, read by all.
struct Piece {
    int b, h, mt;
    long off, len;     // off: cost already covered by earlier CTAs
    long per;          // the length of a full piece
};

__host__ __device__ inline long piece_len(long total, int n_cta, int min_len)
{
    return lmax((total + n_cta - 1) / n_cta, min_len);
}

template <int BM, int BN>
struct Units : Cost<BM> {
    using Cost<BM>::kUnitCost;
    // 32-bit arithmetic: a sequence has at most 2^30 rows
    static __host__ __device__ __forceinline__ int tiles(const Seq &s, int G, int mt)
    {
        const unsigned rows = (unsigned)s.n * G, end = ((unsigned)mt + 1) * BM;
        const unsigned last = (rows < end ? rows : end) - 1;              // last row of the tile
        return (int)((s.ctx + last / (unsigned)G + 1 + BN - 1) / BN);
    }
    static __host__ __device__ __forceinline__ int weight(const Seq &s, int G, int mt)
    {
        return BM == 256 && s.n * G - mt * BM > BM / 2 ? 2 : 1;
    }
    static __host__ __device__ __forceinline__ int cost(const Seq &s, int G, int mt)
    {
        return tiles(s, G, mt) * weight(s, G, mt) + kUnitCost;
    }
    static __host__ __device__ __forceinline__ int mtiles(const Seq &s, int G) { return (s.n * G + BM - 1) / BM; }
    static __host__ __device__ __forceinline__ long head_cost(const Seq &s, int G)
    {
        long c = 0;
        const int m = mtiles(s, G);
        for (int i = 0; i < m; ++i) c += cost(s, G, i);
        return c;
    }
    // head, row tile and offset of cost unit x of a sequence (hc: head_cost)
    static __host__ __device__ __forceinline__ void place(const Seq &s, int G, long hc, long x, Piece &out)
    {
        out.h = (int)(x / hc);
        x -= out.h * hc;
        int mt = 0;
        for (;;) {
            const int t = cost(s, G, mt);
            if (x < t) break;
            x -= t;
            ++mt;
        }
        out.mt = mt;
        out.off = x;
    }
};

// By one warp, 32 sequences at a time, the next ones' lengths being read under
// the arithmetic.  A first round (lo < 0) adds up the costs and keeps those of
// the first 32 chunks of 32 sequences, one per lane, so that the second one,
// which finds the sequence that holds the piece's beginning, can go straight to
// its chunk.  One loop serves both: code that runs once is paid for in
// instruction fetches.
template <int BM, int BN>
__device__ __forceinline__ void find_piece(const Pool &P, const WorkDim &W, int cta, int n_cta, Piece *out)
{
    using U = Units<BM, BN>;
    const int lane = threadIdx.x & 31, chunks = (P.B + 31) / 32;
    auto fetch = [&](int c) {
        const int b = 32 * c + lane;
        return b < P.B ? raw_seq(W.q_start, W.ctx_len, b) : RawSeq{0, 0, 0};
    };
    if (lane == 0) out->len = 0;
    long lo = -1, hi = 0, per = 0, before = 0, chunk = 0;
    int c = 0;
    RawSeq next = fetch(0);
#pragma unroll 1
    for (;;) {
        const Seq s = check_seq(P, next, W.T);
        if (c + 1 < chunks) next = fetch(c + 1);
        const long hc = U::head_cost(s, W.G), x = hc * P.Hkv;
        long incl = x;                               // inclusive over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const long sum = __shfl_sync(0xffffffffu, incl, 31), start = before + incl - x;
        if (lo >= 0) {
            const bool here = start <= lo && lo < start + x;
            if (here) {
                U::place(s, W.G, hc, lo - start, *out);
                out->b = 32 * c + lane;
                out->per = per;
                out->len = hi - lo;
            }
            if (__any_sync(0xffffffffu, here)) break;
        } else if (c == lane) {
            chunk = before + sum;                    // the running total
        }
        before += sum;
        if (++c < chunks) continue;
        if (lo >= 0) break;                          // not reached: lo lies below the total
        per = piece_len(before, n_cta, U::kMinPiece);
        lo = per * cta;
        hi = lmin(before, lo + per);
        if (lo >= hi) break;
        c = __popc(__ballot_sync(0xffffffffu, lane < chunks && chunk <= lo));   // chunks that end at or before lo
        before = c ? __shfl_sync(0xffffffffu, chunk, c - 1) : 0;
        next = fetch(c);
    }
    __syncwarp();
}

// One unit, or the part of it that falls to this CTA.
struct Item {
    int b, h, mt;
    int tok0, n, ctx;      // the sequence
    int rows;              // valid rows of the tile
    int t_lo, t_hi;        // key tiles of this part
    bool whole;            // the part is the whole unit: written to the output
    bool head;             // a partial unit's first part
    int parts;             // head: how many CTAs share the unit
};

// Walks a piece; every role of a CTA walks it alike.
template <int BM, int BN>
struct Walk {
    using U = Units<BM, BN>;
    int b, h, mt;
    long off, left, per;
    Seq s;
    int m;

    __host__ __device__ __forceinline__ void start(const Pool &P, const WorkDim &W, const Piece &p)
    {
        b = p.b;
        h = p.h;
        mt = p.mt;
        off = p.off;
        left = p.len;
        per = p.per;
        if (left > 0) {
            s = load_seq(P, W.q_start, W.ctx_len, W.T, b);
            m = U::mtiles(s, W.G);
        }
    }
    // The next part with at least one key tile; false at the piece's end.
    __host__ __device__ __forceinline__ bool next(const Pool &P, const WorkDim &W, Item &it)
    {
        while (left > 0) {
            const int cost = U::cost(s, W.G, mt), weight = U::weight(s, W.G, mt);
            const long take = lmin(left, (long)cost - off);
            const bool uncut = cost <= U::kWhole, mine = !uncut || (off <= cost / 2 && cost / 2 < off + take);
            const long a = uncut ? 0 : off, e = uncut ? cost : off + take;
            it.b = b;
            it.h = h;
            it.mt = mt;
            it.tok0 = s.tok0;
            it.n = s.n;
            it.ctx = s.ctx;
            it.rows = (int)lmin((long)BM, (long)s.n * W.G - (long)mt * BM);
            // the unit's first kUnitCost cost units carry no tile
            it.t_lo = (int)(lmax(a - U::kUnitCost, 0) / weight);
            it.t_hi = (int)(lmax(e - U::kUnitCost, 0) / weight);
            const bool starts = it.t_lo == 0, ends = e == cost;
            it.head = starts;
            it.whole = starts && ends;
            it.parts = 0;
            if (starts && !ends) it.parts = 1 + (int)((cost - e + per - 1) / per);
            left -= take;
            off = 0;
            if (++mt == m) {
                mt = 0;
                if (++h == P.Hkv) {
                    h = 0;
                    m = 0;
                    while (left > 0 && m == 0 && ++b < P.B) {
                        s = load_seq(P, W.q_start, W.ctx_len, W.T, b);
                        m = U::mtiles(s, W.G);
                    }
                    if (m == 0) left = 0;
                }
            }
            if (mine && it.t_hi > it.t_lo) return true;
        }
        return false;
    }
};

// ----- partial results ------------------------------------------------------------
// A CTA takes part in at most two units that others share: one that began in
// an earlier CTA (slot 0; it is the first of the piece) and one whose first
// part it holds (slot 1; it is the last of the piece).  desc[c] describes the
// latter: its parts are slot 1 of CTA c and slot 0 of CTAs c + 1 ..
// c + parts - 1; parts = 0 when there is none.
struct PartDesc {
    int parts, tok0, h, row0, rows, pad[3];
};

struct Parts {
    PartDesc *desc;    // [n_cta]
    float2 *ml;        // [n_cta][2][rows_cap]: running maximum (log2 domain) and sum
    float *o;          // [n_cta][2][rows_cap][d], not divided by the sum
    int rows_cap;

    __device__ __forceinline__ size_t row(int cta, int slot, int r) const
    {
        return ((size_t)cta * 2 + slot) * rows_cap + r;
    }
};

// ----- pieces of the tensor-core kernels ----------------------------------------------
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A place in a ring of N buffers and the parity of its current round.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++slot == N) slot = 0, phase ^= 1;
    }
    __device__ __forceinline__ Ring after() const
    {
        Ring r = *this;
        r.next();
        return r;
    }
};

// A bounded wait by one thread: on a timeout it is reported and the CTA's
// other roles, whose waits then run out too, leave as well.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, int32_t *status, int where)
{
    if (mbar_wait(bar, parity)) return true;
    report_timeout(status, where);
    return false;
}
// The same by a whole warp, which stays together.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, int32_t *status, int where)
{
    return __all_sync(0xffffffffu, wait_bar(bar, parity, status, where));
}

// ----- launchers ----------------------------------------------------------------------
// paged_attn_simt.cu: fp32 on the CUDA cores
constexpr int kSimtKeys = 32;      // the smallest key tile of its variants
int simt_rows(int T, int G, int B);
int simt_ctas();
cudaError_t attn_simt(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, void *out, float *lse,
                      const Parts &parts, cudaStream_t st);
cudaError_t mass_simt(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, const float *lse,
                      float *scores, int scores_stride, cudaStream_t st);

// paged_attn_tc.cu: bf16 on the tensor cores, row tiles of 256
constexpr int kTcRows = 256, kTcKeys = 128;
int tc_ctas();
// s_out (or null): the products q . k of every row, s_stride apart (a multiple
// of 128, at least the table's slots)
cudaError_t attn_tc(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, void *out, float *lse,
                    float *s_out, long s_stride, const Parts &parts, int32_t *status, cudaStream_t st);

// paged_mass_tc.cu: scores += the attention weight of every slot, lse (log2
// domain) of every row given
cudaError_t mass_tc(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, const float *lse,
                    float *scores, int scores_stride, int32_t *status, cudaStream_t st);

// paged_attn.cu: attention, with scores != null also the attention mass
size_t attn_ws_bytes(vc_dtype dt, int d, int T, int Hq, int Hkv, int B, long cap, bool mass);
cudaError_t attn(const Pool &P, vc_dtype dt, int d, const void *q, const int32_t *q_start, const int32_t *ctx_len,
                 int T, int Hq, float sm_scale, void *out, float *scores, int scores_stride, void *ws, cudaStream_t st);

// paged_append.cu
cudaError_t append(const Pool &P, vc_dtype dt, int d, const void *qkv, const void *q_gain, const void *k_gain,
                   float eps, const vc_rope &rope, const int32_t *positions, const int32_t *q_start,
                   const int32_t *ctx_len, int T, int Hq, void *q_out, cudaStream_t st);

// paged_evict.cu
cudaError_t evict(const Pool &S, const Pool &Dp, int row_bytes, const float *scores, int scores_stride,
                  const int32_t *src_len, long top, long recent, int32_t *dst_len, int32_t *kept_idx, int kept_stride,
                  float *scores_out, int out_stride, cudaStream_t st);

}  // namespace paged
}  // namespace vc
