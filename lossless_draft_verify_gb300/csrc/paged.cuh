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
    uint8_t *k_scale, *v_scale;    // 8-bit pages: [n_pages][Hkv][page], else null

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

    // row i sees keys 0 .. last(i); the sequence has len() of them
    __host__ __device__ __forceinline__ int last(int i) const { return ctx + i; }
    __host__ __device__ __forceinline__ int len() const { return ctx + n; }
};

// An entry of a planned batch (paged_shared.cu): rows and keys of its own.
// The keys are the slots from `base` (a page's first) of sequence b's table; row
// i sees keys 0 .. ctx + step i, step 1 for a sequence's own slots, 0 for a prefix,
// which all rows see whole.  Results go to row out0 + i.
struct alignas(8) VSeq {
    int tok0, n, ctx, step, base, b, out0, pad;

    __host__ __device__ __forceinline__ int last(int i) const { return ctx + step * i; }
    __host__ __device__ __forceinline__ int len() const { return step ? ctx + n : ctx + 1; }
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

// The sequence that packed row `tok` belongs to: the last one that starts at or
// before it, by one warp (32 probes a step); -1: none does.
__device__ __forceinline__ int find_seq(const int32_t *__restrict__ q_start, int B, int tok)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = B;
    for (;;) {
        const int step = (hi - lo + 31) / 32, b = lo + lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, b < hi && q_start[b] <= tok);
        if (le == 0) return -1;
        lo += (31 - __clz(le)) * step;
        hi = min(hi, lo + step);
        if (step == 1) return lo;
    }
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
    const VSeq *plan;      // a planned batch's entries, else null
    int n_plan;
};

// Entries of a batch: its sequences, or those of its plan.
template <typename S>
struct Source;
template <>
struct Source<Seq> {
    using Raw = RawSeq;
    static __host__ __device__ __forceinline__ int count(const Pool &P, const WorkDim &) { return P.B; }
    static __host__ __device__ __forceinline__ Raw raw(const WorkDim &W, int b) { return raw_seq(W.q_start, W.ctx_len, b); }
    static __host__ __device__ __forceinline__ Raw none() { return RawSeq{0, 0, 0}; }
    static __host__ __device__ __forceinline__ Seq check(const Pool &P, const WorkDim &W, const Raw &r) { return check_seq(P, r, W.T); }
};
template <>
struct Source<VSeq> {
    using Raw = VSeq;
    static __host__ __device__ __forceinline__ int count(const Pool &, const WorkDim &W) { return W.n_plan; }
    static __host__ __device__ __forceinline__ Raw raw(const WorkDim &W, int i) { return W.plan[i]; }
    static __host__ __device__ __forceinline__ Raw none() { return VSeq{0, 0, 0, 1, 0, 0, 0, 0}; }
    static __host__ __device__ __forceinline__ VSeq check(const Pool &, const WorkDim &, const Raw &r) { return r; }
};
template <typename S>
__host__ __device__ __forceinline__ S load_entry(const Pool &P, const WorkDim &W, int i)
{
    return Source<S>::check(P, W, Source<S>::raw(W, i));
}

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
    static constexpr bool kByTiles = false;
    static constexpr int kUnitCost = BM == 256 ? 16 : 1;
    static constexpr int kMinPiece = BM == 256 ? 10 : 2;
    static constexpr int kWhole = BM == 256 ? 20 : 3;
    static constexpr int kSlack = 0;
};
// Pieces of one warp each, in tiles of few_keys() (paged_attn_few.cuh).  A lone warp
// takes about 1 us for a tile, so small batches are cut finely: unit cost, least piece
// and whole units of 3, 8, 12, of 2, 2, 4 and of 2, 1, 3, one token of one sequence over
// 1000 (32/8 heads of 128) 23.9, 11.6 and 10.7 us, of 16 over 500 21.5, 12.8 and 12.6, of
// 16 over 32768 the same.  A unit that is little longer (kSlack) than a piece is not cut
// either: of units longer than a piece a piece holds one middle at most, so that a warp
// takes at most kSlack tiles more, some 4 us, and the batch needs no parts, whose merge
// takes about as long.  (Of shorter units a piece can hold several middles, and one taken
// whole may be another unit's length too much; they are cut.)  Cutting, and without, 128
// sequences of 150 tokens 26.5 and 19.9 us, 96 20.8 and 17.8, 128 of 250 30.3 and 27.0.
struct CostFew {
    static constexpr bool kByTiles = true;
    static constexpr int kUnitCost = 2;
    static constexpr int kMinPiece = 1;
    static constexpr int kWhole = 3;
    static constexpr int kSlack = 4;
};
// fp32 rows, whose tiles take longer, and planned batches, whose pieces pass from long
// units to short ones: with a slack four chunks up to 17 over 2000 21.0 us for 16.5, 32
// sequences in two groups over 8-bit pages 80.9 for 78.3.
struct CostFewCut : CostFew {
    static constexpr int kSlack = 0;
};

// What one CTA has to do: from unit (b, h, mt), cost offset `off` within it,
// `len` cost units on.  Written to shared memory by one warp, read by all.
struct Piece {
    int b, h, mt;
    long off, len;     // off: cost already covered by earlier CTAs
    long per;          // the length of a full piece
};

// With the entry that it begins in.
template <typename S>
struct PieceOf : Piece {
    S s;
};

// a / b of numbers that are not negative: 64-bit division takes a hundred instructions.
// For the kernel of few rows; the tensor-core kernel gains nothing from it, nor from the
// entry found with the piece (a verify batch of nine chunks 384 us, with that 391).
__host__ __device__ inline long quotient(long a, long b)
{
    return (unsigned long)(a | b) >> 32 == 0 ? (long)((unsigned)a / (unsigned)b) : a / b;
}

__host__ __device__ inline long piece_len(long total, int n_cta, int min_len)
{
    return lmax((total + n_cta - 1) / n_cta, min_len);
}

template <int BM, int BN, typename C = Cost<BM>>
struct Units : C {
    using C::kUnitCost;
    // 32-bit arithmetic: a sequence has at most 2^30 rows
    template <typename S>
    static __host__ __device__ __forceinline__ int tiles(const S &s, int G, int mt)
    {
        const unsigned rows = (unsigned)s.n * G, end = ((unsigned)mt + 1) * BM;
        const unsigned last = (rows < end ? rows : end) - 1;              // last row of the tile
        return (int)(((unsigned)s.last((int)(last / (unsigned)G)) + 1 + BN - 1) / BN);
    }
    template <typename S>
    static __host__ __device__ __forceinline__ int weight(const S &s, int G, int mt)
    {
        return BM == 256 && s.n * G - mt * BM > BM / 2 ? 2 : 1;
    }
    template <typename S>
    static __host__ __device__ __forceinline__ int cost(const S &s, int G, int mt)
    {
        return tiles(s, G, mt) * weight(s, G, mt) + kUnitCost;
    }
    template <typename S>
    static __host__ __device__ __forceinline__ int mtiles(const S &s, int G) { return (s.n * G + BM - 1) / BM; }
    // Row tiles of few rows are many, and many have the same tiles: how many take
    // `t` tiles at most.
    template <typename S>
    static __host__ __device__ __forceinline__ int upto(const S &s, int G, int t, int m, int last)
    {
        if (t >= last) return m;
        const long tok = (long)t * BN - s.ctx;               // tokens whose last key lies in the first t tiles
        return tok <= 0 ? 0 : (int)lmin((tok * G) / BM, m);
    }
    template <typename S>
    static __host__ __device__ __forceinline__ long head_cost(const S &s, int G)
    {
        if constexpr (C::kByTiles) {
            const int m = mtiles(s, G);
            if (m == 0) return 0;
            long c = (long)m * kUnitCost;
            const int first = tiles(s, G, 0), last = tiles(s, G, m - 1);
            for (int t = first, before = 0; t <= last; ++t) {
                const int n = upto(s, G, t, m, last);
                c += (long)(n - before) * t;
                before = n;
            }
            return c;
        }
        long c = 0;
        const int m = mtiles(s, G);
        for (int i = 0; i < m; ++i) c += cost(s, G, i);
        return c;
    }
    // head, row tile and offset of cost unit x of a sequence (hc: head_cost)
    template <typename S>
    static __host__ __device__ __forceinline__ void place(const S &s, int G, long hc, long x, Piece &out)
    {
        out.h = (int)(C::kByTiles ? quotient(x, hc) : x / hc);
        x -= out.h * hc;
        int mt = 0;
        if constexpr (C::kByTiles) {                         // past the row tiles of fewer tiles
            const int m = mtiles(s, G), last = tiles(s, G, m - 1);
            for (int t = tiles(s, G, 0); t <= last; ++t) {
                const int n = upto(s, G, t, m, last);
                const long c = (long)(n - mt) * (t + kUnitCost);
                if (x < c) {
                    const int i = (int)quotient(x, t + kUnitCost);
                    mt += i;
                    x -= (long)i * (t + kUnitCost);
                    break;
                }
                x -= c;
                mt = n;
            }
            out.mt = mt;
            out.off = x;
            return;
        }
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
// instruction fetches.  A round trip saved here is one less of a small call's few: of
// one token over 200 (8-bit pages) the kernel took 7 us, 2.1 of them here and 1.6 up to
// the first request for keys.
template <int BM, int BN, typename S = Seq, typename C = Cost<BM>>
__device__ __forceinline__ void find_piece(const Pool &P, const WorkDim &W, int cta, int n_cta, PieceOf<S> *out)
{
    using U = Units<BM, BN, C>;
    using Src = Source<S>;
    const int lane = threadIdx.x & 31, count = Src::count(P, W), chunks = (count + 31) / 32;
    auto fetch = [&](int c) {
        const int b = 32 * c + lane;
        return b < count ? Src::raw(W, b) : Src::none();
    };
    if (lane == 0) out->len = 0;
    long lo = -1, hi = 0, per = 0, before = 0, chunk = 0;
    int c = 0;
    typename Src::Raw next = fetch(0);
#pragma unroll 1
    for (;;) {
        const S s = Src::check(P, W, next);
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
                out->s = s;
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
        per = C::kByTiles ? lmax(quotient(before + n_cta - 1, n_cta), U::kMinPiece) : piece_len(before, n_cta, U::kMinPiece);
        lo = per * cta;
        hi = lmin(before, lo + per);
        if (lo >= hi) break;
        c = __popc(__ballot_sync(0xffffffffu, lane < chunks && chunk <= lo));   // chunks that end at or before lo
        before = c ? __shfl_sync(0xffffffffu, chunk, c - 1) : 0;
        if (chunks > 1) next = fetch(c);
    }
    __syncwarp();
}

// One unit, or the part of it that falls to this CTA.
template <typename S>
struct ItemOf;
template <>
struct ItemOf<Seq> {
    int b, h, mt;
    int tok0, n, ctx;      // the sequence
    int rows;              // valid rows of the tile
    int t_lo, t_hi;        // key tiles of this part
    bool whole;            // the part is the whole unit: written to the output
    bool head;             // a partial unit's first part
    int parts;             // head: how many CTAs share the unit

    __host__ __device__ __forceinline__ int last(int i) const { return ctx + i; }
    __host__ __device__ __forceinline__ int len() const { return ctx + n; }
    __host__ __device__ __forceinline__ int first_slot() const { return 0; }
    __host__ __device__ __forceinline__ int out_tok0() const { return tok0; }
    __host__ __device__ __forceinline__ void set(int entry, const Seq &s) { b = entry, tok0 = s.tok0, n = s.n, ctx = s.ctx; }
};
template <>
struct ItemOf<VSeq> : ItemOf<Seq> {
    int step, base, out0;

    __host__ __device__ __forceinline__ int last(int i) const { return ctx + step * i; }
    __host__ __device__ __forceinline__ int len() const { return step ? ctx + n : ctx + 1; }
    __host__ __device__ __forceinline__ int first_slot() const { return base; }
    __host__ __device__ __forceinline__ int out_tok0() const { return out0; }
    __host__ __device__ __forceinline__ void set(int, const VSeq &s)
    {
        b = s.b, tok0 = s.tok0, n = s.n, ctx = s.ctx, step = s.step, base = s.base, out0 = s.out0;
    }
};
using Item = ItemOf<Seq>;

// Walks a piece; every role of a CTA walks it alike.
template <int BM, int BN, typename S = Seq, typename C = Cost<BM>>
struct Walk {
    using U = Units<BM, BN, C>;
    int b, h, mt;          // b: the entry
    long off, left, per;
    S s;
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
            s = load_entry<S>(P, W, b);
            m = U::mtiles(s, W.G);
        }
    }
    __host__ __device__ __forceinline__ void start(const WorkDim &W, const PieceOf<S> &p)
    {
        b = p.b;
        h = p.h;
        mt = p.mt;
        off = p.off;
        left = p.len;
        per = p.per;
        if (left > 0) {
            s = p.s;
            m = U::mtiles(s, W.G);
        }
    }
    // The next part with at least one key tile; false at the piece's end.
    __host__ __device__ __forceinline__ bool next(const Pool &P, const WorkDim &W, ItemOf<S> &it)
    {
        while (left > 0) {
            const int cost = U::cost(s, W.G, mt), weight = U::weight(s, W.G, mt);
            const long take = lmin(left, (long)cost - off);
            const bool uncut = cost <= U::kWhole || (C::kByTiles && cost > per && cost <= per + C::kSlack), mine = !uncut || (off <= cost / 2 && cost / 2 < off + take);
            const long a = uncut ? 0 : off, e = uncut ? cost : off + take;
            it.set(b, s);
            it.h = h;
            it.mt = mt;
            it.rows = (int)lmin((long)BM, (long)s.n * W.G - (long)mt * BM);
            // the unit's first kUnitCost cost units carry no tile
            it.t_lo = (int)(lmax(a - U::kUnitCost, 0) / weight);
            it.t_hi = (int)(lmax(e - U::kUnitCost, 0) / weight);
            const bool starts = it.t_lo == 0, ends = e == cost;
            it.head = starts;
            it.whole = starts && ends;
            it.parts = 0;
            if (starts && !ends) {
                const long rest = cost - e + per - 1;
                it.parts = 1 + (int)(C::kByTiles ? quotient(rest, per) : rest / per);
            }
            left -= take;
            off = 0;
            if (++mt == m) {
                mt = 0;
                if (++h == P.Hkv) {
                    h = 0;
                    m = 0;
                    while (left > 0 && m == 0 && ++b < Source<S>::count(P, W)) {
                        s = load_entry<S>(P, W, b);
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
    int rows_cap, n_cta;

    __device__ __forceinline__ size_t row(int cta, int slot, int r) const
    {
        return ((size_t)cta * 2 + slot) * rows_cap + r;
    }
};

// Where a row of a planned batch's halves is: in the output (parts 0), or in parts as
// PartDesc has them, row r of each.  Written with the row's first part.
struct Place {
    uint32_t cta_parts, r;     // cta | parts << 16

    static __host__ __device__ __forceinline__ Place in_output() { return Place{0, 0}; }
    static __host__ __device__ __forceinline__ Place in_parts(int cta, int parts, int r)
    {
        return Place{(uint32_t)cta | (uint32_t)parts << 16, (uint32_t)r};
    }
    __host__ __device__ __forceinline__ int cta() const { return (int)(cta_parts & 0xffffu); }
    __host__ __device__ __forceinline__ int parts() const { return (int)(cta_parts >> 16); }
    // Whether it names parts that are there: not where a wait ran out (reported) before
    // it was written, and the workspace holds whatever it did.
    __host__ __device__ __forceinline__ bool fits(const Parts &p) const
    {
        return parts() > 0 && cta() + parts() <= p.n_cta && r < (uint32_t)p.rows_cap;
    }
};
// What a planned batch's attention leaves: o (normalised) and lse of the rows that
// are not in parts, and every row's place.
struct Halves {
    float *o;                  // [2][T][Hq][d], the prefix's half first
    float *lse;                // [2][T][Hq]
    Place *place;              // [2][T][Hq]
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
int simt_rows(int T, int G, int B, bool planned);
int simt_ctas();
cudaError_t attn_simt(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, void *out, float *lse,
                      const Parts &parts, cudaStream_t st, Place *place = nullptr);
cudaError_t mass_simt(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, const float *lse,
                      float *scores, int scores_stride, cudaStream_t st);

// paged_attn_tc.cu: bf16 on the tensor cores, row tiles of 256
constexpr int kTcRows = 256, kTcKeys = 128;
int tc_ctas();
// s_out (or null): the products q . k of every row, s_stride apart (a multiple
// of 128, at least the table's slots)
cudaError_t attn_tc(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, void *out, float *lse,
                    float *s_out, long s_stride, const Parts &parts, int32_t *status, cudaStream_t st);
// A planned batch's attention (W.plan)
cudaError_t attn_tc_planned(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, const Halves &H,
                            const Parts &parts, int32_t *status, cudaStream_t st);
// paged_attn_few.cuh: for batches of few rows: pieces per warp, row tiles of few_rows()
// (0: the batch has too many), of fp32 rows 8 or 16 in all batches.  The host knows the
// batch's average only (lengths lie on the device), and each kernel does badly what the
// other is for: 8-bit pages, 32/8 heads of 128, 31 decoding sequences over 4000 with one
// chunk of 97 over 30000 (16 rows on average) 360 us here, with one of 98 192 on the tensor
// cores, as two calls 57 and 77; 127 over 1000 with one of 385 1223, 386 499, apart 61 and
// 288; 15 over 32768 with one of 2048 over 30000 1694, apart 169 and 763.  The bound is that
// of batches of one kind: at 16 rows 70 us here and 122 there, from 24 on there is nothing
// between them.  Over 8-bit pages,
// and planned batches over bf16 ones: begun beside the kernel launched before, which
// is waited for at the end only, unless it is the plan's (first)
constexpr int few_keys(int d, bool kv8) { return 4096 / (kv8 ? d : 2 * d); }      // of a tile: 4 KB
int few_pieces(int rows);
inline int few_rows(int T, int G, int B) { return (long)T * G <= 8l * B ? 8 : (long)T * G <= 16l * B ? 16 : 0; }
cudaError_t attn8_few(const Pool &P, const WorkDim &W, vc_dtype dt, int d, int rows, const void *q, int Hq, float sl2,
                      void *out, const Parts &parts, int32_t *status, cudaStream_t st);
cudaError_t attn8_few_planned(const Pool &P, const WorkDim &W, vc_dtype dt, int d, int rows, const void *q, int Hq,
                              float sl2, const Halves &H, bool first, const Parts &parts, int32_t *status,
                              cudaStream_t st);
cudaError_t attn_few_planned(const Pool &P, const WorkDim &W, int d, int rows, const void *q, int Hq, float sl2,
                             const Halves &H, bool first, const Parts &parts, int32_t *status, cudaStream_t st);

// paged_attn8_tc.cu: both over 8-bit pages
cudaError_t attn8_tc(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, void *out,
                     const Parts &parts, int32_t *status, cudaStream_t st);
cudaError_t attn8_tc_planned(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, const Halves &H,
                             const Parts &parts, int32_t *status, cudaStream_t st);

// paged_mass_tc.cu: scores += the attention weight of every slot, lse (log2
// domain) of every row given
cudaError_t mass_tc(const Pool &P, const WorkDim &W, int d, const void *q, int Hq, float sl2, const float *lse,
                    float *scores, int scores_stride, int32_t *status, cudaStream_t st);

// paged_shared.cu: groups of sequences [first[g], first[g + 1]) that share the
// first prefix[g] tokens.  The plan: an entry per group, then one per sequence.
struct Groups {
    const int32_t *first, *prefix;
    int n;
};
cudaError_t plan_shared(const Pool &P, const int32_t *q_start, const int32_t *ctx_len, int T, const Groups &G,
                        VSeq *plan, cudaStream_t st);
// out from the halves of every row; seqs: the plan's entries of the sequences; pre,
// own: the parts of the prefixes' half and of the other
cudaError_t join_shared(const Pool &P, vc_dtype dt, int d, const int32_t *q_start, int T, int Hq, const VSeq *seqs,
                        const Halves &H, const Parts &pre, const Parts &own, void *out, cudaStream_t st);

// paged_attn.cu: attention, with scores != null also the attention mass; shared:
// that of groups (scores null, n_groups those of its workspace)
size_t attn_ws_bytes(vc_dtype dt, int d, int T, int Hq, int Hkv, int B, long cap, bool mass, bool kv8);
size_t attn_shared_ws_bytes(vc_dtype dt, int d, int T, int Hq, int Hkv, int B, long cap, int n_groups, bool kv8);
cudaError_t attn(const Pool &P, vc_dtype dt, int d, const void *q, const int32_t *q_start, const int32_t *ctx_len,
                 int T, int Hq, float sm_scale, void *out, float *scores, int scores_stride, void *ws, cudaStream_t st);
cudaError_t attn_shared(const Pool &P, vc_dtype dt, int d, const void *q, const Groups &G, const int32_t *q_start,
                        const int32_t *ctx_len, int T, int Hq, float sm_scale, void *out, void *ws, cudaStream_t st);

// paged8_read.cu: rows back; the batch's pages as bf16 pages [B][max_blocks] with their table
cudaError_t expand8(const Pool &P, int d, const int32_t *q_start, const int32_t *ctx_len, int T, void *k_out,
                    void *v_out, int32_t *table_out, cudaStream_t st);
cudaError_t read8(const Pool &P, vc_dtype dt, int d, const int32_t *q_start, const int32_t *ctx_len, int T, void *k_out,
                  void *v_out, cudaStream_t st);

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
