// sv_tree_attend.cu -- attention of drafted tokens, a tree or a chain, over the
// paged cache (spec_tree_attend).
//
// For a key head the query rows of one sequence are its nodes times the G
// query heads that share the head: out[r] = sum_k p[r][k] V[k] / sum_k p[r][k],
// p = exp(scale q[r] . K[k]) over the keys row r sees.  One pass over the keys
// with the running maximum m and sum l of each row: a tile of keys gives
// S = Q K^T (tensor cores, fp32), p = 2^(c S - c m) with c = scale log2(e),
// l += sum p and O += P V (tensor cores, O fp32 in tensor memory); when m grows
// by more than 2^8 would allow, O and l are scaled down first.  P is rounded to
// the 16-bit type, the only one that meets a 16-bit V in an MMA: half an ulp of
// each p (2^-9 of it in bf16), while l takes p before the rounding.  In f16, whose
// smallest number is 2^-24, p and l are taken 2^7 times as large, the most that
// leaves p below the type's end: a long context's many p of 2^-25 add up.
//
// The bound is HBM for up to about 256 rows per key head (each key's 4 D bytes
// are read once per 256 rows and cost 4 D products per row), the tensor cores
// beyond.  So:
//  * Rows are tiles of 128: floor(128 / G) nodes times G heads, the M of the
//    MMA, whatever their number: the tensor pipe has time for 128 rows while
//    the keys stream, so few rows need no other form.
//  * Work items are (key head, sequence, group of row tiles).  All items' key
//    tiles in a row are cut into ranges of equal cost, one per SM, whatever the
//    batch: a long cache with few rows fills the machine, a ragged batch is
//    balanced, and the lengths are read on the GPU.  An item cut by a range's
//    end leaves partial sums (O, m, l) that k_tree_combine joins.  The key head
//    comes first, so that the SMs of all heads go through the same pages
//    together.
//  * A CTA has a scheduling warp (it walks the range and hands the others one
//    segment of an item at a time, which keeps that state out of their
//    registers), two producer warps (tensor-map copies of whole pages into
//    rings of 128-byte-swizzled key and value tiles; what few rows of Q leave
//    free is more stages), an MMA issuer and one or two softmax warpgroups, a
//    thread per row.
//  * Heads up to 128 elements have two streams (an O in tensor memory, the
//    scores of a tile of 128 keys, and a warpgroup): an item of one row tile
//    gives its even key tiles to one and its odd ones to the other (own m, l, O;
//    joined at the end, each warpgroup half of the columns), an item of two row
//    tiles gives each stream a row tile and reads the keys once for both.
//    Probabilities take the place of their scores and are handed over in halves:
//    the first meets its values while the warpgroup is at the second.  Tiles of
//    128 keys, as one MMA reads Q from shared memory once for 128 keys (64
//    cycles against twice 48).  Larger heads fill tensor memory with one stream,
//    whose two score buffers of 64 keys take turns.
//
// Measured (bf16, 8 key heads of 128 elements, 8 query heads to each where
// nothing else is said, L2 flushed; bytes of K and V once):
//   256 sequences of one token over 100 to 4000 keys: 347-355 us, 6.1-6.2 TB/s
//     (0.89-0.91 of a copy);
//   64 of up to 9 tokens over 100 to 4100 keys: 123-126 us, 4.5-4.6 TB/s;
//   one of 32 tokens over 260000 keys: 206-218 us, 4.9-5.2 TB/s and 1.3 PFLOP/s.
//     The chain scores, softmax, values of 256 rows takes some 3200 cycles a tile,
//     of which the MMAs are 2048;
//   16 of up to 64 tokens over 4000 to 8191 keys: 175-177 us, 1.0 PFLOP/s.  Both items
//     of a key head read the keys from HBM: 836 MB where they are 403;
//   6 chains of up to 333 f16 tokens of 7 heads of 80 elements: 61-69 us;
//   one token of 4 heads to a key head over 500 keys: 17.5-19.6 us (14.5 warm).
// An item costs some four tiles beside its keys: its masked tile, its output and
// the first softmax of the next item are a chain that the rings cover in part.
// Two warpgroups a stream, half of a tile's keys each, were slower (238 us where
// this takes 204): the softmax of 64 columns takes 421 cycles with one warp on a
// scheduler, 704 with the two that there are now and 1350 with four.  The 2^x are
// the largest part of it (4 cycles a warp and instruction, 512 of the 704), but the
// chain is the bound: with two row tiles their unit works 27 % of the time, the
// tensor cores 59 %.
//
// What a row does not see must not touch it, whatever it holds: scores are
// replaced by -inf before the maximum, but P V multiplies hidden values by a
// zero probability, and 0 x NaN is NaN.  In the tiles that some row sees only
// in part the softmax warps zero the rows beyond the sequence and every
// non-finite value in shared memory; rows that see a node with such values
// (rare) add them afterwards.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "sv_tcgen.cuh"
#include "sv_tree.cuh"

namespace sv {

constexpr int ATT_ROWS = 128;                 // rows of a row tile: M of the MMA
constexpr int ATT_SMEM = 227 * 1024;          // shared memory of a CTA
constexpr int ATT_MISC = 4096;                // of it: barriers and small tables
constexpr uint32_t ATT_TMEM_COLS = 512;
constexpr int ATT_SEGS = 4;                   // segments handed out ahead
constexpr uint32_t ATT_WAIT_POLLS = 1u << 17;  // limit of a wait: some seconds (a poll sleeps for microseconds)
constexpr uint32_t ATT_STALL_POLLS = 4096;    // SPEC_FAULT_STALL_STREAM
constexpr float ATT_LAZY = 8.f;               // log2 growth of the maximum that O takes unscaled
// log2 of what p, l and O are multiplied by: f16 ends at 2^16, and p is at most 2^ATT_LAZY
__host__ __device__ constexpr float att_up(bool f16) { return f16 ? 15.f - ATT_LAZY : 0.f; }
// natural logarithm of a row's sum l in units of its maximum m
template <bool F16>
__device__ __forceinline__ float att_lse(float m, float scale, float l)
{
    return fmaf(m, scale, logf(l * (F16 ? 1.f / (1 << (int)att_up(true)) : 1.f)));
}

constexpr int ATT_STAGES = 8;                 // most stages of a ring

template <int DP>
struct Att {                                  // DP: head size rounded up to 64
    static constexpr int NH = DP / 64;        // 64-column (128-byte) boxes of a row
    static constexpr int NS = DP <= 128 ? 2 : 1;     // streams (softmax warpgroups)
    static constexpr int KT = 64 * NS;        // keys of a tile: two halves of 64, or one
    static constexpr int UNIT = KT * DP * 2;  // bytes of a K or V tile
    static constexpr int ROOM = ATT_SMEM - 1024 - ATT_MISC;  // bytes for Q and the rings
    static constexpr int THREADS = 128 + 128 * NS;   // four warps, and the softmax warpgroups
    // scores of stream s: 128 columns, a tile's or (one stream) two buffers of a tile
    __host__ __device__ static constexpr uint32_t s_col(int s) { return 128u * s; }
    __host__ __device__ static constexpr uint32_t o_col(int s) { return NS == 2 ? 256u + 128u * s : 128u; }
    static_assert((ROOM - NS * ATT_ROWS * DP * 2) / UNIT >= 4, "the rings fit");
};

// one segment: the key tiles tile0 .. tile0 + nt - 1 of an item (nt = 0: the range's end)
struct __align__(16) AttSeg {
    int32_t b, hk;
    int32_t ctx, n;
    int32_t t0, ntok;           // the item's first node, and nodes
    int32_t tile0, nt;
    int32_t limit;              // keys any of its rows may see
    int32_t mask_from;          // keys below are seen by all its rows
    int32_t dual;               // two row tiles
    int32_t whole;              // all of the item's tiles
};

struct __align__(16) AttMisc {
    uint64_t k_full[ATT_STAGES], k_empty[ATT_STAGES];  // key tiles: copied; read by the MMAs
    uint64_t v_full[ATT_STAGES], v_empty[ATT_STAGES];  // value tiles
    uint64_t v_clean[ATT_STAGES];    // a masked value tile may meet the MMAs
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2][2];         // [stream][buffer] a tile's scores are in tensor memory
    uint64_t p_ready[2][2];        // [stream][half or buffer] probabilities are (and O is scaled)
    uint64_t o_full[2], o_empty[2];  // the segment's O is complete; has been read
    uint64_t j_full[4];            // [quarter] both streams' (m, l) are in ml
    uint64_t seg_full[ATT_SEGS], seg_empty[ATT_SEGS];
    uint64_t drain;
    AttSeg seg[ATT_SEGS];
    uint32_t nf[ATT_STAGES][4];    // (masked) value rows of the tile with non-finite elements
    float2 ml[2][ATT_ROWS];        // [stream] (m, l) of a row, for the join
    uint32_t tmem;
    int32_t failed;
};
static_assert(sizeof(AttMisc) <= ATT_MISC, "barriers and tables fit");

// ------------------------------------------------------------------------- //
// the work: items, and a CTA's range of key tiles                           //
// ------------------------------------------------------------------------- //
struct AttGeom {
    int G, tpt, group;  // heads per key head, nodes per row tile, nodes per item
    int Hkv;
};

// The ranges are equal in cost, not in tiles: an item costs its key tiles and
// ATT_ITEM_COST more (its first scores, its masked tile and its output).  With
// 2, 3, 4 and 5, 6 chains of 333 tokens take 65.6, 57.8, 55.5 and 57.6 us, a
// prompt of 4 x 1500 tokens 199, 192, 191 and 189 us, long caches the same.
constexpr int ATT_ITEM_COST = 4;

// keys that some row of item `rp` of a sequence sees: a chain's rows see
// nothing past their last node
__device__ __forceinline__ int att_limit(const TreeAttendParams& p, const AttGeom& g, int ctx, int n, int rp)
{
    return ctx + (p.mask ? n : min(n, (rp + 1) * g.group));
}
// key tiles of an item; its keys may reach 2^31 - 1
template <int KT>
__device__ __forceinline__ int att_tiles(int limit)
{
    return (int)(((uint32_t)limit + KT - 1) / KT);
}
template <int KT>
__device__ __forceinline__ int att_cost(const TreeAttendParams& p, const AttGeom& g, int ctx, int n, int rp)
{
    return att_tiles<KT>(att_limit(p, g, ctx, n, rp)) + ATT_ITEM_COST;
}
// cost of all items of one key head of a sequence
template <int KT>
__device__ __forceinline__ int att_head_cost(const TreeAttendParams& p, const AttGeom& g, int ctx, int n)
{
    if (n <= g.group) return n ? att_cost<KT>(p, g, ctx, n, 0) : 0;
    const int nrp = (n + g.group - 1) / g.group;
    if (p.mask) return nrp * att_cost<KT>(p, g, ctx, n, 0);
    int t = 0;
    for (int rp = 0; rp < nrp; ++rp) t += att_cost<KT>(p, g, ctx, n, rp);
    return t;
}

// `total` cut into `ctas` ranges that differ by one at most
struct AttSplit {
    int total, ctas, q, r;
    __device__ __forceinline__ AttSplit(int total_, int ctas_) : total(total_), ctas(min(ctas_, total_))
    {
        q = ctas ? total / ctas : 0;
        r = total - q * ctas;
    }
    __device__ __forceinline__ int start(int c) const { return c * q + min(c, r); }
    __device__ __forceinline__ int owner(int x) const
    {
        const int wide = r * (q + 1);
        return x < wide ? x / (q + 1) : r + (x - wide) / q;
    }
};

// the segments of a CTA: parts of items, in order of (key head, sequence, group)
template <int KT>
struct AttIter {
    int pos, end;               // cost positions in the order of all items
    int b, hk, rp;              // the item
    int at;                     // cost position of its begin
    int ctx, n;
    int t0, ntok;               // its first node and nodes
    int ntiles, tile0, tile1;   // its key tiles, and this segment's (none: tile0 >= tile1)
    int limit;                  // keys some of its rows see

    __device__ __forceinline__ bool more() const { return pos < end; }
    __device__ __forceinline__ void load_item(const TreeAttendParams& p, const AttGeom& g)
    {
        t0 = rp * g.group;
        ntok = min(g.group, n - t0);
        limit = att_limit(p, g, ctx, n, rp);
        ntiles = att_tiles<KT>(limit);
        tile0 = max(pos - at - ATT_ITEM_COST, 0);
        tile1 = min(end - at - ATT_ITEM_COST, ntiles);
    }
    __device__ __forceinline__ void load_seq(const TreeAttendParams& p)
    {
        const SeqLen l = tree_len(p.s, b);
        ctx = l.ctx;
        n = l.n;
    }
    // head0: key head of the range's begin; off: cost of sequence b0 before it
    __device__ __forceinline__ void start(const TreeAttendParams& p, const AttGeom& g, int pos0, int end0, int head0,
                                          int b0, int off)
    {
        pos = pos0;
        end = end0;
        if (!more()) return;
        hk = head0;
        b = b0;
        load_seq(p);
        rp = 0;
        if (n > g.group)
            for (int t; off >= (t = att_cost<KT>(p, g, ctx, n, rp)); ++rp) off -= t;
        at = pos - off;
        load_item(p, g);
        if (tile0 >= tile1) next(p, g);
    }
    __device__ __forceinline__ void next(const TreeAttendParams& p, const AttGeom& g)
    {
        do {
            at += ntiles + ATT_ITEM_COST;
            pos = at;
            if (!more()) return;
            if ((++rp) * g.group >= n) {
                rp = 0;
                do {
                    if (++b == p.s.B) {
                        b = 0;
                        ++hk;
                    }
                    load_seq(p);
                } while (n == 0);
            }
            load_item(p, g);
        } while (tile0 >= tile1);
    }
};

// A task of k_tree_combine: some rows and columns (number `sub` of its item's
// tasks) of an item whose tiles the CTAs first .. last share.
struct __align__(16) AttJoin {
    int32_t first, last;
    int32_t b, hk, t0, rows;
    int32_t sub;
    int32_t pad;
};
// Up to `few` parts: a task is 8 warps times 32 rows by 32 columns; more: 32 rows
// by 8.  A batch's cuts leave two or three parts, whose loads a warp has in flight
// at once; one sequence's long cache leaves up to one per SM, which one warp would
// add one after the other.  Always the first form: 8 tokens on one key head over
// 100000 keys take 110 us and not 25; always the second: 16 x 64 tokens over 8000
// keys 247 us and not 168.  Where all tasks of the second form have a CTA each,
// nothing is gained by the first (one token over 500 keys: 14.5 us, with it 16.5).
constexpr int ATT_FEW = 8;
__host__ __device__ __forceinline__ int att_join_tasks(int parts, int rows, int D, int few)
{
    const int rb = (rows + 31) / 32;
    return parts <= few ? (rb * ((D + 31) / 32) + 7) / 8 : rb * (D / 8);
}

struct AttWork {
    TreeAttendParams p;
    AttGeom g;
    float* part_o;      // [2 * CTAs][DP / 4][NS * 128] float4: O of a part, per 4 columns all rows
    float2* part_ml;    // [2 * CTAs][NS * 128]: (m, l) of a part's rows
    AttJoin* joins;     // the tasks of k_tree_combine
    unsigned* n_joins;  // their number; back at 0 after it
    unsigned* n_done;   // its CTAs that are done
    unsigned* err;
    int32_t page_box;   // tokens of one copied box: min(page, KT)
    int32_t k_stages, v_stages;
    uint32_t k_inv, v_inv;  // 2^32 over them, rounded up: a product's upper word is the quotient (tiles < 2^29)
    uint32_t g_inv;         // 2^16 over G, rounded up (row numbers are below 128)
    int32_t q_rows;     // rows of Q a buffer holds, a multiple of 8 (the MMA's other rows are never used)
    int32_t q_box;      // nodes of one copied box of Q
    int32_t few;        // most parts that are joined in the first form
    int32_t stall;
};

__device__ __forceinline__ bool att_wait(uint64_t* bar, uint32_t parity, const volatile int32_t* failed, uint32_t limit)
{
    for (uint32_t i = 0; i < limit; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 63u && *failed) return false;
    }
    return false;
}

// bits of the keys k0 .. k0 + 31 that node t sees
__device__ __forceinline__ uint32_t att_low(int count) { return count <= 0 ? 0u : count >= 32 ? ~0u : (1u << count) - 1u; }
__device__ __forceinline__ uint32_t att_sees(const TreeAttendParams& p, int b, int t, int ctx, int n, int k0)
{
    if (!p.mask) return att_low(ctx + t + 1 - k0);
    uint32_t v = att_low(ctx - k0);
    const uint32_t* m = p.mask + ((int64_t)b * p.s.T + t) * p.words;
    const int node = k0 - ctx;  // of bit 0
    if (node >= 0) {
        const int w = node >> 5;
        const uint32_t lo = w < p.words ? __ldg(m + w) : 0u, hi = w + 1 < p.words ? __ldg(m + w + 1) : 0u;
        v |= __funnelshift_r(lo, hi, node & 31);
    } else if (node > -32) {
        v |= __ldg(m) << -node;
    }
    return v & att_low(ctx + n - k0);
}

template <bool F16>
__device__ __forceinline__ bool att_nonfinite(uint16_t h)
{
    const uint32_t e = F16 ? 0x7C00u : 0x7F80u;
    return (h & e) == e;
}

// the segment's first tile that some row sees only in part
template <int KT>
__device__ __forceinline__ int att_first_masked(const AttSeg& sg)
{
    return max(0, sg.mask_from / KT - sg.tile0);
}

// zeroes the non-finite ones of a word's two values; true when there was one
template <bool F16>
__device__ __forceinline__ bool clean_word(uint32_t& v)
{
    const bool lo = att_nonfinite<F16>((uint16_t)v), hi = att_nonfinite<F16>((uint16_t)(v >> 16));
    if (lo) v &= 0xFFFF0000u;
    if (hi) v &= 0x0000FFFFu;
    return lo || hi;
}

// + 0 x v in both halves: what is not finite makes the sum NaN
template <bool F16>
__device__ __forceinline__ uint32_t add_zero_times(uint32_t v, uint32_t sum)
{
    if (F16) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(sum) : "r"(v), "r"(0u), "r"(sum));
    else asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(sum) : "r"(v), "r"(0u), "r"(sum));
    return sum;
}

// One warp's part of cleaning a masked value tile (keys from kb on): rows from
// key `end` on become 0, and so does what is not finite, noted in nf.  A tile
// that both warpgroups read is shared between them.  Eight rows at a time, every
// fourth or eighth eight a warp's, eight lanes per 128-byte row of a box.
template <bool F16, int DP>
__device__ __forceinline__ void att_clean(AttMisc& ms, unsigned char* tile, uint32_t st, int kb, int from, int end,
                                          bool shared, int s, int quarter, int lane)
{
    using A = Att<DP>;
#pragma unroll 1
    for (int g = (shared ? s * 4 : 0) + quarter; g < A::KT / 8; g += shared ? 8 : 4) {
        uint32_t bits = 0;
        if (kb + 8 * g + 7 >= from) {
            uint4* const a0 = (uint4*)(tile + (8 * g + (lane >> 3)) * 128) + (lane & 7);
            auto at = [&](int i, int h) { return a0 + (h * A::KT + 4 * i) * 8; };
            const int key0 = kb + 8 * g + (lane >> 3);
            uint32_t sum = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < A::NH; ++h) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (key0 + 4 * i >= end) *at(i, h) = v;
                    else if (key0 + 4 * i >= from) v = *at(i, h);
                    sum = add_zero_times<F16>(v.x, sum);
                    sum = add_zero_times<F16>(v.y, sum);
                    sum = add_zero_times<F16>(v.z, sum);
                    sum = add_zero_times<F16>(v.w, sum);
                }
            if (__any_sync(0xffffffffu, sum != 0)) {  // rare
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    bool found = false;
#pragma unroll 1
                    for (int h = 0; h < A::NH && key0 + 4 * i >= from; ++h) {
                        uint4 v = *at(i, h);
                        const bool bad = clean_word<F16>(v.x) | clean_word<F16>(v.y) | clean_word<F16>(v.z) |
                                         clean_word<F16>(v.w);
                        if (bad) *at(i, h) = v;
                        found = found || bad;
                    }
                    const uint32_t v = __ballot_sync(0xffffffffu, found);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if ((v >> (8 * j)) & 0xFFu) bits |= 1u << (4 * i + j);
                }
            }
        }
        if (lane == 0) ((uint8_t*)ms.nf[st])[g] = (uint8_t)bits;
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_n(&ms.v_clean[st], A::NS == 2 && !shared ? 2 : 1);
}

// O += the non-finite values of the keys kb + i whose bits i are set in see0, see1
template <bool F16>
__device__ __noinline__ void att_add_nonfinite(const TreeAttendParams& p, uint32_t see0, uint32_t see1, int b, int hk,
                                               int kb, uint32_t o_addr)
{
#pragma unroll 1
    for (int y = 0; y < 2; ++y) {
        const uint32_t mine = y ? see1 : see0;
        for (uint32_t any = __reduce_or_sync(0xffffffffu, mine); any; any &= any - 1) {
            const int bit = __ffs(any) - 1, key = kb + 32 * y + bit;
            const int page = __ldg(p.table + (int64_t)b * p.s.width + (key >> p.s.page_log2));
            if (page < 0 || page >= p.s.num_pages) continue;
            const uint16_t* v = (const uint16_t*)p.c.v + page * p.c.page +
                                (key & ((1 << p.s.page_log2) - 1)) * p.c.token + hk * p.c.head;
#pragma unroll 1
            for (int d = 0; d < p.s.D; d += 16) {
                uint32_t o[16];
                tmem_ld<16>(o_addr + d, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint16_t e = __ldg(v + d + i);
                    if (att_nonfinite<F16>(e) && ((mine >> bit) & 1u))
                        o[i] = __float_as_uint(__uint_as_float(o[i]) + Half2<F16>::one(e));
                }
                tmem_st<16>(o_addr + d, o);
            }
            tmem_wait_st();
        }
    }
}

template <bool F16, int DP>
__global__ void __launch_bounds__(Att<DP>::THREADS, 1)
    k_tree_attend(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const AttWork w)
{
    using A = Att<DP>;
    using H = Half2<F16>;
    constexpr int KT = A::KT, NS = A::NS, NH = A::NH;
    const uint32_t KS = w.k_stages, VS = w.v_stages;
    auto k_round_of = [&](uint32_t i) { return __umulhi(i, w.k_inv); };
    auto v_round_of = [&](uint32_t i) { return __umulhi(i, w.v_inv); };
    auto v_stage_of = [&](uint32_t i) { return i - v_round_of(i) * VS; };
    extern __shared__ unsigned char att_raw[];
    const uint32_t raw = smem_u32(att_raw);
    // tables, Q buffers, rings; Q's unused rows reach into the rings
    unsigned char* const q_smem = att_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t q_bytes = w.q_rows * DP * 2;
    unsigned char* const k_smem = q_smem + NS * q_bytes;
    unsigned char* const v_smem = k_smem + KS * A::UNIT;
    AttMisc& ms = *reinterpret_cast<AttMisc*>(q_smem + A::ROOM);
    const TreeAttendParams& p = w.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t limit = w.stall ? ATT_STALL_POLLS : ATT_WAIT_POLLS;
    const volatile int32_t* failed = &ms.failed;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        tma_prefetch_map(&map_k);
        tma_prefetch_map(&map_q);
        tma_prefetch_map(&map_v);
    }
    if (warp == 2) tmem_alloc(&ms.tmem, ATT_TMEM_COLS);
    if (warp == 1) {
        if (lane < ATT_STAGES) {
            mbar_init(&ms.k_full[lane], 1);
            mbar_init(&ms.k_empty[lane], NS);
            mbar_init(&ms.v_full[lane], 1);
            mbar_init(&ms.v_empty[lane], 1);
            mbar_init(&ms.v_clean[lane], 4 * NS);
        }
        if (lane < 2) {
            mbar_init(&ms.q_full[lane], 1);
            mbar_init(&ms.q_empty[lane], 1);
            for (int j = 0; j < 2; ++j) {
                mbar_init(&ms.s_full[lane][j], 1);
                mbar_init(&ms.p_ready[lane][j], 4);
            }
            mbar_init(&ms.o_full[lane], 1);
            mbar_init(&ms.o_empty[lane], 4 * NS);
        }
        if (lane < ATT_SEGS) {
            mbar_init(&ms.seg_full[lane], 1);
            mbar_init(&ms.seg_empty[lane], 3 + 4 * NS);
            mbar_init(&ms.j_full[lane], 2);
        }
        if (lane == 0) {
            mbar_init(&ms.drain, 1);
            ms.failed = 0;
        }
        fence_barrier_init();
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = ms.tmem;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {  // whole warp
        if (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1u)))
            ok = ok && __all_sync(0xffffffffu, att_wait(bar, parity & 1u, failed, limit));
    };
    auto until = [&](uint64_t* bar, uint32_t parity) {  // one thread
        if (!mbar_try_wait(bar, parity & 1u)) ok = ok && att_wait(bar, parity & 1u, failed, limit);
    };
    // the k-th segment; done with it
    auto segment = [&](uint32_t k) -> const AttSeg& {
        wait(&ms.seg_full[k % ATT_SEGS], k / ATT_SEGS);
        return ms.seg[k % ATT_SEGS];
    };
    auto release = [&](uint32_t k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.seg_empty[k % ATT_SEGS]);
    };

    if (warp == 3) {
        // ---------------- scheduler: finds the range by a scan of the sequences' costs,
        // a run of sequences per lane (in one warp: the others need no barrier for it)
        const int per = (p.s.B + 31) / 32, seq0 = min(p.s.B, lane * per), seq1 = min(p.s.B, seq0 + per);
        int sum = 0;
#pragma unroll 4
        for (int b = seq0; b < seq1; ++b) {
            const SeqLen l = tree_len(p.s, b);
            sum += att_head_cost<KT>(p, w.g, l.ctx, l.n);
        }
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += v;
        }
        const int per_head = __shfl_sync(0xffffffffu, before, 31);
        before -= sum;
        const AttSplit split(per_head * w.g.Hkv, gridDim.x);
        const bool busy = (int)blockIdx.x < split.ctas;
        const int pos0 = split.start(blockIdx.x), head0 = busy ? pos0 / per_head : 0, in_head = pos0 - head0 * per_head;
        int first_b = seq0, off = in_head - before;
        const bool mine = busy && off >= 0 && off < sum;
        if (mine)
            for (;; ++first_b) {
                const SeqLen l = tree_len(p.s, first_b);
                const int t = att_head_cost<KT>(p, w.g, l.ctx, l.n);
                if (off < t) break;
                off -= t;
            }
        const int who = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        first_b = __shfl_sync(0xffffffffu, first_b, max(who, 0));
        off = __shfl_sync(0xffffffffu, off, max(who, 0));
        AttIter<KT> it;
        it.start(p, w.g, busy ? pos0 : 0, busy ? split.start(blockIdx.x + 1) : 0, head0, first_b, off);
        for (uint32_t k = 0; ok; ++k) {
            const uint32_t slot = k % ATT_SEGS;
            if (k >= ATT_SEGS) wait(&ms.seg_empty[slot], k / ATT_SEGS - 1);
            if (!ok) break;
            const bool more = it.more();
            if (lane == 0) {
                AttSeg& sg = ms.seg[slot];
                sg.nt = more ? it.tile1 - it.tile0 : 0;
                if (more) {
                    sg.b = it.b;
                    sg.hk = it.hk;
                    sg.ctx = it.ctx;
                    sg.n = it.n;
                    sg.t0 = it.t0;
                    sg.ntok = it.ntok;
                    sg.tile0 = it.tile0;
                    sg.limit = it.limit;
                    sg.mask_from = p.mask ? it.ctx : it.ctx + it.t0 + 1;
                    sg.dual = it.ntok > w.g.tpt;
                    sg.whole = it.tile0 == 0 && it.tile1 == it.ntiles;
                }
                mbar_arrive(&ms.seg_full[slot]);
            }
            __syncwarp();
            if (!more) break;
            if (k == 0 && it.tile0 > 0) {
                // the item began in an earlier range.  Where that is the one before,
                // this is the first cut of the item, and its join is announced here.
                const int first = split.owner(it.at + ATT_ITEM_COST);
                if (first == (int)blockIdx.x - 1) {
                    const int last = split.owner(it.at + ATT_ITEM_COST + it.ntiles - 1), rows = it.ntok * w.g.G;
                    const int tasks = att_join_tasks(last - first + 1, rows, p.s.D, w.few);
                    unsigned at = 0;
                    if (lane == 0) at = atomicAdd(w.n_joins, (unsigned)tasks);
                    at = __shfl_sync(0xffffffffu, at, 0);
                    for (int i = lane; i < tasks; i += 32)
                        w.joins[at + i] = AttJoin{first, last, it.b, it.hk, it.t0, rows, i, 0};
                }
            }
            it.next(p, w.g);
        }
        if (!ok && lane == 0) ms.failed = 1;
    } else if (warp == 0 || warp == 2) {
        // ---------------- producers: warp 0 keys and the rows of Q, warp 2 values
        const bool is_k = warp == 0;
        const CUtensorMap* map = is_k ? &map_k : &map_v;
        unsigned char* const ring = is_k ? k_smem : v_smem;
        uint64_t *const full = is_k ? ms.k_full : ms.v_full, *const empty = is_k ? ms.k_empty : ms.v_empty;
        const uint32_t stages = is_k ? KS : VS;
        const int page_mask = (1 << p.s.page_log2) - 1;
        uint32_t n = 0, st = 0, round = 0, qi = 0;  // stages filled, the next one; row tiles of Q
        for (uint32_t k = 0; ok && !w.stall; ++k) {
            const AttSeg& sg = segment(k);
            const int nt = sg.nt, b = sg.b, hk = sg.hk, tile0 = sg.tile0;
            if (!ok || nt == 0) break;
            const int last_key = sg.limit;
            // page ids come 32 at a time, one load per block of the table row and one
            // block ahead: a lookup per tile would put its latency between the copies
            const int32_t* table = p.table + (int64_t)b * p.s.width;
            const int pages = (last_key + page_mask) >> p.s.page_log2;
            auto ids = [&](int blk) {
                const int i = blk * 32 + lane;
                return i < pages ? __ldg(table + i) : -1;
            };
            int blk = (tile0 * KT >> p.s.page_log2) >> 5, cur = ids(blk), ahead = ids(blk + 1);
            for (int t = 0; t < nt; ++t) {
                const int kb = (tile0 + t) * KT, first = kb >> p.s.page_log2;
                if ((first >> 5) != blk) {
                    ++blk;
                    cur = ahead;
                    ahead = ids(blk + 1);
                }
                wait(&empty[st], round + 1);  // at once in the first round
                if (!ok) break;
                const int boxes = (min(KT, last_key - kb) + w.page_box - 1) / w.page_box;
                if (elect_one()) mbar_arrive_expect_tx(&full[st], (uint32_t)(boxes * w.page_box * 128 * NH));
                // a tile's pages (at most 16) lie in one block
                const uint32_t key = (uint32_t)kb + lane * w.page_box;  // of no meaning from lane `boxes` on
                const int page = __shfl_sync(0xffffffffu, cur, (key >> p.s.page_log2) & 31);
                unsigned char* dst = ring + st * A::UNIT + lane * w.page_box * 128;
                if (lane < boxes)
                    for (int h = 0; h < NH; ++h)
                        tma_4d(dst + h * KT * 128, map, h * 64, hk, (int)(key & page_mask), page, &full[st]);
                ++n;
                if (++st == stages) st = 0, ++round;
                if (t > 0 || !is_k) continue;
                for (int s = 0; s <= sg.dual; ++s) {
                    const uint32_t qb = qi % NS;
                    wait(&ms.q_empty[qb], qi / NS + 1);
                    if (!ok) break;
                    ++qi;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&ms.q_full[qb], (uint32_t)(w.q_box * w.g.G * 128 * NH));
                        for (int h = 0; h < NH; ++h)
                            tma_4d(q_smem + qb * q_bytes + h * w.q_rows * 128, &map_q, h * 64, hk * w.g.G,
                                   sg.t0 + s * w.g.tpt, b, &ms.q_full[qb]);
                    }
                }
            }
            release(k);
        }
        // drain: every tile and row tile of Q has been read by the MMAs, so no
        // copy or commit is still on its way when the CTA leaves
        const uint32_t n0 = n > stages ? n - stages : 0, q0 = qi > NS ? qi - NS : 0;
        for (uint32_t i = n0; ok && i < n; ++i) wait(&empty[i % stages], i / stages);
        for (uint32_t i = q0; ok && i < qi; ++i) wait(&ms.q_empty[i % NS], i / NS);
        if (!ok) {
            // a role gave up: at least every copy issued has landed
            if (lane == 0) ms.failed = 1;
            for (uint32_t i = n0; i < n; ++i) mbar_wait_n(&full[i % stages], (i / stages) & 1, limit);
            for (uint32_t i = q0; i < qi; ++i) mbar_wait_n(&ms.q_full[i % NS], (i / NS) & 1, limit);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer: one thread, whose every step (a poll, a commit)
        // keeps the tensor cores waiting: few commits, state in registers, and code
        // that fits the first instruction fetches.  Elected, not picked by its number:
        // the MMAs of a branch that the compiler knows to be one thread's issue in a
        // third of the cycles (17 against 52 each, measured).
        if (elect_one()) {
            const uint32_t id_o = umma_idesc(F16, true, ATT_ROWS, 0) | ((uint32_t)(p.s.D >> 3) << 17);
            const int dk = p.s.D / 16;  // k-steps of the scores
            uint32_t k_st = 0, k_round = 0, v_st = 0, v_round = 0, qi = 0;  // rings; row tiles of Q
            uint32_t cleaned = 0;             // bit per stage, phases of v_clean so far
            uint32_t n[2] = {0, 0};           // tiles of each stream so far
            uint32_t emptied = 0, used = 0;   // bit s: phases of o_empty; the stream has had a segment
            // Q and K are K-major with 8-row groups 1024 bytes apart; V is N-major,
            // 64-column boxes KT rows apart, 8-row groups 1024 bytes apart
            const uint64_t q_desc = umma_desc(smem_u32(q_smem), 16, 1024);
            const uint64_t k_desc = umma_desc(smem_u32(k_smem), 16, 1024);
            const uint64_t v_desc = umma_desc(smem_u32(v_smem), KT * 128, 1024);
            const uint32_t q_half = w.q_rows * 8;  // a box of Q, in 16 bytes
            for (uint32_t k = 0; ok; ++k) {
                const AttSeg& sg = ms.seg[k % ATT_SEGS];
                until(&ms.seg_full[k % ATT_SEGS], k / ATT_SEGS);
                if (!ok || sg.nt == 0) break;
                const int nt = sg.nt, masked = att_first_masked<KT>(sg);
                const bool dual = sg.dual != 0;
                mbar_arrive(&ms.seg_empty[k % ATT_SEGS]);
                // the scores of tile t, stream s's i-th from its next
                auto scores = [&](auto stream, int t, uint32_t i) {
                    constexpr int s = decltype(stream)::value;
                    if (t >= nt || !ok) return;
                    const uint32_t q = qi + (dual ? s : 0), qb = q % NS, buf = NS == 1 ? (n[s] + i) & 1 : 0;
                    if (!dual || s == 0) until(&ms.k_full[k_st], k_round);
                    if (t == 0) until(&ms.q_full[qb], q / NS);
                    if (!ok) return;
                    tmem_fence_after();
                    const uint64_t a = q_desc + qb * (q_bytes / 16), b = k_desc + k_st * (A::UNIT / 16);
                    const uint32_t d = tmem + A::s_col(s) + 64 * buf;
                    constexpr uint32_t ID = umma_idesc(F16, false, ATT_ROWS, KT);
                    auto mma = [&](int x) {
                        umma_ss(d, a + (x / 4) * q_half + (x % 4) * 2, b + ((x / 4) * KT * 128 + (x % 4) * 32) / 16, ID,
                                x > 0);
                    };
                    // at most 3 k-steps of the padded head are past the head's own
#pragma unroll
                    for (int x = 0; x < DP / 16 - 3; ++x) mma(x);
                    if (dk > DP / 16 - 3) mma(DP / 16 - 3);
                    if (dk > DP / 16 - 2) mma(DP / 16 - 2);
                    if (dk > DP / 16 - 1) mma(DP / 16 - 1);
                    umma_commit(&ms.s_full[s][buf]);  // the warpgroup releases the key stage
                    if (t == nt - 1) umma_commit(&ms.q_empty[qb]);
                    if ((!dual || s == 1) && ++k_st == KS) k_st = 0, ++k_round;
                };
                // scores of all buffers, then tile by tile the values and the scores that
                // take the place of what they read
                const std::integral_constant<int, 0> c0{};
                const std::integral_constant<int, NS - 1> c1{};
                scores(c0, 0, 0);
                if (NS == 1) scores(c0, 1, 1);
                else scores(c1, dual ? 0 : 1, 0);
                for (int t = 0; ok && t < nt; ++t) {
                    if (t >= masked) {
                        until(&ms.v_clean[v_st], cleaned >> v_st);
                        cleaned ^= 1u << v_st;
                    } else {
                        until(&ms.v_full[v_st], v_round);
                    }
                    const uint64_t b = v_desc + v_st * (A::UNIT / 16);
                    auto values = [&](auto stream) {
                        constexpr int s = decltype(stream)::value;
                        const bool first = t == (NS == 2 && !dual ? s : 0);
                        if (first) {
                            if ((used >> s) & 1u) {
                                until(&ms.o_empty[s], emptied >> s);
                                emptied ^= 1u << s;
                            }
                            used |= 1u << s;
                        }
                        const uint32_t buf = NS == 1 ? n[s] & 1 : 0, a = tmem + A::s_col(s) + 64 * buf;
                        // half by half: the first meets its values while the warpgroup is at
                        // the second
#pragma unroll
                        for (int h = 0; h < NS; ++h) {
                            until(&ms.p_ready[s][NS == 1 ? buf : h], NS == 1 ? n[s] >> 1 : n[s]);
                            if (!ok) return;
                            tmem_fence_after();
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                umma_ts(tmem + A::o_col(s), a + 64 * h + x * 8, b + (4 * h + x) * 128, id_o,
                                        !first || h + x > 0);
                        }
                        ++n[s];
                        if (!dual || s == 1) umma_commit(&ms.v_empty[v_st]);
                        if (t + (NS == 2 && !dual ? 2 : 1) >= nt) umma_commit(&ms.o_full[s]);
                        if (NS == 1) scores(c0, t + 2, 1);
                        else scores(stream, dual ? t + 1 : t + 2, 0);
                    };
                    if (NS == 1 || dual || !(t & 1)) values(c0);
                    if (NS == 2 && (dual || (t & 1))) values(c1);
                    if (++v_st == VS) v_st = 0, ++v_round;
                }
                qi += dual ? 2 : 1;
            }
            if (!ok) {
                ms.failed = 1;
                umma_commit(&ms.drain);  // no MMA is in flight when the CTA leaves
                mbar_wait_n(&ms.drain, 0, limit);
            }
        }
        __syncwarp();
    } else {
        // ---------------- softmax: warpgroup s, thread = row
        const int s = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t o_addr = tmem + A::o_col(s) + lanes;
        const float c = p.scale * 1.4426950408889634f;
        const int T = p.s.T, Hq = p.s.Hq, D = p.s.D, G = w.g.G;
        auto node_of = [&]() { return (int)((uint32_t)row * w.g_inv >> 16); };  // row / G
        // nodes that do not exist: zero rows
        {
            const int rows = p.s.B * T, ws = gridDim.x * NS * 4, per = (rows + ws - 1) / ws;
            const int r0 = min(rows, ((int)blockIdx.x * NS * 4 + warp - 4) * per), r1 = min(rows, r0 + per);
            for (int r = r0, b = r0 / T; r < r1; ++r) {
                if (r >= (b + 1) * T) ++b;
                if (r - b * T < tree_len(p.s, b).n) continue;
                uint4* o = (uint4*)((char*)p.out + (int64_t)r * Hq * D * 2);
                for (int i = lane; i < Hq * D / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
                if (p.lse)
                    for (int i = lane; i < Hq; i += 32) p.lse[(int64_t)r * Hq + i] = -INFINITY;
            }
        }
        uint32_t base = 0, cleaned = 0;              // tiles, phases of v_clean (bit per stage)
        uint32_t n_unit = 0;                         // own tiles
        uint32_t n_o = 0, n_join = 0;                // segments of the stream, joins
        for (uint32_t k = 0; ok; ++k) {
            const AttSeg& sg = segment(k);
            const int nt = sg.nt;
            if (!ok || nt == 0) break;
            const bool dual = sg.dual != 0;
            const int t_first = sg.t0 + (dual ? s * w.g.tpt : 0);
            const int rows = min(w.g.tpt, sg.t0 + sg.ntok - t_first) * G;
            const bool active = (warp & 3) * 32 < rows;
            float m = -INFINITY, l = 0.f;
            int masked = att_first_masked<KT>(sg);  // later: the first masked tile not counted in `cleaned`

            const int t_begin = dual ? 0 : s, stride = dual ? 1 : NS;  // all tiles, or alternate ones
            for (int tile = t_begin; tile < nt && ok; tile += stride, ++n_unit) {
                const bool part = tile >= masked;  // some row sees the tile only in part
                const int kb = (sg.tile0 + tile) * KT;
                const uint32_t buf = NS == 1 ? n_unit & 1 : 0, phase = NS == 1 ? n_unit >> 1 : n_unit;
                const uint32_t s_addr = tmem + A::s_col(s) + lanes + 64 * buf;
                uint32_t see[KT / 32], some = 0;
                if (part) {
                    // on their way while the scores are computed
                    const int t = min(t_first + node_of(), sg.n - 1);  // rows past the last are never stored
#pragma unroll
                    for (int y = 0; y < KT / 32; ++y) see[y] = att_sees(p, sg.b, t, sg.ctx, sg.n, kb + 32 * y);
                }
                wait(&ms.s_full[s][buf], phase);
                if (!ok) break;
                tmem_fence_after();
                // the scores are there, so their keys have been read
                if (warp == 4 + 4 * s && lane == 0)
                    mbar_arrive_n(&ms.k_empty[base + tile - k_round_of(base + tile) * KS], NS == 2 && !dual ? 2 : 1);
                const uint32_t vi = base + tile, v_round = v_round_of(vi), vst = v_stage_of(vi);
                if (part) {
                    // phases of v_clean of the tiles before this one (the other stream's)
                    for (; masked < tile; ++masked) cleaned ^= 1u << v_stage_of(base + masked);
                    ++masked;
                    wait(&ms.v_full[vst], v_round);
                    if (!ok) break;
                    att_clean<F16, DP>(ms, v_smem + vst * A::UNIT, vst, kb, sg.mask_from, sg.ctx + sg.n, dual, s,
                                       warp & 3, lane);
                    wait(&ms.v_clean[vst], cleaned >> vst);
                    if (!ok) break;
                    cleaned ^= 1u << vst;
                    // hidden scores become -inf in tensor memory
                    if (active) {
#pragma unroll 1
                        for (int y = 0; y < KT / 32; ++y) {
                            const uint32_t sees = y == 0 ? see[0] : y == 1 ? see[1] : y == 2 ? see[KT / 32 - 2]
                                                                                          : see[KT / 32 - 1];
                            if (__all_sync(0xffffffffu, sees == ~0u)) continue;
                            uint32_t x[32];
                            tmem_ld<32>(s_addr + 32 * y, x);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((sees >> i) & 1u)) x[i] = 0xFF800000u;
                            tmem_st<32>(s_addr + 32 * y, x);
                        }
                        tmem_wait_st();
                    }
                    // seen keys with non-finite values (before the tile is handed over: its
                    // stage may be filled anew after that)
#pragma unroll
                    for (int y = 0; y < KT / 32; ++y) some |= see[y] &= *(volatile uint32_t*)&ms.nf[vst][y];
                }
                if (active) {
                    // the row's maximum, found by the loads
                    uint32_t x[64];
                    float top = tmem_ld_max<64>(s_addr + KT - 64, x);
                    if (NS == 2) top = fmaxf(top, tmem_ld_max<64>(s_addr, x));
                    // O and l stay in units of the old maximum while the new one is
                    // less than 2^8 above it: p then stays below 2^8
                    const bool grow = top * c > m * c + ATT_LAZY || (m == -INFINITY && top > m);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = grow ? ex2_fast((m - top) * c) : 1.f;
                        if (grow) m = top;
                        l *= f;
                        if (tile > t_begin) {
                            // every P V before has to be complete.  With two streams it is:
                            // these scores were issued after the stream's last.
                            if (NS == 1) wait(&ms.v_empty[v_stage_of(vi - 1)], v_round_of(vi - 1));
                            if (!ok) break;
                            tmem_fence_after();
#pragma unroll 1
                            for (int d = 0; d < D; d += 16) {
                                uint32_t o[16];
                                tmem_ld<16>(o_addr + d, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st<16>(o_addr + d, o);
                            }
                        }
                    }
                    const float mc = m == -INFINITY ? 0.f : m * c;
                    const uint64_t c2 = pack2(c, c), mc2 = pack2(att_up(F16) - mc, att_up(F16) - mc);
                    uint64_t sum[2] = {0ull, 0ull};  // two pairs of partial sums
#pragma unroll 1
                    for (int h = 0; h < NS; ++h) {
                        if (h > 0) tmem_ld<64>(s_addr + 64 * h, x);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            float2 e = unpack2(fma2(pack2u(x[2 * i], x[2 * i + 1]), c2, mc2));
                            e.x = ex2_fast(e.x);
                            e.y = ex2_fast(e.y);
                            sum[i & 1] = add2(sum[i & 1], pack2(e.x, e.y));
                            x[i] = H::pack(e.x, e.y);
                        }
                        tmem_st<32>(s_addr + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(&x));
                        tmem_wait_st();
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0 && (NS == 1 || h == 0)) mbar_arrive(&ms.p_ready[s][NS == 1 ? buf : 0]);
                    }
                    const float2 sums = unpack2(add2(sum[0], sum[1]));
                    l += sums.x + sums.y;
                } else if (lane == 0) {
                    mbar_arrive(&ms.p_ready[s][buf]);
                }
                if (NS == 2 && lane == 0) mbar_arrive(&ms.p_ready[s][1]);
                if (part && __any_sync(0xffffffffu, active && some)) {
                    // rare: once P V is done (it saw zeros there), O += those values
                    wait(&ms.v_empty[vst], v_round);
                    if (!ok) break;
                    tmem_fence_after();
                    att_add_nonfinite<F16>(p, see[0], see[1], sg.b, sg.hk, kb, o_addr);
                    if (NS == 2)
                        att_add_nonfinite<F16>(p, see[KT / 32 - 2], see[KT / 32 - 1], sg.b, sg.hk, kb + 64, o_addr);
                }
            }
            for (; masked < nt; ++masked) cleaned ^= 1u << v_stage_of(base + masked);
            base += nt;
            if (!ok) break;

            // ---- the segment's end: O of the streams that had tiles
            const bool two = dual || nt > 1;            // stream 1 had some
            const bool join = NS == 2 && !dual && two;  // one row tile in two streams
            if (s == 0 || two) {
                wait(&ms.o_full[s], n_o++);
                if (!ok) break;
                tmem_fence_after();
                float m1 = -INFINITY, l1 = 0.f;
                int d0 = 0, d1 = D;
                if (join) {
                    // the streams' maxima and sums meet, and each gives out half of the
                    // columns.  ml is free again: its readers' o_empty came before this o_full
                    ms.ml[s][row] = make_float2(m, l);
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.j_full[warp & 3]);
                    wait(&ms.j_full[warp & 3], n_join++);
                    if (!ok) break;
                    tmem_fence_after();
                    m = ms.ml[0][row].x;
                    l = ms.ml[0][row].y;
                    m1 = ms.ml[1][row].x;
                    l1 = ms.ml[1][row].y;
                    const int half = (D / 16 + 1) / 2 * 16;
                    (s ? d0 : d1) = half;
                }
                if (active) {
                    const float mm = fmaxf(m, m1), mr = mm == -INFINITY ? 0.f : mm;
                    float f0 = m == -INFINITY ? 0.f : ex2_fast((m - mr) * c);
                    float f1 = m1 == -INFINITY ? 0.f : ex2_fast((m1 - mr) * c);
                    // a NaN sum stays NaN, and so does that of an infinite maximum
                    const float ll = l * f0 + (join ? l1 * f1 : 0.f);
                    const bool none = ll == 0.f, whole = sg.whole != 0, mine = row < rows;
                    if (whole) {
                        const float inv = none ? 0.f : 1.f / ll;
                        f0 *= inv;
                        f1 *= inv;
                    }
                    const int64_t orow = ((int64_t)sg.b * T + t_first + node_of()) * Hq + sg.hk * G + row - node_of() * G;
                    const int64_t slot = (int64_t)blockIdx.x * 2 + (sg.tile0 > 0 ? 0 : 1);
                    const int prow = (dual ? s * ATT_ROWS : 0) + row;
#pragma unroll 1
                    for (int d = d0; d < d1; d += 16) {
                        uint32_t o[16];
                        if (join) {
                            uint32_t o1[16];
                            tmem_ld_2x16(tmem + A::o_col(0) + lanes + d, tmem + A::o_col(NS - 1) + lanes + d, o, o1);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * f0 + __uint_as_float(o1[i]) * f1);
                        } else {
                            tmem_ld<16>(o_addr + d, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0);
                        }
                        auto y = [&](int i) { return __uint_as_float(o[i]); };
                        if (!mine) continue;
                        if (whole) {
                            uint4* o16 = (uint4*)((char*)p.out + (orow * D + d) * 2);
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                o16[i] = none ? make_uint4(0, 0, 0, 0)
                                              : make_uint4(H::pack(y(8 * i), y(8 * i + 1)),
                                                           H::pack(y(8 * i + 2), y(8 * i + 3)),
                                                           H::pack(y(8 * i + 4), y(8 * i + 5)),
                                                           H::pack(y(8 * i + 6), y(8 * i + 7)));
                        } else {
                            float4* o32 = (float4*)w.part_o + (slot * (DP / 4) + d / 4) * (NS * ATT_ROWS) + prow;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                o32[i * NS * ATT_ROWS] =
                                    make_float4(y(4 * i), y(4 * i + 1), y(4 * i + 2), y(4 * i + 3));
                        }
                    }
                    const bool first = s == 0 || dual;
                    if (first && mine && whole && p.lse) p.lse[orow] = none ? -INFINITY : att_lse<F16>(mr, p.scale, ll);
                    if (first && mine && !whole) w.part_ml[slot * NS * ATT_ROWS + prow] = make_float2(mm, ll);
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_n(&ms.o_empty[s], NS == 2 && !join ? 2 : 1);
                    if (join) mbar_arrive(&ms.o_empty[1 - s]);
                }
            }
            release(k);
        }
        if (!ok && lane == 0) ms.failed = 1;
    }
    tmem_fence_before();
    __syncthreads();
    if (tid == 0 && ms.failed) atomicOr(w.err, 1u);
    tmem_fence_after();
    if (warp == 2) tmem_free(tmem, ATT_TMEM_COLS);
}

// ------------------------------------------------------------------------- //
// k_tree_combine                                                            //
// ------------------------------------------------------------------------- //
// Joins the parts of an item cut between CTAs: out = sum_i 2^(m_i - m) O_i /
// sum_i 2^(m_i - m) l_i (m here in log2 units).  Lane = row.  Where the parts
// are few a warp takes 32 rows by 32 columns, all loads of a thread
// independent; where they are many (few items, long caches) a CTA takes 32
// rows by 8 columns, every eighth part a warp's, and the warps' sums meet in
// shared memory.  The tasks are those that k_tree_attend announced: only the
// GPU knows which ranges cut items.  Parts are summed in their order, whatever
// the order of the tasks.
constexpr int COMB_THREADS = 256, COMB_CTAS_PER_SM = 2;

template <bool F16>
__global__ void __launch_bounds__(COMB_THREADS, COMB_CTAS_PER_SM)
    k_tree_combine(const AttWork w, int DP, int prows)
{
    using H = Half2<F16>;
    __shared__ float4 acc_s[8][2][32];
    __shared__ float2 ml_s[8][32];
    const TreeAttendParams& p = w.p;
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int D = p.s.D, G = w.g.G, first_rows = w.g.tpt * G;
    const float c = p.scale * 1.4426950408889634f;
    auto weight = [&](float m, float ref) { return m == -INFINITY ? 0.f : ex2_fast((m - ref) * c); };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    AttJoin next = w.joins[blockIdx.x];  // of no meaning past the tasks' number
    const int tasks = (int)__ldcg(w.n_joins);
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
        const AttJoin jn = next;
        if (task + (int)gridDim.x < tasks) next = w.joins[task + gridDim.x];
        const int n = jn.last - jn.first + 1;
        auto slot = [&](int i) { return (int64_t)(jn.first + i) * 2 + (i == 0 ? 1 : 0); };
        // rows of the second row tile lie behind the first's 128
        auto part_row = [&](int r) { return r < first_rows ? r : ATT_ROWS + r - first_rows; };
        auto out_row = [&](int r) {
            const int node = r / G;
            return ((int64_t)jn.b * p.s.T + jn.t0 + node) * p.s.Hq + jn.hk * G + r - node * G;
        };
        if (n <= w.few) {
            const int c32 = (D + 31) / 32, sub = jn.sub * 8 + g, rb = sub / c32, col4 = (sub - rb * c32) * 8;
            const int r = rb * 32 + lane, pr = part_row(r);
            if (r >= jn.rows) continue;
            // the parts' maxima, sums and columns are loaded together; the running
            // maximum keeps the sums in its units
            float ref = -INFINITY, l = 0.f;
            float4 acc[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int i = 0; i < n; ++i) {
                const float2 v = w.part_ml[slot(i) * prows + pr];
                const float4* src = (const float4*)w.part_o + (slot(i) * (DP / 4) + col4) * prows + pr;
                float4 o[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if ((col4 + k) * 4 < D) o[k] = src[k * prows];
                const float top = fmaxf(ref, v.x), m = top == -INFINITY ? 0.f : top;
                const float f = weight(ref, m), e = weight(v.x, m);
                ref = top;
                l = l * f + v.y * e;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if ((col4 + k) * 4 < D) {
                        acc[k].x = acc[k].x * f + o[k].x * e;
                        acc[k].y = acc[k].y * f + o[k].y * e;
                        acc[k].z = acc[k].z * f + o[k].z * e;
                        acc[k].w = acc[k].w * f + o[k].w * e;
                    }
            }
            if (ref == -INFINITY) ref = 0.f;
            const bool none = l == 0.f;
            const float inv = none ? 0.f : 1.f / l;
            const int64_t orow = out_row(r);
            uint4* o16 = (uint4*)((char*)p.out + (orow * D + col4 * 4) * 2);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 a = acc[2 * k], b = acc[2 * k + 1];
                if ((col4 + 2 * k) * 4 < D)
                    o16[k] = none ? make_uint4(0, 0, 0, 0)
                                  : make_uint4(H::pack(a.x * inv, a.y * inv), H::pack(a.z * inv, a.w * inv),
                                               H::pack(b.x * inv, b.y * inv), H::pack(b.z * inv, b.w * inv));
            }
            if (p.lse && col4 == 0) p.lse[orow] = none ? -INFINITY : att_lse<F16>(ref, p.scale, l);
            continue;
        }
        const int c8 = D / 8, rb = jn.sub / c8, col4 = (jn.sub - rb * c8) * 2;
        const int r = min(rb * 32 + lane, jn.rows - 1), pr = part_row(r);
        float top = -INFINITY, l = 0.f;
#pragma unroll 4
        for (int i = g; i < n; i += 8) top = fmaxf(top, w.part_ml[slot(i) * prows + pr].x);
        const float own = top == -INFINITY ? 0.f : top;
        float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 4
        for (int i = g; i < n; i += 8) {
            const float2 v = w.part_ml[slot(i) * prows + pr];
            const float f = weight(v.x, own);
            l += v.y * f;
            const float4* src = (const float4*)w.part_o + (slot(i) * (DP / 4) + col4) * prows + pr;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 o = src[k * prows];
                acc[k].x += f * o.x, acc[k].y += f * o.y, acc[k].z += f * o.z, acc[k].w += f * o.w;
            }
        }
        __syncthreads();  // the tables of the task before have been read
        ml_s[g][lane] = make_float2(top, l);
        acc_s[g][0][lane] = acc[0];
        acc_s[g][1][lane] = acc[1];
        __syncthreads();
        if (g < 2) {  // warp g joins its four columns
            top = -INFINITY;
            l = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fmaxf(top, ml_s[k][lane].x);
            const float ref = top == -INFINITY ? 0.f : top;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 v = ml_s[k][lane];
                const float f = weight(v.x, ref);
                const float4 o = acc_s[k][g][lane];
                l += v.y * f;
                y.x += f * o.x, y.y += f * o.y, y.z += f * o.z, y.w += f * o.w;
            }
            const bool none = l == 0.f;
            const float inv = none ? 0.f : 1.f / l;
            if (rb * 32 + lane < jn.rows) {
                const int64_t orow = out_row(r);
                *(uint2*)((char*)p.out + (orow * D + (col4 + g) * 4) * 2) =
                    none ? make_uint2(0, 0)
                         : make_uint2(H::pack(y.x * inv, y.y * inv), H::pack(y.z * inv, y.w * inv));
                if (p.lse && col4 == 0 && g == 0)
                    p.lse[orow] = none ? -INFINITY : att_lse<F16>(ref, p.scale, l);
            }
        }
    }
    // the last CTA to finish leaves the list empty
    if (threadIdx.x == 0 && atomicInc(w.n_done, gridDim.x - 1) == gridDim.x - 1) *w.n_joins = 0;
}

// ------------------------------------------------------------------------- //
// host side                                                                 //
// ------------------------------------------------------------------------- //
static int att_dp(int D) { return (D + 63) / 64 * 64; }
static int att_part_rows(int DP) { return (DP <= 128 ? 2 : 1) * ATT_ROWS; }

// workspace: partial O, (m, l) and joins of `ctas` CTAs, and the joins' two counters
size_t tree_attend_bytes(int D, int ctas, size_t* ml_at, size_t* join_at)
{
    const int DP = att_dp(D);
    const size_t slots = 2 * (size_t)ctas, o = slots * att_part_rows(DP) * DP * sizeof(float);
    const size_t ml = slots * att_part_rows(DP) * sizeof(float2);
    *ml_at = o;
    *join_at = o + ml;
    const int most = att_join_tasks(1, att_part_rows(DP), DP, 0);  // of a cut
    return o + ml + 16 + (size_t)ctas * most * sizeof(AttJoin);
}

// a tensor [d3, d2, d1, D] of 16-bit elements as a 4-D map with boxes of 64
// columns, box1 x box2 rows; false when the driver refuses it
static bool att_map(CUtensorMap* map, bool f16, const void* ptr, int D, const int64_t (&dims)[3],
                    const int64_t (&strides)[3], int box1, int box2)
{
    EncodeTiledFn enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t d[4] = {(cuuint64_t)D, (cuuint64_t)dims[0], (cuuint64_t)dims[1], (cuuint64_t)dims[2]};
    cuuint64_t st[3];
    // the stride of a dimension of size 1 is never used, but may not be 0
    for (int i = 0; i < 3; ++i) st[i] = dims[i] == 1 ? 16 * (cuuint64_t)((D + 7) / 8) : (cuuint64_t)strides[i] * 2;
    // L2 fetches 256 bytes at a time where a head's row is a multiple of that (256
    // sequences of one token, D = 128: 343 us, by 64 bytes 354), else by 64: the rest
    // of a wider fetch is other heads' (22 x 2 tokens over 7000 keys, 4 key heads, L2
    // flushed: D = 64 62 -> 52 us, 80 81 -> 67, 96 85 -> 73, 112 99 -> 86, 192 118 -> 110)
    const auto promotion = D % 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    const cuuint32_t box[4] = {64, (cuuint32_t)box1, (cuuint32_t)box2, 1}, one[4] = {1, 1, 1, 1};
    return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void*>(ptr), d, st, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool F16, int DP>
static cudaError_t att_launch(AttWork w, int num_sms, cudaStream_t s)
{
    using A = Att<DP>;
    static DeviceOnce once;  // per device: the shared-memory opt-in
    cudaError_t e = cuda_once(once, nullptr, [](int, int*) {
        return cudaFuncSetAttribute(k_tree_attend<F16, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, ATT_SMEM);
    });
    if (e != cudaSuccess) return e;
    const TreeShape& sh = w.p.s;
    w.g.group = A::NS * w.g.tpt;
    w.page_box = min(1 << sh.page_log2, A::KT);
    w.q_box = min(w.g.tpt, sh.T);
    // what Q does not need is for the rings: few rows leave room for more tiles on their way
    w.q_rows = (w.q_box * w.g.G + 7) / 8 * 8;
    const int stages = (A::ROOM - A::NS * w.q_rows * DP * 2) / A::UNIT;
    w.k_stages = min((stages + 1) / 2, ATT_STAGES);
    w.v_stages = min(stages / 2, ATT_STAGES);
    w.k_inv = 0xFFFFFFFFu / w.k_stages + 1;
    w.v_inv = 0xFFFFFFFFu / w.v_stages + 1;
    w.g_inv = 0xFFFFu / w.g.G + 1;
    CUtensorMap mq, mk, mv;
    const int64_t qd[3] = {sh.Hq, sh.T, sh.B}, qs[3] = {w.p.q.head, w.p.q.token, w.p.q.seq};
    const int64_t cd[3] = {sh.Hkv, 1 << sh.page_log2, sh.num_pages}, cs[3] = {w.p.c.head, w.p.c.token, w.p.c.page};
    if (!att_map(&mq, F16, w.p.q.ptr, sh.D, qd, qs, w.g.G, w.q_box) ||
        !att_map(&mk, F16, w.p.c.k, sh.D, cd, cs, 1, w.page_box) ||
        !att_map(&mv, F16, w.p.c.v, sh.D, cd, cs, 1, w.page_box))
        return cudaErrorInvalidValue;
    // an item's parts may lie in all ranges; the second form has the more tasks
    const int64_t items = (int64_t)sh.B * sh.Hkv * ((sh.T + w.g.group - 1) / w.g.group);
    const int64_t tasks = items * att_join_tasks(1, w.q_rows * A::NS, sh.D, 0), ctas = num_sms * COMB_CTAS_PER_SM;
    w.few = tasks <= ctas ? 0 : ATT_FEW;
    k_tree_attend<F16, DP><<<num_sms, A::THREADS, ATT_SMEM, s>>>(mq, mk, mv, w);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)std::min(tasks, ctas));  // no more CTAs than there can be tasks
    cfg.blockDim = dim3(COMB_THREADS);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_tree_combine<F16>, w, DP, A::NS * ATT_ROWS);
    if (e != cudaSuccess) cudaMemsetAsync(w.n_joins, 0, sizeof(unsigned), s);  // nobody empties the list
    return e;
}

bool tree_attend_fits(const TreeShape& sh)
{
    const int64_t group = (sh.D <= 128 ? 2 : 1) * (ATT_ROWS / (sh.Hq / sh.Hkv));
    const int64_t groups = (sh.T + group - 1) / group;
    const int64_t tiles = (((int64_t)sh.width << sh.page_log2) + 63) / 64 + ATT_ITEM_COST;
    return (double)sh.B * sh.Hkv * groups * tiles < 2147483648.0;
}

cudaError_t launch_tree_attend(const TreeAttendParams& p, int dtype, int num_sms, void* ws, unsigned* err, bool stall,
                               cudaStream_t s)
{
    size_t ml_at, join_at;
    tree_attend_bytes(p.s.D, num_sms, &ml_at, &join_at);
    AttWork w = {};
    w.p = p;
    w.g.G = p.s.Hq / p.s.Hkv;
    w.g.tpt = ATT_ROWS / w.g.G;
    w.g.Hkv = p.s.Hkv;
    w.part_o = (float*)ws;
    w.part_ml = (float2*)((char*)ws + ml_at);
    w.n_joins = (unsigned*)((char*)ws + join_at);
    w.n_done = w.n_joins + 1;
    w.joins = (AttJoin*)((char*)ws + join_at + 16);
    w.err = err;
    w.stall = stall;
    const bool f16 = dtype == SPEC_F16;
    switch (att_dp(p.s.D)) {
    case 64: return f16 ? att_launch<true, 64>(w, num_sms, s) : att_launch<false, 64>(w, num_sms, s);
    case 128: return f16 ? att_launch<true, 128>(w, num_sms, s) : att_launch<false, 128>(w, num_sms, s);
    case 192: return f16 ? att_launch<true, 192>(w, num_sms, s) : att_launch<false, 192>(w, num_sms, s);
    default: return f16 ? att_launch<true, 256>(w, num_sms, s) : att_launch<false, 256>(w, num_sms, s);
    }
}

}  // namespace sv
