// sv_tree_attend.cu -- attention of drafted tokens, a tree or a chain, over the
// paged cache (spec_tree_attend).
//
// For a key head the query rows of one sequence are its nodes times the G
// query heads that share the head: out[r] = sum_k p[r][k] V[k] / sum_k p[r][k],
// p = exp(scale q[r] . K[k]) over the keys row r sees.  One pass over the keys
// with the running maximum m and sum l of each row: a tile of KT keys gives
// S = Q K^T (tensor cores, fp32), p = 2^(c S - c m) with c = scale log2(e),
// l += sum p and O += P V (tensor cores, P rounded to the 16-bit type, O fp32
// in tensor memory); when m grows by more than 2^8 would allow, O and l are
// scaled down first.
//
// The bound is HBM for up to about 256 rows per key head (each key's 4 D bytes
// are read once per 256 rows and cost 4 D products per row), the tensor cores
// beyond.  So:
//  * Rows are tiles of 128: floor(128 / G) nodes times G heads, the M of the
//    MMA, whatever their number: the tensor pipe has time for 128 rows while
//    the keys stream, so few rows need no other form.
//  * Work items are (key head, sequence, group of row tiles).  All items' key
//    tiles in a row are cut into equal ranges, one per SM, whatever the batch:
//    a long cache with few rows fills the machine, a ragged batch is balanced,
//    and the lengths are read on the GPU.  An item cut by a range's end leaves
//    partial sums (O, m, l) that k_tree_combine joins.  The key head comes
//    first, so that the SMs of all heads go through the same pages together.
//  * A CTA has two producer warps (tensor-map copies of whole pages into rings
//    of 128-byte-swizzled key and value tiles), an MMA warp and one or two
//    softmax warpgroups, a thread per row.  With heads up
//    to 128 elements two streams of (S, O) share tensor memory's 512 columns:
//    an item of one row tile gives its even key tiles to one and its odd ones
//    to the other (own m, l, O; joined at the end), an item of two row tiles
//    gives each stream a row tile and reads the keys once for both; either way
//    one stream's exponentials hide behind the other's MMAs.  Larger heads
//    fill tensor memory with one stream of 64-key tiles.
//
// What a row does not see must not touch it, whatever it holds: scores are
// replaced by -inf before the maximum, but P V multiplies hidden values by a
// zero probability, and 0 x NaN is NaN.  In the tiles that some row sees only
// in part the softmax warps zero the rows beyond the sequence and every
// non-finite value in shared memory; rows that see a node with such values
// (rare) add them afterwards.
#include <math.h>

#include "sv_tcgen.cuh"
#include "sv_tree.cuh"

namespace sv {

constexpr int ATT_ROWS = 128;                 // rows of a row tile: M of the MMA
constexpr int ATT_SMEM = 227 * 1024;          // shared memory of a CTA
constexpr int ATT_MISC = 2048;                // of it: barriers and small tables
constexpr uint32_t ATT_TMEM_COLS = 512;
constexpr uint32_t ATT_WAIT_POLLS = 1u << 17;  // limit of a wait: some seconds (a poll sleeps for microseconds)
constexpr uint32_t ATT_STALL_POLLS = 4096;    // SPEC_FAULT_STALL_STREAM
constexpr float ATT_LAZY = 8.f;               // log2 growth of the maximum that O takes unscaled

template <int DP>
struct Att {                                  // DP: head size rounded up to 64
    static constexpr int NH = DP / 64;        // 64-column (128-byte) boxes of a row
    static constexpr int NS = DP <= 128 ? 2 : 1;     // streams (softmax warpgroups)
    static constexpr int KT = DP <= 128 ? 128 : 64;  // keys per tile
    static constexpr int UNIT = KT * DP * 2;         // bytes of a K or V tile
    static constexpr int QB = ATT_ROWS * DP * 2;     // bytes of a row tile of Q
    static constexpr int STAGES = (ATT_SMEM - 1024 - ATT_MISC - NS * QB) / UNIT;
    static constexpr int KS = (STAGES + 1) / 2, VS = STAGES / 2;  // of them for keys, for values
    static constexpr int SMEM = 1024 + NS * QB + STAGES * UNIT + ATT_MISC;
    static constexpr int THREADS = 128 + 128 * NS;
    __host__ __device__ static constexpr uint32_t s_col(int s) { return 128u * s; }
    __host__ __device__ static constexpr uint32_t o_col(int s) { return NS == 2 ? 256u + 128u * s : 128u; }
    static_assert(STAGES >= 4 && SMEM <= ATT_SMEM, "the ring fits");
};

struct __align__(16) AttMisc {
    uint64_t k_full[8], k_empty[8];  // key tiles: copied; read by the MMAs
    uint64_t v_full[8], v_empty[8];  // value tiles
    uint64_t v_clean[8];             // a masked value tile may meet the MMAs
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2];            // scores of the stream's unit are in tensor memory
    uint64_t p_ready[2];           // its probabilities are (and O is scaled)
    uint64_t o_full[2], o_empty[2];  // the segment's O is complete; has been read
    uint64_t ml_full, ml_empty;    // stream 1's (m, l) for the join
    uint64_t drain;
    uint32_t nf[8][4];             // (masked) value rows of the tile with non-finite elements
    float2 ml[ATT_ROWS];
    int32_t scan[16];
    int32_t first, first_b;        // the range's first sequence, and its cost before the range
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
// ATT_ITEM_COST more (its first scores, its masked tile and its output).
constexpr int ATT_ITEM_COST = 1;

// keys that some row of item `rp` of a sequence sees: a chain's rows see
// nothing past their last node
__device__ __forceinline__ int att_limit(const TreeAttendParams& p, const AttGeom& g, int ctx, int n, int rp)
{
    return ctx + (p.mask ? n : min(n, (rp + 1) * g.group));
}
template <int KT>
__device__ __forceinline__ int att_cost(const TreeAttendParams& p, const AttGeom& g, int ctx, int n, int rp)
{
    return (att_limit(p, g, ctx, n, rp) + KT - 1) / KT + ATT_ITEM_COST;
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
    int limit;                  // keys any of its rows may see
    int mask_from;              // keys below are seen by all its rows
    bool dual;                  // two row tiles

    __device__ __forceinline__ bool more() const { return pos < end; }
    __device__ __forceinline__ void load_item(const TreeAttendParams& p, const AttGeom& g)
    {
        t0 = rp * g.group;
        ntok = min(g.group, n - t0);
        dual = ntok > g.tpt;
        limit = att_limit(p, g, ctx, n, rp);
        ntiles = (limit + KT - 1) / KT;
        mask_from = p.mask ? ctx : ctx + t0 + 1;
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
    __device__ __forceinline__ int tiles() const { return tile1 - tile0; }
    // the segment's first tile that some row sees only in part
    __device__ __forceinline__ int first_masked() const { return max(0, mask_from / KT - tile0); }
    __device__ __forceinline__ bool whole() const { return tile0 == 0 && tile1 == ntiles; }
};

// an item's tiles cut by the start of CTA c's range; c is the first such cut
struct __align__(16) AttCut {
    int32_t first, last;  // CTAs with parts of it; first < 0: nothing to join here
    int32_t b, hk, t0, rows;
};

struct AttWork {
    TreeAttendParams p;
    AttGeom g;
    float* part_o;      // [2 * CTAs][DP / 4][NS * 128] float4: O of a part, per 4 columns all rows
    float2* part_ml;    // [2 * CTAs][NS * 128]: (m, l) of a part's rows
    AttCut* cuts;       // [CTAs]
    unsigned* err;
    int32_t page_box;   // tokens of one copied box: min(page, KT)
    int32_t q_box;      // nodes of one copied box of Q
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

// zeroes the non-finite ones of a word's two values; true when there was one
template <bool F16>
__device__ __forceinline__ bool clean_word(uint32_t& v)
{
    const bool lo = att_nonfinite<F16>((uint16_t)v), hi = att_nonfinite<F16>((uint16_t)(v >> 16));
    if (lo) v &= 0xFFFF0000u;
    if (hi) v &= 0x0000FFFFu;
    return lo || hi;
}

template <bool F16, int DP>
__global__ void __launch_bounds__(Att<DP>::THREADS, 1)
    k_tree_attend(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const AttWork w)
{
    using A = Att<DP>;
    using H = Half2<F16>;
    constexpr int KT = A::KT, NS = A::NS, NH = A::NH, KS = A::KS, VS = A::VS;
    extern __shared__ unsigned char att_raw[];
    const uint32_t raw = smem_u32(att_raw);
    unsigned char* const q_smem = att_raw + (((raw + 1023u) & ~1023u) - raw);
    unsigned char* const k_smem = q_smem + NS * A::QB;
    unsigned char* const v_smem = k_smem + KS * A::UNIT;
    AttMisc& ms = *reinterpret_cast<AttMisc*>(v_smem + VS * A::UNIT);
    const TreeAttendParams& p = w.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t limit = w.stall ? ATT_STALL_POLLS : ATT_WAIT_POLLS;
    const volatile int32_t* failed = &ms.failed;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 64) {
        tma_prefetch_map(&map_k);
        tma_prefetch_map(&map_q);
        tma_prefetch_map(&map_v);
    }
    if (warp == 0) tmem_alloc(&ms.tmem, ATT_TMEM_COLS);
    if (tid == 32) {
        for (int i = 0; i < KS; ++i) {
            mbar_init(&ms.k_full[i], 1);
            mbar_init(&ms.k_empty[i], 1);
        }
        for (int i = 0; i < VS; ++i) {
            mbar_init(&ms.v_full[i], 1);
            mbar_init(&ms.v_empty[i], 1);
            mbar_init(&ms.v_clean[i], 4 * NS);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.q_full[i], 1);
            mbar_init(&ms.q_empty[i], 1);
            mbar_init(&ms.s_full[i], 1);
            mbar_init(&ms.p_ready[i], 4);
            mbar_init(&ms.o_full[i], 1);
            mbar_init(&ms.o_empty[i], 4);
        }
        mbar_init(&ms.ml_full, 4);
        mbar_init(&ms.ml_empty, 4);
        mbar_init(&ms.drain, 1);
        ms.failed = 0;
        fence_barrier_init();
    }
    // ---- this CTA's range: a scan of the sequences' costs
    int total = 0, per_head = 0, head0 = 0;
    {
        const int per = (p.s.B + A::THREADS - 1) / A::THREADS;
        const int s0 = min(p.s.B, tid * per), s1 = min(p.s.B, s0 + per);
        int sum = 0;
        for (int b = s0; b < s1; ++b) {
            const SeqLen l = tree_len(p.s, b);
            sum += att_head_cost<KT>(p, w.g, l.ctx, l.n);
        }
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) ms.scan[warp] = inc;
        __syncthreads();
        int before = inc - sum;
#pragma unroll
        for (int i = 0; i < A::THREADS / 32; ++i) {
            const int v = ms.scan[i];
            if (i < warp) before += v;
            total += v;
        }
        per_head = total;
        total *= w.g.Hkv;
        const int pos0 = AttSplit(total, gridDim.x).start(blockIdx.x);
        head0 = per_head ? pos0 / per_head : 0;
        const int in_head = pos0 - head0 * per_head;
        if (sum > 0 && in_head >= before && in_head < before + sum) {
            int b = s0, off = in_head - before;
            for (;; ++b) {
                const SeqLen l = tree_len(p.s, b);
                const int t = att_head_cost<KT>(p, w.g, l.ctx, l.n);
                if (off < t) break;
                off -= t;
            }
            ms.first_b = b;
            ms.first = off;
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = ms.tmem;
    const AttSplit split(total, gridDim.x);
    const bool busy = (int)blockIdx.x < split.ctas;
    AttIter<KT> it;
    it.start(p, w.g, busy ? split.start(blockIdx.x) : 0, busy ? split.start(blockIdx.x + 1) : 0, head0,
             ms.first_b, ms.first);
    bool ok = true;

    if (warp == 0 || warp == 2) {
        // ---------------- producers: warp 0 keys and the rows of Q, warp 2 values
        const bool is_k = warp == 0;
        const CUtensorMap* map = is_k ? &map_k : &map_v;
        unsigned char* const ring = is_k ? k_smem : v_smem;
        uint64_t *const full = is_k ? ms.k_full : ms.v_full, *const empty = is_k ? ms.k_empty : ms.v_empty;
        const uint32_t stages = is_k ? KS : VS;
        uint32_t n = 0, st = 0, round = 0, qi = 0;  // tiles so far, the next one's stage; row tiles of Q
        // page ids come 32 at a time, one load per block of the table row and one
        // block ahead: a lookup per tile would put its latency between the copies
        int blk = -2, cur = 0, ahead = 0;  // ids of blocks blk and blk + 1 of the item's row
        auto ids = [&](int k) {
            const int i = k * 32 + lane, pages = (it.limit + (1 << p.s.page_log2) - 1) >> p.s.page_log2;
            return i < pages ? __ldg(p.table + (int64_t)it.b * p.s.width + i) : -1;
        };
        auto copy = [&](int t) {
            const int kb = (it.tile0 + t) * KT, first = kb >> p.s.page_log2;
            if ((first >> 5) != blk) {
                cur = (first >> 5) == blk + 1 ? ahead : ids(first >> 5);
                blk = first >> 5;
                ahead = ids(blk + 1);
            }
            if (n >= stages) ok = ok && __all_sync(0xffffffffu, att_wait(&empty[st], (round - 1) & 1, failed, limit));
            if (!ok || w.stall) return;
            const int boxes = (min(KT, it.limit - kb) + w.page_box - 1) / w.page_box;
            if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(boxes * w.page_box * 128 * NH));
            // a tile's pages (at most 16) lie in one block
            const int key = kb + lane * w.page_box;
            const int page = __shfl_sync(0xffffffffu, cur, (key >> p.s.page_log2) & 31);
            unsigned char* dst = ring + st * A::UNIT + lane * w.page_box * 128;
            if (lane < boxes)
                for (int h = 0; h < NH; ++h)
                    tma_4d(dst + h * KT * 128, map, h * 64, it.hk, key & ((1 << p.s.page_log2) - 1), page, &full[st]);
            ++n;
            if (++st == stages) st = 0, ++round;
        };
        for (; ok && it.more() && !w.stall; it.next(p, w.g)) {
            const int nt = it.tiles();
            blk = -2;
            copy(0);
            if (is_k)
                for (int s = 0; s < (it.dual ? 2 : 1); ++s) {
                    const uint32_t qb = qi % NS;
                    if (qi >= NS)
                        ok = ok &&
                             __all_sync(0xffffffffu, att_wait(&ms.q_empty[qb], (qi / NS - 1) & 1, failed, limit));
                    if (!ok) break;
                    ++qi;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&ms.q_full[qb], (uint32_t)(w.q_box * w.g.G * 128 * NH));
                        for (int h = 0; h < NH; ++h)
                            tma_4d(q_smem + qb * A::QB + h * ATT_ROWS * 128, &map_q, h * 64, it.hk * w.g.G,
                                   it.t0 + s * w.g.tpt, it.b, &ms.q_full[qb]);
                    }
                }
            for (int t = 1; ok && t < nt; ++t) copy(t);
        }
        // drain: every tile and row tile of Q has been read by the MMAs, so no
        // copy or commit is still on its way when the CTA leaves
        const uint32_t n0 = n > stages ? n - stages : 0, q0 = qi > NS ? qi - NS : 0;
        for (uint32_t i = n0; ok && i < n; ++i) ok = att_wait(&empty[i % stages], (i / stages) & 1, failed, limit);
        for (uint32_t i = q0; ok && i < qi; ++i) ok = att_wait(&ms.q_empty[i % NS], (i / NS) & 1, failed, limit);
        if (!ok) {
            // a role gave up: at least every copy issued has landed
            if (lane == 0) ms.failed = 1;
            for (uint32_t i = n0; i < n; ++i) mbar_wait_n(&full[i % stages], (i / stages) & 1, limit);
            for (uint32_t i = q0; i < qi; ++i) mbar_wait_n(&ms.q_full[i % NS], (i / NS) & 1, limit);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer: the whole warp waits, one lane issues
        constexpr uint32_t ID_S = umma_idesc(F16, false, ATT_ROWS, KT);
        constexpr uint32_t ID_O = umma_idesc(F16, true, ATT_ROWS, DP);
        uint32_t base = 0, qi = 0, cleaned = 0;  // cleaned: bit per stage, phases of v_clean so far
        uint32_t n_unit[2] = {0, 0}, n_seg[2] = {0, 0};  // units and segments of each stream so far
        // descriptors: Q and K are K-major with 8-row groups 1024 bytes apart; V is
        // N-major, 64-column boxes KT rows apart, 8-row groups 1024 bytes apart
        const uint64_t q_desc = umma_desc(smem_u32(q_smem), 16, 1024), k_desc = umma_desc(smem_u32(k_smem), 16, 1024);
        const uint64_t v_desc = umma_desc(smem_u32(v_smem), KT * 128, 1024);
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, att_wait(bar, parity & 1, failed, limit));
        };
        for (; ok && it.more(); it.next(p, w.g)) {
            const bool dual = it.dual;
            const int nt = it.tiles(), units = dual ? 2 * nt : nt, masked = it.first_masked();
            auto scores = [&](int u) {
                const int s = NS == 2 ? u & 1 : 0, t = dual ? u >> 1 : u;
                const uint32_t i = base + t, st = i % KS;
                const uint32_t q = qi + (dual ? s : 0), qb = q % NS;
                if (!dual || s == 0) wait(&ms.k_full[st], i / KS);
                if (t == 0 && (dual || u == 0)) wait(&ms.q_full[qb], q / NS);
                if (!ok) return;
                tmem_fence_after();
                if (elect_one()) {
                    const uint64_t a = q_desc + qb * (A::QB / 16), b = k_desc + st * (A::UNIT / 16);
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k)
                        umma_ss(tmem + A::s_col(s), a + ((k / 4) * ATT_ROWS * 128 + (k % 4) * 32) / 16,
                                b + ((k / 4) * KT * 128 + (k % 4) * 32) / 16, ID_S, k > 0);
                    umma_commit(&ms.s_full[s]);
                    if (!dual || s == 1) umma_commit(&ms.k_empty[st]);
                    if (t == nt - 1) umma_commit(&ms.q_empty[qb]);
                }
                __syncwarp();
            };
            auto values = [&](int u) {
                const int s = NS == 2 ? u & 1 : 0, t = dual ? u >> 1 : u;
                const uint32_t i = base + t, st = i % VS;
                const bool first = u < NS;
                if (!dual || s == 0) {
                    if (t >= masked) {
                        wait(&ms.v_clean[st], cleaned >> st);
                        cleaned ^= 1u << st;
                    } else {
                        wait(&ms.v_full[st], i / VS);
                    }
                }
                if (first && n_seg[s] > 0) wait(&ms.o_empty[s], n_seg[s] - 1);
                wait(&ms.p_ready[s], n_unit[s]);
                if (!ok) return;
                ++n_unit[s];
                if (first) ++n_seg[s];
                tmem_fence_after();
                if (elect_one()) {
                    const uint64_t b = v_desc + st * (A::UNIT / 16);
#pragma unroll
                    for (int k = 0; k < KT / 16; ++k)
                        umma_ts(tmem + A::o_col(s), tmem + A::s_col(s) + k * 8, b + k * 128, ID_O, !first || k > 0);
                    if (!dual || s == 1) umma_commit(&ms.v_empty[st]);
                    if (u + NS >= units) umma_commit(&ms.o_full[s]);
                }
                __syncwarp();
            };
            for (int u = 0; ok && u < min(NS, units); ++u) scores(u);
            for (int u = 0; ok && u < units; ++u) {
                values(u);
                if (ok && u + NS < units) scores(u + NS);
            }
            base += nt;
            qi += dual ? 2 : 1;
        }
        if (!ok) {
            // no MMA is in flight when the CTA leaves (one lane issued them all: the
            // election takes the same lane of a full warp every time)
            if (elect_one()) {
                ms.failed = 1;
                umma_commit(&ms.drain);
                mbar_wait_n(&ms.drain, 0, limit);
            }
            __syncwarp();
        }
    } else if (warp == 3) {
        // ---------------- this range's first item, where it began in an earlier
        // range: the one before it, or the cut is not the first of the item
        if (lane == 0) {
            AttCut cut{-1, 0, 0, 0, 0, 0};
            if (it.more() && it.tile0 > 0) {
                const int first = split.owner(it.at + ATT_ITEM_COST);
                if (first == (int)blockIdx.x - 1)
                    cut = AttCut{first, split.owner(it.at + ATT_ITEM_COST + it.ntiles - 1), it.b, it.hk, it.t0,
                                 it.ntok * w.g.G};
            }
            w.cuts[blockIdx.x] = cut;
        }
    } else {
        // ---------------- softmax: warpgroup s, thread = row
        const int s = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const float c = p.scale * 1.4426950408889634f;
        const int T = p.s.T, Hq = p.s.Hq, D = p.s.D, G = w.g.G;
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
        uint32_t base = 0, n_unit = 0, n_seg[2] = {0, 0}, n_ml = 0, cleaned = 0;
        for (; ok && it.more(); it.next(p, w.g)) {
            const bool dual = it.dual;
            const int nt = it.tiles(), units = dual ? 2 * nt : nt;
            const int tbase = it.t0 + (dual ? s * w.g.tpt : 0);
            const int rows = min(w.g.tpt, it.t0 + it.ntok - tbase) * G;
            const bool active = (warp & 3) * 32 < rows;
            const int t = min(tbase + row / G, it.n - 1);  // rows past the last are computed, never stored
            const bool mine = row < rows;
            float m = -INFINITY, l = 0.f;
            uint32_t pend[KT / 32] = {};  // seen keys with non-finite values, of the tile at pend_kb
            int pend_kb = -1;
            int masked = it.first_masked();  // later: the first masked tile not counted in `cleaned`
            const uint32_t o_addr = tmem + A::o_col(s) + lanes, s_addr = tmem + A::s_col(s) + lanes;

            // the rows of a masked value tile beyond the sequence become 0, and so does
            // what is not finite (noted in nf); the warpgroups share the tile where
            // both read it.  Eight lanes per 128-byte row of a box.
            auto clean = [&](uint32_t st, int kb, bool shared) {
                const int per = shared ? KT / 8 : KT / 4, r0 = ((shared ? s * 4 : 0) + (warp & 3)) * per;
                uint32_t bits = 0;
#pragma unroll 1
                for (int i = 0; i < per; i += 4) {
                    const int r = r0 + i + (lane >> 3), key = kb + r;
                    bool found = false;
                    if (key >= it.mask_from) {
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            uint4* a = (uint4*)(v_smem + st * A::UNIT + (h * KT + r) * 128) + (lane & 7);
                            if (key >= it.ctx + it.n) {
                                *a = make_uint4(0, 0, 0, 0);
                                continue;
                            }
                            uint4 x = *a;
                            const bool bad = clean_word<F16>(x.x) | clean_word<F16>(x.y) | clean_word<F16>(x.z) |
                                             clean_word<F16>(x.w);
                            if (bad) *a = x;
                            found = found || bad;
                        }
                    }
                    const uint32_t v = __ballot_sync(0xffffffffu, found);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if ((v >> (8 * j)) & 0xFFu) bits |= 1u << (i + j);
                }
                fence_async_smem();
                if (lane < per / 16) ((uint16_t*)ms.nf[st])[r0 / 16 + lane] = (uint16_t)(bits >> (16 * lane));
                __syncwarp();
                if (lane == 0) mbar_arrive_n(&ms.v_clean[st], NS == 2 && !shared ? 2 : 1);
            };
            // O += the non-finite values of pend's keys (the MMA saw zeros there)
            auto add_nonfinite = [&]() {
                for (int x = 0; x < KT / 32; ++x) {
                    uint32_t any = __reduce_or_sync(0xffffffffu, pend[x]);
                    for (; any; any &= any - 1) {
                        const int bit = __ffs(any) - 1, key = pend_kb + 32 * x + bit;
                        const int page = __ldg(p.table + (int64_t)it.b * p.s.width + (key >> p.s.page_log2));
                        if (page < 0 || page >= p.s.num_pages) continue;
                        const uint16_t* v = (const uint16_t*)p.c.v + page * p.c.page +
                                            (key & ((1 << p.s.page_log2) - 1)) * p.c.token + it.hk * p.c.head;
                        for (int d = 0; d < D; d += 16) {
                            uint32_t o[16];
                            tmem_ld<16>(o_addr + d, o);
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const uint16_t e = __ldg(v + d + k);
                                if (att_nonfinite<F16>(e) && ((pend[x] >> bit) & 1u))
                                    o[k] = __float_as_uint(__uint_as_float(o[k]) + H::one(e));
                            }
                            tmem_st<16>(o_addr + d, o);
                        }
                        tmem_wait_st();
                    }
                    pend[x] = 0;
                }
                pend_kb = -1;
            };

            for (int u = s; u < units && ok; u += NS) {
                const int tile = dual ? u >> 1 : u, kb = (it.tile0 + tile) * KT;
                ok = __all_sync(0xffffffffu, att_wait(&ms.s_full[s], n_unit & 1, failed, limit));
                if (!ok) break;
                ++n_unit;
                tmem_fence_after();
                const uint32_t vi = base + tile, vst = vi % VS;
                const bool part = kb + KT > it.mask_from;
                if (part) {
                    // phases of v_clean of the tiles before this one (the other stream's)
                    for (; masked < tile; ++masked) cleaned ^= 1u << ((base + masked) % VS);
                    ++masked;
                    ok = __all_sync(0xffffffffu, att_wait(&ms.v_full[vst], (vi / VS) & 1, failed, limit));
                    if (!ok) break;
                    clean(vst, kb, dual);
                    ok = __all_sync(0xffffffffu, att_wait(&ms.v_clean[vst], (cleaned >> vst) & 1, failed, limit));
                    if (!ok) break;
                    cleaned ^= 1u << vst;
                }
                if (active) {
                    // every earlier P V of the stream is complete: the scores were issued after it
                    if (pend_kb >= 0) add_nonfinite();
                    if (part) {
                        // hidden scores become -inf in tensor memory, before the passes over them
                        uint32_t some = 0;
#pragma unroll 1
                        for (int y = 0; y < KT / 32; ++y) {
                            const uint32_t see = att_sees(p, it.b, t, it.ctx, it.n, kb + 32 * y);
                            if (__all_sync(0xffffffffu, see == ~0u)) continue;
                            some |= see & *(volatile uint32_t*)&ms.nf[vst][y];
                            uint32_t x[32];
                            tmem_ld<32>(s_addr + 32 * y, x);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((see >> k) & 1u)) x[k] = 0xFF800000u;
                            tmem_st<32>(s_addr + 32 * y, x);
                        }
                        tmem_wait_st();
                        pend_kb = -1;
                        if (__any_sync(0xffffffffu, some)) {
                            pend_kb = kb;
#pragma unroll
                            for (int y = 0; y < KT / 32; ++y)
                                pend[y] = att_sees(p, it.b, t, it.ctx, it.n, kb + 32 * y) &
                                          *(volatile uint32_t*)&ms.nf[vst][y];
                        }
                    }
                    // the row's maximum, then its exponentials: two passes over the
                    // scores in tensor memory take fewer registers than one that
                    // holds all of them, and no spills
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int y = 0; y < KT; y += 64) {
                        uint32_t x[64];
                        tmem_ld<64>(s_addr + y, x);
#pragma unroll
                        for (int k = 0; k < 64; k += 8)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mx[j] = fmaxf(mx[j], fmaxf(__uint_as_float(x[k + 2 * j]),
                                                           __uint_as_float(x[k + 2 * j + 1])));
                    }
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    // O and l stay in units of the old maximum while the new one is
                    // less than 2^8 above it: p then stays below 2^8
                    const bool grow = top * c > m * c + ATT_LAZY || (m == -INFINITY && top > m);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = grow ? ex2_fast((m - top) * c) : 1.f;
                        if (grow) m = top;
                        l *= f;
                        if (u >= NS) {
                            for (int d = 0; d < D; d += 16) {
                                uint32_t o[16];
                                tmem_ld<16>(o_addr + d, o);
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                tmem_st<16>(o_addr + d, o);
                            }
                        }
                    }
                    const float mc = m == -INFINITY ? 0.f : m * c;
                    const uint64_t c2 = pack2(c, c), mc2 = pack2(-mc, -mc);
                    uint64_t sum[2] = {0ull, 0ull};  // two pairs of partial sums
#pragma unroll
                    for (int y = 0; y < KT; y += 64) {
                        uint32_t x[64];
                        tmem_ld<64>(s_addr + y, x);
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            float2 e = unpack2(fma2(pack2u(x[2 * k], x[2 * k + 1]), c2, mc2));
                            e.x = ex2_fast(e.x);
                            e.y = ex2_fast(e.y);
                            sum[k & 1] = add2(sum[k & 1], pack2(e.x, e.y));
                            x[k] = H::pack(e.x, e.y);
                        }
                        tmem_st<32>(s_addr + y / 2, *reinterpret_cast<uint32_t(*)[32]>(&x));
                    }
                    const float2 sums = unpack2(add2(sum[0], sum[1]));
                    l += sums.x + sums.y;
                    tmem_wait_st();
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.p_ready[s]);
            }
            for (; masked < nt; ++masked) cleaned ^= 1u << ((base + masked) % VS);
            base += nt;
            if (!ok) break;

            // ---- the segment's end: O of the streams with units
            const int units1 = dual ? nt : units / 2;  // of stream 1 (NS == 2)
            const bool join = NS == 2 && !dual && units1 > 0;  // one row tile in two streams
            const bool has = s == 0 || units1 > 0;
            if (has)
                ok = __all_sync(0xffffffffu, att_wait(&ms.o_full[s], n_seg[s] & 1, failed, limit));
            if (!ok) break;
            tmem_fence_after();
            if (has && active && pend_kb >= 0) add_nonfinite();
            if (join && s == 1) {
                // stream 1 hands its maximum and sum over; its O stays until stream 0 has read it
                if (n_ml > 0) ok = __all_sync(0xffffffffu, att_wait(&ms.ml_empty, (n_ml - 1) & 1, failed, limit));
                if (!ok) break;
                ms.ml[row] = make_float2(m, l);
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.ml_full);
            }
            float m1 = -INFINITY, l1 = 0.f;
            if (join && s == 0) {
                ok = __all_sync(0xffffffffu, att_wait(&ms.o_full[1], n_seg[1] & 1, failed, limit) &&
                                                 att_wait(&ms.ml_full, n_ml & 1, failed, limit));
                if (!ok) break;
                tmem_fence_after();
                const float2 o = ms.ml[row];
                m1 = o.x;
                l1 = o.y;
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.ml_empty);
            }
            if (join) ++n_ml;
            ++n_seg[0];
            if (units1 > 0) ++n_seg[1];
            if (active && (s == 0 || dual)) {
                const float mm = fmaxf(m, m1), mr = mm == -INFINITY ? 0.f : mm;
                float f0 = ex2_fast((m - mr) * c), f1 = ex2_fast((m1 - mr) * c);
                if (m == -INFINITY) f0 = 0.f;
                if (m1 == -INFINITY) f1 = 0.f;
                // a NaN sum stays NaN; an infinite maximum (0 x inf above) too
                float ll = l * f0 + (join ? l1 * f1 : 0.f);
                const bool none = ll == 0.f, whole = it.whole();
                if (whole) {
                    const float inv = none ? 0.f : 1.f / ll;
                    f0 *= inv;
                    f1 *= inv;
                }
                const int head = it.hk * G + row % G;
                const int64_t orow = ((int64_t)it.b * T + t) * Hq + head;
                const int64_t slot = (int64_t)blockIdx.x * 2 + (it.tile0 > 0 ? 0 : 1);
                const int prow = (dual ? s * ATT_ROWS : 0) + row;
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                    uint32_t o[32];
                    float y[32];
                    if (join) {
                        uint32_t o1[32];
                        tmem_ld_2x32(o_addr + d, tmem + A::o_col(NS - 1) + lanes + d, o, o1);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            y[k] = __uint_as_float(o[k]) * f0 + __uint_as_float(o1[k]) * f1;
                    } else {
                        tmem_ld<32>(o_addr + d, o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(o[k]) * f0;
                    }
                    if (!mine) continue;
                    if (whole) {
                        uint4* o16 = (uint4*)((char*)p.out + (orow * D + d) * 2);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (d + 8 * k < D)
                                o16[k] = none ? make_uint4(0, 0, 0, 0)
                                              : make_uint4(H::pack(y[8 * k], y[8 * k + 1]),
                                                           H::pack(y[8 * k + 2], y[8 * k + 3]),
                                                           H::pack(y[8 * k + 4], y[8 * k + 5]),
                                                           H::pack(y[8 * k + 6], y[8 * k + 7]));
                    } else {
                        float4* o32 = (float4*)w.part_o + (slot * (DP / 4) + d / 4) * (NS * ATT_ROWS) + prow;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (d + 4 * k < D)
                                o32[k * NS * ATT_ROWS] =
                                    make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
                    }
                }
                if (mine && whole && p.lse) p.lse[orow] = none ? -INFINITY : fmaf(mr, p.scale, logf(ll));
                if (mine && !whole) w.part_ml[slot * NS * ATT_ROWS + prow] = make_float2(mm, ll);
            }
            if (s == 0 || dual) {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&ms.o_empty[s]);
                    if (join) mbar_arrive(&ms.o_empty[1]);
                }
            }
        }
        if (!ok && lane == 0) ms.failed = 1;
    }
    tmem_fence_before();
    __syncthreads();
    if (tid == 0 && ms.failed) atomicOr(w.err, 1u);
    tmem_fence_after();
    if (warp == 0) tmem_free(tmem, ATT_TMEM_COLS);
}

// ------------------------------------------------------------------------- //
// k_tree_combine                                                            //
// ------------------------------------------------------------------------- //
// Joins the parts of an item cut between CTAs: out = sum_i 2^(m_i - m) O_i /
// sum_i 2^(m_i - m) l_i.  Grid (cut, 32 rows, 32 columns); a thread has one row,
// four columns and one in eight of the parts, or all parts of few.
constexpr int COMB_THREADS = 256;

template <bool F16>
__global__ void __launch_bounds__(COMB_THREADS) k_tree_combine(const AttWork w, int DP, int prows)
{
    using H = Half2<F16>;
    __shared__ float4 part[8][32];
    __shared__ float2 part_ml[8][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const AttCut cut = w.cuts[blockIdx.x + 1];
    const int r = blockIdx.y * 32 + (threadIdx.x & 31), g8 = threadIdx.x >> 5;
    if (cut.first < 0 || (int)blockIdx.y * 32 >= cut.rows) return;
    const TreeAttendParams& p = w.p;
    const float c = p.scale * 1.4426950408889634f;
    const int G = w.g.G, D = p.s.D;
    // rows of the second row tile lie behind the first's 128
    const int first_rows = w.g.tpt * G, pr = r < first_rows ? r : ATT_ROWS + r - first_rows;
    const bool on = r < cut.rows;
    const int64_t orow = ((int64_t)cut.b * p.s.T + cut.t0 + r / G) * p.s.Hq + cut.hk * G + r % G;
    const int n = cut.last - cut.first + 1;
    auto slot = [&](int i) { return (int64_t)(cut.first + i) * 2 + (i == 0 ? 1 : 0); };
    auto ml = [&](int i) { return on ? w.part_ml[slot(i) * prows + pr] : make_float2(-INFINITY, 0.f); };
    auto weight = [&](float m, float top) { return m == -INFINITY ? 0.f : ex2_fast((m - top) * c); };
    const int step = n > 8 ? 8 : 1, i0 = n > 8 ? g8 : 0;
    float top = -INFINITY;
    for (int i = i0; i < n; i += step) top = fmaxf(top, ml(i).x);
    if (step == 8) {
        part_ml[g8][threadIdx.x & 31].x = top;
        __syncthreads();
        for (int k = 0; k < 8; ++k) top = fmaxf(top, part_ml[k][threadIdx.x & 31].x);
        __syncthreads();
    }
    const float ref = top == -INFINITY ? 0.f : top;
    float l = 0.f;
    for (int i = i0; i < n; i += step) {
        const float2 v = ml(i);
        l += v.y * weight(v.x, ref);
    }
    if (step == 8) {
        part_ml[g8][threadIdx.x & 31].y = l;
        __syncthreads();
        l = 0.f;
        for (int k = 0; k < 8; ++k) l += part_ml[k][threadIdx.x & 31].y;
    }
    const bool none = l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
    auto store = [&](int col4, float4 y) {
        if (!on || col4 * 4 >= D) return;
        uint2 h = make_uint2(H::pack(y.x * inv, y.y * inv), H::pack(y.z * inv, y.w * inv));
        if (none) h = make_uint2(0, 0);
        *(uint2*)((char*)p.out + (orow * D + col4 * 4) * 2) = h;
    };
    auto sum = [&](int col4, int from, int by) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on && col4 * 4 < D)
#pragma unroll 4
            for (int i = from; i < n; i += by) {
                const float f = weight(ml(i).x, ref);
                const float4 v = ((const float4*)w.part_o)[(slot(i) * (DP / 4) + col4) * prows + pr];
                y.x += f * v.x, y.y += f * v.y, y.z += f * v.z, y.w += f * v.w;
            }
        return y;
    };
    if (step == 1) {
        store(blockIdx.z * 8 + g8, sum(blockIdx.z * 8 + g8, 0, 1));
    } else {
        for (int k = 0; k < 8; ++k) {
            __syncthreads();
            part[g8][threadIdx.x & 31] = sum(blockIdx.z * 8 + k, g8, 8);
            __syncthreads();
            if (g8 == 0) {
                float4 y = part[0][threadIdx.x];
                for (int x = 1; x < 8; ++x) {
                    const float4 v = part[x][threadIdx.x];
                    y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
                }
                store(blockIdx.z * 8 + k, y);
            }
        }
    }
    if (p.lse && on && g8 == 0 && blockIdx.z == 0) p.lse[orow] = none ? -INFINITY : fmaf(ref, p.scale, logf(l));
}

// ------------------------------------------------------------------------- //
// host side                                                                 //
// ------------------------------------------------------------------------- //
static int att_dp(int D) { return (D + 63) / 64 * 64; }
static int att_part_rows(int DP) { return (DP <= 128 ? 2 : 1) * ATT_ROWS; }

// workspace: partial O, (m, l) and cuts of `ctas` CTAs
size_t tree_attend_bytes(int D, int ctas, size_t* ml_at, size_t* cut_at)
{
    const int DP = att_dp(D);
    const size_t slots = 2 * (size_t)ctas, o = slots * att_part_rows(DP) * DP * sizeof(float);
    const size_t ml = slots * att_part_rows(DP) * sizeof(float2);
    *ml_at = o;
    *cut_at = o + ml;
    return o + ml + (size_t)ctas * sizeof(AttCut);
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
    const cuuint32_t box[4] = {64, (cuuint32_t)box1, (cuuint32_t)box2, 1}, one[4] = {1, 1, 1, 1};
    return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void*>(ptr), d, st, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool F16, int DP>
static cudaError_t att_launch(AttWork w, int num_sms, cudaStream_t s)
{
    using A = Att<DP>;
    static DeviceOnce once;  // per device: the shared-memory opt-in
    cudaError_t e = cuda_once(once, nullptr, [](int, int*) {
        return cudaFuncSetAttribute(k_tree_attend<F16, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, A::SMEM);
    });
    if (e != cudaSuccess) return e;
    const TreeShape& sh = w.p.s;
    w.g.group = A::NS * w.g.tpt;
    w.page_box = min(1 << sh.page_log2, A::KT);
    w.q_box = min(w.g.tpt, sh.T);
    CUtensorMap mq, mk, mv;
    const int64_t qd[3] = {sh.Hq, sh.T, sh.B}, qs[3] = {w.p.q.head, w.p.q.token, w.p.q.seq};
    const int64_t cd[3] = {sh.Hkv, 1 << sh.page_log2, sh.num_pages}, cs[3] = {w.p.c.head, w.p.c.token, w.p.c.page};
    if (!att_map(&mq, F16, w.p.q.ptr, sh.D, qd, qs, w.g.G, w.q_box) ||
        !att_map(&mk, F16, w.p.c.k, sh.D, cd, cs, 1, w.page_box) ||
        !att_map(&mv, F16, w.p.c.v, sh.D, cd, cs, 1, w.page_box))
        return cudaErrorInvalidValue;
    k_tree_attend<F16, DP><<<num_sms, A::THREADS, A::SMEM, s>>>(mq, mk, mv, w);
    if ((e = cudaGetLastError()) != cudaSuccess || num_sms == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    const int rows = min(w.g.group, sh.T) * w.g.G;
    cfg.gridDim = dim3((unsigned)num_sms - 1, (unsigned)((rows + 31) / 32), (unsigned)((sh.D + 31) / 32));
    cfg.blockDim = dim3(COMB_THREADS);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_tree_combine<F16>, w, DP, A::NS * ATT_ROWS);
}

bool tree_attend_fits(const TreeShape& sh)
{
    const int64_t kt = sh.D <= 128 ? 128 : 64, group = (sh.D <= 128 ? 2 : 1) * (ATT_ROWS / (sh.Hq / sh.Hkv));
    const int64_t groups = (sh.T + group - 1) / group;
    const int64_t tiles = (((int64_t)sh.width << sh.page_log2) + kt - 1) / kt + ATT_ITEM_COST;
    return (double)sh.B * sh.Hkv * groups * tiles < 2147483648.0;
}

cudaError_t launch_tree_attend(const TreeAttendParams& p, int dtype, int num_sms, void* ws, unsigned* err, bool stall,
                               cudaStream_t s)
{
    size_t ml_at, cut_at;
    tree_attend_bytes(p.s.D, num_sms, &ml_at, &cut_at);
    AttWork w = {};
    w.p = p;
    w.g.G = p.s.Hq / p.s.Hkv;
    w.g.tpt = ATT_ROWS / w.g.G;
    w.g.Hkv = p.s.Hkv;
    w.part_o = (float*)ws;
    w.part_ml = (float2*)((char*)ws + ml_at);
    w.cuts = (AttCut*)((char*)ws + cut_at);
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
