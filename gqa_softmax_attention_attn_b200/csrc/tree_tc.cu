// tree_tc.cu -- bf16 decode of a tree of drafted tokens per sequence on the
// sm_100a tensor cores (tcgen05, accumulators in tensor memory, TMA-staged K/V),
// over contiguous and paged caches.
//
// The mathematics is tree_simt.cu's: per row (drafted token, query head) the
// online softmax over the keys the row sees, in one pass over a chunk of them,
// without the sink, which joins once in the combine of the splits (or here,
// when a sequence needs one split).  The softmax statistics are fp32; P is
// rounded to bf16 for P V (unnormalised, so its relative rounding, half a step
// of bf16, is what reaches the output) and the row sum adds the unrounded P.
//
// Design: T drafted tokens times G query heads of a KV group share every K/V
// byte, T G 64 flop a byte: with up to 64 rows a KV head the kernel is bound by
// HBM, beyond that by the softmax (one exponential per 256 flop).
//  * The work is one line of 64-key tiles, sequence by sequence, cut evenly over
//    teams of CTAs, whatever the lengths: as many as fit the GPU at once (two CTAs
//    per SM, 256 TMEM columns each).  A team has a CTA for every row tile and KV
//    head, which walk the same tokens at the same time, so that row tiles meet in L2 and the
//    heads' 128-byte rows of a token are read from one DRAM page (with the heads one
//    after the other on the line, 64 sequences of 8 tokens took 558 us instead of 400);
//    of groups of KV heads, where all of them would leave too many SMs idle.  A team's
//    stretch covers a few segments (stretches of one sequence); a segment
//    that is not the whole of its sequence leaves a partial (m, l, o) in the
//    workspace, at most two per CTA, and the join kernel adds them up.  (With a grid of
//    fixed chunks the last wave, the starts and the partials took a third of the time:
//    16 sequences of 61 tokens 209 us unsplit, 235 in chunks of 2048 keys, 266 in 1024.)
//  * A row tile is 128 / C rows, held C times in the 128 lanes of the MMA tile
//    (C = 4, 2, 1 for up to 32, 64, more rows): copy k's threads take the
//    k-th part of every tile's keys and write zeros of P elsewhere, once, so
//    that few rows still keep all four softmax warps busy and each has 1/C of
//    the exponentials in its dependent chain; the copies' sums join through
//    shared memory at the end.  The tensor pipe does C times the work, of
//    which it has plenty to spare while HBM is the limit.
//  * Warps 0-3, one row (copy) a thread, do the softmax; warps 4 and 5 stream K and
//    V in tiles of 64 keys (128-byte-swizzled TMA boxes, one a page for small
//    pages) through rings of kNS stages; warp 6 issues S = Q K^T and O += P V, Q and P read from
//    tensor memory, S double-buffered there, so that neither product is in the
//    softmax warps' chain: S(t + 2) follows P V(t).  One warp issues both, in order, so S(t + 2) being
//    complete means P V(t) is.
//    (Four chains an SM with single buffers, P written over S, hid less: from P
//    to the next S 1000 to 1700 cycles a tile were in each chain, 1060 cycles a
//    tile and SM in all.)
//  * The reference maximum moves in whole powers of two, and only when a tile's
//    exponentials sum past kSumLimit: scaling what is already summed or
//    multiplied by it is then exact.
//  * Masks: a thread's visible keys of a tile are one 64-bit word -- the cached
//    prefix as a range, the drafted keys as the row's ancestor bits shifted
//    into place -- and only tiles some row does not see in full apply it.
//  * Key and value rows no row of the sequence sees may hold anything: their
//    scores are selected away, their V rows zeroed in shared memory.
//  * Every wait is bounded; on expiry the CTA raises the device status bit, waits
//    (bounded) for its own loads and MMAs, frees tensor memory and exits.
//  * The host divides the GPU for max_q tokens in every sequence: a CTA whose row tile
//    a sequence does not reach skips it, so a bound above the drafts, or one long draft among
//    short ones, leaves that part of the GPU idle (64 sequences of 8 tokens 404 us with a bound
//    of 8, 850 with 32, 5912 with 256).
// Measured (64 query and 8 KV heads): 64 sequences of 1024 to 32768 keys in pages of
// 16, 8 tokens each, 370 to 407 us, 5.5 to 6.0 TB/s, bound by HBM in short runs.  Repeated
// for seconds it takes 425 to 475 us: HBM, the products and the exponentials
// together reach the 1000 W limit and the clock falls to 1.2 to 1.4 GHz (without
// the products 360 us).  Beyond 64 rows a KV head the softmax warps' chain
// bounds it: 16 sequences of 61 tokens 202 to 211 us, one of 131072 keys with 32 tokens 119 to 130
// us; a tile is 1500 to 1650 cycles of it, 880 in the pass of the exponentials (two CTAs'
// warps share a scheduler; 440 without the exponentials) and 600 in its waits, votes,
// loads and arrivals, 90 to 180 each.  Of the 318000 cycles of a CTA of the first, 182 us at the
// 1.7 to 1.8 GHz that it runs at, 282000 are its 172 tiles, 9000 epilogues, 5000 the plan, 1000
// first scores and 20000 the segments' starts (Q, paths) and end; of 200000 of the second (116 us)
// 184000 are its 114 tiles.  (Not bounded by the S products: with three S buffers
// 201 us; nor by the load of S: with the next tile's scores loaded during the pass 225 us.)
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include "kernels.h"
#include "sm100_ptx.cuh"
#include "tree_path.cuh"

namespace attn_sink {
namespace {

constexpr int kM = 128;
constexpr int kD = 64;
constexpr int kBN = kTreeTile;
constexpr int kNS = 5;         // K/V ring stages
constexpr int kThreads = 224;  // warps: 4 softmax, K loads, V loads, MMA issue
constexpr int kCtasPerSm = 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// exponentials that sum past this move the row's reference maximum
constexpr float kSumLimit = 1024.f;

constexpr int kTileBytes = kBN * kD * 2;
constexpr int kOffRed = 0;  // [128][32] half of the copies' O, joined after the last tile
constexpr int kOffK = kM * 32 * 4;
constexpr int kOffV = kOffK + kNS * kTileBytes;
constexpr int kOffPath = kOffV + kNS * kTileBytes;         // [128][kPathWords] ancestor bits
constexpr int kOffDepth = kOffPath + kM * kPathWords * 4;  // [128] depths
constexpr int kOffPar = kOffDepth + kM * 2;                // [256] parents
constexpr int kOffMl = kOffPar + kTreeMaxTokens * 2;       // [128] (m, l) of the copies
constexpr int kOffBar = kOffMl + kM * 8;
// k_full[], k_empty[], v_full[], v_empty[], s_full[2], p_full[2], o_done, o_last, q_full
constexpr int kNumBar = 4 * kNS + 7;
constexpr int kOffPlan = kOffBar + (kNumBar + 1) / 2 * 16;  // TreeSpan, then the scan's warp sums
constexpr int kOffMisc = kOffPlan + 32 + 8 * 8;             // TMEM address, abort flag
constexpr int kSmemBytes = kOffMisc + 16 + 1024;
static_assert(kOffBar % 8 == 0, "barriers on 8 bytes");
static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory");
// tensor memory: S double-buffered, O, Q (bf16, 32 columns), and P (bf16): over S with one copy of the rows (the
// tensor pipe runs one thread's MMAs in order, so the next S there follows P V), else a buffer of its own, whose
// zeros in the other copies' keys stay
constexpr int kTmS = 0, kTmO = 2 * kBN, kTmQ = kTmO + kD, kTmP = kTmQ + kD / 2, kTmCols = 256;
static_assert(kTmP + kBN / 2 <= kTmCols && kCtasPerSm * kTmCols <= 512, "tensor memory");
// shortest stretch of the line; units up to kTreeSnapTiles are never cut
constexpr int kTreeMinTiles = 4, kTreeSnapTiles = 8;

struct TreeTcParams {
    TreeShape s;
    int G, row_tiles, copies, box_rows;
    unsigned g_magic;   // ceil(2^32 / G), for row_token()
    int page_shift;     // page_size = 2^page_shift, or -1
    int heads, head_groups;  // KV heads of a team; groups of them (units of the line) per sequence
    int teams;   // stretches of the line; a team is heads * row_tiles CTAs
    int q_min;   // shortest stretch, in tiles
    int snap;    // whole units (sequence, group of KV heads) only: no partials
    float c_log2;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    float *lse, *ws_o, *ws_ml;
    long long *plan;  // [0] tiles a stretch, [1 + b] tiles in front of sequence b (B + 1 entries)
    unsigned *status;
    long long timeout_ns;
};

// Runtime divisions cost 100 cycles (32 bits) to 250 (64 bits), one after the other in front of a CTA's first
// load; these are their cheap cases.
__device__ __forceinline__ long long div64(long long a, long long b)
{
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
// row / G by the high word of row * ceil(2^32 / G): the product is off by row * (less than G), which stays below
// 2^32 for rows and G below 2^16
__device__ __forceinline__ int row_token(const TreeTcParams &p, int row)
{
    if (p.G == 1) return row;
    return (row | p.G) >> 16 ? row / p.G : (int)__umulhi((unsigned)row, p.g_magic);
}
__device__ __forceinline__ int key_page(const TreeTcParams &p, int key)
{
    return p.page_shift >= 0 ? key >> p.page_shift : key / p.s.page_size;
}

// tiles of one unit of sequence b: the keys some row of it sees, at least one (a sequence without keys gets
// its output from a tile that is masked altogether); none without rows
__device__ __forceinline__ int unit_tiles(const TreeSeq &q)
{
    return q.T <= 0 ? 0 : max(1, (q.len - q.lo_al + kBN - 1) / kBN);
}

// A CTA's stretch [pos, end) of the line, starting in sequence b, which begins at tile base.
struct TreeSpan {
    long long pos, end, base;
    int b;
};

__device__ __forceinline__ bool wait_noabort(uint64_t *bar, uint32_t parity, unsigned *status, long long tmo)
{
    int never = 0;
    return mbar_wait(bar, parity, &never, status, tmo > 1000000000LL ? tmo : 1000000000LL);
}

// keys [lo, hi) of the 64 from key 0 on
__device__ __forceinline__ uint64_t range_bits(int lo, int hi)
{
    lo = max(lo, 0);
    hi = min(hi, 64);
    if (hi <= lo) return 0;
    return (~0ull >> (64 - (hi - lo))) << lo;
}

// bits [at, at + 64) of a path (at may be negative)
__device__ __forceinline__ uint64_t path_bits(const uint32_t *path, int at)
{
    if (at <= -64 || at >= kTreeMaxTokens) return 0;
    auto word = [&](int w) -> uint64_t { return w >= 0 && w < kPathWords ? path[w] : 0u; };
    const int w = at >> 5, sh = at & 31;
    const uint64_t lo = word(w) | word(w + 1) << 32;
    return sh == 0 ? lo : (lo >> sh) | (word(w + 2) << (64 - sh));
}

template <int C>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const TreeTcParams p)
{
    grid_dep_launch();  // the join may start its set-up; it waits for this grid
    constexpr int kRows = kM / C;  // rows of a tile
    constexpr int kC = kBN / C;    // keys of a tile per thread
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *k_empty = k_full + kNS, *v_full = k_empty + kNS, *v_empty = v_full + kNS;
    uint64_t *s_full = v_empty + kNS, *p_full = s_full + 2, *o_done = p_full + 2, *o_last = o_done + 1;
    uint64_t *q_full = o_last + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 4);

    long long *scan = reinterpret_cast<long long *>(smem + kOffPlan + 32);
    TreeSpan *span_s = reinterpret_cast<TreeSpan *>(smem + kOffPlan);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rt = blockIdx.x % p.row_tiles, head = blockIdx.x / p.row_tiles % p.heads;
    const int team = blockIdx.x / p.row_tiles / p.heads, r0 = rt * kRows;

    // the first try and its vote keep the warp converged when the phase is over, or ends while the try is
    // suspended; only a try that runs out takes the bounded polling loop
    auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        return __all_sync(0xffffffffu, mbar_wait_slow(bar, parity, abort_flag, p.status, p.timeout_ns));
    };

    // ---- the plan: every CTA scans the batch's lengths (a thread a run of sequences) and takes its stretch
    // (the barriers and tensor memory are set up meanwhile)
    if (warp == 4 && lane == 0) {
        for (int i = 0; i < kNS; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);  // the softmax warps
        }
        mbar_init(o_done, 1);
        mbar_init(o_last, 1);
        mbar_init(q_full, 4);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 6) {
        tmem_alloc(tmem_slot, kTmCols);
        tmem_relinquish();
    }
    grid_dep_wait();  // the grid ahead: what it wrote is read from here on
    TreeSpan span;
    {
        const int run = (p.s.B + kThreads - 1) / kThreads;
        const int b0 = min((int)threadIdx.x * run, p.s.B), b1 = min(b0 + run, p.s.B);
        long long mine = 0;
        int nt0 = 0;  // of the thread's first sequence (its only one in batches of up to kThreads)
        for (int b = b0; b < b1; ++b) {
            const int nt = unit_tiles(tree_seq(p.s, b));
            if (b == b0) nt0 = nt;
            mine += (long long)nt * p.head_groups;
        }
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) scan[warp] = incl;
        if (threadIdx.x == 0) span_s->b = -1;
        __syncthreads();
        long long before = incl - mine, total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += scan[w];
            total += scan[w];
        }
        const long long q = max(div64(total + p.teams - 1, p.teams), (long long)p.q_min);
        const long long first = q * team, last = min(first + q, total);
        // (snap: the units that start in [first, last), whole)
        long long at = before;
        for (int b = b0; b < b1; ++b) {
            const int nt = b == b0 ? nt0 : unit_tiles(tree_seq(p.s, b));
            const long long len = (long long)nt * p.head_groups;
            if (blockIdx.x == 0 && p.plan) p.plan[1 + b] = at;
            if (first < last && at <= first && first < at + len) {
                span_s->pos = p.snap ? at + div64(first - at + nt - 1, nt) * nt : first;
                span_s->end = last;
                span_s->base = at;
                span_s->b = b;
            }
            at += len;
        }
        if (blockIdx.x == 0 && p.plan && b1 == p.s.B && b0 < b1) {
            p.plan[0] = q;
            p.plan[1 + p.s.B] = total;
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        span = *span_s;
    }
    const uint32_t tmem = *tmem_slot;
    // segment by segment: f(sequence, its number, KV head, first tile, tiles, all tiles of the unit); stops at false
    auto for_segments = [&](auto f) {
        if (span.b < 0) return;  // no work
        long long pos = span.pos, base = span.base;
        int b = span.b;
        TreeSeq sq = tree_seq(p.s, b);
        int nt = unit_tiles(sq);
        while (pos < span.end) {
            while (pos >= base + (long long)nt * p.head_groups) {
                base += (long long)nt * p.head_groups;
                sq = tree_seq(p.s, ++b);
                nt = unit_tiles(sq);
            }
            const int u = p.head_groups == 1 ? 0 : (int)div64(pos - base, nt);
            const int g = u * p.heads + head, ta = (int)(pos - base - (long long)u * nt);
            const int n = p.snap ? nt : (int)min((long long)(nt - ta), span.end - pos);
            if (r0 < min(sq.T, p.s.max_q) * p.G && !f(sq, b, g, ta, n, nt, pos == span.pos)) return;
            pos += n;
        }
    };

    // ---- producers.  The whole warp runs the loop, so that every operand is warp-uniform, and one elected
    // lane issues (from a lane == 0 branch an issue took twice as long).
    int pt = 0;  // tiles issued
    auto produce = [&](const CUtensorMap &map, uint64_t *full, uint64_t *empty, uint32_t ring) {
        const int ps = p.s.page_size, nb = kBN / p.box_rows, per = 32 / nb;  // boxes of a tile, tiles of a batch
        int st = 0;
        uint32_t ph = 1;
        if (elect_one()) tma_prefetch_desc(&map);
        for_segments([&](const TreeSeq &sq, int b, int g, int ta, int n, int, bool) -> bool {
            const int key0 = sq.lo_al + ta * kBN;
            // the pages of 32 boxes from tile t of the segment on, one a lane; boxes behind the sequence
            // (masked) reuse its last page, so the table is only read within the sequence's own entries
            auto pages = [&](int t) -> int {
                const int lp = key_page(p, min(key0 + t * kBN + lane * p.box_rows, max(sq.len - 1, 0)));
                return p.s.page_table[(size_t)b * p.s.max_pages + lp];
            };
            // a tile's slot in its page: 0 for pages of at most a tile, else it advances with the tiles
            int slot = ps > 0 ? key0 - key_page(p, key0) * ps : key0, in_batch = 0;
            int page = 0, next_page = 0;
            if (ps > 0) {
                page = pages(0);
                if (per < n) next_page = pages(per);
            }
            for (int t = 0; t < n; ++t) {
                int outer[kBN / 8];
                outer[0] = b;
                if (ps > 0) {
                    if (in_batch == per) {
                        in_batch = 0;
                        page = next_page;  // loaded a batch ahead
                        if (t + per < n) next_page = pages(t + per);
                    }
#pragma unroll
                    for (int i = 0; i < kBN / 8; ++i)
                        if (i < nb) outer[i] = __shfl_sync(0xffffffffu, page, in_batch * nb + i);
                    ++in_batch;
                }
                if (!wait_all(&empty[st], ph)) return false;
                if (elect_one()) {
                    const uint32_t dst = ring + st * kTileBytes, bar = smem_u32(&full[st]);
                    mbar_arrive_expect_tx(&full[st], kTileBytes);
                    tma_load_4d_at(dst, &map, 0, g, slot, outer[0], bar);
#pragma unroll
                    for (int i = 1; i < kBN / 8; ++i)
                        if (i < nb) tma_load_4d_at(dst + i * p.box_rows * kD * 2, &map, 0, g, slot, outer[i], bar);
                }
                __syncwarp();
                if (ps == 0 || ps > kBN) {
                    slot += kBN;
                    if (slot == ps) slot = 0;
                }
                ++pt;
                if (++st == kNS) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            return true;
        });
        // every load issued must land before the CTA may exit
        for (int x = 0; x < kNS && x < pt; ++x)
            wait_noabort(&full[x], (uint32_t)((pt - 1 - x) / kNS) & 1u, p.status, p.timeout_ns);
    };

    if (warp == 4) {
        produce(tmK, k_full, k_empty, smem_u32(smem + kOffK));
    } else if (warp == 5) {
        produce(tmV, v_full, v_empty, smem_u32(smem + kOffV));
    } else if (warp == 6) {
        // ------------------------------------------------------------ MMA issuer (converged, one lane issues)
        constexpr uint32_t id_s = idesc_bf16_f32(kM, kBN, 0), id_pv = idesc_bf16_f32(kM, kD, 1);
        const uint64_t k_desc = smem_desc_sw128(smem_u32(smem + kOffK), 16, 1024);
        const uint64_t v_desc = smem_desc_sw128(smem_u32(smem + kOffV), kBN * 128, 1024);
        int kst = 0, st = 0;  // stages of the next K, of the next V, and their phases
        uint32_t kph = 0, ph = 0;
        uint32_t sn = 0, n_seg = 0;            // tiles of S so far; segments
        bool pending = false;                  // products issued that no o_last covers
        auto issue_s = [&]() {  // one lane
            const uint64_t kd = k_desc + (uint64_t)((uint32_t)(kst * kTileBytes) >> 4);
            const uint32_t ts = tmem + kTmS + (sn & 1) * kBN;
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk)
                mma_ts(ts, tmem + kTmQ + kk * 8, kd + (uint64_t)(kk * 32 >> 4), id_s, kk > 0 ? 1u : 0u);
            mma_commit(&s_full[sn & 1]);
            mma_commit(&k_empty[kst]);
        };
        auto next_k = [&]() {
            ++sn;
            if (++kst == kNS) {
                kst = 0;
                kph ^= 1u;
            }
        };
        uint32_t n = 0;  // tiles of P V so far
        for_segments([&](const TreeSeq &sq, int, int, int ta, int nt, int, bool) -> bool {
            if (!wait_all(q_full, n_seg & 1u)) return false;
            tc_fence_after();
            int ahead = 0;  // tiles of this segment with S issued
            for (; ahead < min(nt, 2); ++ahead) {
                if (!wait_all(&k_full[kst], kph)) return false;
                tc_fence_after();
                if (elect_one()) issue_s();
                __syncwarp();
                pending = true;
                next_k();
            }
            for (int t = 0; t < nt; ++t, ++n) {
                // before P is there: the waits for this V and the K after the next, V's zeros
                const bool more = ahead < nt;
                if (!wait_all(&v_full[st], ph) || (more && !wait_all(&k_full[kst], kph))) return false;
                const int j0 = sq.lo_al + (ta + t) * kBN;
                if (j0 < sq.lo || j0 + kBN > sq.len) {
                    // value rows no row sees may hold anything (0 x NaN is NaN): zeros
                    uint4 *vt = reinterpret_cast<uint4 *>(smem + kOffV + st * kTileBytes);
                    for (int e = lane; e < kBN * 8; e += 32) {
                        const int j = j0 + (e >> 3);
                        if (j < sq.lo || j >= sq.len) vt[e] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                // (the first P of a segment: O of the one before has been read, too)
                if (!wait_all(&p_full[n & 1], (n >> 1) & 1u)) return false;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t vd = v_desc + (uint64_t)((uint32_t)(st * kTileBytes) >> 4);
                    const uint32_t tp = tmem + (C == 1 ? kTmS + (n & 1) * kBN : kTmP);
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk)
                        mma_ts(tmem + kTmO, tp + kk * 8, vd + (uint64_t)(kk * 2048 >> 4), id_pv,
                               (t > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(o_done);
                    mma_commit(&v_empty[st]);
                    if (more) issue_s();  // P(t) being there, S(t) has been read
                    // last of all: once the last o_last is over, no arrival on this CTA's barriers is to come
                    if (t == nt - 1) mma_commit(o_last);
                }
                __syncwarp();
                if (more) {
                    next_k();
                    ++ahead;
                }
                if (++st == kNS) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            ++n_seg;
            pending = false;
            return true;
        });
        // given up half way: what is in flight must still end before tensor memory is freed (nobody else
        // waits for o_last then)
        if (pending) {
            if (elect_one()) mma_commit(o_last);
            __syncwarp();
            ++n_seg;
        }
        if (n_seg > 0) wait_noabort(o_last, (n_seg - 1) & 1u, p.status, p.timeout_ns);
    } else {
        // ------------------------------------------------------------ softmax + epilogue
        const int lrow = warp * 32 + lane;                // TMEM lane
        const int r = lrow % kRows, copy = lrow / kRows;  // row of the tile, copy of it
        const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
        uint32_t(*path)[kPathWords] = reinterpret_cast<uint32_t(*)[kPathWords]>(smem + kOffPath);
        int16_t *depth = reinterpret_cast<int16_t *>(smem + kOffDepth);
        if (C > 1) {
            // P of the keys of the other copies stays zero
            uint32_t z[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) z[k] = 0u;
#pragma unroll
            for (int k = 0; k < kBN / 32; ++k) tmem_st16(trow + kTmP + 16 * k, z);
            tmem_wait_st();
        }
        const float2 C2 = make_float2(p.c_log2, p.c_log2);
        uint32_t n = 0, n_seg = 0;  // tiles, segments so far
        for_segments([&](const TreeSeq &sq, int, int g, int ta, int nt, int nt_unit, bool is_first) -> bool {
        const int rows = min(sq.T, p.s.max_q) * p.G, nrow = min(kRows, rows - r0);
        const bool valid = r < nrow;
        const bool active = (warp * 32) % kRows < nrow;  // some row of this warp exists
        const int row = r0 + (valid ? r : 0), row_tok = row_token(p, row);
        const int i0 = row_token(p, r0), tok = row_tok - i0, h = g * p.G + row - row_tok * p.G;
        const size_t at = (size_t)(sq.row0 + row_tok) * p.s.Hq + h;
        {
            // Q: this thread's row into tensor memory (rows that do not exist: zeros).  From shared memory every S
            // product read its 16 KB again: 64 sequences of 1 and of 4 tokens 2 to 4 % longer at the power limit, more
            // tokens 1 %.
            const uint4 *src = reinterpret_cast<const uint4 *>(p.q + at * kD);
            uint32_t x[2][16];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint4 v = valid ? src[k] : make_uint4(0u, 0u, 0u, 0u);
                x[k >> 2][4 * (k & 3)] = v.x;
                x[k >> 2][4 * (k & 3) + 1] = v.y;
                x[k >> 2][4 * (k & 3) + 2] = v.z;
                x[k >> 2][4 * (k & 3) + 3] = v.w;
            }
            tmem_st16(trow + kTmQ, x[0]);
            tmem_st16(trow + kTmQ + 16, x[1]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        const int kfirst = sq.lo_al + ta * kBN;  // first key of the segment
        const float sink2 = p.s.sinks[h] * kLog2e;
        // reference maximum in log2 units, a whole number: next to the sink's until a tile moves it
        float m = rintf(sink2);
        float l = 0.f;   // running sum, without the sink
        int vis_lo = 0;  // first cached key this row sees
        if (p.s.window > 0 || kfirst + nt * kBN > sq.cached) {
            tree_paths(p.s, sq, i0, row_token(p, r0 + nrow - 1) - i0 + 1, lrow, 128,
                       reinterpret_cast<int16_t *>(smem + kOffPar), path, depth, [] { named_bar_sync(1, 128); });
            if (p.s.window > 0) vis_lo = max(0, sq.cached + depth[tok] - p.s.window + 1);
        }
        bool ok = true;
        for (int t = 0; t < nt; ++t, ++n) {
            const int sb = n & 1;
            const int j0 = kfirst + t * kBN;
            // S(t) is complete, and with it P V(t - 2)
            if (!wait_all(&s_full[sb], (n >> 1) & 1u)) {
                ok = false;
                break;
            }
            if (!active) {  // no row here: P's values do not matter, only the barrier
                if (lane == 0) mbar_arrive(&p_full[sb]);
                continue;
            }
            tc_fence_after();
            uint32_t sr[kC / 16][16];
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) tmem_ld16(trow + kTmS + sb * kBN + copy * kC + 16 * k, sr[k]);
            tmem_wait_ld();
            float sv[kC];
#pragma unroll
            for (int k = 0; k < kC; ++k) sv[k] = __uint_as_float(sr[k / 16][k % 16]);
            if (__any_sync(0xffffffffu, j0 < vis_lo || j0 + kBN > sq.cached)) {
                uint64_t see = range_bits(vis_lo - j0, sq.cached - j0);
                if (j0 + kBN > sq.cached) see |= path_bits(path[tok], j0 - sq.cached) & range_bits(0, sq.len - j0);
                see >>= copy * kC;
                const uint32_t see0 = (uint32_t)see, see1 = (uint32_t)(see >> 32);
#pragma unroll
                for (int k = 0; k < kC; ++k)
                    sv[k] = ((k < 32 ? see0 : see1) >> (k & 31)) & 1u ? sv[k] : -INFINITY;
            }
            // P = exp2(S C - m) against the reference, without looking for the tile's maximum: every
            // exponential is at most their sum, and a sum within kSumLimit (NaN fails the test) keeps the
            // reference
            const uint32_t tp = trow + (C == 1 ? kTmS + sb * kBN : kTmP + copy * (kC / 2));
            float2 acc[2];
            auto exp_pass = [&](float neg_m) -> bool {
                const float2 M2 = make_float2(neg_m, neg_m);
                acc[0] = acc[1] = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) {
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 x = ffma2(make_float2(sv[16 * k + 2 * e], sv[16 * k + 2 * e + 1]), C2, M2);
                        const float2 pe = make_float2(ex2(x.x), ex2(x.y));
                        acc[e & 1] = fadd2(acc[e & 1], pe);
                        pk[e] = pack_bf16x2(pe.x, pe.y);
                    }
                    // one buffer of P: P V(t - 1) must have read it
                    if (C > 1 && k == 0 && n > 0 && !wait_all(o_done, (n - 1) & 1u)) return false;
                    tmem_st8(tp + 8 * k, pk);
                }
                return true;
            };
            if (!exp_pass(m == -INFINITY ? 0.f : -m)) {
                ok = false;
                break;
            }
            float sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
            const bool big = !(sum <= kSumLimit) || m == -INFINITY;
            if (__any_sync(0xffffffffu, big)) {
                float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
                for (int k = 4; k < kC; k += 4)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], sv[k + e]);
                const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c_log2;
                const bool move = big && tmax > m;
                if (__any_sync(0xffffffffu, move)) {
                    // up by a whole number of powers of two, so that the scaling is exact (by more than 126, from
                    // a sink far below or none: what was summed is 0 against the new reference)
                    const float m_new = !move ? m : tmax - m > 126.f ? ceilf(tmax) : m + ceilf(tmax - m);
                    const float d = m_new - m;  // 0 where the reference stays, infinite where there was none
                    const float alpha = d > 126.f ? 0.f : __uint_as_float((uint32_t)(127 - (int)d) << 23);
                    m = m_new;
                    l *= alpha;
                    exp_pass(m == -INFINITY ? 0.f : -m);
                    sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                    if (t > 0) {
                        // O must hold the tile before, too.  (P V(t - 2) is complete, P V(t) not issued:
                        // the parity is unambiguous although other phases go unobserved.)
                        if (C == 1 && !wait_all(o_done, (n - 1) & 1u)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < kD / 16; ++k) {
                            uint32_t o[16];
                            tmem_ld16(trow + kTmO + 16 * k, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st16(trow + kTmO + 16 * k, o);
                        }
                    }
                }
            }
            l += sum;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[sb]);
        }
        // -------------------------------------------------------- epilogue
        // (every warp waits: Q, which S reads, is free then, too)
        ok = ok && wait_all(o_last, n_seg & 1u);
        ++n_seg;
        tc_fence_after();
        const bool whole = nt == nt_unit;
        // a segment of a unit leaves a partial: the CTA's first segment in its first slot, its last in the second
        const size_t part = ((size_t)blockIdx.x * 2 + (is_first ? 0 : 1)) * kRows + r;
        float L = l, scale_o = 1.f;
        // the row's statistics are final: a partial, or the sink's share and the norm
        auto finish_row = [&](bool write) {
            if (!whole) {
                if (write) *reinterpret_cast<float2 *>(p.ws_ml + part * 2) = make_float2(m, L);
                return;
            }
            // m starts next to the sink and only grows
            L += sink2 == -INFINITY ? 0.f : ex2(sink2 - m);
            scale_o = L > 0.f ? 1.f / L : 0.f;
            if (write) p.lse[at] = L > 0.f ? (m + log2f(L)) * kLn2 : -INFINITY;
        };
        // 8 columns of the row from column d on
        auto store_o = [&](int d, const float *o) {
            if (!whole) {
                float4 *dst = reinterpret_cast<float4 *>(p.ws_o + part * kD + d);
                dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                dst[1] = make_float4(o[4], o[5], o[6], o[7]);
            } else {
                *reinterpret_cast<uint4 *>(p.out + at * kD + d) =
                    make_uint4(pack_bf16x2(o[0] * scale_o, o[1] * scale_o), pack_bf16x2(o[2] * scale_o, o[3] * scale_o),
                               pack_bf16x2(o[4] * scale_o, o[5] * scale_o), pack_bf16x2(o[6] * scale_o, o[7] * scale_o));
            }
        };
        auto load_o = [&](int k, float (&o)[16]) {  // 16 columns of O
            uint32_t x[16];
            tmem_ld16(trow + kTmO + 16 * k, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(x[e]);
        };
        if (C == 1) {
            if (ok && active) {
                if (valid) finish_row(true);
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    float o[16];
                    load_o(k, o);
                    if (valid) {
                        store_o(16 * k, o);
                        store_o(16 * k + 8, o + 8);
                    }
                }
            }
        } else {
            // The copies of a row join through shared memory, 32 columns at a time (element c of a row at c ^ row:
            // no bank conflicts); thread (row, copy) takes the copy-th part of them.  The barriers are
            // reached by all 128 threads, after an expired wait too.
            float *red = reinterpret_cast<float *>(smem + kOffRed);
            float2 *ml = reinterpret_cast<float2 *>(smem + kOffMl);
            if (!ok) *abort_flag = 1;
            ml[lrow] = make_float2(m, l);
            float f[C];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (ok && active) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float o[16];
                        load_o(2 * half + k, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) red[lrow * 32 + ((16 * k + e) ^ lane)] = o[e];
                    }
                }
                named_bar_sync(1, 128);
                if (*abort_flag == 0 && valid) {
                    if (half == 0) {
                        m = -INFINITY;
#pragma unroll
                        for (int k = 0; k < C; ++k) {
                            f[k] = ml[k * kRows + r].x;
                            m = fmaxf(m, f[k]);
                        }
                        L = 0.f;
#pragma unroll
                        for (int k = 0; k < C; ++k) {
                            f[k] = f[k] == -INFINITY ? 0.f : ex2(f[k] - m);
                            L = fmaf(f[k], ml[k * kRows + r].y, L);
                        }
                        finish_row(copy == 0);
                    }
#pragma unroll
                    for (int x = 0; x < 32 / C / 8; ++x) {
                        const int d = copy * (32 / C) + 8 * x;
                        float o[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
                        for (int k = 0; k < C; ++k)
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                o[e] = fmaf(f[k], red[(k * kRows + r) * 32 + ((d + e) ^ (r & 31))], o[e]);
                        store_o(32 * half + d, o);
                    }
                }
                named_bar_sync(1, 128);
            }
        }
        // all 128 threads go on or none does: the next segment has barriers among them
        return !named_bar_or(1, 128, !ok);
        });
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 6) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmCols);
    }
}

}  // namespace

namespace {

// One warp per (token, query head) of sequence blockIdx.y, for units that were cut: M = max(sink, max_c m_c),
// L = 2^(sink - M) + sum_c l_c 2^(m_c - M), o = sum_c 2^(m_c - M) o_c / L, the pieces in the order of their keys.
__global__ void __launch_bounds__(128) tree_join_kernel(const TreeTcParams p)
{
    grid_dep_launch();  // the next call's set-up beside this kernel: 4 sequences of 4 tokens 18.4 -> 17.2 us a call
    grid_dep_wait();    // the partials and the plan of the grid ahead (programmatic dependent launch)
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const int w = blockIdx.x * 4 + (threadIdx.x >> 5);  // (token, head) of the sequence
    const SeqRows sr = seq_rows(p.s.cu_q, b, 0, p.s.total_q);
    if (w >= min(sr.len, p.s.max_q) * p.s.Hq) return;
    const int tok = w / p.s.Hq, h = w - tok * p.s.Hq, g = row_token(p, h), row = tok * p.G + h - g * p.G;
    const int per_tile = kM / p.copies, rt = row / per_tile, r = row - rt * per_tile;
    const int team_head = p.head_groups == 1 ? g : g % p.heads;
    const long long q = p.plan[0], base = p.plan[1 + b], all = p.plan[2 + b] - base;
    const long long nt = p.head_groups == 1 ? all : div64(all, p.head_groups);
    const long long u0 = base + (p.head_groups == 1 ? 0 : g / p.heads * nt);  // the unit's first tile
    const int j0 = (int)div64(u0, q), j1 = (int)div64(u0 + nt - 1, q);        // the teams it was cut over
    if (j0 == j1) return;  // written in one piece
    auto slot = [&](int j) -> size_t {
        const int second = j == j0 && u0 != j0 * q;  // not the first segment of its CTA
        return ((size_t)((j * p.heads + team_head) * p.row_tiles + rt) * 2 + second) * per_tile + r;
    };
    const float sk = p.s.sinks[h] * kLog2e;
    float M = sk;
    for (int j = j0 + lane; j <= j1; j += 32) M = fmaxf(M, p.ws_ml[slot(j) * 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    float2 acc = make_float2(0.f, 0.f);
    for (int jb = j0; jb <= j1; jb += 32) {
        float f = 0.f;  // weight of piece jb + lane
        if (jb + lane <= j1) {
            const float2 ml = *reinterpret_cast<const float2 *>(p.ws_ml + slot(jb + lane) * 2);
            f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
            L = fmaf(f, ml.y, L);
        }
        const int n = min(32, j1 - jb + 1);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, k);
            const float2 o = reinterpret_cast<const float2 *>(p.ws_o + slot(jb + k) * kD)[lane];
            acc.x = fmaf(fk, o.x, acc.x);
            acc.y = fmaf(fk, o.y, acc.y);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    L += sk == -INFINITY ? 0.f : ex2(sk - M);
    const float inv = L > 0.f ? 1.f / L : 0.f;
    const size_t at = (size_t)sr.row0 * p.s.Hq + w;
    reinterpret_cast<uint32_t *>(p.out + at * kD)[lane] = pack_bf16x2(acc.x * inv, acc.y * inv);
    if (lane == 0) p.lse[at] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

// How the line is cut, from what the host knows.
struct TreePlan {
    int copies, row_tiles, heads, teams, q_min, snap;
    size_t plan_bytes, ml_floats, o_floats;
};
TreePlan tree_plan(const TreeShape &s, int num_splits)
{
    TreePlan t;
    const long long rows = (long long)s.max_q * (s.Hq / s.Hkv);
    t.copies = rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
    t.row_tiles = (int)((rows * t.copies + kM - 1) / kM);
    // tiles of the longest possible unit
    const long long lw = s.window > 0 ? (long long)s.window - 1 + s.max_q + kBN - 1 : (long long)s.Lmax;
    const long long most = ((lw < s.Lmax ? lw : s.Lmax) + kBN - 1) / kBN;
    t.snap = num_splits == 0 && most <= kTreeSnapTiles;
    // all KV heads in a team, or the largest part of them that keeps nine SMs of ten busy
    const int fit = 148 * kCtasPerSm;
    t.heads = 1;
    for (int h = s.Hkv; h >= 1; --h) {
        const long long team = (long long)h * t.row_tiles;
        if (s.Hkv % h == 0 && team <= fit && fit / team * team * 10 >= fit * 9) {
            t.heads = h;
            break;
        }
    }
    const long long line = most * (s.Hkv / t.heads) * s.B;
    long long teams = fit / ((long long)t.heads * t.row_tiles);
    t.q_min = kTreeMinTiles;
    if (num_splits > 0) {
        t.q_min = (int)((most + num_splits - 1) / num_splits);
        teams = (line + t.q_min - 1) / t.q_min;
        const long long cap = 4096 / t.heads;  // (the stretches are then longer)
        if (teams > cap) teams = cap;
    }
    const long long useful = t.snap ? line : (line + t.q_min - 1) / t.q_min;
    if (teams > useful) teams = useful;
    t.teams = (int)(teams < 1 ? 1 : teams);
    const size_t slots = t.snap ? 0 : (size_t)t.teams * t.heads * t.row_tiles * 2 * (kM / t.copies);
    t.plan_bytes = t.snap ? 0 : ((size_t)s.B + 2) * 8 + 15 & ~(size_t)15;
    t.ml_floats = slots * 2;
    t.o_floats = slots * kD;
    return t;
}

}  // namespace

size_t tree_tc_workspace_bytes(const TreeShape &s, int num_splits)
{
    const TreePlan t = tree_plan(s, num_splits);
    return t.plan_bytes + (t.ml_floats + t.o_floats) * sizeof(float);
}

cudaError_t launch_tree_tc(const void *q, const void *kc, const void *vc, void *out, float *lse, const TreeShape &s,
                           int num_splits, void *ws, cudaStream_t st)
{
    const TreePlan t = tree_plan(s, num_splits);
    TreeTcParams p;
    p.s = s;
    p.G = s.Hq / s.Hkv;
    p.g_magic = p.G > 1 ? (unsigned)((0x100000000ull + p.G - 1) / p.G) : 0;
    p.page_shift = -1;
    for (int x = 3; x < 31; ++x)
        if (s.page_size == 1 << x) p.page_shift = x;
    p.copies = t.copies;
    p.row_tiles = t.row_tiles;
    p.heads = t.heads;
    p.head_groups = s.Hkv / t.heads;
    p.teams = t.teams;
    p.q_min = t.q_min;
    p.snap = t.snap;
    p.box_rows = s.page_size > 0 && s.page_size < kBN ? s.page_size : kBN;
    p.c_log2 = s.scale * kLog2e;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.plan = t.snap ? nullptr : static_cast<long long *>(ws);
    p.ws_o = t.snap ? nullptr : reinterpret_cast<float *>(static_cast<char *>(ws) + t.plan_bytes);
    p.ws_ml = t.snap ? nullptr : p.ws_o + t.o_floats;
    p.status = device_status_ptr();
    p.timeout_ns = wait_timeout_ns();
    const long long ctas = (long long)t.teams * t.heads * t.row_tiles;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    alignas(64) CUtensorMap mk, mv;
    // contiguous: [B][Lmax][Hkv][64]; paged pool: [num_pages][page_size][Hkv][64]
    const bool paged = s.page_size > 0;
    const uint64_t krows = paged ? (uint64_t)s.page_size : (uint64_t)s.Lmax;
    const uint64_t dims[4] = {(uint64_t)kD, (uint64_t)s.Hkv, krows, paged ? (uint64_t)s.num_pages : (uint64_t)s.B};
    const uint64_t strides[3] = {(uint64_t)kD * 2, (uint64_t)s.Hkv * kD * 2, krows * s.Hkv * kD * 2};
    const uint32_t box[4] = {(uint32_t)kD, 1u, (uint32_t)p.box_rows, 1u};
    if (!encode_tensor_map_4d(&mk, const_cast<void *>(kc), 2, dims, strides, box, true) ||
        !encode_tensor_map_4d(&mv, const_cast<void *>(vc), 2, dims, strides, box, true))
        return cudaErrorInvalidValue;
    auto kern = t.copies == 4 ? tree_tc_kernel<4> : t.copies == 2 ? tree_tc_kernel<2> : tree_tc_kernel<1>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    e = launch_chained(kern, dim3((unsigned)ctas), kThreads, kSmemBytes, st, mk, mv, p);
    if (e != cudaSuccess || t.snap) return e;
    return launch_chained(tree_join_kernel, dim3((unsigned)(((long long)s.max_q * s.Hq + 3) / 4), (unsigned)s.B), 128, 0,
                          st, p);
}

}  // namespace attn_sink
