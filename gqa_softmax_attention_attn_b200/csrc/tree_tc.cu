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
// byte, T G 64 flop a byte: with up to 128 rows a KV head the kernel is bound by
// HBM, beyond that by the softmax (one exponential per 256 flop).
//  * CTA = (row tile, KV head, split, sequence); row tiles of one chunk and the
//    KV heads of one token range are neighbours in the grid, so their K/V rows
//    meet in L2.  Two CTAs per SM (256 TMEM columns each).
//  * A row tile is 128 / C rows, held C times in the 128 lanes of the MMA tile
//    (C = 4, 2, 1 for up to 32, 64, more rows): copy k's threads take the
//    k-th part of every tile's keys and write zeros of P elsewhere, once, so
//    that few rows still keep all four softmax warps busy and each has 1/C of
//    the exponentials in its dependent chain; the copies' sums join through
//    shared memory at the end.  The tensor pipe does C times the work, of
//    which it has plenty to spare while HBM is the limit.
//  * Warp 0 streams K and V in tiles of 64 keys (128-byte-swizzled TMA boxes, one
//    a page for small pages, issued by as many lanes) through a ring of kNS
//    stages; warp 1 issues S = Q K^T into a double-buffered TMEM tile and O += P V
//    with P from TMEM; warps 2-5, one row (copy) a thread, do the softmax.
//  * Masks: a thread's visible keys of a tile are one 64-bit word -- the cached
//    prefix as a range, the drafted keys as the row's ancestor bits shifted
//    into place -- and only tiles some row does not see in full apply it.
//  * Key and value rows no row of the sequence sees may hold anything: their
//    scores are selected away, their V rows zeroed in shared memory.
//  * Every wait is bounded; on expiry the CTA raises the device status bit, waits
//    (bounded) for its own loads and MMAs, frees tensor memory and exits.
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
constexpr int kNS = 5;  // K/V ring stages
constexpr int kThreads = 192;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// a tile whose exponentials sum past this moves the row's reference maximum
constexpr float kSumLimit = 1024.f;

constexpr int kTileBytes = kBN * kD * 2;
constexpr int kOffQ = 0;
constexpr int kOffK = kM * kD * 2;
constexpr int kOffV = kOffK + kNS * kTileBytes;
constexpr int kOffPath = kOffV + kNS * kTileBytes;                 // [128][kPathWords] ancestor bits
constexpr int kOffDepth = kOffPath + kM * kPathWords * 4;          // [128] depths
constexpr int kOffPar = kOffDepth + kM * 2;                        // [256] parents
constexpr int kOffBar = kOffPar + kTreeMaxTokens * 2;
// q_full, k_full[], k_empty[], v_full[], v_empty[], s_full[2], p_full[2], o_done, drain
constexpr int kNumBar = 1 + 4 * kNS + 4 + 2;
constexpr int kOffMisc = kOffBar + kNumBar * 8;                    // TMEM address, abort flag
constexpr int kSmemBytes = kOffMisc + 16 + 1024;
constexpr int kRedStride = 67;                                     // floats a row of the copies' exchange
static_assert(kM * kRedStride * 4 <= 2 * kNS * kTileBytes, "the exchange reuses the K/V ring");
static_assert(kOffBar % 8 == 0, "barriers on 8 bytes");
// tensor memory: S and P double-buffered, O
constexpr int kTmS = 0, kTmP = 2 * kBN, kTmO = kTmP + kBN, kTmCols = 256;
static_assert(kTmO + kD <= kTmCols, "tensor memory");

struct TreeTcParams {
    TreeShape s;
    int G, row_tiles, box_rows;
    float c_log2;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    float *lse, *ws_o, *ws_ml;
    unsigned *status;
    long long timeout_ns;
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
__global__ void __launch_bounds__(kThreads, 2)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const TreeTcParams p)
{
    grid_dep_launch();  // the combine may start its set-up; it waits for this grid
    constexpr int kRows = kM / C;  // rows of a tile
    constexpr int kC = kBN / C;    // keys of a tile per thread
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *k_full = q_full + 1, *k_empty = k_full + kNS, *v_full = k_empty + kNS, *v_empty = v_full + kNS;
    uint64_t *s_full = v_empty + kNS, *p_full = s_full + 2, *o_done = p_full + 2, *drain = o_done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int rest = blockIdx.x;
    const int rt = rest % p.row_tiles;
    rest /= p.row_tiles;
    const int g = rest % p.s.Hkv;
    rest /= p.s.Hkv;
    const int c = rest % p.s.splits, b = rest / p.s.splits;
    const TreeSeq sq = tree_seq(p.s, b);
    const int rows = min(sq.T, p.s.max_q) * p.G, r0 = rt * kRows;
    if (c >= sq.nsplit || r0 >= rows) return;  // uniform over the CTA
    const int nrow = min(kRows, rows - r0);
    const int kbeg = sq.lo_al + c * p.s.chunk;
    const int kend = min((long long)sq.len, (long long)kbeg + p.s.chunk);
    const int n_tiles = kend > kbeg ? (kend - kbeg + kBN - 1) / kBN : 0;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 128);
        for (int i = 0; i < kNS; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
        }
        mbar_init(o_done, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer (the whole warp)
        const int nb = kBN / p.box_rows;  // boxes of a tile, one lane each for K and V
        const int box = lane % nb, is_v = lane / nb;
        const int batch = 32 / nb;        // tiles whose page entries one load per lane fetches
        const int ps = p.s.page_size;
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        int page = 0, t = 0;
        for (; t < n_tiles; ++t) {
            const int st = t % kNS;
            const uint32_t ph = (uint32_t)(t / kNS) & 1u;
            if (ps > 0 && t % batch == 0) {
                // the next 32 boxes' pages; boxes behind the sequence (masked) reuse its last page, so
                // the table is only read within the sequence's own entries
                const int key = min(kbeg + t * kBN + lane * p.box_rows, sq.len - 1);
                page = p.s.page_table[(size_t)b * p.s.max_pages + key / ps];
            }
            const int my_page = __shfl_sync(0xffffffffu, page, (t % batch) * nb + box);
            if (!__all_sync(0xffffffffu, mbar_wait(&k_empty[st], ph ^ 1u, abort_flag, p.status, p.timeout_ns) &&
                                             mbar_wait(&v_empty[st], ph ^ 1u, abort_flag, p.status, p.timeout_ns)))
                break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&k_full[st], kTileBytes);
                mbar_arrive_expect_tx(&v_full[st], kTileBytes);
            }
            __syncwarp();
            if (is_v < 2) {
                const int key = kbeg + t * kBN + box * p.box_rows;
                uint8_t *dst = smem + (is_v ? kOffV : kOffK) + st * kTileBytes + box * p.box_rows * kD * 2;
                tma_load_4d(dst, is_v ? &tmV : &tmK, 0, g, ps > 0 ? key % ps : key, ps > 0 ? my_page : b,
                            is_v ? &v_full[st] : &k_full[st]);
            }
        }
        // every load issued must land before the CTA may exit
        for (int st = 0; st < kNS && st < t; ++st) {
            const uint32_t ph = (uint32_t)((t - 1 - st) / kNS) & 1u;
            wait_noabort(&k_full[st], ph, p.status, p.timeout_ns);
            wait_noabort(&v_full[st], ph, p.status, p.timeout_ns);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (converged, one lane issues)
        const uint32_t id_s = idesc_bf16_f32(kM, kBN, 0), id_pv = idesc_bf16_f32(kM, kD, 1);
        const uint32_t q_addr = smem_u32(smem + kOffQ), k_addr = smem_u32(smem + kOffK);
        auto wait_all = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, p.timeout_ns));
        };
        // O += P(t) V(t)
        auto issue_pv = [&](int t) -> bool {
            const int sb = t & 1, st = t % kNS;
            if (!wait_all(&p_full[sb], (uint32_t)(t >> 1) & 1u)) return false;
            if (!wait_all(&v_full[st], (uint32_t)(t / kNS) & 1u)) return false;
            uint8_t *vt = smem + kOffV + st * kTileBytes;
            const int j0 = kbeg + t * kBN;
            if (j0 < sq.lo || j0 + kBN > sq.len) {
                // value rows no row sees may hold anything (0 x NaN is NaN): zeros
                for (int e = lane; e < kBN * 8; e += 32) {
                    const int j = j0 + (e >> 3);
                    if (j < sq.lo || j >= sq.len) reinterpret_cast<uint4 *>(vt)[e] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            tc_fence_after();
            if (elect_one()) {
                const uint32_t va = smem_u32(vt);
#pragma unroll
                for (int kk = 0; kk < kBN / 16; ++kk)
                    mma_ts(tmem + kTmO, tmem + kTmP + sb * (kBN / 2) + kk * 8,
                           smem_desc_sw128(va + kk * 2048, kBN * 128, 1024), id_pv, (t > 0 || kk > 0) ? 1u : 0u);
                mma_commit(o_done);
                mma_commit(&v_empty[st]);
            }
            __syncwarp();
            return true;
        };
        bool ok = n_tiles > 0 && wait_all(q_full, 0);
        for (int t = 0; t < n_tiles && ok; ++t) {
            const int st = t % kNS, sb = t & 1;
            if (!wait_all(&k_full[st], (uint32_t)(t / kNS) & 1u)) break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t kb = k_addr + st * kTileBytes;
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk)
                    mma_ss(tmem + kTmS + sb * kBN, smem_desc_sw128(q_addr + kk * 32, 16, 1024),
                           smem_desc_sw128(kb + kk * 32, 16, 1024), id_s, kk > 0 ? 1u : 0u);
                mma_commit(&s_full[sb]);
                mma_commit(&k_empty[st]);
            }
            __syncwarp();
            if (t >= 1) ok = issue_pv(t - 1);
            if (ok && t == n_tiles - 1) ok = issue_pv(t);
        }
        if (elect_one()) mma_commit(drain);
        __syncwarp();
        wait_noabort(drain, 0, p.status, p.timeout_ns);
    } else {
        // ------------------------------------------------------------ softmax + epilogue
        const int tid = threadIdx.x - 64;
        const int quad = warp & 3;
        const int lrow = quad * 32 + lane;               // TMEM lane
        const int r = lrow % kRows, copy = lrow / kRows;  // row of the tile, copy of it
        const bool valid = r < nrow;
        const bool active = (quad * 32) % kRows < nrow;  // some row of this warp exists
        const int row = r0 + (valid ? r : 0);
        const int i0 = r0 / p.G, tok = row / p.G - i0, h = g * p.G + row % p.G;
        const size_t at = (size_t)(sq.row0 + row / p.G) * p.s.Hq + h;
        const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);

        // Q: this thread's row into the 128-byte-swizzled operand tile (rows that do not exist: zeros)
        {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.q + at * kD);
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = valid ? src[k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4 *>(smem + kOffQ + lrow * 128 + ((k ^ (lrow & 7)) << 4)) = v[k];
            fence_proxy_async_smem();
            mbar_arrive(q_full);
        }
        if (C > 1) {
            // P of the keys of the other copies stays zero
            uint32_t z[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) z[k] = 0u;
#pragma unroll
            for (int k = 0; k < kBN / 16; ++k) tmem_st16(trow + kTmP + 16 * k, z);
        }
        const float sink2 = p.s.sinks[h] * kLog2e;
        float m = sink2;  // reference maximum, log2 units: the sink's, until a tile moves it
        float l = 0.f;    // running sum, without the sink
        uint32_t(*path)[kPathWords] = reinterpret_cast<uint32_t(*)[kPathWords]>(smem + kOffPath);
        int16_t *depth = reinterpret_cast<int16_t *>(smem + kOffDepth);
        int vis_lo = 0;  // first cached key this row sees
        if (p.s.window > 0 || kend > sq.cached) {
            tree_paths(p.s, sq, i0, (r0 + nrow - 1) / p.G - i0 + 1, tid, 128,
                       reinterpret_cast<int16_t *>(smem + kOffPar), path, depth, [] { named_bar_sync(1, 128); });
            if (p.s.window > 0) vis_lo = max(0, sq.cached + depth[tok] - p.s.window + 1);
        }
        const float2 C2 = make_float2(p.c_log2, p.c_log2);
        bool ok = true;
        for (int t = 0; t < n_tiles; ++t) {
            const int sb = t & 1;
            if (!__all_sync(0xffffffffu,
                            mbar_wait(&s_full[sb], (uint32_t)(t >> 1) & 1u, abort_flag, p.status, p.timeout_ns))) {
                ok = false;
                break;
            }
            if (!active) {  // no row here: P's values do not matter, only its barrier
                mbar_arrive(&p_full[sb]);
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
            const int j0 = kbeg + t * kBN;
            const bool edge = j0 < vis_lo || j0 + kBN > sq.cached;
            if (__any_sync(0xffffffffu, edge)) {
                uint64_t see = range_bits(vis_lo - j0, sq.cached - j0);
                if (j0 + kBN > sq.cached)
                    see |= path_bits(path[tok], j0 - sq.cached) & range_bits(0, sq.len - j0);
                see >>= copy * kC;
                const uint32_t see0 = (uint32_t)see, see1 = (uint32_t)(see >> 32);
#pragma unroll
                for (int k = 0; k < kC; ++k)
                    sv[k] = ((k < 32 ? see0 : see1) >> (k & 31)) & 1u ? sv[k] : -INFINITY;
            }
            // P = exp2(S C - m) against the reference maximum, without looking for the tile's: every
            // exponential is at most their sum, and a sum within kSumLimit (NaN fails the test) keeps
            // the reference
            float2 acc[2];
            auto exp_pass = [&](float neg_m) {
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
                    tmem_st8(trow + kTmP + sb * (kBN / 2) + copy * (kC / 2) + 8 * k, pk);
                }
            };
            exp_pass(m == -INFINITY ? 0.f : -m);
            float tsum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
            const bool big = !(tsum <= kSumLimit) || m == -INFINITY;
            bool rescale = false;
            float alpha = 1.f;
            if (__any_sync(0xffffffffu, big)) {
                float mx[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) mx[k] = -INFINITY;
#pragma unroll
                for (int k = 0; k < kC; k += 16)
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx[e] = fmax3(mx[e], sv[k + e], sv[k + 8 + e]);
                const float tmax = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                const float m_new = fmaxf(m, tmax * p.c_log2);
                rescale = big && m_new > m;
                if (__any_sync(0xffffffffu, rescale)) {
                    if (rescale) {
                        alpha = m == -INFINITY ? 0.f : ex2(m - m_new);
                        m = m_new;
                    }
                    exp_pass(m == -INFINITY ? 0.f : -m);
                    tsum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                }
            }
            l = l * alpha + tsum;
            if (t > 0) {
                // O holds the products of the tiles before once P V(t - 1) completes; waited on at every
                // tile, so that the parity is never more than one phase behind
                if (!__all_sync(0xffffffffu,
                                mbar_wait(o_done, (uint32_t)(t - 1) & 1u, abort_flag, p.status, p.timeout_ns))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (__any_sync(0xffffffffu, rescale)) {
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
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_full[sb]);
        }
        if (ok && active && n_tiles > 0)
            ok = __all_sync(0xffffffffu, mbar_wait(o_done, (uint32_t)(n_tiles - 1) & 1u, abort_flag, p.status,
                                                   p.timeout_ns));
        // -------------------------------------------------------- epilogue
        constexpr int kOut = kD / C;  // output columns of a thread: [copy kOut, + kOut)
        float o[kD];
        if (ok && active && n_tiles > 0) {
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kD / 16; ++k) {
                uint32_t x[16];
                tmem_ld16(trow + kTmO + 16 * k, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[16 * k + e] = __uint_as_float(x[e]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kD; ++k) o[k] = 0.f;
        }
        if (C > 1) {
            // the copies' statistics and sums join, each thread its part of the columns.  Every load
            // and product of the ring has completed: it is free.
            // (an expired wait leaves the exchange unused: the barrier below is reached by all 128)
            float *red = reinterpret_cast<float *>(smem + kOffK);
            if (active) {
                float *me = red + lrow * kRedStride;
#pragma unroll
                for (int k = 0; k < kD; ++k) me[k] = o[k];
                me[kD] = m;
                me[kD + 1] = l;
            }
            if (!ok) *abort_flag = 1;
            named_bar_sync(1, 128);
            if (*abort_flag) ok = false;
            if (ok && active) {
                float M = -INFINITY;
#pragma unroll
                for (int k = 0; k < C; ++k) M = fmaxf(M, red[(k * kRows + r) * kRedStride + kD]);
                l = 0.f;
#pragma unroll
                for (int e = 0; e < kOut; ++e) o[e] = 0.f;
#pragma unroll
                for (int k = 0; k < C; ++k) {
                    const float *you = red + (k * kRows + r) * kRedStride;
                    const float f = you[kD] == -INFINITY ? 0.f : ex2(you[kD] - M);
                    l = fmaf(f, you[kD + 1], l);
#pragma unroll
                    for (int e = 0; e < kOut; ++e) o[e] = fmaf(f, you[copy * kOut + e], o[e]);
                }
                m = M;
            }
        }
        if (ok && valid) {
            if (sq.nsplit == 1) {
                // m starts at the sink, so it is the larger of the two
                const float L = l + (sink2 == -INFINITY ? 0.f : ex2(sink2 - m));
                const float inv = L > 0.f ? 1.f / L : 0.f;
                uint4 *dst = reinterpret_cast<uint4 *>(p.out + at * kD + copy * kOut);
#pragma unroll
                for (int k = 0; k < kOut / 8; ++k)
                    dst[k] = make_uint4(pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv),
                                        pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                        pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                                        pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
                if (copy == 0) p.lse[at] = L > 0.f ? (m + log2f(L)) * kLn2 : -INFINITY;
            } else {
                const size_t slot = at * p.s.splits + c;
                float4 *dst = reinterpret_cast<float4 *>(p.ws_o + slot * kD + copy * kOut);
#pragma unroll
                for (int k = 0; k < kOut / 4; ++k)
                    dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                if (copy == 0) {
                    p.ws_ml[slot * 2] = m;
                    p.ws_ml[slot * 2 + 1] = l;
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmCols);
    }
}

}  // namespace

cudaError_t launch_tree_tc(const void *q, const void *kc, const void *vc, void *out, float *lse, const TreeShape &s,
                           float *ws_o, float *ws_ml, cudaStream_t st)
{
    TreeTcParams p;
    p.s = s;
    p.G = s.Hq / s.Hkv;
    const long long rows = (long long)s.max_q * p.G;
    const int copies = rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
    p.row_tiles = (int)((rows * copies + kM - 1) / kM);
    p.box_rows = s.page_size > 0 && s.page_size < kBN ? s.page_size : kBN;
    p.c_log2 = s.scale * kLog2e;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.ws_o = ws_o;
    p.ws_ml = ws_ml;
    p.status = device_status_ptr();
    p.timeout_ns = wait_timeout_ns();
    const long long ctas = (long long)p.row_tiles * s.Hkv * s.splits * s.B;
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
    auto kern = copies == 4 ? tree_tc_kernel<4> : copies == 2 ? tree_tc_kernel<2> : tree_tc_kernel<1>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)ctas, kThreads, kSmemBytes, st>>>(mk, mv, p);
    return cudaGetLastError();
}

}  // namespace attn_sink
