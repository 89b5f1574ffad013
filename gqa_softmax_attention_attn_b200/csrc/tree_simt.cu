// tree_simt.cu -- decode of a tree of drafted tokens per sequence on the CUDA
// cores (the exact fp32 path), and the combine of its splits.
//
// Row (token i, query head h) of sequence b sits at position p = cached +
// depth(i), sees the cached keys j > p - window and, among the drafted tokens'
// own keys (the sequence's last), those of its ancestors and itself fewer than
// `window` levels up; its softmax carries the head's sink:
//   m = max_j s_j, l = sum_j exp(s_j - m), o = sum_j exp(s_j - m) v_j
// per split of the keys, in log2 units and without the sink, which joins once
// in the combine (or here, when a sequence needs one split).
//
// CTA = (16 rows of one KV head, split, sequence): keys in tiles of 32, lane =
// key for the scores and lane = (d, d + 32) for the output, so that K and V
// are read once for 16 rows.  Every score and sum is fp32, each exponential
// exp2f.  A warp's four rows go side by side (16 sequences of 61 tokens, 6 query and
// 2 KV heads, 2000 to 4000 keys: 608 -> 412 us, 11 TFLOP/s; with 64 and 8 heads 3924 us,
// 12 TFLOP/s, against 74 at two flop a lane and cycle).  Where rows are many, bound by issue:
// the products of Q K^T feed on shared memory, and two FMAs of P V bring a shuffle
// and two selects with them.  Where they are few, bound by the latency of
// a tile's chain, so the keys are cut into chunks of a single tile if need be
// until there are sixteen CTAs an SM, of which it runs four at a time (128 registers a
// thread): 3 sequences of 7 tokens 12.3 us a call on the
// device, 60 us a call in chunks of 16 tiles.
#include <cuda_bf16.h>
#include <math.h>

#include "kernels.h"
#include "sm100_ptx.cuh"
#include "tree_path.cuh"

namespace attn_sink {
namespace {

constexpr int kD = 64;
constexpr int kRows = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float warp_max(float x)
{
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float warp_sum(float x)
{
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// element offset of (key j, KV head g) in a cache, or -1 (a page outside the pool: zeros)
__device__ __forceinline__ long long kv_offset(const TreeShape &s, int b, int j, int g)
{
    if (s.page_size == 0) return (((long long)b * s.Lmax + j) * s.Hkv + g) * kD;
    const int page = s.page_table[(size_t)b * s.max_pages + j / s.page_size];
    if (page < 0 || page >= s.num_pages) return -1;
    return (((long long)page * s.page_size + j % s.page_size) * s.Hkv + g) * kD;
}

__global__ void __launch_bounds__(128) tree_simt_kernel(const float *q, const float *kc, const float *vc, float *out,
                                                        float *lse, float *ws_o, float *ws_ml, const TreeShape s,
                                                        int row_tiles)
{
    grid_dep_launch();  // the combine may start its set-up; it waits for this grid
    grid_dep_wait();    // (as this one for the grid ahead)
    __shared__ __align__(16) float qs[kRows][kD];
    __shared__ float ks[32][kD + 1];
    __shared__ __align__(16) float vs[32][kD];
    __shared__ int16_t par[kTreeMaxTokens], depth[kRows];
    __shared__ uint32_t path[kRows][kPathWords];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rt = blockIdx.x % row_tiles, rest = blockIdx.x / row_tiles;
    const int g = rest % s.Hkv, c = rest / s.Hkv % s.splits, b = rest / s.Hkv / s.splits;
    const int G = s.Hq / s.Hkv;
    const TreeSeq sq = tree_seq(s, b);
    const int nsplit = tree_splits(s, sq);
    const int rows = min(sq.T, s.max_q) * G, r0 = rt * kRows;
    if (c >= nsplit || r0 >= rows) return;  // uniform over the CTA
    const int nrow = min(kRows, rows - r0);
    const int kbeg = max(sq.lo, sq.lo_al + c * s.chunk), kend = min(sq.len, sq.lo_al + (c + 1) * s.chunk);

    // a tile's K and V, a quarter of a key's row a thread, loaded a tile ahead (the first beside the paths and q)
    const int jj0 = tid >> 2, d0 = (tid & 3) * 16;
    float4 kv[4], vv[4];
    auto load = [&](int j0) {
        const long long at = j0 + jj0 < kend ? kv_offset(s, b, j0 + jj0, g) : -1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            kv[e] = at >= 0 ? *reinterpret_cast<const float4 *>(kc + at + d0 + 4 * e) : make_float4(0.f, 0.f, 0.f, 0.f);
            vv[e] = at >= 0 ? *reinterpret_cast<const float4 *>(vc + at + d0 + 4 * e) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    load(kbeg);
    const int i0 = r0 / G, ntok = (r0 + nrow - 1) / G - i0 + 1;
    tree_paths(s, sq, i0, ntok, tid, 128, par, path, depth, [] { __syncthreads(); });
    for (int e = tid; e < nrow * kD; e += 128) {
        const int r = r0 + e / kD;
        qs[e / kD][e % kD] = q[((size_t)(sq.row0 + r / G) * s.Hq + g * G + r % G) * kD + e % kD];
    }

    float m[4], l[4], o0[4], o1[4];
    int tok[4], vis_lo[4];
#pragma unroll
    for (int rr = 0; rr < 4; ++rr) {
        m[rr] = -INFINITY;
        l[rr] = o0[rr] = o1[rr] = 0.f;
        const int r = min(r0 + warp * 4 + rr, rows - 1);
        tok[rr] = r / G - i0;
        vis_lo[rr] = s.window > 0 ? sq.cached + depth[tok[rr]] - s.window + 1 : 0;
    }
    const float C = s.scale * kLog2e;
    for (int j0 = kbeg; j0 < kend; j0 += 32) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float *k = &ks[jj0][d0 + 4 * e];
            k[0] = kv[e].x;
            k[1] = kv[e].y;
            k[2] = kv[e].z;
            k[3] = kv[e].w;
            *reinterpret_cast<float4 *>(&vs[jj0][d0 + 4 * e]) = vv[e];
        }
        __syncthreads();
        if (j0 + 32 < kend) load(j0 + 32);
        // the warp's four rows side by side (rows that do not exist are computed and not stored): each K and V
        // value is read once for them, and their reductions overlap
        const int j = j0 + lane, a = j - sq.cached;
        float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int d = 0; d < kD; d += 4) {
            float4 q4[4];
#pragma unroll
            for (int rr = 0; rr < 4; ++rr) q4[rr] = *reinterpret_cast<const float4 *>(&qs[warp * 4 + rr][d]);
            const float k0 = ks[lane][d], k1 = ks[lane][d + 1], k2 = ks[lane][d + 2], k3 = ks[lane][d + 3];
#pragma unroll
            for (int rr = 0; rr < 4; ++rr)
                sc[rr] = fmaf(q4[rr].w, k3, fmaf(q4[rr].z, k2, fmaf(q4[rr].y, k1, fmaf(q4[rr].x, k0, sc[rr]))));
        }
        float pj[4];
#pragma unroll
        for (int rr = 0; rr < 4; ++rr) {
            bool see = j < kend && j >= vis_lo[rr];
            if (a >= 0) see = j < kend && a < kTreeMaxTokens && ((path[tok[rr]][a >> 5] >> (a & 31)) & 1u);
            const float x = see ? sc[rr] * C : -INFINITY;
            const float mn = fmaxf(m[rr], warp_max(x));
            const float sub = mn == -INFINITY ? 0.f : mn;  // no finite score so far
            const float alpha = m[rr] == -INFINITY ? 0.f : exp2f(m[rr] - sub);
            pj[rr] = see ? exp2f(x - sub) : 0.f;
            l[rr] = l[rr] * alpha + warp_sum(pj[rr]);
            o0[rr] *= alpha;
            o1[rr] *= alpha;
            m[rr] = mn;
        }
#pragma unroll 8
        for (int jj = 0; jj < 32; ++jj) {
            const float v0 = vs[jj][lane], v1 = vs[jj][lane + 32];
#pragma unroll
            for (int rr = 0; rr < 4; ++rr) {
                const float w = __shfl_sync(0xffffffffu, pj[rr], jj);
                // a key the row does not see stays out, whatever its value row holds
                o0[rr] = w != 0.f ? fmaf(w, v0, o0[rr]) : o0[rr];
                o1[rr] = w != 0.f ? fmaf(w, v1, o1[rr]) : o1[rr];
            }
        }
    }
#pragma unroll
    for (int rr = 0; rr < 4; ++rr) {
        const int r = r0 + warp * 4 + rr;
        if (r >= rows) continue;
        const int h = g * G + r % G;
        const size_t at = (size_t)(sq.row0 + r / G) * s.Hq + h;
        if (nsplit == 1) {
            const float sk = s.sinks[h] * kLog2e, M = fmaxf(m[rr], sk);
            const float fo = m[rr] == -INFINITY ? 0.f : exp2f(m[rr] - M);
            const float L = l[rr] * fo + (sk == -INFINITY ? 0.f : exp2f(sk - M));
            const float inv = L > 0.f ? fo / L : 0.f;
            out[at * kD + lane] = o0[rr] * inv;
            out[at * kD + lane + 32] = o1[rr] * inv;
            if (lane == 0) lse[at] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
        } else {
            const size_t slot = at * s.splits + c;
            ws_o[slot * kD + lane] = o0[rr];
            ws_o[slot * kD + lane + 32] = o1[rr];
            if (lane == 0) {
                ws_ml[slot * 2] = m[rr];
                ws_ml[slot * 2 + 1] = l[rr];
            }
        }
    }
}

// One warp per (token, query head): M = max(sink, max_c m_c), L = 2^(sink - M)
// + sum_c l_c 2^(m_c - M), o = sum_c 2^(m_c - M) o_c / L, the splits in order
// (so the result does not depend on which finished first).
__global__ void __launch_bounds__(128) tree_combine_kernel(float *out, float *lse, const float *ws_o,
                                                           const float *ws_ml, const TreeShape s)
{
    grid_dep_wait();  // the partials of the grid ahead (programmatic dependent launch)
    const TreeSeq sq = tree_seq(s, blockIdx.y);
    const int nsplit = tree_splits(s, sq);
    const int lane = threadIdx.x & 31;
    const int w = blockIdx.x * 4 + (threadIdx.x >> 5);  // (token, head) of the sequence
    if (nsplit <= 1 || w >= min(sq.T, s.max_q) * s.Hq) return;
    const size_t at = (size_t)sq.row0 * s.Hq + w, slot0 = at * s.splits;
    const float sk = s.sinks[w % s.Hq] * kLog2e;
    float mc[kTreeMaxSplits / 32], M = sk;
#pragma unroll
    for (int k = 0; k < kTreeMaxSplits / 32; ++k) {
        const int c = 32 * k + lane;
        mc[k] = c < nsplit ? ws_ml[(slot0 + c) * 2] : -INFINITY;
        M = fmaxf(M, mc[k]);
    }
    M = warp_max(M);
    float L = 0.f;
#pragma unroll
    for (int k = 0; k < kTreeMaxSplits / 32; ++k) {
        const int c = 32 * k + lane;
        mc[k] = mc[k] == -INFINITY ? 0.f : exp2f(mc[k] - M);  // from here on the split's weight
        if (c < nsplit) L += ws_ml[(slot0 + c) * 2 + 1] * mc[k];
    }
    L = warp_sum(L) + (sk == -INFINITY ? 0.f : exp2f(sk - M));
    const float inv = L > 0.f ? 1.f / L : 0.f;
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kTreeMaxSplits / 32; ++k) {
        const int n = min(32, nsplit - 32 * k);
#pragma unroll 4
        for (int c = 0; c < n; ++c) {
            const float f = __shfl_sync(0xffffffffu, mc[k], c);
            const float2 o = reinterpret_cast<const float2 *>(ws_o + (slot0 + 32 * k + c) * kD)[lane];
            acc.x = fmaf(f, o.x, acc.x);
            acc.y = fmaf(f, o.y, acc.y);
        }
    }
    reinterpret_cast<float2 *>(out + at * kD)[lane] = make_float2(acc.x * inv, acc.y * inv);
    if (lane == 0) lse[at] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

}  // namespace

cudaError_t launch_tree_simt(const float *q, const float *kc, const float *vc, float *out, float *lse,
                             const TreeShape &s, float *ws_o, float *ws_ml, cudaStream_t st)
{
    const int row_tiles = (s.max_q * (s.Hq / s.Hkv) + kRows - 1) / kRows;
    const long long ctas = (long long)row_tiles * s.Hkv * s.splits * s.B;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_chained(tree_simt_kernel, dim3((unsigned)ctas), 128, 0, st, q, kc, vc, out, lse, ws_o,
                                         ws_ml, s, row_tiles);
    if (e != cudaSuccess || s.splits <= 1) return e;
    return launch_chained(tree_combine_kernel, dim3((unsigned)(((long long)s.max_q * s.Hq + 3) / 4), (unsigned)s.B), 128,
                          0, st, out, lse, (const float *)ws_o, (const float *)ws_ml, s);
}

}  // namespace attn_sink
