// page_map.cu -- what a paged step needs to know about its requests, from their
// lengths alone: lengths and offsets for the attention calls, a position and a
// cache row for every new token, and the new pages' entries of the page table.
//
// Request b holds c_b cached tokens in ceil(c_b / ps) pages and gets n_b new
// ones.  With N_b = sum_{a < b} n_a and F_b = sum_{a < b} take_a (take_b the
// pages it needs beyond the ones it has), token i of request b is row N_b + i
// of the step, sits at position c_b + depth(i) and goes to slot
// (c_b + i) mod ps of logical page (c_b + i) / ps; its new pages are the free
// pages from F_b on.
//
// Design: launch latency is all there is (a few bytes a request and a token),
// so one kernel without a second pass: every CTA scans the requests' lengths
// itself, kChunk at a time (read from L2, two numbers a request), which costs
// less than handing sums from CTA to CTA, then fills its own kTokens tokens
// by a binary search of the scanned offsets in shared memory.  CTA 0 writes
// the per-request results, and the new pages' entries are dealt out evenly.
// Bound by latency: two dependent trips to L2, a scan over the CTA and a search
// of 10 steps.  64 requests of 8 tokens 4.9 us on the device, 1000 requests of
// mixed lengths 5.7 us (back to back from a graph; 7.0 us with the next grid let in early, whose
// waiting CTAs then share the SMs with this one's).
#include "kernels.h"
#include "sm100_ptx.cuh"

namespace attn_sink {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;                   // requests per thread and chunk
constexpr int kChunk = kThreads * kPer;   // requests scanned at a time
constexpr int kTokens = 256;              // tokens per CTA

struct MapParams {
    PageMapShape s;
    const int *cached, *fresh, *parents, *free_pages;
    int *page_table, *seqlens, *cu, *positions, *rows, *stats;
};

struct Request {
    long long len;  // cached and new tokens
    int cached, fresh, have, take;
};
__device__ __forceinline__ Request request_at(const MapParams &p, int b)
{
    Request r{0, 0, 0, 0, 0};
    if (b >= p.s.B) return r;
    r.cached = max(p.cached[b], 0);
    r.fresh = max(p.fresh[b], 0);
    r.len = (long long)r.cached + r.fresh;
    const int ps = p.s.page_size;
    r.have = (int)min((r.cached + (long long)ps - 1) / ps, (long long)p.s.max_pages);
    r.take = (int)min((r.len + ps - 1) / ps, (long long)p.s.max_pages) - r.have;
    return r;
}

// index of the last entry of a[0 .. n) at or below x (a[0] <= x, a ascending)
__device__ __forceinline__ int last_at_or_below(const int *a, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) page_map_kernel(const MapParams p)
{
    __shared__ int tok0[kChunk + 1], page0[kChunk + 1];  // N_b and F_b of the chunk's requests
    __shared__ int cached_s[kChunk], have_s[kChunk];
    __shared__ int par[kTreeMaxTokens + kTokens];
    __shared__ long long wsum[kThreads / 32];
    __shared__ int wtake[kThreads / 32], wover[kThreads / 32];
    grid_dep_wait();  // the grid ahead
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.x * kTokens;
    const int ps = p.s.page_size;

    // the parents of this CTA's tokens and of the ones before them a tree may reach back to
    if (p.parents)
        for (int i = tid; i < kTreeMaxTokens + kTokens; i += kThreads) {
            const int t = t0 - kTreeMaxTokens + i;
            par[i] = t >= 0 && t < p.s.total_tokens ? p.parents[t] : -1;
        }

    long long tok_base = 0;
    int page_base = 0, over = 0;
    bool filled = t0 + tid >= p.s.total_tokens;
    for (int b0 = 0; b0 < p.s.B; b0 += kChunk) {
        // exclusive sums of the chunk's new tokens and new pages
        Request r[kPer];
        long long n = 0;
        int f = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            r[k] = request_at(p, b0 + tid * kPer + k);
            n += r[k].fresh;
            f += r[k].take;
            over += r[k].len > (long long)p.s.max_pages * ps;
        }
        long long ni = n;
        int fi = f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long nu = __shfl_up_sync(0xffffffffu, ni, o);
            const int fu = __shfl_up_sync(0xffffffffu, fi, o);
            if (lane >= o) {
                ni += nu;
                fi += fu;
            }
        }
        __syncthreads();  // the previous chunk's readers are done
        if (lane == 31) {
            wsum[warp] = ni;
            wtake[warp] = fi;
        }
        __syncthreads();
        long long nb = tok_base + ni - n;
        int fb = page_base + fi - f;
        long long ntot = 0;
        int ftot = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) {
                nb += wsum[w];
                fb += wtake[w];
            }
            ntot += wsum[w];
            ftot += wtake[w];
        }
        const int nreq = min(kChunk, p.s.B - b0);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = tid * kPer + k, b = b0 + i;
            tok0[i] = (int)min(nb, 0x7fffffffLL);
            page0[i] = fb;
            cached_s[i] = r[k].cached;
            have_s[i] = r[k].have;
            if (blockIdx.x == 0 && b < p.s.B) {
                p.cu[b] = (int)min(nb, (long long)p.s.total_tokens);
                p.seqlens[b] = (int)min(r[k].len, 0x7fffffffLL);
            }
            nb += r[k].fresh;
            fb += r[k].take;
        }
        if (tid == 0) {
            tok0[nreq] = (int)min(tok_base + ntot, 0x7fffffffLL);
            page0[nreq] = page_base + ftot;
        }
        __syncthreads();
        // the new pages' entries, dealt out over the grid (a page the free list does not hold: -1)
        for (unsigned x = page_base + blockIdx.x * kThreads + tid; x < (unsigned)page0[nreq];
             x += gridDim.x * kThreads) {  // (32 bits without a sign: a last step may pass 2^31)
            const int e = (int)x, i = last_at_or_below(page0, nreq, e);
            p.page_table[(size_t)(b0 + i) * p.s.max_pages + have_s[i] + (e - page0[i])] =
                e < p.s.n_free ? p.free_pages[e] : -1;
        }
        // this thread's token, once its request is in the chunk
        const int t = t0 + tid;
        if (!filled && t < tok0[nreq]) {
            filled = true;
            const int i = last_at_or_below(tok0, nreq, t);
            const int at = t - tok0[i], n_req = tok0[i + 1] - tok0[i];
            int depth = at;
            if (p.parents && n_req <= kTreeMaxTokens) {
                depth = 0;
                const int base = kTreeMaxTokens + tid - at;  // the request's first token in par
                for (int a = at;;) {
                    const int up = par[base + a];
                    if (up < 0 || up >= a) break;
                    a = up;
                    ++depth;
                }
            }
            p.positions[t] = (int)min((long long)cached_s[i] + depth, 0x7fffffffLL);
            const long long j = (long long)cached_s[i] + at, lp = j / ps;
            int page = -1;
            if (lp < have_s[i]) {
                page = p.page_table[(size_t)(b0 + i) * p.s.max_pages + lp];
            } else if (lp < p.s.max_pages) {
                const long long e = page0[i] + (lp - have_s[i]);
                page = e < p.s.n_free ? p.free_pages[e] : -1;
            }
            p.rows[t] = page >= 0 && page < p.s.num_pages ? page * ps + (int)(j % ps) : -1;
        }
        tok_base += ntot;
        page_base += ftot;
    }
    if (!filled) {  // behind the last request: no cache row
        p.positions[t0 + tid] = 0;
        p.rows[t0 + tid] = -1;
    }
    if (blockIdx.x == 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) over += __shfl_xor_sync(0xffffffffu, over, o);
        if (lane == 0) wover[warp] = over;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kThreads / 32; ++w) over += wover[w];
            p.cu[p.s.B] = (int)min(tok_base, (long long)p.s.total_tokens);
            p.stats[0] = (int)min(tok_base, 0x7fffffffLL);
            p.stats[1] = page_base;
            p.stats[2] = max(page_base - p.s.n_free, 0);
            p.stats[3] = over;
        }
    }
}

}  // namespace

cudaError_t launch_page_map(const int *cached_lens, const int *new_lens, const int *parents, const int *free_pages,
                            int *page_table, int *seqlens, int *cu_seqlens, int *positions, int *kv_rows, int *stats,
                            const PageMapShape &s, cudaStream_t st)
{
    const MapParams p{s, cached_lens, new_lens, parents, free_pages, page_table, seqlens, cu_seqlens, positions,
                      kv_rows, stats};
    return launch_chained(page_map_kernel, dim3((unsigned)((s.total_tokens - 1) / kTokens + 1)), kThreads, 0, st, p);
}

}  // namespace attn_sink
