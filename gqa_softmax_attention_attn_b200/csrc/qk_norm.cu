// qk_norm.cu -- the QKV prologue of models that normalise every query and key
// head before the rotation, forward and backward.
//
// Forward, for every token t and head with row y = qkv + bias (D = 64 values):
//   q and k heads: r = 1 / sqrt(mean(y^2) + eps), z = R_t (w o y r), with w the
//   weight of q or of k and R_t the (YaRN-scaled) rotation of t's position;
//   v heads: z = y.  k and v may go to any row of their outputs.
// Backward, from dz (of the rotated heads): u = R_t^T dz, n = y r,
//   dw_d   = sum over tokens and heads of u_d n_d
//   dy     = r (w o u - n mean(w o u o n)),  dy = dz for v,
//   dbias  = sum over tokens of dy, and dqkv = dy rounded to bf16.
// Sums and norms are fp32; dbias and the weights' gradients sum the unrounded
// dy and u n.
//
// A head's row is 8 chunks of 16 bytes and is worked on by 4 lanes, lane l
// holding pairs 8l .. 8l + 7 (both halves of each pair: two chunks), so the
// rotation needs no exchange and a sum over the head is two shuffles.
//
// Bound by HBM and instruction issue together (64 + 8 + 8 heads): forward of
// 4096 tokens 16.0 to 16.6 us, 5.1 TB/s; backward of 65536 tokens 340 to 346 us, 5.9 TB/s (359 to 378
// in runs of seconds, at the power limit, the clock down to 1.7 to 1.8 GHz); of 1003
// tokens 10.8 to 11.4 us, two launches and the latency of one slab.  Two pairs per
// instruction, the asynchronous ring and slabs as many as run at once brought
// 4096 tokens from 26.6 us and 65536 tokens backward from 614 us, addresses step by
// step the last 4 and 6 %; starting while
// the grid ahead ends took 512 tokens from 4.5 to 4.1 us, now 3.9.
#include <cuda_bf16.h>
#include <math.h>

#include "kernels.h"
#include "sm100_ptx.cuh"

namespace attn_sink {
namespace {

constexpr int kD = 64;
constexpr int kPairs = kD / 2;
constexpr int kThreads = 256;

struct NormParams {
    const __nv_bfloat16 *qkv;
    const float *bias;  // [(Hq + 2 Hkv) * D] or nullptr
    const float *qw, *kw;
    const int *pos, *kv_rows;
    float eps;
    int T, Hq, Hkv, kv_rows_total;
    float attn_factor;
    double turns[kPairs];  // rotary frequency of each pair, in turns per position
};

struct BwdParams {
    NormParams n;
    const __nv_bfloat16 *dq, *dk, *dv;
    __nv_bfloat16 *dqkv;
    float *dbias, *dqw, *dkw;
    float *ws;
    int slabs, groups;
};

// cos and sin (times the attention factor) of pair i at position pos, to out[i] and out[kPairs + i].  The
// angle is formed in turns and reduced in fp64 (a position of 131071 leaves
// fp32 too few bits of phase); its fraction, at most half a turn, is then
// rounded to fp32, an error of at most 2^-24 of half a turn.
__device__ __forceinline__ void rotation(const NormParams &p, int pos, int i, float *out)
{
    const double x = (double)pos * p.turns[i];
    float sn, cs;
    sincospif((float)(2.0 * (x - rint(x))), &sn, &cs);
    out[i] = cs * p.attn_factor;
    out[kPairs + i] = sn * p.attn_factor;
}

// element offsets of lane l's two chunks of a head's row.  In registers the lane's eight pairs are two
// arrays, a[i] the first halves of pairs 8l + 2i and 8l + 2i + 1 and b[i] their second halves, so that
// every operation takes two pairs at a time (fp32 x 2 instructions: half the issue slots).
template <bool kInter>
__device__ __forceinline__ constexpr int chunk0(int l) { return kInter ? 16 * l : 8 * l; }
template <bool kInter>
__device__ __forceinline__ constexpr int chunk1(int l) { return kInter ? 16 * l + 8 : kPairs + 8 * l; }

__device__ __forceinline__ float2 bf2(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <bool kInter>
__device__ __forceinline__ void unpack(const uint4 &c0, const uint4 &c1, float2 (&a)[4], float2 (&b)[4])
{
    const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kInter) {
            a[i] = make_float2(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i + 1] << 16));
            b[i] = make_float2(__uint_as_float(w[2 * i] & 0xffff0000u), __uint_as_float(w[2 * i + 1] & 0xffff0000u));
        } else {
            a[i] = bf2(w[i]);
            b[i] = bf2(w[4 + i]);
        }
    }
}
template <bool kInter>
__device__ __forceinline__ void pack(const float2 (&a)[4], const float2 (&b)[4], uint4 &c0, uint4 &c1)
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[kInter ? 2 * i : i] = kInter ? pack_bf16x2(a[i].x, b[i].x) : pack_bf16x2(a[i].x, a[i].y);
        w[kInter ? 2 * i + 1 : 4 + i] = kInter ? pack_bf16x2(a[i].y, b[i].y) : pack_bf16x2(b[i].x, b[i].y);
    }
    c0 = make_uint4(w[0], w[1], w[2], w[3]);
    c1 = make_uint4(w[4], w[5], w[6], w[7]);
}

// lane l's 16 of a head's 64 fp32 values (bias, weight, partial sums)
template <bool kInter>
__device__ __forceinline__ void load_pairs(const float *p, int l, float2 (&a)[4], float2 (&b)[4])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 u = reinterpret_cast<const float4 *>(p + chunk0<kInter>(l))[i];
        const float4 v = reinterpret_cast<const float4 *>(p + chunk1<kInter>(l))[i];
        if (kInter) {
            a[i] = make_float2(u.x, u.z);
            b[i] = make_float2(u.y, u.w);
            a[2 + i] = make_float2(v.x, v.z);
            b[2 + i] = make_float2(v.y, v.w);
        } else {
            a[2 * i] = make_float2(u.x, u.y);
            a[2 * i + 1] = make_float2(u.z, u.w);
            b[2 * i] = make_float2(v.x, v.y);
            b[2 * i + 1] = make_float2(v.z, v.w);
        }
    }
}
template <bool kInter>
__device__ __forceinline__ void store_pairs(float *p, int l, const float2 (&a)[4], const float2 (&b)[4])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        reinterpret_cast<float4 *>(p + chunk0<kInter>(l))[i] =
            kInter ? make_float4(a[i].x, b[i].x, a[i].y, b[i].y)
                   : make_float4(a[2 * i].x, a[2 * i].y, a[2 * i + 1].x, a[2 * i + 1].y);
        reinterpret_cast<float4 *>(p + chunk1<kInter>(l))[i] =
            kInter ? make_float4(a[2 + i].x, b[2 + i].x, a[2 + i].y, b[2 + i].y)
                   : make_float4(b[2 * i].x, b[2 * i].y, b[2 * i + 1].x, b[2 * i + 1].y);
    }
}

// A token's rotations in shared memory: cosines, then sines of its 32 pairs.
__device__ __forceinline__ void load_rotation(const float *rot, int l, float2 (&c)[4], float2 (&s)[4])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 u = reinterpret_cast<const float4 *>(rot + 8 * l)[i];
        const float4 v = reinterpret_cast<const float4 *>(rot + kPairs + 8 * l)[i];
        c[2 * i] = make_float2(u.x, u.y);
        c[2 * i + 1] = make_float2(u.z, u.w);
        s[2 * i] = make_float2(v.x, v.y);
        s[2 * i + 1] = make_float2(v.z, v.w);
    }
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }

// sum over a head (its 4 lanes) of the products of two rows
__device__ __forceinline__ float head_dot(const float2 (&a)[4], const float2 (&b)[4], const float2 (&c)[4],
                                          const float2 (&d)[4])
{
    float2 s = fmul2(a[0], c[0]), t = fmul2(b[0], d[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        s = ffma2(a[i], c[i], s);
        t = ffma2(b[i], d[i], t);
    }
    s = fadd2(s, t);
    float x = s.x + s.y;
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// Both kernels: CTA = (16 heads, a slab of tokens), 4 tokens x 16 heads x 4 lanes a step, so a thread keeps
// its head, and with it the bias and the weights of its 16 columns, in registers.  The slabs are as many as
// run at once.  The rows come through a ring in shared memory, each thread copying (asynchronously)
// the bytes it will read itself, so that no barrier and no register holds a load in flight.  The rotations
// of kBTok tokens at a time are formed in shared memory, one angle a thread, a batch ahead.
constexpr int kHeads = 16;
constexpr int kTokLanes = kThreads / (4 * kHeads);
constexpr int kBTok = 16;
__host__ __device__ __forceinline__ int head_groups(int heads) { return (heads + kHeads - 1) / kHeads; }
// slabs of T tokens for `ctas` CTAs in all; at least a step's tokens each
__host__ __forceinline__ int num_slabs(int T, int groups, int ctas)
{
    const int most = (T + kTokLanes - 1) / kTokLanes, fit = ctas / groups > 0 ? ctas / groups : 1;
    return most < fit ? most : fit;
}

__device__ __forceinline__ void copy16_async(uint32_t smem_dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(src) : "memory");
}

// ------------------------------------------------------------------ forward
constexpr int kFwdRing = 4, kFwdPerSm = 3;

template <bool kInter>
__global__ void __launch_bounds__(kThreads, kFwdPerSm) qk_norm_fwd_kernel(const NormParams p, int slabs,
                                                                          __nv_bfloat16 *q, __nv_bfloat16 *k,
                                                                          __nv_bfloat16 *v)
{
    grid_dep_launch();
    grid_dep_wait();  // the grid ahead
    __shared__ __align__(16) float rot[2][kBTok][2 * kPairs];
    extern __shared__ __align__(16) uint8_t ring_raw[];  // [kFwdRing][2 chunks][kThreads] of 16 bytes
    const int heads = p.Hq + 2 * p.Hkv, groups = head_groups(heads);
    const int slab = blockIdx.x / groups;
    const int l = threadIdx.x & 3, h = blockIdx.x % groups * kHeads + (threadIdx.x >> 2) % kHeads;
    const int tl = threadIdx.x / (4 * kHeads);
    const bool live_h = h < heads;
    const int hc = live_h ? h : 0;
    const long long tb = (long long)p.T * slab / slabs;
    const int nt = (int)((long long)p.T * (slab + 1) / slabs - tb);  // tokens of the slab
    // (addresses step by step: with products of 64 bits and remainders 4096 tokens took 17.3 us instead of 16.6)
    const size_t ss = (size_t)heads * kD;
    const __nv_bfloat16 *src = p.qkv + (tb + tl) * ss + hc * kD + chunk0<kInter>(l);
    const uint32_t ring = smem_u32(ring_raw) + threadIdx.x * 16;
    int fetched = tl, put = 0, get = 0;  // the lane's next token to fetch; places of the next step in and out
    auto fetch = [&]() {
        if (fetched < nt) {
            const uint32_t dst = ring + put * (2 * kThreads * 16);
            copy16_async(dst, src);
            copy16_async(dst + kThreads * 16, src + (chunk1<kInter>(0) - chunk0<kInter>(0)));
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        fetched += kTokLanes;
        src += kTokLanes * ss;
        put = put + 1 == kFwdRing ? 0 : put + 1;
    };
    auto rotations = [&](int t0) {  // of tokens [t0, t0 + kBTok) of the slab
        for (int a = threadIdx.x; a < kBTok * kPairs; a += kThreads)
            if (t0 + a / kPairs < nt)
                rotation(p, p.pos[tb + t0 + a / kPairs], a % kPairs, rot[t0 / kBTok & 1][a / kPairs]);
    };
#pragma unroll
    for (int s = 0; s < kFwdRing - 1; ++s) fetch();
    float2 ba[4], bb[4], wa[4], wb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) ba[j] = bb[j] = make_float2(0.f, 0.f);
    if (p.bias) load_pairs<kInter>(p.bias + hc * kD, l, ba, bb);
    load_pairs<kInter>(h < p.Hq ? p.qw : p.kw, l, wa, wb);
    rotations(0);
    // where its rows go: q by token, k and v by cache row
    const bool is_q = h < p.Hq;
    __nv_bfloat16 *out = is_q ? q + h * kD : h < p.Hq + p.Hkv ? k + (h - p.Hq) * kD : v + (h - p.Hq - p.Hkv) * kD;
    const unsigned stride = (unsigned)(is_q ? p.Hq : p.Hkv) * kD;
    for (int t0 = 0; t0 < nt; t0 += kBTok) {
        __syncthreads();  // this batch's rotations are there, and the other buffer's readers done
        if (t0 + kBTok < nt) rotations(t0 + kBTok);
        const int n = min(kBTok, nt - t0);
#pragma unroll 1
        for (int x = 0; x < n; x += kTokLanes) {  // (the shuffles need whole warps: no lane leaves)
            const int tt = x + tl;
            const bool live = live_h && tt < n;
            const int t = (int)tb + t0 + tt;
            const int row = !is_q && p.kv_rows && live ? p.kv_rows[t] : t;
            asm volatile("cp.async.wait_group %0;" ::"n"(kFwdRing - 2) : "memory");
            const uint4 *mine = reinterpret_cast<const uint4 *>(ring_raw) + get * (2 * kThreads) + threadIdx.x;
            get = get + 1 == kFwdRing ? 0 : get + 1;
            float2 a[4], b[4];
            unpack<kInter>(mine[0], mine[kThreads], a, b);
            fetch();  // into the step before's place
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] = fadd2(a[j], ba[j]);
                b[j] = fadd2(b[j], bb[j]);
            }
            const float r = rsqrtf(head_dot(a, b, a, b) * (1.f / kD) + p.eps);
            if (h < p.Hq + p.Hkv) {
                float2 c[4], s[4];
                load_rotation(rot[t0 / kBTok & 1][tt], l, c, s);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = fmul2(fmul2(a[j], both(r)), wa[j]), y = fmul2(fmul2(b[j], both(r)), wb[j]);
                    a[j] = ffma2(x, c[j], neg2(fmul2(y, s[j])));
                    b[j] = ffma2(y, c[j], fmul2(x, s[j]));
                }
            }
            if (live && (is_q || (row >= 0 && row < p.kv_rows_total))) {
                __nv_bfloat16 *dst = out + (size_t)(unsigned)row * stride;
                uint4 o0, o1;
                pack<kInter>(a, b, o0, o1);
                *reinterpret_cast<uint4 *>(dst + chunk0<kInter>(l)) = o0;
                *reinterpret_cast<uint4 *>(dst + chunk1<kInter>(l)) = o1;
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------------ backward
// A thread's dbias and weight sums stay in its registers over its slab.  The four token lanes then add up
// through shared memory and the CTA stores one partial row; a second kernel sums the slabs in order, so the
// gradients are the same from run to run.
constexpr int kRing = 3, kBwdPerSm = 2;
constexpr int kBwdSmem = kRing * 4 * kThreads * 16;

template <bool kInter>
__global__ void __launch_bounds__(kThreads, kBwdPerSm) qk_norm_bwd_kernel(const BwdParams bp)
{
    grid_dep_launch();  // the finish kernel may start; it waits for this grid
    grid_dep_wait();    // (as this one for the grid ahead)
    const NormParams &p = bp.n;
    __shared__ __align__(16) float rot[2][kBTok][2 * kPairs];
    extern __shared__ __align__(16) uint8_t ring_raw[];  // [kRing][4 chunks][kThreads] of 16 bytes
    static_assert(kTokLanes * kHeads * kD * 4 <= kBwdSmem, "the sums' exchange reuses the ring");
    float *red = reinterpret_cast<float *>(ring_raw);  // [kTokLanes][kHeads * kD]
    const int heads = p.Hq + 2 * p.Hkv;
    const int group = blockIdx.x % bp.groups, slab = blockIdx.x / bp.groups;
    const int l = threadIdx.x & 3, hs = (threadIdx.x >> 2) % kHeads, tl = threadIdx.x / (4 * kHeads);
    const int h = group * kHeads + hs;
    const bool is_q = h < p.Hq, rotated = h < p.Hq + p.Hkv, live_h = h < heads;
    const int hc = live_h ? h : 0;
    const long long tb = (long long)p.T * slab / bp.slabs, te = (long long)p.T * (slab + 1) / bp.slabs;
    const int nt = (int)(te - tb);  // tokens of the slab
    // this thread's rows: token tb + tl of the inputs and of the gradient of its head, and their strides
    const __nv_bfloat16 *src = p.qkv + ((size_t)(tb + tl) * heads + hc) * kD + chunk0<kInter>(l);
    const size_t gs = is_q || !live_h ? (size_t)p.Hq * kD : (size_t)p.Hkv * kD, ss = (size_t)heads * kD;
    const __nv_bfloat16 *gsrc = (is_q || !live_h ? bp.dq + (live_h ? h : 0) * kD
                                 : rotated       ? bp.dk + (h - p.Hq) * kD
                                                 : bp.dv + (h - p.Hq - p.Hkv) * kD) + (tb + tl) * gs + chunk0<kInter>(l);
    constexpr int kOther = chunk1<kInter>(0) - chunk0<kInter>(0);  // from a lane's first chunk to its second
    const uint32_t ring = smem_u32(ring_raw) + threadIdx.x * 16;
    int fetched = tl, put = 0, get = 0;  // the lane's next token to fetch; places of the next step in and out
    auto fetch = [&]() {
        if (fetched < nt) {
            const uint32_t dst = ring + put * (4 * kThreads * 16);
            copy16_async(dst, src);
            copy16_async(dst + kThreads * 16, src + kOther);
            copy16_async(dst + 2 * kThreads * 16, gsrc);
            copy16_async(dst + 3 * kThreads * 16, gsrc + kOther);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        fetched += kTokLanes;
        src += kTokLanes * ss;
        gsrc += kTokLanes * gs;
        put = put + 1 == kRing ? 0 : put + 1;
    };
    __nv_bfloat16 *dst = bp.dqkv + ((size_t)(tb + tl) * heads + hc) * kD + chunk0<kInter>(l);
    auto rotations = [&](int t0) {  // of tokens [t0, t0 + kBTok) of the slab
        for (int a = threadIdx.x; a < kBTok * kPairs; a += kThreads)
            if (t0 + a / kPairs < nt)
                rotation(p, p.pos[tb + t0 + a / kPairs], a % kPairs, rot[t0 / kBTok & 1][a / kPairs]);
    };
#pragma unroll
    for (int s = 0; s < kRing - 1; ++s) fetch();
    float2 ba[4], bb[4], wa[4], wb[4], sa[4], sb[4], ga[4], gb[4];  // bias, weight, dbias sums, weight sums
#pragma unroll
    for (int j = 0; j < 4; ++j) ba[j] = bb[j] = sa[j] = sb[j] = ga[j] = gb[j] = make_float2(0.f, 0.f);
    if (p.bias) load_pairs<kInter>(p.bias + hc * kD, l, ba, bb);
    load_pairs<kInter>(is_q ? p.qw : p.kw, l, wa, wb);
    rotations(0);
    for (int t0 = 0; t0 < nt; t0 += kBTok) {
        __syncthreads();  // this batch's rotations are there, and the other buffer's readers done
        if (t0 + kBTok < nt) rotations(t0 + kBTok);
#pragma unroll 1
        for (int x = 0; x < min(kBTok, nt - t0); x += kTokLanes, dst += kTokLanes * ss) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
            const int tt = x + tl;
            const bool live = live_h && t0 + tt < nt;
            const uint4 *mine = reinterpret_cast<const uint4 *>(ring_raw) + get * (4 * kThreads) + threadIdx.x;
            get = get + 1 == kRing ? 0 : get + 1;
            float2 a[4], b[4], ua[4], ub[4];
            unpack<kInter>(mine[0], mine[kThreads], a, b);
            unpack<kInter>(mine[2 * kThreads], mine[3 * kThreads], ua, ub);
            fetch();  // into the step before's place
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] = fadd2(a[j], ba[j]);
                b[j] = fadd2(b[j], bb[j]);
            }
            const float r = rsqrtf(head_dot(a, b, a, b) * (1.f / kD) + p.eps);
            if (rotated) {
                float2 c[4], s[4];
                load_rotation(rot[t0 / kBTok & 1][tt], l, c, s);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = ffma2(ua[j], c[j], fmul2(ub[j], s[j]));
                    const float2 y = ffma2(ub[j], c[j], neg2(fmul2(ua[j], s[j])));
                    a[j] = fmul2(a[j], both(r));  // n
                    b[j] = fmul2(b[j], both(r));
                    if (live) {
                        ga[j] = ffma2(x, a[j], ga[j]);
                        gb[j] = ffma2(y, b[j], gb[j]);
                    }
                    ua[j] = fmul2(x, wa[j]);
                    ub[j] = fmul2(y, wb[j]);
                }
            }
            const float2 mean = both(-head_dot(ua, ub, a, b) * (1.f / kD));
            if (rotated) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ua[j] = fmul2(both(r), ffma2(mean, a[j], ua[j]));
                    ub[j] = fmul2(both(r), ffma2(mean, b[j], ub[j]));
                }
            }
            if (live) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sa[j] = fadd2(sa[j], ua[j]);
                    sb[j] = fadd2(sb[j], ub[j]);
                }
                uint4 c0, c1;
                pack<kInter>(ua, ub, c0, c1);
                *reinterpret_cast<uint4 *>(dst) = c0;
                *reinterpret_cast<uint4 *>(dst + kOther) = c1;
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // partial rows: [slab][groups * kHeads * D] dbias, then [slab][groups][2][D] weights
    const size_t wide = (size_t)bp.groups * kHeads * kD;
    __syncthreads();
    store_pairs<kInter>(red + (tl * kHeads + hs) * kD, l, sa, sb);
    __syncthreads();
    for (int c = threadIdx.x; c < kHeads * kD; c += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kTokLanes; ++w) s += red[w * kHeads * kD + c];
        bp.ws[slab * wide + (size_t)group * kHeads * kD + c] = s;
    }
    __syncthreads();
    store_pairs<kInter>(red + (tl * kHeads + hs) * kD, l, ga, gb);
    __syncthreads();
    if (threadIdx.x < 2 * kD) {
        const int which = threadIdx.x / kD, d = threadIdx.x % kD;  // 0: q, 1: k
        float s = 0.f;
        for (int x = 0; x < kHeads; ++x) {
            const int hh = group * kHeads + x;
            if (which == 0 ? hh < p.Hq : hh >= p.Hq && hh < p.Hq + p.Hkv)
#pragma unroll
                for (int w = 0; w < kTokLanes; ++w) s += red[(w * kHeads + x) * kD + d];
        }
        bp.ws[bp.slabs * wide + (((size_t)slab * bp.groups + group) * 2 + which) * kD + d] = s;
    }
}

// Column sums over the slabs, in order: a CTA takes 64 columns, 16 threads of four columns for each of 16
// parts of the slabs; the last two CTAs take the weights.
__global__ void __launch_bounds__(kThreads) qk_norm_finish_kernel(const BwdParams bp)
{
    constexpr int kParts = kThreads / (kD / 4);
    __shared__ __align__(16) float red[kParts][kD];
    const size_t wide = (size_t)bp.groups * kHeads * kD;
    const int bias_ctas = gridDim.x - 2, which = (int)blockIdx.x - bias_ctas;  // which >= 0: q's, k's weights
    const int col = threadIdx.x % (kD / 4) * 4, part = threadIdx.x / (kD / 4);
    const float *src = which < 0 ? bp.ws + (size_t)blockIdx.x * kD : bp.ws + bp.slabs * wide + which * kD;
    const size_t stride = which < 0 ? wide : 2 * kD;
    const int n = which < 0 ? bp.slabs : bp.slabs * bp.groups;
    grid_dep_launch();
    grid_dep_wait();
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int x = part; x < n; x += kParts) {
        const float4 v = *reinterpret_cast<const float4 *>(src + x * stride + col);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    *reinterpret_cast<float4 *>(&red[part][col]) = s;
    __syncthreads();
    if (threadIdx.x >= kD) return;
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kParts; ++w) t += red[w][threadIdx.x];
    if (which < 0)
        bp.dbias[(size_t)blockIdx.x * kD + threadIdx.x] = t;
    else
        (which == 0 ? bp.dqw : bp.dkw)[threadIdx.x] = t;
}

NormParams norm_params(const void *qkv, const float *bias, const QkNorm &n, const int *positions, const int *kv_rows,
                       int T, int Hq, int Hkv, int kv_rows_total, const RopeParams &r)
{
    NormParams p;
    p.qkv = static_cast<const __nv_bfloat16 *>(qkv);
    p.bias = bias;
    p.qw = n.q_weight;
    p.kw = n.k_weight;
    p.eps = n.eps;
    p.pos = positions;
    p.kv_rows = kv_rows;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.kv_rows_total = kv_rows_total;
    p.attn_factor = (float)rope_attention_factor(r);
    rope_frequencies(r, p.turns);
    for (int i = 0; i < kPairs; ++i) p.turns[i] /= 2.0 * M_PI;
    return p;
}

}  // namespace

cudaError_t launch_qk_norm_prologue(const void *qkv, const float *bias, const QkNorm &n, const int *positions,
                                    const int *kv_rows, void *q, void *k, void *v, int T, int Hq, int Hkv,
                                    int kv_rows_total, const RopeParams &r, cudaStream_t st)
{
    const NormParams p = norm_params(qkv, bias, n, positions, kv_rows, T, Hq, Hkv, kv_rows_total, r);
    const int groups = head_groups(Hq + 2 * Hkv), slabs = num_slabs(T, groups, kFwdPerSm * 148);
    auto kern = r.interleaved ? qk_norm_fwd_kernel<true> : qk_norm_fwd_kernel<false>;
    constexpr int smem = kFwdRing * 2 * kThreads * 16;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_chained(kern, dim3((unsigned)(slabs * groups)), kThreads, smem, st, p, slabs,
                          static_cast<__nv_bfloat16 *>(q), static_cast<__nv_bfloat16 *>(k),
                          static_cast<__nv_bfloat16 *>(v));
}

size_t qk_norm_bwd_workspace_bytes(int T, int Hq, int Hkv)
{
    const int groups = head_groups(Hq + 2 * Hkv);
    return (size_t)num_slabs(T, groups, kBwdPerSm * 148) * groups * (kHeads + 2) * kD * sizeof(float);
}

cudaError_t launch_qk_norm_bwd(const void *qkv, const float *bias, const QkNorm &n, const int *positions,
                               const void *dq, const void *dk, const void *dv, void *dqkv, float *dbias,
                               float *dq_weight, float *dk_weight, int T, int Hq, int Hkv, const RopeParams &r,
                               float *ws, cudaStream_t st)
{
    BwdParams p;
    p.n = norm_params(qkv, bias, n, positions, nullptr, T, Hq, Hkv, T, r);
    p.dq = static_cast<const __nv_bfloat16 *>(dq);
    p.dk = static_cast<const __nv_bfloat16 *>(dk);
    p.dv = static_cast<const __nv_bfloat16 *>(dv);
    p.dqkv = static_cast<__nv_bfloat16 *>(dqkv);
    p.dbias = dbias;
    p.dqw = dq_weight;
    p.dkw = dk_weight;
    p.ws = ws;
    p.groups = head_groups(Hq + 2 * Hkv);
    p.slabs = num_slabs(T, p.groups, kBwdPerSm * 148);
    auto kern = r.interleaved ? qk_norm_bwd_kernel<true> : qk_norm_bwd_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdSmem);
    if (e != cudaSuccess) return e;
    e = launch_chained(kern, dim3((unsigned)(p.slabs * p.groups)), kThreads, kBwdSmem, st, p);
    if (e != cudaSuccess) return e;
    return launch_chained(qk_norm_finish_kernel, dim3((unsigned)((dbias ? Hq + 2 * Hkv : 0) + 2)), kThreads, 0, st, p);
}

}  // namespace attn_sink
