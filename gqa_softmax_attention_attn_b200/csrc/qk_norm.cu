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
    const __nv_bfloat16 *__restrict__ qkv;
    const float *__restrict__ bias;  // [(Hq + 2 Hkv) * D] or nullptr
    const float *__restrict__ qw, *__restrict__ kw;
    const int *__restrict__ pos, *__restrict__ kv_rows;
    float eps;
    int T, Hq, Hkv, kv_rows_total;
    float attn_factor;
    double turns[kPairs];  // rotary frequency of each pair, in turns per position
};

struct BwdParams {
    NormParams n;
    const __nv_bfloat16 *__restrict__ dq, *__restrict__ dk, *__restrict__ dv;
    __nv_bfloat16 *__restrict__ dqkv;
    float *__restrict__ dbias, *__restrict__ dqw, *__restrict__ dkw;
    float *__restrict__ ws;
    int slabs, groups;
};

// cos and sin (times the attention factor) of pair i at position pos.  The
// angle is formed in turns and reduced in fp64 (a position of 131071 leaves
// fp32 too few bits of phase); its fraction, at most half a turn, is then
// rounded to fp32, an error of at most 2^-24 of half a turn.
__device__ __forceinline__ float2 rotation(const NormParams &p, int pos, int i)
{
    const double x = (double)pos * p.turns[i];
    float sn, cs;
    sincospif((float)(2.0 * (x - rint(x))), &sn, &cs);
    return make_float2(cs * p.attn_factor, sn * p.attn_factor);
}

// element offsets of lane l's two chunks of a head's row, and their layout in
// registers: a[j], b[j] are the two halves of pair 8l + j
template <bool kInter>
__device__ __forceinline__ void unpack(const uint4 &c0, const uint4 &c1, float (&a)[8], float (&b)[8])
{
    const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j]));
        if (kInter) {
            a[j] = f.x;
            b[j] = f.y;
        } else if (j < 4) {
            a[2 * j] = f.x;
            a[2 * j + 1] = f.y;
        } else {
            b[2 * (j - 4)] = f.x;
            b[2 * (j - 4) + 1] = f.y;
        }
    }
}
template <bool kInter>
__device__ __forceinline__ void pack(const float (&a)[8], const float (&b)[8], uint4 &c0, uint4 &c1)
{
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        w[j] = kInter ? pack_bf16x2(a[j], b[j])
                      : (j < 4 ? pack_bf16x2(a[2 * j], a[2 * j + 1]) : pack_bf16x2(b[2 * (j - 4)], b[2 * (j - 4) + 1]));
    c0 = make_uint4(w[0], w[1], w[2], w[3]);
    c1 = make_uint4(w[4], w[5], w[6], w[7]);
}
template <bool kInter>
__device__ __forceinline__ int chunk0(int l) { return kInter ? 16 * l : 8 * l; }
template <bool kInter>
__device__ __forceinline__ int chunk1(int l) { return kInter ? 16 * l + 8 : kPairs + 8 * l; }

// lane l's 16 of a head's 64 fp32 values (bias, weight, partial sums), in pairs
template <bool kInter>
__device__ __forceinline__ void load_pairs(const float *p, int l, float (&a)[8], float (&b)[8])
{
    float x[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 v = reinterpret_cast<const float4 *>(p + (j < 2 ? chunk0<kInter>(l) : chunk1<kInter>(l)))[j & 1];
        x[4 * j] = v.x;
        x[4 * j + 1] = v.y;
        x[4 * j + 2] = v.z;
        x[4 * j + 3] = v.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        a[j] = kInter ? x[2 * j] : x[j];
        b[j] = kInter ? x[2 * j + 1] : x[8 + j];
    }
}
template <bool kInter>
__device__ __forceinline__ void store_pairs(float *p, int l, const float (&a)[8], const float (&b)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float4 v;
        if (kInter)
            v = make_float4(a[2 * j], b[2 * j], a[2 * j + 1], b[2 * j + 1]);
        else
            v = j < 2 ? make_float4(a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3])
                      : make_float4(b[4 * j - 8], b[4 * j - 7], b[4 * j - 6], b[4 * j - 5]);
        reinterpret_cast<float4 *>(p + (j < 2 ? chunk0<kInter>(l) : chunk1<kInter>(l)))[j & 1] = v;
    }
}

__device__ __forceinline__ float head_sum(float x)  // over a head's 4 lanes
{
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
__device__ __forceinline__ float dot16(const float (&a)[8], const float (&b)[8], const float (&c)[8],
                                       const float (&d)[8])
{
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(a[j], c[j], fmaf(b[j], d[j], s));
    return s;
}

// ------------------------------------------------------------------ forward
// kTok tokens per CTA: their rotations into shared memory (one angle a
// thread), then 64 heads at a time.
constexpr int kTok = 8;

template <bool kInter>
__global__ void __launch_bounds__(kThreads) qk_norm_fwd_kernel(const NormParams p, __nv_bfloat16 *__restrict__ q,
                                                               __nv_bfloat16 *__restrict__ k,
                                                               __nv_bfloat16 *__restrict__ v)
{
    __shared__ float2 rot[kTok][kPairs];
    const int t0 = blockIdx.x * kTok;
    for (int a = threadIdx.x; a < kTok * kPairs; a += kThreads)
        if (t0 + a / kPairs < p.T) rot[a / kPairs][a % kPairs] = rotation(p, p.pos[t0 + a / kPairs], a % kPairs);
    __syncthreads();
    const int heads = p.Hq + 2 * p.Hkv, l = threadIdx.x & 3;
    const int units = min(kTok, p.T - t0) * heads;
    for (int base = 0; base < units; base += kThreads / 4) {  // uniform: the shuffles need whole warps
        const int u = base + (threadIdx.x >> 2);
        const bool live = u < units;
        const int tt = live ? u / heads : 0, h = live ? u % heads : 0, t = t0 + tt;
        const int kr = p.kv_rows && h >= p.Hq ? p.kv_rows[t] : t;
        const __nv_bfloat16 *src = p.qkv + ((size_t)t * heads + h) * kD;
        float a[8], b[8];
        unpack<kInter>(*reinterpret_cast<const uint4 *>(src + chunk0<kInter>(l)),
                       *reinterpret_cast<const uint4 *>(src + chunk1<kInter>(l)), a, b);
        if (p.bias) {
            float ba[8], bb[8];
            load_pairs<kInter>(p.bias + h * kD, l, ba, bb);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] += ba[j];
                b[j] += bb[j];
            }
        }
        const float r = rsqrtf(head_sum(dot16(a, b, a, b)) * (1.f / kD) + p.eps);
        if (h < p.Hq + p.Hkv) {
            float wa[8], wb[8];
            load_pairs<kInter>(h < p.Hq ? p.qw : p.kw, l, wa, wb);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 cs = rot[tt][8 * l + j];
                const float x = a[j] * r * wa[j], y = b[j] * r * wb[j];
                a[j] = x * cs.x - y * cs.y;
                b[j] = y * cs.x + x * cs.y;
            }
        }
        if (!live || (h >= p.Hq && (kr < 0 || kr >= p.kv_rows_total))) continue;
        __nv_bfloat16 *dst = h < p.Hq              ? q + ((size_t)t * p.Hq + h) * kD
                             : h < p.Hq + p.Hkv ? k + ((size_t)kr * p.Hkv + (h - p.Hq)) * kD
                                                : v + ((size_t)kr * p.Hkv + (h - p.Hq - p.Hkv)) * kD;
        uint4 c0, c1;
        pack<kInter>(a, b, c0, c1);
        *reinterpret_cast<uint4 *>(dst + chunk0<kInter>(l)) = c0;
        *reinterpret_cast<uint4 *>(dst + chunk1<kInter>(l)) = c1;
    }
}

// ------------------------------------------------------------------ backward
// CTA = (16 heads, slab of tokens): 4 tokens x 16 heads x 4 lanes at a time, so
// a thread keeps its head and its 16 columns, whose dbias and weight sums stay
// in its registers over the slab.  The four token lanes then add up through
// shared memory and the CTA stores one partial row; a second kernel sums the
// slabs in order, so the gradients are the same from run to run.
constexpr int kHeads = 16;
constexpr int kTokLanes = kThreads / (4 * kHeads);
constexpr int kBTok = 8;           // tokens whose rotations are formed at a time
constexpr int kMaxSlabs = 256;

__host__ __device__ __forceinline__ int head_groups(int heads) { return (heads + kHeads - 1) / kHeads; }
__host__ __forceinline__ int num_slabs(int T)
{
    const int s = (T + kBTok - 1) / kBTok;
    return s < kMaxSlabs ? s : kMaxSlabs;
}

template <bool kInter>
__global__ void __launch_bounds__(kThreads) qk_norm_bwd_kernel(const BwdParams bp)
{
    grid_dep_launch();
    const NormParams &p = bp.n;
    __shared__ float2 rot[kBTok][kPairs];
    __shared__ float red[kTokLanes][kHeads * kD];
    const int heads = p.Hq + 2 * p.Hkv;
    const int group = blockIdx.x % bp.groups, slab = blockIdx.x / bp.groups;
    const int l = threadIdx.x & 3, hs = (threadIdx.x >> 2) % kHeads, tl = threadIdx.x / (4 * kHeads);
    const int h = group * kHeads + hs;
    const bool is_q = h < p.Hq, rotated = h < p.Hq + p.Hkv, live_h = h < heads;
    const int hc = live_h ? h : 0;
    const long long tb = (long long)p.T * slab / bp.slabs, te = (long long)p.T * (slab + 1) / bp.slabs;
    float ba[8], bb[8], wa[8], wb[8], sa[8], sb[8], ga[8], gb[8];  // bias, weight, dbias sums, weight sums
#pragma unroll
    for (int j = 0; j < 8; ++j) ba[j] = bb[j] = sa[j] = sb[j] = ga[j] = gb[j] = 0.f;
    if (p.bias) load_pairs<kInter>(p.bias + hc * kD, l, ba, bb);
    load_pairs<kInter>(is_q ? p.qw : p.kw, l, wa, wb);
    for (long long t0 = tb; t0 < te; t0 += kBTok) {
        __syncthreads();
        for (int a = threadIdx.x; a < kBTok * kPairs; a += kThreads)
            if (t0 + a / kPairs < te) rot[a / kPairs][a % kPairs] = rotation(p, p.pos[t0 + a / kPairs], a % kPairs);
        __syncthreads();
        for (int tt = tl; tt < kBTok; tt += kTokLanes) {
            const bool live = live_h && t0 + tt < te;
            const size_t t = live ? t0 + tt : tb;
            const __nv_bfloat16 *src = p.qkv + (t * heads + hc) * kD;
            const __nv_bfloat16 *gsrc = is_q || !live_h ? bp.dq + (t * p.Hq + (live_h ? h : 0)) * kD
                                        : rotated     ? bp.dk + (t * p.Hkv + (h - p.Hq)) * kD
                                                      : bp.dv + (t * p.Hkv + (h - p.Hq - p.Hkv)) * kD;
            float a[8], b[8], ua[8], ub[8];
            unpack<kInter>(*reinterpret_cast<const uint4 *>(src + chunk0<kInter>(l)),
                           *reinterpret_cast<const uint4 *>(src + chunk1<kInter>(l)), a, b);
            unpack<kInter>(*reinterpret_cast<const uint4 *>(gsrc + chunk0<kInter>(l)),
                           *reinterpret_cast<const uint4 *>(gsrc + chunk1<kInter>(l)), ua, ub);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] += ba[j];
                b[j] += bb[j];
            }
            const float r = rsqrtf(head_sum(dot16(a, b, a, b)) * (1.f / kD) + p.eps);
            if (rotated) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 cs = rot[tt][8 * l + j];
                    const float x = ua[j] * cs.x + ub[j] * cs.y, y = ub[j] * cs.x - ua[j] * cs.y;
                    a[j] *= r;  // n
                    b[j] *= r;
                    if (live) {
                        ga[j] = fmaf(x, a[j], ga[j]);
                        gb[j] = fmaf(y, b[j], gb[j]);
                    }
                    ua[j] = x * wa[j];
                    ub[j] = y * wb[j];
                }
            }
            const float mean = head_sum(dot16(ua, ub, a, b)) * (1.f / kD);
            if (rotated) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    ua[j] = r * fmaf(-mean, a[j], ua[j]);
                    ub[j] = r * fmaf(-mean, b[j], ub[j]);
                }
            }
            if (live) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sa[j] += ua[j];
                    sb[j] += ub[j];
                }
                uint4 c0, c1;
                pack<kInter>(ua, ub, c0, c1);
                __nv_bfloat16 *dst = bp.dqkv + (t * heads + h) * kD;
                *reinterpret_cast<uint4 *>(dst + chunk0<kInter>(l)) = c0;
                *reinterpret_cast<uint4 *>(dst + chunk1<kInter>(l)) = c1;
            }
        }
    }
    // partial rows: [slab][groups * kHeads * D] dbias, then [slab][groups][2][D] weights
    const size_t wide = (size_t)bp.groups * kHeads * kD;
    __syncthreads();
    store_pairs<kInter>(&red[tl][hs * kD], l, sa, sb);
    __syncthreads();
    for (int c = threadIdx.x; c < kHeads * kD; c += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kTokLanes; ++w) s += red[w][c];
        bp.ws[slab * wide + (size_t)group * kHeads * kD + c] = s;
    }
    __syncthreads();
    store_pairs<kInter>(&red[tl][hs * kD], l, ga, gb);
    __syncthreads();
    if (threadIdx.x < 2 * kD) {
        const int which = threadIdx.x / kD, d = threadIdx.x % kD;  // 0: q, 1: k
        float s = 0.f;
        for (int x = 0; x < kHeads; ++x) {
            const int hh = group * kHeads + x;
            if (which == 0 ? hh < p.Hq : hh >= p.Hq && hh < p.Hq + p.Hkv)
#pragma unroll
                for (int w = 0; w < kTokLanes; ++w) s += red[w][x * kD + d];
        }
        bp.ws[bp.slabs * wide + (((size_t)slab * bp.groups + group) * 2 + which) * kD + d] = s;
    }
}

// column sums over the slabs, in order; the last two CTAs take the weights
__global__ void __launch_bounds__(kThreads) qk_norm_finish_kernel(const BwdParams bp)
{
    grid_dep_wait();
    const int heads = bp.n.Hq + 2 * bp.n.Hkv;
    const size_t wide = (size_t)bp.groups * kHeads * kD;
    __shared__ float red[kThreads];
    const int bias_ctas = gridDim.x - 2;
    const int col = threadIdx.x % kD, part = threadIdx.x / kD;
    constexpr int kParts = kThreads / kD;
    float s = 0.f;
    if ((int)blockIdx.x < bias_ctas) {
        for (int x = part; x < bp.slabs; x += kParts) s += bp.ws[x * wide + (size_t)blockIdx.x * kD + col];
    } else {
        const int which = blockIdx.x - bias_ctas;
        const float *w = bp.ws + bp.slabs * wide;
        for (int x = part; x < bp.slabs * bp.groups; x += kParts) s += w[((size_t)x * 2 + which) * kD + col];
    }
    red[threadIdx.x] = s;
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int w = 1; w < kParts; ++w) s += red[w * kD + col];
    if ((int)blockIdx.x < bias_ctas) {
        if ((int)blockIdx.x < heads) bp.dbias[(size_t)blockIdx.x * kD + col] = s;
    } else {
        (blockIdx.x == (unsigned)bias_ctas ? bp.dqw : bp.dkw)[col] = s;
    }
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
    for (int i = 0; i < kPairs; ++i) p.turns[i] = rope_frequency(r, i) / (2.0 * M_PI);
    return p;
}

}  // namespace

cudaError_t launch_qk_norm_prologue(const void *qkv, const float *bias, const QkNorm &n, const int *positions,
                                    const int *kv_rows, void *q, void *k, void *v, int T, int Hq, int Hkv,
                                    int kv_rows_total, const RopeParams &r, cudaStream_t st)
{
    const NormParams p = norm_params(qkv, bias, n, positions, kv_rows, T, Hq, Hkv, kv_rows_total, r);
    auto kern = r.interleaved ? qk_norm_fwd_kernel<true> : qk_norm_fwd_kernel<false>;
    kern<<<(T + kTok - 1) / kTok, kThreads, 0, st>>>(p, static_cast<__nv_bfloat16 *>(q),
                                                     static_cast<__nv_bfloat16 *>(k),
                                                     static_cast<__nv_bfloat16 *>(v));
    return cudaGetLastError();
}

size_t qk_norm_bwd_workspace_bytes(int T, int Hq, int Hkv)
{
    const size_t groups = head_groups(Hq + 2 * Hkv);
    return (size_t)num_slabs(T) * groups * (kHeads + 2) * kD * sizeof(float);
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
    p.slabs = num_slabs(T);
    p.groups = head_groups(Hq + 2 * Hkv);
    auto kern = r.interleaved ? qk_norm_bwd_kernel<true> : qk_norm_bwd_kernel<false>;
    kern<<<p.slabs * p.groups, kThreads, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((dbias ? Hq + 2 * Hkv : 0) + 2));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qk_norm_finish_kernel, p);
}

}  // namespace attn_sink
