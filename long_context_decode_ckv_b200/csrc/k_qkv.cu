// k_qkv.cu -- rows into the caches: the norm of queries and keys for each
// head with the position rotation in the same pass, rows written to 16/32-bit
// caches or quantised into 4-bit caches, and 4-bit rows read back.
//
// For a row x of 128 channels at position p:
//   y   = x / sqrt(mean(x^2) + eps) * w          (w null: y = x)
//   a'  = (a cos - b sin) scale, b' = (b cos + a sin) scale
// for the pairs (a, b) of the first `rot` channels: (i, i + rot/2), or
// (2i, 2i+1) when interleaved, with the angle p * inv_freq[i].  All of it in
// 32 bits with one rounding at the end, except the angle: it is formed in
// revolutions in 64 bits (p * inv_freq / 2 pi) and reduced to [-1/2, 1/2], and
// its cosine and sine are rounded once, since a 32-bit angle at position
// 131072 would be off by up to 2^-8 radians.
//
// 16 lanes hold one row, 8 channels each (one 16-byte load of bfloat16); a
// warp holds two rows at a time and walks the rows of its share of one token,
// so the token's angles are formed once.  Memory bound: (Hq + 2 Hkv) rows
// read and written once per token.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv4.cuh"

namespace ckv {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kQkvWarps = 4;

template <bool BF16>
struct Row8 {
    static __device__ __forceinline__ void load(const void* base, int64_t elem, float (&x)[8])
    {
        if (BF16) {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + elem);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
            const float4 a = p[0], b = p[1];
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        }
    }
    static __device__ __forceinline__ void store(void* base, int64_t elem, const float (&x)[8])
    {
        if (BF16) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + elem) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
            p[0] = make_float4(x[0], x[1], x[2], x[3]);
            p[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    }
    // the value a cache of this type would hold
    static __device__ __forceinline__ float rounded(float v)
    {
        return BF16 ? __bfloat162float(__float2bfloat16_rn(v)) : v;
    }
};

// cosines and sines of a lane's 8 channels (interleaved: of its 4 pairs, in [0, 4))
struct Angles {
    float c[8], s[8];
};

// All lanes call.  Lane i forms the angles of pairs i and i + 32 in 64 bits
// and rounds them once; the lanes then fetch those of their channels.
__device__ __forceinline__ void make_angles(const QkvArgs& a, int pos, int lane, Angles& g)
{
    const int l = lane & 15, half = a.rot / 2;
    float c[2] = {1.f, 1.f}, s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = lane + 32 * k;
        if (i < half) {
            const double t = (double)pos * a.turn[i];
            double sn, cs;
            sincospi(2.0 * (t - rint(t)), &sn, &cs);
            c[k] = (float)cs * a.rot_scale;
            s[k] = (float)sn * a.rot_scale;
        }
    }
    const int i0 = a.interleaved ? 4 * l : (8 * l < half ? 8 * l : 8 * l - half);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int at = i0 + i;                          // lanes from rot on fetch what they do not use
        const float c0 = __shfl_sync(kAll, c[0], at & 31), c1 = __shfl_sync(kAll, c[1], at & 31);
        const float s0 = __shfl_sync(kAll, s[0], at & 31), s1 = __shfl_sync(kAll, s[1], at & 31);
        g.c[i] = at & 32 ? c1 : c0;
        g.s[i] = at & 32 ? s1 : s0;
    }
}

// Sum of the 128 squares of a row over its 16 lanes, in a fixed order: four
// neighbours one after the other, then the 32 sums of four by halves (i with
// i + 16, i + 8, ..).  torch's mean over a row of 128 was measured to add in
// this order, so rows, and with them 4-bit codes, where one rounding can move
// a whole group, equal those of an eager norm and not only nearly.
__device__ __forceinline__ float sum_squares(const float (&x)[8])
{
    float s[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        s[k] = __fmul_rn(x[4 * k], x[4 * k]);
#pragma unroll
        for (int i = 1; i < 4; ++i) s[k] = __fadd_rn(s[k], __fmul_rn(x[4 * k + i], x[4 * k + i]));
    }
#pragma unroll
    for (int off = 8; off; off >>= 1) {
        s[0] = __fadd_rn(s[0], __shfl_xor_sync(kAll, s[0], off));
        s[1] = __fadd_rn(s[1], __shfl_xor_sync(kAll, s[1], off));
    }
    return __fadd_rn(s[0], s[1]);
}

// every lane calls; lanes at or above rot keep their channels.  Products and
// sums are rounded one by one, as the formula has them.
__device__ __forceinline__ void rotate8(const QkvArgs& a, int lane, float (&x)[8], const Angles& g)
{
    const int l = lane & 15;
    if (a.rot == 0) return;
    if (a.interleaved) {
        if (8 * l < a.rot) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = x[2 * i], v = x[2 * i + 1];
                x[2 * i] = __fsub_rn(__fmul_rn(u, g.c[i]), __fmul_rn(v, g.s[i]));
                x[2 * i + 1] = __fadd_rn(__fmul_rn(v, g.c[i]), __fmul_rn(u, g.s[i]));
            }
        }
        return;
    }
    const int step = a.rot / 16;                       // lanes between a pair's halves
    const bool first = l < step, in = 8 * l < a.rot;
    const int from = in ? (first ? lane + step : lane - step) : lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float o = __fmul_rn(__shfl_sync(kAll, x[i], from), g.s[i]), u = __fmul_rn(x[i], g.c[i]);
        if (in) x[i] = first ? __fsub_rn(u, o) : __fadd_rn(u, o);
    }
}

// One warp: rows [r0, r1) of one token (q heads, then k heads, then v
// heads), two at a time.
template <bool BF16>
__global__ void __launch_bounds__(32 * kQkvWarps) k_qkv(const __grid_constant__ QkvArgs a, int per_warp, int slices)
{
    using Row = Row8<BF16>;
    const int lane = threadIdx.x & 31, l = lane & 15, half = lane >> 4;
    const int64_t w = (int64_t)blockIdx.x * kQkvWarps + (threadIdx.x >> 5);
    const int64_t token = w / slices;
    if (token >= (int64_t)a.B * a.T) return;
    const int b = (int)(token / a.T), t = (int)(token % a.T);
    const int pos = a.pos ? a.pos[token] : t;
    if (pos < 0 || pos >= a.n_max) return;             // padding: nothing of this token is written
    const int nq = a.q.data ? a.Hq : 0, rows = nq + 2 * a.Hkv;
    const int r0 = (int)(w % slices) * per_warp, r1 = min(r0 + per_warp, rows);
    Angles g;
    if (a.rot) make_angles(a, pos, lane, g);
    float wq[8], wk[8];
    if (a.q_weight) Row::load(a.q_weight, 8 * l, wq);
    if (a.k_weight) Row::load(a.k_weight, 8 * l, wk);
    for (int rr = r0; rr < r1; rr += 2) {
        const int r = rr + half;
        const bool live = r < r1;
        // the two halves of a warp may hold rows of different kinds, so every
        // step that shuffles is run by all lanes
        const int kind = r < nq ? 0 : r < nq + a.Hkv ? 1 : 2;
        const int h = kind == 0 ? r : kind == 1 ? r - nq : r - nq - a.Hkv;
        const RowSource& src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        const bool has = live && src.data;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
        if (has) Row::load(src.data, b * src.batch + t * src.token + h * src.head + 8 * l, x);
        if (a.q_weight || a.k_weight) {
            const float r = rsqrtf(fmaf(sum_squares(x), 1.f / kD, a.eps));
            const bool normed = kind == 0 ? a.q_weight != nullptr : kind == 1 && a.k_weight != nullptr;
            if (normed) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (kind == 0 ? wq[i] : wk[i]);
            }
        }
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i];
        rotate8(a, lane, y, g);
        if (kind < 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = y[i];
        }
        if (has && kind == 0)
            Row::store(a.q_out, b * a.q_out_batch + t * a.q_out_token + h * a.q_out_head + 8 * l, x);
        const int64_t unit = (int64_t)b * a.Hkv + h;
        void* cache = kind == 1 ? a.K : a.V;
        if (has && kind && cache) Row::store(cache, (unit * a.n_max + pos) * kD + 8 * l, x);
        if (a.group) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = Row::rounded(x[i]);
            uint32_t params;
            const uint32_t word = kv4_quantise(x, a.group, params);
            if (has && kind == 1) kv4_store<false>(a.K4, unit * a.K4.R + pos, a.group, l, word, params);
            if (has && kind == 2) kv4_store<true>(a.V4, unit * a.V4.R + pos, a.group, l, word, params);
        }
    }
}

template <bool BF16>
__global__ void __launch_bounds__(256) k_kv4_read(Kv4ReadArgs a)
{
    const int l = threadIdx.x & 15;
    const int64_t i = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    if (i >= a.units * a.count) return;
    const int64_t unit = i / a.count;
    const int64_t row = a.first + i % a.count;
    float x[8];
    if (a.K) {
        kv4_load<false>(a.K4, unit * a.K4.R + row, a.group, l, x);
        Row8<BF16>::store(a.K, (unit * a.n_max + row) * kD + 8 * l, x);
    }
    if (a.V) {
        kv4_load<true>(a.V4, unit * a.V4.R + row, a.group, l, x);
        Row8<BF16>::store(a.V, (unit * a.n_max + row) * kD + 8 * l, x);
    }
}

}  // namespace

cudaError_t launch_qkv(const QkvArgs& a, int bf16, int sms, cudaStream_t st)
{
    const int rows = (a.q.data ? a.Hq : 0) + 2 * a.Hkv;
    const int64_t tokens = (int64_t)a.B * a.T;
    const int per_warp = tokens * rows <= (int64_t)sms * 64 ? 2 : rows;
    const int slices = (rows + per_warp - 1) / per_warp;
    const int64_t grid = (tokens * slices + kQkvWarps - 1) / kQkvWarps;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    if (bf16) k_qkv<true><<<(unsigned)grid, 32 * kQkvWarps, 0, st>>>(a, per_warp, slices);
    else k_qkv<false><<<(unsigned)grid, 32 * kQkvWarps, 0, st>>>(a, per_warp, slices);
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int bf16, cudaStream_t st)
{
    const int64_t grid = (a.units * a.count + 15) / 16;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    if (bf16) k_kv4_read<true><<<(unsigned)grid, 256, 0, st>>>(a);
    else k_kv4_read<false><<<(unsigned)grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace ckv
