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
// 16 lanes hold one row, 8 channels each; a warp holds two rows at a time and
// walks its share of one token's rows.  Memory bound where nothing is
// quantised: (Hq + 2 Hkv) rows read and written once per token (16384 tokens
// of 32 + 16 heads, 403 MB: 82 us, 4.9 TB/s; without norm and rotation 70 us,
// a plain copy of as much 62 us).  Quantised rows are bound by instructions,
// about 200 for two rows (16384 x 16 rows to groups of 32: 36 us, 2.5 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv4.cuh"

namespace ckv {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kQkvWarps = 4;                   // at least 2: 64 threads fetch the frequencies

// Quantisation of the group that holds this lane's 8 channels: the 16 lanes
// of a row call together; group / 8 neighbouring lanes share a group.
//   scale  = the smallest bfloat16 >= (max - min) / 15
//   middle = min + 8 scale, rounded to float and then to bfloat16
//   code   = clamp(rint((x - middle) / scale), -8, 7), ties to even
// A group that holds an infinity or a NaN gets scale 0 and middle NaN.
// The results are those of the formulas and do not depend on how 32 bits
// round: 32-bit steps decide only where they cannot be wrong, the others
// (a middle of more than 200 scales, where a code may leave its range, very
// small or very large groups, and what kv4_quantise names) are taken again in
// 64 bits.

// the float, or the NaN, of a group's extremes: lo and hi over its lanes
template <int GROUP>
__device__ __forceinline__ void group_extremes(float& lo, float& hi)
{
#pragma unroll
    for (int off = 1; off < GROUP / 8; off <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(kAll, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(kAll, hi, off));
    }
}
// the same for a lane's 8 bfloat16 (4 pairs): two at a time, NaN wins
template <int GROUP>
__device__ __forceinline__ void group_extremes(const uint32_t (&w)[4], float& lo, float& hi)
{
    const auto h = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); };
    __nv_bfloat162 mn = __hmin2_nan(__hmin2_nan(h(w[0]), h(w[1])), __hmin2_nan(h(w[2]), h(w[3])));
    __nv_bfloat162 mx = __hmax2_nan(__hmax2_nan(h(w[0]), h(w[1])), __hmax2_nan(h(w[2]), h(w[3])));
#pragma unroll
    for (int off = 1; off < GROUP / 8; off <<= 1) {
        mn = __hmin2_nan(mn, h(__shfl_xor_sync(kAll, *reinterpret_cast<uint32_t*>(&mn), off)));
        mx = __hmax2_nan(mx, h(__shfl_xor_sync(kAll, *reinterpret_cast<uint32_t*>(&mx), off)));
    }
    lo = __bfloat162float(__hmin_nan(__low2bfloat16(mn), __high2bfloat16(mn)));
    hi = __bfloat162float(__hmax_nan(__low2bfloat16(mx), __high2bfloat16(mx)));
}

// scale and middle from the extremes, in 64 bits
__device__ __noinline__ uint32_t kv4_params_exact(float lo, float hi)
{
    constexpr float kBfMax = 3.3895313892515355e38f;
    const double range = (double)hi - (double)lo;
    uint32_t sb = (__float_as_uint((float)(range * (1.0 / 15.0))) + 0xffffu) & 0xffff0000u;
    if (15.0 * (double)__uint_as_float(sb) < range) sb += 0x10000u;
    else if (sb && 15.0 * (double)__uint_as_float(sb - 0x10000u) >= range) sb -= 0x10000u;
    const float mid = __bfloat162float(__float2bfloat16_rn(fminf(fmaxf(fmaf(8.f, __uint_as_float(sb), lo), -kBfMax), kBfMax)));
    return (__float_as_uint(mid) & 0xffff0000u) | (sb >> 16);
}
// one code, in 64 bits
__device__ __noinline__ int kv4_code_exact(float x, float s, float mid)
{
    const double d = (double)x - (double)mid;
    double c = rint(d / (double)s);                        // off by one at most next to a border
    c = c < -8.0 ? -8.0 : c > 7.0 ? 7.0 : c;
    const double e = fma(c, -(double)s, d), twice = 2.0 * fabs(e);   // exact
    if (twice > (double)s || (twice == (double)s && ((int)c & 1))) c += e > 0.0 ? 1.0 : -1.0;
    return (int)(c < -8.0 ? -8.0 : c > 7.0 ? 7.0 : c);
}

// This lane's codes, four to a register as bytes: channels 0 .. 3 and 4 .. 7
// (K), or the even and the odd ones (V); params: its group's parameters.
// bfloat16 values lie on few points, so that exact ties are common (some lane
// of every second warp has one): their quotients are rounded correctly (a
// quotient that is not a tie is further from one than half a step of its last
// bit), given that x - middle is exact, which is looked at.  Of float values
// x - middle is seldom exact and ties are rare: quotients within 2^-14 of a
// border are looked at again.
template <bool BF16, bool VALUES>
__device__ __forceinline__ void kv4_quantise(const float (&x)[8], float lo, float hi, uint32_t& params, uint32_t (&code)[2])
{
    constexpr float kMagic = 12582912.f;                   // 1.5 * 2^23: adding it rounds to an integer, kept in the low bits
    float bits[8];
    code[0] = code[1] = 0u;
    const float range = hi - lo;
    if (!(fmaxf(fabsf(hi), fabsf(lo)) <= 3.4028234e38f) || hi != hi) {
        params = 0x7fc00000u;                              // scale 0, middle NaN
        return;
    }
    const bool plain = range > 1.0842022e-19f /* 2^-63 */ && fmaxf(fabsf(lo), fabsf(hi)) < 1e38f;
    if (plain) {
        // hi - lo = range + rest exactly; 15 s - range is exact for s next to range / 15
        const float back = range - hi, rest = (hi - (range - back)) - (lo + back);
        uint32_t sb = (__float_as_uint(range * (1.f / 15.f)) + 0xffffu) & 0xffff0000u;
        if (fmaf(15.f, __uint_as_float(sb), -range) < rest) sb += 0x10000u;
        else if (fmaf(15.f, __uint_as_float(sb - 0x10000u), -range) >= rest) sb -= 0x10000u;
        const float mid = __bfloat162float(__float2bfloat16_rn(fmaf(8.f, __uint_as_float(sb), lo)));
        params = (__float_as_uint(mid) & 0xffff0000u) | (sb >> 16);
    } else {
        params = kv4_params_exact(lo, hi);
        if (!(params & 0xffffu)) return;                   // all equal
    }
    const float s = __uint_as_float(params << 16), mid = __uint_as_float(params & 0xffff0000u);
    bool again = !(plain && fabsf(mid) <= 200.f * s);
    const float inv = __frcp_rn(s);
    if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = x[i] - mid;
            again |= d + mid != x[i];
            const float q = d * inv;
            bits[i] = fmaf(fmaf(-q, s, d), inv, q) + kMagic;
        }
    } else {
        const float at0 = -mid * inv;
        float worst = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = fmaf(x[i], inv, at0);          // |q| <= 208: off by 208 * 2^-23 at most
            bits[i] = q + kMagic;
            worst = fmaxf(worst, fabsf(q - (bits[i] - kMagic)));
        }
        again |= !(worst <= 0.5f - 6.103515625e-5f);
    }
    if (again) {
#pragma unroll
        for (int i = 0; i < 8; ++i) bits[i] = kMagic + (float)kv4_code_exact(x[i], s, mid);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i0 = VALUES ? k : 4 * k, step = VALUES ? 2 : 1;
        const uint32_t a = __byte_perm(__float_as_uint(bits[i0]), __float_as_uint(bits[i0 + step]), 0x0040);
        const uint32_t b = __byte_perm(__float_as_uint(bits[i0 + 2 * step]), __float_as_uint(bits[i0 + 3 * step]), 0x0040);
        code[k] = __byte_perm(a, b, 0x5410);
    }
}

// Lane l (0..15) of a row: stores its 8 codes and, on a group's first lane,
// the group's parameters.
template <int GROUP, bool VALUES>
__device__ __forceinline__ void kv4_store(const Kv4& c, int64_t row, int l, const uint32_t (&code)[2], uint32_t params)
{
    unsigned char* p = c.codes + row * kRowCodes;
    const int j = l >> 2, t = l & 3;
    const uint32_t word = (code[0] & 0x0f0f0f0fu) | ((code[1] << 4) & 0xf0f0f0f0u);
    if (VALUES) {
        // channels 8 l .. 8 l + 7 are those of g = 2 t and 2 t + 1: 2 bytes each
        *reinterpret_cast<uint16_t*>(p + 16 * t + 2 * j) = (uint16_t)word;
        *reinterpret_cast<uint16_t*>(p + 16 * t + 8 + 2 * j) = (uint16_t)(word >> 16);
    } else {
        *reinterpret_cast<uint32_t*>(p + 16 * t + 4 * j) = word;
    }
    constexpr int lanes = GROUP / 8;
    if (l % lanes == 0) c.params[row * (kD / GROUP) + l / lanes] = params;
}

// the inverse: lane l's 8 values of a row
template <int GROUP, bool VALUES>
__device__ __forceinline__ void kv4_load(const Kv4& c, int64_t row, int l, float (&x)[8])
{
    const unsigned char* p = c.codes + row * kRowCodes;
    const int j = l >> 2, t = l & 3;
    uint32_t w;
    if (VALUES)
        w = *reinterpret_cast<const uint16_t*>(p + 16 * t + 2 * j) |
            (uint32_t) * reinterpret_cast<const uint16_t*>(p + 16 * t + 8 + 2 * j) << 16;
    else
        w = *reinterpret_cast<const uint32_t*>(p + 16 * t + 4 * j);
    const uint32_t params = c.params[row * (kD / GROUP) + l / (GROUP / 8)];
    const float s = __uint_as_float(params << 16), mid = __uint_as_float(params & 0xffff0000u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // channel i: byte i / 2, nibble i % 2 (V), or byte i % 4, nibble i / 4 (K)
        const int at = VALUES ? 4 * i : 8 * (i & 3) + 4 * (i >> 2);
        x[i] = fmaf(s, (float)((int32_t)(w << (28 - at)) >> 28), mid);
    }
}

// 8 channels of a row as they lie in memory, in two chunks of 4.  Lane l of
// the row's 16 holds channels 8 l .. 8 l + 7 (whole), or 4 l .. 4 l + 3 and
// 64 + 4 l .. 64 + 4 l + 3 (split).
template <bool BF16, bool SPLIT>
struct Raw {
    static constexpr int W = BF16 ? 2 : 4;                 // words of a chunk
    uint32_t w[2 * W];

    static __device__ __forceinline__ int64_t at(int l) { return SPLIT ? 4 * l : 8 * l; }
    __device__ __forceinline__ void load(const void* base, int64_t elem)
    {
        const char* p = static_cast<const char*>(base) + elem * (BF16 ? 2 : 4);
        if constexpr (BF16 && !SPLIT) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const char* q = p + i * (SPLIT ? 64 * (BF16 ? 2 : 4) : 16);
                if constexpr (BF16) {
                    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(q));
                    w[2 * i] = v.x; w[2 * i + 1] = v.y;
                } else {
                    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(q));
                    w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
                }
            }
        }
    }
    __device__ __forceinline__ void store(void* base, int64_t elem) const
    {
        char* p = static_cast<char*>(base) + elem * (BF16 ? 2 : 4);
        if constexpr (BF16 && !SPLIT) {
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                char* q = p + i * (SPLIT ? 64 * (BF16 ? 2 : 4) : 16);
                if constexpr (BF16) *reinterpret_cast<uint2*>(q) = make_uint2(w[2 * i], w[2 * i + 1]);
                else *reinterpret_cast<uint4*>(q) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
        }
    }
    __device__ __forceinline__ void floats(float (&x)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = BF16 ? __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16) : __uint_as_float(w[i]);
    }
    // rounded to the cache's type
    __device__ __forceinline__ void set(const float (&x)[8])
    {
        if constexpr (BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
        }
    }
    template <int GROUP>
    __device__ __forceinline__ void extremes(const float (&x)[8], float& lo, float& hi) const
    {
        if constexpr (BF16) {
            group_extremes<GROUP>(w, lo, hi);
        } else {
            float nan = 0.f;
            lo = hi = x[0];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lo = fminf(lo, x[i]);
                hi = fmaxf(hi, x[i]);
                nan = fmaf(x[i], 0.f, nan);
            }
            if (nan != 0.f) hi = INFINITY;     // a NaN, or an infinity
            group_extremes<GROUP>(lo, hi);
        }
    }
};

// Cosine and sine of t revolutions in 64 bits, rounded once: t less the
// nearest quarter, then the Taylor series to the 14th and 15th power of the
// angle, at most pi / 4 (the next terms are below 2^-49).
__device__ __forceinline__ void turn_by(double t, float& c, float& s)
{
    t -= rint(t);
    const double quarter = rint(4.0 * t);
    const double x = (t - 0.25 * quarter) * 6.283185307179586476925286766559, z = x * x;
    const double sn = x * fma(z, fma(z, fma(z, fma(z, fma(z, fma(z, -1.0 / 1307674368000.0 * z + 1.0 / 6227020800.0,
                      -1.0 / 39916800.0), 1.0 / 362880.0), -1.0 / 5040.0), 1.0 / 120.0), -1.0 / 6.0), 1.0);
    const double cs = fma(z, fma(z, fma(z, fma(z, fma(z, fma(z, fma(z, -1.0 / 87178291200.0, 1.0 / 479001600.0),
                      -1.0 / 3628800.0), 1.0 / 40320.0), -1.0 / 720.0), 1.0 / 24.0), -0.5), 1.0);
    const int q = (int)quarter & 3;
    const float a = (float)(q & 1 ? sn : cs), b = (float)(q & 1 ? cs : sn);
    c = q == 1 || q == 2 ? -a : a;
    s = q >= 2 ? -b : b;
}

// A token's cosines and sines: lane (l, half) = (lane % 16, lane / 16) has
// those of pairs 4 l + 2 half and + 1.
struct Turns {
    float c[2], s[2];
    // freq: the frequencies in shared memory (read by lane from the kernel's
    // arguments, they would come one lane at a time)
    __device__ __forceinline__ Turns(const QkvArgs& a, const double* freq, int pos)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = 4 * (lane & 15) + 2 * (lane >> 4) + k;
            c[k] = 1.f;
            s[k] = 0.f;
            if (i < a.rot / 2) {
                turn_by((double)pos * freq[i], c[k], s[k]);
                c[k] *= a.rot_scale;
                s[k] *= a.rot_scale;
            }
        }
    }
    // those of pair i; all lanes call
    __device__ __forceinline__ void of(int i, float& ci, float& si) const
    {
        const int from = (i >> 2) + 8 * (i & 2);
        const float c0 = __shfl_sync(kAll, c[0], from), c1 = __shfl_sync(kAll, c[1], from);
        const float s0 = __shfl_sync(kAll, s[0], from), s1 = __shfl_sync(kAll, s[1], from);
        ci = i & 1 ? c1 : c0;
        si = i & 1 ? s1 : s0;
    }
};

// Sum of the 128 squares of a row over its 16 lanes, in a fixed order: four
// neighbours one after the other, then the 32 sums of four by halves (i with
// i + 16, i + 8, ..).  torch's mean over a row of 128 was measured to add in
// this order, so rows, and with them 4-bit codes, where one rounding can move
// a whole group, equal those of an eager norm and not only nearly.
template <bool SPLIT>
__device__ __forceinline__ float sum_squares(const float (&x)[8])
{
    float s[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        s[k] = __fmul_rn(x[4 * k], x[4 * k]);
#pragma unroll
        for (int i = 1; i < 4; ++i) s[k] = __fadd_rn(s[k], __fmul_rn(x[4 * k + i], x[4 * k + i]));
    }
    if constexpr (SPLIT) {
        // sums l and l + 16 are this lane's
        float t = __fadd_rn(s[0], s[1]);
#pragma unroll
        for (int off = 8; off; off >>= 1) t = __fadd_rn(t, __shfl_xor_sync(kAll, t, off));
        return t;
    } else {
        // sums 2 l and 2 l + 1
#pragma unroll
        for (int off = 8; off; off >>= 1) {
            s[0] = __fadd_rn(s[0], __shfl_xor_sync(kAll, s[0], off));
            s[1] = __fadd_rn(s[1], __shfl_xor_sync(kAll, s[1], off));
        }
        return __fadd_rn(s[0], s[1]);
    }
}

// The rotation of a lane's channels: x[e] c[e] + partner s[e], s with its sign.
// Products and sums are rounded one by one, as the formula has them.
template <bool SPLIT>
struct Rotation {
    float c[8], s[8];        // interleaved: of the lane's 4 pairs, in [0, 4)

    static __device__ __forceinline__ int channel(int l, int e) { return SPLIT ? (e < 4 ? 4 * l + e : 60 + 4 * l + e) : 8 * l + e; }
    __device__ __forceinline__ void make(const QkvArgs& a, const double* freq, int pos)
    {
        const Turns turns(a, freq, pos);
        const int l = threadIdx.x & 15, half = a.rot / 2;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (a.interleaved && e >= 4) break;
            const int ch = channel(l, a.interleaved ? 2 * e : e);
            const int pair = a.interleaved ? ch / 2 : ch < half ? ch : ch - half;
            turns.of(pair & 63, c[e], s[e]);
            if (!a.interleaved && ch < half) s[e] = -s[e];
            if (ch >= a.rot) { c[e] = 1.f; s[e] = 0.f; }
        }
    }
    // all lanes call
    __device__ __forceinline__ void apply(const QkvArgs& a, float (&x)[8]) const
    {
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (channel(threadIdx.x & 15, 2 * i) >= a.rot) continue;   // kept as they are, an infinity or a NaN too
                const float u = x[2 * i], v = x[2 * i + 1];
                x[2 * i] = __fsub_rn(__fmul_rn(u, c[i]), __fmul_rn(v, s[i]));
                x[2 * i + 1] = __fadd_rn(__fmul_rn(v, c[i]), __fmul_rn(u, s[i]));
            }
            return;
        }
        const int lane = threadIdx.x & 31, l = lane & 15, half = a.rot / 2;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int ch = channel(l, e), other = ch >= a.rot ? ch : ch < half ? ch + half : ch - half;
            float o;
            if (SPLIT) {
                // half is a multiple of 8, so the partner is element e % 4 of a chunk
                const int from = (lane & 16) + (other & 63) / 4;
                const float lo = __shfl_sync(kAll, x[e & 3], from), hi = __shfl_sync(kAll, x[4 + (e & 3)], from);
                o = other < 64 ? lo : hi;
            } else {
                o = __shfl_sync(kAll, x[e], (lane & 16) + other / 8);
            }
            y[e] = ch < a.rot ? __fadd_rn(__fmul_rn(x[e], c[e]), __fmul_rn(o, s[e])) : x[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = y[e];
    }
};
// All 128 channels in pairs (i, i + 64) of split rows: both are the lane's.
struct Halves {
    float c[4], s[4];

    __device__ __forceinline__ void make(const QkvArgs& a, const double* freq, int pos)
    {
        const Turns turns(a, freq, pos);
        const bool high = threadIdx.x & 16;                // this lane's own pairs are 4 l + 2 and + 3
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float oc = __shfl_xor_sync(kAll, turns.c[k], 16), os = __shfl_xor_sync(kAll, turns.s[k], 16);
            c[k] = high ? oc : turns.c[k];
            s[k] = high ? os : turns.s[k];
            c[2 + k] = high ? turns.c[k] : oc;
            s[2 + k] = high ? turns.s[k] : os;
        }
    }
    __device__ __forceinline__ void apply(const QkvArgs&, float (&x)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = x[i], v = x[i + 4];
            x[i] = __fsub_rn(__fmul_rn(u, c[i]), __fmul_rn(v, s[i]));
            x[i + 4] = __fadd_rn(__fmul_rn(v, c[i]), __fmul_rn(u, s[i]));
        }
    }
};
struct NoTurn {
    __device__ __forceinline__ void make(const QkvArgs&, const double*, int) {}
    __device__ __forceinline__ void apply(const QkvArgs&, float (&)[8]) const {}
};

enum { kQuery = 0, kKey = 1, kValue = 2 };

// A warp: heads [h0, h1) of one token's queries, keys or values, two at a
// time (16 lanes a row), kAhead loads under way: where no warp has more than
// 8 rows (not LONG), all of them are before the token's angles are made.
// Rows that are not quantised are held split, where a pair (i, i + 64) is one
// lane's; a group of a quantised row lies in few lanes only if they are whole.
template <bool BF16, int KIND, int GROUP, bool LONG, bool NORM, class Turn>
__device__ __forceinline__ void do_rows(const QkvArgs& a, const double* freq, int b, int t, int pos, int h0, int h1)
{
    constexpr bool SPLIT = GROUP == 0;
    constexpr int ESZ = BF16 ? 2 : 4, kAhead = GROUP ? 1 : 4;
    using R = Raw<BF16, SPLIT>;
    const int lane = threadIdx.x & 31, l = lane & 15, half = lane >> 4;
    const RowSource& src = KIND == kQuery ? a.q : KIND == kKey ? a.k : a.v;
    const char* from = static_cast<const char*>(src.data) + (b * src.batch + t * src.token + (h0 + half) * src.head + R::at(l)) * ESZ;
    const int64_t step = 2 * src.head * ESZ;
    // where the row goes: q_out, or the cache's row of this position
    char* to = static_cast<char*>(KIND == kQuery ? a.q_out : KIND == kKey ? a.K : a.V);
    const bool plain = to != nullptr;
    const int64_t to_step = 2 * (KIND == kQuery ? a.q_out_head : (int64_t)a.n_max * kD) * ESZ;
    const int64_t unit0 = (int64_t)b * a.Hkv + h0 + half;
    if (KIND == kQuery) to += (b * a.q_out_batch + t * a.q_out_token + (h0 + half) * a.q_out_head + R::at(l)) * ESZ;
    else to += ((unit0 * a.n_max + pos) * kD + R::at(l)) * ESZ;
    const Kv4& four = KIND == kKey ? a.K4 : a.V4;
    int64_t row4 = unit0 * four.R + pos;
    R next[kAhead], w;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        if (h0 + half + 2 * i < h1) next[i].load(from, 0);
        from += step;
    }
    if (NORM) w.load(KIND == kQuery ? a.q_weight : a.k_weight, R::at(l));
    Turn turn;
    turn.make(a, freq, pos);
    for (int left = h1 - h0; left > 0;) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (left <= 0) break;
            R raw = next[i];
            if (LONG) {
                if (half + 2 * kAhead < left) next[i].load(from, 0);
                from += step;
            }
            const bool live = half < left;
            float x[8];
            if (KIND != kValue || GROUP) raw.floats(x);
            if (KIND != kValue) {
                if (NORM) {
                    const float r = rsqrtf(fmaf(sum_squares<SPLIT>(x), 1.f / kD, a.eps));
                    float f[8];
                    w.floats(f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = x[e] * r * f[e];
                }
                turn.apply(a, x);
                raw.set(x);
            }
            if (plain) {
                if (live) raw.store(to, 0);
                to += to_step;
            }
            if constexpr (GROUP != 0 && KIND != kQuery) {
                if (KIND == kKey) raw.floats(x);           // as the cache rounds them
                float lo, hi;
                uint32_t params, code[2];
                raw.template extremes<GROUP>(x, lo, hi);
                // not the lanes beside a last odd row: whatever their registers
                // hold would take the warp through the 64-bit steps (2 x 88410
                // rows of one head: 170 us, 70 without)
                if (live) {
                    kv4_quantise<BF16, KIND == kValue>(x, lo, hi, params, code);
                    kv4_store<GROUP, KIND == kValue>(four, row4, l, code, params);
                }
                row4 += 2 * four.R;
            }
            left -= 2;
        }
        if (!LONG) break;
    }
}

// queries or keys: with or without a norm, and by the kind of rotation
template <bool BF16, int KIND, int GROUP, bool LONG>
__device__ __forceinline__ void do_turned(const QkvArgs& a, const double* freq, int b, int t, int pos, int h0, int h1)
{
    const bool norm = (KIND == kQuery ? a.q_weight : a.k_weight) != nullptr;
    if constexpr (GROUP == 0) {
        if (a.rot == kD && !a.interleaved) {
            if (norm) do_rows<BF16, KIND, GROUP, LONG, true, Halves>(a, freq, b, t, pos, h0, h1);
            else do_rows<BF16, KIND, GROUP, LONG, false, Halves>(a, freq, b, t, pos, h0, h1);
            return;
        }
    }
    if (a.rot) {
        if (norm) do_rows<BF16, KIND, GROUP, LONG, true, Rotation<GROUP == 0>>(a, freq, b, t, pos, h0, h1);
        else do_rows<BF16, KIND, GROUP, LONG, false, Rotation<GROUP == 0>>(a, freq, b, t, pos, h0, h1);
    } else {
        if (norm) do_rows<BF16, KIND, GROUP, LONG, true, NoTurn>(a, freq, b, t, pos, h0, h1);
        else do_rows<BF16, KIND, GROUP, LONG, false, NoTurn>(a, freq, b, t, pos, h0, h1);
    }
}

// One warp: rows [r0, r1) of one token, q heads, then k heads, then v heads.
// Few rows to a warp: what the machine works on at once then lies within some
// megabytes of each tensor, which the memory needs for its bandwidth (without
// norm and rotation, 16384 tokens of 32 + 16 heads: 84 us with a token to a
// warp, whatever the depth of its loads).
template <bool BF16, int GROUP>
__global__ void __launch_bounds__(32 * kQkvWarps, GROUP || BF16 ? 8 : 6) k_qkv(const __grid_constant__ QkvArgs a, int per_warp, int slices)
{
    constexpr bool LONG = GROUP != 0;
    __shared__ double freq[kD / 2];
    if (threadIdx.x < a.rot / 2) freq[threadIdx.x] = a.turn[threadIdx.x];
    if (a.rot) __syncthreads();
    const int64_t w = (int64_t)blockIdx.x * kQkvWarps + (threadIdx.x >> 5);
    const int token = (int)(w / slices);
    if (token >= a.B * a.T) return;
    const int b = token / a.T, t = token - b * a.T;
    const int pos = a.pos ? a.pos[token] : t;
    if (pos < 0 || pos >= a.n_max) return;             // padding: nothing of this token is written
    const int nq = a.q.data ? a.Hq : 0, nk = nq + a.Hkv, rows = nk + a.Hkv;
    const int r0 = (int)(w - (int64_t)token * slices) * per_warp, r1 = min(r0 + per_warp, rows);
    if (r0 < nq) do_turned<BF16, kQuery, 0, LONG>(a, freq, b, t, pos, r0, min(r1, nq));
    if (r0 < nk && r1 > nq) do_turned<BF16, kKey, GROUP, LONG>(a, freq, b, t, pos, max(r0, nq) - nq, min(r1, nk) - nq);
    if (r1 > nk) do_rows<BF16, kValue, GROUP, LONG, false, NoTurn>(a, freq, b, t, pos, max(r0, nk) - nk, r1 - nk);
}

// 16 lanes a row, kReadRows rows 16 apart for each lane: their K, their V, or
// both, all loaded before the first is stored
constexpr int kReadRows = 2;
template <bool BF16, int GROUP>
__global__ void __launch_bounds__(256) k_kv4_read(const __grid_constant__ Kv4ReadArgs a)
{
    const int l = threadIdx.x & 15;
    const int i0 = blockIdx.x * (16 * kReadRows) + (threadIdx.x >> 4);   // row of the unit's range
    const int64_t unit = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (unit >= a.units) return;
    const int64_t row0 = a.first + i0;
    float x[kReadRows][8], y[kReadRows][8];
#pragma unroll
    for (int k = 0; k < kReadRows; ++k) {
        if (i0 + 16 * k >= a.count) break;
        if (a.K) kv4_load<GROUP, false>(a.K4, unit * a.K4.R + row0 + 16 * k, l, x[k]);
        if (a.V) kv4_load<GROUP, true>(a.V4, unit * a.V4.R + row0 + 16 * k, l, y[k]);
    }
    const int64_t to = (unit * a.n_max + row0) * kD + 8 * l;
    Raw<BF16, false> raw;
#pragma unroll
    for (int k = 0; k < kReadRows; ++k) {
        if (i0 + 16 * k >= a.count) break;
        if (a.K) {
            raw.set(x[k]);
            raw.store(a.K, to + 16 * k * kD);
        }
        if (a.V) {
            raw.set(y[k]);
            raw.store(a.V, to + 16 * k * kD);
        }
    }
}

template <bool BF16>
cudaError_t launch_qkv_t(const QkvArgs& a, int sms, cudaStream_t st)
{
    const int rows = (a.q.data ? a.Hq : 0) + 2 * a.Hkv;
    const int64_t tokens = (int64_t)a.B * a.T;
    // Few rows: two to a warp, spread over the machine.  Many: eight, which
    // share the work on the token's angles; rows to quantise are bound by
    // their arithmetic, so as many of a token as leave 32 warps to an SM
    // (16384 tokens of 32 + 16 heads: 101 us, eight to a warp 140 us; 2000
    // tokens: a whole token to a warp 20.7 us).
    const int64_t all = tokens * rows;
    int per_warp = all <= (int64_t)sms * 128 ? 2 : 8;
    if (a.group && per_warp == 8) {
        const int64_t fair = all / ((int64_t)sms * 32) / 2 * 2;
        per_warp = fair < 8 ? 8 : fair < rows ? (int)fair : rows;
    }
    const int slices = (rows + per_warp - 1) / per_warp;
    const int64_t grid = (tokens * slices + kQkvWarps - 1) / kQkvWarps;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    auto fn = a.group == 0 ? k_qkv<BF16, 0> : a.group == 32 ? k_qkv<BF16, 32> : a.group == 64 ? k_qkv<BF16, 64> : k_qkv<BF16, 128>;
    return launch_kernel(fn, dim3((unsigned)grid), 32 * kQkvWarps, 0, st, a, per_warp, slices);
}

template <bool BF16>
cudaError_t launch_read_t(const Kv4ReadArgs& a, cudaStream_t st)
{
    const int64_t y = a.units < 32768 ? a.units : 32768, z = (a.units + y - 1) / y;
    const dim3 grid((unsigned)((a.count - 1) / (16 * kReadRows) + 1), (unsigned)y, (unsigned)z);
    auto fn = a.group == 32 ? k_kv4_read<BF16, 32> : a.group == 64 ? k_kv4_read<BF16, 64> : k_kv4_read<BF16, 128>;
    return launch_kernel(fn, grid, 256, 0, st, a);
}

}  // namespace

cudaError_t launch_qkv(const QkvArgs& a, int bf16, int sms, cudaStream_t st)
{
    return bf16 ? launch_qkv_t<true>(a, sms, st) : launch_qkv_t<false>(a, sms, st);
}

cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int bf16, cudaStream_t st)
{
    return bf16 ? launch_read_t<true>(a, st) : launch_read_t<false>(a, st);
}

}  // namespace ckv
