// kv4.cuh -- the 4-bit KV cache: its format, the quantisation of one row by
// 16 lanes, and the launchers of the kernels that write, read and attend to it.
//
// One cache (K or V) is one buffer: codes [B][Hkv][R][64 bytes], then params
// [B][Hkv][R][D / group] of 4 bytes (low half: bfloat16 scale, high half:
// bfloat16 middle), R = n_max rounded up to 16 rows, so that every run of 16
// rows starts and ends on 16 bytes in both parts.  A channel's value is
// middle + scale * code, code in [-8, 7] as a two's complement nibble.
//
// Byte order within a row, chosen for the attention kernel's fragments (h = 0
// is the low nibble):
//   K: channel 32 j + 8 t + 4 h + i  ->  byte 16 t + 4 j + i.  Lane t of a
//      quad loads its 16 bytes at once; word j is its share of channels
//      32 j .. 32 j + 31 (the integer MMA's k32 step j), the two nibble
//      halves are the step's two B registers.
//   V: channel 32 j + 4 g + 2 i + h  ->  byte 8 g + 2 j + i.  Lane group g
//      loads its 8 bytes at once and holds 4 channels of each block of 32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ckv_internal.cuh"

namespace ckv {

constexpr int kRowCodes = kD / 2;              // code bytes of one row

__host__ __device__ inline int64_t kv4_rows(int n_max) { return ((int64_t)n_max + 15) / 16 * 16; }

// one 4-bit cache as the kernels see it
struct Kv4 {
    unsigned char* codes;    // [units][R][64]
    uint32_t* params;        // [units][R][D / group]
    int64_t R;
};

__host__ inline Kv4 kv4_view(void* buf, int64_t units, int n_max)
{
    const int64_t R = kv4_rows(n_max);
    unsigned char* p = static_cast<unsigned char*>(buf);
    return Kv4{p, reinterpret_cast<uint32_t*>(p + units * R * kRowCodes), R};
}

// Parameters of the group that holds this lane's 8 channels, and their codes
// as 8 nibbles (channel e in bits 4e .. 4e+3).  The 16 lanes of a row call
// together; group / 8 neighbouring lanes share a group.
//   scale  = the smallest bfloat16 >= (max - min) / 15
//   middle = min + 8 scale, rounded to float and then to bfloat16
//   code   = clamp(rint((x - middle) / scale), -8, 7), ties to even
// A group that holds an infinity or a NaN gets scale 0 and middle NaN.
// The scale and every code next to a rounding border are decided in 64 bits,
// so they are those of the formulas and do not depend on how a division
// rounds; 32 bits decide only codes that lie 2^-14 or more from a border,
// which is above the 2^-20 that the 32-bit quotient can be off.
__device__ __forceinline__ uint32_t kv4_quantise(const float (&x)[8], int group, uint32_t& params)
{
    constexpr float kBfMax = 3.3895313892515355e38f;
    float lo = x[0], hi = x[0], nan = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        nan = fmaf(x[i], 0.f, nan);            // NaN as soon as one value is not finite
    }
    if (nan != 0.f) hi = INFINITY;             // (NaN != 0 is true)
    for (int off = 1; off < group / 8; off <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    if (hi == INFINITY) {
        params = 0x7fc00000u;                  // scale 0, middle NaN
        return 0u;
    }
    const double range = (double)hi - (double)lo;
    uint32_t sb = (__float_as_uint((float)(range * (1.0 / 15.0))) + 0xffffu) & 0xffff0000u;
    if (15.0 * (double)__uint_as_float(sb) < range) sb += 0x10000u;
    else if (sb && 15.0 * (double)__uint_as_float(sb - 0x10000u) >= range) sb -= 0x10000u;
    const float s = __uint_as_float(sb);
    const float mid = __bfloat162float(__float2bfloat16_rn(fminf(fmaxf(fmaf(8.f, s, lo), -kBfMax), kBfMax)));
    params = (__float_as_uint(mid) & 0xffff0000u) | (sb >> 16);
    if (sb == 0u) return 0u;
    // very small scales are moved up by a power of two, so that 1 / scale exists
    const float up = s < 8.6736174e-19f /* 2^-60 */ ? 18446744073709551616.f /* 2^64 */ : 1.f;
    const float inv = 1.f / (s * up);
    uint32_t word = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = (x[i] - mid) * up * inv;
        float c = rintf(q);
        if (fabsf(q - c) > 0.5f - 6.103515625e-5f) {
            const double e = fma((double)c, -(double)s, (double)x[i] - (double)mid);   // exact
            const double twice = 2.0 * fabs(e);
            if (twice > (double)s || (twice == (double)s && ((int)c & 1))) c += e > 0.0 ? 1.f : -1.f;
        }
        const int code = (int)fminf(fmaxf(c, -8.f), 7.f);
        word |= (uint32_t)(code & 15) << (4 * i);
    }
    return word;
}

// 8 nibbles (channel e at bits 4e) -> the K row's word (codes e and e + 4 share byte e)
__device__ __forceinline__ uint32_t kv4_k_word(uint32_t w)
{
    uint32_t r = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= ((w >> (4 * i)) & 15u) << (8 * i) | ((w >> (4 * i + 16)) & 15u) << (8 * i + 4);
    return r;
}
// and back
__device__ __forceinline__ uint32_t kv4_k_nibbles(uint32_t r)
{
    uint32_t w = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= ((r >> (8 * i)) & 15u) << (4 * i) | ((r >> (8 * i + 4)) & 15u) << (4 * i + 16);
    return w;
}

// Lane l (0..15) of a row: stores its 8 codes and, on a group's first lane,
// the group's parameters.
template <bool VALUES>
__device__ __forceinline__ void kv4_store(const Kv4& c, int64_t row, int group, int l, uint32_t word, uint32_t params)
{
    unsigned char* p = c.codes + row * kRowCodes;
    const int j = l >> 2, t = l & 3;
    if (VALUES) {
        // channels 8 l .. 8 l + 7 are those of g = 2 t and 2 t + 1: 2 bytes each
        *reinterpret_cast<uint16_t*>(p + 16 * t + 2 * j) = (uint16_t)word;
        *reinterpret_cast<uint16_t*>(p + 16 * t + 8 + 2 * j) = (uint16_t)(word >> 16);
    } else {
        *reinterpret_cast<uint32_t*>(p + 16 * t + 4 * j) = kv4_k_word(word);
    }
    const int lanes = group / 8;
    if (l % lanes == 0) c.params[row * (kD / group) + l / lanes] = params;
}

// the inverse: lane l's 8 values of a row
template <bool VALUES>
__device__ __forceinline__ void kv4_load(const Kv4& c, int64_t row, int group, int l, float (&x)[8])
{
    const unsigned char* p = c.codes + row * kRowCodes;
    const int j = l >> 2, t = l & 3;
    uint32_t w;
    if (VALUES)
        w = *reinterpret_cast<const uint16_t*>(p + 16 * t + 2 * j) |
            (uint32_t) * reinterpret_cast<const uint16_t*>(p + 16 * t + 8 + 2 * j) << 16;
    else
        w = kv4_k_nibbles(*reinterpret_cast<const uint32_t*>(p + 16 * t + 4 * j));
    const uint32_t params = c.params[row * (kD / group) + l / (group / 8)];
    const float s = __uint_as_float(params << 16), mid = __uint_as_float(params & 0xffff0000u);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(s, (float)((int32_t)(w << (28 - 4 * i)) >> 28), mid);
}

// ---- rows into the caches (k_qkv.cu) -------------------------------------
// one source of rows [B][T][heads][D] by strides in elements; null data = no rows
struct RowSource {
    const void* data;
    int64_t batch, token, head;
};

struct QkvArgs {
    RowSource q, k, v;
    int B, T, Hq, Hkv, n_max;
    const int32_t* pos;              // [B][T], or null: 0 .. T-1
    const void *q_weight, *k_weight; // [D], or null: no norm
    float eps;
    int rot;                         // rotated channels (0: none)
    int interleaved;
    float rot_scale;
    double turn[kD / 2];             // revolutions per position of each pair: inv_freq / (2 pi)
    void* q_out;
    int64_t q_out_batch, q_out_token, q_out_head;
    void *K, *V;                     // caches [B][Hkv][n_max][D], or null
    Kv4 K4, V4;                      // 4-bit caches (codes null: none)
    int group;
};
cudaError_t launch_qkv(const QkvArgs& a, int bf16, int sms, cudaStream_t st);

struct Kv4ReadArgs {
    Kv4 K4, V4;
    int64_t units;
    int n_max, first, count, group;
    void *K, *V;                     // either may be null
};
cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int bf16, cudaStream_t st);

// ---- attention over a 4-bit cache (k_kv4.cu) -----------------------------
struct Kv4AttendArgs {
    const void* q;                   // [B][Hq][D]
    Kv4 K4, V4;
    int B, Hq, Hkv;
    int U, NH;                       // units (lists of rows) and query heads of each
    int n;                           // most positions of a sequence
    int group;
    const int32_t* lens;             // [B], or null: n for every sequence
    const int32_t* rows;             // [U][max_rows], or null: dense
    const int32_t* n_rows;           // [U]
    int max_rows, S;
    float* part;                     // o [U + kKv4MaxCtas][NH][D], then (m, l) [U + kKv4MaxCtas][NH][2]
    unsigned* cnt;                   // [U] arrivals, 0 between calls
    float* out;                      // [B][Hq][D]
    float* lse;                      // [B][Hq] or null
};
constexpr int kKv4MaxCtas = 640;     // most CTAs of the attention grid (slots of the workspace)
constexpr int kKv4MaxHeads = 8;      // query heads of a unit
cudaError_t launch_kv4_attend(const Kv4AttendArgs& a, int bf16, int sms, cudaStream_t st);

}  // namespace ckv
