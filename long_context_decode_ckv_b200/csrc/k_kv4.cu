// k_kv4.cu -- decode attention over a 4-bit KV cache (format: kv4.cuh):
// every position of a sequence, or the sinks, a given list of rows and the
// new token.
//
// Per query head h and allowed row j: z_j = q_h.k_j / sqrt(D), softmax over
// the rows, out = sum_j p_j v_j, lse = m + ln(l).  With c the codes, s the
// scales and m the middles of a row's groups G,
//   q.k = sum_G s_G (q_G.c_G) + m_G sum(q_G),
//   sum_j p_j v_j = sum_j p_j (s_jG c_jG) + sum_j p_j m_jG per group G,
// so the keys' codes go to the tensor cores as they are and their scales are
// applied to 4 logits a lane, not to 128 channels a row.  Both products are
// exact but for the rounding of their float operands and sums:
//   q.c on the 8-bit integer MMA: q as 28-bit fixed point of its head's
//     largest channel, four signed base-128 digits in the rows of A (4 heads x
//     4 digits), a nibble in the high half of a byte as the code times 16;
//     unpacking 8 codes takes 3 instructions and no conversion.
//   p.(s c) on the fp16 MMA: a scale has 8 bits and a code at most 3 (or is
//     -8), so s c is an fp16 number, exactly, once s is brought into fp16's
//     range by a power of two c_G that keeps the largest of its group below
//     2^13.  p, 2^9 for the largest weight, is two fp16 numbers in the 8
//     columns of B (4 heads x 2 parts): p1 = fp16(p) and 2^13 (p - p1), whose
//     sums are put together when the piece ends.  So a weight has 22 bits down
//     to 2^-24 of the largest one and loses at most 2^-47 of that (half of
//     fp16's last step, 2^-25, over 2^13 and 2^9), and a scale keeps its 8 bits
//     down to 2^-29 of the largest of its group.  Scales multiplied into the
//     weights' parts, both without the factor 2^13, take fewer instructions
//     (2 % less time in groups of 32 at the size below, 5 % and 7 % in groups
//     of 64 and 128), but weights and scales then share one range: a weight
//     2^-20 of the largest keeps 14 bits, and with a scale 2^-17 of the largest
//     none.
//
// Work split: one unit per (batch, KV head), or per row list.  Units' tiles of
// 32 rows are laid end to end and split evenly over the grid; a CTA's share
// is one or more pieces (a run of one unit's tiles), and its warps take the
// tiles of a piece in turn, each through its own ring of cp.async stages.  A
// piece's (m, l, o) per head goes to a slot of its own; the unit's last piece
// to arrive merges the slots in their order, so the result does not depend on
// which one that is.
//
// Measured: 32 units of 131072 rows in groups of 32 (671 MB) take 169 us, 3.97
// TB/s, where the memory would take 103; in groups of 64 148, of 128 140; with
// eight heads of a KV head 253.  By length, 32 units of 16384, 32768, 65536,
// 131072 and 262144 rows take 33, 52, 89, 168 and 340 us: about 14 us that do
// not grow (start, queries, merge) and 1.2 us for 1000 rows, 1.3 beyond 131072.
// What bounds the part that grows: 472 instructions for 16 rows of a warp are 118
// cycles of an SM at full issue, about what the memory takes (111), but 16
// warps, which is what the registers allow, keep 68 % of the issue slots busy.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "kv4.cuh"
#include "warp_mma.cuh"

namespace ckv {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;                 // rows of a tile: two MMA tiles of 16
constexpr int kStages = 2;                // tiles of a warp's ring
constexpr int kRed = kD + 2 + 4;          // a warp's result per head: o[D], m, l, the middles' sums
constexpr float kLog2Scale = (float)(0.08838834764831845 * 1.4426950408889634);   // log2(e) / sqrt(128)

// what a unit attends to
struct Unit {
    int b, kvh, head0;     // sequence, KV head, first query head
    int len;               // positions of the sequence
    int sinks, listed;     // rows mode: sinks and list entries before the new token
    int count;             // entries, some of them possibly masked
};

__device__ __forceinline__ int seq_len(const Kv4AttendArgs& a, int b)
{
    return a.lens ? min(max(a.lens[b], 0), a.n) : a.n;
}

__device__ __forceinline__ Unit unit_of(const Kv4AttendArgs& a, int u)
{
    Unit x;
    const int per = a.U / a.B;            // units of a sequence
    x.b = u / per;
    x.head0 = (u % per) * a.NH;
    x.kvh = x.head0 / (a.Hq / a.Hkv);
    x.len = seq_len(a, x.b);
    x.sinks = x.listed = 0;
    x.count = x.len;
    if (a.rows) {
        x.sinks = min(a.S, x.len);
        x.listed = x.len > a.S ? min(max(a.n_rows[u], 0), a.max_rows) : 0;
        x.count = x.sinks + x.listed + (x.len > a.S ? 1 : 0);
    }
    return x;
}

// position of entry e of a unit; -1 where there is none
__device__ __forceinline__ int entry_row(const Kv4AttendArgs& a, const Unit& x, int u, int e)
{
    if (e >= x.count) return -1;
    if (!a.rows || e < x.sinks) return e;
    if (e == x.sinks + x.listed) return x.len - 1;
    const int r = a.rows[(int64_t)u * a.max_rows + (e - x.sinks)];
    return r >= a.S && r < x.len - 1 ? r : -1;
}

__device__ __forceinline__ int tiles_of(int count) { return (count + kTile - 1) / kTile; }

// the CTA whose share [lo(p), lo(p+1)), lo(p) = p * TT / P, holds tile x
__device__ __forceinline__ int owner_of(long long x, long long TT, int P)
{
    return (int)(((x + 1) * (long long)P - 1) / TT);
}

__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const int (&c)[4])
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%10,%11,%12,%13};\n"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c[0]), "r"(c[1]), "r"(c[2]),
                   "r"(c[3]));
}
// c + a b, the product rounded on its own and added to c to nearest: the MMA
// adds to its accumulator with truncation, which over the 100 MMAs of a long
// sequence took 2^-17 off the sums (9.5e-6 at 131072 rows, 8.5e-7 like this;
// it costs 8 us of 169)
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    float d[4];
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%10,%10,%10,%10};\n"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] += d[i];
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (lo, hi) -> fp16 pair, and an fp16 pair's halves
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// 4-bit codes of two rows (one per 16-bit half of x) as an fp16 pair: with
// magic 0x6488 in both halves, a masked low nibble n becomes 1024 + 128 +
// (n ^ 8) = 1160 + code, a high one 1024 + 16 (n ^ 8) + 8 = 16 (72.5 + code).
__device__ __forceinline__ uint32_t codes_low(uint32_t x, uint32_t magic)
{
    const uint32_t u = (x & 0x000f000fu) ^ magic, k = 0xe488e488u;          // -1160
    const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&k));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t codes_high(uint32_t x, uint32_t magic, uint32_t offset)
{
    const uint32_t u = (x & 0x00f000f0u) ^ magic, f = 0x2c002c00u;          // 1/16; offset: -72.5
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&f),
                              *reinterpret_cast<const __half2*>(&offset));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// a constant that stays in a register: an instruction takes one immediate,
// and the compiler, which cannot see through the shuffle, would otherwise
// rebuild the other one at every use
__device__ __forceinline__ uint32_t held(uint32_t v) { return __shfl_sync(kFull, v, 0); }
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float scale_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float middle_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <int N>
struct Words {
    uint32_t w[N];
};
template <int N>
__device__ __forceinline__ Words<N> lds(const unsigned char* p)
{
    Words<N> r;
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r.w[0] = v.x; r.w[1] = v.y;
    } else {
        r.w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
    return r;
}
template <int N>
__device__ __forceinline__ void sts(unsigned char* p, const Words<N>& r)
{
    if constexpr (N == 4) *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else if constexpr (N == 2) *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
    else *reinterpret_cast<uint32_t*>(p) = r.w[0];
}
template <int N>
__device__ __forceinline__ void cp_async_bytes(uint32_t dst, const void* src)
{
    if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(dst), "l"(src), "n"(N) : "memory");
}

// One stage of a warp's ring: a tile's K codes, V codes, K parameters, V
// parameters and the rows' mask.  V's 16-byte chunks of rows 4-7 and 12-15 of
// 16 are swapped by halves, so that the 8-byte reads of four rows that a half
// warp makes at once fall into different banks.
template <int NG>
struct Stage {
    static constexpr int K = 0, V = K + kTile * kRowCodes, KP = V + kTile * kRowCodes, VP = KP + kTile * 4 * NG,
                         MASK = VP + kTile * 4 * NG, bytes = MASK + 32;
};
// a tile's unpacked parameters: K scales, K middles, V middles as floats
// [32 rows][NG], V scales times c_G as fp16 pairs [16 pairs of rows][NG]
template <int NG>
struct Unpacked {
    static constexpr int KS = 0, KM = kTile * 4 * NG, VM = 2 * KM, VS = 3 * KM, bytes = VS + kTile * 2 * NG;
};
// a warp's shared memory: its ring, and a tile's unpacked parameters
template <int NG>
constexpr int kWarpSmem = (kStages * Stage<NG>::bytes + Unpacked<NG>::bytes + 127) / 128 * 128;
// Weights are powers of two of z - max + kRef: 2^kRef for the largest logit
// when the reference was set, at most 2^kMost before it is set again (a new
// maximum moves it only then; each move costs a pass over the sums).
constexpr float kRef = 9.f, kMost = 14.f;
// What a weight's second part is multiplied by (p <= 2^14 leaves p - p1 <= 4, so
// the part stays below fp16's 65504), and the border that value scales are kept
// below (8 times the largest 8-bit number under it is 65280).
constexpr float kSecond = 8192.f, kTopScale = 8192.f;

// NG: groups of a row.  NT: blocks of 4 query heads.  A lane is (g, t) =
// (lane / 4, lane % 4).
template <int NG, int NT>
struct Warp {
    static constexpr int NGH = NG > 1 ? NG / 2 : 1;    // groups whose middles this lane's half (g / 4) sums

    uint32_t qa[NT][4][4];   // digits of q: A of the k32 step j
    float qs[NT][NGH];       // this lane half's share of the sum of q over a group
    float unit[NT], unit128[NT], zero[NT];   // one step of the lane's second digit, of its first one, and minus the offsets of both
    float F[NT];             // logit (in powers of two) of a product of 1
    float m[NT], l[NT];      // kRef - the maximum referred to, and this lane's share of the sum: head 4 nt + g % 4
    float Z[NT][NGH];        // this lane's share of sum p * middle
    float acc[NT][8][4];     // sum (p's part) (s c_G code): [channel block J, pair of channels][..]
    uint32_t magic, offset;  // of codes_low and codes_high
    int base[4];             // what integer sums start at
    float c[NG];             // the powers of two c_G

    // ---- the unit's queries
    __device__ __forceinline__ void start(const Kv4AttendArgs& a, const Unit& x, bool bf16)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = 4 * nt + (g & 3);
            float q[4][8];
            float top_q = 0.f, nan = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t at = ((int64_t)x.b * a.Hq + x.head0 + h) * kD + 32 * j + 8 * t;
                if (h >= a.NH) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) q[j][i] = 0.f;
                } else if (bf16) {
                    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) { q[j][2 * i] = bf_lo(w[i]); q[j][2 * i + 1] = bf_hi(w[i]); }
                } else {
                    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
                    const float4 u = p[0], v = p[1];
                    q[j][0] = u.x; q[j][1] = u.y; q[j][2] = u.z; q[j][3] = u.w;
                    q[j][4] = v.x; q[j][5] = v.y; q[j][6] = v.z; q[j][7] = v.w;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    top_q = fmaxf(top_q, fabsf(q[j][i]));
                    nan = fmaf(q[j][i], 0.f, nan);
                }
            }
#pragma unroll
            for (int off = 1; off <= 2; off <<= 1) {
                top_q = fmaxf(top_q, __shfl_xor_sync(kFull, top_q, off));
                nan += __shfl_xor_sync(kFull, nan, off);
            }
            const bool bad = nan != 0.f;                       // an infinity or a NaN in the head
            if (bad) top_q = 0.f;
            // |q| < 2^e; q = X 2^(e - 27), the power of two in two factors (each a float)
            const bool small = top_q < 1.5777218e-30f;         // 2^-99
            int e = (int)(__float_as_uint(small ? top_q * 1.8446744e19f : top_q) >> 23) - 126 - (small ? 64 : 0);
            if (top_q == 0.f) e = 0;
            const int half = (27 - e) / 2;
            const float up1 = __uint_as_float((uint32_t)(127 + half) << 23), up2 = __uint_as_float((uint32_t)(127 + 27 - e - half) << 23);
            float sum[4];                                      // over 32 channels, in units of 4 X
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t d[4] = {0u, 0u, 0u, 0u};              // [channels 4..7 / 0..3 of 8 t ..][first / second digit]
                int part = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int X = bad ? 0 : __float2int_rn(q[j][i] * up1 * up2);
                    part += X;                                 // 8 * 2^27 at most
                    const int d3 = ((X + 64) & 127) - 64, X1 = (X - d3) >> 7;
                    const int d2 = ((X1 + 64) & 127) - 64, X2 = (X1 - d2) >> 7;
                    const int d1 = ((X2 + 64) & 127) - 64, d0 = (X2 - d1) >> 7;
                    const int hi = g < 4 ? d0 : d2, lo = g < 4 ? d1 : d3;
                    d[i < 4 ? 2 : 0] |= (uint32_t)(hi & 255) << (8 * (i & 3));
                    d[i < 4 ? 3 : 1] |= (uint32_t)(lo & 255) << (8 * (i & 3));
                }
                // rows g and g + 8 of A: the lane half's first and second digit
#pragma unroll
                for (int i = 0; i < 4; ++i) qa[nt][j][i] = d[i];
                part >>= 2;                                    // so that four of them fit; 2^-25 of the largest channel
                part += __shfl_xor_sync(kFull, part, 1);
                part += __shfl_xor_sync(kFull, part, 2);
                sum[j] = (float)part;
            }
            // a lane's integer logit counts 2^14 X (first half) or X, times 16
            // (the codes).  It is turned into q.c itself, and not left in those
            // units until the scales are applied: keys near the largest float
            // would overflow with small q.  The power of two is kept where
            // neither it nor the offsets leave the floats; F has the rest.
            const int E = e - 27 + (g < 4 ? 10 : -4), kept = min(max(E, -100), 84);
            unit[nt] = __uint_as_float((uint32_t)(127 + kept) << 23);
            unit128[nt] = 128.f * unit[nt];
            zero[nt] = -129.f * 12582912.f * unit[nt];
            // the middles' share: half of q's sum each where there is one group
            const float in_units = (g < 4 ? 1.f / 16384.f : 1.f) * 64.f * unit[nt];
            if constexpr (NG == 4) {
                qs[nt][0] = (g < 4 ? sum[0] : sum[2]) * in_units;
                qs[nt][1] = (g < 4 ? sum[1] : sum[3]) * in_units;
            } else if constexpr (NG == 2) {
                qs[nt][0] = (g < 4 ? sum[0] + sum[1] : sum[2] + sum[3]) * in_units;
            } else {
                qs[nt][0] = ((sum[0] + sum[1]) + (sum[2] + sum[3])) * (0.5f * in_units);
            }
            F[nt] = bad ? NAN : kLog2Scale * __uint_as_float((uint32_t)(127 + E - kept) << 23);
            m[nt] = FLT_MAX;
            l[nt] = 0.f;
#pragma unroll
            for (int j = 0; j < NGH; ++j) Z[nt][j] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[nt][i][r] = 0.f;
        }
        magic = held(0x64886488u);
        offset = held(0xd488d488u);
#pragma unroll
        for (int i = 0; i < 4; ++i) base[i] = (int)held(0x4b400000u);
#pragma unroll
        for (int j = 0; j < NG; ++j) c[j] = 5.1922969e33f;      // 2^112: scales below 2^-99
    }

    // ---- larger value scales than so far (this lane's row has sc): c_G down, sums with it
    __device__ __forceinline__ void raise(const float (&sc)[NG])
    {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const uint32_t most = __reduce_max_sync(kFull, __float_as_uint(sc[j]));
            // scale < 2^e; the format's scales are below 2^126
            int e = (int)((most >> 23) & 255u) - 126;
            e = e < -99 ? -99 : e > 126 ? 126 : e;
            const float now = fminf(c[j], __uint_as_float((uint32_t)(127 + 13 - e) << 23)), f = now / c[j];
            c[j] = now;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int J = 0; J < 4; ++J)
                    if (J * NG / 4 == j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) { acc[nt][2 * J][r] *= f; acc[nt][2 * J + 1][r] *= f; }
        }
    }

    // ---- a tile's parameters (of stage st) into un, each row's unpacked by
    // one lane and not by the eight that use them; valid: the tile's rows (bit
    // = row).  Before the tile's rows16(), after the tile before.
    __device__ __forceinline__ void unpack(const unsigned char* st, unsigned char* un, uint32_t valid)
    {
        using S = Stage<NG>;
        using U = Unpacked<NG>;
        const int lane = threadIdx.x & 31;
        Words<NG> kw = lds<NG>(st + S::KP + 4 * NG * lane), vw = lds<NG>(st + S::VP + 4 * NG * lane);
        if (!((valid >> lane) & 1u)) {
            // a row that is not there: its parameters may be anything
#pragma unroll
            for (int j = 0; j < NG; ++j) kw.w[j] = vw.w[j] = 0u;
        }
        float sc[NG];
        bool more = false;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            sc[j] = scale_of(vw.w[j]);
            more |= sc[j] * c[j] >= kTopScale;
        }
        if (__any_sync(kFull, more)) raise(sc);
        // the pair (columns 2 t', 2 t' + 1) that the row belongs to, and which of the two it is
        const int pair = lane >> 1, side = (lane & 1) ^ (pair & 1);
        Words<NG> ks, km, vm;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            ks.w[j] = __float_as_uint(scale_of(kw.w[j]));
            km.w[j] = __float_as_uint(middle_of(kw.w[j]));
            vm.w[j] = __float_as_uint(middle_of(vw.w[j]));
            reinterpret_cast<__half*>(un + U::VS)[2 * (pair * NG + j) + side] = __float2half_rn(sc[j] * c[j]);
        }
        sts<NG>(un + U::KS + 4 * NG * lane, ks);
        sts<NG>(un + U::KM + 4 * NG * lane, km);
        sts<NG>(un + U::VM + 4 * NG * lane, vm);
    }

    // ---- rows 16 sub .. 16 sub + 15 of a tile; valid: which are there
    __device__ __forceinline__ void rows16(const unsigned char* st, const unsigned char* un, int sub, uint32_t valid)
    {
        using S = Stage<NG>;
        using U = Unpacked<NG>;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        // the rows of this lane's logits: columns 2 t and 2 t + 1 of the two
        // MMAs; their order within the pair alternates with t (see Stage)
        const int ra = 2 * t + (t & 1), rb = 2 * t + 1 - (t & 1);
        const int rows[4] = {16 * sub + ra, 16 * sub + rb, 16 * sub + ra + 8, 16 * sub + rb + 8};
        const int half = NG > 1 ? (g >> 2) * (4 * NGH) : 0;    // bytes to this lane half's middles
        // ---- logits
        float z[NT][4];
        {
            float ks[4][NG], km[4][NGH];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Words<NG> w = lds<NG>(un + U::KS + rows[e] * (4 * NG));
                const Words<NGH> h = lds<NGH>(un + U::KM + rows[e] * (4 * NG) + half);
#pragma unroll
                for (int j = 0; j < NG; ++j) ks[e][j] = __uint_as_float(w.w[j]);
#pragma unroll
                for (int j = 0; j < NGH; ++j) km[e][j] = __uint_as_float(h.w[j]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[nt][e] = km[e][0] * qs[nt][0];
#pragma unroll
                    for (int j = 1; j < NGH; ++j) z[nt][e] = fmaf(km[e][j], qs[nt][j], z[nt][e]);
                }
            // column n of MMA a is row 8 a + rowof(n): lane g loads that row
            const int kr = 2 * (g >> 1) + ((g & 1) ^ ((g >> 1) & 1));
            // The sums start at the bits of 1.5 * 2^23, so that they are floats
            // 1.5 * 2^23 + v for |v| < 2^22: no conversion.  128 v0 + v1, the two
            // digits' sums, is then one FMA that also takes the offsets off
            // (exact) and one that rounds.
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const Words<4> w = lds<4>(st + S::K + (16 * sub + 8 * a + kr) * kRowCodes + 16 * t);
                int d[NT][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b0 = w.w[j] & 0xf0f0f0f0u, b1 = (w.w[j] << 4) & 0xf0f0f0f0u;
                    constexpr int per = 4 / NG;                // k32 steps of a group
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (j % per == 0) mma_s8(d[nt], qa[nt][j], b0, b1, base);
                        else mma_s8(d[nt], qa[nt][j], b0, b1, d[nt]);
                        if (j % per == per - 1) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float v = fmaf(__int_as_float(d[nt][2 + i]), unit[nt], fmaf(__int_as_float(d[nt][i]), unit128[nt], zero[nt]));
                                z[nt][2 * a + i] = fmaf(ks[2 * a + i][j / per], v, z[nt][2 * a + i]);
                            }
                        }
                    }
                }
            }
        }
        // ---- values: A is 16 channels x 16 rows
        Words<2> v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = rows[e], chunk = (g >> 1) ^ ((r >> 1) & 2);
            v[e] = lds<2>(st + S::V + r * kRowCodes + 16 * chunk + 8 * (g & 1));
        }
        bool more = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                z[nt][e] *= F[nt];
                z[nt][e] += __shfl_xor_sync(kFull, z[nt][e], 16);
            }
            if (valid != 0xffffu) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!((valid >> (rows[e] & 15)) & 1u)) z[nt][e] = -INFINITY;
            }
            more |= fmaxf(fmaxf(z[nt][0], z[nt][1]), fmaxf(z[nt][2], z[nt][3])) + m[nt] > kMost;
        }
        // ---- a new maximum: sums down
        if (__any_sync(kFull, more)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float mx = fmaxf(fmaxf(z[nt][0], z[nt][1]), fmaxf(z[nt][2], z[nt][3]));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
                // rounded down: where logits step by 16 (from 2^27 on), to
                // nearest would leave 2^16 for the largest weight, which fp16
                // does not hold
                const float mn = fminf(m[nt], __fsub_rd(kRef, mx)), f = ex2(mn - m[nt]);
                m[nt] = mn;
                l[nt] *= f;
#pragma unroll
                for (int j = 0; j < NGH; ++j) Z[nt][j] *= f;
                // columns 2 t and 2 t + 1 of the sums: heads 2 t % 4 and + 1
                const float f0 = __shfl_sync(kFull, f, ((2 * t) & 3) * 4), f1 = __shfl_sync(kFull, f, ((2 * t + 1) & 3) * 4);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[nt][i][0] *= f0;
                    acc[nt][i][2] *= f0;
                    acc[nt][i][1] *= f1;
                    acc[nt][i][3] *= f1;
                }
            }
        }
        // ---- weights: this lane's column of B holds the first parts (g < 4) or
        // the second ones, (p - 0) 1 or (p - p1) 2^13
        uint32_t pb[NT][2];
        {
            const float minus = g < 4 ? 0.f : -1.f, times = g < 4 ? 1.f : kSecond;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = ex2(z[nt][e] + m[nt]);
                l[nt] += (p[0] + p[1]) + (p[2] + p[3]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 f = unpack_f16(pack_f16(p[2 * k], p[2 * k + 1]));
                    pb[nt][k] = pack_f16(fmaf(minus, f.x, p[2 * k]) * times, fmaf(minus, f.y, p[2 * k + 1]) * times);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const Words<NGH> h = lds<NGH>(un + U::VM + rows[e] * (4 * NG) + half);
#pragma unroll
                    for (int j = 0; j < NGH; ++j) Z[nt][j] = fmaf(p[e], __uint_as_float(h.w[j]), Z[nt][j]);
                }
            }
        }
        // A is 16 channels x 16 rows: codes times their rows' scales
        Words<NG> vs[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) vs[k] = lds<NG>(un + U::VS + (8 * sub + t + 4 * k) * (4 * NG));
#pragma unroll
        for (int J = 0; J < 4; ++J) {
            const uint32_t sel = J & 1 ? 0x7632u : 0x5410u;
            uint32_t x = __byte_perm(v[0].w[J >> 1], v[1].w[J >> 1], sel), y = __byte_perm(v[2].w[J >> 1], v[3].w[J >> 1], sel);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t sx = vs[0].w[J * NG / 4], sy = vs[1].w[J * NG / 4];
                const uint32_t a0 = mul2(codes_low(x, magic), sx), a1 = mul2(codes_high(x, magic, offset), sx);
                const uint32_t a2 = mul2(codes_low(y, magic), sy), a3 = mul2(codes_high(y, magic, offset), sy);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_f16(acc[nt][2 * J + k], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                x >>= 8;
                y >>= 8;
            }
        }
    }

    // ---- this warp's sums per head: o without the middles, m, l, the middles' sums
    __device__ __forceinline__ void finish(float* red)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int J = 0; J < 4; ++J) {
                const float inv = 1.f / c[J * NG / 4] * (t < 2 ? 1.f : 1.f / kSecond);   // columns of first or second parts
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float v = acc[nt][2 * J + k][r] * inv;
                        v += __shfl_xor_sync(kFull, v, 2);
                        if (t < 2) red[(4 * nt + 2 * t + (r & 1)) * kRed + 32 * J + 4 * g + 2 * k + (r >> 1)] = v;
                    }
            }
            float s = l[nt];
            s += __shfl_xor_sync(kFull, s, 1);
            s += __shfl_xor_sync(kFull, s, 2);
            float* r = red + (4 * nt + (g & 3)) * kRed + kD;
            if (t == 0 && g < 4) { r[0] = -m[nt]; r[1] = s; }
#pragma unroll
            for (int j = 0; j < NGH; ++j) {
                float v = Z[nt][j];
                v += __shfl_xor_sync(kFull, v, 1);
                v += __shfl_xor_sync(kFull, v, 2);
                if (t == 0 && (NG > 1 || g < 4)) r[2 + (NG > 1 ? (g >> 2) * NGH : 0) + j] = v;
            }
        }
    }
};

// weight of a part with maximum m and sum l in a merge with maximum M; a part without rows has l = 0
__device__ __forceinline__ float part_weight(float m, float l, float M) { return l == 0.f ? 0.f : ex2(m - M); }

// channel d of head h over the CTA's warps, and their maximum and sum
template <int NG>
__device__ __forceinline__ float merge_warps(const float* red, int stride, int h, int d, float& M, float& L)
{
    const float* r = red + h * kRed;
    float O = 0.f;
    M = -FLT_MAX;
    L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, r[w * stride + kD]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float* rw = r + w * stride;
        const float f = part_weight(rw[kD], rw[kD + 1], M);
        L += f * rw[kD + 1];
        O += f * (rw[d] + rw[kD + 2 + d * NG / kD]);
    }
    return O;
}

__device__ __forceinline__ void store_out(const Kv4AttendArgs& a, const Unit& x, int h, int d, float O, float M, float L)
{
    const int64_t hq = (int64_t)x.b * a.Hq + x.head0 + h;
    a.out[hq * kD + d] = L == 0.f ? 0.f : O / L;
    if (d == 0 && a.lse) a.lse[hq] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// The CTA merges slots u + pf .. u + pf + ns - 1 of unit u.  First a warp per
// head turns the slots' (m, l) into weights, a lane a slot; then a thread
// takes 4 channels of a head and every k-th slot, with independent loads.
__device__ __forceinline__ void merge_slots(const Kv4AttendArgs& a, const Unit& x, int u, int pf, int ns, float* sh)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float* weight = sh;                                    // [NH][ns]
    float* total = weight + a.NH * ns;                     // [NH][2]: m, l
    float4* part = reinterpret_cast<float4*>(sh + kKv4MaxHeads * (kKv4MaxCtas + 2));   // [kThreads]
    const float2* sm = reinterpret_cast<const float2*>(a.part + (int64_t)(a.U + kKv4MaxCtas) * a.NH * kD) + (int64_t)(u + pf) * a.NH;
    const float4* so = reinterpret_cast<const float4*>(a.part + (int64_t)(u + pf) * a.NH * kD);
    for (int h = warp; h < a.NH; h += kWarps) {
        float M = -FLT_MAX, L = 0.f;
        float2 v = make_float2(-FLT_MAX, 0.f);             // this lane's first slot
        if (lane < ns) v = __ldcg(sm + (int64_t)lane * a.NH + h);
        M = v.x;
        for (int s = lane + 32; s < ns; s += 32) M = fmaxf(M, __ldcg(sm + (int64_t)s * a.NH + h).x);
#pragma unroll
        for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, off));
        for (int s = lane; s < ns; s += 32) {
            if (s >= 32) v = __ldcg(sm + (int64_t)s * a.NH + h);
            const float f = part_weight(v.x, v.y, M);
            weight[h * ns + s] = f;
            L += f * v.y;
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) L += __shfl_xor_sync(kFull, L, off);
        if (lane == 0) { total[2 * h] = M; total[2 * h + 1] = L; }
    }
    __syncthreads();
    constexpr int kQuads = kD / 4;
    const int items = a.NH * kQuads, ways = kThreads / items;   // NH <= 8: one item a thread at most
    const int item = tid % items, way = tid / items;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (way < ways) {
        const float* w = weight + item / kQuads * ns;
#pragma unroll 4
        for (int s = way; s < ns; s += ways) {
            const float4 v = __ldcg(so + (int64_t)s * items + item);
            const float f = w[s];
            o.x += f * v.x;
            o.y += f * v.y;
            o.z += f * v.z;
            o.w += f * v.w;
        }
        part[tid] = o;
    }
    __syncthreads();
    if (tid < items) {
        for (int i = 1; i < ways; ++i) {
            const float4 v = part[i * items + tid];
            o.x += v.x;
            o.y += v.y;
            o.z += v.z;
            o.w += v.w;
        }
        const int h = tid / kQuads;
        const int64_t hq = (int64_t)x.b * a.Hq + x.head0 + h;
        const float L = total[2 * h + 1];
        if (L == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
        else { o.x /= L; o.y /= L; o.z /= L; o.w /= L; }
        reinterpret_cast<float4*>(a.out)[hq * kQuads + tid % kQuads] = o;
        if (a.lse && tid % kQuads == 0) a.lse[hq] = L == 0.f ? -INFINITY : (total[2 * h] + log2f(L)) * 0.6931471805599453f;
    }
}

// CTAs of an SM: two while a warp's sums fit 128 registers (4 heads).  With 8
// heads of a unit, 4 x 131072 rows of 8 KV heads in groups of 32 took 256 us
// with one CTA of 8 warps, 282 with 12 warps, 442 with two CTAs: the sums spill.
template <int NT>
constexpr int kCtasPerSM = NT == 1 ? 2 : 1;

template <int NG, int NT, bool ROWS>
__global__ void __launch_bounds__(kThreads, kCtasPerSM<NT>) k_kv4_attend(const __grid_constant__ Kv4AttendArgs a, int bf16)
{
    using S = Stage<NG>;
    static_assert(4 * NT * kRed * 4 <= kWarpSmem<NG>, "a warp's results must fit its ring");
    static_assert(kWarpSmem<NG> % 128 == 0, "aligned warps");
    static_assert(kKv4MaxHeads * (kKv4MaxCtas + 2) * 4 + kThreads * 16 <= kWarps * kWarpSmem<NG>, "the merge must fit");
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long s_scan[kWarps];
    __shared__ long long s_first[2];       // first unit of this CTA's share, tiles before that unit
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned char* ring = smem + warp * kWarpSmem<NG>;
    float* red = reinterpret_cast<float*>(smem);
    constexpr int kRedWarp = kWarpSmem<NG> / 4;            // floats between two warps' results
    const int p = blockIdx.x;

    // ---- the share: tiles of all units, and the unit the share starts in
    long long TT;
    int P;
    long long lo, hi;
    if (!ROWS && !a.lens) {
        const long long per = tiles_of(a.n);
        TT = per * a.U;
        P = TT < gridDim.x ? (int)TT : (int)gridDim.x;
        lo = p < P ? p * TT / P : TT;
        hi = p < P ? (p + 1) * TT / P : TT;
        if (tid == 0) { s_first[0] = lo / per; s_first[1] = lo / per * per; }
    } else {
        const int per = (a.U + kThreads - 1) / kThreads;
        const int u0 = min(tid * per, a.U), u1 = min(u0 + per, a.U);
        long long mine = 0;
        for (int u = u0; u < u1; ++u) mine += tiles_of(unit_of(a, u).count);
        long long upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long o = __shfl_up_sync(kFull, upto, off);
            if (lane >= off) upto += o;
        }
        if (lane == 31) s_scan[warp] = upto;
        __syncthreads();
        TT = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) upto += TT;
            TT += s_scan[w];
        }
        // no more shares than tiles: the arrivals of a unit count every CTA
        // between its first and its last tile's owner
        P = TT < gridDim.x ? (int)(TT > 0 ? TT : 1) : (int)gridDim.x;
        lo = p < P ? p * TT / P : TT;
        hi = p < P ? (p + 1) * TT / P : TT;
        if (lo < hi && lo >= upto - mine && lo < upto) {
            long long at = upto - mine;
            int u = u0;
            for (;; ++u) {
                const int n = tiles_of(unit_of(a, u).count);
                if (lo < at + n) break;
                at += n;
            }
            s_first[0] = u;
            s_first[1] = at;
        }
        // units with nothing to attend to: 0 and -inf
        for (int u = p; u < a.U; u += gridDim.x) {
            const Unit x = unit_of(a, u);
            if (x.count) continue;
            for (int i = tid; i < a.NH * kD; i += kThreads) a.out[((int64_t)x.b * a.Hq + x.head0) * kD + i] = 0.f;
            if (a.lse && tid < a.NH) a.lse[(int64_t)x.b * a.Hq + x.head0 + tid] = -INFINITY;
        }
    }
    __syncthreads();
    if (lo >= hi) return;

    int u = (int)s_first[0];
    long long before = s_first[1];
    for (long long at = lo; at < hi; ++u) {
        // ---- one piece: tiles [t0, t1) of unit u
        const Unit x = unit_of(a, u);
        const long long end = before + tiles_of(x.count);
        if (end == before) continue;
        const int t0 = (int)(at - before), t1 = (int)((hi < end ? hi : end) - before);
        {
            const int first = t0 + warp;
            const int nb = t1 > first ? (t1 - first + kWarps - 1) / kWarps : 0;
            const int64_t row0 = ((int64_t)x.b * a.Hkv + x.kvh) * a.K4.R;
            const int r8 = lane >> 2, ch = lane & 3;
            // this lane's bytes of the first tile (dense) or of row 0 (rows)
            const int64_t from = row0 + (ROWS ? 0 : (int64_t)first * kTile);
            const unsigned char* kc = a.K4.codes + (from + (ROWS ? 0 : r8)) * kRowCodes + 16 * ch;
            const unsigned char* vc = a.V4.codes + (from + (ROWS ? 0 : r8)) * kRowCodes + 16 * ch;
            const uint32_t* kp = a.K4.params + (from + (ROWS ? 0 : lane)) * NG;
            const uint32_t* vp = a.V4.params + (from + (ROWS ? 0 : lane)) * NG;
            const uint32_t ring_at = smem_u32(ring);
            const uint32_t to_k = r8 * kRowCodes + 16 * ch, to_v = S::V + r8 * kRowCodes + 16 * (ch ^ ((r8 >> 1) & 2));
            const uint32_t to_p = S::KP + lane * (4 * NG);
            // entry `lane` of the warp's tile i: its position, -1 for none
            auto entry = [&](int i) { return i < nb ? entry_row(a, x, u, (first + i * kWarps) * kTile + lane) : -1; };
            // copies of the next tile to stage offset `to`, if there is one
            int ahead = x.count - first * kTile;               // entries from that tile's first one on, if it is this warp's
            int tiles_left = nb;
            auto issue = [&](uint32_t to, int row) {
                if (tiles_left > 0) {
                    const uint32_t st = ring_at + to;
                    if (ROWS) {
                        const uint32_t mask = __ballot_sync(kFull, row >= 0);
                        row = max(row, 0);                     // a row that is not there: row 0, which is never used
                        if (lane == 0) *reinterpret_cast<uint32_t*>(ring + to + S::MASK) = mask;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int64_t k = (int64_t)__shfl_sync(kFull, row, r8 + 8 * i) * kRowCodes;
                            cp_async_bytes<16>(st + to_k + 8 * i * kRowCodes, kc + k);
                            cp_async_bytes<16>(st + to_v + 8 * i * kRowCodes, vc + k);
                        }
                        cp_async_bytes<4 * NG>(st + to_p, kp + (int64_t)row * NG);
                        cp_async_bytes<4 * NG>(st + to_p + kTile * 4 * NG, vp + (int64_t)row * NG);
                    } else {
                        // rows behind the sequence are not read: the last tile may
                        // reach past the end of the cache
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (r8 + 8 * i < ahead) {
                                cp_async_bytes<16>(st + to_k + 8 * i * kRowCodes, kc + 8 * i * kRowCodes);
                                cp_async_bytes<16>(st + to_v + 8 * i * kRowCodes, vc + 8 * i * kRowCodes);
                            }
                        if (lane < ahead) {
                            cp_async_bytes<4 * NG>(st + to_p, kp);
                            cp_async_bytes<4 * NG>(st + to_p + kTile * 4 * NG, vp);
                        }
                        kc += kWarps * kTile * kRowCodes;
                        vc += kWarps * kTile * kRowCodes;
                        kp += kWarps * kTile * NG;
                        vp += kWarps * kTile * NG;
                    }
                }
                ahead -= kWarps * kTile;
                --tiles_left;
                cp_async_commit();
            };
            int row = 0;
            if (ROWS) row = entry(0);
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) {
                const int now = row;
                if (ROWS) row = entry(i + 1);
                issue(i * S::bytes, now);
            }
            Warp<NG, NT> w;
            w.start(a, x, bf16 != 0);
            // the rows of the tile at stage offset `at`; left: entries from its first one on
            auto valid_of = [&](uint32_t at, int left) -> uint32_t {
                if (ROWS) return *reinterpret_cast<const uint32_t*>(ring + at + S::MASK);
                return left < kTile ? (1u << left) - 1u : 0xffffffffu;
            };
            int left = x.count - first * kTile;
            uint32_t cur = 0u;
            unsigned char* un = ring + kStages * S::bytes;
            for (int i = 0; i < nb; ++i) {
                // this tile's copies have arrived and are seen by the warp
                cp_async_wait<kStages - 2>();
                __syncwarp();
                const uint32_t valid = valid_of(cur, left);
                const int now = row;
                if (ROWS) row = entry(i + kStages);
                issue(S::bytes - cur, now);                    // into the other stage, read by the tile before
                w.unpack(ring + cur, un, valid);
                __syncwarp();
                w.rows16(ring + cur, un, 0, valid & 0xffffu);
                if (valid >> 16) w.rows16(ring + cur, un, 1, valid >> 16);
                cur = S::bytes - cur;
                left -= kWarps * kTile;
            }
            static_assert(kStages == 2, "cur alternates between two stages");
            cp_async_wait<0>();
            __syncwarp();
            w.finish(reinterpret_cast<float*>(ring));          // the ring is drained
        }
        __syncthreads();
        const int pf = owner_of(before, TT, P), pl = owner_of(end - 1, TT, P);
        if (pf == pl) {
            // the unit is this piece
            for (int i = tid; i < a.NH * kD; i += kThreads) {
                float M, L;
                const float O = merge_warps<NG>(red, kRedWarp, i / kD, i % kD, M, L);
                store_out(a, x, i / kD, i % kD, O, M, L);
            }
        } else {
            // ---- the piece's slot
            float* so = a.part + (int64_t)(u + p) * a.NH * kD;
            float2* sm = reinterpret_cast<float2*>(a.part + (int64_t)(a.U + kKv4MaxCtas) * a.NH * kD) + (int64_t)(u + p) * a.NH;
            for (int i = tid; i < a.NH * kD; i += kThreads) {
                float M, L;
                so[i] = merge_warps<NG>(red, kRedWarp, i / kD, i % kD, M, L);
                if (i % kD == 0) sm[i / kD] = make_float2(M, L);
            }
            // ---- arrival; the unit's last piece merges every slot.  A unit of
            // several pieces is the last one of its first CTA's share, so that
            // CTA's counter is this unit's alone.  The barrier orders the CTA's
            // stores before thread 0's fence, which makes them visible before
            // its arrival; likewise the other way.
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                s_last = atomicAdd(a.cnt + pf, 1u) == (unsigned)(pl - pf);
                __threadfence();
            }
            __syncthreads();
            if (s_last) {
                merge_slots(a, x, u, pf, pl - pf + 1, red);
                if (tid == 0) a.cnt[pf] = 0;
            }
        }
        __syncthreads();   // the rings are written again by the next piece
        at = before + t1;
        before = end;
    }
}

// How many tiles the units of a call have: all `tiles` (dense, one length), at
// most that and mostly near it (row lists), at most that (sequences of their
// own lengths).
enum Extent { kEqual, kLists, kLengths };

// CTAs for U units; `most` of them run at once, `sms` of them with an SM each.
// Measured at 4 heads, groups of 32, 148 SMs.
//
// Equal units: shares that end with units (k of them each), or as many shares
// as CTAs run at once, wherever their borders fall.  Costs are in rounds of a
// warp's tile, which take 1.6 us with one CTA on an SM and 1.7 times that
// with two.  A merge through slots costs 2.2 rounds (3.7 with two CTAs on an
// SM) and a little for each slot; borders within units 6 (7.2), since CTAs
// then start, end and merge twice, and more for each further unit of a share; a
// second wave of CTAs 3.5.  32 units of 1250 tiles take 60 us in 288 shares and 67
// in 296, of 375 tiles 28 and 35; 80 of 118 tiles 26 us in 240 shares, 33 in 80
// and 32 in 296; 112 of 73 tiles 24 in 112 and 30 in 296; 8 of 600 tiles 19 in
// 144 and 22 in 296; 256 of 19 tiles 17 in 256 and 26 in 296.
//
// Lists and lengths: shares end with units only if these turn out equal, which
// happens often enough that the number is a multiple of U where one covers the
// machine (32 units of 150 tiles in 128 and 148 shares: equal ones 19 and 25
// us, within a tenth of one another 27 and 26, lengths from an eighth on 23 and
// 23).  A CTA for each unit while a warp has up to 3 tiles, then one CTA to an
// SM, but two where U takes more than half of the SMs (80 units of 60 tiles in
// 80, 148 and 240 shares: equal ones 21, 25 and 20 us, lengths apart 33, 28 and
// 27; of 30 tiles 14, 22 and 16, and 28, 25 and 24: from 6 tiles a warp on) or a
// warp has four tiles on the whole machine.  More units than SMs: two CTAs to
// an SM, but a CTA for each list of a tile a warp (160 of 4: 12 us, 23 in 296).
long long grid_of(long long U, long long tiles, Extent extent, long long sms, long long most)
{
    const long long total = U * tiles;
    if (extent != kEqual) {
        const long long each = tiles <= 3 * kWarps ? 1 : (tiles + kWarps - 1) / kWarps, aligned = U <= most ? most / U * U : 0;
        if (total > most * kWarps * 4) return 20 * aligned >= 19 * most ? aligned : most;
        if (U >= sms) return extent == kLists && U <= most && tiles <= kWarps ? U : most;
        if (2 * U <= sms) return U * (each < sms / U ? each : sms / U);
        if (each <= 6) return U;
        return 4 * aligned >= 3 * most ? aligned : most;
    }
    const auto rounds = [](double t) { return t <= 4 * kWarps ? ceil(t / kWarps) : t / kWarps + 0.5; };
    const auto pace = [&](long long ctas) { return ctas <= sms ? 1.0 : 1.7; };
    const double over = (double)U / (double)most;
    double best = rounds((double)total / (double)most) * pace(most) + (most > sms ? 7.2 : 6.0) + 0.02 / over +
                  (over > 1.0 ? 8.0 * (over - 1.0) : 0.0);
    long long P = most;
    const auto offer = [&](long long k) {
        if (k < 1 || U * k > (k == 1 ? kKv4MaxCtas : most)) return;
        const long long waves = U * k / most, rest = U * k % most;
        const double paces = (double)waves * pace(most) + (rest ? pace(rest) : 0.0);
        double cost = rounds((double)((tiles + k - 1) / k)) * paces + 3.5 * (double)(waves + (rest != 0) - 1);
        if (k > 1) cost += (U * k > sms ? 3.7 : 2.2) + 0.02 * (double)k;
        if (cost < best) {
            best = cost;
            P = U * k;
        }
    };
    offer(1);
    for (int r = 1; r <= 4; ++r) offer((tiles + r * kWarps - 1) / (r * kWarps));
    offer(sms / U);
    offer(most / U);
    return P;
}

template <int NG, int NT, bool ROWS>
cudaError_t launch_attend_t(const Kv4AttendArgs& a, int bf16, int sms, cudaStream_t st)
{
    auto fn = k_kv4_attend<NG, NT, ROWS>;
    static std::atomic<uint64_t> prepared{0};              // devices (bit = ordinal) that know the kernel's shared memory
    if (!(prepared.load(std::memory_order_acquire) >> a.device & 1)) {
        cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kWarps * kWarpSmem<NG>);
        if (e != cudaSuccess) return e;
        prepared.fetch_or(uint64_t(1) << a.device, std::memory_order_release);
    }
    const long long tiles = ROWS ? ((long long)a.S + a.max_rows + 1 + kTile - 1) / kTile : (a.n + kTile - 1) / kTile;
    const Extent extent = ROWS ? kLists : a.lens && a.B > 1 ? kLengths : kEqual;
    const long long most = kCtasPerSM<NT> * sms < kKv4MaxCtas ? kCtasPerSM<NT> * sms : kKv4MaxCtas;
    const long long P = grid_of(a.U, tiles, extent, sms, most);
    return launch_kernel(fn, dim3((unsigned)P), kThreads, kWarps * kWarpSmem<NG>, st, a, bf16);
}

template <bool ROWS>
cudaError_t launch_attend_g(const Kv4AttendArgs& a, int bf16, int sms, cudaStream_t st)
{
    if (a.NH <= 4) {
        if (a.group == 32) return launch_attend_t<4, 1, ROWS>(a, bf16, sms, st);
        if (a.group == 64) return launch_attend_t<2, 1, ROWS>(a, bf16, sms, st);
        return launch_attend_t<1, 1, ROWS>(a, bf16, sms, st);
    }
    if (a.group == 32) return launch_attend_t<4, 2, ROWS>(a, bf16, sms, st);
    if (a.group == 64) return launch_attend_t<2, 2, ROWS>(a, bf16, sms, st);
    return launch_attend_t<1, 2, ROWS>(a, bf16, sms, st);
}

}  // namespace

cudaError_t launch_kv4_attend(const Kv4AttendArgs& a, int bf16, int sms, cudaStream_t st)
{
    return a.rows ? launch_attend_g<true>(a, bf16, sms, st) : launch_attend_g<false>(a, bf16, sms, st);
}

}  // namespace ckv
