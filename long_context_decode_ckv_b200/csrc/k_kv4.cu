// k_kv4.cu -- decode attention over a 4-bit KV cache (format: kv4.cuh):
// every position of a sequence, or the sinks, a given list of rows and the
// new token.
//
// Per query head h and allowed row j: z_j = q_h.k_j / sqrt(D), softmax over
// the rows, out = sum_j p_j v_j, lse = m + ln(l).  With c the codes, s the
// scales and m the middles of a row's groups G,
//   q.k = sum_G s_G (q_G.c_G) + m_G sum(q_G),
//   sum_j p_j v_j = sum_j (p_j s_jG) c_jG + sum_j p_j m_jG per group G.
//
// Work split: one unit per (batch, KV head), or per row list.  Units' tiles of
// 16 rows are laid end to end and split evenly over the grid; a CTA's share
// is one or more pieces (a run of one unit's tiles), and its warps take the
// tiles of a piece in turn.  A piece's (m, l, o) per head goes to a slot of
// its own; the unit's last piece to arrive merges the slots in their order,
// so the result does not depend on which one that is.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kv4.cuh"
#include "warp_mma.cuh"

namespace ckv {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;                 // rows of a tile
constexpr int kSlot = 2 + kD;             // slot row per head: m, l, o[D]
constexpr float kScale = 0.08838834764831845f;   // 1 / sqrt(128)

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

template <bool BF16>
__device__ __forceinline__ float load_q(const void* q, int64_t i)
{
    return BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(q)[i]) : static_cast<const float*>(q)[i];
}

// One warp: rows of tiles t0 + warp, t0 + warp + kWarps, ... of [t0, t1); lane l holds channels 4 l .. 4 l + 3.
template <bool BF16>
__device__ __forceinline__ void warp_rows(const Kv4AttendArgs& a, const Unit& x, int u, int t0, int t1,
                                          float (&m)[kKv4MaxHeads], float (&l)[kKv4MaxHeads],
                                          float (&o)[kKv4MaxHeads][4])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int NG = kD / a.group;
    const int64_t base = ((int64_t)x.b * a.Hkv + x.kvh) * a.K4.R;
    const int j = lane >> 3;
    float q[kKv4MaxHeads][4];
    for (int h = 0; h < kKv4MaxHeads; ++h)
        for (int i = 0; i < 4; ++i)
            q[h][i] = h < a.NH ? load_q<BF16>(a.q, ((int64_t)x.b * a.Hq + x.head0 + h) * kD + 4 * lane + i) : 0.f;
    for (int tile = t0 + warp; tile < t1; tile += kWarps)
        for (int e = tile * kTile; e < tile * kTile + kTile; ++e) {
            const int row = entry_row(a, x, u, e);
            if (row < 0) continue;
            const int64_t at = base + row;
            // K: channels 32 j + 8 t + 4 h + i at bytes 16 t + 4 j + i
            const int t = (lane & 7) >> 1, hi = lane & 1;
            const uint32_t kw = *reinterpret_cast<const uint32_t*>(a.K4.codes + at * kRowCodes + 16 * t + 4 * j) >> (4 * hi);
            const uint32_t vw = *reinterpret_cast<const uint16_t*>(a.V4.codes + at * kRowCodes + 8 * (lane & 7) + 2 * j);
            const uint32_t kp = a.K4.params[at * NG + 4 * lane / a.group], vp = a.V4.params[at * NG + 4 * lane / a.group];
            float k[4], v[4];
            for (int i = 0; i < 4; ++i) {
                k[i] = fmaf(__uint_as_float(kp << 16), (float)((int)(kw << (28 - 8 * i)) >> 28), __uint_as_float(kp & 0xffff0000u));
                v[i] = fmaf(__uint_as_float(vp << 16), (float)((int)(vw << (28 - 4 * i)) >> 28), __uint_as_float(vp & 0xffff0000u));
            }
            for (int h = 0; h < a.NH; ++h) {
                float z = q[h][0] * k[0] + q[h][1] * k[1] + q[h][2] * k[2] + q[h][3] * k[3];
                for (int off = 16; off; off >>= 1) z += __shfl_xor_sync(kFull, z, off);
                z *= kScale;
                const float mn = fmaxf(m[h], z);
                const float al = m[h] == -INFINITY ? 0.f : expf(m[h] - mn), p = expf(z - mn);
                l[h] = l[h] * al + p;
                for (int i = 0; i < 4; ++i) o[h][i] = o[h][i] * al + p * v[i];
                m[h] = mn;
            }
        }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_kv4_attend(const __grid_constant__ Kv4AttendArgs a)
{
    __shared__ float red[kWarps][kSlot];
    __shared__ long long s_scan[kThreads + 1];
    __shared__ long long s_first[2];       // first unit of this CTA's share, tiles before that unit
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int p = blockIdx.x;

    // ---- the share: tiles of all units, and the unit the share starts in
    const int per = (a.U + kThreads - 1) / kThreads;
    const int u0 = min(tid * per, a.U), u1 = min(u0 + per, a.U);
    long long mine = 0;
    for (int u = u0; u < u1; ++u) mine += tiles_of(unit_of(a, u).count);
    s_scan[tid + 1] = mine;
    if (tid == 0) s_scan[0] = 0;
    __syncthreads();
    if (tid == 0)
        for (int i = 1; i <= kThreads; ++i) s_scan[i] += s_scan[i - 1];
    __syncthreads();
    const long long TT = s_scan[kThreads];
    // no more shares than tiles: the arrivals of a unit count every CTA
    // between its first and its last tile's owner
    const int P = TT < gridDim.x ? (int)(TT > 0 ? TT : 1) : (int)gridDim.x;
    const long long lo = p < P ? p * TT / P : TT, hi = p < P ? (p + 1) * TT / P : TT;
    if (lo < hi && lo >= s_scan[tid] && lo < s_scan[tid + 1]) {
        long long at = s_scan[tid];
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
        float m[kKv4MaxHeads], l[kKv4MaxHeads], o[kKv4MaxHeads][4];
        for (int h = 0; h < kKv4MaxHeads; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.f;
            for (int i = 0; i < 4; ++i) o[h][i] = 0.f;
        }
        warp_rows<BF16>(a, x, u, t0, t1, m, l, o);
        float* slot = a.part + (int64_t)(u + p) * a.NH * kSlot;
        for (int h = 0; h < a.NH; ++h) {
            __syncthreads();
            if (lane == 0) { red[warp][0] = m[h]; red[warp][1] = l[h]; }
            for (int i = 0; i < 4; ++i) red[warp][2 + 4 * lane + i] = o[h][i];
            __syncthreads();
            if (tid < kD) {
                float M = -INFINITY, L = 0.f, O = 0.f;
                for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red[w][0]);
                for (int w = 0; w < kWarps; ++w) {
                    const float c = red[w][0] == -INFINITY ? (red[w][1] == 0.f ? 0.f : 1.f) : expf(red[w][0] - M);
                    L += c * red[w][1];
                    O += c * red[w][2 + tid];
                }
                slot[h * kSlot + 2 + tid] = O;
                if (tid == 0) { slot[h * kSlot] = M; slot[h * kSlot + 1] = L; }
            }
        }
        __threadfence();
        __syncthreads();
        // ---- arrival; the unit's last piece merges every slot
        const int pf = owner_of(before, TT, P), pl = owner_of(end - 1, TT, P);
        if (tid == 0) s_last = atomicAdd(a.cnt + u, 1u) == (unsigned)(pl - pf);
        __syncthreads();
        if (s_last) {
            __threadfence();
            const float* s0 = a.part + (int64_t)(u + pf) * a.NH * kSlot;
            for (int i = tid; i < a.NH * kD; i += kThreads) {
                const int h = i / kD, d = i % kD;
                float M = -INFINITY, L = 0.f, O = 0.f;
                for (int s = 0; s <= pl - pf; ++s) M = fmaxf(M, __ldcg(s0 + ((int64_t)s * a.NH + h) * kSlot));
                for (int s = 0; s <= pl - pf; ++s) {
                    const float* q = s0 + ((int64_t)s * a.NH + h) * kSlot;
                    const float ms = __ldcg(q), ls = __ldcg(q + 1);
                    const float c = ms == -INFINITY ? (ls == 0.f ? 0.f : 1.f) : expf(ms - M);
                    L += c * ls;
                    O += c * __ldcg(q + 2 + d);
                }
                const int64_t hq = (int64_t)x.b * a.Hq + x.head0 + h;
                a.out[hq * kD + d] = L == 0.f ? 0.f : O / L;
                if (d == 0 && a.lse) a.lse[hq] = L == 0.f ? -INFINITY : M + logf(L);
            }
            if (tid == 0) a.cnt[u] = 0;
        }
        at = before + t1;
        before = end;
    }
}

}  // namespace

cudaError_t launch_kv4_attend(const Kv4AttendArgs& a, int bf16, int sms, cudaStream_t st)
{
    long long tiles = a.rows ? ((long long)a.S + a.max_rows + 1 + kTile - 1) / kTile : (a.n + kTile - 1) / kTile;
    tiles *= a.U;
    long long P = (tiles + kWarps - 1) / kWarps;
    P = P < 4LL * sms ? P : 4LL * sms;
    P = P < kKv4MaxCtas ? P : kKv4MaxCtas;
    if (bf16) k_kv4_attend<true><<<(unsigned)P, kThreads, 0, st>>>(a);
    else k_kv4_attend<false><<<(unsigned)P, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace ckv
