// kv4.cuh -- the 4-bit KV cache: its format, and the launchers of the kernels
// that write, read and attend to it.
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

// A launch's own status.  cudaGetLastError() after <<<>>> would also report,
// as this call's, what an earlier call of the thread that failed left behind.
template <class... Params, class... Args>
cudaError_t launch_kernel(void (*fn)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, const Args&... args)
{
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    return cudaLaunchKernelEx(&c, fn, args...);
}

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
    int device;                      // ordinal, below 64
    const int32_t* lens;             // [B], or null: n for every sequence
    const int32_t* rows;             // [U][max_rows], or null: dense
    const int32_t* n_rows;           // [U]
    int max_rows, S;
    float* part;                     // o [U + kKv4MaxCtas][NH][D], then (m, l) [U + kKv4MaxCtas][NH][2]
    unsigned* cnt;                   // [kKv4MaxCtas] arrivals, 0 between calls
    float* out;                      // [B][Hq][D]
    float* lse;                      // [B][Hq] or null
};
constexpr int kKv4MaxCtas = 640;     // most CTAs of the attention grid (slots of the workspace)
constexpr int kKv4MaxHeads = 8;      // query heads of a unit
cudaError_t launch_kv4_attend(const Kv4AttendArgs& a, int bf16, int sms, cudaStream_t st);

}  // namespace ckv
