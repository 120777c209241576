// ckv_kv4.cu -- C ABI of the rows' way into the caches and of the 4-bit
// cache (declared in include/ckv.h): argument checks and launches.  None of
// these calls needs a context or allocates; they run on cfg->device whatever
// the current device is, only enqueue work, and can be captured into a graph.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "device_guard.h"
#include "kv4.cuh"

#define CKV_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr int kMaxDevices = 64;

// what these calls read of a configuration
bool valid_shape(const ckv_config* c)
{
    if (!c || c->batch < 1 || c->n_q_heads < 1 || c->n_kv_heads < 1 || c->n_q_heads % c->n_kv_heads) return false;
    if (c->head_dim != ckv::kD || c->n_max < 1 || c->n_max > INT32_MAX - 1023) return false;
    if (c->kv_dtype != CKV_F32 && c->kv_dtype != CKV_BF16) return false;
    if ((int64_t)c->batch * c->n_q_heads > (1 << 20)) return false;
    return c->device >= 0 && c->device < kMaxDevices;
}

bool valid_group(int group) { return group == 32 || group == 64 || group == 128; }

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// multiprocessors of a device; looked up once per device
ckv_status device_sms(int device, int* sms)
{
    static std::atomic<int> known[kMaxDevices];
    int n = known[device].load(std::memory_order_relaxed);
    if (!n) {
        int count = 0;
        if (cudaGetDeviceCount(&count) != cudaSuccess || device >= count) return CKV_ERR_INVALID_ARG;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return CKV_ERR_CUDA;
        known[device].store(n, std::memory_order_relaxed);
    }
    *sms = n;
    return CKV_OK;
}

ckv_status status_of(cudaError_t e)
{
    if (e == cudaSuccess) return CKV_OK;
    cudaGetLastError();                                    // reported here, not again by the next call
    return e == cudaErrorInvalidValue ? CKV_ERR_INVALID_ARG : CKV_ERR_CUDA;
}

int64_t kv_units(const ckv_config* c) { return (int64_t)c->batch * c->n_kv_heads; }

// rows [batch][tokens][heads]: 16-byte loads need 16-byte rows; the stride of
// a single one does not matter
bool valid_rows(const void* p, const int64_t* stride, int batch, int tokens, int heads, int esz)
{
    const int size[3] = {batch, tokens, heads};
    if (!aligned(p, 16)) return false;
    for (int i = 0; i < 3; ++i)
        if (size[i] > 1 && stride[i] % (16 / esz)) return false;
    return true;
}

// rows that are written: no two at one address by a stride of zero, and where
// they start with the rows that are read, they are those (in place)
bool valid_out(const ckv_qkv* x, int batch, int tokens, int heads)
{
    const int size[3] = {batch, tokens, heads};
    for (int i = 0; i < 3; ++i)
        if (size[i] > 1 && (x->q_out_stride[i] == 0 || (x->q_out == x->q && x->q_out_stride[i] != x->q_stride[i])))
            return false;
    return true;
}

// The counters at the head of a workspace, as many for every configuration:
// where they end may not depend on the call, since one call's partial results
// would lie where the next one, of another batch, expects zeros.
constexpr size_t kCounterBytes = ckv::kKv4MaxCtas * sizeof(unsigned);
static_assert(kCounterBytes % 256 == 0, "aligned partial results");

// everything of an attention call but its row lists
ckv_status attend(const ckv_config* cfg, int group, const void* q, const void* K4, const void* V4, int n,
                  const int32_t* lens, const int32_t* rows, const int32_t* n_rows, int max_rows, bool listed,
                  void* workspace, float* out, float* lse, void* stream)
{
    if (!valid_shape(cfg) || !valid_group(group) || !q || !K4 || !V4 || !workspace || !out) return CKV_ERR_INVALID_ARG;
    if (n < 1 || n > cfg->n_max) return CKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(K4, 16) || !aligned(V4, 16) || !aligned(workspace, 16) || !aligned(out, 16) ||
        !aligned(lens, 4) || !aligned(rows, 4) || !aligned(n_rows, 4) || !aligned(lse, 4))
        return CKV_ERR_INVALID_ARG;
    const int Gq = cfg->n_q_heads / cfg->n_kv_heads;
    const bool per_head = listed && cfg->mode == CKV_PER_HEAD;
    if (listed) {
        if (cfg->mode != CKV_PER_HEAD && cfg->mode != CKV_QUERY_GROUP) return CKV_ERR_INVALID_ARG;
        if (cfg->n_sinks < 0 || max_rows < 0 || (int64_t)cfg->n_sinks + max_rows > INT32_MAX - 1023) return CKV_ERR_INVALID_ARG;
        if (!n_rows || (max_rows > 0 && !rows)) return CKV_ERR_INVALID_ARG;
    }
    const int NH = per_head ? 1 : Gq;
    if (NH > ckv::kKv4MaxHeads) return CKV_ERR_INVALID_ARG;
    int sms = 0;
    if (ckv_status s = device_sms(cfg->device, &sms)) return s;
    ckv::DeviceGuard guard;
    if (guard.enter(cfg->device) != cudaSuccess) return CKV_ERR_CUDA;
    ckv::Kv4AttendArgs a{};
    a.q = q;
    a.K4 = ckv::kv4_view(const_cast<void*>(K4), kv_units(cfg), cfg->n_max);
    a.V4 = ckv::kv4_view(const_cast<void*>(V4), kv_units(cfg), cfg->n_max);
    a.B = cfg->batch;
    a.Hq = cfg->n_q_heads;
    a.Hkv = cfg->n_kv_heads;
    a.NH = NH;
    a.U = cfg->batch * cfg->n_q_heads / NH;
    a.n = n;
    a.group = group;
    a.device = cfg->device;
    a.lens = lens;
    if (listed) {
        // without a list the kernel still needs a non-null pointer to know the mode
        a.rows = rows ? rows : n_rows;
        a.n_rows = n_rows;
        a.max_rows = max_rows;
        a.S = cfg->n_sinks;
    }
    a.cnt = static_cast<unsigned*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kCounterBytes);
    a.out = out;
    a.lse = lse;
    return status_of(ckv::launch_kv4_attend(a, cfg->kv_dtype == CKV_BF16, sms, (cudaStream_t)stream));
}

}  // namespace

CKV_API size_t ckv_kv4_bytes(const ckv_config* cfg, int group)
{
    if (!valid_shape(cfg) || !valid_group(group)) return 0;
    return (size_t)kv_units(cfg) * ckv::kv4_rows(cfg->n_max) * (ckv::kRowCodes + ckv::kD / group * 4);
}

CKV_API size_t ckv_kv4_workspace(const ckv_config* cfg)
{
    if (!valid_shape(cfg)) return 0;
    const size_t Hq = cfg->n_q_heads, NH = Hq / cfg->n_kv_heads;
    return kCounterBytes + (cfg->batch * Hq + ckv::kKv4MaxCtas * NH) * (2 + ckv::kD) * sizeof(float);
}

CKV_API ckv_status ckv_qk_norm_rope(const ckv_config* cfg, const ckv_qkv* x, void* stream)
{
    if (!valid_shape(cfg) || !x) return CKV_ERR_INVALID_ARG;
    if (x->n_tokens < 0 || (int64_t)cfg->batch * x->n_tokens > INT32_MAX) return CKV_ERR_INVALID_ARG;
    // an array of no tokens may have no address
    if (x->n_tokens > 0 && (!x->q || !x->k || !x->v || !x->pos || !x->q_out)) return CKV_ERR_INVALID_ARG;
    if ((x->K == nullptr) != (x->V == nullptr) || (x->K4 == nullptr) != (x->V4 == nullptr)) return CKV_ERR_INVALID_ARG;
    if (!x->K && !x->K4) return CKV_ERR_INVALID_ARG;
    if (x->K4 && !valid_group(x->group)) return CKV_ERR_INVALID_ARG;
    if (x->rot_dim < 0 || x->rot_dim > ckv::kD || x->rot_dim % 16 || (x->rot_dim && !x->inv_freq_host))
        return CKV_ERR_INVALID_ARG;
    if (!(x->eps >= 0.f) || isinf(x->eps) || !isfinite(x->rot_scale)) return CKV_ERR_INVALID_ARG;
    const int esz = cfg->kv_dtype == CKV_BF16 ? 2 : 4;
    const int B = cfg->batch, T = x->n_tokens, Hq = cfg->n_q_heads, Hkv = cfg->n_kv_heads;
    if (!valid_rows(x->q, x->q_stride, B, T, Hq, esz) || !valid_rows(x->k, x->k_stride, B, T, Hkv, esz) ||
        !valid_rows(x->v, x->v_stride, B, T, Hkv, esz) || !valid_rows(x->q_out, x->q_out_stride, B, T, Hq, esz) ||
        !valid_out(x, B, T, Hq))
        return CKV_ERR_INVALID_ARG;
    if (!aligned(x->K, 16) || !aligned(x->V, 16) || !aligned(x->K4, 16) || !aligned(x->V4, 16) ||
        !aligned(x->q_weight, 16) || !aligned(x->k_weight, 16) || !aligned(x->pos, 4))
        return CKV_ERR_INVALID_ARG;
    ckv::QkvArgs a{};
    for (int i = 0; i < x->rot_dim / 2; ++i) {
        if (!isfinite(x->inv_freq_host[i])) return CKV_ERR_INVALID_ARG;
        a.turn[i] = x->inv_freq_host[i] / 6.283185307179586476925286766559;
    }
    if (x->n_tokens == 0) return CKV_OK;
    a.q = {x->q, x->q_stride[0], x->q_stride[1], x->q_stride[2]};
    a.k = {x->k, x->k_stride[0], x->k_stride[1], x->k_stride[2]};
    a.v = {x->v, x->v_stride[0], x->v_stride[1], x->v_stride[2]};
    a.B = cfg->batch;
    a.T = x->n_tokens;
    a.Hq = cfg->n_q_heads;
    a.Hkv = cfg->n_kv_heads;
    a.n_max = cfg->n_max;
    a.pos = x->pos;
    a.q_weight = x->q_weight;
    a.k_weight = x->k_weight;
    a.eps = x->eps;
    a.rot = x->rot_dim;
    a.interleaved = x->interleaved != 0;
    a.rot_scale = x->rot_scale;
    a.q_out = x->q_out;
    a.q_out_batch = x->q_out_stride[0];
    a.q_out_token = x->q_out_stride[1];
    a.q_out_head = x->q_out_stride[2];
    a.K = x->K;
    a.V = x->V;
    if (x->K4) {
        a.K4 = ckv::kv4_view(x->K4, kv_units(cfg), cfg->n_max);
        a.V4 = ckv::kv4_view(x->V4, kv_units(cfg), cfg->n_max);
        a.group = x->group;
    }
    int sms = 0;
    if (ckv_status s = device_sms(cfg->device, &sms)) return s;
    ckv::DeviceGuard guard;
    if (guard.enter(cfg->device) != cudaSuccess) return CKV_ERR_CUDA;
    return status_of(ckv::launch_qkv(a, cfg->kv_dtype == CKV_BF16, sms, (cudaStream_t)stream));
}

CKV_API ckv_status ckv_kv4_write(const ckv_config* cfg, int group, const void* k, const int64_t* k_stride_host,
                                 const void* v, const int64_t* v_stride_host, int n_tokens, const int32_t* pos,
                                 void* K4, void* V4, void* stream)
{
    if (!valid_shape(cfg) || !valid_group(group) || !k_stride_host || !v_stride_host || !K4 || !V4)
        return CKV_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!k || !v)) return CKV_ERR_INVALID_ARG;
    if (n_tokens < 0 || (int64_t)cfg->batch * n_tokens > INT32_MAX || (!pos && n_tokens > cfg->n_max))
        return CKV_ERR_INVALID_ARG;
    const int esz = cfg->kv_dtype == CKV_BF16 ? 2 : 4;
    if (!valid_rows(k, k_stride_host, cfg->batch, n_tokens, cfg->n_kv_heads, esz) ||
        !valid_rows(v, v_stride_host, cfg->batch, n_tokens, cfg->n_kv_heads, esz) || !aligned(K4, 16) || !aligned(V4, 16) ||
        !aligned(pos, 4))
        return CKV_ERR_INVALID_ARG;
    if (n_tokens == 0) return CKV_OK;
    ckv::QkvArgs a{};
    a.k = {k, k_stride_host[0], k_stride_host[1], k_stride_host[2]};
    a.v = {v, v_stride_host[0], v_stride_host[1], v_stride_host[2]};
    a.B = cfg->batch;
    a.T = n_tokens;
    a.Hkv = cfg->n_kv_heads;
    a.n_max = cfg->n_max;
    a.pos = pos;
    a.K4 = ckv::kv4_view(K4, kv_units(cfg), cfg->n_max);
    a.V4 = ckv::kv4_view(V4, kv_units(cfg), cfg->n_max);
    a.group = group;
    int sms = 0;
    if (ckv_status s = device_sms(cfg->device, &sms)) return s;
    ckv::DeviceGuard guard;
    if (guard.enter(cfg->device) != cudaSuccess) return CKV_ERR_CUDA;
    return status_of(ckv::launch_qkv(a, cfg->kv_dtype == CKV_BF16, sms, (cudaStream_t)stream));
}

CKV_API ckv_status ckv_kv4_read(const ckv_config* cfg, int group, const void* K4, const void* V4, int first, int count,
                                void* K, void* V, void* stream)
{
    if (!valid_shape(cfg) || !valid_group(group) || (!K && !V) || (K && !K4) || (V && !V4)) return CKV_ERR_INVALID_ARG;
    if (first < 0 || count < 0 || first > cfg->n_max - count) return CKV_ERR_INVALID_ARG;
    if (!aligned(K4, 16) || !aligned(V4, 16) || !aligned(K, 16) || !aligned(V, 16)) return CKV_ERR_INVALID_ARG;
    if (count == 0) return CKV_OK;
    ckv::Kv4ReadArgs a{};
    a.units = kv_units(cfg);
    if (K) a.K4 = ckv::kv4_view(const_cast<void*>(K4), a.units, cfg->n_max);
    if (V) a.V4 = ckv::kv4_view(const_cast<void*>(V4), a.units, cfg->n_max);
    a.n_max = cfg->n_max;
    a.first = first;
    a.count = count;
    a.group = group;
    a.K = K;
    a.V = V;
    int sms = 0;
    if (ckv_status s = device_sms(cfg->device, &sms)) return s;
    ckv::DeviceGuard guard;
    if (guard.enter(cfg->device) != cudaSuccess) return CKV_ERR_CUDA;
    return status_of(ckv::launch_kv4_read(a, cfg->kv_dtype == CKV_BF16, (cudaStream_t)stream));
}

CKV_API ckv_status ckv_kv4_dense_decode(const ckv_config* cfg, int group, const void* q, const void* K4, const void* V4,
                                        int n, const int32_t* lens, void* workspace, float* out, float* lse, void* stream)
{
    return attend(cfg, group, q, K4, V4, n, lens, nullptr, nullptr, 0, false, workspace, out, lse, stream);
}

CKV_API ckv_status ckv_kv4_attend_rows(const ckv_config* cfg, int group, const void* q, const void* K4, const void* V4,
                                       int n, const int32_t* lens, const int32_t* rows, const int32_t* n_rows,
                                       int max_rows, void* workspace, float* out, float* lse, void* stream)
{
    return attend(cfg, group, q, K4, V4, n, lens, rows, n_rows, max_rows, true, workspace, out, lse, stream);
}
