// api.cu -- the extern "C" entry points declared in include/w4moe.h: argument
// validation on the host, then kernel launches on the caller's stream.  No
// device allocation, no synchronisation, no device-to-host reads.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/w4moe.h"
#include "launch.h"
#include "strides.h"

namespace w4 {
PipelineTestHooks &pipeline_test_hooks()
{
    thread_local PipelineTestHooks hooks;
    return hooks;
}
}  // namespace w4

namespace {

thread_local char g_detail[512] = "";

int fail(int status, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_detail, sizeof(g_detail), fmt, ap);
    va_end(ap);
    return status;
}

int cuda_fail(cudaError_t err, const char *what)
{
    return fail(W4_ERR_CUDA, "%s: %s", what, cudaGetErrorString(err));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned2(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

cudaStream_t as_stream(w4_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// The cubin targets sm_103a only; refuse anything else up front.
int check_device()
{
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return cuda_fail(err, "cudaGetDevice");
    static std::atomic<uint64_t> known{0};       // devices found to be sm_103
    if (dev < 64 && (known.load(std::memory_order_relaxed) >> dev & 1u))
        return W4_OK;
    int major = 0, minor = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (major != 10 || minor != 3)
        return fail(W4_ERR_NO_DEVICE, "device %d is sm_%d%d; this library is built for sm_103a",
                    dev, major, minor);
    if (dev < 64)
        known.fetch_or(1ull << dev, std::memory_order_relaxed);
    return W4_OK;
}

bool valid_block_m(int bm) { return bm == 16 || bm == 32 || bm == 64 || bm == 128 || bm == 256; }

int64_t align_capacity(int M, int k, int E, int bm)
{
    const int64_t A = static_cast<int64_t>(M) * k;
    const int64_t cap = A + static_cast<int64_t>(E) * (bm - 1);
    return (cap + bm - 1) / bm * bm;
}

// Shared checks for the two grouped GEMMs.
int check_gemm_common(int M, int d, int m, int E, int k, int block_m, const void *act,
                      const void *q, const void *s, const void *z, const void *sorted_ids,
                      const void *offsets, const void *out)
{
    if (!act || !q || !s || !z || !sorted_ids || !offsets || !out)
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (M < 0 || d <= 0 || m <= 0 || E <= 0 || k <= 0)
        return fail(W4_ERR_INVALID_ARG, "sizes must be positive (M >= 0)");
    if (!valid_block_m(block_m))
        return fail(W4_ERR_INVALID_ARG, "block_m must be 16, 32, 64, 128 or 256 (got %d)", block_m);
    if (d % 128 || m % 64)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need d %% 128 == 0 and m %% 64 == 0 (d=%d, m=%d)", d,
                    m);
    if (d > 8192 || m > 1024)
        return fail(W4_ERR_UNSUPPORTED_SHAPE,
                    "need d <= 8192 and m <= 1024: the group sums of xg and h fill at most one "
                    "64-column block (d=%d, m=%d)", d, m);
    if (E > 1024 || k > E)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need k <= E <= 1024");
    const int64_t A = static_cast<int64_t>(M) * k;
    if (A > (1ll << 30) || static_cast<int64_t>(E) * 2 * m > (1ll << 30) ||
        static_cast<int64_t>(E) * d > (1ll << 30))
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "problem too large for 32-bit indexing");
    if (!aligned16(act) || !aligned16(q) || !aligned16(s) || !aligned16(z) || !aligned16(out))
        return fail(W4_ERR_MISALIGNED, "activation, weight, scale, zero and output pointers "
                                       "must be 16-byte aligned");
    if (!aligned4(sorted_ids) || !aligned4(offsets))
        return fail(W4_ERR_MISALIGNED, "index arrays must be 4-byte aligned");
    return W4_OK;
}

}  // namespace

int w4::check_device_sm103() { return check_device(); }

int w4::set_error_detail(int status, const char *detail)
{
    return fail(status, "%s", detail);
}

extern "C" {

const char *w4_status_string(int status)
{
    switch (status) {
    case W4_OK: return "W4_OK";
    case W4_ERR_INVALID_ARG: return "W4_ERR_INVALID_ARG";
    case W4_ERR_UNSUPPORTED_SHAPE: return "W4_ERR_UNSUPPORTED_SHAPE";
    case W4_ERR_MISALIGNED: return "W4_ERR_MISALIGNED";
    case W4_ERR_CUDA: return "W4_ERR_CUDA";
    case W4_ERR_NO_DEVICE: return "W4_ERR_NO_DEVICE";
    case W4_ERR_WORKSPACE: return "W4_ERR_WORKSPACE";
    default: return "W4_ERR_UNKNOWN";
    }
}

const char *w4_last_error_detail(void) { return g_detail; }

int w4_abi_version(void) { return W4MOE_ABI_VERSION; }

int w4_quantize(const float *W, int E, int N, int K, int group, uint8_t *q, uint16_t *s,
                uint16_t *z, w4_stream_t stream)
{
    if (!W || !q || !s || !z)
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (E < 0 || N < 0 || K <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes E=%d N=%d K=%d", E, N, K);
    if (group != 64 && group != 128 && group != 256)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "group must be 64, 128 or 256 (got %d)", group);
    if (K % group)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "group %d does not divide K=%d", group, K);
    if (!aligned16(W) || !aligned4(q) || !aligned4(s) || !aligned4(z))
        return fail(W4_ERR_MISALIGNED, "W must be 16-byte aligned, outputs 4-byte aligned");
    if (int rc = check_device())
        return rc;
    const int64_t rows = static_cast<int64_t>(E) * N;
    cudaError_t err = w4::launch_quantize(W, rows, K, group, q, s, z, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "quantize launch");
}

int w4_moe_route(const float *logits, int M, int E, int k, int32_t *topk_ids, float *topk_weights,
                 w4_stream_t stream)
{
    if (!logits || !topk_ids || !topk_weights)
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (M < 0 || E <= 0 || k <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes M=%d E=%d k=%d", M, E, k);
    if (k > 32 || k > E || E > 1024)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need 1 <= k <= 32, k <= E <= 1024");
    if (!aligned4(logits) || !aligned4(topk_ids) || !aligned4(topk_weights))
        return fail(W4_ERR_MISALIGNED, "pointers must be 4-byte aligned");
    if (int rc = check_device())
        return rc;
    cudaError_t err = w4::launch_route(logits, M, E, k, topk_ids, topk_weights, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "route launch");
}

int64_t w4_moe_align_capacity(int M, int k, int E, int block_m)
{
    if (M < 0 || k <= 0 || E <= 0 || !valid_block_m(block_m))
        return -1;
    return align_capacity(M, k, E, block_m);
}

int w4_moe_align(const int32_t *topk_ids, int M, int k, int E, int block_m, int32_t *sorted_ids,
                 int32_t *block_expert, int32_t *expert_offsets, int32_t *num_padded,
                 int32_t *dev_status, w4_stream_t stream)
{
    if (!sorted_ids || !block_expert || !expert_offsets || !num_padded || (M > 0 && !topk_ids))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (M < 0 || k <= 0 || E <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes M=%d k=%d E=%d", M, k, E);
    if (!valid_block_m(block_m))
        return fail(W4_ERR_INVALID_ARG, "block_m must be 16, 32, 64, 128 or 256 (got %d)", block_m);
    if (E > 1024)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "E must be <= 1024");
    const int64_t cap = align_capacity(M, k, E, block_m);
    if (cap > (1ll << 30))
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "too many assignments");
    if (int rc = check_device())
        return rc;
    cudaError_t err = w4::launch_align(topk_ids, M, k, E, block_m, cap, sorted_ids, block_expert,
                                       expert_offsets, num_padded, dev_status, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "align launch");
}

int w4_gather_activations(const uint16_t *x, int M, int d, int k, int E, int block_m,
                          const int32_t *sorted_ids, const int32_t *num_padded, uint16_t *xg,
                          int32_t *dev_status, w4_stream_t stream)
{
    if (!xg || !sorted_ids || !num_padded || (M > 0 && !x))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (M < 0 || d <= 0 || k <= 0 || E <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes M=%d d=%d k=%d E=%d", M, d, k, E);
    if (!valid_block_m(block_m))
        return fail(W4_ERR_INVALID_ARG, "block_m must be 16, 32, 64, 128 or 256 (got %d)", block_m);
    if (d % 128 || d > 8192)
        return fail(W4_ERR_UNSUPPORTED_SHAPE,
                    "d must be a multiple of 128 and at most 8192 (its group sums fill one "
                    "64-column block)");
    if (!aligned16(x) || !aligned16(xg) || !aligned4(sorted_ids) || !aligned4(num_padded))
        return fail(W4_ERR_MISALIGNED, "x and xg must be 16-byte aligned");
    if (int rc = check_device())
        return rc;
    const int64_t cap = align_capacity(M, k, E, block_m);
    cudaError_t err =
        w4::launch_gather(x, M, d, k, cap, sorted_ids, num_padded, xg, dev_status,
                          as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "gather launch");
}

int w4_moe_align_gather(const int32_t *topk_ids, const uint16_t *x, int M, int d, int k, int E,
                        int block_m, int32_t *sorted_ids, int32_t *block_expert,
                        int32_t *expert_offsets, int32_t *num_padded, uint16_t *xg,
                        int32_t *dev_status, w4_stream_t stream)
{
    if (!sorted_ids || !block_expert || !expert_offsets || !num_padded || !xg ||
        (M > 0 && (!topk_ids || !x)))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (M < 0 || d <= 0 || k <= 0 || E <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes M=%d d=%d k=%d E=%d", M, d, k, E);
    if (!valid_block_m(block_m))
        return fail(W4_ERR_INVALID_ARG, "block_m must be 16, 32, 64, 128 or 256 (got %d)", block_m);
    if (E > 1024 || d % 128 || d > 8192)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need E <= 1024, d %% 128 == 0 and d <= 8192");
    if (!aligned16(x) || !aligned16(xg))
        return fail(W4_ERR_MISALIGNED, "x and xg must be 16-byte aligned");
    const int64_t cap = align_capacity(M, k, E, block_m);
    if (cap > (1ll << 30))
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "too many assignments");
    if (int rc = check_device())
        return rc;
    cudaError_t err;
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (w4::align_gather_smem_bytes(M, k, E, sms) <= 200 * 1024) {
        err = w4::launch_align_gather(topk_ids, M, k, E, block_m, cap, sorted_ids, block_expert,
                                      expert_offsets, num_padded, dev_status, x, d, xg, sms,
                                      as_stream(stream));
    } else {   // too many assignments to keep their slots in shared memory
        err = w4::launch_align(topk_ids, M, k, E, block_m, cap, sorted_ids, block_expert,
                               expert_offsets, num_padded, dev_status, as_stream(stream));
        if (err == cudaSuccess)
            err = w4::launch_gather(x, M, d, k, cap, sorted_ids, num_padded, xg, dev_status,
                                    as_stream(stream));
    }
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "align+gather launch");
}

int w4_moe_route_align_gather(const float *logits, const uint16_t *x, int M, int d, int k, int E,
                              int block_m, int32_t *topk_ids, float *topk_weights,
                              int32_t *sorted_ids, int32_t *block_expert,
                              int32_t *expert_offsets, int32_t *num_padded, uint16_t *xg,
                              int32_t *dev_status, w4_stream_t stream)
{
    if (!topk_ids || !topk_weights || (M > 0 && !logits))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (k > 32 || k > E || E > 1024)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need 1 <= k <= 32, k <= E <= 1024");
    if (!aligned4(logits) || !aligned4(topk_ids) || !aligned4(topk_weights))
        return fail(W4_ERR_MISALIGNED, "logits, ids and weights must be 4-byte aligned");
    if (!sorted_ids || !block_expert || !expert_offsets || !num_padded || !xg ||
        (M > 0 && !x))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (M < 0 || d <= 0 || k <= 0 || E <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes M=%d d=%d k=%d E=%d", M, d, k, E);
    if (!valid_block_m(block_m))
        return fail(W4_ERR_INVALID_ARG, "block_m must be 16, 32, 64, 128 or 256 (got %d)", block_m);
    if (d % 128 || d > 8192)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need d %% 128 == 0 and d <= 8192");
    if (!aligned16(x) || !aligned16(xg))
        return fail(W4_ERR_MISALIGNED, "x and xg must be 16-byte aligned");
    if (int rc = check_device())
        return rc;
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (M > 0 && w4::route_align_gather_fits(M, k, E, sms)) {
        const int64_t cap = align_capacity(M, k, E, block_m);
        cudaError_t err = w4::launch_route_align_gather(
            logits, M, k, E, block_m, cap, topk_ids, topk_weights, sorted_ids, block_expert,
            expert_offsets, num_padded, dev_status, x, d, xg, sms, as_stream(stream));
        return err == cudaSuccess ? W4_OK : cuda_fail(err, "route+align+gather launch");
    }
    // larger shapes: the router launch, then the fused alignment and gather
    if (int rc = w4_moe_route(logits, M, E, k, topk_ids, topk_weights, stream))
        return rc;
    return w4_moe_align_gather(topk_ids, x, M, d, k, E, block_m, sorted_ids, block_expert,
                               expert_offsets, num_padded, xg, dev_status, stream);
}

}  // extern "C"

namespace {
// The layer's combine folded into the GEMMs (w4_moe_layer only; comb_cnt
// NULL elsewhere): see GroupedGemmProblem.
struct FoldedCombine {
    const int32_t *topk_ids = nullptr;
    const float *topk_w = nullptr;
    int32_t *cnt = nullptr;
    uint16_t *out = nullptr;
};

int grouped_gemm_gate_up(const uint16_t *xg, int M, int d, int m, int E, int k, int block_m,
                         const uint8_t *gu_q, const uint16_t *gu_s, const uint16_t *gu_z,
                         int group, const int32_t *sorted_ids, const int32_t *expert_offsets,
                         uint16_t *h, int32_t *dev_status, w4_stream_t stream,
                         const FoldedCombine &fc)
{
    if (int rc = check_gemm_common(M, d, m, E, k, block_m, xg, gu_q, gu_s, gu_z, sorted_ids,
                                   expert_offsets, h))
        return rc;
    if (group != 128)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "gate_up group must be 128 (got %d)", group);
    if (int rc = check_device())
        return rc;
    w4::GroupedGemmProblem p{};
    p.gate_up = true;
    p.act = xg;
    p.wq = gu_q;
    p.ws = gu_s;
    p.wz = gu_z;
    p.sorted_ids = sorted_ids;
    p.expert_offsets = expert_offsets;
    p.out = h;
    p.dev_status = dev_status;
    p.M = M;
    p.k = k;
    p.E = E;
    p.K = d;
    p.R = 2 * m;
    p.group = group;
    p.out_cols = m;
    p.cap = align_capacity(M, k, E, block_m);
    p.topk_ids = fc.topk_ids;
    p.comb_cnt = fc.cnt;
    p.comb_out = fc.out;
    p.comb_d = d;
    p.wait_ns = w4::pipeline_test_hooks().wait_ns;
    p.test_withhold_sz = w4::pipeline_test_hooks().withhold_sz;
    if (M == 0)
        return W4_OK;
    const char *why = nullptr;
    cudaError_t err = w4::launch_grouped_gemm(p, as_stream(stream), &why);
    if (why)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "%s", why);
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "gate_up launch");
}

// early_schedule: see GroupedGemmProblem (set only by w4_moe_layer, where the
// alignment is two launches back and gate_up waits for it before triggering)
int grouped_gemm_down(const uint16_t *h, int M, int d, int m, int E, int k, int block_m,
                      const uint8_t *dn_q, const uint16_t *dn_s, const uint16_t *dn_z, int group,
                      const int32_t *sorted_ids, const int32_t *expert_offsets, float *y,
                      int32_t *dev_status, w4_stream_t stream, bool early_schedule,
                      const FoldedCombine &fc)
{
    if (int rc = check_gemm_common(M, d, m, E, k, block_m, h, dn_q, dn_s, dn_z, sorted_ids,
                                   expert_offsets, y))
        return rc;
    if (group != 64)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "down group must be 64 (got %d)", group);
    if (int rc = check_device())
        return rc;
    w4::GroupedGemmProblem p{};
    p.gate_up = false;
    p.act = h;
    p.wq = dn_q;
    p.ws = dn_s;
    p.wz = dn_z;
    p.sorted_ids = sorted_ids;
    p.expert_offsets = expert_offsets;
    p.out = y;
    p.dev_status = dev_status;
    p.M = M;
    p.k = k;
    p.E = E;
    p.K = m;
    p.R = d;
    p.group = group;
    p.out_cols = d;
    p.cap = align_capacity(M, k, E, block_m);
    p.early_schedule = early_schedule;
    p.topk_ids = fc.topk_ids;
    p.topk_w = fc.topk_w;
    p.comb_cnt = fc.cnt;
    p.comb_out = fc.out;
    p.comb_d = d;
    p.wait_ns = w4::pipeline_test_hooks().wait_ns;
    p.test_withhold_sz = w4::pipeline_test_hooks().withhold_sz;
    if (M == 0)
        return W4_OK;
    const char *why = nullptr;
    cudaError_t err = w4::launch_grouped_gemm(p, as_stream(stream), &why);
    if (why)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "%s", why);
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "down launch");
}
}  // namespace

extern "C" {

int w4_grouped_gemm_gate_up(const uint16_t *xg, int M, int d, int m, int E, int k, int block_m,
                            const uint8_t *gu_q, const uint16_t *gu_s, const uint16_t *gu_z,
                            int group, const int32_t *sorted_ids, const int32_t *expert_offsets,
                            uint16_t *h, int32_t *dev_status, w4_stream_t stream)
{
    return grouped_gemm_gate_up(xg, M, d, m, E, k, block_m, gu_q, gu_s, gu_z, group, sorted_ids,
                                expert_offsets, h, dev_status, stream, FoldedCombine{});
}

int w4_grouped_gemm_down(const uint16_t *h, int M, int d, int m, int E, int k, int block_m,
                         const uint8_t *dn_q, const uint16_t *dn_s, const uint16_t *dn_z, int group,
                         const int32_t *sorted_ids, const int32_t *expert_offsets, float *y,
                         int32_t *dev_status, w4_stream_t stream)
{
    return grouped_gemm_down(h, M, d, m, E, k, block_m, dn_q, dn_s, dn_z, group, sorted_ids,
                             expert_offsets, y, dev_status, stream, false, FoldedCombine{});
}

int w4_grouped_gemm_down_combine(const uint16_t *h, int M, int d, int m, int E, int k,
                                 int block_m, const uint8_t *dn_q, const uint16_t *dn_s,
                                 const uint16_t *dn_z, int group, const int32_t *sorted_ids,
                                 const int32_t *expert_offsets, const int32_t *topk_ids,
                                 const float *topk_weights, int32_t *counters, float *y,
                                 uint16_t *out, int32_t *dev_status, w4_stream_t stream)
{
    if (M > 0 && (!topk_ids || !topk_weights || !counters || !out))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if ((reinterpret_cast<uintptr_t>(out) & 7u) || !aligned4(topk_ids) ||
        !aligned4(topk_weights) || !aligned4(counters))
        return fail(W4_ERR_MISALIGNED, "out must be 8-byte and topk_ids, topk_weights and "
                                       "counters 4-byte aligned");
    FoldedCombine fc;
    fc.topk_ids = topk_ids;
    fc.topk_w = topk_weights;
    fc.cnt = counters;
    fc.out = out;
    return grouped_gemm_down(h, M, d, m, E, k, block_m, dn_q, dn_s, dn_z, group, sorted_ids,
                             expert_offsets, y, dev_status, stream, false, fc);
}

int w4_test_pipeline_hooks(uint64_t wait_limit_ns, int withhold_first_scales)
{
    w4::PipelineTestHooks &h = w4::pipeline_test_hooks();
    h.wait_ns = wait_limit_ns ? wait_limit_ns : 1000000000ull;
    h.withhold_sz = withhold_first_scales != 0;
    return W4_OK;
}

int w4_moe_combine_prepare(const int32_t *topk_ids, int M, int k, int E, int d,
                           int32_t *counters, uint16_t *out, w4_stream_t stream)
{
    if (M > 0 && (!topk_ids || !counters || !out))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (M < 0 || k <= 0 || d <= 0 || E <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes M=%d k=%d d=%d E=%d", M, k, d, E);
    if (d % 128)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "d must be a multiple of 128 (got %d)", d);
    if (static_cast<int64_t>(M) * k >= (1ll << 31) || static_cast<int64_t>(M) * d >= (1ll << 31))
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "M * k and M * d must be below 2^31");
    if ((reinterpret_cast<uintptr_t>(out) & 7u) || !aligned4(topk_ids) || !aligned4(counters))
        return fail(W4_ERR_MISALIGNED, "out must be 8-byte and topk_ids and counters 4-byte "
                                       "aligned");
    if (M == 0)
        return W4_OK;
    if (int rc = check_device())
        return rc;
    cudaError_t err = w4::launch_combine_prepare(topk_ids, M, k, E, d, counters, out,
                                                 as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "combine prepare launch");
}

int w4_moe_combine_fixed_order(const float *y, const int32_t *topk_ids, const float *topk_weights,
                               int M, int k, int d, int E, uint16_t *out, w4_stream_t stream)
{
    if (!out || (M > 0 && (!y || !topk_ids || !topk_weights)))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (M < 0 || k <= 0 || d <= 0 || E <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes M=%d k=%d d=%d E=%d", M, k, d, E);
    if (d % 4)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "d must be a multiple of 4");
    if (!aligned16(y) || (reinterpret_cast<uintptr_t>(out) & 7u))
        return fail(W4_ERR_MISALIGNED, "y must be 16-byte and out 8-byte aligned");
    if (int rc = check_device())
        return rc;
    cudaError_t err =
        w4::launch_combine(y, topk_ids, topk_weights, M, k, d, E, out, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "combine launch");
}

}  // extern "C"

// Workspace layout of w4_moe_layer (each piece 256-byte aligned):
//   sorted_ids [cap] i32 | block_expert [cap/bm] i32 | expert_offsets [E+1] i32 |
//   num_padded [1] i32 | xg [cap, d + 64] fp16 | h [cap, m + 64] fp16 |
//   y [M*k, d] fp32
//   (xg and h rows end in their 64-column group-sum block)
namespace {
struct LayerWs {
    size_t sorted, block, offs, npad, xg, h, y, total;
};
size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
LayerWs layer_ws(int M, int d, int m, int E, int k, int bm)
{
    const size_t cap = static_cast<size_t>(align_capacity(M, k, E, bm));
    LayerWs w;
    w.sorted = 0;
    w.block = up256(w.sorted + 4 * cap);
    w.offs = up256(w.block + 4 * (cap / bm));
    w.npad = up256(w.offs + 4 * (static_cast<size_t>(E) + 1));
    w.xg = up256(w.npad + 4);
    w.h = up256(w.xg + 2 * cap * (static_cast<size_t>(d) + 64));
    w.y = up256(w.h + 2 * cap * (static_cast<size_t>(m) + 64));
    w.total = up256(w.y + 4 * static_cast<size_t>(M) * k * d);
    return w;
}

// The checks of the layer's GEMM and combine arguments, made before its
// first launch (the workspace pieces stand in for the intermediates).
int check_layer(int M, int d, int m, int E, int k, int block_m, const uint8_t *gu_q,
                const uint16_t *gu_s, const uint16_t *gu_z, int gu_group, const uint8_t *dn_q,
                const uint16_t *dn_s, const uint16_t *dn_z, int dn_group, const uint8_t *ws,
                const LayerWs &L, const float *topk_weights, const uint16_t *out)
{
    if (int rc = check_gemm_common(M, d, m, E, k, block_m, ws + L.xg, gu_q, gu_s, gu_z,
                                   ws + L.sorted, ws + L.offs, ws + L.h))
        return rc;
    if (int rc = check_gemm_common(M, d, m, E, k, block_m, ws + L.h, dn_q, dn_s, dn_z,
                                   ws + L.sorted, ws + L.offs, ws + L.y))
        return rc;
    if (gu_group != 128 || dn_group != 64)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need gate_up group 128 and down group 64 (got %d, %d)",
                    gu_group, dn_group);
    if (int rc = check_device())
        return rc;
    if (!w4::grouped_gemm_fits(true, d, gu_group, E) || !w4::grouped_gemm_fits(false, m, dn_group, E))
        return fail(W4_ERR_UNSUPPORTED_SHAPE,
                    "the grouped GEMMs' scale/zero stages do not fit shared memory (d=%d, m=%d, "
                    "E=%d; gate_up takes d up to about 3584 at E = 128)", d, m, E);
    if (M > 0 && (!out || !topk_weights))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if ((reinterpret_cast<uintptr_t>(out) & 7u) || !aligned4(topk_weights))
        return fail(W4_ERR_MISALIGNED, "out must be 8-byte and topk_weights 4-byte aligned");
    return W4_OK;
}

// gate_up (which also sets the combine counters) and down with the combine
// folded into its epilogue: the layer's launches after alignment+gather
int layer_gemms(const int32_t *topk_ids, const float *topk_weights, int M,
                int d, int m, int E, int k, int block_m, const uint8_t *gu_q,
                const uint16_t *gu_s, const uint16_t *gu_z, int gu_group, const uint8_t *dn_q,
                const uint16_t *dn_s, const uint16_t *dn_z, int dn_group, uint8_t *ws,
                const LayerWs &L, uint16_t *out, int32_t *dev_status, w4_stream_t stream)
{
    const int32_t *sorted = reinterpret_cast<const int32_t *>(ws + L.sorted);
    const int32_t *offs = reinterpret_cast<const int32_t *>(ws + L.offs);
    const uint16_t *xg = reinterpret_cast<const uint16_t *>(ws + L.xg);
    uint16_t *h = reinterpret_cast<uint16_t *>(ws + L.h);
    float *y = reinterpret_cast<float *>(ws + L.y);
    // The combine runs as its own launch: folded into the down GEMM
    // (w4_grouped_gemm_down_combine) the completed tokens gather on the CTAs
    // that finish last and their y reads (23 MB at M = 256, d = 2816, top-8)
    // run in those CTAs' tails, which measured ~13 us slower per layer than
    // the standalone fixed-order combine, which reads the same bytes with the
    // whole GPU and overlaps its start with the down GEMM's end.
    int rc = grouped_gemm_gate_up(xg, M, d, m, E, k, block_m, gu_q, gu_s, gu_z, gu_group, sorted,
                                  offs, h, dev_status, stream, FoldedCombine{});
    if (rc)
        return rc;
    rc = grouped_gemm_down(h, M, d, m, E, k, block_m, dn_q, dn_s, dn_z, dn_group, sorted, offs, y,
                           dev_status, stream, true, FoldedCombine{});
    if (rc)
        return rc;
    cudaError_t err = w4::launch_combine(y, topk_ids, topk_weights, M, k, d, E, out,
                                         as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "combine launch");
}
}  // namespace

extern "C" {

size_t w4_moe_layer_workspace_size(int M, int d, int m, int E, int k, int block_m)
{
    if (M < 0 || d <= 0 || m <= 0 || E <= 0 || k <= 0 || !valid_block_m(block_m))
        return 0;
    return layer_ws(M, d, m, E, k, block_m).total;
}

int w4_moe_layer(const uint16_t *x, const int32_t *topk_ids, const float *topk_weights, int M,
                 int d, int m, int E, int k, int block_m, const uint8_t *gu_q,
                 const uint16_t *gu_s, const uint16_t *gu_z, int gu_group, const uint8_t *dn_q,
                 const uint16_t *dn_s, const uint16_t *dn_z, int dn_group, void *workspace,
                 size_t workspace_bytes, uint16_t *out, int32_t *dev_status, w4_stream_t stream)
{
    if (!valid_block_m(block_m))
        return fail(W4_ERR_INVALID_ARG, "block_m must be 16, 32, 64, 128 or 256 (got %d)", block_m);
    if (M < 0 || d <= 0 || m <= 0 || E <= 0 || k <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes");
    const LayerWs L = layer_ws(M, d, m, E, k, block_m);
    if (!workspace || workspace_bytes < L.total)
        return fail(W4_ERR_WORKSPACE, "workspace needs %zu bytes", L.total);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(W4_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (int rc = check_layer(M, d, m, E, k, block_m, gu_q, gu_s, gu_z, gu_group, dn_q, dn_s, dn_z,
                             dn_group, ws, L, topk_weights, out))
        return rc;
    int32_t *sorted = reinterpret_cast<int32_t *>(ws + L.sorted);
    int32_t *block = reinterpret_cast<int32_t *>(ws + L.block);
    int32_t *offs = reinterpret_cast<int32_t *>(ws + L.offs);
    int32_t *npad = reinterpret_cast<int32_t *>(ws + L.npad);
    uint16_t *xg = reinterpret_cast<uint16_t *>(ws + L.xg);
    // alignment and the activation gather share one launch
    if (int rc0 = w4_moe_align_gather(topk_ids, x, M, d, k, E, block_m, sorted, block, offs, npad,
                                      xg, dev_status, stream))
        return rc0;
    if (M == 0)
        return W4_OK;
    return layer_gemms(topk_ids, topk_weights, M, d, m, E, k, block_m, gu_q, gu_s, gu_z,
                       gu_group, dn_q, dn_s, dn_z, dn_group, ws, L, out, dev_status, stream);
}

// Staging buffers of w4_moe_layer_host after the layer's workspace.
struct HostStaging {
    size_t x, ids, w, out, total;
};

static HostStaging host_staging(size_t base, int M, int d, int k)
{
    auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
    HostStaging h;
    h.x = up(base);
    h.ids = up(h.x + 2 * static_cast<size_t>(M) * d);
    h.w = up(h.ids + 4 * static_cast<size_t>(M) * k);
    h.out = up(h.w + 4 * static_cast<size_t>(M) * k);
    h.total = up(h.out + 2 * static_cast<size_t>(M) * d);
    return h;
}

size_t w4_moe_layer_host_workspace_size(int M, int d, int m, int E, int k, int block_m)
{
    if (M < 0 || d <= 0 || m <= 0 || E <= 0 || k <= 0 || !valid_block_m(block_m))
        return 0;
    return host_staging(layer_ws(M, d, m, E, k, block_m).total, M, d, k).total;
}

int w4_moe_layer_host(const uint16_t *x_host, const int32_t *topk_ids_host,
                      const float *topk_weights_host, int M, int d, int m, int E, int k,
                      int block_m, const uint8_t *gu_q, const uint16_t *gu_s,
                      const uint16_t *gu_z, int gu_group, const uint8_t *dn_q,
                      const uint16_t *dn_s, const uint16_t *dn_z, int dn_group, void *workspace,
                      size_t workspace_bytes, uint16_t *out_host, int32_t *dev_status,
                      w4_stream_t stream)
{
    if (!valid_block_m(block_m))
        return fail(W4_ERR_INVALID_ARG, "block_m must be 16, 32, 64, 128 or 256 (got %d)", block_m);
    if (M < 0 || d <= 0 || m <= 0 || E <= 0 || k <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes");
    if (M > 0 && (!x_host || !topk_ids_host || !topk_weights_host || !out_host))
        return fail(W4_ERR_INVALID_ARG, "NULL host buffer");
    const LayerWs L = layer_ws(M, d, m, E, k, block_m);
    const HostStaging H = host_staging(L.total, M, d, k);
    if (!workspace || workspace_bytes < H.total)
        return fail(W4_ERR_WORKSPACE, "workspace needs %zu bytes", H.total);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(W4_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    if (M == 0)   // no rows to copy or compute
        return W4_OK;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint16_t *x_d = reinterpret_cast<uint16_t *>(ws + H.x);
    int32_t *ids_d = reinterpret_cast<int32_t *>(ws + H.ids);
    float *w_d = reinterpret_cast<float *>(ws + H.w);
    uint16_t *out_d = reinterpret_cast<uint16_t *>(ws + H.out);
    const cudaStream_t s = as_stream(stream);
    const size_t nx = 2 * static_cast<size_t>(M) * d, nk = 4 * static_cast<size_t>(M) * k;
    cudaError_t err = cudaMemcpyAsync(x_d, x_host, nx, cudaMemcpyHostToDevice, s);
    if (err == cudaSuccess)
        err = cudaMemcpyAsync(ids_d, topk_ids_host, nk, cudaMemcpyHostToDevice, s);
    if (err == cudaSuccess)
        err = cudaMemcpyAsync(w_d, topk_weights_host, nk, cudaMemcpyHostToDevice, s);
    if (err != cudaSuccess)
        return fail(W4_ERR_CUDA, "host-to-device copy: %s", cudaGetErrorString(err));
    if (int rc = w4_moe_layer(x_d, ids_d, w_d, M, d, m, E, k, block_m, gu_q, gu_s, gu_z, gu_group,
                              dn_q, dn_s, dn_z, dn_group, workspace, L.total, out_d, dev_status,
                              stream))
        return rc;
    err = cudaMemcpyAsync(out_host, out_d, nx, cudaMemcpyDeviceToHost, s);
    if (err != cudaSuccess)
        return fail(W4_ERR_CUDA, "device-to-host copy: %s", cudaGetErrorString(err));
    return W4_OK;
}

int w4_moe_layer_from_logits(const uint16_t *x, const float *logits, int M, int d, int m, int E,
                             int k, int block_m, const uint8_t *gu_q, const uint16_t *gu_s,
                             const uint16_t *gu_z, int gu_group, const uint8_t *dn_q,
                             const uint16_t *dn_s, const uint16_t *dn_z, int dn_group,
                             void *workspace, size_t workspace_bytes, int32_t *topk_ids,
                             float *topk_weights, uint16_t *out, int32_t *dev_status,
                             w4_stream_t stream)
{
    if (!valid_block_m(block_m))
        return fail(W4_ERR_INVALID_ARG, "block_m must be 16, 32, 64, 128 or 256 (got %d)", block_m);
    if (M < 0 || d <= 0 || m <= 0 || E <= 0 || k <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes");
    const LayerWs L = layer_ws(M, d, m, E, k, block_m);
    if (!workspace || workspace_bytes < L.total)
        return fail(W4_ERR_WORKSPACE, "workspace needs %zu bytes", L.total);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(W4_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (int rc = check_layer(M, d, m, E, k, block_m, gu_q, gu_s, gu_z, gu_group, dn_q, dn_s, dn_z,
                             dn_group, ws, L, topk_weights, out))
        return rc;
    int32_t *sorted = reinterpret_cast<int32_t *>(ws + L.sorted);
    int32_t *block = reinterpret_cast<int32_t *>(ws + L.block);
    int32_t *offs = reinterpret_cast<int32_t *>(ws + L.offs);
    int32_t *npad = reinterpret_cast<int32_t *>(ws + L.npad);
    uint16_t *xg = reinterpret_cast<uint16_t *>(ws + L.xg);
    // router, alignment and activation gather share one launch
    if (int rc0 = w4_moe_route_align_gather(logits, x, M, d, k, E, block_m, topk_ids,
                                            topk_weights, sorted, block, offs, npad, xg,
                                            dev_status, stream))
        return rc0;
    if (M == 0)
        return W4_OK;
    return layer_gemms(topk_ids, topk_weights, M, d, m, E, k, block_m, gu_q, gu_s, gu_z,
                       gu_group, dn_q, dn_s, dn_z, dn_group, ws, L, out, dev_status, stream);
}

}  // extern "C"

// ------------------------------------------------- the layer for a few tokens
namespace {
int check_few(const void *x, int M, int d, int m, int E, int k, const void *gu_q,
              const void *gu_s, const void *gu_z, int gu_group, const void *dn_q,
              const void *dn_s, const void *dn_z, int dn_group, const void *workspace,
              size_t workspace_bytes, const void *ids, const void *w, const void *out)
{
    if (M < 0 || d <= 0 || m <= 0 || E <= 0 || k <= 0)
        return fail(W4_ERR_INVALID_ARG, "sizes must be positive (M >= 0)");
    if (!gu_q || !gu_s || !gu_z || !dn_q || !dn_s || !dn_z ||
        (M > 0 && (!x || !ids || !w || !out)))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (d % 128 || m % 64 || gu_group != 128 || dn_group != 64)
        return fail(W4_ERR_UNSUPPORTED_SHAPE,
                    "need d %% 128 == 0, m %% 64 == 0 and groups of 128 and 64 (d=%d, m=%d, "
                    "groups %d and %d)", d, m, gu_group, dn_group);
    if (E > 1024 || k > 32)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need E <= 1024 and k <= 32");
    if (!w4::few_supported(M, d, m, k))
        return fail(W4_ERR_UNSUPPORTED_SHAPE,
                    "need M <= 32, M * k <= 256 and rows that fit shared memory (M=%d, k=%d, d=%d, "
                    "m=%d)", M, k, d, m);
    if (!aligned16(x) || !aligned16(gu_q) || !aligned16(gu_s) || !aligned16(gu_z) ||
        !aligned16(dn_q) || !aligned16(dn_s) || !aligned16(dn_z) || !aligned16(out))
        return fail(W4_ERR_MISALIGNED, "x, weights, scales, zeros and out must be 16-byte aligned");
    if (!aligned4(ids) || !aligned4(w))
        return fail(W4_ERR_MISALIGNED, "ids and weights must be 4-byte aligned");
    const size_t need = w4_moe_layer_few_workspace_size(M, d, m, E, k);
    if (M > 0 && (!workspace || workspace_bytes < need))
        return fail(W4_ERR_WORKSPACE, "workspace needs %zu bytes", need);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(W4_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    return W4_OK;
}

int run_few(const uint16_t *x, const float *logits, int M, int d, int m, int E, int k,
            const uint8_t *gu_q, const uint16_t *gu_s, const uint16_t *gu_z, const uint8_t *dn_q,
            const uint16_t *dn_s, const uint16_t *dn_z, void *workspace, int32_t *ids, float *w,
            uint16_t *out, int32_t *dev_status, w4_stream_t stream)
{
    if (M == 0)
        return W4_OK;
    if (int rc = check_device())
        return rc;
    w4::FewProblem p{};
    p.x = x;
    p.logits = logits;
    p.ids = ids;
    p.w = w;
    p.gu_q = gu_q;
    p.gu_s = gu_s;
    p.gu_z = gu_z;
    p.dn_q = dn_q;
    p.dn_s = dn_s;
    p.dn_z = dn_z;
    p.workspace = workspace;
    p.out = out;
    p.dev_status = dev_status;
    p.M = M;
    p.d = d;
    p.m = m;
    p.E = E;
    p.k = k;
    cudaError_t err = w4::launch_few(p, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "few-token layer launch");
}
}  // namespace

size_t w4_moe_layer_few_workspace_size(int M, int d, int m, int E, int k)
{
    if (M < 0 || d <= 0 || m <= 0 || E <= 0 || k <= 0)
        return 0;
    return w4::few_workspace_bytes(M, d, m, k);
}

int w4_moe_layer_few(const uint16_t *x, const int32_t *topk_ids, const float *topk_weights, int M,
                     int d, int m, int E, int k, const uint8_t *gu_q, const uint16_t *gu_s,
                     const uint16_t *gu_z, int gu_group, const uint8_t *dn_q, const uint16_t *dn_s,
                     const uint16_t *dn_z, int dn_group, void *workspace, size_t workspace_bytes,
                     uint16_t *out, int32_t *dev_status, w4_stream_t stream)
{
    if (int rc = check_few(x, M, d, m, E, k, gu_q, gu_s, gu_z, gu_group, dn_q, dn_s, dn_z, dn_group,
                           workspace, workspace_bytes, topk_ids, topk_weights, out))
        return rc;
    // read only: without logits the kernels write neither
    return run_few(x, nullptr, M, d, m, E, k, gu_q, gu_s, gu_z, dn_q, dn_s, dn_z, workspace,
                   const_cast<int32_t *>(topk_ids), const_cast<float *>(topk_weights), out,
                   dev_status, stream);
}

int w4_moe_layer_few_from_logits(const uint16_t *x, const float *logits, int M, int d, int m, int E,
                                 int k, const uint8_t *gu_q, const uint16_t *gu_s,
                                 const uint16_t *gu_z, int gu_group, const uint8_t *dn_q,
                                 const uint16_t *dn_s, const uint16_t *dn_z, int dn_group,
                                 void *workspace, size_t workspace_bytes, int32_t *topk_ids,
                                 float *topk_weights, uint16_t *out, int32_t *dev_status,
                                 w4_stream_t stream)
{
    if (int rc = check_few(x, M, d, m, E, k, gu_q, gu_s, gu_z, gu_group, dn_q, dn_s, dn_z, dn_group,
                           workspace, workspace_bytes, topk_ids, topk_weights, out))
        return rc;
    if (M > 0 && !logits)
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (k > E)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need k <= E (k=%d, E=%d)", k, E);
    if (!aligned4(logits))
        return fail(W4_ERR_MISALIGNED, "logits must be 4-byte aligned");
    return run_few(x, logits, M, d, m, E, k, gu_q, gu_s, gu_z, dn_q, dn_s, dn_z, workspace,
                   topk_ids, topk_weights, out, dev_status, stream);
}

// -------------------------------------------------------------- paged cache
namespace {
int check_kv_state(const void *table, int B, int W, const void *lens, const void *refs, int P)
{
    if (!table || !lens || !refs)
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (B <= 0 || W <= 0 || P <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes B=%d W=%d P=%d", B, W, P);
    if (static_cast<int64_t>(B) * W >= (1ll << 30) || P >= (1 << 30))
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need B * W and P below 2^30");
    if (!aligned4(table) || !aligned4(lens) || !aligned4(refs))
        return fail(W4_ERR_MISALIGNED, "table, lens and refs must be 4-byte aligned");
    return W4_OK;
}

int check_kv_pool(const void *pool, int planes, int64_t page_bytes, int page_size)
{
    if (!pool)
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (planes <= 0 || page_bytes <= 0 || page_size <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes planes=%d page_bytes=%lld page_size=%d", planes,
                    static_cast<long long>(page_bytes), page_size);
    if (planes > 65535 || page_bytes % (16ll * page_size))
        return fail(W4_ERR_UNSUPPORTED_SHAPE,
                    "need at most 65535 planes and tokens of a multiple of 16 bytes");
    if (!aligned16(pool))
        return fail(W4_ERR_MISALIGNED, "the pool must be 16-byte aligned");
    return W4_OK;
}

int check_kv_workspace(const void *workspace, size_t bytes, int P, int n)
{
    const size_t need = w4_kv_workspace_size(P, n);
    if (!workspace || bytes < need)
        return fail(W4_ERR_WORKSPACE, "workspace needs %zu bytes", need);
    if (!aligned16(workspace))
        return fail(W4_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    return W4_OK;
}
}  // namespace

size_t w4_kv_workspace_size(int P, int n)
{
    return P < 0 || n < 0 ? 0 : w4::kv_workspace_bytes(P, n);
}

int w4_kv_reserve(int32_t *table, int B, int W, int32_t *lens, int32_t *refs, int P,
                  const int32_t *slots, const int32_t *new_lens, int n, int page_size,
                  int32_t *dev_status, w4_stream_t stream)
{
    if (int rc = check_kv_state(table, B, W, lens, refs, P))
        return rc;
    if (n < 0 || page_size <= 0 || (n > 0 && (!slots || !new_lens)))
        return fail(W4_ERR_INVALID_ARG, "bad n=%d, page_size=%d or NULL slots", n, page_size);
    if (n > 1024)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "at most 1024 slots per call (got %d)", n);
    if (n == 0)
        return W4_OK;
    if (int rc = check_device())
        return rc;
    cudaError_t err = w4::launch_kv_reserve(table, B, W, lens, refs, P, slots, new_lens, n,
                                            page_size, dev_status, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "kv_reserve launch");
}

int w4_kv_free(int32_t *table, int B, int W, int32_t *lens, int32_t *refs, int P,
               const int32_t *slots, int n, int32_t *dev_status, w4_stream_t stream)
{
    if (int rc = check_kv_state(table, B, W, lens, refs, P))
        return rc;
    if (n < 0 || (n > 0 && !slots))
        return fail(W4_ERR_INVALID_ARG, "bad n=%d or NULL slots", n);
    if (n == 0)
        return W4_OK;
    if (int rc = check_device())
        return rc;
    cudaError_t err = w4::launch_kv_free(table, B, W, lens, refs, P, slots, n, dev_status,
                                         as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "kv_free launch");
}

int w4_kv_fork(void *pool, int planes, int64_t page_bytes, int32_t *table, int B, int W,
               int32_t *lens, int32_t *refs, int P, const int32_t *parents,
               const int32_t *children, int n, int page_size, void *workspace,
               size_t workspace_bytes, int32_t *dev_status, w4_stream_t stream)
{
    if (int rc = check_kv_state(table, B, W, lens, refs, P))
        return rc;
    if (int rc = check_kv_pool(pool, planes, page_bytes, page_size))
        return rc;
    if (n < 0 || (n > 0 && (!parents || !children)))
        return fail(W4_ERR_INVALID_ARG, "bad n=%d or NULL slots", n);
    if (n > 1024)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "at most 1024 forks per call (got %d)", n);
    if (n == 0)
        return W4_OK;
    if (int rc = check_kv_workspace(workspace, workspace_bytes, P, n))
        return rc;
    if (int rc = check_device())
        return rc;
    cudaError_t err = w4::launch_kv_fork(static_cast<uint8_t *>(pool), planes, page_bytes, table, B,
                                         W, lens, refs, P, parents, children, n, page_size,
                                         workspace, dev_status, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "kv_fork launch");
}

int w4_kv_copy_pages(void *pool, int planes, int64_t page_bytes, int P, const int32_t *src,
                     const int32_t *dst, int n, int32_t *dev_status, w4_stream_t stream)
{
    if (int rc = check_kv_pool(pool, planes, page_bytes, 1))
        return rc;
    if (P <= 0 || n < 0 || (n > 0 && (!src || !dst)))
        return fail(W4_ERR_INVALID_ARG, "bad P=%d, n=%d or NULL lists", P, n);
    if (n == 0)
        return W4_OK;
    if (int rc = check_device())
        return rc;
    cudaError_t err = w4::launch_kv_copy(static_cast<uint8_t *>(pool), planes, page_bytes, P, src,
                                         dst, n, dev_status, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "kv_copy_pages launch");
}

int w4_kv_compact(void *pool, int planes, int64_t page_bytes, const int32_t *table, int B, int W,
                  const int32_t *refs, int P, int32_t *table_out, int32_t *refs_out,
                  void *workspace, size_t workspace_bytes, int32_t *dev_status, w4_stream_t stream)
{
    if (int rc = check_kv_state(table, B, W, refs, refs, P))
        return rc;
    if (!table_out || !refs_out)
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned4(table_out) || !aligned4(refs_out))
        return fail(W4_ERR_MISALIGNED, "table_out and refs_out must be 4-byte aligned");
    if (int rc = check_kv_pool(pool, planes, page_bytes, 1))
        return rc;
    if (int rc = check_kv_workspace(workspace, workspace_bytes, P, 0))
        return rc;
    if (int rc = check_device())
        return rc;
    cudaError_t err = w4::launch_kv_compact(static_cast<uint8_t *>(pool), planes, page_bytes, table,
                                            static_cast<int64_t>(B) * W, refs, P, table_out,
                                            refs_out, workspace, dev_status, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "kv_compact launch");
}

int w4_kv_append(uint16_t *k_pages, uint16_t *v_pages, int64_t page_stride, int64_t tok_stride,
                 int64_t head_stride, int P, int page_size, int Hkv, int D, const int32_t *table,
                 int B, int W, const int32_t *lens, const uint16_t *k, int64_t k_tok_stride,
                 int64_t k_head_stride, const uint16_t *v, int64_t v_tok_stride,
                 int64_t v_head_stride, const int32_t *q_offsets, int T, int32_t *dev_status,
                 w4_stream_t stream)
{
    if (int rc = check_kv_state(table, B, W, lens, lens, P))
        return rc;
    if (!k_pages || !v_pages || !q_offsets || (T > 0 && (!k || !v)))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (page_size <= 0 || Hkv <= 0 || D <= 0 || T < 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes page_size=%d Hkv=%d D=%d T=%d", page_size, Hkv,
                    D, T);
    if (D % 8 || static_cast<int64_t>(Hkv) * D >= (1ll << 30))
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "D must be a multiple of 8 (got %d)", D);
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k) || !aligned16(v) ||
        (page_stride | tok_stride | head_stride | k_tok_stride | k_head_stride | v_tok_stride |
         v_head_stride) & 7 || !aligned4(q_offsets))
        return fail(W4_ERR_MISALIGNED, "pointers must be 16-byte aligned and strides multiples of "
                                       "8 elements");
    if (T == 0)
        return W4_OK;
    if (int rc = check_device())
        return rc;
    w4::KvAppend a{};
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.page_stride = page_stride;
    a.tok_stride = tok_stride;
    a.head_stride = head_stride;
    a.k = k;
    a.v = v;
    a.k_tok = k_tok_stride;
    a.k_head = k_head_stride;
    a.v_tok = v_tok_stride;
    a.v_head = v_head_stride;
    a.table = table;
    a.lens = lens;
    a.q_offsets = q_offsets;
    a.dev_status = dev_status;
    a.P = P;
    a.page = page_size;
    a.Hkv = Hkv;
    a.D = D;
    a.B = B;
    a.W = W;
    a.T = T;
    cudaError_t err = w4::launch_kv_append(a, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "kv_append launch");
}

int w4_kv_keep(void *pool, int planes, int64_t page_bytes, const int32_t *table, int B, int W,
               const int32_t *lens, const int32_t *refs, int P, const int32_t *q_offsets,
               const int32_t *kept, const int32_t *kept_offsets, int n_kept, int page_size,
               int32_t *lens_out, int32_t *dev_status, w4_stream_t stream)
{
    if (n_kept < 0 || B < 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes n_kept=%d B=%d", n_kept, B);
    if (B == 0)
        return W4_OK;
    if (int rc = check_kv_state(table, B, W, lens, refs, P))
        return rc;
    if (int rc = check_kv_pool(pool, planes, page_bytes, page_size))
        return rc;
    if (!q_offsets || !kept_offsets || !lens_out || (n_kept > 0 && !kept))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned4(q_offsets) || !aligned4(kept) || !aligned4(kept_offsets) || !aligned4(lens_out))
        return fail(W4_ERR_MISALIGNED, "index arrays must be 4-byte aligned");
    if (static_cast<int64_t>(W) * page_size >= (1ll << 31) || B > (1 << 24))
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need W * page_size below 2^31 and B up to 2^24");
    if (int rc = check_device())
        return rc;
    w4::KvKeep k{};
    k.pool = static_cast<uint8_t *>(pool);
    k.page_bytes = page_bytes;
    k.table = table;
    k.lens = lens;
    k.refs = refs;
    k.q_offsets = q_offsets;
    k.kept = kept;
    k.kept_offsets = kept_offsets;
    k.lens_out = lens_out;
    k.dev_status = dev_status;
    k.planes = planes;
    k.P = P;
    k.B = B;
    k.W = W;
    k.page = page_size;
    k.n_kept = n_kept;
    cudaError_t err = w4::launch_kv_keep(k, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "kv_keep launch");
}

// --------------------------------------------------- norms and rotation
int w4_rope_steps(int rot, double base, int method, double factor, double trained_len, double low,
                  double high, int64_t *steps)
{
    if (rot < 0 || rot % 2 || (rot > 0 && !steps))
        return fail(W4_ERR_INVALID_ARG, "rot must be even (got %d) and steps not NULL", rot);
    if (!(base > 0.0) || !std::isfinite(base) || !(factor > 0.0) || !std::isfinite(factor))
        return fail(W4_ERR_INVALID_ARG, "base and factor must be positive and finite");
    if (method != W4_ROPE_LINEAR && method != W4_ROPE_BASE && method != W4_ROPE_PARTS)
        return fail(W4_ERR_INVALID_ARG, "unknown method %d", method);
    if (method == W4_ROPE_PARTS && (!(trained_len > 0.0) || !std::isfinite(trained_len) ||
                                    !(high > low) || !std::isfinite(high) || !std::isfinite(low)))
        return fail(W4_ERR_INVALID_ARG, "need trained_len > 0 and low < high");
    if (method == W4_ROPE_BASE && rot == 2)
        return fail(W4_ERR_INVALID_ARG, "raising the base needs rot > 2");
    constexpr double kTurn = 6.283185307179586476925286766559;
    const double b =
        method == W4_ROPE_BASE && rot > 2 ? base * std::pow(factor, rot / (rot - 2.0)) : base;
    for (int i = 0; i < rot / 2; i++) {
        const double f = std::pow(b, -2.0 * i / rot);
        double scaled = method == W4_ROPE_LINEAR ? f / factor : f;
        if (method == W4_ROPE_PARTS) {
            const double turns = trained_len * f / kTurn;
            const double x = (turns - low) / (high - low), keep = x < 0.0 ? 0.0 : x > 1.0 ? 1.0 : x;
            scaled = f * keep + f / factor * (1.0 - keep);
        }
        // the fraction of a turn: whole turns at integer positions change nothing
        const double turns = scaled / kTurn, part = turns - std::floor(turns);
        const double bits = std::ldexp(part, 64);
        steps[i] = static_cast<int64_t>(bits < 18446744073709551616.0 ? static_cast<uint64_t>(bits)
                                                                      : 0);
    }
    return W4_OK;
}

namespace {
// What both rotations ask of queries, keys, weights and steps.
int check_rope(const w4::RopeProblem &r, float eps)
{
    if (r.T < 0 || r.Hq < 0 || r.Hkv < 0 || r.D <= 0 || r.rot < 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes T=%d Hq=%d Hkv=%d D=%d rot=%d", r.T, r.Hq,
                    r.Hkv, r.D, r.rot);
    if (!(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(r.amplitude))
        return fail(W4_ERR_INVALID_ARG, "eps must not be negative, eps and amplitude finite");
    if (r.D % 8 || r.D > 256)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "D must be a multiple of 8 up to 256 (got %d)", r.D);
    if (r.rot % 16 || r.rot > r.D)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "rot must be a multiple of 16 up to D (got %d of %d)",
                    r.rot, r.D);
    if (static_cast<int64_t>(r.Hq) + 2ll * r.Hkv > 65535)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need Hq + 2 Hkv up to 65535 (got %d, %d)", r.Hq,
                    r.Hkv);
    if (r.T > 0 && ((r.Hq > 0 && (!r.q || !r.q_out)) || (r.Hkv > 0 && !r.k) ||
                    (r.rot > 0 && !r.steps)))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(r.q) || !aligned16(r.k) || !aligned16(r.q_out) || !aligned16(r.q_weight) ||
        !aligned16(r.k_weight) ||
        (r.q_tok | r.q_head | r.k_tok | r.k_head | r.q_out_tok | r.q_out_head) & 7)
        return fail(W4_ERR_MISALIGNED, "queries, keys and weights must be 16-byte aligned and "
                                       "strides multiples of 8 elements");
    if (!aligned4(r.positions) || (reinterpret_cast<uintptr_t>(r.steps) & 7u))
        return fail(W4_ERR_MISALIGNED, "positions must be 4-byte, steps 8-byte aligned");
    if (w4::rows_overlap(r.T, r.Hq, r.D, r.q_out_tok, r.q_out_head))
        return fail(W4_ERR_INVALID_ARG, "tokens or heads of q_out overlap");
    return W4_OK;
}
}  // namespace

int w4_qk_norm_rope(const uint16_t *q, int64_t q_tok_stride, int64_t q_head_stride,
                    const uint16_t *k, int64_t k_tok_stride, int64_t k_head_stride,
                    const int32_t *positions, const int64_t *steps, const uint16_t *q_weight,
                    const uint16_t *k_weight, int T, int Hq, int Hkv, int D, int rot,
                    int interleaved, int dtype, float eps, float amplitude, uint16_t *q_out,
                    int64_t q_out_tok_stride, int64_t q_out_head_stride, uint16_t *k_out,
                    int64_t k_out_tok_stride, int64_t k_out_head_stride, w4_stream_t stream)
{
    w4::RopeProblem r{};
    r.q = q;
    r.q_tok = q_tok_stride;
    r.q_head = q_head_stride;
    r.k = k;
    r.k_tok = k_tok_stride;
    r.k_head = k_head_stride;
    r.q_out = q_out;
    r.q_out_tok = q_out_tok_stride;
    r.q_out_head = q_out_head_stride;
    r.k_out = k_out;
    r.k_out_tok = k_out_tok_stride;
    r.k_out_head = k_out_head_stride;
    r.positions = positions;
    r.steps = steps;
    r.q_weight = q_weight;
    r.k_weight = k_weight;
    r.T = T;
    r.Hq = Hq;
    r.Hkv = Hkv;
    r.D = D;
    r.rot = rot;
    r.interleaved = interleaved != 0;
    r.bf16 = dtype == 0;
    r.eps = eps;
    r.amplitude = amplitude;
    if (dtype != 0 && dtype != 1)
        return fail(W4_ERR_INVALID_ARG, "dtype must be 0 or 1 (got %d)", dtype);
    if (int rc = check_rope(r, eps))
        return rc;
    if (T == 0 || Hq + Hkv == 0)
        return W4_OK;
    if (!positions || (Hkv > 0 && !k_out))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(k_out) || (k_out_tok_stride | k_out_head_stride) & 7)
        return fail(W4_ERR_MISALIGNED, "outputs must be 16-byte aligned and their strides multiples "
                                       "of 8 elements");
    if (w4::rows_overlap(T, Hkv, D, k_out_tok_stride, k_out_head_stride))
        return fail(W4_ERR_INVALID_ARG, "tokens or heads of k_out overlap");
    if (int rc = check_device())
        return rc;
    cudaError_t err = w4::launch_rope(r, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "qk_norm_rope launch");
}

int w4_kv_append_rope(uint16_t *k_pages, uint16_t *v_pages, int64_t page_stride, int64_t tok_stride,
                      int64_t head_stride, int P, int page_size, const int32_t *table, int B, int W,
                      const int32_t *lens, const uint16_t *q, int64_t q_tok_stride,
                      int64_t q_head_stride, const uint16_t *k, int64_t k_tok_stride,
                      int64_t k_head_stride, const uint16_t *v, int64_t v_tok_stride,
                      int64_t v_head_stride, const int32_t *q_offsets, const int32_t *positions,
                      const int64_t *steps, const uint16_t *q_weight, const uint16_t *k_weight,
                      int T, int Hq, int Hkv, int D, int rot, int interleaved, int dtype, float eps,
                      float amplitude, uint16_t *q_out, int64_t q_out_tok_stride,
                      int64_t q_out_head_stride, int32_t *dev_status, w4_stream_t stream)
{
    w4::RopeProblem r{};
    r.q = q;
    r.q_tok = q_tok_stride;
    r.q_head = q_head_stride;
    r.k = k;
    r.k_tok = k_tok_stride;
    r.k_head = k_head_stride;
    r.v = v;
    r.v_tok = v_tok_stride;
    r.v_head = v_head_stride;
    r.q_out = q_out;
    r.q_out_tok = q_out_tok_stride;
    r.q_out_head = q_out_head_stride;
    r.k_pages = k_pages;
    r.v_pages = v_pages;
    r.page_stride = page_stride;
    r.tok_stride = tok_stride;
    r.head_stride = head_stride;
    r.table = table;
    r.lens = lens;
    r.q_offsets = q_offsets;
    r.positions = positions;
    r.steps = steps;
    r.q_weight = q_weight;
    r.k_weight = k_weight;
    r.dev_status = dev_status;
    r.T = T;
    r.Hq = Hq;
    r.Hkv = Hkv;
    r.D = D;
    r.rot = rot;
    r.interleaved = interleaved != 0;
    r.P = P;
    r.page = page_size;
    r.B = B;
    r.W = W;
    r.bf16 = dtype == 0;
    r.eps = eps;
    r.amplitude = amplitude;
    if (dtype != 0 && dtype != 1)
        return fail(W4_ERR_INVALID_ARG, "dtype must be 0 or 1 (got %d)", dtype);
    if (int rc = check_kv_state(table, B, W, lens, lens, P))
        return rc;
    if (int rc = check_rope(r, eps))
        return rc;
    if (!k_pages || !v_pages || !q_offsets || (T > 0 && !v))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (page_size <= 0 || Hkv <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes page_size=%d Hkv=%d", page_size, Hkv);
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(v) ||
        (page_stride | tok_stride | head_stride | v_tok_stride | v_head_stride) & 7 ||
        !aligned4(q_offsets))
        return fail(W4_ERR_MISALIGNED, "pointers must be 16-byte aligned and strides multiples of "
                                       "8 elements");
    if (T == 0)
        return W4_OK;
    if (int rc = check_device())
        return rc;
    cudaError_t err = w4::launch_rope(r, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "kv_append_rope launch");
}

// ---------------------------------------------------------------- attention
size_t w4_attn_shared_prefix_workspace_size(int T, int B, int G, int max_q, int Hq, int Hkv, int D)
{
    if (T < 0 || B < 0 || G < 0 || max_q <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || D <= 0)
        return 0;
    return w4::attn_workspace_bytes(T, B, G, max_q, Hq, Hkv, D);
}

// Both attentions; tree NULL: causal counts.
static int run_attn(const uint16_t *q, int64_t q_tok_stride, int64_t q_head_stride,
                    const uint16_t *k_pages, const uint16_t *v_pages, int64_t page_stride,
                    int64_t tok_stride, int64_t head_stride, int P, int page_size,
                    const int32_t *table, int W, const int32_t *lens, const int32_t *q_offsets,
                    int T, int B, int max_q, const int32_t *group_offsets,
                    const int32_t *shared_lens, int G, int Hq, int Hkv, int D, int dtype,
                    int causal, const uint32_t *tree, int tree_words, float scale,
                    void *workspace, size_t workspace_bytes, uint16_t *out, int32_t *dev_status,
                    w4_stream_t stream)
{
    if (T < 0 || B < 0 || G < 0 || max_q <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || P <= 0 ||
        W <= 0 || (dtype != 0 && dtype != 1))
        return fail(W4_ERR_INVALID_ARG, "bad sizes or dtype (T=%d B=%d G=%d max_q=%d Hq=%d Hkv=%d "
                    "D=%d P=%d W=%d dtype=%d)", T, B, G, max_q, Hq, Hkv, D, P, W, dtype);
    if (!(scale > 0.0f) || scale > 1e30f)
        return fail(W4_ERR_INVALID_ARG, "scale must be positive and finite");
    if (D != 64 && D != 128)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "D must be 64 or 128 (got %d)", D);
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "page_size must be 16, 32, 64 or 128 (got %d)",
                    page_size);
    if (Hq % Hkv)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "Hkv must divide Hq (%d, %d)", Hkv, Hq);
    if (static_cast<int64_t>(B) + G > 4000)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need B + G <= 4000 (got %d + %d)", B, G);
    const int64_t rows = static_cast<int64_t>(T) * Hq;
    const int64_t keys = static_cast<int64_t>(W) * page_size;
    const int64_t items = 2 * (rows / 128 + 1) + (static_cast<int64_t>(B) + G) * Hkv;
    if (rows * D >= (1ll << 31) || keys >= (1ll << 30) || items * (keys / 128 + 4) >= (1ll << 31) ||
        static_cast<int64_t>(max_q) * Hq >= (1ll << 30))
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "problem too large for 32-bit counts");
    if (T == 0 || B == 0)
        return W4_OK;
    if (!q || !k_pages || !v_pages || !table || !lens || !q_offsets || !out ||
        (G > 0 && (!group_offsets || !shared_lens)))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) ||
        (q_tok_stride | q_head_stride | page_stride | tok_stride | head_stride) & 7)
        return fail(W4_ERR_MISALIGNED, "q, the pages and out must be 16-byte aligned and strides "
                                       "multiples of 8 elements");
    if (!aligned4(table) || !aligned4(lens) || !aligned4(q_offsets) || !aligned4(group_offsets) ||
        !aligned4(shared_lens))
        return fail(W4_ERR_MISALIGNED, "index arrays must be 4-byte aligned");
    if (page_stride <= 0 || tok_stride <= 0 || head_stride <= 0)
        return fail(W4_ERR_INVALID_ARG, "the pages' strides must be positive");
    const size_t need = w4_attn_shared_prefix_workspace_size(T, B, G, max_q, Hq, Hkv, D);
    if (!workspace || workspace_bytes < need)
        return fail(W4_ERR_WORKSPACE, "workspace needs %zu bytes", need);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(W4_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    if (int rc = check_device())
        return rc;
    w4::AttnProblem p{};
    p.q = q;
    p.q_tok = q_tok_stride;
    p.q_head = q_head_stride;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.page_stride = page_stride;
    p.tok_stride = tok_stride;
    p.head_stride = head_stride;
    p.table = table;
    p.lens = lens;
    p.q_offsets = q_offsets;
    p.group_offsets = group_offsets;
    p.shared = shared_lens;
    p.workspace = workspace;
    p.out = out;
    p.dev_status = dev_status;
    p.T = T;
    p.B = B;
    p.G = G;
    p.W = W;
    p.P = P;
    p.page = page_size;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.max_q = max_q;
    p.causal = causal != 0;
    p.tree = tree;
    p.tree_words = tree_words;
    p.bf16 = dtype == 0;
    p.scale = scale;
    cudaError_t err = w4::launch_attn(p, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "attention launch");
}

int w4_attn_shared_prefix(const uint16_t *q, int64_t q_tok_stride, int64_t q_head_stride,
                          const uint16_t *k_pages, const uint16_t *v_pages, int64_t page_stride,
                          int64_t tok_stride, int64_t head_stride, int P, int page_size,
                          const int32_t *table, int W, const int32_t *lens,
                          const int32_t *q_offsets, int T, int B, int max_q,
                          const int32_t *group_offsets, const int32_t *shared_lens, int G, int Hq,
                          int Hkv, int D, int dtype, int causal, float scale, void *workspace,
                          size_t workspace_bytes, uint16_t *out, int32_t *dev_status,
                          w4_stream_t stream)
{
    return run_attn(q, q_tok_stride, q_head_stride, k_pages, v_pages, page_stride, tok_stride,
                    head_stride, P, page_size, table, W, lens, q_offsets, T, B, max_q,
                    group_offsets, shared_lens, G, Hq, Hkv, D, dtype, causal, nullptr, 0, scale,
                    workspace, workspace_bytes, out, dev_status, stream);
}

int w4_attn_tree(const uint16_t *q, int64_t q_tok_stride, int64_t q_head_stride,
                 const uint16_t *k_pages, const uint16_t *v_pages, int64_t page_stride,
                 int64_t tok_stride, int64_t head_stride, int P, int page_size,
                 const int32_t *table, int W, const int32_t *lens, const int32_t *q_offsets, int T,
                 int B, int max_q, const uint32_t *tree, int tree_words,
                 const int32_t *group_offsets, const int32_t *shared_lens, int G, int Hq, int Hkv,
                 int D, int dtype, float scale, void *workspace, size_t workspace_bytes,
                 uint16_t *out, int32_t *dev_status, w4_stream_t stream)
{
    if (tree_words < 0 || (max_q > 0 && tree_words < (max_q - 1) / 32 + 1))
        return fail(W4_ERR_INVALID_ARG, "a row of tree must have a bit for each of max_q tokens "
                    "(max_q=%d tree_words=%d)", max_q, tree_words);
    if (T > 0 && B > 0 && !tree)
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned4(tree))
        return fail(W4_ERR_MISALIGNED, "tree must be 4-byte aligned");
    return run_attn(q, q_tok_stride, q_head_stride, k_pages, v_pages, page_stride, tok_stride,
                    head_stride, P, page_size, table, W, lens, q_offsets, T, B, max_q,
                    group_offsets, shared_lens, G, Hq, Hkv, D, dtype, 0, tree, tree_words, scale,
                    workspace, workspace_bytes, out, dev_status, stream);
}

// ------------------------------------------------------------------ RMSNorm
int w4_rmsnorm(const uint16_t *x, const uint16_t *weight, int M, int d, float eps, uint16_t *y,
               w4_stream_t stream)
{
    if (!weight || (M > 0 && (!x || !y)))
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (M < 0 || d <= 0 || !(eps >= 0.0f))
        return fail(W4_ERR_INVALID_ARG, "bad sizes or eps (M=%d d=%d)", M, d);
    if (d % 8)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "d must be a multiple of 8 (got %d)", d);
    if (static_cast<int64_t>(M) * d >= (1ll << 31))
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "M * d must be below 2^31");
    if (!aligned16(x) || !aligned16(weight) || !aligned16(y))
        return fail(W4_ERR_MISALIGNED, "x, weight and y must be 16-byte aligned");
    if (M == 0)
        return W4_OK;
    if (int rc = check_device())
        return rc;
    cudaError_t err = w4::launch_rmsnorm(x, weight, M, d, eps, y, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "rmsnorm launch");
}

// ------------------------------------------------------------------ sampler
size_t w4_sample_logits_workspace_size(int M, int64_t V)
{
    if (M <= 0 || V <= 0 || V >= (1ll << 31))
        return 0;
    return w4::sampler_workspace_bytes(M, V);
}

int w4_sample_logits(const float *logits, int M, int64_t V, uint64_t seed, uint64_t offset,
                     float *entropy, int64_t *sample, int64_t *argmax, void *workspace,
                     size_t workspace_bytes, w4_stream_t stream)
{
    if (M < 0 || V <= 0 || V >= (1ll << 31))
        return fail(W4_ERR_INVALID_ARG, "need M >= 0 and 0 < V < 2^31 (M=%d V=%lld)", M,
                    static_cast<long long>(V));
    if (M == 0)
        return W4_OK;
    if (!logits)
        return fail(W4_ERR_INVALID_ARG, "NULL logits");
    if (!entropy && !sample && !argmax)
        return fail(W4_ERR_INVALID_ARG, "no output requested");
    if (!aligned4(logits))
        return fail(W4_ERR_MISALIGNED, "logits must be 4-byte aligned");
    if (!workspace || workspace_bytes < w4::sampler_workspace_bytes(M, V) || !aligned16(workspace))
        return fail(W4_ERR_WORKSPACE, "workspace must be 16-byte aligned and hold %zu bytes",
                    w4::sampler_workspace_bytes(M, V));
    if (int rc = check_device())
        return rc;
    cudaError_t err = w4::launch_sampler(logits, M, V, seed, offset, entropy, sample, argmax,
                                         workspace, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "sampler launch");
}

int w4_fused_entropy(const float *logits, int M, int64_t V, float *entropy, void *workspace,
                     size_t workspace_bytes, w4_stream_t stream)
{
    if (!entropy)
        return fail(W4_ERR_INVALID_ARG, "NULL entropy");
    return w4_sample_logits(logits, M, V, 0, 0, entropy, nullptr, nullptr, workspace,
                            workspace_bytes, stream);
}

int w4_gumbel_argmax_sample(const float *logits, int M, int64_t V, uint64_t seed,
                            uint64_t offset, int64_t *sample, int64_t *argmax, void *workspace,
                            size_t workspace_bytes, w4_stream_t stream)
{
    if (!sample)
        return fail(W4_ERR_INVALID_ARG, "NULL sample");
    return w4_sample_logits(logits, M, V, seed, offset, nullptr, sample, argmax, workspace,
                            workspace_bytes, stream);
}

// ----------------------------------------------------------- dense linear
// Workspace of w4_w4a16_linear (each piece 256-byte aligned):
//   sorted_ids [padded] i32 | offsets [2] i32 | xg [padded, K] fp16 |
//   partial sums [splits, M, N] fp32 (dense kernel with a split contraction)
// with padded = M rounded up to 16 (the one expert's slots).
namespace {
constexpr int kLinearBlockM = 16;
struct LinearWs {
    size_t sorted, offs, xg, part, total;
    int padded;
};
LinearWs linear_ws(int M, int K, int N, int group)
{
    LinearWs w;
    w.padded = (M + kLinearBlockM - 1) / kLinearBlockM * kLinearBlockM;
    w.sorted = 0;
    w.offs = up256(4 * static_cast<size_t>(w.padded));
    w.xg = up256(w.offs + 8);
    w.part = up256(w.xg + 2 * static_cast<size_t>(w.padded) * K);
    const bool split = M > 0 && w4::dense_gemm_supported(M, N, K, group);
    w.total = up256(w.part + (split ? w4::dense_gemm_partial_bytes(M, N, K) : 0));
    return w;
}
}  // namespace

size_t w4_w4a16_linear_workspace_size(int M, int K, int N, int group)
{
    if (M < 0 || K <= 0 || N <= 0)
        return 0;
    return linear_ws(M, K, N, group).total;
}

int w4_w4a16_linear(const uint16_t *x, int M, int K, int N, const uint8_t *q, const uint16_t *s,
                    const uint16_t *z, int group, void *workspace, size_t workspace_bytes,
                    uint16_t *y, int32_t *dev_status, w4_stream_t stream)
{
    if (M < 0 || K <= 0 || N <= 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes M=%d K=%d N=%d", M, K, N);
    if (M == 0)
        return W4_OK;
    if (!x || !q || !s || !z || !y)
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (group != 64 && group != 128)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "group must be 64 or 128 (got %d)", group);
    if (K % group || K % 64 || K < 256 || N % 128 || K / group > 32)
        return fail(W4_ERR_UNSUPPORTED_SHAPE,
                    "need K >= 256, a multiple of the group and of 64, with at most 32 groups, "
                    "N a multiple of 128 (K=%d N=%d group=%d)", K, N, group);
    if (static_cast<int64_t>(M) * K > (1ll << 30) || static_cast<int64_t>(M) * N > (1ll << 30) ||
        static_cast<int64_t>(N) * K > (1ll << 31))
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "problem too large for 32-bit indexing");
    if (!aligned16(x) || !aligned16(q) || !aligned16(s) || !aligned16(z) || !aligned16(y))
        return fail(W4_ERR_MISALIGNED, "x, q, s, z and y must be 16-byte aligned");
    const LinearWs L = linear_ws(M, K, N, group);
    if (!workspace || workspace_bytes < L.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return fail(W4_ERR_WORKSPACE, "workspace must be 256-byte aligned and hold %zu bytes",
                    L.total);
    if (int rc = check_device())
        return rc;
    char *ws = static_cast<char *>(workspace);
    int32_t *sorted = reinterpret_cast<int32_t *>(ws + L.sorted);
    int32_t *offs = reinterpret_cast<int32_t *>(ws + L.offs);
    uint16_t *xg = reinterpret_cast<uint16_t *>(ws + L.xg);
    // every token in the one "expert" that is the whole matrix, one slot each
    cudaError_t err = w4::launch_identity_align_gather(x, M, K, L.padded, sorted, offs, xg,
                                                       as_stream(stream));
    if (err != cudaSuccess)
        return cuda_fail(err, "identity alignment launch");
    w4::DenseGemmProblem d{};
    d.xg = xg;
    d.q = q;
    d.s = s;
    d.z = z;
    d.y = y;
    d.partials = reinterpret_cast<float *>(ws + L.part);
    d.dev_status = dev_status;
    d.M = M;
    d.N = N;
    d.K = K;
    d.group = group;
    const char *why = nullptr;
    err = w4::launch_dense_gemm(d, as_stream(stream), &why);
    if (why)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "%s", why);
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "dense GEMM launch");
}

int w4_w4a16_linear_few(const uint16_t *x, int M, int K, int N, const uint8_t *q,
                        const uint16_t *s, const uint16_t *z, int group, uint16_t *y,
                        int32_t *dev_status, w4_stream_t stream)
{
    if (M < 0 || K <= 0 || N < 0)
        return fail(W4_ERR_INVALID_ARG, "bad sizes M=%d K=%d N=%d", M, K, N);
    if (M == 0 || N == 0)
        return W4_OK;
    if (!x || !q || !s || !z || !y)
        return fail(W4_ERR_INVALID_ARG, "NULL pointer argument");
    if (group != 64 && group != 128)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "group must be 64 or 128 (got %d)", group);
    if (M > 32 || K % group || K > 11264)
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need M <= 32 and K a multiple of the group up to "
                                              "11264 (M=%d K=%d group=%d)", M, K, group);
    if (N >= (1 << 30) || static_cast<int64_t>(N) * K >= (1ll << 33))
        return fail(W4_ERR_UNSUPPORTED_SHAPE, "need N below 2^30 and N * K below 2^33");
    if (!aligned16(x) || !aligned16(q) || !aligned2(s) || !aligned2(z) || !aligned4(y))
        return fail(W4_ERR_MISALIGNED, "x and q must be 16-byte aligned, y 4-byte, s and z 2-byte aligned");
    if (int rc = check_device())
        return rc;
    w4::FewLinearProblem l{};
    l.x = x;
    l.q = q;
    l.s = s;
    l.z = z;
    l.y = y;
    l.dev_status = dev_status;
    l.M = M;
    l.K = K;
    l.N = N;
    l.group = group;
    cudaError_t err = w4::launch_few_linear(l, as_stream(stream));
    return err == cudaSuccess ? W4_OK : cuda_fail(err, "few-token linear launch");
}
