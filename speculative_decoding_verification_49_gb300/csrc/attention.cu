// attention.cu -- the verifier's attention of new tokens over the KV cache.
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "spec_verify_cache.h"
#include "sv_device.cuh"

namespace {

using namespace sv;

constexpr int kMaxT = 128;

struct Params {
    sv_attention_args a;
};

__device__ __forceinline__ float code_scale(uint8_t s)
{
    return s ? __int_as_float((int)s << 23) : __int_as_float(0x00400000);
}

template <int E> __device__ __forceinline__ void load_row(const void *base, const uint8_t *scale, size_t row, int lane, int D, float *x)
{
    if (!scale) {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(base) + row * D + lane * E;
#pragma unroll
        for (int i = 0; i < E; ++i)
            x[i] = __bfloat162float(p[i]);
    } else {
        const __nv_fp8_storage_t *p = static_cast<const __nv_fp8_storage_t *>(base) + row * D + lane * E;
        const float s = code_scale(scale[row]);
#pragma unroll
        for (int i = 0; i < E; ++i)
            x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3))) * s;
    }
}

// One warp per query row, one pass over the keys with the running maximum and sum.
template <int E> __global__ void __launch_bounds__(128) sv_attention_kernel(Params p)
{
    const sv_attention_args &a = p.a;
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int T = (int)a.T, Hq = (int)a.heads_q, Hk = (int)a.heads_kv, D = 32 * E;
    if (row >= a.B * T * Hq)
        return;
    const int hq = (int)(row % Hq), t = (int)(row / Hq % T);
    const long long b = row / Hq / T;
    const int h = hq / (Hq / Hk);
    float q[E], o[E], m = -INFINITY, l = 0.0f;
    bool poison = false;
    const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q) + b * a.q_stride_b + t * a.q_stride_t + hq * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        q[i] = __bfloat162float(qp[i]);
        o[i] = 0.0f;
    }
    const float c = (float)(a.softmax_scale * 1.4426950408889634);
    auto step = [&](const float *k, const float *v) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i)
            s = fmaf(q[i], k[i], s);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= c;
        const float mn = fmax_nan(m, s), mu = mn == -INFINITY ? 0.0f : mn;
        const float f = exp2f(m - mu), w = exp2f(s - mu);
        l = l * f + w;
#pragma unroll
        for (int i = 0; i < E; ++i)
            o[i] = fmaf(w, v[i], o[i] * f);
        m = mn;
    };
    float k[E], v[E];
    const bool e4 = a.format == SV_KV_E4M3;
    for (long long j = 0; j < a.prefix_len; ++j) {
        const size_t r = (size_t)j * Hk + h;
        load_row<E>(a.k_prefix, e4 ? a.k_prefix_scale : nullptr, r, lane, D, k);
        load_row<E>(a.v_prefix, e4 ? a.v_prefix_scale : nullptr, r, lane, D, v);
        step(k, v);
    }
    long long len = a.max_len > 0 ? a.cache_len[b] : 0;
    if (len < 0 || len > a.max_len) {
        if (lane == 0 && a.status)
            atomicOr(a.status, SV_ATTN_BAD_LEN);
        len = 0;
        poison = true;
    }
    for (long long j = 0; j < len; ++j) {
        const size_t r = ((size_t)b * a.max_len + j) * Hk + h;
        load_row<E>(a.k_cache, e4 ? a.k_scale : nullptr, r, lane, D, k);
        load_row<E>(a.v_cache, e4 ? a.v_scale : nullptr, r, lane, D, v);
        step(k, v);
    }
    if (a.k_new) {
        const int32_t *par = a.parent ? a.parent + b * T : nullptr;
        if (par) {
            bool bad = false;
            for (int n = lane; n < T; n += 32)
                bad |= n == 0 ? par[n] != -1 : par[n] < 0 || par[n] >= n;
            if (__any_sync(0xffffffffu, bad)) {
                if (lane == 0 && a.status)
                    atomicOr(a.status, SV_ATTN_BAD_TREE);
                poison = true;
            }
        }
        for (int j = t; j >= 0 && !poison; j = par ? par[j] : j - 1) {
            const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(a.k_new) + b * a.new_stride_b + j * a.new_stride_t + h * D + lane * E;
            const __nv_bfloat16 *vp = static_cast<const __nv_bfloat16 *>(a.v_new) + b * a.new_stride_b + j * a.new_stride_t + h * D + lane * E;
            bool nf = false;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                k[i] = __bfloat162float(kp[i]);
                v[i] = __bfloat162float(vp[i]);
                nf |= !isfinite(v[i]);
            }
            if (__any_sync(0xffffffffu, nf))
                l = __int_as_float(0x7fc00000);
            step(k, v);
        }
    }
    const bool empty = m == -INFINITY && l == 0.0f;
    const float nan = __int_as_float(0x7fc00000);
    const float inv = poison ? nan : empty ? 0.0f : 1.0f / l;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + row * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i)
        out[i] = __float2bfloat16(o[i] * inv);
    if (a.lse && lane == 0)
        a.lse[row] = poison ? nan : (m + log2f(l)) * 0.69314718055994531f;
}

sv_status check(const sv_attention_args *a)
{
    if (!a || a->B < 0 || a->T < 1 || a->T > kMaxT || a->heads_kv < 1 || a->heads_q < 1 ||
        a->heads_q % a->heads_kv != 0 || a->max_len < 0 || a->prefix_len < 0)
        return SV_ERR_INVALID_ARG;
    if (a->head_dim != 64 && a->head_dim != 128)
        return SV_ERR_SHAPE;
    if (a->format != SV_KV_BF16 && a->format != SV_KV_E4M3)
        return SV_ERR_DTYPE;
    if (!(a->softmax_scale > 0.0) || !std::isfinite((float)a->softmax_scale) || !((float)a->softmax_scale > 0.0f))
        return SV_ERR_INVALID_ARG;
    return SV_OK;
}

bool al16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

} // namespace

extern "C" sv_status spec_verify_attention_workspace(const sv_attention_args *args, int64_t *bytes)
{
    const sv_status st = check(args);
    if (st != SV_OK)
        return st;
    if (!bytes)
        return SV_ERR_INVALID_ARG;
    *bytes = 16;
    return SV_OK;
}

extern "C" sv_status spec_verify_attention(const sv_attention_args *args, void *stream)
{
    sv_status st = check(args);
    if (st != SV_OK)
        return st;
    const sv_attention_args &a = *args;
    if (a.B == 0)
        return SV_OK;
    const bool e4 = a.format == SV_KV_E4M3;
    if (!a.q || !a.out || (a.max_len > 0 && (!a.k_cache || !a.v_cache || !a.cache_len || (e4 && (!a.k_scale || !a.v_scale)))) ||
        (a.prefix_len > 0 && (!a.k_prefix || !a.v_prefix || (e4 && (!a.k_prefix_scale || !a.v_prefix_scale)))) ||
        (!a.k_new) != (!a.v_new))
        return SV_ERR_INVALID_ARG;
    if (!al16(a.q) || !al16(a.out) || !al16(a.k_cache) || !al16(a.v_cache) || !al16(a.k_prefix) || !al16(a.v_prefix) ||
        !al16(a.k_new) || !al16(a.v_new) || !al16(a.workspace))
        return SV_ERR_INVALID_ARG;
    const int64_t qrow = a.heads_q * a.head_dim, nrow = a.heads_kv * a.head_dim;
    if ((a.B > 1 && a.q_stride_b < qrow) || (a.T > 1 && a.q_stride_t < qrow) ||
        (a.k_new && ((a.B > 1 && a.new_stride_b < nrow) || (a.T > 1 && a.new_stride_t < nrow))))
        return SV_ERR_INVALID_ARG;
    if (!a.workspace || a.workspace_bytes < 16)
        return SV_ERR_INVALID_ARG;
    if (a.q_stride_b % 8 || a.q_stride_t % 8 || (a.k_new && (a.new_stride_b % 8 || a.new_stride_t % 8)))
        return SV_ERR_INVALID_ARG;
    if (a.B > INT_MAX / a.T / a.heads_q || a.B * ((a.max_len + 127) / 128 + 1) > INT_MAX / a.heads_kv)
        return SV_ERR_TOO_LARGE;
    Params p{a};
    const unsigned grid = (unsigned)((a.B * a.T * a.heads_q + 3) / 4);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.head_dim == 64)
        sv_attention_kernel<2><<<grid, 128, 0, s>>>(p);
    else
        sv_attention_kernel<4><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
