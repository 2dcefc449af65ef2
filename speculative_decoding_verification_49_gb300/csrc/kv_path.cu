// kv_path.cu -- commit of the accepted path into a bf16 or e4m3 KV cache, and
// the read-back of an e4m3 cache, for sm_103a.
//
// "Speculative decoding -- draft, verify, repeat" (factory.pai-world.com,
// lesson 07-16), section "KV cache dance": after the verify the accepted
// entries are appended and the others dropped.  The 8-bit format is this
// library's own.
//
// Commit.  One (row, head) vector x of D elements becomes codes
// round_e4m3(x * 2^-e) and the scale byte e + 127, e the smallest whole number
// in [-40, 120] with max|x| <= 448 * 2^e: with max|x| = (1 + f) * 2^E, e = E - 8,
// plus 1 when f > 0.75 (448 = 1.75 * 2^8), read off the bf16 bits.  A lane holds
// 8 elements (one 16-byte load), D / 8 lanes share a vector (rounded up to a
// power of two, the rest idle) and find its maximum by xor shuffles.
// A cluster of CTAs serves one sequence in all planes, so one launch does the
// copy and the new length: every CTA reads cache_len, the cluster barrier's
// arrival follows, and one thread writes the length after the barrier, which
// allows out_len == cache_len.
// Bound: HBM on rows * heads * (2 D in + D + 1 out) bytes; at a serving batch the
// rows are few, so launch and load latency count first.
//
// Read-back.  A sequence's rows are contiguous in a plane, so a thread takes 16
// codes (one 16-byte load) at a time and writes 32 bytes; HBM bound on 3 D + 1
// bytes per vector.
#include <climits>
#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "spec_verify_cache.h"
#include "sv_device.cuh"

namespace {

using namespace sv;

constexpr int kPathThreads = 256;
constexpr int kPathUnroll = 4;  // vectors of a lane group in flight
constexpr int kPathMaxT = 1024;
constexpr int kReadThreads = 256;
constexpr int kReadUnroll = 4;  // 16-code chunks of a thread in flight
constexpr int kEMin = -40, kEMax = 120;  // range of a scale's exponent

struct PathParams {
    const unsigned char *rows;  // bf16 [P][B][T][heads][D]
    unsigned char *cache;
    uint8_t *scale;
    const int32_t *cache_len;
    int32_t *out_len;
    const int32_t *nacc, *path;
    int32_t *status;
    int P, B, T, lead, max_len, heads, D;
};

// A vector's scale exponent from the largest magnitude of its finite elements
// (the 15 low bits of a bf16).
__device__ __forceinline__ int scale_exponent(unsigned m)
{
    const int e = (int)(m >> 7) - 127 - 8 + ((m & 127u) > 96u ? 1 : 0);
    return min(max(e, kEMin), kEMax);
}

__device__ __forceinline__ float pow2i(int e)
{
    return __int_as_float((e + 127) << 23);
}

// 8 bf16 (four words) times s as 8 e4m3 codes; NaN and infinities become NaN.
__device__ __forceinline__ uint2 quantise8(const unsigned *w, float s)
{
    unsigned out[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        unsigned c[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const unsigned u = w[2 * i + j];
            float lo = __uint_as_float(u << 16), hi = __uint_as_float(u & 0xffff0000u);
            lo = (u & 0x7f80u) == 0x7f80u ? __int_as_float(0x7fc00000) : lo * s;
            hi = (u & 0x7f800000u) == 0x7f800000u ? __int_as_float(0x7fc00000) : hi * s;
            c[j] = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
        }
        out[i] = c[0] | (c[1] << 16);
    }
    return make_uint2(out[0], out[1]);
}

// Grid: x = CTAs of a sequence (one cluster), y = sequence.  LPV lanes serve one vector.
template <bool E4M3, int LPV>
__global__ void __launch_bounds__(kPathThreads) sv_kv_path_kernel(PathParams k)
{
    grid_dependency_wait();
    const int b = blockIdx.y;
    const int len = __ldg(&k.cache_len[b]), a = __ldg(&k.nacc[b]);
    int rows = a < 0 ? 0 : k.lead + a, bits = 0;
    if (a >= 0) {
        if (a > k.T - k.lead)
            bits = SV_KV_BAD_COUNT;
        else if (len < 0 || len > k.max_len - rows)
            bits = SV_KV_OVERFLOW;
    }
    __shared__ int32_t src_row[kPathMaxT];  // scratch row of each committed row
    bool bad = false;
    if (!bits)
        for (int i = threadIdx.x; i < rows; i += kPathThreads) {
            int r = i;
            if (i >= k.lead && k.path)
                r = __ldg(&k.path[(size_t)b * k.T + (i - k.lead)]);
            bad |= (unsigned)r >= (unsigned)k.T;
            src_row[i] = r;
        }
    if (__syncthreads_or(bad))
        bits = SV_KV_BAD_PATH;
    if (bits)
        rows = 0;
    // every thread of the cluster has read the old length once this barrier completes
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    const unsigned sub = threadIdx.x % LPV;
    const bool active = (int)sub * 8 < k.D;
    const unsigned nvec = (unsigned)k.P * (unsigned)rows * (unsigned)k.heads;  // below 2^31
    const unsigned per = kPathThreads / LPV * gridDim.x;  // vectors the cluster takes at a time
    const unsigned first = blockIdx.x * (kPathThreads / LPV) + threadIdx.x / LPV;
    const unsigned hr = (unsigned)k.heads * (unsigned)rows;
    bool nonfinite = false;
    for (unsigned v0 = first - threadIdx.x / LPV; v0 < nvec; v0 += per * kPathUnroll) {  // uniform over the CTA
        uint4 x[kPathUnroll];
        size_t dst[kPathUnroll];
#pragma unroll
        for (int j = 0; j < kPathUnroll; ++j) {
            const unsigned v = v0 + threadIdx.x / LPV + j * per;
            x[j] = make_uint4(0, 0, 0, 0);
            if (v < nvec) {
                const unsigned p = v / hr, ih = v - p * hr, i = ih / (unsigned)k.heads, h = ih - i * (unsigned)k.heads;
                const size_t seq = (size_t)p * k.B + b;
                dst[j] = (seq * k.max_len + (size_t)(len + (int)i)) * k.heads + h;
                if (active)
                    x[j] = __ldcs(reinterpret_cast<const uint4 *>(
                        k.rows + ((((seq * k.T + src_row[i]) * k.heads + h) * k.D) + sub * 8) * 2));
            }
        }
#pragma unroll
        for (int j = 0; j < kPathUnroll; ++j) {
            const unsigned v = v0 + threadIdx.x / LPV + j * per;
            if constexpr (E4M3) {
                const unsigned w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                unsigned m = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const unsigned lo = w[q] & 0x7fffu, hi = (w[q] >> 16) & 0x7fffu;
                    nonfinite |= lo >= 0x7f80u || hi >= 0x7f80u;
                    m = max(m, max(lo >= 0x7f80u ? 0u : lo, hi >= 0x7f80u ? 0u : hi));
                }
#pragma unroll
                for (int o = LPV / 2; o >= 1; o >>= 1)
                    m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                const int e = scale_exponent(m);
                if (v < nvec) {
                    if (active)
                        *reinterpret_cast<uint2 *>(k.cache + dst[j] * k.D + sub * 8) = quantise8(w, pow2i(-e));
                    if (sub == 0)
                        k.scale[dst[j]] = (uint8_t)(e + 127);
                }
            } else if (v < nvec && active) {
                *reinterpret_cast<uint4 *>(k.cache + (dst[j] * k.D + sub * 8) * 2) = x[j];
            }
        }
    }
    if (nonfinite && k.status)
        atomicOr(k.status, SV_KV_NONFINITE);
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        k.out_len[b] = len + rows;
        if (bits && k.status)
            atomicOr(k.status, bits);
    }
}

struct ReadParams {
    const unsigned char *cache;
    const uint8_t *scale;
    const int32_t *cache_len, *start;
    unsigned char *out;
    int32_t *status;
    int P, B, n, max_len, heads, D;
};

// Two codes (the low 16 bits) times s as two bf16.
__device__ __forceinline__ unsigned dequant2(unsigned short c, float s)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * s, f.y * s);
    return *reinterpret_cast<const unsigned *>(&r);
}

// Grid: x = blocks of 16-code chunks of one sequence in one plane, y = sequence, z = plane.
__global__ void __launch_bounds__(kReadThreads) sv_kv_read_kernel(ReadParams k)
{
    grid_dependency_wait();
    const unsigned long long chunk0 = (unsigned long long)blockIdx.x * (kReadThreads * kReadUnroll) + threadIdx.x;
    const unsigned cpv = (unsigned)k.D / 16u;  // chunks of a (row, head) vector
    for (int b = blockIdx.y; b < k.B; b += gridDim.y) {
        const int len = __ldg(&k.cache_len[b]), st = k.start ? __ldg(&k.start[b]) : 0;
        if (len < 0 || len > k.max_len || st < 0) {
            if (k.status && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.z == 0)
                atomicOr(k.status, SV_KV_OVERFLOW);
            continue;
        }
        const long long rows = min((long long)len - st, (long long)k.n);
        if (rows <= 0)
            continue;
        const unsigned long long total = (unsigned long long)rows * k.heads * cpv;
        for (int p = blockIdx.z; p < k.P; p += gridDim.z) {
            const size_t seq = (size_t)p * k.B + b;
            const size_t v_in = (seq * k.max_len + st) * k.heads, v_out = seq * k.n * k.heads;
            const uint4 *src = reinterpret_cast<const uint4 *>(k.cache + v_in * k.D);
            uint4 *dst = reinterpret_cast<uint4 *>(k.out + v_out * k.D * 2);
            uint4 x[kReadUnroll];
            uint8_t s[kReadUnroll];
#pragma unroll
            for (int j = 0; j < kReadUnroll; ++j) {
                const unsigned long long c = chunk0 + j * kReadThreads;
                if (c < total) {
                    x[j] = __ldcs(src + c);
                    s[j] = __ldg(k.scale + v_in + c / cpv);
                }
            }
#pragma unroll
            for (int j = 0; j < kReadUnroll; ++j) {
                const unsigned long long c = chunk0 + j * kReadThreads;
                if (c < total) {
                    const unsigned w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                    unsigned o[8];
                    // a scale byte of 0 or 255 is never written by the commit; 0 reads as 2^-127
                    const float f = s[j] ? __int_as_float((int)s[j] << 23) : __int_as_float(0x00400000);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        o[2 * q] = dequant2((unsigned short)(w[q] & 0xffffu), f);
                        o[2 * q + 1] = dequant2((unsigned short)(w[q] >> 16), f);
                    }
                    __stcs(dst + 2 * c, make_uint4(o[0], o[1], o[2], o[3]));
                    __stcs(dst + 2 * c + 1, make_uint4(o[4], o[5], o[6], o[7]));
                }
            }
        }
    }
}

bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// planes * B * rows * heads * D * 2 fits in 62 bits
bool fits(int planes, int B, long long rows, int heads, int D)
{
    const unsigned long long a = (unsigned long long)planes * (unsigned long long)B;
    const unsigned long long c = (unsigned long long)heads * (unsigned long long)D * 2ull;
    return rows == 0 || a == 0 || a <= (1ull << 62) / c / (unsigned long long)rows;
}

template <bool E4M3, int LPV> cudaError_t launch_path(const cudaLaunchConfig_t &cfg, const PathParams &k)
{
    return cudaLaunchKernelEx(&cfg, sv_kv_path_kernel<E4M3, LPV>, k);
}

template <bool E4M3> cudaError_t launch_path(const cudaLaunchConfig_t &cfg, const PathParams &k)
{
    const int lanes = k.D / 8;
    return lanes <= 2 ? launch_path<E4M3, 2>(cfg, k)
         : lanes <= 4 ? launch_path<E4M3, 4>(cfg, k)
         : lanes <= 8 ? launch_path<E4M3, 8>(cfg, k)
         : lanes <= 16 ? launch_path<E4M3, 16>(cfg, k)
                       : launch_path<E4M3, 32>(cfg, k);
}

} // namespace

extern "C" sv_status spec_verify_kv_commit_path(const void *rows, void *cache, uint8_t *scale,
                                                const int32_t *cache_len, int32_t *out_len,
                                                const int32_t *num_accepted, const int32_t *path, int32_t *status,
                                                int planes, int B, int T, int lead, int max_len, int heads,
                                                int head_dim, sv_kv_format format, void *stream)
{
    if (planes < 1 || B < 0 || T < 0 || lead < 0 || lead > T || max_len < 0 || heads < 1 || head_dim < 16 ||
        head_dim > 256 || head_dim % 16 != 0)
        return SV_ERR_INVALID_ARG;
    if (format != SV_KV_BF16 && format != SV_KV_E4M3)
        return SV_ERR_DTYPE;
    if (B == 0)
        return SV_OK;
    if (!cache_len || !out_len || !num_accepted || (T > 0 && (!rows || !cache)) ||
        (T > 0 && format == SV_KV_E4M3 && !scale))
        return SV_ERR_INVALID_ARG;
    if (!aligned16(rows) || !aligned16(cache))
        return SV_ERR_INVALID_ARG;
    if (B > 65535 || T > kPathMaxT || !fits(planes, B, T > max_len ? T : max_len, heads, head_dim) ||
        (long long)planes * T > INT_MAX / 64 / heads)
        return SV_ERR_TOO_LARGE;
    PathParams k = {static_cast<const unsigned char *>(rows), static_cast<unsigned char *>(cache), scale, cache_len,
                    out_len, num_accepted, path, status, planes, B, T, lead, max_len, heads, head_dim};
    // CTAs of a sequence: enough that the batch covers the SMs twice, none without a round of vectors
    int cs = 8;
    while (cs > 1 && ((long long)B * cs > 1216 || (long long)planes * T * heads * head_dim <= (long long)(cs / 2) * kPathThreads * 8))
        cs >>= 1;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cs, (unsigned)B);
    cfg.blockDim = dim3(kPathThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if ((format == SV_KV_E4M3 ? launch_path<true>(cfg, k) : launch_path<false>(cfg, k)) != cudaSuccess) {
        cudaGetLastError();
        return SV_ERR_CUDA;
    }
    return SV_OK;
}

extern "C" sv_status spec_verify_kv_read(const void *cache, const uint8_t *scale, const int32_t *cache_len,
                                         const int32_t *start, void *out, int32_t *status, int planes, int B, int n,
                                         int max_len, int heads, int head_dim, void *stream)
{
    if (planes < 1 || B < 0 || n < 0 || max_len < 0 || heads < 1 || head_dim < 16 || head_dim > 256 ||
        head_dim % 16 != 0)
        return SV_ERR_INVALID_ARG;
    if (B == 0 || n == 0)
        return SV_OK;
    if (!cache_len || !out || (max_len > 0 && (!cache || !scale)) || !aligned16(cache) || !aligned16(out))
        return SV_ERR_INVALID_ARG;
    if (B > 65535 || !fits(planes, B, n > max_len ? n : max_len, heads, head_dim))
        return SV_ERR_TOO_LARGE;
    const unsigned long long chunks = (unsigned long long)(n < max_len ? n : max_len) * heads * (head_dim / 16);
    const unsigned long long nx = (chunks + kReadThreads * kReadUnroll - 1) / (kReadThreads * kReadUnroll);
    if (nx > (unsigned long long)INT_MAX)
        return SV_ERR_TOO_LARGE;
    ReadParams k = {static_cast<const unsigned char *>(cache), scale, cache_len, start,
                    static_cast<unsigned char *>(out), status, planes, B, n, max_len, heads, head_dim};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(nx ? (unsigned)nx : 1u, (unsigned)B, (unsigned)(planes < 65535 ? planes : 65535));
    cfg.blockDim = dim3(kReadThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, sv_kv_read_kernel, k) != cudaSuccess) {
        cudaGetLastError();
        return SV_ERR_CUDA;
    }
    return SV_OK;
}
