// Residual addition, root-mean-square norm and row-wise int8 quantization
// before an LLM.int8() linear, and the recovery of values from row codes.
//
//   h = x + residual, rounded to the input type (the new residual stream)
//   y = fp16(h * rstd * w),  rstd = 1 / sqrt(mean(h^2) + eps) in fp32
//   codes, row absmax, outlier bitmap of y: as llmint8_quantize_rowwise gives
//   them for the stored y (page "Hugging Face 将 LLM.int8() 8-bit 量化集成进
//   transformers 与 accelerate", sections "模型量化简介" and "MatMul 内部")
//
// Bound by HBM: per element two 2-byte reads, a 2-byte h, a 2-byte y and a
// 1-byte code written.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "llmint8.h"

namespace llmint8 {
namespace {

constexpr int kVec = 4;             // 16-byte vectors a thread holds of its row
constexpr int kMaxRowThreads = 1024; // so rows of up to 32768 columns stay in registers

// h = x + residual in fp32, rounded once.
template <bool BF16>
__device__ __forceinline__ uint4 add8(const uint4 &x, const uint4 &r)
{
    const uint32_t *a = reinterpret_cast<const uint32_t *>(&x), *b = reinterpret_cast<const uint32_t *>(&r);
    uint4 o;
    uint32_t *p = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = up2<BF16>(a[i]), v = up2<BF16>(b[i]);
        p[i] = down2<BF16>(u.x + v.x, u.y + v.y);
    }
    return o;
}

template <bool BF16>
__device__ __forceinline__ float squares8(const uint4 &h)
{
    const uint32_t *a = reinterpret_cast<const uint32_t *>(&h);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = up2<BF16>(a[i]);
        s0 = fmaf(u.x, u.x, s0);
        s1 = fmaf(u.y, u.y, s1);
    }
    return s0 + s1;
}

// y = fp16(h * w * rstd). The product of two 16-bit values is exact in fp32
// (at most 22 significant bits), so y is off by rstd's rounding and one more.
template <bool BF16>
__device__ __forceinline__ uint4 norm8(const uint4 &h, const uint4 &w, float rstd)
{
    const uint32_t *a = reinterpret_cast<const uint32_t *>(&h), *b = reinterpret_cast<const uint32_t *>(&w);
    uint4 o;
    uint32_t *p = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = up2<BF16>(a[i]), v = up2<BF16>(b[i]);
        p[i] = down2<false>(u.x * v.x * rstd, u.y * v.y * rstd);
    }
    return o;
}

template <bool MAX>
__device__ __forceinline__ float warp_all(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    return v;
}

// Sum or maximum over the CTA, the same value in every thread. `s` holds one
// float a warp; two buffers used in turn need no barrier between uses.
template <bool MAX>
__device__ __forceinline__ float block_all(float v, float *s, int nwarps)
{
    v = warp_all<MAX>(v);
    if (nwarps == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        s[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = lane < nwarps ? s[lane] : 0.f; // squares and magnitudes: 0 changes neither
    return warp_all<MAX>(v);
}

struct NormParams {
    const uint4 *x, *res, *w;
    uint4 *h, *y; // null: not stored
    uint2 *codes;
    float *absmax;
    int64_t rows;
    int cols;
    float eps;
    __half t16;
    uint32_t *sets, *calls, *ticket, *bitmap_out;
    int alone; // one row: its own outlier columns are all there are
};

// One CTA per row, the row in registers from its one read to its codes. With
// THR a row is coded against the outlier columns it has itself; what other
// rows add to the set is put right by k_norm_fix.
template <bool BF16, bool THR>
__global__ void __launch_bounds__(kMaxRowThreads) k_norm_quant(const NormParams p)
{
    __shared__ float s_red[2][32];
    const int tid = threadIdx.x, nwarps = blockDim.x >> 5;
    const int nvec = p.cols >> 3;
    griddep_wait();
    griddep_release();
    uint32_t *set = nullptr;
    if (THR)
        set = p.sets + (*reinterpret_cast<volatile uint32_t *>(p.calls) & 1u) * kSetWords;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const uint4 *xr = p.x + r * nvec;
        uint4 v[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = tid + i * blockDim.x;
            v[i] = c < nvec ? __ldcs(xr + c) : make_uint4(0, 0, 0, 0);
        }
        if (p.res) {
            const uint4 *rr = p.res + r * nvec;
            uint4 u[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int c = tid + i * blockDim.x;
                u[i] = c < nvec ? __ldcs(rr + c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                v[i] = add8<BF16>(v[i], u[i]);
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = tid + i * blockDim.x;
            if (p.h && c < nvec)
                p.h[r * nvec + c] = v[i];
            ss += squares8<BF16>(v[i]);
        }
        ss = block_all<false>(ss, s_red[0], nwarps);
        const float rstd = 1.0f / sqrtf(ss / (float)p.cols + p.eps);
        float amax = 0.f;
        __half2 m2 = __float2half2_rn(0.f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = tid + i * blockDim.x;
            if (c < nvec) {
                v[i] = norm8<BF16>(v[i], __ldg(p.w + c), rstd);
                if (p.y)
                    p.y[r * nvec + c] = v[i];
                __half2 a[4];
                __half2 m = vec_abs_max(v[i], a);
                if (THR && __hge(__hmax(__low2half(m), __high2half(m)), p.t16)) {
                    const uint32_t hit = hit_mask8(v[i], p.t16);
                    const uint32_t bits = hit << ((c & 3) * 8);
                    if ((__ldcg(set + (c >> 2)) & bits) != bits)
                        atomicOr(set + (c >> 2), bits);
                    mask_known(v[i], hit);
                    m = vec_abs_max(v[i], a);
                }
                m2 = __hmax2(m2, m);
            }
        }
        amax = block_all<true>(fmaxf(__low2float(m2), __high2float(m2)), s_red[1], nwarps);
        const float s = amax > 0.f ? __fdiv_rn(127.0f, amax) : 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = tid + i * blockDim.x;
            if (c < nvec)
                p.codes[r * nvec + c] = codes8(v[i], s);
        }
        if (tid == 0)
            p.absmax[r] = amax;
    }
}

// Rows wider than the registers hold: the same steps, each pass reading h (or
// x) again.
template <bool BF16, bool THR>
__global__ void __launch_bounds__(kMaxRowThreads) k_norm_quant_wide(const NormParams p)
{
    __shared__ float s_red[2][32];
    const int tid = threadIdx.x, nwarps = blockDim.x >> 5;
    const int nvec = p.cols >> 3;
    griddep_wait();
    griddep_release();
    uint32_t *set = nullptr;
    if (THR)
        set = p.sets + (*reinterpret_cast<volatile uint32_t *>(p.calls) & 1u) * kSetWords;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        float ss = 0.f;
        auto hidden = [&](int c) {
            uint4 v = p.x[r * nvec + c];
            if (p.res)
                v = add8<BF16>(v, p.res[r * nvec + c]);
            return v;
        };
        for (int c = tid; c < nvec; c += blockDim.x)
            ss += squares8<BF16>(hidden(c));
        ss = block_all<false>(ss, s_red[0], nwarps);
        const float rstd = 1.0f / sqrtf(ss / (float)p.cols + p.eps);
        __half2 m2 = __float2half2_rn(0.f);
        for (int c = tid; c < nvec; c += blockDim.x) {
            uint4 v = norm8<BF16>(hidden(c), __ldg(p.w + c), rstd);
            __half2 a[4];
            if (THR) {
                const uint32_t hit = hit_mask8(v, p.t16);
                if (hit) {
                    atomicOr(set + (c >> 2), hit << ((c & 3) * 8));
                    mask_known(v, hit);
                }
            }
            m2 = __hmax2(m2, vec_abs_max(v, a));
        }
        const float amax = block_all<true>(fmaxf(__low2float(m2), __high2float(m2)), s_red[1], nwarps);
        const float s = amax > 0.f ? __fdiv_rn(127.0f, amax) : 0.f;
        // h may take the place of x or the residual: it is stored last, each
        // vector by the thread that read it.
        for (int c = tid; c < nvec; c += blockDim.x) {
            const uint4 h = hidden(c);
            uint4 v = norm8<BF16>(h, __ldg(p.w + c), rstd);
            if (p.h)
                p.h[r * nvec + c] = h;
            if (p.y)
                p.y[r * nvec + c] = v;
            if (THR)
                mask_known(v, hit_mask8(v, p.t16));
            p.codes[r * nvec + c] = codes8(v, s);
        }
        if (tid == 0)
            p.absmax[r] = amax;
    }
}

// After every row has added its outlier columns to the set: the columns of
// the set get code 0 in every row, and a row whose absmax is attained in one
// of them is coded again. All other codes stand: a row's absmax and codes
// depend on the set only through those columns. The last CTA to finish moves
// the call counter on, so that the next call finds the other set, cleared
// here, and the counter untouched until everyone has read it.
__global__ void __launch_bounds__(256) k_norm_fix(const NormParams p)
{
    extern __shared__ uint32_t s_dyn[];
    const int nwords = (p.cols + 31) >> 5, nvec = p.cols >> 3;
    uint32_t *s_set = s_dyn;
    int *s_col = reinterpret_cast<int *>(s_dyn + nwords); // the first kListed columns
    constexpr int kListed = 1024;
    __shared__ int s_count;
    const int tid = threadIdx.x, lane = tid & 31;
    griddep_wait();
    griddep_release();
    const uint32_t call = *reinterpret_cast<volatile uint32_t *>(p.calls);
    const uint32_t *set = p.sets + (call & 1u) * kSetWords;
    uint32_t *next = p.sets + ((call + 1u) & 1u) * kSetWords;
    if (tid == 0)
        s_count = 0;
    __syncthreads();
    for (int w = tid; w < nwords; w += blockDim.x) {
        uint32_t v = __ldcg(set + w);
        s_set[w] = v;
        if (blockIdx.x == 0)
            p.bitmap_out[w] = v;
        while (v) {
            const int b = __ffs(v) - 1;
            v &= v - 1u;
            const int at = atomicAdd(&s_count, 1);
            if (at < kListed)
                s_col[at] = w * 32 + b;
        }
    }
    if (blockIdx.x == 0)
        for (int w = tid; w < (int)kSetWords; w += blockDim.x)
            next[w] = 0u;
    __syncthreads();
    const int count = s_count;
    const __half *Y = reinterpret_cast<const __half *>(p.y);
    if (count) {
        const int64_t nw = (int64_t)gridDim.x * (blockDim.x >> 5);
        for (int64_t r = (int64_t)blockIdx.x * (blockDim.x >> 5) + (tid >> 5); r < p.rows; r += nw) {
            const float old = __ldcg(p.absmax + r);
            bool stale = count > kListed;
            if (!stale)
                for (int i = lane; i < count; i += 32) {
                    const int c = s_col[i];
                    const float a = fabsf(__half2float(Y[r * (int64_t)p.cols + c]));
                    if (a < __half2float(p.t16)) {
                        reinterpret_cast<int8_t *>(p.codes)[r * (int64_t)p.cols + c] = 0;
                        stale |= a == old;
                    }
                }
            if (!__any_sync(0xffffffffu, stale))
                continue;
            const uint4 *yr = p.y + r * nvec;
            __half2 m2 = __float2half2_rn(0.f);
            for (int c = lane; c < nvec; c += 32) {
                uint4 v = yr[c];
                mask_known(v, (s_set[c >> 2] >> ((c & 3) * 8)) & 0xFFu);
                __half2 a[4];
                m2 = __hmax2(m2, vec_abs_max(v, a));
            }
            const float amax = warp_all<true>(fmaxf(__low2float(m2), __high2float(m2)));
            const float s = amax > 0.f ? __fdiv_rn(127.0f, amax) : 0.f;
            for (int c = lane; c < nvec; c += 32) {
                uint4 v = yr[c];
                mask_known(v, (s_set[c >> 2] >> ((c & 3) * 8)) & 0xFFu);
                p.codes[r * nvec + c] = codes8(v, s);
            }
            if (lane == 0)
                p.absmax[r] = amax;
        }
    }
    __syncthreads();
    if (tid == 0 && atomicAdd(p.ticket, 1u) == gridDim.x - 1u) {
        *p.ticket = 0u;
        *reinterpret_cast<volatile uint32_t *>(p.calls) = call + 1u;
    }
}

// value = code * (absmax / 127), 16 codes a thread.
template <bool BF16>
__global__ void __launch_bounds__(256) k_dequant_rows(const uint4 *__restrict__ codes,
                                                      const float *__restrict__ absmax, int64_t n16, int row16,
                                                      uint4 *__restrict__ out)
{
    griddep_wait();
    griddep_release();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n16; i += (int64_t)gridDim.x * blockDim.x) {
        const uint4 c = codes[i];
        const float s = __fdiv_rn(absmax[i / row16], 127.0f);
        const int8_t *b = reinterpret_cast<const int8_t *>(&c);
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o[j] = down2<BF16>((float)b[2 * j] * s, (float)b[2 * j + 1] * s);
        out[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
        out[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

} // namespace

cudaError_t launch_norm_quant(const NormArgs &a, const Workspace &ws, const DeviceInfo &dev, cudaStream_t stream)
{
    const bool thr = a.t > 0.f;
    NormParams p{};
    p.x = static_cast<const uint4 *>(a.x);
    p.res = static_cast<const uint4 *>(a.res);
    p.w = static_cast<const uint4 *>(a.w);
    p.h = static_cast<uint4 *>(a.h);
    p.y = static_cast<uint4 *>(a.y);
    p.codes = reinterpret_cast<uint2 *>(a.codes);
    p.absmax = a.absmax;
    p.rows = a.rows;
    p.cols = (int)a.cols;
    p.eps = a.eps;
    p.t16 = threshold_fp16(a.t);
    p.sets = ws.sets;
    p.calls = ws.calls;
    p.ticket = ws.ticket;
    p.bitmap_out = a.bitmap;
    const int nvec = p.cols >> 3;
    const int threads = std::min(kMaxRowThreads, (nvec + 32 * kVec - 1) / (32 * kVec) * 32);
    const bool wide = nvec > kMaxRowThreads * kVec;
    auto kern = wide ? (a.bf16 ? (thr ? k_norm_quant_wide<true, true> : k_norm_quant_wide<true, false>)
                               : (thr ? k_norm_quant_wide<false, true> : k_norm_quant_wide<false, false>))
                     : (a.bf16 ? (thr ? k_norm_quant<true, true> : k_norm_quant<true, false>)
                               : (thr ? k_norm_quant<false, true> : k_norm_quant<false, false>));
    const int64_t grid = std::min<int64_t>(a.rows, (int64_t)dev.num_sms * std::max(1, 2048 / threads));
    cudaError_t e = launch_pdl(kern, dim3((unsigned)grid), threads, 0, stream, p);
    if (e != cudaSuccess || !thr)
        return e;
    const size_t smem = ((size_t)(p.cols + 31) / 32 + 1024) * 4;
    const int64_t fgrid = std::min<int64_t>((a.rows + 7) / 8, (int64_t)dev.num_sms * 8);
    return launch_pdl(k_norm_fix, dim3((unsigned)fgrid), 256, smem, stream, p);
}

cudaError_t launch_dequant_rows(const int8_t *codes, const float *absmax, int64_t rows, int64_t cols, void *out,
                                bool bf16, const DeviceInfo &dev, cudaStream_t stream)
{
    const int64_t n16 = rows * cols / 16;
    const int64_t grid = std::min<int64_t>((n16 + 255) / 256, (int64_t)dev.num_sms * 16);
    return launch_pdl(bf16 ? k_dequant_rows<true> : k_dequant_rows<false>, dim3((unsigned)grid), 256, 0, stream,
                      reinterpret_cast<const uint4 *>(codes), absmax, n16, (int)(cols / 16),
                      static_cast<uint4 *>(out));
}

} // namespace llmint8
