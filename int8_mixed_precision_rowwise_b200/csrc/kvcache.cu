// Writing tokens to the paged int8 key/value cache and reading them back.
//
// A page holds page_size tokens of every head; each (page, head) has one
// absmax for its keys and one for its values ("absmax quantization", page
// "Hugging Face 将 LLM.int8() 8-bit 量化集成进 transformers 与 accelerate",
// section "模型量化简介", with a block of tokens of one head in the place of a
// row): value = code * (absmax / 127).
//
// Appending to a page that holds earlier tokens keeps their scale unless a
// new value exceeds it: S = max(old absmax, max |new|), earlier codes become
// rint(code * (old / S)), new ones rint(x * (127 / S)), all in fp32.
//
// Both directions are bound by HBM: 2 bytes in and 1 out per value written,
// 1 in and 2 out per value read.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "attention.cuh"
#include "common.cuh"
#include "internal.h"
#include "kvcache.cuh"

namespace llmint8 {
namespace {

// Below this absmax 127 / absmax is not finite in fp32: the block's codes are 0.
constexpr float kTinyAbsmax = 4e-37f;

template <bool BF16>
__device__ __forceinline__ float amax8(const uint4 &v)
{
    const uint32_t *a = reinterpret_cast<const uint32_t *>(&v);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = up2<BF16>(a[i]);
        m = fmaxf(m, fmaxf(fabsf(u.x), fabsf(u.y)));
    }
    return m;
}

template <bool BF16>
__device__ __forceinline__ uint2 kv_codes8(const uint4 &v, float s)
{
    const uint32_t *a = reinterpret_cast<const uint32_t *>(&v);
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = up2<BF16>(a[i]);
        b[2 * i] = __float_as_uint(__fadd_rn(__fmul_rn(f.x, s), 12582912.0f));
        b[2 * i + 1] = __float_as_uint(__fadd_rn(__fmul_rn(f.y, s), 12582912.0f));
    }
    return make_uint2(pack4(b[0], b[1], b[2], b[3]), pack4(b[4], b[5], b[6], b[7]));
}

struct AppendParams {
    KvView c;
    const uint4 *src[2];
    int64_t token[2], head[2]; // strides in 16-byte vectors
    int64_t tokens;
};

constexpr int kWindow = 16; // packed tokens a CTA looks at

// A warp takes one (page, head) of the keys or the values: the run of new
// tokens that starts at a page's first slot or at the sequence's first new
// token. A CTA covers the runs that start in kWindow packed tokens.
template <bool BF16, int D>
__global__ void __launch_bounds__(128) k_kv_append(const AppendParams p)
{
    constexpr int kLanes = D / 8;        // lanes a token's row takes
    constexpr int kRows = 32 / kLanes;   // rows a warp reads at once
    const KvView &c = p.c;
    const int h = blockIdx.y, kv = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = lane / kLanes, vec = lane % kLanes;
    griddep_wait();
    griddep_release();
    const uint4 *src = p.src[kv] + (int64_t)h * p.head[kv] + vec;
    for (int i = warp; i < kWindow; i += 4) {
        const int64_t t = (int64_t)blockIdx.x * kWindow + i;
        if (t >= p.tokens)
            break;
        const int b = sequence_of(c, t);
        if (b < 0)
            continue;
        const int begin = __ldg(c.cu + b), end = __ldg(c.cu + b + 1);
        if (t < begin || t >= end)
            continue; // offsets that decrease
        const int64_t pos64 = (int64_t)__ldg(c.lens + b) - (end - t);
        if (pos64 < 0)
            continue;
        const int pos = (int)pos64;
        const int slot = pos & (c.page_size - 1);
        if (t != begin && slot != 0)
            continue;
        const int page = page_of(c, b, pos);
        if (page < 0)
            continue;
        const int n = (int)min((int64_t)min(c.page_size - slot, end - (int)t), p.tokens - t);
        float amax = 0.f;
        for (int r = row; r < n; r += kRows)
            amax = fmaxf(amax, amax8<BF16>(__ldg(src + (t + r) * p.token[kv])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int64_t block = (int64_t)page * c.heads + h;
        float *scale = (kv ? c.va : c.ka) + block;
        int8_t *dst = (kv ? c.v : c.k) + block * c.page_size * D;
        const float old = slot ? *scale : 0.f;
        if (old > amax)
            amax = old;
        if (slot && old < amax) {
            const float ratio = __fdiv_rn(old, amax);
            for (int j = lane; j < slot * (D / 16); j += 32) {
                uint4 v = reinterpret_cast<uint4 *>(dst)[j];
                int8_t *e = reinterpret_cast<int8_t *>(&v);
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    e[k] = (int8_t)__float2int_rn((float)e[k] * ratio);
                reinterpret_cast<uint4 *>(dst)[j] = v;
            }
        }
        const float s = amax > kTinyAbsmax ? __fdiv_rn(127.0f, amax) : 0.f;
        for (int r = row; r < n; r += kRows)
            *reinterpret_cast<uint2 *>(dst + (slot + r) * D + vec * 8) =
                kv_codes8<BF16>(__ldg(src + (t + r) * p.token[kv]), s);
        __syncwarp();
        if (lane == 0)
            *scale = amax;
    }
}

// 16 codes a thread.
template <bool BF16>
__global__ void __launch_bounds__(256) k_kv_read(const KvView c, uint4 *k_out, uint4 *v_out, int64_t tokens, int d16)
{
    griddep_wait();
    griddep_release();
    const int64_t per = (int64_t)c.heads * d16;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < tokens * per;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = i / per;
        const int e = (int)(i - t * per), h = e / d16, x = e - h * d16;
        const int b = sequence_of(c, t);
        if (b < 0)
            continue;
        const int begin = __ldg(c.cu + b), end = __ldg(c.cu + b + 1);
        const int64_t pos = (int64_t)__ldg(c.lens + b) - (end - t);
        if (t < begin || t >= end || pos < 0)
            continue;
        const int page = page_of(c, b, (int)pos);
        if (page < 0)
            continue;
        const int64_t block = (int64_t)page * c.heads + h;
        const int64_t at = (block * c.page_size + (pos & (c.page_size - 1))) * d16 + x;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            uint4 *out = kv ? v_out : k_out;
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(kv ? c.v : c.k) + at);
            const float s = __fdiv_rn(__ldg((kv ? c.va : c.ka) + block), 127.0f);
            const int8_t *a = reinterpret_cast<const int8_t *>(&v);
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j] = down2<BF16>((float)a[2 * j] * s, (float)a[2 * j + 1] * s);
            out[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
            out[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

} // namespace

KvView kv_view(const llmint8_kv_cache &c, uint32_t *status)
{
    KvView v{};
    v.k = c.k_codes;
    v.v = c.v_codes;
    v.ka = c.k_absmax;
    v.va = c.v_absmax;
    v.pages = (int)c.pages;
    v.heads = c.heads;
    v.page_size = c.page_size;
    while ((1 << v.page_shift) < c.page_size)
        ++v.page_shift;
    v.batch = c.batch;
    v.table_width = c.table_width;
    v.table_stride = c.table_stride;
    v.table = c.page_table;
    v.lens = c.seq_lens;
    v.cu = c.cu_rows;
    v.status = status;
    return v;
}

bool encode_map_codes(CUtensorMap *map, const void *base, int64_t rows, int head_dim, int box_rows)
{
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static std::atomic<Encode> encode{nullptr};
    Encode f = encode.load();
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return false;
        f = reinterpret_cast<Encode>(p);
        encode.store(f);
    }
    cuuint64_t dims[2] = {(cuuint64_t)head_dim, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)head_dim};
    cuuint32_t box[2] = {(cuuint32_t)head_dim, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_kv_append(const llmint8_kv_cache &c, const KvRows &rows, uint32_t *status, const DeviceInfo &,
                             cudaStream_t stream)
{
    AppendParams p{};
    p.c = kv_view(c, status);
    p.src[0] = static_cast<const uint4 *>(rows.k);
    p.src[1] = static_cast<const uint4 *>(rows.v);
    p.token[0] = rows.k_token / 8;
    p.token[1] = rows.v_token / 8;
    p.head[0] = rows.k_head / 8;
    p.head[1] = rows.v_head / 8;
    p.tokens = rows.tokens;
    auto kern = c.head_dim == 128 ? (rows.bf16 ? k_kv_append<true, 128> : k_kv_append<false, 128>)
                                  : (rows.bf16 ? k_kv_append<true, 64> : k_kv_append<false, 64>);
    const dim3 grid((unsigned)((rows.tokens + kWindow - 1) / kWindow), (unsigned)c.heads, 2);
    return launch_pdl(kern, grid, 128, 0, stream, p);
}

cudaError_t launch_kv_read(const llmint8_kv_cache &c, void *k, void *v, int64_t tokens, bool bf16, uint32_t *status,
                           const DeviceInfo &dev, cudaStream_t stream)
{
    const int64_t n = tokens * c.heads * (c.head_dim / 16);
    const int64_t grid = std::min<int64_t>((n + 255) / 256, (int64_t)dev.num_sms * 64);
    return launch_pdl(bf16 ? k_kv_read<true> : k_kv_read<false>, dim3((unsigned)grid), 256, 0, stream,
                      kv_view(c, status), static_cast<uint4 *>(k), static_cast<uint4 *>(v), tokens, c.head_dim / 16);
}

} // namespace llmint8
