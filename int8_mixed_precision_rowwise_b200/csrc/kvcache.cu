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
// 1 in and 2 out per value read. On B200, 2048 tokens of 112 heads of 128 in
// pages of 16: 33 us written, 29 us read, 5.7 TB/s together (a copy: 6.5).
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

// Magnitudes of 16-bit floats are in the order of their bits.
__device__ __forceinline__ uint32_t max_bits8(uint32_t m, const uint4 &v)
{
    m = __vmaxu2(__vmaxu2(m, v.x & 0x7FFF7FFFu), __vmaxu2(v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu));
    return __vmaxu2(m, v.w & 0x7FFF7FFFu);
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
    int window; // packed tokens a CTA takes
};

constexpr int kHeads = 8;   // heads a CTA takes
constexpr int kWindow = 16; // packed tokens a CTA takes

// The places of a CTA's packed tokens [t0, t0 + n): page (-1: none), position
// and the end of the sequence's rows, each found by one lane.
struct Places {
    int page[kWindow], slot[kWindow], begin[kWindow], end[kWindow];
};

__device__ __forceinline__ void find_places(const KvView &c, int64_t t0, int n, int64_t tokens, Places &s)
{
    const int i = threadIdx.x;
    if (i < kWindow) {
        int page = -1, slot = 0, begin = 0, end = 0;
        const int64_t t = t0 + i;
        const int b = i < n && t < tokens ? sequence_of(c, t) : -1;
        if (b >= 0) {
            begin = c.cu[b];
            end = c.cu[b + 1];
            const int64_t pos = (int64_t)c.lens[b] - (end - t);
            if (t >= begin && t < end && pos >= 0) { // offsets that decrease have no rows
                page = page_of(c, b, (int)pos);
                slot = (int)pos & (c.page_size - 1);
            }
        }
        s.page[i] = page;
        s.slot[i] = slot;
        s.begin[i] = begin;
        s.end[i] = end;
    }
    __syncthreads();
}

// A warp takes a (page, head) of the keys or the values: the run of new tokens
// that starts at a page's first slot or at the sequence's first new token. A
// CTA covers the runs that start in its `window` packed tokens, for kHeads
// heads; a run of up to 16 tokens is read once, into registers, a longer one
// (pages of more) a second time, from the caches.
template <bool BF16, int D>
__global__ void __launch_bounds__(kHeads * 32, 4) k_kv_append(const AppendParams p)
{
    constexpr int kLanes = D / 8;      // lanes a token's row takes
    constexpr int kRows = 32 / kLanes; // rows a warp reads at once
    constexpr int kHeld = 16 / kRows;  // vectors of 16 rows in a lane
    __shared__ Places s;
    const KvView &c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y * kHeads + warp, kv = blockIdx.z;
    const int row = lane / kLanes, vec = lane % kLanes;
    const int64_t t0 = (int64_t)blockIdx.x * p.window;
    const int64_t step = p.token[kv];
    const uint4 *src = p.src[kv] + (int64_t)h * p.head[kv] + vec;
    griddep_wait();
    griddep_release();
    // The window's rows on their way while their places are looked up: most of
    // them are this CTA's.
    if (h < c.heads && vec % 8 == 0)
        for (int r = row; r < p.window && t0 + r < p.tokens; r += kRows)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(src + (t0 + r) * step));
    find_places(c, t0, p.window, p.tokens, s);
    if (h >= c.heads)
        return;
    // The window's tokens that start a run.
    const bool starts = lane < p.window && s.page[lane % kWindow] >= 0 &&
                        (s.slot[lane % kWindow] == 0 || t0 + lane == s.begin[lane % kWindow]);
    for (uint32_t runs = __ballot_sync(0xffffffffu, starts); runs; runs &= runs - 1u) {
        const int i = __ffs(runs) - 1, page = s.page[i], slot = s.slot[i];
        const int64_t t = t0 + i;
        const int len = (int)min((int64_t)min(c.page_size - slot, s.end[i] - (int)t), p.tokens - t);
        const int64_t block = (int64_t)page * c.heads + h;
        float *scale = (kv ? c.va : c.ka) + block;
        int8_t *dst = (kv ? c.v : c.k) + block * c.page_size * D;
        const float old = slot ? __ldcg(scale) : 0.f;
        const uint4 *rows = src + t * step;
        uint4 held[kHeld];
        uint32_t bits = 0u;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int r = row + k * kRows;
            held[k] = r < len ? rows[r * step] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            bits = max_bits8(bits, held[k]);
#pragma unroll 8
        for (int r = 16 + row; r < len; r += kRows)
            bits = max_bits8(bits, rows[r * step]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            bits = __vmaxu2(bits, __shfl_xor_sync(0xffffffffu, bits, o));
        const float2 top = up2<BF16>(bits);
        float amax = fmaxf(top.x, top.y);
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
        const float m = amax > kTinyAbsmax ? __fdiv_rn(127.0f, amax) : 0.f;
        uint2 *to = reinterpret_cast<uint2 *>(dst + slot * D + vec * 8);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int r = row + k * kRows;
            if (r < len)
                to[r * (D / 8)] = kv_codes8<BF16>(held[k], m);
        }
        for (int r0 = 16 + row; r0 < len; r0 += 4 * kRows) {
            uint4 u[4]; // all under way before the first is stored
#pragma unroll
            for (int k = 0; k < 4; ++k)
                u[k] = r0 + k * kRows < len ? rows[(r0 + k * kRows) * step] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (r0 + k * kRows < len)
                    to[(r0 + k * kRows) * (D / 8)] = kv_codes8<BF16>(u[k], m);
        }
        __syncwarp();
        if (lane == 0)
            *scale = amax;
    }
}

// kWindow packed tokens of kHeads heads a CTA and turn, 8 codes a thread and
// step: tokens of a page lie one after the other, and whole sectors are stored.
template <bool BF16, int D>
__global__ void __launch_bounds__(256, 4) k_kv_read(const KvView c, uint4 *k_out, uint4 *v_out, int64_t tokens)
{
    constexpr int kPieces = D / 8, kSteps = kHeads * kWindow * kPieces / 256;
    __shared__ Places s;
    const int64_t t0 = (int64_t)blockIdx.x * kWindow;
    griddep_wait();
    griddep_release();
    find_places(c, t0, kWindow, tokens, s);
    // Which piece of which token of each 256 / kPieces is the same in all steps.
    constexpr int kTokens = 256 / kPieces; // a step's (token, head) pairs
    const int x = threadIdx.x % kPieces, pair = threadIdx.x / kPieces;
    for (int h0 = blockIdx.y * kHeads; h0 < c.heads; h0 += gridDim.y * kHeads) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint2 *codes = reinterpret_cast<const uint2 *>(kv ? c.v : c.k);
            const float *absmax = kv ? c.va : c.ka;
            uint4 *out = kv ? v_out : k_out;
            uint2 v[kSteps];
            float f[kSteps];
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int e = pair + i * kTokens, r = e % kWindow, h = h0 + e / kWindow;
                if (s.page[r] >= 0 && h < c.heads) {
                    const int block = s.page[r] * c.heads + h; // fits: pages * heads * page_size < 2^31
                    v[i] = __ldcg(codes + ((int64_t)(block * c.page_size + s.slot[r])) * kPieces + x);
                    f[i] = __ldcg(absmax + block);
                }
            }
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int e = pair + i * kTokens, r = e % kWindow, h = h0 + e / kWindow;
                if (s.page[r] >= 0 && h < c.heads) {
                    const float m = __fdiv_rn(f[i], 127.0f);
                    const uint2 a = code_values4<BF16>(v[i].x, m), b = code_values4<BF16>(v[i].y, m);
                    out[((t0 + r) * c.heads + h) * kPieces + x] = make_uint4(a.x, a.y, b.x, b.y);
                }
            }
        }
    }
}

// CTAs over the heads' groups: enough for two rounds of three an SM; a CTA
// that takes more of them looks its tokens up once.
int head_groups(int64_t windows, int heads, const DeviceInfo &dev)
{
    const int64_t groups = (heads + kHeads - 1) / kHeads;
    return (int)std::max<int64_t>(1, std::min<int64_t>(groups, (6 * dev.num_sms + windows - 1) / windows));
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
    // A step of single tokens has a run in each: one token a CTA, or its warps
    // would take 16 runs one after the other.
    p.window = rows.tokens <= 4 * (int64_t)c.batch ? 1 : kWindow;
    auto kern = c.head_dim == 128 ? (rows.bf16 ? k_kv_append<true, 128> : k_kv_append<false, 128>)
                                  : (rows.bf16 ? k_kv_append<true, 64> : k_kv_append<false, 64>);
    const int64_t windows = (rows.tokens + p.window - 1) / p.window;
    const dim3 grid((unsigned)windows, (unsigned)((c.heads + kHeads - 1) / kHeads), 2);
    return launch_pdl(kern, grid, kHeads * 32, 0, stream, p);
}

cudaError_t launch_kv_read(const llmint8_kv_cache &c, void *k, void *v, int64_t tokens, bool bf16, uint32_t *status,
                           const DeviceInfo &dev, cudaStream_t stream)
{
    auto kern = c.head_dim == 128 ? (bf16 ? k_kv_read<true, 128> : k_kv_read<false, 128>)
                                  : (bf16 ? k_kv_read<true, 64> : k_kv_read<false, 64>);
    const int64_t windows = (tokens + kWindow - 1) / kWindow;
    const dim3 grid((unsigned)windows, (unsigned)head_groups(windows, c.heads, dev));
    return launch_pdl(kern, grid, 256, 0, stream, kv_view(c, status), static_cast<uint4 *>(k), static_cast<uint4 *>(v),
                      tokens);
}

} // namespace llmint8
