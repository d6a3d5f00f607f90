// Attention of new tokens over the paged int8 key/value cache.
//
//   s_ij = scale * q_i . kc_j * (ka / 127)  [+ slope_h * (j - pos_i)]
//   out_i = sum_j softmax(s_i)_j * vc_j * (va / 127)
//
// over the keys j <= pos_i (causal) or all of the sequence's, with codes kc,
// vc and one absmax ka, va per (page, head).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "kvcache.cuh"

namespace llmint8 {

KvView kv_view(const llmint8_kv_cache &c, uint32_t *status);

namespace {

struct AttnParams {
    KvView c;
    const void *q;
    int64_t q_token, q_head, tokens;
    int heads, group;
    float scale;
    const float *slopes;
    void *out;
    float *lse;
    int causal;
};

// One warp per (new token, head): 32 keys at a time, each lane a key's score,
// then each lane D / 32 of the output's dimensions.
template <bool BF16, int D>
__global__ void __launch_bounds__(128) k_attn_simple(const AttnParams p)
{
    __shared__ float s_q[4][D];
    const KvView &c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + warp;
    if (w >= p.tokens * p.heads)
        return;
    const int64_t t = w / p.heads;
    const int head = (int)(w % p.heads), h = head / p.group;
    const int b = sequence_of(c, t);
    if (b < 0)
        return;
    const int begin = __ldg(c.cu + b), end = __ldg(c.cu + b + 1), len = __ldg(c.lens + b);
    if (t < begin || t >= end)
        return;
    const int64_t pos = (int64_t)len - (end - t);
    const int64_t last = p.causal ? pos : len - 1;
    const uint16_t *q = static_cast<const uint16_t *>(p.q) + t * p.q_token + head * p.q_head;
    for (int d = lane; d < D; d += 32)
        s_q[warp][d] = BF16 ? __uint_as_float((uint32_t)q[d] << 16) : __half2float(reinterpret_cast<const __half *>(q)[d]);
    __syncwarp();
    constexpr int DL = D / 32;
    float o[DL] = {}, m = -INFINITY, l = 0.f;
    const float slope = p.slopes ? p.slopes[head] : 0.f;
    for (int64_t j0 = 0; pos >= 0 && j0 <= last; j0 += 32) {
        const int64_t j = j0 + lane;
        float s = -INFINITY, vs = 0.f;
        int page = -1;
        if (j <= last)
            page = page_of(c, b, (int)j);
        const int64_t block = (int64_t)page * c.heads + h;
        const int64_t at = (block * c.page_size + (j & (c.page_size - 1))) * D;
        if (page >= 0) {
            float dot = 0.f;
            for (int d = 0; d < D; ++d)
                dot = fmaf(s_q[warp][d], (float)c.k[at + d], dot);
            s = dot * (c.ka[block] / 127.0f) * p.scale + slope * (float)(j - pos);
            vs = c.va[block] / 127.0f;
        }
        float top = s;
        for (int x = 16; x; x >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float mn = fmaxf(m, top);
        if (mn == -INFINITY)
            continue;
        const float keep = m == -INFINITY ? 0.f : expf(m - mn);
        const float e = page >= 0 ? expf(s - mn) : 0.f;
        float sum = e;
        for (int x = 16; x; x >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l = l * keep + sum;
        m = mn;
        for (int d = 0; d < DL; ++d)
            o[d] *= keep;
        for (int x = 0; x < 32; ++x) {
            const int pg = __shfl_sync(0xffffffffu, page, x);
            const float wgt = __shfl_sync(0xffffffffu, e * vs, x);
            const int64_t a = __shfl_sync(0xffffffffu, at, x);
            if (pg >= 0)
                for (int d = 0; d < DL; ++d)
                    o[d] = fmaf(wgt, (float)c.v[a + d * 32 + lane], o[d]);
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int d = 0; d < DL; ++d) {
        const int64_t at = w * D + d * 32 + lane;
        if (BF16)
            static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(o[d] * inv);
        else
            static_cast<__half *>(p.out)[at] = __float2half_rn(o[d] * inv);
    }
    if (p.lse && lane == 0)
        p.lse[w] = l > 0.f ? m + logf(l) : -INFINITY;
}

} // namespace

cudaError_t launch_kv_attention(const llmint8_kv_cache &c, const AttnArgs &a, const Workspace &ws, const DeviceInfo &,
                                cudaStream_t stream)
{
    AttnParams p{};
    p.c = kv_view(c, ws.status);
    p.q = a.q;
    p.q_token = a.q_token;
    p.q_head = a.q_head;
    p.tokens = a.tokens;
    p.heads = a.heads;
    p.group = a.heads / c.heads;
    p.scale = a.scale;
    p.slopes = a.slopes;
    p.out = a.out;
    p.lse = a.lse;
    p.causal = a.causal ? 1 : 0;
    auto kern = c.head_dim == 128 ? (a.bf16 ? k_attn_simple<true, 128> : k_attn_simple<false, 128>)
                                  : (a.bf16 ? k_attn_simple<true, 64> : k_attn_simple<false, 64>);
    const int64_t grid = (a.tokens * a.heads + 3) / 4;
    kern<<<(unsigned)grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

} // namespace llmint8
