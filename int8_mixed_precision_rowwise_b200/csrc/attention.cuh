// What the kernels of the attention over the int8 key/value cache share: their
// parameters, the even split of all work over the CTAs, and the conversions.
#pragma once

#include <cstdint>

#include "internal.h"
#include "kvcache.cuh"

namespace llmint8 {

struct AttnParams {
    KvView c;
    const void *q;
    int64_t q_token, q_head, tokens;
    int heads, group;
    float scale_log2; // scale * log2(e)
    const float *slopes;
    void *out;
    float *lse;
    int causal, bf16;
    int tile_rows, unit;  // rows of a row tile, keys of a work unit
    int rows_from, rows_to; // sequences with so many rows (tokens x group) are this launch's
    float *slots;         // parked parts of split items
    uint32_t *arrived;    // arrivals per split item, 0 between calls
};

// One sequence's share of the work: tiles * chunks units per key/value head.
struct SeqShape {
    int n, len;  // new tokens, and all of them
    int keys;    // of which the table has the pages
    int rows, tiles, chunks;
};

__device__ __forceinline__ SeqShape seq_shape(const AttnParams &p, int b)
{
    const KvView &c = p.c;
    SeqShape s;
    const int begin = __ldg(c.cu + b), end = __ldg(c.cu + b + 1);
    s.n = begin >= 0 && end > begin && end <= p.tokens ? end - begin : 0;
    s.len = max(0, __ldg(c.lens + b));
    s.keys = min(s.len, c.table_width << c.page_shift);
    s.rows = (int)min((int64_t)s.n * p.group, (int64_t)INT32_MAX);
    const bool mine = s.rows >= p.rows_from && s.rows <= p.rows_to;
    s.tiles = mine ? (s.rows + p.tile_rows - 1) / p.tile_rows : 0;
    s.chunks = max(1, (s.keys + p.unit - 1) / p.unit);
    return s;
}

__device__ __forceinline__ int64_t seq_units(const AttnParams &p, int b)
{
    const SeqShape s = seq_shape(p, b);
    if (s.tiles && s.len > s.keys)
        atomicOr(p.c.status, LLMINT8_DEV_BAD_PAGE);
    return (int64_t)s.tiles * s.chunks * p.c.heads;
}

// A CTA's units [u0, u1) of `total`, split evenly over `parts` CTAs; the first
// lies in sequence b, `off` units into it.
struct Range {
    int64_t u0, u1, total, off;
    int b, parts;
};

// Every thread sums the units of a run of sequences, a scan over the threads
// gives the total and the run that the CTA's first unit lies in.
template <int THREADS>
__device__ __forceinline__ Range my_range(const AttnParams &p, void *scratch, int64_t *s_start)
{
    int64_t *s_sum = static_cast<int64_t *>(scratch); // [THREADS / 32]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int batch = p.c.batch;
    const int per = (batch + THREADS - 1) / THREADS;
    const int b0 = min(batch, tid * per), b1 = min(batch, b0 + per);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b)
        sum += seq_units(p, b);
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        s_sum[warp] = incl;
    __syncthreads();
    int64_t base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp)
            base += s_sum[w];
        total += s_sum[w];
    }
    incl += base;
    Range r;
    r.total = total;
    r.parts = (int)min((int64_t)gridDim.x, total);
    r.u0 = r.u1 = 0;
    if ((int)blockIdx.x < r.parts) {
        r.u0 = total * blockIdx.x / r.parts;
        r.u1 = total * (blockIdx.x + 1) / r.parts;
    }
    const int64_t excl = incl - sum;
    if (r.u0 < r.u1 && r.u0 >= excl && r.u0 < incl) {
        int64_t off = r.u0 - excl;
        int b = b0;
        for (;; ++b) {
            const int64_t n = seq_units(p, b);
            if (off < n)
                break;
            off -= n;
        }
        s_start[0] = b;
        s_start[1] = off;
    }
    __syncthreads();
    r.b = (int)s_start[0];
    r.off = s_start[1];
    __syncthreads();
    return r;
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ int warp_min(int v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// fp16 pairs from int8 codes, exactly: a code with its sign bit flipped is
// c + 128, as the low byte of an fp16 in [1024, 2048) it is 1152 + c.
__device__ __forceinline__ uint32_t minus_1152(uint32_t v)
{
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&v), __float2half2_rn(1152.f));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// One word of four codes as two pairs.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &p0, uint32_t &p1)
{
    w ^= 0x80808080u;
    p0 = minus_1152(__byte_perm(w, 0x64646464u, 0x4140));
    p1 = minus_1152(__byte_perm(w, 0x64646464u, 0x4342));
}

// Two words of four codes each (two keys, the same dimensions): for each
// dimension the pair of both keys.
__device__ __forceinline__ void code_pairs_to_f16(uint32_t a, uint32_t b, uint32_t (&out)[4])
{
    const uint32_t x = __byte_perm(a, b, 0x5140) ^ 0x80808080u, y = __byte_perm(a, b, 0x7362) ^ 0x80808080u;
    out[0] = minus_1152(__byte_perm(x, 0x64646464u, 0x4140));
    out[1] = minus_1152(__byte_perm(x, 0x64646464u, 0x4342));
    out[2] = minus_1152(__byte_perm(y, 0x64646464u, 0x4140));
    out[3] = minus_1152(__byte_perm(y, 0x64646464u, 0x4342));
}

// A row of bf16 query values spread over the four lanes of a quad (N words in
// each) as fp16: scaled by a power of two that puts the largest below 2^14, so
// that bf16's 8 significant bits survive down to 2^-38 of it. Returns the
// factor that undoes the scaling (the exponents add up in fp32).
template <int N>
__device__ __forceinline__ float bf16_row_to_f16(uint32_t (&w)[N])
{
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 f = up2<true>(w[i]);
        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^(13 - exponent(top)), kept where both it and its inverse are normal
    int e = 13 - ((int)(__float_as_uint(top) >> 23) - 127);
    e = max(-126, min(126, e));
    const float up = __uint_as_float((uint32_t)(e + 127) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 f = up2<true>(w[i]);
        w[i] = down2<false>(f.x * up, f.y * up);
    }
    return down;
}

// Four output values of row R (token R / group, head h * group + R % group) of
// a sequence whose rows start at out_row / heads, and its lse.
template <int D>
__device__ __forceinline__ void finish_row(const AttnParams &p, int64_t out_row, int h, int R, int chunk, float4 acc,
                                           float M, float l)
{
    const int tok = R / p.group, head = h * p.group + (R - tok * p.group);
    const int64_t row = out_row + (int64_t)tok * p.heads + head;
    const float inv = l > 0.f ? 1.0f / l : 0.f;
    uint2 v;
    if (p.bf16)
        v = make_uint2(down2<true>(acc.x * inv, acc.y * inv), down2<true>(acc.z * inv, acc.w * inv));
    else
        v = make_uint2(down2<false>(acc.x * inv, acc.y * inv), down2<false>(acc.z * inv, acc.w * inv));
    reinterpret_cast<uint2 *>(p.out)[row * (D / 4) + chunk] = v;
    if (p.lse && chunk == 0)
        p.lse[row] = l > 0.f ? (M + log2f(l)) * 0.69314718f : -INFINITY;
}

// Row-major codes [rows x head_dim] as a 2-D TMA map of whole rows, swizzled by
// their width (128 or 64 bytes).
bool encode_map_codes(CUtensorMap *map, const void *base, int64_t rows, int head_dim, int box_rows);

cudaError_t launch_attn_decode(AttnParams p, const llmint8_kv_cache &c, bool r8, const DeviceInfo &dev,
                               cudaStream_t stream);

} // namespace llmint8
