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

// One sequence: its rows (token, head of a group) lie in `tiles` row tiles; an
// item is one of them with one key/value head.
struct SeqShape {
    int n, len;  // new tokens, and all of them
    int keys;    // of which the table has the pages
    int rows, tiles;
};

__device__ __forceinline__ SeqShape seq_shape(const AttnParams &p, int b)
{
    const KvView &c = p.c;
    SeqShape s;
    const int begin = c.cu[b], end = c.cu[b + 1];
    s.n = begin >= 0 && end > begin && end <= p.tokens ? end - begin : 0;
    s.len = max(0, c.lens[b]);
    s.keys = min(s.len, c.table_width << c.page_shift);
    s.rows = (int)min((int64_t)s.n * p.group, (int64_t)INT32_MAX);
    const bool mine = s.rows >= p.rows_from && s.rows <= p.rows_to;
    s.tiles = mine ? (s.rows + p.tile_rows - 1) / p.tile_rows : 0;
    return s;
}

// Keys that the rows of tile r see (its last row sees the most).
__device__ __forceinline__ int tile_keys(const AttnParams &p, const SeqShape &s, int r)
{
    if (!p.causal)
        return s.keys;
    const int last = (int)min((int64_t)(r + 1) * p.tile_rows, (int64_t)s.rows) - 1;
    return max(0, min(s.keys, s.len - s.n + last / p.group + 1));
}

// Units of tile r: at least one, so that rows without keys are written too.
__device__ __forceinline__ int tile_units(const AttnParams &p, const SeqShape &s, int r)
{
    return max(1, (tile_keys(p, s, r) + p.unit - 1) / p.unit);
}

__device__ __forceinline__ int64_t head_units(const AttnParams &p, const SeqShape &s)
{
    int64_t n = 0;
    for (int r = 0; r < s.tiles; ++r)
        n += tile_units(p, s, r);
    return n;
}

__device__ __forceinline__ int64_t seq_units(const AttnParams &p, int b)
{
    const SeqShape s = seq_shape(p, b);
    if (s.tiles && s.len > s.keys)
        atomicOr(p.c.status, LLMINT8_DEV_BAD_PAGE);
    return head_units(p, s) * p.c.heads;
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

// Keys [t0, t1), units [c0, c1) of an item: sequence b, head h, row tile r.
struct Seg {
    int b, h, r;
    int row0, rows;        // rows of the tile, of n * group
    int n, len, keys;      // of the sequence
    int t0, t1;
    int c0, c1, chunks;    // of the item's units
};

// The segments of units [u, u1), one after the other.
struct Walk {
    int64_t u, u1;
    int b, h, r, c, chunks;
    SeqShape s;

    __device__ __forceinline__ void start(const AttnParams &p, const Range &range)
    {
        u = range.u0;
        u1 = range.u1;
        b = range.b;
        s = seq_shape(p, b);
        const int64_t per = head_units(p, s);
        h = (int)(range.off / per);
        int64_t off = range.off - h * per;
        r = 0;
        for (;; ++r) {
            chunks = tile_units(p, s, r);
            if (off < chunks)
                break;
            off -= chunks;
        }
        c = (int)off;
    }
    __device__ __forceinline__ bool next(const AttnParams &p, Seg &g)
    {
        if (u >= u1)
            return false;
        if (c == chunks) {
            c = 0;
            if (++r == s.tiles) {
                r = 0;
                if (++h == p.c.heads) {
                    h = 0;
                    do { // there is one more: u < u1
                        ++b;
                        s = seq_shape(p, b);
                    } while (s.tiles == 0);
                }
            }
            chunks = tile_units(p, s, r);
        }
        g.b = b;
        g.h = h;
        g.r = r;
        g.row0 = r * p.tile_rows;
        g.rows = min(p.tile_rows, s.rows - g.row0);
        g.n = s.n;
        g.len = s.len;
        g.keys = s.keys;
        g.chunks = chunks;
        g.c0 = c;
        g.c1 = (int)min((int64_t)chunks, c + (u1 - u));
        const int keys = tile_keys(p, s, r);
        g.t0 = min(g.c0 * p.unit, keys);
        g.t1 = min(g.c1 * p.unit, keys);
        u += g.c1 - c;
        c = g.c1;
        return true;
    }
};

// The keys and values of a warp's walk, for the warp that loads them: lane j
// (of 16) looks after 16-key group j % 8 of each unit, its keys for j < 8 and
// its values for the others. Page numbers are requested two units ahead and
// scales one, so that no lookup is waited for.
struct UnitLoad {
    bool some, want; // there is a unit; this lane's group has keys in it
    bool first;      // of its segment
    int page;        // -1: none
    int h, slot;
    float scale;
};

struct LoadWalk {
    Walk walk;
    Seg q;
    int c;
    bool more, bad;

    __device__ __forceinline__ void start(const AttnParams &p, const Range &range)
    {
        walk.start(p, range);
        more = walk.next(p, q);
        c = q.c0;
        bad = false;
    }
    __device__ __forceinline__ void fetch(const AttnParams &p, UnitLoad &u)
    {
        const KvView &kv = p.c;
        const int lane = threadIdx.x & 31;
        if (more && c == q.c1) {
            more = walk.next(p, q);
            c = q.c0;
        }
        u.some = more;
        u.page = -1;
        u.want = false;
        if (!more)
            return;
        const int key = c * p.unit + (lane & 7) * 16;
        u.want = lane < 16 && key < q.t1;
        u.first = c == q.c0;
        const int j = key >> kv.page_shift;
        if (u.want && j < kv.table_width)
            u.page = kv.table[q.b * kv.table_stride + j];
        u.h = q.h;
        u.slot = key & (kv.page_size - 1);
        ++c;
    }
    __device__ __forceinline__ void scale(const AttnParams &p, UnitLoad &u)
    {
        const KvView &kv = p.c;
        if (u.want && (unsigned)u.page >= (unsigned)kv.pages) {
            bad = true;
            u.page = -1;
        }
        u.scale = u.page >= 0 ? __ldcg(((threadIdx.x & 31) >= 8 ? kv.va : kv.ka) + (u.page * kv.heads + u.h)) : 0.f;
    }
};

// What the scores need of a 16-key group, by its two lanes: the keys' scale in
// log2 units, log2 of the values' scale and its inverse, over what the weights
// start at. A group without a page weighs nothing: scale 0, weight 2^-inf.
__device__ __forceinline__ void store_meta(float *meta, const UnitLoad &u, float scale_log2, float start)
{
    const int lane = threadIdx.x & 31;
    if (lane < 8) {
        meta[0] = u.scale * (1.0f / 127.0f) * scale_log2;
    } else if (lane < 16) {
        const float vs = fmaxf(u.scale * (1.0f / 127.0f), 1e-30f);
        meta[1] = u.page >= 0 ? log2f(vs) : -INFINITY;
        meta[2] = u.page >= 0 ? 1.0f / vs / start : 0.f;
    }
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// A warpgroup's share of the registers that the block was launched with.
template <int N>
__device__ __forceinline__ void regs_more()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void regs_less()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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

// bf16 query values of a row that LANES neighbouring lanes share, N words each,
// as fp16: scaled by a power of two that puts the largest
// below 2^14, so that bf16's 8 significant bits survive down to 2^-30 of it.
// Returns the factor that undoes the scaling.
template <int LANES, int N>
__device__ __forceinline__ float bf16_to_f16(uint32_t (&w)[N])
{
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 f = up2<true>(w[i]);
        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
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

// One part of a split item (its maximum, sum of weights, weighted values) onto
// the parts before it.
__device__ __forceinline__ void add_part(float &M, float &l, float4 &acc, float2 ml, float4 v)
{
    const float mn = fmaxf(M, ml.x), mu = mn == -INFINITY ? 0.f : mn;
    const float fa = exp2_approx(M - mu), fb = exp2_approx(ml.x - mu);
    M = mn;
    l = fmaf(l, fa, ml.y * fb);
    acc.x = fmaf(acc.x, fa, v.x * fb);
    acc.y = fmaf(acc.y, fa, v.y * fb);
    acc.z = fmaf(acc.z, fa, v.z * fb);
    acc.w = fmaf(acc.w, fa, v.w * fb);
}

// Four output values of row R (token R / group, head h * group + R % group) of
// a sequence whose rows start at out_row / heads, and its lse. The values are
// weighted with what the weights start at, their sum l is not.
template <int D>
__device__ __forceinline__ void finish_row(const AttnParams &p, int64_t out_row, int h, int R, int chunk, float4 acc,
                                           float M, float l, float start)
{
    const int tok = R / p.group, head = h * p.group + (R - tok * p.group);
    const int64_t row = out_row + (int64_t)tok * p.heads + head;
    const float inv = l > 0.f ? 1.0f / l / start : 0.f;
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

cudaError_t launch_attn_prefill(AttnParams p, const llmint8_kv_cache &c, const DeviceInfo &dev, cudaStream_t stream);
cudaError_t launch_attn_decode(AttnParams p, const llmint8_kv_cache &c, bool r8, const DeviceInfo &dev,
                               cudaStream_t stream);

} // namespace llmint8
