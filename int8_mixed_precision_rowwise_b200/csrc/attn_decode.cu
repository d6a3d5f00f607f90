// Attention of few new tokens over the paged int8 key/value cache: a row tile
// of 8 or 16 (token, head) rows that share one key/value head, against that
// head's keys and values. Bound by HBM: every cached byte is read once (per
// row tile) and there are 2 to 64 flops for it.
//
// Mathematics. With codes kc, vc (exact as fp16), page scales ka / 127 and
// va / 127, and everything per key in log2 units:
//   x_j = (q . kc_j) * (ka_j / 127 * scale * log2 e) [+ slope * (j - p) * log2 e]
//   e_j = x_j + log2(va_j / 127),  w_j = 2^(e_j - m),  m the running maximum of e
//   o = sum_j w_j vc_j,  l = sum_j w_j * (127 / va_j),  out = o / l
// The value scale rides on the exponent, so that the weights that enter the
// product are at most 1 (no overflow of fp16) and the codes stay exact.
// q . kc and w . vc run on the tensor cores (fp16 in, fp32 sums). With row
// tiles of 8 the other 8 rows of the m16 tile carry what rounding w to fp16
// left over (w = hi + lo), which the matrix instruction then adds for free;
// with 16 rows the weights are fp16 (off by at most 2^-11 of themselves).
//
// Work. Unit: 128 keys of one (sequence, head, row tile). The units of all of
// them in order are split evenly over the CTAs, whatever the lengths; a CTA
// runs through its units in segments of one item. An item that lies in one
// CTA is finished there; of one that is split every CTA parks its part (o, m,
// l) in the workspace, and the last to arrive adds the parts in order (so the
// result does not depend on the order of arrival).
//
// Each of the four warps takes every fourth 32 keys of a segment and streams
// them through a ring of its own: lane 0 issues the TMA loads of the pages two
// or three steps ahead (page numbers and scales are fetched a step earlier
// still, so that no lane waits for them), the codes land in swizzled shared
// memory, and each lane's 16-byte reads of them are free of bank conflicts and
// already hold what the lane's operand fragments need.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "attention.cuh"

namespace llmint8 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSub = 32;              // keys a warp takes at once
constexpr int kUnit = kSub * kWarps;  // keys of a unit
constexpr int kStages = 3;
constexpr int kMergeRows = 8;

template <int D>
struct Smem {
    static constexpr int kTile = kSub * D;                       // codes of one operand
    static constexpr int kRing = kWarps * kStages * 2 * kTile;
    static constexpr int kMerge = kWarps * kMergeRows * D * 4;
    static constexpr int kMeta = kWarps * kStages * 2 * 2 * 4;   // (key scale, value scale) per 16 keys
    static constexpr int kBars = kWarps * kStages * 8;
    static constexpr int kStats = kWarps * 16 * 2 * 4;
    static constexpr int kTotal = kRing + kMerge + kMeta + kBars + kStats + 64;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

// Keys [t0, t1), chunks [c0, c1) of an item: sequence b, head h, row tile r.
struct Seg {
    int b, h, r;
    int row0, rows;    // rows of the tile, of n * group
    int n, len, keys;  // of the sequence
    int t0, t1;
    int c0, c1, chunks;
};

// The segments of units [u, u1), one after the other.
template <int TR>
struct Walk {
    const AttnParams *p;
    int64_t u, u1;
    int b, h, r, c;
    SeqShape s;

    __device__ __forceinline__ void start(const AttnParams &params, int64_t u0, int64_t end, int b0, int64_t off)
    {
        p = &params;
        u = u0;
        u1 = end;
        b = b0;
        if (u >= u1)
            return;
        s = seq_shape(params, b);
        c = (int)(off % s.chunks);
        off /= s.chunks;
        r = (int)(off % s.tiles);
        h = (int)(off / s.tiles);
    }
    __device__ __forceinline__ bool next(Seg &g)
    {
        if (u >= u1)
            return false;
        if (c == s.chunks) {
            c = 0;
            if (++r == s.tiles) {
                r = 0;
                if (++h == p->c.heads) {
                    h = 0;
                    do {
                        ++b;
                        s = seq_shape(*p, b);
                    } while (s.tiles == 0);
                }
            }
        }
        g.b = b;
        g.h = h;
        g.r = r;
        g.row0 = r * TR;
        g.rows = min(TR, s.rows - g.row0);
        g.n = s.n;
        g.len = s.len;
        g.keys = s.keys;
        g.chunks = s.chunks;
        g.c0 = c;
        g.c1 = (int)min((int64_t)s.chunks, c + (u1 - u));
        int keys = s.keys;
        if (p->causal) // the tile's last row sees the most
            keys = max(0, min(keys, s.len - s.n + (g.row0 + g.rows - 1) / p->group + 1));
        g.t0 = min(g.c0 * kUnit, keys);
        g.t1 = min(g.c1 * kUnit, keys);
        u += g.c1 - c;
        c = g.c1;
        return true;
    }
};

template <int D, bool R8, bool ALIBI>
__global__ void __launch_bounds__(kThreads, 2) k_attn_decode(const __grid_constant__ CUtensorMap km,
                                                             const __grid_constant__ CUtensorMap vm,
                                                             const AttnParams p)
{
    using L = Smem<D>;
    constexpr int TR = R8 ? 8 : 16;
    constexpr int KS = D / 16;       // k-steps of q . k, and words a lane holds of a key
    constexpr int NT = D / 8;        // n-tiles of w . v
    constexpr uint32_t kTile = L::kTile;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t ring = smem_u32(smem);
    float *s_merge = reinterpret_cast<float *>(smem + L::kRing);
    float2 *s_meta = reinterpret_cast<float2 *>(smem + L::kRing + L::kMerge);
    uint64_t *s_bars = reinterpret_cast<uint64_t *>(smem + L::kRing + L::kMerge + L::kMeta);
    float2 *s_ml = reinterpret_cast<float2 *>(smem + L::kRing + L::kMerge + L::kMeta + L::kBars); // [warp][16]
    int64_t *s_start = reinterpret_cast<int64_t *>(smem + L::kTotal - 64);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const KvView &c = p.c;

    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < kStages; ++s)
            mbar_init(smem_u32(&s_bars[warp * kStages + s]), 1);
        fence_barrier_init();
        if (warp == 0) {
            tma_prefetch_desc(&km);
            tma_prefetch_desc(&vm);
        }
    }
    griddep_wait();
    griddep_release();

    // ---- this CTA's units: [U i / G, U (i + 1) / G), G = min(grid, U)
    const Range range = my_range<kThreads>(p, s_merge, s_start);
    if (range.u0 >= range.u1)
        return;

    const int page_shift = c.page_shift;
    const int box = page_shift >= 5 ? 32 : 16; // rows a TMA load brings
    const uint32_t bar0 = smem_u32(&s_bars[warp * kStages]);
    const uint32_t ring_w = ring + warp * (kStages * 2 * kTile);
    float2 *meta_w = s_meta + warp * kStages * 2;

    // ---- the loads: a cursor that runs ahead of the computation
    Walk<TR> ahead;
    Seg a;
    ahead.start(p, range.u0, range.u1, range.b, range.off);
    int at = 0;                 // next key of the cursor
    bool more = ahead.next(a);  // the cursor has a segment
    if (more)
        at = a.t0 + warp * kSub;
    auto settle = [&] { // on to a segment with keys for this warp
        while (more && at >= a.t1) {
            more = ahead.next(a);
            if (more)
                at = a.t0 + warp * kSub;
        }
    };
    settle();
    const int half = (lane & 1) * 16; // lanes look after the 16 keys of their parity
    auto page_at = [&](int key) { // page of `key`, -1 if it has none
        const int j = key >> page_shift;
        int page = -1;
        if (j < c.table_width)
            page = __ldg(c.table + a.b * c.table_stride + j);
        return page;
    };
    int page_next = more && at + half < a.t1 ? page_at(at + half) : -1;
    float ka_pend = 0.f, va_pend = 0.f; // scales fetched for the last issue, stored at the next
    int stage_pend = -1;
    bool bad_pend = false;
    int issued = 0;
    uint32_t bad_any = 0;
    auto store_meta = [&] {
        if (stage_pend >= 0 && lane < 2) {
            // An absent page weighs nothing: scale 0, weight 2^-inf.
            const float ks = ka_pend * (1.0f / 127.0f) * p.scale_log2;
            const float vs = bad_pend ? -1.f : fmaxf(va_pend * (1.0f / 127.0f), 1e-30f);
            meta_w[stage_pend * 2 + lane] = make_float2(bad_pend ? 0.f : ks, vs);
        }
        stage_pend = -1;
    };
    auto issue = [&] {
        store_meta();
        if (!more)
            return;
        const int s = issued % kStages;
        const bool want = at + half < a.t1;
        const bool ok = want && (unsigned)page_next < (unsigned)c.pages;
        if (want && !ok)
            bad_any = 1;
        const int block = page_next * c.heads + a.h; // fits: pages * heads * page_size < 2^31
        ka_pend = ok ? __ldg(c.ka + block) : 0.f;
        va_pend = ok ? __ldg(c.va + block) : 0.f;
        bad_pend = !ok;
        stage_pend = s;
        const int y = (block << page_shift) + ((at + half) & (c.page_size - 1));
        const uint32_t dst = ring_w + s * 2 * kTile, bar = bar0 + s * 8;
        const bool ok1 = __shfl_sync(0xffffffffu, ok, 1);
        if (box == 32) {
            if (lane == 0) {
                if (ok) {
                    mbar_arrive_expect_tx(bar, 2 * kTile);
                    tma_load_2d(dst, &km, bar, 0, y);
                    tma_load_2d(dst + kTile, &vm, bar, 0, y);
                } else {
                    mbar_arrive(bar);
                }
            }
        } else {
            if (lane == 0)
                mbar_arrive_expect_tx(bar, ((ok ? 1u : 0u) + (ok1 ? 1u : 0u)) * kTile);
            __syncwarp();
            if (lane < 2 && ok) {
                tma_load_2d(dst + lane * (kTile / 2), &km, bar, 0, y);
                tma_load_2d(dst + kTile + lane * (kTile / 2), &vm, bar, 0, y);
            }
        }
        ++issued;
        at += kUnit;
        settle();
        page_next = more && at + half < a.t1 ? page_at(at + half) : -1;
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s)
        issue();

    // ---- the computation
    Walk<TR> walk;
    Seg q;
    walk.start(p, range.u0, range.u1, range.b, range.off);
    int used = 0;
    bool failed = false;
    while (walk.next(q)) {
        // Rows of this lane: g, and g + 8 with 16-row tiles.
        uint32_t qa[KS][R8 ? 2 : 4];
        float fac[R8 ? 1 : 2], slope[R8 ? 1 : 2];
        int limit[R8 ? 1 : 2], pos[R8 ? 1 : 2]; // last key a row sees
#pragma unroll
        for (int i = 0; i < (R8 ? 1 : 2); ++i) {
            const int row = g + 8 * i;
            const bool live = row < q.rows;
            const int R = q.row0 + (live ? row : 0);
            const int tok = R / p.group, head = q.h * p.group + (R - tok * p.group);
            pos[i] = q.len - q.n + tok;
            limit[i] = !live ? INT32_MAX // nobody reads its result
                       : pos[i] < 0 ? -1 : p.causal ? min(pos[i], q.keys - 1) : q.keys - 1;
            slope[i] = ALIBI ? __ldg(p.slopes + head) * 1.44269504f : 0.f;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                static_cast<const uint16_t *>(p.q) + (__ldg(c.cu + q.b) + (int64_t)tok) * p.q_token + head * p.q_head +
                t * (D / 4));
            uint32_t w[2 * KS];
#pragma unroll
            for (int v = 0; v < KS / 2; ++v)
                reinterpret_cast<uint4 *>(w)[v] = live ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
            fac[i] = 1.f;
            if (p.bf16)
                fac[i] = bf16_row_to_f16<2 * KS>(w);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qa[k][i] = w[2 * k];
                qa[k][(R8 ? 1 : 2) + i] = w[2 * k + 1];
            }
        }
        const int lim_min = warp_min(R8 ? limit[0] : min(limit[0], limit[1]));
        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[n][e] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (int key = q.t0 + warp * kSub; key < q.t1; key += kUnit) {
            issue();
            const int s = used % kStages;
            failed |= !mbar_wait(bar0 + s * 8, (used / kStages) & 1);
            ++used;
            __syncwarp();
            const uint32_t kb = ring_w + s * 2 * kTile, vb = kb + kTile;
            const float2 m0 = meta_w[s * 2], m1 = meta_w[s * 2 + 1];
            float sc[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sc[j][e] = 0.f;
                const int row = 8 * j + g;
                uint32_t w[KS];
                if (D == 128) {
                    *reinterpret_cast<uint4 *>(w) = lds128(kb + row * 128 + (((2 * t) ^ g) << 4));
                    *reinterpret_cast<uint4 *>(w + 4) = lds128(kb + row * 128 + (((2 * t + 1) ^ g) << 4));
                } else {
                    *reinterpret_cast<uint4 *>(w) = lds128(kb + row * 64 + ((t ^ ((g >> 1) & 3)) << 4));
                }
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t b0, b1;
                    codes_to_f16(w[k], b0, b1);
                    mma_16816(sc[j], qa[k][0], R8 ? 0u : qa[k][1], R8 ? qa[k][1] : qa[k][2], R8 ? 0u : qa[k][3], b0, b1);
                }
            }
            // ---- scores to weights
            const float lv0 = m0.y < 0.f ? -INFINITY : __log2f(m0.y), lv1 = m1.y < 0.f ? -INFINITY : __log2f(m1.y);
            const float iv0 = m0.y < 0.f ? 0.f : __frcp_rn(m0.y), iv1 = m1.y < 0.f ? 0.f : __frcp_rn(m1.y);
            const bool edge = key + kSub - 1 > lim_min;
            uint32_t pa[4][R8 ? 2 : 2]; // [n-tile][row g: hi / row g + 8 (or lo)]
            float alpha[2];
#pragma unroll
            for (int i = 0; i < (R8 ? 1 : 2); ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float ks = (j < 2 ? m0.x : m1.x) * fac[i], lv = j < 2 ? lv0 : lv1;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int kk = key + 8 * j + 2 * t + e;
                        float x = sc[j][2 * i + e] * ks;
                        if (ALIBI)
                            x = fmaf(slope[i], (float)(kk - pos[i]), x);
                        x += lv;
                        if (edge && kk > limit[i])
                            x = -INFINITY;
                        sc[j][2 * i + e] = x;
                        top = fmaxf(top, x);
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float mn = fmaxf(m[i], top);
                const float mu = mn == -INFINITY ? 0.f : mn;
                alpha[i] = exp2_approx(m[i] - mu);
                m[i] = mn;
                float sum[2] = {0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float w0 = exp2_approx(sc[j][2 * i] - mu), w1 = exp2_approx(sc[j][2 * i + 1] - mu);
                    sum[j >> 1] += w0 + w1;
                    const uint32_t hi = down2<false>(w0, w1);
                    pa[j][i] = hi;
                    if (R8) {
                        const float2 h = up2<false>(hi);
                        pa[j][1] = down2<false>(w0 - h.x, w1 - h.y);
                    }
                }
                l[i] = fmaf(l[i], alpha[i], fmaf(sum[0], iv0, sum[1] * iv1));
            }
            if (R8)
                alpha[1] = alpha[0];
            if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][0] *= alpha[0];
                    o[n][1] *= alpha[0];
                    o[n][2] *= alpha[1];
                    o[n][3] *= alpha[1];
                }
            }
            // ---- weights times values
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const int r0 = 16 * ks + 2 * t;
                uint32_t v0[NT / 4], v1[NT / 4], v2[NT / 4], v3[NT / 4];
                if (D == 128) {
                    const uint32_t ra = vb + r0 * 128, x0 = (g ^ (r0 & 7)) << 4, x1 = (g ^ ((r0 + 1) & 7)) << 4;
                    *reinterpret_cast<uint4 *>(v0) = lds128(ra + x0);
                    *reinterpret_cast<uint4 *>(v1) = lds128(ra + 128 + x1);
                    *reinterpret_cast<uint4 *>(v2) = lds128(ra + 1024 + x0);
                    *reinterpret_cast<uint4 *>(v3) = lds128(ra + 1152 + x1);
                } else {
                    const uint32_t ra = vb + r0 * 64 + (((g >> 1) ^ ((r0 >> 1) & 3)) << 4) + (g & 1) * 8;
                    *reinterpret_cast<uint2 *>(v0) = lds64(ra);
                    *reinterpret_cast<uint2 *>(v1) = lds64(ra + 64);
                    *reinterpret_cast<uint2 *>(v2) = lds64(ra + 512);
                    *reinterpret_cast<uint2 *>(v3) = lds64(ra + 576);
                }
                const uint32_t a0 = pa[2 * ks][0], a1 = pa[2 * ks][1], a2 = pa[2 * ks + 1][0], a3 = pa[2 * ks + 1][1];
#pragma unroll
                for (int w = 0; w < NT / 4; ++w) {
                    uint32_t b0[4], b1[4];
                    code_pairs_to_f16(v0[w], v1[w], b0);
                    code_pairs_to_f16(v2[w], v3[w], b1);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mma_16816(o[4 * w + e], a0, a1, a2, a3, b0[e], b1[e]);
                }
            }
            __syncwarp(); // the stage is read: the next issue may overwrite it
        }

        // ---- the four warps' parts into one, 8 rows at a time
#pragma unroll
        for (int i = 0; i < (R8 ? 1 : 2); ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (t == 0)
                s_ml[warp * 16 + g + 8 * i] = make_float2(m[i], l[i]);
        }
        const bool whole = q.c0 == 0 && q.c1 == q.chunks;
        const int64_t out_row = (int64_t)__ldg(c.cu + q.b) * p.heads;
        float *slot = p.slots + ((int64_t)blockIdx.x * 2 + (q.c0 == 0 ? 1 : 0)) * (16 * (D + 2));
#pragma unroll
        for (int i = 0; i < (R8 ? 1 : 2); ++i) {
            if (i)
                __syncthreads();
            // This lane's dimensions of row g: the 2 NT from t D/4 on (n-tile
            // n holds dimension n of each of its two columns' blocks).
            float *dst = s_merge + (warp * kMergeRows + g) * D;
#pragma unroll
            for (int n = 0; n < NT; n += 4)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float4 v;
                    if (R8)
                        v = make_float4(o[n][e] + o[n][2 + e], o[n + 1][e] + o[n + 1][2 + e],
                                        o[n + 2][e] + o[n + 2][2 + e], o[n + 3][e] + o[n + 3][2 + e]);
                    else
                        v = make_float4(o[n][2 * i + e], o[n + 1][2 * i + e], o[n + 2][2 * i + e],
                                        o[n + 3][2 * i + e]);
                    // 16-byte chunks swizzled by row: rows are a multiple of all banks apart
                    const int chunk = ((2 * t + e) * NT + n) / 4;
                    reinterpret_cast<float4 *>(dst)[chunk ^ g] = v;
                }
            __syncthreads();
            for (int x = tid; x < kMergeRows * D / 4; x += kThreads) {
                const int rr = x / (D / 4), ch = x % (D / 4), row = rr + 8 * i;
                if (row >= q.rows)
                    break;
                float2 ml[kWarps];
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    ml[w] = s_ml[w * 16 + row];
                    M = fmaxf(M, ml[w].x);
                }
                const float mu = M == -INFINITY ? 0.f : M;
                float lsum = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = exp2_approx(ml[w].x - mu);
                    const float4 v =
                        reinterpret_cast<const float4 *>(s_merge + (w * kMergeRows + rr) * D)[ch ^ rr];
                    lsum = fmaf(ml[w].y, f, lsum);
                    acc.x = fmaf(v.x, f, acc.x);
                    acc.y = fmaf(v.y, f, acc.y);
                    acc.z = fmaf(v.z, f, acc.z);
                    acc.w = fmaf(v.w, f, acc.w);
                }
                if (whole) {
                    finish_row<D>(p, out_row, q.h, q.row0 + row, ch, acc, M, lsum);
                } else {
                    reinterpret_cast<float4 *>(slot)[row * (D / 4) + ch] = acc;
                    if (ch == 0)
                        reinterpret_cast<float2 *>(slot + 16 * D)[row] = make_float2(M, lsum);
                }
            }
        }
        if (!whole) {
            // Parts lie in CTA `first` (its opening slot) and all CTAs to
            // `last` (their other slots). The last to arrive adds them.
            const int64_t begin = walk.u - q.c1, G = range.parts;
            const int first = (int)(((begin + 1) * G - 1) / range.total);
            const int last = (int)(((begin + q.chunks) * G - 1) / range.total);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const uint32_t old = atomicAdd(p.arrived + first, 1u);
                const bool all = old == (uint32_t)(last - first);
                if (all)
                    p.arrived[first] = 0u;
                *reinterpret_cast<int *>(s_start) = all ? 1 : 0;
            }
            __syncthreads();
            if (*reinterpret_cast<volatile int *>(s_start)) {
                __threadfence();
                for (int x = tid; x < q.rows * (D / 4); x += kThreads) {
                    const int row = x / (D / 4), ch = x % (D / 4);
                    float M = -INFINITY, lsum = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int i = first; i <= last; ++i) {
                        const float *part = p.slots + ((int64_t)i * 2 + (i == first ? 1 : 0)) * (16 * (D + 2));
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(part + 16 * D) + row);
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(part) + row * (D / 4) + ch);
                        const float mn = fmaxf(M, ml.x), mu = mn == -INFINITY ? 0.f : mn;
                        const float fa = exp2_approx(M - mu), fb = exp2_approx(ml.x - mu);
                        M = mn;
                        lsum = fmaf(lsum, fa, ml.y * fb);
                        acc.x = fmaf(acc.x, fa, v.x * fb);
                        acc.y = fmaf(acc.y, fa, v.y * fb);
                        acc.z = fmaf(acc.z, fa, v.z * fb);
                        acc.w = fmaf(acc.w, fa, v.w * fb);
                    }
                    finish_row<D>(p, out_row, q.h, q.row0 + row, ch, acc, M, lsum);
                }
            }
        }
        __syncthreads(); // the merge buffers are free
    }
    if (bad_any)
        atomicOr(c.status, LLMINT8_DEV_BAD_PAGE);
    if (failed && lane == 0)
        atomicOr(c.status, LLMINT8_DEV_TIMEOUT_PRODUCER);
}

template <int D, bool R8>
cudaError_t launch(const AttnParams &p, const CUtensorMap &km, const CUtensorMap &vm, int grid, int device,
                   cudaStream_t stream)
{
    auto kern = p.slopes ? k_attn_decode<D, R8, true> : k_attn_decode<D, R8, false>;
    static std::atomic<uint64_t> configured[2];
    const uint64_t bit = 1ull << (device & 63);
    if (!(configured[p.slopes ? 1 : 0].load() & bit)) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kTotal);
        if (e != cudaSuccess)
            return e;
        configured[p.slopes ? 1 : 0].fetch_or(bit);
    }
    return launch_pdl(kern, dim3((unsigned)grid), kThreads, Smem<D>::kTotal, stream, km, vm, p);
}

} // namespace

cudaError_t launch_attn_decode(AttnParams p, const llmint8_kv_cache &c, bool r8, const DeviceInfo &dev,
                               cudaStream_t stream)
{
    CUtensorMap km, vm;
    const int64_t rows = c.pages * c.heads * c.page_size;
    const int box = c.page_size >= 32 ? 32 : 16;
    if (!encode_map_codes(&km, c.k_codes, rows, c.head_dim, box) ||
        !encode_map_codes(&vm, c.v_codes, rows, c.head_dim, box))
        return cudaErrorInvalidValue;
    p.tile_rows = r8 ? 8 : 16;
    p.unit = kUnit;
    const int grid = std::min(kAttnMaxCtas, 2 * dev.num_sms);
    if (c.head_dim == 128)
        return r8 ? launch<128, true>(p, km, vm, grid, dev.device, stream)
                  : launch<128, false>(p, km, vm, grid, dev.device, stream);
    return r8 ? launch<64, true>(p, km, vm, grid, dev.device, stream)
              : launch<64, false>(p, km, vm, grid, dev.device, stream);
}

} // namespace llmint8
