// Attention of few new tokens over the paged int8 key/value cache: a row tile
// of 8 or 16 (token, head) rows that share one key/value head, against that
// head's keys and values. Bound by HBM: every cached byte is read once (per
// row tile) and there are 2 to 64 flops for it.
//
// Mathematics. With codes kc, vc (exact as fp16), page scales ka / 127 and
// va / 127, and everything per key in log2 units:
//   x_j = (q . kc_j) * (ka_j / 127 * scale * log2 e) [+ slope * (j - p) * log2 e]
//   e_j = x_j + log2(va_j / 127),  w_j = 2^(e_j - m + 8),  m the running maximum of e
//   o = sum_j w_j vc_j,  l = sum_j w_j * (127 / va_j) / 2^8,  out = o / 2^8 / l
// The value scale rides on the exponent, so that the weights that enter the
// product are about 2^8 at most (no overflow of fp16) and the codes stay exact.
// They start there and not at 1 because fp16 ends at 2^-24: in a long sequence
// with one heavy key all others weigh little.
// q . kc and w . vc run on the tensor cores (fp16 in, fp32 sums). With row
// tiles of 8 the weights enter as hi + lo, what rounding to fp16 left over in
// a second product (off by at most 2^-22 of themselves or 2^-33 of the largest):
// there the matrix instructions have time to spare. With 16 rows the weights
// are fp16 (off by at most 2^-11 of themselves, or 2^-33 of the largest).
//
// Work. Unit: 128 keys of one (sequence, head, row tile). The units of all of
// them in order are split evenly over the CTAs, whatever the lengths; a CTA
// runs through its units in segments of one item. An item that lies in one
// CTA is finished there; of one that is split every CTA parks its part (o, m,
// l) in the workspace, and the last to arrive adds the parts in order (so the
// result does not depend on the order of arrival).
//
// One warp loads: its lanes look up the pages and scales of a unit's 16-key
// groups two units ahead (so that no lookup is waited for) and issue one TMA
// load each into a ring of two or three units. Four warps compute, 32 keys each. The
// products are taken transposed, keys (then dimensions) as the m16 side and
// the row tile as n8, so that no part of an instruction is spent on padding
// when 8 rows or fewer share a head. Shared memory is swizzled by the TMA, a
// lane's 16-byte reads are free of bank conflicts and hold exactly the codes
// of its operand fragments: the order of the dimensions within a product and
// of the output rows is free, and chosen for that.
//
// The running maximum m moves only when a score exceeds it by more than 2^6
// in weight (fp16 holds that as well): then no maximum is reduced over the
// warp and nothing rescaled for most units.
//
// On B200: 64 sequences of 100 to 8000 tokens, 32 heads over 8, pages of 16:
// 100 us, 5.3 TB/s of the cache (5.9 without the 9 us that a call of any size
// takes); 16 sequences of up to 2048, 112 heads with position biases: 116 us,
// 5.1 TB/s; two of 131072 and 100000, 16 rows a head: 98 us, 4.8 TB/s.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "attention.cuh"

namespace llmint8 {
namespace {

constexpr int kWarps = 4;             // that compute
constexpr int kSub = 32;              // keys a warp takes at once
constexpr int kUnit = kSub * kWarps;  // keys of a unit
constexpr int kGroups = kUnit / 16;   // 16 keys lie in one page
constexpr float kStart = 8.f;         // log2 of the weight at the running maximum
constexpr float kSlack = 6.f;         // log2 of how far a weight may exceed that: 2^14 at most, fp16 holds it

// With row tiles of 8 the registers allow three CTAs an SM, with 16 two; the
// ring takes what shared memory that leaves (192 KB an SM either way).
template <int D, int NQ>
struct Smem {
    static constexpr int kCtas = NQ == 1 ? 3 : 2;
    // With 16 rows the computing warps take registers from the loading one,
    // which for that comes with three idle ones (a warpgroup each; 2 x 128
    // threads x 128 at launch).
    static constexpr int kThreads = NQ == 1 ? (kWarps + 1) * 32 : 256;
    static constexpr int kStages = NQ == 1 ? 2 : 3;
    static constexpr int kTile = kUnit * D; // a unit's codes of one operand
    static constexpr int kRing = kStages * 2 * kTile;
    static constexpr int kMerge = kWarps * 4 * D * 4; // 4 rows at a time
    static constexpr int kMeta = kStages * kGroups * 16; // key scale, log2 value scale, 1 / value scale
    static constexpr int kBars = kStages * 2 * 8;
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

// The 8 x 8 matrix of 16-bit values spread over the warp (lane 4 r + c holds
// columns 2 c, 2 c + 1 of row r), transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
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

template <int D, int NQ, bool ALIBI>
__global__ void __launch_bounds__(Smem<D, NQ>::kThreads, Smem<D, NQ>::kCtas)
    k_attn_decode(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm, const AttnParams p)
{
    using L = Smem<D, NQ>;
    constexpr int kStages = L::kStages;
    constexpr bool kLo = NQ == 1;
    constexpr int KS = D / 16;  // k-steps of q . k, and words a lane holds of a key
    constexpr int MT = D / 16;  // m-tiles of w . v
    constexpr uint32_t kTile = L::kTile;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t ring = smem_u32(smem);
    float *s_merge = reinterpret_cast<float *>(smem + L::kRing);
    float *s_meta = reinterpret_cast<float *>(smem + L::kRing + L::kMerge);
    uint64_t *s_bars = reinterpret_cast<uint64_t *>(smem + L::kRing + L::kMerge + L::kMeta);
    float2 *s_ml = reinterpret_cast<float2 *>(smem + L::kRing + L::kMerge + L::kMeta + L::kBars); // [warp][16]
    int64_t *s_start = reinterpret_cast<int64_t *>(smem + L::kTotal - 64);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const KvView &c = p.c;
    const uint32_t full = smem_u32(s_bars), empty = full + kStages * 8;

    if (tid == 0) {
#pragma unroll
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s * 8, 1);
            mbar_init(empty + s * 8, kWarps);
        }
        fence_barrier_init();
        tma_prefetch_desc(&km);
        tma_prefetch_desc(&vm);
    }
    griddep_wait();
    griddep_release();

    // ---- this CTA's units: [U i / G, U (i + 1) / G), G = min(grid, U)
    const Range range = my_range<L::kThreads>(p, s_merge, s_start);
    if (range.u0 >= range.u1)
        return;

    if (warp >= kWarps) {
        // ------------------------------------------------ the loads
        if (NQ > 1) {
            regs_less<56>();
            if (warp > kWarps)
                return;
        }
        const int group = lane & 7, page_shift = c.page_shift;
        const bool is_v = lane >= 8;
        const int box = page_shift >= 5 ? 32 : 16; // rows a TMA load brings
        const bool loads = lane < 16 && (group * 16) % box == 0;
        LoadWalk units;
        units.start(p, range);
        bool failed = false;
        UnitLoad u0, u1, u2;
        units.fetch(p, u0);
        units.fetch(p, u1);
        units.scale(p, u0);
        for (int i = 0; u0.some; ++i) {
            units.fetch(p, u2);
            units.scale(p, u1);
            const int s = i % kStages;
            if (i >= kStages && !mbar_wait(empty + s * 8, ((i / kStages) - 1) & 1))
                failed = true;
            const bool load = loads && u0.page >= 0;
            const uint32_t n = __popc(__ballot_sync(0xffffffffu, load));
            failed = __any_sync(0xffffffffu, failed);
            if (failed)
                break;
            const uint32_t bar = full + s * 8;
            if (lane == 0)
                mbar_expect_tx(bar, n * box * D);
            __syncwarp();
            if (load)
                tma_load_2d(ring + (s * 2 + (is_v ? 1 : 0)) * kTile + group * 16 * D, is_v ? &vm : &km, bar, 0,
                            ((u0.page * c.heads + u0.h) << page_shift) + u0.slot);
            store_meta(s_meta + (s * kGroups + group) * 4, u0, p.scale_log2, exp2f(kStart));
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar);
            u0 = u1;
            u1 = u2;
        }
        if (units.bad)
            atomicOr(c.status, LLMINT8_DEV_BAD_PAGE);
        if (failed && lane == 0)
            atomicOr(c.status, LLMINT8_DEV_TIMEOUT_PRODUCER);
        return;
    }

    // ---------------------------------------------------- the computation
    if (NQ > 1)
        regs_more<200>();
    const int g = lane >> 2, t = lane & 3;
    int used = 0;
    bool failed = false;
    Walk walk;
    Seg q;
    walk.start(p, range);
    while (walk.next(p, q)) {
        // As an operand this lane holds dimensions t D/4 .. of row g (of each
        // 8); of the scores it has rows 2 t and 2 t + 1.
        uint32_t qb[NQ][KS][2];
        float fac[NQ][2], slope[NQ][2];
        int limit[NQ][2], pos[NQ][2]; // last key a row sees
        const int64_t first_row = c.cu[q.b];
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const int row = g + 8 * i;
            const bool live = row < q.rows;
            const int R = q.row0 + (live ? row : 0);
            const int tok = R / p.group, head = q.h * p.group + (R - tok * p.group);
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) +
                                                               (first_row + tok) * p.q_token + head * p.q_head +
                                                               t * (D / 4));
            uint32_t w[2 * KS];
#pragma unroll
            for (int v = 0; v < KS / 2; ++v)
                reinterpret_cast<uint4 *>(w)[v] = live ? src[v] : make_uint4(0, 0, 0, 0);
            float f = 1.f;
            if (p.bf16)
                f = bf16_to_f16<4>(w);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qb[i][k][0] = w[2 * k];
                qb[i][k][1] = w[2 * k + 1];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r2 = 2 * t + e;
                fac[i][e] = __shfl_sync(0xffffffffu, f, 4 * r2);
                const bool live2 = r2 + 8 * i < q.rows;
                const int R2 = q.row0 + (live2 ? r2 + 8 * i : 0);
                const int tok2 = R2 / p.group;
                pos[i][e] = q.len - q.n + tok2;
                limit[i][e] = !live2 ? INT32_MAX // nobody reads its result
                              : pos[i][e] < 0 ? -1 : p.causal ? min(pos[i][e], q.keys - 1) : q.keys - 1;
                slope[i][e] = ALIBI ? __ldg(p.slopes + q.h * p.group + (R2 - tok2 * p.group)) * 1.44269504f : 0.f;
            }
        }
        int lim_min = INT32_MAX;
#pragma unroll
        for (int i = 0; i < NQ; ++i)
            lim_min = min(lim_min, min(limit[i][0], limit[i][1]));
        lim_min = warp_min(lim_min);
        float o[NQ][MT][4];
        float m[NQ][2], l[NQ][2];
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            m[i][0] = m[i][1] = -INFINITY;
            l[i][0] = l[i][1] = 0.f;
#pragma unroll
            for (int n = 0; n < MT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[i][n][e] = 0.f;
        }

        for (int n = q.c0; n < q.c1; ++n, ++used) {
            const int s = used % kStages;
            if (!failed) // one wait that runs out is enough
                failed = !mbar_wait(full + s * 8, (used / kStages) & 1);
            __syncwarp();
            const int key = n * kUnit + warp * kSub;
            if (key < q.t1) {
                const uint32_t kb = ring + s * 2 * kTile + warp * kSub * D, vb = kb + kTile;
                const float4 m0 = *reinterpret_cast<const float4 *>(s_meta + (s * kGroups + 2 * warp) * 4);
                const float4 m1 = *reinterpret_cast<const float4 *>(s_meta + (s * kGroups + 2 * warp + 1) * 4);
                // ---- scores: two m-tiles of 16 keys
                float sc[NQ][2][4];
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    uint32_t w0[KS], w1[KS]; // codes of keys 16 a + g and 8 further
                    if (D == 128) {
                        const uint32_t ra = kb + (16 * a + g) * 128, x0 = ((2 * t) ^ g) << 4, x1 = x0 ^ 16;
                        *reinterpret_cast<uint4 *>(w0) = lds128(ra + x0);
                        *reinterpret_cast<uint4 *>(w0 + 4) = lds128(ra + x1);
                        *reinterpret_cast<uint4 *>(w1) = lds128(ra + 1024 + x0);
                        *reinterpret_cast<uint4 *>(w1 + 4) = lds128(ra + 1024 + x1);
                    } else {
                        const uint32_t ra = kb + (16 * a + g) * 64 + ((t ^ ((g >> 1) & 3)) << 4);
                        *reinterpret_cast<uint4 *>(w0) = lds128(ra);
                        *reinterpret_cast<uint4 *>(w1) = lds128(ra + 512);
                    }
#pragma unroll
                    for (int i = 0; i < NQ; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sc[i][a][e] = 0.f;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        uint32_t a0, a1, a2, a3;
                        codes_to_f16(w0[k], a0, a2);
                        codes_to_f16(w1[k], a1, a3);
#pragma unroll
                        for (int i = 0; i < NQ; ++i)
                            mma_16816(sc[i][a], a0, a1, a2, a3, qb[i][k][0], qb[i][k][1]);
                    }
                }
                // ---- to weights. sc[.][a][e]: key 16 a + g + 8 (e / 2), row 2 t + e % 2
                const bool edge = key + kSub - 1 > lim_min;
                uint32_t hi[NQ][2][2], lo[NQ][2][2];
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    bool over = false;
#pragma unroll
                    for (int a = 0; a < 2; ++a)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int kk = key + 16 * a + g + 8 * (e >> 1);
                            float x = sc[i][a][e];
                            if (ALIBI) {
                                x = fmaf(x, (a ? m1.x : m0.x) * fac[i][e & 1], a ? m1.y : m0.y);
                                x = fmaf(slope[i][e & 1], (float)(kk - pos[i][e & 1]), x);
                            } else {
                                x = fmaf(x, (a ? m1.x : m0.x) * fac[i][e & 1], a ? m1.y : m0.y);
                            }
                            if (edge && kk > limit[i][e & 1])
                                x = -INFINITY;
                            sc[i][a][e] = x;
                            over |= x > m[i][e & 1] + kSlack;
                        }
                    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float top = fmaxf(fmaxf(sc[i][0][e], sc[i][0][2 + e]), fmaxf(sc[i][1][e], sc[i][1][2 + e]));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                            const float mn = fmaxf(m[i][e], top);
                            const float alpha = mn == -INFINITY ? 1.f : exp2_approx(m[i][e] - mn);
                            m[i][e] = mn;
                            l[i][e] *= alpha;
#pragma unroll
                            for (int n = 0; n < MT; ++n) {
                                o[i][n][e] *= alpha;
                                o[i][n][2 + e] *= alpha;
                            }
                        }
                    }
                    const float mu[2] = {(m[i][0] == -INFINITY ? 0.f : m[i][0]) - kStart,
                                         (m[i][1] == -INFINITY ? 0.f : m[i][1]) - kStart};
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        const float iv = a ? m1.z : m0.z;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sc[i][a][e] = exp2_approx(sc[i][a][e] - mu[e & 1]);
                        l[i][0] = fmaf(sc[i][a][0] + sc[i][a][2], iv, l[i][0]);
                        l[i][1] = fmaf(sc[i][a][1] + sc[i][a][3], iv, l[i][1]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t h = down2<false>(sc[i][a][2 * e], sc[i][a][2 * e + 1]);
                            if (kLo) {
                                const float2 f = up2<false>(h);
                                lo[i][a][e] = transpose8x8(
                                    down2<false>(sc[i][a][2 * e] - f.x, sc[i][a][2 * e + 1] - f.y));
                            }
                            hi[i][a][e] = transpose8x8(h);
                        }
                    }
                }
                // ---- weights times values: m-tile n holds this lane's dimensions
                // 2 n (rows g) and 2 n + 1 (rows g + 8) of D / 8
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const int r0 = 16 * a + 2 * t;
                    uint32_t v0[MT / 2], v1[MT / 2], v2[MT / 2], v3[MT / 2];
                    if (D == 128) {
                        const uint32_t ra = vb + r0 * 128, x0 = (g ^ (r0 & 7)) << 4, x1 = x0 ^ 16;
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
#pragma unroll
                    for (int w = 0; w < MT / 2; ++w) {
                        uint32_t e0[4], e1[4];
                        code_pairs_to_f16(v0[w], v1[w], e0);
                        code_pairs_to_f16(v2[w], v3[w], e1);
#pragma unroll
                        for (int i = 0; i < NQ; ++i) {
                            mma_16816(o[i][2 * w], e0[0], e0[1], e1[0], e1[1], hi[i][a][0], hi[i][a][1]);
                            mma_16816(o[i][2 * w + 1], e0[2], e0[3], e1[2], e1[3], hi[i][a][0], hi[i][a][1]);
                            if (kLo) {
                                mma_16816(o[i][2 * w], e0[0], e0[1], e1[0], e1[1], lo[i][a][0], lo[i][a][1]);
                                mma_16816(o[i][2 * w + 1], e0[2], e0[3], e1[2], e1[3], lo[i][a][0], lo[i][a][1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(empty + s * 8);
        }

        // ---- the four warps' parts into one: each lane's rows 2 t, then its
        // rows 2 t + 1, of each 8
        const bool whole = q.c0 == 0 && q.c1 == q.chunks;
        const int64_t out_row = first_row * p.heads;
        float *slot = p.slots + ((int64_t)blockIdx.x * 2 + (q.c0 == 0 ? 1 : 0)) * (16 * (D + 2));
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[i][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                if (g == 0)
                    s_ml[warp * 16 + 2 * t + e + 8 * i] = make_float2(m[i][e], sum);
                // 16-byte chunks swizzled by row: rows are a multiple of all banks apart
                float4 *dst = reinterpret_cast<float4 *>(s_merge + (warp * 4 + t) * D);
#pragma unroll
                for (int n = 0; n < MT; n += 2)
                    dst[(g * (D / 32) + n / 2) ^ t] =
                        make_float4(o[i][n][e], o[i][n][2 + e], o[i][n + 1][e], o[i][n + 1][2 + e]);
                named_barrier_sync(1, kWarps * 32);
                for (int x = tid; x < 4 * D / 4; x += kWarps * 32) {
                    const int rr = x / (D / 4), ch = x % (D / 4), row = 2 * rr + e + 8 * i;
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
                        const float4 v = reinterpret_cast<const float4 *>(s_merge + (w * 4 + rr) * D)[ch ^ rr];
                        lsum = fmaf(ml[w].y, f, lsum);
                        acc.x = fmaf(v.x, f, acc.x);
                        acc.y = fmaf(v.y, f, acc.y);
                        acc.z = fmaf(v.z, f, acc.z);
                        acc.w = fmaf(v.w, f, acc.w);
                    }
                    if (whole) {
                        finish_row<D>(p, out_row, q.h, q.row0 + row, ch, acc, M, lsum, exp2f(kStart));
                    } else {
                        reinterpret_cast<float4 *>(slot)[row * (D / 4) + ch] = acc;
                        if (ch == 0)
                            reinterpret_cast<float2 *>(slot + 16 * D)[row] = make_float2(M, lsum);
                    }
                }
                named_barrier_sync(1, kWarps * 32); // the buffer is free
            }
        if (!whole) {
            // Parts lie in CTA `first` (its opening slot) and all CTAs to
            // `last` (their other slots). The last to arrive adds them.
            const int64_t begin = walk.u - q.c1, G = range.parts;
            const int first = (int)(((begin + 1) * G - 1) / range.total);
            const int last = (int)(((begin + q.chunks) * G - 1) / range.total);
            __threadfence();
            named_barrier_sync(1, kWarps * 32);
            if (tid == 0) {
                const uint32_t old = atomicAdd(p.arrived + first, 1u);
                const bool all = old == (uint32_t)(last - first);
                if (all)
                    p.arrived[first] = 0u;
                *reinterpret_cast<volatile int *>(s_start) = all ? 1 : 0;
            }
            named_barrier_sync(1, kWarps * 32);
            if (*reinterpret_cast<volatile int *>(s_start)) {
                __threadfence();
                for (int x = tid; x < q.rows * (D / 4); x += kWarps * 32) {
                    const int row = x / (D / 4), ch = x % (D / 4);
                    float M = -INFINITY, lsum = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int i = first; i <= last; ++i) {
                        const float *part = p.slots + ((int64_t)i * 2 + (i == first ? 1 : 0)) * (16 * (D + 2));
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(part + 16 * D) + row);
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(part) + row * (D / 4) + ch);
                        add_part(M, lsum, acc, ml, v);
                    }
                    finish_row<D>(p, out_row, q.h, q.row0 + row, ch, acc, M, lsum, exp2f(kStart));
                }
            }
            named_barrier_sync(1, kWarps * 32);
        }
    }
    if (failed && lane == 0)
        atomicOr(c.status, LLMINT8_DEV_TIMEOUT_EPILOGUE);
}

template <int D, int NQ>
cudaError_t launch(const AttnParams &p, const CUtensorMap &km, const CUtensorMap &vm, int grid, int device,
                   cudaStream_t stream)
{
    auto kern = p.slopes ? k_attn_decode<D, NQ, true> : k_attn_decode<D, NQ, false>;
    static std::atomic<uint64_t> configured[2];
    const uint64_t bit = 1ull << (device & 63);
    if (!(configured[p.slopes ? 1 : 0].load() & bit)) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, NQ>::kTotal);
        if (e != cudaSuccess)
            return e;
        configured[p.slopes ? 1 : 0].fetch_or(bit);
    }
    return launch_pdl(kern, dim3((unsigned)grid), Smem<D, NQ>::kThreads, Smem<D, NQ>::kTotal, stream, km, vm, p);
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
    const int grid = std::min(kAttnMaxCtas, (r8 ? 3 : 2) * dev.num_sms);
    if (c.head_dim == 128)
        return r8 ? launch<128, 1>(p, km, vm, grid, dev.device, stream)
                  : launch<128, 2>(p, km, vm, grid, dev.device, stream);
    return r8 ? launch<64, 1>(p, km, vm, grid, dev.device, stream)
              : launch<64, 2>(p, km, vm, grid, dev.device, stream);
}

} // namespace llmint8
