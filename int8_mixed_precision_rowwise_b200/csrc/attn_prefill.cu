// Attention of many new tokens over the paged int8 key/value cache: row tiles
// of 256 (token, head) rows that share one key/value head, on tcgen05 tensor
// cores. Bound by the tensor cores and, with them, by the exponentials: 128
// keys take a tile four 128 x 128 x D products and 2 x 128 x 128 powers of 2.
//
// The mathematics is that of the kernel for few rows (attn_decode.cu): codes
// exact as fp16, page scales on the scores and the exponents, fp16 weights
// of at most 2^13 together, a running maximum that moves only when it must.
//
// Work. Unit: 128 keys of one item, split evenly over the CTAs (one an SM) as
// there; a causal item has the units that its last row sees.
//
// Roles. Two warpgroups compute the weights of 128 rows each, a thread a row:
// its 128 scores come from tensor memory into registers, its weights go back
// there (over the scores) as fp16 and are the first operand of the value
// product; no reduction crosses threads. While one warpgroup computes, the
// tensor cores work for the other. A third warpgroup turns the codes into fp16
// tiles, keys and values alike [key][dimension] in 128-byte swizzled rows: the
// score product reads them along the dimensions, the value product across
// (the transposed form of the operand), so neither is transposed. One warp
// loads the codes with TMA, one thread issues the products.
//
// On B200, chunks of 2048 and 1500 tokens over 8192 and 6000, 32 heads over 8:
// 430 to 440 us, 840 to 860 TFLOP/s, 0.50 to 0.51 of the measured bf16 rate. A unit takes about 3950
// cycles; the special function unit and the tensor cores are busy for 2048 of
// them each, the chain scores -> weights (2600 for a row half, with both halves
// and the codes' conversion sharing the issue slots) -> products decides.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "attention.cuh"

namespace llmint8 {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 256;     // of a tile
constexpr int kUnit = 128;     // keys
constexpr int kGroups = 8;     // of 16 keys
constexpr int kMetaRing = 8;   // units whose scales are kept: more than can be under way
constexpr float kMostWeight = 8192.f; // of 128 weights together, before the maximum moves (fp16 holds 65504)
// Registers a thread of each role; 128 at launch, 2 x 128 x 192 + 128 x 56 +
// 128 x 72 = 512 x 128.
constexpr int kRegsRows = 192, kRegsCodes = 56, kRegsLoad = 72;
static_assert(2 * kRegsRows + kRegsCodes + kRegsLoad == 4 * 128, "register split");
constexpr int kHalf = 128 * 128; // bytes of 128 rows of 64 fp16 values

template <int D>
struct Smem {
    static constexpr int NH = D / 64;
    static constexpr int Q = 0;                       // [2 row halves][NH]
    static constexpr int K = Q + 2 * NH * kHalf;      // [2 stages][NH]
    static constexpr int V = K + 2 * NH * kHalf;      // [2 stages][NH]
    static constexpr int RAW = V + 2 * NH * kHalf;    // codes: keys, values
    static constexpr int META = RAW + 2 * kUnit * D;
    static constexpr int UNITS = META + kMetaRing * kGroups * 16; // what the units are (UnitInfo)
    static constexpr int BARS = UNITS + kMetaRing * 64;
    static constexpr int MISC = BARS + 40 * 8;
    static constexpr int TOTAL = MISC + 64;
};

// A unit, as the loading warp announces it to the other roles.
struct UnitInfo {
    int key;               // first key; < 0: there are no more units
    int first, last;       // of its segment
    int subs;              // row halves with rows
    int b, h, row0, rows, n, len, keys, chunks, whole; // of its segment
    int pad[3];
};
static_assert(sizeof(UnitInfo) == 64, "laid out in shared memory");

enum Bar { RAW_FULL = 0, RAW_EMPTY = 2, K_FULL = 4, K_EMPTY = 6, V_FULL = 8, V_EMPTY = 10, S_FULL = 12, P_FULL = 14,
           O_FULL = 16, Q_FULL = 18, META_FULL = 20, META_EMPTY = 28, DONE = 36,
           SYNC = 37 };

// D[tmem] (+)= A . B^T with fp16 operands and fp32 sums: A from shared memory,
// or from tensor memory (16-bit pairs, one row a lane).
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// Instruction descriptor of kind::f16: fp16 A and B, fp32 D; B along its rows
// (K-major) or across them.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_across)
{
    return (1u << 4) | ((b_across ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Operand read across its 128-byte swizzled rows (N contiguous): 64 values of
// N a row, 8-row atoms 1024 bytes apart along K, the next 64 of N kHalf bytes
// further (the leading offset).
__device__ __forceinline__ uint64_t smem_desc_across(uint32_t saddr)
{
    uint64_t d = smem_desc_k128(saddr);
    d &= ~((uint64_t)0x3FFFu << 16);
    d |= (uint64_t)(kHalf >> 4) << 16;
    return d;
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
        " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(r))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
          "l"(reinterpret_cast<uint64_t &>(c)));
    return r;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(r))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return r;
}

// A bounded wait that every later one gives up with: after the first that runs
// out, all roles go on to the end without loading or multiplying, so that
// every barrier between warps is still met.
// The roles on the chain from scores to weights to sums poll: waking from a
// suspended wait would cost them more than the issue slots.
template <bool POLL>
struct Waiter {
    volatile int *abort;
    uint32_t *status;
    uint32_t bit;
    __device__ __forceinline__ void operator()(uint32_t bar, int parity) const
    {
        if (POLL ? mbar_try_wait_poll(bar, parity) : mbar_try_wait(bar, parity))
            return;
        const uint64_t t0 = global_timer_ns();
        while (!*abort && !(POLL ? mbar_try_wait_poll(bar, parity) : mbar_try_wait(bar, parity))) {
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                *abort = 1;
                atomicOr(status, bit);
            }
        }
    }
};

template <int D, bool ALIBI>
__global__ void __launch_bounds__(kThreads, 1) k_attn_prefill(const __grid_constant__ CUtensorMap km,
                                                              const __grid_constant__ CUtensorMap vm,
                                                              const AttnParams p)
{
    using L = Smem<D>;
    constexpr int NH = L::NH;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem), bars = base + L::BARS;
    auto bar = [&](int which) { return bars + which * 8; };
    float *s_meta = reinterpret_cast<float *>(smem + L::META);
    UnitInfo *s_info = reinterpret_cast<UnitInfo *>(smem + L::UNITS);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + L::MISC);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + L::MISC + 4);
    volatile int *s_last = reinterpret_cast<volatile int *>(smem + L::MISC + 8);
    int64_t *s_start = reinterpret_cast<int64_t *>(smem + L::MISC + 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const KvView &c = p.c;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(RAW_FULL + i), 1);
            mbar_init(bar(RAW_EMPTY + i), 4);
            mbar_init(bar(K_FULL + i), 4);
            mbar_init(bar(K_EMPTY + i), 1);
            mbar_init(bar(V_FULL + i), 4);
            mbar_init(bar(V_EMPTY + i), 1);
            mbar_init(bar(S_FULL + i), 1);
            mbar_init(bar(P_FULL + i), 4);
            mbar_init(bar(O_FULL + i), 1);
            mbar_init(bar(Q_FULL + i), 4);
        }
        for (int i = 0; i < kMetaRing; ++i) {
            mbar_init(bar(META_FULL + i), 1);
            mbar_init(bar(META_EMPTY + i), 8);
        }
        mbar_init(bar(DONE), 1);
        mbar_init(bar(SYNC), 8);
        fence_barrier_init();
        *s_abort = 0;
        tma_prefetch_desc(&km);
        tma_prefetch_desc(&vm);
    }
    griddep_wait();
    griddep_release();
    const Range range = my_range<kThreads>(p, smem + L::META, s_start);
    if (range.u0 >= range.u1)
        return;
    if (warp == 12) {
        tmem_alloc(smem_u32(s_tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(s_tmem);

    if (warp < 8) {
        // ------------------------------------------------ weights and output
        regs_more<kRegsRows>();
        const int sub = warp >> 2, r = tid & 127; // row half, row in it = lane of tensor memory
        const Waiter<true> wait{s_abort, c.status, LLMINT8_DEV_TIMEOUT_EPILOGUE};
        const uint32_t t_s = tmem + ((uint32_t)(warp & 3) << 21) + sub * 128, t_o = t_s + 256;
        int mine = 0;  // units of this row half so far
        float m = -INFINITY, l = 0.f, fac = 1.f, slope = 0.f;
        int limit = 0, lim_min = 0, pos = 0;
        int64_t walked = range.u0; // units of the whole list up to this one
        int syncs = 0;
        auto sync = [&] { // of both warpgroups; bounded, as every wait here
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(SYNC));
            wait(bar(SYNC), syncs++ & 1);
            __syncwarp();
        };
        for (int i = 0;; ++i) {
            const int slot = i % kMetaRing;
            wait(bar(META_FULL + slot), (i / kMetaRing) & 1);
            __syncwarp();
            const volatile UnitInfo *info = s_info + slot;
            const int key = info->key;
            if (__any_sync(0xffffffffu, key < 0 || *s_abort)) // the whole warp or none of it
                break;
            ++walked;
            const bool active = sub < info->subs, first = info->first, last = info->last;
            if (active && first) {
                // The row into swizzled shared memory. All products of the
                // segment before are complete (its last scores were read).
                const int row = sub * 128 + r;
                const bool live = row < info->rows;
                const int R = info->row0 + (live ? row : 0), h = info->h;
                const int tok = R / p.group, head = h * p.group + (R - tok * p.group);
                pos = info->len - info->n + tok;
                limit = !live ? INT32_MAX : pos < 0 ? -1 : p.causal ? min(pos, info->keys - 1) : info->keys - 1;
                lim_min = warp_min(limit);
                slope = ALIBI ? __ldg(p.slopes + head) * 1.44269504f : 0.f;
                m = -INFINITY;
                l = 0.f;
                fac = 1.f;
                // D / 8 lanes read a row, 32 of a warp's rows in as many steps
                // as that takes; a row's place comes from the lane that has it.
                constexpr int kLanes = D / 8, kSteps = kLanes;
                const uint64_t src = reinterpret_cast<uint64_t>(
                    static_cast<const uint16_t *>(p.q) + (c.cu[info->b] + (int64_t)tok) * p.q_token +
                    head * p.q_head);
                const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u; // scores grow with the products
                uint4 w[kSteps];
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const int from = k * (32 / kLanes) + lane / kLanes;
                    const uint64_t at = __shfl_sync(0xffffffffu, src, from);
                    const bool there = __shfl_sync(0xffffffffu, (int)live, from);
                    w[k] = there ? reinterpret_cast<const uint4 *>(at)[lane % kLanes] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const int of = k * (32 / kLanes) + lane / kLanes; // row of the warp
                    if (p.bf16) {
                        const float f = bf16_to_f16<kLanes>(reinterpret_cast<uint32_t (&)[4]>(w[k]));
                        const float g = __shfl_sync(0xffffffffu, f, (lane % (32 / kLanes)) * kLanes);
                        if (lane / (32 / kLanes) == k)
                            fac = g;
                    }
                    const int rr = (warp & 3) * 32 + of, ch = lane % kLanes;
                    *reinterpret_cast<uint4 *>(smem + L::Q + (sub * NH + ch / 8) * kHalf + rr * 128 +
                                               (((ch & 7) ^ (rr & 7)) << 4)) =
                        make_uint4(w[k].x ^ flip, w[k].y ^ flip, w[k].z ^ flip, w[k].w ^ flip);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(Q_FULL + sub));
            }
            if (active) {
                const float4 *meta = reinterpret_cast<const float4 *>(s_meta + slot * kGroups * 4);
                wait(bar(S_FULL + sub), mine & 1);
                __syncwarp();
                tc_fence_after();
                // Scores of a group share one scale; where keys are masked or
                // have a position term the exponents are formed one by one,
                // scale 1 from there.
                const bool each = ALIBI || key + kUnit - 1 > lim_min;
                // The maximum so far mostly will do: that none of the weights
                // is too large shows in their sum. If one is, the scores (still
                // in tensor memory) are read again and the maximum moves. A row
                // that has not met a key yet has none.
                bool move = first || __any_sync(0xffffffffu, m == -INFINITY);
                uint32_t w16[64];
                float sum_l;
                for (;;) {
                    uint32_t s[4][32];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tmem_ld_32x32b_x32(t_s + k * 32, s[k]);
                    tmem_wait_ld();
                    if (each) {
#pragma unroll
                        for (int j = 0; j < kGroups; ++j) {
                            const float4 mt = meta[j];
                            const float a = mt.x * fac;
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                uint32_t &v = s[j >> 1][(j & 1) * 16 + e];
                                const int kk = key + j * 16 + e;
                                float x = fmaf(__uint_as_float(v), a, mt.y);
                                if (ALIBI)
                                    x = fmaf(slope, (float)(kk - pos), x);
                                if (kk > limit)
                                    x = -INFINITY;
                                v = __float_as_uint(x);
                            }
                        }
                    }
                    if (move) {
                        float top = -INFINITY;
#pragma unroll
                        for (int j = 0; j < kGroups; ++j) {
                            const float4 mt = meta[j];
                            float g0 = -INFINITY, g1 = -INFINITY;
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const uint32_t *v = &s[j >> 1][(j & 1) * 16 + e];
                                g0 = max3(g0, __uint_as_float(v[0]), __uint_as_float(v[1]));
                                g1 = max3(g1, __uint_as_float(v[2]), __uint_as_float(v[3]));
                            }
                            g0 = fmaxf(g0, g1);
                            top = fmaxf(top, each ? g0 : fmaf(g0, mt.x * fac, mt.y));
                        }
                        const float mn = fmaxf(m, top);
                        const float alpha = mn == -INFINITY ? 1.f : exp2_approx(m - mn);
                        m = mn;
                        l *= alpha;
                        if (!first) { // the sums so far, with all products before complete
                            wait(bar(O_FULL + sub), (mine - 1) & 1);
                            __syncwarp();
                            tc_fence_after();
#pragma unroll 1
                            for (int k = 0; k < D / 16; ++k) {
                                uint32_t o[16];
                                tmem_ld_32x32b_x16(t_o + k * 16, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st_32x32b_x16(t_o + k * 16, o);
                            }
                        }
                    }
                    const float mu = m == -INFINITY ? 0.f : m;
                    sum_l = 0.f;
                    float all = 0.f;
#pragma unroll
                    for (int j = 0; j < kGroups; ++j) {
                        const float4 mt = meta[j];
                        const float a = each ? 1.f : mt.x * fac, b = each ? -mu : mt.y - mu;
                        const float2 a2 = make_float2(a, a), b2 = make_float2(b, b);
                        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const uint32_t *v = &s[j >> 1][(j & 1) * 16 + e];
                            float2 x = fma2(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), a2, b2);
                            x.x = exp2_approx(x.x);
                            x.y = exp2_approx(x.y);
                            sum = add2(sum, x);
                            w16[j * 8 + e / 2] = down2<false>(x.x, x.y);
                        }
                        sum.x += sum.y;
                        all += sum.x;
                        sum_l = fmaf(sum.x, mt.z, sum_l);
                    }
                    if (move || !__any_sync(0xffffffffu, all > kMostWeight))
                        break;
                    move = true;
                }
                l += sum_l;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    tmem_st_32x32b_x32(t_s + h * 32, reinterpret_cast<const uint32_t (&)[32]>(w16[h * 32]));
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(P_FULL + sub));
                ++mine;
            }
            if (!last) {
                __syncwarp(); // all lanes have read what the slot says
                if (lane == 0)
                    mbar_arrive(bar(META_EMPTY + slot));
                continue;
            }

            // ---- the segment's sums out
            const int c1 = key / kUnit + 1; // its units are [c0, c1) of the item
            const bool whole = info->whole;
            const int64_t out_row = (int64_t)c.cu[info->b] * p.heads;
            // An item's first part goes to the CTA's second slot.
            const int64_t begin = walked - c1; // of the item
            float *part = p.slots + ((int64_t)blockIdx.x * 2 + (begin >= range.u0 ? 1 : 0)) * (kRows * (D + 2));
            if (active) {
                const int row = sub * 128 + r;
                const bool live = row < info->rows;
                const int R = info->row0 + (live ? row : 0), h = info->h;
                const int tok = R / p.group;
                const int64_t at = out_row + (int64_t)tok * p.heads + h * p.group + (R - tok * p.group);
                wait(bar(O_FULL + sub), (mine - 1) & 1);
                __syncwarp();
                tc_fence_after();
                // Through the query area, free now, in its layout: each warp its
                // own rows, as the next segment's queries may come into the
                // others' already. 2 D bytes of a row at a time, so that whole
                // lines are written.
                const float inv = whole ? (l > 0.f ? 1.0f / l : 0.f) : 1.f;
                uint8_t *stage = smem + L::Q + sub * NH * kHalf + (warp & 3) * 32 * 128;
                auto staged = [&](int row, int ch) {
                    return reinterpret_cast<uint4 *>(stage + (ch / 8) * kHalf + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
                };
                constexpr int kRowBytes = D * 2, kCh = kRowBytes / 16; // 16-byte pieces of a staged row
                const uint64_t to = whole ? reinterpret_cast<uint64_t>(static_cast<uint16_t *>(p.out) + at * D)
                                          : reinterpret_cast<uint64_t>(part + row * D);
#pragma unroll 1
                for (int pass = 0; pass < (whole ? 1 : 2); ++pass) {
#pragma unroll 1
                    for (int k = 0; k < (whole ? D : D / 2); k += 16) {
                        uint32_t o[16];
                        tmem_ld_32x32b_x16(t_o + pass * (D / 2) + k, o);
                        tmem_wait_ld();
                        if (whole) {
                            uint32_t v[8];
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                const float y = __uint_as_float(o[2 * x]) * inv, z = __uint_as_float(o[2 * x + 1]) * inv;
                                v[x] = p.bf16 ? down2<true>(y, z) : down2<false>(y, z);
                            }
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                *staged(lane, k / 8 + x) =
                                    make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                        } else {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                *staged(lane, k / 4 + x) =
                                    make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < kCh; ++k) {
                        const int of = k * (32 / kCh) + lane / kCh, ch = lane % kCh;
                        const uint64_t dst = __shfl_sync(0xffffffffu, to, of);
                        if (__shfl_sync(0xffffffffu, (int)live, of))
                            *reinterpret_cast<uint4 *>(dst + pass * kRowBytes + ch * 16) = *staged(of, ch);
                    }
                    __syncwarp();
                }
                tc_fence_before(); // read before the next segment's products write there
                if (live && whole && p.lse)
                    p.lse[at] = l > 0.f ? (m + log2f(l)) * 0.69314718f : -INFINITY;
                if (live && !whole)
                    reinterpret_cast<float2 *>(part + kRows * D)[row] = make_float2(m, l);
            }
            if (!whole) {
                // As in the kernel for few rows: the last part to arrive adds
                // them all, in order.
                const int64_t G = range.parts;
                const int from = (int)(((begin + 1) * G - 1) / range.total);
                const int to = (int)(((begin + info->chunks) * G - 1) / range.total);
                __threadfence();
                sync();
                if (tid == 0) {
                    const bool all = atomicAdd(p.arrived + from, 1u) == (uint32_t)(to - from);
                    if (all)
                        p.arrived[from] = 0u;
                    *s_last = all ? 1 : 0;
                }
                sync();
                if (*s_last) {
                    __threadfence();
                    const int rows = info->rows, row0 = info->row0, h = info->h;
                    // Sixteen rows at a time, all their loads under way at once.
                    constexpr int kLanes = D / 4, kStep = 256 / kLanes; // lanes a row takes, rows a step
                    const int ch = tid % kLanes;
                    constexpr int kAt = 16;
                    for (int r0 = tid / kLanes; r0 < rows; r0 += kAt * kStep) {
                        float M[kAt], lsum[kAt];
                        float4 acc[kAt];
#pragma unroll
                        for (int x = 0; x < kAt; ++x) {
                            M[x] = -INFINITY;
                            lsum[x] = 0.f;
                            acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                        for (int k = from; k <= to; ++k) {
                            const float *it = p.slots + ((int64_t)k * 2 + (k == from ? 1 : 0)) * (kRows * (D + 2));
                            float2 ml[kAt];
                            float4 v[kAt];
#pragma unroll
                            for (int x = 0; x < kAt; ++x) {
                                const int rr = min(r0 + x * kStep, rows - 1);
                                ml[x] = __ldcg(reinterpret_cast<const float2 *>(it + kRows * D) + rr);
                                v[x] = __ldcg(reinterpret_cast<const float4 *>(it) + rr * kLanes + ch);
                            }
#pragma unroll
                            for (int x = 0; x < kAt; ++x)
                                add_part(M[x], lsum[x], acc[x], ml[x], v[x]);
                        }
#pragma unroll
                        for (int x = 0; x < kAt; ++x)
                            if (r0 + x * kStep < rows)
                                finish_row<D>(p, out_row, h, row0 + r0 + x * kStep, ch, acc[x], M[x], lsum[x], 1.f);
                    }
                }
                sync(); // s_last is free
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(META_EMPTY + slot));
        }
    } else if (warp < 12) {
        // ------------------------------------------------ codes to fp16 tiles
        regs_less<kRegsCodes>();
        const Waiter<true> wait{s_abort, c.status, LLMINT8_DEV_TIMEOUT_PRODUCER};
        const int r = tid & 127; // a key each
        for (int i = 0;; ++i) {
            wait(bar(META_FULL + i % kMetaRing), (i / kMetaRing) & 1);
            const int key = reinterpret_cast<const volatile UnitInfo *>(s_info)[i % kMetaRing].key;
            if (__any_sync(0xffffffffu, key < 0 || *s_abort))
                break;
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
                const int st = i & 1;
                wait(bar(RAW_FULL + kv), i & 1);
                if (i >= 2)
                    wait(bar((kv ? V_EMPTY : K_EMPTY) + st), ((i >> 1) - 1) & 1);
                const uint8_t *src = smem + L::RAW + kv * kUnit * D + r * D;
                uint8_t *dst = smem + (kv ? L::V : L::K) + st * NH * kHalf + r * 128;
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const int sw = D == 128 ? x ^ (r & 7) : x ^ ((r >> 1) & 3);
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + (sw << 4));
                    uint4 a, b;
                    codes_to_f16(v.x, a.x, a.y);
                    codes_to_f16(v.y, a.z, a.w);
                    codes_to_f16(v.z, b.x, b.y);
                    codes_to_f16(v.w, b.z, b.w);
                    uint8_t *d = dst + (x / 4) * kHalf;
                    *reinterpret_cast<uint4 *>(d + (((2 * (x & 3)) ^ (r & 7)) << 4)) = a;
                    *reinterpret_cast<uint4 *>(d + (((2 * (x & 3) + 1) ^ (r & 7)) << 4)) = b;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar((kv ? V_FULL : K_FULL) + st));
                    mbar_arrive(bar(RAW_EMPTY + kv));
                }
            }
        }
    } else {
        regs_less<kRegsLoad>();
        if (warp == 12) {
            // -------------------------------------------- the products
            // The whole warp runs the loop, on values that are the same in
            // every lane (descriptors in uniform registers: with one lane in a
            // branch of its own each product took 150 cycles to issue, more
            // than it takes to compute); one elected lane issues.
            const Waiter<true> wait{s_abort, c.status, LLMINT8_DEV_TIMEOUT_MMA};
            constexpr uint32_t id_s = idesc_f16(128, kUnit, false), id_o = idesc_f16(128, D, true);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            auto scores = [&](int sub, int st) {
                const uint64_t a = smem_desc_k128(base + L::Q + sub * NH * kHalf);
                const uint64_t b = smem_desc_k128(base + L::K + st * NH * kHalf);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = (uint32_t)((k / 4) * kHalf + (k & 3) * 32) >> 4;
                        mma_f16_ss(tm + sub * 128, a + off, b + off, id_s, k > 0);
                    }
                    mma_commit(bar(S_FULL + sub));
                }
                __syncwarp();
            };
            auto values = [&](int sub, int st, uint32_t add) {
                const uint64_t b = smem_desc_across(base + L::V + st * NH * kHalf);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kUnit / 16; ++k)
                        mma_f16_ts(tm + 256 + sub * 128, tm + sub * 128 + k * 8, b + (uint32_t)((k * 2048) >> 4), id_o,
                                   k > 0 ? 1u : add);
                    mma_commit(bar(O_FULL + sub));
                }
                __syncwarp();
            };
            auto commit = [&](int which) {
                if (elect_one())
                    mma_commit(bar(which));
                __syncwarp();
            };
            int segs0 = 0, segs1 = 0, done0 = 0, done1 = 0;
            for (int i = 0;; ++i) {
                const int slot = i % kMetaRing, st = i & 1, nst = st ^ 1;
                wait(bar(META_FULL + slot), (i / kMetaRing) & 1);
                const volatile UnitInfo *info = s_info + slot;
                if (__any_sync(0xffffffffu, info->key < 0 || *s_abort))
                    break;
                const bool both = __any_sync(0xffffffffu, info->subs == 2);
                const bool first = __any_sync(0xffffffffu, info->first), last = __any_sync(0xffffffffu, info->last);
                if (first) {
                    wait(bar(K_FULL + st), (i >> 1) & 1);
                    wait(bar(Q_FULL), segs0++ & 1);
                    __syncwarp();
                    tc_fence_after();
                    scores(0, st);
                    if (both) {
                        wait(bar(Q_FULL + 1), segs1++ & 1);
                        __syncwarp();
                        tc_fence_after();
                        scores(1, st);
                    }
                    commit(K_EMPTY + st);
                }
                wait(bar(V_FULL + st), (i >> 1) & 1);
                wait(bar(P_FULL), done0++ & 1);
                __syncwarp();
                tc_fence_after();
                values(0, st, first ? 0u : 1u);
                if (!last) {
                    wait(bar(K_FULL + nst), ((i + 1) >> 1) & 1);
                    __syncwarp();
                    tc_fence_after();
                    scores(0, nst);
                }
                if (both) {
                    wait(bar(P_FULL + 1), done1++ & 1);
                    __syncwarp();
                    tc_fence_after();
                    values(1, st, first ? 0u : 1u);
                    if (!last)
                        scores(1, nst);
                }
                commit(V_EMPTY + st);
                if (!last)
                    commit(K_EMPTY + nst);
            }
            commit(DONE); // everything issued is complete before the memory goes
            mbar_wait(bar(DONE), 0);
        } else if (warp == 13) {
            // -------------------------------------------- the loads
            const Waiter<true> wait{s_abort, c.status, LLMINT8_DEV_TIMEOUT_PRODUCER};
            const int group = lane & 7;
            const bool is_v = lane >= 8;
            const int box = c.page_shift >= 5 ? 32 : 16;
            const bool loads = lane < 16 && (group * 16) % box == 0;
            LoadWalk units;
            units.start(p, range);
            // Unit n: requested, and announced but for `last`, which the next
            // one tells.
            auto fetch = [&](UnitLoad &u, int n) {
                units.fetch(p, u);
                if (!u.some)
                    return;
                if (n >= kMetaRing)
                    wait(bar(META_EMPTY + n % kMetaRing), (n / kMetaRing - 1) & 1);
                __syncwarp();
                if (lane == 0) {
                    UnitInfo &o = s_info[n % kMetaRing];
                    const Seg &q = units.q;
                    o.key = (units.c - 1) * kUnit;
                    o.first = u.first;
                    o.subs = q.rows > 128 ? 2 : 1;
                    o.b = q.b;
                    o.h = q.h;
                    o.row0 = q.row0;
                    o.rows = q.rows;
                    o.n = q.n;
                    o.len = q.len;
                    o.keys = q.keys;
                    o.chunks = q.chunks;
                    o.whole = q.c0 == 0 && q.c1 == q.chunks;
                }
            };
            UnitLoad u0, u1, u2;
            fetch(u0, 0);
            fetch(u1, 1);
            units.scale(p, u0);
            int i = 0;
            for (; u0.some; ++i) {
                fetch(u2, i + 2);
                units.scale(p, u1);
                if (lane == 0)
                    s_info[i % kMetaRing].last = !u1.some || u1.first;
                store_meta(s_meta + ((i % kMetaRing) * kGroups + group) * 4, u0, fabsf(p.scale_log2), 1.f);
                const bool load = loads && u0.page >= 0;
                const uint32_t which = __ballot_sync(0xffffffffu, load);
                __syncwarp(); // all lanes' scales are written
                if (lane == 0)
                    mbar_arrive(bar(META_FULL + i % kMetaRing));
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    if (i > 0)
                        wait(bar(RAW_EMPTY + kv), (i - 1) & 1);
                    const bool go = __all_sync(0xffffffffu, !*s_abort);
                    const uint32_t full = bar(RAW_FULL + kv);
                    if (lane == 0 && go)
                        mbar_arrive_expect_tx(full, __popc(which & (kv ? 0xFF00u : 0xFFu)) * box * D);
                    __syncwarp();
                    if (load && go && is_v == (kv == 1))
                        tma_load_2d(base + L::RAW + kv * kUnit * D + group * 16 * D, kv ? &vm : &km, full, 0,
                                    ((u0.page * c.heads + u0.h) << c.page_shift) + u0.slot);
                }
                u0 = u1;
                u1 = u2;
            }
            if (i >= kMetaRing)
                wait(bar(META_EMPTY + i % kMetaRing), (i / kMetaRing - 1) & 1);
            if (lane == 0) {
                s_info[i % kMetaRing].key = -1;
                mbar_arrive(bar(META_FULL + i % kMetaRing));
            }
            if (units.bad)
                atomicOr(c.status, LLMINT8_DEV_BAD_PAGE);
            // After an aborted run: the loads under way land before the CTA ends.
            if (*s_abort && i > 0)
                for (int kv = 0; kv < 2; ++kv)
                    mbar_wait(bar(RAW_FULL + kv), (i - 1) & 1);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool ALIBI>
cudaError_t launch(const AttnParams &p, const CUtensorMap &km, const CUtensorMap &vm, int grid, int device,
                   cudaStream_t stream)
{
    auto kern = k_attn_prefill<D, ALIBI>;
    static std::atomic<uint64_t> configured{0};
    const uint64_t bit = 1ull << (device & 63);
    if (!(configured.load() & bit)) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::TOTAL);
        if (e != cudaSuccess)
            return e;
        configured.fetch_or(bit);
    }
    return launch_pdl(kern, dim3((unsigned)grid), kThreads, Smem<D>::TOTAL, stream, km, vm, p);
}

} // namespace

cudaError_t launch_attn_prefill(AttnParams p, const llmint8_kv_cache &c, const DeviceInfo &dev, cudaStream_t stream)
{
    CUtensorMap km, vm;
    const int64_t rows = c.pages * c.heads * c.page_size;
    const int box = c.page_size >= 32 ? 32 : 16;
    if (!encode_map_codes(&km, c.k_codes, rows, c.head_dim, box) ||
        !encode_map_codes(&vm, c.v_codes, rows, c.head_dim, box))
        return cudaErrorInvalidValue;
    p.tile_rows = kRows;
    p.unit = kUnit;
    const int grid = std::min(kAttnPrefillCtas, dev.num_sms);
    if (c.head_dim == 128)
        return p.slopes ? launch<128, true>(p, km, vm, grid, dev.device, stream)
                        : launch<128, false>(p, km, vm, grid, dev.device, stream);
    return p.slopes ? launch<64, true>(p, km, vm, grid, dev.device, stream)
                    : launch<64, false>(p, km, vm, grid, dev.device, stream);
}

} // namespace llmint8
