// Residual addition, root-mean-square norm and row-wise int8 quantization
// before an LLM.int8() linear, and the recovery of values from row codes.
//
//   h = x + residual, rounded to the input type (the new residual stream)
//   y = fp16(fp32(h * w / sqrt(mean(h^2) + eps))), as from 64 bits
//   codes, row absmax, outlier bitmap of y: as llmint8_quantize_rowwise gives
//   them for the stored y (page "Hugging Face 将 LLM.int8() 8-bit 量化集成进
//   transformers 与 accelerate", sections "模型量化简介" and "MatMul 内部")
//
// Bound by HBM: per element two 2-byte reads, a 2-byte h, a 2-byte y and a
// 1-byte code written. On B200, 4001 x 14336 with a residual and outlier
// columns: 107 us, 4.8 TB/s (a copy runs at 6.5): a row's two reductions and
// about 275 instructions per 8 columns (issue slots 53% taken) keep the loads
// waiting; 32 x 14336: 9 us. The codes' values again: 26 us, 6.7 TB/s. The sum
// of squares as a pair costs 3% of that (130 -> 133 us both together; 2048 x
// 4096, codes only, 15.4 -> 16.9); in doubles, reduced by shuffles, 142 and 18.9.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "llmint8.h"

namespace llmint8 {
namespace {

constexpr int kVec = 4;             // 16-byte vectors a thread holds of its row
constexpr int kMaxRowThreads = 1024; // so rows of up to 32768 columns stay in registers

// h = x + residual, rounded once (what an fp32 sum rounded to 16 bits gives as
// well: 24 bits are enough for the second rounding to change nothing).
template <bool BF16>
__device__ __forceinline__ uint4 add8(const uint4 &x, const uint4 &r)
{
    uint4 o;
    if (BF16) {
        const __nv_bfloat162 *a = reinterpret_cast<const __nv_bfloat162 *>(&x);
        const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<__nv_bfloat162 *>(&o)[i] = __hadd2(a[i], b[i]);
    } else {
        const __half2 *a = reinterpret_cast<const __half2 *>(&x), *b = reinterpret_cast<const __half2 *>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<__half2 *>(&o)[i] = __hadd2(a[i], b[i]);
    }
    return o;
}

// Two fp32 values side by side: one instruction a pair.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(r))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
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

// Largest magnitudes of packed 16-bit values, NaN if one is.
template <bool BF16>
__device__ __forceinline__ uint32_t top2(uint32_t a, uint32_t b)
{
    if (BF16) {
        const __nv_bfloat162 r = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162 *>(&a)),
                                             __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&b)));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    const __half2 r = __hmax2_nan(__habs2(*reinterpret_cast<const __half2 *>(&a)),
                                  __habs2(*reinterpret_cast<const __half2 *>(&b)));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Two fp32 values: what `hi` leaves of a sum or product is in `lo`.
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair operator+(Pair a, Pair b)
{
    const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
    const float left = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t)); // of a.hi + b.hi, exact
    return {s, __fadd_rn(__fadd_rn(a.lo, b.lo), left)};
}

// y must come out as from 64 bits: one step of fp16 in y can move a code by
// one, and a code's step is half of the values' rms in rows with a large
// column. So the sum of squares and its root are pairs.
//
// Sum of the squares of a warp's vectors, N a thread, off by about 2^-38 of
// itself, the same in all lanes. A square of 16-bit values is exact in fp32;
// added to `acc`, which starts at a power of two above all of them, it splits
// into what acc takes up and the rest, both exact. What acc took up is a whole
// number of units, the rests nearly are of smaller ones, and whole numbers are
// added over the warp by one instruction. NaN where the squares leave fp32's
// range (of bf16 values), or for infinities and NaN.
template <bool BF16, int N>
__device__ __forceinline__ Pair warp_squares(const uint4 (&h)[N])
{
    uint32_t bits = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i)
        bits = top2<BF16>(bits, top2<BF16>(top2<BF16>(h[i].x, h[i].y), top2<BF16>(h[i].z, h[i].w)));
    bits = __reduce_max_sync(0xffffffffu, max(bits & 0xFFFFu, bits >> 16));
    const float top = up2<BF16>(bits).x;
    if (bits == 0u)
        return {0.f, 0.f};
    if (!(top > 1e-12f && top < 1e15f))
        return {NAN, NAN};
    const uint32_t start_exp = (__float_as_uint(top * top) >> 23) + 3u;
    const float start = __uint_as_float(start_exp << 23), unit = __uint_as_float((start_exp - 23u) << 23);
    const float per_unit = __uint_as_float((277u - start_exp) << 23);
    float2 acc = make_float2(start, start), rest = make_float2(0.f, 0.f);
    const float2 one = make_float2(1.f, 1.f), minus = make_float2(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < N * 4; ++i) {
        const float2 u = up2<BF16>(reinterpret_cast<const uint32_t *>(h)[i]);
        const float2 next = fma2(u, u, acc);
        const float2 back = fma2(next, minus, acc); // what acc took up, negative
        rest = fma2(fma2(u, u, back), one, rest);
        acc = next;
    }
    // Of acc at most 2^25 units a component, so less than 2^31 in a warp.
    const uint32_t n = __reduce_add_sync(0xffffffffu, (uint32_t)(__float2int_rn((acc.x - start) * per_unit) +
                                                                 __float2int_rn((acc.y - start) * per_unit)));
    const float r = rest.x + rest.y;
    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(r))) >> 23;
    const uint32_t up = min(253u, 278u - most); // the rests times 2^(up - 127) are below 2^25
    const int m = __reduce_add_sync(0xffffffffu, __float2int_rn(r * __uint_as_float(up << 23)));
    const float nh = __uint2float_rn(n), nl = (float)(int)(n - (uint32_t)nh);
    return {nh * unit, fmaf(nl, unit, (float)m * __uint_as_float((254u - up) << 23))};
}

// 1 / sqrt(mean + eps) as hi + lo, off by about 2^-40 of itself; `far`: where the
// fp32 steps that use it could leave fp32's range, only `r` counts.
struct RowScale {
    float hi, lo;
    bool far;
    double r;
};

// One Newton step from fp32's root, with its error term as a pair.
__device__ __forceinline__ RowScale row_scale(Pair sum, Pair inv_cols, float eps)
{
    const float mean = __fmul_rn(sum.hi, inv_cols.hi);
    const float left = __fmaf_rn(sum.hi, inv_cols.hi, -mean);
    Pair m = Pair{mean, __fadd_rn(left, __fmaf_rn(sum.hi, inv_cols.lo, __fmul_rn(sum.lo, inv_cols.hi)))} +
             Pair{eps, 0.f};
    const float whole = __fadd_rn(m.hi, m.lo); // m.lo may reach 2^-14 of m.hi
    m = {whole, __fsub_rn(m.lo, __fsub_rn(whole, m.hi))};
    const float r = rsqrtf(m.hi), q = __fmul_rn(r, r), ql = __fmaf_rn(r, r, -q);
    const float p = __fmul_rn(m.hi, q), pl = __fmaf_rn(m.hi, q, -p);
    const float e = __fsub_rn(__fsub_rn(__fsub_rn(1.f, p), pl), __fmaf_rn(m.hi, ql, __fmul_rn(m.lo, q)));
    const float add = __fmul_rn(__fmul_rn(r, e), __fmaf_rn(0.375f, e, 0.5f));
    const float hi = __uint_as_float(__float_as_uint(r) - 8u); // so that lo is above 0
    return {hi, __fadd_rn(__fsub_rn(r, hi), add), !(m.hi > 1e-18f && m.hi < 1e18f), 0.0};
}

template <bool BF16>
__device__ __noinline__ double squares_far(const uint4 h)
{
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = up2<BF16>(reinterpret_cast<const uint32_t *>(&h)[i]);
        sum += (double)u.x * u.x + (double)u.y * u.y;
    }
    return sum;
}

template <bool BF16>
__device__ __noinline__ uint4 norm8_far(const uint4 h, const uint4 w, double r)
{
    uint4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = up2<BF16>(reinterpret_cast<const uint32_t *>(&h)[i]);
        const float2 b = up2<BF16>(reinterpret_cast<const uint32_t *>(&w)[i]);
        reinterpret_cast<uint32_t *>(&o)[i] = down2<false>((float)((double)a.x * r * b.x), (float)((double)a.y * r * b.y));
    }
    return o;
}

// y = h * w / sqrt(mean(h^2) + eps), rounded to fp32 and then to fp16. The
// product of two 16-bit values is exact in fp32 (at most 22 significant bits);
// the second of its products with hi and lo is far below the first and the sum
// is rounded once. An infinite product (of an infinite weight, or bf16 values)
// stays one, as lo is above 0.
template <bool BF16>
__device__ __forceinline__ uint4 norm8(const uint4 &h, const uint4 &w, const RowScale &s)
{
    const uint32_t *a = reinterpret_cast<const uint32_t *>(&h), *b = reinterpret_cast<const uint32_t *>(&w);
    const float2 hi = make_float2(s.hi, s.hi), lo = make_float2(s.lo, s.lo);
    uint4 o;
    uint32_t *p = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 g = mul2(up2<BF16>(a[i]), up2<BF16>(b[i]));
        const float2 y = fma2(g, hi, mul2(g, lo));
        p[i] = down2<false>(y.x, y.y);
    }
    return o;
}

// Of the block's warps, each lane one; lanes that are left over take one again
// or `none`, so that all get the result.
template <typename T, typename F>
__device__ __forceinline__ T over_warps(T v, T *s, int nwarps, T none, F join)
{
    if (nwarps == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        s[threadIdx.x >> 5] = v;
    __syncthreads();
    const int all = 1 << (32 - __clz(nwarps - 1)), from = threadIdx.x & (all - 1);
    v = from < nwarps ? s[from] : none;
    for (int o = 1; o < all; o <<= 1)
        v = join(v, o);
    return v;
}

// Maximum of magnitudes, and sums, over the CTA, the same value in every thread.
// `s` holds one value a warp; two buffers used in turn need no barrier between
// uses.
__device__ __forceinline__ float warp_max(float v)
{
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(v, 0.f))));
}

__device__ __forceinline__ float block_max(float v, float *s, int nwarps)
{
    v = warp_max(v);
    if (nwarps == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        s[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_max(lane < nwarps ? s[lane] : 0.f);
}

__device__ __forceinline__ Pair block_sum(Pair v, Pair *s, int nwarps)
{
    return over_warps(v, s, nwarps, Pair{0.f, 0.f}, [](Pair a, int o) {
        return a + Pair{__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
    });
}

__device__ __noinline__ double block_sum_far(double v, double *s, int nwarps)
{
    auto join = [](double a, int o) { return a + __shfl_xor_sync(0xffffffffu, a, o); };
    for (int o = 1; o < 32; o <<= 1)
        v = join(v, o);
    return over_warps(v, s, nwarps, 0.0, join);
}

// What a row's values are multiplied with before they are rounded to codes:
// 127 / absmax, as in quantize_rowwise. Where the codes are all that is asked
// for (no Y that a quantizer could be given) it is 127 * (1 / absmax), what
// torch's `127.0 / absmax` gives; the two part where a value lies exactly
// between two codes (2048 x 4096: 24 to 87 of 8.4 million codes).
__device__ __forceinline__ float code_multiplier(float amax, bool codes_only)
{
    if (!(amax > 0.f))
        return 0.f;
    return codes_only ? __fmul_rn(127.0f, __frcp_rn(amax)) : __fdiv_rn(127.0f, amax);
}

struct NormParams {
    const uint4 *x, *res, *w;
    uint4 *h, *y; // null: not stored
    uint2 *codes;
    float *absmax;
    int64_t rows;
    int cols;
    float eps;
    Pair inv_cols;
    __half t16;
    uint32_t *sets, *calls, *sync, *grown, *bitmap_out, *status;
};

// The scale of a row that is `far`.
__device__ __noinline__ double root_far(double sum, int cols, float eps)
{
    return 1.0 / sqrt(sum / cols + eps);
}

constexpr int kListed = 1024; // outlier columns that the fix-up visits one by one

// After every CTA has added its rows' outlier columns to the set: the complete
// set into shared memory, the first kListed of its columns listed; CTA 0 also
// writes it out, clears the other set for the next call and moves the call
// counter on (everyone read it before the barrier). Returns the set's size,
// or -1 if the barrier ran out.
__device__ __forceinline__ int complete_set(const NormParams &p, uint32_t call, uint32_t *s_set, int *s_col)
{
    __shared__ int s_count;
    const int nwords = (p.cols + 31) >> 5, tid = threadIdx.x;
    __threadfence();
    __syncthreads();
    if (tid == 0)
        s_count = grid_barrier(p.sync, gridDim.x) ? 0 : -1 - 133143;
    __syncthreads();
    const uint32_t *set = p.sets + (call & 1u) * kSetWords;
    for (int w = tid; w < nwords; w += blockDim.x) {
        uint32_t v = __ldcg(set + w);
        s_set[w] = v;
        if (blockIdx.x == 0)
            p.bitmap_out[w] = v;
        while (v) {
            const int b = __ffs(v) - 1;
            v &= v - 1u;
            const int at = atomicAdd(&s_count, 1);
            if (at >= 0 && at < kListed)
                s_col[at] = w * 32 + b;
        }
    }
    if (blockIdx.x == 0) {
        uint32_t *next = p.sets + ((call + 1u) & 1u) * kSetWords;
        for (int w = tid; w < (int)kSetWords; w += blockDim.x)
            next[w] = 0u;
        if (tid == 0)
            *reinterpret_cast<volatile uint32_t *>(p.calls) = call + 1u;
    }
    __syncthreads();
    const int count = s_count;
    if (count < 0 && tid == 0)
        atomicOr(p.status, LLMINT8_DEV_TIMEOUT_QUANT);
    return count;
}

// Outlier columns of a vector into the set; a column that is new to it moves
// the growth counter on (after the set: who reads the counter and then the set
// sees the column).
__device__ __forceinline__ void add_hits(const NormParams &p, uint32_t *set, int c, uint32_t hit)
{
    const uint32_t bits = hit << ((c & 3) * 8);
    if ((atomicOr(set + (c >> 2), bits) & bits) != bits) {
        __threadfence();
        atomicAdd(p.grown, 1u);
    }
}

// Rows first, first + gridDim.x, .. < end of this CTA were coded before the
// set was complete. Their codes in the set's columns become 0, and a row whose
// absmax was attained in one of them is coded again, by the whole CTA. All
// other codes stand: a row's absmax and codes depend on the set only through
// those columns. A warp looks at a row's listed columns.
__device__ __forceinline__ void fix_rows(const NormParams &p, int64_t first, int64_t end, int count,
                                         const uint32_t *s_set, const int *s_col, float *s_max)
{
    __shared__ int s_stale[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5, nvec = p.cols >> 3;
    const float t = __half2float(p.t16);
    for (int64_t r0 = first; r0 < end; r0 += (int64_t)nwarps * gridDim.x) {
        const int64_t mine = r0 + (int64_t)warp * gridDim.x;
        if (mine < end) {
            const __half *Y = reinterpret_cast<const __half *>(p.y) + mine * p.cols;
            int8_t *codes = reinterpret_cast<int8_t *>(p.codes) + mine * p.cols;
            const float old = p.absmax[mine];
            bool stale = count > kListed;
            if (!stale)
                for (int i = lane; i < count; i += 32) {
                    const int c = s_col[i];
                    const float a = fabsf(__half2float(Y[c]));
                    if (a < t && codes[c] != 0) {
                        codes[c] = 0;
                        stale |= a == old;
                    }
                }
            stale = __any_sync(0xffffffffu, stale);
            if (lane == 0)
                s_stale[warp] = stale;
        }
        __syncthreads();
        for (int w = 0; w < nwarps; ++w) {
            const int64_t r = r0 + (int64_t)w * gridDim.x;
            if (r >= end || !s_stale[w])
                continue;
            const uint4 *yr = p.y + r * nvec;
            __half2 m2 = __float2half2_rn(0.f);
            for (int c = tid; c < nvec; c += blockDim.x) {
                uint4 v = yr[c];
                mask_known(v, (s_set[c >> 2] >> ((c & 3) * 8)) & 0xFFu);
                __half2 a[4];
                m2 = __hmax2(m2, vec_abs_max(v, a));
            }
            const float amax = block_max(fmaxf(__low2float(m2), __high2float(m2)), s_max, nwarps);
            const float s = code_multiplier(amax, false);
            for (int c = tid; c < nvec; c += blockDim.x) {
                uint4 v = yr[c];
                mask_known(v, (s_set[c >> 2] >> ((c & 3) * 8)) & 0xFFu);
                p.codes[r * nvec + c] = codes8(v, s);
            }
            if (tid == 0)
                p.absmax[r] = amax;
            __syncthreads(); // s_max is free
        }
        __syncthreads(); // and s_stale
    }
}

// One CTA per row, the row in registers from its one read to its codes. With
// THR a row is coded against the outlier columns known by then (its own and
// what earlier rows of any CTA have found); after all rows a grid barrier
// makes the set complete. The CTA's last row is still in registers and is
// coded again from there where the set has grown; with many rows the columns
// are known after the first few, so the others rarely need fix_row's work.
template <bool BF16, bool THR, int MAXT>
__global__ void __launch_bounds__(MAXT, 1024 / MAXT) k_norm_quant(const NormParams p)
{
    __shared__ float s_red[2][32];
    __shared__ Pair s_sum[32];
    __shared__ double s_far[32];
    extern __shared__ uint32_t s_dyn[]; // THR: the set, then its listed columns
    const int tid = threadIdx.x, nwarps = blockDim.x >> 5;
    const int nvec = p.cols >> 3;
    griddep_wait();
    griddep_release();
    uint32_t call = 0u, *set = nullptr;
    if (THR) {
        call = *reinterpret_cast<volatile uint32_t *>(p.calls);
        set = p.sets + (call & 1u) * kSetWords;
    }
    const __half2 t2 = __half2half2(p.t16);
    uint4 v[kVec];
    float amax = 0.f;
    uint32_t known = 0u; // outlier columns of this thread's vectors, a byte each
    uint32_t grown = 0u; // thread 0: the growth counter, and the first row that was
    int64_t since = -1;  // coded against the set it stands for
    int64_t r = blockIdx.x;
    for (int n = 0; r < p.rows; r += gridDim.x, ++n) {
        const uint4 *xr = p.x + r * nvec;
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
        // The CTA's next row on its way to L2 while this one is worked on.
        if (r + gridDim.x < p.rows)
            for (int line = tid * 8; line < nvec; line += blockDim.x * 8) {
                asm volatile("prefetch.global.L2 [%0];" ::"l"(xr + (int64_t)gridDim.x * nvec + line));
                if (p.res)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.res + (r + gridDim.x) * nvec + line));
            }
        // Most columns are found by the first rows: look often then, and later
        // now and again.
        if (THR && n > 0 && (n < 4 || (n & 7) == 0)) {
            if (tid == 0) {
                const uint32_t now = *reinterpret_cast<volatile uint32_t *>(p.grown);
                if (now != grown || since < 0) {
                    grown = now;
                    since = r;
                }
                __threadfence();
            }
            __syncthreads(); // the counter is read before the set
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int c = tid + i * blockDim.x;
                if (c < nvec)
                    known |= ((__ldcg(set + (c >> 2)) >> ((c & 3) * 8)) & 0xFFu) << (8 * i);
            }
        }
        RowScale scale = row_scale(block_sum(warp_squares<BF16>(v), s_sum, nwarps), p.inv_cols, p.eps);
        if (scale.far) { // the same in all threads
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                sum += squares_far<BF16>(v[i]);
            scale.r = root_far(block_sum_far(sum, s_far, nwarps), p.cols, p.eps);
        }
        if (p.h) {
            uint4 *hr = p.h + r * nvec;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int c = tid + i * blockDim.x;
                if (c < nvec)
                    hr[c] = v[i];
            }
        }
        if (scale.far) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int c = tid + i * blockDim.x;
                if (c < nvec)
                    v[i] = norm8_far<BF16>(v[i], __ldg(p.w + c), scale.r);
            }
        }
        __half2 m2 = __float2half2_rn(0.f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = tid + i * blockDim.x;
            if (c < nvec) {
                if (!scale.far)
                    v[i] = norm8<BF16>(v[i], __ldg(p.w + c), scale);
                if (p.y)
                    p.y[r * nvec + c] = v[i];
                __half2 a[4];
                __half2 m = vec_abs_max(v[i], a);
                if (THR) {
                    // a new column is rare, a known one in few vectors
                    if (!__hblt2(m, t2)) { // some |y| >= t
                        const uint32_t hit = hit_mask8(v[i], p.t16);
                        if (hit & ~(known >> (8 * i)))
                            add_hits(p, set, c, hit);
                        known |= hit << (8 * i);
                    }
                    if ((known >> (8 * i)) & 0xFFu) {
                        mask_known(v[i], (known >> (8 * i)) & 0xFFu);
                        m = vec_abs_max(v[i], a);
                    }
                }
                m2 = __hmax2(m2, m);
            }
        }
        amax = block_max(fmaxf(__low2float(m2), __high2float(m2)), s_red[0], nwarps);
        const float s = code_multiplier(amax, !THR && !p.y);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = tid + i * blockDim.x;
            if (c < nvec)
                p.codes[r * nvec + c] = codes8(v[i], s);
        }
        if (tid == 0)
            p.absmax[r] = amax;
    }
    if (THR) {
        uint32_t *s_set = s_dyn;
        int *s_col = reinterpret_cast<int *>(s_set + ((p.cols + 31) >> 5));
        const int count = complete_set(p, call, s_set, s_col);
        if (count <= 0)
            return;
        // The last row, from registers.
        bool more = false;
        __half2 m2 = __float2half2_rn(0.f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = tid + i * blockDim.x;
            if (c < nvec) {
                const uint4 was = v[i];
                mask_known(v[i], (s_set[c >> 2] >> ((c & 3) * 8)) & 0xFFu);
                more |= was.x != v[i].x || was.y != v[i].y || was.z != v[i].z || was.w != v[i].w;
                __half2 a[4];
                m2 = __hmax2(m2, vec_abs_max(v[i], a));
            }
        }
        r -= gridDim.x; // this CTA's last row
        if (__syncthreads_or(more)) {
            amax = block_max(fmaxf(__low2float(m2), __high2float(m2)), s_red[1], nwarps);
            const float s = code_multiplier(amax, false);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int c = tid + i * blockDim.x;
                if (c < nvec)
                    p.codes[r * nvec + c] = codes8(v[i], s);
            }
            if (tid == 0)
                p.absmax[r] = amax;
        }
        __shared__ int64_t s_since;
        if (tid == 0) // the counter no longer moves
            s_since = since >= 0 && *reinterpret_cast<volatile uint32_t *>(p.grown) == grown ? min(since, r) : r;
        __syncthreads();
        fix_rows(p, blockIdx.x, s_since, count, s_set, s_col, s_red[0]);
    }
}

// Rows wider than the registers hold: the same steps, each pass reading h (or
// x) again.
template <bool BF16, bool THR>
__global__ void __launch_bounds__(kMaxRowThreads, 1) k_norm_quant_wide(const NormParams p)
{
    __shared__ float s_red[32];
    __shared__ Pair s_sum[32];
    __shared__ double s_far[32];
    extern __shared__ uint32_t s_words[];
    const int tid = threadIdx.x, nwarps = blockDim.x >> 5;
    const int nvec = p.cols >> 3;
    griddep_wait();
    griddep_release();
    uint32_t call = 0u, *set = nullptr;
    if (THR) {
        call = *reinterpret_cast<volatile uint32_t *>(p.calls);
        set = p.sets + (call & 1u) * kSetWords;
    }
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        auto hidden = [&](int c) {
            uint4 v = p.x[r * nvec + c];
            if (p.res)
                v = add8<BF16>(v, p.res[r * nvec + c]);
            return v;
        };
        Pair squares{0.f, 0.f};
        for (int c0 = 0; c0 < nvec; c0 += blockDim.x) { // whole warps
            const uint4 h[1] = {c0 + tid < nvec ? hidden(c0 + tid) : make_uint4(0, 0, 0, 0)};
            squares = squares + warp_squares<BF16>(h);
        }
        RowScale scale = row_scale(block_sum(squares, s_sum, nwarps), p.inv_cols, p.eps);
        if (scale.far) { // the same in all threads
            double sum = 0.0;
            for (int c = tid; c < nvec; c += blockDim.x)
                sum += squares_far<BF16>(hidden(c));
            scale.r = root_far(block_sum_far(sum, s_far, nwarps), p.cols, p.eps);
        }
        auto normed = [&](const uint4 &h, int c) {
            const uint4 w = __ldg(p.w + c);
            return scale.far ? norm8_far<BF16>(h, w, scale.r) : norm8<BF16>(h, w, scale);
        };
        __half2 m2 = __float2half2_rn(0.f);
        for (int c = tid; c < nvec; c += blockDim.x) {
            uint4 v = normed(hidden(c), c);
            __half2 a[4];
            if (THR) {
                const uint32_t hit = hit_mask8(v, p.t16);
                if (hit) {
                    add_hits(p, set, c, hit);
                    mask_known(v, hit);
                }
            }
            m2 = __hmax2(m2, vec_abs_max(v, a));
        }
        const float amax = block_max(fmaxf(__low2float(m2), __high2float(m2)), s_red, nwarps);
        const float s = code_multiplier(amax, !THR && !p.y);
        // h may take the place of x or the residual: it is stored last, each
        // vector by the thread that read it.
        for (int c = tid; c < nvec; c += blockDim.x) {
            const uint4 h = hidden(c);
            uint4 v = normed(h, c);
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
    if (THR) {
        uint32_t *s_set = s_words;
        int *s_col = reinterpret_cast<int *>(s_words + ((p.cols + 31) >> 5));
        const int count = complete_set(p, call, s_set, s_col);
        if (count > 0)
            fix_rows(p, blockIdx.x, p.rows, count, s_set, s_col, s_red);
    }
}

// value = code * (absmax / 127). A thread takes four vectors of 8 codes, a CTA's
// width apart: 8-byte loads, all under way at once, and whole sectors stored. A
// vector's row is carried along, not divided for.
template <bool BF16>
__global__ void __launch_bounds__(256) k_dequant_rows(const uint2 *codes, const float *absmax, int64_t n8, int row8,
                                                      uint4 *out)
{
    griddep_wait();
    griddep_release();
    const int dr = 256 / row8, dc = 256 - dr * row8;
    for (int64_t i0 = (int64_t)blockIdx.x * 1024 + threadIdx.x; i0 < n8; i0 += (int64_t)gridDim.x * 1024) {
        int64_t row = n8 < ((int64_t)1 << 32) ? (int64_t)((uint32_t)i0 / (uint32_t)row8) : i0 / row8;
        int col = (int)(i0 - row * row8);
        uint2 c[4];
        float s[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (i0 + k * 256 < n8) {
                c[k] = __ldcs(codes + i0 + k * 256);
                s[k] = absmax[row];
            }
            row += dr;
            col += dc;
            if (col >= row8) {
                col -= row8;
                ++row;
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * 256 < n8) {
                const float m = __fdiv_rn(s[k], 127.0f);
                const uint2 a = code_values4<BF16>(c[k].x, m), b = code_values4<BF16>(c[k].y, m);
                out[i0 + k * 256] = make_uint4(a.x, a.y, b.x, b.y);
            }
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
    p.inv_cols.hi = (float)(1.0 / (double)a.cols);
    p.inv_cols.lo = (float)(1.0 / (double)a.cols - (double)p.inv_cols.hi);
    p.t16 = threshold_fp16(a.t);
    p.sets = ws.sets;
    p.calls = ws.calls;
    p.sync = ws.sync;
    p.grown = ws.grown;
    p.bitmap_out = a.bitmap;
    p.status = ws.status;
    const int nvec = p.cols >> 3;
    const int threads = std::min(kMaxRowThreads, (nvec + 32 * kVec - 1) / (32 * kVec) * 32);
    const int size = nvec > kMaxRowThreads * kVec ? 2 : threads > 512 ? 1 : 0; // wide rows; large CTAs
    using Kernel = void (*)(NormParams);
    static const Kernel kernels[3][2][2] = {
        {{k_norm_quant<false, false, 512>, k_norm_quant<false, true, 512>},
         {k_norm_quant<true, false, 512>, k_norm_quant<true, true, 512>}},
        {{k_norm_quant<false, false, kMaxRowThreads>, k_norm_quant<false, true, kMaxRowThreads>},
         {k_norm_quant<true, false, kMaxRowThreads>, k_norm_quant<true, true, kMaxRowThreads>}},
        {{k_norm_quant_wide<false, false>, k_norm_quant_wide<false, true>},
         {k_norm_quant_wide<true, false>, k_norm_quant_wide<true, true>}}};
    const Kernel kern = kernels[size][a.bf16][thr];
    // As many CTAs an SM as their registers (at most 64 a thread) leave room
    // for: the grid barrier needs them all resident.
    const int per_sm = size == 2 ? 1 : std::max(1, std::min(1024 / threads, 16));
    const size_t smem = thr ? ((size_t)(p.cols + 31) / 32 + kListed) * 4 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(a.rows, (int64_t)dev.num_sms * per_sm));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = thr && cfg.gridDim.x > 1 ? 2 : 1; // one CTA is resident anyhow
    return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_dequant_rows(const int8_t *codes, const float *absmax, int64_t rows, int64_t cols, void *out,
                                bool bf16, const DeviceInfo &dev, cudaStream_t stream)
{
    const int64_t n8 = rows * cols / 8;
    const int64_t grid = std::min<int64_t>((n8 + 1023) / 1024, (int64_t)dev.num_sms * 32);
    return launch_pdl(bf16 ? k_dequant_rows<true> : k_dequant_rows<false>, dim3((unsigned)grid), 256, 0, stream,
                      reinterpret_cast<const uint2 *>(codes), absmax, n8, (int)(cols / 8), static_cast<uint4 *>(out));
}

} // namespace llmint8
