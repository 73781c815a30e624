// paged_fp8_append.cuh -- new K/V rows quantized into a paged 8-bit cache.
//
// A page holds page_size rows of each head as e4m3 codes under one scale per
// (page, head): value = e4m3(code) * scale.  Scales are powers of two,
//   s = 2^max(-60, e),   e the smallest integer with amax <= 448 * 2^e.
// A floating-point code loses nothing by that (a wider scale only shifts its
// exponent), and when a later row of the page needs a larger scale, the codes
// already there move to it by an exact shift: only codes that leave e4m3's
// normal range (below 2^-6 of the new scale) are rounded again, by at most
// half a subnormal step, 2^-10 of the scale.
//
// Work split.  A run is a maximal stretch of consecutive tokens whose slots
// lie in one page.  One unit of W warps takes a run of one head of K or V:
// the largest finite |x| of the new rows, the scale, the old rows if the
// scale grew, the new rows.  New rows are read once and stay in registers (up
// to 16 * W rows at d = 128; longer runs read the rest again from L2).  W goes
// by the page size, so that a full page's rows are held by their unit.  A unit
// looks for the starts of its runs among `chunk` tokens; chunk is 1 while
// there are too few units to fill the GPU (a decode step) and grows to 16 (a
// prefill, where most tokens start no run).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "dev_prims.cuh"

namespace fattn {

struct AppendParams {
    const __nv_bfloat16* x[2];  // new rows of K, V: [T, H, d], token strides below
    long long stride[2];
    uint8_t* pages[2];          // [num_pages, page_size, H, d]
    float* scales[2];           // [num_pages, H]
    const long long* slots;     // [T]
    long long num_slots;        // num_pages * page_size
    int T, H, page_shift, chunk;
    long long units;
};

constexpr int kMinScaleExp = -60;

// The power-of-two scale of rows whose largest finite magnitude has these
// float bits: 448 = 1.75 * 2^8.
__device__ __forceinline__ float pow2_scale(uint32_t amax_bits) {
    int e = static_cast<int>(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = e < kMinScaleExp ? kMinScaleExp : e;
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Eight bf16 to eight codes; an infinity or a NaN becomes e4m3's NaN (x - x is
// 0 for a finite x and NaN otherwise).
__device__ __forceinline__ uint2 quantize8(const uint4& r, float inv) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = __uint_as_float(w[e] << 16), b = __uint_as_float(w[e] & 0xFFFF0000u);
        f[2 * e] = fmaf(a, inv, a - a);
        f[2 * e + 1] = fmaf(b, inv, b - b);
    }
    return make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
}

// Two codes (low byte first) as two halves: exact, e4m3 is a subset of f16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}

__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
    float2 f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float ratio) {
    const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(codes)), b = f16x2_to_float2(e4m3x2_hi_to_f16x2(codes));
    return pack_e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

template <int D, int W>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) append_paged_fp8_kernel(const AppendParams p) {
    constexpr int UNITS = W == 1 ? 4 : 1;  // units per CTA
    constexpr int LPR = D / 8;             // lanes per row, 8 elements each
    constexpr int RPS = 32 / LPR;          // rows per warp step
    constexpr int HOLD = 8;                // steps held in registers
    __shared__ uint32_t sm_amax[W];
    const int lane = threadIdx.x & 31;
    const int wu = W == 1 ? 0 : threadIdx.x >> 5;  // warp of the unit
    const long long unit = static_cast<long long>(blockIdx.x) * UNITS + (W == 1 ? threadIdx.x >> 5 : 0);
    if (unit >= p.units) return;  // the whole unit
    const int kv = static_cast<int>(unit % 2);
    const long long u2 = unit / 2;
    const int h = static_cast<int>(u2 % p.H);
    const long long t_lo = (u2 / p.H) * p.chunk;
    const long long t_hi = t_lo + p.chunk < p.T ? t_lo + p.chunk : p.T;
    const int shift = p.page_shift;
    const long long page_mask = (1LL << shift) - 1;
    const __nv_bfloat16* x = (kv ? p.x[1] : p.x[0]) + static_cast<long long>(h) * D + (lane % LPR) * 8;
    const long long stride = kv ? p.stride[1] : p.stride[0];
    uint8_t* pages = (kv ? p.pages[1] : p.pages[0]) + static_cast<long long>(h) * D + (lane % LPR) * 8;
    float* scales = (kv ? p.scales[1] : p.scales[0]) + h;
    const long long row_bytes = static_cast<long long>(p.H) * D;

    // page of a token, -1 for one that is not stored (a negative slot, or one beyond the pool)
    auto page_of = [&](long long t) -> long long {
        const long long s = __ldg(p.slots + t);
        return s >= 0 && s < p.num_slots ? s >> shift : -1;
    };
    for (long long t = t_lo; t < t_hi;) {
        const long long page = page_of(t);
        const bool start = page >= 0 && (t == 0 || page_of(t - 1) != page);
        if (!start) {
            ++t;
            continue;
        }
        // the run's end, its lowest row, and whether its slots rise by one
        long long n = 0;
        int first = 0x7fffffff;
        bool dense = true;
        for (;;) {
            const long long i = t + n + lane;
            long long s = -1;
            if (i < p.T && page_of(i) == page) s = __ldg(p.slots + i);
            const unsigned in = __ballot_sync(0xffffffffu, s >= 0);
            const int m = in == 0xffffffffu ? 32 : __ffs(~in) - 1;
            int off = lane < m ? static_cast<int>(s & page_mask) : 0x7fffffff;
            if (lane < m && n + lane > 0 && s != __ldg(p.slots + i - 1) + 1) dense = false;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const int y = __shfl_xor_sync(0xffffffffu, off, o);
                off = y < off ? y : off;
            }
            first = off < first ? off : first;
            n += m;
            if (m < 32) break;
        }
        dense = __all_sync(0xffffffffu, dense);

        const long long r0 = wu * RPS + lane / LPR;  // this lane's row in step 0
        constexpr long long RSTEP = static_cast<long long>(W) * RPS;
        uint4 hold[HOLD];
        uint32_t amax = 0;  // the largest finite magnitude, as bf16 bits
        auto take = [&](const uint4& v) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t a = w[e] & 0x7FFF7FFFu;
                a &= ~__vcmpgeu2(a, 0x7F807F80u);
                amax = __vmaxu2(amax, a);
            }
        };
#pragma unroll
        for (int i = 0; i < HOLD; ++i) {
            const long long r = r0 + i * RSTEP;
            hold[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < n) hold[i] = __ldg(reinterpret_cast<const uint4*>(x + (t + r) * stride));
        }
        // the scale before: read by every thread, written by one after the barrier below
        const float s_old = first > 0 ? scales[page * p.H] : 0.f;
#pragma unroll
        for (int i = 0; i < HOLD; ++i) take(hold[i]);
        for (long long r = r0 + HOLD * RSTEP; r < n; r += RSTEP)
            take(__ldg(reinterpret_cast<const uint4*>(x + (t + r) * stride)));
        amax = __vmaxu2(amax, amax >> 16) & 0xFFFFu;
        amax = __reduce_max_sync(0xffffffffu, amax);
        if constexpr (W > 1) {
            __syncthreads();  // the previous run's reads of sm_amax
            if (lane == 0) sm_amax[wu] = amax;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < W; ++w) amax = sm_amax[w] > amax ? sm_amax[w] : amax;
        } else {
            __syncwarp();
        }
        const float s = fmaxf(s_old, pow2_scale(amax << 16));
        const float inv = __frcp_rn(s);
        if (wu == 0 && lane == 0) scales[page * p.H] = s;
        uint8_t* page_rows = pages + (page << shift) * row_bytes;
        if (first > 0 && s != s_old) {
            const float ratio = s_old * inv;
            for (long long r = r0; r < first; r += RSTEP) {
                uint2* q = reinterpret_cast<uint2*>(page_rows + r * row_bytes);
                const uint2 c = *q;
                *q = make_uint2(rescale4(c.x, ratio), rescale4(c.y, ratio));
            }
        }
        auto put = [&](long long r, const uint4& v) {
            const long long slot = __ldg(p.slots + t + r);
            if (!dense) {
                // a slot named again by a later token of the run keeps that token's row
                for (long long i = r + 1; i < n; ++i)
                    if (__ldg(p.slots + t + i) == slot) return;
            }
            *reinterpret_cast<uint2*>(page_rows + (slot & page_mask) * row_bytes) = quantize8(v, inv);
        };
#pragma unroll
        for (int i = 0; i < HOLD; ++i) {
            const long long r = r0 + i * RSTEP;
            if (r < n) put(r, hold[i]);
        }
        for (long long r = r0 + HOLD * RSTEP; r < n; r += RSTEP)
            put(r, __ldg(reinterpret_cast<const uint4*>(x + (t + r) * stride)));
        t += n;
    }
}

}  // namespace fattn
