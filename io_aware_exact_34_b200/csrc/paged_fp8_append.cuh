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
// lie in one page; of every run and head the work is: the largest finite |x| of
// the new rows, the scale, the old rows if the scale grew, the new rows.  A CTA
// takes `chunk` tokens of one head of K or V and the runs that start there.
// It has a warp for every 16 rows of a page (1 to 4): where its runs are long
// they share the rows of one run after the other, where there are as many runs
// as warps (decode steps) each warp takes runs of its own.  The first 16 rows of
// a warp (d = 128) stay in registers between the two passes, the rest comes
// again from L2, 16 rows in flight at once.  17.8k tokens of 8 heads of 128 take
// 22, 23, 26, 26 and 31 us in pages of 16, 32, 64, 128 and 256 (16.7 for the
// bytes alone): what is left is the chain of a run, slots -> rows -> maximum ->
// codes, and 60 % of the issue slots.  chunk grows from 1 (a decode step, too
// few tokens to fill the GPU) to a page (a prefill, where most tokens start no
// run).
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
};

constexpr int kMinScaleExp = -60;

// The power-of-two scale of rows whose largest finite magnitude has these
// float bits: 448 = 1.75 * 2^8.
__device__ __forceinline__ float pow2_scale(uint32_t amax_bits) {
    int e = static_cast<int>(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = e < kMinScaleExp ? kMinScaleExp : e;
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Eight bf16 to eight codes.  kAll: an infinity or a NaN may be among them and
// becomes e4m3's NaN (x - x is 0 for a finite x and NaN otherwise).
template <bool kAll>
__device__ __forceinline__ uint2 quantize8(const uint4& r, float inv) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = __uint_as_float(w[e] << 16), b = __uint_as_float(w[e] & 0xFFFF0000u);
        f[2 * e] = kAll ? fmaf(a, inv, a - a) : a * inv;
        f[2 * e + 1] = kAll ? fmaf(b, inv, b - b) : b * inv;
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

template <int D, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 32 / WARPS) append_paged_fp8_kernel(const AppendParams p) {
    constexpr int LPR = D / 8;   // lanes per row, 8 elements each
    constexpr int RPS = 32 / LPR;  // rows per warp step
    constexpr int HOLD = 8;      // steps held in registers
    __shared__ uint32_t sm_amax[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // CTA = (chunk of tokens, head, K or V), K and V fastest
    const int kv = blockIdx.x & 1;
    const int h = (blockIdx.x >> 1) % p.H;
    const unsigned int T = p.T, t_lo = (blockIdx.x >> 1) / p.H * p.chunk;
    const unsigned int t_hi = T - t_lo < static_cast<unsigned int>(p.chunk) ? T : t_lo + p.chunk;
    const int shift = p.page_shift;
    const long long page_mask = (1LL << shift) - 1;
    const __nv_bfloat16* x = (kv ? p.x[1] : p.x[0]) + static_cast<long long>(h) * D + (lane % LPR) * 8;
    const long long stride = kv ? p.stride[1] : p.stride[0];
    uint8_t* pages = (kv ? p.pages[1] : p.pages[0]) + static_cast<long long>(h) * D + (lane % LPR) * 8;
    float* scales = (kv ? p.scales[1] : p.scales[0]) + h;
    const long long row_bytes = static_cast<long long>(p.H) * D;

    // One run of tokens from t (in slot0) on, by `warps` warps of which this one is `w`.
    auto do_run = [&](unsigned int t, long long slot0, int w, int warps) {
        const long long page = slot0 >> shift;
        const unsigned long long base = static_cast<unsigned long long>(page) << shift;
        // the run's end, its lowest row, and whether its slots rise by one
        int n = 0;  // at most T
        int first = static_cast<int>(slot0 & page_mask), low = first;
        bool dense = true;
        for (bool more = true; more;) {
            constexpr int AHEAD = 4;  // loads in flight: 128 tokens
            long long s[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const unsigned int i = t + n + 32 * k + lane;
                s[k] = i < T ? __ldg(p.slots + i) : -1;
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (!more) break;
                const unsigned long long off = static_cast<unsigned long long>(s[k]) - base;  // in the page, or beyond its rows
                const unsigned out = __ballot_sync(0xffffffffu, off >= (1ull << shift));
                const int m = out == 0 ? 32 : __ffs(out) - 1;
                const int row = static_cast<int>(off);
                if (lane < m) {
                    dense = dense && row == first + n + lane;
                    low = row < low ? row : low;
                }
                n += m;
                more = m == 32;
            }
        }
        dense = __all_sync(0xffffffffu, dense);
        if (!dense) first = __reduce_min_sync(0xffffffffu, low);

        const int r0 = w * RPS + lane / LPR;  // this lane's row in step 0
        const int rstep = warps * RPS;
        const __nv_bfloat16* x_row = x + static_cast<long long>(t + r0) * stride;
        const long long x_step = rstep * stride;
        uint4 hold[HOLD];
        // the largest over the lanes of the run's warps
        auto over_unit = [&](uint32_t v) {
            v = __reduce_max_sync(0xffffffffu, v);
            if (WARPS > 1 && warps > 1) {
                __syncthreads();  // the reads of the time before
                if (lane == 0) sm_amax[warp] = v;
                __syncthreads();
#pragma unroll
                for (int k = 0; k < WARPS; ++k) v = sm_amax[k] > v ? sm_amax[k] : v;
            } else {
                __syncwarp();
            }
            return v;
        };
        uint32_t amax = 0;  // the largest magnitude, as two bf16; 0x7F80 and above: not a finite number
        auto take = [&](const uint4& v) {
            amax = __vmaxu2(amax, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                           __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
        };
        auto row = [&](int r) { return __ldg(reinterpret_cast<const uint4*>(x + static_cast<long long>(t + r) * stride)); };
        auto take_finite = [&](const uint4& v) {
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = u[e] & 0x7FFFu, hi = (u[e] >> 16) & 0x7FFFu;
                amax = lo < 0x7F80u && lo > amax ? lo : amax;
                amax = hi < 0x7F80u && hi > amax ? hi : amax;
            }
        };
        // rows that will not stay in registers come first, as many at once
#pragma unroll 1
        for (int r = r0 + HOLD * rstep; r < n; r += HOLD * rstep) {
#pragma unroll
            for (int i = 0; i < HOLD; ++i) {
                hold[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r + i * rstep < n) hold[i] = row(r + i * rstep);
            }
#pragma unroll
            for (int i = 0; i < HOLD; ++i) take(hold[i]);
        }
#pragma unroll
        for (int i = 0; i < HOLD; ++i) {
            hold[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r0 + i * rstep < n) hold[i] = __ldg(reinterpret_cast<const uint4*>(x_row + i * x_step));
        }
        // the scale before: read by every thread, written by one after the barrier below
        const float s_old = first > 0 ? scales[page * p.H] : 0.f;
#pragma unroll
        for (int i = 0; i < HOLD; ++i) take(hold[i]);
        amax = over_unit((amax >> 16) > (amax & 0xFFFFu) ? amax >> 16 : amax & 0xFFFFu);
        const bool all = amax >= 0x7F80u;  // infinities or NaN among the rows: the largest finite one
        if (all) {
            amax = 0;
            for (int r = r0; r < n; r += rstep) take_finite(row(r));
            amax = over_unit(amax);
        }
        const float s = fmaxf(s_old, pow2_scale(amax << 16));
        const float inv = __frcp_rn(s);
        if (w == 0 && lane == 0) scales[page * p.H] = s;
        uint8_t* page_rows = pages + (page << shift) * row_bytes;
        if (first > 0 && s != s_old) {
            const float ratio = s_old * inv;
            for (int r = r0; r < first; r += rstep) {
                uint2* q = reinterpret_cast<uint2*>(page_rows + r * row_bytes);
                const uint2 c = *q;
                *q = make_uint2(rescale4(c.x, ratio), rescale4(c.y, ratio));
            }
        }
        auto store = [&](uint8_t* at, const uint4& v) {
            *reinterpret_cast<uint2*>(at) = all ? quantize8<true>(v, inv) : quantize8<false>(v, inv);
        };
        if (dense) {
            uint8_t* at = page_rows + (first + r0) * row_bytes;
            const long long step = rstep * row_bytes;
#pragma unroll 1
            for (int r = r0;;) {
#pragma unroll
                for (int i = 0; i < HOLD; ++i)
                    if (r + i * rstep < n) store(at + i * step, hold[i]);
                r += HOLD * rstep;
                if (r >= n) break;
                at += HOLD * step;
#pragma unroll
                for (int i = 0; i < HOLD; ++i)
                    if (r + i * rstep < n) hold[i] = row(r + i * rstep);
            }
        } else {
            for (int r = r0; r < n; r += rstep) {
                // a slot named again by a later token of the run keeps that token's row; looking only as far as the
                // next such token, all looks of a slot together pass the run once: n * page_size steps at most, not n * n
                const long long slot = __ldg(p.slots + t + r);
                bool again = false;
                for (int i = r + 1; i < n && !again; ++i) again = __ldg(p.slots + t + i) == slot;
                if (!again) store(page_rows + (slot & page_mask) * row_bytes, row(r));
            }
        }
    };

    for (unsigned int t32 = t_lo; t32 < t_hi; t32 += 32) {
        // the tokens of these 32 that start a run (the same in every warp)
        bool start = false;
        long long slot = -1;
        if (t32 + lane < t_hi) {
            // stored (not a negative slot nor one beyond the pool), and in another page than the token before
            slot = __ldg(p.slots + t32 + lane);
            start = static_cast<unsigned long long>(slot) < static_cast<unsigned long long>(p.num_slots) &&
                    (t32 + lane == 0 || (static_cast<unsigned long long>(slot ^ __ldg(p.slots + t32 + lane - 1)) >> shift) != 0);
        }
        unsigned starts = __ballot_sync(0xffffffffu, start);
        const bool own = __popc(starts) >= WARPS;
        for (int k = 0; starts != 0; starts &= starts - 1, ++k) {
            if (own && k % WARPS != warp) continue;
            const int at = __ffs(starts) - 1;
            do_run(t32 + at, __shfl_sync(0xffffffffu, slot, at), own ? 0 : warp, own ? 1 : WARPS);
        }
    }
}

}  // namespace fattn
