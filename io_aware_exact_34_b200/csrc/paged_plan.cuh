// paged_plan.cuh -- block tables and slot maps of a paged KV cache, built on
// the GPU from the requests' lengths.
//
// With cu = prefix sums of the new token counts, token t of the packed batch
// belongs to the sequence b with cu[b] <= t < cu[b+1], sits at position
// pos = seqlens_k[b] + t - cu[b] and in logical page pos / page_size.  Pages
// below ceil(seqlens_k[b] / page_size) are there already (the last one may be
// partly filled); the others are taken from the free list in the order of the
// sequences: sequence b takes them from free_pages[taken[b]] on, taken = prefix
// sums of the pages each sequence needs.
//
// The work is a few bytes a token, so latency decides: one launch, no
// communication between CTAs.  Every CTA scans all sequences' counts into
// shared memory by itself (B <= 16384: two 4-byte sums each), then maps its
// 1024 tokens by binary search.  The token at offset 0 of a new page writes
// that page's table entry; entries of pages held before are only read, so no
// entry is both read and written in one launch.
#pragma once

#include <stdint.h>

namespace fattn {

constexpr int PLAN_MAX_SEQ = 16384;
constexpr int PLAN_THREADS = 256;
constexpr int PLAN_TOKENS = 1024;  // tokens per CTA

struct PlanParams {
    const int* seqlens_k;    // [B]
    const int* seqlens_new;  // [B]
    const int* free_pages;   // [num_free]
    int* block_table;        // [B, max_pages]
    long long* slot_map;     // [max_tokens]
    int* cu_seqlens;         // [B + 1]
    int* seqlens_out;        // [B]
    int* counts;             // [2]: tokens, pages needed
    int B, max_pages, page_shift, num_free, max_tokens;
};

__device__ __forceinline__ int plan_saturate(long long x) { return x > 0x7fffffffLL ? 0x7fffffff : static_cast<int>(x); }

__global__ void __launch_bounds__(PLAN_THREADS) paged_plan_kernel(const PlanParams p) {
    extern __shared__ int plan_sm[];
    int* cu = plan_sm;                // [B + 1]
    int* taken = plan_sm + p.B + 1;   // [B + 1]
    __shared__ long long warp_tok[PLAN_THREADS / 32], warp_pag[PLAN_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = p.B, shift = p.page_shift;
    const long long page_mask = (1LL << shift) - 1;

    // Exclusive prefix sums over the sequences in 64 bits; what is kept is
    // saturated to 31 bits, beyond every capacity the indices are compared with.
    const int per = (B + PLAN_THREADS - 1) / PLAN_THREADS;
    const int b_lo = tid * per < B ? tid * per : B, b_hi = b_lo + per < B ? b_lo + per : B;
    auto counts_of = [&](int b, long long& tok, long long& pag) {
        const int len = __ldg(p.seqlens_k + b), add = __ldg(p.seqlens_new + b);
        const long long l = len > 0 ? len : 0;
        tok = add > 0 ? add : 0;
        pag = ((l + tok + page_mask) >> shift) - ((l + page_mask) >> shift);
    };
    long long tok = 0, pag = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        long long t, g;
        counts_of(b, t, g);
        tok += t;
        pag += g;
    }
    long long tok_in = tok, pag_in = pag;  // inclusive over the warp
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, tok_in, o), g = __shfl_up_sync(0xffffffffu, pag_in, o);
        if (lane >= o) {
            tok_in += t;
            pag_in += g;
        }
    }
    if (lane == 31) {
        warp_tok[warp] = tok_in;
        warp_pag[warp] = pag_in;
    }
    __syncthreads();
    long long tok_at = tok_in - tok, pag_at = pag_in - pag;
    for (int w = 0; w < warp; ++w) {
        tok_at += warp_tok[w];
        pag_at += warp_pag[w];
    }
    for (int b = b_lo; b < b_hi; ++b) {
        cu[b] = plan_saturate(tok_at);
        taken[b] = plan_saturate(pag_at);
        long long t, g;
        counts_of(b, t, g);
        tok_at += t;
        pag_at += g;
    }
    if (tid == PLAN_THREADS - 1) {
        cu[B] = plan_saturate(tok_at);
        taken[B] = plan_saturate(pag_at);
    }
    __syncthreads();

    if (blockIdx.x == 0) {
        for (int b = tid; b <= B; b += PLAN_THREADS) {
            p.cu_seqlens[b] = cu[b];
            if (b < B) {
                const int len = __ldg(p.seqlens_k + b), add = __ldg(p.seqlens_new + b);
                p.seqlens_out[b] = plan_saturate((len > 0 ? len : 0LL) + (add > 0 ? add : 0LL));
            }
        }
        if (tid == 0) {
            p.counts[0] = cu[B];
            p.counts[1] = taken[B];
        }
    }

    const long long t0 = static_cast<long long>(blockIdx.x) * PLAN_TOKENS;
#pragma unroll
    for (int i = 0; i < PLAN_TOKENS / PLAN_THREADS; ++i) {
        const long long t = t0 + i * PLAN_THREADS + tid;
        if (t >= p.max_tokens) break;
        long long slot = -1;
        if (t < cu[B]) {
            int lo = 0, hi = B - 1;  // the last b with cu[b] <= t: it has tokens
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            const int len = __ldg(p.seqlens_k + lo);
            const long long l = len > 0 ? len : 0;
            const long long pos = l + t - cu[lo];
            const long long at = pos >> shift, have = (l + page_mask) >> shift;
            if (at < p.max_pages) {
                int* entry = p.block_table + static_cast<long long>(lo) * p.max_pages + at;
                int page = -1;
                if (at >= have) {
                    const long long idx = taken[lo] + (at - have);
                    if (idx < p.num_free) {
                        page = __ldg(p.free_pages + idx);
                        if ((pos & page_mask) == 0) *entry = page;
                    }
                } else {
                    page = *entry;
                }
                if (page >= 0) slot = (static_cast<long long>(page) << shift) + (pos & page_mask);
            }
        }
        p.slot_map[t] = slot;
    }
}

}  // namespace fattn
