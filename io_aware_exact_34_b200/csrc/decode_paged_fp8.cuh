// decode_paged_fp8.cuh -- attention of few query rows per sequence over a paged
// 8-bit cache: split-KV decode, and short runs of new tokens (verification).
//
// For a kv head h and its group of g = Hq / Hkv query heads, the rows of one
// sequence are (new token i, group head j) -> row i*g + j.  With block scales
// ks, vs (one per page and kv head) and codes K, V,
//   x = scale * ks * (q . K_code),   p = 2^(x log2e),   l = sum p,
//   o = (sum p * vs * V_code) / l.
// The scale of V goes into the exponent, y = x log2e + log2 vs, and the
// running reference my follows y, not x: p' = 2^(y - my + 7) <= 2^15 goes into
// the P V product as f16, l sums p' / vs in fp32, and o = acc / l,
// lse = my + log2 l - 7.  So one exponential serves both sums, and the largest
// p * vs of the numerator always sits in f16's normal range, whatever the pages'
// scales are.  A smaller one is rounded by 2^-11 of itself down to p' = 2^-14, 2^-21
// of the largest, and by half a subnormal step below, 2^-25: 2^-32 of the largest.
// The reference moves only when some y passes it by more than 8 (as in the
// prefill kernels), which keeps reductions out of the loop.
//
// Products run on mma.sync m16n8k16 with f16 operands and fp32 accumulation:
// e4m3 is a subset of f16, so codes convert exactly; a query row is scaled by
// a power of two to a largest magnitude in [1, 2) before it becomes f16 (11
// bits against bf16's 8, so nothing is lost down to 2^-14 of the row's
// largest element); P is rounded to f16 (see above).  The key rows are the
// M operand and 8 query rows the N operand: S^T = K Q^T and O^T = V^T P^T waste
// nothing at 8 rows a group, where Q as the M operand would pay for 16.
// (mma.sync on e4m3 operands, with Q as two e4m3 terms, was measured: it is
// expanded to conversions and f16 products, 9 % more instructions.)  A decode
// step reads 2*d bytes per key and kv head and is bound by that and by the
// conversions; tcgen05 would add nothing here but the round trip through
// tensor memory.
//
// Loads: a warp takes 16 keys a step (16 divides every page, so one page and
// one pair of scales per step) through its own ring of cp.async stages in
// shared memory.  Each copy instruction covers whole rows (128 bytes to eight
// lanes): on B200 that streams 6.9 TB/s, while copies laid out like the
// fragments, half a row or a column of rows at a time, stop at 5.3 TB/s.  The
// 16-byte chunks are swizzled so that the fragment reads are free of bank
// conflicts, and the fragments need no transposition:
//   K: lane (r = lane/4, c = lane%4) reads 16 bytes of rows r and r + 8 per
//      64-byte half; the product's k index runs over d in that order, for Q too;
//   V: the lane reads D/8 bytes of rows 2c, 2c+1, 2c+8, 2c+9; PRMT pairs the
//      bytes of two rows, and a pair converts to one A register of V^T;
//   P: S^T's accumulator transposes to the B operand of O^T by movmatrix.
// Rows outside the keys that some row of the tile may see are filled with
// zeros, so stale codes there (NaN too) never reach a product.
//
// Split: a sequence's key blocks are divided evenly over at most S CTAs of 4
// warps (by the sequence's own length, not the table's width).  Where all CTAs
// fit the GPU at once, up to 8 splits are the CTAs of one thread-block cluster
// and combine their (o, lse) through distributed shared memory (one sequence of
// 4097 keys: 9.6 us in 8 splits, 11.2 through the workspace, 10.6 in 16 splits).
// Longer work goes through the workspace and a merge kernel that starts by
// programmatic launch: there the heads of one key range stand next to each
// other in the grid and read the same DRAM pages together (32 x 32768 keys: 345
// us a call, 360-390 with the splits of a head, or one split of all sequences,
// next to each other).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "dev_prims.cuh"
#include "paged_fp8_append.cuh"

namespace fattn {

constexpr int DP8_WARPS = 4;
constexpr int DP8_BLOCK = 16;       // keys per warp step
constexpr int DP8_MIN_BLOCKS = 16;   // key blocks of the smallest split: 256 keys
constexpr int DP8_ROUND_BLOCKS = 4;  // a split's blocks: as many for each warp
constexpr int DP8_MAX_CLUSTER = 8;  // splits that merge inside a cluster
constexpr float kDp8Shift = 7.f;    // p' = 2^(y - my + 7)
constexpr float kDp8Slack = 8.f;
constexpr float kMinValueScale = 8.271806125530277e-25f;  // 2^-80: smaller V scales count as this, so that sums of p' / vs stay finite

struct PagedFp8Params {
    const __nv_bfloat16* q;     // rows (token, query head) of d elements
    const uint8_t *k, *v;       // [num_pages, page_size, Hkv, d]
    const float *ks, *vs;       // [num_pages, Hkv]
    const int* block_table;     // [B, max_pages]
    const int* seqlens_k;       // [B]
    const int* cu_q;            // [B + 1], or null: one token per sequence, token b
    __nv_bfloat16* o;
    float* lse;                 // or null
    float *ws_o, *ws_lse;       // partials [row][split][d], [row][split]; rows of the output, or of the pairs that are cut
    long long lse_tok, lse_head;  // strides of lse
    int B, Hq, Hkv, g, total_q, max_q;
    int max_pages, page_shift, num_pages;
    int S, row_tiles;
    int cluster;  // the S splits are one cluster
    int causal, window_left, window_right;
    float scale_log2;
};

// One sequence: first token, tokens, keys.  Lengths stay below 2^31, so all of
// this is 32-bit arithmetic (a 64-bit division costs as much as a key block).
struct SeqSpan {
    int q0, n, len;
};

__device__ __forceinline__ SeqSpan seq_span(const PagedFp8Params& p, int b) {
    SeqSpan s;
    if (p.cu_q != nullptr) {
        auto clampi = [](int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); };
        s.q0 = clampi(__ldg(p.cu_q + b), 0, p.total_q);
        s.n = clampi(__ldg(p.cu_q + b + 1), s.q0, p.total_q) - s.q0;
    } else {
        s.q0 = b;
        s.n = 1;
    }
    const int cap = p.max_pages << p.page_shift;
    const int len = __ldg(p.seqlens_k + b);
    s.len = len < 0 ? 0 : (len > cap ? cap : len);
    return s;
}

// Keys [lo, hi) that the token i of the sequence may see; both rise with i.
__device__ __forceinline__ void key_range(const PagedFp8Params& p, const SeqSpan& s, int i, int* lo, int* hi) {
    const int pos = i + (s.len - s.n);  // at most len - 1
    const int room = s.len - 1 - pos;   // keys behind the token's own
    const int right = p.causal ? 0 : p.window_right;
    int h = s.len, l = 0;
    if (right >= 0 && right < room) h = pos + right + 1;
    if (p.window_left >= 0 && pos > p.window_left) l = pos - p.window_left;
    *lo = l;
    *hi = h > l ? h : l;
}

// The key blocks of the rows' union and this split's share.
struct SplitSpan {
    int k_lo, k_hi;   // union of the rows' keys
    int first, last;  // blocks of this split
    int active;       // splits that hold blocks
};

__device__ __forceinline__ SplitSpan split_span(const PagedFp8Params& p, const SeqSpan& s, int tok_lo, int tok_hi, int split) {
    SplitSpan r;
    int lo0, hi0, lo1, hi1;
    key_range(p, s, tok_lo, &lo0, &hi0);
    key_range(p, s, tok_hi, &lo1, &hi1);
    r.k_lo = lo0;
    r.k_hi = hi1;
    r.first = r.last = 0;
    r.active = 0;
    if (r.k_hi <= r.k_lo) return r;
    const int b0 = r.k_lo / DP8_BLOCK, b1 = (r.k_hi - 1) / DP8_BLOCK + 1;
    int per = (b1 - b0 + p.S - 1) / p.S;
    per = (per + DP8_ROUND_BLOCKS - 1) / DP8_ROUND_BLOCKS * DP8_ROUND_BLOCKS;
    per = per < DP8_MIN_BLOCKS ? DP8_MIN_BLOCKS : per;
    r.active = (b1 - b0 + per - 1) / per;
    const long long first = b0 + static_cast<long long>(split) * per;
    r.first = first < b1 ? static_cast<int>(first) : b1;
    r.last = r.first + per < b1 ? r.first + per : b1;
    return r;
}

template <int D>
struct Dp8Traits {
    static constexpr int STAGES = 3;
    static constexpr int VB = D / 8;                        // bytes of a V row per lane
    static constexpr int KV_BYTES = 2 * DP8_BLOCK * D;      // one step of one warp
    static constexpr int WARP_BYTES = STAGES * KV_BYTES;
    static constexpr int RING_BYTES = DP8_WARPS * WARP_BYTES;
    static constexpr int SCALE_BYTES = DP8_WARPS * STAGES * 8;
    static constexpr int SMEM_BYTES = RING_BYTES + SCALE_BYTES;
    static constexpr int CPR = D / 16;   // 16-byte chunks per row
    static constexpr int RPC = 32 / CPR; // rows per copy instruction
    // Place of a 16-byte chunk in a stage: rows back to back, chunks exchanged
    // inside each 128-byte line so that the eight lanes of a read phase (K: two
    // rows of four chunks; V: rows 0, 2, 4, 6 of two chunks) hit all banks.
    __device__ static __forceinline__ uint32_t k_at(int row, int chunk) {
        return D == 128 ? row * 128 + ((chunk ^ ((row & 1) << 2)) << 4) : row * 64 + (chunk << 4);
    }
    __device__ static __forceinline__ uint32_t v_at(int row, int chunk) {
        const int line = D == 128 ? row : row >> 1, pos = D == 128 ? chunk : (row & 1) * 4 + chunk;
        return DP8_BLOCK * D + line * 128 + ((pos ^ (((row >> 1) & 3) << 1)) << 4);
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds_u4(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ uint2 lds_u2(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ float2 lds_f2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}

// All threads of the cluster's CTAs that have not left.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Shared memory of the cluster's CTA `rank`, by an address of this CTA's own.
__device__ __forceinline__ uint32_t cluster_map(uint32_t a, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}

__device__ __forceinline__ float cluster_lds_f32(uint32_t a, int rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_map(a, rank)));
    return v;
}

__device__ __forceinline__ float4 cluster_lds_f4(uint32_t a, int rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_map(a, rank)));
    return v;
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// True if one of the four bytes is e4m3's NaN (0x7F with either sign).
__device__ __forceinline__ bool has_nan4(uint32_t w) { return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0; }

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The exponent of a row's largest magnitude: the row times 2^-e has it in [1, 2).
__device__ __forceinline__ int row_exponent(float amax) {
    const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
    return e < -100 ? -100 : (e > 126 ? 126 : e);
}

// CTAs that an SM holds: 48 KB of ring at d = 128, 24 KB at 64, and registers.
__host__ __device__ constexpr int dp8_resident(int d, int tile_rows, bool masked) {
    return d == 128 ? (tile_rows > 8 ? (masked ? 2 : 3) : 4) : (tile_rows > 8 ? (masked ? 3 : 4) : (masked ? 4 : 6));
}

// NT tiles of 8 query rows per CTA.  kMasked: rows of the tile may see
// different keys (more than one token per sequence).
template <int D, int NT, bool kMasked>
__global__ void __launch_bounds__(32 * DP8_WARPS, dp8_resident(D, 8 * NT, kMasked)) decode_paged_fp8_kernel(const PagedFp8Params p) {
    using T = Dp8Traits<D>;
    constexpr int ROWS = 8 * NT;
    constexpr int HALVES = D / 64;
    constexpr int MT = D / 16;  // 16-row tiles of O^T
    extern __shared__ __align__(16) uint8_t dp8_smem[];
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r8 = lane >> 2, c4 = lane & 3;

    // CTA = (sequence, split, kv head, row tile), or with the splits fastest where they are a cluster
    unsigned int x = blockIdx.x;
    int split = 0;
    if (p.cluster) {
        split = x % p.S;
        x /= p.S;
    }
    const int rt = x % p.row_tiles;
    x /= p.row_tiles;
    const int h = x % p.Hkv;
    x /= p.Hkv;
    int b = x;
    if (!p.cluster) {
        split = x % p.S;
        b = x / p.S;
    }
    const SeqSpan sq = seq_span(p, b);
    const int n_tok = sq.n < p.max_q ? sq.n : p.max_q;
    const int row0 = rt * ROWS, rows = n_tok * p.g - row0 < ROWS ? n_tok * p.g - row0 : ROWS;  // valid rows of the tile
    if (rows <= 0) return;
    const SplitSpan sp = split_span(p, sq, row0 / p.g, (row0 + rows - 1) / p.g, split);
    if (split > 0 && split >= sp.active) return;

    // element offset of a row in q and o, and its place in lse
    auto row_q = [&](int r) -> long long {
        const int i = (row0 + r) / p.g, j = (row0 + r) - i * p.g;
        return ((static_cast<long long>(sq.q0) + i) * p.Hq + static_cast<long long>(h) * p.g + j) * D;
    };
    auto row_lse = [&](int r) -> long long {
        const int i = (row0 + r) / p.g, j = (row0 + r) - i * p.g;
        return (static_cast<long long>(sq.q0) + i) * p.lse_tok + (static_cast<long long>(h) * p.g + j) * p.lse_head;
    };

    const uint32_t ring = smem_addr(dp8_smem) + warp * T::WARP_BYTES;
    const uint32_t sring = smem_addr(dp8_smem) + T::RING_BYTES + warp * T::STAGES * 8;
    const int nblk = sp.last - sp.first;
    const int nsteps = nblk <= warp ? 0 : (nblk - warp + DP8_WARPS - 1) / DP8_WARPS;
    const int shift = p.page_shift;
    const long long head_row = static_cast<long long>(p.Hkv) * D;  // bytes between a head's rows
    const int* table = p.block_table + static_cast<long long>(b) * p.max_pages;

    // keys of a step relative to the union's first; the union holds k_len keys
    const int k_len = sp.k_hi - sp.k_lo;
    const int rel_first = (sp.first + warp) * DP8_BLOCK - sp.k_lo;
    auto rel_of = [&](int i) { return rel_first + i * (DP8_WARPS * DP8_BLOCK); };
    const int page_mask = (1 << shift) - 1;
    const int key_first = (sp.first + warp) * DP8_BLOCK;  // absolute
    const int cr = lane / T::CPR, cc = lane % T::CPR;  // row and chunk of this lane in a copy
    const long long lane_off = static_cast<long long>(h) * D + cr * head_row + cc * 16;
    const uint8_t *k_lane = p.k + lane_off, *v_lane = p.v + lane_off;
    const long long copy_step = T::RPC * head_row;
    int table_lane = 0;  // lane i: the page of step 32*(issued/32) + i
    auto issue = [&](int i) {
        if ((i & 31) == 0) {
            const int mine = i + lane;
            if (mine < nsteps) {
                const int pg = __ldg(table + ((key_first + mine * (DP8_WARPS * DP8_BLOCK)) >> shift));
                table_lane = pg < 0 ? 0 : (pg >= p.num_pages ? p.num_pages - 1 : pg);
            }
        }
        if (i < nsteps) {
            const int page = __shfl_sync(0xffffffffu, table_lane, i & 31);
            const int off = (key_first + i * (DP8_WARPS * DP8_BLOCK)) & page_mask;
            const long long at = ((static_cast<long long>(page) << shift) + off) * head_row;
            const uint8_t *kp = k_lane + at, *vp = v_lane + at;
            const uint32_t slot = ring + (i % T::STAGES) * T::KV_BYTES;
            const int rel = rel_of(i);
            if (rel >= 0 && rel + DP8_BLOCK <= k_len) {
#pragma unroll
                for (int e = 0; e < DP8_BLOCK / T::RPC; ++e) {
                    cp_async16(slot + T::k_at(e * T::RPC + cr, cc), kp);
                    cp_async16(slot + T::v_at(e * T::RPC + cr, cc), vp);
                    kp += copy_step;
                    vp += copy_step;
                }
            } else {
#pragma unroll
                for (int e = 0; e < DP8_BLOCK / T::RPC; ++e) {
                    const int r = rel + e * T::RPC + cr;
                    const int bytes = r >= 0 && r < k_len ? 16 : 0;
                    cp_async16(slot + T::k_at(e * T::RPC + cr, cc), kp, bytes);
                    cp_async16(slot + T::v_at(e * T::RPC + cr, cc), vp, bytes);
                    kp += copy_step;
                    vp += copy_step;
                }
            }
            const uint32_t sslot = sring + (i % T::STAGES) * 8;
            if (lane < 2) cp_async4(sslot + 4 * lane, (lane == 0 ? p.ks : p.vs) + static_cast<long long>(page) * p.Hkv + h);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < T::STAGES - 1; ++i) issue(i);

    // Q^T fragments: column r8 of tile nt, d in the order of the K fragments
    uint32_t qf[NT][HALVES][4][2];
    float cq[NT][2];  // scale * log2e * 2^e of the rows 2*c4, 2*c4 + 1
    [[maybe_unused]] int klo[NT][2], khi[NT][2];  // keys of those rows, relative to the union's first key
    [[maybe_unused]] int full_lo = 0, full_hi = 0;  // keys every row may see, relative too
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + r8;
        uint4 raw[HALVES][2];
        float amax = 0.f;
#pragma unroll
        for (int hh = 0; hh < HALVES; ++hh)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                raw[hh][e] = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows) raw[hh][e] = __ldg(reinterpret_cast<const uint4*>(p.q + row_q(r) + hh * 64 + c4 * 16 + e * 8));
                const uint32_t w[4] = {raw[hh][e].x, raw[hh][e].y, raw[hh][e].z, raw[hh][e].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
            }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e2 = row_exponent(amax);
        const float down = amax == CUDART_INF_F ? CUDART_NAN_F : pow2f(-e2);  // a row with an infinity becomes NaN
        const float up = p.scale_log2 * pow2f(e2);
        cq[nt][0] = __shfl_sync(0xffffffffu, up, 8 * c4);
        cq[nt][1] = __shfl_sync(0xffffffffu, up, 8 * c4 + 4);
#pragma unroll
        for (int hh = 0; hh < HALVES; ++hh)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4& v = raw[hh][j >> 1];
                const uint32_t w0 = (j & 1) ? v.z : v.x, w1 = (j & 1) ? v.w : v.y;
                qf[nt][hh][j][0] = pack_f16x2(__uint_as_float(w0 << 16) * down, __uint_as_float(w0 & 0xFFFF0000u) * down);
                qf[nt][hh][j][1] = pack_f16x2(__uint_as_float(w1 << 16) * down, __uint_as_float(w1 & 0xFFFF0000u) * down);
            }
        if constexpr (kMasked) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = nt * 8 + 2 * c4 + e;
                int lo = sp.k_lo, hi = sp.k_lo;  // rows of the padding see nothing
                if (rr < rows) key_range(p, sq, (row0 + rr) / p.g, &lo, &hi);
                klo[nt][e] = lo - sp.k_lo;
                khi[nt][e] = hi - sp.k_lo;
            }
        }
    }
    if constexpr (kMasked) {
        int lo0, hi0, lo1, hi1;
        key_range(p, sq, row0 / p.g, &lo0, &hi0);
        key_range(p, sq, (row0 + rows - 1) / p.g, &lo1, &hi1);
        full_lo = lo1 - sp.k_lo;
        full_hi = hi0 - sp.k_lo;
    }

    float my[NT][2], l[NT][2], acc[NT][MT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        my[nt][0] = my[nt][1] = -CUDART_INF_F;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][i][e] = 0.f;
    }

#pragma unroll 1
    for (int i = 0; i < nsteps; ++i) {
        cp_async_wait<T::STAGES - 2>();
        __syncwarp();  // a lane reads what others copied
        issue(i + T::STAGES - 1);
        const uint32_t slot = ring + (i % T::STAGES) * T::KV_BYTES;
        const float2 sc = lds_f2(sring + (i % T::STAGES) * 8);
        const int rel = rel_of(i);

        // S^T = K Q^T
        float s[NT][2][4];  // two chains of products, summed below
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][0][e] = s[nt][1][e] = 0.f;
#pragma unroll
        for (int hh = 0; hh < HALVES; ++hh) {
            const uint4 ka = lds_u4(slot + T::k_at(r8, hh * 4 + c4)), kb = lds_u4(slot + T::k_at(r8 + 8, hh * 4 + c4));
            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a0 = e4m3x2_to_f16x2(wa[j]), a2 = e4m3x2_hi_to_f16x2(wa[j]);
                const uint32_t a1 = e4m3x2_to_f16x2(wb[j]), a3 = e4m3x2_hi_to_f16x2(wb[j]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16_16816(s[nt][j & 1], a0, a1, a2, a3, qf[nt][hh][j][0], qf[nt][hh][j][1]);
            }
        }

        // V codes of this lane's rows and columns
        uint32_t vw[4][T::VB / 4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 2 * c4 + (e & 1) + 8 * (e >> 1);
            if constexpr (D == 128) {
                const uint4 v = lds_u4(slot + T::v_at(r, r8));
                vw[e][0] = v.x, vw[e][1] = v.y, vw[e][2] = v.z, vw[e][3] = v.w;
            } else {
                const uint2 v = lds_u2(slot + T::v_at(r, r8 >> 1) + (r8 & 1) * 8);
                vw[e][0] = v.x, vw[e][1] = v.y;
            }
        }

        // y = x log2e + log2 vs, with keys a row may not see at -inf
        float y[NT][4];
        const float vs = sc.y < kMinValueScale ? kMinValueScale : sc.y;
        const float lvs = fast_log2(vs), rvs = __fdividef(1.f, vs);
        const bool whole = kMasked ? rel >= full_lo && rel + DP8_BLOCK <= full_hi : rel >= 0 && rel + DP8_BLOCK <= k_len;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[nt][e] = fmaf(s[nt][0][e] + s[nt][1][e], cq[nt][e & 1] * sc.x, lvs);
        if (!whole) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int k = rel + r8 + 8 * (e >> 1);
                    if constexpr (kMasked) {
                        if (k < klo[nt][e & 1] || k >= khi[nt][e & 1]) y[nt][e] = -CUDART_INF_F;
                    } else {
                        if (k < 0 || k >= k_len) y[nt][e] = -CUDART_INF_F;
                    }
                }
        }
        bool raise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) raise |= fmaxf(y[nt][e], y[nt][e + 2]) > my[nt][e] + kDp8Slack;
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = fmaxf(y[nt][e], y[nt][e + 2]);
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    m = fmaxf(m, my[nt][e]);
                    const float alpha = m == my[nt][e] ? 1.f : fast_exp2(my[nt][e] - m);
                    my[nt][e] = m;
                    l[nt][e] *= alpha;
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        acc[nt][t][e] *= alpha;
                        acc[nt][t][e + 2] *= alpha;
                    }
                }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float sh0 = kDp8Shift - (my[nt][0] == -CUDART_INF_F ? 0.f : my[nt][0]);
            const float sh1 = kDp8Shift - (my[nt][1] == -CUDART_INF_F ? 0.f : my[nt][1]);
            const float p0 = fast_exp2(y[nt][0] + sh0), p1 = fast_exp2(y[nt][1] + sh1);
            const float p2 = fast_exp2(y[nt][2] + sh0), p3 = fast_exp2(y[nt][3] + sh1);
            l[nt][0] = fmaf(p0 + p2, rvs, l[nt][0]);
            l[nt][1] = fmaf(p1 + p3, rvs, l[nt][1]);
            pf[nt][0] = movmatrix_trans(pack_f16x2(p0, p1));
            pf[nt][1] = movmatrix_trans(pack_f16x2(p2, p3));
        }

        if constexpr (kMasked) {
            // A NaN in a V row that some rows of the tile may not see: take it
            // out of the product and put it into the rows that see it.
            if (!whole) {
                bool bad = false;
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int w = 0; w < T::VB / 4; ++w) bad |= has_nan4(vw[e][w]);
                if (__any_sync(0xffffffffu, bad)) {
#pragma unroll
                    for (int w = 0; w < T::VB / 4; ++w)
#pragma unroll
                        for (int byte = 0; byte < 4; ++byte) {
                            unsigned keys = 0;  // keys of the step whose element w*4 + byte is NaN
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (((vw[e][w] >> (8 * byte)) & 0x7Fu) == 0x7Fu) {
                                    keys |= 1u << (2 * c4 + (e & 1) + 8 * (e >> 1));
                                    vw[e][w] &= ~(0xFFu << (8 * byte));
                                }
                            keys |= __shfl_xor_sync(0xffffffffu, keys, 1);
                            keys |= __shfl_xor_sync(0xffffffffu, keys, 2);
                            // element of this lane: 2t + e of O^T tile t
                            const int el = w * 4 + byte;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    bool seen = false;
                                    for (int k = 0; k < DP8_BLOCK; ++k)
                                        seen |= ((keys >> k) & 1u) && rel + k >= klo[nt][e] && rel + k < khi[nt][e];
                                    if (seen) acc[nt][el / 2][e + 2 * (el & 1)] = CUDART_NAN_F;
                                }
                        }
                }
            }
        }

        // O^T += V^T P^T
#pragma unroll
        for (int w = 0; w < T::VB / 4; ++w) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t sel = e == 0 ? 0x5140u : 0x7362u;
                const uint32_t lo = __byte_perm(vw[0][w], vw[1][w], sel), hi = __byte_perm(vw[2][w], vw[3][w], sel);
                const uint32_t a0 = e4m3x2_to_f16x2(lo), a1 = e4m3x2_hi_to_f16x2(lo);
                const uint32_t a2 = e4m3x2_to_f16x2(hi), a3 = e4m3x2_hi_to_f16x2(hi);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16_16816(acc[nt][2 * w + e], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
            }
        }
    }
    cp_async_wait<0>();

    // The warps' states through shared memory (the ring is free now).
    float* sm_m = reinterpret_cast<float*>(dp8_smem);           // [warp][row]
    float* sm_l = sm_m + DP8_WARPS * ROWS;                      // [warp][row]
    float* sm_acc = sm_l + DP8_WARPS * ROWS;                    // [warp][row][D + 4]
    constexpr int LD = D + 4;
    float* sm_part = sm_acc + DP8_WARPS * ROWS * LD;            // [row][D]: this split's o
    float* sm_part_lse = sm_part + ROWS * D;                    // [row]
    static_assert((DP8_WARPS * ROWS * (LD + 2) + ROWS * (D + 1)) * 4 <= T::RING_BYTES, "the warps' states fit the ring");
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float t = l[nt][e];
            t += __shfl_xor_sync(0xffffffffu, t, 4);
            t += __shfl_xor_sync(0xffffffffu, t, 8);
            t += __shfl_xor_sync(0xffffffffu, t, 16);
            const int r = nt * 8 + 2 * c4 + e;
            if (r >= rows) continue;
            if (r8 == 0) {
                sm_m[warp * ROWS + r] = my[nt][e];
                sm_l[warp * ROWS + r] = t;
            }
            float4* dst = reinterpret_cast<float4*>(sm_acc + (warp * ROWS + r) * LD + r8 * T::VB);
#pragma unroll
            for (int i = 0; i < MT / 2; ++i)
                dst[i] = make_float4(acc[nt][2 * i][e], acc[nt][2 * i][e + 2], acc[nt][2 * i + 1][e], acc[nt][2 * i + 1][e + 2]);
        }
    __syncthreads();
    // Eight elements of a row per thread.
    for (int w = threadIdx.x; w < rows * (D / 8); w += 32 * DP8_WARPS) {
        const int r = w / (D / 8), d0 = (w % (D / 8)) * 8;
        float M = -CUDART_INF_F;
        bool nan = false;
#pragma unroll
        for (int k = 0; k < DP8_WARPS; ++k) M = fmaxf(M, sm_m[k * ROWS + r]);
        float L = 0.f, f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
#pragma unroll
        for (int k = 0; k < DP8_WARPS; ++k) {
            const float mk = sm_m[k * ROWS + r], lk = sm_l[k * ROWS + r];
            // a warp whose scores are all NaN has no reference: its l is NaN
            const float wt = mk == -CUDART_INF_F ? (lk == 0.f ? 0.f : lk) : fast_exp2(mk - M);
            nan |= wt != wt;
            L = fmaf(wt, lk, L);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fmaf(wt, sm_acc[(k * ROWS + r) * LD + d0 + e], f[e]);
        }
        const bool empty = M == -CUDART_INF_F && !nan;
        const float inv = empty ? 0.f : 1.f / L;
        const float lse2 = empty ? -CUDART_INF_F : M + fast_log2(L) - kDp8Shift;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = empty ? 0.f : f[e] * inv;
        if (sp.active <= 1) {
            *reinterpret_cast<uint4*>(p.o + row_q(r) + d0) =
                make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
            if (d0 == 0 && p.lse != nullptr) p.lse[row_lse(r)] = lse2 * 0.6931471805599453f;
        } else if (p.cluster) {
            float4* dst = reinterpret_cast<float4*>(sm_part + r * D + d0);
            dst[0] = make_float4(f[0], f[1], f[2], f[3]);
            dst[1] = make_float4(f[4], f[5], f[6], f[7]);
            if (d0 == 0) sm_part_lse[r] = lse2;
        } else {
            const long long at = (row_q(r) / D) * p.S + split;
            float4* dst = reinterpret_cast<float4*>(p.ws_o + at * D + d0);
            dst[0] = make_float4(f[0], f[1], f[2], f[3]);
            dst[1] = make_float4(f[4], f[5], f[6], f[7]);
            if (d0 == 0) p.ws_lse[at] = lse2;
        }
    }
    if (sp.active <= 1 || !p.cluster) return;

    // The splits of the cluster (its first `active` CTAs; the others have left):
    // eight elements of a row per thread, the rows dealt over the CTAs.
    cluster_sync();
    const uint32_t part_s = smem_addr(sm_part), part_lse_s = smem_addr(sm_part_lse);
    for (int w = split * 32 * DP8_WARPS + threadIdx.x; w < rows * (D / 8); w += sp.active * 32 * DP8_WARPS) {
        const int r = w / (D / 8), d0 = (w % (D / 8)) * 8;
        float ls[DP8_MAX_CLUSTER], M = -CUDART_INF_F, W = 0.f, f[8];
        bool nan = false;
#pragma unroll
        for (int k = 0; k < DP8_MAX_CLUSTER; ++k) {
            ls[k] = k < sp.active ? cluster_lds_f32(part_lse_s + 4 * r, k) : -CUDART_INF_F;
            nan |= ls[k] != ls[k];
            M = fmaxf(M, ls[k]);
        }
        const float safe = M == -CUDART_INF_F ? 0.f : M;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
#pragma unroll
        for (int k = 0; k < DP8_MAX_CLUSTER; ++k) {
            if (k >= sp.active) continue;
            const float4 a = cluster_lds_f4(part_s + (r * D + d0) * 4, k), b4 = cluster_lds_f4(part_s + (r * D + d0) * 4 + 16, k);
            const float wt = fast_exp2(ls[k] - safe);
            W += wt;
            f[0] = fmaf(wt, a.x, f[0]), f[1] = fmaf(wt, a.y, f[1]), f[2] = fmaf(wt, a.z, f[2]), f[3] = fmaf(wt, a.w, f[3]);
            f[4] = fmaf(wt, b4.x, f[4]), f[5] = fmaf(wt, b4.y, f[5]), f[6] = fmaf(wt, b4.z, f[6]), f[7] = fmaf(wt, b4.w, f[7]);
        }
        const bool empty = M == -CUDART_INF_F && !nan;
        const float inv = empty ? 0.f : 1.f / W;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= inv;
        *reinterpret_cast<uint4*>(p.o + row_q(r) + d0) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        if (d0 == 0 && p.lse != nullptr) p.lse[row_lse(r)] = empty ? -CUDART_INF_F : (M + fast_log2(W)) * 0.6931471805599453f;
    }
    cluster_sync();  // nobody leaves while its part may still be read
}

// One warp: the row of packed token tok and query head hq from its `active` partial (o, lse) pairs, those of the workspace's row
// ws_row, which has room for `stride` of them.  kMany: more than 64 of them may be active (for one variant of both, 16 x 5 drafted tokens take 23.8 us instead of 23.4).
template <int D, bool kMany>
__device__ __forceinline__ void merge_row(const PagedFp8Params& p, long long tok, int hq, long long ws_row, int active, int stride) {
    constexpr int EPL = D / 32;  // elements per lane
    const int lane = threadIdx.x & 31;
    const long long r = tok * p.Hq + hq;
    const float* ls = p.ws_lse + ws_row * stride;
    // lane s holds the lse of parts s and s + 32
    const float x0 = lane < active ? ls[lane] : -CUDART_INF_F, x1 = lane + 32 < active ? ls[lane + 32] : -CUDART_INF_F;
    float M = fmaxf(x0, x1);
    bool nan = x0 != x0 || x1 != x1;
    if constexpr (kMany) {
        for (int s = 64 + lane; s < active; s += 32) {
            M = fmaxf(M, ls[s]);
            nan |= ls[s] != ls[s];
        }
    }
    nan = __any_sync(0xffffffffu, nan);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float safe = M == -CUDART_INF_F ? 0.f : M;
    const float w0 = fast_exp2(x0 - safe), w1 = fast_exp2(x1 - safe);
    float W = 0.f, f[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) f[e] = 0.f;
    const float* src = p.ws_o + ws_row * stride * D + lane * EPL;
    auto add = [&](float wt, bool some) {
        W += wt;
        // a part without a key of this row may not have written its o
        if constexpr (EPL == 4) {
            const float4 v = some ? *reinterpret_cast<const float4*>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
            f[0] = fmaf(wt, v.x, f[0]), f[1] = fmaf(wt, v.y, f[1]), f[2] = fmaf(wt, v.z, f[2]), f[3] = fmaf(wt, v.w, f[3]);
        } else {
            const float2 v = some ? *reinterpret_cast<const float2*>(src) : make_float2(0.f, 0.f);
            f[0] = fmaf(wt, v.x, f[0]), f[1] = fmaf(wt, v.y, f[1]);
        }
        src += D;
    };
    const int held = kMany && active > 64 ? 64 : active;
#pragma unroll 8
    for (int s = 0; s < held; ++s)
        add(__shfl_sync(0xffffffffu, s < 32 ? w0 : w1, s & 31), __shfl_sync(0xffffffffu, s < 32 ? x0 : x1, s & 31) != -CUDART_INF_F);
    if constexpr (kMany) {
#pragma unroll 1
        for (int s = 64; s < active; ++s) add(fast_exp2(ls[s] - safe), ls[s] != -CUDART_INF_F);
    }
    const bool empty = M == -CUDART_INF_F && !nan;
    const float inv = empty ? 0.f : 1.f / W;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + r * D + lane * EPL);
    dst[0] = pack_bf16x2(f[0] * inv, f[1] * inv);
    if constexpr (EPL == 4) dst[1] = pack_bf16x2(f[2] * inv, f[3] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[tok * p.lse_tok + static_cast<long long>(hq) * p.lse_head] =
            empty ? -CUDART_INF_F : (M + fast_log2(W)) * 0.6931471805599453f;
}

// One row (token, query head) per warp: merge its splits.
template <int D, bool kMany>
__global__ void __launch_bounds__(128) merge_paged_fp8_kernel(const PagedFp8Params p, int tile_rows) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const unsigned item = blockIdx.x * 4 + (threadIdx.x >> 5), per_seq = p.max_q * p.Hq;
    const int b = item / per_seq, w = item - b * per_seq;
    if (b >= p.B) return;
    const SeqSpan sq = seq_span(p, b);
    const int i = w / p.Hq, hq = w - i * p.Hq;
    const int n_tok = sq.n < p.max_q ? sq.n : p.max_q;
    if (i >= n_tok) return;
    // the tile of this row, whose union of keys was split
    const int row = i * p.g + hq % p.g;
    const int row0 = row / tile_rows * tile_rows;
    const int rows = n_tok * p.g - row0 < tile_rows ? n_tok * p.g - row0 : tile_rows;
    const SplitSpan sp = split_span(p, sq, row0 / p.g, (row0 + rows - 1) / p.g, 0);
    const long long tok = static_cast<long long>(sq.q0) + i;
    if (sp.active > 1) merge_row<D, kMany>(p, tok, hq, tok * p.Hq + hq, sp.active, p.S);  // else written by the split kernel
}

}  // namespace fattn
