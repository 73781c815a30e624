// attn_paged_fp8_sm100.cuh -- attention of long runs of new tokens over a paged
// 8-bit cache (chunked prefill) on the 5th-generation tensor cores.
//
// The recurrence, the masks and the block scales are those of
// decode_paged_fp8.cuh: y = x log2e + log2 vs against a lazily moved reference
// my, p' = 2^(y - my + 7), l = sum p' / vs, o = acc / l.  The pipeline is that of
// attn_fwd_sm100.cuh (one persistent CTA per SM, a pair of 128-row tiles that
// share every K/V tile), with three differences that the cache brings:
//
//   Rows.  The g query heads of a kv head stand in one tile: row r of a tile is
//   token r / g, head r % g, so a K/V tile is loaded and converted once for all
//   of them.  A tile holds floor(128 / g) tokens.
//   S = Q K^T takes K's codes as they are (kind::f8f6f4).  A query row is split
//   into two e4m3 terms, q 2^-e = hi + lo, largest magnitude at 224 .. 448, and
//   both go through the same accumulator: 2 x 4 products of 32 elements, the
//   time of one bf16 product, with no conversion of K.  The split is exact down
//   to 2^-10 of the row's largest element, and off by at most 2^-18 of it below.
//   O += P V runs on f16 (kind::f16): p * vs keeps 11 bits down to 2^-21 of the
//   row's largest and is off by up to 2^-32 of it below (e4m3 would lose long
//   tails), V's codes convert exactly.  Two
//   warps convert each V tile once for both row tiles, from its 8-bit stage into
//   an f16 tile in the 128-byte-swizzled layout the tensor core reads.
//
//   warp 0        page lookups, TMA loads of K and V tiles (one box per page,
//                 one lane per box), the scales of the tile's 16-key blocks
//   warp 1        MMA issuer (one thread)
//   warps 2, 3    V tiles to f16; rows no query of the pair may see become zeros
//   warps 4-11    softmax, one thread per row; each thread also loads, splits
//                 and stores its own query row
//
// TMEM: S0 [0,128), S1 [128,256), O0, O1 from 256; P (f16) over its S tile.
//
// NaN in V rows that only some rows may see: in a tile with a mask the
// converter takes NaN codes out of the product and raises a flag, and the
// epilogue of that item looks the codes up and sets the columns of the rows
// that see them.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "decode_paged_fp8.cuh"
#include "dev_prims.cuh"
#include "sched.cuh"

namespace fattn {

constexpr int EXT_MIN_TILES = 4;  // key tiles of the smallest part: 512 keys

// One item: a pair of row tiles of one sequence and kv head, and a part of the
// key tiles they visit.  The loading warp works it out and hands it to the other
// roles through shared memory.
struct alignas(16) ExtItem {
    int item;                     // its number, -1: there are no more
    int b, h;
    int split, active;            // this part, and the parts that hold tiles
    int q0, n, len;               // first token, tokens and keys of the sequence
    int tok[2], tok_end[2];       // tokens of the tiles
    int lo_t[2], hi_t[2], lo, hi; // their key tiles, and the union
    int full_lo[2], full_hi[2];   // keys every row of a tile may see
    int k_lo, k_hi;               // keys that some row of the pair may see
};
constexpr int EXT_ITEM_BYTES = sizeof(ExtItem);

template <int D>
struct ExtTraits {
    static constexpr int THREADS = 384;
    static constexpr int NSTAGE = 6;                 // even: K in even slots, V in odd ones
    static constexpr int KV_BYTES = 128 * D;         // an 8-bit tile of 128 keys
    static constexpr int Q_BYTES = 2 * 128 * D;      // hi and lo of one row tile
    static constexpr int V16_BYTES = 128 * D * 2;
    static constexpr int SCALE_SLOTS = 4;
    static constexpr int SMEM_Q_OFF = 0;
    static constexpr int SMEM_V16_OFF = 2 * Q_BYTES;
    static constexpr int SMEM_RING_OFF = SMEM_V16_OFF + 2 * V16_BYTES;
    static constexpr int SMEM_SCALE_OFF = SMEM_RING_OFF + NSTAGE * KV_BYTES;  // float4 [slots][8]: ks, log2 vs, 1 / vs
    static constexpr int SMEM_BAR_OFF = SMEM_SCALE_OFF + SCALE_SLOTS * 8 * 16;
    // kv_full, kv_empty[NSTAGE]; v16_full, v16_empty, q_full, s_full, p_ready, o_full, item_full, item_empty[2];
    // sc_full, sc_empty[SCALE_SLOTS]; drain
    static constexpr int NBAR = 2 * NSTAGE + 16 + 2 * SCALE_SLOTS + 1;
    static constexpr int SMEM_ITEM_OFF = (SMEM_BAR_OFF + NBAR * 8 + 15) / 16 * 16;  // two ExtItem
    static constexpr int SMEM_MISC_OFF = SMEM_ITEM_OFF + 2 * EXT_ITEM_BYTES;
    // misc words: TMEM address, abort flag, unused[2], NaN rounds[4] (an item is dealt once every
    // role has read the item two rounds before it, so a round's entry outlives its epilogue)
    static constexpr int SMEM_BYTES = SMEM_MISC_OFF + 32 + 1024;  // + alignment slack
    static_assert(SMEM_BYTES <= 232448, "shared memory");
    // Register split as attn_fwd_sm100.cuh: 128 * 80 + 256 * 208 = 63488 <= 384 * 168.
    static constexpr uint32_t REGS_LOW = 80, REGS_HIGH = 208;
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr int KSTEPS = D / 32;  // products of 32 elements per term of Q
};

struct ExtParams {
    PagedFp8Params c;       // the cache, the rows, the mask
    unsigned int* counter;  // zeroed before the launch: the next item to deal
    int toks;               // tokens per row tile: floor(128 / g)
    int n_pairs, n_items;   // pairs of row tiles per sequence at most; items
    int n_whole;            // pairs (in the items' order) that are one item; the others are `splits` items each
    int box_rows;           // keys per TMA box: min(page_size, 128)
    int splits;             // parts that a pair's key tiles are cut into at most
    int o_vec32;            // o is 32-byte aligned: rows are written 32 bytes at a time
};

// Instruction descriptor of kind::f16 with f16 A and B (format 0), fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Matrix descriptor of 64-byte rows with 64-byte swizzle (eight rows are 512
// bytes), layout 4 in bits 61-63.
constexpr uint32_t kSdescHiSw64Sbo512 = (512u >> 4) | (1u << 14) | (4u << 29);

// Keys [lo, hi) of token i, as key_range.
__device__ __forceinline__ void ext_keys(const PagedFp8Params& c, int n, int len, int i, int* lo, int* hi) {
    const int pos = i + (len - n);
    const long long right = c.causal ? 0 : c.window_right;
    int h = len, l = 0;
    if (right >= 0 && pos + right + 1 < h) h = static_cast<int>(pos + right + 1);
    if (c.window_left >= 0 && pos > c.window_left) l = pos - c.window_left;
    *lo = l;
    *hi = h > l ? h : l;
}

__device__ __forceinline__ ExtItem ext_pair(const ExtParams& p, int b, int h, int pair, int split, int splits) {
    ExtItem it;
    it.item = 0;
    it.b = b;
    it.h = h;
    it.split = split;
    const SeqSpan sq = seq_span(p.c, b);
    it.q0 = sq.q0;
    it.n = sq.n;
    it.len = sq.len;
    // rows behind max_seqlen_q are not computed, but they count for the alignment
    const int n_tok = it.n < p.c.max_q ? it.n : p.c.max_q;
    it.lo = it.k_lo = 0x7fffffff;
    it.hi = it.k_hi = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const long long first = static_cast<long long>(2 * pair + t) * p.toks;
        it.tok[t] = first < n_tok ? static_cast<int>(first) : n_tok;
        it.tok_end[t] = first + p.toks < n_tok ? static_cast<int>(first + p.toks) : n_tok;
        it.lo_t[t] = it.hi_t[t] = it.full_lo[t] = it.full_hi[t] = 0;
        if (it.tok[t] < it.tok_end[t]) {
            int lo0, hi0, lo1, hi1;  // of the first and the last token: both ends rise with the token
            ext_keys(p.c, it.n, it.len, it.tok[t], &lo0, &hi0);
            ext_keys(p.c, it.n, it.len, it.tok_end[t] - 1, &lo1, &hi1);
            it.full_lo[t] = lo1;
            it.full_hi[t] = hi0;
            if (lo0 < hi1) {
                it.lo_t[t] = lo0 >> 7;
                it.hi_t[t] = (hi1 + 127) >> 7;
                it.lo = it.lo_t[t] < it.lo ? it.lo_t[t] : it.lo;
                it.hi = it.hi_t[t] > it.hi ? it.hi_t[t] : it.hi;
                it.k_lo = lo0 < it.k_lo ? lo0 : it.k_lo;
                it.k_hi = hi1 > it.k_hi ? hi1 : it.k_hi;
            }
        }
    }
    it.active = 0;
    if (it.lo >= it.hi) {
        it.lo = it.hi = 0;
        return it;
    }
    int per = (it.hi - it.lo + splits - 1) / splits;
    per = per < EXT_MIN_TILES ? EXT_MIN_TILES : per;
    it.active = (it.hi - it.lo + per - 1) / per;
    if (it.active > 1) {
        const int first = it.lo + split * per, last = first + per < it.hi ? first + per : it.hi;
        it.lo = first < last ? first : 0;
        it.hi = first < last ? last : 0;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            it.lo_t[t] = it.lo_t[t] > it.lo ? it.lo_t[t] : it.lo;
            it.hi_t[t] = it.hi_t[t] < it.hi ? it.hi_t[t] : it.hi;
            if (it.lo_t[t] >= it.hi_t[t]) it.lo_t[t] = it.hi_t[t] = 0;
        }
    } else if (split > 0) {
        it.lo = it.hi = it.lo_t[0] = it.hi_t[0] = it.lo_t[1] = it.hi_t[1] = 0;
    }
    return it;
}

// Pairs run through a sequence and head from its last one (the longest under
// causal masking), then the heads; the last ones are cut into parts.
__device__ __forceinline__ ExtItem ext_item(const ExtParams& p, int item) {
    int pb = item, split = 0, splits = 1;
    if (item >= p.n_whole) {
        splits = p.splits;
        pb = p.n_whole + (item - p.n_whole) / splits;
        split = (item - p.n_whole) % splits;
    }
    const int bh = pb / p.n_pairs;
    ExtItem it = ext_pair(p, bh / p.c.Hkv, bh % p.c.Hkv, p.n_pairs - 1 - pb % p.n_pairs, split, splits);
    it.item = item;
    return it;
}

// Whether some row of a tile that visits key tile j may not see all of it.
__device__ __forceinline__ bool ext_edge(const ExtItem& it, int j) {
    bool edge = false;
#pragma unroll
    for (int t = 0; t < 2; ++t)
        if (j >= it.lo_t[t] && j < it.hi_t[t]) edge |= j * 128 < it.full_lo[t] || j * 128 + 128 > it.full_hi[t];
    return edge;
}

__device__ __forceinline__ int ext_page(const PagedFp8Params& c, int b, long long key) {
    long long at = key >> c.page_shift;
    at = at < c.max_pages ? at : c.max_pages - 1;
    const int pg = __ldg(c.block_table + static_cast<long long>(b) * c.max_pages + at);
    return pg < 0 ? 0 : (pg >= c.num_pages ? c.num_pages - 1 : pg);
}

// Columns [32 ch, 32 ch + 32) in which a V row of a masked tile that this row
// may see holds a NaN code.
template <int D>
__device__ __noinline__ uint32_t ext_nan_columns(const ExtParams& p, int item, int t, int tok, int ch) {
    const ExtItem it = ext_item(p, item);
    int key_lo, key_hi;
    ext_keys(p.c, it.n, it.len, tok, &key_lo, &key_hi);
    uint32_t cols = 0;
    for (int j = it.lo_t[t]; j < it.hi_t[t]; ++j) {
        if (!ext_edge(it, j)) continue;
        for (int k = j * 128 > key_lo ? j * 128 : key_lo; k < key_hi && k < j * 128 + 128; ++k) {
            const long long row = (static_cast<long long>(ext_page(p.c, it.b, k)) << p.c.page_shift) + (k & ((1 << p.c.page_shift) - 1));
            const uint32_t* src = reinterpret_cast<const uint32_t*>(p.c.v + (row * p.c.Hkv + it.h) * D + ch * 32);
            for (int w = 0; w < 8; ++w) {
                const uint32_t v = __ldg(src + w);
                for (int e = 0; e < 4; ++e)
                    if (((v >> (8 * e)) & 0x7Fu) == 0x7Fu) cols |= 1u << (4 * w + e);
            }
        }
    }
    return cols;
}

__device__ __forceinline__ void sts_u2(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

// Two halves as hi + lo, both e4m3 (two codes in the low 16 bits).
__device__ __forceinline__ void split_f16x2(uint32_t x, uint32_t& hi, uint32_t& lo) {
    unsigned short h, l;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(x));
    const uint32_t rest = e4m3x2_to_f16x2(h);
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(rest));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(d));
    hi = h;
    lo = l;
}

// 16 codes to 16 halves, written as two 16-byte chunks.
__device__ __forceinline__ void sts_f16x16(uint32_t a0, uint32_t a1, const uint4& v) {
    sts128(a0, e4m3x2_to_f16x2(v.x), e4m3x2_hi_to_f16x2(v.x), e4m3x2_to_f16x2(v.y), e4m3x2_hi_to_f16x2(v.y));
    sts128(a1, e4m3x2_to_f16x2(v.z), e4m3x2_hi_to_f16x2(v.z), e4m3x2_to_f16x2(v.w), e4m3x2_hi_to_f16x2(v.w));
}

// The bytes of w that are not NaN codes.
__device__ __forceinline__ uint32_t drop_nan4(uint32_t w) {
    const uint32_t hit = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    return w & ~((hit >> 7) * 0xFFu);
}

template <int D>
__global__ void __launch_bounds__(384, 1)
    attn_paged_fp8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const __grid_constant__ ExtParams p) {
    using T = ExtTraits<D>;
    extern __shared__ uint8_t ext_smem_raw[];
    const uint32_t raw = smem_addr(ext_smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = ext_smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;");  // the merge, if there is one, may be set up

    const uint32_t sQ = base + T::SMEM_Q_OFF, sV16 = base + T::SMEM_V16_OFF, sRing = base + T::SMEM_RING_OFF;
    const uint32_t sScale = base + T::SMEM_SCALE_OFF;
    const uint32_t bar0 = base + T::SMEM_BAR_OFF;
    const uint32_t kv_full0 = bar0, kv_empty0 = kv_full0 + 8 * T::NSTAGE;
    const uint32_t v16_full0 = kv_empty0 + 8 * T::NSTAGE, v16_empty0 = v16_full0 + 16;
    const uint32_t q_full0 = v16_empty0 + 16, s_full0 = q_full0 + 16, p_ready0 = s_full0 + 16, o_full0 = p_ready0 + 16;
    const uint32_t item_full0 = o_full0 + 16, item_empty0 = item_full0 + 16;
    const uint32_t sc_full0 = item_empty0 + 16, sc_empty0 = sc_full0 + 8 * T::SCALE_SLOTS;
    const uint32_t drain_bar = sc_empty0 + 8 * T::SCALE_SLOTS;
    const uint32_t misc = base + T::SMEM_MISC_OFF;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(gbase + T::SMEM_MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + T::SMEM_MISC_OFF + 4);
    ExtItem* items = reinterpret_cast<ExtItem*>(gbase + T::SMEM_ITEM_OFF);
    volatile int* nan_round = reinterpret_cast<volatile int*>(gbase + T::SMEM_MISC_OFF + 16);
    int* status = &g_fattn_status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < T::NSTAGE; ++s) {
            mbar_init(kv_full0 + 8 * s, 1);
            mbar_init(kv_empty0 + 8 * s, (s & 1) ? 2 : 1);  // V: the converter warps; K: an MMA commit
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(v16_full0 + 8 * t, 2);
            mbar_init(v16_empty0 + 8 * t, 1);
            mbar_init(q_full0 + 8 * t, 4);
            mbar_init(s_full0 + 8 * t, 1);
            mbar_init(p_ready0 + 8 * t, 128);
            mbar_init(o_full0 + 8 * t, 1);
            mbar_init(item_full0 + 8 * t, 1);
            mbar_init(item_empty0 + 8 * t, 11);  // MMA thread, 2 converter and 8 softmax warps
        }
        for (int s = 0; s < T::SCALE_SLOTS; ++s) {
            mbar_init(sc_full0 + 8 * s, 1);
            mbar_init(sc_empty0 + 8 * s, 8);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        for (int e = 0; e < 4; ++e) nan_round[e] = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_holder), T::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
    auto tm_s = [&](int t) { return tmem + static_cast<uint32_t>(t) * 128u; };
    auto tm_o = [&](int t) { return tmem + 256u + static_cast<uint32_t>(t) * D; };
    // A wait of a whole warp; false once anybody gave up.
    auto warp_wait = [&](uint32_t bar, uint32_t parity) {
        const bool ok = mbar_wait(bar, parity, abort_flag, status, -6);
        return __all_sync(0xffffffffu, ok) != 0;
    };
    // The item of a round, from the loading warp's two entries (whole warps): false
    // if there are no more.
    auto next_item = [&](int round, ExtItem& it) {
        const int e = round & 1;
        if (!warp_wait(item_full0 + 8 * e, (round >> 1) & 1)) return false;
        it = items[e];
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty0 + 8 * e);
        return it.item >= 0;
    };

    if (warp < 4) {
        warpgroup_reg_lower<T::REGS_LOW>();
        if (warp == 0) {
            // -------------------------------------------------------- loads
            uint32_t ring = 0, sc = 0;
            bool ok = true;
            const int boxes = 128 / p.box_rows;  // lane i < boxes loads keys [i*box_rows, (i+1)*box_rows) of a tile
            for (int round = 0; ok; ++round) {
                // the first item by the CTA's index, further ones from the counter
                int item = blockIdx.x;
                if (round > 0) {
                    if (lane == 0) item = static_cast<int>(gridDim.x + atomicAdd(p.counter, 1u));
                    item = __shfl_sync(0xffffffffu, item, 0);
                }
                if (item >= p.n_items || item < 0) item = -1;
                const int e = round & 1;
                ExtItem it{};
                if (item >= 0) it = ext_item(p, item);
                else it.item = -1;
                if (round >= 2) {
                    ok = warp_wait(item_empty0 + 8 * e, ((round >> 1) - 1) & 1);
                    if (!ok) break;
                }
                if (lane == 0) {
                    items[e] = it;
                    mbar_arrive(item_full0 + 8 * e);
                }
                if (item < 0) break;
                if (it.lo < it.hi) {
                    // the pair's query rows on their way to L2: the heads of a token stand next to each other
                    const int toks = it.tok_end[1] - it.tok[0], lines = (p.c.g * D * 2 + 127) / 128;
                    const __nv_bfloat16* q = p.c.q + ((static_cast<long long>(it.q0) + it.tok[0]) * p.c.Hq + static_cast<long long>(it.h) * p.c.g) * D;
                    for (int x = lane; x < toks * lines; x += 32)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(q + static_cast<long long>(x / lines) * p.c.Hq * D + x % lines * 64));
                }
                // lanes 0-7: the page of their box; lanes 8-15: of their 16-key block
                const int mine = lane < 8 ? lane * p.box_rows : (lane & 7) * 16;
                int page = it.lo < it.hi && lane < 16 ? ext_page(p.c, it.b, static_cast<long long>(it.lo) * 128 + mine) : 0;
                for (int j = it.lo; j < it.hi && ok; ++j) {
                    const long long k0 = static_cast<long long>(j) * 128;
                    float ks = 0.f, vs = 0.f;
                    if (lane >= 8 && lane < 16) {
                        const long long at = static_cast<long long>(page) * p.c.Hkv + it.h;
                        ks = __ldg(p.c.ks + at);
                        vs = __ldg(p.c.vs + at);
                        if (k0 + mine >= it.k_hi || k0 + mine + 16 <= it.k_lo) ks = vs = 1.f;  // a block nobody sees
                    }
                    const int row = (page << p.c.page_shift) + static_cast<int>((k0 + mine) & ((1LL << p.c.page_shift) - 1));
                    if (j + 1 < it.hi && lane < 16) page = ext_page(p.c, it.b, k0 + 128 + mine);
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t slot = ring % T::NSTAGE, use = ring / T::NSTAGE;
                        if (use > 0) {
                            ok = warp_wait(kv_empty0 + 8 * slot, (use - 1) & 1u);
                            if (!ok) break;
                        }
                        const uint32_t fb = kv_full0 + 8 * slot;
                        if (lane == 0) mbar_arrive_expect_tx(fb, T::KV_BYTES);
                        __syncwarp();
                        if (lane < boxes)
                            tma_load_3d(sRing + slot * T::KV_BYTES + lane * p.box_rows * D, kv ? &tm_v : &tm_k, fb, 0, it.h, row);
                        __syncwarp();
                        ++ring;
                    }
                    if (!ok) break;
                    const uint32_t ss = sc % T::SCALE_SLOTS, su = sc / T::SCALE_SLOTS;
                    if (su > 0) {
                        ok = warp_wait(sc_empty0 + 8 * ss, (su - 1) & 1u);
                        if (!ok) break;
                    }
                    if (lane >= 8 && lane < 16) {
                        vs = vs < kMinValueScale ? kMinValueScale : vs;
                        sts128(sScale + (ss * 8 + (lane & 7)) * 16, __float_as_uint(ks), __float_as_uint(fast_log2(vs)),
                               __float_as_uint(__fdividef(1.f, vs)), 0u);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sc_full0 + 8 * ss);
                    ++sc;
                }
            }
            // No TMA write may still be landing in shared memory when the CTA exits.
            for (uint32_t s = 0; s < T::NSTAGE; ++s)
                if (ring > s) mbar_wait(kv_full0 + 8 * s, ((ring - 1 - s) / T::NSTAGE) & 1u, nullptr, status, -6);
        } else if (warp == 1) {
            // -------------------------------------------------------- MMA issuer
            if (lane == 0) {
                constexpr uint32_t idesc_s = idesc_e4m3_f32(128, 128, 0, 0);
                constexpr uint32_t idesc_pv = idesc_f16_f32(128, D, 0, 1);  // V: d contiguous
                uint32_t ring = 0, v16 = 0, p_cnt[2] = {0u, 0u}, q_cnt[2] = {0u, 0u};
                bool ok = true;
                for (int round = 0; ok; ++round) {
                    const int e = round & 1;
                    ok = mbar_wait(item_full0 + 8 * e, (round >> 1) & 1, abort_flag, status, -6);
                    if (!ok) break;
                    const ExtItem it = items[e];
                    mbar_arrive(item_empty0 + 8 * e);
                    if (it.item < 0) break;
                    const uint32_t ring0 = ring, v16_0 = v16;
                    bool q_seen[2] = {false, false};
                    for (int j = it.lo; j <= it.hi && it.lo < it.hi && ok; ++j) {
                        const bool haveK = j < it.hi, haveV = j > it.lo;
                        const uint32_t rK = ring0 + 2u * static_cast<uint32_t>(j - it.lo);
                        const uint32_t iV = v16_0 + static_cast<uint32_t>(j - 1 - it.lo);  // V16 tile of key tile j - 1
                        if (haveK) ok = mbar_wait(kv_full0 + 8 * (rK % T::NSTAGE), (rK / T::NSTAGE) & 1u, abort_flag, status, -6);
                        if (ok && haveV) ok = mbar_wait(v16_full0 + 8 * (iV & 1u), (iV >> 1) & 1u, abort_flag, status, -6);
                        if (!ok) break;
                        tc_fence_after_sync();
                        for (int t = 0; t < 2 && ok; ++t) {
                            if (haveV && j - 1 >= it.lo_t[t] && j - 1 < it.hi_t[t]) {
                                ok = mbar_wait(p_ready0 + 8 * t, p_cnt[t] & 1u, abort_flag, status, -6);
                                ++p_cnt[t];
                                if (!ok) break;
                                tc_fence_after_sync();
                                const bool first = j - 1 == it.lo_t[t];
                                const uint32_t v_lo = sdesc_lo(sV16 + (iV & 1u) * T::V16_BYTES, 128 * 128);
#pragma unroll
                                for (int ks = 0; ks < 8; ++ks)
                                    // 16 keys: 8 TMEM columns of P, 16 rows of 128 bytes of V
                                    mma_bf16_ts(tm_o(t), tm_s(t) + ks * 8, sdesc_from_lo(v_lo + ks * (2048 >> 4)), idesc_pv,
                                                (first && ks == 0) ? 0u : 1u);
                                if (j == it.hi_t[t]) mma_commit(o_full0 + 8 * t);
                            }
                            if (haveK && j >= it.lo_t[t] && j < it.hi_t[t]) {
                                if (!q_seen[t]) {
                                    ok = mbar_wait(q_full0 + 8 * t, q_cnt[t] & 1u, abort_flag, status, -6);
                                    ++q_cnt[t];
                                    if (!ok) break;
                                    q_seen[t] = true;
                                    tc_fence_after_sync();
                                }
                                const uint32_t k_lo = sdesc_lo(sRing + (rK % T::NSTAGE) * T::KV_BYTES, 16);
                                const uint32_t q_lo = sdesc_lo(sQ + t * T::Q_BYTES, 16);
#pragma unroll
                                for (int term = 0; term < 2; ++term)
#pragma unroll
                                    for (int ks = 0; ks < T::KSTEPS; ++ks) {
                                        // d = 128: hi and lo are tiles of their own; d = 64: the halves of a 128-byte row
                                        const uint32_t qo = (D == 128 ? term * 128 * 128 + ks * 32 : term * 64 + ks * 32) >> 4;
                                        const uint32_t k_hi = D == 128 ? kSdescHiSw128Sbo1024 : kSdescHiSw64Sbo512;
                                        mma_fp8_ss(tm_s(t), sdesc_from_lo(q_lo + qo),
                                                   (static_cast<uint64_t>(k_hi) << 32) | (k_lo + ((ks * 32) >> 4)), idesc_s,
                                                   (term | ks) ? 1u : 0u);
                                    }
                                mma_commit(s_full0 + 8 * t);
                            }
                        }
                        if (!ok) break;
                        if (haveV) mma_commit(v16_empty0 + 8 * (iV & 1u));
                        if (haveK) mma_commit(kv_empty0 + 8 * (rK % T::NSTAGE));
                    }
                    ring = ring0 + 2u * static_cast<uint32_t>(it.hi - it.lo);
                    v16 = v16_0 + static_cast<uint32_t>(it.hi - it.lo);
                }
            }
        } else {
            // -------------------------------------------------------- V to f16
            uint32_t ring = 1, v16 = 0;  // V tiles take the odd slots
            bool ok = true;
            for (int round = 0; ok; ++round) {
                ExtItem it;
                if (!next_item(round, it)) break;
                for (int j = it.lo; j < it.hi; ++j, ring += 2, ++v16) {
                    const uint32_t slot = ring % T::NSTAGE, buf = v16 & 1u;
                    ok = warp_wait(kv_full0 + 8 * slot, (ring / T::NSTAGE) & 1u);
                    if (ok && v16 >= 2) ok = warp_wait(v16_empty0 + 8 * buf, ((v16 >> 1) - 1) & 1u);
                    if (!ok) break;
                    const bool edge = ext_edge(it, j);
                    const uint32_t src = sRing + slot * T::KV_BYTES, dst = sV16 + buf * T::V16_BYTES;
                    bool nan = false;
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        const int r = half * 64 + (warp - 2) * 32 + lane;  // key row
                        const int key = j * 128 + r;
                        const bool seen = key >= it.k_lo && key < it.k_hi;
                        // 16 codes: chunk c of the row, exchanged by the TMA swizzle (128-byte rows: by row % 8, 64-byte
                        // rows: by row / 2 % 4); as f16, chunks 2c, 2c + 1 of 64-element (128-byte) columns of 128 rows
                        auto code_at = [&](int c) { return src + r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4); };
                        auto put = [&](int c, const uint4& v) {
                            const uint32_t row = dst + (c >> 2) * (128 * 128) + r * 128;
                            const int q = (2 * c) & 7;
                            sts_f16x16(row + ((q ^ (r & 7)) << 4), row + (((q + 1) ^ (r & 7)) << 4), v);
                        };
                        const uint32_t keep = seen ? 0xFFFFFFFFu : 0u;
                        uint32_t hit = 0;  // bit 7 of every byte: a NaN code
                        if (edge) {
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                const uint4 v = lds_u4(code_at(c));
                                hit |= ((v.x & 0x7F7F7F7Fu) + 0x01010101u) | ((v.y & 0x7F7F7F7Fu) + 0x01010101u) |
                                       ((v.z & 0x7F7F7F7Fu) + 0x01010101u) | ((v.w & 0x7F7F7F7Fu) + 0x01010101u);
                            }
                            hit &= 0x80808080u & keep;
                        }
                        if (!__any_sync(0xffffffffu, hit != 0)) {
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) {
                                const uint4 v = lds_u4(code_at(c));
                                put(c, make_uint4(v.x & keep, v.y & keep, v.z & keep, v.w & keep));
                            }
                        } else {
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                const uint4 v = lds_u4(code_at(c));
                                put(c, make_uint4(drop_nan4(v.x & keep), drop_nan4(v.y & keep), drop_nan4(v.z & keep), drop_nan4(v.w & keep)));
                            }
                            nan |= hit != 0;
                        }
                    }
                    if (nan) nan_round[round & 3] = round + 1;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(kv_empty0 + 8 * slot);
                        mbar_arrive(v16_full0 + 8 * buf);
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        warpgroup_reg_raise<T::REGS_HIGH>();
        const int t = (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t taddr_s = tm_s(t) + lane_off, taddr_o = tm_o(t) + lane_off;
        const uint32_t s_full = s_full0 + 8 * t, p_ready = p_ready0 + 8 * t, o_full = o_full0 + 8 * t;
        const int tok_of_row = row / p.c.g, head_of_row = row % p.c.g;
        uint32_t s_phase = 0, o_phase = 0, sc = 0;

        // One turn: take an item (its row, and its query into shared memory), finish
        // the item before (wait for its last product, write O), do the new item's
        // key tiles.  So the tensor core starts on an item's first scores during the
        // epilogue of the one before.
        bool ok = true, pending = false;
        // of the item in hand
        int item = -1, tok = 0, split = 0, active = 0, round_of = 0;
        bool valid = false, visited = false;  // a row of the problem; its tile has keys
        long long q_row = 0;                  // row (token, query head) of q and o
        float my = 0.f, l = 0.f;
        for (int round = 0; ok; ++round) {
            ExtItem it;
            const bool have = next_item(round, it);
            int n_tok = 0, lo = 0, hi = 0, full_lo = 0, full_hi = 0, key_lo = 0, key_hi = 0;
            bool n_valid = false;
            long long n_row = 0;
            float n_c = 0.f;
            if (have) {
                const int tok0 = t == 0 ? it.tok[0] : it.tok[1], tok1 = t == 0 ? it.tok_end[0] : it.tok_end[1];
                lo = t == 0 ? it.lo_t[0] : it.lo_t[1], hi = t == 0 ? it.hi_t[0] : it.hi_t[1];
                full_lo = t == 0 ? it.full_lo[0] : it.full_lo[1], full_hi = t == 0 ? it.full_hi[0] : it.full_hi[1];
                n_tok = tok0 + tok_of_row;
                n_valid = tok_of_row < p.toks && n_tok < tok1;
                if (n_valid) ext_keys(p.c, it.n, it.len, n_tok, &key_lo, &key_hi);
                n_row = (static_cast<long long>(it.q0) + n_tok) * p.c.Hq + static_cast<long long>(it.h) * p.c.g + head_of_row;
                if (lo < hi) {
                    // The warp's 32 query rows as two e4m3 terms each, RPL rows at a time with 16 bytes
                    // to a lane: whole rows per load (a thread loading its own row touches 32 lines per
                    // instruction).  The tile's products of the item before are done.
                    constexpr int LPR = D / 8, RPL = 32 / LPR;
                    const int sub = lane / LPR, v = lane % LPR;
                    int e2_mine = 0;
                    uint4 raw_q[LPR];  // all of them in flight
#pragma unroll
                    for (int k = 0; k < LPR; ++k) {
                        const long long src = __shfl_sync(0xffffffffu, n_row, k * RPL + sub);
                        const bool there = __shfl_sync(0xffffffffu, n_valid ? 1 : 0, k * RPL + sub) != 0;
                        raw_q[k] = there ? __ldg(reinterpret_cast<const uint4*>(p.c.q + src * D) + v) : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += RPL) {
                        const uint4 x = raw_q[i / RPL];
                        // the largest magnitude as bf16 bits: an infinity or a NaN is above every number
                        uint32_t ab = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
#pragma unroll
                        for (int o = LPR / 2; o > 0; o >>= 1) ab = __vmaxu2(ab, __shfl_xor_sync(0xffffffffu, ab, o));
                        ab = (ab >> 16) > (ab & 0xFFFFu) ? ab >> 16 : ab & 0xFFFFu;
                        // the row's largest magnitude <= 448 * 2^e2, e2 within [-100, 120]
                        int e2 = static_cast<int>(ab >> 7) - 127 - 8 + ((ab & 0x7Fu) > 0x60u ? 1 : 0);
                        e2 = e2 < -100 ? -100 : (e2 > 120 ? 120 : e2);
                        const float down = ab >= 0x7F80u ? CUDART_NAN_F : pow2f(-e2);  // a row that is not finite becomes NaN
                        const int e2_of = __shfl_sync(0xffffffffu, e2, (lane % RPL) * LPR);
                        if (lane / RPL == i / RPL) e2_mine = e2_of;
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                        uint32_t h8[4], l8[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            // f16 holds the scaled bf16 exactly (down to 2^-24), and so the difference
                            split_f16x2(pack_f16x2(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xFFFF0000u) * down), h8[k], l8[k]);
                        // 8 bytes of each term, in 128-byte rows swizzled by row % 8
                        const int r = quarter * 32 + i + sub;
                        const uint32_t q_base = sQ + t * T::Q_BYTES + r * 128 + (v & 1) * 8;
                        const uint32_t hi_at = q_base + (((v >> 1) ^ (r & 7)) << 4);
                        // d = 128: the terms are tiles of their own; d = 64: the halves of a row
                        const uint32_t lo_at = D == 128 ? hi_at + 128 * 128 : q_base + (((4 + (v >> 1)) ^ (r & 7)) << 4);
                        sts_u2(hi_at, h8[0] | (h8[1] << 16), h8[2] | (h8[3] << 16));
                        sts_u2(lo_at, l8[0] | (l8[1] << 16), l8[2] | (l8[3] << 16));
                    }
                    n_c = p.c.scale_log2 * pow2f(e2_mine);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(q_full0 + 8 * t);
                }
            }
            if (pending) {
                const bool part = active > 1;  // a part writes its (o, lse) to the workspace
                long long ws_row = 0;  // its place in the workspace, which has the rows of the cut pairs alone
                if (part) {
                    const int cut = static_cast<int>(static_cast<unsigned>(item - p.n_whole) / static_cast<unsigned>(p.splits));
                    ws_row = static_cast<long long>((cut * 2 + t) * p.toks * p.c.g + row) * p.splits + split;
                }
                float* lse = nullptr;
                if (p.c.lse != nullptr) lse = p.c.lse + q_row / p.c.Hq * p.c.lse_tok + q_row % p.c.Hq * p.c.lse_head;
                if (!visited) {
                    // no key for any row of this tile
                    if (valid && part) {
                        if (split < active) p.c.ws_lse[ws_row] = -CUDART_INF_F;
                    } else if (valid && split == 0) {
                        uint4* dst = reinterpret_cast<uint4*>(p.c.o + q_row * D);
#pragma unroll
                        for (int v = 0; v < D / 8; ++v) dst[v] = make_uint4(0u, 0u, 0u, 0u);
                        if (lse) *lse = -CUDART_INF_F;
                    }
                } else {
                    // O = acc / l, LSE = (my + log2 l - 7) ln 2
                    ok = warp_wait(o_full, o_phase & 1u);
                    ++o_phase;
                    if (!ok) break;
                    tc_fence_after_sync();
                    const bool empty = my == -CUDART_INF_F && l == 0.f;
                    const float inv_l = empty ? 0.f : 1.f / l;
                    const bool nan = nan_round[round_of & 3] == round_of + 1;
                    __nv_bfloat16* orow = p.c.o + q_row * D;
                    float* wrow = part ? p.c.ws_o + ws_row * D : nullptr;
#pragma unroll 1
                    for (int ch = 0; ch < D / 32; ++ch) {
                        uint32_t orr[32];
                        tmem_ld32(taddr_o + ch * 32, orr);
                        tmem_wait_ld();
                        reg_fence(orr);
                        if (valid) {
                            const uint32_t cols = nan ? ext_nan_columns<D>(p, item, t, tok, ch) : 0u;
                            float f[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(orr[e]) * inv_l;
                            if (cols != 0) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if ((cols >> e) & 1u) f[e] = CUDART_NAN_F;
                            }
                            if (part) {
#pragma unroll
                                for (int v = 0; v < 4; ++v)
                                    stg256(wrow + ch * 32 + 8 * v, __float_as_uint(f[8 * v]), __float_as_uint(f[8 * v + 1]),
                                           __float_as_uint(f[8 * v + 2]), __float_as_uint(f[8 * v + 3]), __float_as_uint(f[8 * v + 4]),
                                           __float_as_uint(f[8 * v + 5]), __float_as_uint(f[8 * v + 6]), __float_as_uint(f[8 * v + 7]));
                            } else {
                                uint32_t o16[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) o16[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
                                if (p.o_vec32) {
                                    stg256(orow + ch * 32, o16[0], o16[1], o16[2], o16[3], o16[4], o16[5], o16[6], o16[7]);
                                    stg256(orow + ch * 32 + 16, o16[8], o16[9], o16[10], o16[11], o16[12], o16[13], o16[14], o16[15]);
                                } else {
#pragma unroll
                                    for (int v = 0; v < 4; ++v)
                                        reinterpret_cast<uint4*>(orow + ch * 32)[v] = make_uint4(o16[4 * v], o16[4 * v + 1], o16[4 * v + 2], o16[4 * v + 3]);
                                }
                            }
                        }
                    }
                    if (valid) {
                        const float lse2 = empty ? -CUDART_INF_F : my + fast_log2(l) - kDp8Shift;
                        if (part) p.c.ws_lse[ws_row] = lse2;
                        else if (lse) *lse = lse2 * 0.6931471805599453f;
                    }
                    // the next item's first product overwrites O only once this tile's P is ready again,
                    // which this warp signals after the reads above
                    tc_fence_before_sync();
                }
            }
            if (!have) break;
            item = it.item, tok = n_tok, split = it.split, active = it.active, round_of = round;
            const int lo_u = it.lo, hi_u = it.hi;
            valid = n_valid, visited = lo < hi, q_row = n_row, pending = true;
            const float c_row = n_c;
            my = -CUDART_INF_F;
            l = 0.f;
            for (int j = lo_u; j < hi_u; ++j, ++sc) {
                const uint32_t ss = sc % T::SCALE_SLOTS;
                ok = warp_wait(sc_full0 + 8 * ss, (sc / T::SCALE_SLOTS) & 1u);
                if (!ok) break;
                if (j < lo || j >= hi) {
                    // a key tile of the other row tile still counts in the scale ring
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sc_empty0 + 8 * ss);
                    continue;
                }
                ok = warp_wait(s_full, s_phase & 1u);
                ++s_phase;
                if (!ok) break;
                tc_fence_after_sync();
                uint32_t sr[4][32];
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) tmem_ld32(taddr_s + q4 * 32, sr[q4]);
                tmem_wait_ld();
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) reg_fence(sr[q4]);
                const int k0 = j * 128;
                if (k0 < full_lo || k0 + 128 > full_hi) {
                    const int lo_col = key_lo - k0, hi_col = key_hi - k0;  // columns [lo_col, hi_col)
#pragma unroll
                    for (int blk = 0; blk < 8; ++blk) {
                        // most blocks of a masked tile are whole for all of a warp's rows
                        if (!__any_sync(0xffffffffu, blk * 16 < lo_col || blk * 16 + 16 > hi_col)) continue;
#pragma unroll
                        for (int c = blk * 16; c < blk * 16 + 16; ++c)
                            if (c < lo_col || c >= hi_col) sr[c >> 5][c & 31] = __float_as_uint(-CUDART_INF_F);
                    }
                }
                // the largest y, block by block
                const uint32_t sblk = sScale + ss * 128;
                float fk[8], mx = -CUDART_INF_F;
#pragma unroll
                for (int blk = 0; blk < 8; ++blk) {
                    const float2 s2 = lds_f2(sblk + blk * 16);
                    // never 0, so that a masked score stays -inf
                    fk[blk] = fmaxf(c_row * s2.x, 1e-37f);
                    float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = blk * 16 + 4 * i;
                        m0 = fmax3(m0, __uint_as_float(sr[c >> 5][c & 31]), __uint_as_float(sr[c >> 5][(c & 31) + 1]));
                        m1 = fmax3(m1, __uint_as_float(sr[c >> 5][(c & 31) + 2]), __uint_as_float(sr[c >> 5][(c & 31) + 3]));
                    }
                    mx = fmaxf(mx, fmaf(fmaxf(m0, m1), fk[blk], s2.y));
                }
                float alpha = 1.f;
                bool resc = false;
                if (mx > my + kDp8Slack) {
                    alpha = fast_exp2(my - mx);  // 0 when my is -inf
                    resc = j > lo && my != -CUDART_INF_F;
                    my = mx;
                    l *= alpha;
                }
                const float shift = kDp8Shift - (my == -CUDART_INF_F ? 0.f : my);
                uint32_t pk[2][32];
#pragma unroll
                for (int blk = 0; blk < 8; ++blk) {
                    const float4 s4 = lds128(sblk + blk * 16);  // ks, log2 vs, 1 / vs
                    const uint64_t f2 = f2_pack(fk[blk], fk[blk]);
                    const float sh = s4.y + shift;
                    const uint64_t sh2 = f2_pack(sh, sh);
                    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int c = blk * 16 + 2 * i;
                        const uint64_t y2 = f2_fma(f2_pack(__uint_as_float(sr[c >> 5][c & 31]), __uint_as_float(sr[c >> 5][(c & 31) + 1])), f2, sh2);
                        float y0, y1;
                        f2_unpack(y2, y0, y1);
                        const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
                        sum[i & 1] = f2_add(sum[i & 1], f2_pack(p0, p1));
                        pk[c >> 6][(c >> 1) & 31] = pack_f16x2(p0, p1);
                    }
                    float a, b;
                    f2_unpack(f2_add(sum[0], sum[1]), a, b);
                    l = fmaf(a + b, s4.z, l);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_empty0 + 8 * ss);
                tmem_st32(taddr_s, pk[0]);
                tmem_st32(taddr_s + 32, pk[1]);
                if (__any_sync(0xffffffffu, resc)) {
                    const float a = resc ? alpha : 1.f;
#pragma unroll 1
                    for (int ch = 0; ch < D / 32; ++ch) {
                        uint32_t orr[32];
                        tmem_ld32(taddr_o + ch * 32, orr);
                        tmem_wait_ld();
                        reg_fence(orr);
#pragma unroll
                        for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * a);
                        tmem_st32(taddr_o + ch * 32, orr);
                    }
                }
                tmem_wait_st();
                tc_fence_before_sync();
                mbar_arrive(p_ready);
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        if (lane == 0) {
            mma_commit(drain_bar);
            mbar_wait(drain_bar, 0, nullptr, status, -6);
        }
        __syncwarp();
        tmem_dealloc(tmem, T::TMEM_COLS);
    }
}

// 16 rows of a pair of row tiles per CTA, two to a warp: merge their parts.
template <int D>
__global__ void __launch_bounds__(256) merge_ext_kernel(const __grid_constant__ ExtParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int cut = blockIdx.x >> 4, pb = p.n_whole + cut;
    const int bh = pb / p.n_pairs, h = bh % p.c.Hkv;
    const ExtItem it = ext_pair(p, bh / p.c.Hkv, h, p.n_pairs - 1 - pb % p.n_pairs, 0, p.splits);
    if (it.active <= 1) return;
    const int rows = (it.tok_end[1] - it.tok[0]) * p.c.g;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = (blockIdx.x & 15) * 16 + e * 8 + (threadIdx.x >> 5);
        if (r < rows)
            merge_row<D, false>(p.c, static_cast<long long>(it.q0) + it.tok[0] + r / p.c.g, h * p.c.g + r % p.c.g,
                                static_cast<long long>(cut) * 2 * p.toks * p.c.g + r, it.active, p.splits);
    }
}

}  // namespace fattn
