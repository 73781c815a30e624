// paged_api.cuh -- C ABI of the paged 8-bit cache: plan, append, decode and
// multi-token attention (declared in include/fattn.h).  Included by
// fattn_api.cu, whose helpers it uses.
#pragma once

namespace {

bool pow2_page(int page_size) { return page_size >= 16 && (page_size & (page_size - 1)) == 0; }

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Query rows of one sequence and kv head that a CTA of the split kernel takes, 8
// or 16.  Two tiles of 8 read the keys twice (the second time from L2) but need
// half the registers: with several tokens a sequence that pays up to 32 rows (16
// sequences of up to 2048 keys, 20 rows: 24.8 us in tiles of 8, 26.9 in tiles of
// 16; 48 rows: 39.4 and 36.9).
int dp8_tile_rows(long long rows, bool masked) { return rows <= (masked ? 32 : 8) ? 8 : 16; }

constexpr long long kSms = 148;

// Splits of a sequence's keys at most; tiles = sequences x kv heads x row tiles,
// keys = the most that a row may see: the lengths are on the device, so the
// table's width stands for them (1 x 4097 keys in a table of 4128: 16.4 us from
// cold caches, in one of 131072: 17.4; 32 x 1-8192 keys: 71 and 77).
int dp8_auto_splits(long long tiles, int keys, int d, int tile_rows, bool masked) {
    // at least 256 keys to a split (the kernel keeps to that by each sequence's own length)
    const long long most = (static_cast<long long>(keys) + DP8_MIN_BLOCKS * DP8_BLOCK - 1) / (DP8_MIN_BLOCKS * DP8_BLOCK);
    const long long slots = kSms * dp8_resident(d, tile_rows, masked), room = slots / tiles;  // splits that fit the GPU at once
    long long S = 1;
    if (room >= 2 && keys <= (room < 16 ? 16384 : 8192)) {
        // one wave, merged inside clusters: 9.6 us for one sequence of 4097 keys and 8 heads (room 74), 58 for 32
        // sequences of 1-8192 keys (room 2; 61-64 in 3 to 9 splits through the workspace), 27 for 24 sequences in a
        // window of 2048 keys with 16 heads of 64 (room 2; 29-37)
        S = room < DP8_MAX_CLUSTER ? room : DP8_MAX_CLUSTER;
    } else if (room >= 8) {
        // one wave: 8192 keys, 32 rows (room 18): 18 us in 18 splits, 25 in 40
        S = room < 64 ? room : 64;
    } else {
        // One wave whole or several in parts.  A CTA's time in keys: its share and a fixed part.  The lengths may all be
        // the longest (whole waves count) or lie anywhere below it (the work balances, half a CTA's time stays over):
        // the mean of both decides, and parts past one wave pay for the workspace.  Against the fullest last wave alone:
        // 128 sequences of up to 2048 keys, 8 heads, 62 -> 56 us, all of 2048 keys 104 -> 92; 64 of up to 8192 keys
        // 114 -> 101, all of 8192 keys 171 -> 181; 40 of up to 1024 keys with 4 tokens each 25.3 -> 20.7, full 45.5 ->
        // 33.3.  32 x 32768 keys: 340-347 us at 4, 9 and 16 splits, 351-363 at 6, 7 and 12, 387 at 5.  More keys never
        // give fewer splits: of two costs, each linear in the keys, the larger S has the larger constant.
        const double fixed = tile_rows == 8 ? 200.0 : 500.0;
        double best = 0.0;
        for (int k = 1; k <= 16; ++k) {
            const double waves = static_cast<double>(tiles * k) / static_cast<double>(slots);
            const double share = static_cast<double>(keys) / k;
            const double whole = std::ceil(waves) * (fixed + share);
            const double ragged = waves <= 1.0 ? whole : waves * (fixed + 0.5 * share) + 0.5 * (fixed + share);
            const double cost = whole + ragged + (waves > 1.0 && k > 1 ? 600.0 : 0.0);
            if (k == 1 || cost < best) {
                best = cost;
                S = k;
            }
        }
    }
    S = S > most ? most : S;
    return static_cast<int>(S < 1 ? 1 : S);
}

// Of parts that go through memory.
size_t parts_bytes(long long rows, int S, int d) {
    return S <= 1 ? 0 : static_cast<size_t>(rows) * S * (static_cast<size_t>(d) + 1) * sizeof(float);
}

template <int D, int NT, bool kMasked>
int launch_dp8_kernel(const PagedFp8Params& p, unsigned grid, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(32 * DP8_WARPS);
    cfg.dynamicSmemBytes = Dp8Traits<D>::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.S;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster;
    if (cudaLaunchKernelEx(&cfg, decode_paged_fp8_kernel<D, NT, kMasked>, p) != cudaSuccess) {
        cudaGetLastError();
        return FATTN_ERR_CUDA;
    }
    return FATTN_OK;
}

// A merge kernel, set up while the kernel before it runs.
template <typename... Args>
int launch_merge(void (*kernel)(Args...), long long grid, int threads, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return FATTN_ERR_CUDA;
    }
    return FATTN_OK;
}

// Checks shared by the two attention entry points (host only).
int check_paged_fp8(const void* q, const void* k, const void* v, const float* ks, const float* vs, const int* table,
                    int max_pages, int page_size, int num_pages, const void* o, const float* lse, const int* seqlens_k,
                    int B, int Hq, int Hkv, int d, float scale) {
    if (!q || !k || !v || !ks || !vs || !table || !seqlens_k || !o) return FATTN_ERR_INVALID_ARG;
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_pages < 1 || num_pages < 1) return FATTN_ERR_INVALID_ARG;
    if (!pow2_page(page_size)) return FATTN_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return FATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FATTN_ERR_UNSUPPORTED;
    if (B > 65535 || Hq > 65535 || Hq / Hkv > 128) return FATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(max_pages) * page_size > 0x7fffff00 ||
        static_cast<long long>(num_pages) * page_size > (1LL << 40))
        return FATTN_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return FATTN_ERR_MISALIGNED;
    if (misaligned4(ks) || misaligned4(vs) || misaligned4(table) || misaligned4(seqlens_k) || (lse && misaligned4(lse)))
        return FATTN_ERR_MISALIGNED;
    return FATTN_OK;
}

// The split kernel over the rows of every sequence, and the merge.
int launch_dp8(PagedFp8Params p, int d, int num_splits, void* workspace, size_t workspace_bytes, void* stream) {
    const long long rows = static_cast<long long>(p.max_q) * p.g;
    const int tile_rows = dp8_tile_rows(rows, p.max_q > 1);
    const long long row_tiles = (rows + tile_rows - 1) / tile_rows;
    const long long tiles = static_cast<long long>(p.B) * p.Hkv * row_tiles;
    const int Lk = p.max_pages << p.page_shift;
    const bool masked = p.max_q > 1;
    int keys = Lk;
    if (p.window_left >= 0 && (p.causal || p.window_right >= 0)) {
        const long long seen = 1LL + p.window_left + (p.causal ? 0 : p.window_right);
        keys = seen < Lk ? static_cast<int>(seen) : Lk;
    }
    // fewer keys never mean more splits, so that a workspace sized without the window suffices
    p.S = num_splits > 0 ? num_splits : dp8_auto_splits(tiles, keys, d, tile_rows, masked);
    p.cluster = p.S > 1 && p.S <= DP8_MAX_CLUSTER && tiles * p.S <= kSms * dp8_resident(d, tile_rows, masked) ? 1 : 0;
    if (p.S > Lk) return FATTN_ERR_INVALID_ARG;
    if (rows > 0x7fffff00LL || tiles * p.S > 0x7fffffffLL || static_cast<long long>(p.B) * p.max_q * p.Hq > 0x7fffffffLL) return FATTN_ERR_UNSUPPORTED;
    p.row_tiles = static_cast<int>(row_tiles);
    const long long all_rows = static_cast<long long>(p.total_q) * p.Hq;
    const size_t need = parts_bytes(all_rows, p.S, d);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return FATTN_ERR_WORKSPACE;
        if (!aligned16(workspace)) return FATTN_ERR_MISALIGNED;
        p.ws_o = static_cast<float*>(workspace);
        p.ws_lse = p.ws_o + all_rows * p.S * d;
    }
    DeviceInfo di;
    int st = device_ready(&di);
    if (st != FATTN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = static_cast<unsigned>(tiles * p.S);
    if (d == 128) {
        if (tile_rows == 8) st = masked ? launch_dp8_kernel<128, 1, true>(p, grid, s) : launch_dp8_kernel<128, 1, false>(p, grid, s);
        else st = masked ? launch_dp8_kernel<128, 2, true>(p, grid, s) : launch_dp8_kernel<128, 2, false>(p, grid, s);
    } else {
        if (tile_rows == 8) st = masked ? launch_dp8_kernel<64, 1, true>(p, grid, s) : launch_dp8_kernel<64, 1, false>(p, grid, s);
        else st = masked ? launch_dp8_kernel<64, 2, true>(p, grid, s) : launch_dp8_kernel<64, 2, false>(p, grid, s);
    }
    if (st != FATTN_OK || p.S == 1 || p.cluster) return st;
    const long long merge_grid = (static_cast<long long>(p.B) * p.max_q * p.Hq + 3) / 4;  // a warp per row
    if (p.S > 64)
        return d == 128 ? launch_merge(merge_paged_fp8_kernel<128, true>, merge_grid, 128, s, p, tile_rows)
                        : launch_merge(merge_paged_fp8_kernel<64, true>, merge_grid, 128, s, p, tile_rows);
    return d == 128 ? launch_merge(merge_paged_fp8_kernel<128, false>, merge_grid, 128, s, p, tile_rows)
                    : launch_merge(merge_paged_fp8_kernel<64, false>, merge_grid, 128, s, p, tile_rows);
}

// Rows (new tokens x group heads) of a sequence from which its tiles go to the
// tensor-core kernel.
constexpr long long kExtMinRows = 49;
// Its TMA coordinates are 32-bit rows of the pool.
constexpr long long kExtMaxPoolRows = 0x7fffff00LL;

bool ext_path(long long max_q, int g) { return max_q * g >= kExtMinRows; }

// Pairs of row tiles of one sequence.
long long ext_pairs(long long max_q, int g) {
    const long long toks = 128 / g;
    return ((max_q + toks - 1) / toks + 1) / 2;
}

// How the pairs of row tiles become items: the whole rounds of one pair per SM
// stay whole, the pairs of the last, incomplete round are cut into parts of the
// keys where a model of the kernel's time says so.  Measured on B200: 2.0 us a
// key tile, 8 us more an item, 5 us for the merge and 1.6 TB/s for the parts'
// (o, lse).  16 pairs over 64 tiles: 47 us in 8 parts, 62 in 10, 64 in 16; 128
// pairs over 16 tiles: 52 us whole, 57 in 2 parts, 64 in 3.
int ext_splits(long long pairs, long long tiles, int toks, int g, int d) {
    const long long tail = pairs % kSms;
    const double part_bytes = static_cast<double>(tail) * 2 * toks * g * (d + 1) * 8;
    int best = 1;
    double least = 0.0;
    for (int S = 1; S <= 32 && (S == 1 || static_cast<long long>(S) * EXT_MIN_TILES <= tiles); ++S) {
        const double rounds = std::ceil(static_cast<double>(tail) * S / kSms);
        double us = rounds * (std::ceil(static_cast<double>(tiles) / S) * 2.0 + 8.0);
        if (S > 1) us += 5.0 + part_bytes * S / 1.6e6;
        if (S == 1 || us < least) {
            least = us;
            best = S;
        }
    }
    return best;
}

// Rows of the pairs that are cut into parts: those of the last, incomplete round.
long long ext_cut_rows(long long pairs, int g) { return pairs % kSms * 2 * (128 / g) * g; }

// The item counter, then the parts' (o, lse) of those rows (2048 tokens of 32 heads over 131072 keys: 57 MB).
constexpr size_t kExtCounterBytes = 32;
size_t ext_workspace(long long pairs, int S, int g, int d) { return kExtCounterBytes + parts_bytes(ext_cut_rows(pairs, g), S, d); }

// The pool [num_pages * page_size, Hkv, d] of codes: boxes of box_rows keys of one head.
int encode_map_pages(CUtensorMap* map, const void* base, int d, int Hkv, long long rows, int box_rows) {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(Hkv), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(Hkv) * d};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(d), 1, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FATTN_OK : FATTN_ERR_CUDA;
}

int launch_ext(const PagedFp8Params& c, int d, long long pool_rows, void* workspace, size_t workspace_bytes, void* stream) {
    ExtParams p{};
    p.c = c;
    p.toks = 128 / c.g;
    p.n_pairs = static_cast<int>(ext_pairs(c.max_q, c.g));
    const long long pairs = static_cast<long long>(c.B) * c.Hkv * p.n_pairs;
    const long long all_tiles = ((static_cast<long long>(c.max_pages) << c.page_shift) + 127) / 128;
    p.splits = ext_splits(pairs, all_tiles, p.toks, c.g, d);  // what the workspace is sized for
    if (c.window_left >= 0 && (c.causal || c.window_right >= 0)) {
        // a pair of row tiles sees the window and its own tokens
        const long long seen = (static_cast<long long>(c.window_left) + (c.causal ? 0 : c.window_right) + 2LL * p.toks + 255) / 128;
        const int S = ext_splits(pairs, seen < all_tiles ? seen : all_tiles, p.toks, c.g, d);
        p.splits = S < p.splits ? S : p.splits;
    }
    p.n_whole = static_cast<int>(p.splits == 1 ? pairs : pairs - pairs % kSms);
    const long long cut = pairs - p.n_whole, n_items = p.n_whole + cut * p.splits;
    if (pairs > 0x07ffffffLL) return FATTN_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < ext_workspace(pairs, p.splits, c.g, d)) return FATTN_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 31u) return FATTN_ERR_MISALIGNED;
    p.counter = static_cast<unsigned int*>(workspace);
    p.c.ws_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + kExtCounterBytes);
    p.c.ws_lse = p.c.ws_o + ext_cut_rows(pairs, c.g) * p.splits * d;
    p.n_items = static_cast<int>(n_items);
    const int page_size = 1 << c.page_shift;
    p.box_rows = page_size < 128 ? page_size : 128;
    p.o_vec32 = (reinterpret_cast<uintptr_t>(c.o) & 31u) == 0 ? 1 : 0;
    DeviceInfo di;
    int st = device_ready(&di);
    if (st != FATTN_OK) return st;
    if (!di.ext_regs_ok) return FATTN_ERR_UNSUPPORTED;
    CUtensorMap mk, mv;
    if (encode_map_pages(&mk, c.k, d, c.Hkv, pool_rows, p.box_rows) != FATTN_OK ||
        encode_map_pages(&mv, c.v, d, c.Hkv, pool_rows, p.box_rows) != FATTN_OK)
        return FATTN_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(p.counter, 0, sizeof(unsigned int), s) != cudaSuccess) {
        cudaGetLastError();
        return FATTN_ERR_CUDA;
    }
    const unsigned grid = static_cast<unsigned>(n_items < di.num_sms ? n_items : di.num_sms);
    if (d == 128) attn_paged_fp8_kernel<128><<<grid, ExtTraits<128>::THREADS, ExtTraits<128>::SMEM_BYTES, s>>>(mk, mv, p);
    else attn_paged_fp8_kernel<64><<<grid, ExtTraits<64>::THREADS, ExtTraits<64>::SMEM_BYTES, s>>>(mk, mv, p);
    if (cudaGetLastError() != cudaSuccess) return FATTN_ERR_CUDA;
    if (p.splits == 1) return FATTN_OK;
    return d == 128 ? launch_merge(merge_ext_kernel<128>, 16 * cut, 256, s, p) : launch_merge(merge_ext_kernel<64>, 16 * cut, 256, s, p);
}

template <int D, int WARPS>
int launch_append(const AppendParams& p, cudaStream_t s) {
    const long long grid = (static_cast<long long>(p.T) + p.chunk - 1) / p.chunk * p.H * 2;
    if (grid > 0x7fffffffLL) return FATTN_ERR_UNSUPPORTED;
    append_paged_fp8_kernel<D, WARPS><<<static_cast<unsigned>(grid), 32 * WARPS, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

int attn_paged_plan(const int* seqlens_k, const int* seqlens_new, int B, const int* free_pages, int num_free,
                    int* block_table, int max_pages, int page_size, long long* slot_map, int max_tokens,
                    int* cu_seqlens, int* seqlens_out, int* counts, void* stream) {
    if (!seqlens_k || !seqlens_new || !block_table || !slot_map || !cu_seqlens || !seqlens_out || !counts)
        return FATTN_ERR_INVALID_ARG;
    if (B < 1 || num_free < 0 || (num_free > 0 && !free_pages) || max_pages < 1 || max_tokens < 1) return FATTN_ERR_INVALID_ARG;
    if (!pow2_page(page_size)) return FATTN_ERR_INVALID_ARG;
    if (B > PLAN_MAX_SEQ || max_tokens > 0x7fffff00) return FATTN_ERR_UNSUPPORTED;
    if (misaligned4(seqlens_k) || misaligned4(seqlens_new) || misaligned4(free_pages) || misaligned4(block_table) ||
        misaligned4(cu_seqlens) || misaligned4(seqlens_out) || misaligned4(counts) ||
        (reinterpret_cast<uintptr_t>(slot_map) & 7u))
        return FATTN_ERR_MISALIGNED;
    // the lengths are read while the outputs are written
    const size_t nb = static_cast<size_t>(B) * 4;
    if (overlap(seqlens_out, nb, seqlens_k, nb) || overlap(seqlens_out, nb, seqlens_new, nb) ||
        overlap(cu_seqlens, nb + 4, seqlens_k, nb) || overlap(cu_seqlens, nb + 4, seqlens_new, nb))
        return FATTN_ERR_INVALID_ARG;
    DeviceInfo di;
    const int st = device_ready(&di);
    if (st != FATTN_OK) return st;
    PlanParams p{seqlens_k, seqlens_new, free_pages, block_table, slot_map, cu_seqlens, seqlens_out, counts,
                 B, max_pages, log2_of(page_size), num_free, max_tokens};
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(max_tokens) + PLAN_TOKENS - 1) / PLAN_TOKENS);
    paged_plan_kernel<<<grid, PLAN_THREADS, 2 * (nb + 4), static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

int attn_append_paged_fp8(const void* k, const void* v, long long k_stride, long long v_stride, const long long* slot_map,
                          int num_tokens, void* k_pages, void* v_pages, float* k_scales, float* v_scales, int num_pages,
                          int page_size, int H, int d, void* stream) {
    if (!k || !v || !slot_map || !k_pages || !v_pages || !k_scales || !v_scales) return FATTN_ERR_INVALID_ARG;
    if (num_tokens < 1 || num_pages < 1 || H < 1 || !pow2_page(page_size)) return FATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FATTN_ERR_UNSUPPORTED;
    const long long row = static_cast<long long>(H) * d;
    if (H > 65535 || num_tokens > 0x7fffff00 || static_cast<long long>(num_pages) * page_size > (1LL << 40))
        return FATTN_ERR_UNSUPPORTED;
    if (num_tokens > 1 && (k_stride < row || v_stride < row)) return FATTN_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) || k_stride % 8 != 0 || v_stride % 8 != 0 ||
        misaligned4(k_scales) || misaligned4(v_scales) || (reinterpret_cast<uintptr_t>(slot_map) & 7u))
        return FATTN_ERR_MISALIGNED;
    const size_t pool = static_cast<size_t>(num_pages) * page_size * row, sc = static_cast<size_t>(num_pages) * H * 4;
    if (overlap(k_pages, pool, v_pages, pool) || overlap(k_scales, sc, v_scales, sc)) return FATTN_ERR_INVALID_ARG;
    DeviceInfo di;
    const int st = device_ready(&di);
    if (st != FATTN_OK) return st;
    AppendParams p{};
    p.x[0] = static_cast<const __nv_bfloat16*>(k);
    p.x[1] = static_cast<const __nv_bfloat16*>(v);
    p.stride[0] = k_stride;
    p.stride[1] = v_stride;
    p.pages[0] = static_cast<uint8_t*>(k_pages);
    p.pages[1] = static_cast<uint8_t*>(v_pages);
    p.scales[0] = k_scales;
    p.scales[1] = v_scales;
    p.slots = slot_map;
    p.num_slots = static_cast<long long>(num_pages) * page_size;
    p.T = num_tokens;
    p.H = H;
    p.page_shift = log2_of(page_size);
    // A warp for every 16 rows of a page, at most 4 (17.8k tokens in pages of 128: 27 us, 30 with 8 warps, 31 with 2).
    // Tokens to a CTA so that the warps, counted up to 8, are about one wave of 64 an SM: larger pages have fewer runs.
    const int rows16 = page_size / 16, W = rows16 < 4 ? rows16 : 4;
    const long long chunk = (2LL * H * num_tokens * (rows16 < 8 ? rows16 : 8) + 64LL * di.num_sms - 1) / (64LL * di.num_sms);
    p.chunk = static_cast<int>(chunk < 1 ? 1 : (chunk > page_size ? page_size : chunk));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d == 128) return W == 1 ? launch_append<128, 1>(p, s) : W == 2 ? launch_append<128, 2>(p, s) : launch_append<128, 4>(p, s);
    return W == 1 ? launch_append<64, 1>(p, s) : W == 2 ? launch_append<64, 2>(p, s) : launch_append<64, 4>(p, s);
}

int attn_decode_paged_fp8_auto_splits(int B, int Hq, int Hkv, int Lk, int d) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Lk < 1 || (d != 64 && d != 128)) return FATTN_ERR_INVALID_ARG;
    const long long g = Hq / Hkv;
    const int t = dp8_tile_rows(g, false);
    return dp8_auto_splits(static_cast<long long>(B) * Hkv * ((g + t - 1) / t), Lk, d, t, false);
}

int attn_decode_paged_fp8(const void* q, const void* k_pages, const void* v_pages, const float* k_scales,
                          const float* v_scales, const int* block_table, int max_pages, int page_size, int num_pages,
                          void* o, float* lse, const int* seqlens_k, int B, int Hq, int Hkv, int d, float scale,
                          int window_left, int num_splits, void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, block_table, max_pages, page_size, num_pages, o,
                                   lse, seqlens_k, B, Hq, Hkv, d, scale);
    if (st != FATTN_OK) return st;
    if (num_splits < 0) return FATTN_ERR_INVALID_ARG;
    PagedFp8Params p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const uint8_t*>(k_pages);
    p.v = static_cast<const uint8_t*>(v_pages);
    p.ks = k_scales;
    p.vs = v_scales;
    p.block_table = block_table;
    p.seqlens_k = seqlens_k;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.lse_tok = Hq;
    p.lse_head = 1;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.g = Hq / Hkv;
    p.total_q = B;
    p.max_q = 1;
    p.max_pages = max_pages;
    p.page_shift = log2_of(page_size);
    p.num_pages = num_pages;
    p.causal = 1;
    p.window_left = window_left < 0 ? -1 : window_left;
    p.window_right = -1;
    p.scale_log2 = scale * 1.4426950408889634f;
    return launch_dp8(p, d, num_splits, workspace, workspace_bytes, stream);
}

size_t attn_fwd_paged_fp8_workspace_bytes(int B, int total_q, int max_seqlen_q, int Hq, int Hkv, int Lk, int d) {
    if (B < 1 || total_q < 1 || max_seqlen_q < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Lk < 1 || (d != 64 && d != 128))
        return 0;
    const long long max_q = max_seqlen_q < total_q ? max_seqlen_q : total_q;
    const int g = Hq / Hkv;
    const long long rows = max_q * g, all = static_cast<long long>(total_q) * Hq;
    if (g <= 128 && ext_path(max_q, g)) {
        const long long pairs = static_cast<long long>(B) * Hkv * ext_pairs(max_q, g);
        return ext_workspace(pairs, ext_splits(pairs, (static_cast<long long>(Lk) + 127) / 128, 128 / g, g, d), g, d);
    }
    const int t = dp8_tile_rows(rows, max_q > 1);
    return parts_bytes(all, dp8_auto_splits(static_cast<long long>(B) * Hkv * ((rows + t - 1) / t), Lk, d, t, max_q > 1), d);
}

int attn_fwd_paged_fp8(const void* q, const void* k_pages, const void* v_pages, const float* k_scales,
                       const float* v_scales, const int* block_table, int max_pages, int page_size, int num_pages,
                       void* o, float* lse, const int* seqlens_k, const int* cu_seqlens_q, int B, int total_q,
                       int max_seqlen_q, int Hq, int Hkv, int d, float scale, int causal, int window_left,
                       int window_right, void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, block_table, max_pages, page_size, num_pages, o,
                                   lse, seqlens_k, B, Hq, Hkv, d, scale);
    if (st != FATTN_OK) return st;
    if (!cu_seqlens_q || total_q < 1 || max_seqlen_q < 1) return FATTN_ERR_INVALID_ARG;
    if (misaligned4(cu_seqlens_q)) return FATTN_ERR_MISALIGNED;
    if (total_q > 0x7fffff00 || max_seqlen_q > 0x7fffff00) return FATTN_ERR_UNSUPPORTED;
    PagedFp8Params p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const uint8_t*>(k_pages);
    p.v = static_cast<const uint8_t*>(v_pages);
    p.ks = k_scales;
    p.vs = v_scales;
    p.block_table = block_table;
    p.seqlens_k = seqlens_k;
    p.cu_q = cu_seqlens_q;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.lse_tok = 1;
    p.lse_head = total_q;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.g = Hq / Hkv;
    p.total_q = total_q;
    p.max_q = max_seqlen_q < total_q ? max_seqlen_q : total_q;
    p.max_pages = max_pages;
    p.page_shift = log2_of(page_size);
    p.num_pages = num_pages;
    p.causal = causal ? 1 : 0;
    p.window_left = window_left < 0 ? -1 : window_left;
    p.window_right = window_right < 0 ? -1 : window_right;
    p.scale_log2 = scale * 1.4426950408889634f;
    if (ext_path(p.max_q, p.g)) {
        const long long pool_rows = static_cast<long long>(num_pages) * page_size;
        if (pool_rows <= kExtMaxPoolRows) return launch_ext(p, d, pool_rows, workspace, workspace_bytes, stream);
        return launch_dp8(p, d, 1, nullptr, 0, stream);  // a pool beyond the tensor map's coordinates
    }
    return launch_dp8(p, d, 0, workspace, workspace_bytes, stream);
}

}  // extern "C"
