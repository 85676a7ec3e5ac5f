// tree_sm100.cuh -- split-KV attention of a tree of drafted tokens over a KV
// cache, on the tcgen05 tensor cores.
//
// What it computes: sequence b has n = seqlens[b] cached rows, the last n_b of
// them the nodes of a tree (n_b = tree_lens[b], or T).  With c = n - n_b, query
// row (h, i) of node i < n_b sees the rows below c and, of the tree, the rows
// c + j whose bit j is set in mask[b][i]:
//
//   O[h, i] = sum_r w_r V_r / sum_r w_r,   w_r = 2^(scale log2e q.K_r - m) over those r,
//   LSE[h, i] = ln sum_r e^(scale q.K_r)
//
// A row that sees nothing (an empty mask on an empty context, a node >= n_b)
// gets O = 0 and LSE = -inf.
//
// The G x T query rows of a KV head are cut into blocks of 128, the M rows of the MMAs.  The
// work is balanced from the lengths on the device: the tiles of all (sequence, KV head) pairs
// in one line are cut into equal ranges, one CTA for each range and query block, as many CTAs
// as the GPU holds at once.  A CTA walks its range segment by segment (a segment: the part of
// one pair's tiles in the range); the CTAs of one range read the same K and V side by side, so
// all but one of them find them in the L2.  A segment that is a whole pair writes the result;
// the others write a normalised partial (at most two a CTA) that a combine kernel merges.  The
// loads run on across segments.
//
// P is rounded to bf16 for the MMA (its A operand has V's type, and two bf16 parts would double
// P V); O is divided by the sum of the rounded P, so that a weight's rounding moves O by at most
// 2^-8 of the weight times V's distance from O, and the log-sum-exp takes the unrounded sum.
// Against 64 bits the bf16 result is off by 0.0021 (500 rows) to 0.0023 (1K to 32K) relative to
// its norm; with weights in fp32 it would be 0.0017, the result's own rounding.
//
// Per tile of 64 cache rows S = Q K^T, P = 2^(S scale log2 e - m) and O += P V, with two S
// buffers, so that S of the next tile is computed under the softmax of this one, as
// attn_decode_tc_kernel.  D = 64 and 128: Q in shared memory, two CTAs on an SM.  D = 256: O
// takes half the TMEM, one CTA on an SM; Q lies in TMEM, which leaves its 64 KB of shared
// memory to K and V.
//
// What bounds it, one B200.  64 requests of 1K to 32K rows, 32 heads over 8 KV heads, 16 nodes, head
// dim 128 (4.45 GB, 687 us at the copy rate): the CTAs take 625 to 655 us, 6.9 TB/s, the cache read,
// the same at 1.5 and 1.6 GHz.  A grid of splits of the longest cache instead of equal ranges took
// 838 us.  8 requests of 3K to 16K rows, 32 heads over 4, 63 nodes, head dim 256 (four query blocks;
// 117 GFLOP, 70 us at the bf16 rate): 156 us for a CTA of one segment and 10 more for each further
// one, about 2260 cycles a tile.  The MMAs are 1376 of them (an MMA of N = 64 costs 54 cycles, not
// 32); what is left is the issuing warp going from one commit to the next wait.  Not faster: tiles
// of 128 rows in two streams, each with a softmax warpgroup, on one CTA an SM (head dim 128, 770 us
// for 683); looking for P and V half-way through Q K^T; waiting for K and V under P V (342K cycles
// for 306K); head dim 256 with Q in shared memory (331K for 306K, with a shallower ring).  Tiles of
// 128 rows at head dim 256 (O and two S fill the TMEM, Q back in shared memory) were not tried.
//
// The mask costs nothing over the committed rows: only a tile that reaches past c builds the
// 64 visibility bits of its rows, each thread (one query row) shifting them out of its own
// mask words.
//
// A tree row that one node sees and another does not may hold infinities or NaN
// in V.  The MMA would carry 0 * NaN into the nodes that do not see it, so the
// MMA warp replaces non-finite elements of tree rows by zero in shared memory
// first, and the epilogue adds them back, read from the cache, to the outputs
// of the nodes that see the row.
#pragma once

#include "decode_sm100.cuh"
#include "decode_tc_sm100.cuh"
#include "device_error.cuh"
#include "ptx_sm100.cuh"
#include "ring_order.cuh"

namespace attn {

constexpr int kTreeMaxNodes = 1024;

struct TreeParams {
    DecodeParams d;              // d.Lq = T; o_part / lse_part: see tree_part; chunk, n_splits unused
    const uint32_t* mask;        // [B or 1, T, W]
    size_t mask_batch;           // words from one sequence's mask to the next's (0: one mask for all)
    const int* tree_lens;        // [B], or nullptr (every tree has T nodes)
    const __nv_bfloat16* v;      // the V cache (non-finite elements of tree rows)
    __nv_bfloat16* out;
    float* lse;                  // or nullptr
    long long* tiles_before;     // [B + 1] workspace: tiles of the sequences before b (one KV head); [B]: tiles a range
    int W;                       // words per mask row, (T + 31) / 32
    int n_mblk;                  // 128-row blocks of a KV head's G x T query rows
    int n_ranges;
};

// Tiles of a sequence (rows of a tile: TreeCfg<D>::kTile).
template <int TILE>
__device__ __forceinline__ int tree_tiles(int seqlen) {
    return seqlen / TILE + (seqlen % TILE != 0);
}

// The partial that range `range` wrote for query block mblk in slot 0 (its first segment) or 1
// (its last), of min(128, G x T) rows.
__device__ __forceinline__ size_t tree_part(const TreeParams& p, long long range, int mblk, int slot) {
    return (static_cast<size_t>(range) * p.n_mblk + mblk) * 2 + slot;
}

// Element (row r, column c) of a partial of `box` rows: four columns of all rows, then the next four,
// so that the epilogue (a thread per row) writes, and the combine (a lane per row) reads, 512
// contiguous bytes a warp.  (Row after row, a warp's stores met 32 lines each: two requests of 1500
// and 3000 rows, 16 nodes, head dim 256 took 30 us for 24.)
__device__ __forceinline__ size_t tree_part_at(int box, int r, int c) {
    return (static_cast<size_t>(c >> 2) * box + r) * 4 + (c & 3);
}

__device__ __forceinline__ int tree_len(const TreeParams& p, int b) {
    if (p.tree_lens == nullptr) return p.d.Lq;
    int n = p.tree_lens[b];
    if (n < 0 || n > p.d.Lq) {
        atomicOr(&g_attn_err, kDevErrIndex);
        n = n < 0 ? 0 : p.d.Lq;
    }
    return n;
}

// Bits 0 .. n-1 (n may be negative or past 64).
__device__ __forceinline__ uint64_t low_bits(int n) {
    return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull);
}

// Which of cache rows key0 .. key0 + 63 a node sees: all below ctx, and row
// ctx + j where bit j of its mask words is set.  Bits at or past W * 32 are 0.
__device__ __forceinline__ uint64_t tree_visible(const uint32_t* words, int W, int ctx, int key0) {
    uint64_t vis = low_bits(ctx - key0);
    const int c = key0 - ctx;                      // tree column of the tile's first row
    if (c > -64) {
        const int w = c >= 0 ? c >> 5 : 0;
        const uint32_t w0 = w < W ? __ldg(words + w) : 0u;
        const uint32_t w1 = w + 1 < W ? __ldg(words + w + 1) : 0u;
        const uint64_t lo = (static_cast<uint64_t>(w1) << 32) | w0;
        if (c <= 0) {
            vis |= lo << -c;
        } else {
            const uint32_t w2 = w + 2 < W ? __ldg(words + w + 2) : 0u;
            const int sh = c & 31;
            vis |= sh == 0 ? lo : (lo >> sh) | (static_cast<uint64_t>(w2) << (64 - sh));
        }
    }
    return vis;
}

// Cache row `row` of sequence b, KV head g, as a row of the [.., D] cache.
__device__ __forceinline__ size_t tree_cache_row(const DecodeParams& p, int b, int g, int row) {
    if (p.block_table == nullptr) return (static_cast<size_t>(b) * p.Hkv + g) * p.Lmax + row;
    int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + row / p.page_size);
    if (page < 0 || page >= p.n_pages) page = 0;       // as the producer does
    return (static_cast<size_t>(page) * p.Hkv + g) * p.page_size + row % p.page_size;
}

// Adds the non-finite elements of the tree rows in [k_begin, k_end) that this
// thread's node sees to its output or partial (any positive weight times them is
// themselves); element c of the row at dst[(c / 4) step + c % 4].
template <typename T>
__device__ __noinline__ void tree_add_nonfinite(const TreeParams& tp, int b, int g, const uint32_t* words, int ctx,
                                                int k_begin, int k_end, int D, T* dst, int step) {
    for (int row = max(max(ctx, 0), k_begin); row < k_end; ++row) {
        const int j = row - ctx;
        if (!(words[j >> 5] >> (j & 31) & 1u)) continue;
        const __nv_bfloat16* src = tp.v + tree_cache_row(tp.d, b, g, row) * D;
        for (int c = 0; c < D; ++c) {
            const float x = __bfloat162float(src[c]);
            T& y = dst[static_cast<size_t>(c >> 2) * step + (c & 3)];
            if (!isfinite(x)) y = static_cast<T>(static_cast<float>(y) + x);
        }
    }
}

// All ones over the halves of a bf16 pair that are infinite or NaN.
__device__ __forceinline__ uint32_t nonfinite_bf16x2(uint32_t x) {
    return ((x & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((x & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

template <int D>
struct TreeCfg {
    static constexpr int kKB = D / 64;
    static constexpr int kCtasPerSm = D == 256 ? 1 : 2;
    static constexpr bool kQTmem = D == 256;
    static constexpr int kTile = 64;                          // cache rows of a tile: the TMA boxes' (kDecKT), pages hold whole ones
    static constexpr int kThreads = 192;                      // softmax warps 0-3, producer, MMA issuer
    static constexpr int kProducerWarp = 4;
    static constexpr int kMmaWarp = 5;
    // TMEM columns: S0, S1 (P over the first half of each), Q (D = 256), O
    static constexpr uint32_t kTmemCols = D == 256 ? 512 : 256;
    static constexpr uint32_t kTmemQ = 128, kTmemO = D == 256 ? 256 : 128;
    // shared memory: Q as 128 rows x 128 bytes per 64 columns, then the ring of K and V tiles
    static constexpr int kQBlockBytes = 128 * 128;
    static constexpr int kQBytes = kQTmem ? 0 : 128 * D * 2;
    static constexpr int kBlockBytes = kTile * 128;           // a tile's rows x 128 bytes per 64 columns
    static constexpr int kTileBytes = kTile * D * 2;
    // as many tiles as fit beside Q when kCtasPerSm CTAs share the SM's 228 KB (1 KB reserved per
    // CTA, 1 KB alignment slack, 1 KB for what follows the ring), at most 16
    static constexpr int kStagesFit = (233472 / kCtasPerSm - 3 * 1024 - kQBytes) / kTileBytes;
    static constexpr int kStages = kStagesFit > 16 ? 16 : kStagesFit;
    static constexpr int kKVOff = kQBytes;
    static constexpr int kBarOff = kKVOff + kStages * kTileBytes;
    // q_full, q_empty, full[S], empty[S], s_full[2], p_full[2], drain
    static constexpr int kNumBars = 2 + 2 * kStages + 4 + 1;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;   // tmem base, abort flag, patched[2]
    static constexpr int kTagOff = kMiscOff + 16;             // debug builds: ring entry -> item
    static constexpr int kAlloc = kTagOff + 4 * kStages + 1024;
    static_assert(kTagOff + 4 * kStages - kBarOff <= 768, "barriers and flags");
    static_assert(kAlloc <= 232448 - 256, "dynamic shared memory per CTA");
    static_assert(kStages >= 4, "ring too shallow");
};

// Part of one (sequence, KV head) pair's tiles in a CTA's range.
struct TreeSeg {
    long long x, x_end;       // tiles of the line still to do: this segment starts at x
    int b, g;
    int seqlen, tiles;        // of the pair
    int t0, t1;               // the segment's tiles
    int n;                    // segments before it
};

// The segment after s; false when the range is done.
template <int TILE>
__device__ __forceinline__ bool tree_next(const TreeParams& tp, TreeSeg& s) {
    s.x += s.t1 - s.t0;
    if (s.x >= s.x_end) return false;
    ++s.n;
    s.t0 = 0;
    if (++s.g == tp.d.Hkv) {
        s.g = 0;
        do {
            if (++s.b == tp.d.B) return false;     // (the lengths changed under the kernel)
            s.seqlen = decode_seqlen(tp.d, s.b);
            s.tiles = tree_tiles<TILE>(s.seqlen);
        } while (s.tiles == 0);
    }
    s.t1 = static_cast<int>(min(static_cast<long long>(s.tiles), s.x_end - s.x));
    return true;
}

// Tiles that a range has at least, where there are fewer than the GPU could hold ranges for.  Longer
// ranges cost a tile's time each, shorter ones partials: their bytes, written and read, and rounds of
// 32 of a pair's partials in the combine.  With r tiles a range the sum is t r + c / r, least at
// r = sqrt(c / t); t, the byte rate and a round's time are fitted to the device times of ten small
// trees with r = 1, 2 and 4, of which it takes the fastest or one within 0.1 us: one request of 375
// rows, 8 nodes of 32 heads, D 64 9.8 us (r = 1) for 10.5 (2) and 12.8 (4); 64 nodes of 8 heads of one
// KV head on 6000 rows 15.6 (4) for 20.7 (1, 2); 4 rows on 12000 12.8 (2) for 16.3 (1) and 13.7 (4);
// D 256, two requests of 1500 and 3000 rows 19.2 (1) for 24.2 (2).
template <int D>
__device__ __forceinline__ long long tree_least_tiles(const TreeParams& tp, long long total) {
    constexpr float kTileUs = D == 256 ? 4.0f : 0.75f, kBytesPerUs = 5e6f, kRoundUs = 0.7f;
    const float tiles = static_cast<float>(total);
    const float bytes = tiles * static_cast<float>(tp.d.G * tp.d.Lq) * static_cast<float>(D * 4 * 2);
    const float rounds = tiles / (static_cast<float>(tp.d.B) * static_cast<float>(tp.d.Hkv)) / 32.0f;
    const float r = sqrtf((bytes / kBytesPerUs + rounds * kRoundUs) / kTileUs);
    return max(1ll, static_cast<long long>(r + 0.5f));
}

template <int D>
__global__ void __launch_bounds__(TreeCfg<D>::kThreads, TreeCfg<D>::kCtasPerSm)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const TreeParams tp) {
    grid_dep_release();   // the combine launch may be scheduled now
    using L = TreeCfg<D>;
    constexpr int kTile = L::kTile, kWarps = L::kThreads / 32;
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long s_warp[kWarps], s_before;
    __shared__ int s_b;
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_base);

    const DecodeParams& p = tp.d;
    const int range = blockIdx.x / tp.n_mblk, mblk = blockIdx.x % tp.n_mblk;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // ---- this CTA's range of the line of tiles ----
    const int per_thread = (p.B + L::kThreads - 1) / L::kThreads;
    const int my_b = min(p.B, static_cast<int>(threadIdx.x) * per_thread), my_end = min(p.B, my_b + per_thread);
    long long mine = 0;
    for (int b = my_b; b < my_end; ++b) mine += tree_tiles<kTile>(decode_seqlen(p, b));
    long long before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
    }
    if (lane == 31) s_warp[warp] = before;
    before -= mine;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    total *= p.Hkv;
    const long long per = max((total + tp.n_ranges - 1) / tp.n_ranges, tree_least_tiles<D>(tp, total));
    if (blockIdx.x == 0) {                        // for the combine
        long long t = before;
        for (int b = my_b; b < my_end; ++b) {
            tp.tiles_before[b] = t;
            t += tree_tiles<kTile>(decode_seqlen(p, b));
        }
        if (threadIdx.x == 0) tp.tiles_before[p.B] = per;
    }
    TreeSeg first;
    first.x = range * per;
    first.x_end = min(first.x + per, total);
    if (first.x >= first.x_end) return;           // uniform: nothing left for this range
    if (before * p.Hkv <= first.x && first.x < (before + mine) * p.Hkv) {
        int b = my_b;
        for (int t; first.x >= (before + (t = tree_tiles<kTile>(decode_seqlen(p, b)))) * p.Hkv; ++b) before += t;
        s_b = b;
        s_before = before;
    }

    const int RG = p.G * p.Lq;                     // query rows of a KV head
    const int R = min(128, RG - mblk * 128);       // of this block
    const int box = min(128, RG);                  // rows TMA loads (past the block's: another head's, or 0)

    const uint32_t sQ = base;
    const uint32_t sKV = base + L::kKVOff;
    const uint32_t bar0 = base + L::kBarOff;
    const uint32_t bar_q_full = bar0, bar_q_empty = bar0 + 8u;
    auto bar_full = [&](int s) { return bar0 + 8u * (2 + s); };
    auto bar_empty = [&](int s) { return bar0 + 8u * (2 + L::kStages + s); };
    constexpr uint32_t kB2 = 2 + 2 * L::kStages;
    auto bar_s_full = [&](int i) { return bar0 + 8u * (kB2 + i); };
    auto bar_p_full = [&](int i) { return bar0 + 8u * (kB2 + 2 + i); };
    const uint32_t bar_drain = bar0 + 8u * (kB2 + 4);
    uint32_t* tmem_base_ptr = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
    // segment n whose tree rows lost non-finite elements: n + 1 in entry n % 2 (the MMA warp is
    // at most one segment ahead of the epilogue)
    volatile int* v_patched = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 8);
    // (debug builds) the item the producer put in each ring entry, checked by the MMA warp
    volatile int* ring_tag = reinterpret_cast<volatile int*>(smem + L::kTagOff);

    if (threadIdx.x == 0) {
        mbar_init(bar_q_full, L::kQTmem ? 128 : 1);
        mbar_init(bar_q_empty, 1);
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar_full(s), 1);
            mbar_init(bar_empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_s_full(i), 1);
            mbar_init(bar_p_full(i), 128);
            v_patched[i] = 0;
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    // query rows past the box are not loaded: make them zero (finite) for the MMA
    if (!L::kQTmem && box < 128) {
        const int pad = (128 - box) * 128;
        for (int kb = 0; kb < L::kKB; ++kb) {
            uint8_t* blk = smem + kb * L::kQBlockBytes + box * 128;
            for (int i = threadIdx.x * 16; i < pad; i += L::kThreads * 16)
                *reinterpret_cast<uint4*>(blk + i) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
    }
    if (warp == L::kMmaWarp) {
        tmem_alloc(smem_u32(tmem_base_ptr), L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_base_ptr;
    auto tS = [&](int buf) { return tmem + static_cast<uint32_t>(kTile * buf); };
    const uint32_t tO = tmem + L::kTmemO;

    first.n = 0;
    first.b = s_b;
    first.seqlen = decode_seqlen(p, first.b);
    first.tiles = tree_tiles<kTile>(first.seqlen);
    {
        const long long in_b = first.x - s_before * p.Hkv;
        first.g = static_cast<int>(in_b / first.tiles);
        first.t0 = static_cast<int>(in_b - static_cast<long long>(first.g) * first.tiles);
        first.t1 = static_cast<int>(min(static_cast<long long>(first.tiles), first.t0 + (first.x_end - first.x)));
    }

    // The ring's items, K and V tiles, are numbered through the whole range: segment after
    // segment, in each K_0 K_1 V_0 K_2 V_1 ... (ring_order.cuh), which is also the order in
    // which the MMAs use them.  Tile jj of the range (counted through all segments) has S
    // buffer jj % 2.
    struct RingPos {
        int e = 0, item = 0;
        uint32_t par = 0;
        __device__ __forceinline__ void next() {
            ++item;
            if (++e == L::kStages) {
                e = 0;
                par ^= 1u;
            }
        }
    };

    if (warp == L::kProducerWarp) {
        // ================= TMA producer (lane 0 issues; the warp looks the pages up) =================
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
        RingPos at;
        bool ok = true;
        auto wait_bar = [&](uint32_t bar, uint32_t parity) {       // the warp goes on, or stops, together
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &g_attn_err, kDevErrTimeout)) != 0;
        };
        TreeSeg s = first;
        do {
            const int n_tiles = s.t1 - s.t0;
            if (!L::kQTmem) {
                // (the last Q K^T of a segment is issued two tiles before its end)
                ok = wait_bar(bar_q_empty, (s.n & 1) ^ 1u);
                if (!ok) break;
                if (lane == 0) {
                    const size_t row0 = (static_cast<size_t>(s.b) * p.Hq + static_cast<size_t>(s.g) * p.G) * p.Lq + mblk * 128;
                    mbar_arrive_expect_tx(bar_q_full, static_cast<uint32_t>(L::kKB * box * 128));
                    for (int kb = 0; kb < L::kKB; ++kb)
                        tma_load_3d(sQ + kb * L::kQBlockBytes, &tm_q, bar_q_full, kb * 64, static_cast<int>(row0), 0);
                }
                __syncwarp();
            }
            // Pages of the segment's tiles, a window of 32 in the warp's lanes and the next one on its way:
            // looked up tile by tile they held the loads back (with tiles of 128 rows, 978 us for 869 at 64
            // requests of 1K to 32K rows).
            int window = s.t0, here = 0, after = 0;
            auto lookup = [&](int tile0) {
                const int i = tile0 + lane;
                if (p.block_table == nullptr || i >= s.t1) return 0;
                const int page = __ldg(p.block_table + static_cast<size_t>(s.b) * p.max_pages +
                                       static_cast<int>(static_cast<long long>(i) * kTile / p.page_size));
                if (page >= 0 && page < p.n_pages) return page;
                atomicOr(&g_attn_err, kDevErrPage);
                return 0;
            };
            here = lookup(window);
            after = lookup(window + 32);
            for (int i = 0; i < 2 * n_tiles; ++i) {
                bool is_v;
                int j;
                ring_tile<1>(i, n_tiles, is_v, j);
                ATTN_CHECK(j >= 0 && j < n_tiles && s.b < p.B && s.g < p.Hkv);
                const int tile = s.t0 + j;
                if (is_v && tile >= window + 32) {             // (K is at most two tiles ahead of V)
                    window += 32;
                    here = after;
                    after = lookup(window + 32);
                }
                ok = wait_bar(bar_empty(at.e), at.par ^ 1u);
                if (!ok) break;
                if (lane == 0) {
                    if (ATTN_DEBUG_BOUNDS) ring_tag[at.e] = at.item;
                    mbar_arrive_expect_tx(bar_full(at.e), static_cast<uint32_t>(L::kTileBytes));
                }
                const CUtensorMap* map = is_v ? &tm_v : &tm_k;
                const int k = tile - window;
                const int page = __shfl_sync(0xffffffffu, k < 32 ? here : after, k & 31);
                if (lane == 0) {
                    int row = tile * kTile, outer = s.b * p.Hkv + s.g;
                    if (p.block_table != nullptr) {
                        row %= p.page_size;
                        outer = page * p.Hkv + s.g;
                    }
                    decode_check_tile(p, row, outer);
                    const uint32_t dst = sKV + at.e * L::kTileBytes;
                    for (int kb = 0; kb < L::kKB; ++kb)
                        tma_load_3d(dst + kb * L::kBlockBytes, map, bar_full(at.e), kb * 64, row, outer);
                }
                at.next();
            }
        } while (ok && tree_next<kTile>(tp, s));
        if (!ok && lane == 0) {
            // unwinding after a timeout: let issued copies land first
            for (int k = min(at.item, L::kStages); k > 0; --k) {
                const int t = at.item - k;
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(bar_full(t % L::kStages), static_cast<uint32_t>(t / L::kStages) & 1u) &&
                       global_timer_ns() - t0 < 100000000ull) {
                }
            }
            const uint64_t t0 = global_timer_ns();
            while (!L::kQTmem && !mbar_try_wait(bar_q_full, s.n & 1) && global_timer_ns() - t0 < 100000000ull) {
            }
        }
        __syncwarp();
    } else if (warp == L::kMmaWarp) {
        // ================= MMA issuer (lane 0 issues; the warp mends V rows) =================
        constexpr uint32_t kIdescQK = umma_idesc_bf16_f32(128, kTile, false);
        constexpr uint32_t kIdescPV = umma_idesc_bf16_f32(128, D, true);
        const uint64_t dQ = umma_sdesc_sw128(sQ, 16, 1024);
        const uint64_t dK0 = umma_sdesc_sw128(sKV, 16, 1024);
        const uint64_t dV0 = umma_sdesc_sw128(sKV, L::kBlockBytes, 1024);
        constexpr uint64_t kEntryStep = L::kTileBytes >> 4;
        RingPos at;
        // Every step is the warp's, with one thread issuing, and every wait's outcome the warp's vote
        const uint32_t leader = lane == 0 ? 1u : 0u;
        auto wait_bar = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &g_attn_err, kDevErrTimeout)) != 0;
        };
        auto wait_item = [&]() {
            const bool got = wait_bar(bar_full(at.e), at.par);
            if (got) ATTN_CHECK(ring_tag[at.e] == at.item);   // (debug builds) the entry holds that item
            return got;
        };
        bool ok = true;
        int tile0 = 0;                             // tiles of the segments before
        TreeSeg s = first;
        do {
            const int n_tiles = s.t1 - s.t0;
            // S(j) = Q K_j^T (N = kTile cache rows)
            auto qk = [&](int j) {
                if (!wait_item()) return false;
                tc_fence_after_sync();
                const uint32_t d = tS((tile0 + j) & 1);
                const uint64_t b0 = dK0 + static_cast<uint64_t>(at.e) * kEntryStep;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t koff = static_cast<uint64_t>(((kk >> 2) * L::kBlockBytes + (kk & 3) * 32) >> 4);
                    if constexpr (L::kQTmem) {
                        umma_ts_by(leader, d, tmem + L::kTmemQ + kk * 8, b0 + koff, kIdescQK, kk > 0 ? 1u : 0u);
                    } else {
                        const uint64_t qoff = static_cast<uint64_t>(((kk >> 2) * L::kQBlockBytes + (kk & 3) * 32) >> 4);
                        umma_ss_by(leader, d, dQ + qoff, b0 + koff, kIdescQK, kk > 0 ? 1u : 0u);
                    }
                }
                umma_commit_by(leader, bar_s_full((tile0 + j) & 1));
                umma_commit_by(leader, bar_empty(at.e));
                if (!L::kQTmem && j + 1 == n_tiles) umma_commit_by(leader, bar_q_empty);
                at.next();
                return true;
            };
            const int ctx = s.seqlen - tree_len(tp, s.b);
            const int k_end = min(s.t1 * kTile, s.seqlen);
            ok = wait_bar(bar_q_full, s.n & 1);
            if (ok) ok = qk(0);
            if (ok && n_tiles > 1) ok = qk(1);
            for (int j = 0; j < n_tiles && ok; ++j) {
                const int jj = tile0 + j, buf = jj & 1;
                ok = wait_item();
                if (!ok) break;
                const int key0 = (s.t0 + j) * kTile;
                const int valid = min(kTile, k_end - key0);
                // rows of the tree, or past the last one: seldom
                if (key0 + kTile > ctx || valid < kTile) {
                    uint8_t* ent = smem + L::kKVOff + at.e * L::kTileBytes;
                    // non-finite elements of tree rows: zero, and noted for the epilogue
                    const int tree_lo = max(0, ctx - key0);
                    for (int kb = 0; kb < L::kKB; ++kb) {
                        uint8_t* blk = ent + kb * L::kBlockBytes;
#pragma unroll 4
                        for (int i = tree_lo * 128 + lane * 16; i < valid * 128; i += 32 * 16) {
                            uint4 x = *reinterpret_cast<const uint4*>(blk + i);
                            const uint32_t bad[4] = {nonfinite_bf16x2(x.x), nonfinite_bf16x2(x.y), nonfinite_bf16x2(x.z),
                                                     nonfinite_bf16x2(x.w)};
                            if (bad[0] | bad[1] | bad[2] | bad[3]) {
                                x = make_uint4(x.x & ~bad[0], x.y & ~bad[1], x.z & ~bad[2], x.w & ~bad[3]);
                                *reinterpret_cast<uint4*>(blk + i) = x;
                                v_patched[s.n & 1] = s.n + 1;
                            }
                        }
                        // V rows past the last row: zero (P is 0 there, but 0 * NaN is NaN)
                        for (int i = valid * 128 + lane * 16; i < L::kBlockBytes; i += 32 * 16)
                            *reinterpret_cast<uint4*>(blk + i) = make_uint4(0, 0, 0, 0);
                    }
                    __threadfence_block();
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                // P(j) is written, and, for the first tile, the epilogue before has read O
                ok = wait_bar(bar_p_full(buf), static_cast<uint32_t>(jj >> 1) & 1u);
                if (!ok) break;
                tc_fence_after_sync();
                // O += P(j) V_j: steps of 16 cache rows.  (A commit holds the tensor pipe up by about 100
                // cycles: the entry's release is also what the softmax waits on for O.)
                const uint64_t b0 = dV0 + static_cast<uint64_t>(at.e) * kEntryStep;
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    umma_ts_by(leader, tO, tS(buf) + kk * 8, b0 + static_cast<uint64_t>((kk * 2048) >> 4), kIdescPV,
                               (j > 0 || kk > 0) ? 1u : 0u);
                umma_commit_by(leader, bar_empty(at.e));
                at.next();
                if (j + 2 < n_tiles) ok = qk(j + 2);
            }
            tile0 += n_tiles;
        } while (ok && tree_next<kTile>(tp, s));
        if (lane == 0) {
            // Drain: no MMA may still be running when TMEM is released.
            umma_commit(bar_drain);
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(bar_drain, 0) && global_timer_ns() - t0 < 100000000ull) {
            }
        }
        __syncwarp();
    } else {
        // ================= softmax warpgroup (thread = row = TMEM lane) =================
        const int r = threadIdx.x;               // 0..127
        const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
        const uint32_t tOr = tO + lane_off;
        const int node = (mblk * 128 + r) % p.Lq;
        const float sl2 = p.scale_log2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        // A warp whose 32 rows are all padding (row >= R) only keeps the pipeline
        // moving: its P rows are never read into a real output row (the MMA keeps
        // rows apart), so it skips the softmax and just signals.
        const bool idle_warp = warp * 32 >= R;
        bool ok = true;
        int tile0 = 0;
        TreeSeg s = first;
        do {
            const int n_tiles = s.t1 - s.t0;
            const size_t row = (static_cast<size_t>(s.b) * p.Hq + static_cast<size_t>(s.g) * p.G) * p.Lq + mblk * 128 +
                               (r < R ? r : 0);
            if constexpr (L::kQTmem) {
                // Q's row to TMEM (the last S of the segment before is complete, so its Q is used)
                const uint4* src = reinterpret_cast<const uint4*>(p.q + row * D);
                uint4 x[D / 8];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) x[i] = r < R ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < D / 8; i += 8)
                    tmem_st_32x32b_x32(tmem + L::kTmemQ + lane_off + i * 4, reinterpret_cast<const uint32_t*>(x + i));
                tmem_wait_st();
                tc_fence_before_sync();
                mbar_arrive(bar_q_full);
            }
            const int n_tree = tree_len(tp, s.b);
            const int ctx = s.seqlen - n_tree;     // rows every node sees (negative: the tree's first rows are not cached)
            const int k_end = min(s.t1 * kTile, s.seqlen);
            const bool live = r < R && node < n_tree;
            const uint32_t* words = tp.mask + static_cast<size_t>(s.b) * tp.mask_batch + static_cast<size_t>(node) * tp.W;
            const int free_end = min(ctx, k_end);  // rows below it need no mask
            // O += P V of tile j is done: V_j's ring entry is released.  (The entry cannot be released
            // again before this wait: what comes into it next is used after P of a later tile.)
            auto wait_o = [&](int j) {
                const int item = 2 * tile0 + ring_pos_v<1>(j, n_tiles);
                return mbar_wait(bar_empty(item % L::kStages), static_cast<uint32_t>(item / L::kStages) & 1u, abort_flag,
                                 &g_attn_err, kDevErrTimeout);
            };
            // l_run: row sum of P as rounded to bf16 (normalises O); l_exact: of the
            // unrounded exponentials (for the log-sum-exp)
            float m_run = -INFINITY, l_run = 0.0f, l_exact = 0.0f;
            for (int j = 0; j < n_tiles; ++j) {
                const int jj = tile0 + j, buf = jj & 1;
                ok = mbar_wait(bar_s_full(buf), static_cast<uint32_t>(jj >> 1) & 1u, abort_flag, &g_attn_err,
                               kDevErrTimeout);
                if (!ok) break;
                tc_fence_after_sync();
                if (idle_warp) {
                    tc_fence_before_sync();
                    mbar_arrive(bar_p_full(buf));
                    continue;
                }
                const uint32_t tSr = tS(buf) + lane_off;
                const int key0 = (s.t0 + j) * kTile;
                // the tile's scores of this row, read from TMEM once
                uint32_t v[kTile];
                tmem_ld_32x32b_x32(tSr, v);
                tmem_ld_32x32b_x32(tSr + 32, v + 32);
                tmem_wait_ld();
                reg_fence<kTile>(v);
                if (key0 + kTile > free_end) {
                    const uint64_t vis = tree_visible(words, tp.W, ctx, key0) & low_bits(k_end - key0);
                    const uint32_t vlo = static_cast<uint32_t>(vis), vhi = static_cast<uint32_t>(vis >> 32);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (!(vlo >> i & 1u)) v[i] = __float_as_uint(-INFINITY);
                        if (!(vhi >> i & 1u)) v[32 + i] = __float_as_uint(-INFINITY);
                    }
                }
                float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                for (int i = 0; i < kTile; i += 8) {
                    mx0 = fmax3(mx0, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                    mx1 = fmax3(mx1, __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                    mx2 = fmax3(mx2, __uint_as_float(v[i + 4]), __uint_as_float(v[i + 5]));
                    mx3 = fmax3(mx3, __uint_as_float(v[i + 6]), __uint_as_float(v[i + 7]));
                }
                const float m_tile = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * sl2;
                float factor = 1.0f;
                if (m_tile > m_run + kDtcRescaleLog2) {
                    factor = (m_run == -INFINITY) ? 0.0f : ex2_approx(m_run - m_tile);
                    m_run = m_tile;
                    l_run *= factor;
                    l_exact *= factor;
                }
                if (j > 0 && __any_sync(0xffffffffu, factor != 1.0f)) {
                    // O must hold the tiles before: the last one's O += P V is the only one that can be in flight
                    if (!wait_o(j - 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint64_t f2 = f2_pack(factor, factor);
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld_32x32b_x16(tOr + c, o);
                        tmem_wait_ld();
                        reg_fence<16>(o);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float a0, a1;
                            f2_unpack(f2_mul(f2_pack(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), f2), a0, a1);
                            o[i] = __float_as_uint(a0);
                            o[i + 1] = __float_as_uint(a1);
                        }
                        tmem_st_32x32b_x16(tOr + c, o);
                    }
                    tmem_wait_st();
                }
                // exponentials, row sums, P (bf16) over the S columns already read
                const float m_sub = (m_run == -INFINITY) ? 0.0f : m_run;
                const uint64_t negm2 = f2_pack(-m_sub, -m_sub);
                uint64_t acc_r = 0ull, acc_e = 0ull;
#pragma unroll
                for (int c = 0; c < kTile; c += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t t = f2_fma(f2_pack(__uint_as_float(v[c + 2 * i]), __uint_as_float(v[c + 2 * i + 1])),
                                                  sl2x2, negm2);
                        float t0, t1;
                        f2_unpack(t, t0, t1);
                        const float e0 = ex2_approx(t0), e1 = ex2_approx(t1);
                        pk[i] = pack_bf16x2(e0, e1);
                        acc_e = f2_add(acc_e, f2_pack(e0, e1));
                        acc_r = f2_add(acc_r, bf16x2_to_f2(pk[i]));   // P as the MMA sees it
                    }
                    tmem_st_32x32b_x16(tSr + c / 2, pk);
                }
                tmem_wait_st();
                tc_fence_before_sync();
                mbar_arrive(bar_p_full(buf));
                float a0, a1, e0, e1;
                f2_unpack(acc_r, a0, a1);
                f2_unpack(acc_e, e0, e1);
                l_run += a0 + a1;
                l_exact += e0 + e1;
            }
            if (!ok) break;
            // ---- the segment's O / l and log-sum-exp per row: the result, or a partial (fp32, log2) ----
            ok = wait_o(n_tiles - 1);
            if (!ok) break;
            tc_fence_after_sync();
            if (!idle_warp) {
                const bool whole = s.t0 == 0 && s.t1 == s.tiles;
                const bool row_valid = r < R;
                // a row that saw nothing here, or is no node: 0, and weight 0 in the combine
                const bool seen = live && !(l_exact == 0.0f);
                const float inv_l = seen ? 1.0f / l_run : 0.0f;
                const float lse2 = seen ? m_run + __log2f(l_exact) : -INFINITY;
                const size_t part = tree_part(tp, range, mblk, s.n == 0 ? 0 : 1);
                float* const o_part = p.o_part + part * box * D + tree_part_at(box, row_valid ? r : 0, 0);
                ATTN_CHECK(row < static_cast<size_t>(p.B) * p.Hq * p.Lq);
                ATTN_CHECK(whole || part < static_cast<size_t>(tp.n_ranges) * tp.n_mblk * 2);
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(tOr + c, o);
                    tmem_wait_ld();
                    reg_fence<32>(o);
                    float x[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) x[k] = seen ? __uint_as_float(o[k]) * inv_l : 0.0f;
                    if (row_valid && whole) {
                        __nv_bfloat16* dst = tp.out + row * D + c;
#pragma unroll
                        for (int k = 0; k < 32; k += 8)
                            *reinterpret_cast<uint4*>(dst + k) =
                                make_uint4(pack_bf16x2(x[k], x[k + 1]), pack_bf16x2(x[k + 2], x[k + 3]),
                                           pack_bf16x2(x[k + 4], x[k + 5]), pack_bf16x2(x[k + 6], x[k + 7]));
                    } else if (row_valid) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4*>(o_part + static_cast<size_t>(c + k) * box) =
                                make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
                    }
                }
                // elements that the node sees and that are not finite
                if (seen && v_patched[s.n & 1] == s.n + 1) {
                    if (whole)
                        tree_add_nonfinite(tp, s.b, s.g, words, ctx, 0, k_end, D, tp.out + row * D, 4);
                    else
                        tree_add_nonfinite(tp, s.b, s.g, words, ctx, s.t0 * kTile, k_end, D, o_part, box * 4);
                }
                if (row_valid) {
                    if (!whole)
                        p.lse_part[part * box + r] = lse2;
                    else if (tp.lse != nullptr)
                        tp.lse[row] = lse2 * kLn2;
                }
            }
            // O is read: the arrival on P of the next segment's first tile lets it be written
            tc_fence_before_sync();
            tile0 += n_tiles;
        } while (tree_next<kTile>(tp, s));
    }

    // ---- teardown ----
    tc_fence_before_sync();
    __syncthreads();
    if (warp == L::kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// Where the partials of a (sequence, KV head) pair lie.
struct TreeParts {
    long long r0;             // their first range
    int n;                    // how many; 0: the sequence has no rows, 1: the result is written
    bool late;                // the first one is its range's last segment

    template <int TILE>
    __device__ __forceinline__ void find(const TreeParams& tp, int pair) {
        const int b = pair / tp.d.Hkv, g = pair - b * tp.d.Hkv;
        const int tiles = tree_tiles<TILE>(decode_seqlen(tp.d, b));
        const long long per = tp.tiles_before[tp.d.B];
        const long long start = tp.tiles_before[b] * tp.d.Hkv + static_cast<long long>(g) * tiles;
        r0 = 0;
        n = 0;
        late = false;
        if (tiles > 0) {
            r0 = start / per;
            n = static_cast<int>((start + tiles - 1) / per - r0) + 1;
            late = start != r0 * per;
        }
    }
    // partial k of query block mblk (past the last one: the last one)
    __device__ __forceinline__ size_t at(const TreeParams& tp, int k, int mblk) const {
        k = min(k, n - 1);
        return tree_part(tp, r0 + k, mblk, k == 0 && late ? 1 : 0);
    }
};

// Running maximum, sum and O (C groups of four columns) of one row's partials.
template <int C>
struct TreeMerge {
    float M = -INFINITY, sum = 0.0f;
    float4 acc[C] = {};

    __device__ __forceinline__ void scale(float f) {
        sum *= f;
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] = make_float4(acc[i].x * f, acc[i].y * f, acc[i].z * f, acc[i].w * f);
    }
    // weight w: a partial that saw nothing has 0 and may hold anything
    __device__ __forceinline__ void add(float w, float part_sum, const float4 (&o)[C]) {
        sum = w == 0.0f ? sum : fmaf(w, part_sum, sum);
        if (w != 0.0f) {
#pragma unroll
            for (int i = 0; i < C; ++i)
                acc[i] = make_float4(fmaf(w, o[i].x, acc[i].x), fmaf(w, o[i].y, acc[i].y), fmaf(w, o[i].z, acc[i].z),
                                     fmaf(w, o[i].w, acc[i].w));
        }
    }
    template <int N>
    __device__ __forceinline__ void add(const float (&ls)[N], const float4 (&ov)[N][C]) {
        float top = M;
#pragma unroll
        for (int u = 0; u < N; ++u) top = fmaxf(top, ls[u]);
        scale(M == -INFINITY ? 1.0f : ex2_approx(M - top));   // (M = -inf: sum is 0, or NaN to stay)
        M = top;
#pragma unroll
        for (int u = 0; u < N; ++u) add(ls[u] == -INFINITY ? 0.0f : ex2_approx(ls[u] - M), 1.0f, ov[u]);
    }
    // a sum of 0: the row saw nothing; NaN: a score was
    __device__ __forceinline__ float lse() const { return sum == 0.0f ? -INFINITY : (M + __log2f(sum)) * kLn2; }
    __device__ __forceinline__ float inv() const { return sum == 0.0f ? 0.0f : 1.0f / sum; }
};

// out = sum_k 2^(lse_k - lse) O_k, lse = log2 sum_k 2^lse_k over the partials of a pair that lies in
// several ranges; rows of sequences without rows get 0 and -inf; the rows of other pairs are there
// already.  A lane takes a row, a warp 16 columns of 32 rows.  WPP = 1: all partials, two at a time,
// the CTA's four warps 64 columns.  WPP = 4: every fourth partial, four at a time, the CTA's warps the
// same 16 columns; they meet in shared memory.
constexpr int kTreeCombineRows = 32;

template <int D, int WPP>
__global__ void __launch_bounds__(128) attn_tree_combine_kernel(const TreeParams tp) {
    grid_dep_wait();   // launched as a programmatic dependent of attn_tree_kernel
    constexpr int kColCtas = D / 16 / (4 / WPP), C = 4, kInFlight = WPP == 1 ? 2 : 4;
    const DecodeParams& p = tp.d;
    const int RG = p.G * p.Lq, box = min(128, RG);
    const int slices = (RG + kTreeCombineRows - 1) / kTreeCombineRows;      // (128 is a multiple of their rows)
    const int unit = blockIdx.x / kColCtas, pair = unit / slices;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = WPP == 1 ? 0 : warp;
    const int rr = (unit - pair * slices) * kTreeCombineRows + lane;
    const int col0 = (static_cast<int>(blockIdx.x % kColCtas) * (4 / WPP) + (WPP == 1 ? warp : 0)) * 16;
    TreeParts parts;
    parts.find<TreeCfg<D>::kTile>(tp, pair);
    if (parts.n == 1) return;                      // uniform over the CTA
    const int row = min(rr, RG - 1), mblk = row / 128, r = row % 128;
    TreeMerge<C> m;
    for (int k0 = sub; k0 < parts.n; k0 += WPP * kInFlight) {
        float ls[kInFlight];
        float4 ov[kInFlight][C];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int k = k0 + u * WPP;
            const size_t part = parts.at(tp, k, mblk);
            ls[u] = k < parts.n ? p.lse_part[part * box + r] : -INFINITY;
            const float* src = p.o_part + part * box * D + tree_part_at(box, r, col0);
#pragma unroll
            for (int i = 0; i < C; ++i) ov[u][i] = *reinterpret_cast<const float4*>(src + static_cast<size_t>(i) * box * 4);
        }
        m.add(ls, ov);
    }
    if constexpr (WPP > 1) {
        __shared__ float s_m[WPP][32], s_sum[WPP][32];
        __shared__ float4 s_acc[WPP][C][32];
        s_m[warp][lane] = m.M;
        s_sum[warp][lane] = m.sum;
#pragma unroll
        for (int i = 0; i < C; ++i) s_acc[warp][i][lane] = m.acc[i];
        __syncthreads();
        if (warp != 0) return;
        m = TreeMerge<C>();
#pragma unroll
        for (int w = 0; w < WPP; ++w) m.M = fmaxf(m.M, s_m[w][lane]);
#pragma unroll
        for (int w = 0; w < WPP; ++w) {
            float4 o[C];
#pragma unroll
            for (int i = 0; i < C; ++i) o[i] = s_acc[w][i][lane];
            m.add(s_m[w][lane] == -INFINITY ? 1.0f : ex2_approx(s_m[w][lane] - m.M), s_sum[w][lane], o);   // (-inf: sum 0, or NaN)
        }
    }
    if (rr >= RG) return;
    const float inv = m.inv();
    const size_t orow = static_cast<size_t>(pair) * RG + rr;
    uint4* o = reinterpret_cast<uint4*>(tp.out + orow * D + col0);
#pragma unroll
    for (int i = 0; i < C; i += 2)
        o[i / 2] = make_uint4(pack_bf16x2(m.acc[i].x * inv, m.acc[i].y * inv), pack_bf16x2(m.acc[i].z * inv, m.acc[i].w * inv),
                              pack_bf16x2(m.acc[i + 1].x * inv, m.acc[i + 1].y * inv),
                              pack_bf16x2(m.acc[i + 1].z * inv, m.acc[i + 1].w * inv));
    if (tp.lse != nullptr && col0 == 0) tp.lse[orow] = m.lse();
}

// The same for pairs of fewer rows than a warp has lanes: a lane takes four columns of a row (32 lanes:
// neighbours in the partial, whatever its rows), the CTA's four warps every fourth partial, eight at a
// time, and they meet in shared memory.
template <int D>
__global__ void __launch_bounds__(128) attn_tree_combine_few_rows_kernel(const TreeParams tp) {
    grid_dep_wait();
    constexpr int kInFlight = 8;
    const DecodeParams& p = tp.d;
    const int RG = p.G * p.Lq, box = min(128, RG), groups = box * (D / 4), ctas = (groups + 31) / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = blockIdx.x / ctas, pair = unit / tp.n_mblk, mblk = unit - pair * tp.n_mblk;
    const int e = min(static_cast<int>(blockIdx.x - unit * ctas) * 32 + lane, groups - 1), c4 = e / box, r = e - c4 * box;
    TreeParts parts;
    parts.find<TreeCfg<D>::kTile>(tp, pair);
    if (parts.n == 1) return;                      // uniform over the CTA
    TreeMerge<1> m;
    for (int k0 = warp; k0 < parts.n; k0 += 4 * kInFlight) {
        float ls[kInFlight];
        float4 ov[kInFlight][1];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int k = k0 + 4 * u;
            const size_t part = parts.at(tp, k, mblk);
            ls[u] = k < parts.n ? p.lse_part[part * box + r] : -INFINITY;
            ov[u][0] = *reinterpret_cast<const float4*>(p.o_part + (part * box * (D / 4) + e) * 4);
        }
        m.add(ls, ov);
    }
    __shared__ float s_m[4][32], s_sum[4][32];
    __shared__ float4 s_acc[4][32];
    s_m[warp][lane] = m.M;
    s_sum[warp][lane] = m.sum;
    s_acc[warp][lane] = m.acc[0];
    __syncthreads();
    if (warp != 0 || mblk * 128 + r >= RG) return;
    TreeMerge<1> all;
#pragma unroll
    for (int w = 0; w < 4; ++w) all.M = fmaxf(all.M, s_m[w][lane]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float4 o[1] = {s_acc[w][lane]};
        all.add(s_m[w][lane] == -INFINITY ? 1.0f : ex2_approx(s_m[w][lane] - all.M), s_sum[w][lane], o);   // (-inf: sum 0, or NaN)
    }
    const float inv = all.inv();
    const size_t orow = static_cast<size_t>(pair) * RG + mblk * 128 + r;
    *reinterpret_cast<uint2*>(tp.out + orow * D + c4 * 4) =
        make_uint2(pack_bf16x2(all.acc[0].x * inv, all.acc[0].y * inv), pack_bf16x2(all.acc[0].z * inv, all.acc[0].w * inv));
    if (tp.lse != nullptr && c4 == 0) tp.lse[orow] = all.lse();
}

}  // namespace attn
