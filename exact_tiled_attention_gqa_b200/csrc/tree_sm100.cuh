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
// The G x T query rows of a KV head are cut into blocks of 128, the M rows of the MMAs
// (S = Q K^T and O += P V on 64-row tiles, as attn_decode_tc_kernel: two S buffers, P over
// S in TMEM, lazy maximum).  The work is balanced from the lengths on the device: the 64-row
// tiles of all (sequence, KV head) pairs in one line are cut into equal ranges, one CTA for
// each range and query block, as many CTAs as the GPU holds at once.  A CTA walks its range
// segment by segment (a segment: the part of one pair's tiles in the range); the CTAs of one
// range read the same K and V side by side, so all but one of them find them in the L2.  A
// segment that is a whole pair writes the result; the others write a normalised partial (at
// most two a CTA) that attn_tree_combine_kernel merges.  The loads run on across segments.
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
    int min_tiles;               // a range is no shorter
};

__device__ __forceinline__ int tree_tiles(int seqlen) { return seqlen / 64 + (seqlen % 64 != 0); }

// Row r of the partial that range `range` wrote for query block mblk in slot 0 (its first
// segment) or 1 (its last).
__device__ __forceinline__ size_t tree_part(const TreeParams& p, long long range, int mblk, int slot, int r) {
    return ((static_cast<size_t>(range) * p.n_mblk + mblk) * 2 + slot) * min(128, p.d.G * p.d.Lq) + r;
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
// themselves).
template <typename T>
__device__ __noinline__ void tree_add_nonfinite(const TreeParams& tp, int b, int g, const uint32_t* words, int ctx,
                                                int k_begin, int k_end, int D, T* dst) {
    for (int row = max(ctx, k_begin); row < k_end; ++row) {
        const int j = row - ctx;
        if (!(words[j >> 5] >> (j & 31) & 1u)) continue;
        const __nv_bfloat16* src = tp.v + tree_cache_row(tp.d, b, g, row) * D;
        for (int c = 0; c < D; ++c) {
            const float x = __bfloat162float(src[c]);
            if (!isfinite(x)) dst[c] = static_cast<T>(static_cast<float>(dst[c]) + x);
        }
    }
}

// All ones over the halves of a bf16 pair that are infinite or NaN.
__device__ __forceinline__ uint32_t nonfinite_bf16x2(uint32_t x) {
    return ((x & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((x & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

template <int D>
struct TreeSmem : DecodeTcSmem<D> {
    using B = DecodeTcSmem<D>;
    static constexpr int kNumBars = B::kNumBars + 1;                  // and q_empty
    static constexpr int kMiscOff = B::kBarOff + kNumBars * 8;        // tmem base, abort flag, patched[2]
    static constexpr int kTagOff = kMiscOff + 16;
    static constexpr int kAlloc = kTagOff + 4 * B::kStages + 1024;
    static_assert(kAlloc <= 232448, "dynamic shared memory per CTA");
};

// Part of one (sequence, KV head) pair's tiles in a CTA's range.
struct TreeSeg {
    long long x, x_end;       // tiles of the line still to do: this segment starts at x
    int b, g;
    int seqlen, tiles;        // of the pair
    int t0, t1;               // the segment's tiles
    int n;                    // segments before it
};

// The segment at s.x; false when the range is done.  s.b, s.g, s.seqlen and s.tiles are set.
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
            s.tiles = tree_tiles(s.seqlen);
        } while (s.tiles == 0);
    }
    s.t1 = static_cast<int>(min(static_cast<long long>(s.tiles), s.x_end - s.x));
    return true;
}

template <int D>
__global__ void __launch_bounds__(kDtcThreads, DecodeTcSmem<D>::kCtasPerSm)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const TreeParams tp) {
    grid_dep_release();   // the combine launch may be scheduled now
    using L = TreeSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long s_warp[kDtcThreads / 32], s_before;
    __shared__ int s_b;
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_base);

    const DecodeParams& p = tp.d;
    const int range = blockIdx.x / tp.n_mblk, mblk = blockIdx.x % tp.n_mblk;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // ---- this CTA's range of the line of tiles ----
    const int per_thread = (p.B + kDtcThreads - 1) / kDtcThreads;
    const int my_b = min(p.B, static_cast<int>(threadIdx.x) * per_thread), my_end = min(p.B, my_b + per_thread);
    long long mine = 0;
    for (int b = my_b; b < my_end; ++b) mine += tree_tiles(decode_seqlen(p, b));
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
    for (int w = 0; w < kDtcThreads / 32; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    total *= p.Hkv;
    const long long per = max((total + tp.n_ranges - 1) / tp.n_ranges, static_cast<long long>(tp.min_tiles));
    if (blockIdx.x == 0) {                        // for the combine
        long long t = before;
        for (int b = my_b; b < my_end; ++b) {
            tp.tiles_before[b] = t;
            t += tree_tiles(decode_seqlen(p, b));
        }
        if (threadIdx.x == 0) tp.tiles_before[p.B] = per;
    }
    TreeSeg first;
    first.x = range * per;
    first.x_end = min(first.x + per, total);
    if (first.x >= first.x_end) return;           // uniform: nothing left for this range
    if (before * p.Hkv <= first.x && first.x < (before + mine) * p.Hkv) {
        int b = my_b;
        for (int t; first.x >= (before + (t = tree_tiles(decode_seqlen(p, b)))) * p.Hkv; ++b) before += t;
        s_b = b;
        s_before = before;
    }

    const int RG = p.G * p.Lq;                     // query rows of a KV head
    const int R = min(128, RG - mblk * 128);       // of this block
    const int box = min(128, RG);                  // rows TMA loads (past the block's: another head's, or 0)

    const uint32_t sQ = base + L::kQOff;
    const uint32_t sKV = base + L::kKVOff;
    const uint32_t bar0 = base + L::kBarOff;
    const uint32_t bar_q_full = bar0;
    auto bar_full = [&](int s) { return bar0 + 8u * (1 + s); };
    auto bar_empty = [&](int s) { return bar0 + 8u * (1 + L::kStages + s); };
    auto bar_s_full = [&](int i) { return bar0 + 8u * (1 + 2 * L::kStages + i); };
    auto bar_p_full = [&](int i) { return bar0 + 8u * (3 + 2 * L::kStages + i); };
    const uint32_t bar_o_ready = bar0 + 8u * (5 + 2 * L::kStages);
    const uint32_t bar_o_done = bar_o_ready + 8u;
    const uint32_t bar_drain = bar_o_ready + 16u;
    const uint32_t bar_q_empty = bar_o_ready + 24u;
    uint32_t* tmem_base_ptr = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
    // segment n whose tree rows lost non-finite elements: n + 1 in entry n % 2 (the MMA warp is
    // at most one segment ahead of the epilogue)
    volatile int* v_patched = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 8);
    // (debug builds) the ring position the producer put in each entry, checked by the MMA warp
    volatile int* ring_tag = reinterpret_cast<volatile int*>(smem + L::kTagOff);

    if (threadIdx.x == 0) {
        mbar_init(bar_q_full, 1);
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
        mbar_init(bar_o_ready, 1);
        mbar_init(bar_o_done, 1);
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    // query rows past the box are not loaded: make them zero (finite) for the MMA
    if (box < 128) {
        const int pad = (128 - box) * 128;
        for (int kb = 0; kb < L::kKB; ++kb) {
            uint8_t* blk = smem + L::kQOff + kb * L::kQBlockBytes + box * 128;
            for (int i = threadIdx.x * 16; i < pad; i += kDtcThreads * 16)
                *reinterpret_cast<uint4*>(blk + i) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
    }
    if (warp == kDtcMmaWarp) {
        tmem_alloc(smem_u32(tmem_base_ptr), L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_base_ptr;
    const uint32_t tS[2] = {tmem, tmem + 64u};    // S buffers (P over the first 32 columns)
    const uint32_t tO = tmem + 128u;               // O

    first.n = 0;
    first.b = s_b;
    first.seqlen = decode_seqlen(p, first.b);
    first.tiles = tree_tiles(first.seqlen);
    {
        const long long in_b = first.x - s_before * p.Hkv;
        first.g = static_cast<int>(in_b / first.tiles);
        first.t0 = static_cast<int>(in_b - static_cast<long long>(first.g) * first.tiles);
        first.t1 = static_cast<int>(min(static_cast<long long>(first.tiles), first.t0 + (first.x_end - first.x)));
    }

    // The ring's items are numbered through the whole range; a segment's, from 2 x its tiles before:
    // K_0 K_1 V_0 K_2 V_1 ...
    auto slot_of = [&](int t) { return t % L::kStages; };
    auto par_of = [&](int t) { return static_cast<uint32_t>(t / L::kStages) & 1u; };

    if (warp == kDtcProducerWarp) {
        // ================= TMA producer =================
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
            int issued = 0;
            bool ok = true;
            TreeSeg s = first;
            do {
                const int n_tiles = s.t1 - s.t0, item0 = issued;
                // (its last Q K^T is two tiles before the end of the segment before)
                ok = mbar_wait(bar_q_empty, (s.n & 1) ^ 1u, abort_flag, &g_attn_err, kDevErrTimeout);
                if (!ok) break;
                const size_t row0 = (static_cast<size_t>(s.b) * p.Hq + static_cast<size_t>(s.g) * p.G) * p.Lq + mblk * 128;
                mbar_arrive_expect_tx(bar_q_full, static_cast<uint32_t>(L::kKB * box * 128));
                for (int kb = 0; kb < L::kKB; ++kb)
                    tma_load_3d(sQ + kb * L::kQBlockBytes, &tm_q, bar_q_full, kb * 64, static_cast<int>(row0), 0);
                for (int i = 0; i < 2 * n_tiles; ++i) {
                    const int t = item0 + i, e = slot_of(t);
                    ok = mbar_wait(bar_empty(e), par_of(t) ^ 1u, abort_flag, &g_attn_err, kDevErrTimeout);
                    if (!ok) break;
                    bool is_v;
                    int j;
                    ring_tile<1>(i, n_tiles, is_v, j);
                    const int key0 = (s.t0 + j) * kDtcBN;
                    int row = key0, outer = s.b * p.Hkv + s.g;
                    if (p.block_table != nullptr) {
                        int page = __ldg(p.block_table + static_cast<size_t>(s.b) * p.max_pages + key0 / p.page_size);
                        if (page < 0 || page >= p.n_pages) {
                            atomicOr(&g_attn_err, kDevErrPage);
                            page = 0;
                        }
                        row = key0 % p.page_size;
                        outer = page * p.Hkv + s.g;
                    }
                    decode_check_tile(p, row, outer);
                    ATTN_CHECK(j >= 0 && j < n_tiles && s.b < p.B && s.g < p.Hkv);
                    if (ATTN_DEBUG_BOUNDS) ring_tag[e] = t;
                    mbar_arrive_expect_tx(bar_full(e), L::kHalfBytes);
                    const CUtensorMap* map = is_v ? &tm_v : &tm_k;
                    const uint32_t dst = sKV + e * L::kHalfBytes;
                    for (int kb = 0; kb < L::kKB; ++kb)
                        tma_load_3d(dst + kb * L::kHalfBlockBytes, map, bar_full(e), kb * 64, row, outer);
                    issued = t + 1;
                }
            } while (ok && tree_next(tp, s));
            if (!ok) {
                // unwinding after a timeout: let issued copies land first
                for (int t = max(0, issued - L::kStages); t < issued; ++t) {
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait(bar_full(slot_of(t)), par_of(t)) && global_timer_ns() - t0 < 100000000ull) {
                    }
                }
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(bar_q_full, s.n & 1) && global_timer_ns() - t0 < 100000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == kDtcMmaWarp) {
        // ================= MMA issuer (lane 0 issues; the warp mends V rows) =================
        constexpr uint32_t kIdescQK = umma_idesc_bf16_f32(128, kDtcBN, false);
        constexpr uint32_t kIdescPV = umma_idesc_bf16_f32(128, D, true);
        const uint64_t dQ = umma_sdesc_sw128(sQ, 16, 1024);
        const uint64_t dK0 = umma_sdesc_sw128(sKV, 16, 1024);
        const uint64_t dV0 = umma_sdesc_sw128(sKV, L::kHalfBlockBytes, 1024);
        constexpr uint64_t kSlotStep = L::kHalfBytes >> 4;
        auto wait_item = [&](int it) {
            const bool got = mbar_wait(bar_full(slot_of(it)), par_of(it), abort_flag, &g_attn_err, kDevErrTimeout);
            if (got) ATTN_CHECK(ring_tag[slot_of(it)] == it);   // (debug builds) the entry holds that item
            return got;
        };
        bool ok = true;
        int tile0 = 0;                             // tiles of the segments before
        TreeSeg s = first;
        do {
            const int n_tiles = s.t1 - s.t0, item0 = 2 * tile0;
            // S(j) = Q K_j^T into the buffer of tile tile0 + j (N = 64 cache rows)
            auto qk = [&](int j) {
                const int it = item0 + ring_pos_k<1>(j), buf = (tile0 + j) & 1;
                if (!wait_item(it)) return false;
                tc_fence_after_sync();
                if (lane == 0) {
                    const uint64_t b0 = dK0 + static_cast<uint64_t>(slot_of(it)) * kSlotStep;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t qoff = static_cast<uint64_t>(((kk >> 2) * L::kQBlockBytes + (kk & 3) * 32) >> 4);
                        const uint64_t koff = static_cast<uint64_t>(((kk >> 2) * L::kHalfBlockBytes + (kk & 3) * 32) >> 4);
                        umma_ss(tS[buf], dQ + qoff, b0 + koff, kIdescQK, kk > 0 ? 1u : 0u);
                    }
                    umma_commit(bar_empty(slot_of(it)));
                    umma_commit(bar_s_full(buf));
                    if (j + 1 == n_tiles) umma_commit(bar_q_empty);
                }
                __syncwarp();
                return true;
            };
            const int ctx = s.seqlen - tree_len(tp, s.b);
            const int k_end = min(s.t1 * kDtcBN, s.seqlen);
            ok = mbar_wait(bar_q_full, s.n & 1, abort_flag, &g_attn_err, kDevErrTimeout);
            if (ok) ok = qk(0);
            if (ok && n_tiles > 1) ok = qk(1);
            for (int j = 0; j < n_tiles && ok; ++j) {
                const int buf = (tile0 + j) & 1;
                const int itv = item0 + ring_pos_v<1>(j, n_tiles);
                ok = wait_item(itv);
                if (!ok) break;
                const int key0 = (s.t0 + j) * kDtcBN;
                const int valid = k_end - key0;
                uint8_t* ent = smem + L::kKVOff + slot_of(itv) * L::kHalfBytes;
                bool wrote = false;
                // non-finite elements of tree rows: zero, and noted for the epilogue
                const int tree_lo = max(0, ctx - key0), tree_hi = min(kDtcBN, valid);
                if (tree_lo < tree_hi) {
                    for (int kb = 0; kb < L::kKB; ++kb) {
                        uint8_t* blk = ent + kb * L::kHalfBlockBytes;
#pragma unroll 4
                        for (int i = tree_lo * 128 + lane * 16; i < tree_hi * 128; i += 32 * 16) {
                            uint4 x = *reinterpret_cast<const uint4*>(blk + i);
                            const uint32_t bad[4] = {nonfinite_bf16x2(x.x), nonfinite_bf16x2(x.y), nonfinite_bf16x2(x.z),
                                                     nonfinite_bf16x2(x.w)};
                            if (bad[0] | bad[1] | bad[2] | bad[3]) {
                                x = make_uint4(x.x & ~bad[0], x.y & ~bad[1], x.z & ~bad[2], x.w & ~bad[3]);
                                *reinterpret_cast<uint4*>(blk + i) = x;
                                wrote = true;
                                v_patched[s.n & 1] = s.n + 1;
                            }
                        }
                    }
                }
                // V rows past the last row: zero (P is 0 there, but 0 * NaN is NaN)
                if (valid < kDtcBN) {
                    for (int kb = 0; kb < L::kKB; ++kb) {
                        uint8_t* blk = ent + kb * L::kHalfBlockBytes + valid * 128;
                        for (int i = lane * 16; i < (kDtcBN - valid) * 128; i += 32 * 16)
                            *reinterpret_cast<uint4*>(blk + i) = make_uint4(0, 0, 0, 0);
                    }
                    wrote = true;
                }
                if (__any_sync(0xffffffffu, wrote)) {
                    __threadfence_block();
                    fence_proxy_async_smem();
                }
                __syncwarp();
                // P(j) is written, and, for the first tile, the epilogue before has read O
                ok = mbar_wait(bar_p_full(buf), static_cast<uint32_t>((tile0 + j) >> 1) & 1u, abort_flag, &g_attn_err,
                               kDevErrTimeout);
                if (!ok) break;
                __syncwarp();
                tc_fence_after_sync();
                if (lane == 0) {
                    // O += P(j) V_j: 4 steps of 16 cache rows
                    const uint64_t b0 = dV0 + static_cast<uint64_t>(slot_of(itv)) * kSlotStep;
#pragma unroll
                    for (int kk = 0; kk < kDtcBN / 16; ++kk)
                        umma_ts(tO, tS[buf] + kk * 8, b0 + static_cast<uint64_t>((kk * 2048) >> 4), kIdescPV,
                                (j > 0 || kk > 0) ? 1u : 0u);
                    umma_commit(bar_o_ready);
                    if (j + 1 == n_tiles) umma_commit(bar_o_done);
                    umma_commit(bar_empty(slot_of(itv)));
                }
                __syncwarp();
                if (j + 2 < n_tiles) ok = qk(j + 2);
            }
            tile0 += n_tiles;
        } while (ok && tree_next(tp, s));
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
            const int n_tree = tree_len(tp, s.b);
            const int ctx = s.seqlen - n_tree;     // rows every node sees (negative: the tree's first rows are not cached)
            const int k_end = min(s.t1 * kDtcBN, s.seqlen);
            const bool live = r < R && node < n_tree;
            const uint32_t* words = tp.mask + static_cast<size_t>(s.b) * tp.mask_batch + static_cast<size_t>(node) * tp.W;
            const int free_end = min(ctx, k_end);  // rows below it need no mask
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
                const uint32_t tSr = tS[buf] + lane_off;
                const int key0 = (s.t0 + j) * kDtcBN;
                const bool masked = key0 + kDtcBN > free_end;
                // the tile's 64 scores of this row, read from TMEM once
                uint32_t v[kDtcBN];
                tmem_ld_32x32b_x32(tSr, v);
                tmem_ld_32x32b_x32(tSr + 32, v + 32);
                tmem_wait_ld();
                reg_fence<kDtcBN>(v);
                if (masked) {
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
                for (int i = 0; i < kDtcBN; i += 8) {
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
                    // O must hold the tiles before: O += P V of the last one is the only one that can be in flight
                    if (!mbar_wait(bar_o_ready, static_cast<uint32_t>(jj - 1) & 1u, abort_flag, &g_attn_err,
                                   kDevErrTimeout)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint64_t f2 = f2_pack(factor, factor);
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(tOr + c, o);
                        tmem_wait_ld();
                        reg_fence<32>(o);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float a0, a1;
                            f2_unpack(f2_mul(f2_pack(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), f2), a0, a1);
                            o[i] = __float_as_uint(a0);
                            o[i + 1] = __float_as_uint(a1);
                        }
                        tmem_st_32x32b_x32(tOr + c, o);
                    }
                    tmem_wait_st();
                }
                // exponentials, row sums, P (bf16) over the S columns already read
                const float m_sub = (m_run == -INFINITY) ? 0.0f : m_run;
                const uint64_t negm2 = f2_pack(-m_sub, -m_sub);
                uint64_t acc_r = 0ull, acc_e = 0ull;
#pragma unroll
                for (int c = 0; c < kDtcBN; c += 32) {
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
            ok = mbar_wait(bar_o_done, s.n & 1, abort_flag, &g_attn_err, kDevErrTimeout);
            if (!ok) break;
            tc_fence_after_sync();
            if (!idle_warp) {
                const bool whole = s.t0 == 0 && s.t1 == s.tiles;
                const bool row_valid = r < R;
                // a row that saw nothing here, or is no node: 0, and weight 0 in the combine
                const bool seen = live && !(l_exact == 0.0f);
                const float inv_l = seen ? 1.0f / l_run : 0.0f;
                const float lse2 = seen ? m_run + __log2f(l_exact) : -INFINITY;
                const size_t row = (static_cast<size_t>(s.b) * p.Hq + static_cast<size_t>(s.g) * p.G) * p.Lq + mblk * 128 +
                                   (row_valid ? r : 0);
                const size_t prow = tree_part(tp, range, mblk, s.n == 0 ? 0 : 1, row_valid ? r : 0);
                ATTN_CHECK(row < static_cast<size_t>(p.B) * p.Hq * p.Lq);
                ATTN_CHECK(whole || prow < static_cast<size_t>(tp.n_ranges) * tp.n_mblk * 2 * box);
                // (seen by this row's node, and not finite)
                const bool add = seen && v_patched[s.n & 1] == s.n + 1;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(tOr + c, o);
                    tmem_wait_ld();
                    reg_fence<32>(o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = seen ? __float_as_uint(__uint_as_float(o[i]) * inv_l) : 0u;
                    if (row_valid && whole) {
                        __nv_bfloat16* dst = tp.out + row * D + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            float x[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(o[i + k]);
                            *reinterpret_cast<uint4*>(dst + i) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
                        }
                    } else if (row_valid) {
                        float* dst = p.o_part + prow * D + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<uint4*>(dst + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    }
                }
                if (row_valid && whole) {
                    if (tp.lse != nullptr) tp.lse[row] = lse2 * kLn2;
                    if (add) tree_add_nonfinite(tp, s.b, s.g, words, ctx, 0, k_end, D, tp.out + row * D);
                } else if (row_valid) {
                    p.lse_part[prow] = lse2;
                    if (add) tree_add_nonfinite(tp, s.b, s.g, words, ctx, s.t0 * kDtcBN, k_end, D, p.o_part + prow * D);
                }
            }
            // O is read: the arrival on P of the next segment's first tile lets it be written
            tc_fence_before_sync();
            tile0 += n_tiles;
        } while (tree_next(tp, s));
    }

    // ---- teardown ----
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kDtcMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// out = sum_k 2^(lse_k - lse) O_k, lse = log2 sum_k 2^lse_k over the partials of a (sequence,
// KV head) pair that lies in several ranges; rows of sequences without rows get 0 and -inf;
// the rows of other pairs are there already.  WPR warps per row (4: one row per CTA, for
// pairs over many ranges), D / 32 columns per lane, kInFlight partials loaded at a time.
template <int D, int WPR>
__global__ void __launch_bounds__(128) attn_tree_combine_kernel(const TreeParams tp) {
    grid_dep_wait();   // launched as a programmatic dependent of attn_tree_kernel
    constexpr int kPer = D / 32;
    constexpr int kInFlight = 8;
    const DecodeParams& p = tp.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x * (4 / WPR) + warp / WPR;
    const int sub = warp % WPR;
    if (row >= p.B * p.Hq * p.Lq) return;          // (uniform over a CTA when WPR = 4)
    const int RG = p.G * p.Lq;
    const int pair = row / RG, rr = row - pair * RG;
    const int b = pair / p.Hkv, g = pair - b * p.Hkv;
    const int mblk = rr / 128, r = rr % 128;
    const int tiles = tree_tiles(decode_seqlen(p, b));
    const long long per = tp.tiles_before[p.B];
    const long long start = tp.tiles_before[b] * p.Hkv + static_cast<long long>(g) * tiles;
    long long r0 = 0;
    int n = 0;                                     // partials
    if (tiles > 0) {
        r0 = start / per;
        n = static_cast<int>((start + tiles - 1) / per - r0) + 1;
        if (n == 1) return;
    }
    auto part = [&](int k) { return tree_part(tp, r0 + k, mblk, k == 0 && start != r0 * per ? 1 : 0, r); };
    float M = -INFINITY, Lsum = 0.0f, acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
    for (int k0 = sub; k0 < n; k0 += WPR * kInFlight) {
        float ls[kInFlight], ov[kInFlight][kPer];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int k = k0 + u * WPR;
            ls[u] = -INFINITY;
#pragma unroll
            for (int i = 0; i < kPer; ++i) ov[u][i] = 0.0f;
            if (k < n) {
                const size_t at = part(k);
                ls[u] = p.lse_part[at];
                const float* src = p.o_part + at * D + lane * kPer;
#pragma unroll
                for (int i = 0; i < kPer; i += 2) {
                    const float2 v = *reinterpret_cast<const float2*>(src + i);
                    ov[u][i] = v.x;
                    ov[u][i + 1] = v.y;
                }
            }
        }
        float top = M;
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) top = fmaxf(top, ls[u]);
        const float f = M == -INFINITY ? 0.0f : ex2_approx(M - top);
        M = top;
        Lsum *= f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] *= f;
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const float w = ls[u] == -INFINITY ? 0.0f : ex2_approx(ls[u] - M);
            Lsum += w;
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] = w == 0.0f ? acc[i] : fmaf(w, ov[u][i], acc[i]);
        }
    }
    if constexpr (WPR > 1) {
        __shared__ float red_m[WPR], red_l[WPR], red_acc[WPR][D];
#pragma unroll
        for (int i = 0; i < kPer; ++i) red_acc[sub][lane * kPer + i] = acc[i];
        if (lane == 0) {
            red_m[sub] = M;
            red_l[sub] = Lsum;
        }
        __syncthreads();
        if (sub != 0) return;
        float top = M;
#pragma unroll
        for (int w = 1; w < WPR; ++w) top = fmaxf(top, red_m[w]);
        Lsum = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            // (a warp that saw only NaN has M = -inf and a NaN sum)
            const float f = red_m[w] == -INFINITY ? 1.0f : ex2_approx(red_m[w] - top);
            Lsum += red_l[w] * f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] = f == 0.0f ? acc[i] : fmaf(f, red_acc[w][lane * kPer + i], acc[i]);
        }
        M = top;
    }
    // a sum of 0: no row was seen; NaN: a score was
    const float inv = Lsum == 0.0f ? 0.0f : 1.0f / Lsum;
    __nv_bfloat16* o = tp.out + static_cast<size_t>(row) * D + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) *reinterpret_cast<uint32_t*>(o + i) = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
    if (tp.lse != nullptr && lane == 0) tp.lse[row] = Lsum == 0.0f ? -INFINITY : (M + __log2f(Lsum)) * kLn2;
}

}  // namespace attn
