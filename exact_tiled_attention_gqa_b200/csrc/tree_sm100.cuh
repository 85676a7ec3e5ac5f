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
// The G x T query rows of a KV head are cut into blocks of 128, the M rows of
// the MMAs; a CTA owns one block and `chunk` cache rows and writes a normalised
// partial output and log2-sum-exp per row, which attn_decode_combine_kernel
// merges.  The mask costs nothing over the committed rows: only a tile that
// reaches past c builds the 64 visibility bits of its rows, each thread (one
// query row) shifting them out of its own mask words.
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
    DecodeParams d;              // d.Lq = T
    const uint32_t* mask;        // [B or 1, T, W]
    size_t mask_batch;           // words from one sequence's mask to the next's (0: one mask for all)
    const int* tree_lens;        // [B], or nullptr (every tree has T nodes)
    const __nv_bfloat16* v;      // the V cache (non-finite elements of tree rows)
    int W;                       // words per mask row, (T + 31) / 32
    int n_mblk;                  // 128-row blocks of a KV head's G x T query rows
};

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
// thread's node sees to its partial output (any positive weight times them is
// themselves).
__device__ __noinline__ void tree_add_nonfinite(const TreeParams& tp, int b, int g, const uint32_t* words, int ctx,
                                                int k_begin, int k_end, int D, float* dst) {
    for (int row = max(ctx, k_begin); row < k_end; ++row) {
        const int j = row - ctx;
        if (!(words[j >> 5] >> (j & 31) & 1u)) continue;
        const __nv_bfloat16* src = tp.v + tree_cache_row(tp.d, b, g, row) * D;
        for (int c = 0; c < D; ++c) {
            const float x = __bfloat162float(src[c]);
            if (!isfinite(x)) dst[c] += x;
        }
    }
}

// All ones over the halves of a bf16 pair that are infinite or NaN.
__device__ __forceinline__ uint32_t nonfinite_bf16x2(uint32_t x) {
    return ((x & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((x & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

template <int D>
__global__ void __launch_bounds__(kDtcThreads, DecodeTcSmem<D>::kCtasPerSm)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const TreeParams tp) {
    grid_dep_release();   // the combine launch may be scheduled now
    using L = DecodeTcSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_base);

    const DecodeParams& p = tp.d;
    const int split = blockIdx.x, g = blockIdx.y / tp.n_mblk, mblk = blockIdx.y % tp.n_mblk, b = blockIdx.z;
    const int seqlen = decode_seqlen(p, b);
    const int k_begin = split * p.chunk;
    if (k_begin >= seqlen) return;   // uniform: this split has no rows
    const int k_end = min(k_begin + p.chunk, seqlen);
    const int n_tiles = (k_end - k_begin + kDtcBN - 1) / kDtcBN;
    const int RG = p.G * p.Lq;                     // query rows of the KV head
    const int R = min(128, RG - mblk * 128);       // of this block
    const int box = min(128, RG);                  // rows TMA loads (past the block's: another head's, or 0)
    const int n_tree = tree_len(tp, b);
    const int ctx = seqlen - n_tree;               // rows every node sees (negative: the tree's first rows are not cached)
    const size_t row0 = (static_cast<size_t>(b) * p.Hq + static_cast<size_t>(g) * p.G) * p.Lq + mblk * 128;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    uint32_t* tmem_base_ptr = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
    volatile int* v_patched = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 8);   // tree rows lost non-finite elements
    // (debug builds) the ring position the producer put in each entry, checked by the MMA warp
    volatile int* ring_tag = reinterpret_cast<volatile int*>(smem + L::kTagOff);

    if (threadIdx.x == 0) {
        mbar_init(bar_q_full, 1);
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar_full(s), 1);
            mbar_init(bar_empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_s_full(i), 1);
            mbar_init(bar_p_full(i), 128);
        }
        mbar_init(bar_o_ready, 1);
        mbar_init(bar_o_done, 1);
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        *v_patched = 0;
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

    // ring entry t holds the tile at ring position t (K_0 K_1 V_0 K_2 V_1 ...)
    const int n_items = 2 * n_tiles;
    auto slot_of = [&](int t) { return t % L::kStages; };
    auto par_of = [&](int t) { return static_cast<uint32_t>(t / L::kStages) & 1u; };

    if (warp == kDtcProducerWarp) {
        // ================= TMA producer =================
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
            mbar_arrive_expect_tx(bar_q_full, static_cast<uint32_t>(L::kKB * box * 128));
            for (int kb = 0; kb < L::kKB; ++kb)
                tma_load_3d(sQ + kb * L::kQBlockBytes, &tm_q, bar_q_full, kb * 64, static_cast<int>(row0), 0);
            int issued = 0;
            for (int t = 0; t < n_items; ++t) {
                const int s = slot_of(t);
                if (!mbar_wait(bar_empty(s), par_of(t) ^ 1u, abort_flag, &g_attn_err, kDevErrTimeout)) break;
                bool is_v;
                int j;
                ring_tile<1>(t, n_tiles, is_v, j);
                const int key0 = k_begin + j * kDtcBN;   // split starts are multiples of 64
                int row = key0, outer = b * p.Hkv + g;
                if (p.block_table != nullptr) {
                    int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + key0 / p.page_size);
                    if (page < 0 || page >= p.n_pages) {
                        atomicOr(&g_attn_err, kDevErrPage);
                        page = 0;
                    }
                    row = key0 % p.page_size;
                    outer = page * p.Hkv + g;
                }
                decode_check_tile(p, row, outer);
                ATTN_CHECK(j >= 0 && j < n_tiles);
                if (ATTN_DEBUG_BOUNDS) ring_tag[s] = t;
                mbar_arrive_expect_tx(bar_full(s), L::kHalfBytes);
                const CUtensorMap* map = is_v ? &tm_v : &tm_k;
                const uint32_t dst = sKV + s * L::kHalfBytes;
                for (int kb = 0; kb < L::kKB; ++kb)
                    tma_load_3d(dst + kb * L::kHalfBlockBytes, map, bar_full(s), kb * 64, row, outer);
                issued = t + 1;
            }
            if (issued < n_items) {
                // unwinding after a timeout: let issued copies land first
                for (int t = max(0, issued - L::kStages); t < issued; ++t) {
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait(bar_full(slot_of(t)), par_of(t)) && global_timer_ns() - t0 < 100000000ull) {
                    }
                }
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(bar_q_full, 0) && global_timer_ns() - t0 < 100000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == kDtcMmaWarp) {
        // ================= MMA issuer (lane 0 issues; the warp clears stale V rows) =================
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
        // S(j) = Q K_j^T into buffer j % 2 (N = 64 cache rows)
        auto qk = [&](int j) {
            const int it = ring_pos_k<1>(j);
            if (!wait_item(it)) return false;
            tc_fence_after_sync();
            if (lane == 0) {
                const uint64_t b0 = dK0 + static_cast<uint64_t>(slot_of(it)) * kSlotStep;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t qoff = static_cast<uint64_t>(((kk >> 2) * L::kQBlockBytes + (kk & 3) * 32) >> 4);
                    const uint64_t koff = static_cast<uint64_t>(((kk >> 2) * L::kHalfBlockBytes + (kk & 3) * 32) >> 4);
                    umma_ss(tS[j & 1], dQ + qoff, b0 + koff, kIdescQK, kk > 0 ? 1u : 0u);
                }
                umma_commit(bar_empty(slot_of(it)));
                umma_commit(bar_s_full(j & 1));
            }
            __syncwarp();
            return true;
        };
        bool ok = mbar_wait(bar_q_full, 0, abort_flag, &g_attn_err, kDevErrTimeout);
        if (ok) ok = qk(0);
        if (ok && n_tiles > 1) ok = qk(1);
        for (int j = 0; j < n_tiles && ok; ++j) {
            const int buf = j & 1;
            const uint32_t ph = static_cast<uint32_t>(j >> 1) & 1u;
            const int itv = ring_pos_v<1>(j, n_tiles);
            ok = wait_item(itv) && mbar_wait(bar_p_full(buf), ph, abort_flag, &g_attn_err, kDevErrTimeout);
            if (!ok) break;
            const int key0 = k_begin + j * kDtcBN;
            const int valid = k_end - key0;
            // non-finite elements of tree rows: zero, and noted for the epilogue
            bool patched = false;
            const int tree_lo = max(0, ctx - key0), tree_hi = min(kDtcBN, valid);
            if (tree_lo < tree_hi) {
                for (int kb = 0; kb < L::kKB; ++kb) {
                    uint8_t* blk = smem + L::kKVOff + slot_of(itv) * L::kHalfBytes + kb * L::kHalfBlockBytes;
#pragma unroll 4
                    for (int i = tree_lo * 128 + lane * 16; i < tree_hi * 128; i += 32 * 16) {
                        uint4 x = *reinterpret_cast<const uint4*>(blk + i);
                        const uint32_t bad = nonfinite_bf16x2(x.x) | nonfinite_bf16x2(x.y) | nonfinite_bf16x2(x.z) | nonfinite_bf16x2(x.w);
                        if (bad) {
                            x.x &= ~nonfinite_bf16x2(x.x);
                            x.y &= ~nonfinite_bf16x2(x.y);
                            x.z &= ~nonfinite_bf16x2(x.z);
                            x.w &= ~nonfinite_bf16x2(x.w);
                            *reinterpret_cast<uint4*>(blk + i) = x;
                            patched = true;
                        }
                    }
                }
                if (patched) *v_patched = 1;
                if (__any_sync(0xffffffffu, patched)) {
                    __threadfence_block();
                    fence_proxy_async_smem();
                }
            }
            // V rows past this split's last row: zero them (P is 0 there, but 0 * NaN is NaN)
            if (valid < kDtcBN) {
                uint8_t* ent = smem + L::kKVOff + slot_of(itv) * L::kHalfBytes;
                for (int kb = 0; kb < L::kKB; ++kb) {
                    uint8_t* blk = ent + kb * L::kHalfBlockBytes + valid * 128;
                    for (int i = lane * 16; i < (kDtcBN - valid) * 128; i += 32 * 16)
                        *reinterpret_cast<uint4*>(blk + i) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
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
        const bool live = r < R && node < n_tree;
        const uint32_t* words = tp.mask + static_cast<size_t>(b) * tp.mask_batch + static_cast<size_t>(node) * tp.W;
        const int free_end = min(ctx, k_end);          // rows below it need no mask
        const float sl2 = p.scale_log2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        // l_run: row sum of P as rounded to bf16 (normalises O); l_exact: of the
        // unrounded exponentials (for the log-sum-exp)
        float m_run = -INFINITY, l_run = 0.0f, l_exact = 0.0f;
        // A warp whose 32 rows are all padding (row >= R) only keeps the pipeline
        // moving: its P rows are never read into a real output row (the MMA keeps
        // rows apart), so it skips the softmax and just signals.
        const bool idle_warp = warp * 32 >= R;
        bool ok = true;
        for (int j = 0; j < n_tiles; ++j) {
            const int buf = j & 1;
            ok = mbar_wait(bar_s_full(buf), static_cast<uint32_t>(j >> 1) & 1u, abort_flag, &g_attn_err,
                           kDevErrTimeout);
            if (!ok) break;
            tc_fence_after_sync();
            if (idle_warp) {
                tc_fence_before_sync();
                mbar_arrive(bar_p_full(buf));
                continue;
            }
            const uint32_t tSr = tS[buf] + lane_off;
            const int key0 = k_begin + j * kDtcBN;
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
                // O must hold tiles 0..j-1: O += P(j-1) V_{j-1} is the only one that can be in flight
                if (!mbar_wait(bar_o_ready, static_cast<uint32_t>(j - 1) & 1u, abort_flag, &g_attn_err,
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
        // ---- this split's partial: O / l (fp32) and m + log2 l per row ----
        bool have_o = ok && n_tiles > 0;
        if (have_o) {
            have_o = mbar_wait(bar_o_done, 0, abort_flag, &g_attn_err, kDevErrTimeout);
            tc_fence_after_sync();
        }
        const bool row_valid = r < R;
        // a row that saw nothing here, or is no node: weight 0 in the combine
        const bool seen = live && !(l_exact == 0.0f);
        const float inv_l = seen ? 1.0f / l_run : 0.0f;
        const size_t prow = (row0 + static_cast<size_t>(row_valid ? r : 0)) * p.n_splits + split;
        decode_check_prow(p, prow);
        float* dst = p.o_part + prow * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            if (have_o) {
                tmem_ld_32x32b_x32(tOr + c, o);
                tmem_wait_ld();
                reg_fence<32>(o);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0u;
            }
            if (row_valid) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<float4*>(dst + c + i) =
                        seen ? make_float4(__uint_as_float(o[i]) * inv_l, __uint_as_float(o[i + 1]) * inv_l,
                                           __uint_as_float(o[i + 2]) * inv_l, __uint_as_float(o[i + 3]) * inv_l)
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
        }
        if (seen && have_o && *v_patched != 0) tree_add_nonfinite(tp, b, g, words, ctx, k_begin, k_end, D, dst);
        if (row_valid) p.lse_part[prow] = seen ? m_run + __log2f(l_exact) : -INFINITY;
    }

    // ---- teardown ----
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kDtcMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

}  // namespace attn
