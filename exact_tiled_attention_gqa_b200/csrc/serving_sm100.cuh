// serving_sm100.cuh -- the calls around a paged cache in a serving step: pages
// and slots from request lengths (page_plan, page_release), rotary positions
// with the write of K and V to their slots (rope_append), and the move of an
// accepted tree path to the end of its sequence (tree_commit).
#pragma once

#include <cuda_fp8.h>

#include "device_error.cuh"
#include "ptx_sm100.cuh"

namespace attn {

// ---------------------------------------------------------------------------
// page_plan / page_release
//
// Request b has s_b rows and gets n_b more; with pages of P rows it holds
// u_b = ceil(s_b / P) pages and needs ceil((s_b + n_b) / P) - u_b new ones.
// New page k of the step (requests in order) is free[n_free - 1 - k], the stack's
// top first; a request whose inclusive sum of needs passes n_free is refused.
// ---------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;

struct PlanParams {
    const int* seqlens;      // [B] rows each request holds
    const int* new_lens;     // [B] rows it gets (plan) or keeps (release)
    int* table;              // [B, max_pages]
    int* free_pages;         // [capacity]
    const int* n_free;       // [1]
    int* slots;              // [B, L]
    int* out_seqlens;        // [B]
    int* out_n_free;         // [1]
    int* status;             // [B]
    int B, L, page_size, max_pages, capacity, n_pages;
};

__device__ __forceinline__ int plan_n_free(const PlanParams& p) {
    int n = *p.n_free;
    if (n < 0 || n > p.capacity) {
        if (threadIdx.x == 0) atomicOr(&g_attn_err, kDevErrPage);
        n = n < 0 ? 0 : p.capacity;
    }
    return n;
}

__device__ __forceinline__ int pages_of(int rows, int page_size) {
    return rows / page_size + (rows % page_size != 0);
}

// Exclusive sum over the block's threads (in order); `total` for all.
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
    long long inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();               // the sums of the scan before are read
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        long long w = lane < n_warps ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warp_sums[lane] = w;       // 32 entries
    }
    __syncthreads();
    total = warp_sums[31];
    return inc - x + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// One CTA: the scan, the table's new entries and the lengths, requests in chunks of
// the block.  Every input of a chunk is read before its outputs are written, so
// out_seqlens may be seqlens and out_n_free n_free.
__global__ void __launch_bounds__(kPlanThreads) attn_page_plan_kernel(const PlanParams p) {
    grid_dep_release();
    __shared__ long long warp_sums[32];
    __shared__ int s_used[kPlanThreads], s_total[kPlanThreads], s_first[kPlanThreads];
    const int n_free = plan_n_free(p);
    long long before = 0;          // pages asked for by earlier chunks
    long long taken = 0;           // pages given
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int used = 0, total = 0, have = 0, want = 0;
        bool fits = false;
        if (b < p.B) {
            have = p.seqlens[b];
            want = p.new_lens[b];
            const long long cap = static_cast<long long>(p.max_pages) * p.page_size;
            // a length that cannot be: nothing is given, the error word says so
            fits = have >= 0 && want >= 0 && want <= p.L && have <= cap;
            if (!fits) atomicOr(&g_attn_err, kDevErrSeqlen);
            fits = fits && static_cast<long long>(have) + want <= cap;
            if (fits) {
                used = pages_of(have, p.page_size);
                total = pages_of(have + want, p.page_size);
            }
        }
        const int need = total - used;
        long long asked;
        const long long first = before + block_scan(need, warp_sums, asked);
        const bool served = fits && (need == 0 || first + need <= n_free);
        long long given;
        block_scan(served ? need : 0, warp_sums, given);
        s_used[threadIdx.x] = used;
        s_total[threadIdx.x] = served ? total : used;
        s_first[threadIdx.x] = served ? static_cast<int>(first) : 0;
        if (b < p.B) {
            p.out_seqlens[b] = served ? have + want : have;
            p.status[b] = served ? 0 : 1;
        }
        __syncthreads();
        for (int i = warp; i < min(kPlanThreads, p.B - b0); i += kPlanThreads / 32) {
            int* row = p.table + static_cast<size_t>(b0 + i) * p.max_pages;
            for (int c = s_used[i] + lane; c < s_total[i]; c += 32)
                row[c] = p.free_pages[n_free - 1 - (s_first[i] + c - s_used[i])];
        }
        before += asked;
        taken += given;
    }
    if (threadIdx.x == 0) *p.out_n_free = n_free - static_cast<int>(taken);
}

// The slot of every new row, from the table and lengths attn_page_plan_kernel wrote.
__global__ void __launch_bounds__(256) attn_page_slots_kernel(const PlanParams p) {
    grid_dep_wait();
    const size_t n = static_cast<size_t>(p.B) * p.L;
    for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < n;
         i += static_cast<size_t>(gridDim.x) * blockDim.x) {
        const int b = static_cast<int>(i / p.L), j = static_cast<int>(i % p.L);
        int slot = -1;
        const int want = p.new_lens[b];
        if (p.status[b] == 0 && j < want) {
            const int row = p.out_seqlens[b] - want + j;
            const int page = p.table[static_cast<size_t>(b) * p.max_pages + row / p.page_size];
            if (page < 0 || page >= p.n_pages)
                atomicOr(&g_attn_err, kDevErrPage);
            else
                slot = page * p.page_size + row % p.page_size;
        }
        p.slots[i] = slot;
    }
}

// Pages past the rows a request keeps go back on the stack, requests and pages in order.
__global__ void __launch_bounds__(kPlanThreads) attn_page_release_kernel(const PlanParams p) {
    __shared__ long long warp_sums[32];
    __shared__ int s_used[kPlanThreads], s_kept[kPlanThreads], s_first[kPlanThreads];
    const int n_free = plan_n_free(p);
    long long before = n_free;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int used = 0, kept = 0;
        if (b < p.B) {
            const int have = p.seqlens[b], keep = p.new_lens[b];
            if (have < 0 || keep < 0 || keep > have || have > static_cast<long long>(p.max_pages) * p.page_size) {
                atomicOr(&g_attn_err, kDevErrSeqlen);
            } else {
                used = pages_of(have, p.page_size);
                kept = pages_of(keep, p.page_size);
            }
        }
        long long gone;
        const long long first = before + block_scan(used - kept, warp_sums, gone);
        s_used[threadIdx.x] = used;
        s_kept[threadIdx.x] = kept;
        s_first[threadIdx.x] = static_cast<int>(first);
        __syncthreads();
        for (int i = warp; i < min(kPlanThreads, p.B - b0); i += kPlanThreads / 32) {
            const int* row = p.table + static_cast<size_t>(b0 + i) * p.max_pages;
            for (int c = s_kept[i] + lane; c < s_used[i]; c += 32) {
                if (row[c] < 0 || row[c] >= p.n_pages) atomicOr(&g_attn_err, kDevErrPage);
                const long long at = static_cast<long long>(s_first[i]) + c - s_kept[i];
                if (at < p.capacity) p.free_pages[at] = row[c];
            }
        }
        before += gone;
    }
    if (threadIdx.x == 0) {
        if (before > p.capacity) atomicOr(&g_attn_err, kDevErrPage);
        *p.out_n_free = static_cast<int>(min(before, static_cast<long long>(p.capacity)));
    }
}

// ---------------------------------------------------------------------------
// rope_append
//
// Pair i of a head is turned by the angle position[axis(i)] * inv_freq[i]:
//   a' = a cos - b sin,  b' = b cos + a sin
// The angle is held as a fraction of a turn in 64-bit fixed point: f = inv_freq /
// 2 pi in double, its fractional part times 2^64, times the integer position
// modulo 2^64.  f's double has a relative error of 2^-52, so the product is the
// exact angle's to |position| * f * 2^-52 + 2^-33 turns: 3e-10 turns at a
// position of a million and f = 1 / 2 pi, where position * inv_freq in fp32
// would be off by position * inv_freq * 2^-24 radians (0.06).
// ---------------------------------------------------------------------------

constexpr int kRopeThreads = 256;
constexpr int kCacheBf16 = 0;      // else ATTN_KV_E4M3 = 1, ATTN_KV_Q8_0 = 2

struct RopeParams {
    const __nv_bfloat16 *q, *k, *v;
    long long q_tok, k_tok, v_tok;      // elements from one token to the next
    const int* positions;               // [n_axes, N]
    const float* inv_freq;              // [rot / 2]
    const int* slots;                   // [N]
    __nv_bfloat16* q_out;               // [B, Hq, L, D]
    void *k_cache, *v_cache;            // [n_outer, Hkv, page_size, D]
    void *k_scale, *v_scale;            // E4M3: fp32 [Hkv]; q8_0: fp16 [n_outer, Hkv, page_size, D / 32]
    int B, L, Hq, Hkv, D, rot, page_size;
    long long n_slots;                  // n_outer * page_size
    int n_axes, sections[4];
    int cycle;                          // axes taken in turn, not in blocks
};

__device__ __forceinline__ int rope_axis(const RopeParams& p, int pair) {
    if (p.cycle) {
        const int a = pair % p.n_axes;
        return (a > 0 && pair / p.n_axes < p.sections[a]) ? a : 0;
    }
    int a = 0, end = p.sections[0];
    while (a + 1 < p.n_axes && pair >= end) end += p.sections[++a];
    return a;
}

// {cos, sin} of position * inv_freq
__device__ __forceinline__ float2 rope_turn(int position, float inv_freq) {
    if (!isfinite(inv_freq)) return make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));   // NaN
    const double turns = static_cast<double>(inv_freq) * 0.15915494309189533577;   // / 2 pi
    const double frac = turns - floor(turns);
    const unsigned long long step = static_cast<unsigned long long>(frac * 18446744073709551616.0);
    const unsigned long long at = step * static_cast<unsigned long long>(static_cast<long long>(position));
    const int top = static_cast<int>((at + 0x80000000ull) >> 32);
    float s, c;
    sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &c);   // 2^-31 half turns
    return make_float2(c, s);
}

__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
    f2_unpack(bf16x2_to_f2(u.x), x[0], x[1]);
    f2_unpack(bf16x2_to_f2(u.y), x[2], x[3]);
    f2_unpack(bf16x2_to_f2(u.z), x[4], x[5]);
    f2_unpack(bf16x2_to_f2(u.w), x[6], x[7]);
}

__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// One CTA per token: its rot / 2 angles once, then its Hq + 2 Hkv rows, D / 16 threads a
// row, 16 elements a thread: the two halves of 8 pairs ("half": elements i and i + rot / 2
// pair up) or 16 neighbours ("adjacent": elements 2i and 2i + 1).
template <int D, int FMT, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads) attn_rope_append_kernel(const RopeParams p) {
    constexpr int TPR = D / 16;                    // threads per row
    constexpr int RPP = kRopeThreads / TPR;        // rows per pass
    __shared__ float2 turn[D / 2];
    __shared__ unsigned int amax[FMT == 2 ? RPP * (D / 32) : 1];
    const int N = p.B * p.L;
    const int tok = blockIdx.x;
    const int b = tok / p.L, l = tok % p.L;
    for (int i = threadIdx.x; i < p.rot / 2; i += kRopeThreads)
        turn[i] = rope_turn(p.positions[static_cast<size_t>(rope_axis(p, i)) * N + tok], p.inv_freq[i]);
    long long slot = p.slots[tok];
    if (slot >= p.n_slots) {
        if (threadIdx.x == 0) atomicOr(&g_attn_err, kDevErrPage);
        slot = -1;
    }
    __syncthreads();
    const int sub = threadIdx.x % TPR, rloc = threadIdx.x / TPR;
    const int rows = p.Hq + 2 * p.Hkv;
    for (int r0 = 0; r0 < rows; r0 += RPP) {
        const int r = r0 + rloc;
        const bool is_q = r < p.Hq, is_k = !is_q && r < p.Hq + p.Hkv;
        const bool on = r < rows && (is_q || slot >= 0);
        const int head = is_q ? r : (is_k ? r - p.Hq : r - p.Hq - p.Hkv);
        // element offsets of this thread's two runs of 8
        const bool turned = (is_q || is_k) && sub * 16 < p.rot;
        int ea = sub * 16, eb = ea + 8;
        if (!ADJ && turned) {
            ea = sub * 8;
            eb = ea + p.rot / 2;
        }
        float xa[8], xb[8];
        if (on) {
            const __nv_bfloat16* src = is_q ? p.q + tok * p.q_tok : (is_k ? p.k + tok * p.k_tok : p.v + tok * p.v_tok);
            src += static_cast<size_t>(head) * D;
            unpack8(*reinterpret_cast<const uint4*>(src + ea), xa);
            unpack8(*reinterpret_cast<const uint4*>(src + eb), xb);
            if (turned) {
                if (ADJ) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 ta = turn[sub * 8 + i / 2], tb = turn[sub * 8 + 4 + i / 2];
                        const float a0 = xa[i], b0 = xb[i];
                        xa[i] = a0 * ta.x - xa[i + 1] * ta.y;
                        xa[i + 1] = xa[i + 1] * ta.x + a0 * ta.y;
                        xb[i] = b0 * tb.x - xb[i + 1] * tb.y;
                        xb[i + 1] = xb[i + 1] * tb.x + b0 * tb.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 t = turn[sub * 8 + i];
                        const float a0 = xa[i];
                        xa[i] = a0 * t.x - xb[i] * t.y;
                        xb[i] = xb[i] * t.x + a0 * t.y;
                    }
                }
            }
        }
        if (on && is_q) {
            __nv_bfloat16* dst = p.q_out + ((static_cast<size_t>(b) * p.Hq + head) * p.L + l) * D;
            *reinterpret_cast<uint4*>(dst + ea) = pack8(xa);
            *reinterpret_cast<uint4*>(dst + eb) = pack8(xb);
        }
        const bool store = on && !is_q;
        // row of the cache: [outer, Hkv, page_size, D]
        size_t crow = 0;
        if (store)
            crow = (static_cast<size_t>(slot / p.page_size) * p.Hkv + head) * p.page_size + slot % p.page_size;
        if constexpr (FMT == kCacheBf16) {
            if (store) {
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_k ? p.k_cache : p.v_cache) + crow * D;
                *reinterpret_cast<uint4*>(dst + ea) = pack8(xa);
                *reinterpret_cast<uint4*>(dst + eb) = pack8(xb);
            }
        } else if constexpr (FMT == 1) {
            // E4M3 of x / scale, rounded to the nearest, saturating at 448
            if (store) {
                uint8_t* dst = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) + crow * D;
                const float sc = static_cast<const float*>(is_k ? p.k_scale : p.v_scale)[head];
                auto codes = [&](const float* x) {
                    uint32_t w[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * h] / sc, x[4 * h + 1] / sc), __NV_SATFINITE, __NV_E4M3);
                        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * h + 2] / sc, x[4 * h + 3] / sc), __NV_SATFINITE, __NV_E4M3);
                        w[h] = lo | (hi << 16);
                    }
                    return make_uint2(w[0], w[1]);
                };
                *reinterpret_cast<uint2*>(dst + ea) = codes(xa);
                *reinterpret_cast<uint2*>(dst + eb) = codes(xb);
            }
        } else {
            // q8_0: per 32 elements the scale fp16(max |x| / 127), codes rint(x / scale).  The
            // 8-element runs of a block meet in shared memory: |x| as bits orders like |x|, NaN above all.
            unsigned int* am = amax + rloc * (D / 32);
            if (sub < D / 32) am[sub] = 0u;
            __syncwarp();
            if (store) {
                unsigned int ma = 0u, mb = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ma = max(ma, __float_as_uint(fabsf(xa[i])));
                    mb = max(mb, __float_as_uint(fabsf(xb[i])));
                }
                atomicMax(am + ea / 32, ma);
                atomicMax(am + eb / 32, mb);
            }
            __syncwarp();
            if (store) {
                int8_t* dst = static_cast<int8_t*>(is_k ? p.k_cache : p.v_cache) + crow * D;
                __half* scales = static_cast<__half*>(is_k ? p.k_scale : p.v_scale) + crow * (D / 32);
                auto scale_of = [&](int e) {
                    const float m = __uint_as_float(am[e / 32]) / 127.0f;
                    return __float2half_rn(m > 65504.0f ? 65504.0f : m);      // NaN stays
                };
                auto codes = [&](const float* x, float sc) {
                    uint32_t w[2] = {0u, 0u};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float c = sc > 0.0f ? fminf(fmaxf(rintf(x[i] / sc), -127.0f), 127.0f) : 0.0f;
                        w[i >> 2] |= (static_cast<uint32_t>(static_cast<int>(c)) & 0xffu) << (8 * (i & 3));
                    }
                    return make_uint2(w[0], w[1]);
                };
                const __half sa = scale_of(ea), sb = scale_of(eb);
                *reinterpret_cast<uint2*>(dst + ea) = codes(xa, __half2float(sa));
                *reinterpret_cast<uint2*>(dst + eb) = codes(xb, __half2float(sb));
                if (ea % 32 == 0) scales[ea / 32] = sa;
                if (eb % 32 == 0) scales[eb / 32] = sb;
            }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------------------
// tree_commit
//
// With c = seqlens[b] - n_b, cache row c + j becomes row c + accept[b][j] for j <
// n_accept[b].  accept increases, so accept[j] >= j and rows move down: a thread
// that owns a 16-byte column of a head reads ahead of what it writes.
// ---------------------------------------------------------------------------

constexpr int kCommitThreads = 256;
constexpr int kCommitBatch = 8;    // rows a thread holds between reading and writing

struct CommitParams {
    uint4 *k_cache, *v_cache;      // [n_outer, Hkv, page_size, D] bf16
    const int* table;              // [B, max_pages], or nullptr (outer = b)
    const int* seqlens;            // [B]
    const int* tree_lens;          // [B] or nullptr
    const int* accept;             // [B, A]
    const int* n_accept;           // [B]
    int* out_seqlens;              // [B]
    int B, Hkv, T, A, D, page_size, max_pages, n_pages;
};

// One CTA per sequence (it alone reads and writes the sequence's length).
__global__ void __launch_bounds__(kCommitThreads) attn_tree_commit_kernel(const CommitParams p) {
    const int b = blockIdx.x;
    const int seqlen = p.seqlens[b];
    const int n_b = p.tree_lens != nullptr ? p.tree_lens[b] : p.T;
    const int n = p.n_accept[b];
    const int* path = p.accept + static_cast<size_t>(b) * p.A;
    const long long cap = p.table != nullptr ? static_cast<long long>(p.max_pages) * p.page_size : p.page_size;
    unsigned int err = 0u;
    if (seqlen < 0 || seqlen > cap || n_b < 0 || n_b > p.T || n_b > seqlen) err = kDevErrSeqlen;
    if (n < 0 || n > p.A || n > n_b) err |= kDevErrIndex;
    if (err == 0u)
        for (int j = threadIdx.x; j < n; j += kCommitThreads)
            if (path[j] < 0 || path[j] >= n_b || (j > 0 && path[j] <= path[j - 1])) err = kDevErrIndex;
    if (__syncthreads_or(static_cast<int>(err))) {     // a path that cannot be: nothing moves
        if (err) atomicOr(&g_attn_err, err);
        if (threadIdx.x == 0) p.out_seqlens[b] = seqlen;
        return;
    }
    const int ctx = seqlen - n_b;
    if (threadIdx.x == 0) p.out_seqlens[b] = ctx + n;
    const int cpr = p.D / 8;                           // 16-byte columns per row
    // the 16-byte element of (row, head, column), or -1 where the page is bad
    auto at = [&](int row, int head, int col) -> long long {
        long long outer = b;
        if (p.table != nullptr) {
            outer = p.table[static_cast<size_t>(b) * p.max_pages + row / p.page_size];
            if (outer < 0 || outer >= p.n_pages) {
                atomicOr(&g_attn_err, kDevErrPage);
                return -1;
            }
            row %= p.page_size;
        }
        return ((outer * p.Hkv + head) * p.page_size + row) * cpr + col;
    };
    const int units = 2 * p.Hkv * cpr;
    for (int u = threadIdx.x; u < units; u += kCommitThreads) {
        const int col = u % cpr, head = u / cpr % p.Hkv;
        uint4* cache = u < p.Hkv * cpr ? p.k_cache : p.v_cache;
        for (int j0 = 0; j0 < n; j0 += kCommitBatch) {
            uint4 hold[kCommitBatch];
            long long to[kCommitBatch];
#pragma unroll
            for (int i = 0; i < kCommitBatch; ++i) {
                to[i] = -1;
                const int j = j0 + i;
                if (j < n && path[j] != j) {
                    const long long from = at(ctx + path[j], head, col);
                    if (from >= 0) {
                        to[i] = at(ctx + j, head, col);
                        hold[i] = cache[from];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kCommitBatch; ++i)
                if (to[i] >= 0) cache[to[i]] = hold[i];
        }
    }
}

}  // namespace attn
