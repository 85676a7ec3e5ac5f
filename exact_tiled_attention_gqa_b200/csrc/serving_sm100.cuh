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
// page_plan / page_release: bound by the launch and a few round trips to memory (64
// requests, one row each: 4.0 us on the device; 512 prompts of up to 4096 rows, 8.5 MB
// of slots: 10.9 us in two launches; release of 512 requests' 33K pages: 7.5 us).
//
// Request b has s_b rows and gets n_b more; with pages of P rows it holds
// u_b = ceil(s_b / P) pages and needs ceil((s_b + n_b) / P) - u_b new ones.
// New page k of the step (requests in order) is free[n_free - 1 - k], the stack's
// top first; a request whose inclusive sum of needs passes n_free is refused.
// ---------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;

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
    int* granted;            // [B] or nullptr; may be new_lens
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

// All CTAs of the launch (one cluster, or a single CTA) have come here.
__device__ __forceinline__ void plan_sync() {
    if (gridDim.x == 1) {
        __syncthreads();
    } else {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}

// Whether any thread of the launch's CTAs says so, for the threads of CTA 0, after all CTAs' writes; the
// others come back at once, for their end.  `flag` of CTA 0 is 0 since before an earlier plan_sync.
__device__ __forceinline__ bool plan_any(bool mine, int* flag) {
    if (gridDim.x == 1) return __syncthreads_or(mine) != 0;
    if (mine) {
        uint32_t first;
        asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(first) : "r"(smem_u32(flag)));
        asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(first) : "memory");
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (blockIdx.x != 0) return false;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    return *static_cast<volatile int*>(flag) != 0;
}

// One warp's share of a copy of runs: entries lo[i] .. hi[i] - 1 of request i for
// i = w, w + step, ... < n; load(i, c) gives a value, store(i, c, value) puts it.
// kPlanInFlight rows of 32 entries are loaded before the first of them is stored:
// one at a time, each request of a warp costs a round trip to memory (512 requests
// of 64 pages: 15.6 us on one CTA one at a time).
constexpr int kPlanInFlight = 8;

template <typename Load, typename Store>
__device__ __forceinline__ void plan_copy_runs(const int* lo, const int* hi, int w, int step, int n, Load load,
                                               Store store) {
    const int lane = threadIdx.x & 31;
    int i = w, c = w < n ? lo[w] : 0;
    while (i < n) {
        int value[kPlanInFlight], at_i[kPlanInFlight], at_c[kPlanInFlight];
#pragma unroll
        for (int u = 0; u < kPlanInFlight; ++u) {
            while (i < n && c >= hi[i]) {
                i += step;
                if (i < n) c = lo[i];
            }
            at_i[u] = -1;
            if (i < n) {
                if (c + lane < hi[i]) {
                    at_i[u] = i;
                    at_c[u] = c + lane;
                    value[u] = load(i, c + lane);
                }
                c += 32;
            }
        }
#pragma unroll
        for (int u = 0; u < kPlanInFlight; ++u)
            if (at_i[u] >= 0) store(at_i[u], at_c[u], value[u]);
    }
}

// The scan, the table's new entries, the lengths and, with SLOTS, the slots; requests in
// chunks of the block.  One CTA, or a cluster of kPlanCluster CTAs that all scan (the
// lengths are few) and share the copies.  Every CTA has read a chunk's lengths, and n_free,
// before any writes that chunk's outputs, so out_seqlens may be seqlens, granted new_lens and
// out_n_free n_free.
template <bool SLOTS>
__global__ void __launch_bounds__(kPlanThreads) attn_page_plan_kernel(const PlanParams p) {
    grid_dep_release();
    __shared__ long long warp_sums[32];
    __shared__ int s_have[kPlanThreads], s_rows[kPlanThreads];      // rows held, rows given
    __shared__ int s_used[kPlanThreads], s_total[kPlanThreads], s_first[kPlanThreads];
    const int n_free = plan_n_free(p);
    const int rank = blockIdx.x, n_cta = gridDim.x;
    long long before = 0;          // pages asked for by earlier chunks
    long long taken = 0;           // pages given
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        const int n = min(kPlanThreads, p.B - b0);
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
        // requests are refused from the first one the pages do not reach for, so the pages given
        // are the served needs' sum
        long long given;
        if (before + asked <= n_free)
            given = asked;
        else
            block_scan(served ? need : 0, warp_sums, given);
        s_have[threadIdx.x] = have;
        s_rows[threadIdx.x] = served ? want : 0;
        s_used[threadIdx.x] = used;
        s_total[threadIdx.x] = served ? total : used;
        s_first[threadIdx.x] = served ? static_cast<int>(first) : 0;
        plan_sync();
        if (rank == 0 && b < p.B) {
            p.out_seqlens[b] = served ? have + want : have;
            p.status[b] = served ? 0 : 1;
            if (p.granted != nullptr) p.granted[b] = served ? want : 0;
        }
        auto popped = [&](int i, int c) { return __ldg(p.free_pages + (n_free - 1 - (s_first[i] + c - s_used[i]))); };
        plan_copy_runs(
            s_used, s_total, rank * (kPlanThreads / 32) + (threadIdx.x >> 5), n_cta * (kPlanThreads / 32), n, popped,
            [&](int i, int c, int page) { p.table[static_cast<size_t>(b0 + i) * p.max_pages + c] = page; });
        if (SLOTS) {
            for (int k = rank * kPlanThreads + threadIdx.x; k < n * p.L; k += n_cta * kPlanThreads) {
                const int i = k / p.L, j = k - i * p.L;
                int slot = -1;
                if (j < s_rows[i]) {
                    const int row = s_have[i] + j, c = row / p.page_size;
                    const int page = c < s_used[i] ? p.table[static_cast<size_t>(b0 + i) * p.max_pages + c] : popped(i, c);
                    if (page < 0 || page >= p.n_pages)
                        atomicOr(&g_attn_err, kDevErrPage);
                    else
                        slot = page * p.page_size + row % p.page_size;
                }
                p.slots[static_cast<size_t>(b0) * p.L + k] = slot;
            }
        }
        before += asked;
        taken += given;
    }
    if (rank == 0 && threadIdx.x == 0) *p.out_n_free = n_free - static_cast<int>(taken);
}

// The slot of every new row, from the table and lengths attn_page_plan_kernel wrote: units of
// kSlotRun rows of one request.  (new_lens may be `granted` by now: the same where a request was
// served.)
constexpr int kSlotThreads = 256;
constexpr int kSlotRun = 4 * kSlotThreads;

__global__ void __launch_bounds__(kSlotThreads) attn_page_slots_kernel(const PlanParams p) {
    grid_dep_wait();
    const int runs = (p.L + kSlotRun - 1) / kSlotRun;
    const long long units = static_cast<long long>(p.B) * runs;
    for (long long unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int b = static_cast<int>(unit / runs), j0 = static_cast<int>(unit % runs) * kSlotRun;
        const int want = p.new_lens[b];
        const int given = p.status[b] == 0 ? want : 0;
        const int row0 = p.out_seqlens[b] - want;
        const int* table = p.table + static_cast<size_t>(b) * p.max_pages;
        int* slots = p.slots + static_cast<size_t>(b) * p.L;
        int page[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + u * kSlotThreads + static_cast<int>(threadIdx.x);
            page[u] = j < given ? table[(row0 + j) / p.page_size] : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + u * kSlotThreads + static_cast<int>(threadIdx.x);
            int slot = -1;
            if (j < given) {
                if (page[u] < 0 || page[u] >= p.n_pages)
                    atomicOr(&g_attn_err, kDevErrPage);
                else
                    slot = page[u] * p.page_size + (row0 + j) % p.page_size;
            }
            if (j < p.L) slots[j] = slot;
        }
    }
}

// Pages a request holds and keeps; none where the lengths cannot be.
__device__ __forceinline__ bool release_pages(const PlanParams& p, int b, int& used, int& kept) {
    const int have = p.seqlens[b], keep = p.new_lens[b];
    used = kept = 0;
    if (have < 0 || keep < 0 || keep > have || have > static_cast<long long>(p.max_pages) * p.page_size) return false;
    used = pages_of(have, p.page_size);
    kept = pages_of(keep, p.page_size);
    return true;
}

// Pages past the rows a request keeps go back on the stack, requests and pages in order.
// One CTA or a cluster, as attn_page_plan_kernel.  A page's place is the count of those before
// it, good or bad; where a bad one turns up (an entry outside the pool, which must not be handed
// out again), one warp writes the stack anew without them.
__global__ void __launch_bounds__(kPlanThreads) attn_page_release_kernel(const PlanParams p) {
    __shared__ long long warp_sums[32];
    __shared__ int s_used[kPlanThreads], s_kept[kPlanThreads], s_first[kPlanThreads], s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    const int n_free = plan_n_free(p);
    const int rank = blockIdx.x, n_cta = gridDim.x;
    long long before = n_free;
    bool bad = false;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int used = 0, kept = 0;
        if (b < p.B && !release_pages(p, b, used, kept)) atomicOr(&g_attn_err, kDevErrSeqlen);
        long long gone;
        const long long first = before + block_scan(used - kept, warp_sums, gone);
        s_used[threadIdx.x] = used;
        s_kept[threadIdx.x] = kept;
        s_first[threadIdx.x] = static_cast<int>(first);
        plan_sync();
        plan_copy_runs(
            s_kept, s_used, rank * (kPlanThreads / 32) + (threadIdx.x >> 5), n_cta * (kPlanThreads / 32),
            min(kPlanThreads, p.B - b0),
            [&](int i, int c) { return __ldg(p.table + static_cast<size_t>(b0 + i) * p.max_pages + c); },
            [&](int i, int c, int page) {
                bad |= page < 0 || page >= p.n_pages;
                const long long at = static_cast<long long>(s_first[i]) + c - s_kept[i];
                if (at < p.capacity) p.free_pages[at] = page;
            });
        before += gone;
    }
    if (rank == 0 && threadIdx.x == 0) *p.out_n_free = static_cast<int>(min(before, static_cast<long long>(p.capacity)));
    bad = plan_any(bad, &s_bad);
    if (rank != 0) return;
    if (bad && threadIdx.x < 32) {
        before = n_free;
        for (int b = 0; b < p.B; ++b) {
            int used, kept;
            release_pages(p, b, used, kept);
            for (int c = kept + static_cast<int>(threadIdx.x); __any_sync(0xffffffffu, c < used); c += 32) {
                const int page = c < used ? __ldg(p.table + static_cast<size_t>(b) * p.max_pages + c) : -1;
                const bool good = page >= 0 && page < p.n_pages;
                const unsigned int goods = __ballot_sync(0xffffffffu, good);
                const long long at = before + __popc(goods & ((1u << threadIdx.x) - 1u));
                if (good && at < p.capacity) p.free_pages[at] = page;
                before += __popc(goods);
            }
        }
        if (threadIdx.x == 0) {
            atomicOr(&g_attn_err, kDevErrPage);
            *p.out_n_free = static_cast<int>(min(before, static_cast<long long>(p.capacity)));
        }
    }
    if (threadIdx.x == 0 && before > p.capacity) atomicOr(&g_attn_err, kDevErrPage);
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
constexpr int kRopeRows = 2;       // rows of a thread in flight
constexpr int kRopeTokens = 8;     // tokens of a CTA, where there are many
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
    int B, L, Hq, Hkv, rot, page_size;
    long long n_slots;                  // n_outer * page_size
    int n_axes, sections[4];
    int cycle;                          // axes taken in turn, not in blocks
    unsigned int row_div;               // 2^32 / (Hq + 2 Hkv), rounded up
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

// A CTA takes TOK tokens: their TOK x rot / 2 angles once, to shared memory, then their
// TOK x (Hq + 2 Hkv) rows, D / 16 threads a row, 16 elements a thread: the two halves of 8
// pairs ("half": elements i and i + rot / 2 pair up) or 16 neighbours ("adjacent": elements
// 2i and 2i + 1).  A thread loads kRopeRows rows before it turns the first.
//
// Bound by the bytes of q, k and v in and q, K and V out, and by the issue of the turn
// itself.  8192 tokens, 5461 of them stored (32 + 8 heads of 128, E4M3 cache, 168 MB, 25.9 us at the
// copy rate): one token a CTA and one row at a time 46.4 us; four tokens and two rows 41.1; the angles
// laid out so that a row's reads of them meet no bank twice 37.1; no division per row 35.9;
// eight tokens 35.5.  Four rows in flight at fewer CTAs 39.1, one row at more 35.9.
template <int D, int FMT, bool ADJ, int TOK>
__global__ void __launch_bounds__(kRopeThreads, 4) attn_rope_append_kernel(const RopeParams p) {
    constexpr int TPR = D / 16;                    // threads per row
    constexpr int RPP = kRopeThreads / TPR;        // rows per pass
    // pair i at [i % 8][i / 8]: a thread's 8 pairs are 8 reads, each of neighbouring words across the row
    __shared__ float2 turn[TOK][8][D / 16];
    __shared__ int s_outer[TOK], s_row[TOK];       // cache slab and row of a token (slab -1: not stored)
    __shared__ size_t s_q[TOK];                    // row of q_out of its head 0
    __shared__ unsigned int amax[FMT == 2 ? RPP * (D / 32) : 1];
    const int N = p.B * p.L;
    const int tok0 = blockIdx.x * TOK;
    const int n_tok = min(TOK, N - tok0);
    const int sub = threadIdx.x % TPR, rloc = threadIdx.x / TPR;
    const int rows = p.Hq + 2 * p.Hkv;
    const int half = p.rot / 2;
    if (threadIdx.x < n_tok) {
        const int tok = tok0 + threadIdx.x;
        int slot = p.slots[tok];
        if (slot >= p.n_slots) {
            atomicOr(&g_attn_err, kDevErrPage);
            slot = -1;
        }
        s_outer[threadIdx.x] = slot < 0 ? -1 : slot / p.page_size;
        s_row[threadIdx.x] = slot < 0 ? 0 : slot % p.page_size;
        s_q[threadIdx.x] = static_cast<size_t>(tok / p.L) * p.Hq * p.L + tok % p.L;
    }
    for (int i = threadIdx.x; i < n_tok * half; i += kRopeThreads) {
        const int t = i / half, pair = i - t * half;
        turn[t][pair % 8][pair / 8] = rope_turn(p.positions[static_cast<size_t>(rope_axis(p, pair)) * N + tok0 + t], p.inv_freq[pair]);
    }
    __syncthreads();
    // element offsets of this thread's two runs of 8, in a turned row and in V's
    const bool turns = sub * 16 < p.rot;
    const int va = sub * 16, vb = va + 8;
    const int ta = !ADJ && turns ? sub * 8 : va, tb = !ADJ && turns ? ta + half : vb;
    const int n_rows = n_tok * rows;
    for (int r0 = rloc; r0 - rloc < n_rows; r0 += kRopeRows * RPP) {
        uint4 ua[kRopeRows], ub[kRopeRows];
        int tk[kRopeRows], rr[kRopeRows];
#pragma unroll
        for (int u = 0; u < kRopeRows; ++u) {
            const int it = r0 + u * RPP;
            tk[u] = -1;
            if (it < n_rows) {
                // it / rows: exact while TOK rows^2 < 2^32, which the launch sees to
                const int t = TOK == 1 ? 0 : static_cast<int>(__umulhi(static_cast<unsigned int>(it), p.row_div)), r = it - t * rows;
                const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hkv;
                if (is_q || s_outer[t] >= 0) {
                    const long long tok = tok0 + t;
                    const __nv_bfloat16* src = is_q ? p.q + tok * p.q_tok + static_cast<size_t>(r) * D
                                               : is_v ? p.v + tok * p.v_tok + static_cast<size_t>(r - p.Hq - p.Hkv) * D
                                                      : p.k + tok * p.k_tok + static_cast<size_t>(r - p.Hq) * D;
                    tk[u] = t;
                    rr[u] = r;
                    ua[u] = __ldg(reinterpret_cast<const uint4*>(src + (is_v ? va : ta)));
                    ub[u] = __ldg(reinterpret_cast<const uint4*>(src + (is_v ? vb : tb)));
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kRopeRows; ++u) {
            const bool on = tk[u] >= 0;
            const int t = on ? tk[u] : 0, r = on ? rr[u] : 0;
            const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hkv;
            const int ea = is_v ? va : ta, eb = is_v ? vb : tb;
            float xa[8], xb[8];
            if (on) {
                unpack8(ua[u], xa);
                unpack8(ub[u], xb);
                if (turns && !is_v) {
                    if (ADJ) {
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            const float2 w = turn[t][i / 2][sub], z = turn[t][4 + i / 2][sub];
                            const float a0 = xa[i], b0 = xb[i];
                            xa[i] = a0 * w.x - xa[i + 1] * w.y;
                            xa[i + 1] = xa[i + 1] * w.x + a0 * w.y;
                            xb[i] = b0 * z.x - xb[i + 1] * z.y;
                            xb[i + 1] = xb[i + 1] * z.x + b0 * z.y;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 w = turn[t][i][sub];
                            const float a0 = xa[i];
                            xa[i] = a0 * w.x - xb[i] * w.y;
                            xb[i] = xb[i] * w.x + a0 * w.y;
                        }
                    }
                }
            }
            if (on && is_q) {
                __nv_bfloat16* dst = p.q_out + (s_q[t] + static_cast<size_t>(r) * p.L) * D;
                *reinterpret_cast<uint4*>(dst + ea) = pack8(xa);
                *reinterpret_cast<uint4*>(dst + eb) = pack8(xb);
            }
            const bool store = on && !is_q;
            const int head = is_v ? r - p.Hq - p.Hkv : r - p.Hq;
            // row of the cache: [outer, Hkv, page_size, D]
            const size_t crow = store ? (static_cast<size_t>(s_outer[t]) * p.Hkv + head) * p.page_size + s_row[t] : 0;
            if constexpr (FMT == kCacheBf16) {
                if (store) {
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? p.v_cache : p.k_cache) + crow * D;
                    *reinterpret_cast<uint4*>(dst + ea) = pack8(xa);
                    *reinterpret_cast<uint4*>(dst + eb) = pack8(xb);
                }
            } else if constexpr (FMT == 1) {
                // E4M3 of x / scale, rounded to the nearest, saturating at 448
                if (store) {
                    uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + crow * D;
                    const float sc = __ldg(static_cast<const float*>(is_v ? p.v_scale : p.k_scale) + head);
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
                    int8_t* dst = static_cast<int8_t*>(is_v ? p.v_cache : p.k_cache) + crow * D;
                    __half* scales = static_cast<__half*>(is_v ? p.v_scale : p.k_scale) + crow * (D / 32);
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

// One CTA per sequence (it alone reads and writes the sequence's length), a 16-byte column of
// a head per thread, kCommitBatch rows in flight: bound by the round trips lengths -> path ->
// pages -> rows (64 sequences, up to 9 rows of 8 heads of 128, paged: 5.9 us; 8 contiguous
// ones, up to 5 rows: 2.8 us).
__global__ void __launch_bounds__(kCommitThreads) attn_tree_commit_kernel(const CommitParams p) {
    const int b = blockIdx.x;
    const int seqlen = p.seqlens[b];
    const int n_b = p.tree_lens != nullptr ? p.tree_lens[b] : p.T;
    const int n = n_b == 0 ? 0 : p.n_accept[b];        // no tree (its rows were refused, say): nothing to accept
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
