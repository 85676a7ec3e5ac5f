// serving_api.cuh -- the C ABI of the serving-step calls (tree attention, page
// plan and release, rotary append, tree commit): argument checks and launches.
// Included by attn_gqa.cu, whose helpers it uses.
#pragma once

namespace attn {
namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// ---- tree attention ----

struct TreeLayout {
    int n_mblk = 0, n_ranges = 0;
    size_t lse_off = 0, tiles_off = 0, total = 0;
};

// Sizes the calls accept (the workspace size of others is 0).
bool tree_sizes_ok(int B, int Hq, int Hkv, int T, int Lmax, int D) {
    return B >= 0 && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && T >= 1 && T <= kTreeMaxNodes && Lmax >= 1 &&
           Lmax <= 0x7ff00000 && (D == 64 || D == 128 || D == 256) &&
           static_cast<long long>(B) * Hq * T <= 0x7fffffffLL;
}

// Depends on the arguments only: 148 SMs, one CTA (D = 256) or two on each.
TreeLayout tree_layout(int B, int Hq, int Hkv, int T, int Lmax, int D) {
    TreeLayout t;
    const long long rg = static_cast<long long>(Hq / Hkv) * T;
    t.n_mblk = static_cast<int>((rg + 127) / 128);
    const long long tiles = static_cast<long long>(B) * Hkv * ((Lmax + 63LL) / 64);
    const long long ctas = 148LL * (D == 256 ? TreeCfg<256>::kCtasPerSm : TreeCfg<128>::kCtasPerSm);
    t.n_ranges = static_cast<int>(std::max(1LL, std::min(ctas / t.n_mblk, tiles)));
    const size_t rows = static_cast<size_t>(t.n_ranges) * t.n_mblk * 2 * static_cast<size_t>(std::min(128LL, rg));
    t.lse_off = align256(rows * D * sizeof(float));
    t.tiles_off = t.lse_off + align256(rows * sizeof(float));
    t.total = t.tiles_off + align256((static_cast<size_t>(B) + 1) * sizeof(long long));
    return t;
}

template <int D>
int launch_tree(const void* q, const void* kc, const void* vc, const TreeParams& tp, const TreeLayout& lay,
                cudaStream_t stream) {
    static int smem_done[64];
    using L = TreeCfg<D>;
    const DecodeParams& prm = tp.d;
    const uint64_t rows = prm.block_table ? static_cast<uint64_t>(prm.page_size) : static_cast<uint64_t>(prm.Lmax);
    const uint64_t outer = static_cast<uint64_t>(prm.block_table ? prm.n_pages : prm.B) * prm.Hkv;
    const int box = std::min(128, prm.G * prm.Lq);
    CUtensorMap tq, tk, tv;
    int st;
    if ((st = encode_bf16_3d(&tq, q, D, static_cast<uint64_t>(prm.B) * prm.Hq * prm.Lq, 1, 64, box, 1, "q")) != ATTN_OK)
        return st;
    if ((st = encode_bf16_3d(&tk, kc, D, rows, outer, 64, kDecKT, 1, "k_cache")) != ATTN_OK) return st;
    if ((st = encode_bf16_3d(&tv, vc, D, rows, outer, 64, kDecKT, 1, "v_cache")) != ATTN_OK) return st;
    if ((st = ensure_smem(attn_tree_kernel<D>, L::kAlloc, smem_done)) != ATTN_OK) return st;
    attn_tree_kernel<D><<<static_cast<unsigned>(lay.n_ranges) * lay.n_mblk, L::kThreads, L::kAlloc, stream>>>(tq, tk, tv, tp);
    if ((st = check_launch("attn_tree_kernel")) != ATTN_OK) return st;
    const long long pairs = static_cast<long long>(prm.B) * prm.Hkv, rows_per_pair = static_cast<long long>(prm.G) * prm.Lq;
    const long long slices = (rows_per_pair + kTreeCombineRows - 1) / kTreeCombineRows;
    // n_ranges / pairs, at most the partials of a pair on average, decides how the combine spreads them.  Over the warps
    // against all by one: 8 requests of 9000 rows, 63 nodes, D 64 (32 pairs) 66 us and 61; 6 of 6000 rows, 21 nodes, 8 heads
    // a KV head, D 128 (12 pairs) 7.7 us of combine, by four columns a lane 13.4; 4 rows on 12000 12.8 us a call by four
    // columns a lane, by rows 15.3.
    const unsigned few_rows = static_cast<unsigned>(pairs * ((rows_per_pair * (D / 4) + 31) / 32));
    const unsigned one = static_cast<unsigned>(pairs * slices * (D / 64)), four = static_cast<unsigned>(pairs * slices * (D / 16));
    const cudaError_t e =
        rows_per_pair < kTreeCombineRows && lay.n_ranges > pairs
            ? launch_dependent(attn_tree_combine_few_rows_kernel<D>, few_rows, 128u, stream, tp)
        : lay.n_ranges > 4 * pairs ? launch_dependent(attn_tree_combine_kernel<D, 4>, four, 128u, stream, tp)
                                   : launch_dependent(attn_tree_combine_kernel<D, 1>, one, 128u, stream, tp);
    if (e != cudaSuccess) return fail(ATTN_ERR_CUDA, "attn_tree_combine_kernel launch failed: %s", cudaGetErrorString(e));
    return check_launch("attn_tree_combine_kernel");
}

int tree_checked(const void* q, const void* kc, const void* vc, const int32_t* block_table, const int32_t* seqlens,
                 const uint32_t* tree_mask, int mask_per_seq, const int32_t* tree_lens, void* out, float* lse, int B,
                 int Hq, int Hkv, int T, int n_pages, int page_size, int max_pages, int Lmax, int D, float scale,
                 void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_common(q, kc, vc, out, lse, B, Hq, Hkv, T, Lmax, D, scale, "T", "Lmax");
    if (st != ATTN_OK) return st;
    if (T < 1 || Lmax < 1) return fail(ATTN_ERR_INVALID_ARG, "T and Lmax must be >= 1 (T=%d Lmax=%d)", T, Lmax);
    if (B > 0 && (!seqlens || !tree_mask)) return fail(ATTN_ERR_INVALID_ARG, "null seqlens or tree_mask");
    if (!aligned4(seqlens) || !aligned4(tree_mask) || !aligned4(tree_lens) || !aligned4(block_table))
        return fail(ATTN_ERR_INVALID_ARG, "seqlens, tree_mask, tree_lens and block_table must be 4-byte aligned");
    if (T > kTreeMaxNodes) return fail(ATTN_ERR_UNSUPPORTED, "T=%d nodes (built: up to %d)", T, kTreeMaxNodes);
    if (!tree_sizes_ok(B, Hq, Hkv, T, Lmax, D)) return fail(ATTN_ERR_UNSUPPORTED, "B*Hq*T or Lmax too large");
    if (B == 0) return ok();
    const TreeLayout lay = tree_layout(B, Hq, Hkv, T, Lmax, D);
    if (!workspace || workspace_bytes < lay.total)
        return fail(ATTN_ERR_WORKSPACE, "tree attention workspace needs %zu bytes, got %zu", lay.total,
                    workspace ? workspace_bytes : static_cast<size_t>(0));
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(ATTN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    TreeParams tp;
    DecodeParams& prm = tp.d;
    prm.q = static_cast<const __nv_bfloat16*>(q);
    prm.seqlens = seqlens;
    prm.o_part = static_cast<float*>(workspace);
    prm.lse_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + lay.lse_off);
    prm.B = B;
    prm.Hq = Hq;
    prm.Hkv = Hkv;
    prm.Lmax = Lmax;
    prm.G = Hq / Hkv;
    prm.Lq = T;
    prm.block_table = block_table;
    prm.page_size = page_size;
    prm.max_pages = max_pages;
    prm.n_pages = n_pages;
    prm.chunk = prm.n_splits = 0;
    prm.scale_log2 = scale * kLog2e;
    tp.out = static_cast<__nv_bfloat16*>(out);
    tp.lse = lse;
    tp.tiles_before = reinterpret_cast<long long*>(static_cast<uint8_t*>(workspace) + lay.tiles_off);
    tp.n_ranges = lay.n_ranges;
    tp.mask = tree_mask;
    tp.W = (T + 31) / 32;
    tp.mask_batch = mask_per_seq ? static_cast<size_t>(T) * tp.W : 0;
    tp.tree_lens = tree_lens;
    tp.v = static_cast<const __nv_bfloat16*>(vc);
    tp.n_mblk = lay.n_mblk;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = (D == 256)   ? launch_tree<256>(q, kc, vc, tp, lay, s)
         : (D == 128) ? launch_tree<128>(q, kc, vc, tp, lay, s)
                      : launch_tree<64>(q, kc, vc, tp, lay, s);
    return st == ATTN_OK ? ok() : st;
}

// Sizes of a pool of pages, shared by the calls that read or write one.
int check_pool(int n_pages, int page_size, int max_pages) {
    if (page_size < 64 || page_size % 64 != 0)
        return fail(ATTN_ERR_INVALID_ARG, "page_size=%d must be a positive multiple of 64", page_size);
    if (n_pages < 1 || max_pages < 1) return fail(ATTN_ERR_INVALID_ARG, "n_pages and max_pages must be >= 1");
    if (static_cast<long long>(page_size) * max_pages > 0x7fffffffLL) return fail(ATTN_ERR_UNSUPPORTED, "page pool too large");
    return ATTN_OK;
}

}  // namespace
}  // namespace attn

extern "C" size_t attn_decode_tree_workspace_size(int B, int Hq, int Hkv, int T, int Lmax, int D) {
    if (B < 1 || !tree_sizes_ok(B, Hq, Hkv, T, Lmax, D)) return 0;
    return tree_layout(B, Hq, Hkv, T, Lmax, D).total;
}

extern "C" int attn_decode_tree(const void* q, const void* k_cache, const void* v_cache, const int32_t* seqlens,
                                const uint32_t* tree_mask, int mask_per_seq, const int32_t* tree_lens, void* out,
                                float* lse, int B, int Hq, int Hkv, int T, int Lmax, int D, float scale,
                                void* workspace, size_t workspace_bytes, void* stream) {
    if (static_cast<long long>(B) * Hkv > 0x7fffffffLL) return fail(ATTN_ERR_UNSUPPORTED, "B*Hkv too large");
    return tree_checked(q, k_cache, v_cache, nullptr, seqlens, tree_mask, mask_per_seq, tree_lens, out, lse, B, Hq, Hkv,
                        T, 0, 0, 0, Lmax, D, scale, workspace, workspace_bytes, stream);
}

extern "C" size_t attn_decode_tree_paged_workspace_size(int B, int Hq, int Hkv, int T, int page_size, int max_pages,
                                                         int D) {
    if (page_size < 64 || page_size % 64 != 0 || max_pages < 1 ||
        static_cast<long long>(page_size) * max_pages > 0x7fffffffLL)
        return 0;
    return attn_decode_tree_workspace_size(B, Hq, Hkv, T, page_size * max_pages, D);
}

extern "C" int attn_decode_tree_paged(const void* q, const void* k_pages, const void* v_pages,
                                      const int32_t* block_table, const int32_t* seqlens, const uint32_t* tree_mask,
                                      int mask_per_seq, const int32_t* tree_lens, void* out, float* lse, int B, int Hq,
                                      int Hkv, int T, int n_pages, int page_size, int max_pages, int D, float scale,
                                      void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_pool(n_pages, page_size, max_pages);
    if (st != ATTN_OK) return st;
    if (static_cast<long long>(n_pages) * Hkv > 0x7fffffffLL) return fail(ATTN_ERR_UNSUPPORTED, "page pool too large");
    if (B > 0 && !block_table) return fail(ATTN_ERR_INVALID_ARG, "null block_table");
    return tree_checked(q, k_pages, v_pages, block_table, seqlens, tree_mask, mask_per_seq, tree_lens, out, lse, B, Hq,
                        Hkv, T, n_pages, page_size, max_pages, page_size * max_pages, D, scale, workspace,
                        workspace_bytes, stream);
}

// ---- page plan and release ----

namespace attn {
namespace {
// Sizes and pointers both calls share.
int check_plan(const PlanParams& p) {
    if (p.B < 0 || p.L < 0 || p.page_size < 1 || p.max_pages < 1 || p.n_pages < 1 || p.capacity < 0)
        return fail(ATTN_ERR_INVALID_ARG, "bad size (B=%d L=%d page_size=%d max_pages=%d n_pages=%d capacity=%d)", p.B, p.L,
                    p.page_size, p.max_pages, p.n_pages, p.capacity);
    if (!p.n_free || !p.out_n_free || (!p.free_pages && p.capacity > 0))
        return fail(ATTN_ERR_INVALID_ARG, "null free_pages, n_free or out_n_free");
    if (p.B > 0 && (!p.seqlens || !p.new_lens || !p.table)) return fail(ATTN_ERR_INVALID_ARG, "null lengths or block_table");
    if (!aligned4(p.seqlens) || !aligned4(p.new_lens) || !aligned4(p.table) || !aligned4(p.free_pages) ||
        !aligned4(p.n_free) || !aligned4(p.slots) || !aligned4(p.out_seqlens) || !aligned4(p.out_n_free) || !aligned4(p.status) ||
        !aligned4(p.granted))
        return fail(ATTN_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    if (static_cast<long long>(p.n_pages) * p.page_size > 0x7fffffffLL)
        return fail(ATTN_ERR_UNSUPPORTED, "n_pages * page_size too large for 32-bit slots");
    if (static_cast<long long>(p.max_pages) * p.page_size > 0x7fffffffLL ||
        static_cast<long long>(p.B) * p.max_pages > 0x3fffffffLL || p.capacity > 0x3fffffff || p.L > 0x3fffffff)
        return fail(ATTN_ERR_UNSUPPORTED, "block table, page stack or L too large");
    return ATTN_OK;
}
// attn_page_plan_kernel writes up to this many slots itself, a second kernel on the whole GPU more.  Device time
// of the call, both ways, on the cluster: 8192 slots of 512 requests 5.1 and 6.0 us, 8192 of 64 5.3 and 5.5,
// 16384 of 64 5.8 and 5.6, 32768 of 512 7.2 and 6.0.
constexpr long long kPlanSlots = 8192;
// One CTA does a step of up to so many requests and slots (64 requests of a row 4.1 us, on the cluster 4.5; of 16
// rows 4.5 and 4.9), the cluster of eight larger ones (512 of a row 5.0 us, on one CTA 5.3; 64 of 64 rows 5.0 and 6.7).
constexpr int kPlanOneB = 128;
constexpr long long kPlanOneSlots = 1024;
// page_release does not know how many pages go, only how many could: one CTA where the table is small, else the cluster
// (512 requests of up to 256 pages 15.6 us on one CTA and 7.5).  A wide table of which little goes pays for the cluster:
// 64 requests of up to 64 pages 4.1 us in a table of 64 columns, 4.3 in one of 512; of up to 16 pages 3.8 and 4.4.
constexpr long long kReleaseEntries = 4096;

int launch_plan(void (*kernel)(const PlanParams), bool one, cudaStream_t s, const PlanParams& p, const char* what) {
    cudaLaunchAttribute attr[1];
    const unsigned n = one ? 1 : kPlanCluster;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess) return fail(ATTN_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
    return check_launch(what);
}

}  // namespace
}  // namespace attn

extern "C" int attn_page_plan(const int32_t* seqlens, const int32_t* new_lens, int32_t* block_table,
                              const int32_t* free_pages, const int32_t* n_free, int32_t* slots, int32_t* out_seqlens,
                              int32_t* out_n_free, int32_t* status, int B, int L, int page_size, int max_pages,
                              int capacity, int n_pages, void* stream) {
    return attn_page_plan_granted(seqlens, new_lens, block_table, free_pages, n_free, slots, out_seqlens, out_n_free, status,
                                  nullptr, B, L, page_size, max_pages, capacity, n_pages, stream);
}

extern "C" int attn_page_plan_granted(const int32_t* seqlens, const int32_t* new_lens, int32_t* block_table,
                                      const int32_t* free_pages, const int32_t* n_free, int32_t* slots,
                                      int32_t* out_seqlens, int32_t* out_n_free, int32_t* status, int32_t* granted, int B,
                                      int L, int page_size, int max_pages, int capacity, int n_pages, void* stream) {
    PlanParams p = {seqlens, new_lens, block_table, const_cast<int32_t*>(free_pages), n_free, slots, out_seqlens,
                    out_n_free, status, granted, B, L, page_size, max_pages, capacity, n_pages};
    int st = check_plan(p);
    if (st != ATTN_OK) return st;
    if (B > 0 && (!out_seqlens || !status || (!slots && L > 0)))
        return fail(ATTN_ERR_INVALID_ARG, "null slots, out_seqlens or status");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long n = static_cast<long long>(B) * L;
    const bool slots_too = n <= kPlanSlots;
    const bool one = B <= kPlanOneB && n <= kPlanOneSlots;
    if ((st = slots_too ? launch_plan(attn_page_plan_kernel<true>, one, s, p, "attn_page_plan_kernel")
                        : launch_plan(attn_page_plan_kernel<false>, one, s, p, "attn_page_plan_kernel")) != ATTN_OK)
        return st;
    if (!slots_too) {
        const long long units = static_cast<long long>(B) * ((L + static_cast<long long>(kSlotRun) - 1) / kSlotRun);
        const unsigned grid = static_cast<unsigned>(std::min<long long>(units, 148 * 64));
        const cudaError_t e = launch_dependent(attn_page_slots_kernel, grid, static_cast<unsigned>(kSlotThreads), s, p);
        if (e != cudaSuccess) return fail(ATTN_ERR_CUDA, "attn_page_slots_kernel launch failed: %s", cudaGetErrorString(e));
        if ((st = check_launch("attn_page_slots_kernel")) != ATTN_OK) return st;
    }
    return ok();
}

extern "C" int attn_page_release(const int32_t* seqlens, const int32_t* keep_lens, const int32_t* block_table,
                                 int32_t* free_pages, const int32_t* n_free, int32_t* out_n_free, int B, int page_size,
                                 int max_pages, int capacity, int n_pages, void* stream) {
    PlanParams p = {seqlens, keep_lens, const_cast<int32_t*>(block_table), free_pages, n_free, nullptr, nullptr,
                    out_n_free, nullptr, nullptr, B, 0, page_size, max_pages, capacity, n_pages};
    int st = check_plan(p);
    if (st != ATTN_OK) return st;
    st = launch_plan(attn_page_release_kernel, static_cast<long long>(B) * max_pages <= kReleaseEntries, static_cast<cudaStream_t>(stream), p,
                     "attn_page_release_kernel");
    return st == ATTN_OK ? ok() : st;
}

// ---- rotary append ----

namespace attn {
namespace {
// Eight tokens a CTA once that leaves four CTAs to each of 148 SMs, else one (and
// where a token's rows are so many that the kernel's division would not be exact).
constexpr long long kRopeManyTokens = 148LL * 4 * kRopeTokens;

template <int D, int FMT, int TOK>
int launch_rope_tokens(const RopeParams& p, bool adjacent, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.B) * p.L + TOK - 1) / TOK);
    if (adjacent)
        attn_rope_append_kernel<D, FMT, true, TOK><<<grid, kRopeThreads, 0, s>>>(p);
    else
        attn_rope_append_kernel<D, FMT, false, TOK><<<grid, kRopeThreads, 0, s>>>(p);
    return check_launch("attn_rope_append_kernel");
}
template <int D, int FMT>
int launch_rope(const RopeParams& p, bool adjacent, cudaStream_t s) {
    return static_cast<long long>(p.B) * p.L >= kRopeManyTokens && p.Hq + 2 * p.Hkv < 16384 ? launch_rope_tokens<D, FMT, kRopeTokens>(p, adjacent, s)
                                                                : launch_rope_tokens<D, FMT, 1>(p, adjacent, s);
}
template <int D>
int launch_rope_fmt(const RopeParams& p, int fmt, bool adjacent, cudaStream_t s) {
    if (fmt == kCacheBf16) return launch_rope<D, kCacheBf16>(p, adjacent, s);
    if constexpr (D <= 128)
        return fmt == ATTN_KV_E4M3 ? launch_rope<D, ATTN_KV_E4M3>(p, adjacent, s) : launch_rope<D, ATTN_KV_Q8_0>(p, adjacent, s);
    return fail(ATTN_ERR_UNSUPPORTED, "8-bit caches are built for D = 64 and 128");
}
}  // namespace
}  // namespace attn

extern "C" int attn_rope_append(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                                long long v_stride, const int32_t* positions, const float* inv_freq,
                                const int32_t* slots, void* q_out, void* k_cache, void* v_cache, void* k_scale,
                                void* v_scale, int kv_format, int B, int L, int Hq, int Hkv, int D, int rot,
                                int n_outer, int page_size, int n_axes, const int* sections, int axis_cycle,
                                int adjacent, void* stream) {
    if (B < 0 || L < 0 || Hq < 1 || Hkv < 1 || n_outer < 0 || page_size < 1)
        return fail(ATTN_ERR_INVALID_ARG, "bad size (B=%d L=%d Hq=%d Hkv=%d page_size=%d)", B, L, Hq, Hkv, page_size);
    if (D != 64 && D != 128 && D != 256) return fail(ATTN_ERR_UNSUPPORTED, "head dim D=%d (built: 64, 128, 256)", D);
    if (kv_format != 0 && kv_format != ATTN_KV_E4M3 && kv_format != ATTN_KV_Q8_0)
        return fail(ATTN_ERR_INVALID_ARG, "kv_format=%d (0: bf16, ATTN_KV_E4M3, ATTN_KV_Q8_0)", kv_format);
    if (kv_format != 0 && D > 128) return fail(ATTN_ERR_UNSUPPORTED, "8-bit caches are built for D = 64 and 128");
    if (rot < 0 || rot > D || rot % 16 != 0)
        return fail(ATTN_ERR_INVALID_ARG, "rot=%d must be a multiple of 16 in [0, D]", rot);
    if (n_axes < 1 || n_axes > 4 || !sections) return fail(ATTN_ERR_INVALID_ARG, "1 to 4 axes with their sections");
    int sum = 0;
    for (int a = 0; a < n_axes; ++a) {
        if (sections[a] < 0 || sections[a] > rot / 2)
            return fail(ATTN_ERR_INVALID_ARG, "sections[%d]=%d outside [0, rot / 2]", a, sections[a]);
        sum += sections[a];
        if (axis_cycle && a > 0 && sections[a] > 0 && a + n_axes * (sections[a] - 1) >= rot / 2)
            return fail(ATTN_ERR_INVALID_ARG, "axis %d in turn has no room for %d pairs", a, sections[a]);
    }
    if (sum != rot / 2) return fail(ATTN_ERR_INVALID_ARG, "sections sum to %d, not rot / 2 = %d", sum, rot / 2);
    const long long n = static_cast<long long>(B) * L;
    if (n > 0x7fffffffLL || static_cast<long long>(Hq) + 2LL * Hkv > 0xffffffLL)
        return fail(ATTN_ERR_UNSUPPORTED, "too many tokens or heads");
    if (static_cast<long long>(n_outer) * page_size > 0x7fffffffLL)
        return fail(ATTN_ERR_UNSUPPORTED, "cache too large for 32-bit slots");
    if (n == 0) return ok();
    if (!q || !q_out || !k || !v || !slots) return fail(ATTN_ERR_INVALID_ARG, "null q, k, v, slots or q_out");
    if ((!k_cache || !v_cache) && n_outer > 0) return fail(ATTN_ERR_INVALID_ARG, "null k_cache or v_cache");
    if (kv_format != 0 && (!k_scale || !v_scale)) return fail(ATTN_ERR_INVALID_ARG, "null k_scale or v_scale");
    if (rot > 0 && (!positions || !inv_freq)) return fail(ATTN_ERR_INVALID_ARG, "null positions or inv_freq");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache))
        return fail(ATTN_ERR_INVALID_ARG, "tensor base addresses must be 16-byte aligned");
    if (!aligned4(positions) || !aligned4(inv_freq) || !aligned4(slots) || !aligned4(k_scale) || !aligned4(v_scale))
        return fail(ATTN_ERR_INVALID_ARG, "positions, inv_freq, slots and scales must be 4-byte aligned");
    if (q_stride < static_cast<long long>(Hq) * D || q_stride % 8 != 0 || k_stride < static_cast<long long>(Hkv) * D ||
        k_stride % 8 != 0 || v_stride < static_cast<long long>(Hkv) * D || v_stride % 8 != 0)
        return fail(ATTN_ERR_INVALID_ARG, "token strides must be multiples of 8 elements and hold a token's heads");
    RopeParams p;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.q_tok = q_stride;
    p.k_tok = k_stride;
    p.v_tok = v_stride;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.slots = slots;
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.B = B;
    p.L = L;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.rot = rot;
    p.page_size = page_size;
    p.n_slots = static_cast<long long>(n_outer) * page_size;
    p.n_axes = n_axes;
    for (int a = 0; a < 4; ++a) p.sections[a] = a < n_axes ? sections[a] : 0;
    p.cycle = axis_cycle ? 1 : 0;
    p.row_div = static_cast<unsigned int>(0xffffffffu / static_cast<unsigned int>(Hq + 2 * Hkv)) + 1u;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool adj = adjacent != 0;
    const int st = (D == 256)   ? launch_rope_fmt<256>(p, kv_format, adj, s)
                   : (D == 128) ? launch_rope_fmt<128>(p, kv_format, adj, s)
                                : launch_rope_fmt<64>(p, kv_format, adj, s);
    return st == ATTN_OK ? ok() : st;
}

// ---- tree commit ----

extern "C" int attn_tree_commit(void* k_cache, void* v_cache, const int32_t* block_table, const int32_t* seqlens,
                                const int32_t* tree_lens, const int32_t* accept, const int32_t* n_accept,
                                int32_t* out_seqlens, int B, int Hkv, int T, int A, int D, int n_outer, int page_size,
                                int max_pages, void* stream) {
    if (B < 0 || Hkv < 1 || T < 1 || A < 0) return fail(ATTN_ERR_INVALID_ARG, "bad size (B=%d Hkv=%d T=%d A=%d)", B, Hkv, T, A);
    if (D != 64 && D != 128 && D != 256) return fail(ATTN_ERR_UNSUPPORTED, "head dim D=%d (built: 64, 128, 256)", D);
    if (T > kTreeMaxNodes) return fail(ATTN_ERR_UNSUPPORTED, "T=%d nodes (built: up to %d)", T, kTreeMaxNodes);
    if (Hkv > 0xffffff) return fail(ATTN_ERR_UNSUPPORTED, "too many heads (Hkv=%d)", Hkv);
    if (n_outer < 0 || page_size < 1 || (block_table && (n_outer < 1 || max_pages < 1)) || (!block_table && n_outer < B))
        return fail(ATTN_ERR_INVALID_ARG, "bad cache size (outer=%d rows=%d max_pages=%d)", n_outer, page_size, max_pages);
    if (block_table && static_cast<long long>(page_size) * max_pages > 0x7fffffffLL)
        return fail(ATTN_ERR_UNSUPPORTED, "page pool too large");
    if (B == 0) return ok();
    if (!k_cache || !v_cache || !seqlens || !n_accept || !out_seqlens || (!accept && A > 0))
        return fail(ATTN_ERR_INVALID_ARG, "null cache, seqlens, accept, n_accept or out_seqlens");
    if (!aligned16(k_cache) || !aligned16(v_cache)) return fail(ATTN_ERR_INVALID_ARG, "caches must be 16-byte aligned");
    if (!aligned4(block_table) || !aligned4(seqlens) || !aligned4(tree_lens) || !aligned4(accept) || !aligned4(n_accept) ||
        !aligned4(out_seqlens))
        return fail(ATTN_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    CommitParams p = {static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), block_table, seqlens, tree_lens, accept,
                      n_accept, out_seqlens, B, Hkv, T, A, D, page_size, max_pages, n_outer};
    attn_tree_commit_kernel<<<static_cast<unsigned>(B), kCommitThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    const int st = check_launch("attn_tree_commit_kernel");
    return st == ATTN_OK ? ok() : st;
}
