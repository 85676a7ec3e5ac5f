// torch_calls.cpp -- the Python binding of the serving-step calls of
// include/attn_gqa.h: argument checks, results and workspaces on torch tensors,
// and the call of the C function on the current stream.  No computation.
//
// These calls come at every layer or step, and on small batches the host bounds
// them, which is why they are bound here and not through ctypes: a page_plan of
// 64 requests takes 10 us of host time so and 16 through ctypes, a tree_commit 5 and 11.  The C functions' addresses
// come from the loaded library (bind), so both of its builds are reached alike.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <cmath>
#include <optional>
#include <string>

#include "../../include/attn_gqa.h"

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

namespace {

struct Calls {
    decltype(&attn_page_plan_granted) page_plan = nullptr;
    decltype(&attn_page_release) page_release = nullptr;
    decltype(&attn_rope_append) rope_append = nullptr;
    decltype(&attn_decode_tree) decode_tree = nullptr;
    decltype(&attn_decode_tree_workspace_size) tree_size = nullptr;
    decltype(&attn_decode_tree_paged) decode_tree_paged = nullptr;
    decltype(&attn_decode_tree_paged_workspace_size) tree_paged_size = nullptr;
    decltype(&attn_tree_commit) tree_commit = nullptr;
} calls;
// raises AttnError(status, description); lives as long as the interpreter
PyObject* check_status = nullptr;

void bind(const py::dict& addresses, const py::object& check) {
    auto get = [&](auto& fn, const char* name) {
        fn = reinterpret_cast<std::decay_t<decltype(fn)>>(py::cast<uintptr_t>(addresses[name]));
    };
    get(calls.page_plan, "attn_page_plan_granted");
    get(calls.page_release, "attn_page_release");
    get(calls.rope_append, "attn_rope_append");
    get(calls.decode_tree, "attn_decode_tree");
    get(calls.tree_size, "attn_decode_tree_workspace_size");
    get(calls.decode_tree_paged, "attn_decode_tree_paged");
    get(calls.tree_paged_size, "attn_decode_tree_paged_workspace_size");
    get(calls.tree_commit, "attn_tree_commit");
    check_status = check.inc_ref().ptr();
}

// The C call f(), without the interpreter's lock (a launch can wait for the device).
template <typename F>
void call(const char* what, F f) {
    int status;
    {
        const py::gil_scoped_release unlocked;
        status = f();
    }
    if (status != ATTN_OK) py::reinterpret_borrow<py::object>(check_status)(status, what);
}

std::string shape_of(at::IntArrayRef s) {
    std::string out = "(";
    for (size_t i = 0; i < s.size(); ++i) out += (i ? ", " : "") + std::to_string(s[i]);
    return out + (s.size() == 1 ? ",)" : ")");
}

// t is a contiguous CUDA tensor of this type and dimension, on `dev` where that is given
void need(const char* name, const Tensor& t, at::ScalarType type, int64_t dim, const c10::Device* dev) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be on a CUDA device");
    TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.dim() == dim, name, " must be ", dim, "-d, got shape ", shape_of(t.sizes()));
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    TORCH_CHECK_VALUE(dev == nullptr || t.device() == *dev, name, " is on ", t.device(), ", but the call's tensors are on ",
                      *dev);
}

// A caller's result tensor, checked against the shape the call writes, or a new one.
Tensor result(const char* name, const Maybe& given, at::ScalarType type, at::IntArrayRef shape, const c10::Device& dev) {
    if (!given) return at::empty(shape, at::TensorOptions(dev).dtype(type));
    need(name, *given, type, static_cast<int64_t>(shape.size()), &dev);
    TORCH_CHECK_VALUE(given->sizes() == shape, name, " must have shape ", shape_of(shape), ", got ", shape_of(given->sizes()));
    return *given;
}

int to_int(const char* name, int64_t x) {
    TORCH_CHECK_VALUE(x >= 0 && x <= 0x7fffffff, name, "=", x, " must lie in [0, 2^31 - 1]");
    return static_cast<int>(x);
}

template <typename T = int32_t>
T* ptr(const Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}
template <typename T = int32_t>
T* ptr(const Maybe& t) {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

void* current_stream(const c10::Device& dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// ---- pages ----

int64_t check_pages(const Tensor& seqlens, const Tensor& lens, const char* lens_name, const Tensor& table, const Tensor& free_pages,
                    const Tensor& n_free) {
    need("seqlens", seqlens, at::kInt, 1, nullptr);
    const c10::Device dev = seqlens.device();
    need(lens_name, lens, at::kInt, 1, &dev);
    need("block_table", table, at::kInt, 2, &dev);
    need("free_pages", free_pages, at::kInt, 1, &dev);
    need("n_free", n_free, at::kInt, 1, &dev);
    const int64_t B = seqlens.size(0);
    TORCH_CHECK_VALUE(lens.size(0) == B && table.size(0) == B && n_free.size(0) == 1, "shape mismatch between seqlens, ", lens_name,
                      ", block_table and n_free");
    return B;
}

std::tuple<Tensor, Tensor, Tensor, Tensor> page_plan(const Tensor& seqlens, const Tensor& new_lens, const Tensor& table,
                                                     const Tensor& free_pages, const Tensor& n_free, int64_t L, int64_t page_size,
                                                     int64_t n_pages, const Maybe& slots_, const Maybe& out_seqlens_,
                                                     const Maybe& out_n_free_, const Maybe& status_, const Maybe& granted) {
    const int l = to_int("L", L), page = to_int("page_size", page_size), pages = to_int("n_pages", n_pages);
    const int64_t B = check_pages(seqlens, new_lens, "new_lens", table, free_pages, n_free);
    const c10::Device dev = seqlens.device();
    const c10::cuda::CUDAGuard guard(dev);
    if (granted) result("granted", granted, at::kInt, {B}, dev);
    Tensor slots = result("slots", slots_, at::kInt, {B, L}, dev), lens = result("out_seqlens", out_seqlens_, at::kInt, {B}, dev);
    Tensor left = result("out_n_free", out_n_free_, at::kInt, {1}, dev), status = result("status", status_, at::kInt, {B}, dev);
    call("attn_page_plan", [&] {
        return calls.page_plan(ptr(seqlens), ptr(new_lens), ptr(table), ptr(free_pages), ptr(n_free), ptr(slots), ptr(lens), ptr(left),
                               ptr(status), ptr(granted), to_int("B", B), l, page, to_int("max_pages", table.size(1)),
                               to_int("capacity", free_pages.size(0)), pages, current_stream(dev));
    });
    return {slots, lens, left, status};
}

Tensor page_release(const Tensor& seqlens, const Tensor& keep_lens, const Tensor& table, const Tensor& free_pages, const Tensor& n_free,
                    int64_t page_size, int64_t n_pages, const Maybe& out_n_free_) {
    const int page = to_int("page_size", page_size), pages = to_int("n_pages", n_pages);
    const int64_t B = check_pages(seqlens, keep_lens, "keep_lens", table, free_pages, n_free);
    const c10::Device dev = seqlens.device();
    const c10::cuda::CUDAGuard guard(dev);
    Tensor left = result("out_n_free", out_n_free_, at::kInt, {1}, dev);
    call("attn_page_release", [&] {
        return calls.page_release(ptr(seqlens), ptr(keep_lens), ptr(table), ptr(free_pages), ptr(n_free), ptr(left), to_int("B", B),
                                  page, to_int("max_pages", table.size(1)), to_int("capacity", free_pages.size(0)), pages,
                                  current_stream(dev));
    });
    return left;
}

// ---- rotary append ----

// Elements from one token of t [B,L,H,D] to the next, heads dense.
int64_t token_stride(const char* name, const Tensor& t, const c10::Device& dev) {
    TORCH_CHECK_VALUE(t.is_cuda() && t.scalar_type() == at::kBFloat16 && t.dim() == 4 && t.device() == dev, name,
                      " must be a 4-d bf16 CUDA tensor [B,L,H,D], on the device of q");
    const int64_t B = t.size(0), L = t.size(1), H = t.size(2), D = t.size(3);
    if (B * L == 0) return H * D;
    TORCH_CHECK_VALUE((t.stride(3) == 1 || D <= 1) && (t.stride(2) == D || H <= 1), "the heads of a token of ", name,
                      " must be contiguous");
    const int64_t step = L > 1 ? t.stride(1) : B > 1 ? t.stride(0) : H * D;
    TORCH_CHECK_VALUE(B <= 1 || L <= 1 || t.stride(0) == L * step, "the tokens of ", name,
                      " must lie one stride apart (as in a part of one projection's output)");
    return step;
}

Tensor rope_append(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& positions, const Tensor& inv_freq, const Tensor& slots,
                   const Tensor& k_cache, const Tensor& v_cache, const std::optional<std::vector<int64_t>>& sections_, bool cycle,
                   bool adjacent, const Maybe& k_scale, const Maybe& v_scale, const Maybe& out_) {
    const c10::Device dev = q.device();
    const int64_t qs = token_stride("q", q, dev), ks = token_stride("k", k, dev), vs = token_stride("v", v, dev);
    const int64_t B = q.size(0), L = q.size(1), Hq = q.size(2), D = q.size(3), Hkv = k.size(2);
    TORCH_CHECK_VALUE(k.size(0) == B && k.size(1) == L && k.size(3) == D && v.sizes() == k.sizes(), "shape mismatch: q ",
                      shape_of(q.sizes()), " k ", shape_of(k.sizes()), " v ", shape_of(v.sizes()));
    const bool one_axis = positions.dim() == 2;                   // [B,L]
    need("positions", positions, at::kInt, one_axis ? 2 : 3, &dev);
    need("inv_freq", inv_freq, at::kFloat, 1, &dev);
    need("slots", slots, at::kInt, 2, &dev);
    const int64_t n_axes = one_axis ? 1 : positions.size(0), rot = 2 * inv_freq.size(0);
    TORCH_CHECK_VALUE(positions.size(-2) == B && positions.size(-1) == L && slots.size(0) == B && slots.size(1) == L,
                      "positions must be [n_axes,B,L] and slots [B,L]");
    const at::ScalarType type = k_cache.scalar_type();
    TORCH_CHECK_TYPE(type == at::kBFloat16 || type == at::kFloat8_e4m3fn || type == at::kChar,
                     "k_cache must be a bfloat16, float8_e4m3fn or int8 tensor");
    need("k_cache", k_cache, type, 4, &dev);
    need("v_cache", v_cache, type, 4, &dev);
    const int64_t n_outer = k_cache.size(0), rows = k_cache.size(2);
    TORCH_CHECK_VALUE(k_cache.size(1) == Hkv && k_cache.size(3) == D && v_cache.sizes() == k_cache.sizes(), "the caches must be [n,", Hkv,
                      ",rows,", D, "]");
    const int fmt = type == at::kBFloat16 ? 0 : type == at::kChar ? ATTN_KV_Q8_0 : ATTN_KV_E4M3;
    TORCH_CHECK_VALUE(k_scale.has_value() == (fmt != 0) && v_scale.has_value() == (fmt != 0),
                      "k_scale and v_scale go with an 8-bit cache, and only with one");
    if (fmt != 0) {
        const std::vector<int64_t> want = fmt == ATTN_KV_E4M3 ? std::vector<int64_t>{Hkv} : std::vector<int64_t>{n_outer, Hkv, rows, D / 32};
        for (const auto& [name, t] : {std::pair<const char*, const Tensor&>{"k_scale", *k_scale}, {"v_scale", *v_scale}}) {
            need(name, t, fmt == ATTN_KV_E4M3 ? at::kFloat : at::kHalf, static_cast<int64_t>(want.size()), &dev);
            TORCH_CHECK_VALUE(t.sizes() == at::IntArrayRef(want), name, " must have shape ", shape_of(want));
        }
    }
    std::vector<int> sections;
    if (!sections_)
        sections.push_back(to_int("sections", rot / 2));
    else
        for (const int64_t x : *sections_) sections.push_back(to_int("sections", x));
    TORCH_CHECK_VALUE(static_cast<int64_t>(sections.size()) == n_axes, n_axes, " position axes need as many sections, got ", sections.size());
    const c10::cuda::CUDAGuard guard(dev);
    Tensor out = result("out", out_, at::kBFloat16, {B, Hq, L, D}, dev);
    call("attn_rope_append", [&] {
        return calls.rope_append(ptr<void>(q), ptr<void>(k), ptr<void>(v), qs, ks, vs, ptr(positions), ptr<float>(inv_freq), ptr(slots),
                                 ptr<void>(out), ptr<void>(k_cache), ptr<void>(v_cache), ptr<void>(k_scale), ptr<void>(v_scale), fmt,
                                 to_int("B", B), to_int("L", L), to_int("Hq", Hq), to_int("Hkv", Hkv), to_int("D", D), to_int("rot", rot),
                                 to_int("n", n_outer), to_int("rows", rows), to_int("n_axes", n_axes), sections.data(), cycle, adjacent,
                                 current_stream(dev));
    });
    return out;
}

// ---- tree attention ----

// q, the caches (contiguous, or pools with a block table), seqlens and the tree's arrays; table may be none
std::tuple<Tensor, Maybe> decode_tree(const Tensor& q, const Tensor& k, const Tensor& v, const Maybe& table, const Tensor& seqlens,
                                      const Tensor& mask, const Maybe& tree_lens, std::optional<double> scale_, const Maybe& out_,
                                      const Maybe& lse_, bool want_lse, const Maybe& workspace_) {
    need("q", q, at::kBFloat16, 4, nullptr);
    const c10::Device dev = q.device();
    const char *k_name = table ? "k_pages" : "k_cache", *v_name = table ? "v_pages" : "v_cache";
    need(k_name, k, at::kBFloat16, 4, &dev);
    need(v_name, v, at::kBFloat16, 4, &dev);
    if (table) need("block_table", *table, at::kInt, 2, &dev);
    need("seqlens", seqlens, at::kInt, 1, &dev);
    const int64_t B = q.size(0), Hq = q.size(1), T = q.size(2), D = q.size(3);
    TORCH_CHECK_VALUE(k.size(3) == D && v.sizes() == k.sizes() && (table ? table->size(0) : k.size(0)) == B && seqlens.size(0) == B,
                      "shape mismatch between q, the ", table ? "page pools, block_table" : "caches", " and seqlens");
    TORCH_CHECK_VALUE(mask.dim() == 2 || mask.dim() == 3, "tree_mask must be a tensor [B,T,W] or [T,W]");
    const bool per_seq = mask.dim() == 3;
    need("tree_mask", mask, at::kInt, mask.dim(), &dev);
    TORCH_CHECK_VALUE((!per_seq || mask.size(0) == B) && mask.size(-2) == T && mask.size(-1) == (T + 31) / 32,
                      "tree_mask must have shape ", per_seq ? "[B,T,W]" : "[T,W]", " with T=", T, ", W=", (T + 31) / 32, ", got ",
                      shape_of(mask.sizes()));
    if (tree_lens) {
        need("tree_lens", *tree_lens, at::kInt, 1, &dev);
        TORCH_CHECK_VALUE(tree_lens->size(0) == B, "tree_lens must have ", B, " entries");
    }
    const int b = to_int("B", B), hq = to_int("Hq", Hq), hkv = to_int("Hkv", k.size(1)), t = to_int("T", T), d = to_int("D", D);
    const int rows = to_int("rows", k.size(2)), n_outer = to_int("n", k.size(0));
    const int max_pages = table ? to_int("max_pages", table->size(1)) : 0;
    const float scale = static_cast<float>(scale_ ? *scale_ : 1.0 / std::sqrt(static_cast<double>(D)));
    const c10::cuda::CUDAGuard guard(dev);
    Tensor out = out_ ? result("out", out_, at::kBFloat16, q.sizes(), dev) : at::empty_like(q);
    Maybe lse;
    if (lse_ || want_lse) lse = result("lse", lse_, at::kFloat, {B, Hq, T}, dev);
    const size_t size = table ? calls.tree_paged_size(b, hq, hkv, t, rows, max_pages, d) : calls.tree_size(b, hq, hkv, t, rows, d);
    Tensor workspace;
    size_t bytes = size;
    if (workspace_) {
        TORCH_CHECK_VALUE(workspace_->is_contiguous() && workspace_->device() == dev, "workspace must be a contiguous tensor on ", dev);
        workspace = *workspace_;
        bytes = static_cast<size_t>(workspace.numel()) * workspace.element_size();
    } else {
        workspace = at::empty({static_cast<int64_t>(std::max<size_t>(size, 1))}, at::TensorOptions(dev).dtype(at::kByte));
    }
    const uint32_t* words = ptr<uint32_t>(mask);
    if (table)
        call("attn_decode_tree_paged", [&] {
            return calls.decode_tree_paged(ptr<void>(q), ptr<void>(k), ptr<void>(v), ptr(*table), ptr(seqlens), words, per_seq, ptr(tree_lens),
                                           ptr<void>(out), ptr<float>(lse), b, hq, hkv, t, n_outer, rows, max_pages, d, scale,
                                           ptr<void>(workspace), bytes, current_stream(dev));
        });
    else
        call("attn_decode_tree", [&] {
            return calls.decode_tree(ptr<void>(q), ptr<void>(k), ptr<void>(v), ptr(seqlens), words, per_seq, ptr(tree_lens), ptr<void>(out),
                                     ptr<float>(lse), b, hq, hkv, t, rows, d, scale, ptr<void>(workspace), bytes, current_stream(dev));
        });
    return {out, lse};
}

// ---- tree commit ----

Tensor tree_commit(const Tensor& k, const Tensor& v, const Tensor& seqlens, const Tensor& accept, const Tensor& n_accept, int64_t T,
                   const Maybe& table, const Maybe& tree_lens, const Maybe& out_seqlens_) {
    const int t = to_int("T", T);
    need("k_cache", k, at::kBFloat16, 4, nullptr);
    const c10::Device dev = k.device();
    need("v_cache", v, at::kBFloat16, 4, &dev);
    need("seqlens", seqlens, at::kInt, 1, &dev);
    need("accept", accept, at::kInt, 2, &dev);
    need("n_accept", n_accept, at::kInt, 1, &dev);
    const int64_t B = seqlens.size(0);
    TORCH_CHECK_VALUE(v.sizes() == k.sizes() && accept.size(0) == B && n_accept.size(0) == B,
                      "shape mismatch between the caches, seqlens, accept and n_accept");
    if (table) need("block_table", *table, at::kInt, 2, &dev);
    if (tree_lens) need("tree_lens", *tree_lens, at::kInt, 1, &dev);
    TORCH_CHECK_VALUE((table ? table->size(0) : k.size(0)) == B && (!tree_lens || tree_lens->size(0) == B),
                      "shape mismatch between seqlens, the caches, block_table and tree_lens");
    const c10::cuda::CUDAGuard guard(dev);
    Tensor out = result("out_seqlens", out_seqlens_, at::kInt, {B}, dev);
    call("attn_tree_commit", [&] {
        return calls.tree_commit(ptr<void>(k), ptr<void>(v), ptr(table), ptr(seqlens), ptr(tree_lens), ptr(accept), ptr(n_accept), ptr(out),
                                 to_int("B", B), to_int("Hkv", k.size(1)), t, to_int("A", accept.size(1)), to_int("D", k.size(3)),
                                 to_int("n", k.size(0)), to_int("rows", k.size(2)), table ? to_int("max_pages", table->size(1)) : 0,
                                 current_stream(dev));
    });
    return out;
}

}  // namespace

PYBIND11_MODULE(_torch_calls, m) {
    m.def("bind", &bind);
    m.def("page_plan", &page_plan);
    m.def("page_release", &page_release);
    m.def("rope_append", &rope_append);
    m.def("decode_tree", &decode_tree);
    m.def("tree_commit", &tree_commit);
}
