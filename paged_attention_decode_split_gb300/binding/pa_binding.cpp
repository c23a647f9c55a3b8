// pa_binding.cpp -- the compiled half of the Python binding: each call checks
// its tensors against the attention description (element type, shape, CUDA
// device, contiguity) and hands their pointers to the C ABI of
// include/pagedattn.h.  It computes nothing.
//
// The C ABI sees bare pointers and cannot tell a buffer's size, so a tensor of
// the wrong type or shape would be read or written past its end; the checks
// come before the call.  They run here rather than in Python because a
// decode step is one call per layer and the Python attribute lookups of eleven
// tensors cost more host time per call than the kernel takes on the GPU.
//
// The library is not linked: the Python side passes the addresses of the C
// entry points it loaded (set_entry), so the process holds one copy of the
// library and its host-side state (last plan, tensor-map cache).
#include <torch/extension.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <array>
#include <initializer_list>
#include <string>
#include <utility>
#include <vector>

#include "pagedattn.h"

namespace {

using at::Tensor;
using c10::optional;

using AttnFn = pa_status (*)(const void *, const void *, const void *, const int32_t *, const int32_t *,
                             const pa_attn_desc *, void *, void *, size_t, int32_t *, void *);
using AttnFp8Fn = pa_status (*)(const void *, const void *, const void *, const float *, const float *,
                                const int32_t *, const int32_t *, const pa_attn_desc *, void *, void *, size_t,
                                int32_t *, void *);
using AppendFn = pa_status (*)(const void *, const void *, const void *, void *, void *, const int32_t *,
                               const int32_t *, const pa_attn_desc *, void *, void *, size_t, int32_t *, void *);
using AppendFp8Fn = pa_status (*)(const void *, const void *, const void *, void *, void *, const float *,
                                  const float *, const int32_t *, const int32_t *, const pa_attn_desc *, void *,
                                  void *, size_t, int32_t *, void *);
using NoAllocFn = pa_status (*)(const void *, const void *, const void *, const int32_t *, const int32_t *,
                                const pa_attn_desc *, void *, int32_t *, void *);
using ReshapeFn = pa_status (*)(const void *, const void *, void *, void *, const int64_t *, int32_t, int32_t,
                                int32_t, int32_t, int64_t, int32_t *, void *);
using ReshapeFp8Fn = pa_status (*)(const void *, const void *, void *, void *, const int64_t *, const float *,
                                   const float *, int32_t, int32_t, int32_t, int32_t, int64_t, int32_t *, void *);

using GatherFn = pa_status (*)(const void *, const void *, const int64_t *, const float *, const float *, void *,
                               void *, int32_t, int32_t, int32_t, int32_t, int32_t, int64_t, int32_t *, void *);
using ExtendFn = pa_status (*)(const int32_t *, const int32_t *, int32_t *, const int32_t *, const int32_t *, int32_t,
                               int32_t, int32_t, int64_t, int32_t, int32_t *, int64_t *, int32_t *, int32_t *, void *);
using ReleaseFn = pa_status (*)(const int32_t *, const int32_t *, const int32_t *, int32_t *, const int32_t *, int32_t,
                                int32_t, int32_t, int64_t, int32_t *, int32_t *, int32_t *, void *);

using SharedFn = pa_status (*)(const void *, const void *, const void *, const int32_t *, const int32_t *,
                               const int32_t *, const int32_t *, const pa_attn_desc *, const pa_prefix_desc *, void *,
                               void *, size_t, int32_t *, void *);
using SharedQuantFn = pa_status (*)(const void *, const void *, const void *, const float *, const float *,
                                    const int32_t *, const int32_t *, const int32_t *, const int32_t *,
                                    const pa_attn_desc *, const pa_prefix_desc *, void *, void *, size_t, int32_t *,
                                    void *);
using RotaryFn = pa_status (*)(const void *, const void *, const int32_t *, const int64_t *, void *, void *,
                               const pa_rotary_desc *, void *);
using RotaryCacheFn = pa_status (*)(const void *, const void *, const void *, const int32_t *, const int64_t *, void *,
                                    void *, void *, const int64_t *, const pa_rotary_desc *, int32_t, int64_t,
                                    int32_t *, void *);
using RotaryQuantFn = pa_status (*)(const void *, const void *, const void *, const int32_t *, const int64_t *, void *,
                                    void *, void *, const int64_t *, const float *, const float *,
                                    const pa_rotary_desc *, int32_t, int64_t, int32_t *, void *);
using ForkFn = pa_status (*)(const int32_t *, const int32_t *, int32_t *, const int32_t *, const int32_t *,
                             const int32_t *, int32_t, int32_t, int32_t, int64_t, int32_t *, int32_t *, int32_t *,
                             int32_t *, int32_t *, int32_t *, int32_t *, void *);
using ReleaseSharedFn = pa_status (*)(const int32_t *, const int32_t *, const int32_t *, int32_t *, const int32_t *,
                                      const int32_t *, int32_t, int32_t, int32_t, int64_t, int32_t *, int32_t *,
                                      int32_t *, int32_t *, void *);
using CompactFn = pa_status (*)(const int32_t *, int32_t *, const int32_t *, const int32_t *, const int32_t *, int32_t,
                                int32_t, int32_t, int64_t, int32_t, int32_t *, int32_t *, int32_t *, int32_t *,
                                int32_t *, int32_t *, int32_t *, int32_t *, void *);
using CopyFn = pa_status (*)(void *const *, int32_t, const int32_t *, const int32_t *, const int32_t *, int32_t, int32_t,
                             int64_t, int32_t, int64_t, int32_t *, void *);

struct Entries {
    AttnFn decode = nullptr, verify = nullptr;
    AttnFp8Fn decode_fp8 = nullptr, verify_fp8 = nullptr;
    AppendFn decode_append = nullptr;
    AppendFp8Fn decode_append_fp8 = nullptr;
    NoAllocFn decode_noalloc = nullptr;
    ReshapeFn reshape = nullptr;
    ReshapeFp8Fn reshape_fp8 = nullptr;
    AttnFp8Fn decode_fp4 = nullptr, verify_fp4 = nullptr;
    AppendFp8Fn decode_append_fp4 = nullptr;
    ReshapeFp8Fn reshape_fp4 = nullptr;
    GatherFn gather_fp4 = nullptr;
    ExtendFn extend_tables = nullptr;
    ReleaseFn release_tables = nullptr;
    SharedFn shared = nullptr;
    SharedQuantFn shared_fp8 = nullptr, shared_fp4 = nullptr;
    RotaryFn rotary = nullptr;
    RotaryCacheFn rotary_and_cache = nullptr;
    RotaryQuantFn rotary_and_cache_fp8 = nullptr, rotary_and_cache_fp4 = nullptr;
    ForkFn fork_tables = nullptr;
    ReleaseSharedFn release_shared = nullptr;
    CompactFn compact_tables = nullptr;
    CopyFn copy_pages = nullptr;
} g_entries;

void set_entry(const std::string &name, int64_t addr) {
    void *p = reinterpret_cast<void *>(addr);
    if (name == "pa_paged_attention_decode") g_entries.decode = reinterpret_cast<AttnFn>(p);
    else if (name == "pa_paged_attention_verify") g_entries.verify = reinterpret_cast<AttnFn>(p);
    else if (name == "pa_paged_attention_decode_fp8") g_entries.decode_fp8 = reinterpret_cast<AttnFp8Fn>(p);
    else if (name == "pa_paged_attention_verify_fp8") g_entries.verify_fp8 = reinterpret_cast<AttnFp8Fn>(p);
    else if (name == "pa_paged_attention_decode_append") g_entries.decode_append = reinterpret_cast<AppendFn>(p);
    else if (name == "pa_paged_attention_decode_append_fp8")
        g_entries.decode_append_fp8 = reinterpret_cast<AppendFp8Fn>(p);
    else if (name == "pa_paged_attention_decode_noalloc") g_entries.decode_noalloc = reinterpret_cast<NoAllocFn>(p);
    else if (name == "pa_reshape_and_cache") g_entries.reshape = reinterpret_cast<ReshapeFn>(p);
    else if (name == "pa_reshape_and_cache_fp8") g_entries.reshape_fp8 = reinterpret_cast<ReshapeFp8Fn>(p);
    else if (name == "pa_paged_attention_decode_fp4") g_entries.decode_fp4 = reinterpret_cast<AttnFp8Fn>(p);
    else if (name == "pa_paged_attention_verify_fp4") g_entries.verify_fp4 = reinterpret_cast<AttnFp8Fn>(p);
    else if (name == "pa_paged_attention_decode_append_fp4")
        g_entries.decode_append_fp4 = reinterpret_cast<AppendFp8Fn>(p);
    else if (name == "pa_reshape_and_cache_fp4") g_entries.reshape_fp4 = reinterpret_cast<ReshapeFp8Fn>(p);
    else if (name == "pa_gather_cache_fp4") g_entries.gather_fp4 = reinterpret_cast<GatherFn>(p);
    else if (name == "pa_extend_block_tables") g_entries.extend_tables = reinterpret_cast<ExtendFn>(p);
    else if (name == "pa_release_block_tables") g_entries.release_tables = reinterpret_cast<ReleaseFn>(p);
    else if (name == "pa_paged_attention_decode_shared") g_entries.shared = reinterpret_cast<SharedFn>(p);
    else if (name == "pa_paged_attention_decode_shared_fp8") g_entries.shared_fp8 = reinterpret_cast<SharedQuantFn>(p);
    else if (name == "pa_paged_attention_decode_shared_fp4") g_entries.shared_fp4 = reinterpret_cast<SharedQuantFn>(p);
    else if (name == "pa_rotary") g_entries.rotary = reinterpret_cast<RotaryFn>(p);
    else if (name == "pa_rotary_and_cache") g_entries.rotary_and_cache = reinterpret_cast<RotaryCacheFn>(p);
    else if (name == "pa_rotary_and_cache_fp8") g_entries.rotary_and_cache_fp8 = reinterpret_cast<RotaryQuantFn>(p);
    else if (name == "pa_rotary_and_cache_fp4") g_entries.rotary_and_cache_fp4 = reinterpret_cast<RotaryQuantFn>(p);
    else if (name == "pa_fork_block_tables") g_entries.fork_tables = reinterpret_cast<ForkFn>(p);
    else if (name == "pa_release_shared_block_tables") g_entries.release_shared = reinterpret_cast<ReleaseSharedFn>(p);
    else if (name == "pa_compact_block_tables") g_entries.compact_tables = reinterpret_cast<CompactFn>(p);
    else if (name == "pa_copy_cache_pages") g_entries.copy_pages = reinterpret_cast<CopyFn>(p);
    else TORCH_CHECK_VALUE(false, "unknown entry point ", name);
}

bool is_fp8_cache_type(at::ScalarType t) { return t == at::kByte || t == at::ScalarType::Float8_e4m3fn; }

// Element type and shape (when `check_shape`) of one tensor.  The device and
// layout checks come after every tensor's type and shape (`placed`), so that a
// call's first error names the argument that does not fit the description.
void expect(const Tensor &t, const char *name, bool type_ok, const char *want, c10::IntArrayRef shape,
            bool check_shape = true) {
    TORCH_CHECK_VALUE(type_ok, name, ": dtype ", t.scalar_type(), "; expected ", want);
    if (check_shape) TORCH_CHECK_VALUE(t.sizes().equals(shape), name, ": shape ", t.sizes(), "; expected ", shape);
}

// The library launches on the current device, so every tensor must live there.
void placed(std::initializer_list<std::pair<const Tensor *, const char *>> ts) {
    int dev = -1;
    for (const auto &[t, name] : ts) {
        if (t == nullptr) continue;
        TORCH_CHECK_VALUE(t->is_cuda(), name, ": a CUDA tensor is required (got ", t->device(), ")");
        if (dev < 0) dev = c10::cuda::current_device();
        TORCH_CHECK_VALUE(t->get_device() == dev, name, ": on ", t->device(), ", but the current device is cuda:", dev);
        TORCH_CHECK_VALUE(t->is_contiguous(), name, ": the tensor must be contiguous");
    }
}

const Tensor *opt(const optional<Tensor> &t) { return t.has_value() ? &*t : nullptr; }

void *stream_of(int64_t s) {
    return s == -1 ? static_cast<void *>(c10::cuda::getCurrentCUDAStream().stream()) : reinterpret_cast<void *>(s);
}

template <typename T>
T *ptr_of(const optional<Tensor> &t) {
    return t.has_value() ? static_cast<T *>(t->data_ptr()) : nullptr;
}

enum Kind {
    kDecode = 0, kDecodeAppend, kVerify, kDecodeFp8, kDecodeAppendFp8, kVerifyFp8, kDecodeNoAlloc, kDecodeFp4,
    kDecodeAppendFp4, kVerifyFp4, kShared, kSharedFp8, kSharedFp4
};

// One attention call of the given kind (the C entry point it maps to is in the
// switch below); returns the pa_status of the call.
int64_t attention(int64_t kind, const Tensor &q, const Tensor &k_cache, const Tensor &v_cache,
                  const optional<Tensor> &k_scale, const optional<Tensor> &v_scale, const optional<Tensor> &k_new,
                  const optional<Tensor> &v_new, const Tensor &block_table, const Tensor &seq_lens,
                  int64_t desc_addr, const Tensor &out, const optional<Tensor> &workspace,
                  const optional<Tensor> &status, int64_t stream, const optional<Tensor> &group_starts = {},
                  const optional<Tensor> &prefix_lens = {}, int64_t prefix_addr = 0) {
    TORCH_CHECK_VALUE(desc_addr != 0, "desc: a description is required");
    const pa_attn_desc *d = reinterpret_cast<const pa_attn_desc *>(desc_addr);
    const bool fp8 = kind == kDecodeFp8 || kind == kDecodeAppendFp8 || kind == kVerifyFp8 || kind == kSharedFp8;
    const bool fp4 = kind == kDecodeFp4 || kind == kDecodeAppendFp4 || kind == kVerifyFp4 || kind == kSharedFp4;
    const bool shared = kind == kShared || kind == kSharedFp8 || kind == kSharedFp4;
    const pa_prefix_desc *x = reinterpret_cast<const pa_prefix_desc *>(prefix_addr);
    const bool append = kind == kDecodeAppend || kind == kDecodeAppendFp8 || kind == kDecodeAppendFp4;
    const int64_t rows = static_cast<int64_t>(d->num_seqs) * d->q_len;
    const std::array<int64_t, 3> row_shape{rows, d->num_q_heads, d->head_dim};
    std::array<int64_t, 4> cache_shape{d->num_pages, d->block_size, d->num_kv_heads, d->head_dim};
    if (fp4) cache_shape = {d->num_pages, d->num_kv_heads, d->block_size / 16, 9 * int64_t(d->head_dim)};
    expect(q, "q", q.scalar_type() == at::kBFloat16, "bfloat16", row_shape);
    auto cache_ok = [&](const Tensor &t) {
        return fp4 ? t.scalar_type() == at::kByte
                   : fp8 ? is_fp8_cache_type(t.scalar_type()) : t.scalar_type() == at::kBFloat16;
    };
    const bool kc_ok = cache_ok(k_cache), vc_ok = cache_ok(v_cache);
    const char *cache_want = fp4 ? "uint8 (fp4 records)" : fp8 ? "uint8 or float8_e4m3fn (e4m3 codes)" : "bfloat16";
    expect(k_cache, "k_cache", kc_ok, cache_want, cache_shape);
    expect(v_cache, "v_cache", vc_ok, cache_want, cache_shape);
    expect(block_table, "block_table", block_table.scalar_type() == at::kInt, "int32",
           std::array<int64_t, 2>{d->num_seqs, d->max_pages_per_seq});
    expect(seq_lens, "seq_lens", seq_lens.scalar_type() == at::kInt, "int32", std::array<int64_t, 1>{d->num_seqs});
    const bool out_bf16 = d->out_dtype == PA_OUT_BF16;
    expect(out, "out", out.scalar_type() == (out_bf16 ? at::kBFloat16 : at::kFloat), out_bf16 ? "bfloat16" : "float32",
           row_shape);
    const std::array<int64_t, 1> scale_shape{d->num_kv_heads};
    TORCH_CHECK_VALUE(!(fp8 || fp4) || (k_scale.has_value() && v_scale.has_value()), "k_scale, v_scale: ",
                      fp4 ? "an fp4" : "an e4m3", " cache needs both");
    if (k_scale.has_value()) expect(*k_scale, "k_scale", k_scale->scalar_type() == at::kFloat, "float32", scale_shape);
    if (v_scale.has_value()) expect(*v_scale, "v_scale", v_scale->scalar_type() == at::kFloat, "float32", scale_shape);
    if (append) {
        TORCH_CHECK_VALUE(k_new.has_value() && v_new.has_value(), "k_new, v_new: the new rows are required");
        const std::array<int64_t, 3> new_shape{d->num_seqs, d->num_kv_heads, d->head_dim};
        expect(*k_new, "k_new", k_new->scalar_type() == at::kBFloat16, "bfloat16", new_shape);
        expect(*v_new, "v_new", v_new->scalar_type() == at::kBFloat16, "bfloat16", new_shape);
    }
    if (shared) {
        TORCH_CHECK_VALUE(x != nullptr, "prefix: a description is required");
        TORCH_CHECK_VALUE(group_starts.has_value() && prefix_lens.has_value(), "group_starts, prefix_lens: both are required");
        expect(*group_starts, "group_starts", group_starts->scalar_type() == at::kInt, "int32",
               std::array<int64_t, 1>{int64_t(x->num_groups) + 1});
        expect(*prefix_lens, "prefix_lens", prefix_lens->scalar_type() == at::kInt, "int32",
               std::array<int64_t, 1>{d->num_seqs});
    }
    size_t ws_bytes = 0;
    if (workspace.has_value()) ws_bytes = workspace->numel() * workspace->element_size();
    if (status.has_value())
        expect(*status, "status", status->scalar_type() == at::kInt && status->numel() >= 1, "int32 (one element)",
               {}, false);
    placed({{&q, "q"}, {&k_cache, "k_cache"}, {&v_cache, "v_cache"}, {&block_table, "block_table"},
            {&seq_lens, "seq_lens"}, {&out, "out"}, {opt(k_scale), "k_scale"}, {opt(v_scale), "v_scale"},
            {opt(k_new), "k_new"}, {opt(v_new), "v_new"}, {opt(workspace), "workspace"}, {opt(status), "status"},
            {opt(group_starts), "group_starts"}, {opt(prefix_lens), "prefix_lens"}});

    const void *qp = q.data_ptr();
    void *kc = k_cache.data_ptr(), *vc = v_cache.data_ptr(), *op = out.data_ptr(), *wp = ptr_of<void>(workspace);
    const int32_t *bt = block_table.data_ptr<int32_t>(), *sl = seq_lens.data_ptr<int32_t>();
    int32_t *st = ptr_of<int32_t>(status);
    const float *ks = ptr_of<float>(k_scale), *vs = ptr_of<float>(v_scale);
    const void *kn = ptr_of<void>(k_new), *vn = ptr_of<void>(v_new);
    void *s = stream_of(stream);
    switch (kind) {
        case kDecode:
            TORCH_CHECK(g_entries.decode, "entry point not set");
            return g_entries.decode(qp, kc, vc, bt, sl, d, op, wp, ws_bytes, st, s);
        case kVerify:
            TORCH_CHECK(g_entries.verify, "entry point not set");
            return g_entries.verify(qp, kc, vc, bt, sl, d, op, wp, ws_bytes, st, s);
        case kDecodeFp8:
            TORCH_CHECK(g_entries.decode_fp8, "entry point not set");
            return g_entries.decode_fp8(qp, kc, vc, ks, vs, bt, sl, d, op, wp, ws_bytes, st, s);
        case kVerifyFp8:
            TORCH_CHECK(g_entries.verify_fp8, "entry point not set");
            return g_entries.verify_fp8(qp, kc, vc, ks, vs, bt, sl, d, op, wp, ws_bytes, st, s);
        case kDecodeAppend:
            TORCH_CHECK(g_entries.decode_append, "entry point not set");
            return g_entries.decode_append(qp, kn, vn, kc, vc, bt, sl, d, op, wp, ws_bytes, st, s);
        case kDecodeAppendFp8:
            TORCH_CHECK(g_entries.decode_append_fp8, "entry point not set");
            return g_entries.decode_append_fp8(qp, kn, vn, kc, vc, ks, vs, bt, sl, d, op, wp, ws_bytes, st, s);
        case kDecodeFp4:
            TORCH_CHECK(g_entries.decode_fp4, "entry point not set");
            return g_entries.decode_fp4(qp, kc, vc, ks, vs, bt, sl, d, op, wp, ws_bytes, st, s);
        case kVerifyFp4:
            TORCH_CHECK(g_entries.verify_fp4, "entry point not set");
            return g_entries.verify_fp4(qp, kc, vc, ks, vs, bt, sl, d, op, wp, ws_bytes, st, s);
        case kDecodeAppendFp4:
            TORCH_CHECK(g_entries.decode_append_fp4, "entry point not set");
            return g_entries.decode_append_fp4(qp, kn, vn, kc, vc, ks, vs, bt, sl, d, op, wp, ws_bytes, st, s);
        case kDecodeNoAlloc:
            TORCH_CHECK(g_entries.decode_noalloc, "entry point not set");
            return g_entries.decode_noalloc(qp, kc, vc, bt, sl, d, op, st, s);
    }
    if (shared) {
        const int32_t *gs = group_starts->data_ptr<int32_t>(), *pl = prefix_lens->data_ptr<int32_t>();
        if (kind == kShared) {
            TORCH_CHECK(g_entries.shared, "entry point not set");
            return g_entries.shared(qp, kc, vc, bt, sl, gs, pl, d, x, op, wp, ws_bytes, st, s);
        }
        const SharedQuantFn fn = fp4 ? g_entries.shared_fp4 : g_entries.shared_fp8;
        TORCH_CHECK(fn, "entry point not set");
        return fn(qp, kc, vc, ks, vs, bt, sl, gs, pl, d, x, op, wp, ws_bytes, st, s);
    }
    TORCH_CHECK_VALUE(false, "unknown call kind ", kind);
    return PA_ERR_INVALID_ARG;
}

// reshape_and_cache (bf16) or reshape_and_cache_fp8: the geometry comes from
// the cache tensor itself.
int64_t reshape(bool fp8, const Tensor &k_new, const Tensor &v_new, const Tensor &k_cache, const Tensor &v_cache,
                const Tensor &slot_mapping, const optional<Tensor> &k_scale, const optional<Tensor> &v_scale,
                const optional<Tensor> &status, int64_t stream) {
    TORCH_CHECK_VALUE(k_cache.dim() == 4, "k_cache: a [pages, block_size, kv_heads, head_dim] tensor is required");
    TORCH_CHECK_VALUE(slot_mapping.dim() == 1, "slot_mapping: a one-dimensional tensor is required");
    const int64_t n = slot_mapping.size(0), hkv = k_cache.size(2), dim = k_cache.size(3);
    const char *cache_want = fp8 ? "uint8 or float8_e4m3fn (e4m3 codes)" : "bfloat16";
    expect(k_cache, "k_cache", fp8 ? is_fp8_cache_type(k_cache.scalar_type()) : k_cache.scalar_type() == at::kBFloat16,
           cache_want, {}, false);
    expect(v_cache, "v_cache", v_cache.scalar_type() == k_cache.scalar_type(), cache_want, k_cache.sizes());
    const std::array<int64_t, 3> new_shape{n, hkv, dim};
    expect(k_new, "k_new", k_new.scalar_type() == at::kBFloat16, "bfloat16", new_shape);
    expect(v_new, "v_new", v_new.scalar_type() == at::kBFloat16, "bfloat16", new_shape);
    expect(slot_mapping, "slot_mapping", slot_mapping.scalar_type() == at::kLong, "int64", {}, false);
    const std::array<int64_t, 1> scale_shape{hkv};
    TORCH_CHECK_VALUE(!fp8 || (k_scale.has_value() && v_scale.has_value()), "k_scale, v_scale: an e4m3 cache needs both");
    if (k_scale.has_value()) expect(*k_scale, "k_scale", k_scale->scalar_type() == at::kFloat, "float32", scale_shape);
    if (v_scale.has_value()) expect(*v_scale, "v_scale", v_scale->scalar_type() == at::kFloat, "float32", scale_shape);
    if (status.has_value())
        expect(*status, "status", status->scalar_type() == at::kInt && status->numel() >= 1, "int32 (one element)",
               {}, false);
    placed({{&k_new, "k_new"}, {&v_new, "v_new"}, {&k_cache, "k_cache"}, {&v_cache, "v_cache"},
            {&slot_mapping, "slot_mapping"}, {opt(k_scale), "k_scale"}, {opt(v_scale), "v_scale"},
            {opt(status), "status"}});
    int32_t *st = ptr_of<int32_t>(status);
    void *s = stream_of(stream);
    if (fp8) {
        TORCH_CHECK(g_entries.reshape_fp8, "entry point not set");
        return g_entries.reshape_fp8(k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                     slot_mapping.data_ptr<int64_t>(), ptr_of<float>(k_scale), ptr_of<float>(v_scale),
                                     static_cast<int32_t>(n), static_cast<int32_t>(hkv), static_cast<int32_t>(dim),
                                     static_cast<int32_t>(k_cache.size(1)), k_cache.size(0), st, s);
    }
    TORCH_CHECK(g_entries.reshape, "entry point not set");
    return g_entries.reshape(k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                             slot_mapping.data_ptr<int64_t>(), static_cast<int32_t>(n), static_cast<int32_t>(hkv),
                             static_cast<int32_t>(dim), static_cast<int32_t>(k_cache.size(1)), k_cache.size(0), st, s);
}

// The rows, slots and scales of an fp4 cache call; the geometry comes from the
// cache tensor [pages, kv_heads, block_size / 16, 9 * head_dim].
struct Fp4Geometry {
    int32_t n, hkv, dim, block_size;
    int64_t pages;
};
Fp4Geometry fp4_geometry(const Tensor &k_cache, const Tensor &v_cache, const Tensor &slot_mapping,
                         const Tensor &k_scale, const Tensor &v_scale, const optional<Tensor> &status) {
    TORCH_CHECK_VALUE(k_cache.dim() == 4 && k_cache.size(3) % 9 == 0,
                      "k_cache: a [pages, kv_heads, block_size / 16, 9 * head_dim] tensor is required");
    TORCH_CHECK_VALUE(slot_mapping.dim() == 1, "slot_mapping: a one-dimensional tensor is required");
    expect(k_cache, "k_cache", k_cache.scalar_type() == at::kByte, "uint8 (fp4 records)", {}, false);
    expect(v_cache, "v_cache", v_cache.scalar_type() == at::kByte, "uint8 (fp4 records)", k_cache.sizes());
    expect(slot_mapping, "slot_mapping", slot_mapping.scalar_type() == at::kLong, "int64", {}, false);
    for (int i = 0; i < 4; ++i)
        TORCH_CHECK_VALUE(k_cache.size(i) <= INT32_MAX / 16, "k_cache: dimension ", i, " is too large");
    TORCH_CHECK_VALUE(slot_mapping.size(0) <= INT32_MAX, "slot_mapping: too many tokens");
    const std::array<int64_t, 1> scale_shape{k_cache.size(1)};
    expect(k_scale, "k_scale", k_scale.scalar_type() == at::kFloat, "float32", scale_shape);
    expect(v_scale, "v_scale", v_scale.scalar_type() == at::kFloat, "float32", scale_shape);
    if (status.has_value())
        expect(*status, "status", status->scalar_type() == at::kInt && status->numel() >= 1, "int32 (one element)",
               {}, false);
    return {static_cast<int32_t>(slot_mapping.size(0)), static_cast<int32_t>(k_cache.size(1)),
            static_cast<int32_t>(k_cache.size(3) / 9), static_cast<int32_t>(k_cache.size(2) * 16), k_cache.size(0)};
}

int64_t reshape_fp4(const Tensor &k_new, const Tensor &v_new, const Tensor &k_cache, const Tensor &v_cache,
                    const Tensor &slot_mapping, const Tensor &k_scale, const Tensor &v_scale,
                    const optional<Tensor> &status, int64_t stream) {
    const Fp4Geometry g = fp4_geometry(k_cache, v_cache, slot_mapping, k_scale, v_scale, status);
    const std::array<int64_t, 3> new_shape{g.n, g.hkv, g.dim};
    expect(k_new, "k_new", k_new.scalar_type() == at::kBFloat16, "bfloat16", new_shape);
    expect(v_new, "v_new", v_new.scalar_type() == at::kBFloat16, "bfloat16", new_shape);
    placed({{&k_new, "k_new"}, {&v_new, "v_new"}, {&k_cache, "k_cache"}, {&v_cache, "v_cache"},
            {&slot_mapping, "slot_mapping"}, {&k_scale, "k_scale"}, {&v_scale, "v_scale"}, {opt(status), "status"}});
    TORCH_CHECK(g_entries.reshape_fp4, "entry point not set");
    return g_entries.reshape_fp4(k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                 slot_mapping.data_ptr<int64_t>(), k_scale.data_ptr<float>(),
                                 v_scale.data_ptr<float>(), g.n, g.hkv, g.dim, g.block_size, g.pages,
                                 ptr_of<int32_t>(status), stream_of(stream));
}

int64_t gather_fp4(const Tensor &k_cache, const Tensor &v_cache, const Tensor &slot_mapping, const Tensor &k_scale,
                   const Tensor &v_scale, const Tensor &k_out, const Tensor &v_out, const optional<Tensor> &status,
                   int64_t stream) {
    const Fp4Geometry g = fp4_geometry(k_cache, v_cache, slot_mapping, k_scale, v_scale, status);
    const std::array<int64_t, 3> out_shape{g.n, g.hkv, g.dim};
    const bool bf = k_out.scalar_type() == at::kBFloat16;
    expect(k_out, "k_out", bf || k_out.scalar_type() == at::kFloat, "bfloat16 or float32", out_shape);
    expect(v_out, "v_out", v_out.scalar_type() == k_out.scalar_type(), "the type of k_out", out_shape);
    placed({{&k_cache, "k_cache"}, {&v_cache, "v_cache"}, {&slot_mapping, "slot_mapping"}, {&k_scale, "k_scale"},
            {&v_scale, "v_scale"}, {&k_out, "k_out"}, {&v_out, "v_out"}, {opt(status), "status"}});
    TORCH_CHECK(g_entries.gather_fp4, "entry point not set");
    return g_entries.gather_fp4(k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr<int64_t>(),
                                k_scale.data_ptr<float>(), v_scale.data_ptr<float>(), k_out.data_ptr(),
                                v_out.data_ptr(), bf ? PA_OUT_BF16 : PA_OUT_F32, g.n, g.hkv, g.dim, g.block_size,
                                g.pages, ptr_of<int32_t>(status), stream_of(stream));
}

// The int32 tensors of a block-table call.
void expect_tables(const Tensor &lens, const char *lens_name, const Tensor &count, const char *count_name,
                   const Tensor &block_table, const Tensor &free_pages, const Tensor &num_free, int64_t block_size,
                   const Tensor &lens_out, const char *out_name, const Tensor &num_free_out,
                   const optional<Tensor> &status) {
    TORCH_CHECK_VALUE(block_table.dim() == 2, "block_table: a [num_seqs, max_pages] tensor is required");
    TORCH_CHECK_VALUE(free_pages.dim() == 1, "free_pages: a one-dimensional tensor is required");
    TORCH_CHECK_VALUE(block_size >= 1 && block_size <= INT32_MAX, "block_size: ", block_size, " is out of range");
    const std::array<int64_t, 1> seqs{block_table.size(0)}, one{1};
    auto i32 = [](const Tensor &t) { return t.scalar_type() == at::kInt; };
    expect(block_table, "block_table", i32(block_table), "int32", {}, false);
    expect(lens, lens_name, i32(lens), "int32", seqs);
    expect(count, count_name, i32(count), "int32", seqs);
    expect(free_pages, "free_pages", i32(free_pages), "int32", {}, false);
    expect(num_free, "num_free", i32(num_free), "int32", one);
    expect(lens_out, out_name, i32(lens_out), "int32", seqs);
    expect(num_free_out, "num_free_out", i32(num_free_out), "int32", one);
    TORCH_CHECK_VALUE(block_table.size(0) <= INT32_MAX && block_table.size(1) <= INT32_MAX,
                      "block_table: too large");
    if (status.has_value())
        expect(*status, "status", status->scalar_type() == at::kInt && status->numel() >= 1, "int32 (one element)",
               {}, false);
}

int64_t extend_tables(const Tensor &context_lens, const Tensor &num_new, const Tensor &block_table,
                      const Tensor &free_pages, const Tensor &num_free, int64_t block_size, const Tensor &seq_lens,
                      const Tensor &slot_mapping, const Tensor &num_free_out, const optional<Tensor> &status,
                      int64_t stream) {
    expect_tables(context_lens, "context_lens", num_new, "num_new", block_table, free_pages, num_free, block_size,
                  seq_lens, "seq_lens", num_free_out, status);
    expect(slot_mapping, "slot_mapping", slot_mapping.scalar_type() == at::kLong && slot_mapping.dim() == 1,
           "int64, one-dimensional", {}, false);
    TORCH_CHECK_VALUE(slot_mapping.size(0) <= INT32_MAX, "slot_mapping: too many tokens");
    placed({{&context_lens, "context_lens"}, {&num_new, "num_new"}, {&block_table, "block_table"},
            {&free_pages, "free_pages"}, {&num_free, "num_free"}, {&seq_lens, "seq_lens"},
            {&slot_mapping, "slot_mapping"}, {&num_free_out, "num_free_out"}, {opt(status), "status"}});
    TORCH_CHECK(g_entries.extend_tables, "entry point not set");
    return g_entries.extend_tables(
        context_lens.data_ptr<int32_t>(), num_new.data_ptr<int32_t>(), block_table.data_ptr<int32_t>(),
        free_pages.data_ptr<int32_t>(), num_free.data_ptr<int32_t>(), static_cast<int32_t>(block_table.size(0)),
        static_cast<int32_t>(block_table.size(1)), static_cast<int32_t>(block_size), free_pages.size(0),
        static_cast<int32_t>(slot_mapping.size(0)), seq_lens.data_ptr<int32_t>(), slot_mapping.data_ptr<int64_t>(),
        num_free_out.data_ptr<int32_t>(), ptr_of<int32_t>(status), stream_of(stream));
}

int64_t release_tables(const Tensor &seq_lens, const Tensor &finished, const Tensor &block_table,
                       const Tensor &free_pages, const Tensor &num_free, int64_t block_size,
                       const Tensor &seq_lens_out, const Tensor &num_free_out, const optional<Tensor> &status,
                       int64_t stream) {
    expect_tables(seq_lens, "seq_lens", finished, "finished", block_table, free_pages, num_free, block_size,
                  seq_lens_out, "seq_lens_out", num_free_out, status);
    placed({{&seq_lens, "seq_lens"}, {&finished, "finished"}, {&block_table, "block_table"},
            {&free_pages, "free_pages"}, {&num_free, "num_free"}, {&seq_lens_out, "seq_lens_out"},
            {&num_free_out, "num_free_out"}, {opt(status), "status"}});
    TORCH_CHECK(g_entries.release_tables, "entry point not set");
    return g_entries.release_tables(
        seq_lens.data_ptr<int32_t>(), finished.data_ptr<int32_t>(), block_table.data_ptr<int32_t>(),
        free_pages.data_ptr<int32_t>(), num_free.data_ptr<int32_t>(), static_cast<int32_t>(block_table.size(0)),
        static_cast<int32_t>(block_table.size(1)), static_cast<int32_t>(block_size), free_pages.size(0),
        seq_lens_out.data_ptr<int32_t>(), num_free_out.data_ptr<int32_t>(), ptr_of<int32_t>(status),
        stream_of(stream));
}

// ---- pages with several holders -----------------------------------------------

void expect_i32(const Tensor &t, const char *name, int64_t n) {
    expect(t, name, t.scalar_type() == at::kInt, "int32", std::array<int64_t, 1>{n});
}

// The block table, pool and counts of a call; returns the number of pages.
int64_t expect_pool(const Tensor &block_table, const Tensor &free_pages, const Tensor &num_free,
                    const Tensor &share_counts, int64_t block_size, const Tensor &share_counts_out,
                    const Tensor &num_free_out, const optional<Tensor> &status) {
    TORCH_CHECK_VALUE(block_table.dim() == 2, "block_table: a [num_seqs, max_pages] tensor is required");
    TORCH_CHECK_VALUE(free_pages.dim() == 1, "free_pages: a one-dimensional tensor is required");
    TORCH_CHECK_VALUE(block_size >= 1 && block_size <= INT32_MAX, "block_size: ", block_size, " is out of range");
    TORCH_CHECK_VALUE(block_table.size(0) <= INT32_MAX && block_table.size(1) <= INT32_MAX, "block_table: too large");
    const int64_t pages = free_pages.size(0);
    expect(block_table, "block_table", block_table.scalar_type() == at::kInt, "int32", {}, false);
    expect_i32(free_pages, "free_pages", pages);
    expect_i32(num_free, "num_free", 1);
    expect_i32(share_counts, "share_counts", pages);
    expect_i32(share_counts_out, "share_counts_out", pages);
    expect_i32(num_free_out, "num_free_out", 1);
    if (status.has_value())
        expect(*status, "status", status->scalar_type() == at::kInt && status->numel() >= 1, "int32 (one element)",
               {}, false);
    return pages;
}

int64_t fork_tables(const Tensor &seq_lens, const Tensor &parent, const Tensor &block_table, const Tensor &free_pages,
                    const Tensor &num_free, const Tensor &share_counts, int64_t block_size, const Tensor &seq_lens_out,
                    const Tensor &share_counts_out, const Tensor &copy_src, const Tensor &copy_dst,
                    const Tensor &copy_tokens, const Tensor &num_free_out, const optional<Tensor> &status,
                    int64_t stream) {
    const int64_t pages = expect_pool(block_table, free_pages, num_free, share_counts, block_size, share_counts_out,
                                      num_free_out, status);
    const int64_t n = block_table.size(0);
    expect_i32(seq_lens, "seq_lens", n);
    expect_i32(parent, "parent", n);
    expect_i32(seq_lens_out, "seq_lens_out", n);
    expect_i32(copy_src, "copy_src", n);
    expect_i32(copy_dst, "copy_dst", n);
    expect_i32(copy_tokens, "copy_tokens", n);
    placed({{&seq_lens, "seq_lens"}, {&parent, "parent"}, {&block_table, "block_table"}, {&free_pages, "free_pages"},
            {&num_free, "num_free"}, {&share_counts, "share_counts"}, {&seq_lens_out, "seq_lens_out"},
            {&share_counts_out, "share_counts_out"}, {&copy_src, "copy_src"}, {&copy_dst, "copy_dst"},
            {&copy_tokens, "copy_tokens"}, {&num_free_out, "num_free_out"}, {opt(status), "status"}});
    TORCH_CHECK(g_entries.fork_tables, "entry point not set");
    return g_entries.fork_tables(
        seq_lens.data_ptr<int32_t>(), parent.data_ptr<int32_t>(), block_table.data_ptr<int32_t>(),
        free_pages.data_ptr<int32_t>(), num_free.data_ptr<int32_t>(), share_counts.data_ptr<int32_t>(),
        static_cast<int32_t>(n), static_cast<int32_t>(block_table.size(1)), static_cast<int32_t>(block_size), pages,
        seq_lens_out.data_ptr<int32_t>(), share_counts_out.data_ptr<int32_t>(), copy_src.data_ptr<int32_t>(),
        copy_dst.data_ptr<int32_t>(), copy_tokens.data_ptr<int32_t>(), num_free_out.data_ptr<int32_t>(),
        ptr_of<int32_t>(status), stream_of(stream));
}

int64_t release_shared(const Tensor &seq_lens, const Tensor &finished, const Tensor &block_table,
                       const Tensor &free_pages, const Tensor &num_free, const Tensor &share_counts, int64_t block_size,
                       const Tensor &seq_lens_out, const Tensor &share_counts_out, const Tensor &num_free_out,
                       const optional<Tensor> &status, int64_t stream) {
    const int64_t pages = expect_pool(block_table, free_pages, num_free, share_counts, block_size, share_counts_out,
                                      num_free_out, status);
    const int64_t n = block_table.size(0);
    expect_i32(seq_lens, "seq_lens", n);
    expect_i32(finished, "finished", n);
    expect_i32(seq_lens_out, "seq_lens_out", n);
    placed({{&seq_lens, "seq_lens"}, {&finished, "finished"}, {&block_table, "block_table"},
            {&free_pages, "free_pages"}, {&num_free, "num_free"}, {&share_counts, "share_counts"},
            {&seq_lens_out, "seq_lens_out"}, {&share_counts_out, "share_counts_out"}, {&num_free_out, "num_free_out"},
            {opt(status), "status"}});
    TORCH_CHECK(g_entries.release_shared, "entry point not set");
    return g_entries.release_shared(
        seq_lens.data_ptr<int32_t>(), finished.data_ptr<int32_t>(), block_table.data_ptr<int32_t>(),
        free_pages.data_ptr<int32_t>(), num_free.data_ptr<int32_t>(), share_counts.data_ptr<int32_t>(),
        static_cast<int32_t>(n), static_cast<int32_t>(block_table.size(1)), static_cast<int32_t>(block_size), pages,
        seq_lens_out.data_ptr<int32_t>(), share_counts_out.data_ptr<int32_t>(), num_free_out.data_ptr<int32_t>(),
        ptr_of<int32_t>(status), stream_of(stream));
}

int64_t compact_tables(const Tensor &seq_lens, const Tensor &block_table, const Tensor &free_pages,
                       const Tensor &num_free, const Tensor &share_counts, int64_t block_size,
                       const Tensor &free_pages_out, const Tensor &num_free_out, const Tensor &share_counts_out,
                       const Tensor &page_map, const Tensor &copy_src, const Tensor &copy_dst, const Tensor &extent,
                       const optional<Tensor> &status, int64_t stream) {
    const int64_t pages = expect_pool(block_table, free_pages, num_free, share_counts, block_size, share_counts_out,
                                      num_free_out, status);
    TORCH_CHECK_VALUE(copy_src.dim() == 1 && copy_src.size(0) <= INT32_MAX, "copy_src: a one-dimensional tensor is required");
    expect_i32(seq_lens, "seq_lens", block_table.size(0));
    expect_i32(free_pages_out, "free_pages_out", pages);
    expect_i32(page_map, "page_map", pages);
    expect_i32(copy_src, "copy_src", copy_src.size(0));
    expect_i32(copy_dst, "copy_dst", copy_src.size(0));
    expect_i32(extent, "extent", 1);
    placed({{&seq_lens, "seq_lens"}, {&block_table, "block_table"}, {&free_pages, "free_pages"},
            {&num_free, "num_free"}, {&share_counts, "share_counts"}, {&free_pages_out, "free_pages_out"},
            {&num_free_out, "num_free_out"}, {&share_counts_out, "share_counts_out"}, {&page_map, "page_map"},
            {&copy_src, "copy_src"}, {&copy_dst, "copy_dst"}, {&extent, "extent"}, {opt(status), "status"}});
    TORCH_CHECK(g_entries.compact_tables, "entry point not set");
    return g_entries.compact_tables(
        seq_lens.data_ptr<int32_t>(), block_table.data_ptr<int32_t>(), free_pages.data_ptr<int32_t>(),
        num_free.data_ptr<int32_t>(), share_counts.data_ptr<int32_t>(), static_cast<int32_t>(block_table.size(0)),
        static_cast<int32_t>(block_table.size(1)), static_cast<int32_t>(block_size), pages,
        static_cast<int32_t>(copy_src.size(0)), free_pages_out.data_ptr<int32_t>(), num_free_out.data_ptr<int32_t>(),
        share_counts_out.data_ptr<int32_t>(), page_map.data_ptr<int32_t>(), copy_src.data_ptr<int32_t>(),
        copy_dst.data_ptr<int32_t>(), extent.data_ptr<int32_t>(), ptr_of<int32_t>(status), stream_of(stream));
}

// Copies inside caches of one shape: [pages, block_size, kv_heads, head_dim]
// (bf16, e4m3) or fp4 records [pages, kv_heads, block_size / 16, 9 * head_dim].
int64_t copy_pages(bool fp4, const std::vector<Tensor> &caches, const Tensor &copy_src, const Tensor &copy_dst,
                   const optional<Tensor> &copy_tokens, const optional<Tensor> &status, int64_t stream) {
    TORCH_CHECK_VALUE(!caches.empty(), "caches: at least one cache is required");
    TORCH_CHECK_VALUE(caches.size() <= PA_MAX_COPY_CACHES, "caches: at most ", PA_MAX_COPY_CACHES, " in one call");
    const Tensor &c0 = caches[0];
    TORCH_CHECK_VALUE(c0.dim() == 4, "caches: 4-dimensional cache tensors are required");
    for (const Tensor &c : caches) {
        const bool ok = fp4 ? c.scalar_type() == at::kByte
                            : c.scalar_type() == at::kBFloat16 || is_fp8_cache_type(c.scalar_type());
        expect(c, "caches", ok && c.element_size() == c0.element_size(),
               fp4 ? "uint8 (fp4 records)" : "bfloat16, or uint8 or float8_e4m3fn, the same for all", c0.sizes());
    }
    TORCH_CHECK_VALUE(copy_src.dim() == 1 && copy_src.size(0) <= INT32_MAX, "copy_src: a one-dimensional tensor is required");
    const int64_t n = copy_src.size(0);
    expect_i32(copy_src, "copy_src", n);
    expect_i32(copy_dst, "copy_dst", n);
    if (copy_tokens.has_value()) expect_i32(*copy_tokens, "copy_tokens", n);
    if (status.has_value())
        expect(*status, "status", status->scalar_type() == at::kInt && status->numel() >= 1, "int32 (one element)",
               {}, false);
    for (int i = 0; i < 4; ++i)
        TORCH_CHECK_VALUE(c0.size(i) >= 1 && c0.size(i) <= INT32_MAX / 16, "caches: dimension ", i, " is out of range");
    for (const Tensor &c : caches) placed({{&c, "caches"}});
    placed({{&copy_src, "copy_src"}, {&copy_dst, "copy_dst"}, {opt(copy_tokens), "copy_tokens"}, {opt(status), "status"}});
    std::vector<void *> ptrs;
    for (const Tensor &c : caches) ptrs.push_back(c.data_ptr());
    const int64_t parts = fp4 ? c0.size(1) : 1, block_size = fp4 ? c0.size(2) * 16 : c0.size(1);
    const int64_t chunk = fp4 ? c0.size(3) : 16 * c0.size(2) * c0.size(3) * c0.element_size();
    TORCH_CHECK(g_entries.copy_pages, "entry point not set");
    return g_entries.copy_pages(ptrs.data(), static_cast<int32_t>(ptrs.size()), copy_src.data_ptr<int32_t>(),
                                copy_dst.data_ptr<int32_t>(), ptr_of<int32_t>(copy_tokens), static_cast<int32_t>(n),
                                static_cast<int32_t>(parts), chunk, static_cast<int32_t>(block_size), c0.size(0),
                                ptr_of<int32_t>(status), stream_of(stream));
}

// ---- rotary positions ---------------------------------------------------------

// Rows [n, heads, dim] of bf16 whose heads are dense; returns their stride in
// elements.  (Not required to be contiguous: q, k and v are often rows of one
// projection's output.)
int64_t expect_rows(const Tensor &t, const char *name, int64_t n, int64_t heads, int64_t dim) {
    expect(t, name, t.scalar_type() == at::kBFloat16, "bfloat16", std::array<int64_t, 3>{n, heads, dim});
    return n > 1 ? t.stride(0) : heads * dim;
}

void placed_rows(std::initializer_list<std::pair<const Tensor *, const char *>> ts) {
    int dev = -1;
    for (const auto &[t, name] : ts) {
        if (t == nullptr) continue;
        TORCH_CHECK_VALUE(t->is_cuda(), name, ": a CUDA tensor is required (got ", t->device(), ")");
        if (dev < 0) dev = c10::cuda::current_device();
        TORCH_CHECK_VALUE(t->get_device() == dev, name, ": on ", t->device(), ", but the current device is cuda:", dev);
        TORCH_CHECK_VALUE((t->size(2) <= 1 || t->stride(2) == 1) && (t->size(1) <= 1 || t->stride(1) == t->size(2)),
                          name, ": the heads of a row must be contiguous");
    }
}

pa_rotary_desc rotary_desc(const Tensor &q, const Tensor *k, const Tensor &positions, const Tensor &freqs,
                           const Tensor &q_out, int64_t flags, double factor, int64_t offset) {
    TORCH_CHECK_VALUE(q.dim() == 3, "q: a [tokens, heads, head_dim] tensor is required");
    TORCH_CHECK_VALUE(k == nullptr || k->dim() == 3, "k: a [tokens, heads, head_dim] tensor is required");
    TORCH_CHECK_VALUE(freqs.dim() == 1, "freqs: a one-dimensional tensor is required");
    TORCH_CHECK_VALUE(offset >= INT32_MIN && offset <= INT32_MAX, "position_offset: out of range");
    for (int i = 0; i < 3; ++i)
        TORCH_CHECK_VALUE(q.size(i) <= INT32_MAX && (k == nullptr || k->size(i) <= INT32_MAX), "q, k: too large");
    TORCH_CHECK_VALUE(freqs.size(0) <= INT32_MAX / 2, "freqs: too large");
    const int64_t n = q.size(0), dim = q.size(2);
    pa_rotary_desc d{};
    d.num_tokens = static_cast<int32_t>(n);
    d.num_q_heads = static_cast<int32_t>(q.size(1));
    d.num_kv_heads = k ? static_cast<int32_t>(k->size(1)) : 0;
    d.head_dim = static_cast<int32_t>(dim);
    d.rotary_dim = static_cast<int32_t>(2 * freqs.size(0));
    d.flags = static_cast<int32_t>(flags);
    d.position_offset = static_cast<int32_t>(offset);
    d.factor = static_cast<float>(factor);
    d.q_stride = expect_rows(q, "q", n, q.size(1), dim);
    if (k) d.k_stride = expect_rows(*k, "k", n, k->size(1), dim);
    d.q_out_stride = expect_rows(q_out, "q_out", n, q.size(1), dim);
    expect_i32(positions, "positions", n);
    expect(freqs, "freqs", freqs.scalar_type() == at::kLong, "int64", {}, false);
    return d;
}

int64_t rotary(const Tensor &q, const optional<Tensor> &k, const Tensor &positions, const Tensor &freqs,
               const Tensor &q_out, const optional<Tensor> &k_out, int64_t flags, double factor, int64_t offset,
               int64_t stream) {
    TORCH_CHECK_VALUE(k.has_value() == k_out.has_value(), "k, k_out: both or neither");
    pa_rotary_desc d = rotary_desc(q, opt(k), positions, freqs, q_out, flags, factor, offset);
    if (k_out.has_value()) d.k_out_stride = expect_rows(*k_out, "k_out", d.num_tokens, d.num_kv_heads, d.head_dim);
    placed_rows({{&q, "q"}, {opt(k), "k"}, {&q_out, "q_out"}, {opt(k_out), "k_out"}});
    placed({{&positions, "positions"}, {&freqs, "freqs"}});
    TORCH_CHECK(g_entries.rotary, "entry point not set");
    return g_entries.rotary(q.data_ptr(), ptr_of<void>(k), positions.data_ptr<int32_t>(), freqs.data_ptr<int64_t>(),
                            q_out.data_ptr(), ptr_of<void>(k_out), &d, stream_of(stream));
}

// kind: 0 bf16, 1 e4m3, 2 fp4
int64_t rotary_and_cache(int64_t kind, const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &positions,
                         const Tensor &freqs, const Tensor &q_out, const Tensor &k_cache, const Tensor &v_cache,
                         const Tensor &slot_mapping, const optional<Tensor> &k_scale, const optional<Tensor> &v_scale,
                         int64_t flags, double factor, int64_t offset, const optional<Tensor> &status, int64_t stream) {
    pa_rotary_desc d = rotary_desc(q, &k, positions, freqs, q_out, flags, factor, offset);
    d.v_stride = expect_rows(v, "v", d.num_tokens, d.num_kv_heads, d.head_dim);
    TORCH_CHECK_VALUE(k_cache.dim() == 4, "k_cache: a 4-dimensional cache tensor is required");
    const bool fp4 = kind == 2, quant = kind != 0;
    const int64_t block_size = fp4 ? k_cache.size(2) * 16 : k_cache.size(1);
    std::array<int64_t, 4> shape{k_cache.size(0), block_size, d.num_kv_heads, d.head_dim};
    if (fp4) shape = {k_cache.size(0), d.num_kv_heads, block_size / 16, 9 * int64_t(d.head_dim)};
    auto cache_ok = [&](const Tensor &t) {
        return fp4 ? t.scalar_type() == at::kByte
                   : quant ? is_fp8_cache_type(t.scalar_type()) : t.scalar_type() == at::kBFloat16;
    };
    const char *want = fp4 ? "uint8 (fp4 records)" : quant ? "uint8 or float8_e4m3fn (e4m3 codes)" : "bfloat16";
    expect(k_cache, "k_cache", cache_ok(k_cache), want, shape);
    expect(v_cache, "v_cache", cache_ok(v_cache), want, shape);
    TORCH_CHECK_VALUE(block_size <= INT32_MAX, "k_cache: block_size is too large");
    expect(slot_mapping, "slot_mapping", slot_mapping.scalar_type() == at::kLong, "int64",
           std::array<int64_t, 1>{d.num_tokens});
    const std::array<int64_t, 1> scale_shape{d.num_kv_heads};
    TORCH_CHECK_VALUE(!quant || (k_scale.has_value() && v_scale.has_value()), "k_scale, v_scale: ",
                      fp4 ? "an fp4" : "an e4m3", " cache needs both");
    if (k_scale.has_value()) expect(*k_scale, "k_scale", k_scale->scalar_type() == at::kFloat, "float32", scale_shape);
    if (v_scale.has_value()) expect(*v_scale, "v_scale", v_scale->scalar_type() == at::kFloat, "float32", scale_shape);
    if (status.has_value())
        expect(*status, "status", status->scalar_type() == at::kInt && status->numel() >= 1, "int32 (one element)",
               {}, false);
    placed_rows({{&q, "q"}, {&k, "k"}, {&v, "v"}, {&q_out, "q_out"}});
    placed({{&positions, "positions"}, {&freqs, "freqs"}, {&k_cache, "k_cache"}, {&v_cache, "v_cache"},
            {&slot_mapping, "slot_mapping"}, {opt(k_scale), "k_scale"}, {opt(v_scale), "v_scale"},
            {opt(status), "status"}});
    const int32_t bs = static_cast<int32_t>(block_size), *pos = positions.data_ptr<int32_t>();
    const int64_t *fr = freqs.data_ptr<int64_t>(), *slots = slot_mapping.data_ptr<int64_t>();
    void *kc = k_cache.data_ptr(), *vc = v_cache.data_ptr(), *s = stream_of(stream);
    if (!quant) {
        TORCH_CHECK(g_entries.rotary_and_cache, "entry point not set");
        return g_entries.rotary_and_cache(q.data_ptr(), k.data_ptr(), v.data_ptr(), pos, fr, q_out.data_ptr(), kc, vc,
                                          slots, &d, bs, k_cache.size(0), ptr_of<int32_t>(status), s);
    }
    const RotaryQuantFn fn = fp4 ? g_entries.rotary_and_cache_fp4 : g_entries.rotary_and_cache_fp8;
    TORCH_CHECK(fn, "entry point not set");
    return fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), pos, fr, q_out.data_ptr(), kc, vc, slots, ptr_of<float>(k_scale),
              ptr_of<float>(v_scale), &d, bs, k_cache.size(0), ptr_of<int32_t>(status), s);
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
    m.def("set_entry", &set_entry);
    m.def("attention", &attention, py::arg("kind"), py::arg("q"), py::arg("k_cache"), py::arg("v_cache"),
          py::arg("k_scale"), py::arg("v_scale"), py::arg("k_new"), py::arg("v_new"), py::arg("block_table"),
          py::arg("seq_lens"), py::arg("desc"), py::arg("out"), py::arg("workspace"), py::arg("status"),
          py::arg("stream"), py::arg("group_starts") = py::none(), py::arg("prefix_lens") = py::none(),
          py::arg("prefix") = 0);
    m.def("reshape", &reshape);
    m.def("reshape_fp4", &reshape_fp4);
    m.def("gather_fp4", &gather_fp4);
    m.def("extend_tables", &extend_tables);
    m.def("release_tables", &release_tables);
    m.def("fork_tables", &fork_tables);
    m.def("release_shared", &release_shared);
    m.def("compact_tables", &compact_tables);
    m.def("copy_pages", &copy_pages);
    m.def("rotary", &rotary);
    m.def("rotary_and_cache", &rotary_and_cache);
}
