// attn_api.cu — the C ABI of the attention operators (include/moe_attention.h):
// argument checks, workspace sizes and launches.
#include <algorithm>
#include <cmath>

#include "attn_mma.cuh"

namespace moe {
namespace attn {
bool make_tmap_heads(CUtensorMap* map, const Heads& h, int T, int H, int D, uint32_t box_heads,
                     uint32_t box_tokens) {
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                          static_cast<cuuint64_t>(T)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(h.hs) * 2, static_cast<cuuint64_t>(h.ts) * 2};
    cuuint32_t box[3] = {64, box_heads, box_tokens};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, h.p, dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace attn
}  // namespace moe

using namespace moe;
using namespace moe::attn;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int kMaxTokens = 1 << 24;
constexpr int kMaxCached = 1 << 30;  // of a sequence: token arithmetic stays within 32 bits

int check_attn(const moe_attn_shape& a) {
    if (a.Hq < 1 || a.Hkv < 1 || a.D < 1) return MOE_ERR_INVALID_ARG;
    if (a.Hq % a.Hkv != 0 || a.Hq / a.Hkv > 64 || a.Hq > 1024 || a.D % 8 != 0 || a.D > 128)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

int check_tokens(int32_t T) {
    return T < 0 ? MOE_ERR_INVALID_ARG : T > kMaxTokens ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}

// A view of [T, H, D]. The strides of an axis of one (or no) element are not used, and
// are replaced by ones that a tensor map accepts.
int check_heads(moe_heads* v, int T, int H, int D, bool output) {
    if (!v->data) return T == 0 ? MOE_OK : MOE_ERR_INVALID_ARG;
    if (!aligned16(v->data)) return MOE_ERR_MISALIGNED;
    if (H <= 1) v->head_stride = D;
    if (T <= 1) v->token_stride = static_cast<int64_t>(H > 1 ? (H - 1) * v->head_stride : 0) + D;
    const int64_t ts = v->token_stride, hs = v->head_stride, most = int64_t{1} << 38;
    if (ts < D || hs < D || ts > most || hs > most) return MOE_ERR_INVALID_ARG;
    if (ts % 8 != 0 || hs % 8 != 0) return MOE_ERR_MISALIGNED;
    if (output && T > 1 && H > 1 && ts < (H - 1) * hs + D && hs < (T - 1) * ts + D)
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

int check_rope(const moe_attn_shape& a, const moe_rope& r, const int32_t* positions) {
    if (r.dims == 0) return MOE_OK;
    if (r.dims < 0 || r.dims % 2 != 0 || r.dims > a.D || r.positions < 1 || !r.table ||
        !positions || (r.layout != MOE_ROPE_HALF && r.layout != MOE_ROPE_INTERLEAVED))
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(r.table) || !aligned4(positions)) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

int check_norm(const float* wq, const float* wk, float eps) {
    if ((wq == nullptr) != (wk == nullptr)) return MOE_ERR_INVALID_ARG;
    if (wq && !(eps >= 0.f && std::isfinite(eps))) return MOE_ERR_INVALID_ARG;
    if (!aligned16(wq) || !aligned16(wk)) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

int check_cache(const moe_attn_shape& a, const moe_kv_cache& c, int* shift) {
    if (!c.k || !c.v || c.pages < 1 || c.page_size < 1) return MOE_ERR_INVALID_ARG;
    if (!aligned16(c.k) || !aligned16(c.v)) return MOE_ERR_MISALIGNED;
    if (c.page_size < 8 || c.page_size > 256 || (c.page_size & (c.page_size - 1)) != 0 ||
        static_cast<int64_t>(c.pages) * a.Hkv * c.page_size >= (int64_t{1} << 31))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    int s = 0;
    while ((1 << s) < c.page_size) ++s;
    *shift = s;
    return MOE_OK;
}

int check_packed(const moe_packed& s) {
    if (s.B < 0 || s.max_q < 0 || s.max_k < 0 || (s.causal != 0 && s.causal != 1))
        return MOE_ERR_INVALID_ARG;
    for (int32_t T : {s.Tq, s.Tk})
        if (const int rc = check_tokens(T)) return rc;
    if (s.B > 65535) return MOE_ERR_UNSUPPORTED_SHAPE;
    if ((!s.cu_q || !s.cu_k) && s.B > 0) return MOE_ERR_INVALID_ARG;
    if (!aligned4(s.cu_q) || !aligned4(s.cu_k)) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

int check_scale(float scale) {
    return scale > 0.f && std::isfinite(scale) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

#define ATTN_TRY(expr)               \
    do {                             \
        if (const int _rc = (expr)) return _rc; \
    } while (0)

int launched(cudaError_t e) { return e == cudaSuccess ? MOE_OK : cuda_error_status(e); }

// No exception (the kernel timer's allocations) crosses the C boundary.
template <class F>
int guarded(F&& f) noexcept {
    try {
        return f();
    } catch (...) {
        return MOE_ERR_CUDA;
    }
}

NormRope norm_rope_of(const moe_attn_shape& a, int32_t T, const moe_heads& q, const moe_heads& k,
                      const float* wq, const float* wk, float eps, const int32_t* positions,
                      const moe_rope& r, int* err) {
    NormRope p{};
    p.a = a;
    p.T = T;
    p.q = heads(q);
    p.k = heads(k);
    p.wq = wq;
    p.wk = wk;
    p.eps = eps;
    p.positions = positions;
    p.table = reinterpret_cast<const float2*>(r.table);
    p.table_rows = r.positions;
    p.rot = r.dims;
    p.interleaved = r.layout == MOE_ROPE_INTERLEAVED;
    p.err = err;
    return p;
}

// No sequence is longer than its array, so a larger stated bound says no more than that.
Packed packed_of(const moe_packed& s) {
    return {s.B, s.Tq, s.Tk, std::min(s.max_q, s.Tq), std::min(s.max_k, s.Tk), s.causal, s.cu_q,
            s.cu_k};
}

}  // namespace

extern "C" {

int moe_rope_table(int32_t positions, int32_t dims, const double* inv_freq, double scale,
                   float* table, void* stream) {
    return guarded([&]() -> int {
        if (positions < 0 || dims < 0 || dims % 2 != 0 || !std::isfinite(scale))
            return MOE_ERR_INVALID_ARG;
        if (positions > kMaxTokens || dims > 128) return MOE_ERR_UNSUPPORTED_SHAPE;
        if (positions == 0 || dims == 0) return MOE_OK;
        if (!inv_freq || !table) return MOE_ERR_INVALID_ARG;
        if (!aligned16(inv_freq) || !aligned16(table)) return MOE_ERR_MISALIGNED;
        int* err = device_status_word();
        if (!err) return MOE_ERR_NO_DEVICE;
        return launched(launch_rope_table(positions, dims / 2, inv_freq, scale,
                                          reinterpret_cast<float2*>(table), err,
                                          static_cast<cudaStream_t>(stream)));
    });
}

int moe_norm_rope(moe_attn_shape a, int32_t T, moe_heads q, moe_heads k, const float* wq,
                  const float* wk, float eps, const int32_t* positions, moe_rope rope,
                  moe_heads q_out, moe_heads k_out, void* stream) {
    return guarded([&]() -> int {
        ATTN_TRY(check_attn(a));
        ATTN_TRY(check_tokens(T));
        if (T == 0) return MOE_OK;
        ATTN_TRY(check_rope(a, rope, positions));
        ATTN_TRY(check_norm(wq, wk, eps));
        ATTN_TRY(check_heads(&q, T, a.Hq, a.D, false));
        ATTN_TRY(check_heads(&q_out, T, a.Hq, a.D, true));
        if (k.data) {
            ATTN_TRY(check_heads(&k, T, a.Hkv, a.D, false));
            ATTN_TRY(check_heads(&k_out, T, a.Hkv, a.D, true));
        }
        int* err = device_status_word();
        if (!err) return MOE_ERR_NO_DEVICE;
        NormRope p = norm_rope_of(a, T, q, k, wq, wk, eps, positions, rope, err);
        p.q_out = heads(q_out);
        p.k_out = heads(k_out);
        return launched(launch_norm_rope(p, false, static_cast<cudaStream_t>(stream)));
    });
}

size_t moe_norm_rope_workspace_size(moe_attn_shape a, int32_t T) {
    if (check_attn(a) || check_tokens(T)) return 0;
    return sizeof(float) * 2 * a.D * static_cast<size_t>(norm_rope_parts(a, T));
}

int moe_norm_rope_backward(moe_attn_shape a, int32_t T, moe_heads dq_out, moe_heads dk_out,
                           moe_heads q, moe_heads k, const float* wq, const float* wk, float eps,
                           const int32_t* positions, moe_rope rope, moe_heads dq, moe_heads dk,
                           float* dwq, float* dwk, void* ws, size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        ATTN_TRY(check_attn(a));
        ATTN_TRY(check_tokens(T));
        if (T > 0) ATTN_TRY(check_rope(a, rope, positions));
        ATTN_TRY(check_norm(wq, wk, eps));
        const bool with_k = k.data != nullptr;
        if (T > 0) {
            ATTN_TRY(check_heads(&dq_out, T, a.Hq, a.D, false));
            ATTN_TRY(check_heads(&q, T, a.Hq, a.D, false));
            ATTN_TRY(check_heads(&dq, T, a.Hq, a.D, true));
            if (with_k) {
                ATTN_TRY(check_heads(&dk_out, T, a.Hkv, a.D, false));
                ATTN_TRY(check_heads(&k, T, a.Hkv, a.D, false));
                ATTN_TRY(check_heads(&dk, T, a.Hkv, a.D, true));
            }
        }
        if (wq) {
            if (!dwq || (!dwk && with_k) || !ws) return MOE_ERR_INVALID_ARG;
            if (!aligned16(ws) || !aligned4(dwq) || !aligned4(dwk)) return MOE_ERR_MISALIGNED;
            if (ws_bytes < moe_norm_rope_workspace_size(a, T)) return MOE_ERR_WORKSPACE_TOO_SMALL;
        } else if (T == 0) {
            return MOE_OK;
        }
        int* err = device_status_word();
        if (!err) return MOE_ERR_NO_DEVICE;
        if (T == 0) {
            // no launch reads the heads: the weight gradients are empty sums
            q.data = k.data = nullptr;
        }
        NormRope p = norm_rope_of(a, T, q, k, wq, wk, eps, positions, rope, err);
        p.q_out = heads(dq);
        p.k_out = heads(dk);
        return launched(launch_norm_rope_backward(p, heads(dq_out), heads(dk_out),
                                                  static_cast<float*>(ws), dwq, dwk,
                                                  static_cast<cudaStream_t>(stream)));
    });
}

int moe_kv_append(moe_attn_shape a, int32_t T, moe_heads q, moe_heads k, moe_heads v,
                  const float* wq, const float* wk, float eps, const int32_t* positions,
                  moe_rope rope, const int64_t* slots, moe_heads q_out, moe_kv_cache cache,
                  void* stream) {
    return guarded([&]() -> int {
        ATTN_TRY(check_attn(a));
        ATTN_TRY(check_tokens(T));
        int shift = 0;
        ATTN_TRY(check_cache(a, cache, &shift));
        if (T == 0) return MOE_OK;
        ATTN_TRY(check_rope(a, rope, positions));
        ATTN_TRY(check_norm(wq, wk, eps));
        ATTN_TRY(check_heads(&q, T, a.Hq, a.D, false));
        ATTN_TRY(check_heads(&k, T, a.Hkv, a.D, false));
        ATTN_TRY(check_heads(&v, T, a.Hkv, a.D, false));
        ATTN_TRY(check_heads(&q_out, T, a.Hq, a.D, true));
        if (!slots) return MOE_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(slots) & 7u) return MOE_ERR_MISALIGNED;
        int* err = device_status_word();
        if (!err) return MOE_ERR_NO_DEVICE;
        NormRope p = norm_rope_of(a, T, q, k, wq, wk, eps, positions, rope, err);
        p.v = heads(v);
        p.q_out = heads(q_out);
        p.slots = slots;
        p.k_pages = static_cast<bf16*>(cache.k);
        p.v_pages = static_cast<bf16*>(cache.v);
        p.pages = cache.pages;
        p.page_shift = shift;
        return launched(launch_norm_rope(p, true, static_cast<cudaStream_t>(stream)));
    });
}

int moe_attention_forward(moe_attn_shape a, moe_packed s, float scale, moe_heads q, moe_heads k,
                          moe_heads v, moe_heads out, float* lse, void* stream) {
    return guarded([&]() -> int {
        ATTN_TRY(check_attn(a));
        ATTN_TRY(check_packed(s));
        ATTN_TRY(check_scale(scale));
        if (s.Tq == 0 || s.B == 0) return MOE_OK;
        ATTN_TRY(check_heads(&q, s.Tq, a.Hq, a.D, false));
        ATTN_TRY(check_heads(&k, s.Tk, a.Hkv, a.D, false));
        ATTN_TRY(check_heads(&v, s.Tk, a.Hkv, a.D, false));
        ATTN_TRY(check_heads(&out, s.Tq, a.Hq, a.D, true));
        if (!lse) return MOE_ERR_INVALID_ARG;
        if (!aligned16(lse)) return MOE_ERR_MISALIGNED;
        int* err = device_status_word();
        if (!err) return MOE_ERR_NO_DEVICE;
        Attention p{};
        p.a = a;
        p.s = packed_of(s);
        p.scale = scale;
        p.q = heads(q);
        p.k = heads(k);
        p.v = heads(v);
        p.out = heads(out);
        p.lse = lse;
        p.err = err;
        return launched(launch_attention_forward(p, static_cast<cudaStream_t>(stream)));
    });
}

size_t moe_attention_backward_workspace_size(moe_attn_shape a, moe_packed s) {
    if (check_attn(a) || check_tokens(s.Tq)) return 0;
    return 2 * sizeof(float) * static_cast<size_t>(s.Tq) * a.Hq;
}

int moe_attention_backward(moe_attn_shape a, moe_packed s, float scale, moe_heads dout,
                           moe_heads q, moe_heads k, moe_heads v, moe_heads out,
                           const float* lse, moe_heads dq, moe_heads dk, moe_heads dv, void* ws,
                           size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        ATTN_TRY(check_attn(a));
        ATTN_TRY(check_packed(s));
        ATTN_TRY(check_scale(scale));
        if (s.B == 0 || (s.Tq == 0 && s.Tk == 0)) return MOE_OK;
        ATTN_TRY(check_heads(&dout, s.Tq, a.Hq, a.D, false));
        ATTN_TRY(check_heads(&q, s.Tq, a.Hq, a.D, false));
        ATTN_TRY(check_heads(&k, s.Tk, a.Hkv, a.D, false));
        ATTN_TRY(check_heads(&v, s.Tk, a.Hkv, a.D, false));
        ATTN_TRY(check_heads(&out, s.Tq, a.Hq, a.D, false));
        ATTN_TRY(check_heads(&dq, s.Tq, a.Hq, a.D, true));
        ATTN_TRY(check_heads(&dk, s.Tk, a.Hkv, a.D, true));
        ATTN_TRY(check_heads(&dv, s.Tk, a.Hkv, a.D, true));
        if (s.Tq > 0 && (!lse || !ws)) return MOE_ERR_INVALID_ARG;
        if (!aligned16(lse) || !aligned16(ws)) return MOE_ERR_MISALIGNED;
        if (ws_bytes < moe_attention_backward_workspace_size(a, s))
            return MOE_ERR_WORKSPACE_TOO_SMALL;
        int* err = device_status_word();
        if (!err) return MOE_ERR_NO_DEVICE;
        Attention p{};
        p.a = a;
        p.s = packed_of(s);
        p.scale = scale;
        p.q = heads(q);
        p.k = heads(k);
        p.v = heads(v);
        p.out = heads(out);
        p.dout = heads(dout);
        p.dq = heads(dq);
        p.dk = heads(dk);
        p.dv = heads(dv);
        p.lse = const_cast<float*>(lse);
        p.delta = static_cast<float*>(ws);
        p.err = err;
        return launched(launch_attention_backward(p, static_cast<cudaStream_t>(stream)));
    });
}

size_t moe_attention_decode_workspace_size(moe_attn_shape a, int32_t B, int32_t n,
                                           int32_t max_kv) {
    if (check_attn(a) || B < 1 || n < 1 || max_kv < 1 || max_kv > kMaxCached ||
        static_cast<int64_t>(B) * n > kMaxTokens)
        return 0;
    return sizeof(float) * decode_ws_floats(a, B, n, max_kv);
}

int moe_attention_decode(moe_attn_shape a, int32_t B, int32_t n, int32_t max_kv, float scale,
                         moe_heads q, moe_kv_cache cache, const int32_t* block_table,
                         int32_t table_stride, const int32_t* kv_lens, moe_heads out, void* ws,
                         size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        ATTN_TRY(check_attn(a));
        int shift = 0;
        ATTN_TRY(check_cache(a, cache, &shift));
        ATTN_TRY(check_scale(scale));
        if (B < 0 || n < 1 || max_kv < 0) return MOE_ERR_INVALID_ARG;
        if (static_cast<int64_t>(B) * n > kMaxTokens || max_kv > kMaxCached)
            return MOE_ERR_UNSUPPORTED_SHAPE;
        if (B == 0) return MOE_OK;
        const int32_t T = B * n;
        ATTN_TRY(check_heads(&q, T, a.Hq, a.D, false));
        ATTN_TRY(check_heads(&out, T, a.Hq, a.D, true));
        if (!block_table || !kv_lens) return MOE_ERR_INVALID_ARG;
        if (!aligned4(block_table) || !aligned4(kv_lens)) return MOE_ERR_MISALIGNED;
        if (table_stride < 0 ||
            (static_cast<int64_t>(max_kv) + cache.page_size - 1) / cache.page_size > table_stride)
            return MOE_ERR_INVALID_ARG;
        const size_t need = moe_attention_decode_workspace_size(a, B, n, max_kv);
        if (need > 0 && !ws) return MOE_ERR_INVALID_ARG;
        if (!aligned16(ws)) return MOE_ERR_MISALIGNED;
        if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
        int* err = device_status_word();
        if (!err) return MOE_ERR_NO_DEVICE;
        Decode p{};
        p.a = a;
        p.B = B;
        p.n = n;
        p.max_kv = max_kv;
        p.scale = scale;
        p.q = heads(q);
        p.out = heads(out);
        p.k_pages = static_cast<const bf16*>(cache.k);
        p.v_pages = static_cast<const bf16*>(cache.v);
        p.pages = cache.pages;
        p.page_shift = shift;
        p.block_table = block_table;
        p.table_stride = table_stride;
        p.kv_lens = kv_lens;
        p.part = static_cast<float*>(ws);
        p.err = err;
        return launched(launch_attention_decode(p, static_cast<cudaStream_t>(stream)));
    });
}

}  // extern "C"
