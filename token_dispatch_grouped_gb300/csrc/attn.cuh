// attn.cuh — shared internals of the attention operators (include/moe_attention.h):
// head views, device helpers and the kernel launchers' signatures.
#pragma once
#include "../../include/moe_attention.h"
#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {
namespace attn {

using bf16 = __nv_bfloat16;

// A moe_heads on the device.
struct Heads {
    bf16* p;
    long long ts, hs;
    __device__ __forceinline__ bf16* row(long long t, int h) const { return p + t * ts + h * hs; }
};
inline Heads heads(const moe_heads& h) {
    return {static_cast<bf16*>(h.data), static_cast<long long>(h.token_stride),
            static_cast<long long>(h.head_stride)};
}

// The packed sequences of one call on the device.
struct Packed {
    int B, Tq, Tk, max_q, max_k, causal;
    const int32_t *cu_q, *cu_k;
};

// launch_k for kernels that are launched programmatically by default, as the grouped GEMMs.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled(true) ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Whether the attention kernels stop. A bad index concerns its row or sequence alone, and
// every kernel checks the indices that it uses, so the others go on with the rest of the call
// and with later calls; any other error may have left anything behind it.
__device__ __forceinline__ bool stopped(const int* err) {
    const int code = *reinterpret_cast<const volatile int*>(err);
    return code != MOE_OK && code != MOE_ERR_BAD_INDEX;
}
// A wait that ran out concerns the call, and is reported over a bad index.
__device__ __forceinline__ void raise_timeout(int* err) {
    if (atomicCAS(err, MOE_OK, MOE_ERR_TIMEOUT) == MOE_ERR_BAD_INDEX)
        atomicCAS(err, MOE_ERR_BAD_INDEX, MOE_ERR_TIMEOUT);
}

// Sequence b's rows [q0, q0 + nq) and [k0, k0 + nk). False (and MOE_ERR_BAD_INDEX)
// if its offsets do not ascend within the arrays or it is longer than stated.
__device__ __forceinline__ bool sequence_of(const Packed& s, int b, int& q0, int& nq, int& k0,
                                            int& nk, int* err) {
    q0 = s.cu_q[b];
    k0 = s.cu_k[b];
    const int q1 = s.cu_q[b + 1], k1 = s.cu_k[b + 1];
    nq = q1 - q0;
    nk = k1 - k0;
    const bool ok = q0 >= 0 && k0 >= 0 && q1 >= q0 && k1 >= k0 && q1 <= s.Tq && k1 <= s.Tk &&
                    nq <= s.max_q && nk <= s.max_k;
    if (!ok) raise_error(err, MOE_ERR_BAD_INDEX);
    return ok;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ void fma2v(float& d0, float& d1, float b, float c0, float c1) {  // d = d b + c
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 c, {%3, %4};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1) {  // d += a b
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 d, {%0, %1};\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "fma.rn.f32x2 d, a, b, d;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1) {  // d *= a
    asm("{\n\t.reg .b64 a, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 d, {%0, %1};\n\t"
        "mul.rn.f32x2 d, d, a;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {  // d += a
    asm("{\n\t.reg .b64 a, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 d, {%0, %1};\n\t"
        "add.rn.f32x2 d, d, a;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}

// ---------------------------------------------------------------- norm_rope.cu
struct NormRope {
    moe_attn_shape a;
    int T;
    Heads q, k, v, q_out, k_out;  // v and the cache: append only
    const float *wq, *wk;         // nullptr: no norm
    float eps;
    const int32_t* positions;
    const float2* table;
    int table_rows, rot, interleaved;
    const int64_t* slots;  // append only
    bf16 *k_pages, *v_pages;
    int pages, page_shift;
    int* err;
};
cudaError_t launch_rope_table(int positions, int half, const double* inv_freq, double scale,
                              float2* table, int* err, cudaStream_t st);
cudaError_t launch_norm_rope(const NormRope& p, bool append, cudaStream_t st);
// p.q, p.k: the inputs; dq_out, dk_out: upstream gradients; p.q_out, p.k_out: dq, dk.
int norm_rope_parts(const moe_attn_shape& a, int T);
cudaError_t launch_norm_rope_backward(const NormRope& p, Heads dq_out, Heads dk_out, float* part,
                                      float* dwq, float* dwk, cudaStream_t st);

// ---------------------------------------------------------------- attention.cu
struct Attention {
    moe_attn_shape a;
    Packed s;
    float scale;
    Heads q, k, v, out, dout, dq, dk, dv;
    float* lse;
    float* delta;  // backward scratch, 2 x [Hkv][Tq][G]
    int* err;
};
cudaError_t launch_attention_forward(const Attention& p, cudaStream_t st);
cudaError_t launch_attention_backward(const Attention& p, cudaStream_t st);

// ---------------------------------------------------------------- decode.cu
struct Decode {
    moe_attn_shape a;
    int B, n, max_kv;
    float scale;
    Heads q, out;
    const void *k_pages, *v_pages;      // bf16, or e4m3 with scales
    const float *k_scale, *v_scale;     // nullptr: bf16
    int pages, page_shift;
    const int32_t* block_table;
    int table_stride;
    const int32_t* kv_lens;
    float* weights;                     // nullptr: not kept
    int fresh;
    float* ws;
    int* err;
};
size_t decode_ws_floats(const moe_attn_shape& a, int B, int n, int max_kv, bool e8, bool weights);
cudaError_t launch_attention_decode(const Decode& p, cudaStream_t st);

// ---------------------------------------------------------------- cache8.cu
// p: the keys (and values) of a NormRope without q, slots and pages.
struct Append8 {
    NormRope r;
    int B, max_kv;
    const int32_t *cu, *lens, *block_table;
    int table_stride;
    uint8_t *k_pages, *v_pages;
    float *k_scale, *v_scale;
};
cudaError_t launch_append8(const Append8& p, cudaStream_t st);

// ---------------------------------------------------------------- evict.cu
struct Evict {
    int Hkv, D, B, max_kv, keep, recent;
    uint8_t *k_pages, *v_pages;    // rows of D values of 1 or 2 bytes
    float *k_scale, *v_scale;      // nullptr: bf16
    float* weights;
    int pages, page_shift;
    const int32_t *block_table, *lens, *new_table;
    int table_stride, new_stride;
    int32_t *new_lens, *kept;
    int* err;
};
cudaError_t launch_evict(const Evict& p, cudaStream_t st);

// ---------------------------------------------------------------- e4m3
// Two values rounded to e4m3 (the first in the low byte), NaN where they are not finite.
__device__ __forceinline__ float finite_or_nan(float x) {
    return fabsf(x) <= 3.402823466e+38f ? x : __int_as_float(0x7fffffff);
}
__device__ __forceinline__ uint32_t round_e4m3x2(float lo, float hi) {  // NaN stays; no infinities
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    return round_e4m3x2(finite_or_nan(lo), finite_or_nan(hi));
}
// Four e4m3 values as two pairs in fp16 (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}
// 16 e4m3 values times f <= 1, rounded to e4m3 again. By a power of two the product is formed in
// fp16: exact from 2^-11 up, and everything below rounds to zero either way.
__device__ __forceinline__ uint4 rescale_e4m3x16(const uint4& v, float f) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if ((__float_as_uint(f) & 0x7fffffu) == 0) {
        const __half2 f2 = __float2half2_rn(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[2];
            e4m3x4_to_f16(w[i], h[0], h[1]);
            uint16_t r[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&h[j]), f2);
                asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;"
                    : "=h"(r[j])
                    : "r"(*reinterpret_cast<const uint32_t*>(&y)));
            }
            w[i] = static_cast<uint32_t>(r[0]) | static_cast<uint32_t>(r[1]) << 16;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo, hi;
            e4m3x4_to_f16(w[i], lo, hi);
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            w[i] = round_e4m3x2(x.x * f, x.y * f) | round_e4m3x2(y.x * f, y.y * f) << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace attn
}  // namespace moe
