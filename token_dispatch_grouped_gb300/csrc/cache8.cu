// cache8.cu — new tokens' keys (normed and rotated) and values into a paged cache of e4m3
// values with one scale for each page and head.
//
// A CTA takes the rows that a page gets of one head's keys or values: x in fp32 to shared
// memory with their largest |x|, then p = the smallest power of two with |x| <= 448 p, the
// page's scale = max(scale, p) (p alone where the page begins), the rows already there moved
// to it if it grew, and the new ones as e4m3(x / scale). The scales are powers of two: e4m3 is a
// floating format, so they cost no precision, and rows that move are not rounded twice. The page
// is the CTA's, so no atomics and one launch. By its bytes (3 a value) 4096 tokens of 8 heads of
// 128 need 4 us; they take 19.4, the chain offsets -> lengths -> rows -> rotation of a page's
// CTA over two and a half waves of them (22.5 with one row's load in flight a lane). The queries
// are norm_rope's.
#include "norm_rope.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kAhead = 4;  // rows of a lane whose loads are in flight at once

// The page tasks of sequence b are numbered from here: the pages that n rows touch are no
// more than floor((r + n) / P) - floor(r / P) + 2 for any r.
__device__ __forceinline__ long long first_task(const int32_t* cu, int b, int shift) {
    return static_cast<long long>(cu[b] >> shift) + 2ll * b;
}

// The largest b < B with first_task(b) <= task: 32 candidates a step.
__device__ __forceinline__ int sequence_of_task(const Append8& p, long long task, int lane) {
    int lo = 0, hi = p.B;  // lo holds, hi does not
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool holds = at < hi && first_task(p.cu, at, p.r.page_shift) <= task;
        const unsigned votes = __ballot_sync(~0u, holds);
        const int k = votes == 0 ? 0 : 31 - __clz(votes);
        lo += k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Exponent of the smallest power of two p with a <= 448 p: 448 = 7/4 2^8.
__device__ __forceinline__ float scale_for(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
    return __uint_as_float(static_cast<uint32_t>(min(120, max(-100, e)) + 127) << 23);
}

template <int LPR, int SWAP>
__global__ void __launch_bounds__(kWarps * 32, 3) append8_kernel(const Append8 p) {
    constexpr int RPW = 32 / LPR;
    extern __shared__ __align__(16) float s_x[];  // [rows of the page][LPR * 8]
    __shared__ __align__(16) bf16 s_buf[SWAP == SWAP_ROW ? kWarps * RPW * 128 : 8];
    __shared__ float s_top[kWarps];
    pdl_wait();
    pdl_trigger();
    const NormRope& r = p.r;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int piece = lane % LPR, sub = lane / LPR;
    const int D = r.a.D, Hkv = r.a.Hkv, sh = r.page_shift;
    const bool value = blockIdx.y >= Hkv;
    const int hk = static_cast<int>(blockIdx.y) - (value ? Hkv : 0);
    // what needs no other load comes first
    const bool live = piece * 8 < D;
    const bool norm = !value && r.wq != nullptr;
    float w[8], wp[8];  // the norm weights of this lane's values and of their partners
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = wp[e] = 1.f;
    if (norm && live) {
        load_weights(r.wk, piece, w);
        if constexpr (SWAP == SWAP_OWN) {
#pragma unroll
            for (int e = 0; e < 8; ++e) wp[e] = w[e ^ 1];
        } else if constexpr (SWAP == SWAP_LANE) {
            const int hop = r.rot >> 4;
            load_weights(r.wk, piece < hop ? piece + hop : piece < 2 * hop ? piece - hop : piece, wp);
        } else if constexpr (SWAP == SWAP_ROW) {
#pragma unroll
            for (int e = 0; e < 8; ++e) wp[e] = __ldg(r.wk + partner_of(piece * 8 + e, r.rot, r.interleaved));
        }
    }
    if (__syncthreads_or(stopped(r.err))) return;
    if (blockIdx.x == 0 && blockIdx.y == 0)  // every sequence's offsets, whatever tasks they get
        for (int b = threadIdx.x; b < p.B; b += kWarps * 32) {
            const int q0 = p.cu[b], q1 = p.cu[b + 1], len = p.lens[b];
            if (q0 < 0 || q1 < q0 || q1 > r.T || len > p.max_kv || (q1 - q0) > len)
                raise_error(r.err, MOE_ERR_BAD_INDEX);
        }
    // the rows of this task (the same in every thread)
    const int b = sequence_of_task(p, blockIdx.x, lane);
    const int q0 = p.cu[b], q1 = p.cu[b + 1], len = p.lens[b];
    const int n = q1 - q0;
    if (q0 < 0 || q1 <= q0 || q1 > r.T || len > p.max_kv || n > len) return;
    const long long j = blockIdx.x - first_task(p.cu, b, sh);
    const int before = len - n;
    const long long pg = (before >> sh) + j;
    if (j < 0 || pg << sh >= len) return;
    const int lo = max(before, static_cast<int>(pg << sh));
    const int rows = min(len, static_cast<int>((pg + 1) << sh)) - lo;
    const int o = lo & ((1 << sh) - 1);
    const int row0 = q0 + lo - before;
    const int page = p.block_table[static_cast<long long>(b) * p.table_stride + pg];
    const Heads src = value ? r.v : r.k;
    uint4 in[kAhead];
    int pos[kAhead];
    const auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * kWarps * RPW + sub;
            in[u] = make_uint4(0u, 0u, 0u, 0u);
            if (i < rows && live) in[u] = *reinterpret_cast<const uint4*>(src.row(row0 + i, hk) + piece * 8);
            pos[u] = SWAP != SWAP_NONE && !value && i < rows ? r.positions[row0 + i] : 0;
        }
    };
    load(warp * RPW);
    if (page < 0 || page >= r.pages) {
        if (threadIdx.x == 0) raise_error(r.err, MOE_ERR_BAD_INDEX);
        return;
    }
    float* scale_at = (value ? p.v_scale : p.k_scale) + static_cast<long long>(page) * Hkv + hk;
    const float old = o > 0 ? *scale_at : 0.f;
    bf16* buf = s_buf + (SWAP == SWAP_ROW ? (warp * RPW + sub) * 128 : 0);
    float top = 0.f;
    const float inv_d = 1.f / static_cast<float>(D);
    for (int i0 = warp * RPW; i0 < rows; i0 += kAhead * kWarps * RPW) {
        if (i0 > warp * RPW) load(i0);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * kWarps * RPW + sub;
            if (i - sub >= rows) break;  // the whole warp
            float x[8];
            unpack8(in[u], x);
            if (!value) {
                float rr = 1.f;
                if (norm) {
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; e += 2) fma2(s0, s1, x[e], x[e + 1], x[e], x[e + 1]);
                    rr = rsqrtf(row_sum<LPR>(s0 + s1) * inv_d + r.eps);
                }
                float a[8], c[8], y[8];
                bool bad = false;
                if constexpr (SWAP != SWAP_NONE) {
                    bad = pos[u] < 0 || pos[u] >= r.table_rows;
                    if (bad && piece == 0) raise_error(r.err, MOE_ERR_BAD_INDEX);
                    load_rotation<SWAP>(r.table + static_cast<long long>(bad ? 0 : pos[u]) * (r.rot >> 1), r.rot,
                                        r.interleaved, piece, a, c);
                    float other[8];
                    partners<LPR, SWAP>(in[u], x, r.rot, r.interleaved, piece, buf, other);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = (x[e] * (w[e] * a[e]) + other[e] * (wp[e] * c[e])) * rr;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = x[e] * w[e] * rr;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = bad ? 0.f : y[e];  // a refused row has no say in the scale
            }
            if (i < rows && live) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (fabsf(x[e]) <= 3.402823466e+38f) top = fmaxf(top, fabsf(x[e]));
                float4* dst = reinterpret_cast<float4*>(s_x + i * (LPR * 8) + piece * 8);
                dst[0] = make_float4(x[0], x[1], x[2], x[3]);
                dst[1] = make_float4(x[4], x[5], x[6], x[7]);
            }
        }
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, k));
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kWarps; ++k) top = fmaxf(top, s_top[k]);
    const float scale = fmaxf(old, scale_for(top));
    uint8_t* dst = (value ? p.v_pages : p.k_pages) + (((static_cast<long long>(page) * Hkv + hk) << sh) * D);
    if (o > 0 && scale != old) {
        if (threadIdx.x == 0) *scale_at = scale;
        const float f = old / scale;
        for (int i = threadIdx.x; i < o * (D / 16); i += kWarps * 32) {
            uint4* at = reinterpret_cast<uint4*>(dst) + i;
            *at = rescale_e4m3x16(*at, f);
        }
    } else if (o == 0 && threadIdx.x == 0) {
        *scale_at = scale;
    }
    const float inv = 1.f / scale;  // a power of two, unless the page came with another scale
    for (int i = warp * RPW + sub; i < rows; i += kWarps * RPW) {
        if (!live) continue;
        const float4* from = reinterpret_cast<const float4*>(s_x + i * (LPR * 8) + piece * 8);
        const float4 x = from[0], y = from[1];
        uint2 v;
        v.x = to_e4m3x2(x.x * inv, x.y * inv) | to_e4m3x2(x.z * inv, x.w * inv) << 16;
        v.y = to_e4m3x2(y.x * inv, y.y * inv) | to_e4m3x2(y.z * inv, y.w * inv) << 16;
        *reinterpret_cast<uint2*>(dst + static_cast<long long>(o + i) * D + piece * 8) = v;
    }
}

template <int LPR, int SWAP>
cudaError_t append8(const Append8& p, cudaStream_t st) {
    const int smem = (LPR * 8 * 4) << p.r.page_shift;
    auto kfn = append8_kernel<LPR, SWAP>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    const long long tasks = (p.r.T >> p.r.page_shift) + 2ll * p.B;
    LaunchScope ls("kv8_append", st);
    return launch_pdl(kfn, dim3(static_cast<unsigned>(tasks), 2 * p.r.a.Hkv), dim3(kWarps * 32), smem, st, p);
}

}  // namespace

cudaError_t launch_append8(const Append8& p, cudaStream_t st) {
    const bool narrow = p.r.a.D <= 64;
    switch (swap_of(p.r)) {
        case SWAP_NONE: return narrow ? append8<8, SWAP_NONE>(p, st) : append8<16, SWAP_NONE>(p, st);
        case SWAP_OWN: return narrow ? append8<8, SWAP_OWN>(p, st) : append8<16, SWAP_OWN>(p, st);
        case SWAP_LANE: return narrow ? append8<8, SWAP_LANE>(p, st) : append8<16, SWAP_LANE>(p, st);
        default: return narrow ? append8<8, SWAP_ROW>(p, st) : append8<16, SWAP_ROW>(p, st);
    }
}

}  // namespace attn
}  // namespace moe
