// norm_rope.cuh — the pieces of a head row that the norm and rotation kernels share
// (norm_rope.cu, cache8.cu): how a row's lanes get the rotation, the partners of their values
// and the row's sum.
#pragma once
#include "attn.cuh"

namespace moe {
namespace attn {

enum Swap { SWAP_NONE = 0, SWAP_OWN = 1, SWAP_LANE = 2, SWAP_ROW = 3 };

inline Swap swap_of(const NormRope& p) {
    if (p.rot == 0) return SWAP_NONE;
    if (p.interleaved) return p.rot % 8 == 0 ? SWAP_OWN : SWAP_ROW;
    return p.rot % 16 == 0 ? SWAP_LANE : SWAP_ROW;
}

// The other value of i's pair.
__device__ __forceinline__ int partner_of(int i, int rot, int interleaved) {
    if (i >= rot) return i;
    if (interleaved) return i ^ 1;
    const int half = rot >> 1;
    return i < half ? i + half : i - half;
}

// cos and sin' of a lane's piece at one position (1 and 0 past the rotated dims).
template <int SWAP>
__device__ __forceinline__ void load_rotation(const float2* row, int rot, int interleaved, int piece,
                                              float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        c[e] = 1.f;
        s[e] = 0.f;
    }
    if constexpr (SWAP == SWAP_OWN) {
        if (piece * 8 < rot) {
            const float4* t = reinterpret_cast<const float4*>(row + piece * 4);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float4 v = __ldg(t + u);
                c[4 * u] = c[4 * u + 1] = v.x;
                s[4 * u] = -v.y;
                s[4 * u + 1] = v.y;
                c[4 * u + 2] = c[4 * u + 3] = v.z;
                s[4 * u + 2] = -v.w;
                s[4 * u + 3] = v.w;
            }
        }
    } else if constexpr (SWAP == SWAP_LANE) {
        const int hop = rot >> 4;  // pieces in half of the rotated dims
        if (piece < 2 * hop) {
            const bool lo = piece < hop;
            const float4* t = reinterpret_cast<const float4*>(row + (lo ? piece : piece - hop) * 8);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 v = __ldg(t + u);
                c[2 * u] = v.x;
                s[2 * u] = lo ? -v.y : v.y;
                c[2 * u + 1] = v.z;
                s[2 * u + 1] = lo ? -v.w : v.w;
            }
        }
    } else if constexpr (SWAP == SWAP_ROW) {
        const int half = rot >> 1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = piece * 8 + e;
            if (i >= rot) continue;
            const float2 v = __ldg(row + (interleaved ? i >> 1 : i < half ? i : i - half));
            const bool firstv = interleaved ? (i & 1) == 0 : i < half;
            c[e] = v.x;
            s[e] = firstv ? -v.y : v.y;
        }
    }
}

// The partners of a lane's 8 values (0 past the rotated dims, where they have no part).
// buf: this row's 128 bf16 of shared memory (SWAP_ROW). Every lane of the warp calls this.
template <int LPR, int SWAP>
__device__ __forceinline__ void partners(const uint4& in, const float (&x)[8], int rot,
                                         int interleaved, int piece, bf16* buf, float (&o)[8]) {
    if constexpr (SWAP == SWAP_OWN) {
        const bool on = piece * 8 < rot;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = on ? x[e ^ 1] : 0.f;
    } else if constexpr (SWAP == SWAP_LANE) {
        const int hop = rot >> 4;
        const bool on = piece < 2 * hop;
        const int from = !on ? piece : piece < hop ? piece + hop : piece - hop;
        uint4 v;
        v.x = __shfl_sync(0xffffffffu, in.x, from, LPR);
        v.y = __shfl_sync(0xffffffffu, in.y, from, LPR);
        v.z = __shfl_sync(0xffffffffu, in.z, from, LPR);
        v.w = __shfl_sync(0xffffffffu, in.w, from, LPR);
        if (!on) v = make_uint4(0u, 0u, 0u, 0u);
        unpack8(v, o);
    } else if constexpr (SWAP == SWAP_ROW) {
        __syncwarp();
        *reinterpret_cast<uint4*>(buf + piece * 8) = in;
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = piece * 8 + e;
            o[e] = i < rot ? __bfloat162float(buf[partner_of(i, rot, interleaved)]) : 0.f;
        }
    }
}

__device__ __forceinline__ void load_weights(const float* w, int piece, float (&v)[8]) {
    const float4* s = reinterpret_cast<const float4*>(w + piece * 8);
    const float4 x = __ldg(s), y = __ldg(s + 1);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace attn
}  // namespace moe
