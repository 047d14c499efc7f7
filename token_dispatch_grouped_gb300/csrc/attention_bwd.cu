// attention_bwd.cu — the backward of softmax attention over packed sequences.
//
//   S = scale q k^T, lse = log sum_j exp S_j, P = exp(S - lse), out = P v;
//   dP = dout v^T, delta = sum_i dout_i out_i, dS = P (dP - delta),
//   dv = P^T dout, dq = scale dS k, dk = scale dS^T q.
//
// One warp per row (of q, or of k and v for their gradients): the lanes take 32 rows
// of the other side at a time for the dot products, then 4 of the D columns each for
// the weighted sums, in one pass with a running maximum and sum.
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxD = 128;

// The sequence of packed row t (offsets cu, `rows` of them at most), or false.
__device__ bool find(const int32_t* cu, int B, int t, int& b) {
    int lo = 0, hi = B;  // last b with cu[b] <= t
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (cu[m] <= t) lo = m;
        else hi = m;
    }
    b = lo;
    return t >= cu[lo] && t < cu[lo + 1];
}

// One warp of the grid looks all sequences over.
__device__ void check_sequences(const Packed& s, int lane, int* err) {
    int q0, nq, k0, nk;
    for (int b = lane; b < s.B; b += 32) sequence_of(s, b, q0, nq, k0, nk, err);
}

__device__ __forceinline__ float dot(const float* q, const bf16* row, int D) {
    float s = 0.f;
    for (int i = 0; i < D; i += 8) {
        float v[8];
        unpack8(*reinterpret_cast<const uint4*>(row + i), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += q[i + e] * v[e];
    }
    return s;
}

__device__ __forceinline__ void stage(float* dst, const bf16* row, int D, int lane) {
    __syncwarp();
    for (int i = lane; i < D; i += 32) dst[i] = __bfloat162float(row[i]);
    __syncwarp();
}

// delta and dq of one query row.
__global__ void __launch_bounds__(kWarps * 32) dq_kernel(const Attention p) {
    __shared__ float s_q[kWarps][kMaxD], s_do[kWarps][kMaxD];
    pdl_wait();
    pdl_trigger();
    if (has_error(p.err)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0 && warp == 0) check_sequences(p.s, lane, p.err);
    const int Hq = p.a.Hq, D = p.a.D;
    const long long row = static_cast<long long>(blockIdx.x) * kWarps + warp;
    if (row >= static_cast<long long>(p.s.Tq) * Hq) return;
    const int t = static_cast<int>(row / Hq), h = static_cast<int>(row % Hq);
    const int hk = h / (Hq / p.a.Hkv);
    int b, q0, nq, k0, nk;
    if (!find(p.s.cu_q, p.s.B, t, b) || !sequence_of(p.s, b, q0, nq, k0, nk, p.err)) return;
    stage(s_q[warp], p.q.row(t, h), D, lane);
    stage(s_do[warp], p.dout.row(t, h), D, lane);
    float delta = 0.f;
    for (int i = lane; i < D; i += 32) delta += s_do[warp][i] * __bfloat162float(p.out.row(t, h)[i]);
    for (int o = 16; o > 0; o >>= 1) delta += __shfl_xor_sync(~0u, delta, o);
    if (lane == 0) p.delta[row] = delta;
    const float lse = p.lse[row];
    const int seen = lse == -INFINITY ? 0 : p.s.causal ? min(nk, t - q0 + nk - nq + 1) : nk;
    float acc[kMaxD / 32] = {};
    for (int j0 = 0; j0 < seen; j0 += 32) {
        const int j = j0 + lane;
        float ds = 0.f;
        if (j < seen) {
            const float w = __expf(p.scale * dot(s_q[warp], p.k.row(k0 + j, hk), D) - lse);
            ds = w * (dot(s_do[warp], p.v.row(k0 + j, hk), D) - delta);
        }
        for (int i = 0; i < min(32, seen - j0); ++i) {
            const float di = __shfl_sync(~0u, ds, i);
            const bf16* k = p.k.row(k0 + j0 + i, hk);
            for (int c = 0; c < kMaxD / 32; ++c)
                if (c * 32 + lane < D) acc[c] += di * __bfloat162float(k[c * 32 + lane]);
        }
    }
    for (int c = 0; c < kMaxD / 32; ++c)
        if (c * 32 + lane < D) p.dq.row(t, h)[c * 32 + lane] = __float2bfloat16(p.scale * acc[c]);
}

// dk and dv of one key row, over the queries that see it in each head of its group.
__global__ void __launch_bounds__(kWarps * 32) dkv_kernel(const Attention p) {
    __shared__ float s_k[kWarps][kMaxD], s_v[kWarps][kMaxD];
    pdl_wait();
    pdl_trigger();
    if (has_error(p.err)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int Hq = p.a.Hq, Hkv = p.a.Hkv, D = p.a.D, G = Hq / Hkv;
    const long long row = static_cast<long long>(blockIdx.x) * kWarps + warp;
    if (row >= static_cast<long long>(p.s.Tk) * Hkv) return;
    const int t = static_cast<int>(row / Hkv), hk = static_cast<int>(row % Hkv);
    int b, q0, nq, k0, nk;
    if (!find(p.s.cu_k, p.s.B, t, b) || !sequence_of(p.s, b, q0, nq, k0, nk, p.err)) return;
    stage(s_k[warp], p.k.row(t, hk), D, lane);
    stage(s_v[warp], p.v.row(t, hk), D, lane);
    const int first = p.s.causal ? max(0, t - k0 + nq - nk) : 0;
    float ak[kMaxD / 32] = {}, av[kMaxD / 32] = {};
    for (int g = 0; g < G; ++g) {
        const int h = hk * G + g;
        for (int i0 = first; i0 < nq; i0 += 32) {
            const int i = q0 + i0 + lane;
            float w = 0.f, ds = 0.f;
            if (i0 + lane < nq) {
                const long long r = static_cast<long long>(i) * Hq + h;
                w = __expf(p.scale * dot(s_k[warp], p.q.row(i, h), D) - p.lse[r]);
                ds = w * (dot(s_v[warp], p.dout.row(i, h), D) - p.delta[r]);
            }
            for (int u = 0; u < min(32, nq - i0); ++u) {
                const float wu = __shfl_sync(~0u, w, u), du = __shfl_sync(~0u, ds, u);
                const bf16 *q = p.q.row(q0 + i0 + u, h), *dd = p.dout.row(q0 + i0 + u, h);
                for (int c = 0; c < kMaxD / 32; ++c)
                    if (c * 32 + lane < D) {
                        av[c] += wu * __bfloat162float(dd[c * 32 + lane]);
                        ak[c] += du * __bfloat162float(q[c * 32 + lane]);
                    }
            }
        }
    }
    for (int c = 0; c < kMaxD / 32; ++c)
        if (c * 32 + lane < D) {
            p.dk.row(t, hk)[c * 32 + lane] = __float2bfloat16(p.scale * ak[c]);
            p.dv.row(t, hk)[c * 32 + lane] = __float2bfloat16(av[c]);
        }
}

dim3 row_grid(long long rows) { return dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps)); }

}  // namespace

cudaError_t launch_attention_backward(const Attention& p, cudaStream_t st) {
    if (p.s.Tq > 0) {
        LaunchScope ls("attention_dq", st);
        const cudaError_t e = launch_k(dq_kernel, row_grid(static_cast<long long>(p.s.Tq) * p.a.Hq),
                                       dim3(kWarps * 32), 0, st, p);
        if (e != cudaSuccess) return e;
    }
    if (p.s.Tk == 0) return cudaSuccess;
    LaunchScope ls("attention_dkv", st);
    return launch_k(dkv_kernel, row_grid(static_cast<long long>(p.s.Tk) * p.a.Hkv),
                    dim3(kWarps * 32), 0, st, p);
}

}  // namespace attn
}  // namespace moe
