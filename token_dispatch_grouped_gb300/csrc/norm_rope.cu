// norm_rope.cu — RMS norm of every query and key head with the rotary positions in
// the same pass, its backward, and the form that appends to a paged cache.
//
// Forward, per head row x of D values at position p:
//   r = (mean(x^2) + eps)^(-1/2),   y = x r w,
//   out_i = y_i cos_i + y_{partner(i)} sin'_i,
// where partner(i) is the other value of i's rotated pair and sin' is -sin for the
// pair's first value and +sin for its second; values past the rotated dims stay y.
// Backward: dy is the upstream gradient rotated by -p, and with n = x r:
//   dx = r (dy w - n mean(dy w n)),   dw = sum over rows of dy n.
//
// Both directions are bound by memory (2 or 3 x 2 bytes a value, a few flops each).
// A head row is read as 16-byte pieces of 8 values, so D / 8 lanes (8 or 16 with
// padding) hold one row and a warp holds 2 to 4 rows at once. A lane keeps the same
// piece of every head of a token, so it reads its (cos, sin) once per token and keeps
// them in registers over the token's heads. Pairs of the half layout lie in another
// lane's registers: a shuffle fetches them when dims / 2 is a multiple of 8 (whole
// pieces swap), else the row passes through shared memory.
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 8;

// Where a lane's rotated partners are: none (no rotation), in its own registers
// (interleaved), in another lane (half layout, whole pieces) or anywhere in the row.
enum Swap { SWAP_NONE = 0, SWAP_OWN = 1, SWAP_LANE = 2, SWAP_ROW = 3 };

Swap swap_of(const NormRope& p) {
    if (p.rot == 0) return SWAP_NONE;
    if (p.interleaved) return SWAP_OWN;
    return (p.rot / 2) % 8 == 0 ? SWAP_LANE : SWAP_ROW;
}

// A lane's rotation factors of one token.
template <int SWAP>
struct Rotation {
    float c[8], s[8];
    // piece: first value / 8; dir: +1 rotates by the position, -1 back.
    __device__ __forceinline__ void load(const float2* row, int rot, int piece, float dir) {
        if constexpr (SWAP == SWAP_NONE) return;
        const int half = rot >> 1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = piece * 8 + e;
            int at;
            float sign;
            if constexpr (SWAP == SWAP_OWN) {
                at = i >> 1;
                sign = (e & 1) ? dir : -dir;
            } else {
                at = i < half ? i : i - half;
                sign = i < half ? -dir : dir;
            }
            const float2 cs = i < rot ? __ldg(row + at) : make_float2(1.f, 0.f);
            c[e] = cs.x;
            s[e] = sign * cs.y;
        }
    }
    // buf: this row's 128 floats of shared memory (SWAP_ROW); every lane of the warp
    // calls this.
    template <int LPR>
    __device__ __forceinline__ void apply(float (&y)[8], int rot, int piece, float* buf) const {
        if constexpr (SWAP == SWAP_NONE) return;
        float o[8];
        if constexpr (SWAP == SWAP_OWN) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = y[e ^ 1];
        } else if constexpr (SWAP == SWAP_LANE) {
            const int hop = rot >> 4;  // pieces in half of the rotated dims
            const int from = piece < hop ? piece + hop : piece < 2 * hop ? piece - hop : piece;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(0xffffffffu, y[e], from, LPR);
        } else {
            const int half = rot >> 1;
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) buf[piece * 8 + e] = y[e];
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = piece * 8 + e;
                o[e] = buf[i < half ? i + half : i < rot ? i - half : i];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (piece * 8 + e < rot) y[e] = y[e] * c[e] + o[e] * s[e];
    }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One warp per (token, run of its rows): rows 0 .. Hq are queries, then Hkv keys, then
// (append) Hkv values, which are only copied.
template <int LPR, int SWAP, bool APPEND>
__global__ void __launch_bounds__(kWarps * 32)
norm_rope_kernel(const NormRope p, int runs, int run_rows) {
    constexpr int RPW = 32 / LPR;  // rows of a warp at once
    constexpr int U = 4;           // loads in flight per lane
    __shared__ float s_buf[SWAP == SWAP_ROW ? kWarps * RPW * 128 : 1];
    pdl_wait();
    pdl_trigger();
    if (has_error(p.err)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long task = static_cast<long long>(blockIdx.x) * kWarps + warp;
    const int t = static_cast<int>(task / runs);
    if (t >= p.T) return;
    const int piece = lane % LPR, sub = lane / LPR;
    const int D = p.a.D, Hq = p.a.Hq, Hkv = p.a.Hkv;
    const int rows = Hq + (p.k.p ? Hkv : 0) + (APPEND ? Hkv : 0);
    const int r0 = static_cast<int>(task % runs) * run_rows, r1 = min(rows, r0 + run_rows);
    const bool live = piece * 8 < D;

    long long cache_row = -1;  // (page * Hkv) * page_size + row of the page, head 0
    if constexpr (APPEND) {
        const long long slot = p.slots[t];
        if (slot >= (static_cast<long long>(p.pages) << p.page_shift)) {
            if (lane == 0) raise_error(p.err, MOE_ERR_BAD_INDEX);
        } else if (slot >= 0) {
            const long long page = slot >> p.page_shift;
            cache_row = ((page * Hkv) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
        }
    }
    Rotation<SWAP> rot;
    bool bad = false;
    if constexpr (SWAP != SWAP_NONE) {
        const int pos = p.positions[t];
        bad = pos < 0 || pos >= p.table_rows;
        if (bad) {
            if (lane == 0) raise_error(p.err, MOE_ERR_BAD_INDEX);
        } else {
            rot.load(p.table + static_cast<long long>(pos) * (p.rot >> 1), p.rot, piece, 1.f);
        }
    }
    if (bad) return;  // the whole warp: one token
    const bool norm = p.wq != nullptr;
    float* buf = s_buf + (SWAP == SWAP_ROW ? (warp * RPW + sub) * 128 : 0);

    for (int rb = r0; rb < r1; rb += RPW * U) {
        uint4 in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = rb + u * RPW + sub;
            in[u] = make_uint4(0, 0, 0, 0);
            if (r < r1 && live) {
                const bf16* src = r < Hq ? p.q.row(t, r)
                                  : !APPEND || r < Hq + Hkv ? p.k.row(t, r - Hq)
                                                            : p.v.row(t, r - Hq - Hkv);
                in[u] = *reinterpret_cast<const uint4*>(src + piece * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (rb + u * RPW >= r1) break;  // the same for the whole warp
            const int r = rb + u * RPW + sub;
            float y[8];
            unpack8(in[u], y);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += y[e] * y[e];
            ss = row_sum<LPR>(ss);
            if (norm && live) {
                const float rr = rsqrtf(ss / static_cast<float>(D) + p.eps);
                const float4* w = reinterpret_cast<const float4*>((r < Hq ? p.wq : p.wk) + piece * 8);
                const float4 w0 = __ldg(w), w1 = __ldg(w + 1);
                const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = y[e] * rr * wv[e];
            }
            rot.template apply<LPR>(y, p.rot, piece, buf);
            if (r >= r1 || !live) continue;
            if (r < Hq) {
                *reinterpret_cast<uint4*>(p.q_out.row(t, r) + piece * 8) = pack8(y);
            } else if constexpr (APPEND) {
                if (cache_row < 0) continue;
                const bool key = r < Hq + Hkv;
                const int h = r - Hq - (key ? 0 : Hkv);
                const long long at = (cache_row + (static_cast<long long>(h) << p.page_shift)) * D;
                *reinterpret_cast<uint4*>((key ? p.k_pages : p.v_pages) + at + piece * 8) =
                    key ? pack8(y) : in[u];
            } else {
                *reinterpret_cast<uint4*>(p.k_out.row(t, r - Hq) + piece * 8) = pack8(y);
            }
        }
    }
}

// Backward: warps walk the (token, run) tasks with the grid's stride and keep their
// piece of the two weight gradients in registers; a CTA adds its warps' sums in warp
// order and writes one partial row [2][D].
template <int LPR, int SWAP>
__global__ void __launch_bounds__(kWarps * 32)
norm_rope_backward_kernel(const NormRope p, Heads dq_out, Heads dk_out, float* part, int runs,
                          int run_rows) {
    constexpr int RPW = 32 / LPR;
    constexpr int U = 2;  // two rows' x and dout in flight per lane
    __shared__ float s_buf[SWAP == SWAP_ROW ? kWarps * RPW * 128 : 1];
    __shared__ float s_dw[kWarps][2][128];
    pdl_wait();
    pdl_trigger();
    if (has_error(p.err)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int piece = lane % LPR, sub = lane / LPR;
    const int D = p.a.D, Hq = p.a.Hq;
    const int rows = Hq + (p.k.p ? p.a.Hkv : 0);
    const bool live = piece * 8 < D;
    const bool norm = p.wq != nullptr;
    float* buf = s_buf + (SWAP == SWAP_ROW ? (warp * RPW + sub) * 128 : 0);
    float aq[8], ak[8], wq[8], wk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        aq[e] = ak[e] = 0.f;
        wq[e] = norm && live ? p.wq[piece * 8 + e] : 1.f;
        wk[e] = norm && live ? p.wk[piece * 8 + e] : 1.f;
    }
    const long long tasks = static_cast<long long>(p.T) * runs;
    const long long step = static_cast<long long>(gridDim.x) * kWarps;
    for (long long task = static_cast<long long>(blockIdx.x) * kWarps + warp; task < tasks;
         task += step) {
        const int t = static_cast<int>(task / runs);
        const int r0 = static_cast<int>(task % runs) * run_rows, r1 = min(rows, r0 + run_rows);
        Rotation<SWAP> rot;
        if constexpr (SWAP != SWAP_NONE) {
            const int pos = p.positions[t];
            if (pos < 0 || pos >= p.table_rows) {
                if (lane == 0) raise_error(p.err, MOE_ERR_BAD_INDEX);
                continue;
            }
            rot.load(p.table + static_cast<long long>(pos) * (p.rot >> 1), p.rot, piece, -1.f);
        }
        for (int rb = r0; rb < r1; rb += RPW * U) {
            uint4 xin[U], gin[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = rb + u * RPW + sub;
                xin[u] = gin[u] = make_uint4(0, 0, 0, 0);
                if (r < r1 && live) {
                    const bf16* x = r < Hq ? p.q.row(t, r) : p.k.row(t, r - Hq);
                    const bf16* g = r < Hq ? dq_out.row(t, r) : dk_out.row(t, r - Hq);
                    xin[u] = *reinterpret_cast<const uint4*>(x + piece * 8);
                    gin[u] = *reinterpret_cast<const uint4*>(g + piece * 8);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (rb + u * RPW >= r1) break;  // the same for the whole warp
                const int r = rb + u * RPW + sub;
                const bool isq = r < Hq;
                float x[8], dy[8];
                unpack8(xin[u], x);
                unpack8(gin[u], dy);
                rot.template apply<LPR>(dy, p.rot, piece, buf);
                if (norm) {
                    float ss = 0.f, sd = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        ss += x[e] * x[e];
                        sd += dy[e] * (isq ? wq[e] : wk[e]) * x[e];
                    }
                    ss = row_sum<LPR>(ss);
                    sd = row_sum<LPR>(sd);
                    const float rr = rsqrtf(ss / static_cast<float>(D) + p.eps);
                    const float m = sd * rr / static_cast<float>(D);  // mean(dy w n)
                    const bool mine = r < r1 && live;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float n = x[e] * rr;
                        if (mine && isq) aq[e] += dy[e] * n;
                        if (mine && !isq) ak[e] += dy[e] * n;
                        dy[e] = rr * (dy[e] * (isq ? wq[e] : wk[e]) - n * m);
                    }
                }
                if (r < r1 && live)
                    *reinterpret_cast<uint4*>((isq ? p.q_out.row(t, r) : p.k_out.row(t, r - Hq)) +
                                              piece * 8) = pack8(dy);
            }
        }
    }
    if (!norm) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) {
            aq[e] += __shfl_xor_sync(0xffffffffu, aq[e], o);
            ak[e] += __shfl_xor_sync(0xffffffffu, ak[e], o);
        }
        if (sub == 0 && live) {
            s_dw[warp][0][piece * 8 + e] = aq[e];
            s_dw[warp][1][piece * 8 + e] = ak[e];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
        const int which = i / D, col = i % D;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += s_dw[w][which][col];
        part[static_cast<long long>(blockIdx.x) * 2 * D + i] = s;
    }
}

// dw[col] = sum of the partial rows: 32 threads a column take every 32nd row, then add
// in thread order pairs (a fixed tree).
__global__ void __launch_bounds__(1024)
norm_rope_dw_kernel(const float* part, int parts, int D, float* dwq, float* dwk, int* err) {
    __shared__ float s[32][33];
    pdl_wait();
    pdl_trigger();
    if (has_error(err)) return;
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + cx;
    float v = 0.f;
    if (col < 2 * D)
        for (int i = ry; i < parts; i += 32) v += part[static_cast<long long>(i) * 2 * D + col];
    s[ry][cx] = v;
    __syncthreads();
    v = s[cx][ry];  // warp ry now holds column ry's 32 sums
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int out = blockIdx.x * 32 + ry;
    if (cx == 0 && out < 2 * D) {
        if (out < D) dwq[out] = v;
        else if (dwk != nullptr) dwk[out - D] = v;
    }
}

__global__ void rope_table_kernel(long long n, int half, const double* inv_freq, double scale,
                                  float2* table, int* err) {
    pdl_wait();
    pdl_trigger();
    if (has_error(err)) return;
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= n) return;
    double s, c;
    sincos(static_cast<double>(i / half) * inv_freq[i % half], &s, &c);
    table[i] = make_float2(static_cast<float>(scale * c), static_cast<float>(scale * s));
}

// How a token's rows are cut into runs (one warp each): whole tokens when there are
// enough of them to fill the GPU, else pieces down to the rows a warp holds at once.
struct Runs {
    int runs, rows;
};
Runs plan_runs(int T, int rows, int rpw) {
    const int groups = (rows + rpw - 1) / rpw;  // warp-wide row groups of a token
    const long long want = static_cast<long long>(num_sms()) * 32;
    long long runs = T > 0 ? (want + T - 1) / T : 1;
    if (runs > groups) runs = groups;
    const int per = static_cast<int>((groups + runs - 1) / runs);
    return {(groups + per - 1) / per, per * rpw};
}

template <int LPR, int SWAP>
cudaError_t fwd(const NormRope& p, bool append, cudaStream_t st) {
    const int rows = p.a.Hq + (p.k.p ? p.a.Hkv : 0) + (append ? p.a.Hkv : 0);
    const Runs r = plan_runs(p.T, rows, 32 / LPR);
    const long long tasks = static_cast<long long>(p.T) * r.runs;
    const dim3 grid(static_cast<unsigned>((tasks + kWarps - 1) / kWarps));
    LaunchScope ls(append ? "kv_append" : "norm_rope", st);
    return append ? launch_k(norm_rope_kernel<LPR, SWAP, true>, grid, dim3(kWarps * 32), 0, st, p,
                             r.runs, r.rows)
                  : launch_k(norm_rope_kernel<LPR, SWAP, false>, grid, dim3(kWarps * 32), 0, st, p,
                             r.runs, r.rows);
}

template <int LPR, int SWAP>
cudaError_t bwd(const NormRope& p, Heads dq_out, Heads dk_out, float* part, cudaStream_t st) {
    const int rows = p.a.Hq + (p.k.p ? p.a.Hkv : 0);
    const Runs r = plan_runs(p.T, rows, 32 / LPR);
    LaunchScope ls("norm_rope_backward", st);
    return launch_k(norm_rope_backward_kernel<LPR, SWAP>, dim3(norm_rope_parts(p.a, p.T)),
                    dim3(kWarps * 32), 0, st, p, dq_out, dk_out, part, r.runs, r.rows);
}

}  // namespace

cudaError_t launch_rope_table(int positions, int half, const double* inv_freq, double scale,
                              float2* table, int* err, cudaStream_t st) {
    const long long n = static_cast<long long>(positions) * half;
    LaunchScope ls("rope_table", st);
    return launch_k(rope_table_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, st,
                    n, half, inv_freq, scale, table, err);
}

cudaError_t launch_norm_rope(const NormRope& p, bool append, cudaStream_t st) {
    const bool narrow = p.a.D <= 64;
    switch (swap_of(p)) {
        case SWAP_NONE: return narrow ? fwd<8, SWAP_NONE>(p, append, st) : fwd<16, SWAP_NONE>(p, append, st);
        case SWAP_OWN: return narrow ? fwd<8, SWAP_OWN>(p, append, st) : fwd<16, SWAP_OWN>(p, append, st);
        case SWAP_LANE: return narrow ? fwd<8, SWAP_LANE>(p, append, st) : fwd<16, SWAP_LANE>(p, append, st);
        default: return narrow ? fwd<8, SWAP_ROW>(p, append, st) : fwd<16, SWAP_ROW>(p, append, st);
    }
}

// CTAs of the backward (each writes one partial row): four per SM, fewer when there
// are fewer rows.
int norm_rope_parts(const moe_attn_shape& a, int T) {
    const int rpw = a.D <= 64 ? 4 : 2;
    const long long groups = static_cast<long long>(T) * ((a.Hq + a.Hkv + rpw - 1) / rpw);
    const long long ctas = (groups + kWarps - 1) / kWarps;
    const long long most = 4ll * num_sms();
    return static_cast<int>(ctas < 1 ? 1 : ctas < most ? ctas : most);
}

cudaError_t launch_norm_rope_backward(const NormRope& p, Heads dq_out, Heads dk_out, float* part,
                                      float* dwq, float* dwk, cudaStream_t st) {
    const bool narrow = p.a.D <= 64;
    cudaError_t e;
    switch (swap_of(p)) {
        case SWAP_NONE: e = narrow ? bwd<8, SWAP_NONE>(p, dq_out, dk_out, part, st) : bwd<16, SWAP_NONE>(p, dq_out, dk_out, part, st); break;
        case SWAP_OWN: e = narrow ? bwd<8, SWAP_OWN>(p, dq_out, dk_out, part, st) : bwd<16, SWAP_OWN>(p, dq_out, dk_out, part, st); break;
        case SWAP_LANE: e = narrow ? bwd<8, SWAP_LANE>(p, dq_out, dk_out, part, st) : bwd<16, SWAP_LANE>(p, dq_out, dk_out, part, st); break;
        default: e = narrow ? bwd<8, SWAP_ROW>(p, dq_out, dk_out, part, st) : bwd<16, SWAP_ROW>(p, dq_out, dk_out, part, st); break;
    }
    if (e != cudaSuccess || p.wq == nullptr) return e;
    LaunchScope ls("norm_rope_dw", st);
    return launch_k(norm_rope_dw_kernel, dim3((2 * p.a.D + 31) / 32), dim3(1024), 0, st,
                    static_cast<const float*>(part), norm_rope_parts(p.a, p.T), p.a.D, dwq, dwk,
                    p.err);
}

}  // namespace attn
}  // namespace moe
