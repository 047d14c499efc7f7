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
// Both directions are bound by memory (2 or 3 x 2 bytes a value), if their instructions
// are few: a head row is read as 16-byte pieces of 8 values, so D / 8 lanes (8 or 16 with
// padding) hold one row and a warp holds 2 to 4 rows at once. A warp takes rows of one
// kind (queries, keys or values) of one token, so what they share is formed once, in
// registers: out_i = r (x_i A_i + x_{partner(i)} B_i) with A = w cos, B = w_{partner} sin'.
// The partner's values are exchanged as they were read, two bf16 a register: from the
// lane's own registers (interleaved), by shuffles (half layout, when whole pieces swap), or
// through shared memory (any other number of rotated dims). Arithmetic is two fp32
// operations an instruction. (One weight load and one fp32 shuffle a value, at half the
// warps: 34.8 us for 4096 tokens of 32/8 heads of 128 against 19.)
#include "attn.cuh"
#include "ptx.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 8;

enum Swap { SWAP_NONE = 0, SWAP_OWN = 1, SWAP_LANE = 2, SWAP_ROW = 3 };

Swap swap_of(const NormRope& p) {
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

// Which rows of which token a warp takes: a token has q runs of its queries, k of its keys
// and v of its values (append), of at most `rows` rows.
struct Runs {
    int q, k, v, rows;
    int total() const { return q + k + v; }
};

// U: row loads in flight per lane; NT: tokens that a warp takes, one after the other. A block
// takes one run of kWarps * NT tokens.
template <int LPR, int SWAP, bool APPEND, int U, int NT>
__global__ void __launch_bounds__(kWarps * 32, U == 2 ? 4 : 3)
norm_rope_kernel(const NormRope p, const Runs rn) {
    constexpr int RPW = 32 / LPR;  // rows of a warp at once
    __shared__ __align__(16) bf16 s_buf[SWAP == SWAP_ROW ? kWarps * RPW * 128 : 8];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = (blockIdx.x * kWarps + warp) * NT;
    if (t0 >= p.T) return;
    int run = blockIdx.y, kind = 0;  // 0 queries, 1 keys, 2 values
    if (run >= rn.q) {
        run -= rn.q;
        kind = 1;
        if (APPEND && run >= rn.k) {
            run -= rn.k;
            kind = 2;
        }
    }
    const int piece = lane % LPR, sub = lane / LPR;
    const int D = p.a.D, Hkv = p.a.Hkv;
    const int r0 = run * rn.rows, r1 = min(kind == 0 ? p.a.Hq : Hkv, r0 + rn.rows);
    const bool live = piece * 8 < D;
    const Heads src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    const bf16* in_row = src.row(t0, r0 + sub) + piece * 8;

    uint4 in[U];
    const auto load = [&](const bf16* row, int rb) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            in[u] = make_uint4(0u, 0u, 0u, 0u);
            if (rb + u * RPW + sub < r1 && live)
                in[u] = *reinterpret_cast<const uint4*>(row + (rb - r0 + u * RPW) * src.hs);
        }
    };
    // what does not depend on another load comes first, all of it in flight at once
    load(in_row, r0);
    const bool skip = stopped(p.err);
    int positions = 0;  // lane i: of token t0 + i
    if (SWAP != SWAP_NONE && kind < 2 && lane < NT && t0 + lane < p.T) positions = p.positions[t0 + lane];
    const long long slot = APPEND && kind > 0 ? p.slots[t0] : 0;
    const bool norm = p.wq != nullptr;
    float w[8], wp[8];  // the weights of this lane's values and of their partners
    if (norm && kind < 2) {
        const float* wr = kind == 0 ? p.wq : p.wk;
        load_weights(wr, live ? piece : 0, w);
        if constexpr (SWAP == SWAP_LANE) {
            const int hop = p.rot >> 4;
            load_weights(wr, !live ? 0 : piece < hop ? piece + hop : piece < 2 * hop ? piece - hop : piece, wp);
        } else if constexpr (SWAP == SWAP_ROW) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                wp[e] = __ldg(wr + (live ? partner_of(piece * 8 + e, p.rot, p.interleaved) : 0));
        }
    }
    if (skip) return;

    // where the rows go
    bf16* out = (kind == 0 ? p.q_out : p.k_out).row(t0, r0 + sub) + piece * 8;
    const long long out_ts = (kind == 0 ? p.q_out : p.k_out).ts;
    long long out_hs = (kind == 0 ? p.q_out : p.k_out).hs;
    if constexpr (APPEND) {
        static_assert(NT == 1, "a slot per task");
        if (kind > 0) {
            if (slot >= (static_cast<long long>(p.pages) << p.page_shift)) {
                if (lane == 0) raise_error(p.err, MOE_ERR_BAD_INDEX);
                return;
            }
            if (slot < 0) return;
            const long long page = slot >> p.page_shift;
            out_hs = static_cast<long long>(D) << p.page_shift;
            out = (kind == 1 ? p.k_pages : p.v_pages) + (page * Hkv + r0 + sub) * out_hs +
                  (slot & ((1 << p.page_shift) - 1)) * D + piece * 8;
        }
        if (kind == 2) {
            for (int rb = r0; rb < r1; rb += RPW * U) {
                if (rb > r0) load(in_row, rb);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (rb + u * RPW + sub < r1 && live)
                        *reinterpret_cast<uint4*>(out + (rb - r0 + u * RPW) * out_hs) = in[u];
            }
            return;
        }
    }
    bf16* buf = s_buf + (SWAP == SWAP_ROW ? (warp * RPW + sub) * 128 : 0);
    const float inv_d = 1.f / static_cast<float>(D);
#pragma unroll 1
    for (int i = 0; i < NT && t0 + i < p.T; ++i) {
        float a[8], b[8];  // A and B
        bool bad = false;
        if constexpr (SWAP != SWAP_NONE) {
            const int pos = __shfl_sync(0xffffffffu, positions, i);
            bad = pos < 0 || pos >= p.table_rows;  // the whole warp: one token
            if (bad && lane == 0) raise_error(p.err, MOE_ERR_BAD_INDEX);
            load_rotation<SWAP>(p.table + static_cast<long long>(bad ? 0 : pos) * (p.rot >> 1), p.rot,
                                p.interleaved, piece, a, b);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = 1.f;
        }
        if (norm) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                mul2(a[e], a[e + 1], w[e], w[e + 1]);
                if constexpr (SWAP == SWAP_OWN) mul2(b[e], b[e + 1], w[e + 1], w[e]);
                if constexpr (SWAP == SWAP_LANE || SWAP == SWAP_ROW)
                    mul2(b[e], b[e + 1], wp[e], wp[e + 1]);
            }
        }
        for (int rb = r0; rb < r1; rb += RPW * U) {
            if (rb > r0) load(in_row, rb);
            uint4 rows[U];
#pragma unroll
            for (int u = 0; u < U; ++u) rows[u] = in[u];
            if (NT > 1 && rb + RPW * U >= r1 && i + 1 < NT && t0 + i + 1 < p.T) {
                in_row += src.ts;  // the next token's first rows
                load(in_row, r0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[8], y[8];
                unpack8(rows[u], x);
                float rr = 1.f;
                if (norm) {
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; e += 2) fma2(s0, s1, x[e], x[e + 1], x[e], x[e + 1]);
                    rr = rsqrtf(row_sum<LPR>(s0 + s1) * inv_d + p.eps);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = x[e];
#pragma unroll
                for (int e = 0; e < 8; e += 2) mul2(y[e], y[e + 1], a[e], a[e + 1]);
                if constexpr (SWAP != SWAP_NONE) {
                    float o[8];
                    partners<LPR, SWAP>(rows[u], x, p.rot, p.interleaved, piece, buf, o);
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        fma2(y[e], y[e + 1], o[e], o[e + 1], b[e], b[e + 1]);
                }
#pragma unroll
                for (int e = 0; e < 8; e += 2) mul2(y[e], y[e + 1], rr, rr);
                if (rb + u * RPW + sub < r1 && live && !bad)
                    *reinterpret_cast<uint4*>(out + (rb - r0 + u * RPW) * out_hs) = pack8(y);
            }
        }
        out += out_ts;
    }
}

// Backward: with the upstream gradient g rotated back, dy_i = g_i cos_i - g_partner sin'_i,
// and q = sum dy w x: dx = r dy w - x r^3 q / D, dw += r dy x. A warp walks (token, run)
// tasks of the queries, then of the keys, with the grid's stride, and keeps its piece of
// that weight gradient in registers; a CTA adds its warps' sums in warp order and writes
// one partial row [2][D]. The rows come through a ring in shared memory that each lane
// fills (cp.async) and reads for itself, kAhead batches ahead: the registers that the
// sums take leave 16 warps an SM, too few to hide the loads by themselves (62 us for 16384
// tokens of 16/4 heads of 128 without the ring, against 52).
constexpr int kBatch = 2;  // row groups of a batch
constexpr int kAhead = 4;  // slots of the ring
constexpr int kRing = kWarps * kAhead * kBatch * 2 * 512;

template <int LPR, int SWAP>
__global__ void __launch_bounds__(kWarps * 32, 2)
norm_rope_backward_kernel(const NormRope p, Heads dq_out, Heads dk_out, float* part, const Runs rn) {
    constexpr int RPW = 32 / LPR, U = kBatch;
    extern __shared__ __align__(16) uint8_t s_ring[];  // [warp][slot][group][x, g][lane]
    __shared__ __align__(16) bf16 s_buf[SWAP == SWAP_ROW ? kWarps * RPW * 128 : 8];
    __shared__ float s_dw[kWarps][2][128];
    pdl_wait();
    pdl_trigger();
    if (stopped(p.err)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int piece = lane % LPR, sub = lane / LPR;
    const int D = p.a.D;
    const bool live = piece * 8 < D;
    const bool norm = p.wq != nullptr;
    bf16* buf = s_buf + (SWAP == SWAP_ROW ? (warp * RPW + sub) * 128 : 0);
    uint4* ring = reinterpret_cast<uint4*>(s_ring) + warp * (kAhead * U * 2 * 32) + lane;
    const float inv_d = 1.f / static_cast<float>(D);
    const long long step = static_cast<long long>(gridDim.x) * kWarps;
    const long long start = static_cast<long long>(blockIdx.x) * kWarps + warp;
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        float acc[8], w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            acc[e] = 0.f;
            w[e] = norm && live ? (kind == 0 ? p.wq : p.wk)[piece * 8 + e] : 1.f;
        }
        const Heads xs = kind == 0 ? p.q : p.k, gs = kind == 0 ? dq_out : dk_out;
        const Heads os = kind == 0 ? p.q_out : p.k_out;
        const int runs = max(1, kind == 0 ? rn.q : rn.k);
        const int rows = kind == 0 ? p.a.Hq : p.k.p ? p.a.Hkv : 0;
        const int step_t = static_cast<int>(step / runs), step_r = static_cast<int>(step % runs);
        // A batch of this warp: rows rb .. of run `run` of token t.
        struct At {
            int t, run, rb;
        };
        const auto next_task = [&](At& a) {
            a.t += step_t;
            a.run += step_r;
            if (a.run >= runs) {
                a.run -= runs;
                ++a.t;
            }
            a.rb = a.run * rn.rows;
        };
        const auto last_row = [&](const At& a) { return min(rows, (a.run + 1) * rn.rows); };
        At in{static_cast<int>(start / runs), static_cast<int>(start % runs), 0};
        in.rb = in.run * rn.rows;
        if (rows == 0) in.t = p.T;
        At at = in;
        int slot_in = 0, slot = 0;
        const auto issue = [&]() {  // the next batch into the ring (empty past the last)
            if (in.t < p.T) {
                const int r1 = last_row(in);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = in.rb + u * RPW + sub;
                    if (r < r1 && live) {
                        uint4* dst = ring + (slot_in * U + u) * 64;
                        ptx::cp_async16(ptx::smem_u32(dst), xs.row(in.t, r) + piece * 8, 16);
                        ptx::cp_async16(ptx::smem_u32(dst + 32), gs.row(in.t, r) + piece * 8, 16);
                    }
                }
                in.rb += RPW * U;
                if (in.rb >= r1) next_task(in);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            slot_in = slot_in + 1 == kAhead ? 0 : slot_in + 1;
        };
#pragma unroll
        for (int i = 0; i < kAhead - 1; ++i) issue();
        int pos = 0;
        if (SWAP != SWAP_NONE && at.t < p.T) pos = p.positions[at.t];
        while (at.t < p.T) {
            const At task = at;
            const int r1 = last_row(at);
            next_task(at);
            const int pos_now = pos;
            float c[8], s[8];
            bool bad = false;
            if constexpr (SWAP != SWAP_NONE) {
                if (at.t < p.T) pos = p.positions[at.t];  // of the next task
                bad = pos_now < 0 || pos_now >= p.table_rows;
                if (bad && lane == 0) raise_error(p.err, MOE_ERR_BAD_INDEX);
                load_rotation<SWAP>(p.table + static_cast<long long>(bad ? 0 : pos_now) * (p.rot >> 1),
                                    p.rot, p.interleaved, piece, c, s);
            }
            bf16* orow = os.row(task.t, task.rb + sub) + piece * 8;
            for (int rb = task.rb; rb < r1; rb += RPW * U) {
                issue();
                asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
                uint4 xin[U], gin[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    xin[u] = gin[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (rb + u * RPW + sub < r1 && live) {
                        xin[u] = ring[(slot * U + u) * 64];
                        gin[u] = ring[(slot * U + u) * 64 + 32];
                    }
                }
                slot = slot + 1 == kAhead ? 0 : slot + 1;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float x[8], dy[8];
                    unpack8(xin[u], x);
                    unpack8(gin[u], dy);
                    if constexpr (SWAP != SWAP_NONE) {
                        float o[8];
                        partners<LPR, SWAP>(gin[u], dy, p.rot, p.interleaved, piece, buf, o);
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            mul2(dy[e], dy[e + 1], c[e], c[e + 1]);
                            fma2(dy[e], dy[e + 1], o[e], o[e + 1], -s[e], -s[e + 1]);
                        }
                    }
                    const bool mine = rb + u * RPW + sub < r1 && !bad;
                    if (norm) {
                        float s0 = 0.f, s1 = 0.f, q0 = 0.f, q1 = 0.f, g[8];
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            fma2(s0, s1, x[e], x[e + 1], x[e], x[e + 1]);
                            g[e] = dy[e];
                            g[e + 1] = dy[e + 1];
                            mul2(g[e], g[e + 1], x[e], x[e + 1]);           // dy x
                            fma2(q0, q1, g[e], g[e + 1], w[e], w[e + 1]);
                        }
                        // rows past the run (zeros) and rows left out add nothing
                        float rr = rsqrtf(row_sum<LPR>(s0 + s1) * inv_d + p.eps);
                        // (r^3 alone would leave fp32 where r is beyond 2^42 either way)
                        const float k = -(rr * rr) * (rr * (row_sum<LPR>(q0 + q1) * inv_d));
                        if (mine) {
#pragma unroll
                            for (int e = 0; e < 8; e += 2) {
                                fma2(acc[e], acc[e + 1], g[e], g[e + 1], rr, rr);
                                mul2(dy[e], dy[e + 1], w[e], w[e + 1]);
                                mul2(dy[e], dy[e + 1], rr, rr);
                                fma2(dy[e], dy[e + 1], x[e], x[e + 1], k, k);
                            }
                        }
                    }
                    if (mine && live)
                        *reinterpret_cast<uint4*>(orow + (rb - task.rb + u * RPW) * os.hs) = pack8(dy);
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
            if (sub == 0 && live) s_dw[warp][kind][piece * 8 + e] = acc[e];
        }
    }
    if (!norm) return;
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
// in a fixed tree.
__global__ void __launch_bounds__(1024)
norm_rope_dw_kernel(const float* part, int parts, int D, float* dwq, float* dwk, int* err) {
    __shared__ float s[32][33];
    pdl_wait();
    pdl_trigger();
    if (stopped(err)) return;
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
    if (stopped(err)) return;
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= n) return;
    double s, c;
    sincos(static_cast<double>(i / half) * inv_freq[i % half], &s, &c);
    table[i] = make_float2(static_cast<float>(scale * c), static_cast<float>(scale * s));
}

// Rows of a run: two batches of loads where there are many tokens, fewer (down to the rows
// that a warp holds at once) until the warps fill the GPU.
Runs plan_runs(const NormRope& p, int rpw, int batch, bool append) {
    Runs r{};
    for (r.rows = 2 * batch * rpw;; r.rows /= 2) {
        const int kv = (p.a.Hkv + r.rows - 1) / r.rows;
        r.q = (p.a.Hq + r.rows - 1) / r.rows;
        r.k = p.k.p ? kv : 0;
        r.v = append ? kv : 0;
        if (r.rows <= rpw || static_cast<long long>(p.T) * r.total() >= num_sms() * 32ll) return r;
    }
}

template <int LPR, int SWAP, bool APPEND, int U, int NT>
cudaError_t fwd_u(const NormRope& p, const Runs& r, cudaStream_t st) {
    constexpr int TOKENS = kWarps * NT;
    const dim3 grid(static_cast<unsigned>((p.T + TOKENS - 1) / TOKENS), r.total());
    return launch_k(norm_rope_kernel<LPR, SWAP, APPEND, U, NT>, grid, dim3(kWarps * 32), 0, st, p, r);
}

// Two loads in flight per lane where a token's heads of a kind are no more than that (fewer
// registers, so more warps), else four; and several tokens a warp where there are so many
// tokens that they fill the GPU all the same (65536 tokens of 8/8 heads of 64: 88 us with
// four loads and one token, 72 with two and one, 56 with two and four).
template <int LPR, int SWAP>
cudaError_t fwd(const NormRope& p, bool append, cudaStream_t st) {
    constexpr int RPW = 32 / LPR;
    const Runs r = plan_runs(p, RPW, 4, append);
    const bool few = p.a.Hq <= 2 * RPW || r.rows <= 2 * RPW;
    LaunchScope ls(append ? "kv_append" : "norm_rope", st);
    if (append)
        return few ? fwd_u<LPR, SWAP, true, 2, 1>(p, r, st) : fwd_u<LPR, SWAP, true, 4, 1>(p, r, st);
    if (!few) return fwd_u<LPR, SWAP, false, 4, 1>(p, r, st);
    return static_cast<long long>(p.T) * r.total() >= num_sms() * 32ll * 8
               ? fwd_u<LPR, SWAP, false, 2, 4>(p, r, st)
               : fwd_u<LPR, SWAP, false, 2, 1>(p, r, st);
}

template <int LPR, int SWAP>
cudaError_t bwd(const NormRope& p, Heads dq_out, Heads dk_out, float* part, cudaStream_t st) {
    const Runs r = plan_runs(p, 32 / LPR, 4, false);
    auto kfn = norm_rope_backward_kernel<LPR, SWAP>;
    const cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
    if (e != cudaSuccess) return e;
    LaunchScope ls("norm_rope_backward", st);
    return launch_k(kfn, dim3(norm_rope_parts(p.a, p.T)), dim3(kWarps * 32), kRing, st, p, dq_out,
                    dk_out, part, r);
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

// CTAs of the backward (each writes one partial row): two per SM, fewer when there
// are fewer rows.
int norm_rope_parts(const moe_attn_shape& a, int T) {
    const int rpw = a.D <= 64 ? 4 : 2;
    const long long groups = static_cast<long long>(T) * ((a.Hq + a.Hkv + rpw - 1) / rpw);
    const long long ctas = (groups + kWarps - 1) / kWarps;
    const long long most = 2ll * num_sms();
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
    return launch_pdl(norm_rope_dw_kernel, dim3((2 * p.a.D + 31) / 32), dim3(1024), 0, st,
                    static_cast<const float*>(part), norm_rope_parts(p.a, p.T), p.a.D, dwq, dwk,
                    p.err);
}

}  // namespace attn
}  // namespace moe
