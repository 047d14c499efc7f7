// attention_bwd.cu — the backward of softmax attention over packed sequences.
//
//   P = exp(scale q k^T - lse),  delta = sum_i dout_i out_i,  dP = dout v^T,
//   dS = P (dP - delta),  dq = scale dS k,  dk = scale dS^T q,  dv = P^T dout.
//
// Two kernels, so that every gradient is summed by one CTA in one order (a single kernel
// over key tiles would need atomics, or fp32 partials of dq larger than all other
// traffic). The scores and dP are formed in both: 7 products against the least 5.
//   dq_kernel   a tile of 128 query rows (the G heads of 128 / G tokens) over its key
//               tiles: S = Q K^T, dP = dO V^T, dQ += dS K. It also writes delta and lse of
//               its rows in tile order for the second kernel.
//   dkv_kernel  a tile of 128 keys over the query tiles that see it, transposed so that
//               keys are rows: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.
//               The G heads of a group are rows of the same tiles, so their sum is the
//               product's.
// Roles as in the forward: a TMA warp, a warp that issues the tcgen05 products, and four
// groups of four warps that turn scores into weights, each for 32 of the 128 columns of
// every row; P and dS go back to TMEM as bf16 operands over the columns that their group
// has read. (Two groups of 64 columns: 652 against 629 us for dq, 697 against 700 for dkv,
// 8192 tokens, 32/8 heads of 128.) The order of the products leaves the tensor cores work
// while the other warps compute: in dkv_kernel (dP, [P] dV, next S, [dS] dK) P while dP
// runs and dS while dV and the next S run; in dq_kernel the next S and dP run while dS is
// formed. TMEM: dq_kernel S, dP twice, dQ; dkv_kernel S, dP, dV, dK (4 x 128 columns).
//
// P and dS are rounded to bf16 (the operand type), everything else is fp32; scale enters
// dq and dk once at the end. Masked weights are zero by selection, and rows of an operand
// that lie past the sequence are zeroed in shared memory where they are summed over.
#include <algorithm>

#include "attn_mma.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kGroups = 4;            // of four warps, kCols columns of every row each
constexpr int kCols = kRows / kGroups;
constexpr int kCompute = 4 * kGroups;  // warps
constexpr int kThreads = (kCompute + 3) * 32;  // and tensor cores, TMA, row data
constexpr float kLog2e = 1.44269504088896341f;

struct Params {
    moe_attn_shape a;
    Packed s;
    float scale;
    Heads out, dout, dq, dk, dv;
    const float* lse;
    float *row_lse, *row_delta;  // [Hkv][Tq][G]: -lse * log2(e) (-inf: no key) and -delta
    int* err;
    int tpt;    // tokens of a 128-row query tile
    int items;  // upper bound of a head's query tiles (dq_kernel)
};

template <int DP>
struct Cfg {
    static constexpr int PIECES = DP / 64;
    static constexpr int TILE = PIECES * kPiece;
    static constexpr int R0 = 3, R1 = 2;  // ring stages: the operand used twice, the other
    static constexpr int TILES = (2 + R0 + R1) * TILE;
    static constexpr int SMEM_Q = TILES + kGroups * 512 + 512;  // parts of delta, barriers
    static constexpr int SMEM_KV = TILES + 2 * 2 * 512 + 256;  // two slots of lse and delta
};

// A group's columns of TMEM as fp32.
__device__ __forceinline__ void load_cols(uint32_t t, float (&v)[kCols]) {
#pragma unroll
    for (int i = 0; i < kCols; i += 32) tmem_ld32(t + i, *reinterpret_cast<uint32_t(*)[32]>(v + i));
    tmem_ld_wait();
}
// A group's columns as kCols / 2 columns of bf16 pairs.
__device__ __forceinline__ void store_cols(uint32_t t, const float (&v)[kCols]) {
#pragma unroll
    for (int h = 0; h < kCols; h += 32) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack2(v[h + 2 * i], v[h + 2 * i + 1]);
        tmem_st16(t + h / 2, w);
    }
    tmem_st_wait();
}
// k-th 16 columns of a bf16 operand that the groups wrote: group g's columns in the
// kCols / 2 TMEM columns at t + kCols g, over scores that it has read itself.
__device__ __forceinline__ uint32_t operand(uint32_t t, int k) {
    constexpr int per = kCols / 16;
    return t + kCols * (k / per) + 8 * (k % per);
}

// ---------------------------------------------------------------------- dq
// One tile of 128 query rows and the key tiles that it sees.
struct Item {
    int q0, nq, k0, nk;
    int first, hk;    // first token (in the sequence), key/value head (-1: no more work)
    int steps, seen;  // key tiles and keys that some row sees
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
dq_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapDO,
          const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
          const Params p) {
    using C = Cfg<DP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sQ = smem_u32(smem), sDO = sQ + C::TILE;
    const uint32_t sK = sDO + C::TILE, sV = sK + C::R0 * C::TILE;
    float* part_delta = reinterpret_cast<float*>(smem + C::TILES);  // [kGroups][128]
    uint8_t* misc = smem + C::TILES + kGroups * 512;
    const uint32_t bars = smem_u32(misc);
    // Phases run on through all items of a CTA: steps are counted from its first item on,
    // q, do, q_free, dq, dq_free and tail per item that has steps (tail: that needs it).
    const auto k_full = [&](int s) { return bars + 8u * s; };
    const auto k_empty = [&](int s) { return bars + 8u * (3 + s); };
    const auto v_full = [&](int s) { return bars + 8u * (6 + s); };
    const auto dp_bar = [&](int s) { return bars + 8u * (8 + s); };    // dP written (V read)
    const auto w_full = [&](int s) { return bars + 8u * (10 + s); };   // an item is in its slot
    const uint32_t q_bar = bars + 8u * 12, do_bar = bars + 8u * 13, q_free = bars + 8u * 14,
                   s_bar = bars + 8u * 15, dq_bar = bars + 8u * 16, tail_bar = bars + 8u * 17,
                   done_bar = bars + 8u * 18;
    const uint32_t s_read = bars + 8u * 19, delta_bar = bars + 8u * 20, dq_free = bars + 8u * 21;
    // dS written: two, as the dS of two steps can be finished before the products' thread
    // looks again (a wait that is passed by two phases would not return)
    const auto ds_bar = [&](int s) { return bars + 8u * (22 + s); };
    const auto w_free = [&](int s) { return bars + 8u * (24 + s); };   // an item's slot read
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 8 * 26);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    Item* ring = reinterpret_cast<Item*>(misc + 8 * 27);  // two slots
    constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DQ = 384;  // dP twice

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 19; ++i) mbar_init(bars + 8 * i, 1);
        for (int i = 19; i < 24; ++i) mbar_init(bars + 8 * i, kCompute);
        for (int i = 24; i < 26; ++i) mbar_init(bars + 8 * i, kCompute + 2);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kCompute) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    if (warp == kCompute + 1 && lane == 0) {
        prefetch_tensormap(&mapQ);
        prefetch_tensormap(&mapDO);
        prefetch_tensormap(&mapK);
        prefetch_tensormap(&mapV);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    const int tpt = p.tpt, G = p.a.Hq / p.a.Hkv;
    const auto item_there = [&](int i) -> bool {
        wait_phase(w_full(i & 1), (i >> 1) & 1, abort_flag);
        return ring[i & 1].hk >= 0 && *abort_flag == 0;
    };
    const auto item_done = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(w_free(i & 1));
    };

    if (warp == kCompute + 2) {
        // --------------------------------------------- items, one ahead of the others
        const bool off = (sQ & 1023u) != 0;  // the swizzle's unit
        if (off) raise_error(p.err, MOE_ERR_MISALIGNED);
        const bool skip = __any_sync(~0u, off || stopped(p.err));
        for (int i = 0;; ++i) {
            // snake order: forwards through the CTAs, then backwards
            const int index = i * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            Item it{};
            it.hk = -1;
            if (index < p.items * p.a.Hkv) {
                const Work w = find_work<false>(p.s, tpt, index / p.a.Hkv, lane, p.err);
                it.q0 = w.q0, it.nq = w.nq, it.k0 = w.k0, it.nk = w.nk;
                it.first = w.item * tpt;
                if (w.items > 0 && !skip) it.hk = index % p.a.Hkv;
                it.seen = p.s.causal ? max(0, min(w.nk, min(it.first + tpt, w.nq) + w.nk - w.nq)) : w.nk;
                it.steps = (it.seen + kRows - 1) / kRows;
            }
            if (i >= 2) warp_wait(w_free(i & 1), (i / 2 - 1) & 1, abort_flag);
            if (lane == 0) {
                ring[i & 1] = it;
                mbar_arrive(w_full(i & 1));
            }
            if (__any_sync(~0u, it.hk < 0 || *abort_flag != 0)) break;
        }
        if (blockIdx.x == 0) check_sequences(p.s, lane, p.err);
    } else if (warp == kCompute + 1) {
        // ---------------------------------------------------------------------- loads
        const auto load = [&](uint32_t dst, const CUtensorMap* m, uint32_t bar, int h, int t) {
            for (int c = 0; c < C::PIECES; ++c) tma_load_3d(dst + c * kPiece, m, bar, 64 * c, h, t);
        };
        const uint32_t qbytes = C::PIECES * 128 * G * tpt;
        int gk = 0, gv = 0, had = 0, dos = 0;  // K and V tiles, Q and dO tiles loaded so far
        for (int i = 0; __all_sync(~0u, item_there(i)); ++i) {
            const Item it = ring[i & 1];
            item_done(i);
            if (lane == 0 && it.steps > 0) {
                for (int j = 0; j < it.steps; ++j) {
                    int s = gk % C::R0;
                    if (gk >= C::R0) wait_phase(k_empty(s), (gk / C::R0 - 1) & 1, abort_flag);
                    if (*abort_flag) break;
                    mbar_arrive_expect_tx(k_full(s), C::TILE);
                    load(sK + s * C::TILE, &mapK, k_full(s), it.hk, it.k0 + j * kRows);
                    ++gk;
                    if (j == 0) {
                        if (had > 0) wait_phase(q_free, (had - 1) & 1, abort_flag);
                        if (*abort_flag) break;
                        ++had;
                        mbar_arrive_expect_tx(q_bar, qbytes);
                        load(sQ, &mapQ, q_bar, it.hk * G, it.q0 + it.first);
                        ++dos;
                        mbar_arrive_expect_tx(do_bar, qbytes);
                        load(sDO, &mapDO, do_bar, it.hk * G, it.q0 + it.first);
                    }
                    s = gv % C::R1;  // V tile g - 2 has been read when its dP is there
                    if (gv >= C::R1) wait_phase(dp_bar(s), (gv / C::R1 - 1) & 1, abort_flag);
                    if (*abort_flag) break;
                    mbar_arrive_expect_tx(v_full(s), C::TILE);
                    load(sV + s * C::TILE, &mapV, v_full(s), it.hk, it.k0 + j * kRows);
                    ++gv;
                }
            }
            __syncwarp();
            if (it.seen % kRows != 0) {  // the last K tile has rows past the keys
                const int last = __shfl_sync(~0u, gk, 0) - 1;
                if (last >= 0) {
                    warp_wait(k_full(last % C::R0), (last / C::R0) & 1, abort_flag);
                    zero_tail(sK + last % C::R0 * C::TILE, C::PIECES, it.seen % kRows, lane);
                }
                if (lane == 0) mbar_arrive(tail_bar);
            }
        }
        if (lane == 0) {  // nothing is in flight when the CTA leaves
            if (had > 0) drain(q_bar, (had - 1) & 1);
            if (dos > 0) drain(do_bar, (dos - 1) & 1);
            for (int j = max(0, gk - C::R0); j < gk; ++j) drain(k_full(j % C::R0), (j / C::R0) & 1);
            for (int j = max(0, gv - C::R1); j < gv; ++j) drain(v_full(j % C::R1), (j / C::R1) & 1);
        }
        __syncwarp();
    } else if (warp == kCompute && elect_one()) {
        // ------------------------------------------------- tensor cores (one thread)
        constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0), id_q = idesc_bf16(128, DP, 0, 1);
        const uint64_t qd = desc_d(sQ), dod = desc_d(sDO);
        int g = 0, had = 0, tails = 0;
        for (int i = 0; item_there(i); ++i) {
            const int n = ring[i & 1].steps;
            const bool ragged = ring[i & 1].seen % kRows != 0;
            mbar_arrive(w_free(i & 1));
            // S and dP of step t (the item's last: `last`), once their keys and values are
            // there (rows of K past the keys zeroed: dQ sums over them); S may be
            // overwritten once it is in registers, and dP has two places
            const auto scores = [&](int t, bool last) {
                if (t > 0) wait_phase(s_read, (t - 1) & 1, abort_flag);
                wait_phase(k_full(t % C::R0), (t / C::R0) & 1, abort_flag);
                if (last && ragged) wait_phase(tail_bar, tails & 1, abort_flag);
                tc_fence_after();
                const uint64_t bd = desc_d(sK + t % C::R0 * C::TILE);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    mma_bf16(tmem + TM_S, qd + kd(k), bd + kd(k), id_s, k > 0);
                mma_commit(s_bar);
            };
            const auto dprob = [&](int t, bool last) {
                wait_phase(v_full(t & 1), (t >> 1) & 1, abort_flag);
                tc_fence_after();
                const uint64_t bd = desc_d(sV + (t & 1) * C::TILE);
                const uint32_t dst = tmem + TM_DP + 128 * (t & 1);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) mma_bf16(dst, dod + kd(k), bd + kd(k), id_s, k > 0);
                mma_commit(dp_bar(t & 1));
                if (last) mma_commit(q_free);
            };
            if (n == 0) continue;
            wait_phase(q_bar, had & 1, abort_flag);
            scores(g, n == 1);
            wait_phase(do_bar, had & 1, abort_flag);
            dprob(g, n == 1);
            for (int j = 0; j < n; ++j, ++g) {
                // the next tile's products run while dS is formed
                if (j + 1 < n) {
                    scores(g + 1, j + 2 == n);
                    dprob(g + 1, j + 2 == n);
                }
                // the last item's dQ has been read
                if (j == 0 && had > 0) wait_phase(dq_free, (had - 1) & 1, abort_flag);
                wait_phase(ds_bar(g & 1), (g >> 1) & 1, abort_flag);
                tc_fence_after();
                const uint64_t kdesc = desc_r(sK + g % C::R0 * C::TILE);
                const uint32_t add = j > 0, src = tmem + TM_DP + 128 * (g & 1);
#pragma unroll
                for (int k = 0; k < kRows / 16; ++k)
                    mma_bf16_ta(tmem + TM_DQ, operand(src, k), kdesc + kr(k), id_q, k > 0 ? 1u : add);
                mma_commit(k_empty(g % C::R0));
            }
            mma_commit(dq_bar);
            ++had;
            tails += ragged;
        }
        mma_commit(done_bar);
        drain(done_bar, 0);
    } else if (warp < kCompute) {
        // -------------------------------------------------------------- weights to dS
        const int grp = warp >> 2, row = threadIdx.x & 127, rtok = row / G, head = row % G;
        const float c = p.scale * kLog2e;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        constexpr int W = DP / kGroups;  // columns of dq that a group stores
        int g = 0, had = 0;
        for (int i = 0; __all_sync(~0u, item_there(i)); ++i) {
            const Item it = ring[i & 1];
            item_done(i);
            const int n = it.steps, token = it.first + rtok;
            const bool valid = row < G * tpt && token < it.nq;
            const int mine = !valid ? 0 : p.s.causal ? min(it.nk, token + 1 + it.nk - it.nq) : it.nk;
            const int open = p.s.causal ? it.first + 1 + it.nk - it.nq : it.nk;  // seen by every row
            const long long t = it.q0 + token;
            const int h = it.hk * G + head;
            float delta = 0.f, neg_lse = -INFINITY;
            if (valid) {
                const float e = p.lse[t * p.a.Hq + h];
                neg_lse = e == -INFINITY ? e : -e * kLog2e;
            }
            // The sum of all groups' parts of delta. (Those of the last item have been read:
            // its dQ is complete.)
            const auto sum_parts = [&](float part) {
                part_delta[grp * 128 + row] = part;
                __syncwarp();
                if (lane == 0) mbar_arrive(delta_bar);
                warp_wait(delta_bar, had & 1, abort_flag);
                float sum = part_delta[row];
#pragma unroll
                for (int u = 1; u < kGroups; ++u) sum += part_delta[u * 128 + row];
                return sum;
            };
            // delta of rows that see more than one key tile is that of the rounded out, each
            // group's part of the columns with all loads at once. Rows that see one tile
            // have all their weights here, and delta is summed from those (below): with few
            // keys the rounding of out weighs as much as that of dS (2.6e-3 against 2.4e-3
            // of dq over sequences of 143 to 297 tokens). Rows without a key have out 0.
            if (n > 1) {
                constexpr int V = W / 8;
                uint4 o[V], d[V];
                const bf16* po = p.out.row(t, h);
                const bf16* pd = p.dout.row(t, h);
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    const int col = (grp * V + u) * 8;
                    o[u] = d[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (valid && col < p.a.D) {
                        o[u] = *reinterpret_cast<const uint4*>(po + col);
                        d[u] = *reinterpret_cast<const uint4*>(pd + col);
                    }
                }
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    float a[8], b[8];
                    unpack8(o[u], a);
                    unpack8(d[u], b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) delta += a[e] * b[e];
                }
                delta = sum_parts(delta);
            }
            for (int j = 0; j < n; ++j, ++g) {
                warp_wait(s_bar, g & 1, abort_flag);
                tc_fence_after();
                float s[kCols], d[kCols];
                load_cols(lanes + TM_S + kCols * grp, s);
                warp_arrive(s_read, lane);
#pragma unroll
                for (int e = 0; e < kCols; e += 2) {
                    fma2v(s[e], s[e + 1], c, neg_lse, neg_lse);
                    s[e] = exp2_fast(s[e]);
                    s[e + 1] = exp2_fast(s[e + 1]);
                }
                warp_wait(dp_bar(g & 1), (g >> 1) & 1, abort_flag);
                tc_fence_after();
                const uint32_t tD = lanes + TM_DP + 128 * (g & 1) + kCols * grp;
                load_cols(tD, d);
                const bool masked = (j + 1) * kRows > open;
                const int lim = mine - j * kRows - kCols * grp;
                if (n == 1) {
                    float d0 = 0.f, d1 = 0.f;
#pragma unroll
                    for (int e = 0; e < kCols; e += 2) {
                        d0 += !masked || e < lim ? s[e] * d[e] : 0.f;
                        d1 += !masked || e + 1 < lim ? s[e + 1] * d[e + 1] : 0.f;
                    }
                    delta = sum_parts(d0 + d1);
                }
#pragma unroll
                for (int e = 0; e < kCols; e += 2) {
                    add2(d[e], d[e + 1], -delta, -delta);
                    mul2(d[e], d[e + 1], s[e], s[e + 1]);
                }
                if (masked) {
#pragma unroll
                    for (int e = 0; e < kCols; ++e) d[e] = e < lim ? d[e] : 0.f;
                }
                store_cols(tD, d);
                warp_arrive(ds_bar(g & 1), lane);
            }
            if (valid && grp == 0) {
                const long long at = (static_cast<long long>(it.hk) * p.s.Tq + t) * G + head;
                p.row_lse[at] = neg_lse;
                p.row_delta[at] = -delta;
            }
            if (n > 0) {
                warp_wait(dq_bar, had & 1, abort_flag);
                ++had;
                tc_fence_after();
            }
            bf16* dst = p.dq.row(t, h);
#pragma unroll
            for (int q = 0; q < W; q += 16) {
                uint32_t o[16];
                if (n > 0) {
                    tmem_ld16(lanes + TM_DQ + grp * W + q, o);
                    tmem_ld_wait();
                    if (q + 16 == W) warp_arrive(dq_free, lane);
                }
#pragma unroll
                for (int u = 0; u < 16; u += 8) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = n > 0 ? __uint_as_float(o[u + e]) * p.scale : 0.f;
                    if (valid && grp * W + q + u < p.a.D)
                        *reinterpret_cast<uint4*>(dst + grp * W + q + u) = pack8(v);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && *abort_flag) raise_timeout(p.err);
    if (warp == kCompute) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------- dk, dv
template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
dkv_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapDO,
           const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
           const Params p) {
    using C = Cfg<DP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sK = smem_u32(smem), sV = sK + C::TILE;
    const uint32_t sQ = sV + C::TILE, sDO = sQ + C::R0 * C::TILE;
    float* rowdata = reinterpret_cast<float*>(smem + C::TILES);  // [2][lse, delta][128]
    uint8_t* misc = smem + C::TILES + 2 * 2 * 512;
    const uint32_t bars = smem_u32(misc);
    const auto q_full = [&](int s) { return bars + 8u * s; };
    const auto q_empty = [&](int s) { return bars + 8u * (3 + s); };
    const auto do_full = [&](int s) { return bars + 8u * (6 + s); };
    const auto do_empty = [&](int s) { return bars + 8u * (8 + s); };
    const auto r_full = [&](int s) { return bars + 8u * (10 + s); };
    const uint32_t kv_bar = bars + 96, s_bar = bars + 104, p_bar = bars + 112, dp_bar = bars + 120,
                   ds_bar = bars + 128, done_bar = bars + 136;
    const auto r_empty = [&](int s) { return bars + 144 + 8u * s; };
    const uint32_t tail_bar = bars + 160;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 168);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    Work* found = reinterpret_cast<Work*>(tmem_slot + 2);
    constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 256 + DP;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 10; ++i) mbar_init(bars + 8 * i, 1);
        mbar_init(r_full(0), 32);
        mbar_init(r_full(1), 32);
        mbar_init(r_empty(0), kCompute);
        mbar_init(r_empty(1), kCompute);
        mbar_init(kv_bar, 1);
        mbar_init(s_bar, 1);
        mbar_init(p_bar, kCompute);
        mbar_init(dp_bar, 1);
        mbar_init(ds_bar, kCompute);
        mbar_init(done_bar, 1);
        mbar_init(tail_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kCompute) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    const int hk = blockIdx.x % p.a.Hkv, tpt = p.tpt, G = p.a.Hq / p.a.Hkv;
    if (G * tpt < kRows && warp < C::R0 + C::R1)  // rows that no load writes: zeros in the sums
        zero_tail(sQ + warp * C::TILE, C::PIECES, G * tpt, lane);
    pdl_wait();
    pdl_trigger();
    if (warp == 0) {
        const bool off = (sK & 1023u) != 0;  // the swizzle's unit
        if (off) raise_error(p.err, MOE_ERR_MISALIGNED);
        const bool skip = __any_sync(~0u, off || stopped(p.err));
        Work w = find_work<true>(p.s, tpt, blockIdx.x / p.a.Hkv, lane, p.err);
        if (skip) w.items = 0;
        if (lane == 0) *found = w;
    }
    if (warp == 1 && blockIdx.x == 0) check_sequences(p.s, lane, p.err);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Work w = *found;
    if (w.items > 0) {
        const int q0 = w.q0, nq = w.nq, k0 = w.k0, nk = w.nk;
        const int kv0 = w.item * kRows;
        // query tiles [i0, i0 + n)
        const int i0 = (p.s.causal ? max(0, kv0 - (nk - nq)) : 0) / tpt;
        const int n = max(0, (nq + tpt - 1) / tpt - i0);
        const auto rows_of = [&](int i) { return G * min(tpt, nq - (i0 + i) * tpt); };

        const bool ragged = n > 0 && rows_of(n - 1) < G * tpt;  // the last tile passes the queries
        if (warp == kCompute + 1) {
            if (lane == 0 && n > 0) {
                const auto load = [&](uint32_t dst, const CUtensorMap* m, uint32_t bar, int h, int t) {
                    for (int c = 0; c < C::PIECES; ++c)
                        tma_load_3d(dst + c * kPiece, m, bar, 64 * c, h, t);
                };
                const uint32_t qbytes = C::PIECES * 128 * G * tpt;
                mbar_arrive_expect_tx(kv_bar, 2 * C::TILE);
                load(sK, &mapK, kv_bar, hk, k0 + kv0);
                load(sV, &mapV, kv_bar, hk, k0 + kv0);
                int iq = 0, id = 0;
                for (int i = 0; i < n; ++i) {
                    const int t = q0 + (i0 + i) * tpt;
                    int s = i % C::R0;
                    if (i >= C::R0) wait_phase(q_empty(s), (i / C::R0 - 1) & 1, abort_flag);
                    if (*abort_flag) break;
                    mbar_arrive_expect_tx(q_full(s), qbytes);
                    load(sQ + s * C::TILE, &mapQ, q_full(s), hk * G, t);
                    ++iq;
                    s = i % C::R1;
                    if (i >= C::R1) wait_phase(do_empty(s), (i / C::R1 - 1) & 1, abort_flag);
                    if (*abort_flag) break;
                    mbar_arrive_expect_tx(do_full(s), qbytes);
                    load(sDO + s * C::TILE, &mapDO, do_full(s), hk * G, t);
                    ++id;
                }
                // nothing is in flight when the CTA leaves
                drain(kv_bar, 0);
                for (int i = max(0, iq - C::R0); i < iq; ++i) drain(q_full(i % C::R0), (i / C::R0) & 1);
                for (int i = max(0, id - C::R1); i < id; ++i) drain(do_full(i % C::R1), (i / C::R1) & 1);
            }
            __syncwarp();
            if (ragged) {
                // the last tiles have landed (or the CTA has given up)
                zero_tail(sQ + (n - 1) % C::R0 * C::TILE, C::PIECES, rows_of(n - 1), lane);
                zero_tail(sDO + (n - 1) % C::R1 * C::TILE, C::PIECES, rows_of(n - 1), lane);
                if (lane == 0) mbar_arrive(tail_bar);
            }
        } else if (warp == kCompute + 2) {
            // -lse and -delta of each query tile's rows; a row past the sequence or without
            // a key has -lse = -inf (its weights are 0) and delta 0
            for (int i = 0; i < n; ++i) {
                if (i >= 2) warp_wait(r_empty(i & 1), (i / 2 - 1) & 1, abort_flag);
                const int rows = rows_of(i);
                const long long at =
                    (static_cast<long long>(hk) * p.s.Tq + q0 + (i0 + i) * tpt) * G;
                float* dst = rowdata + (i & 1) * 256;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int r = u * 32 + lane;
                    dst[r] = r < rows ? p.row_lse[at + r] : -INFINITY;
                    dst[128 + r] = r < rows ? p.row_delta[at + r] : 0.f;
                }
                mbar_arrive(r_full(i & 1));
            }
        } else if (warp == kCompute && elect_one()) {
            constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0), id_g = idesc_bf16(128, DP, 0, 1);
            const uint64_t kdesc = desc_d(sK), vd = desc_d(sV);
            // S^T_i, once its queries are there (rows past them zeroed: dK sums over them)
            const auto scores = [&](int i) {
                const int s = i % C::R0;
                wait_phase(q_full(s), (i / C::R0) & 1, abort_flag);
                if (i + 1 == n && ragged) wait_phase(tail_bar, 0, abort_flag);
                tc_fence_after();
                const uint64_t bd = desc_d(sQ + s * C::TILE);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    mma_bf16(tmem + TM_S, kdesc + kd(k), bd + kd(k), id_s, k > 0);
                mma_commit(s_bar);
            };
            if (n > 0) {
                wait_phase(kv_bar, 0, abort_flag);
                scores(0);
            }
            for (int i = 0; i < n; ++i) {
                const int sd = i % C::R1, sq = i % C::R0;
                const uint64_t dod = desc_d(sDO + sd * C::TILE), dor = desc_r(sDO + sd * C::TILE);
                const uint64_t qr = desc_r(sQ + sq * C::TILE);
                const uint32_t add = i > 0;
                wait_phase(do_full(sd), (i / C::R1) & 1, abort_flag);
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    mma_bf16(tmem + TM_DP, vd + kd(k), dod + kd(k), id_s, k > 0);
                mma_commit(dp_bar);
                wait_phase(p_bar, i & 1, abort_flag);
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kRows / 16; ++k)
                    mma_bf16_ta(tmem + TM_DV, operand(tmem + TM_S, k), dor + kr(k), id_g,
                                k > 0 ? 1u : add);
                mma_commit(do_empty(sd));
                if (i + 1 < n) scores(i + 1);
                wait_phase(ds_bar, i & 1, abort_flag);
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kRows / 16; ++k)
                    mma_bf16_ta(tmem + TM_DK, operand(tmem + TM_DP, k), qr + kr(k), id_g,
                                k > 0 ? 1u : add);
                mma_commit(q_empty(sq));
            }
            mma_commit(done_bar);
            drain(done_bar, 0);
        } else if (warp < kCompute) {
            const int grp = warp >> 2, row = threadIdx.x & 127;
            const int key = kv0 + row;  // in its sequence
            const float c = p.scale * kLog2e;
            const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            for (int i = 0; i < n; ++i) {
                const float* rd = rowdata + (i & 1) * 256 + kCols * grp;
                // the first token of the tile that sees this key, as the first such column
                const int from = p.s.causal ? (key - (nk - nq) - (i0 + i) * tpt) * G - kCols * grp : 0;
                const bool diag = p.s.causal && kv0 + kRows - 1 - (nk - nq) > (i0 + i) * tpt;
                warp_wait(r_full(i & 1), (i >> 1) & 1, abort_flag);
                warp_wait(s_bar, i & 1, abort_flag);
                tc_fence_after();
                float s[kCols], d[kCols];
                load_cols(lanes + TM_S + kCols * grp, s);
#pragma unroll
                for (int q = 0; q < kCols; q += 4) {
                    const float4 e = *reinterpret_cast<const float4*>(rd + q);
                    fma2v(s[q], s[q + 1], c, e.x, e.y);
                    fma2v(s[q + 2], s[q + 3], c, e.z, e.w);
#pragma unroll
                    for (int u = 0; u < 4; ++u) s[q + u] = exp2_fast(s[q + u]);
                }
                if (diag) {
#pragma unroll
                    for (int q = 0; q < kCols; ++q) s[q] = q >= from ? s[q] : 0.f;
                }
                store_cols(lanes + TM_S + kCols * grp, s);
                warp_arrive(p_bar, lane);
                warp_wait(dp_bar, i & 1, abort_flag);
                tc_fence_after();
                load_cols(lanes + TM_DP + kCols * grp, d);
#pragma unroll
                for (int q = 0; q < kCols; q += 4) {
                    const float4 e = *reinterpret_cast<const float4*>(rd + 128 + q);
                    add2(d[q], d[q + 1], e.x, e.y);
                    add2(d[q + 2], d[q + 3], e.z, e.w);
                    mul2(d[q], d[q + 1], s[q], s[q + 1]);
                    mul2(d[q + 2], d[q + 3], s[q + 2], s[q + 3]);
                }
                if (diag) {
#pragma unroll
                    for (int q = 0; q < kCols; ++q) d[q] = q >= from ? d[q] : 0.f;
                }
                store_cols(lanes + TM_DP + kCols * grp, d);
                warp_arrive(ds_bar, lane);
                if (lane == 0) mbar_arrive(r_empty(i & 1));
            }
            if (n > 0) warp_wait(done_bar, 0, abort_flag);
            {
                tc_fence_after();
                // the first half of the groups: parts of dv; the others: of dk
                constexpr int PER = kGroups / 2, W = DP / PER;
                const bool is_v = grp < PER;
                const Heads& to = is_v ? p.dv : p.dk;
                store_rows<W>(lanes + (is_v ? TM_DV : TM_DK) + (grp % PER) * W, n > 0,
                              is_v ? 1.f : p.scale, smem + warp * 32 * W * 2, lane,
                              key < nk ? to.row(k0 + key, hk) : nullptr, (grp % PER) * W, p.a.D);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && *abort_flag) raise_timeout(p.err);
    if (warp == kCompute) tmem_dealloc(tmem, 512);
}

template <int DP>
cudaError_t backward(const Attention& p, cudaStream_t st) {
    using C = Cfg<DP>;
    const int G = p.a.Hq / p.a.Hkv, D = p.a.D, tpt = kRows / G;
    float* second = p.delta + static_cast<size_t>(p.s.Tq) * p.a.Hq;
    const Params prm{p.a, p.s, p.scale, p.out, p.dout, p.dq, p.dk, p.dv, p.lse, p.delta, second,
                     p.err, tpt, static_cast<int>(tile_bound(p.s.Tq, p.s.B, p.s.max_q, tpt))};
    CUtensorMap mq, md, mk, mv;
    if (p.s.Tq > 0 && (!make_tmap_heads(&mq, p.q, p.s.Tq, p.a.Hq, D, G, tpt) ||
                       !make_tmap_heads(&md, p.dout, p.s.Tq, p.a.Hq, D, G, tpt)))
        return cudaErrorInvalidValue;
    if (p.s.Tk > 0 && (!make_tmap_heads(&mk, p.k, p.s.Tk, p.a.Hkv, D, 1, kRows) ||
                       !make_tmap_heads(&mv, p.v, p.s.Tk, p.a.Hkv, D, 1, kRows)))
        return cudaErrorInvalidValue;
    // without queries or without keys no tile is loaded
    if (p.s.Tq == 0) mq = md = mk;
    if (p.s.Tk == 0) mk = mv = mq;
    const long long items = static_cast<long long>(prm.items) * p.a.Hkv;
    if (p.s.Tq > 0) {
        auto kfn = dq_kernel<DP>;
        cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             C::SMEM_Q);
        if (e != cudaSuccess) return e;
        LaunchScope ls("attention_dq", st);
        e = launch_pdl(kfn, dim3(static_cast<unsigned>(std::min<long long>(items, num_sms()))), dim3(kThreads), C::SMEM_Q, st,
                     mq, md, mk, mv, prm);
        if (e != cudaSuccess) return e;
    }
    if (p.s.Tk == 0) return cudaSuccess;
    const long long ki = tile_bound(p.s.Tk, p.s.B, p.s.max_k, kRows);
    auto kfn = dkv_kernel<DP>;
    const cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               C::SMEM_KV);
    if (e != cudaSuccess) return e;
    LaunchScope ls("attention_dkv", st);
    return launch_pdl(kfn, dim3(static_cast<unsigned>(ki * p.a.Hkv)), dim3(kThreads), C::SMEM_KV, st,
                    mq, md, mk, mv, prm);
}

}  // namespace

cudaError_t launch_attention_backward(const Attention& p, cudaStream_t st) {
    return p.a.D <= 64 ? backward<64>(p, st) : backward<128>(p, st);
}

}  // namespace attn
}  // namespace moe
