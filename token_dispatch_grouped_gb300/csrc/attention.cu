// attention.cu — softmax attention over packed sequences, forward.
//
//   S = q k^T,  lse = log sum_j exp(scale S_j),  P = exp(scale S - lse),  out = P v,
//
// in one pass over the keys per tile of queries: with the running maximum m and
// c = scale log2(e), weights p = 2^(c S - c m), sum l += sum p, O += p v, and O and l
// scaled by 2^(c m_old - c m_new) when m moves; out = O / l, lse = scale m + ln l.
//
// A CTA owns two tiles of 128 query rows of one key/value head. A tile's rows are the G
// query heads of 128 / G tokens (token-major), so grouped heads share every key and value
// tile that is loaded, and a short sequence still fills its tiles. Both tiles use each
// 128-key tile of K and V from shared memory. Roles:
//   warp 9     loads: Q once, then K and V tiles by TMA, two or three in flight of each;
//   warp 8     the tensor cores: S_x = Q_x K^T (both from shared memory) into TMEM,
//              O_x += P_x V with P_x as the TMEM operand;
//   warps 0-3  softmax of tile 0, warps 4-7 of tile 1, one row a thread: S_x to registers,
//              p as bf16 over S_x's first 64 TMEM columns, handed over in two halves so
//              that the first products run while the second half is formed.
// While one tile is in softmax the tensor cores run the other tile's products (1024 cycles
// at D = 128). A step lasts as long as one tile's chain of softmax, PV and the next S, so
// everything that the products do not wait for (the row sums) comes after the hand-over.
// Two threads a row (16 warps) measured slower (721 against 692 us for 16384 tokens, 16/4
// heads of 128): the exponentials of a tile share the same units, and more warps slow the
// issue of the products. TMEM: S_0, S_1 (128 columns each), O_0, O_1 (D each), fp32.
//
// m moves only when the new maximum exceeds it by 2^8 in weight (c (max - m) > 8): p stays
// at most 256, exact in the fp32 sum, and the pass over O in TMEM is rare after the first
// tiles. p is rounded to bf16 for the product (the operand type of the tensor cores, as v),
// l sums the unrounded p. Masks: a row's keys past its limit get S = -inf, by selection,
// so what those rows hold does not matter; rows of V past the last key of the CTA are
// zeroed in shared memory, since 0 * NaN would reach the sum.
#include "attn_mma.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = 320;

template <int DP>  // D padded to 64 or 128
struct Cfg {
    static constexpr int PIECES = DP / 64;
    static constexpr int TILE = PIECES * kPiece;
    static constexpr int KR = 3, VR = 2;  // tiles of K and V in shared memory
    static constexpr int TILES = (2 + KR + VR) * TILE;
    static constexpr int SMEM = TILES + 256;
    static constexpr uint32_t TM_S = 0, TM_O = 256;
};

struct Params {
    moe_attn_shape a;
    Packed s;
    float scale;
    Heads out;
    float* lse;
    int* err;
    int tpt;  // tokens of a 128-row tile
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
attention_forward_kernel(const __grid_constant__ CUtensorMap mapQ,
                         const __grid_constant__ CUtensorMap mapK,
                         const __grid_constant__ CUtensorMap mapV, const Params p) {
    using C = Cfg<DP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sQ = smem_u32(smem), sK = sQ + 2 * C::TILE, sV = sK + C::KR * C::TILE;
    uint8_t* misc = smem + C::TILES;
    const uint32_t bars = smem_u32(misc);
    const auto k_full = [&](int s) { return bars + 8u * s; };
    const auto v_full = [&](int s) { return bars + 8u * (3 + s); };
    const auto step = [&](int s) { return bars + 8u * (5 + s); };         // step j's products done
    const auto q_bar = [&](int x) { return bars + 8u * (7 + x); };
    const auto s_bar = [&](int x) { return bars + 8u * (9 + x); };        // S_x written
    const auto o_bar = [&](int x) { return bars + 8u * (11 + x); };       // O_x final
    const auto p_bar = [&](int x, int h) { return bars + 8u * (13 + 2 * x + h); };  // half of P_x
    const uint32_t done_bar = bars + 8u * 17, tail_bar = bars + 8u * 18;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 8 * 19);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    Work* found = reinterpret_cast<Work*>(tmem_slot + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 13; ++i) mbar_init(bars + 8 * i, 1);
        for (int i = 13; i < 17; ++i) mbar_init(bars + 8 * i, 4);  // the tile's warps
        mbar_init(done_bar, 1);
        mbar_init(tail_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    if (warp == 9 && lane == 0) {
        prefetch_tensormap(&mapQ);
        prefetch_tensormap(&mapK);
        prefetch_tensormap(&mapV);
    }
    pdl_wait();
    pdl_trigger();
    const int hk = blockIdx.x % p.a.Hkv, tpt = p.tpt, G = p.a.Hq / p.a.Hkv;
    if (warp == 0) {
        if ((sQ & 1023u) != 0) raise_error(p.err, MOE_ERR_MISALIGNED);  // the swizzle's unit
        const bool skip = has_error(p.err);
        Work w = find_work<false>(p.s, 2 * tpt, blockIdx.x / p.a.Hkv, lane, p.err);
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
        const int base = w.item * 2 * tpt;
        // keys that some row of a tile sees, and their tiles
        const auto limit_of = [&](int first) {
            const int last = min(first + tpt, nq) - 1;
            return last < first ? 0 : p.s.causal ? max(0, min(nk, last + 1 + nk - nq)) : nk;
        };
        const int limit0 = limit_of(base), limit1 = limit_of(base + tpt);
        const int tiles0 = (limit0 + kRows - 1) / kRows, tiles1 = (limit1 + kRows - 1) / kRows;
        const int n = max(tiles0, tiles1), seen = max(limit0, limit1);
        const bool ragged = seen % kRows != 0;  // the last V tile has rows past the keys

        if (warp == 9) {
            // ------------------------------------------------------------ loads
            if (lane == 0) {
                const auto load = [&](uint32_t dst, const CUtensorMap* m, uint32_t bar, int h, int t) {
                    for (int c = 0; c < C::PIECES; ++c)
                        tma_load_3d(dst + c * kPiece, m, bar, 64 * c, h, t);
                };
                const uint32_t qbytes = C::PIECES * 128 * G * tpt;
                int jk = 0, jv = 0;
                const auto load_q = [&](int x) {
                    mbar_arrive_expect_tx(q_bar(x), qbytes);
                    load(sQ + x * C::TILE, &mapQ, q_bar(x), hk * G, q0 + base + x * tpt);
                };
                const auto load_k = [&](int j) {
                    mbar_arrive_expect_tx(k_full(j % C::KR), C::TILE);
                    load(sK + j % C::KR * C::TILE, &mapK, k_full(j % C::KR), hk, k0 + j * kRows);
                    ++jk;
                };
                if (tiles0 > 0) load_q(0);
                if (n > 0) load_k(0);
                if (tiles1 > 0) load_q(1);
                for (int j = 0; j < n; ++j) {
                    // step j - 2 is the last that reads V_{j-2}; K_{j-2} was read before it
                    if (j >= 2) wait_phase(step(j & 1), (j / 2 - 1) & 1, abort_flag);
                    if (*abort_flag) break;
                    mbar_arrive_expect_tx(v_full(j & 1), C::TILE);
                    load(sV + (j & 1) * C::TILE, &mapV, v_full(j & 1), hk, k0 + j * kRows);
                    ++jv;
                    if (j + 1 < n) load_k(j + 1);
                }
                // nothing is in flight when the CTA leaves
                if (tiles0 > 0) drain(q_bar(0), 0);
                if (tiles1 > 0) drain(q_bar(1), 0);
                for (int j = max(0, jk - C::KR); j < jk; ++j) drain(k_full(j % C::KR), (j / C::KR) & 1);
                for (int j = max(0, jv - C::VR); j < jv; ++j) drain(v_full(j & 1), (j >> 1) & 1);
            }
            __syncwarp();
            if (ragged) {
                // the last V tile has landed (or the CTA has given up)
                zero_tail(sV + ((n - 1) & 1) * C::TILE, C::PIECES, seen % kRows, lane);
                if (lane == 0) mbar_arrive(tail_bar);
            }
        } else if (warp == 8) {
            // ----------------------------------------------------- tensor cores
            constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, DP, 0, 1);
            const auto scores = [&](int x, int j) {
                const uint64_t ad = desc_d(sQ + x * C::TILE), bd = desc_d(sK + j % C::KR * C::TILE);
                const uint32_t dst = tmem + C::TM_S + 128 * x, bar = s_bar(x);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) mma_bf16(dst, ad + kd(k), bd + kd(k), id_s, k > 0);
                    mma_commit(bar);
                }
                __syncwarp();
            };
            if (n > 0) warp_wait(k_full(0), 0, abort_flag);
            if (tiles0 > 0) {
                warp_wait(q_bar(0), 0, abort_flag);
                tc_fence_after();
                scores(0, 0);
            }
            if (tiles1 > 0) {
                warp_wait(q_bar(1), 0, abort_flag);
                tc_fence_after();
                scores(1, 0);
            }
            for (int j = 0; j < n; ++j) {
                warp_wait(v_full(j & 1), (j >> 1) & 1, abort_flag);
                if (j + 1 < n) warp_wait(k_full((j + 1) % C::KR), ((j + 1) / C::KR) & 1, abort_flag);
                else if (ragged) warp_wait(tail_bar, 0, abort_flag);
                const uint64_t vd = desc_r(sV + (j & 1) * C::TILE);
                const uint32_t add = j > 0;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int tiles = x == 0 ? tiles0 : tiles1;
                    if (j >= tiles) continue;
                    const uint32_t dst = tmem + C::TM_O + DP * x, src = tmem + C::TM_S + 128 * x;
                    const uint32_t bar = o_bar(x);
                    const bool last = j + 1 == tiles;
                    warp_wait(p_bar(x, 0), j & 1, abort_flag);
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16_ta(dst, src + 8 * k, vd + kr(k), id_o, k > 0 ? 1u : add);
                    }
                    __syncwarp();
                    warp_wait(p_bar(x, 1), j & 1, abort_flag);
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 4; k < 8; ++k) mma_bf16_ta(dst, src + 8 * k, vd + kr(k), id_o, 1u);
                        if (last) mma_commit(bar);
                    }
                    __syncwarp();
                    if (!last) scores(x, j + 1);
                }
                const uint32_t bar = step(j & 1);
                if (elect_one()) mma_commit(bar);
                __syncwarp();
            }
            if (elect_one()) mma_commit(done_bar);
            __syncwarp();
            drain(done_bar, 0);
            __syncwarp();
        } else {
            // ---------------------------------------------------------- softmax
            const int x = warp >> 2;
            const int row = threadIdx.x & 127, head = row % G;
            const int first = base + x * tpt, token = first + row / G;  // in the sequence
            const int tiles = x == 0 ? tiles0 : tiles1;
            const bool valid = row < G * tpt && token < nq;
            const int mine = !valid ? 0 : p.s.causal ? min(nk, token + 1 + nk - nq) : nk;
            // every row of the tile sees the keys before this one
            const int open = p.s.causal ? first + 1 + nk - nq : nk;
            const float c = p.scale * 1.44269504088896341f;
            const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            const uint32_t tS = lanes + C::TM_S + 128 * x, tO = lanes + C::TM_O + DP * x;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < tiles; ++j) {
                warp_wait(s_bar(x), j & 1, abort_flag);
                tc_fence_after();
                float s[128];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    tmem_ld32(tS + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * q));
                tmem_ld_wait();
                if ((j + 1) * kRows > open) {
                    const int lim = mine - j * kRows;
#pragma unroll
                    for (int i = 0; i < 128; ++i) s[i] = i < lim ? s[i] : -INFINITY;
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int i = 4; i < 124; i += 8)
#pragma unroll
                    for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], s[i + 2 * u], s[i + 2 * u + 1]);
                const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], s[124], s[125]),
                                       fmaxf(s[126], s[127]));
                if (j == 0) {
                    m = top;
                } else if (__any_sync(~0u, (top - m) * c > 8.f)) {
                    const float mn = fmaxf(m, top);
                    const float keep = m == -INFINITY ? 0.f : exp2_fast((m - mn) * c);
                    m = mn;
                    l *= keep;
#pragma unroll 1
                    for (int q = 0; q < DP; q += 16) {
                        uint32_t o[16];
                        tmem_ld16(tO + q, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                        tmem_st16(tO + q, o);
                    }
                }
                const float shift = m == -INFINITY ? 0.f : -m * c;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int q = 64 * h; q < 64 * h + 64; q += 32) {
                        uint32_t o[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            fma2v(s[q + i], s[q + i + 1], c, shift, shift);
                            s[q + i] = exp2_fast(s[q + i]);
                            s[q + i + 1] = exp2_fast(s[q + i + 1]);
                            o[i / 2] = pack2(s[q + i], s[q + i + 1]);
                        }
                        tmem_st16(tS + q / 2, o);
                    }
                    tmem_st_wait();
                    warp_arrive(p_bar(x, h), lane);
                }
                float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
                for (int i = 0; i < 128; i += 4) {
                    add2(s0, s1, s[i], s[i + 1]);
                    add2(s2, s3, s[i + 2], s[i + 3]);
                }
                l += (s0 + s1) + (s2 + s3);
            }
            if (tiles > 0) warp_wait(o_bar(x), 0, abort_flag);
            if (first < nq) {
                tc_fence_after();
                const long long t = q0 + token;
                const int h = hk * G + head;
                if (valid)
                    p.lse[t * p.a.Hq + h] = l == 0.f ? -INFINITY : fmaf(m, p.scale, logf(l));
                // The rows leave through Q_x, all reads of which are done.
                store_rows<DP>(tO, tiles > 0, l == 0.f ? 0.f : 1.f / l,
                               smem + x * C::TILE + (warp & 3) * 32 * DP * 2, lane,
                               valid ? p.out.row(t, h) : nullptr, 0, p.a.D);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && *abort_flag) raise_error(p.err, MOE_ERR_TIMEOUT);
    if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int DP>
cudaError_t forward(const Attention& p, cudaStream_t st) {
    using C = Cfg<DP>;
    const int G = p.a.Hq / p.a.Hkv, D = p.a.D;
    Params prm{p.a, p.s, p.scale, p.out, p.lse, p.err, kRows / G};
    CUtensorMap mq, mk, mv;
    if (!make_tmap_heads(&mq, p.q, p.s.Tq, p.a.Hq, D, G, prm.tpt)) return cudaErrorInvalidValue;
    mk = mv = mq;  // without keys no tile is loaded
    if (p.s.Tk > 0 && (!make_tmap_heads(&mk, p.k, p.s.Tk, p.a.Hkv, D, 1, kRows) ||
                       !make_tmap_heads(&mv, p.v, p.s.Tk, p.a.Hkv, D, 1, kRows)))
        return cudaErrorInvalidValue;
    const long long items = tile_bound(p.s.Tq, p.s.B, p.s.max_q, 2 * prm.tpt);
    if (items == 0) return cudaSuccess;
    auto kfn = attention_forward_kernel<DP>;
    cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    LaunchScope ls("attention_forward", st);
    return launch_pdl(kfn, dim3(static_cast<unsigned>(items * p.a.Hkv)), dim3(kThreads), C::SMEM, st,
                    mq, mk, mv, prm);
}

}  // namespace

cudaError_t launch_attention_forward(const Attention& p, cudaStream_t st) {
    return p.a.D <= 64 ? forward<64>(p, st) : forward<128>(p, st);
}

}  // namespace attn
}  // namespace moe
