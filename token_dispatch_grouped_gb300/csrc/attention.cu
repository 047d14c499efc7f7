// attention.cu — softmax attention over packed sequences, forward.
//
//   S = q k^T,  lse = log sum_j exp(scale S_j),  P = exp(scale S - lse),  out = P v,
//
// in one pass over the keys per tile of queries: with the running maximum m and
// c = scale log2(e), weights p = 2^(c S - c m), sum l += sum p, O += p v, and O and l
// scaled by 2^(c m_old - c m_new) when m moves; out = O / l, lse = scale m + ln l.
//
// A CTA (one per SM) walks items of work, most steps first, dealt in snake order (dealt in
// one direction the first CTA of 16384 tokens had 15% more steps than the mean); an item
// is two tiles of 128 query rows of one key/value head. A tile's rows are the G
// query heads of 128 / G tokens (token-major), so grouped heads share every key and value
// tile that is loaded, and a short sequence still fills its tiles. Both tiles use each
// 128-key tile of K and V from shared memory. Roles:
//   warp 10    finds the next item while the others work on the last one (a CTA per item
//              spent 7.6 us outside its steps: 53 us for the packed batch of 4096 tokens
//              against 45);
//   warp 9     loads: Q, then K and V tiles by TMA, into the next item as tiles fall free;
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
#include <algorithm>

#include "attn_mma.cuh"

namespace moe {
namespace attn {
namespace {

// Three groups of four warps; the third (warp 11 idle) gives registers to the
// softmax warps, which hold a row of 128 scores each: 256 * 200 + 128 * 104 = 384 * 168.
constexpr int kThreads = 384;
constexpr int kSoftRegs = 200, kOtherRegs = 104;

template <int DP>  // D padded to 64 or 128
struct Cfg {
    static constexpr int PIECES = DP / 64;
    static constexpr int TILE = PIECES * kPiece;
    static constexpr int KR = 3, VR = 2;  // tiles of K and V in shared memory
    static constexpr int TILES = (2 + KR + VR) * TILE;
    static constexpr int SMEM = TILES + 512;
    static constexpr uint32_t TM_S = 0, TM_O = 256;
};

struct Params {
    moe_attn_shape a;
    Packed s;
    float scale;
    Heads out;
    float* lse;
    int* err;
    int tpt;    // tokens of a 128-row tile
    int items;  // upper bound of the work items of a head
};

// One item: two query tiles of a key/value head, and the key tiles that they see.
struct Item {
    int q0, nq, k0, nk;
    int base, hk;           // first token (in the sequence), key/value head (-1: no more work)
    int tiles0, tiles1;     // key tiles that some row of each query tile sees
    int steps, seen;        // the larger of them; keys that some row sees
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
    // Phases run on through all items of a CTA: steps are counted from its first item on
    // (K and V tiles, step), tiles of scores per query tile (s, p), items per query tile
    // that have any (q, q_free, o, o_free).
    const auto k_full = [&](int s) { return bars + 8u * s; };
    const auto v_full = [&](int s) { return bars + 8u * (3 + s); };
    const auto step = [&](int s) { return bars + 8u * (5 + s); };      // a step's products done
    const auto q_full = [&](int x) { return bars + 8u * (7 + x); };
    const auto q_free = [&](int x) { return bars + 8u * (9 + x); };    // Q_x read for the last time
    const auto s_bar = [&](int x) { return bars + 8u * (11 + x); };    // S_x written
    const auto o_bar = [&](int x) { return bars + 8u * (13 + x); };    // O_x final
    const auto w_full = [&](int s) { return bars + 8u * (15 + s); };   // an item is in its slot
    const uint32_t done_bar = bars + 8u * 17;
    const auto p_bar = [&](int x, int h) { return bars + 8u * (19 + 2 * x + h); };  // half of P_x
    const auto o_free = [&](int x) { return bars + 8u * (23 + x); };   // O_x read
    const auto w_free = [&](int s) { return bars + 8u * (25 + s); };   // its slot read
    const auto tail_bar = [&](int s) { return bars + 8u * (27 + s); };  // V's slot zeroed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 8 * 29);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    Item* ring = reinterpret_cast<Item*>(misc + 8 * 30);  // two slots

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 18; ++i) mbar_init(bars + 8 * i, 1);
        mbar_init(tail_bar(0), 1);
        mbar_init(tail_bar(1), 1);
        for (int i = 19; i < 25; ++i) mbar_init(bars + 8 * i, 4);  // the tile's warps
        for (int i = 25; i < 27; ++i) mbar_init(bars + 8 * i, 10);  // warps 0 to 9
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    const int tpt = p.tpt, G = p.a.Hq / p.a.Hkv;
    // Item i of this CTA, for those that only read them (false: no more work), and its
    // slot given back by a warp.
    const auto item_there = [&](int i) -> bool {
        wait_phase(w_full(i & 1), (i >> 1) & 1, abort_flag);
        return ring[i & 1].hk >= 0 && *abort_flag == 0;
    };
    const auto item_done = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(w_free(i & 1));
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 10) {
            // ----------------------------------------- items, one ahead of the others
            const bool off = (sQ & 1023u) != 0;  // the swizzle's unit
            if (off) raise_error(p.err, MOE_ERR_MISALIGNED);
            const bool skip = __any_sync(~0u, off || stopped(p.err));
            for (int i = 0;; ++i) {
                // snake order: forwards through the CTAs, then backwards
                const int index = i * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                Item it{};
                it.hk = -1;
                if (index < p.items * p.a.Hkv) {
                    const Work w = find_work<false>(p.s, 2 * tpt, index / p.a.Hkv, lane, p.err);
                    it.q0 = w.q0, it.nq = w.nq, it.k0 = w.k0, it.nk = w.nk;
                    it.base = w.item * 2 * tpt;
                    if (w.items > 0 && !skip) it.hk = index % p.a.Hkv;
                    const auto limit_of = [&](int first) {  // keys that some row of a tile sees
                        const int last = min(first + tpt, it.nq) - 1;
                        return last < first ? 0
                               : p.s.causal ? max(0, min(it.nk, last + 1 + it.nk - it.nq))
                                            : it.nk;
                    };
                    const int limit0 = limit_of(it.base), limit1 = limit_of(it.base + tpt);
                    it.tiles0 = (limit0 + kRows - 1) / kRows;
                    it.tiles1 = (limit1 + kRows - 1) / kRows;
                    it.steps = max(it.tiles0, it.tiles1);
                    it.seen = max(limit0, limit1);
                }
                if (i >= 2) warp_wait(w_free(i & 1), (i / 2 - 1) & 1, abort_flag);
                if (lane == 0) {
                    ring[i & 1] = it;
                    mbar_arrive(w_full(i & 1));
                }
                if (__any_sync(~0u, it.hk < 0 || *abort_flag != 0)) break;
            }
            if (blockIdx.x == 0) check_sequences(p.s, lane, p.err);
        } else if (warp == 9) {
            // ---------------------------------------------------------------- loads
            const auto load = [&](uint32_t dst, const CUtensorMap* m, uint32_t bar, int h, int t) {
                for (int c = 0; c < C::PIECES; ++c)
                    tma_load_3d(dst + c * kPiece, m, bar, 64 * c, h, t);
            };
            const uint32_t qbytes = C::PIECES * 128 * G * tpt;
            int g = 0, kg = 0, qg0 = 0, qg1 = 0;  // steps, K tiles, Q tiles loaded so far
            for (int i = 0; __all_sync(~0u, item_there(i)); ++i) {
                const Item it = ring[i & 1];
                item_done(i);
                if (lane == 0) {
                    const auto load_q = [&](int x, int& count) {
                        if (count > 0) wait_phase(q_free(x), (count - 1) & 1, abort_flag);
                        if (*abort_flag) return;
                        ++count;
                        mbar_arrive_expect_tx(q_full(x), qbytes);
                        load(sQ + x * C::TILE, &mapQ, q_full(x), it.hk * G, it.q0 + it.base + x * tpt);
                    };
                    const auto load_k = [&](int j) {
                        mbar_arrive_expect_tx(k_full(kg % C::KR), C::TILE);
                        load(sK + kg % C::KR * C::TILE, &mapK, k_full(kg % C::KR), it.hk,
                             it.k0 + j * kRows);
                        ++kg;
                    };
                    // K tile g is loaded when step g - 3 is done: it was waited for at step g - 1
                    if (it.steps > 0 && *abort_flag == 0) load_k(0);
                    if (it.tiles0 > 0) load_q(0, qg0);
                    if (it.tiles1 > 0) load_q(1, qg1);
                    for (int j = 0; j < it.steps; ++j) {
                        // step g - 2 is the last that reads V tile g - 2; K tile g - 2 was read
                        // before it
                        if (g >= 2) wait_phase(step(g & 1), (g / 2 - 1) & 1, abort_flag);
                        if (*abort_flag) break;
                        mbar_arrive_expect_tx(v_full(g & 1), C::TILE);
                        load(sV + (g & 1) * C::TILE, &mapV, v_full(g & 1), it.hk, it.k0 + j * kRows);
                        ++g;
                        if (j + 1 < it.steps) load_k(j + 1);
                    }
                }
                __syncwarp();
                if (it.seen % kRows != 0) {  // the last V tile has rows past the keys
                    const int last = __shfl_sync(~0u, g, 0) - 1;
                    if (last >= 0) {
                        warp_wait(v_full(last & 1), (last >> 1) & 1, abort_flag);
                        zero_tail(sV + (last & 1) * C::TILE, C::PIECES, it.seen % kRows, lane);
                    }
                    if (lane == 0) mbar_arrive(tail_bar(last & 1));
                }
            }
            if (lane == 0) {  // nothing is in flight when the CTA leaves
                if (qg0 > 0) drain(q_full(0), (qg0 - 1) & 1);
                if (qg1 > 0) drain(q_full(1), (qg1 - 1) & 1);
                for (int j = max(0, kg - C::KR); j < kg; ++j) drain(k_full(j % C::KR), (j / C::KR) & 1);
                for (int j = max(0, g - C::VR); j < g; ++j) drain(v_full(j & 1), (j >> 1) & 1);
            }
            __syncwarp();
        } else if (warp == 8 && elect_one()) {
            // ----------------------------------------------- tensor cores (one thread)
            constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, DP, 0, 1);
            int g = 0, had0 = 0, had1 = 0, ps0 = 0, ps1 = 0;  // see the phases above
            uint32_t tails = 0;  // the phase of each slot's next tail
            const auto scores = [&](int x, int kt, bool last) {
                const uint64_t ad = desc_d(sQ + x * C::TILE), bd = desc_d(sK + kt % C::KR * C::TILE);
                const uint32_t dst = tmem + C::TM_S + 128 * x;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) mma_bf16(dst, ad + kd(k), bd + kd(k), id_s, k > 0);
                mma_commit(s_bar(x));
                if (last) mma_commit(q_free(x));
            };
            for (int i = 0; item_there(i); ++i) {
                const Item& it = ring[i & 1];
                const int n = it.steps, tiles0 = it.tiles0, tiles1 = it.tiles1;
                const bool ragged = it.seen % kRows != 0;
                mbar_arrive(w_free(i & 1));
                if (n > 0) wait_phase(k_full(g % C::KR), (g / C::KR) & 1, abort_flag);
                if (tiles0 > 0) {
                    wait_phase(q_full(0), had0 & 1, abort_flag);
                    tc_fence_after();
                    scores(0, g, tiles0 == 1);
                }
                if (tiles1 > 0) {
                    wait_phase(q_full(1), had1 & 1, abort_flag);
                    tc_fence_after();
                    scores(1, g, tiles1 == 1);
                }
                for (int j = 0; j < n; ++j, ++g) {
                    wait_phase(v_full(g & 1), (g >> 1) & 1, abort_flag);
                    if (j + 1 < n) {
                        wait_phase(k_full((g + 1) % C::KR), ((g + 1) / C::KR) & 1, abort_flag);
                    } else if (ragged) {
                        // (a V slot is not loaded again before its step is done, so no
                        // phase of its tail is passed)
                        wait_phase(tail_bar(g & 1), tails >> (g & 1) & 1, abort_flag);
                        tails ^= 1 << (g & 1);
                    }
                    const uint64_t vd = desc_r(sV + (g & 1) * C::TILE);
                    const uint32_t add = j > 0;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int tiles = x == 0 ? tiles0 : tiles1;
                        if (j >= tiles) continue;
                        const int ps = x == 0 ? ps0 : ps1;
                        const int had = x == 0 ? had0 : had1;
                        const uint32_t dst = tmem + C::TM_O + DP * x, src = tmem + C::TM_S + 128 * x;
                        const bool last = j + 1 == tiles;
                        // the last item's O_x has been read
                        if (j == 0 && had > 0) wait_phase(o_free(x), (had - 1) & 1, abort_flag);
                        wait_phase(p_bar(x, 0), ps & 1, abort_flag);
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16_ta(dst, src + 8 * k, vd + kr(k), id_o, k > 0 ? 1u : add);
                        wait_phase(p_bar(x, 1), ps & 1, abort_flag);
                        tc_fence_after();
#pragma unroll
                        for (int k = 4; k < 8; ++k)
                            mma_bf16_ta(dst, src + 8 * k, vd + kr(k), id_o, 1u);
                        if (x == 0) ++ps0;
                        else ++ps1;
                        if (last) mma_commit(o_bar(x));
                        else scores(x, g + 1, j + 2 == tiles);
                    }
                    mma_commit(step(g & 1));
                }
                had0 += tiles0 > 0;
                had1 += tiles1 > 0;
            }
            mma_commit(done_bar);
            drain(done_bar, 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // -------------------------------------------------------------- softmax
        const int x = warp >> 2;
        const int row = threadIdx.x & 127, head = row % G, rtok = row / G;
        const float c = p.scale * 1.44269504088896341f;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t tS = lanes + C::TM_S + 128 * x, tO = lanes + C::TM_O + DP * x;
        int ps = 0, had = 0;
        for (int i = 0; __all_sync(~0u, item_there(i)); ++i) {
            const Item& it = ring[i & 1];
            const int tiles = x == 0 ? it.tiles0 : it.tiles1;
            int mine, open;  // keys that this row sees, and that every row of the tile sees
            {
                const int first = it.base + x * tpt, more = it.nk - it.nq;
                const bool valid = row < G * tpt && first + rtok < it.nq;
                mine = !valid ? 0 : p.s.causal ? min(it.nk, first + rtok + 1 + more) : it.nk;
                open = p.s.causal ? first + 1 + more : it.nk;
            }
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < tiles; ++j, ++ps) {
                warp_wait(s_bar(x), ps & 1, abort_flag);
                tc_fence_after();
                float s[128];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    tmem_ld32(tS + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * q));
                tmem_ld_wait();
                if ((j + 1) * kRows > open) {
                    const int lim = mine - j * kRows;
#pragma unroll
                    for (int e = 0; e < 128; ++e) s[e] = e < lim ? s[e] : -INFINITY;
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int e = 4; e < 124; e += 8)
#pragma unroll
                    for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], s[e + 2 * u], s[e + 2 * u + 1]);
                // (a row that sees no key may hold anything, and has no say in the vote below:
                // m moves in all rows of the warp, and with it how their p is rounded)
                const float top = mine <= 0 ? -INFINITY
                                            : max3(max3(mx[0], mx[1], mx[2]),
                                                   max3(mx[3], s[124], s[125]),
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
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
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
                        for (int e = 0; e < 32; e += 2) {
                            fma2v(s[q + e], s[q + e + 1], c, shift, shift);
                            s[q + e] = exp2_fast(s[q + e]);
                            s[q + e + 1] = exp2_fast(s[q + e + 1]);
                            o[e / 2] = pack2(s[q + e], s[q + e + 1]);
                        }
                        tmem_st16(tS + q / 2, o);
                    }
                    tmem_st_wait();
                    warp_arrive(p_bar(x, h), lane);
                }
                float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
                for (int e = 0; e < 128; e += 4) {
                    add2(s0, s1, s[e], s[e + 1]);
                    add2(s2, s3, s[e + 2], s[e + 3]);
                }
                l += (s0 + s1) + (s2 + s3);
            }
            const int token = it.base + x * tpt + rtok, h = it.hk * G + head;
            const bool valid = row < G * tpt && token < it.nq;
            const long long t = it.q0 + token;
            item_done(i);
            if (valid)
                p.lse[t * p.a.Hq + h] = l == 0.f ? -INFINITY : fmaf(m, p.scale, logf(l));
            const float inv = l == 0.f ? 0.f : 1.f / l;
            bf16* dst = p.out.row(t, h);
            if (tiles > 0) {
                warp_wait(o_bar(x), had & 1, abort_flag);
                ++had;
                tc_fence_after();
            }
#pragma unroll 1
            for (int q = 0; q < DP; q += 32) {
                uint32_t o[32];
                if (tiles > 0) {
                    tmem_ld32(tO + q, o);
                    tmem_ld_wait();
                    if (q + 32 == DP) warp_arrive(o_free(x), lane);
                }
                if (valid) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float v[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            v[u] = tiles > 0 && l != 0.f ? __uint_as_float(o[e + u]) * inv : 0.f;
                        if (q + e < p.a.D) *reinterpret_cast<uint4*>(dst + q + e) = pack8(v);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && *abort_flag) raise_timeout(p.err);
    if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int DP>
cudaError_t forward(const Attention& p, cudaStream_t st) {
    using C = Cfg<DP>;
    const int G = p.a.Hq / p.a.Hkv, D = p.a.D, tpt = kRows / G;
    const long long items = tile_bound(p.s.Tq, p.s.B, p.s.max_q, 2 * tpt);
    Params prm{p.a, p.s, p.scale, p.out, p.lse, p.err, tpt, static_cast<int>(items)};
    CUtensorMap mq, mk, mv;
    if (!make_tmap_heads(&mq, p.q, p.s.Tq, p.a.Hq, D, G, tpt)) return cudaErrorInvalidValue;
    mk = mv = mq;  // without keys no tile is loaded
    if (p.s.Tk > 0 && (!make_tmap_heads(&mk, p.k, p.s.Tk, p.a.Hkv, D, 1, kRows) ||
                       !make_tmap_heads(&mv, p.v, p.s.Tk, p.a.Hkv, D, 1, kRows)))
        return cudaErrorInvalidValue;
    auto kfn = attention_forward_kernel<DP>;
    cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const long long ctas = std::min<long long>(items * p.a.Hkv, num_sms());
    LaunchScope ls("attention_forward", st);
    return launch_pdl(kfn, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), C::SMEM, st, mq, mk, mv,
                      prm);
}

}  // namespace

cudaError_t launch_attention_forward(const Attention& p, cudaStream_t st) {
    return p.a.D <= 64 ? forward<64>(p, st) : forward<128>(p, st);
}

}  // namespace attn
}  // namespace moe
