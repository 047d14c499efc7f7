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
//   warp 9     loads: Q once, then K and V tiles by TMA into a ring of stages;
//   warp 8     the tensor cores: S_x = Q_x K^T (both from shared memory) into TMEM,
//              O_x += P_x V with P_x as the TMEM operand;
//   warps 0-3  softmax of tile 0, warps 4-7 of tile 1, one row a thread: S_x to registers,
//              p as bf16 over S_x's first 64 TMEM columns.
// While one tile is in softmax the tensor cores run the other tile's products. TMEM:
// S_0, S_1 (128 columns each), O_0, O_1 (D each), fp32.
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
    static constexpr int STAGES = DP == 128 ? 5 : 8;
    static constexpr int SMEM = 1024 + 2 * TILE + STAGES * TILE + 256;
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
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t sQ = base, sKV = base + 2 * C::TILE;
    uint8_t* misc = smem_raw + (base - raw) + (2 + C::STAGES) * C::TILE;
    const uint32_t bars = smem_u32(misc);
    const auto full = [&](int s) { return bars + 8u * s; };
    const auto empty = [&](int s) { return bars + 8u * (C::STAGES + s); };
    const auto q_bar = [&](int x) { return bars + 8u * (2 * C::STAGES + x); };
    const auto s_bar = [&](int x) { return bars + 8u * (2 * C::STAGES + 2 + x); };  // S_x written
    const auto p_bar = [&](int x) { return bars + 8u * (2 * C::STAGES + 4 + x); };  // P_x written
    const auto o_bar = [&](int x) { return bars + 8u * (2 * C::STAGES + 6 + x); };  // O_x final
    const uint32_t done_bar = bars + 8u * (2 * C::STAGES + 8);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 8 * (2 * C::STAGES + 9));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* found = reinterpret_cast<int*>(tmem_slot + 2);  // sequence (-1: none), item

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(q_bar(x), 1);
            mbar_init(s_bar(x), 1);
            mbar_init(p_bar(x), kRows);
            mbar_init(o_bar(x), 1);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    const int hk = blockIdx.y, tpt = p.tpt, G = p.a.Hq / p.a.Hkv;
    if (warp == 0) {
        int b = -1, item = 0, items = 0;
        const bool skip = __any_sync(~0u, has_error(p.err));
        if (skip || !find_tile(p.s, false, 2 * tpt, blockIdx.x, lane, b, item, items, p.err)) b = -1;
        if (lane == 0) {
            found[0] = b;
            found[1] = items - 1 - item;  // the longest rows of a sequence first
        }
    }
    if (warp == 1 && blockIdx.x == 0 && hk == 0) check_sequences(p.s, lane, p.err);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int b = found[0];
    if (b >= 0) {
        const int q0 = p.s.cu_q[b], nq = p.s.cu_q[b + 1] - q0;
        const int k0 = p.s.cu_k[b], nk = p.s.cu_k[b + 1] - k0;
        const int first[2] = {found[1] * 2 * tpt, found[1] * 2 * tpt + tpt};
        // keys that some row of tile x sees, and their tiles
        int limit[2], tiles[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int last = min(first[x] + tpt, nq) - 1;
            limit[x] = last < first[x] ? 0 : p.s.causal ? max(0, min(nk, last + 1 + nk - nq)) : nk;
            tiles[x] = (limit[x] + kRows - 1) / kRows;
        }
        const int n = max(tiles[0], tiles[1]);
        const int seen = max(limit[0], limit[1]);

        if (warp == 9) {
            // ------------------------------------------------------------ loads
            if (lane == 0 && n > 0) {
                for (int x = 0; x < 2; ++x) {
                    if (tiles[x] == 0) continue;
                    mbar_arrive_expect_tx(q_bar(x), C::PIECES * 128 * G * tpt);
                    for (int c = 0; c < C::PIECES; ++c)
                        tma_load_3d(sQ + x * C::TILE + c * kPiece, &mapQ, q_bar(x), 64 * c, hk * G,
                                    q0 + first[x]);
                }
                int i = 0;
                for (; i < 2 * n; ++i) {  // K and V tiles in turn
                    const int slot = i % C::STAGES;
                    if (i >= C::STAGES &&
                        !wait_phase(empty(slot), (i / C::STAGES - 1) & 1, abort_flag))
                        break;
                    mbar_arrive_expect_tx(full(slot), C::TILE);
                    for (int c = 0; c < C::PIECES; ++c)
                        tma_load_3d(sKV + slot * C::TILE + c * kPiece, (i & 1) ? &mapV : &mapK,
                                    full(slot), 64 * c, hk, k0 + (i >> 1) * kRows);
                }
                // nothing is in flight when the CTA leaves
                for (int x = 0; x < 2; ++x)
                    if (tiles[x] > 0) drain(q_bar(x), 0);
                for (int j = max(0, i - C::STAGES); j < i; ++j)
                    drain(full(j % C::STAGES), (j / C::STAGES) & 1);
            }
        } else if (warp == 8) {
            // ----------------------------------------------------- tensor cores
            constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, DP, 0, 1);
            const auto scores = [&](int x, int slot) {
                const uint64_t ad = desc_d(sQ + x * C::TILE), bd = desc_d(sKV + slot * C::TILE);
                const uint32_t dst = tmem + C::TM_S + 128 * x, bar = s_bar(x);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) mma_bf16(dst, ad + kd(k), bd + kd(k), id_s, k > 0);
                    mma_commit(bar);
                }
                __syncwarp();
            };
            bool ok = n == 0 || warp_wait(full(0), 0, abort_flag);
            tc_fence_after();
            for (int x = 0; x < 2 && ok; ++x)
                if (tiles[x] > 0) {
                    ok = warp_wait(q_bar(x), 0, abort_flag);
                    if (ok) scores(x, 0);
                }
            if (ok && n > 0 && elect_one()) mma_commit(empty(0));
            __syncwarp();
            for (int j = 0; j < n && ok; ++j) {
                const int iv = 2 * j + 1, ik = 2 * j + 2;
                const int sv = iv % C::STAGES, sk = ik % C::STAGES;
                ok = warp_wait(full(sv), (iv / C::STAGES) & 1, abort_flag);
                if (ok && j + 1 < n) ok = warp_wait(full(sk), (ik / C::STAGES) & 1, abort_flag);
                if (!ok) break;
                if (seen - j * kRows < kRows)
                    zero_tail(sKV + sv * C::TILE, C::PIECES, seen - j * kRows, lane);
                for (int x = 0; x < 2 && ok; ++x) {
                    if (j >= tiles[x]) continue;
                    ok = warp_wait(p_bar(x), j & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vd = desc_r(sKV + sv * C::TILE);
                    const uint32_t dst = tmem + C::TM_O + DP * x, src = tmem + C::TM_S + 128 * x;
                    const uint32_t add = j > 0, bar = o_bar(x);
                    const bool last = j + 1 == tiles[x];
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kRows / 16; ++k)
                            mma_bf16_ta(dst, src + 8 * k, vd + kr(k), id_o, k > 0 ? 1u : add);
                        if (last) mma_commit(bar);
                    }
                    __syncwarp();
                    if (j + 1 < tiles[x]) scores(x, sk);
                }
                if (!ok) break;
                const uint32_t ev = empty(sv), ek = empty(sk);
                const bool more = j + 1 < n;
                if (elect_one()) {
                    mma_commit(ev);
                    if (more) mma_commit(ek);
                }
                __syncwarp();
            }
            if (elect_one()) mma_commit(done_bar);
            __syncwarp();
            drain(done_bar, 0);
            __syncwarp();
        } else {
            // ---------------------------------------------------------- softmax
            const int x = warp >> 2;
            const int row = threadIdx.x & 127;
            const int token = first[x] + row / G;  // in its sequence
            const bool valid = row < G * tpt && token < nq;
            const int mine = !valid ? 0 : p.s.causal ? min(nk, token + 1 + nk - nq) : nk;
            // every row of the tile sees the keys before this one
            const int open = p.s.causal ? first[x] + 1 + nk - nq : nk;
            const float c = p.scale * 1.44269504088896341f;
            const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            const uint32_t tS = lanes + C::TM_S + 128 * x, tO = lanes + C::TM_O + DP * x;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = 0; j < tiles[x]; ++j) {
                ok = warp_wait(s_bar(x), j & 1, abort_flag);
                if (!ok) break;
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
                for (int i = 4; i < 128; ++i) mx[i & 3] = fmaxf(mx[i & 3], s[i]);
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (j == 0) {
                    m = top;
                } else if (__any_sync(~0u, (top - m) * c > 8.f)) {
                    const float mn = fmaxf(m, top);
                    const float keep = m == -INFINITY ? 0.f : exp2_fast((m - mn) * c);
                    m = mn;
                    l *= keep;
#pragma unroll 1
                    for (int q = 0; q < DP; q += 32) {
                        uint32_t o[32];
                        tmem_ld32(tO + q, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                        tmem_st32(tO + q, o);
                    }
                }
                const float shift = m == -INFINITY ? 0.f : -m * c;
                float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float a, d;
                        fma2(a, d, s[64 * h + 2 * i], s[64 * h + 2 * i + 1], c, shift);
                        a = exp2_fast(a);
                        d = exp2_fast(d);
                        if (i & 1) add2(s0, s1, a, d);
                        else add2(s2, s3, a, d);
                        w[i] = pack2(a, d);
                    }
                    tmem_st32(tS + 32 * h, w);
                }
                l += (s0 + s1) + (s2 + s3);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(p_bar(x));
            }
            if (ok && tiles[x] > 0) ok = warp_wait(o_bar(x), 0, abort_flag);
            if (ok && first[x] < nq) {
                tc_fence_after();
                const float inv = l == 0.f ? 0.f : 1.f / l;
                if (valid)
                    p.lse[static_cast<long long>(q0 + token) * p.a.Hq + hk * G + row % G] =
                        l == 0.f ? -INFINITY : fmaf(m, p.scale, logf(l));
                // This warp's 32 rows leave through its part of Q_x (all reads of it are
                // done), 16-byte chunks XORed with the row so that neither side conflicts.
                constexpr int CH = DP / 8;  // chunks of a row
                uint8_t* stg = smem_raw + (base - raw) + x * C::TILE + (warp & 3) * 32 * DP * 2;
#pragma unroll
                for (int q = 0; q < DP; q += 32) {
                    uint32_t o[32];
                    if (tiles[x] > 0) {
                        tmem_ld32(tO + q, o);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            f[e] = tiles[x] > 0 && l != 0.f ? __uint_as_float(o[8 * i + e]) * inv : 0.f;
                        const int ch = (q / 8 + i) ^ (lane & (CH - 1));
                        *reinterpret_cast<uint4*>(stg + lane * DP * 2 + ch * 16) = pack8(f);
                    }
                }
                __syncwarp();
                constexpr int RPI = 32 / CH;  // rows a warp writes at once
#pragma unroll 4
                for (int i = 0; i < 32; i += RPI) {
                    const int rl = i + lane / CH, ch = lane % CH;
                    const int r = (warp & 3) * 32 + rl, t = first[x] + r / G;
                    if (r < G * tpt && t < nq && ch * 8 < p.a.D)
                        *reinterpret_cast<uint4*>(p.out.row(q0 + t, hk * G + r % G) + ch * 8) =
                            *reinterpret_cast<const uint4*>(stg + rl * DP * 2 +
                                                            (ch ^ (rl & (CH - 1))) * 16);
                }
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
    return launch_k(kfn, dim3(static_cast<unsigned>(items), p.a.Hkv), dim3(kThreads), C::SMEM, st,
                    mq, mk, mv, prm);
}

}  // namespace

cudaError_t launch_attention_forward(const Attention& p, cudaStream_t st) {
    return p.a.D <= 64 ? forward<64>(p, st) : forward<128>(p, st);
}

}  // namespace attn
}  // namespace moe
