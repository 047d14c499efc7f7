// decode8.cu — attention of the newest tokens of each sequence over a paged cache of e4m3
// values with a scale for each page and head.
//
// Bound by reading the cached keys and values once: 2 D bytes a token and key/value head, half
// of what decode.cu reads, so everything else has half the time. m16n8k16 products in fp16 with
// 16 tokens (S^T = K q^T) or 16 columns (O^T = V^T P^T) as the rows of the first operand and 8
// query heads x new tokens as the columns of the second: grouped heads fill 8 columns sooner than
// decode.cu's 16 rows, and the weights turn from one product's result into the other's operand
// by movmatrix. An e4m3 value is exact in fp16, so keys and values are converted between ldmatrix
// and the product; queries are brought to fp16's range by a power of two a row; the scales enter
// outside the products, the keys' at the scores and the values' at the weights.
//
// 64 sequences of up to 32768 tokens, 32/8 heads of 128, pages of 64 (2.19 GB):
//   decode.cu's shape (16 rows of queries, 16 tokens a warp and 64-token stage)        406 us
//   32 tokens a warp and 128-token stages: one maximum, one vote, one hand-over for them  358
//   8 columns of queries (about half the instructions a token); keys and values as stages
//   of their own, freed as soon as they are read; CTAs that stay, two on an SM, and take
//   the next part from a count in the workspace (a fixed share for each, 391 before the
//   8 columns, is uneven: CTAs read at different rates)                               316-320
// The last is 6.9 TB/s, 102% of the measured copy. Parts are the same for a sequence whatever
// the lengths of the others, so its bits are too.
#include "decode.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kTokens = 128;  // of a stage
constexpr int kWarps = 4;
constexpr int kOf = kTokens / kWarps;  // tokens of a warp: kX groups of 16
constexpr int kX = kOf / 16;
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kBoxes = kTokens / 8;  // of a stage at most: pages of 8 tokens
constexpr int kMostSlots = 12;
constexpr int kQueue = 2;            // parts that the load warp may be ahead
// P enters its product as weight * kLift, so that the many small weights beside one that is
// near 1 keep their share (fp16 ends at 2^-24, a lifted weight at 2^-39).
constexpr float kLift = 32768.f;

// Slots of the ring and the place of everything behind it, for `rows` rows of a tile in use.
template <int DP>
struct Cfg {
    static constexpr int SLOT = kTokens * DP;  // keys or values of a stage
    static constexpr int PITCH = DP + 4;       // floats of a merged row
    static constexpr int FIXED = 1024 + 2 * kWarps * kRowTile * 4 + kMostSlots * (kBoxes * 4 + 16) +
                                 kQueue * 24 + 16;
    static constexpr int merge(int rows) { return kWarps * rows * PITCH * 4; }
    static constexpr int slots(int rows) {  // of two CTAs an SM
        const int n = (113 * 1024 - FIXED - 4 * (kNumberedSeqs + 1) - merge(rows)) / SLOT;
        return n < kMostSlots ? n : kMostSlots;
    }
};

__device__ __forceinline__ void mma16h(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 block of 16-bit values, turned.
__device__ __forceinline__ uint32_t turned(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// 16-byte chunk c of row r of a stage, whose rows are swizzled over their DP bytes.
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return r * DP + ((DP == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

// A part of a sequence for one key/value head and one tile of rows.
struct Item {
    int b, hk, part, rt, len;
};

// Part `at` of all sequences (first: the numbers of parts before each), or of the grid of
// B * Hkv * parts * row_tiles (first = nullptr), where it may lie past its sequence. b: a
// sequence that is not past it.
__device__ __forceinline__ bool item_of(const DecodeParams& p, const int* first, int at, int& b, Item& it) {
    if (first == nullptr) {
        it.rt = at % p.row_tiles;
        at /= p.row_tiles;
        it.part = at % p.parts;
        at /= p.parts;
        it.hk = at % p.a.Hkv;
        it.b = at / p.a.Hkv;
        it.len = p.lens[it.b];
        if (it.len < 0 || it.len > p.max_kv) return false;
        // an empty sequence has one part, which writes its zeros
        return it.part == 0 || it.part * p.chunk < it.len;
    }
    const int heads = p.a.Hkv * p.row_tiles;
    if (at >= first[p.B] * heads) return false;
    while (first[b + 1] * heads <= at) ++b;
    at -= first[b] * heads;
    const int parts = first[b + 1] - first[b];
    it.b = b;
    it.rt = at % p.row_tiles;  // fastest, so that tiles of the same tokens meet in L2
    at /= p.row_tiles;
    it.part = at % parts;
    it.hk = at / parts;
    it.len = p.lens[b];
    return true;
}

// W: scores are kept for the weights.
template <int DP, int NB, bool W>
__global__ void __launch_bounds__(kThreads, 2)
decode8_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
               const DecodeParams p, const int slots, const int rows_in_use, int* tickets) {
    using C = Cfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* tail = smem_raw + (base - raw) + slots * C::SLOT;
    float* merge = reinterpret_cast<float*>(tail);  // [warp][row in use][PITCH]
    float* s_m = merge + kWarps * rows_in_use * C::PITCH;  // [warp][row]
    float* s_l = s_m + kWarps * kRowTile;
    float* s_scale = s_l + kWarps * kRowTile;  // [slot][box]
    uint8_t* misc = reinterpret_cast<uint8_t*>(s_scale + kMostSlots * kBoxes);
    const uint32_t bars = smem_u32(misc);
    const auto full = [&](int s) { return bars + 8u * s; };
    const auto empty = [&](int s) { return bars + 8u * (kMostSlots + s); };
    const auto item_full = [&](int i) { return bars + 8u * (2 * kMostSlots + i); };
    const auto item_empty = [&](int i) { return bars + 8u * (2 * kMostSlots + kQueue + i); };
    volatile int* s_item = reinterpret_cast<volatile int*>(misc + 16 * kMostSlots + 16 * kQueue);
    volatile int* abort_flag = s_item + 2 * kQueue;
    int* s_first = const_cast<int*>(abort_flag) + 4;  // numbered: [B + 1]
    const bool numbered = tickets != nullptr;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < slots; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kWarps);
        }
        for (int i = 0; i < kQueue; ++i) {
            mbar_init(item_full(i), 1);
            mbar_init(item_empty(i), kWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    if (__syncthreads_or(stopped(p.err))) return;
    // a length out of range is reported by the first CTA; its sequence has no parts
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.B; b += kThreads)
            if (p.lens[b] < 0 || p.lens[b] > p.max_kv) raise_error(p.err, MOE_ERR_BAD_INDEX);
    if (numbered) {
        for (int b = threadIdx.x; b < p.B; b += kThreads) {
            const int len = p.lens[b];
            s_first[b + 1] = len < 0 || len > p.max_kv ? 0 : max(1, (len + p.chunk - 1) / p.chunk);
        }
        __syncthreads();
        if (warp == 0) {
            int sum = 0;
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                int x = b0 + lane < p.B ? s_first[b0 + lane + 1] : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(~0u, x, o);
                    if (lane >= o) x += y;
                }
                if (b0 + lane < p.B) s_first[b0 + lane + 1] = sum + x;
                sum += __shfl_sync(~0u, x, 31);
            }
            if (lane == 0) s_first[0] = 0;
        }
        __syncthreads();
    }
    const int* first = numbered ? s_first : nullptr;
    int cursor = 0;
    const int G = p.a.Hq / p.a.Hkv, R = G * p.n, D = p.a.D;
    Item it;

    if (warp == kWarps) {
        // ---------------------------------------------------------------- pages
        const int sh = p.page_shift, rows = min(1 << sh, kTokens);  // of a box
        int slot = 0, done = 0;  // fills so far
        uint32_t phase = 1;      // of `empty`: a first fill waits for nothing
        bool ok = true;
        int at = blockIdx.x;
        for (int k = 0; ok; ++k) {
            // the part is handed to the other warps (-1: no more), the one after it asked for
            const bool any = at >= 0 && item_of(p, first, at, cursor, it);
            if (k >= kQueue) warp_wait(item_empty(k % kQueue), (k / kQueue - 1) & 1, abort_flag);
            if (lane == 0) {
                s_item[k % kQueue] = any ? at : -1;
                mbar_arrive(item_full(k % kQueue));
            }
            if (!any) break;
            int ticket = -1;
            if (numbered && lane == 0) ticket = static_cast<int>(gridDim.x) + atomicAdd(tickets, 1);
            const int* table = p.table + static_cast<long long>(it.b) * p.table_stride;
            const int t0 = it.part * p.chunk, t1 = min(it.len, t0 + p.chunk);
            const int stages = (t1 - t0 + kTokens - 1) / kTokens;
            // pages are looked up two stages ahead and their scales one, so that no load stands
            // between a free slot and its boxes: lane x has box x, rows x * rows .. of a stage
            const auto page_at = [&](int i) {
                const int tok = t0 + i * kTokens + lane * rows;
                return lane < kTokens / rows && tok < t1 ? table[tok >> sh] : -1;
            };
            const auto there = [&](int page) { return page >= 0 && page < p.pages; };
            const auto scales_of = [&](int page) {
                if (!there(page)) return make_float2(0.f, 0.f);
                const long long at = static_cast<long long>(page) * p.a.Hkv + it.hk;
                return make_float2(p.k_scale[at], p.v_scale[at]);
            };
            int page0 = page_at(0), page1 = page_at(1);
            float2 sc0 = scales_of(page0);
            for (int i = 0; i < stages; ++i) {
                const int page2 = page_at(i + 2);
                const float2 sc1 = scales_of(page1);
                const int tok = t0 + i * kTokens + lane * rows;
                const bool mine = lane < kTokens / rows && tok < t1, load = mine && there(page0);
                if (mine && !load) raise_error(p.err, MOE_ERR_BAD_INDEX);
                const int boxes = __popc(__ballot_sync(~0u, load));
                const int y = load ? ((page0 * p.a.Hkv + it.hk) << sh) + (tok & ((1 << sh) - 1)) : 0;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    if (done >= slots) warp_wait(empty(slot), phase, abort_flag);
                    if (__any_sync(~0u, *abort_flag != 0)) {
                        ok = false;
                        break;
                    }
                    if (lane < kBoxes) s_scale[slot * kBoxes + lane] = v ? sc0.y : sc0.x;  // 0: no box
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(full(slot), boxes * rows * DP);
                    __syncwarp();
                    if (load)
                        tma_load_2d(base + slot * C::SLOT + lane * rows * DP, v ? &mapV : &mapK, full(slot),
                                    0, y);
                    __syncwarp();
                    ++done;
                    if (++slot == slots) slot = 0, phase ^= 1;
                }
                if (!ok) break;
                page0 = page1, page1 = page2, sc0 = sc1;
            }
            at = __shfl_sync(~0u, ticket, 0);
        }
        if (lane == 0)  // nothing is in flight when the CTA leaves
            for (int j = max(0, done - slots); j < done; ++j)
                drain(full(j % slots), (j / slots) & 1);
    } else {
        // -------------------------------------------------------------- products
        int slot = 0;
        uint32_t phase = 0;
        const auto release = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(slot));
            if (++slot == slots) slot = 0, phase ^= 1;
        };
        const int box_shift = min(p.page_shift, 7);
        const int c2 = (lane & 3) * 2;
        for (int k = 0;; ++k) {
            warp_wait(item_full(k % kQueue), (k / kQueue) & 1, abort_flag);
            const int at = *abort_flag ? -1 : s_item[k % kQueue];
            __syncwarp();
            if (lane == 0) mbar_arrive(item_empty(k % kQueue));
            if (!__all_sync(~0u, at >= 0)) break;
            item_of(p, first, at, cursor, it);
            const int b = it.b, hk = it.hk, len = it.len;
            const int t0 = it.part * p.chunk, t1 = min(len, t0 + p.chunk);
            const int stages = (t1 - t0 + kTokens - 1) / kTokens;
            const int r0 = it.rt * 8 * NB;
            uint32_t qb[NB][DP / 16][2];  // of row r0 + 8 nb + lane / 4
            int lim[NB][2];               // of rows r0 + 8 nb + 2 (lane % 4) + u, as all below
            float c[NB][2];               // what turns a product into its score, in powers of two
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int r = r0 + 8 * nb + (lane >> 2);
                const bool valid = r < R;
                const bf16* src = p.q.row(static_cast<long long>(b) * p.n + (valid ? r / G : 0),
                                          hk * G + (valid ? r % G : 0));
                // a lane's four bytes of a key row are four values in a row, two for each half
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const int col = 16 * k + 2 * c2;
                    const uint2 w = valid && col < D ? *reinterpret_cast<const uint2*>(src + col)
                                                     : make_uint2(0u, 0u);
                    qb[nb][k][0] = w.x;
                    qb[nb][k][1] = w.y;
                    const uint32_t x = w.x & 0x7fff7fffu, y = w.y & 0x7fff7fffu;
                    top = max(top, max(max(x & 0xffffu, x >> 16), max(y & 0xffffu, y >> 16)));
                }
                // The row in fp16: divided by the power of two that brings its largest value to
                // [1, 2), where bf16 values down to 2^-17 of the largest are exact and the others
                // off by at most 2^-25 of it.
                top = max(top, __shfl_xor_sync(~0u, top, 1));
                top = max(top, __shfl_xor_sync(~0u, top, 2));
                const int e = min(253, max(1, static_cast<int>(top >> 7)));  // the exponent's field
                const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                const float mine = p.scale * 1.44269504088896341f *
                                   __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const uint32_t w = qb[nb][k][v];
                        qb[nb][k][v] = half2_of(__uint_as_float(w << 16) * inv,
                                                __uint_as_float(w & 0xffff0000u) * inv);
                    }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int row = r0 + 8 * nb + c2 + u;
                    lim[nb][u] = row < R ? min(len, row / G + len - p.n + 1) : 0;
                    c[nb][u] = __shfl_sync(~0u, mine, 4 * (c2 + u));
                }
            }
            // the tokens before this one are seen by every row
            const int open = len - p.n + 1;
            float vr = 0.f, vr_inv = 0.f;  // O is in units of vr, the largest value scale so far
            float m[NB][2], l[NB][2], o[NB][DP / 16][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                m[nb][0] = m[nb][1] = -INFINITY;
                l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
                for (int d = 0; d < DP / 16; ++d) o[nb][d][0] = o[nb][d][1] = o[nb][d][2] = o[nb][d][3] = 0.f;
            }
            for (int i = 0; i < stages; ++i) {
                const int tok = t0 + i * kTokens + kOf * warp;  // this warp's first token
                const bool some = tok < t1;
                // scores: token 16 x + 8 (e / 2) + lane / 4, row e % 2
                float s[kX][NB][4] = {};
                warp_wait(full(slot), phase, abort_flag);
                if (some) {
                    const uint32_t sK = base + slot * C::SLOT;
                    // a chunk of 16 bytes is 16 of K
                    const int row = kOf * warp + (lane >> 4) * 8 + (lane & 7), half = (lane >> 3) & 1;
                    float odd[kX][NB][4] = {};  // half of a short chain of products (NB = 1)
#pragma unroll
                    for (int k = 0; k < DP / 16; k += 2)
#pragma unroll
                        for (int x = 0; x < kX; ++x) {
                            uint32_t kb[4], a[4];
                            ldm4(sK + chunk_at<DP>(row + 16 * x, k + half), kb);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                e4m3x4_to_f16(kb[j], a[0], a[2]);
                                e4m3x4_to_f16(kb[2 + j], a[1], a[3]);
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb)
                                    mma16h(j && NB == 1 ? odd[x][nb] : s[x][nb], a, qb[nb][k + j][0], qb[nb][k + j][1]);
                            }
                        }
#pragma unroll
                    for (int x = 0; x < kX; ++x)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float ks =
                                s_scale[slot * kBoxes + ((kOf * warp + 16 * x + 8 * h) >> box_shift)];
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int u = 0; u < 2; ++u)
                                    s[x][nb][2 * h + u] =
                                        (s[x][nb][2 * h + u] + odd[x][nb][2 * h + u]) * (c[nb][u] * ks);
                        }
                }
                release();
                if (some) {
                    if (tok + kOf > open || tok + kOf > t1) {
#pragma unroll
                        for (int x = 0; x < kX; ++x)
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (tok + 16 * x + 8 * (e >> 1) + (lane >> 2) >= min(t1, lim[nb][e & 1]))
                                        s[x][nb][e] = -INFINITY;
                    }
                    if constexpr (W) {
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int r = r0 + 8 * nb + c2 + u;
                                if (r >= R) continue;
                                float* dst = p.scores +
                                             (static_cast<long long>(b * p.a.Hkv + hk) * R + r) * p.pitch +
                                             tok + (lane >> 2);
#pragma unroll
                                for (int x = 0; x < kX; ++x) {
                                    dst[16 * x] = s[x][nb][u];
                                    dst[16 * x + 8] = s[x][nb][2 + u];
                                }
                            }
                    }
                    bool grew = false;
                    float keep[NB][2];
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float t = fmaxf(s[0][nb][u], s[0][nb][2 + u]);
#pragma unroll
                            for (int x = 1; x < kX; ++x) t = max3(t, s[x][nb][u], s[x][nb][2 + u]);
#pragma unroll
                            for (int w = 4; w < 32; w *= 2) t = fmaxf(t, __shfl_xor_sync(~0u, t, w));
                            const float mn = fmaxf(m[nb][u], t);
                            grew |= mn > m[nb][u];
                            keep[nb][u] = m[nb][u] == -INFINITY ? 0.f : exp2_fast(m[nb][u] - mn);
                            m[nb][u] = mn;
                        }
                    if (__any_sync(~0u, grew)) {
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                l[nb][u] *= keep[nb][u];
#pragma unroll
                                for (int d = 0; d < DP / 16; ++d) {
                                    o[nb][d][u] *= keep[nb][u];
                                    o[nb][d][2 + u] *= keep[nb][u];
                                }
                            }
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float from = m[nb][u] == -INFINITY ? 0.f : m[nb][u];
#pragma unroll
                            for (int x = 0; x < kX; ++x)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    float& y = s[x][nb][2 * h + u];
                                    y = exp2_fast(y - from);
                                    l[nb][u] += y;
                                }
                        }
                }
                warp_wait(full(slot), phase, abort_flag);
                if (some) {
                    const uint32_t sV = base + slot * C::SLOT;
                    if (tok + kOf > t1) {  // rows past the length hold whatever the page held
                        constexpr int CH = DP / 16;
                        for (int x = lane; x < kOf * CH; x += 32) {
                            const int row = kOf * warp + x / CH;
                            if (t0 + i * kTokens + row >= t1)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                                 sV + row * DP + (x % CH) * 16),
                                             "r"(0)
                                             : "memory");
                        }
                        __syncwarp();
                    }
                    float vs[2 * kX], vn = vr;  // the same in every lane
#pragma unroll
                    for (int t = 0; t < 2 * kX; ++t) {
                        vs[t] = s_scale[slot * kBoxes + ((kOf * warp + 8 * t) >> box_shift)];
                        vn = fmaxf(vn, vs[t]);
                    }
                    if (vn > vr) {
                        vr_inv = 1.f / vn;
                        const float f = vr * vr_inv;
                        vr = vn;
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int d = 0; d < DP / 16; ++d)
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[nb][d][e] *= f;
                    }
                    const int row = kOf * warp + ((lane >> 3) & 1) * 8 + (lane & 7), half = lane >> 4;
#pragma unroll
                    for (int x = 0; x < kX; ++x) {
                        uint32_t pb[NB][2];  // weights of token pairs, by turning those of row pairs
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float f = vs[2 * x + h] * vr_inv * kLift;
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                pb[nb][h] = turned(half2_of(s[x][nb][2 * h] * f, s[x][nb][2 * h + 1] * f));
                        }
                        // a transposed pair of bytes is two columns of two tokens: sorted by column
                        // they are rows lane / 4 (the even columns) and 8 + lane / 4 (the odd ones)
#pragma unroll
                        for (int d = 0; d < DP / 16; d += 2) {
                            uint32_t vb[4], a[4];
                            ldm4t(sV + chunk_at<DP>(row + 16 * x, d + half), vb);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                e4m3x4_to_f16(__byte_perm(vb[2 * j], 0u, 0x3120), a[0], a[1]);
                                e4m3x4_to_f16(__byte_perm(vb[2 * j + 1], 0u, 0x3120), a[2], a[3]);
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb)
                                    mma16h(o[nb][d + j], a, pb[nb][0], pb[nb][1]);
                            }
                        }
                    }
                }
                release();
            }
            // the last part's merged rows have been read by every warp
            asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
            const float unit = vr * (1.f / kLift);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int w = 4; w < 32; w *= 2) l[nb][u] += __shfl_xor_sync(~0u, l[nb][u], w);
                    const int r = 8 * nb + c2 + u;
                    if (r >= rows_in_use) continue;
                    if (lane < 4) {
                        s_m[warp * kRowTile + r] = m[nb][u];
                        s_l[warp * kRowTile + r] = l[nb][u];
                    }
                    float* dst = merge + (warp * rows_in_use + r) * C::PITCH + 2 * (lane >> 2);
#pragma unroll
                    for (int d = 0; d < DP / 16; ++d)
                        *reinterpret_cast<float2*>(dst + 16 * d) =
                            make_float2(o[nb][d][u] * unit, o[nb][d][2 + u] * unit);
                }
            asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
            const int rows = min(rows_in_use, R - r0), pieces = D / 8;
            for (int x = threadIdx.x; x < rows * pieces; x += kWarps * 32) {
                const int r = x / pieces, col = x % pieces * 8;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w * kRowTile + r]);
                const float b2 = top == -INFINITY ? 0.f : top;
                float f[kWarps], sum = 0.f, v[8] = {};
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    f[w] = exp2_fast(s_m[w * kRowTile + r] - b2);
                    sum += f[w] * s_l[w * kRowTile + r];
                    const float4* src =
                        reinterpret_cast<const float4*>(merge + (w * rows_in_use + r) * C::PITCH + col);
                    const float4 y = src[0], z = src[1];
                    v[0] += f[w] * y.x, v[1] += f[w] * y.y, v[2] += f[w] * y.z, v[3] += f[w] * y.w;
                    v[4] += f[w] * z.x, v[5] += f[w] * z.y, v[6] += f[w] * z.z, v[7] += f[w] * z.w;
                }
                const long long t = static_cast<long long>(b) * p.n + (r0 + r) / G;
                const int h = hk * G + (r0 + r) % G;
                const long long at = (t * p.a.Hq + h) * p.parts + it.part;
                if (p.parts > 1) {
                    if (col == 0) {
                        p.part_ml[2 * at] = top;
                        p.part_ml[2 * at + 1] = sum;
                    }
                    float4* dst = reinterpret_cast<float4*>(p.part + at * D + col);
                    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                } else {
                    if (W && col == 0) p.lse[t * p.a.Hq + h] = sum == 0.f ? INFINITY : top + log2f(sum);
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = sum == 0.f ? 0.f : v[e] * inv;
                    *reinterpret_cast<uint4*>(p.out.row(t, h) + col) = pack8(v);
                }
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) raise_timeout(p.err);
}

// Tensor map of e4m3 rows [rows, cols] with a box of `box_cols` (64 or 128, its swizzle) x box_rows.
bool make_tmap_e4m3(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t box_cols,
                    uint32_t box_rows) {
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t es[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              box_cols == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, int NB, bool W>
cudaError_t decode8(const Decode& d, cudaStream_t st) {
    using C = Cfg<DP>;
    const DecodePlan pl = decode_plan(d.a, d.B, d.n, d.max_kv, true);
    const long long most = static_cast<long long>(d.B) * d.a.Hkv * pl.parts * pl.row_tiles;
    if (most > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const DecodeParams p = decode_params(d, pl);
    CUtensorMap mk, mv;
    const uint64_t cache_rows = (static_cast<uint64_t>(d.pages) * d.a.Hkv) << d.page_shift;
    const uint32_t box = (1 << d.page_shift) < kTokens ? (1 << d.page_shift) : kTokens;
    if (!make_tmap_e4m3(&mk, d.k_pages, cache_rows, d.a.D, DP, box) ||
        !make_tmap_e4m3(&mv, d.v_pages, cache_rows, d.a.D, DP, box))
        return cudaErrorInvalidValue;
    int* tickets = decode_numbered(d.a, d.B, d.max_kv, pl)
                       ? reinterpret_cast<int*>(d.ws + decode_space(d, pl).total) - 4
                       : nullptr;
    const int g = d.a.Hq / d.a.Hkv * d.n, rows = g < kRowTile ? g : kRowTile;
    const int slots = C::slots(rows);
    const int smem = C::FIXED + slots * C::SLOT + C::merge(rows) + 4 * (kNumberedSeqs + 1);
    auto kfn = decode8_kernel<DP, NB, W>;
    const cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    {
        LaunchScope ls("attention_decode8", st);
        if (tickets != nullptr) {  // (behind a memset there is nothing to overlap with)
            const cudaError_t z = cudaMemsetAsync(tickets, 0, sizeof(int), st);
            if (z != cudaSuccess) return z;
            kfn<<<2 * num_sms(), kThreads, smem, st>>>(mk, mv, p, slots, rows, tickets);
            if (const cudaError_t r = cudaGetLastError()) return r;
        } else if (const cudaError_t r = launch_pdl(kfn, dim3(static_cast<unsigned>(most)), dim3(kThreads),
                                                    smem, st, mk, mv, p, slots, rows, tickets)) {
            return r;
        }
    }
    return launch_decode_rest(p, st);
}

template <int DP, int NB>
cudaError_t decode8_w(const Decode& d, cudaStream_t st) {
    return d.weights != nullptr ? decode8<DP, NB, true>(d, st) : decode8<DP, NB, false>(d, st);
}

}  // namespace

cudaError_t launch_decode8(const Decode& d, cudaStream_t st) {
    const bool few = d.a.Hq / d.a.Hkv * d.n <= 8;
    if (d.a.D <= 64) return few ? decode8_w<64, 1>(d, st) : decode8_w<64, 2>(d, st);
    return few ? decode8_w<128, 1>(d, st) : decode8_w<128, 2>(d, st);
}

}  // namespace attn
}  // namespace moe
