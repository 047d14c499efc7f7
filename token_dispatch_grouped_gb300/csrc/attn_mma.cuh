// attn_mma.cuh — what the tensor-core attention kernels share: tile geometry, the
// tcgen05 forms with an operand in TMEM, waits, and the search for a CTA's sequence.
#pragma once
#include "attn.cuh"
#include "ptx.cuh"

namespace moe {
namespace attn {

using namespace moe::ptx;

// A tile holds 128 rows of 128-byte pieces: 64 of the D columns each, 128-byte swizzle,
// one piece of 16 KB after the other (D <= 64: one, else two; columns past D are zeros).
// The same bytes serve as a K-major operand (rows x D, K = D) and as an MN-major one
// (D x rows, K = rows).
constexpr int kRows = 128;
constexpr int kPiece = kRows * 128;
constexpr uint64_t kWaitNs = 2000000000ull;

// D[tmem] (+)= A[tmem] * B[smem]: A is M = 128 lanes of 16-bit pairs, 8 columns per 16 of K.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One lane of a converged warp (the same one every time), in the form that lets the
// tensor-core instructions take their operands from uniform registers. The role that
// issues the products runs as a whole in such a thread: with 16 busy warps beside it and
// a barrier polled every 8 products, a 128 x 128 x 16 product takes 66 cycles (64 is the
// tensor cores' own time), against 143 with warp-wide waits and an election for every
// group, and 333 under `lane == 0` with a descriptor built for every step. (The queue of
// issued products is short, so what the thread does between them is lost to the tensor
// cores.)
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p)
                 :
                 : "memory");
    return p != 0;
}
// Descriptors of a tile: K-major (K = D; the k-th 16 of K is kd(k) further) and MN-major
// (K = rows; the k-th 16 rows are kr(k) further).
__device__ __forceinline__ uint64_t desc_d(uint32_t tile) { return sdesc_sw128(tile, 16, 1024); }
__device__ __forceinline__ uint64_t desc_r(uint32_t tile) { return sdesc_sw128(tile, kPiece, 1024); }
__device__ __forceinline__ constexpr uint64_t kd(int k) { return ((k >> 2) * kPiece + (k & 3) * 32) / 16; }
__device__ __forceinline__ constexpr uint64_t kr(int k) { return k * 2048 / 16; }

// 16 columns of this warp's 32 TMEM lanes, to and from registers.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// 2^x in the hardware's approximation (relative error about 2^-22; 2^-inf = 0).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// One arrival for a warp whose lanes' earlier TMEM accesses are waited for.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// Waits for a phase, but not longer than kWaitNs or once another role has given up (the
// abort flag): then every later wait returns after 64 polls at most, the loops run out on
// whatever their buffers hold, and the CTA reports the time-out. So no role has to agree
// on a failure with another, and a wait that is already over costs one poll. The roles
// hand tiles over every few hundred cycles, so the polls are plain try_waits without a
// suspend hint (a suspended warp woke late).
__device__ __forceinline__ void wait_phase(uint32_t bar, uint32_t parity, volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return;
    uint64_t t0 = 0;
    for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
        if ((i & 63u) != 0) continue;
        const uint64_t t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (*abort) return;
        if (t - t0 > kWaitNs) {
            *abort = 1;
            return;
        }
    }
}
// The same by a whole warp, which leaves it together.
__device__ __forceinline__ void warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
    wait_phase(bar, parity, abort);
    __syncwarp();
}
// Bounded wait for something in flight before leaving (given up or not).
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_sleep(bar, parity, 20000u))
        if (globaltimer_ns() - t0 > kWaitNs) break;
}

// 32 rows x W columns (fp32, TMEM columns t ..) of one warp, times f, as bf16 rows. dst:
// where this lane's row goes (nullptr: nowhere); only columns before D. stg: 32 x W x 2
// bytes of shared memory, 16-byte chunks XORed with the row so that neither side
// conflicts.
template <int W>
__device__ __forceinline__ void store_rows(uint32_t t, bool any, float f, uint8_t* stg, int lane,
                                           bf16* dst, int col0, int D) {
    constexpr int CH = W / 8;
#pragma unroll
    for (int q = 0; q < W; q += 16) {
        uint32_t o[16];
        if (any) {
            tmem_ld16(t + q, o);
            tmem_ld_wait();
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = any && f != 0.f ? __uint_as_float(o[8 * i + e]) * f : 0.f;
            *reinterpret_cast<uint4*>(stg + lane * W * 2 + ((q / 8 + i) ^ (lane & (CH - 1))) * 16) =
                pack8(v);
        }
    }
    __syncwarp();
    constexpr int RPI = 32 / CH;
    const unsigned long long at = reinterpret_cast<unsigned long long>(dst);
    const int ch = lane % CH;
#pragma unroll
    for (int i = 0; i < 32; i += RPI) {
        const int rl = i + lane / CH;
        const unsigned long long to = __shfl_sync(0xffffffffu, at, rl);
        if (to != 0 && col0 + ch * 8 < D)
            *reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(to) + col0 + ch * 8) =
                *reinterpret_cast<const uint4*>(stg + rl * W * 2 + (ch ^ (rl & (CH - 1))) * 16);
    }
}

// Zeroes rows [first, 128) of a tile (whole 128-byte rows of each piece, so the swizzle
// does not matter) and makes that visible to the tensor cores. One warp.
__device__ __forceinline__ void zero_tail(uint32_t tile, int pieces, int first, int lane) {
    for (int p = 0; p < pieces; ++p)
        for (int i = first * 8 + lane; i < kRows * 8; i += 32)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + p * kPiece + i * 16),
                         "r"(0)
                         : "memory");
    fence_proxy_async_smem();
    __syncwarp();
}

// A CTA's part of the batch: tokens of its sequence and the tile of them that it works on.
struct Work {
    int q0, nq, k0, nk;
    int item, items;  // items 0: nothing to do
};

// Items of one sequence whose steps are v >= 1 or more, out of `items`: tiles of `tile`
// query tokens, whose steps are the 128-key tiles that they see (never fewer from one item
// to the next, so these are the last ones) ...
__device__ __forceinline__ int query_items(const Packed& s, const Work& w, int tile, int v) {
    const int keys = (v - 1) * kRows + 1;  // sees at least as many
    if (!s.causal) return w.nk >= keys ? w.items : 0;
    const int need = keys - (w.nk - w.nq);  // tokens up to the end of the item
    if (need > w.nq) return 0;
    return need <= 0 ? w.items : w.items - ((need + tile - 1) / tile - 1);
}
// ... or tiles of 128 keys, whose steps are the query tiles that see them (never more from
// one item to the next, so these are the first ones).
__device__ __forceinline__ int key_items(const Packed& s, const Work& w, int tile, int v) {
    const int tiles = (w.nq + tile - 1) / tile;
    if (tiles < v) return 0;
    if (!s.causal) return w.items;
    const int keys = (tiles - v + 1) * tile + w.nk - w.nq;  // that start before it
    return keys <= 0 ? 0 : min(w.items, (keys + kRows - 1) / kRows);
}

// Work item `want` of the batch, by one warp. Sequences that are not valid have none.
// Up to 32 sequences (one a lane) the items with the most steps come first, over all of
// them, so that the shortest end the launch: the number of steps at rank `want` is found by
// bisection, then the sequence. Beyond, the items of a sequence follow each other, most
// steps first (16384 tokens of 16/4 heads of 128, causal, random lengths, mean of three:
// 32 sequences 86 us forward and 299 backward, 33 sequences 98 and 339), and every item is
// found by a pass over the offsets again: 70 and 219 us for 128 sequences, 259 and 689 for
// 1024, 2810 and 6430 for 4096, where that pass is nearly all of the time.
template <bool KEYS>
__device__ __forceinline__ Work find_work(const Packed& s, int tile, int want, int lane, int* err) {
    const int size = KEYS ? kRows : tile;
    int before = 0;
    for (int b0 = 0; b0 < s.B; b0 += 32) {
        Work w{0, 0, 0, 0, 0, 0};
        if (b0 + lane < s.B && sequence_of(s, b0 + lane, w.q0, w.nq, w.k0, w.nk, err))
            w.items = ((KEYS ? w.nk : w.nq) + size - 1) / size;
        const auto from_steps = [&](int v) {
            return v < 1 ? w.items : w.items == 0 ? 0 : KEYS ? key_items(s, w, tile, v)
                                                             : query_items(s, w, tile, v);
        };
        int mine = w.items, skipped = 0;  // items of this level (of all), and of higher ones
        if (s.B <= 32 && s.B > 1) {
            if (want >= __reduce_add_sync(0xffffffffu, w.items)) break;
            // the largest v with more than `want` items of v steps or more
            int lo = 0, hi = KEYS ? (w.nq + tile - 1) / tile : (w.nk + kRows - 1) / kRows;
            hi = __reduce_max_sync(0xffffffffu, hi) + 1;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__reduce_add_sync(0xffffffffu, from_steps(mid)) > want) lo = mid;
                else hi = mid;
            }
            skipped = from_steps(lo + 1);
            mine = from_steps(lo) - skipped;
            before = __reduce_add_sync(0xffffffffu, skipped);
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, want < before + incl);
        if (past) {
            const int l = __ffs(past) - 1;
            // rank within the sequence, most steps first
            w.item = want - (before + incl - mine) + skipped;
            if (!KEYS) w.item = w.items - 1 - w.item;
            w.q0 = __shfl_sync(0xffffffffu, w.q0, l);
            w.nq = __shfl_sync(0xffffffffu, w.nq, l);
            w.k0 = __shfl_sync(0xffffffffu, w.k0, l);
            w.nk = __shfl_sync(0xffffffffu, w.nk, l);
            w.item = __shfl_sync(0xffffffffu, w.item, l);
            w.items = __shfl_sync(0xffffffffu, w.items, l);
            return w;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return {0, 0, 0, 0, 0, 0};
}
// Upper bound of the items, known on the host; `longest` <= T. At least one, so that some
// CTA looks the sequences over.
inline long long tile_bound(int T, int B, int longest, int tile) {
    const long long a = static_cast<long long>(T) / tile + B;
    const long long b = static_cast<long long>(B) * ((longest + tile - 1) / tile);
    return a < b ? a : b < 1 ? 1 : b;
}

// One warp looks all sequences over (for the error report).
__device__ __forceinline__ void check_sequences(const Packed& s, int lane, int* err) {
    int q0, nq, k0, nk;
    for (int b = lane; b < s.B; b += 32) sequence_of(s, b, q0, nq, k0, nk, err);
}

// Tensor map of a view [T, H, D] with a box of 64 columns x box_heads x box_tokens and the
// 128-byte swizzle. False on failure.
bool make_tmap_heads(CUtensorMap* map, const Heads& h, int T, int H, int D, uint32_t box_heads,
                     uint32_t box_tokens);

}  // namespace attn
}  // namespace moe
