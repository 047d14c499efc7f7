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

__device__ __forceinline__ uint64_t desc_k(uint32_t tile, int k) {  // K-major, k-th 16 of D
    return sdesc_sw128(tile + (k >> 2) * kPiece + (k & 3) * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int k) {  // MN-major, k-th 16 rows
    return sdesc_sw128(tile + k * 2048, kPiece, 1024);
}

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

// 32 columns of this warp's 32 TMEM lanes, written from registers.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
        "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
        "r"(v[30]), "r"(v[31]), "r"(taddr)
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
// Two fp32 operations in one instruction.
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c) {
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {
    asm("{\n\t.reg .b64 a, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 d, {%0, %1};\n\t"
        "add.rn.f32x2 d, d, a;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}

// A wait of every lane of a warp; false (for all of them) when it ran out or another
// role has given up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, kWaitNs));
}
// Bounded wait for something in flight before leaving (given up or not).
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_sleep(bar, parity, 20000u))
        if (globaltimer_ns() - t0 > kWaitNs) break;
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

// The sequence and tile of work item `want` when sequence b has ceil(n_b / tile) items,
// n_b its query (or key) tokens: one warp. Sequences that are not valid have none.
// Returns false past the last item.
__device__ __forceinline__ bool find_tile(const Packed& s, bool keys, int tile, int want, int lane,
                                          int& b, int& item, int& items, int* err) {
    int before = 0;
    for (int b0 = 0; b0 < s.B; b0 += 32) {
        int n = 0;
        if (b0 + lane < s.B) {
            int q0, nq, k0, nk;
            if (sequence_of(s, b0 + lane, q0, nq, k0, nk, err)) n = ((keys ? nk : nq) + tile - 1) / tile;
        }
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, want < before + incl);
        if (past) {
            const int l = __ffs(past) - 1;
            const int end = __shfl_sync(0xffffffffu, incl, l);
            items = __shfl_sync(0xffffffffu, n, l);
            item = want - (before + end - items);
            b = b0 + l;
            return true;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
}
// Upper bound of the items, known on the host.
inline long long tile_bound(int T, int B, int longest, int tile) {
    const long long a = static_cast<long long>(T) / tile + B;
    const long long b = static_cast<long long>(B) * ((longest + tile - 1) / tile);
    return a < b ? a : b;
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
