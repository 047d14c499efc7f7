// decode.cu — attention of the newest tokens of each sequence over its paged cache.
//
// Bound by reading the cached keys and values once: 4 D bytes a token and key/value head
// against 4 D G n flops. The rows of one product are the G query heads of the n newest
// tokens (16 a CTA), so a cached token is read once for all of them. A CTA takes a part
// of the tokens of one (sequence, key/value head): a warp brings pages by TMA (boxes of
// min(page, 64) rows, 128-byte swizzle) into a ring of 64-token stages, several in flight;
// four warps take 16 tokens of a stage each, S = q K^T and O += P V with m16n8k16 products
// (the rows fill one fragment; tcgen05's 128 rows would be mostly padding), each with its
// own running maximum and sum over the tokens it has seen. They meet in shared memory at
// the end. Where B * Hkv leaves SMs idle or sequences are uneven, the tokens of a sequence
// are cut into parts whose (maximum, sum, O) go to the workspace in fp32, and a second
// kernel joins them in part order.
//
// P is rounded to bf16 for its product; maxima, sums and O are fp32. Tokens past a row's
// limit get weight 0 by selection; rows of V past the length are zeroed in shared memory,
// whatever the page holds there.
#include "attn_mma.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kTokens = 64;   // of a stage
constexpr int kWarps = 4;     // 16 tokens of a stage each
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kRowTile = 16;

template <int DP>
struct Cfg {
    static constexpr int PIECES = DP / 64;
    static constexpr int HALF = PIECES * kTokens * 128;  // K or V of a stage
    static constexpr int STAGE = 2 * HALF;
    static constexpr int STAGES = DP == 128 ? 3 : 6;     // 96 KB: two CTAs an SM
    static constexpr int SMEM = 1024 + STAGES * STAGE + 2 * kWarps * kRowTile * 4 + 256;
    static constexpr int PITCH = DP + 4;                 // floats of a merged row
    static_assert(kWarps * kRowTile * PITCH * 4 <= STAGES * STAGE, "merge area");
};

struct Params {
    moe_attn_shape a;
    int B, n, max_kv;
    float scale;
    Heads q, out;
    int pages, page_shift;
    const int32_t* table;
    int table_stride;
    const int32_t* lens;
    float *part, *part_ml;  // [row][parts][D] and [row][parts][2] (row = token, head)
    int parts, chunk;       // tokens of a part
    int row_tiles;
    int* err;
};

__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 2)
decode_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
              const Params p) {
    using C = Cfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* tail = smem_raw + (base - raw) + C::STAGES * C::STAGE;
    float* s_m = reinterpret_cast<float*>(tail);  // [warp][row]
    float* s_l = s_m + kWarps * kRowTile;
    uint8_t* misc = tail + 2 * kWarps * kRowTile * 4;
    const uint32_t bars = smem_u32(misc);
    const auto full = [&](int s) { return bars + 8u * s; };
    const auto empty = [&](int s) { return bars + 8u * (C::STAGES + s); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 16 * C::STAGES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    // work item: row tile (fastest, so that tiles of the same tokens meet in L2), part,
    // key/value head, sequence
    long long item = blockIdx.x;
    const int rt = static_cast<int>(item % p.row_tiles);
    item /= p.row_tiles;
    const int part = static_cast<int>(item % p.parts);
    item /= p.parts;
    const int hk = static_cast<int>(item % p.a.Hkv);
    const int b = static_cast<int>(item / p.a.Hkv);
    const int G = p.a.Hq / p.a.Hkv, D = p.a.D;
    const int len = p.lens[b];
    const int t0 = part * p.chunk;
    const bool skip = stopped(p.err);
    // an empty sequence has one part, which writes its zeros
    if (__syncthreads_or(skip) || len < 0 || len > p.max_kv || (part > 0 && t0 >= len)) {
        if (threadIdx.x == 0 && (len < 0 || len > p.max_kv)) raise_error(p.err, MOE_ERR_BAD_INDEX);
        return;
    }
    const int t1 = min(len, t0 + p.chunk);
    const int stages = (t1 - t0 + kTokens - 1) / kTokens;

    if (warp == kWarps) {
        // ---------------------------------------------------------------- pages
        const int* table = p.table + static_cast<long long>(b) * p.table_stride;
        const int sh = p.page_shift, rows = min(1 << sh, kTokens);  // of a box
        int i = 0;
        for (; i < stages; ++i) {
            const int slot = i % C::STAGES;
            if (i >= C::STAGES) warp_wait(empty(slot), (i / C::STAGES - 1) & 1, abort_flag);
            if (__any_sync(~0u, *abort_flag != 0)) break;
            // box x of this stage: rows x * rows .. of K and V; lane x has its page
            const int tok = t0 + i * kTokens + lane * rows;
            const bool mine = lane < kTokens / rows && tok < t1;
            int page = mine ? table[tok >> sh] : 0;
            const bool bad = mine && (page < 0 || page >= p.pages);
            if (bad) raise_error(p.err, MOE_ERR_BAD_INDEX);
            const bool load = mine && !bad;
            const int boxes = __popc(__ballot_sync(~0u, load));
            if (lane == 0) mbar_arrive_expect_tx(full(slot), boxes * rows * 128 * C::PIECES * 2);
            __syncwarp();
            if (load) {
                const int y = ((page * p.a.Hkv + hk) << sh) + (tok & ((1 << sh) - 1));
                const uint32_t dst = base + slot * C::STAGE + lane * rows * 128;
#pragma unroll
                for (int c = 0; c < C::PIECES; ++c) {
                    tma_load_2d(dst + c * kTokens * 128, &mapK, full(slot), 64 * c, y);
                    tma_load_2d(dst + C::HALF + c * kTokens * 128, &mapV, full(slot), 64 * c, y);
                }
            }
            __syncwarp();
        }
        if (lane == 0)  // nothing is in flight when the CTA leaves
            for (int j = max(0, i - C::STAGES); j < i; ++j)
                drain(full(j % C::STAGES), (j / C::STAGES) & 1);
    } else {
        // -------------------------------------------------------------- products
        const int r0 = rt * kRowTile + (lane >> 2);  // this thread's rows: r0, r0 + 8
        const int c2 = (lane & 3) * 2;
        uint32_t qa[DP / 16][4];
        int lim[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = r0 + 8 * u;
            const bool valid = r < G * p.n;
            const int i = valid ? r / G : 0;
            lim[u] = valid ? min(len, i + len - p.n + 1) : 0;
            const bf16* src = p.q.row(static_cast<long long>(b) * p.n + i, hk * G + (valid ? r % G : 0));
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int col = 16 * k + 8 * v + c2;
                    qa[k][2 * v + u] = valid && col < D ? *reinterpret_cast<const uint32_t*>(src + col) : 0u;
                }
        }
        // the tokens before this one are seen by every row
        const int open = len - p.n + 1;
        const float c = p.scale * 1.44269504088896341f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float o[DP / 8][4];
#pragma unroll
        for (int d = 0; d < DP / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
        for (int i = 0; i < stages; ++i) {
            const int slot = i % C::STAGES;
            const int tok = t0 + i * kTokens + 16 * warp;  // this warp's first token
            warp_wait(full(slot), (i / C::STAGES) & 1, abort_flag);
            if (tok < t1) {
                const uint32_t sK = base + slot * C::STAGE, sV = sK + C::HALF;
                float s[2][4] = {};
                {
                    const int row = 16 * warp + (lane >> 4) * 8 + (lane & 7), half = (lane >> 3) & 1;
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) {
                        uint32_t kb[4];
                        ldm4(sK + (k >> 2) * kTokens * 128 + row * 128 +
                                 (((2 * (k & 3) + half) ^ (row & 7)) << 4),
                             kb);
                        mma16(s[0], qa[k], kb[0], kb[1]);
                        mma16(s[1], qa[k], kb[2], kb[3]);
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[t][e] *= c;
                if (tok + 16 > open || tok + 16 > t1) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (tok + 8 * t + c2 + (e & 1) >= min(t1, lim[e >> 1])) s[t][e] = -INFINITY;
                    // rows of V past the length hold whatever the page held
                    if (tok + 16 > t1) {
                        for (int x = lane; x < 16 * 8 * C::PIECES; x += 32) {
                            const int row = 16 * warp + (x >> 3) % 16;
                            if (t0 + i * kTokens + row >= t1)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                                 sV + (x >> 7) * kTokens * 128 + row * 128 + (x & 7) * 16),
                                             "r"(0)
                                             : "memory");
                        }
                        __syncwarp();
                    }
                }
                uint32_t pa[4];
                bool grew = false;
                float keep[2], base2[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float t = fmaxf(fmaxf(s[0][2 * u], s[0][2 * u + 1]), fmaxf(s[1][2 * u], s[1][2 * u + 1]));
                    t = fmaxf(t, __shfl_xor_sync(~0u, t, 1));
                    t = fmaxf(t, __shfl_xor_sync(~0u, t, 2));
                    const float mn = fmaxf(m[u], t);
                    grew |= mn > m[u];
                    keep[u] = m[u] == -INFINITY ? 0.f : exp2_fast(m[u] - mn);
                    m[u] = mn;
                    base2[u] = mn == -INFINITY ? 0.f : mn;
                }
                if (__any_sync(~0u, grew)) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        l[u] *= keep[u];
#pragma unroll
                        for (int d = 0; d < DP / 8; ++d) {
                            o[d][2 * u] *= keep[u];
                            o[d][2 * u + 1] *= keep[u];
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float x = exp2_fast(s[t][2 * u] - base2[u]);
                        const float y = exp2_fast(s[t][2 * u + 1] - base2[u]);
                        l[u] += x + y;
                        pa[2 * t + u] = pack2(x, y);
                    }
                const int row = 16 * warp + ((lane >> 3) & 1) * 8 + (lane & 7), half = lane >> 4;
#pragma unroll
                for (int d = 0; d < DP / 16; ++d) {
                    uint32_t vb[4];
                    ldm4t(sV + (d >> 2) * kTokens * 128 + row * 128 +
                              (((2 * (d & 3) + half) ^ (row & 7)) << 4),
                          vb);
                    mma16(o[2 * d], pa, vb[0], vb[1]);
                    mma16(o[2 * d + 1], pa, vb[2], vb[3]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(slot));
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            l[u] += __shfl_xor_sync(~0u, l[u], 1);
            l[u] += __shfl_xor_sync(~0u, l[u], 2);
        }
        // every stage has been read by every warp before the ring is reused
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        float* merge = reinterpret_cast<float*>(smem_raw + (base - raw));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = (lane >> 2) + 8 * u;
            if ((lane & 3) == 0) {
                s_m[warp * kRowTile + r] = m[u];
                s_l[warp * kRowTile + r] = l[u];
            }
#pragma unroll
            for (int d = 0; d < DP / 8; ++d)
                *reinterpret_cast<float2*>(merge + (warp * kRowTile + r) * C::PITCH + 8 * d + c2) =
                    make_float2(o[d][2 * u], o[d][2 * u + 1]);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        // 8 threads a row, each a run of columns in steps of 8 x 4
        const int r = threadIdx.x >> 3, rg = rt * kRowTile + r;
        if (rg < G * p.n) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w * kRowTile + r]);
            const float b2 = top == -INFINITY ? 0.f : top;
            float f[kWarps], sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                f[w] = exp2_fast(s_m[w * kRowTile + r] - b2);
                sum += f[w] * s_l[w * kRowTile + r];
            }
            const long long t = static_cast<long long>(b) * p.n + rg / G;
            const int h = hk * G + rg % G;
            const bool split = p.parts > 1;
            const float inv = split ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
            const long long at = (t * p.a.Hq + h) * p.parts + part;
            if (split && (threadIdx.x & 7) == 0) {
                p.part_ml[2 * at] = top;
                p.part_ml[2 * at + 1] = sum;
            }
            for (int col = (threadIdx.x & 7) * 8; col < D; col += 64) {
                float v[8] = {};
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4* src =
                        reinterpret_cast<const float4*>(merge + (w * kRowTile + r) * C::PITCH + col);
                    const float4 x = src[0], y = src[1];
                    v[0] += f[w] * x.x, v[1] += f[w] * x.y, v[2] += f[w] * x.z, v[3] += f[w] * x.w;
                    v[4] += f[w] * y.x, v[5] += f[w] * y.y, v[6] += f[w] * y.z, v[7] += f[w] * y.w;
                }
                if (split) {
                    float4* dst = reinterpret_cast<float4*>(p.part + at * D + col);
                    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                } else {
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

// Joins the parts of each row, in part order: one warp a row, four columns a lane.
__global__ void __launch_bounds__(128) join_kernel(const Params p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (__any_sync(~0u, stopped(p.err))) return;
    const int n = p.n, Hq = p.a.Hq, D = p.a.D;
    if (row >= static_cast<long long>(p.B) * n * Hq) return;
    const long long t = row / Hq;
    const int len = p.lens[t / n];
    if (len < 0 || len > p.max_kv) return;
    const int parts = max(1, (len + p.chunk - 1) / p.chunk);
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + row * p.parts;
    float top = -INFINITY;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, ml[i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const float b2 = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* src = p.part + row * p.parts * D + lane * 4;
    for (int i0 = 0; i0 < parts; i0 += 32) {
        const float2 e = i0 + lane < parts ? ml[i0 + lane] : make_float2(-INFINITY, 0.f);
        const float f = exp2_fast(e.x - b2);
        const float w = e.y == 0.f ? 0.f : f * e.y;
        const int m = min(32, parts - i0);
        for (int i1 = 0; i1 < m; i1 += 8) {  // eight parts' loads in flight
            float4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i1 + i < m && lane * 4 < D)
                    x[i] = *reinterpret_cast<const float4*>(src + static_cast<long long>(i0 + i1 + i) * D);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float fi = __shfl_sync(~0u, f, i1 + i), wi = __shfl_sync(~0u, w, i1 + i);
                if (i1 + i >= m) break;
                sum += wi;
                acc.x += fi * x[i].x, acc.y += fi * x[i].y, acc.z += fi * x[i].z, acc.w += fi * x[i].w;
            }
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (lane * 4 < D) {
        uint2 v = make_uint2(0u, 0u);
        if (sum != 0.f)
            v = make_uint2(pack2(acc.x * inv, acc.y * inv), pack2(acc.z * inv, acc.w * inv));
        *reinterpret_cast<uint2*>(p.out.row(t, static_cast<int>(row % Hq)) + lane * 4) = v;
    }
}

// Tokens of a part: about eight parts for every CTA that the GPU holds at once, so that
// uneven sequences even out, between 128 tokens (two stages, below which the merge costs
// more than the reads) and 2048 (where writing and reading the partial results of one tile of
// 16 rows moves under 2% of the bytes that the part reads; each further row tile adds as much,
// while its cache reads come from L2).
struct Plan {
    int chunk, parts, row_tiles;
};
Plan plan_of(const moe_attn_shape& a, int B, int n, int max_kv) {
    const int row_tiles = (a.Hq / a.Hkv * n + kRowTile - 1) / kRowTile;
    const long long tokens = static_cast<long long>(B) * a.Hkv * row_tiles * max_kv;
    long long chunk = tokens / (static_cast<long long>(num_sms()) * 2 * 8);
    chunk = chunk < 128 ? 128 : chunk > 2048 ? 2048 : chunk;
    chunk = (chunk + kTokens - 1) / kTokens * kTokens;
    const long long parts = max_kv > 0 ? (max_kv + chunk - 1) / chunk : 1;
    return {static_cast<int>(chunk), static_cast<int>(parts), row_tiles};
}

template <int DP>
cudaError_t decode(const Decode& d, cudaStream_t st) {
    using C = Cfg<DP>;
    const Plan pl = plan_of(d.a, d.B, d.n, d.max_kv);
    const long long rows = static_cast<long long>(d.B) * d.n * d.a.Hq;
    const long long items = static_cast<long long>(d.B) * d.a.Hkv * pl.parts * pl.row_tiles;
    if (items > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const Params p{d.a, d.B, d.n, d.max_kv, d.scale, d.q, d.out, d.pages, d.page_shift, d.block_table,
                   d.table_stride, d.kv_lens, d.part, d.part + rows * pl.parts * d.a.D, pl.parts,
                   pl.chunk, pl.row_tiles, d.err};
    CUtensorMap mk, mv;
    const uint64_t cache_rows = (static_cast<uint64_t>(d.pages) * d.a.Hkv) << d.page_shift;
    const uint32_t box = (1 << d.page_shift) < kTokens ? (1 << d.page_shift) : kTokens;
    if (!make_tmap_bf16(&mk, d.k_pages, cache_rows, d.a.D, 64, box) ||
        !make_tmap_bf16(&mv, d.v_pages, cache_rows, d.a.D, 64, box))
        return cudaErrorInvalidValue;
    auto kfn = decode_kernel<DP>;
    cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    {
        LaunchScope ls("attention_decode", st);
        e = launch_pdl(kfn, dim3(static_cast<unsigned>(items)), dim3(kThreads), C::SMEM, st, mk, mv, p);
        if (e != cudaSuccess || pl.parts == 1) return e;
    }
    LaunchScope ls("attention_join", st);
    return launch_pdl(join_kernel, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, st, p);
}

}  // namespace

size_t decode_ws_floats(const moe_attn_shape& a, int B, int n, int max_kv) {
    const Plan pl = plan_of(a, B, n, max_kv);
    if (pl.parts == 1) return 0;
    return static_cast<size_t>(B) * n * a.Hq * pl.parts * (a.D + 2);
}

cudaError_t launch_attention_decode(const Decode& p, cudaStream_t st) {
    return p.a.D <= 64 ? decode<64>(p, st) : decode<128>(p, st);
}

}  // namespace attn
}  // namespace moe
