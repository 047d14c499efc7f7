// decode.cu — attention of the newest tokens of each sequence over its paged cache.
//
// One warp per query row: the lanes take 32 cached tokens at a time for the dot
// products and 4 of the D columns each for the weighted sum, in one pass with a
// running maximum and sum.
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxD = 128;

__global__ void __launch_bounds__(kWarps * 32) decode_kernel(const Decode p) {
    __shared__ float s_q[kWarps][kMaxD];
    pdl_wait();
    pdl_trigger();
    if (has_error(p.err)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int Hq = p.a.Hq, Hkv = p.a.Hkv, D = p.a.D;
    const long long row = static_cast<long long>(blockIdx.x) * kWarps + warp;
    if (row >= static_cast<long long>(p.B) * p.n * Hq) return;
    const int t = static_cast<int>(row / Hq), h = static_cast<int>(row % Hq);
    const int hk = h / (Hq / Hkv), b = t / p.n;
    const int len = p.kv_lens[b];
    bool bad = len < 0 || len > p.max_kv;
    if (!bad)
        for (int pg = lane; pg << p.page_shift < len; pg += 32) {
            const int id = p.block_table[static_cast<long long>(b) * p.table_stride + pg];
            bad |= id < 0 || id >= p.pages;
        }
    if (__any_sync(~0u, bad)) {
        if (lane == 0) raise_error(p.err, MOE_ERR_BAD_INDEX);
        return;
    }
    for (int i = lane; i < D; i += 32) s_q[warp][i] = __bfloat162float(p.q.row(t, h)[i]);
    __syncwarp();
    auto at = [&](int j) {
        const long long page = p.block_table[static_cast<long long>(b) * p.table_stride + (j >> p.page_shift)];
        return (((page * Hkv + hk) << p.page_shift) + (j & ((1 << p.page_shift) - 1))) * D;
    };
    const int seen = min(len, t % p.n + len - p.n + 1);
    float m = -INFINITY, l = 0.f, acc[kMaxD / 32] = {};
    for (int j0 = 0; j0 < seen; j0 += 32) {
        const int j = j0 + lane;
        float s = -INFINITY;
        if (j < seen) {
            const bf16* k = p.k_pages + at(j);
            s = 0.f;
            for (int i = 0; i < D; i += 8) {
                float v[8];
                unpack8(*reinterpret_cast<const uint4*>(k + i), v);
                for (int e = 0; e < 8; ++e) s += s_q[warp][i + e] * v[e];
            }
            s *= p.scale;
        }
        float mx = s;
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
        const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.f : mn;
        const float w = j < seen ? __expf(s - base) : 0.f, keep = __expf(m - base);
        l = l * keep + w;
        m = mn;
        for (int c = 0; c < kMaxD / 32; ++c) acc[c] *= keep;
        for (int i = 0; i < min(32, seen - j0); ++i) {
            const float wi = __shfl_sync(~0u, w, i);
            const bf16* v = p.v_pages + at(j0 + i);
            for (int c = 0; c < kMaxD / 32; ++c)
                if (c * 32 + lane < D) acc[c] += wi * __bfloat162float(v[c * 32 + lane]);
        }
    }
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
    for (int c = 0; c < kMaxD / 32; ++c)
        if (c * 32 + lane < D)
            p.out.row(t, h)[c * 32 + lane] = __float2bfloat16(seen > 0 ? acc[c] / l : 0.f);
}

}  // namespace

size_t decode_ws_floats(const moe_attn_shape&, int, int, int) { return 0; }

cudaError_t launch_attention_decode(const Decode& p, cudaStream_t st) {
    const long long rows = static_cast<long long>(p.B) * p.n * p.a.Hq;
    LaunchScope ls("attention_decode", st);
    return launch_k(decode_kernel, dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps)),
                    dim3(kWarps * 32), 0, st, p);
}

}  // namespace attn
}  // namespace moe
