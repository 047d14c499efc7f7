// evict.cu — the tokens of each sequence and key/value head that a cache keeps, and their way
// into other pages.
//
// select_kernel, a CTA for each (sequence, head): the weights that compete are read once, as
// whole numbers in their order, into shared memory (again from the pages at every use where a
// sequence is longer than that holds); the m-th largest by a radix select in three passes of 11,
// 11 and 10 bits; then the kept tokens' places in order: each warp counts, and then writes, those
// of a run of its own that are above that weight, and the first of those that have just that.
// gather_kernel, a CTA for each new page of a head: its rows from their old pages, 2 x 2 D bytes
// (D for e4m3) read and written a token; with e4m3 pages the new scale is the largest of the rows'
// and the others are moved to it.
//
// One sequence of 32768 tokens and 8 heads (8 CTAs): select 32 us, of which about 5 for each of
// its five sweeps over a CTA's keys (132 us with a page lookup and a load for each key and sweep);
// 64 sequences of up to 16384 tokens: 50 us. Four copies of the bins, or twice the registers,
// change nothing. Gather of the latter (0.93 GB) about 180 us, 5.2 TB/s: what does not depend on
// another load comes first, as a block's chain is lengths and places -> pages -> rows and scales
// (210 us with scales before rows and products in fp32).
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kSelect = 1024;  // threads
constexpr int kGather = 256;

// Whole numbers in the order of the weights (NaN below all; -0 as 0).
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

constexpr int kBins = 2048;
constexpr int kHeld = 48 * 1024;  // weights in shared memory at most: 192 KB

// How many of a warp's keys are above the last one kept, and at it.
struct Count {
    int more, same;
};

// HELD: keys in shared memory.
template <bool HELD>
__global__ void __launch_bounds__(kSelect, 2) select_kernel(const Evict p) {
    extern __shared__ __align__(16) uint32_t s_key[];
    __shared__ int s_bins[kBins];
    __shared__ int s_warp[kSelect / 32];
    __shared__ Count s_count[kSelect / 32];
    __shared__ int s_digit, s_left;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hk = blockIdx.x % p.Hkv, b = blockIdx.x / p.Hkv;
    const int len = p.lens[b], sh = p.page_shift;
    if (__syncthreads_or(stopped(p.err))) return;
    int* kept = p.kept + static_cast<long long>(blockIdx.x) * p.keep;
    const bool bad = len < 0 || len > p.max_kv;
    if (bad && tid == 0) raise_error(p.err, MOE_ERR_BAD_INDEX);
    if (bad || len <= p.keep) {
        for (int i = tid; i < p.keep; i += kSelect) kept[i] = !bad && i < len ? i : -1;
        return;
    }
    const int rivals = len - p.recent, m = p.keep - p.recent;  // m < rivals
    for (int i = tid; i < p.recent; i += kSelect) kept[m + i] = rivals + i;
    if (m == 0) return;
    const int32_t* table = p.block_table + static_cast<long long>(b) * p.table_stride;
    // four tokens at a time, which share a page; a page that is not there is reported
    const auto page_of = [&](int t) {
        const int page = t < rivals ? table[t >> sh] : 0;
        return page >= 0 && page < p.pages ? page : -1;
    };
    const auto at = [&](int page, int t) {
        const float4 w = *reinterpret_cast<const float4*>(
            p.weights + ((static_cast<long long>(max(page, 0)) * p.Hkv + hk) << sh) + (t & ((1 << sh) - 1)));
        return make_uint4(key_of(w.x), key_of(w.y), key_of(w.z), key_of(w.w));
    };
    const auto read = [&](int t) {
        const int page = page_of(t);
        if (page < 0) raise_error(p.err, MOE_ERR_BAD_INDEX);
        return at(page, t);
    };
    const auto keys = [&](int t, uint32_t (&k)[4]) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (t < rivals) v = HELD ? *reinterpret_cast<const uint4*>(s_key + t) : read(t);
        k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
    };
    for (int i = tid; i < kBins; i += kSelect) s_bins[i] = 0;
    if constexpr (HELD) {
        bool missing = false;
        for (int t0 = 4 * tid; t0 < rivals; t0 += 4 * 4 * kSelect) {  // four loads in flight
            int page[4];
            uint4 k[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) page[u] = page_of(t0 + u * 4 * kSelect);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                missing |= page[u] < 0;
                k[u] = at(page[u], t0 + u * 4 * kSelect);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (t0 + u * 4 * kSelect < rivals)
                    *reinterpret_cast<uint4*>(s_key + t0 + u * 4 * kSelect) = k[u];
        }
        if (missing) raise_error(p.err, MOE_ERR_BAD_INDEX);
    }
    __syncthreads();
    uint32_t last = 0, mask = 0;  // the m-th largest key; `left` of those that have it are kept
    int left = m;
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
        for (int t0 = warp * 128; t0 < rivals; t0 += 4 * kSelect) {
            const int t = t0 + 4 * lane;
            uint32_t k[4];
            keys(t, k);
            int digit[4];
            bool same = true;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = t + e < rivals && (k[e] & mask) == last;
                digit[e] = in ? static_cast<int>((k[e] >> shift) & (bins - 1)) : -1;
                same &= digit[e] == digit[0];
            }
            // equal digits all over the warp (weights that are all alike) are added at once
            const int first = __shfl_sync(~0u, digit[0], 0);
            if (__all_sync(~0u, same && digit[0] == first)) {
                if (lane == 0 && first >= 0) atomicAdd(&s_bins[first], 128);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (digit[e] >= 0) atomicAdd(&s_bins[digit[e]], 1);
            }
        }
        __syncthreads();
        // the bin with the left-th largest: thread i has bins 2 i, 2 i + 1, counted from above
        const int i = bins / 2 - 1 - tid;
        const int hi = i >= 0 ? s_bins[2 * i + 1] : 0, lo = i >= 0 ? s_bins[2 * i] : 0;
        int above = hi + lo;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, above, o);
            if (lane >= o) above += y;
        }
        if (lane == 31) s_warp[warp] = above;
        __syncthreads();
        int before = 0;
#pragma unroll
        for (int w = 0; w < kSelect / 32; ++w) before += w < warp ? s_warp[w] : 0;
        before += above - hi - lo;  // in bins above this thread's
        if (before < left && left <= before + hi + lo) {
            s_digit = 2 * i + (left <= before + hi);
            s_left = left <= before + hi ? left - before : left - before - hi;
        }
        if (i >= 0) s_bins[2 * i] = s_bins[2 * i + 1] = 0;
        __syncthreads();
        last |= static_cast<uint32_t>(s_digit) << shift;
        left = s_left;
        mask |= static_cast<uint32_t>(bins - 1) << shift;
    }
    const int run = (rivals + 4 * kSelect - 1) / (4 * kSelect) * 128;  // tokens of a warp
    const int begin = min(rivals, warp * run), end = min(rivals, begin + run);
    // of four tokens: how many are above `last`, and, in the upper half, how many are at it
    const auto count = [&](int t, const uint32_t (&k)[4]) {
        int n = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (t + e < rivals) n += k[e] > last ? 1 : k[e] == last ? 1 << 16 : 0;
        return n;
    };
    int more = 0, same = 0;
    for (int t0 = begin; t0 < end; t0 += 128) {
        uint32_t k[4];
        keys(t0 + 4 * lane, k);
        const int n = count(t0 + 4 * lane, k);
        more += n & 0xffff;
        same += n >> 16;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        more += __shfl_xor_sync(~0u, more, o);
        same += __shfl_xor_sync(~0u, same, o);
    }
    if (lane == 0) s_count[warp] = Count{more, same};
    __syncthreads();
    more = same = 0;
#pragma unroll
    for (int w = 0; w < kSelect / 32; ++w) {
        more += w < warp ? s_count[w].more : 0;
        same += w < warp ? s_count[w].same : 0;
    }
    for (int t0 = begin; t0 < end; t0 += 128) {
        const int t = t0 + 4 * lane;
        uint32_t k[4];
        keys(t, k);
        const int n = count(t, k);
        int upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, upto, o);
            if (lane >= o) upto += y;
        }
        int above = more + ((upto - n) & 0xffff), ties = same + ((upto - n) >> 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (t + e >= rivals) break;
            const int at = above + min(ties, left);
            if (k[e] > last || (k[e] == last && ties < left)) kept[at] = t + e;
            above += k[e] > last;
            ties += k[e] == last;
        }
        const int all = __shfl_sync(~0u, upto, 31);
        more += all & 0xffff;
        same += all >> 16;
    }
}

template <bool E8>
__global__ void __launch_bounds__(kGather)
gather_kernel(const Evict p, int new_pages, int lane_shift) {
    __shared__ int s_row[256];       // rows of the cache that the new rows come from
    __shared__ float s_old[2][256];  // E8: their scales (keys, values)
    __shared__ float s_top[2][kGather / 32];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int j = static_cast<int>(blockIdx.x % new_pages), unit = static_cast<int>(blockIdx.x / new_pages);
    const int hk = unit % p.Hkv, b = unit / p.Hkv, sh = p.page_shift;
    // what does not depend on another load comes first
    const int len = p.lens[b];
    const int goal = p.new_table[static_cast<long long>(b) * p.new_stride + j];
    const int place = (j << sh) + tid;  // in the new sequence
    int t = -1;
    if (tid < 1 << sh && place < p.keep) t = p.kept[static_cast<long long>(unit) * p.keep + place];
    if (__syncthreads_or(stopped(p.err)) || len < 0 || len > p.max_kv) return;  // reported by select_kernel
    const int n = min(len, p.keep);
    // (new_lens may be the lengths themselves: whichever of the two is read, n is the same)
    if (j == 0 && hk == 0 && tid == 0) p.new_lens[b] = n;
    const int rows = min(1 << sh, n - (j << sh));
    if (rows <= 0) return;
    bool bad = goal < 0 || goal >= p.pages;
    int page = 0;
    if (tid < rows) {
        page = t < 0 || t >= p.max_kv ? -1 : p.block_table[static_cast<long long>(b) * p.table_stride + (t >> sh)];
        bad |= page < 0 || page >= p.pages;
        s_row[tid] = bad ? 0 : ((page * p.Hkv + hk) << sh) + (t & ((1 << sh) - 1));
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) raise_error(p.err, MOE_ERR_BAD_INDEX);
        return;
    }
    // a row's pieces of 16 bytes on 1 << lane_shift lanes, two rows' loads in flight
    const int chunks = p.D * (E8 ? 1 : 2) / 16;
    const int c = tid & ((1 << lane_shift) - 1), step = kGather >> lane_shift;
    uint4 v[2][2];
    const auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = i0 + u * step;
            if (i < rows && c < chunks) {
                const long long at = static_cast<long long>(s_row[i]) * chunks + c;
                v[u][0] = reinterpret_cast<const uint4*>(p.k_pages)[at];
                v[u][1] = reinterpret_cast<const uint4*>(p.v_pages)[at];
            }
        }
    };
    load(tid >> lane_shift);
    const float weight = tid < rows ? p.weights[s_row[tid]] : 0.f;
    const int goal_row = (goal * p.Hkv + hk) << sh;
    float top[2] = {0.f, 0.f};
    if constexpr (E8) {
        if (tid < rows) {
            const long long at = static_cast<long long>(page) * p.Hkv + hk;
            top[0] = s_old[0][tid] = p.k_scale[at];
            top[1] = s_old[1][tid] = p.v_scale[at];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], o));
            if (lane == 0) s_top[x][warp] = top[x];
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int w = 0; w < kGather / 32; ++w) top[x] = fmaxf(top[x], s_top[x][w]);
        if (tid < 2) (tid == 0 ? p.k_scale : p.v_scale)[static_cast<long long>(goal) * p.Hkv + hk] = top[tid];
    }
    if (tid < rows) p.weights[goal_row + tid] = weight;
    for (int i0 = tid >> lane_shift; i0 < rows; i0 += 2 * step) {
        if (i0 >= 2 * step) load(i0);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = i0 + u * step;
            if (i >= rows || c >= chunks) continue;
            if constexpr (E8) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float old = s_old[x][i];
                    if (old != top[x]) v[u][x] = rescale_e4m3x16(v[u][x], old / top[x]);
                }
            }
            const long long at = static_cast<long long>(goal_row + i) * chunks + c;
            reinterpret_cast<uint4*>(p.k_pages)[at] = v[u][0];
            reinterpret_cast<uint4*>(p.v_pages)[at] = v[u][1];
        }
    }
}

}  // namespace

cudaError_t launch_evict(const Evict& p, cudaStream_t st) {
    const int most = p.max_kv < p.keep ? p.max_kv : p.keep;
    const int size = 1 << p.page_shift;
    const int new_pages = most < 1 ? 1 : (most - 1) / size + 1;
    const long long items = static_cast<long long>(p.B) * p.Hkv * new_pages;
    if (items > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    {
        const bool held = p.max_kv <= kHeld;
        const int smem = held ? 4 * p.max_kv + 16 : 0;
        auto kfn = held ? select_kernel<true> : select_kernel<false>;
        cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kHeld + 16);
        if (e != cudaSuccess) return e;
        LaunchScope ls("kv_select", st);
        e = launch_pdl(kfn, dim3(static_cast<unsigned>(p.B * p.Hkv)), dim3(kSelect), smem, st, p);
        if (e != cudaSuccess) return e;
    }
    int lane_shift = 0;
    while ((16 << lane_shift) < p.D * (p.k_scale != nullptr ? 1 : 2)) ++lane_shift;
    LaunchScope ls("kv_gather", st);
    return launch_pdl(p.k_scale != nullptr ? gather_kernel<true> : gather_kernel<false>,
                      dim3(static_cast<unsigned>(items)), dim3(kGather), 0, st, p, new_pages, lane_shift);
}

}  // namespace attn
}  // namespace moe
