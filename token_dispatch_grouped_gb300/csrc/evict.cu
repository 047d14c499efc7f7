// evict.cu — the tokens of each sequence and key/value head that a cache keeps, and their way
// into other pages.
//
// select_kernel, a CTA for each (sequence, head): the m-th largest of the weights that compete
// by a radix select over their bits as ordered whole numbers (8 bits a pass), then the kept
// tokens' places in order, by running counts of the tokens above that weight and of those that
// have just that (the first of them are kept). gather_kernel, a CTA for each new page of a
// head: its rows from their old pages, 2 x 2 D bytes (D for e4m3) read and written a token;
// with e4m3 pages the new scale is the largest of the rows' and the others are moved to it.
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

// Tokens before this thread's whose flag is set, and the block's sum (every thread calls).
__device__ __forceinline__ int count_before(bool flag, int* s_warp, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned votes = __ballot_sync(~0u, flag);
    __syncthreads();
    if (lane == 0) s_warp[warp] = __popc(votes);
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kSelect / 32; ++w) {
        const int c = s_warp[w];
        before += w < warp ? c : 0;
        total += c;
    }
    return before + __popc(votes & ((1u << lane) - 1));
}

__global__ void __launch_bounds__(kSelect) select_kernel(const Evict p) {
    __shared__ int s_hist[256];
    __shared__ int s_warp[kSelect / 32];
    __shared__ uint32_t s_digit;
    __shared__ int s_left;
    pdl_wait();
    pdl_trigger();
    if (__syncthreads_or(stopped(p.err))) return;
    const int tid = threadIdx.x;
    const int hk = blockIdx.x % p.Hkv, b = blockIdx.x / p.Hkv;
    const int len = p.lens[b], sh = p.page_shift;
    int* kept = p.kept + static_cast<long long>(blockIdx.x) * p.keep;
    const bool bad = len < 0 || len > p.max_kv;
    if (bad && tid == 0) raise_error(p.err, MOE_ERR_BAD_INDEX);
    if (bad || len <= p.keep) {
        for (int i = tid; i < p.keep; i += kSelect) kept[i] = !bad && i < len ? i : -1;
        return;
    }
    const int32_t* table = p.block_table + static_cast<long long>(b) * p.table_stride;
    const auto key = [&](int t) {  // a page that is not there is reported by gather or here
        const int page = table[t >> sh];
        if (page < 0 || page >= p.pages) {
            raise_error(p.err, MOE_ERR_BAD_INDEX);
            return 0u;
        }
        return key_of(p.weights[((static_cast<long long>(page) * p.Hkv + hk) << sh) + (t & ((1 << sh) - 1))]);
    };
    const int rivals = len - p.recent, m = p.keep - p.recent;  // m < rivals
    uint32_t last = 0;  // the m-th largest key; `left` of those that have it are kept
    int left = 0;
    if (m > 0) {
        left = m;
        uint32_t mask = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) s_hist[tid] = 0;
            __syncthreads();
            for (int t = tid; t < rivals; t += kSelect) {
                const uint32_t k = key(t);
                if ((k & mask) == last) atomicAdd(&s_hist[k >> shift & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int d = 255, n = left;
                for (; d > 0 && s_hist[d] < n; --d) n -= s_hist[d];
                s_digit = d;
                s_left = n;
            }
            __syncthreads();
            last |= s_digit << shift;
            left = s_left;
            mask |= 255u << shift;
        }
    }
    int at = 0, same = 0;  // tokens kept, and tokens at the last weight, so far
    for (int t0 = 0; t0 < rivals && m > 0; t0 += kSelect) {
        const int t = t0 + tid;
        const uint32_t k = t < rivals ? key(t) : 0u;
        const bool tie = t < rivals && k == last;
        int ties, n;
        const int tie_at = same + count_before(tie, s_warp, ties);
        const bool mine = (t < rivals && k > last) || (tie && tie_at < left);
        const int i = at + count_before(mine, s_warp, n);
        if (mine && i < p.keep) kept[i] = t;
        same += ties;
        at += n;
    }
    for (int i = tid; i < p.recent; i += kSelect) kept[m + i] = rivals + i;
}

template <bool E8>
__global__ void __launch_bounds__(kGather) gather_kernel(const Evict p, int new_pages) {
    __shared__ int s_row[256];     // rows of the cache that the new rows come from
    __shared__ float s_old[2][256];  // E8: their scales (keys, values)
    __shared__ float s_top[2][kGather / 32];
    pdl_wait();
    pdl_trigger();
    if (__syncthreads_or(stopped(p.err))) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long item = blockIdx.x;
    const int j = static_cast<int>(item % new_pages);
    item /= new_pages;
    const int hk = static_cast<int>(item % p.Hkv), b = static_cast<int>(item / p.Hkv);
    const int len = p.lens[b], sh = p.page_shift;
    if (len < 0 || len > p.max_kv) return;  // reported by select_kernel
    const int n = min(len, p.keep);
    // (new_lens may be the lengths themselves: whichever of the two is read, n is the same)
    if (j == 0 && hk == 0 && tid == 0) p.new_lens[b] = n;
    const int rows = min(1 << sh, n - (j << sh));
    if (rows <= 0) return;
    const int goal = p.new_table[static_cast<long long>(b) * p.new_stride + j];
    bool bad = goal < 0 || goal >= p.pages;
    float kt = 0.f, vt = 0.f;
    if (tid < rows) {
        const int t = p.kept[(static_cast<long long>(b) * p.Hkv + hk) * p.keep + (j << sh) + tid];
        const int page = t < 0 || t >= len ? -1
                                           : p.block_table[static_cast<long long>(b) * p.table_stride + (t >> sh)];
        bad |= page < 0 || page >= p.pages;
        if (!bad) {
            s_row[tid] = ((page * p.Hkv + hk) << sh) + (t & ((1 << sh) - 1));
            if constexpr (E8) {
                const long long at = static_cast<long long>(page) * p.Hkv + hk;
                kt = s_old[0][tid] = p.k_scale[at];
                vt = s_old[1][tid] = p.v_scale[at];
            }
        }
    }
    if constexpr (E8) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            kt = fmaxf(kt, __shfl_xor_sync(~0u, kt, o));
            vt = fmaxf(vt, __shfl_xor_sync(~0u, vt, o));
        }
        if (lane == 0) s_top[0][warp] = kt, s_top[1][warp] = vt;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) raise_error(p.err, MOE_ERR_BAD_INDEX);
        return;
    }
    const int goal_row = (goal * p.Hkv + hk) << sh;
    float top[2] = {0.f, 0.f};
    if constexpr (E8) {
#pragma unroll
        for (int w = 0; w < kGather / 32; ++w) {
            top[0] = fmaxf(top[0], s_top[0][w]);
            top[1] = fmaxf(top[1], s_top[1][w]);
        }
        if (tid < 2) (tid == 0 ? p.k_scale : p.v_scale)[static_cast<long long>(goal) * p.Hkv + hk] = top[tid];
    }
    if (tid < rows) p.weights[goal_row + tid] = p.weights[s_row[tid]];
    const int bytes = p.D * (E8 ? 1 : 2), chunks = bytes / 16;
    for (int x = tid; x < 2 * rows * chunks; x += kGather) {
        const int which = x >= rows * chunks, y = which ? x - rows * chunks : x;
        const int i = y / chunks, c = y % chunks;
        uint8_t* pages = which ? p.v_pages : p.k_pages;
        uint4 v = reinterpret_cast<const uint4*>(pages + static_cast<long long>(s_row[i]) * bytes)[c];
        if constexpr (E8) {
            const float old = s_old[which][i];
            if (old != top[which]) {
                const float f = old / top[which];
                v.x = rescale_e4m3x4(v.x, f);
                v.y = rescale_e4m3x4(v.y, f);
                v.z = rescale_e4m3x4(v.z, f);
                v.w = rescale_e4m3x4(v.w, f);
            }
        }
        reinterpret_cast<uint4*>(pages + static_cast<long long>(goal_row + i) * bytes)[c] = v;
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
        LaunchScope ls("kv_select", st);
        const cudaError_t e = launch_pdl(select_kernel, dim3(static_cast<unsigned>(p.B * p.Hkv)),
                                         dim3(kSelect), 0, st, p);
        if (e != cudaSuccess) return e;
    }
    LaunchScope ls("kv_gather", st);
    return launch_pdl(p.k_scale != nullptr ? gather_kernel<true> : gather_kernel<false>,
                      dim3(static_cast<unsigned>(items)), dim3(kGather), 0, st, p, new_pages);
}

}  // namespace attn
}  // namespace moe
