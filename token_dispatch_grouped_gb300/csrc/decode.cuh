// decode.cuh — what the decode kernels over bf16 pages (decode.cu) and e4m3 pages (decode8.cu)
// share: their parameters, the split of the tokens, the workspace, fragments.
#pragma once
#include "attn_mma.cuh"

namespace moe {
namespace attn {

constexpr int kRowTile = 16;  // query heads x new tokens of a CTA

struct DecodeParams {
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
    const float *k_scale, *v_scale;  // e4m3 pages
    float* scores;  // weights: [sequence][head][row of its G n][pitch], base 2, -inf unseen
    float* lse;     // weights: [row], base 2, inf where nothing is seen
    int pitch;
    float* weights;
    int fresh;
};

// Tokens of a part, and how many parts the longest sequence has.
struct DecodePlan {
    int chunk, parts, row_tiles;
};
DecodePlan decode_plan(const moe_attn_shape& a, int B, int n, int max_kv, bool e8);

// Whether decode8.cu's CTAs stay and take numbered parts (with a count of the taken ones in the
// workspace, which a call without cached tokens has not): where the parts are more than the GPU
// holds at once and a CTA can number the sequences in shared memory.
constexpr int kNumberedSeqs = 1024;
inline bool decode_numbered(const moe_attn_shape& a, int B, int max_kv, const DecodePlan& pl) {
    return max_kv > 0 && B <= kNumberedSeqs &&
           static_cast<long long>(B) * a.Hkv * pl.parts * pl.row_tiles > 2 * num_sms();
}

// The workspace: partial results of the parts, then what the weights are summed from.
struct DecodeSpace {
    size_t part, lse, scores, total;  // in floats; each a multiple of 4
    int pitch;
};
DecodeSpace decode_space(const Decode& d, const DecodePlan& pl);
DecodeParams decode_params(const Decode& d, const DecodePlan& pl);

// The kernels behind the decode kernel: the parts joined, the weights summed.
cudaError_t launch_decode_rest(const DecodeParams& p, cudaStream_t st);
cudaError_t launch_decode8(const Decode& d, cudaStream_t st);

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

}  // namespace attn
}  // namespace moe
