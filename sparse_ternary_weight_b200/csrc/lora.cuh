// lora.cuh -- shared by the kernels of the low-rank adapters (lora.cu, prefill.cu,
// dgrad.cu): the token plan, and the splitting of fp32 factors into bf16 terms.
#pragma once

#include "common.cuh"

#include <cuda_bf16.h>

namespace sherry {

constexpr int kLoraTile = 128;  // tokens per tile of the tensor-core kernels

// Tokens by adapter, built on the device from the ids (k_lora_plan).  Bucket a <
// n_adapters holds adapter a's tokens in order, bucket n_adapters those of none
// (any id outside [0, n_adapters)).
struct LoraPlan {
    int32_t* perm;    // [M] token indices, bucket after bucket
    int32_t* offs;    // [n_adapters + 2] where each bucket starts, and M
    int32_t* tile_n;  // [tiles] different adapters among each 128 tokens (in their own order)
    int32_t* tile_a;  // [tiles][kLoraTile] which
};

// Term `which` of x = t0 + t1 (+ t2), each the bf16 nearest to what is left: the
// differences are exact in fp32, so two terms keep 16 significant bits and three all 24.
__device__ __forceinline__ float split_term(float x, int which) {
    float t = __bfloat162float(__float2bfloat16_rn(x));
    for (int i = 0; i < which; ++i) {
        x -= t;
        t = __bfloat162float(__float2bfloat16_rn(x));
    }
    return t;
}
__device__ __forceinline__ uint32_t split_pair(float x, float y, int which) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(split_term(x, which), split_term(y, which));
    return *reinterpret_cast<const uint32_t*>(&h);
}

// What the prefill kernel needs to add the adapters' product
struct LoraArgs {
    const uint16_t* B;  // bf16 [n_adapters][N][R]
    const float* U;     // fp32 [M][R]
    const int32_t* ids;
    int R;
    LoraPlan plan;
};
int prefill_lora_launch(const ProbShape& s, const sherry_linear_desc& d, int64_t M, int y_bf16, const LoraArgs& lora,
                        cudaStream_t stream);

// dX = dY (T alpha) (+ Pm A_a): dY bf16 rows ldy apart (a multiple of 8), lora null for the plain gradient (dgrad.cu)
size_t dgrad_workspace_bytes(int64_t M, int64_t N, int64_t K, int sms);
int dgrad_launch(const ProbShape& s, const uint32_t* idx, const uint8_t* sgn, const float* scales, const uint16_t* dY,
                 int64_t ldy, int64_t M, uint16_t* dX, const LoraPlan* lora, const uint16_t* A, const float* Pm,
                 const int32_t* ids, int R, void* workspace, int sms, cudaStream_t stream);

// bytes of a plan, and the plan laid out in `mem` (256-byte aligned)
size_t lora_plan_bytes(int64_t M, int n_adapters);
LoraPlan lora_plan_in(void* mem, int64_t M, int n_adapters);
int lora_plan_launch(const int32_t* ids, int64_t M, int n_adapters, const LoraPlan& plan, cudaStream_t stream);

// V[m][r] = scaling[a] * sum_c G[m][c] W[a][r][c], a the token's adapter; 0 for tokens of none.
// G bf16 [M] rows ldg apart, W bf16 [n_adapters][R] rows ldw apart; C, ldg, ldw multiples of 8.
int lora_down_launch(const uint16_t* G, int64_t ldg, int64_t M, int64_t C, const uint16_t* W, int64_t ldw, int R,
                     const int32_t* ids, const float* scaling, int n_adapters, const LoraPlan& plan, float* V, int sms,
                     cudaStream_t stream);
// the same for a few tokens, without a plan
int lora_down_few_launch(const uint16_t* G, int64_t ldg, int64_t M, int64_t C, const uint16_t* W, int64_t ldw, int R,
                         const int32_t* ids, const float* scaling, int n_adapters, float* V, cudaStream_t stream);
// Y[m][n] = Yin[m][n] + sum_r U[m][r] B[a][n][r]
int lora_up_launch(const float* Yin, int64_t M, int64_t N, const float* U, const uint16_t* B, int R,
                   const int32_t* ids, int n_adapters, void* Y, int y_bf16, cudaStream_t stream);
// dst[a][r][0..ld) = src[a][n][r] over n, zeros from N on
int lora_transpose_launch(const uint16_t* src, int n_adapters, int64_t N, int R, uint16_t* dst, int64_t ld,
                          cudaStream_t stream);
// dst[m][0..ld) = src[m][0..N), zeros from N on
int lora_pad_launch(const uint16_t* src, int64_t M, int64_t N, uint16_t* dst, int64_t ld, cudaStream_t stream);

// One gradient of the adapters: sum over adapter a's tokens of V[m][r] G[m][c],
// written as [a][r][c] (by_column = 0) or [a][c][r] (by_column = 1); fp32 or bf16.
struct LoraGradJob {
    const float* V;       // fp32 [M][R]
    const uint16_t* G;    // bf16, rows ldg apart (a multiple of 8)
    int64_t ldg, C;
    void* out;
    int by_column;
};
int lora_grad_launch(const LoraGradJob* jobs, int count, int R, int n_adapters, int64_t M, const LoraPlan& plan,
                     int out_bf16, int sms, cudaStream_t stream);

}  // namespace sherry
