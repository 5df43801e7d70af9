// lora.cuh -- shared by the kernels of the low-rank adapters (lora.cu, prefill.cu,
// dgrad.cu): the token plan, and the splitting of fp32 factors into bf16 terms.
#pragma once

#include "common.cuh"

#include <cuda_bf16.h>

namespace sherry {

constexpr int kLoraTile = 128;  // tokens per tile of the tensor-core kernels

// Which adapters each 128-token tile holds, built on the device from the ids (k_lora_plan).
// A slot is one (tile, adapter) pair with a token in it.  Tokens stay where they are while
// the slots are few; where tokens of many adapters alternate they are taken adapter by
// adapter instead (`perm`), tokens of none (any id outside [0, n_adapters)) last, which
// leaves at most tiles + n_adapters slots.  The kernels then read rows that k_lora_rows
// has put in that order, and write to the tokens' own rows.
struct LoraPlan {
    int32_t* head;    // [0]: 1 where tokens are taken in perm's order; [1]: number of slots
    int32_t* perm;    // [M] the token at each position (only where head[0])
    int32_t* tile_b;  // [tiles + 1] first slot of each tile
    int32_t* slot_a;  // [max_slots] the slot's adapter
    int32_t* slot_t;  // [max_slots] its tile
    int32_t* adap_b;  // [n_adapters + 1] where each adapter's slots start in adap_s
    int32_t* adap_s;  // [max_slots] slots, adapter by adapter, in order
    int32_t* bad;     // [n_adapters] 1 where A_a holds a NaN or an infinity (k_lora_down, for the input gradient)
    uint32_t* mask;   // [max_slots][4] which of the tile's 128 tokens the slot has (written by k_lora_down)
    int64_t tiles;
    int max_slots;
    int may_permute;  // 0: the ids cannot make more slots than max_slots
};

// The slot's rows among 128 positions hold U or P split into bf16 terms whose sum is the value to
// 16 (two terms) or 24 (three) bits, zero for tokens of other adapters: [max_slots * 128][terms * rp],
// rp the rank rounded up to 16.
struct LoraImage {
    uint16_t* data;
    int rp, terms;
};
static inline int lora_rp(int R) { return (R + 15) / 16 * 16; }

// the next term of (x, y), each the bf16 nearest to what is left; the differences are exact in fp32, so two
// terms keep 16 significant bits and three all 24.  An infinity or NaN is its own first term.
__device__ __forceinline__ uint32_t split_next(float& x, float& y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    x -= __low2float(h);
    y -= __high2float(h);
    if (!(fabsf(x) < INFINITY)) x = 0.0f;
    if (!(fabsf(y) < INFINITY)) y = 0.0f;
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The input gradient multiplies alpha / unit: unit = (the mean of 32 scales spread over the weight's n) / kGTop, so that
// a per-tensor scale is one bf16 (dgrad.cu), or 1 where that is no ordinary number.  P is held in the same unit.
// Called by whole warps.
constexpr float kGTop = 1.71875f;
__device__ __forceinline__ float dgrad_unit(const float* scales, int64_t n) {
    float a = __ldg(scales + n * (int64_t)(threadIdx.x & 31) / 32);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
    a *= 1.0f / 32.0f;  // (a per-tensor scale: itself, exactly)
    return (a > 1e-30f && a < 1e30f) ? a / kGTop : 1.0f;
}
static inline int64_t scale_count(const ProbShape& s) {
    return s.granularity == SHERRY_PER_TENSOR ? 1 : s.granularity == SHERRY_PER_CHANNEL ? s.N : s.N * (s.K / s.group);
}

// What the prefill kernel needs to add the adapters' product
struct LoraArgs {
    const uint16_t* B;  // bf16 [n_adapters][N][R]
    LoraImage U;
    const uint16_t* Xp; // X in perm's order (null: the plan cannot permute)
    int R, n_adapters;
    LoraPlan plan;
};
int prefill_lora_launch(const ProbShape& s, const sherry_linear_desc& d, int64_t M, int y_bf16, const LoraArgs& lora,
                        cudaStream_t stream);

int64_t prefill_lora_ctas(const ProbShape& s, int64_t M, int sms);  // of that launch

// What the input-gradient kernel needs to add P A_a
struct LoraGradArgs {
    const uint16_t* A;   // bf16 [n_adapters][R][K]
    LoraImage P;         // in dgrad_unit's unit
    const uint16_t* Gp;  // dY in perm's order (null: the plan cannot permute)
    int R, n_adapters;
    LoraPlan plan;
};
int64_t dgrad_ctas(const ProbShape& s, int64_t M, int n_adapters, int R, int sms);  // 0 adapters: the plain gradient
// dX = dY (T alpha) (+ P A_a): dY bf16 rows ldy apart (a multiple of 8), lora null for the plain gradient (dgrad.cu)
size_t dgrad_workspace_bytes(int64_t M, int64_t N, int64_t K, int n_adapters, int R, int sms);
int dgrad_launch(const ProbShape& s, const uint32_t* idx, const uint8_t* sgn, const float* scales, const uint16_t* dY,
                 int64_t ldy, int64_t M, uint16_t* dX, const LoraGradArgs* lora, void* workspace, int sms,
                 cudaStream_t stream);
// where the rows were split over CTAs: dX from their partial sums; otherwise nothing
int dgrad_join_launch(const ProbShape& s, const float* scales, int64_t M, uint16_t* dX, const void* workspace,
                      int n_adapters, int R, int sms, cudaStream_t stream);

// bytes of a plan, and the plan laid out in `mem` (256-byte aligned)
size_t lora_plan_bytes(int64_t M, int n_adapters);
LoraPlan lora_plan_in(void* mem, int64_t M, int n_adapters);
int lora_plan_launch(const int32_t* ids, int64_t M, int n_adapters, const LoraPlan& plan, cudaStream_t stream);
// whether the ids of such a call may need more slots than there are
bool lora_may_permute(int64_t M, int n_adapters);
size_t lora_image_bytes(int64_t M, int n_adapters, int R, int terms);

// dst[p][0..ld) = src[token at position p][0..N), zeros from N on; where the plan does not
// permute, only if `always`
struct LoraRows {
    const uint16_t* src;
    uint16_t* dst;
    int64_t N, ld;
    int always;
};
int lora_rows_launch(const LoraRows* jobs, int count, int64_t M, const LoraPlan& plan, int sms, cudaStream_t stream);

// V[m][r] = scaling[a] * sum_c G[m][c] W_a(r, c), a the token's adapter, as fp32 rows (zero for tokens
// of none) and / or as an image; and the image of rows V2 that are there already.
struct LoraDown {
    const uint16_t* G;   // bf16 [M] rows ldg apart (a multiple of 8)
    const uint16_t* Gp;  // the same in perm's order (null: the plan cannot permute)
    int64_t ldg, C;
    const uint16_t* W;   // bf16 [n_adapters][R][C], or [n_adapters][C][R] with by_row; null: only V2's image
    int by_row;
    const int32_t* ids;
    const float* scaling;
    const float* unit;   // scales of the packed weight: the image holds V / dgrad_unit; or null
    int64_t unit_n;
    float* V;            // or null
    LoraImage img;       // data may be null
    const float* V2;     // or null
    LoraImage img2;
    const uint16_t* A;   // bf16 [n_adapters][R][K] to look through for what is not finite, or null
    int64_t K;
    int64_t beside_ctas; // CTAs (one per SM) of the kernel that follows
};
int lora_down_launch(const LoraDown& d, int64_t M, int R, int n_adapters, const LoraPlan& plan, int sms,
                     cudaStream_t stream);
// The whole operator for few tokens, without a plan (lora_few.cu); U fp32 [M][R] is written
constexpr int64_t kLoraFew = 32;  // tokens of one CTA
int lora_few_launch(const ProbShape& s, const sherry_linear_desc& d, int64_t M, int y_bf16, const uint16_t* A,
                    const uint16_t* B, int R, const int32_t* ids, const float* scaling, int n_adapters, float* U,
                    cudaStream_t stream);
// U alone, likewise
int lora_down_few_launch(const ProbShape& s, const sherry_linear_desc& d, int64_t M, const uint16_t* A, int R,
                         const int32_t* ids, const float* scaling, int n_adapters, float* U, cudaStream_t stream);
// Y[m][n] = Yin[m][n] + sum_r U[m][r] B[a][n][r]
int lora_up_launch(const float* Yin, int64_t M, int64_t N, const float* U, const uint16_t* B, int R,
                   const int32_t* ids, int n_adapters, void* Y, int y_bf16, cudaStream_t stream);

// One gradient of the adapters: sum over adapter a's tokens of V[m][r] G[m][c] (times dgrad_unit of
// `unit` where that is not null), written as [a][r][c] (by_column = 0) or [a][c][r] (by_column = 1).
struct LoraGradJob {
    LoraImage V;
    const uint16_t* G;    // bf16, rows ldg apart (a multiple of 8)
    const uint16_t* Gp;   // the same in perm's order (null: the plan cannot permute)
    int64_t ldg, C;
    void* out;            // fp32 or bf16
    const float* unit;
    int64_t unit_n;
    int by_column;
};
// `beside`: right after dgrad_launch's kernel, whose idle SMs it takes
int lora_grad_launch(const LoraGradJob* jobs, int count, int R, int n_adapters, int64_t M, const LoraPlan& plan,
                     int out_bf16, bool beside, int sms, cudaStream_t stream);
int lora_status_take();  // as stream_status_take

}  // namespace sherry
