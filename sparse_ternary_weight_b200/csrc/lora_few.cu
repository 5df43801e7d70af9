// lora_few.cu -- the packed linear with adapters for a decode step's tokens, in two
// launches: Y[m] = X[m] (T alpha)^T + U[m] B_a^T, U[m] = s_a X[m] A_a^T ("Sherry, Tequila
// and Fairies in Python", section 1.1, has the layer; lora.cu the adapters).
//
// k_lora_down_few makes U, a CTA per token and four ranks.  k_lora_few is the linear
// and the product with B: 16 weight rows per CTA, whose eight warps split K in chunks
// of 128 weights.  The weights are expanded in registers as operand A of mma.sync
// (m16n8k16): a lane of place c takes blocks 2c and 2c + 1 of every word of its two
// rows, so that each block of 4 weights is one pair of k of A and the next, and the same
// order of k gives operand B as 16 bytes of a token's X per word.  Sums per scale group
// are fp32, promoted with alpha, and the warps' are joined in order.  The second
// launch starts beside the first and waits for U only then.
//
// Bound by latency: at 16 tokens x 8192 x 2048 no pipe is full (LSU 57%, a third of that
// bank conflicts between the rows that one load touches; issue slots 28%, DRAM 6%); the
// warps wait for loads 39% of their time, sixteen of them per SM (128 registers a thread), and 512
// CTAs are 1.7 waves.  10 us a call.  (At 1 x 8192 x 8192 the LSU is 80% busy.)  tcgen05's tiles of
// 128 rows would leave most SMs without one; rows of 16 give every SM three CTAs or more.
#include "lora.cuh"
#include "lut.cuh"
#include "tc.cuh"

#include <algorithm>

namespace sherry {

struct FewParams {
    const uint16_t* X;
    const uint16_t* A;
    const float* scaling;
    const int32_t* ids;
    float* U;
    int M, K, R, n_adapters;
};

__global__ void __launch_bounds__(128) k_lora_down_few(const FewParams P) {
    pdl_wait();
    pdl_trigger();  // only now: k_lora_few reads X at once, which the kernel before this one may write
    __shared__ float red[4][4];
    const int m = blockIdx.y, r0 = 4 * blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int a = P.ids[m];
    float* out = P.U + (int64_t)m * P.R + r0;
    if (a < 0 || a >= P.n_adapters) {
        if (threadIdx.x < 4) out[threadIdx.x] = 0.0f;
        return;
    }
    const uint16_t* x = P.X + (int64_t)m * P.K;
    const uint16_t* w = P.A + ((int64_t)a * P.R + r0) * P.K;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
    for (int k = 8 * threadIdx.x; k < P.K; k += 8 * 128) {
        const uint4 xv = __ldg(reinterpret_cast<const uint4*>(x + k));
        const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(w + (int64_t)r * P.K + k));
            const uint32_t vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[r] = fmaf(bf16lo(xs[j]), bf16lo(vs[j]), acc[r]);
                acc[r] = fmaf(bf16hi(xs[j]), bf16hi(vs[j]), acc[r]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) acc[r] += __shfl_xor_sync(kFull, acc[r], o);
        if (lane == 0) red[warp][r] = acc[r];
    }
    __syncthreads();
    if (threadIdx.x < 4) {
        const float s = (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
        out[threadIdx.x] = (P.scaling ? P.scaling[a] : 1.0f) * s;
    }
}

constexpr int kFewWarps = 8;
constexpr int kFewRows = 16;
constexpr int kFewPitch = 20;  // floats between tokens of the partial sums: their writes touch every bank once

struct FewUpParams {
    const uint16_t* X;
    const uint32_t* idx;
    const uint8_t* sgn;
    const float* scales;
    const uint16_t* B;
    const float* U;
    const int32_t* ids;
    void* Y;
    int M, N, K, words;
    int group_words, spr;  // words per scale group, and scales per row (0: one for all)
    int per_tensor;
    int R, n_adapters, y_bf16;
};

__device__ __forceinline__ void few_mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: tiles of 8 tokens.  SCALE: 0 per row or tensor (applied at the end) and 1 groups of whole chunks
// of 128 weights, both for K % 128 == 0; 2 all other shapes (loaded and promoted word by word)
template <int NT, int SCALE>
__global__ void __launch_bounds__(32 * kFewWarps, NT == 1 ? 3 : 2) k_lora_few(const __grid_constant__ FewUpParams P) {
    constexpr bool XAHEAD = NT <= 2;  // X is loaded with the words; for four tiles when it is used (registers)
    pdl_trigger();
    __shared__ __align__(256) uint32_t table[64];  // the 32 patterns' low halves, then high halves
    __shared__ float part[kFewWarps][8 * NT * kFewPitch];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int n0 = blockIdx.x * kFewRows, m0 = blockIdx.y * (8 * NT);  // rows and tokens of this CTA
    if (tid < 32) {
        const uint2 e = decode_block_bf16((uint32_t)tid & 15u, (uint32_t)tid >> 4);
        table[tid] = e.x;
        table[32 + tid] = e.y;
    }
    // B's rows are fetched beside the linear
    for (int o = tid; o < kFewRows * 8 * NT; o += 32 * kFewWarps) {
        const int n = n0 + o % kFewRows, m = m0 + o / kFewRows;
        if (m < P.M && n < P.N) {
            const int a = P.ids[m];
            if (a >= 0 && a < P.n_adapters) {
                const char* p = reinterpret_cast<const char*>(P.B + ((int64_t)a * P.N + n) * P.R);
                for (int b = 0; b < 2 * P.R; b += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + b));
            }
        }
    }
    __syncthreads();
    const uint32_t tab = smem_u32(table);
    // two rows per lane (past the last: the last again, not written)
    const int64_t ra = min(n0 + g, P.N - 1), rb = min(n0 + g + 8, P.N - 1);
    const uint32_t* ia = P.idx + ra * P.words;
    const uint32_t* ib = P.idx + rb * P.words;
    const uint8_t* sa = P.sgn + ra * P.words;
    const uint8_t* sb = P.sgn + rb * P.words;
    const float* al = P.scales + ra * P.spr;
    const float* bl = P.scales + rb * P.spr;
    constexpr bool vec = SCALE != 2;
    const int chunks = (P.words + 3) / 4;
    const int ch0 = chunks * warp / kFewWarps, ch1 = chunks * (warp + 1) / kFewWarps;
    struct Chunk {  // 128 weights of both rows and the tokens' X
        uint32_t a[4], b[4];
        uint32_t sa, sb;
        float al, bl;
        uint4 x[XAHEAD ? 4 : 1][NT];
    };
    const uint16_t* xr[NT];  // the lane's token of each tile (past the last: the last again), at its place in a word
#pragma unroll
    for (int t = 0; t < NT; ++t) xr[t] = P.X + (int64_t)min(m0 + 8 * t + g, P.M - 1) * P.K + 8 * c;
    auto fetch_x = [&](int ch, uint4 (*x)[NT]) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint4* p = reinterpret_cast<const uint4*>(xr[t] + 128 * ch);
#pragma unroll
            for (int j = 0; j < 4; ++j)  // past the row: zero
                x[j][t] = vec || 4 * ch + j < P.words ? __ldg(p + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    int group = 0, left = P.group_words / 4;  // SCALE 1: the fetched chunk's group, and its chunks from there on
    if (SCALE == 1) {
        group = ch0 / left;
        left -= ch0 % left;
    }
    auto fetch = [&](int ch, Chunk& w) {
        if (ch >= ch1) return;
        const int w0 = 4 * ch;
        if (vec) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(ia + w0)), y = __ldg(reinterpret_cast<const uint4*>(ib + w0));
            w.a[0] = x.x, w.a[1] = x.y, w.a[2] = x.z, w.a[3] = x.w;
            w.b[0] = y.x, w.b[1] = y.y, w.b[2] = y.z, w.b[3] = y.w;
            w.sa = __ldg(reinterpret_cast<const uint32_t*>(sa + w0));
            w.sb = __ldg(reinterpret_cast<const uint32_t*>(sb + w0));
        } else {
            w.sa = w.sb = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = w0 + j < P.words;
                w.a[j] = in ? __ldg(ia + w0 + j) : 0u;
                w.b[j] = in ? __ldg(ib + w0 + j) : 0u;
                if (in) {
                    w.sa |= (uint32_t)__ldg(sa + w0 + j) << (8 * j);
                    w.sb |= (uint32_t)__ldg(sb + w0 + j) << (8 * j);
                }
            }
        }
        if (SCALE == 1) {
            w.al = __ldg(al + group);
            w.bl = __ldg(bl + group);
            if (--left == 0) {
                ++group;
                left = P.group_words / 4;
            }
        }
        if (XAHEAD) fetch_x(ch, w.x);
    };
    float sum[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[t][j] = 0.0f;
    auto multiply = [&](int ch, Chunk& w) {
        if (ch >= ch1) return;
        uint4 xl[XAHEAD ? 1 : 4][NT];
        if (!XAHEAD) fetch_x(ch, xl);
        uint4(*x)[NT] = XAHEAD ? w.x : xl;
        float acc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t][j] = SCALE == 0 ? sum[t][j] : 0.0f;
        // byte j of even[q] (odd[q]): 4 * code of block 2c (2c + 1) of row q's word j, code = nibble + 16 * sign
        uint32_t even[2], odd[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t* v = q ? w.b : w.a;
            const uint32_t sg = q ? w.sb : w.sa;
            const uint32_t sel = (uint32_t)c | (uint32_t)(c + 4) << 4;
            const uint32_t bytes = __byte_perm(__byte_perm(v[0], v[1], sel), __byte_perm(v[2], v[3], sel), 0x5410u);
            even[q] = ((bytes << 2) & 0x3c3c3c3cu) | ((sg << (6 - 2 * c)) & 0x40404040u);
            odd[q] = ((bytes >> 2) & 0x3c3c3c3cu) | (__funnelshift_l(sg, sg, (5 - 2 * c) & 31) & 0x40404040u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // blocks 2c and 2c + 1
                uint32_t lo[2], hi[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t at = __byte_perm(h ? odd[q] : even[q], tab, (uint32_t)j | 0x7650u);
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(lo[q]) : "r"(at));
                    asm volatile("ld.shared.u32 %0, [%1+128];" : "=r"(hi[q]) : "r"(at));
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    few_mma(acc[t], lo[0], lo[1], hi[0], hi[1], h ? x[j][t].z : x[j][t].x, h ? x[j][t].w : x[j][t].y);
            }
            if (SCALE == 2) {
                const int at = min(4 * ch + j, P.words - 1) / P.group_words;
                const float fa = __ldg(al + at), fb = __ldg(bl + at);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    sum[t][0] = fmaf(fa, acc[t][0], sum[t][0]);
                    sum[t][1] = fmaf(fa, acc[t][1], sum[t][1]);
                    sum[t][2] = fmaf(fb, acc[t][2], sum[t][2]);
                    sum[t][3] = fmaf(fb, acc[t][3], sum[t][3]);
                    acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
                }
            }
        }
        if (SCALE != 2) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sum[t][j] = SCALE == 0 ? acc[t][j] : fmaf(j < 2 ? w.al : w.bl, acc[t][j], sum[t][j]);
        }
    };
    // two chunks in turn, each loaded again as soon as it is used
    Chunk w0, w1;
    fetch(ch0, w0);
    fetch(ch0 + 1, w1);
#pragma unroll 1
    for (int ch = ch0; ch < ch1; ch += 2) {
        multiply(ch, w0);
        fetch(ch + 2, w0);
        multiply(ch + 1, w1);
        fetch(ch + 3, w1);
    }
    // rows g and g + 8, tokens 2c and 2c + 1 of each tile
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[warp][(8 * t + 2 * c + (j & 1)) * kFewPitch + g + 8 * (j >> 1)] = sum[t][j];
    __syncthreads();
    pdl_wait();
    for (int o = tid; o < kFewRows * 8 * NT; o += 32 * kFewWarps) {
        const int n = n0 + o % kFewRows, m = m0 + o / kFewRows;
        if (m >= P.M || n >= P.N) continue;
        float y = 0.0f;
#pragma unroll
        for (int q = 0; q < kFewWarps; ++q) y += part[q][(m - m0) * kFewPitch + o % kFewRows];
        if (SCALE == 0) y *= __ldg(P.scales + (P.per_tensor ? 0 : n));
        const int a = P.ids[m];
        if (a >= 0 && a < P.n_adapters) {
            const uint4* b = reinterpret_cast<const uint4*>(P.B + ((int64_t)a * P.N + n) * P.R);
            const float4* u = reinterpret_cast<const float4*>(P.U + (int64_t)m * P.R);
            float s = 0.0f;
#pragma unroll 2
            for (int r = 0; r < P.R / 8; ++r) {
                const uint4 v = __ldg(b + r);
                const float4 p = u[2 * r], q = u[2 * r + 1];
                s = fmaf(bf16lo(v.x), p.x, s);
                s = fmaf(bf16hi(v.x), p.y, s);
                s = fmaf(bf16lo(v.y), p.z, s);
                s = fmaf(bf16hi(v.y), p.w, s);
                s = fmaf(bf16lo(v.z), q.x, s);
                s = fmaf(bf16hi(v.z), q.y, s);
                s = fmaf(bf16lo(v.w), q.z, s);
                s = fmaf(bf16hi(v.w), q.w, s);
            }
            y += s;
        }
        if (P.y_bf16)
            reinterpret_cast<__nv_bfloat16*>(P.Y)[(int64_t)m * P.N + n] = __float2bfloat16_rn(y);
        else
            reinterpret_cast<float*>(P.Y)[(int64_t)m * P.N + n] = y;
    }
}

template <int NT>
static int few_launch(const FewUpParams& P, int scale, dim3 grid, cudaStream_t stream) {
    auto kernel = scale == 0 ? k_lora_few<NT, 0> : scale == 1 ? k_lora_few<NT, 1> : k_lora_few<NT, 2>;
    grid.y = (unsigned)((P.M + 8 * NT - 1) / (8 * NT));
    return launch_after(kernel, grid, 32 * kFewWarps, 0, stream, 1, true, P);
}

int lora_down_few_launch(const ProbShape& s, const sherry_linear_desc& d, int64_t M, const uint16_t* A, int R,
                         const int32_t* ids, const float* scaling, int n_adapters, float* U, cudaStream_t stream) {
    const FewParams D{d.X, A, scaling, ids, U, (int)M, (int)s.K, R, n_adapters};
    return launch_after(k_lora_down_few, dim3((unsigned)(R / 4), (unsigned)M), 128, 0, stream, 1, true, D);
}

int lora_few_launch(const ProbShape& s, const sherry_linear_desc& d, int64_t M, int y_bf16, const uint16_t* A,
                    const uint16_t* B, int R, const int32_t* ids, const float* scaling, int n_adapters, float* U,
                    cudaStream_t stream) {
    const int st = lora_down_few_launch(s, d, M, A, R, ids, scaling, n_adapters, U, stream);
    if (st) return st;
    FewUpParams P{};
    P.X = d.X;
    P.idx = d.idx;
    P.sgn = d.sgn;
    P.scales = d.scales;
    P.B = B;
    P.U = U;
    P.ids = ids;
    P.Y = d.Y;
    P.M = (int)M;
    P.N = (int)s.N;
    P.K = (int)s.K;
    P.words = (int)(s.K / 32);
    const bool grouped = s.granularity == SHERRY_PER_GROUP;
    P.group_words = grouped ? s.group / 32 : P.words;
    P.spr = grouped ? (int)(s.K / s.group) : s.granularity == SHERRY_PER_CHANNEL;
    P.per_tensor = s.granularity == SHERRY_PER_TENSOR;
    P.R = R;
    P.n_adapters = n_adapters;
    P.y_bf16 = y_bf16;
    const int64_t grid = (s.N + kFewRows - 1) / kFewRows;
    if (grid > 0x7fffffff || s.N > 0x7fffffff - kFewRows) return SHERRY_ERR_UNSUPPORTED;
    const int scale = s.K % 128 != 0 ? 2 : !grouped ? 0 : s.group % 128 == 0 ? 1 : 2;
    if (M <= 8) return few_launch<1>(P, scale, dim3((unsigned)grid), stream);
    if (M <= 16) return few_launch<2>(P, scale, dim3((unsigned)grid), stream);
    return few_launch<4>(P, scale, dim3((unsigned)grid), stream);
}

}  // namespace sherry
