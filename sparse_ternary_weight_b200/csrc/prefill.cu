// prefill.cu -- packed 3:4 ternary linear for many tokens on the 5th-generation
// tensor cores (tcgen05 + TMEM), Y = X (T alpha)^T ("Sherry: Hardware-Efficient
// 1.25-Bit Ternary Quantization via Fine-grained Sparsification", digest: Y = X
// T alpha; "Sherry, Tequila and Fairies in Python" section 1.1: F.linear).
//
// With many tokens the layer is a dense contraction, so the packed weights are
// expanded to bf16 {-1, 0, +1} and multiplied on the tensor cores; alpha cannot
// be folded into the bf16 weights without losing precision, so each K-group is
// accumulated separately in TMEM and promoted into fp32 registers with alpha
// (per-row scales: once at the end).
//
// CTA tile: 128 weight rows (MMA M, TMEM lanes) x 128 tokens (MMA N); K runs in
// chunks of 256 (four 64-wide MMA steps).  The expanded weights (MMA operand A)
// never touch shared memory: decode threads own one TMEM lane (= weight row)
// each and write their row's 64 bf16 of a step into TMEM with tcgen05.st; only
// the X tiles (operand B) come through shared memory, by TMA (no multicast).
// Synchronisation is per chunk: the MMA thread waits once for the chunk's four A
// stages and once for its X, issues the 16 MMAs, and commits once; that commit
// frees both the X slot and the chunk's A buffer.
//   warps 0..E-1 epilogue (E = 16 for group scales and K <= 4096, else 8): wait for one of two
//                finished group accumulators, tcgen05.ld its share of the tokens
//                (128 / (E / 4) each), acc[token] += alpha(row, group) * D, write
//                Y (row per thread)
//   next 8 warps decode, two groups of four warps: group g expands steps 2g and
//                2g + 1 of every chunk, one pattern-table lookup per block of 4
//                weights; packed words come straight from global memory through
//                a per-thread prefetch ring
//   next warp    TMA: the chunk's four X tiles [128 tokens x 64 K], SWIZZLE_128B
//   last warp    TMEM allocation; one elected thread issues tcgen05.mma
#include "common.cuh"
#include "lora.cuh"
#include "lut.cuh"
#include "tc.cuh"

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>

namespace cg = cooperative_groups;

namespace sherry {

constexpr int kPDecGroups = 2;   // decode groups (two MMA steps of every chunk each)
// epilogue warps EPI (8 or 16; a template parameter of the kernel), then the decode
// warps, the TMA warp and the MMA warp
template <int EPI>
struct PRoles {
    static constexpr int kThreads = 32 * (EPI + 4 * kPDecGroups + 2);
    static constexpr int kTmaWarp = EPI + 4 * kPDecGroups;
    static constexpr int kMmaWarp = kTmaWarp + 1;
};
constexpr int kPBM = 128;     // weight rows per tile
constexpr int kPBN = 128;     // tokens per tile
constexpr int kPBK = 64;      // K per MMA step
constexpr int kPChunkSteps = 4;                  // steps per chunk
constexpr int kPStepB = kPBN * kPBK * 2;         // 16 KB of X per step
constexpr int kPXSlots = 3;                      // X chunks in flight
constexpr int kPABuf = 2;                        // A buffers (chunks) in TMEM
constexpr int kPRing = 2;                        // chunks of packed words in flight per decode thread
constexpr int kPArnSteps = 2, kPArnSlots = 3;    // Arenas: steps per chunk, slots (X and W tiles)
constexpr int kPXBytes = kPXSlots * kPChunkSteps * kPStepB > kPArnSlots * 2 * kPArnSteps * kPStepB
                             ? kPXSlots * kPChunkSteps * kPStepB
                             : kPArnSlots * 2 * kPArnSteps * kPStepB;  // the slots of either form
constexpr int kPTable = 256;                     // 32 weight patterns: low words (128 B), then high words
constexpr int kPSmem = kPXBytes + kPTable + 1024;
constexpr int kPAcc = 2;                         // group accumulators in flight
constexpr int kPTmemCols = 512;                  // 2 x 128 accumulator columns + the A buffers
constexpr int kPAcol = kPAcc * kPBN;             // first TMEM column of the A stages (256)
constexpr int kPAcols = kPBK / 2;                // 32 columns (64 bf16) per A stage
constexpr int kPMaxSlots = kPXSlots > kPArnSlots ? kPXSlots : kPArnSlots;
constexpr int kPMaxABuf = kPABuf > 2 ? kPABuf : 2;
static_assert(kPAcol + kPABuf * kPChunkSteps * kPAcols <= kPTmemCols, "TMEM plan");
static_assert(kPXSlots >= kPABuf + 1, "the decode's A-buffer wait reads the slot barrier of chunk cc - kPABuf");

// bf16 x bf16 -> fp32, both K-major, M = 128, N = 128
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kPBN >> 3) << 17) |
                            ((uint32_t)(kPBM >> 4) << 24);

struct PParams {
    const uint32_t* idx;
    const uint8_t* sgn;
    const float* scales;
    void* Y;
    int M, N, K, words;
    int y_bf16;
    int row_scale, per_tensor, spr;
    int group_steps;  // K-steps per scale group (per-row: all of K)
    float lambda;     // Arenas: weight of the dense product
    // adapters (PMode::kLora)
    LoraPlan plan;
    int rp, terms;     // the rank rounded up to 16, and the bf16 terms that U is split into
};

// Arenas (ARN): the same kernel also accumulates X W^T for a dense bf16 latent
// weight W in a third TMEM accumulator and writes Y = (the promoted ternary sum)
// + lambda * that product.  Its W tiles [128 rows x 64 K] come by TMA into the
// same slots as X: a chunk is then two K-steps of X and two of W (64 KB), and the
// ternary A stages shrink to 2 x 2 steps so that the dense accumulator fits in
// TMEM (columns 384..511).
//
// Adapters (kLora): after a tile's last K-chunk come chunks for its slots (the adapters that
// its tokens have) and each 64 ranks: operand A is B_a's rows, operand B the terms of U, zero
// for tokens of other adapters, all by TMA into one X slot (the terms first, then B_a).  A
// slot is one more accumulator group with scale 1, added for its own tokens alone, so
// that an adapter whose weights are not finite spoils no other request's tokens.
// Where there are fewer tiles than SMs a cluster of CL CTAs shares a tile: each sums its part
// of K (whole groups), the last one adds the slots, and the partial tiles are joined
// in order through distributed shared memory (331 x 2050 x 8192, rank 8: 61 -> 53 us).
constexpr int kPLoraB = 3 * kPStepB;  // where B_a's tile lies in the slot: after at most three terms' tiles
enum class PMode { kPlain, kArenas, kLora };

template <int EPI, PMode MODE>
__global__ void __launch_bounds__(PRoles<EPI>::kThreads, 1)
k_prefill(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
          const __grid_constant__ CUtensorMap bmap, const __grid_constant__ CUtensorMap umap,
          const __grid_constant__ PParams P) {
    constexpr bool ARN = MODE == PMode::kArenas, LORA = MODE == PMode::kLora;
    constexpr int kPTmaWarp = PRoles<EPI>::kTmaWarp, kPMmaWarp = PRoles<EPI>::kMmaWarp;
    constexpr int CS = ARN ? kPArnSteps : kPChunkSteps;   // K-steps per chunk
    constexpr int XS = ARN ? kPArnSlots : kPXSlots;       // chunk slots
    constexpr int AB = ARN ? 2 : kPABuf;                  // A buffers
    constexpr int SLOTB = (ARN ? 2 : 1) * CS * kPStepB;   // bytes per slot (ARN: X, then W tiles)
    constexpr int SPG = CS / kPDecGroups;           // steps each decode group expands per chunk
    constexpr int kWOff = CS * kPStepB;             // W tiles after the X tiles of a slot (ARN)
    constexpr int kDenseCol = kPAcol + AB * CS * kPAcols;  // dense accumulator (ARN)
    static_assert(!ARN || kDenseCol + kPBN <= kPTmemCols, "Arenas plan");
    static_assert(XS * SLOTB <= kPXBytes && XS >= AB + 1 && SLOTB % 1024 == 0, "slot plan");
    extern __shared__ __align__(1024) unsigned char psmem[];
    __shared__ uint64_t bars[2 * kPMaxSlots + kPMaxABuf + 2 * kPAcc + 3];
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (smem_u32(psmem) + 1023u) & ~1023u;
    const uint32_t stX = base;                               // XS slots of SLOTB bytes, 1024-aligned
    const uint32_t table = base + kPXBytes;                  // 256-aligned
    const uint32_t bar0 = smem_u32(&bars[0]);
    auto full_x = [&](int c) { return bar0 + 8u * c; };                    // X (and W) chunk in slot c landed
    auto chunk_empty = [&](int c) { return bar0 + 8u * (XS + c); };  // MMAs of slot c's chunk done
    auto full_a = [&](int h) { return bar0 + 8u * (2 * XS + h); };   // A buffer h written
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * XS + AB + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (2 * XS + AB + kPAcc + b); };
    const uint32_t drain = bar0 + 8u * (2 * XS + AB + 2 * kPAcc);  // the MMA thread's last commit
    const uint32_t dense_full = drain + 8u;    // ARN: a tile's dense product is complete
    const uint32_t dense_empty = drain + 16u;  // ARN: the epilogue has read it

    // persistent: tile t = (weight-row tile t % ntn, token tile t / ntn), strided by the grid;
    // chunk and accumulator phases run on across tiles
    const int ntn = (P.N + kPBM - 1) / kPBM;
    const int ntiles = ntn * ((P.M + kPBN - 1) / kPBN);
    // LORA: CTAs that share a tile (then one tile each), and this one's place
    const int CL = LORA ? (int)cg::this_cluster().num_blocks() : 1;
    const int cr = LORA ? (int)cg::this_cluster().block_rank() : 0;
    const unsigned tile0 = blockIdx.x / CL, tstride = gridDim.x / CL;  // LORA
    // this CTA's steps kb .. kb + nk of K, in groups of gs
    const int ksteps = P.K / kPBK;
    const int unit = LORA && P.row_scale ? 1 : P.group_steps;
    const int kb = LORA ? (int)((int64_t)(ksteps / unit) * cr / CL) * unit : 0;
    const int nk = LORA ? (int)((int64_t)(ksteps / unit) * (cr + 1) / CL) * unit - kb : ksteps;
    const int gs = LORA && P.row_scale ? nk : P.group_steps;
    const int nchunks = (nk + CS - 1) / CS;  // the last one may hold fewer steps
    const int ngroups = nk / gs;
    // LORA: chunks of 64 ranks per slot, and whether the terms of U lie in one tile's 64 columns
    const int lblocks = LORA ? (P.rp + 63) / 64 : 0;
    const bool one_box = LORA && P.terms * P.rp <= 64;
    if (threadIdx.x == 0) {
        abort_s = 0;
        for (int c = 0; c < XS; ++c) {
            mbar_init(full_x(c), 1);
            mbar_init(chunk_empty(c), 1);
        }
        for (int h = 0; h < AB; ++h) mbar_init(full_a(h), 128 * kPDecGroups);
        for (int b = 0; b < kPAcc; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), 32 * EPI);
        }
        mbar_init(drain, 1);
        mbar_init(dense_full, 1);
        mbar_init(dense_empty, 32 * EPI);
        fence_mbar_init();
    }
    if (threadIdx.x < 32) {
        // bf16 patterns of the 32 block codes (entry = nibble + 16 * sign bit): the
        // low halves (weights 0, 1) and the high halves (weights 2, 3) in separate
        // 128-byte tables, so that a warp's lookups never conflict on a bank
        const uint2 e = decode_block_bf16((uint32_t)threadIdx.x & 15u, (uint32_t)threadIdx.x >> 4);
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(table + 4u * threadIdx.x), "r"(e.x) : "memory");
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(table + 128u + 4u * threadIdx.x), "r"(e.y) : "memory");
    }
    if (warp == kPMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_s)),
                     "r"(kPTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    // LORA: the plan, and X in its order, are ready when this kernel is launched (k_lora_down lets it
    // start only then); U's image and the slots' masks are waited for where they are read
    const bool permuted = LORA && P.plan.may_permute && P.plan.head[0] != 0;
    // the slots of tile t; every role loads them at the tile's start and uses them at its end
    auto slots_of = [&](int t) {
        return LORA && cr == CL - 1 ? make_int2(P.plan.tile_b[t / ntn], P.plan.tile_b[t / ntn + 1]) : make_int2(0, 0);
    };

    if (warp < EPI) {
        // ---------------- epilogue: row n = tile row 32*(warp%4) + lane, tokens
        // [kCols*(warp/4), kCols*(warp/4) + kCols) of each tile ----------------
        const int q = warp & 3, half = warp >> 2;
        constexpr int kCols = kPBN / (EPI / 4);
        bool ok = true;
        int b = 0;
        uint32_t bph = 0;  // phase parity of accumulator b's use
        uint32_t dph = 0;  // ARN: phase parity of the dense accumulator's use
        for (int t = LORA ? tile0 : blockIdx.x; t < ntiles && ok; t += LORA ? tstride : gridDim.x) {
            const int n = (t % ntn) * kPBM + q * 32 + lane;
            const int m0 = (t / ntn) * kPBN + half * kCols;
            const int2 sl = slots_of(t);
            uint32_t own0[kCols / 32];  // the first slot's tokens among this thread's; of the first tile after the wait
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c)
                own0[c] = LORA && t != (int)tile0 && sl.x < sl.y ? P.plan.mask[4 * sl.x + half * (kCols / 32) + c] : 0u;
            const bool row_ok = n < P.N;
            const bool gsc = !P.row_scale && row_ok;
            const float* srow = P.scales + (int64_t)(row_ok ? n : 0) * P.spr + (LORA && !P.row_scale ? kb / gs : 0);
            // group scales are loaded two groups ahead of their use
            float a_next = gsc ? __ldg(srow) : 1.0f;
            float a_next2 = (gsc && ngroups > 1) ? __ldg(srow + 1) : 1.0f;
            float acc[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
            for (int g = 0; g < ngroups; ++g) {
                const float a = a_next;
                a_next = a_next2;
                a_next2 = (gsc && g + 2 < ngroups) ? __ldg(srow + g + 2) : 1.0f;
                ok = mbar_wait(acc_full(b), bph, &abort_s);
                if (!ok) break;
                tc_fence_after();
                const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * kPBN + half * kCols);
                // 32 columns per wait (two TMEM loads in flight); the running sums stay in registers
#pragma unroll
                for (int c = 0; c < kCols / 32; ++c) {
                    uint32_t v[16], w[16];
                    SHERRY_TMEM_LD16(t_row + 32 * c, v);
                    SHERRY_TMEM_LD16(t_row + 32 * c + 16, w);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[32 * c + j] = fmaf(a, __uint_as_float(v[j]), acc[32 * c + j]);
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[32 * c + 16 + j] = fmaf(a, __uint_as_float(w[j]), acc[32 * c + 16 + j]);
                }
                tc_fence_before();
                mbar_arrive(acc_empty(b));
                if (++b == kPAcc) { b = 0; bph ^= 1u; }
            }
            if (!ok) break;
            float a = 1.0f;
            if (P.row_scale && row_ok) a = __ldg(P.scales + (P.per_tensor ? 0 : n));
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] *= a;
            if constexpr (LORA) {
                // at the first tile, whether it has slots or not: from the second on the masks are read at the tile's start
                if (t == (int)tile0) pdl_wait();
                if (t == (int)tile0 && sl.x < sl.y) {
#pragma unroll
                    for (int c = 0; c < kCols / 32; ++c) own0[c] = P.plan.mask[4 * sl.x + half * (kCols / 32) + c];
                }
                for (int i = sl.x; i < sl.y; ++i) {
                    uint32_t own[kCols / 32];  // the next slot's are loaded ahead
#pragma unroll
                    for (int c = 0; c < kCols / 32; ++c) {
                        own[c] = own0[c];
                        own0[c] = P.plan.mask[4 * min(i + 1, sl.y - 1) + half * (kCols / 32) + c];
                    }
                    ok = mbar_wait(acc_full(b), bph, &abort_s);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * kPBN + half * kCols);
#pragma unroll
                    for (int c = 0; c < kCols / 16; ++c) {
                        uint32_t v[16];
                        SHERRY_TMEM_LD16(t_row + 16 * c, v);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (own[c / 2] >> (16 * (c & 1) + j) & 1u) acc[16 * c + j] += __uint_as_float(v[j]);
                    }
                    tc_fence_before();
                    mbar_arrive(acc_empty(b));
                    if (++b == kPAcc) { b = 0; bph ^= 1u; }
                }
                if (!ok) break;
            }
            if constexpr (ARN) {
                // Y = the ternary sum + lambda * the dense product
                ok = mbar_wait(dense_full, dph, &abort_s);
                if (!ok) break;
                tc_fence_after();
                const uint32_t t_d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(kDenseCol + half * kCols);
#pragma unroll
                for (int c = 0; c < kCols / 16; ++c) {
                    uint32_t v[16];
                    SHERRY_TMEM_LD16(t_d + 16 * c, v);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[16 * c + j] = fmaf(P.lambda, __uint_as_float(v[j]), acc[16 * c + j]);
                }
                tc_fence_before();
                mbar_arrive(dense_empty);
                dph ^= 1u;
            }
            if (LORA && CL > 1) {
                // the tile as [token][row] in the X slots: every product and load of this CTA is done
                float* part = reinterpret_cast<float*>(psmem + (base - smem_u32(psmem)));
#pragma unroll
                for (int j = 0; j < kCols; ++j) part[(half * kCols + j) * kPBM + q * 32 + lane] = acc[j];
            } else if (row_ok && LORA && permuted) {
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    if (m0 + j < P.M) {
                        const int64_t at = (int64_t)P.plan.perm[m0 + j] * P.N + n;
                        if (P.y_bf16)
                            reinterpret_cast<__nv_bfloat16*>(P.Y)[at] = __float2bfloat16_rn(acc[j]);
                        else
                            reinterpret_cast<float*>(P.Y)[at] = acc[j];
                    }
                }
            } else if (row_ok) {
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    const int m = m0 + j;
                    if (m < P.M) {
                        const float y = acc[j];
                        if (P.y_bf16)
                            reinterpret_cast<__nv_bfloat16*>(P.Y)[(int64_t)m * P.N + n] = __float2bfloat16_rn(y);
                        else
                            reinterpret_cast<float*>(P.Y)[(int64_t)m * P.N + n] = y;
                    }
                }
            }
        }
    } else if (warp < kPTmaWarp) {
        // ---------------- decode: TMEM lane (= tile row) i per thread; group g expands
        // steps SPG*g .. SPG*g + SPG-1 of every chunk into A buffer (cc % AB) ----------------
        const int g = (warp - EPI) >> 2, q = warp & 3;
        const int i = q * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)kPAcol;
        int cc = 0;  // chunks done so far (all tiles)
        bool ok = true;
        for (int t = LORA ? tile0 : blockIdx.x; t < ntiles && ok; t += LORA ? tstride : gridDim.x) {
            const int n = (t % ntn) * kPBM + i;
            const bool row_ok = n < P.N;
            const int2 sl = slots_of(t);
            const uint32_t* idxr = P.idx + (int64_t)(row_ok ? n : 0) * P.words + (LORA ? 2 * kb : 0);
            const uint8_t* sgnr = P.sgn + (int64_t)(row_ok ? n : 0) * P.words + (LORA ? 2 * kb : 0);
            // ring of the next kPRing chunks' packed words: per step 2 idx words + 2 sign bytes
            uint2 rw[kPRing][2];
            uint32_t rs[kPRing][2];
            auto fetch = [&](int ch, uint2* w, uint32_t* sg) {
#pragma unroll
                for (int e = 0; e < SPG; ++e) {
                    const int ks = ch * CS + SPG * g + e;
                    w[e] = make_uint2(0u, 0u);
                    sg[e] = 0u;
                    if (row_ok && ch < nchunks && ks < nk) {
                        w[e] = __ldg(reinterpret_cast<const uint2*>(idxr + 2 * ks));
                        sg[e] = __ldg(reinterpret_cast<const uint16_t*>(sgnr + 2 * ks));
                    }
                }
            };
#pragma unroll
            for (int r = 0; r < kPRing; ++r) fetch(r, rw[r], rs[r]);
            for (int ch0 = 0; ch0 < nchunks && ok; ch0 += kPRing) {
#pragma unroll
                for (int r = 0; r < kPRing; ++r) {
                    const int ch = ch0 + r;
                    if (ch >= nchunks) break;
                    uint2 w[2] = {rw[r][0], rw[r][1]};
                    uint32_t sb[2] = {rs[r][0], rs[r][1]};
                    fetch(ch + kPRing, rw[r], rs[r]);
                    const int hbuf = cc % AB;
                    // a last chunk that ends before this group's steps: the group writes nothing, but
                    // arrives for buffer hbuf all the same, so it too waits for the buffer's last use
                    // (a phase ahead, its arrival would stand in for the other group's)
                    if (ch * CS + SPG * g >= nk && cc >= AB &&
                        !mbar_wait(chunk_empty((cc - AB) % XS), (uint32_t)(((cc - AB) / XS) & 1), &abort_s)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int e = 0; e < SPG; ++e) {
                        const int st = SPG * g + e;
                        if (ch * CS + st >= nk) break;
                        uint32_t v[32];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t wd = h ? w[e].y : w[e].x;
                            const uint32_t sg = (sb[e] >> (8 * h)) & 0xffu;
                            const uint32_t ev = ((wd << 2) & 0x3c3c3c3cu) | (((sg & 0x55u) * 0x01041040u) & 0x40404040u);
                            const uint32_t od = ((wd >> 2) & 0x3c3c3c3cu) | (((sg & 0xaau) * 0x00820820u) & 0x40404040u);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint32_t a = __byte_perm((j & 1) ? od : ev, table, (uint32_t)(j >> 1) | 0x7650u);
                                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[16 * h + 2 * j]) : "r"(a));
                                asm volatile("ld.shared.u32 %0, [%1+128];" : "=r"(v[16 * h + 2 * j + 1]) : "r"(a));
                            }
                        }
                        // A buffer hbuf was last read by the MMAs of chunk cc - AB, whose
                        // completion the MMA thread commits to that chunk's slot barrier
                        if (e == 0 && cc >= AB) {
                            if (!mbar_wait(chunk_empty((cc - AB) % XS), (uint32_t)(((cc - AB) / XS) & 1),
                                           &abort_s)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                        }
                        SHERRY_TMEM_ST32(t_lane + (uint32_t)((hbuf * CS + st) * kPAcols), v);
                    }
                    if (!ok) break;
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    tc_fence_before();
                    mbar_arrive(full_a(hbuf));
                    ++cc;
                }
            }
            if constexpr (LORA) {
                // the adapters' chunks use no A buffer; their turns are waited for all the same, so
                // that no slot barrier gets two phases ahead of this thread
                for (int left = lblocks * (sl.y - sl.x); left > 0 && ok; --left, ++cc)
                    if (cc >= AB)
                        ok = mbar_wait(chunk_empty((cc - AB) % XS), (uint32_t)(((cc - AB) / XS) & 1), &abort_s);
            }
        }
    } else if (warp == kPTmaWarp) {
        // ---------------- TMA producer for X (and, ARN, the latent-weight tiles) ----------------
        if (lane == 0) {
            int c = 0;
            uint32_t cph = 0;  // phase parity of slot c's use
            int issued[XS] = {};  // chunks loaded into each slot (phases of full_x)
            bool ok = true;
            for (int t = LORA ? tile0 : blockIdx.x; t < ntiles && ok; t += LORA ? tstride : gridDim.x) {
                const int m0 = (t / ntn) * kPBN;
                const int n0 = (t % ntn) * kPBM;
                const int2 sl = slots_of(t);
                int a0 = 0, a1 = 0;  // the first slots' adapters, loaded beside the K-chunks
                if (LORA && sl.x < sl.y) {
                    a0 = P.plan.slot_a[sl.x];
                    a1 = P.plan.slot_a[min(sl.x + 1, sl.y - 1)];
                }
                for (int ch = 0; ch < nchunks; ++ch) {
                    if (!mbar_wait(chunk_empty(c), cph ^ 1u, &abort_s)) {
                        ok = false;
                        break;
                    }
                    const int steps = min(CS, nk - ch * CS);
                    mbar_expect_tx(full_x(c), (uint32_t)(steps * kPStepB * (ARN ? 2 : 1)));
                    for (int st = 0; st < steps; ++st) {
                        tma_load_2d(stX + c * SLOTB + st * kPStepB, LORA && permuted ? &wmap : &xmap,
                                    ((LORA ? kb : 0) + ch * CS + st) * kPBK, m0, full_x(c));
                        if constexpr (ARN)
                            tma_load_2d(stX + c * SLOTB + kWOff + st * kPStepB, &wmap, (ch * CS + st) * kPBK, n0,
                                        full_x(c));
                    }
                    ++issued[c];
                    if (++c == XS) { c = 0; cph ^= 1u; }
                }
                if constexpr (LORA) {
                    pdl_wait();
                    for (int i = sl.x; i < sl.y && ok; ++i) {
                        const int a = a0;  // the next slots' adapters are loaded ahead
                        a0 = a1;
                        a1 = P.plan.slot_a[min(i + 2, sl.y - 1)];
                        for (int r0 = 0; r0 < P.rp; r0 += 64) {
                            if (!mbar_wait(chunk_empty(c), cph ^ 1u, &abort_s)) {
                                ok = false;
                                break;
                            }
                            const int boxes = one_box ? 1 : P.terms;
                            const uint32_t slot = stX + c * SLOTB;
                            mbar_expect_tx(full_x(c), (uint32_t)((boxes + 1) * kPStepB));
                            for (int j = 0; j < boxes; ++j)
                                tma_load_2d(slot + j * kPStepB, &umap, j * P.rp + r0, i * kLoraTile, full_x(c));
                            tma_load_3d(slot + kPLoraB, &bmap, r0, n0, a, full_x(c));
                            ++issued[c];
                            if (++c == XS) { c = 0; cph ^= 1u; }
                        }
                    }
                }
            }
            // every load issued must land before the CTA's shared memory goes away
            // (after an abort the MMA thread may not have waited for the last ones)
            for (int s = 0; s < XS; ++s)
                if (issued[s] > 0) mbar_drain(full_x(s), (uint32_t)((issued[s] - 1) & 1));
        }
    } else {
        // ---------------- MMA issuer ----------------
        // A single thread issues every MMA, so its own instruction stream is on the
        // critical path: full chunks take an unrolled path, group boundaries are a
        // count-down, and operand addresses are fixed offsets from the chunk base.
        if (lane == 0) {
            int cc = 0, c = 0, b = 0;
            uint32_t cph = 0, bph = 0;
            uint32_t dph = 0;  // ARN: phase parity of the dense accumulator's use
            uint32_t aph = 0;  // phase parities of the A buffers' uses
            bool ok = true;
            // one MMA step (K = 64: four K = 16 MMAs) into accumulator b, and (ARN) the
            // dense step into the dense accumulator; returns false on a timed-out wait
            auto step = [&](int& gleft, int ks, uint32_t ta, uint64_t db, uint64_t dw) -> bool {
                const bool first = gleft == gs;
                if (first) {
                    if (!mbar_wait(acc_empty(b), bph ^ 1u, &abort_s)) return false;
                    tc_fence_after();
                }
                const uint32_t td = tmem + (uint32_t)(b * kPBN);
                mma_bf16_ts(td, ta, db, kIdesc, first ? 0u : 1u);
#pragma unroll
                for (int kk = 1; kk < kPBK / 16; ++kk)  // K = 16 per MMA: 8 A columns, +32 bytes in the B row
                    mma_bf16_ts(td, ta + (uint32_t)(8 * kk), db + (uint64_t)(2 * kk), kIdesc, 1u);
                if constexpr (ARN) {
                    if (ks == 0) {
                        if (!mbar_wait(dense_empty, dph ^ 1u, &abort_s)) return false;
                        tc_fence_after();
                    }
                    const uint32_t tdd = tmem + (uint32_t)kDenseCol;
#pragma unroll
                    for (int kk = 0; kk < kPBK / 16; ++kk)
                        mma_bf16_ss(tdd, dw + (uint64_t)(2 * kk), db + (uint64_t)(2 * kk), kIdesc,
                                    (ks == 0 && kk == 0) ? 0u : 1u);
                    if (ks == nk - 1) {
                        mma_commit(dense_full);
                        dph ^= 1u;
                    }
                }
                if (--gleft == 0) {
                    mma_commit(acc_full(b));
                    gleft = gs;
                    if (++b == kPAcc) { b = 0; bph ^= 1u; }
                }
                return true;
            };
            for (int t = LORA ? tile0 : blockIdx.x; t < ntiles && ok; t += LORA ? tstride : gridDim.x) {
                int gleft = gs;  // steps left in the current group
                const int2 sl = slots_of(t);
                for (int ch = 0; ch < nchunks; ++ch, ++cc) {
                    const int hbuf = cc % AB;
                    const uint32_t ah = LORA ? (aph >> hbuf) & 1u : (uint32_t)((cc / AB) & 1);
                    if (!mbar_wait(full_a(hbuf), ah, &abort_s)) { ok = false; break; }
                    if constexpr (LORA) aph ^= 1u << hbuf;
                    if (!mbar_wait(full_x(c), cph, &abort_s)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t db0 = smem_desc(stX + c * SLOTB);
                    const uint64_t dw0 = smem_desc(stX + c * SLOTB + kWOff);
                    const uint32_t ta0 = tmem + (uint32_t)(kPAcol + hbuf * CS * kPAcols);
                    const int steps = min(CS, nk - ch * CS);
                    if (steps == CS) {
#pragma unroll
                        for (int st = 0; st < CS; ++st)
                            if (!step(gleft, ch * CS + st, ta0 + (uint32_t)(st * kPAcols),
                                      db0 + (uint64_t)((st * kPStepB) >> 4), dw0 + (uint64_t)((st * kPStepB) >> 4))) {
                                ok = false;
                                break;
                            }
                    } else {
                        for (int st = 0; st < steps; ++st)
                            if (!step(gleft, ch * CS + st, ta0 + (uint32_t)(st * kPAcols),
                                      db0 + (uint64_t)((st * kPStepB) >> 4), dw0 + (uint64_t)((st * kPStepB) >> 4))) {
                                ok = false;
                                break;
                            }
                    }
                    if (!ok) break;
                    mma_commit(chunk_empty(c));
                    if (++c == XS) { c = 0; cph ^= 1u; }
                }
                if constexpr (LORA) {
                    for (int left = sl.y - sl.x; left > 0 && ok; --left) {
                        if (!mbar_wait(acc_empty(b), bph ^ 1u, &abort_s)) { ok = false; break; }
                        const uint32_t td = tmem + (uint32_t)(b * kPBN);
                        for (int r0 = 0; r0 < P.rp; r0 += 64, ++cc) {
                            if (!mbar_wait(full_x(c), cph, &abort_s)) { ok = false; break; }
                            tc_fence_after();
                            const uint64_t du = smem_desc(stX + c * SLOTB), db = smem_desc(stX + c * SLOTB + kPLoraB);
                            const int nk16 = min(4, (P.rp - r0) / 16);
                            for (int i = P.terms - 1; i >= 0; --i)  // the small terms first
                                for (int kk = 0; kk < nk16; ++kk)   // 16 ranks: 32 bytes of a row
                                    mma_bf16_ss(td, db + (uint64_t)(2 * kk),
                                                du + (uint64_t)(one_box ? (i * P.rp) / 8 + 2 * kk
                                                                        : ((i * kPStepB) >> 4) + 2 * kk),
                                                kIdesc, (r0 == 0 && i == P.terms - 1 && kk == 0) ? 0u : 1u);
                            mma_commit(chunk_empty(c));
                            if (++c == XS) { c = 0; cph ^= 1u; }
                        }
                        if (!ok) break;
                        mma_commit(acc_full(b));
                        if (++b == kPAcc) { b = 0; bph ^= 1u; }
                    }
                }
            }
            // all MMAs this thread issued complete before TMEM is freed (after an abort
            // no epilogue has waited for them)
            mma_commit(drain);
            mbar_drain(drain, 0u);
        }
        __syncwarp();
    }

    if constexpr (LORA) {
        if (CL > 1) {
            cg::cluster_group cluster = cg::this_cluster();
            __syncwarp();
            cluster.sync();
            if (warp < EPI) {  // this CTA's share of the tokens
                float* part = reinterpret_cast<float*>(psmem + (base - smem_u32(psmem)));
                const int row = threadIdx.x % kPBM, n = (tile0 % ntn) * kPBM + row, share = kPBN / CL;
#pragma unroll 4
                for (int i = threadIdx.x / kPBM; i < share; i += EPI / 4) {
                    const int j = share * cr + i;
                    int m = (tile0 / ntn) * kPBN + j;
                    if (m >= P.M || n >= P.N) continue;
                    if (permuted) m = P.plan.perm[m];
                    float y = 0.0f;
                    for (int r = 0; r < CL; ++r) y += cluster.map_shared_rank(part, r)[j * kPBM + row];
                    if (P.y_bf16)
                        reinterpret_cast<__nv_bfloat16*>(P.Y)[(int64_t)m * P.N + n] = __float2bfloat16_rn(y);
                    else
                        reinterpret_cast<float*>(P.Y)[(int64_t)m * P.N + n] = y;
                }
            }
            cluster.sync();  // the others' tiles are read until here
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kPMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kPTmemCols));
    }
}

// ---- host side -------------------------------------------------------------------

bool prefill_eligible(const ProbShape& s, int64_t M) {
    if (M < 17 || s.N == 0) return false;
    if (s.K % kPBK != 0) return false;
    if (s.granularity == SHERRY_PER_GROUP && s.group % kPBK != 0) return false;
    if (M > (int64_t)0x7fffffff / 2) return false;
    return true;
}

// SMs that clusters of one CTA per SM can fill, in percent: what is left over in a GPC stays empty
constexpr int kPRoom = 88;

static int64_t prefill_tiles(const ProbShape& s, int64_t M) {
    return ((s.N + kPBM - 1) / kPBM) * ((M + kPBN - 1) / kPBN);
}

// Adapters: K is split while that still gives every CTA an SM, and each of them four chunks or more in whole groups
static int lora_split(const ProbShape& s, int64_t M, int sms) {
    const int64_t steps = s.K / kPBK, tiles = prefill_tiles(s, M);
    const int64_t units = s.granularity == SHERRY_PER_GROUP ? s.K / s.group : steps;
    int cl = 1;
    while (cl < 8 && tiles * cl * 2 <= sms * kPRoom / 100 && units >= 2 * cl && steps >= 16 * cl) cl *= 2;
    return cl;
}

int64_t prefill_lora_ctas(const ProbShape& s, int64_t M, int sms) {
    return std::min<int64_t>(prefill_tiles(s, M), sms) * lora_split(s, M, sms);
}

// Wd: the latent bf16 weight for Arenas; lora: the adapters' part of P (null: the plain linear)
static int prefill_launch_any(const ProbShape& s, const sherry_linear_desc& d, int64_t M, int y_bf16,
                              const uint16_t* Wd, float lambda, const LoraArgs* lora, cudaStream_t stream) {
    CUtensorMap map, wmap;
    int st = encode_2d(&map, d.X, s.K, M, kPBN);
    if (st) return st;
    if (Wd && (st = encode_2d(&wmap, Wd, s.K, s.N, kPBM))) return st;
    if (!Wd) wmap = map;  // unused, or X in the plan's order
    CUtensorMap bmap = map, umap = map;
    PParams P{};
    P.idx = d.idx;
    P.sgn = d.sgn;
    P.scales = d.scales;
    P.Y = d.Y;
    P.M = (int)M;
    P.N = (int)s.N;
    P.K = (int)s.K;
    P.words = (int)(s.K / 32);
    P.y_bf16 = y_bf16;
    P.row_scale = s.granularity != SHERRY_PER_GROUP;
    P.per_tensor = s.granularity == SHERRY_PER_TENSOR;
    P.spr = s.granularity == SHERRY_PER_GROUP ? (int)(s.K / s.group) : 1;
    P.group_steps = s.granularity == SHERRY_PER_GROUP ? s.group / kPBK : (int)(s.K / kPBK);
    P.lambda = lambda;
    if (lora) {
        P.plan = lora->plan;
        P.rp = lora->U.rp;
        P.terms = lora->U.terms;
        if (lora->Xp && (st = encode_2d(&wmap, lora->Xp, s.K, M, kPBN))) return st;
        if ((st = encode_3d(&bmap, lora->B, lora->R, s.N, lora->n_adapters, kPBM))) return st;
        if ((st = encode_2d(&umap, lora->U.data, P.rp * P.terms, (int64_t)lora->plan.max_slots * kLoraTile, kPBN)))
            return st;
    }
    // per device: the shared-memory opt-in of every instantiation, and the SM count
    static PerDevice dev_sms;
    int sms = 0;
    st = per_device(dev_sms, &sms, [](int& v) {
        SHERRY_CUDA_CHECK(cudaFuncSetAttribute(k_prefill<8, PMode::kPlain>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem));
        SHERRY_CUDA_CHECK(cudaFuncSetAttribute(k_prefill<16, PMode::kPlain>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem));
        SHERRY_CUDA_CHECK(cudaFuncSetAttribute(k_prefill<8, PMode::kArenas>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem));
        SHERRY_CUDA_CHECK(cudaFuncSetAttribute(k_prefill<16, PMode::kArenas>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem));
        SHERRY_CUDA_CHECK(cudaFuncSetAttribute(k_prefill<8, PMode::kLora>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem));
        SHERRY_CUDA_CHECK(cudaFuncSetAttribute(k_prefill<16, PMode::kLora>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem));
        int dev = 0;
        SHERRY_CUDA_CHECK(cudaGetDevice(&dev));
        SHERRY_CUDA_CHECK(cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev));
        if (v < 1) v = 1;
        return SHERRY_OK;
    });
    if (st) return st;
    const int64_t tiles = prefill_tiles(s, M);
    const unsigned grid = (unsigned)(tiles < sms ? tiles : sms);
    // 16 epilogue warps (32 token columns each) drain a group accumulator faster; measured on the
    // 3B shapes that pays for group scales up to K = 4096 (+6%) and costs at K = 8192 (-15%) and
    // for per-row scales (one drain per tile; -1.5% at 2048 and 4096 tokens)
    const bool epi16 = s.granularity == SHERRY_PER_GROUP && s.K <= 4096;
    if (lora) {
        const int cl = lora_split(s, M, sms);
        if (epi16)
            return launch_after(k_prefill<16, PMode::kLora>, grid * cl, PRoles<16>::kThreads, kPSmem, stream, cl, true,
                                map, wmap, bmap, umap, P);
        return launch_after(k_prefill<8, PMode::kLora>, grid * cl, PRoles<8>::kThreads, kPSmem, stream, cl, true, map,
                            wmap, bmap, umap, P);
    } else if (Wd) {
        if (epi16)
            k_prefill<16, PMode::kArenas><<<grid, PRoles<16>::kThreads, kPSmem, stream>>>(map, wmap, bmap, umap, P);
        else
            k_prefill<8, PMode::kArenas><<<grid, PRoles<8>::kThreads, kPSmem, stream>>>(map, wmap, bmap, umap, P);
    } else {
        if (epi16)
            k_prefill<16, PMode::kPlain><<<grid, PRoles<16>::kThreads, kPSmem, stream>>>(map, wmap, bmap, umap, P);
        else
            k_prefill<8, PMode::kPlain><<<grid, PRoles<8>::kThreads, kPSmem, stream>>>(map, wmap, bmap, umap, P);
    }
    SHERRY_LAUNCH_CHECK();
    return SHERRY_OK;
}

int prefill_launch(const ProbShape& s, const sherry_linear_desc& d, int64_t M, int y_bf16, cudaStream_t stream) {
    return prefill_launch_any(s, d, M, y_bf16, nullptr, 0.0f, nullptr, stream);
}

bool arenas_eligible(const ProbShape& s, int64_t M) {
    if (M < 1 || s.N == 0 || s.K % kPBK != 0) return false;
    if (s.granularity == SHERRY_PER_GROUP && s.group % kPBK != 0) return false;
    return M <= (int64_t)0x7fffffff / 2 && s.N <= (int64_t)0x7fffffff / 2;
}

int arenas_launch(const ProbShape& s, const sherry_linear_desc& d, int64_t M, int y_bf16, const uint16_t* Wd,
                  float lambda, cudaStream_t stream) {
    return prefill_launch_any(s, d, M, y_bf16, Wd, lambda, nullptr, stream);
}

int prefill_lora_launch(const ProbShape& s, const sherry_linear_desc& d, int64_t M, int y_bf16, const LoraArgs& lora,
                        cudaStream_t stream) {
    return prefill_launch_any(s, d, M, y_bf16, nullptr, 0.0f, &lora, stream);
}

int device_status_take(cudaStream_t stream) {
    SHERRY_CUDA_CHECK(cudaStreamSynchronize(stream));
    const int v = tc_status_take();
    const int w = skinny_status_take();
    const int x = stream_status_take();
    const int y = dgrad_status_take();
    const int z = lora_status_take();
    return v ? v : w ? w : x ? x : y ? y : z;
}

}  // namespace sherry
