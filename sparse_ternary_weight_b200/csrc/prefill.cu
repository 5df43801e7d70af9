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

#include <cuda_bf16.h>

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
    const uint16_t* B;      // bf16 [n_adapters][N][R]
    const float* U;         // fp32 [M][R]
    const int32_t* ids;
    const int32_t* tile_n;  // adapters present in each 128-token tile
    const int32_t* tile_a;  // [tiles][kLoraTile]
    int R, terms;           // rank; bf16 terms that U is split into
};

// Arenas (ARN): the same kernel also accumulates X W^T for a dense bf16 latent
// weight W in a third TMEM accumulator and writes Y = (the promoted ternary sum)
// + lambda * that product.  Its W tiles [128 rows x 64 K] come by TMA into the
// same slots as X: a chunk is then two K-steps of X and two of W (64 KB), and the
// ternary A stages shrink to 2 x 2 steps so that the dense accumulator fits in
// TMEM (columns 384..511).
//
// Adapters (kLora): after a tile's last K-chunk come chunks whose operand A is B_a
// (the rank columns of the tile's weight rows, straight from its rows into TMEM) and
// whose X slot holds U of the tile's tokens, zero for tokens of other adapters.  The
// decode warps write both; each different adapter of the tile and each 16 ranks is
// one K = 16 entry per bf16 term of U, four entries a step.  They form one more
// group, with scale 1.  A tile of one adapter of rank 16 adds 3 K = 16 products to
// K / 16, and a tile whose tokens all differ stays right, at 128 entries a term.
enum class PMode { kPlain, kArenas, kLora };

template <int EPI, PMode MODE>
__global__ void __launch_bounds__(PRoles<EPI>::kThreads, 1)
k_prefill(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
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
    const int nk = P.K / kPBK;
    const int nchunks = (nk + CS - 1) / CS;  // the last one may hold fewer steps
    const int gs = P.group_steps;
    const int ngroups = nk / gs;
    // LORA: K = 16 entries of tile t's adapters, and their steps of four
    const int rb = LORA ? (P.R + 15) / 16 : 1;
    auto lora_entries = [&](int t) -> int { return LORA ? __ldg(P.tile_n + t / ntn) * rb * P.terms : 0; };
    auto lora_steps = [&](int t) -> int { return LORA ? (lora_entries(t) + 3) / 4 : 0; };

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

    if (warp < EPI) {
        // ---------------- epilogue: row n = tile row 32*(warp%4) + lane, tokens
        // [kCols*(warp/4), kCols*(warp/4) + kCols) of each tile ----------------
        const int q = warp & 3, half = warp >> 2;
        constexpr int kCols = kPBN / (EPI / 4);
        bool ok = true;
        int b = 0;
        uint32_t bph = 0;  // phase parity of accumulator b's use
        uint32_t dph = 0;  // ARN: phase parity of the dense accumulator's use
        for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
            const int n = (t % ntn) * kPBM + q * 32 + lane;
            const int m0 = (t / ntn) * kPBN + half * kCols;
            const bool row_ok = n < P.N;
            const bool gsc = !P.row_scale && row_ok;
            const float* srow = P.scales + (int64_t)(row_ok ? n : 0) * P.spr;
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
                if (lora_steps(t) > 0) {
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
                        for (int j = 0; j < 16; ++j) acc[16 * c + j] += __uint_as_float(v[j]);
                    }
                    tc_fence_before();
                    mbar_arrive(acc_empty(b));
                    if (++b == kPAcc) { b = 0; bph ^= 1u; }
                }
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
            if (row_ok) {
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
        for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
            const int n = (t % ntn) * kPBM + i;
            const bool row_ok = n < P.N;
            const uint32_t* idxr = P.idx + (int64_t)(row_ok ? n : 0) * P.words;
            const uint8_t* sgnr = P.sgn + (int64_t)(row_ok ? n : 0) * P.words;
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
                // the adapters' chunks: thread i writes row i of both operands
                const int entries = lora_entries(t), lsteps = lora_steps(t);
                const int64_t m = (int64_t)(t / ntn) * kPBN + i;
                const int my = m < P.M ? __ldg(P.ids + m) : -1;
                for (int st0 = 0; st0 < lsteps && ok; st0 += CS, ++cc) {
                    const int hbuf = cc % AB;
                    // chunk cc - AB done: A buffer hbuf is free, and so is X slot cc % XS (XS > AB)
                    if (cc >= AB &&
                        !mbar_wait(chunk_empty((cc - AB) % XS), (uint32_t)(((cc - AB) / XS) & 1), &abort_s)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int e = 0; e < SPG; ++e) {
                        const int st = SPG * g + e;
                        if (st0 + st >= lsteps) break;
                        uint32_t v[32];
                        const uint32_t xrow = stX + (uint32_t)((cc % XS) * SLOTB + st * kPStepB + (i >> 3) * 1024 +
                                                               (i & 7) * 128);
#pragma unroll
                        for (int el = 0; el < 4; ++el) {
                            const int en = (st0 + st) * 4 + el, qq = en / P.terms, term = en - qq * P.terms;
                            const int r0 = (qq % rb) * 16;
                            const bool in = en < entries;
                            const int a = in ? __ldg(P.tile_a + (int64_t)(t / ntn) * kLoraTile + qq / rb) : -1;
                            uint4 b0 = make_uint4(0u, 0u, 0u, 0u), b1 = b0;
                            if (in && row_ok) {
                                const uint4* src =
                                    reinterpret_cast<const uint4*>(P.B + ((int64_t)a * P.N + n) * P.R + r0);
                                b0 = __ldg(src);
                                if (r0 + 8 < P.R) b1 = __ldg(src + 1);
                            }
                            v[8 * el] = b0.x, v[8 * el + 1] = b0.y, v[8 * el + 2] = b0.z, v[8 * el + 3] = b0.w;
                            v[8 * el + 4] = b1.x, v[8 * el + 5] = b1.y, v[8 * el + 6] = b1.z, v[8 * el + 7] = b1.w;
                            uint32_t h[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) h[j] = 0u;
                            if (in && a == my) {
                                const float4* src = reinterpret_cast<const float4*>(P.U + m * P.R + r0);
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    if (r0 + 4 * j < P.R) {
                                        const float4 f = __ldg(src + j);
                                        h[2 * j] = split_pair(f.x, f.y, term);
                                        h[2 * j + 1] = split_pair(f.z, f.w, term);
                                    }
                            }
#pragma unroll
                            for (int hh = 0; hh < 2; ++hh)
                                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                                 xrow + (uint32_t)(((2 * el + hh) ^ (i & 7)) * 16)),
                                             "r"(h[4 * hh]), "r"(h[4 * hh + 1]), "r"(h[4 * hh + 2]), "r"(h[4 * hh + 3])
                                             : "memory");
                        }
                        SHERRY_TMEM_ST32(t_lane + (uint32_t)((hbuf * CS + st) * kPAcols), v);
                    }
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    tc_fence_before();
                    fence_proxy_async();
                    mbar_arrive(full_a(hbuf));
                }
            }
        }
    } else if (warp == kPTmaWarp) {
        // ---------------- TMA producer for X (and, ARN, the latent-weight tiles) ----------------
        if (lane == 0) {
            int c = 0;
            uint32_t cph = 0;  // phase parity of slot c's use
            int issued[XS] = {};  // chunks loaded into each slot (phases of full_x)
            bool ok = true;
            for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
                const int m0 = (t / ntn) * kPBN;
                const int n0 = (t % ntn) * kPBM;
                for (int ch = 0; ch < nchunks; ++ch) {
                    if (!mbar_wait(chunk_empty(c), cph ^ 1u, &abort_s)) {
                        ok = false;
                        break;
                    }
                    const int steps = min(CS, nk - ch * CS);
                    mbar_expect_tx(full_x(c), (uint32_t)(steps * kPStepB * (ARN ? 2 : 1)));
                    for (int st = 0; st < steps; ++st) {
                        tma_load_2d(stX + c * SLOTB + st * kPStepB, &xmap, (ch * CS + st) * kPBK, m0, full_x(c));
                        if constexpr (ARN)
                            tma_load_2d(stX + c * SLOTB + kWOff + st * kPStepB, &wmap, (ch * CS + st) * kPBK, n0,
                                        full_x(c));
                    }
                    ++issued[c];
                    if (++c == XS) { c = 0; cph ^= 1u; }
                }
                if constexpr (LORA) {
                    // the decode warps fill these slots themselves
                    for (int st0 = 0; st0 < lora_steps(t) && ok; st0 += CS) {
                        if (!mbar_wait(chunk_empty(c), cph ^ 1u, &abort_s)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive(full_x(c));
                        ++issued[c];
                        if (++c == XS) { c = 0; cph ^= 1u; }
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
            for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
                int gleft = gs;  // steps left in the current group
                for (int ch = 0; ch < nchunks; ++ch, ++cc) {
                    const int hbuf = cc % AB;
                    if (!mbar_wait(full_a(hbuf), (uint32_t)((cc / AB) & 1), &abort_s)) { ok = false; break; }
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
                    const int lsteps = lora_steps(t);
                    if (ok && lsteps > 0) {
                        if (!mbar_wait(acc_empty(b), bph ^ 1u, &abort_s)) break;
                        const uint32_t td = tmem + (uint32_t)(b * kPBN);
                        for (int st0 = 0; st0 < lsteps; st0 += CS, ++cc) {
                            const int hbuf = cc % AB;
                            if (!mbar_wait(full_a(hbuf), (uint32_t)((cc / AB) & 1), &abort_s) ||
                                !mbar_wait(full_x(c), cph, &abort_s)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint64_t db0 = smem_desc(stX + c * SLOTB);
                            const uint32_t ta0 = tmem + (uint32_t)(kPAcol + hbuf * CS * kPAcols);
                            const int steps = min(CS, lsteps - st0);
                            for (int st = 0; st < steps; ++st)
#pragma unroll
                                for (int kk = 0; kk < kPBK / 16; ++kk)
                                    mma_bf16_ts(td, ta0 + (uint32_t)(st * kPAcols + 8 * kk),
                                                db0 + (uint64_t)((st * kPStepB) >> 4) + (uint64_t)(2 * kk), kIdesc,
                                                (st0 + st + kk) == 0 ? 0u : 1u);
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

// Wd: the latent bf16 weight for Arenas; lora: the adapters' part of P (null: the plain linear)
static int prefill_launch_any(const ProbShape& s, const sherry_linear_desc& d, int64_t M, int y_bf16,
                              const uint16_t* Wd, float lambda, const LoraArgs* lora, cudaStream_t stream) {
    CUtensorMap map, wmap;
    int st = encode_2d(&map, d.X, s.K, M, kPBN);
    if (st) return st;
    if (Wd && (st = encode_2d(&wmap, Wd, s.K, s.N, kPBM))) return st;
    if (!Wd) wmap = map;  // unused
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
        P.B = lora->B;
        P.U = lora->U;
        P.ids = lora->ids;
        P.tile_n = lora->plan.tile_n;
        P.tile_a = lora->plan.tile_a;
        P.R = lora->R;
        P.terms = y_bf16 ? 2 : 3;  // 16 bits of U under a bf16 result, all 24 under an fp32 one
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
    const int64_t tiles = ((s.N + kPBM - 1) / kPBM) * ((M + kPBN - 1) / kPBN);
    const unsigned grid = (unsigned)(tiles < sms ? tiles : sms);
    // 16 epilogue warps (32 token columns each) drain a group accumulator faster; measured on the
    // 3B shapes that pays for group scales up to K = 4096 (+6%) and costs at K = 8192 (-15%) and
    // for per-row scales (one drain per tile; -1.5% at 2048 and 4096 tokens)
    const bool epi16 = s.granularity == SHERRY_PER_GROUP && s.K <= 4096;
    if (lora) {
        if (epi16)
            k_prefill<16, PMode::kLora><<<grid, PRoles<16>::kThreads, kPSmem, stream>>>(map, wmap, P);
        else
            k_prefill<8, PMode::kLora><<<grid, PRoles<8>::kThreads, kPSmem, stream>>>(map, wmap, P);
    } else if (Wd) {
        if (epi16)
            k_prefill<16, PMode::kArenas><<<grid, PRoles<16>::kThreads, kPSmem, stream>>>(map, wmap, P);
        else
            k_prefill<8, PMode::kArenas><<<grid, PRoles<8>::kThreads, kPSmem, stream>>>(map, wmap, P);
    } else {
        if (epi16)
            k_prefill<16, PMode::kPlain><<<grid, PRoles<16>::kThreads, kPSmem, stream>>>(map, wmap, P);
        else
            k_prefill<8, PMode::kPlain><<<grid, PRoles<8>::kThreads, kPSmem, stream>>>(map, wmap, P);
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
    return v ? v : w ? w : x ? x : y;
}

}  // namespace sherry
