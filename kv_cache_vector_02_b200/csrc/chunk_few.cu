// Attention of few new tokens over the paged compressed cache: the way of tq_chunk_attention
// for verification, short follow-ups and single tokens, where decompressing the pages first
// would cost more than the attention.  Everything happens in the rotated domain, as in the
// decode, on tcgen05 with the packed pages read once:
//   s_t = a_t <q', c_k> + b_t <s, sigma>,  q' = R^T q, s = S q,
//         a_t = scale n_t / sqrt(d),  b_t = scale gamma_t sqrt(pi/2) / d,
//   acc = sum_t p_t (n_t / sqrt(d)) c_v,   o = R acc / sum_t p_t.
//
// few_rotate_kernel   q' and s of every (query, head), fp16 (R^T as fp16 hi + lo), with a factor
//                     for the rows that would pass fp16
// few_attend_kernel   one CTA per (32 or 128 rows, kv head, split of the tokens); a row is a
//                     (query, query head of the group) pair.  Per tile of 128 tokens:
//   coding warps   two threads per token (32 rows: 16 warps, four per token) turn its packed
//                  codes and signs, loaded two tiles ahead, into fp16 levels and +-1 in
//                  registers and store them to swizzled operand tiles; a_t, b_t and the values'
//                  scalar v_t = n_t/sqrt(d) go to shared memory
//   issuing warp   D1 = Q' C_k^T, D2 = S_q Sigma^T, O += P V on tcgen05
//   softmax warps  one thread per row: s = a_t D1 + b_t D2 in fp32 (the score's two scalars are
//                  never rounded), mask, running maximum and sum, P to tensor memory.  With 32
//                  rows four warps share a tile's tokens, 32 each, and P is the weight times
//                  v_t: the maximum runs over s + log2 v_t, P = 2^(s + log2 v_t - m + 7) <= 2^15
//                  whatever the values' size, and the sum takes P / v_t.  One rounding to fp16
//                  instead of three (P, v_t, v_t c); with 128 rows, whose scalars do not fit
//                  beside the tiles, the values' tile holds v_t c
// few_join_kernel     the splits joined, o = R acc / l in fp32
//
// Roundings to fp16: q' and s, P, and what of the values the tile holds: the levels (LevelTable)
// alone, or with 128 rows the scalar v_t and its product with the level too.
//
// Bound (32 sequences, 1 to 8 queries of 32 heads, about 3600 tokens each: 147 us, 1.0 TB/s of
// pages; 130 of it in the attend kernel): a capture has the ALU pipe, the busiest, at 52 % over the
// whole kernel, the issue slots at 52 %, the tensor pipe at 37 %, DRAM at 14 %; the counters do not
// tell lookups from softmax and waiting.  The 16 decoding warps sit on three of the four
// sub-partitions, six on one and five each on the others, and a tile is ready with the last of
// them.  The MMAs of a tile, 24 of 65 cycles whatever the rows, would allow 1560 cycles where it
// takes about 4000.  On the way: decompressing to fp16 first, 305 us; one
// register set and one value buffer, 255; two of each up to 32 rows, 171; four softmax warps, 145.
// Tried: four copies of the rows, one per lane quarter, each with its own softmax warp and a
// single value buffer, 205; half of the exponentials by a polynomial, 149 against 148.
#include <cmath>

#include <cuda.h>

#include "dequant.cuh"
#include "device_util.cuh"
#include "mma_sync.cuh"
#include "sm100.cuh"

namespace tq {
namespace {

using namespace sm100;

constexpr int kFN = 128;                            // tokens of a tile
constexpr uint32_t kFTile = 128 * kDim * 2, kFHalf = kFTile / 2;
// Registers (ROWS = 128): 128 a thread at launch (the launch checks it), moved to the softmax.
constexpr int kFRegs = 128, kFSoftmaxRegs = 208, kFCodeRegs = 112, kFIssueRegs = 80;
static_assert(kFSoftmaxRegs + 2 * kFCodeRegs + kFIssueRegs == 4 * kFRegs, "the block's own registers");
// Shared memory.  At most 32 rows (ROWS = 32): a 64-column block of Q' is 32 rows of 128 bytes,
// and the MMA's other rows read whatever follows (results that nothing looks at); what that
// saves holds a second buffer of values.
template <int ROWS>
struct FewSmem {
    static constexpr int kVBufs = ROWS == 32 ? 2 : 1;
    static constexpr int kSub = ROWS == 32 ? 4 : 2;            // threads per token that decode it
    static constexpr int kThreads = ROWS == 32 ? 768 : 512;
    static constexpr uint32_t kBlock = ROWS * 128;             // 64 columns of Q'
    static constexpr uint32_t kOffQ = 0;                       // q' | s: two blocks each
    static constexpr uint32_t kOffK = 4 * kBlock;              // two buffers of C_k | Sigma
    static constexpr uint32_t kOffV = kOffK + 4 * kFTile;      // C_v n / sqrt(d)
    static constexpr uint32_t kOffScal = kOffV + kVBufs * kFTile;  // float [2][kScalars][128]
    static constexpr bool kWeighted = ROWS == 32;              // P carries the values' scalar (below)
    static constexpr int kScalars = kWeighted ? 4 : 2;
    static constexpr uint32_t kOffBar = kOffScal + 2 * kScalars * 128 * 4;
    static constexpr uint32_t kOffTop = kOffBar + 256;         // float [4][32] (ROWS = 32)
    static constexpr uint32_t kBytes = kOffTop + (ROWS == 32 ? 512 : 0);
    static_assert(kBytes <= 232448, "shared memory budget");
    static_assert(kOffK % 1024 == 0 && kBlock % 1024 == 0, "swizzled tiles");
};
constexpr uint64_t kFWaitNs = 2000000000ull;
constexpr float kFRescale = 8.f;  // log2 of what a weight may grow to before O is rescaled
constexpr float kFPHeadroom = 7.f;  // log2 of P over the weight: fp16 loses weights below 2^-32 of the largest (attend_tc.cu)
// ROWS = 32, where P carries the values' scalar v_t: a value below 2^-40 (a token's fp16 values, if
// any is not 0, give 2^-29 at the least) counts as zero, and its P as if v_t were 2^-40.  That keeps
// its weight in the sum: P is flushed below 2^-126, for such a token when its score is 93 - log2 v
// below that of one of scalar v, a share of 2^-79 up to v = 2^14.
constexpr float kFNoValue = 9.0949470177292824e-13f;
constexpr uint32_t kFColS2 = 128, kFColO = 256, kFColP = 384;

enum : int {
    kFBQ = 0,
    kFBKFull = 1,   // +buffer
    kFBKEmpty = 3,  // +buffer
    kFBVFull = 5,   // +buffer
    kFBVEmpty = 7,  // +buffer
    kFBO = 9,       // a tile's P V added
    kFBS = 10,      // scores in tensor memory
    kFBL = 11,      // scores in registers
    kFBP = 12,      // P in tensor memory
    kFBDrain = 13,
    kFNumBars = 14
};

struct FewArgs {
    const uint8_t* kc;
    const uint8_t* vc;
    int num_blocks;
    const int32_t* block_table;
    int max_blocks;
    const int32_t* cu_q;
    const int32_t* seq_lens;
    int B, total_q, max_kv;
    int Hq, Hkv, G, QT;      // QT = ROWS / G queries per CTA
    ChunkLayout lk, lv;
    LevelTable tk, tv;
    float qscale, sscale;    // scale log2(e) / sqrt(d) (times the key levels' scale), scale log2(e) sqrt(pi/2) / d
    float vscale;            // 1 / sqrt(d) times the value levels' scale
    float vmost;             // the largest scalar whose product with every level of the table fits fp16
    const float* qfactor;    // [total_q * Hq] what q' and s of the row are to be multiplied by (a power of two)
    float* part;             // [splits][total_q * Hq][128] unscaled sums, rotated
    float2* ml;              // [splits][total_q * Hq] maximum (base 2) and sum
    void* out;               // rows of sequences with impossible lengths are zeroed here
    int out_fp32;
    uint32_t* err;
};

// Named barriers of n threads: whether x holds in any of them; plain.
__device__ __forceinline__ bool any_of_threads(int id, int n, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(n), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void sync_threads(int id, int n) { asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

template <int ROWS, int WK, int LK, bool PROD, int WV, int LV>
__global__ void __launch_bounds__(FewSmem<ROWS>::kThreads, 1)
    few_attend_kernel(const __grid_constant__ CUtensorMap q_map, const FewArgs a) {
    using M = FewSmem<ROWS>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (sbase & 1023u) {
        if (threadIdx.x == 0) atomicOr(a.err, TQ_DEVERR_INTERNAL);
        return;
    }
    griddep_wait();  // (nothing above depends on an earlier kernel)
    griddep_launch_dependents();
    const int slot = (int)(blockIdx.x / (unsigned)a.Hkv), hk = (int)(blockIdx.x % (unsigned)a.Hkv);
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        for (int b = threadIdx.x; b < a.B; b += M::kThreads)
            if (a.cu_q[b] < 0 || a.cu_q[b + 1] < a.cu_q[b] || a.cu_q[b + 1] > a.total_q)
                atomicOr(a.err, TQ_DEVERR_SEQLEN);
    }
    const int b = find_tile_seq(a.cu_q, a.B, a.QT, slot, lane);
    const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1];
    if (c0 < 0 || c1 <= c0 || c1 > a.total_q) return;  // (entry by entry: differences of any two may overflow)
    const int nq = c1 - c0;
    const int rank = slot - (c0 / a.QT + b);
    if (rank < 0 || rank >= (nq + a.QT - 1) / a.QT) return;
    const int q0 = rank * a.QT, nrows = min(a.QT, nq - q0) * a.G;
    const int kv_len = a.seq_lens[b];
    auto out_row = [&](int r) { return (size_t)(c0 + q0 + r / a.G) * a.Hq + hk * a.G + r % a.G; };
    if (kv_len < nq || kv_len > a.max_kv) {  // a length that cannot be: zero rows
        if (blockIdx.y) return;
        if (threadIdx.x == 0) atomicOr(a.err, TQ_DEVERR_SEQLEN);
        for (int i = threadIdx.x; i < nrows * kDim; i += M::kThreads) {
            const size_t o = out_row(i / kDim) * kDim + i % kDim;
            if (a.out_fp32) static_cast<float*>(a.out)[o] = 0.f;
            else static_cast<__half*>(a.out)[o] = __ushort_as_half(0);
        }
        return;
    }
    // this split's tiles: j0 .. j0 + n - 1, up to the last query's position
    const int off = kv_len - nq;
    const int last = off + min(q0 + a.QT, nq);  // tokens that its last query attends
    const int all = (last + kFN - 1) / kFN;
    const int share = (all + (int)gridDim.y - 1) / (int)gridDim.y, j0 = min((int)blockIdx.y * share, all);
    const int n = min(share, all - j0);
    const size_t prow0 = (size_t)blockIdx.y * a.total_q * a.Hq;
    if (n <= 0) {
        for (int r = threadIdx.x; r < nrows; r += M::kThreads) a.ml[prow0 + out_row(r)] = make_float2(-INFINITY, 0.f);
        return;
    }
    // roles: with 32 rows four softmax warps, on the one lane quarter that has them, share a
    // tile's tokens; with 128 one per quarter
    constexpr int kParts = ROWS == 32 ? 4 : 1;
    constexpr int kSub = M::kSub, kCoders = 4 * kSub;
    const bool softmax = ROWS == 32 ? warp % 4 == 0 && warp < 16 : warp < 4;
    const int coder = ROWS == 32 ? (warp % 4 == 0 ? kCoders : (warp / 4) * 3 + warp % 4 - 1) : warp - 4;
    constexpr int kWarpIssue = ROWS == 32 ? 16 : 12;
    const int live_warps = ROWS == 32 ? kParts : (nrows + 31) / 32;

    const uint32_t bars = sbase + M::kOffBar;
    auto bar = [&](int i) -> uint32_t { return bars + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + M::kOffBar + 8 * kFNumBars);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + M::kOffBar + 8 * kFNumBars + 4);
    int* first_bad = reinterpret_cast<int*>(smem + M::kOffBar + 8 * kFNumBars + 8);
    uint8_t* page_bad = smem + M::kOffBar + 8 * kFNumBars + 16;  // [2][8]
    auto give_up = [&] {
        *abort = 1;
        atomicOr(a.err, TQ_DEVERR_TIMEOUT);
    };
    if (threadIdx.x == 0) {
        mbar_init(bar(kFBQ), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(kFBKFull + s), kCoders);
            mbar_init(bar(kFBKEmpty + s), (uint32_t)live_warps + 1);  // MMAs done, scalars read
        }
        for (int s = 0; s < M::kVBufs; ++s) {
            mbar_init(bar(kFBVFull + s), kCoders);
            mbar_init(bar(kFBVEmpty + s), 1);
        }
        mbar_init(bar(kFBO), 1);
        mbar_init(bar(kFBS), 1);
        mbar_init(bar(kFBL), (uint32_t)live_warps);
        mbar_init(bar(kFBP), (uint32_t)live_warps);
        mbar_init(bar(kFBDrain), 1);
        *abort = 0;
        *first_bad = 0x7FFFFFFF;
        fence_mbar_init();
        const int box = a.G * a.QT * 128;
        mbar_arrive_expect_tx(bar(kFBQ), (uint32_t)(box * (PROD ? 4 : 2)));
        for (int x = 0; x < (PROD ? 4 : 2); ++x)
            tma_load_3d(sbase + M::kOffQ + x * M::kBlock, &q_map, 64 * x, hk * a.G, c0 + q0, bar(kFBQ));
    }
    if (warp == kWarpIssue) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (!softmax && coder < kCoders) {
        if (ROWS != 32) set_registers_down<kFCodeRegs>();
        // ------------------------------------------------------------ codes to operands
        // the threads of a token side by side, so that a warp reads whole rows
        const int tok = coder * (32 / kSub) + lane / kSub, sub = lane % kSub, r16 = tok % kPage;
        const uint32_t lead = lane == 0;
        struct Raw {  // a tile's packed bytes of this thread's part of its token
            PartRow<WK, kSub> kw;
            PartRow<WV, kSub> vw;
            PartRow<1, kSub> sw;
            float kn, kg, vn;
            int state;  // 0 usable, 1 behind the last token, 2 block out of range
        };
        // Block of the thread's token in tile j (nothing looks at it before fetch does); loads are
        // made whether the token is there or not, from the nearest that is: a value that is loaded
        // on one path only is copied at the paths' end, and waited for there.
        const int32_t* table = a.block_table + (size_t)b * a.max_blocks;
        auto block_of = [&](int j) -> int { return table[min((j0 + j) * kFN + tok, kv_len - 1) / kPage]; };
        const uint8_t* kh = a.kc + (size_t)hk * a.lk.bytes;
        const uint8_t* vh = a.vc + (size_t)hk * a.lv.bytes;
        const size_t kstep = (size_t)a.Hkv * a.lk.bytes, vstep = (size_t)a.Hkv * a.lv.bytes;
        auto fetch = [&](Raw& r, int j, int blk) {
            const bool in = blk >= 0 && blk < a.num_blocks;
            r.state = j >= n || (j0 + j) * kFN + tok >= kv_len ? 1 : in ? 0 : 2;
            const uint8_t* kp = kh + (in ? blk : 0) * kstep;
            const uint8_t* vp = vh + (in ? blk : 0) * vstep;
            r.kw.load(kp + r16 * a.lk.code_row + sub * (16 * WK / kSub));
            if (PROD) r.sw.load(kp + a.lk.signs_off + r16 * (kDim / 8) + sub * (16 / kSub));
            r.vw.load(vp + r16 * a.lv.code_row + sub * (16 * WV / kSub));
            r.kn = reinterpret_cast<const float*>(kp + a.lk.norm_off)[r16];
            if (PROD) r.kg = reinterpret_cast<const float*>(kp + a.lk.gamma_off)[r16];
            r.vn = reinterpret_cast<const float*>(vp + a.lv.norm_off)[r16];
        };
        // 16-byte pieces c = sub * kPer .. of the row, at c ^ (row % 8) within their half
        constexpr int kPer = 16 / kSub;
        const uint32_t row = (uint32_t)tok * 128 + (sub * kPer / 8) * kFHalf;
        const int piece0 = sub * kPer % 8;
        // eight threads that store at once (two or four tokens) hit all eight pieces of the banks:
        // the parts of the second half go in another order
        const int swap = kSub == 4 ? (sub >> 1) * 2 : sub * 4;
        bool ok = true;
        auto tile = [&](Raw& r, int j, int s) {
            if (j > 1 && !mbar_wait_all(bar(kFBKEmpty + s), (uint32_t)(j / 2 - 1) & 1u, abort, kFWaitNs)) {
                give_up();
                ok = false;
                return;
            }
            r.kw.exchange(swap != 0);
            if (PROD) r.sw.exchange(swap != 0);
            r.vw.exchange(swap != 0);
            uint8_t* kt = smem + M::kOffK + s * 2 * kFTile + row;
#pragma unroll
            for (int c = 0; c < kPer; ++c) {
                const uint32_t at = (uint32_t)((piece0 + c) ^ swap ^ (tok & 7)) << 4;
                uint32_t w[4];
                levels8<WK, LK>(r.kw.codes(c), a.tk, w);
                *reinterpret_cast<uint4*>(kt + at) = make_uint4(w[0], w[1], w[2], w[3]);
                if (PROD) {
                    signs8(r.sw.codes(c), 0x3C003C00u, w);
                    *reinterpret_cast<uint4*>(kt + kFTile + at) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (sub == 0) {
                float* scal = reinterpret_cast<float*>(smem + M::kOffScal) + s * (M::kScalars * 128) + tok;
                scal[0] = r.state ? 0.f : r.kn * a.qscale;
                if (PROD) scal[128] = r.state ? 0.f : r.kg * a.sscale;
                if (M::kWeighted) {
                    const float v = fmaxf(fabsf(r.vn * a.vscale), kFNoValue);
                    const bool use = r.state == 0 && v < INFINITY;
                    scal[256] = use ? __log2f(v) : 0.f;
                    scal[384] = use ? __fdividef(1.f, v) : 0.f;
                }
                if (r16 == 0) {
                    page_bad[8 * s + tok / kPage] = r.state == 2;
                    if (r.state == 2) atomicOr(a.err, TQ_DEVERR_BLOCK);
                }
            }
            fence_proxy_async_shared();
            mbar_arrive_lead(lead, bar(kFBKFull + s));
            // the values of a token that are not finite (with 128 rows: that pass fp16 in the tile) are
            // left out here and make the rows that attend it NaN at the end: a masked one must not reach any
            const float vn = r.state ? 0.f : r.vn * a.vscale;
            const bool fine = fabsf(vn) <= (M::kWeighted ? 3.402823466e38f : a.vmost);
            if (!fine && sub == 0) atomicMin(first_bad, (j0 + j) * kFN + tok);
            const __half2 v2 = __float2half2_rn(fine ? vn : 0.f);
            const int vb = j % M::kVBufs, use = j / M::kVBufs;
            if (use > 0 && !mbar_wait_all(bar(kFBVEmpty + vb), (uint32_t)(use - 1) & 1u, abort, kFWaitNs)) {
                give_up();
                ok = false;
                return;
            }
            uint8_t* vt = smem + M::kOffV + vb * kFTile + row;
#pragma unroll
            for (int c = 0; c < kPer; ++c) {
                uint32_t w[4];
                levels8<WV, LV>(r.vw.codes(c), a.tv, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&w[i]), v2);
                    if (!M::kWeighted) w[i] = *reinterpret_cast<const uint32_t*>(&x);
                }
                *reinterpret_cast<uint4*>(vt + ((uint32_t)((piece0 + c) ^ swap ^ (tok & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (M::kWeighted && fabsf(r.vn * a.vscale) < kFNoValue) {
#pragma unroll
                for (int c = 0; c < kPer; ++c)
                    *reinterpret_cast<uint4*>(vt + ((uint32_t)((piece0 + c) ^ swap ^ (tok & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_shared();
            mbar_arrive_lead(lead, bar(kFBVFull + vb));
        };
        // a tile's bytes are asked for two tiles ahead, its block id three
        Raw r0{}, r1{};
        int blk = block_of(0);
        int next = block_of(1);
        fetch(r0, 0, blk);
        blk = block_of(2);
        fetch(r1, 1, next);
#pragma unroll 1
        for (int j = 0; j < n && ok; j += 2) {
            next = block_of(j + 3);
            tile(r0, j, 0);
            fetch(r0, j + 2, blk);
            if (j + 1 >= n || !ok) break;
            blk = block_of(j + 4);
            tile(r1, j + 1, 1);
            fetch(r1, j + 3, next);
        }
    } else if (!softmax) {
        if (ROWS != 32) set_registers_down<kFIssueRegs>();
        if (warp == kWarpIssue) {
            // ------------------------------------------------------------ MMA issuer (converged warp)
            constexpr uint32_t id_s = idesc_f16(128, kFN), id_o = idesc_f16(128, kDim) | (1u << 16);
            const uint32_t lead = elect_lane();
            const uint32_t q_lo = sw128_desc_lo(sbase + M::kOffQ), k_lo = sw128_desc_lo(sbase + M::kOffK);
            // the values as they lie, N-major: 64-coordinate blocks kFHalf apart
            const uint32_t v_lo = (((sbase + M::kOffV) >> 4) & 0x3FFFu) | ((kFHalf >> 4) << 16);
            auto wait = [&](int i, int phase) -> bool {
                if (mbar_wait_all(bar(i), (uint32_t)phase & 1u, abort, kFWaitNs)) return true;
                if (lane == 0) give_up();
                return false;
            };
            auto values = [&](int j) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    umma_ts_warp(lead, kFColO, kFColP + ks * 8, sw128_desc(v_lo + (j % M::kVBufs) * (kFTile >> 4) + ks * (2048 >> 4)),
                                 id_o, (j | ks) > 0);
                umma_commit_warp(lead, bar(kFBO));
                umma_commit_warp(lead, bar(kFBVEmpty + j % M::kVBufs));
            };
            bool ok = tmem == 0;
            if (!ok && lane == 0) {
                *abort = 1;
                atomicOr(a.err, TQ_DEVERR_INTERNAL);
            }
            ok = ok && wait(kFBQ, 0);
            for (int j = 0; ok && j < n; ++j) {
                ok = wait(kFBKFull + (j & 1), j / 2) && (j == 0 || wait(kFBL, j - 1));
                if (!ok) break;
                tc_fence_after();
                const uint32_t kl = k_lo + (j & 1) * (2 * kFTile >> 4);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t o = (uint32_t)(ks & 3) * 2 + (uint32_t)(ks >> 2) * (kFHalf >> 4);
                    const uint32_t qo = (uint32_t)(ks & 3) * 2 + (uint32_t)(ks >> 2) * (M::kBlock >> 4);
                    umma_ss_warp(lead, 0, sw128_desc(q_lo + qo), sw128_desc(kl + o), id_s, ks > 0);
                    if (PROD)
                        umma_ss_warp(lead, kFColS2, sw128_desc(q_lo + (2 * M::kBlock >> 4) + qo),
                                     sw128_desc(kl + (kFTile >> 4) + o), id_s, ks > 0);
                }
                umma_commit_warp(lead, bar(kFBS));
                umma_commit_warp(lead, bar(kFBKEmpty + (j & 1)));
                if (j > 0) {
                    ok = wait(kFBP, j - 1) && wait(kFBVFull + (j - 1) % M::kVBufs, (j - 1) / M::kVBufs);
                    if (!ok) break;
                    tc_fence_after();
                    values(j - 1);
                }
            }
            if (ok) ok = wait(kFBP, n - 1) && wait(kFBVFull + (n - 1) % M::kVBufs, (n - 1) / M::kVBufs);
            if (ok) {
                tc_fence_after();
                values(n - 1);
            }
            umma_commit_warp(lead, bar(kFBDrain));
            const volatile int never = 0;
            mbar_wait(bar(kFBQ), 0, &never, kFWaitNs);
            mbar_wait(bar(kFBDrain), 0, &never, kFWaitNs);
            __syncwarp();
        }
    } else {
        if (ROWS != 32) set_registers_up<kFSoftmaxRegs>();
        if (ROWS == 32 || warp < live_warps) {
            // ------------------------------------------------------------ softmax
            constexpr int kCols = kFN / kParts, kChunks = kCols / 32;  // tokens of this thread
            const int part = ROWS == 32 ? warp / 4 : 0, row = ROWS == 32 ? lane : (int)threadIdx.x;
            const uint32_t lanes = ROWS == 32 ? 0u : (uint32_t)warp << 21, lead = lane == 0;
            const uint32_t ts = tmem + lanes + kCols * part, tp = tmem + kFColP + kCols / 2 * part + lanes;
            const uint32_t to = tmem + kFColO + kCols * part + lanes;
            const bool live = row < nrows;
            const int limit = live ? off + q0 + row / a.G - j0 * kFN : -1;  // its last token, from the split's first
            const int masked_from = (off + q0 + 1) / kFN - j0;             // first tile with a masked pair
            float* tops = reinterpret_cast<float*>(smem + M::kOffTop) + lane;  // [kParts][32]
            // D1 and D2 are 1 / fac of the row's products.  With 32 rows the scores of a warp that has
            // such a row are put right as they come; with 128 the exponent's argument takes the factor.
            const float fac = live ? a.qfactor[out_row(row)] : 1.f;
            const float rest = M::kWeighted ? 1.f : fac;
            const bool scaled = __any_sync(0xffffffffu, fac != 1.f) != 0;
            float m = -INFINITY;
            float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
            bool ok = true;
            // after a wait that gave up the loop goes on without waiting: the parts' barriers need every warp
            auto wait = [&](int x, int phase) {
                if (ok && !mbar_wait_all(bar(x), (uint32_t)phase & 1u, abort, kFWaitNs)) {
                    give_up();
                    ok = false;
                }
            };
            for (int j = 0; j < n; ++j) {
                wait(kFBS, j);
                tc_fence_after();
                uint32_t s[kChunks][32];
                const float4* sc = reinterpret_cast<const float4*>(smem + M::kOffScal + (j & 1) * (M::kScalars * 512)) + kCols / 4 * part;
#pragma unroll
                for (int q = 0; q < 2 * kChunks; ++q) {  // 16 tokens
                    uint32_t d1[16], d2[16];
                    tmem_ld16(ts + 16 * q, d1);
                    if (PROD) tmem_ld16(ts + kFColS2 + 16 * q, d2);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // four tokens
                        const float4 fa = sc[4 * q + e];
                        uint32_t* x = &s[q / 2][16 * (q & 1) + 4 * e];
                        const uint32_t* z = &d1[4 * e];
                        // (-0: nothing added)
                        const float4 fl = M::kWeighted ? sc[64 + 4 * q + e] : make_float4(-0.f, -0.f, -0.f, -0.f);
                        const float2 z01 = make_float2(__uint_as_float(z[0]), __uint_as_float(z[1]));
                        const float2 z23 = make_float2(__uint_as_float(z[2]), __uint_as_float(z[3]));
                        float2 u = __ffma2_rn(make_float2(fa.x, fa.y), z01, make_float2(fl.x, fl.y));
                        float2 v = __ffma2_rn(make_float2(fa.z, fa.w), z23, make_float2(fl.z, fl.w));
                        if (PROD) {
                            const float4 fb = sc[32 + 4 * q + e];
                            const uint32_t* y = &d2[4 * e];
                            u = __ffma2_rn(make_float2(fb.x, fb.y), make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), u);
                            v = __ffma2_rn(make_float2(fb.z, fb.w), make_float2(__uint_as_float(y[2]), __uint_as_float(y[3])), v);
                        }
                        x[0] = __float_as_uint(u.x);
                        x[1] = __float_as_uint(u.y);
                        x[2] = __float_as_uint(v.x);
                        x[3] = __float_as_uint(v.y);
                    }
                }
                if (M::kWeighted && scaled) {  // (seldom)
                    // a rounding of log2 v_t is multiplied too: 2^-24 |log2 v_t| fac, at most 2^-15 |log2 v_t|
#pragma unroll
                    for (int q = 0; q < kCols / 4; ++q) {
                        const float4 fl = sc[64 + q];
                        uint32_t* x = &s[q / 8][4 * (q % 8)];
                        x[0] = __float_as_uint(fmaf(__uint_as_float(x[0]) - fl.x, fac, fl.x));
                        x[1] = __float_as_uint(fmaf(__uint_as_float(x[1]) - fl.y, fac, fl.y));
                        x[2] = __float_as_uint(fmaf(__uint_as_float(x[2]) - fl.z, fac, fl.z));
                        x[3] = __float_as_uint(fmaf(__uint_as_float(x[3]) - fl.w, fac, fl.w));
                    }
                }
                const uint2 pb = *reinterpret_cast<const uint2*>(page_bad + 8 * (j & 1));
                tc_fence_before();
                mbar_arrive_lead(lead, bar(kFBL));
                if (!M::kWeighted) mbar_arrive_lead(lead, bar(kFBKEmpty + (j & 1)));
                if (j >= masked_from) {
                    const int lim = limit - j * kFN - kCols * part;
#pragma unroll
                    for (int q = 0; q < kChunks; ++q)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * q + e > lim) s[q][e] = 0xFF800000u;  // -inf
                }
                if (pb.x | pb.y) {
#pragma unroll
                    for (int q = 0; q < kChunks; ++q) {
                        const int page = 2 * (kChunks * part + q);  // the chunk's first of the tile's eight
                        const uint32_t w = (page < 4 ? pb.x : pb.y) >> (8 * (page & 3));
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if ((w >> (8 * (e / 16))) & 1u) s[q][e] = 0xFF800000u;
                    }
                }
                float top = -INFINITY;
#pragma unroll
                for (int q = 0; q < kChunks; ++q) {
                    float m0 = max3(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]), __uint_as_float(s[q][2]));
                    float m1 = max3(__uint_as_float(s[q][16]), __uint_as_float(s[q][17]), __uint_as_float(s[q][18]));
#pragma unroll
                    for (int e = 3; e < 15; e += 2) {
                        m0 = max3(m0, __uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1]));
                        m1 = max3(m1, __uint_as_float(s[q][16 + e]), __uint_as_float(s[q][17 + e]));
                    }
                    top = max3(top, max3(m0, m0, __uint_as_float(s[q][15])), max3(m1, m1, __uint_as_float(s[q][31])));
                }
                if (!M::kWeighted) top *= rest;
                // a NaN or infinite score makes the row's sum and outputs NaN; the maximum carries it
                if (!(top < INFINITY)) top = NAN;
                auto grows = [&](float t) { return t > m + kFRescale || (m == -INFINITY && t > m) || (t != t && m == m); };
                bool any = grows(top);
                any = kParts > 1 ? any_of_threads(1, 32 * kParts, any) : __any_sync(0xffffffffu, any) != 0;
                if (any) {
                    if (kParts > 1) {
                        tops[32 * part] = top;
                        sync_threads(1, 32 * kParts);
#pragma unroll
                        for (int i = 0; i < kParts; ++i) top = max3(top, top, tops[32 * i]);
                        sync_threads(1, 32 * kParts);
                    }
                    const bool grow = grows(top);
                    const float mn = grow ? top : m;
                    if (j > 0) {
                        const float f = grow ? ex2(m - mn) : 1.f;  // (first maximum: ex2(-inf) = 0)
#pragma unroll
                        for (int q = 0; q < 2; ++q) sum[q] = __fmul2_rn(sum[q], make_float2(f, f));
                        wait(kFBO, j - 1);  // the tile before is in O
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < 2 * kChunks; ++q) {
                            uint32_t o[16];
                            tmem_ld16(to + 16 * q, o);
                            tmem_ld_wait();
                            uint32_t lo[8], hi[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                lo[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                hi[e] = __float_as_uint(__uint_as_float(o[8 + e]) * f);
                            }
                            tmem_st8(to + 16 * q, lo);
                            tmem_st8(to + 16 * q + 8, hi);
                        }
                    }
                    m = mn;
                }
                const float mm = m == -INFINITY ? 0.f : m - kFPHeadroom;
                const float2 nm = make_float2(-mm, -mm);
                uint32_t p[2 * kChunks][8];
#pragma unroll
                for (int q = 0; q < 2 * kChunks; ++q) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i = 16 * q + 2 * e;
                        float2 x = make_float2(__uint_as_float(s[i / 32][i % 32]), __uint_as_float(s[i / 32][i % 32 + 1]));
                        x = M::kWeighted ? __fadd2_rn(x, nm) : __ffma2_rn(x, make_float2(rest, rest), nm);
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        if (M::kWeighted) {  // the weight in the sum is without the value's scalar
                            const float2 iv = reinterpret_cast<const float2*>(sc + 96)[8 * q + e];
                            sum[e & 1] = __ffma2_rn(x, iv, sum[e & 1]);
                        } else {
                            sum[e & 1] = __fadd2_rn(sum[e & 1], x);
                        }
                        const __half2 hp = __floats2half2_rn(x.x, x.y);
                        p[q][e] = *reinterpret_cast<const uint32_t*>(&hp);
                    }
                }
                if (M::kWeighted) mbar_arrive_lead(lead, bar(kFBKEmpty + (j & 1)));  // its scalars are read
                // the tile before's P has been read
                if (j > 0 && !any) wait(kFBO, j - 1);
#pragma unroll
                for (int q = 0; q < 2 * kChunks; ++q) tmem_st8(tp + 8 * q, p[q]);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive_lead(lead, bar(kFBP));
            }
            wait(kFBO, n - 1);
            float l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            if (kParts > 1) {  // the row's sum: the same terms in the same order in every part
                tops[32 * part] = l;
                sync_threads(1, 32 * kParts);
                l = 0.f;
#pragma unroll
                for (int i = 0; i < kParts; ++i) l += tops[32 * i];
            }
            const size_t prow = live ? prow0 + out_row(row) : 0;
            if (live && part == 0) {
                const bool hit = limit + j0 * kFN >= *reinterpret_cast<volatile int*>(first_bad);
                a.ml[prow] = ok ? make_float2(m, hit ? NAN : l) : make_float2(-INFINITY, 0.f);
            }
            if (ok) {
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < kChunks; ++q) {
                    uint32_t o[32];
                    tmem_ld32(to + 32 * q, o);
                    tmem_ld_wait();
                    if (!live) continue;
                    float4* d = reinterpret_cast<float4*>(a.part + prow * kDim + kCols * part + 32 * q);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        d[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                           __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                }
                tc_fence_before();
            }
        }
    }
    __syncthreads();
    if (warp == kWarpIssue) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- rotation of the queries
// q' = R^T q and s = S q of 64 rows and 32 output coordinates per CTA, 16 rows per warp, on
// mma.sync (m16n8k16); R^T as fp16 hi + lo, fp32 sums, rounded once.  The matrices' 16-byte
// pieces lie at k ^ (row % 8).
//
// No coordinate of q' or s is larger than 128 times the query's largest (S has entries +-1), which
// passes fp16 from 512 on.  Rows whose bound passes 61440 are stored times a power of two that
// brings it into 2^14 .. 2^15, and the attention multiplies their products by its inverse, `factor`.
constexpr int kRotThreads = 128, kRotRows = 64, kRotCols = 32;
constexpr uint32_t kRotMat = kRotCols * kDim * 2;

__device__ __forceinline__ uint32_t rot_word(const uint8_t* m, int r, int w) {
    return *reinterpret_cast<const uint32_t*>(m + r * 256 + ((((w >> 2) ^ (r & 7)) << 4) | ((w & 3) << 2)));
}

// The row's factor, 1 if its bound fits (or the row is not finite): the four lanes of a row's group
// hold its coordinates between them.
__device__ __forceinline__ float rot_factor(const uint32_t (&qa)[8][4], int first) {
    __half2 m = __float2half2_rn(0.f);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
        for (int i = first; i < 4; i += 2) m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&qa[ks][i])));
    float most = (float)kDim * __half2float(__hmax(__low2half(m), __high2half(m)));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
    return most > 61440.f && most < INFINITY ? scalbnf(1.f, ilogbf(most) - 14) : 1.f;
}

__global__ void __launch_bounds__(kRotThreads) few_rotate_kernel(const uint16_t* q, long long rows, const uint16_t* RTh,
                                                                 const uint16_t* RTl, const uint16_t* Sh, int prod,
                                                                 uint16_t* out, float* factor) {
    __shared__ __align__(16) uint8_t smem[3 * kRotMat];
    const uint32_t base = smem_u32(smem);
    const uint16_t* src[3] = {RTh, RTl, Sh};
    const int pieces = kRotMat / 16, n0 = blockIdx.y * kRotCols;
    for (int i = threadIdx.x; i < (prod ? 3 : 2) * pieces; i += kRotThreads) {
        const int mtx = i / pieces, o = (i - mtx * pieces) * 16, r = o >> 8, k16 = (o >> 4) & 15;
        cp_async16(base + mtx * (pieces * 16) + r * 256 + ((k16 ^ (r & 7)) << 4),
                   reinterpret_cast<const uint8_t*>(src[mtx]) + n0 * 256 + o);
    }
    cp_async_commit();
    griddep_wait();  // the queries may come from the kernel before
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const long long i0 = (long long)blockIdx.x * kRotRows + 16 * (threadIdx.x >> 5) + g, i1 = i0 + 8;
    const bool r0 = i0 < rows, r1 = i1 < rows;
    const uint32_t* q0 = reinterpret_cast<const uint32_t*>(q + (r0 ? i0 : 0) * kDim);
    const uint32_t* q1 = reinterpret_cast<const uint32_t*>(q + (r1 ? i1 : 0) * kDim);
    uint32_t qa[8][4];
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        qa[ks][0] = r0 ? q0[8 * ks + c] : 0u;
        qa[ks][1] = r1 ? q1[8 * ks + c] : 0u;
        qa[ks][2] = r0 ? q0[8 * ks + c + 4] : 0u;
        qa[ks][3] = r1 ? q1[8 * ks + c + 4] : 0u;
    }
    const float f0 = rot_factor(qa, 0), f1 = rot_factor(qa, 1);
    if (blockIdx.y == 0 && c == 0) {
        if (r0) factor[i0] = f0;
        if (r1) factor[i1] = f1;
    }
    const float u0 = 1.f / f0, u1 = 1.f / f1;
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll 1
    for (int nt = 0; nt < kRotCols / 8; ++nt) {  // output coordinates n0 + 8 nt .. + 7
        const int n = 8 * nt + g;
        float dq[4] = {0.f, 0.f, 0.f, 0.f}, ds[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint8_t* lo = smem + kRotMat;
            mma16816(dq, qa[k][0], qa[k][1], qa[k][2], qa[k][3], rot_word(lo, n, 8 * k + c), rot_word(lo, n, 8 * k + c + 4));
            mma16816(dq, qa[k][0], qa[k][1], qa[k][2], qa[k][3], rot_word(smem, n, 8 * k + c), rot_word(smem, n, 8 * k + c + 4));
            if (prod) {
                const uint8_t* sm = smem + 2 * kRotMat;
                mma16816(ds, qa[k][0], qa[k][1], qa[k][2], qa[k][3], rot_word(sm, n, 8 * k + c), rot_word(sm, n, 8 * k + c + 4));
            }
        }
        uint32_t* o0 = reinterpret_cast<uint32_t*>(out + i0 * 2 * kDim + n0) + 4 * nt + c;
        uint32_t* o1 = reinterpret_cast<uint32_t*>(out + i1 * 2 * kDim + n0) + 4 * nt + c;
        if (r0) {
            o0[0] = f2h2(dq[0] * u0, dq[1] * u0);
            if (prod) o0[kDim / 2] = f2h2(ds[0] * u0, ds[1] * u0);
        }
        if (r1) {
            o1[0] = f2h2(dq[2] * u1, dq[3] * u1);
            if (prod) o1[kDim / 2] = f2h2(ds[2] * u1, ds[3] * u1);
        }
    }
}

// ---------------------------------------------------------------- joining and un-rotation
// PER rows per warp, WARPS of them per block: o = R (sum_s 2^(m_s - m) acc_s) / l.  R^T (fp32) in
// shared memory, a lane takes four output coordinates.
struct JoinArgs {
    const float* part;
    const float2* ml;
    int splits;
    const int32_t* cu_q;
    const int32_t* seq_lens;
    int B, total_q, Hq, max_kv;
    const float* RT;
    void* out;
    int out_fp32;
};
constexpr uint32_t join_smem(int rows) { return kDim * kDim * 4 + rows * kDim * 4; }

template <int WARPS, int PER>
__global__ void __launch_bounds__(32 * WARPS) few_join_kernel(const JoinArgs a) {
    constexpr int kJoinThreads = 32 * WARPS, kJoinPer = PER, kJoinRows = WARPS * PER;
    extern __shared__ __align__(16) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    for (int i = threadIdx.x; i < kDim * kDim / 4; i += kJoinThreads) cp_async16(base + 16 * i, a.RT + 4 * i);
    cp_async_commit();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* acc = reinterpret_cast<float*>(smem + kDim * kDim * 4) + warp * kJoinPer * kDim;
    const size_t rows = (size_t)a.total_q * a.Hq;
    bool live[kJoinPer];
#pragma unroll
    for (int r = 0; r < kJoinPer; ++r) {
        const size_t row = (size_t)blockIdx.x * kJoinRows + kJoinPer * warp + r;
        live[r] = false;
        if (row >= rows) continue;  // (uniform in the warp)
        const int qi = (int)(row / a.Hq);
        const int b = find_row_seq(a.cu_q, a.B, qi, lane);
        const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], len = a.seq_lens[b];
        live[r] = qi >= c0 && qi < c1 && c0 >= 0 && c1 <= a.total_q && len >= c1 - c0 && len <= a.max_kv;
        if (!live[r]) continue;
        // lane s has split s (32 at most); no token of the row in a split: its sums were not written
        const float2 x = lane < a.splits ? a.ml[lane * rows + row] : make_float2(-INFINITY, 0.f);
        float m = x.y != 0.f ? x.x : -INFINITY;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float f = x.y != 0.f ? exp2f(x.x - (m == -INFINITY ? 0.f : m)) : 0.f;
        float l = x.y != 0.f ? f * x.y : 0.f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        const float inv = l != 0.f ? 1.f / l : 0.f;
        uint32_t some = __ballot_sync(0xffffffffu, x.y != 0.f);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4* part = reinterpret_cast<const float4*>(a.part + row * kDim) + lane;
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) {
            const float fs = __shfl_sync(0xffffffffu, f, s);
            if (!((some >> s) & 1u)) continue;
            const float4 v = part[s * rows * (kDim / 4)];
            o.x = fmaf(fs, v.x, o.x);
            o.y = fmaf(fs, v.y, o.y);
            o.z = fmaf(fs, v.z, o.z);
            o.w = fmaf(fs, v.w, o.w);
        }
        reinterpret_cast<float4*>(acc + r * kDim)[lane] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
    cp_async_wait<0>();
    __syncthreads();
    float4 o[kJoinPer] = {};
    const float4* RT = reinterpret_cast<const float4*>(smem) + lane;
#pragma unroll 4
    for (int j = 0; j < kDim; j += 4) {
        float4 x[kJoinPer];
#pragma unroll
        for (int r = 0; r < kJoinPer; ++r) x[r] = *reinterpret_cast<const float4*>(acc + r * kDim + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 w = RT[(j + i) * (kDim / 4)];
#pragma unroll
            for (int r = 0; r < kJoinPer; ++r) {
                const float xi = i == 0 ? x[r].x : i == 1 ? x[r].y : i == 2 ? x[r].z : x[r].w;
                o[r].x = fmaf(w.x, xi, o[r].x);
                o[r].y = fmaf(w.y, xi, o[r].y);
                o[r].z = fmaf(w.z, xi, o[r].z);
                o[r].w = fmaf(w.w, xi, o[r].w);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kJoinPer; ++r) {
        if (!live[r]) continue;
        const size_t row = (size_t)blockIdx.x * kJoinRows + kJoinPer * warp + r;
        if (a.out_fp32) {
            reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kDim)[lane] = o[r];
        } else {
            const __half2 p = __floats2half2_rn(o[r].x, o[r].y), q = __floats2half2_rn(o[r].z, o[r].w);
            reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + row * kDim)[lane] =
                make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
        }
    }
}

// A launch whose setup (what comes before its griddep_wait) may overlap the kernel before.
template <typename... P, typename... A>
cudaError_t launch_after(void (*k)(P...), dim3 grid, int threads, uint32_t smem, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <int WARPS, int PER>
cudaError_t launch_join_shape(const JoinArgs& m, long long rows, cudaStream_t stream) {
    auto k = few_join_kernel<WARPS, PER>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = ready_kernel(k, ready, (int)join_smem(WARPS * PER));
    if (e != cudaSuccess) return e;
    const long long blocks = (rows + WARPS * PER - 1) / (WARPS * PER);
    return launch_after(k, dim3((unsigned)blocks), 32 * WARPS, join_smem(WARPS * PER), stream, m);
}

// Every warp reads the whole matrix (64 KB) from shared memory, so a block takes as long as it
// has warps, and fetches it once whatever their number: the fewest rows per block that keep the
// grid within two blocks per SM.  The whole call in us, with 2 x 1 / 4 x 1 / 4 x 2 / 8 x 2
// (warps x rows): 512 rows 19.6 / 21.3 / 22.7 / 27.1; 1024 rows 35.0 / 33.4 / 34.9 / 39.3;
// 2048 rows - / 62.8 / 59.6 / 63.8; 4096 rows - / 47.1 / 43.1 / 42.2 (300 cached
// tokens a sequence; the first three of 1 query each, the last of 4).
cudaError_t launch_join(const JoinArgs& m, long long rows, cudaStream_t stream) {
    const long long per_block = (rows + 2 * 148 - 1) / (2 * 148);
    if (per_block <= 2) return launch_join_shape<2, 1>(m, rows, stream);
    if (per_block <= 4) return launch_join_shape<4, 1>(m, rows, stream);
    if (per_block <= 8) return launch_join_shape<4, 2>(m, rows, stream);
    return launch_join_shape<8, 2>(m, rows, stream);
}

template <int ROWS, int WK, int LK, bool PROD, int WV, int LV>
cudaError_t launch_few_attend(const CUtensorMap& q, const FewArgs& a, dim3 grid, cudaStream_t stream) {
    auto k = few_attend_kernel<ROWS, WK, LK, PROD, WV, LV>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = ready_kernel(k, ready, (int)FewSmem<ROWS>::kBytes, ROWS == 32 ? 0 : kFRegs);  // (the split has to add up)
    if (e != cudaSuccess) return e;
    return launch_after(k, grid, FewSmem<ROWS>::kThreads, FewSmem<ROWS>::kBytes, stream, q, a);
}

}  // namespace

cudaError_t launch_chunk_few(const tq_ctx* ctx, const ChunkPlan& plan, const ChunkCall& c, cudaStream_t stream) {
    uint8_t* ws = c.workspace;
    const long long most = (long long)c.max_blocks * kPage;
    const long long rows = (long long)c.total_q * c.Hq;
    const bool prod = ctx->lay_key.prod;
    uint16_t* rot = reinterpret_cast<uint16_t*>(ws + plan.k_off);
    float* factor = reinterpret_cast<float*>(ws + plan.v_off);
    const long long rot_blocks = (rows + kRotRows - 1) / kRotRows;
    if (rot_blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    cudaError_t e = launch_after(few_rotate_kernel, dim3((unsigned)rot_blocks, kDim / kRotCols), kRotThreads, 0, stream, c.q,
                                 rows, ctx->dev.RTh, ctx->dev.RTl, ctx->dev.Sh, prod ? 1 : 0, rot, factor);
    if (e != cudaSuccess) return e;

    FewArgs a{};
    a.kc = c.kc;
    a.vc = c.vc;
    a.num_blocks = c.num_blocks;
    a.block_table = c.block_table;
    a.max_blocks = c.max_blocks;
    a.cu_q = c.cu_q;
    a.seq_lens = c.seq_lens;
    a.B = c.B;
    a.total_q = c.total_q;
    a.max_kv = (int)(most < c.max_seq_len ? most : c.max_seq_len);
    a.Hq = c.Hq;
    a.Hkv = c.Hkv;
    a.G = c.Hq / c.Hkv;
    a.QT = plan.rows / a.G;
    a.lk = ctx->lay_key;
    a.lv = ctx->lay_value;
    a.tk = ctx->levels_key;
    a.tv = ctx->levels_value;
    const float scale_log2 = c.scale * 1.4426950408889634f;
    a.vscale = a.tv.scale / std::sqrt((float)kDim);
    // (scalar and level are each rounded up by 2^-11 at most: 65440 (1 + 2^-11)^2 < 65504)
    a.vmost = 65440.f * a.tv.scale / ctx->cb_value.c[ctx->cb_value.levels - 1];
    a.qscale = scale_log2 * a.tk.scale / std::sqrt((float)kDim);
    a.sscale = scale_log2 * 1.2533141373155003f / (float)kDim;
    a.qfactor = factor;
    a.part = reinterpret_cast<float*>(ws + plan.part_off);
    a.ml = reinterpret_cast<float2*>(ws + plan.ml_off);
    a.out = c.out;
    a.out_fp32 = c.out_fp32;
    a.err = ctx->dev_error;
    CUtensorMap qm;
    if (!encode_heads_tmap(&qm, rot, c.Hq, c.total_q, (long long)c.Hq * 2 * kDim, a.G, a.QT, 2 * kDim))
        return cudaErrorInvalidValue;
    const long long slots = (long long)c.total_q / a.QT + c.B;
    if (slots * c.Hkv > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)(slots * c.Hkv), (unsigned)plan.splits);
    const int kb = ctx->host.kbits, vb = ctx->host.vbits;
    e = cudaErrorInvalidValue;
#define TQ_FEW(P, KB, VB, ...)                                                                                  \
    if (prod == P && kb == KB && vb == VB)                                                                       \
        e = plan.rows == 32 ? launch_few_attend<32, __VA_ARGS__>(qm, a, grid, stream)                           \
                            : launch_few_attend<128, __VA_ARGS__>(qm, a, grid, stream);
    TQ_FEW(true, 3, 4, 4, 8, true, 4, 16)
    TQ_FEW(true, 2, 3, 2, 4, true, 4, 8)
    TQ_FEW(true, 1, 2, 1, 2, true, 2, 4)
    TQ_FEW(false, 4, 4, 4, 16, false, 4, 16)
    TQ_FEW(false, 3, 3, 4, 8, false, 4, 8)
    TQ_FEW(false, 2, 2, 2, 4, false, 2, 4)
#undef TQ_FEW
    if (e != cudaSuccess) return e;

    JoinArgs m{};
    m.part = a.part;
    m.ml = a.ml;
    m.splits = plan.splits;
    m.cu_q = c.cu_q;
    m.seq_lens = c.seq_lens;
    m.B = c.B;
    m.total_q = c.total_q;
    m.Hq = c.Hq;
    m.max_kv = a.max_kv;
    m.RT = ctx->dev.RT;
    m.out = c.out;
    m.out_fp32 = c.out_fp32;
    return launch_join(m, rows, stream);
}

}  // namespace tq
