// Causal attention of ragged sequences over fp16 keys and values on the sm_100a tensor
// cores (tcgen05 + TMEM + TMA): the kernel behind tq_prompt_attention (the prompt's own
// keys and values) and, over decompressed pages, behind long chunks of tq_chunk_attention.
//
//   s_ij = scale <q_i, k_j>,   o_i = sum_j softmax(s_i)_j v_j,   j <= off + i,
// off = tokens before the sequence's first query (0 for a whole prompt).
//
// One CTA per (256 rows, kv head).  A row is a (query, query head of the group) pair, the
// group's G heads packed beside each other, so keys and values are read once for all of
// them and a causal tile's waste is that of 128 / G queries, not of 128.  The rows are two
// halves of 128 (one TMEM lane each); each has its own softmax warps:
//   warps 0-3, 4-7  softmax of half 0, 1: one thread per row.  Scores come from tensor
//                   memory into registers, the running maximum and sum are fp32, base 2;
//                   P goes to tensor memory as packed fp16
//   warp 8          MMA issuer: S = Q K^T (A, B in shared memory),
//                   O += P V (A in tensor memory, V as it lies: N-major descriptor)
//   warp 9          TMA producer: Q once, then rings of K and V tiles of 128 tokens
// Tensor memory has no room for both halves' scores beside their P and O (640 columns of
// 512), but scores are there only until their softmax has them in registers: the halves
// share one score buffer in turn, and P has columns of its own.  So the next scores are
// computed while the softmax before them runs, and no softmax waits for the tensor core.
// The warps that are not softmax move their registers to it (200 a thread: 128 scores).
//
// Bound (8192 tokens, 64 query heads over 8: 1.1 ms, 990 TFLOP/s, 59 % of the measured GEMM): a
// pair of 128 x 128 tiles takes 3180 cycles where its MMAs alone take 2080 and its
// exponentials, 16 a cycle and SM, 2050.  What is between is the chain from a softmax over
// the barriers to the MMAs and back (a satisfied wait costs about 100 cycles, an arrive 200)
// and the power limit: the SMs run at about 1.45 GHz.  On the way: scores written over by P,
// one tile in flight per half, 4800 cycles; MMAs issued by a converged warp, and two buffers
// of 64 tokens, 3830 (an MMA of N = 64 takes as long as one of 128); one shared buffer of 128,
// 3180.  Tried on that: two threads per row (3390), an issuer warp each for S and P V (3340 to
// 3700), a branch per stage with constant descriptors (4150), an eighth to a half of the
// exponentials by a polynomial (3390 to 3490), 64 tests of a barrier before the first pause (1189 us for 1123).
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since the one it is
// scaled by, and the sum is exact about it either way.  P carries another 2^7 (as O and the sum
// do), so it stays below 2^15, inside fp16, and a weight is lost in its rounding below 2^-32 of
// the row's largest only: at 2^-25, 131072 tokens of such weights were 0.4 % of the output.
//
// Masked places may hold anything.  Scores are masked by position, whatever their value.
// P there is 0, but 0 * inf or 0 * NaN in V would reach O: tiles with a masked (row,
// token) pair are first looked through by warps 10, 11, which clear non-finite values
// in shared memory and note it; a row's epilogue then adds those values back (v * p is v
// for p > 0 and v infinite or NaN) for the tokens the row does attend.
#include <cuda.h>

#include "device_util.cuh"
#include "sm100.cuh"

namespace tq {
namespace {

using namespace sm100;

constexpr int kAN = 128;                    // tokens of a tile
constexpr uint32_t kATile = 128 * kDim * 2;  // one 128 x 128 fp16 operand
constexpr uint32_t kAHalf = kATile / 2;      // 64 of its columns
constexpr int kAKStages = 3, kAVStages = 2;
constexpr int kAThreads = 384;
// Registers: 168 a thread at launch (the launch checks it), moved from warps 8-11 to the softmax.
constexpr int kARegs = 168, kASoftmaxRegs = 200, kAOtherRegs = 104;
static_assert(2 * kASoftmaxRegs + kAOtherRegs == 3 * kARegs, "the block's own registers");
constexpr uint32_t kAOffQ = 0;
constexpr uint32_t kAOffK = 2 * kATile;
constexpr uint32_t kAOffV = kAOffK + kAKStages * kATile;
constexpr uint32_t kAOffBar = kAOffV + kAVStages * kATile;
constexpr uint32_t kASmem = kAOffBar + 512;
constexpr uint64_t kAWaitNs = 2000000000ull;
constexpr float kRescale = 8.f;              // log2 of what a weight may grow to before O is rescaled
constexpr float kPHeadroom = 7.f;            // log2 of P over the weight
static_assert(kASmem <= 232448, "shared memory budget");

enum : int {
    kABQ = 0,
    kABKFull = 1,    // +stage
    kABKEmpty = 4,   // +stage
    kABVFull = 7,    // +stage
    kABVEmpty = 9,   // +stage
    kABVGo = 11,     // +stage: a masked tile's load has been issued
    kABVClean = 13,  // +stage: a masked tile has been looked through
    kABS = 15,       // +half: the half's scores in the buffer
    kABL = 17,       // +half: the half has them in registers
    kABP = 19,       // +half: P in tensor memory
    kABO = 21,       // +half: P V added
    kABDrain = 23,
    kANumBars = 24
};

// V as the B operand: [token][64 coordinates] rows of 128 bytes, 128-byte swizzle, the
// coordinates (N) contiguous.  LBO: from one 64-coordinate block to the next; SBO: from
// one 8-token group to the next.
__device__ __forceinline__ uint32_t v_desc_lo(uint32_t addr) {
    return ((addr >> 4) & 0x3FFFu) | ((kAHalf >> 4) << 16);
}

struct Args {
    const int32_t* cu_q;      // [B + 1] first query row of each sequence
    const int32_t* kv_lens;   // [B] tokens of each sequence (nullptr: its queries)
    int B, total_q;
    int max_kv;               // largest valid length (kv_lens)
    int kv_pad;               // rows from one sequence's tokens to the next's (kv_lens)
    const uint8_t* pages_ok;  // [B][kv_pad / 128] bit p: page p of the tile can be used (nullptr: all)
    int Hq, heads, head0, G, QT;  // heads: kv heads of this launch, from head0 on; QT = 128 / G queries per half
    float scale_log2;
    const uint16_t* v;        // the values again, for the epilogue's repair
    long long v_stride;       // elements from one token to the next
    void* out;
    int out_fp32;
    float* part;              // [splits][total_q * Hq][128] unscaled sums, or null: one split
    float2* part_ml;          // [splits][total_q * Hq] maximum (base 2) and sum
    uint32_t* err;
};

__global__ void __launch_bounds__(kAThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tq_map, const __grid_constant__ CUtensorMap tk_map,
                     const __grid_constant__ CUtensorMap tv_map, const Args a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (warp: uniform)
    if (sbase & 1023u) {
        if (threadIdx.x == 0) atomicOr(a.err, TQ_DEVERR_INTERNAL);
        return;
    }
    // ---- which rows
    const int slot = (int)(blockIdx.x / (unsigned)a.heads), hk = (int)(blockIdx.x % (unsigned)a.heads);
    const int QC = 2 * a.QT;
    if (blockIdx.x == 0 && blockIdx.y == 0) {  // the whole list is looked through once
        for (int b = threadIdx.x; b < a.B; b += kAThreads)
            if (a.cu_q[b] < 0 || a.cu_q[b + 1] < a.cu_q[b] || a.cu_q[b + 1] > a.total_q)
                atomicOr(a.err, TQ_DEVERR_SEQLEN);
    }
    const int b = find_tile_seq(a.cu_q, a.B, QC, slot, lane);
    const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1];
    if (c0 < 0 || c1 <= c0 || c1 > a.total_q) return;  // (entry by entry: differences of any two may overflow)
    const int nq = c1 - c0;
    const int tiles = (nq + QC - 1) / QC;
    const int rank = slot - (c0 / QC + b);
    if (rank < 0 || rank >= tiles) return;
    const int q0 = (tiles - 1 - rank) * QC;  // this CTA's first query; the sequence's heaviest tile first
    const int kv_len = a.kv_lens ? a.kv_lens[b] : nq;
    if (kv_len < nq || (a.kv_lens && kv_len > a.max_kv)) {  // a length that cannot be: zero rows
        if (blockIdx.y) return;
        if (threadIdx.x == 0) atomicOr(a.err, TQ_DEVERR_SEQLEN);
        const int rows = min(QC, nq - q0) * a.G;
        for (int i = threadIdx.x; i < rows * kDim; i += kAThreads) {
            const int r = i / kDim;
            const size_t o = ((size_t)(c0 + q0 + r / a.G) * a.Hq + (a.head0 + hk) * a.G + r % a.G) * kDim + i % kDim;
            if (a.out_fp32) static_cast<float*>(a.out)[o] = 0.f;
            else static_cast<__half*>(a.out)[o] = __ushort_as_half(0);
        }
        return;
    }
    const int off = kv_len - nq;
    // tiles of each half: up to its last query's position
    auto tiles_of = [&](int h) {
        const int first = q0 + h * a.QT;
        return first < nq ? (off + min(nq, first + a.QT) + kAN - 1) / kAN : 0;
    };
    // this split's share of the tiles, j0 on (counts and tile numbers below are from there)
    const int all = max(tiles_of(0), tiles_of(1));
    const int share = (all + (int)gridDim.y - 1) / (int)gridDim.y, j0 = min((int)blockIdx.y * share, all);
    const int n0 = max(0, min(tiles_of(0) - j0, share)), n1 = max(0, min(tiles_of(1) - j0, share)), n = max(n0, n1);
    const int masked_from = max((off + q0 + 1) / kAN - j0, 0);  // first tile with a masked (row, token) pair
    if (n == 0) {  // nothing for this split
        if (a.part) {
            const int rows = min(QC, nq - q0) * a.G;
            for (int r = threadIdx.x; r < rows; r += kAThreads)
                a.part_ml[(size_t)blockIdx.y * a.total_q * a.Hq + (size_t)(c0 + q0 + r / a.G) * a.Hq +
                          (a.head0 + hk) * a.G + r % a.G] = make_float2(-INFINITY, 0.f);
        }
        return;
    }

    // row of the split's token 0 (the sequence's token j0 * 128)
    const int kv_row = (a.kv_lens ? b * a.kv_pad : c0) + j0 * kAN;

    const uint32_t bars = sbase + kAOffBar;
    auto bar = [&](int i) -> uint32_t { return bars + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kAOffBar + 8 * kANumBars);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + kAOffBar + 8 * kANumBars + 4);
    volatile int* repaired = reinterpret_cast<volatile int*>(smem + kAOffBar + 8 * kANumBars + 8);
    auto give_up = [&] {
        *abort = 1;
        atomicOr(a.err, TQ_DEVERR_TIMEOUT);
    };
    if (threadIdx.x == 0) {
        mbar_init(bar(kABQ), 1);
        for (int s = 0; s < kAKStages; ++s) {
            mbar_init(bar(kABKFull + s), 1);
            mbar_init(bar(kABKEmpty + s), 1);
        }
        for (int s = 0; s < kAVStages; ++s) {
            mbar_init(bar(kABVFull + s), 1);
            mbar_init(bar(kABVEmpty + s), 1);
            mbar_init(bar(kABVClean + s), 2);
            mbar_init(bar(kABVGo + s), 1);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(bar(kABS + h), 1);
            mbar_init(bar(kABL + h), 4);
            mbar_init(bar(kABP + h), 4);
            mbar_init(bar(kABO + h), 1);
        }
        mbar_init(bar(kABDrain), 1);
        *abort = 0;
        *repaired = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    // pages that cannot be used among this split's (seldom: looked up per step only then)
    bool bad_page = false;
    const uint8_t* pages_ok = a.pages_ok ? a.pages_ok + (size_t)b * (a.kv_pad / kAN) + j0 : nullptr;
    if (pages_ok)
        for (int j = threadIdx.x; j < n; j += kAThreads) bad_page |= pages_ok[j] != 0xff;
    tc_fence_before();
    bad_page = __syncthreads_or(bad_page);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    constexpr uint32_t kColP = 128, kColO = 256;  // columns: scores | P0 | P1 (64 each) | O0 | O1 (128 each)

    if (warp >= 8) {
        set_registers_down<kAOtherRegs>();
        if (warp == 9) {
            // ------------------------------------------------------------ producer
            if (lane == 0) {
                int kj = 0, vj = 0;
                const int half_bytes = a.G * a.QT * 128;
                mbar_arrive_expect_tx(bar(kABQ), (uint32_t)(half_bytes * 4));
                for (int h = 0; h < 2; ++h)
                    for (int x = 0; x < 2; ++x)
                        tma_load_3d(sbase + kAOffQ + h * kATile + x * kAHalf, &tq_map, 64 * x, (a.head0 + hk) * a.G,
                                    c0 + q0 + h * a.QT, bar(kABQ));
                auto load = [&](const void* map, int full, int empty, uint32_t at, int stages, int j) -> bool {
                    const int s = j % stages;
                    if (!mbar_wait(bar(empty + s), (uint32_t)(j / stages & 1) ^ 1u, abort, kAWaitNs)) {
                        give_up();
                        return false;
                    }
                    mbar_arrive_expect_tx(bar(full + s), kATile);
                    for (int x = 0; x < 2; ++x)
                        tma_load_3d(sbase + at + s * kATile + x * kAHalf, map, 64 * x, hk, kv_row + j * kAN,
                                    bar(full + s));
                    return true;
                };
                bool ok = load(&tk_map, kABKFull, kABKEmpty, kAOffK, kAKStages, 0);
                kj = ok;
                for (int j = 0; ok && j < n; ++j) {
                    if (j + 1 < n) {
                        ok = load(&tk_map, kABKFull, kABKEmpty, kAOffK, kAKStages, j + 1);
                        kj += ok;
                    }
                    if (ok) {
                        ok = load(&tv_map, kABVFull, kABVEmpty, kAOffV, kAVStages, j);
                        vj += ok;
                        if (ok && j >= masked_from) mbar_arrive(bar(kABVGo + j % kAVStages));
                    }
                }
                // every copy lands before the CTA can exit
                const volatile int never = 0;
                mbar_wait(bar(kABQ), 0, &never, kAWaitNs);
                for (int j = max(0, kj - kAKStages); j < kj; ++j)
                    mbar_wait(bar(kABKFull + j % kAKStages), (uint32_t)(j / kAKStages) & 1u, &never, kAWaitNs);
                for (int j = max(0, vj - kAVStages); j < vj; ++j)
                    mbar_wait(bar(kABVFull + j % kAVStages), (uint32_t)(j / kAVStages) & 1u, &never, kAWaitNs);
            }
            __syncwarp();
        } else if (warp == 8) {
            // ------------------------------------------------------------ MMA issuer
            // (the whole warp, converged: see umma_ss_warp; all 512 columns are ours, from 0 on)
            constexpr uint32_t id_s = idesc_f16(128, kAN), id_o = idesc_f16(128, kDim) | (1u << 16);
            const uint32_t q_lo = sw128_desc_lo(sbase + kAOffQ), k_lo = sw128_desc_lo(sbase + kAOffK);
            const uint32_t v_lo = v_desc_lo(sbase + kAOffV);
            auto wait = [&](int i, uint32_t parity) -> bool {
                if (mbar_wait_all(bar(i), parity & 1u, abort, kAWaitNs)) return true;
                if (lane == 0) give_up();
                return false;
            };
            const uint32_t lead = elect_lane();
            auto scores = [&](int h, int stage) {
                const uint32_t ql = q_lo + h * (kATile >> 4), kl = k_lo + stage * (kATile >> 4);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t o = (uint32_t)(ks & 3) * 2 + (uint32_t)(ks >> 2) * (kAHalf >> 4);
                    umma_ss_warp(lead, 0, sw128_desc(ql + o), sw128_desc(kl + o), id_s, ks > 0);
                }
                umma_commit_warp(lead, bar(kABS + h));
            };
            auto values = [&](int h, int stage, bool first) {
                const uint32_t vl = v_lo + stage * (kATile >> 4);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    umma_ts_warp(lead, kColO + h * 128, kColP + h * 64 + ks * 8, sw128_desc(vl + ks * (2048 >> 4)),
                                 id_o, !(first && ks == 0));
                umma_commit_warp(lead, bar(kABO + h));
            };
            bool ok = tmem == 0;
            if (!ok && lane == 0) {
                *abort = 1;
                atomicOr(a.err, TQ_DEVERR_INTERNAL);
            }
            ok = ok && wait(kABQ, 0) && wait(kABKFull, 0);
            int user = -1;               // whose scores the buffer last held, and of which tile
            uint32_t used = 0;
            auto next_scores = [&](int h, int j, int stage) {
                if (ok && user >= 0) ok = wait(kABL + user, used);
                if (!ok) return;
                tc_fence_after();
                scores(h, stage);
                user = h;
                used = (uint32_t)j;
            };
            if (n0) next_scores(0, 0, 0);
            if (n1) next_scores(1, 0, 0);
            if (ok) umma_commit_warp(lead, bar(kABKEmpty));
            int vs = 0, kn = 0;          // stages of tile j's values and of tile j + 1's keys
            uint32_t vp = 0, kp = 0;     // and their phases
            for (int j = 0; ok && j < n; ++j) {
                if (++kn == kAKStages) {
                    kn = 0;
                    kp ^= 1u;
                }
                if (j + 1 < n) ok = wait(kABKFull + kn, kp);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int nh = h ? n1 : n0;
                    if (j + 1 < nh) next_scores(h, j + 1, kn);
                    if (ok && h == 0)
                        ok = j >= masked_from ? wait(kABVClean + vs, (j - masked_from) / kAVStages)
                                              : wait(kABVFull + vs, vp);
                    if (ok && j < nh) {
                        ok = wait(kABP + h, j);
                        if (ok) {
                            tc_fence_after();
                            values(h, vs, j == 0);
                        }
                    }
                }
                if (!ok) break;
                umma_commit_warp(lead, bar(kABVEmpty + vs));
                if (j + 1 < n) umma_commit_warp(lead, bar(kABKEmpty + kn));
                if (++vs == kAVStages) {
                    vs = 0;
                    vp ^= 1u;
                }
            }
            // nothing is in flight when the CTA exits
            umma_commit_warp(lead, bar(kABDrain));
            const volatile int never = 0;
            mbar_wait(bar(kABDrain), 0, &never, kAWaitNs);
            __syncwarp();
        } else {
            // ------------------------------------------------------------ masked tiles' values
            for (int j = masked_from; j < n; ++j) {
                const int s = j % kAVStages;
                // (these warps do not follow the unmasked tiles' phases of the stage: its load's
                // issue tells them that the phase of this tile is the current one)
                const uint32_t go = (uint32_t)((j - masked_from) / kAVStages) & 1u;
                if (!__all_sync(0xffffffffu, mbar_wait_asleep(bar(kABVGo + s), go, abort, kAWaitNs)) ||
                    !mbar_wait_warp(bar(kABVFull + s), (uint32_t)(j / kAVStages) & 1u, abort, kAWaitNs)) {
                    give_up();
                    break;
                }
                uint4* v = reinterpret_cast<uint4*>(smem + kAOffV + s * kATile);
                bool any = false;
#pragma unroll 4
                for (int i = threadIdx.x - 320; i < (int)(kATile / 16); i += 64) {
                    uint4 x = v[i];
                    uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    bool bad = false;
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        // bit 15 / 31: the half's exponent is all ones
                        const uint32_t e = ((w[p] & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
                        if (e) {
                            bad = true;
                            if (e & 0x8000u) w[p] &= 0xFFFF0000u;
                            if (e & 0x80000000u) w[p] &= 0x0000FFFFu;
                        }
                    }
                    if (bad) {
                        any = true;
                        v[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                if (any) *repaired = 1;
                fence_proxy_async_shared();
                mbar_arrive_warp(bar(kABVClean + s));
            }
        }
    } else {
        set_registers_up<kASoftmaxRegs>();
        // ------------------------------------------------------------ softmax
        const int h = warp >> 2, row = threadIdx.x & 127;
        const int nh = h ? n1 : n0;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes
        const uint32_t ts = tmem + lanes, tp = tmem + kColP + h * 64 + lanes, to = tmem + kColO + h * 128 + lanes;
        const int qi = q0 + h * a.QT + row / a.G;           // this row's query
        const bool live = row < a.G * a.QT && qi < nq;
        const int limit = live ? off + qi - j0 * kAN : -1;  // its last token
        const int half_masked = (off + q0 + h * a.QT + 1) / kAN - j0;  // first tile with a masked pair
        const uint32_t lead = lane == 0;
        const float2 sc = make_float2(a.scale_log2, a.scale_log2);
        float m = -INFINITY;
        float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
        bool ok = true;
        auto wait = [&](int x, int phase) -> bool {
            if (mbar_wait_all(bar(x), (uint32_t)phase & 1u, abort, kAWaitNs)) return true;
            give_up();
            return false;
        };
        for (int j = 0; j < nh; ++j) {
            ok = wait(kABS + h, j);
            if (!ok) break;
            tc_fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, s[q]);
            tmem_ld_wait();
            tc_fence_before();
            mbar_arrive_lead(lead, bar(kABL + h));
            if (j >= half_masked) {
                const int lim = limit - j * kAN;
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * q + e > lim) s[q][e] = 0xFF800000u;  // -inf
            }
            if (bad_page) {
                const int okp = pages_ok[j];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!((okp >> (2 * q + e / 16)) & 1)) s[q][e] = 0xFF800000u;
            }
            float mx[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                mx[q] = max3(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]), __uint_as_float(s[q][2]));
#pragma unroll
                for (int e = 3; e < 31; e += 2)
                    mx[q] = max3(mx[q], __uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1]));
                mx[q] = max3(mx[q], mx[q], __uint_as_float(s[q][31]));
            }
            float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]) * a.scale_log2;
            // a NaN or infinite score makes the row's sum and outputs NaN; the maximum carries it
            if (!(top < INFINITY)) top = NAN;
            const bool grow = top > m + kRescale || (m == -INFINITY && top > m) || (top != top && m == m);
            // the tile before is in O, and its P has been read
            if (j > 0) ok = wait(kABO + h, j - 1);
            if (!ok) break;
            if (__any_sync(0xffffffffu, grow)) {
                const float mn = grow ? top : m;
                if (j > 0) {
                    const float f = grow ? ex2(m - mn) : 1.f;  // (first maximum: ex2(-inf) = 0)
#pragma unroll
                    for (int q = 0; q < 2; ++q) sum[q] = __fmul2_rn(sum[q], make_float2(f, f));
                    tc_fence_after();
#pragma unroll 1
                    for (int q = 0; q < 8; ++q) {
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
            const float mm = m == -INFINITY ? 0.f : m - kPHeadroom;
            const float2 nm = make_float2(-mm, -mm);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t p[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float2 x = make_float2(__uint_as_float(s[2 * q + e / 16][2 * e % 32]),
                                           __uint_as_float(s[2 * q + e / 16][2 * e % 32 + 1]));
                    x = __ffma2_rn(x, sc, nm);
                    x.x = ex2(x.x);
                    x.y = ex2(x.y);
                    sum[e & 1] = __fadd2_rn(sum[e & 1], x);
                    const __half2 hp = __floats2half2_rn(x.x, x.y);
                    p[e] = *reinterpret_cast<const uint32_t*>(&hp);
                }
                tmem_st32(tp + 32 * q, p);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_lead(lead, bar(kABP + h));
        }
        if (ok && nh > 0) ok = wait(kABO + h, nh - 1);
        const float l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        const size_t orow = (size_t)(c0 + qi) * a.Hq + (a.head0 + hk) * a.G + row % a.G;
        const size_t prow = (size_t)blockIdx.y * a.total_q * a.Hq + orow;
        if (a.part && live) a.part_ml[prow] = ok ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
        if (ok && nh > 0) {
            tc_fence_after();
            const float inv = a.part ? 1.f : l != 0.f ? 1.f / l : 0.f;  // (no token: a zero row)
            const bool fix = *repaired != 0;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                uint32_t o[32];
                tmem_ld32(to + 32 * q, o);
                tmem_ld_wait();
                if (!live) continue;
                float f[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * inv;
                if (fix) {
                    for (int t = masked_from * kAN; t <= limit; ++t) {
                        const __half* v =
                            reinterpret_cast<const __half*>(a.v) + (kv_row + t) * a.v_stride + hk * kDim + 32 * q;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float x = __half2float(v[i]);
                            if (!isfinite(x)) f[i] += x;
                        }
                    }
                }
                if (a.part || a.out_fp32) {
                    float4* d = reinterpret_cast<float4*>(
                        (a.part ? a.part + prow * kDim : static_cast<float*>(a.out) + orow * kDim) + 32 * q);
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                } else {
                    uint4* d = reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + orow * kDim + 32 * q);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const __half2 x = __floats2half2_rn(f[8 * i + 2 * p], f[8 * i + 2 * p + 1]);
                            w[p] = *reinterpret_cast<const uint32_t*>(&x);
                        }
                        d[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_attend(const tq_ctx* ctx, const AttendCall& c, cudaStream_t stream) {
    Args a{};
    a.cu_q = c.cu_q;
    a.kv_lens = c.kv_lens;
    a.B = c.B;
    a.total_q = c.total_q;
    a.max_kv = c.max_kv;
    a.kv_pad = c.kv_pad;
    a.pages_ok = c.pages_ok;
    a.Hq = c.Hq;
    a.heads = c.heads;
    a.head0 = c.head0;
    a.G = c.G;
    a.QT = 128 / c.G;
    a.scale_log2 = c.scale * 1.4426950408889634f;
    a.v = c.v;
    a.v_stride = c.v_stride;
    a.out = c.out;
    a.out_fp32 = c.out_fp32;
    a.part = c.splits > 1 ? c.part : nullptr;
    a.part_ml = reinterpret_cast<float2*>(c.part_ml);
    a.err = ctx->dev_error;
    const long long kv_rows = c.kv_lens ? (long long)c.B * c.kv_pad : c.total_q;
    CUtensorMap mq, mk, mv;
    if (!encode_heads_tmap(&mq, c.q, c.Hq, c.total_q, c.q_stride, c.G, a.QT) ||
        !encode_heads_tmap(&mk, c.k, c.heads, kv_rows, c.k_stride, 1, kAN) ||
        !encode_heads_tmap(&mv, c.v, c.heads, kv_rows, c.v_stride, 1, kAN))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = ready_kernel(attend_tc_kernel, ready, (int)kASmem, kARegs);  // (the register split has to add up)
    if (e != cudaSuccess) return e;
    // slots of all sequences: floor(total / q) + B bounds every sequence's last one
    const long long slots = (long long)c.total_q / (2 * a.QT) + c.B;
    if (slots * c.heads > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)(slots * c.heads), (unsigned)(c.splits > 1 ? c.splits : 1));
    attend_tc_kernel<<<grid, kAThreads, kASmem, stream>>>(mq, mk, mv, a);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace tq
