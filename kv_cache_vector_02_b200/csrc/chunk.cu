// Causal attention of ragged chunks over the paged compressed cache (tq_chunk_attention):
// the pages are decompressed to fp16 once, tile by tile of 128 tokens, and the attention
// kernel of attend_tc.cu runs over the result, its tokens split over CTAs and joined again
// where there are few rows.
//
// [FQ-TQ] "FlashQuant：生产级KV缓存压缩方案…", section "注意力计算的特殊挑战与QJL校正"
// (the score estimator; the decompressed key k~ = n/sqrt(d) R c + gamma sqrt(pi/2)/d S^T
// (2 sigma - 1) gives it as a plain inner product), section "架构设计" (decompress).
//
// unpack_tc_kernel, one persistent CTA per SM, per (sequence, tile, kv head):
//   warps 0-7  two threads per token: its packed codes and signs (loaded a tile ahead) become
//              fp16 levels and +-1 in registers and go to three swizzled operand tiles
//   warp 12    D1 = C_k R^T, D2 = Sigma S, D3 = C_v R^T on tcgen05 (R, S resident in shared
//              memory; S as it lies, N-major)
//   warps 8-11 one thread per token: k = n_k D1 + gamma' D2, v = n_v D3, rounded to fp16,
//              staged and written by TMA
// Decompressing once costs 156 + 512 bytes a (token, head) against the 156 of the packed
// pages, but every further row tile then reads fp16 from L2 with no arithmetic, and the
// attention is one MMA per 16 coordinates instead of two (codes and signs).
//
// Which way: up to 128 (query, head of a group) rows a sequence on average, chunk_few.cu;
// above, this one.  Measured on both sides (32 heads over 8; us there and here), rows a sequence:
//   32 sequences of 3600 tokens   32: 166, 287   64: 254, 288   128: 301, 292   192: 518, 312
//   4 sequences of 2000           32: 34, 47     96: 45, 47     128: 47, 49     256: 68, 57
//   1 sequence of 32768           32: 57, 103    64: 74, 107    128: 80, 108    256: 127, 117
// 2048 queries of 4096 tokens (8192 rows), 513 and 131.  The average decides for the whole batch,
// so a long piece among single tokens may go the slower way: 700 queries beside 31 single ones
// over 2000 tokens each (91 rows on average), 240 and 195; 1000 beside 63 over 4096 (66), 707 and
// 662; 800 beside 127 over 4096 (29), 937 and 1234; and where the long piece has most of the
// tokens, 900 queries of 4096 beside 31 of 500 (116), 294 and 136.
//
// Roundings to fp16: R (one image of it, as the operand tiles leave no room for a second), the
// levels (LevelTable) and the decompressed keys and values, which halves what the attention reads
// and lets it be one MMA.  By a model of the arithmetic (4096 tokens, 64 bits but for the rounding
// named; relative to the output): values 2.0e-4, R 2.0e-4, P 2.1e-4, keys 0.7e-4, levels 0.5e-4, an
// fp16 output itself 2.1e-4.
//
// Bound: a tile of the decompression takes about 6500 cycles (HBM would allow 3750): its
// lookups, MMAs and stores take turns on one set of operand tiles.  It is 12 us of the 131 above,
// and 188 of the 1290 that 256 queries of 64 heads take over 131072 tokens; the rest is the
// attention's and the join's.
#include <cmath>
#include <cstdint>

#include <cuda.h>

#include "dequant.cuh"
#include "device_util.cuh"
#include "sm100.cuh"

namespace tq {
namespace {

using namespace sm100;

constexpr int kUN = 128;
constexpr uint32_t kUTile = 128 * kDim * 2, kUHalf = kUTile / 2;
constexpr int kUThreads = 416;
constexpr int kUWarpIssue = 12;
constexpr uint32_t kUOffR = 0, kUOffS = kUTile;
constexpr uint32_t kUOffA = 2 * kUTile;                 // C_k | Sigma | C_v
constexpr uint32_t kUOffOut = kUOffA + 3 * kUTile;      // k | v
constexpr uint32_t kUOffBar = kUOffOut + 2 * kUTile;
constexpr uint32_t kUSmem = kUOffBar + 256;
static_assert(kUSmem <= 232448, "shared memory budget");
constexpr uint64_t kUWaitNs = 2000000000ull;
// At most so many (query, head of a group) rows a sequence on average: chunk_few.cu.
constexpr int kFewRows = 128;
// Keys and values decompressed at a time: as many kv heads as fit, one at the least.
constexpr size_t kDecompressedMost = size_t(1) << 30;

enum : int { kUBConst = 0, kUBA = 1, kUBD = 2, kUBDEmpty = 3, kUNumBars = 4 };

struct UnpackArgs {
    const uint8_t* kc;
    const uint8_t* vc;
    int num_blocks;
    const int32_t* block_table;
    int max_blocks;
    const int32_t* cu_q;
    const int32_t* seq_lens;
    int B, max_kv, tiles;   // tiles per sequence, at most
    int Hkv, heads, head0;  // kv heads of the cache; of this launch
    ChunkLayout lk, lv;
    LevelTable tk, tv;
    float k_scale, v_scale; // 1/sqrt(d), times the level tables' scales
    float g_scale;          // sqrt(pi/2)/d
    uint8_t* pages_ok;
    uint32_t* err;
};

__device__ __forceinline__ void tma_store_3d(const void* tmap, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(tmap),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

template <int WK, int LK, bool PROD, int WV, int LV>
__global__ void __launch_bounds__(kUThreads, 1)
    unpack_tc_kernel(const __grid_constant__ CUtensorMap r_map, const __grid_constant__ CUtensorMap s_map,
                     const __grid_constant__ CUtensorMap ko_map, const __grid_constant__ CUtensorMap vo_map,
                     const UnpackArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (warp: uniform)
    if (sbase & 1023u) {
        if (threadIdx.x == 0) atomicOr(a.err, TQ_DEVERR_INTERNAL);
        return;
    }
    const uint32_t bars = sbase + kUOffBar;
    auto bar = [&](int i) -> uint32_t { return bars + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kUOffBar + 8 * kUNumBars);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + kUOffBar + 8 * kUNumBars + 4);
    auto give_up = [&] {
        *abort = 1;
        atomicOr(a.err, TQ_DEVERR_TIMEOUT);
    };
    if (threadIdx.x == 0) {
        mbar_init(bar(kUBConst), 1);
        mbar_init(bar(kUBA), 8);
        mbar_init(bar(kUBD), 1);
        mbar_init(bar(kUBDEmpty), 4);
        *abort = 0;
        fence_mbar_init();
        mbar_arrive_expect_tx(bar(kUBConst), (PROD ? 2 : 1) * kUTile);
        for (int x = 0; x < 2; ++x) {
            tma_load_2d(sbase + kUOffR + x * kUHalf, &r_map, 64 * x, 0, bar(kUBConst));
            if (PROD) tma_load_2d(sbase + kUOffS + x * kUHalf, &s_map, 64 * x, 0, bar(kUBConst));
        }
    }
    if (warp == kUWarpIssue) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // items (sequence, tile, head), head fastest; those behind a sequence's last token are skipped,
    // and sequences without queries
    const long long items = (long long)a.B * a.tiles * a.heads;
    struct Item {
        int b, j, h, len;
    };
    auto next = [&](long long& i, Item& it) -> bool {  // from i on, this CTA's next item
        while (i < items) {
            const long long bj = i / a.heads;
            it.h = (int)(i - bj * a.heads);
            it.b = (int)(bj / a.tiles);
            it.j = (int)(bj - (long long)it.b * a.tiles);
            it.len = a.cu_q[it.b + 1] > a.cu_q[it.b] ? a.seq_lens[it.b] : 0;
            if (it.len <= a.max_kv && it.j * kUN < it.len) return true;
            // on to this CTA's first item of the next sequence
            const long long left = (long long)(it.b + 1) * a.tiles * a.heads - i;
            i += (left + gridDim.x - 1) / gridDim.x * gridDim.x;
        }
        return false;
    };
    // physical block of token t, -1 where there is none to read
    auto block_of = [&](const Item& it, int t) {
        if (t >= it.len) return -1;
        const int blk = a.block_table[(size_t)it.b * a.max_blocks + t / kPage];
        return blk >= 0 && blk < a.num_blocks ? blk : -1;
    };
    auto chunk = [&](const uint8_t* cache, const ChunkLayout& lay, int blk, int h) {
        return cache + ((size_t)blk * a.Hkv + a.head0 + h) * lay.bytes;
    };

    if (warp < 8) {
        // ------------------------------------------------------------ codes to operands
        const int row = threadIdx.x & 127, sub = warp >> 2, r16 = row % kPage;
        PartRow<WK, 2> kw{};
        PartRow<WV, 2> vw{};
        PartRow<1, 2> sw{};
        auto fetch = [&](const Item& it) {
            const int blk = block_of(it, it.j * kUN + row);
            if (blk < 0) return;
            const uint8_t* kp = chunk(a.kc, a.lk, blk, it.h);
            kw.load(kp + r16 * a.lk.code_row + sub * 8 * WK);
            if (PROD) sw.load(kp + a.lk.signs_off + r16 * (kDim / 8) + sub * 8);
            vw.load(chunk(a.vc, a.lv, blk, it.h) + r16 * a.lv.code_row + sub * 8 * WV);
        };
        long long i = blockIdx.x;
        Item it;
        bool have = next(i, it);
        if (have) fetch(it);
        uint8_t* tile = smem + kUOffA + row * 128 + sub * kUHalf;
        for (int k = 0; have; ++k) {
            if (it.h == 0 && threadIdx.x == 0) {  // the tile's usable pages, once for all heads
                uint32_t m = 0;
                for (int p = 0; p < kUN / kPage; ++p) {
                    const int t = it.j * kUN + p * kPage;
                    const bool ok = t >= it.len || block_of(it, t) >= 0;
                    m |= ok ? 1u << p : 0u;
                }
                a.pages_ok[(size_t)it.b * a.tiles + it.j] = (uint8_t)m;
                if (m != 0xff) atomicOr(a.err, TQ_DEVERR_BLOCK);
            }
            // the previous item's MMAs are done with the tiles
            if (k > 0 && !mbar_wait_warp(bar(kUBD), (uint32_t)(k - 1) & 1u, abort, kUWaitNs)) {
                give_up();
                break;
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint32_t at = (uint32_t)(c ^ (row & 7)) << 4;
                uint32_t w[4];
                levels8<WK, LK>(kw.codes(c), a.tk, w);
                *reinterpret_cast<uint4*>(tile + at) = make_uint4(w[0], w[1], w[2], w[3]);
                if (PROD) {
                    signs8(sw.codes(c), 0x3C003C00u, w);
                    *reinterpret_cast<uint4*>(tile + kUTile + at) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                levels8<WV, LV>(vw.codes(c), a.tv, w);
                *reinterpret_cast<uint4*>(tile + 2 * kUTile + at) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_shared();
            mbar_arrive_warp(bar(kUBA));
            i += gridDim.x;
            have = next(i, it);
            if (have) fetch(it);
        }
    } else if (warp == kUWarpIssue) {
        // ------------------------------------------------------------ MMA issuer
        // (the whole warp, converged: see umma_ss_warp; all 512 columns are ours, from 0 on)
        constexpr uint32_t id_k = idesc_f16(128, kDim), id_n = id_k | (1u << 16);
        auto wait = [&](int x, int phase) {
            if (mbar_wait_all(bar(x), (uint32_t)phase & 1u, abort, kUWaitNs)) return true;
            if (lane == 0) give_up();
            return false;
        };
        const uint32_t A = sw128_desc_lo(sbase + kUOffA), R = sw128_desc_lo(sbase + kUOffR);
        // S[j][i] with the output coordinate i contiguous: 64-coordinate blocks kUHalf apart
        const uint32_t S = (((sbase + kUOffS) >> 4) & 0x3FFFu) | ((kUHalf >> 4) << 16);
        long long i = blockIdx.x;
        Item it;
        const uint32_t lead = elect_lane();
        bool ok = tmem == 0;
        if (!ok && lane == 0) {
            *abort = 1;
            atomicOr(a.err, TQ_DEVERR_INTERNAL);
        }
        ok = ok && wait(kUBConst, 0);
        int issued = 0;
        for (int k = 0; ok && next(i, it); ++k, i += gridDim.x) {
            ok = wait(kUBA, k) && (k == 0 || wait(kUBDEmpty, k - 1));
            if (!ok) break;
            ++issued;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint32_t o = (uint32_t)(ks & 3) * 2 + (uint32_t)(ks >> 2) * (kUHalf >> 4);
                umma_ss_warp(lead, 0, sw128_desc(A + o), sw128_desc(R + o), id_k, ks > 0);
                if (PROD)
                    umma_ss_warp(lead, 128, sw128_desc(A + (kUTile >> 4) + o), sw128_desc(S + ks * (2048 >> 4)), id_n, ks > 0);
                umma_ss_warp(lead, 256, sw128_desc(A + 2 * (kUTile >> 4) + o), sw128_desc(R + o), id_k, ks > 0);
            }
            umma_commit_warp(lead, bar(kUBD));
        }
        // the operand matrices have landed and no MMA is in flight when the CTA exits
        const volatile int never = 0;
        mbar_wait(bar(kUBConst), 0, &never, kUWaitNs);
        if (issued > 0) mbar_wait(bar(kUBD), (uint32_t)(issued - 1) & 1u, &never, kUWaitNs);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ scale, round, store
        const int row = threadIdx.x - 256, r16 = row % kPage;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        long long i = blockIdx.x;
        Item it;
        uint8_t* stage = smem + kUOffOut + row * 128;
        auto join = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
        bool pending = false;
        for (int k = 0; next(i, it); ++k, i += gridDim.x) {
            float kn = 0.f, kg = 0.f, vn = 0.f;
            const int blk = block_of(it, it.j * kUN + row);
            if (blk >= 0) {
                const uint8_t* kp = chunk(a.kc, a.lk, blk, it.h);
                kn = reinterpret_cast<const float*>(kp + a.lk.norm_off)[r16] * a.k_scale;
                if (PROD) kg = reinterpret_cast<const float*>(kp + a.lk.gamma_off)[r16] * a.g_scale;
                vn = reinterpret_cast<const float*>(chunk(a.vc, a.lv, blk, it.h) + a.lv.norm_off)[r16] * a.v_scale;
            }
            // the staging area is free (the copies of the item before have read it).  After a
            // wait that gave up the loop goes on without storing: the barrier needs every warp.
            if (pending && row == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            join();
            const bool ok = mbar_wait_warp(bar(kUBD), (uint32_t)k & 1u, abort, kUWaitNs);
            if (!ok) give_up();
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t d1[32], d2[32];
                tmem_ld32(tmem + lanes + 32 * q, d1);
                if (PROD) tmem_ld32(tmem + lanes + 128 + 32 * q, d2);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const int e = 8 * c + 2 * p;
                        float x = kn * __uint_as_float(d1[e]), y = kn * __uint_as_float(d1[e + 1]);
                        if (PROD) {
                            x = fmaf(kg, __uint_as_float(d2[e]), x);
                            y = fmaf(kg, __uint_as_float(d2[e + 1]), y);
                        }
                        const __half2 hh = __floats2half2_rn(x, y);
                        w[p] = *reinterpret_cast<const uint32_t*>(&hh);
                    }
                    const int cc = 4 * q + c;
                    *reinterpret_cast<uint4*>(stage + (cc / 8) * kUHalf + (((cc % 8) ^ (row & 7)) << 4)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t d3[32];
                tmem_ld32(tmem + lanes + 256 + 32 * q, d3);
                tmem_ld_wait();
                if (q == 3) {  // everything read
                    tc_fence_before();
                    mbar_arrive_warp(bar(kUBDEmpty));
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const int e = 8 * c + 2 * p;
                        const __half2 hh = __floats2half2_rn(vn * __uint_as_float(d3[e]), vn * __uint_as_float(d3[e + 1]));
                        w[p] = *reinterpret_cast<const uint32_t*>(&hh);
                    }
                    const int cc = 4 * q + c;
                    *reinterpret_cast<uint4*>(stage + kUTile + (cc / 8) * kUHalf + (((cc % 8) ^ (row & 7)) << 4)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            fence_proxy_async_shared();
            join();
            if (row == 0 && ok) {
                const int z = (it.b * a.tiles + it.j) * kUN;
                for (int x = 0; x < 2; ++x) {
                    tma_store_3d(&ko_map, sbase + kUOffOut + x * kUHalf, 64 * x, it.h, z);
                    tma_store_3d(&vo_map, sbase + kUOffOut + kUTile + x * kUHalf, 64 * x, it.h, z);
                }
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                pending = true;
            }
        }
        if (row == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    if (warp == kUWarpIssue) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The splits of a row joined: o = sum_s 2^(m_s - m) acc_s / sum_s 2^(m_s - m) l_s.  A warp per
// (query, head); four coordinates per lane.
struct CombineArgs {
    const float* part;
    const float2* ml;
    int splits;
    const int32_t* cu_q;
    const int32_t* seq_lens;
    int B, total_q, Hq, max_kv;
    int col0, cols;  // query heads of this launch
    void* out;
    int out_fp32;
};
__global__ void __launch_bounds__(256) chunk_combine_kernel(const CombineArgs a) {
    const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (w >= (long long)a.total_q * a.cols) return;
    const int qi = (int)(w / a.cols), h = a.col0 + (int)(w - (long long)qi * a.cols);
    const int lo = find_row_seq(a.cu_q, a.B, qi, lane);
    const int c0 = a.cu_q[lo], c1 = a.cu_q[lo + 1], len = a.seq_lens[lo];
    if (qi < c0 || qi >= c1 || c0 < 0 || c1 > a.total_q || len < c1 - c0 || len > a.max_kv) return;
    const size_t rows = (size_t)a.total_q * a.Hq, row = (size_t)qi * a.Hq + h;
    float m = -INFINITY;
    for (int s = 0; s < a.splits; ++s) {
        const float2 x = a.ml[s * rows + row];
        if (x.y != 0.f) m = fmaxf(m, x.x);
    }
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < a.splits; ++s) {
        const float2 x = a.ml[s * rows + row];
        if (x.y == 0.f) continue;  // no token of the row in this split: its sums were not written
        const float f = exp2f(x.x - (m == -INFINITY ? 0.f : m));
        const float4 v = reinterpret_cast<const float4*>(a.part + (s * rows + row) * kDim)[lane];
        l += f * x.y;
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    o.x *= inv;
    o.y *= inv;
    o.z *= inv;
    o.w *= inv;
    if (a.out_fp32) {
        reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kDim)[lane] = o;
    } else {
        const __half2 p = __floats2half2_rn(o.x, o.y), q = __floats2half2_rn(o.z, o.w);
        reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + row * kDim)[lane] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
    }
}

template <int WK, int LK, bool PROD, int WV, int LV>
cudaError_t launch_unpack(const tq_ctx* ctx, const CUtensorMap& ko, const CUtensorMap& vo, const UnpackArgs& a,
                          cudaStream_t stream) {
    auto k = unpack_tc_kernel<WK, LK, PROD, WV, LV>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = ready_kernel(k, ready, (int)kUSmem);
    if (e != cudaSuccess) return e;
    const long long items = (long long)a.B * a.tiles * a.heads;
    const unsigned grid = (unsigned)(items < ctx->sm_count ? items : ctx->sm_count);
    k<<<grid, kUThreads, kUSmem, stream>>>(ctx->map_Rh, ctx->map_Sh, ko, vo, a);
    return cudaGetLastError();
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

// Workspace of the splits' partial results, and of the few-row way.
static size_t part_bytes(int splits, int total_q, int Hq) {
    const size_t rows = (size_t)splits * total_q * Hq;
    return up256(rows * kDim * 4) + up256(rows * 8);
}
static size_t few_bytes(int splits, int total_q, int Hq) {
    return up256((size_t)total_q * Hq * 2 * kDim * 2) + up256((size_t)total_q * Hq * 4) + part_bytes(splits, total_q, Hq) + 256;
}

ChunkPlan plan_chunk(const tq_ctx* ctx, int B, int total_q, int Hq, int Hkv, int max_seq_len, size_t limit) {
    ChunkPlan p{};
    p.few = (long long)total_q * (Hq / Hkv) <= (long long)kFewRows * B;
    const long long tiles = max_seq_len > 0 ? ((long long)max_seq_len + 127) / 128 : 1;
    const long long rows = (long long)B * tiles * 128;
    // TMA coordinates and token numbers are 32-bit; chunk_few.cu counts up to five tiles past the last
    if (rows > 0x7FFFFFFFll - 1024) return p;
    p.kv_pad = (int)(tiles * 128);
    const size_t head_bytes = (size_t)rows * kDim * 2 * 2;
    const size_t fixed = up256((size_t)B * tiles) + 256;  // (many rows: besides tokens and partial results)
    p.heads = Hkv;
    if (!p.few) {
        size_t room = head_bytes > kDecompressedMost ? head_bytes : kDecompressedMost;
        const size_t left = limit > fixed ? limit - fixed : 0;
        if (room > left) room = left;
        if (head_bytes * Hkv > room) p.heads = (int)(room / head_bytes);
        if (p.heads < 1) return p;
    }
    auto bytes = [&](int splits) {
        if (p.few) return few_bytes(splits, total_q, Hq);
        return head_bytes * p.heads + fixed + (splits > 1 ? part_bytes(splits, total_q, Hq) : 0);
    };
    if (bytes(1) > limit) return p;
    // Splits of the tokens: as many as make the waves over the SMs shortest, each split
    // costing about three tiles more (its start and end, and its part of the join); of those
    // that the workspace has room for.
    const int G = Hq / Hkv;
    // rows per CTA: 32 where a sequence has no more on average (chunk_few.cu has more buffers then)
    p.rows = !p.few ? 256 : G <= 32 && (long long)total_q * G <= 32ll * B ? 32 : 128;
    const int QC = p.few ? p.rows / G : 2 * (128 / G);
    long long ctas = (total_q + QC - 1) / QC;
    if (ctas < B) ctas = B;
    ctas *= p.heads;
    p.splits = 1;
    double best = 0.;
    for (int s = 1; s <= 32 && (s == 1 || tiles >= (p.few ? 2 : 4) * s) && bytes(s) <= limit; ++s) {
        const double waves = double((ctas * s + ctx->sm_count - 1) / ctx->sm_count);
        const double cost = waves * (double(tiles) / s + 3.) + (s > 1 ? 2. : 0.);
        if (s == 1 || cost < best) {
            best = cost;
            p.splits = s;
        }
    }
    size_t off = 0;
    auto take = [&](size_t n) {
        const size_t at = off;
        off = up256(off + n);
        return at;
    };
    if (p.few) {
        p.k_off = take((size_t)total_q * Hq * 2 * kDim * 2);  // the rotated queries
        p.v_off = take((size_t)total_q * Hq * 4);             // and their factors
    } else {
        p.k_off = take(head_bytes / 2 * p.heads);
        p.v_off = take(head_bytes / 2 * p.heads);
        p.pages_off = take((size_t)B * tiles);
    }
    if (p.few || p.splits > 1) {
        p.part_off = take((size_t)p.splits * total_q * Hq * kDim * 4);
        p.ml_off = take((size_t)p.splits * total_q * Hq * 8);
    }
    p.bytes = bytes(p.splits);
    return p;
}

// A call of as many sequences with fewer queries or tokens might choose more splits, more heads a
// pass or the other way.  It does with fewer splits and heads where it has to (plan_chunk), and
// then needs no more than this call, but for the few-row way's queries: the most of them are
// counted here.
size_t chunk_workspace(const tq_ctx* ctx, int B, int total_q, int Hq, int Hkv, int max_seq_len) {
    const ChunkPlan p = plan_chunk(ctx, B, total_q, Hq, Hkv, max_seq_len, SIZE_MAX);
    if (p.bytes == 0 || p.few) return p.bytes;
    const long long most = (long long)kFewRows * B / (Hq / Hkv);
    const size_t few = few_bytes(1, (int)(most < total_q ? most : total_q), Hq);
    return few > p.bytes ? few : p.bytes;
}

cudaError_t launch_chunk(const tq_ctx* ctx, const ChunkPlan& plan, const ChunkCall& c, cudaStream_t stream) {
    if (plan.few) return launch_chunk_few(ctx, plan, c, stream);
    uint8_t* ws = c.workspace;
    uint16_t* k = reinterpret_cast<uint16_t*>(ws + plan.k_off);
    uint16_t* v = reinterpret_cast<uint16_t*>(ws + plan.v_off);
    const long long most = (long long)c.max_blocks * kPage;
    const int max_kv = (int)(most < c.max_seq_len ? most : c.max_seq_len);
    const int G = c.Hq / c.Hkv;
    UnpackArgs u{};
    u.kc = c.kc;
    u.vc = c.vc;
    u.num_blocks = c.num_blocks;
    u.block_table = c.block_table;
    u.max_blocks = c.max_blocks;
    u.cu_q = c.cu_q;
    u.seq_lens = c.seq_lens;
    u.B = c.B;
    u.max_kv = max_kv;
    u.tiles = plan.kv_pad / 128;
    u.Hkv = c.Hkv;
    u.lk = ctx->lay_key;
    u.lv = ctx->lay_value;
    u.tk = ctx->levels_key;
    u.tv = ctx->levels_value;
    u.k_scale = u.tk.scale / std::sqrt((float)kDim);
    u.v_scale = u.tv.scale / std::sqrt((float)kDim);
    u.g_scale = 1.2533141373155003f / (float)kDim;
    u.pages_ok = ws + plan.pages_off;
    u.err = ctx->dev_error;
    AttendCall at{};
    at.q = c.q;
    at.k = k;
    at.v = v;
    at.q_stride = (long long)c.Hq * kDim;
    at.cu_q = c.cu_q;
    at.kv_lens = c.seq_lens;
    at.B = c.B;
    at.total_q = c.total_q;
    at.max_kv = max_kv;
    at.kv_pad = plan.kv_pad;
    at.pages_ok = u.pages_ok;
    at.Hq = c.Hq;
    at.G = G;
    at.scale = c.scale;
    at.out = c.out;
    at.out_fp32 = c.out_fp32;
    at.splits = plan.splits;
    at.part = reinterpret_cast<float*>(ws + plan.part_off);
    at.part_ml = reinterpret_cast<float*>(ws + plan.ml_off);
    const int kb = ctx->host.kbits, vb = ctx->host.vbits;
    const bool prod = ctx->lay_key.prod;
    for (int head0 = 0; head0 < c.Hkv; head0 += plan.heads) {
        const int heads = c.Hkv - head0 < plan.heads ? c.Hkv - head0 : plan.heads;
        u.head0 = at.head0 = head0;
        u.heads = at.heads = heads;
        at.k_stride = at.v_stride = (long long)heads * kDim;
        cudaError_t e = cudaSuccess;
        {
            CUtensorMap ko, vo;
            const long long rows = (long long)c.B * plan.kv_pad;
            if (!encode_heads_tmap(&ko, k, heads, rows, at.k_stride, 1, kUN) ||
                !encode_heads_tmap(&vo, v, heads, rows, at.v_stride, 1, kUN))
                return cudaErrorInvalidValue;
            if (prod && kb == 3 && vb == 4) e = launch_unpack<4, 8, true, 4, 16>(ctx, ko, vo, u, stream);
            else if (prod && kb == 2 && vb == 3) e = launch_unpack<2, 4, true, 4, 8>(ctx, ko, vo, u, stream);
            else if (prod && kb == 1 && vb == 2) e = launch_unpack<1, 2, true, 2, 4>(ctx, ko, vo, u, stream);
            else if (!prod && kb == 4 && vb == 4) e = launch_unpack<4, 16, false, 4, 16>(ctx, ko, vo, u, stream);
            else if (!prod && kb == 3 && vb == 3) e = launch_unpack<4, 8, false, 4, 8>(ctx, ko, vo, u, stream);
            else if (!prod && kb == 2 && vb == 2) e = launch_unpack<2, 4, false, 2, 4>(ctx, ko, vo, u, stream);
            else return cudaErrorInvalidValue;
            if (e != cudaSuccess) return e;
            count_launches(1);
        }
        e = launch_attend(ctx, at, stream);
        if (e != cudaSuccess) return e;
        if (plan.splits > 1) {
            CombineArgs m{};
            m.part = at.part;
            m.ml = reinterpret_cast<const float2*>(at.part_ml);
            m.splits = plan.splits;
            m.cu_q = c.cu_q;
            m.seq_lens = c.seq_lens;
            m.B = c.B;
            m.total_q = c.total_q;
            m.Hq = c.Hq;
            m.max_kv = max_kv;
            m.col0 = head0 * G;
            m.cols = heads * G;
            m.out = c.out;
            m.out_fp32 = c.out_fp32;
            const long long blocks = ((long long)c.total_q * m.cols + 7) / 8;
            if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
            chunk_combine_kernel<<<(unsigned)blocks, 256, 0, stream>>>(m);
            e = cudaGetLastError();
            if (e != cudaSuccess) return e;
            count_launches(1);
        }
    }
    return cudaSuccess;
}

}  // namespace tq
