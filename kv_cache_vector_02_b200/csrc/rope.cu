// Rotary positions of queries and keys, before attention and compress.
//
// Pair i of a head (i < rot/2) is turned by the angle a = pos * theta_i:
//   y1 = m (x1 cos a - x2 sin a),   y2 = m (x2 cos a + x1 sin a),
// the rest of the head is copied.  The transposed map (the gradient with respect to x)
// turns by -a.
//
// Angles: the table holds theta_i / 2 pi as a 64-bit fraction of a turn, so pos * turns[i]
// modulo 2^64 is the angle's fraction of a turn, exact up to pos * 2^-64 turns however far
// the position is.  32 bits of it go into sincospif as a float of 24: up to 2^-26 turns
// (9.4e-8 rad) at half a turn, less for smaller angles.  A float product pos * theta would lose the angle from about 10^5 on.
//
// Bound by HBM: every value is read and written once.  A block takes one token (a few where
// they are small): its threads first issue the 16-byte loads of two units each (a unit: 8 pairs in the
// half layout, 8 values in the interleaved one), then one thread per (token, pair) puts
// (cos, sin) into shared memory, and after one barrier every head of the token uses them.
// Computing them per head instead costs Hq + Hkv times the sincospif work.
// 32768 tokens of 72 heads: 186 us, 6.5 TB/s, the measured copy's rate.  Many small blocks carry
// it, their barriers and their loads at different times (before (cos, sin) lay in the lanes' order: 196 to 215 us;
// 265 with blocks of 256 threads and four units, 331 with 512 and two, 246 with 128 and five); a
// division per unit by a runtime number, now a multiplication, cost another 20.  4099 tokens of
// 40 heads, half of each rotated: 20 us, 4.1 TB/s, against 13 for its bytes
// (four units a thread: 22.5).
#include <cuda_fp16.h>

#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kRThreads = 128;
constexpr int kRUnits = 2;      // units in flight per thread
constexpr int kRTokens = 8;     // tokens of a block, at most

struct RopeArgs {
    const uint16_t* q;
    const uint16_t* k;
    uint16_t* qo;
    uint16_t* ko;
    long long qs, ks, qos, kos;  // token strides (elements)
    const int32_t* pos;
    int T, Hq, Hkv;              // Hq / Hkv = 0: no q / k
    int tokens;                  // tokens per block
    int per_head;                // units per head
    uint32_t by_head, by_heads;  // ceil(2^32 / per_head), ceil(2^32 / (Hq + Hkv)) (0: divide by 1)
    float m, ms;                 // factor on cos and on sin (negative: transposed)
    tq_rope_table tab;
};

struct Unit {
    const __half* src;
    __half* dst;
    int tok, lane;
};

// VEC = 8: 16-byte units.  Half layout: unit u < rot/16 holds values [8u, 8u+8) and their
// partners rot/2 further; the units behind them are 8 values that are not turned.
// Interleaved: unit u holds values [8u, 8u+8).
// VEC = 1 (half layout whose rot/2 is no multiple of 8): unit u < rot/2 holds one pair, the
// others one value.
// Place of pair p's (cos, sin): the lanes of a head read theirs side by side.
template <bool HALF, int VEC>
__device__ __forceinline__ int place(int p) {
    return VEC == 1 ? p : HALF ? (p & 7) * 8 + (p >> 3) : (p & 3) * 16 + (p >> 2);
}

template <bool HALF, int VEC>
__global__ void __launch_bounds__(kRThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ float2 cs[kRTokens][kDim / 2];
    __shared__ int live[kRTokens];
    const int t0 = (int)blockIdx.x * a.tokens;
    const int nt = min(a.tokens, a.T - t0);
    const int rot = a.tab.rot_dim, H = a.Hq + a.Hkv;
    const int total = nt * H * a.per_head;
    const int turned = HALF ? rot / (2 * VEC) : (rot + VEC - 1) / VEC;  // units with turned pairs
    auto unit = [&](int u) {
        Unit r;
        // (exact: a block's units times the divisor stay below 2^32)
        const int hu = a.by_head ? (int)__umulhi((uint32_t)u, a.by_head) : u;
        r.lane = u - hu * a.per_head;
        r.tok = a.by_heads ? (int)__umulhi((uint32_t)hu, a.by_heads) : hu;
        const int h = hu - r.tok * H;
        const long long t = t0 + r.tok;
        const bool isq = h < a.Hq;
        const int hh = isq ? h : h - a.Hq;
        r.src = reinterpret_cast<const __half*>(isq ? a.q + t * a.qs : a.k + t * a.ks) + hh * kDim;
        r.dst = reinterpret_cast<__half*>(isq ? a.qo + t * a.qos : a.ko + t * a.kos) + hh * kDim;
        return r;
    };
    bool first = true;
    for (int base = 0; base < total; base += kRThreads * kRUnits) {
        uint4 x[kRUnits][2];
        Unit un[kRUnits];
#pragma unroll
        for (int i = 0; i < kRUnits; ++i) {
            const int u = base + i * kRThreads + (int)threadIdx.x;
            if (u < total) {
                un[i] = unit(u);
                const int l = un[i].lane;
                if (VEC == 8) {
                    const int at = HALF && l >= turned ? rot + 8 * (l - turned) : 8 * l;
                    x[i][0] = *reinterpret_cast<const uint4*>(un[i].src + at);
                    if (HALF && l < turned) x[i][1] = *reinterpret_cast<const uint4*>(un[i].src + at + rot / 2);
                } else {
                    const uint16_t* s = reinterpret_cast<const uint16_t*>(un[i].src);
                    x[i][0].x = s[l < turned ? l : rot + l - turned];
                    if (l < turned) x[i][1].x = s[l + rot / 2];
                }
            }
        }
        if (first) {
            for (int i = threadIdx.x; i < nt * (rot / 2); i += kRThreads) {
                const int t = i / (rot / 2), p = i - t * (rot / 2);
                const int pos = a.pos[t0 + t];
                const uint64_t f = (uint64_t)(int64_t)pos * a.tab.turns[p] + (1ull << 31);
                float s, c;
                sincospif((float)(int32_t)(f >> 32) * 4.656612873077393e-10f /* 2^-31 */, &s, &c);
                cs[t][place<HALF, VEC>(p)] = make_float2(c * a.m, s * a.ms);
                if (p == 0) live[t] = pos >= 0;
            }
            __syncthreads();
            first = false;
        }
#pragma unroll
        for (int i = 0; i < kRUnits; ++i) {
            const int u = base + i * kRThreads + (int)threadIdx.x;
            if (u >= total || !live[un[i].tok]) continue;
            const int l = un[i].lane;
            const float2* w = cs[un[i].tok];
            if (VEC == 8) {
                __half2* p = reinterpret_cast<__half2*>(&x[i][0]);
                __half2* p2 = reinterpret_cast<__half2*>(&x[i][1]);
                if (l >= turned) {
                    if (un[i].src == un[i].dst) continue;
                } else if (HALF) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x1 = __half22float2(p[j]), x2 = __half22float2(p2[j]);
                        const float2 w0 = w[place<HALF, VEC>(8 * l + 2 * j)], w1 = w[place<HALF, VEC>(8 * l + 2 * j + 1)];
                        p[j] = __floats2half2_rn(x1.x * w0.x - x2.x * w0.y, x1.y * w1.x - x2.y * w1.y);
                        p2[j] = __floats2half2_rn(x2.x * w0.x + x1.x * w0.y, x2.y * w1.x + x1.y * w1.y);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (8 * l + 2 * j < rot) {
                            const float2 v = __half22float2(p[j]), wj = w[place<HALF, VEC>(4 * l + j)];
                            p[j] = __floats2half2_rn(v.x * wj.x - v.y * wj.y, v.y * wj.x + v.x * wj.y);
                        }
                    }
                }
                const int at = HALF && l >= turned ? rot + 8 * (l - turned) : 8 * l;
                *reinterpret_cast<uint4*>(un[i].dst + at) = x[i][0];
                if (HALF && l < turned) *reinterpret_cast<uint4*>(un[i].dst + at + rot / 2) = x[i][1];
            } else {
                if (l < turned) {
                    const float x1 = __half2float(__ushort_as_half((unsigned short)x[i][0].x));
                    const float x2 = __half2float(__ushort_as_half((unsigned short)x[i][1].x));
                    const float2 wl = w[l];
                    un[i].dst[l] = __float2half_rn(x1 * wl.x - x2 * wl.y);
                    un[i].dst[l + rot / 2] = __float2half_rn(x2 * wl.x + x1 * wl.y);
                } else {
                    un[i].dst[rot + l - turned] = __ushort_as_half((unsigned short)x[i][0].x);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeCall& c, cudaStream_t stream) {
    RopeArgs a{};
    a.q = c.q;
    a.k = c.k;
    a.qo = c.q_out;
    a.ko = c.k_out;
    a.qs = c.q_stride;
    a.ks = c.k_stride;
    a.qos = c.q_out_stride;
    a.kos = c.k_out_stride;
    a.pos = c.positions;
    a.T = c.T;
    a.Hq = c.q ? c.Hq : 0;
    a.Hkv = c.k ? c.Hkv : 0;
    a.tab = *c.table;
    a.m = c.table->mscale;
    a.ms = c.transpose ? -a.m : a.m;
    const int rot = a.tab.rot_dim;
    const bool half = a.tab.layout == TQ_ROPE_HALF;
    const bool vec = !half || (rot / 2) % 8 == 0;
    a.per_head = !vec ? rot / 2 + (kDim - rot) : half ? rot / 16 + (kDim - rot) / 8 : kDim / 8;
    // as many tokens as fill the threads' units once, at least one
    const long long per_token = (long long)(a.Hq + a.Hkv) * a.per_head;
    long long n = (long long)kRThreads * kRUnits / per_token;
    a.tokens = (int)(n < 1 ? 1 : n > kRTokens ? kRTokens : n);
    // few tokens: one per block, so that they spread over the SMs
    if (a.T < 2 * 148 * a.tokens) a.tokens = 1;
    auto magic = [](int d) { return d == 1 ? 0u : (uint32_t)(((1ull << 32) + d - 1) / d); };
    a.by_head = magic(a.per_head);
    a.by_heads = magic(a.Hq + a.Hkv);
    const unsigned grid = (unsigned)((a.T + a.tokens - 1) / a.tokens);
    if (!half) rope_kernel<false, 8><<<grid, kRThreads, 0, stream>>>(a);
    else if (vec) rope_kernel<true, 8><<<grid, kRThreads, 0, stream>>>(a);
    else rope_kernel<true, 1><<<grid, kRThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace tq
