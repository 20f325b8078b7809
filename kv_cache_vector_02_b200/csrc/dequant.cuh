// Packed codes and signs to fp16, eight coordinates at a time, in registers.
//
// An fp16 level is two bytes; PRMT looks four of them up at once: its selector is four
// nibbles, which is what a word of nibble codes is.  Up to 8 levels one table holds the low
// bytes and one the high bytes; 16 levels use the codebook's symmetry, c[15 - j] = -c[j]:
// the table holds the 8 magnitudes and the sign comes from bit 3 of the code.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

#include "tq_internal.h"

namespace tq {

// One of SUB equal parts of a row of packed codes of W bits: 16 W / SUB bytes.
template <int W, int SUB>
struct PartRow {
    static constexpr int kWords = 4 * W / SUB;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const uint8_t* p) {
        if (kWords % 4 == 0) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 x = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = x.x;
                w[(4 * i + 1) % kWords] = x.y;
                w[(4 * i + 2) % kWords] = x.z;
                w[(4 * i + 3) % kWords] = x.w;
            }
        } else if (kWords == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x;
            w[1 % kWords] = x.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        }
    }
    // Exchanges piece c with piece c ^ (SUB == 4 ? 2 : 4) of the part.
    __device__ __forceinline__ void exchange(bool yes) {
        constexpr int kStep = SUB == 4 ? W / 2 : W;  // words from one to the other
        if (kStep == 0) {                            // (in one word)
            w[0] = yes ? __byte_perm(w[0], 0u, 0x1032) : w[0];
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                if (!(i & (kStep ? kStep : 1))) {
                    const uint32_t x = w[i], y = w[(i + kStep) % kWords];
                    w[i] = yes ? y : x;
                    w[(i + kStep) % kWords] = yes ? x : y;
                }
        }
    }
    // the codes of the part's coordinates 8c .. 8c + 7
    __device__ __forceinline__ uint32_t codes(int c) const { return w[8 * W * c / 32] >> (8 * W * c % 32); }
};

// Bytes of (x, y) picked by the low four nibbles of a selector whose nibbles are below 8.
// (__byte_perm masks the selector first; lookups are bound by the pipe that the mask takes.)
__device__ __forceinline__ uint32_t pick4(uint32_t x, uint32_t y, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(sel));
    return r;
}

// The halves of codes 2i, 2i + 1 (i = 0..3) from eight nibbles below 8.
__device__ __forceinline__ void lookup8(uint32_t nib, const LevelTable& t, uint32_t sign_a, uint32_t sign_b,
                                        uint32_t (&w)[4]) {
    const uint32_t up = nib >> 16;
    const uint32_t la = pick4(t.lo[0], t.lo[1], nib), ha = pick4(t.hi[0], t.hi[1], nib) | sign_a;
    const uint32_t lb = pick4(t.lo[0], t.lo[1], up), hb = pick4(t.hi[0], t.hi[1], up) | sign_b;
    w[0] = __byte_perm(la, ha, 0x5140);
    w[1] = __byte_perm(la, ha, 0x7362);
    w[2] = __byte_perm(lb, hb, 0x5140);
    w[3] = __byte_perm(lb, hb, 0x7362);
}

// +-m (m: fp16 magnitude in both halves, sign bits clear) from eight bits: a set bit is +.
__device__ __forceinline__ void signs8(uint32_t bits, uint32_t m2, uint32_t (&w)[4]) {
    const uint32_t nb = ~bits & 0xffu;
#pragma unroll
    for (int i = 0; i < 4; ++i)  // bit 2i to bit 15, bit 2i + 1 to bit 31
        w[i] = ((nb * ((1u << (15 - 2 * i)) + (1u << (30 - 2 * i)))) & 0x80008000u) | m2;
}

// Eight codes of container width W (4, 2 or 1 bits) in the low bits of `codes`, LEVELS levels.
template <int W, int LEVELS>
__device__ __forceinline__ void levels8(uint32_t codes, const LevelTable& t, uint32_t (&w)[4]) {
    if (W == 4 && LEVELS == 16) {
        const uint32_t neg = ~codes & 0x88888888u;                     // codes below 8
        const uint32_t mag = (codes ^ (neg - (neg >> 3))) & 0x77777777u;  // 7 - j for those, j - 8 for the rest
        const uint32_t even = (neg << 4) & 0x80808080u, odd = neg & 0x80808080u;
        lookup8(mag, t, __byte_perm(even, odd, 0x5140), __byte_perm(even, odd, 0x7362), w);
    } else if (W == 4) {
        lookup8(codes & 0x77777777u, t, 0u, 0u, w);
    } else if (W == 2) {
        uint32_t x = codes & 0xffffu;
        x = (x | (x << 8)) & 0x00ff00ffu;
        x = (x | (x << 4)) & 0x0f0f0f0fu;
        x = (x | (x << 2)) & 0x33333333u;
        lookup8(x, t, 0u, 0u, w);
    } else {
        const uint32_t m = (t.lo[0] & 0xffu) | ((t.hi[0] & 0xffu) << 8);
        signs8(codes, m | (m << 16), w);
    }
}

}  // namespace tq
