// qcache.cuh -- the 4-bit KV cache format shared by the kernels that write it, read
// it back and attend over it.
//
// The cache is one byte tensor [2, num_pages, G, page_size / 16, 10 d]: plane 0 is K
// (normed and rotated), plane 1 raw V.  Every 16 tokens of one KV head form a block of
// 10 d contiguous bytes:
//   codes   [d / 64][16][32 bytes]  one slab of 64 features per token as eight 32-bit
//           words; word w holds features 4w .. 4w+3 in its low half and 32+4w .. 32+4w+3
//           in its high half, the lowest feature in the lowest four bits
//   scales  [d / 32][16] bf16
//   centres [d / 32][16] bf16
// A feature stands for centre + scale * (code - 8): 4 + 2 * 16 / 32 = 5 bits a number.
// A group of 32 features with extremes lo, hi is written as
//   step = (hi - lo) / 15, scale = bf16(step), centre = bf16(lo + 8 step),
//   code - 8 = round-half-even((x - centre) * (1 / scale)) clamped to [-8, 7];
// a group that holds an infinity or a NaN gets scale = centre = NaN.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace gattn {

constexpr int kQcBlock = 16;  // tokens per block
constexpr int kQcGroup = 32;  // features per scale

__host__ __device__ __forceinline__ int64_t qc_block_bytes(int d) { return 10 * (int64_t)d; }

// Byte offset of a block inside one plane.
__device__ __forceinline__ int64_t qc_block_offset(int page, int g, int slot, int G, int page_size, int d) {
    return (((int64_t)page * G + g) * (page_size / kQcBlock) + slot / kQcBlock) * qc_block_bytes(d);
}

// max / min that return NaN when any operand is one
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
    float r;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Scale and centre of a group with extremes lo, hi (as bf16 bits and as the floats they
// stand for) and the reciprocal that turns a distance from the centre into codes.  The
// halves keep hi - lo finite over the whole fp32 range; a scale below the smallest
// normal float stores the group as its centre.
struct QcGroup {
    uint32_t scale_bits, centre_bits;
    float centre, inv;
};
__device__ __forceinline__ QcGroup qc_group(float lo, float hi) {
    const float step = __fmul_rn(__fsub_rn(__fmul_rn(0.5f, hi), __fmul_rn(0.5f, lo)), 2.0f / 15.0f);
    const bool finite = step < INFINITY;  // false for NaN too
    QcGroup q;
    const __nv_bfloat16 s = __float2bfloat16_rn(finite ? step : NAN);
    const __nv_bfloat16 c = __float2bfloat16_rn(finite ? fmaf(8.0f, step, lo) : NAN);
    q.scale_bits = __bfloat16_as_ushort(s);
    q.centre_bits = __bfloat16_as_ushort(c);
    q.centre = __bfloat162float(c);
    const float sf = __bfloat162float(s);
    q.inv = sf >= 1.17549435e-38f ? __frcp_rn(sf) : 0.f;
    return q;
}

// Eight codes of one group as nibbles, lowest feature first.  Adding 1.5 * 2^23 rounds
// the product to an integer half to even in one rounding and leaves code - 8 in the low
// mantissa bits (two's complement); flipping bit 3 of each nibble adds the 8.  CLAMP is
// needed only where a group's own extremes fall outside [-8, 7] (the codes are monotonic
// in x), which takes a centre so large that its rounding is half a step.
constexpr float kQcMagic = 12582912.f;
__device__ __forceinline__ float qc_round(float x, const QcGroup& q) {
    return fmaf(__fsub_rn(x, q.centre), q.inv, kQcMagic);
}
template <bool CLAMP>
__device__ __forceinline__ uint32_t qc_encode8(const float* x, const QcGroup& q) {
    uint32_t b[4];  // byte i: features 2i (low nibble) and 2i + 1; garbage above it
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float t0 = qc_round(x[2 * i], q), t1 = qc_round(x[2 * i + 1], q);
        if (CLAMP) {
            t0 = fminf(fmaxf(t0, kQcMagic - 8.f), kQcMagic + 7.f);
            t1 = fminf(fmaxf(t1, kQcMagic - 8.f), kQcMagic + 7.f);
        }
        const uint32_t hi = __float_as_uint(t1) << 4;
        b[i] = (__float_as_uint(t0) & 15u) | (hi & ~15u);
    }
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410) ^ 0x88888888u;
}

// sin and cos of the RoPE angle pos * f, f in 2^-64 turns: the product modulo one turn is
// exact in integers, so the angle of a far position is as good as that of a near one
// (a float product is off by half an ulp of the angle itself, 2e-3 rad at 32k).
__device__ __forceinline__ void rope_turn_sincos(uint64_t f, int pos, float* s, float* c) {
    const uint32_t t = (uint32_t)(((uint64_t)(int64_t)pos * f) >> 32);  // 2^-32 turns
    const uint32_t q = (t + 0x20000000u) >> 30;                         // nearest quarter turn
    float s0, c0;
    sincospif((float)(int32_t)(t - (q << 30)) * 4.656612873077393e-10f, &s0, &c0);  // 2^-31: half turns
    const bool odd = q & 1u;
    const float a = odd ? c0 : s0, b = odd ? s0 : c0;
    *s = (q & 2u) ? -a : a;
    *c = ((q + 1u) & 2u) ? -b : b;
}

// Sequence of packed token t: the largest b with cu[b] <= t (B >= 1, cu[0] = 0).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int t) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

}  // namespace gattn
