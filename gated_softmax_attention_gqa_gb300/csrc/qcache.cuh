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
#include "qcache_internal.h"

namespace gattn {

constexpr int kQcBlock = 16;  // tokens per block
constexpr int kQcGroup = 32;  // features per scale

__host__ __device__ __forceinline__ int64_t qc_block_bytes(int d) { return 10 * (int64_t)d; }

__device__ __forceinline__ int page_of(int x, const PageDiv& d) {
    return d.mul ? (int)(__umulhi((uint32_t)x, d.mul) >> d.shift) : x;
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

// Scale and centre of a group with extremes lo, hi (scale in the low half of `bits`) and
// the reciprocal that turns a distance from the centre into codes.  The halves keep
// hi - lo finite over the whole fp32 range; a scale below the smallest normal float stores
// the group as its centre.  The reciprocal is one Newton step r (2 - s r) on the hardware
// approximation, which for the 8-bit significands of bf16 is 1 / s rounded to nearest (a
// test puts numbers half way between codes for every significand and 201 exponents).
struct QcGroup {
    uint32_t bits;
    float centre, inv;
};
__device__ __forceinline__ QcGroup qc_group(float lo, float hi) {
    const float step = __fmul_rn(__fsub_rn(__fmul_rn(0.5f, hi), __fmul_rn(0.5f, lo)), 2.0f / 15.0f);
    QcGroup q;
    q.bits = step < INFINITY ? pack_bf16x2(step, fmaf(8.0f, step, lo)) : 0x7FC07FC0u;  // NaN, NaN
    q.centre = bf16_hi(q.bits);
    const float s = bf16_lo(q.bits), r = rcp_approx(s);
    q.inv = s >= 1.17549435e-38f ? fmaf(r, fmaf(-s, r, 1.f), r) : 0.f;
    return q;
}

// Adding 1.5 * 2^23 + 8 to (x - centre) / scale rounds it to an integer half to even, in the
// one rounding of a fused multiply-add, and leaves the code in the low mantissa bits.
constexpr float kQcMagic = 12582912.f;

// sin and cos of the RoPE angle pos * f, f in 2^-64 turns: the product modulo one turn is
// exact in integers, so the angle of a far position is as good as that of a near one
// (a float product is off by half an ulp of the angle itself, 2e-3 rad at 32k).  The rest
// of the nearest quarter turn, at most pi/4, goes through the Taylor series of sine and
// cosine (first terms left out: a^11/11! < 2e-9, a^12/12! < 2e-10).
__device__ __forceinline__ void rope_turn_sincos(uint64_t f, int pos, float* s, float* c) {
    const uint32_t t = __umulhi((uint32_t)pos, (uint32_t)f) + (uint32_t)pos * (uint32_t)(f >> 32);  // 2^-32 turns
    const uint32_t q = (t + 0x20000000u) >> 30;                         // nearest quarter turn
    const float a = (float)(int32_t)(t - (q << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float a2 = a * a;
    const float ps = fmaf(a2, fmaf(a2, fmaf(a2, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f);
    const float pc = fmaf(a2, fmaf(a2, fmaf(a2, fmaf(a2, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f);
    const float s0 = fmaf(a * a2, ps, a), c0 = fmaf(a2, pc, 1.f);
    const float x = q & 1u ? c0 : s0, y = q & 1u ? s0 : c0;
    *s = __uint_as_float(__float_as_uint(x) ^ ((q & 2u) << 30));
    *c = __uint_as_float(__float_as_uint(y) ^ (((q + 1u) & 2u) << 30));
}

// 1 / sqrt(x): the hardware approximation and one Newton step (0 for an infinite x).
__device__ __forceinline__ float inv_sqrt(float x) {
    const float r = rsqrtf(x);
    return x < INFINITY ? fmaf(0.5f * r, fmaf(-x * r, r, 1.f), r) : r;
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

// Launches a kernel that may become resident while the one ahead of it in the stream still
// runs, and that waits for it (griddepcontrol) before it touches what that one may write.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t shared, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace gattn
