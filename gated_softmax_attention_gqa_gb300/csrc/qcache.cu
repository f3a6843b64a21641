// qcache.cu -- writing the 4-bit KV cache and reading it back (format: qcache.cuh).
//
// Both passes move every number once: the write reads 2 (bf16) or 4 (fp32) bytes a
// number and leaves 0.625, the read the reverse, so HBM bounds both as long as the
// arithmetic stays small: at 6.8 TB/s an SM has some 14 instruction slots for a written
// number.  So a lane takes 16 features (half a scale group) of one token and walks its KV
// heads: the token's sines and cosines (made once per warp, in shared memory) and their
// products with the norm weights are shared by all heads, and what a group costs
// (extremes, scale, reciprocal) is shared by 32 numbers and two lanes.  The chain of
// lookups that finds a token's row (sequence, length, page) is walked by one lane per
// token for all the tokens a warp will deal with.
#include "qcache.cuh"

namespace gattn {
namespace {

constexpr int kWarps = 4;

// A lane's sixteen features of a group of 32 are two runs of eight, 16 apart: its
// neighbour (lane ^ 1) has the runs between, so that each 16-byte load or store of the two
// fills whole 32-byte sectors.  (With sixteen in a row every sector passed twice, and the L1
// path, 79% busy, held the write at 104 us where it moves 333 MB.)
__device__ __forceinline__ int first_feature(int lane_of_token) { return 32 * (lane_of_token >> 1) + 8 * (lane_of_token & 1); }

// The sixteen, in pairs for the two-wide fp32 instructions: of each four neighbours
// (quad q) the first and third in p[2q], the second and fourth in p[2q + 1], so that a
// quad's codes combine pair by pair too.
struct Vec16 {
    float2 p[8];
};

// A row's sixteen features as loaded.
template <typename T>
struct Row16;
template <>
struct Row16<bf16> {
    uint4 v[2];
    __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0, 0, 0, 0); }
    // run c (0 or 1) from p
    __device__ __forceinline__ void load8(int c, const bf16* p) { v[c] = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(Vec16& x) const {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                x.p[4 * c + 2 * q] = make_float2(bf16_lo(w[2 * q]), bf16_lo(w[2 * q + 1]));
                x.p[4 * c + 2 * q + 1] = make_float2(bf16_hi(w[2 * q]), bf16_hi(w[2 * q + 1]));
            }
        }
    }
};
template <>
struct Row16<float> {
    float4 v[4];
    __device__ __forceinline__ void zero() { v[0] = v[1] = v[2] = v[3] = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load8(int c, const float* p) {
        v[2 * c] = reinterpret_cast<const float4*>(p)[0];
        v[2 * c + 1] = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void get(Vec16& x) const {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x.p[2 * q] = make_float2(v[q].x, v[q].z);
            x.p[2 * q + 1] = make_float2(v[q].y, v[q].w);
        }
    }
};

__device__ __forceinline__ float to_float(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The codes of eight features (four pairs), lowest feature in the lowest nibble.  CLAMP is
// needed only where a group's own extremes fall outside [-8, 7] (codes are monotonic in x),
// which takes a centre so large that its rounding is half a step.
template <bool CLAMP>
__device__ __forceinline__ uint32_t encode8(const float2* p, const QcGroup& g) {
    uint32_t h[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float2 u[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            u[i] = fma2(add2(p[2 * q + i], both(-g.centre)), both(g.inv), both(kQcMagic + 8.f));
            if (CLAMP)
                u[i] = make_float2(fminf(fmaxf(u[i].x, kQcMagic), kQcMagic + 15.f),
                                   fminf(fmaxf(u[i].y, kQcMagic), kQcMagic + 15.f));
        }
        // the bits of magic + code end in the code: even + 16 odd is a byte, garbage above it
        h[q] = __byte_perm(__float_as_uint(u[0].x) + 16u * __float_as_uint(u[1].x),
                           __float_as_uint(u[0].y) + 16u * __float_as_uint(u[1].y), 0x0040);
    }
    return __byte_perm(h[0], h[1], 0x5410);
}

// Place of packed token t: its position, and its row of the pool.  False for padding and
// for tokens that a length or a table entry keeps out of the cache (the caller reports).
struct Place {
    int pos, page, slot;
};
__device__ __forceinline__ Place place_of(const Place& at, int lane) {
    return Place{__shfl_sync(0xffffffffu, at.pos, lane), __shfl_sync(0xffffffffu, at.page, lane),
                 __shfl_sync(0xffffffffu, at.slot, lane)};
}
enum { kSkip = 0, kLive = 1, kBadLength = 2, kBadPage = 3 };

template <typename P>
__device__ __forceinline__ int find_page(const P& p, int b, Place& at) {
    const int k = page_of(at.pos, p.by_page);
    at.slot = at.pos - k * p.page_size;
    at.page = p.block_table[(int64_t)b * p.max_pages + k];
    return at.page >= 0 && at.page < p.num_pages ? kLive : kBadPage;
}

__device__ __forceinline__ int place_new(const QcacheWriteParams& p, int t, Place& at) {
    at.pos = 0;
    if (t >= p.T) return kSkip;
    int b = t, n = 1, j = 0;
    if (p.cu_seqlens) {
        b = find_sequence(p.cu_seqlens, p.B, t);
        const int c0 = p.cu_seqlens[b];
        n = p.cu_seqlens[b + 1] - c0;
        j = t - c0;
    }
    const int L = p.seqlens[b];
    if (j < 0 || j >= n) return kSkip;
    // a length of 0 marks an unused row of a batch that adds one token to each sequence
    if (!p.cu_seqlens && L == 0) return kSkip;
    if (L > p.max_pages * p.page_size || L < n) return kBadLength;
    at.pos = L - n + j;
    return find_page(p, b, at);
}

__device__ __forceinline__ int place_cached(const QcacheReadParams& p, int t, Place& at) {
    at.pos = 0;
    if (t >= p.T) return kSkip;
    int b = t, n = 1, j = 0;
    if (p.cu_seqlens) {
        b = find_sequence(p.cu_seqlens, p.B, t);
        const int c0 = p.cu_seqlens[b];
        n = p.cu_seqlens[b + 1] - c0;
        j = t - c0;
    }
    if (j < 0 || j >= n) return kSkip;
    const int64_t start = p.starts ? p.starts[b] : 0;
    if (start < 0 || start + n > (int64_t)p.max_pages * p.page_size) return kBadLength;
    at.pos = (int)start + j;
    return find_page(p, b, at);
}

__device__ __forceinline__ bool report(int what, unsigned int* status) {
    if (what == kBadLength) atomicOr(status, GATTN_DEVICE_BAD_SEQLEN);
    if (what == kBadPage) atomicOr(status, GATTN_DEVICE_BAD_PAGE);
    return what == kLive;
}

// Quantise this lane's features of K and of V (neighbouring lanes share a group of 32, four
// a slab) and store them at row `row` of `block` and of the V plane's block.  The two go
// together so that one's chain of extremes, scale and reciprocal fills the other's waits.
// All lanes of the warp.
__device__ __forceinline__ void encode_store(const Vec16 (&x)[2], uint8_t* block, int64_t plane, int row, int lc, int d,
                                             bool live) {
    float hi[2], lo[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        hi[n] = max_nan(x[n].p[0].x, x[n].p[0].y);
        lo[n] = min_nan(x[n].p[0].x, x[n].p[0].y);
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            hi[n] = max_nan(hi[n], x[n].p[i].x, x[n].p[i].y);
            lo[n] = min_nan(lo[n], x[n].p[i].x, x[n].p[i].y);
        }
    }
    QcGroup q[2];
    bool inside = true;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        hi[n] = max_nan(hi[n], __shfl_xor_sync(0xffffffffu, hi[n], 1));
        lo[n] = min_nan(lo[n], __shfl_xor_sync(0xffffffffu, lo[n], 1));
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        q[n] = qc_group(lo[n], hi[n]);
        const float2 ends = fma2(add2(make_float2(lo[n], hi[n]), both(-q[n].centre)), both(q[n].inv), both(kQcMagic + 8.f));
        inside = inside && ends.x >= kQcMagic && ends.y <= kQcMagic + 15.f;
    }
    uint32_t w[2][2];
    if (__all_sync(0xffffffffu, inside)) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            w[n][0] = encode8<false>(x[n].p, q[n]);
            w[n][1] = encode8<false>(x[n].p + 4, q[n]);
        }
    } else {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            w[n][0] = encode8<true>(x[n].p, q[n]);
            w[n][1] = encode8<true>(x[n].p + 4, q[n]);
        }
    }
    // lanes j and j ^ 2 of a slab hold the same features of its two groups, which meet in the
    // words of both runs; the first group's lane stores the words of run 0, the other run 1's
    const int odd = lc & 1, upper = (lc >> 1) & 1;
    const int at = (lc >> 2) * 512 + row * 32 + 16 * upper + 8 * odd;
    const int par = 8 * d + (odd * (d / 2) + (lc >> 1) * 16 + row) * 2;  // the group's lanes: its scale, its centre
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const uint32_t o = __shfl_xor_sync(0xffffffffu, upper ? w[n][0] : w[n][1], 2);
        const uint32_t a = upper ? o : w[n][0], b = upper ? w[n][1] : o;
        if (live) {
            uint8_t* to = block + n * plane;
            *reinterpret_cast<uint2*>(to + at) = make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
            *reinterpret_cast<uint16_t*>(to + par) = (uint16_t)(odd ? q[n].bits >> 16 : q[n].bits);
        }
    }
}

// A token is spread over D / 16 lanes, 32 / (D / 16) tokens to a pass.  `TEAM` of the block's
// warps (one or all) take the same tokens, `passes` passes of them, and every TEAM-th of the
// heads [blockIdx.y heads, ...); they make the sines and cosines together.
template <int D, typename T, int TEAM>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 2 ? 6 : 4)
    qcache_write_kernel(const __grid_constant__ QcacheWriteParams p, int passes, int heads) {
    constexpr int LPR = D / 16, TPW = 32 / LPR;
    // sines and cosines of a pass, {sin, cos} of frequencies 2u, 2u + 1 in element
    // [token][u % 4][u / 4] (lanes of neighbouring features read neighbouring elements), and one
    // element that turns nothing
    __shared__ float4 tables[kWarps / TEAM][TPW * D / 4 + 1];
    // norm weights, and the rotation partners' with the rotation's sign, in Vec16 order
    __shared__ float4 weights[2][4][LPR];
    // their products with cosine and sine for the pass's tokens: each lane's own 32 floats,
    // here rather than in registers, because the kernel lives on warps per SM (with 16 of them
    // it moved 2.9 TB/s, whatever the instructions per warp)
    __shared__ float4 factors[kWarps][8][32];
    pdl_launch_dependents();  // a decode step may set itself up; it waits for this grid before it reads the cache
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mate_id = warp % TEAM, tl = lane / LPR, lc = lane % LPR;
    const int t0 = (blockIdx.x * (kWarps / TEAM) + warp / TEAM) * TPW * passes;
    const int e0 = first_feature(lc), g0 = blockIdx.y * heads + mate_id, g1 = min(p.G, (int)(blockIdx.y + 1) * heads);
    const int half = p.rd >> 1;
    // distance of the rotation partner, eight features at a time (half is a multiple of 8);
    // 0: features past rotary_dim, which are not turned
    auto partner = [&](int e) { return e < half ? half : e < p.rd ? -half : 0; };
    const int mate[2] = {partner(e0), partner(e0 + 16)};
    Place mine;  // of token t0 + lane
    const bool ok = report(lane < passes * TPW ? place_new(p, t0 + lane, mine) : kSkip, p.status);
    if (!ok) mine = Place{0, -1, 0};

    for (int e = threadIdx.x; e < D; e += 32 * kWarps) {
        // run, quad and place of feature e in its lane's Vec16
        const int m = partner(e), q = 2 * ((e >> 4) & 1) + ((e >> 2) & 1), of = 2 * (e >> 5) + ((e >> 3) & 1);
        const int at = (q * LPR + of) * 4 + (e & 1) * 2 + ((e >> 1) & 1);
        const T* w = static_cast<const T*>(p.knorm_w);
        reinterpret_cast<float*>(weights[0])[at] = to_float(w[e]);
        reinterpret_cast<float*>(weights[1])[at] = m > 0 ? -to_float(w[e + m]) : to_float(w[e + m]);
    }
    float4* table = tables[warp / TEAM];
    if (lane == 0) table[TPW * D / 4] = make_float4(0.f, 1.f, 0.f, 1.f);
    const float4* sc[2];
    int step[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int e = e0 + 16 * c;
        sc[c] = table + (mate[c] ? tl * (half / 2) + (e < half ? e : e - half) / 8 : TPW * D / 4);
        step[c] = mate[c] ? half / 8 : 0;
    }
    const int64_t head = (int64_t)(p.page_size / kQcBlock) * qc_block_bytes(D), plane = (int64_t)p.num_pages * p.G * head;
    __syncthreads();

    for (int pass = 0; pass < passes; ++pass) {
        if (TEAM == 1 && t0 + pass * TPW >= p.T) break;
        for (int k = mate_id; k < TPW; k += TEAM) {
            const int pos = __shfl_sync(0xffffffffu, mine.pos, pass * TPW + k);
            for (int i = lane; i < half; i += 32) {
                float s, c;
                rope_turn_sincos(p.turns[i], pos, &s, &c);
                reinterpret_cast<float2*>(table + k * (half / 2) + ((i >> 1) & 3) * (half / 8) + (i >> 3))[i & 1] =
                    make_float2(s, c);
            }
        }
        if (TEAM > 1) __syncthreads(); else __syncwarp();
        // K' = (x wc + partner ws) / rms
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 w = weights[0][q][lc], m = weights[1][q][lc];
            const float4 a = sc[q >> 1][(2 * q & 3) * step[q >> 1]], b = sc[q >> 1][((2 * q & 3) + 1) * step[q >> 1]];
            const float2 c0 = mul2(make_float2(w.x, w.y), make_float2(a.y, b.y));
            const float2 c1 = mul2(make_float2(w.z, w.w), make_float2(a.w, b.w));
            const float2 s0 = mul2(make_float2(m.x, m.y), make_float2(a.x, b.x));
            const float2 s1 = mul2(make_float2(m.z, m.w), make_float2(a.z, b.z));
            factors[warp][q][lane] = make_float4(c0.x, c0.y, c1.x, c1.y);
            factors[warp][4 + q][lane] = make_float4(s0.x, s0.y, s1.x, s1.y);
        }
        if (TEAM > 1) __syncthreads(); else __syncwarp();  // the next pass overwrites the table
        const Place at = place_of(mine, pass * TPW + tl);
        const bool live = at.page >= 0;
        uint8_t* block = p.cache + (live ? (at.page * (int64_t)p.G + g0) * head + (at.slot / kQcBlock) * qc_block_bytes(D) : 0);
        const int row = at.slot % kQcBlock;
        const int64_t t = min(t0 + pass * TPW + tl, p.T - 1);
        const T* kp = static_cast<const T*>(p.k) + t * p.k_tok_stride + g0 * p.k_head_stride + e0;
        const T* vp = static_cast<const T*>(p.v) + t * p.v_tok_stride + g0 * p.v_head_stride + e0;
        for (int g = g0; g < g1; g += TEAM) {
            Row16<T> kr, ko, vr;
            ko.zero();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                kr.load8(c, kp + 16 * c);
                if (mate[c]) ko.load8(c, kp + 16 * c + mate[c]);
                vr.load8(c, vp + 16 * c);
            }
            kp += TEAM * p.k_head_stride;
            vp += TEAM * p.v_head_stride;
            Vec16 x[2], o;
            kr.get(x[0]);
            float2 s2 = mul2(x[0].p[0], x[0].p[0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) s2 = fma2(x[0].p[i], x[0].p[i], s2);
            float ss = s2.x + s2.y;
#pragma unroll
            for (int s = LPR / 2; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
            const float2 rinv = both(inv_sqrt(ss / (float)D + p.eps));
            ko.get(o);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 wc = factors[warp][q][lane], ws = factors[warp][4 + q][lane];
                x[0].p[2 * q] = mul2(fma2(x[0].p[2 * q], make_float2(wc.x, wc.y), mul2(o.p[2 * q], make_float2(ws.x, ws.y))), rinv);
                x[0].p[2 * q + 1] =
                    mul2(fma2(x[0].p[2 * q + 1], make_float2(wc.z, wc.w), mul2(o.p[2 * q + 1], make_float2(ws.z, ws.w))), rinv);
            }
            vr.get(x[1]);
            encode_store(x, block, plane, row, lc, D, live);
            block += TEAM * head;
        }
    }
}

// Eight stored features (their nibbles lowest first) as bf16 or fp32.  bf16: a nibble or-ed
// into 128's mantissa reads as 128 + code; the difference to 136 is exact and the fused
// multiply-add rounds centre + scale (code - 8) once.
__device__ __forceinline__ void decode8(uint32_t n, uint32_t s2, uint32_t c2, bf16* out) {
    uint32_t r[4];  // features i and i + 4
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = ((n >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
        uint32_t u;
        asm("sub.bf16x2 %0, %1, %2;" : "=r"(u) : "r"(v), "r"(0x43084308u));
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r[i]) : "r"(u), "r"(s2), "r"(c2));
    }
    *reinterpret_cast<uint4*>(out) = make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                                                __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
}
__device__ __forceinline__ void decode8(uint32_t n, uint32_t s2, uint32_t c2, float* out) {
    const float s = bf16_lo(s2), c = bf16_lo(c2);
    float x[8];
    // 2^23 + code as a float; the difference to 2^23 + 8 is exact
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = fmaf(s, __uint_as_float(((n >> (4 * k)) & 15u) | 0x4B000000u) - 8388616.f, c);
    reinterpret_cast<float4*>(out)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(out)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// The same layout of work: a lane reads back 16 features of one token, head after head.
template <int D, typename T>
__global__ void __launch_bounds__(32 * kWarps)
    qcache_read_kernel(const __grid_constant__ QcacheReadParams p, int passes, int heads, int team) {
    constexpr int LPR = D / 16, TPW = 32 / LPR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = (blockIdx.x * (kWarps / team) + warp / team) * TPW * passes;
    const int lc = lane % LPR, e0 = first_feature(lc), g0 = blockIdx.y * heads + warp % team, g1 = min(p.G, (int)(blockIdx.y + 1) * heads);
    if (t0 >= p.T || g0 >= g1) return;
    Place mine;  // of token t0 + lane
    const bool ok = report(lane < passes * TPW ? place_cached(p, t0 + lane, mine) : kSkip, p.status);
    if (!ok) mine = Place{0, -1, 0};
    const int64_t head = (int64_t)(p.page_size / kQcBlock) * qc_block_bytes(D), plane = (int64_t)p.num_pages * p.G * head;
    const uint32_t sel = (lc & 2) ? 0x7632 : 0x5410;  // the group's half of a word
    for (int pass = 0; pass < passes; ++pass) {
        const Place at = place_of(mine, pass * TPW + lane / LPR);
        if (at.page < 0) continue;  // no lane of this token goes on; the shuffles above are whole again next time
        const int64_t t = t0 + pass * TPW + lane / LPR;
        const int row = at.slot % kQcBlock;
        const int codes = (lc >> 2) * 512 + row * 32 + 8 * (lc & 1);
        const uint8_t* src = p.cache + (at.page * (int64_t)p.G + g0) * head + (at.slot / kQcBlock) * qc_block_bytes(D) + codes;
        const int par = 8 * D + ((lc >> 1) * 16 + row) * 2 - codes;
        T* kout = static_cast<T*>(p.k) + (t * p.G + g0) * D + e0;
        T* vout = static_cast<T*>(p.v) + (t * p.G + g0) * D + e0;
#pragma unroll 4
        for (int g = g0; g < g1; g += team) {
            uint2 w[2][2];
            uint32_t s[2], c[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // K and V
                w[i][0] = *reinterpret_cast<const uint2*>(src + i * plane);
                w[i][1] = *reinterpret_cast<const uint2*>(src + i * plane + 16);
                s[i] = *reinterpret_cast<const uint16_t*>(src + i * plane + par);
                c[i] = *reinterpret_cast<const uint16_t*>(src + i * plane + par + D);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                T* out = i ? vout : kout;
                const uint32_t s2 = s[i] * 0x10001u, c2 = c[i] * 0x10001u;
                decode8(__byte_perm(w[i][0].x, w[i][0].y, sel), s2, c2, out);
                decode8(__byte_perm(w[i][1].x, w[i][1].y, sel), s2, c2, out + 16);
            }
            src += team * head;
            kout += team * D;
            vout += team * D;
        }
    }
}

// How a call is cut: passes a warp takes (their lookups go together), KV heads of a block,
// warps that share a token's heads.  A call too small to fill the device with one warp for
// all heads of its tokens takes one pass and spreads the heads, over a block's warps first.
// (Passes of a long call: the write of 131072 tokens, 2 x 256, takes 106 us with two and 101
// with four; the read of 211k tokens, 4 x 128, 107 with two and 119 with four.)
struct Cut {
    int passes, heads, team;
    dim3 grid;
};
template <int D>
Cut cut_of(int T, int G, int passes) {
    constexpr int TPW = 32 / (D / 16);
    const int64_t want = 8 * (int64_t)device_sm_count(), groups = ((int64_t)T + TPW - 1) / TPW;
    Cut c{passes, G, 1, dim3()};
    if (groups < passes * want) c.passes = 1;
    if (G > 1 && groups < want) c.team = kWarps;
    while (c.heads > c.team && groups * c.team * ((G + c.heads - 1) / c.heads) < want) c.heads = (c.heads + 1) / 2;
    const int tokens = kWarps / c.team * TPW * c.passes;
    c.grid = dim3((unsigned)((T + tokens - 1) / tokens), (unsigned)((G + c.heads - 1) / c.heads));
    return c;
}

template <int D>
cudaError_t write_d(const QcacheWriteParams& p, bool fp32, cudaStream_t stream) {
    const Cut c = cut_of<D>(p.T, p.G, 4);
    auto kernel = fp32 ? (c.team > 1 ? qcache_write_kernel<D, float, kWarps> : qcache_write_kernel<D, float, 1>)
                       : (c.team > 1 ? qcache_write_kernel<D, bf16, kWarps> : qcache_write_kernel<D, bf16, 1>);
    kernel<<<c.grid, 32 * kWarps, 0, stream>>>(p, c.passes, c.heads);
    return cudaGetLastError();
}

template <int D>
cudaError_t read_d(const QcacheReadParams& p, bool fp32, cudaStream_t stream) {
    const Cut c = cut_of<D>(p.T, p.G, 2);
    auto kernel = fp32 ? qcache_read_kernel<D, float> : qcache_read_kernel<D, bf16>;
    kernel<<<c.grid, 32 * kWarps, 0, stream>>>(p, c.passes, c.heads, c.team);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qcache_write(const QcacheWriteParams& p, bool fp32, cudaStream_t stream) {
    switch (p.d) {
        case 64: return write_d<64>(p, fp32, stream);
        case 128: return write_d<128>(p, fp32, stream);
        case 256: return write_d<256>(p, fp32, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_qcache_read(const QcacheReadParams& p, bool fp32, cudaStream_t stream) {
    switch (p.d) {
        case 64: return read_d<64>(p, fp32, stream);
        case 128: return read_d<128>(p, fp32, stream);
        case 256: return read_d<256>(p, fp32, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gattn
