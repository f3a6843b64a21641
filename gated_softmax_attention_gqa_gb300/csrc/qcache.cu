// qcache.cu -- writing the 4-bit KV cache and reading it back (format: qcache.cuh).
//
// Both passes move every number once: the write reads 2 (bf16) or 4 (fp32) bytes a
// number and leaves 0.625, the read the reverse, so HBM bounds both as long as the
// arithmetic stays small: at 6.8 TB/s an SM has some 14 instruction slots for a written
// number.  So a lane takes 16 features (half a scale group) of one token and walks its KV
// heads: the token's sines and cosines and their products with the norm weights (made once
// per warp, in shared memory) are shared by all heads, and what a group costs
// (extremes, scale, reciprocal) is shared by 32 numbers and two lanes.  The chain of
// lookups that finds a token's row (sequence, length, page) is walked by one lane per
// token for all the tokens a warp will deal with.
//
// Measured, 131072 tokens of 2 heads of 256 in bf16 (353 MB each way): the read 54 us,
// 6.5 TB/s, which is HBM; the write 76 us, 4.6 TB/s, held by instruction issue (two thirds
// of the slots are taken).
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

// Sixteen-byte chunk m of a warp's staged rows lies at chunk m ^ swizzle(m), so that the
// eight lanes of a 128-byte access, which skip every other 16 features, meet all banks.
template <typename T>
__device__ __forceinline__ int staged(int m) {
    return sizeof(T) == 2 ? m ^ ((m >> 2) & 2) : m ^ (((m >> 3) & 1) | ((m >> 2) & 4));
}

// A lane's run c (0 or 1) of eight features, from chunk m of the staged rows on.
__device__ __forceinline__ void load8(Vec16& x, int c, const uint4* rows, int m, bf16) {
    const uint4 v = rows[staged<bf16>(m)];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        x.p[4 * c + 2 * q] = make_float2(bf16_lo(w[2 * q]), bf16_lo(w[2 * q + 1]));
        x.p[4 * c + 2 * q + 1] = make_float2(bf16_hi(w[2 * q]), bf16_hi(w[2 * q + 1]));
    }
}
__device__ __forceinline__ void load8(Vec16& x, int c, const uint4* rows, int m, float) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const float4 v = reinterpret_cast<const float4*>(rows)[staged<float>(m + q)];
        x.p[4 * c + 2 * q] = make_float2(v.x, v.z);
        x.p[4 * c + 2 * q + 1] = make_float2(v.y, v.w);
    }
}

__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float to_float(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The codes of eight features (four pairs), lowest feature in the lowest nibble.  CLAMP is
// needed only where a group's own extremes fall outside [-8, 7], which takes a centre so
// large that its rounding, 2^-8 of it, nears half a step: with |centre| <= 112 scales it is
// 0.44 steps, and the scale's rounding over eight steps 0.03.
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
// K is x[0] * rinv: its group's centre and reciprocal scale are taken to x[0]'s measure
// (rms = 1 / rinv) instead of sixteen numbers to the group's.  All lanes of the warp.
__device__ __forceinline__ void encode_store(const Vec16 (&x)[2], float rinv, float rms, uint8_t* block, int64_t plane,
                                             int row, int lc, int d, bool live) {
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
        q[n] = n ? qc_group(lo[n], hi[n]) : qc_group(lo[n] * rinv, hi[n] * rinv);
        if (n == 0) {
            q[n].centre *= rms;
            q[n].inv *= rinv;
        }
        // false, too, where rinv took the reciprocal past fp32's range (steps below 3e-39 rinv)
        inside = inside && fabsf(q[n].centre) * q[n].inv <= 112.f;
    }
    uint32_t w[2][2];
    if (__all_sync(0xffffffffu, inside)) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            w[n][0] = encode8<false>(x[n].p, q[n]);
            w[n][1] = encode8<false>(x[n].p + 4, q[n]);
        }
    } else {
        Vec16 k = x[0];
        if (!(q[0].inv < INFINITY)) {  // K in its group's measure
            q[0] = qc_group(lo[0] * rinv, hi[0] * rinv);
#pragma unroll
            for (int i = 0; i < 8; ++i) k.p[i] = mul2(k.p[i], both(rinv));
        }
        w[0][0] = encode8<true>(k.p, q[0]);
        w[0][1] = encode8<true>(k.p + 4, q[0]);
        w[1][0] = encode8<true>(x[1].p, q[1]);
        w[1][1] = encode8<true>(x[1].p + 4, q[1]);
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

// Shared memory of a write block.
template <typename T, int TEAM>
struct WriteShared {
    static constexpr int kStages = 2, kChunks = 512 * sizeof(T) / 16;  // a warp's pass: 512 features each of K and V
    // What K' = (x wc + partner ws) / rms takes, products of the norm weights with cosine
    // and sine (the rotation's sign in ws): quads of wc in rows 0-3, of ws in rows 4-7, a
    // float4 a lane in Vec16 order.  The spare two spread a token's features, 32 at a time,
    // over the banks.  In shared memory rather than in 32 registers, which are worth a CTA
    // per SM (131072 tokens, 2 x 256: five hold 87 us, four 92; six spill, 94).
    float4 factors[kWarps / TEAM][8][34];
    float4 plain[8][34];  // the same of features that are not turned (the norm weights, and zeros), a token's lanes
    uint4 rows[kWarps][kStages][2][kChunks];  // K and V as copied, ahead of their use
};

// A token is spread over D / 16 lanes, 32 / (D / 16) tokens to a pass.  `TEAM` of the block's
// warps take the same tokens, `passes` passes of them (one, if they are several), and every TEAM-th of the
// heads [blockIdx.y heads, ...); they make the factors together.  A warp's rows are copied to
// shared memory two heads ahead (with loads straight to registers the warps waited for HBM a
// third of the time: 101 us for 131072 tokens of 2 x 256, 87 with the copies).
template <int D, typename T, int TEAM>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 2 ? 5 : 4)
    qcache_write_kernel(const __grid_constant__ QcacheWriteParams p, int passes, int heads) {
    using S = WriteShared<T, TEAM>;
    constexpr int LPR = D / 16, TPW = 32 / LPR, EPC = 16 / sizeof(T), CPR = D / EPC, CPL = S::kChunks / 32;
    extern __shared__ __align__(16) uint8_t smem[];
    S& sh = *reinterpret_cast<S*>(smem);
    pdl_wait_prerequisites();  // the kernel ahead may not have finished when this one is placed
    // a decode step sets itself up meanwhile, and waits before it reads the cache
    if (p.before_decode) pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mate_id = warp % TEAM, tl = lane / LPR, lc = lane % LPR;
    const int t0 = (blockIdx.x * (kWarps / TEAM) + warp / TEAM) * TPW * passes;
    const int e0 = first_feature(lc), g0 = blockIdx.y * heads + mate_id, g1 = min(p.G, (int)(blockIdx.y + 1) * heads);
    const int mine_heads = g0 < g1 ? (g1 - g0 + TEAM - 1) / TEAM : 0;
    if (TEAM == 1) passes = min(passes, (p.T - t0 + TPW - 1) / TPW);

    // ---- the copies: lane l takes chunks l, l + 32, ... of a pass's tokens, head after head
    const int my_token = lane / CPR;
    const T* kf = static_cast<const T*>(p.k) + (int64_t)(t0 + my_token) * p.k_tok_stride + g0 * p.k_head_stride + lane % CPR * EPC;
    const T* vf = static_cast<const T*>(p.v) + (int64_t)(t0 + my_token) * p.v_tok_stride + g0 * p.v_head_stride + lane % CPR * EPC;
    int left = passes * mine_heads, head_left = mine_heads, token = t0 + my_token;
    auto fetch = [&](int stage) {
        if (left > 0) {
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                // chunk 32 i + lane: CPR chunks a token
                constexpr bool kWide = CPR > 32;
                const int dt = kWide ? i / (CPR / 32) : i * (32 / CPR), de = kWide ? i % (CPR / 32) * 32 * EPC : 0;
                const int at = staged<T>(32 * i + lane);
                if (token + dt < p.T) {  // a token past the end keeps what the buffer holds; it is not stored
                    copy16(&sh.rows[warp][stage][0][at], kf + dt * p.k_tok_stride + de);
                    copy16(&sh.rows[warp][stage][1][at], vf + dt * p.v_tok_stride + de);
                }
            }
            --left;
            kf += TEAM * p.k_head_stride;
            vf += TEAM * p.v_head_stride;
            if (--head_left == 0) {
                head_left = mine_heads;
                token += TPW;
                kf += TPW * p.k_tok_stride - mine_heads * (TEAM * p.k_head_stride);
                vf += TPW * p.v_tok_stride - mine_heads * (TEAM * p.v_head_stride);
            }
        }
        copies_commit();
    };
    fetch(0);
    fetch(1);

    const int half = p.rd >> 1;
    // distance of the rotation partner, eight features at a time (half is a multiple of 8);
    // 0: features past rotary_dim, which are not turned
    auto partner = [&](int e) { return e < half ? half : e < p.rd ? -half : 0; };
    // float of feature e of token k within rows q of `factors` or `plain` (of a token's lanes)
    auto place = [&](int e, int k) {
        const int q = 2 * ((e >> 4) & 1) + ((e >> 2) & 1), of = 2 * (e >> 5) + ((e >> 3) & 1);
        return (q * 34 + k * LPR + of) * 4 + (e & 1) * 2 + ((e >> 1) & 1);
    };
    for (int i = threadIdx.x; i < 4 * 34; i += 32 * kWarps) sh.plain[4][i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int e = threadIdx.x; e < D; e += 32 * kWarps) {
        const float w = to_float(static_cast<const T*>(p.knorm_w)[e]);
        reinterpret_cast<float*>(sh.plain)[place(e, 0)] = w;
    }
    Place mine;  // of token t0 + lane: passes * TPW <= 32 (cut_of)
    const bool ok = report(lane < passes * TPW ? place_new(p, t0 + lane, mine) : kSkip, p.status);
    if (!ok) mine = Place{0, -1, 0};

    float* const factors = reinterpret_cast<float*>(sh.factors[warp / TEAM]);
    constexpr int kSines = 4 * 34 * 4;  // floats from a feature's wc to its ws
    const int mate[2] = {partner(e0), partner(e0 + 16)};
    const float4* wc[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) wc[c] = mate[c] ? &sh.factors[warp / TEAM][2 * c][lane] : &sh.plain[2 * c][lc];
    const int64_t head = (int64_t)(p.page_size / kQcBlock) * qc_block_bytes(D), plane = (int64_t)p.num_pages * p.G * head;
    const int chunk0 = tl * CPR + e0 / EPC;
    const int chunk_o[2] = {chunk0 + mate[0] / EPC, chunk0 + (16 + mate[1]) / EPC};  // the partners'
    __syncthreads();

    // a lane's frequency, the places of its two features' factors, and their norm weights
    // (kept from pass to pass where one round covers them all, rotary_dim <= 64: 131072 tokens
    // of 2 x 256 take 76 us rather than 81)
    uint64_t turn = 0;
    float *lo = factors, *hi = factors, wl = 0.f, wh = 0.f;
    auto aim = [&](int i0) {
        const int i = min(i0 + lane, half - 1);
        turn = p.turns[i];
        wl = reinterpret_cast<const float*>(sh.plain)[place(i, 0)];
        wh = reinterpret_cast<const float*>(sh.plain)[place(i + half, 0)];
        lo = factors + place(i, 0);
        hi = factors + place(i + half, 0);
    };
    int stage = 0;
    for (int pass = 0; pass < passes; ++pass) {
        for (int i0 = 0; i0 < half; i0 += 32) {
            if (i0 + pass == 0 || half > 32) aim(i0);
            for (int k = mate_id; k < TPW; k += TEAM) {
                const int pos = __shfl_sync(0xffffffffu, mine.pos, pass * TPW + k);
                float s, c;
                rope_turn_sincos(turn, pos, &s, &c);
                if (i0 + lane < half) {
                    lo[k * LPR * 4] = wl * c;
                    hi[k * LPR * 4] = wh * c;
                    lo[k * LPR * 4 + kSines] = -wh * s;
                    hi[k * LPR * 4 + kSines] = wl * s;
                }
            }
        }
        if (TEAM > 1) __syncthreads(); else __syncwarp();
        const Place at = place_of(mine, pass * TPW + tl);
        const bool live = at.page >= 0;
        uint8_t* block = p.cache + (live ? (at.page * (int64_t)p.G + g0) * head + (at.slot / kQcBlock) * qc_block_bytes(D) : 0);
        const int row = at.slot % kQcBlock;
        for (int g = g0; g < g1; g += TEAM) {
            copies_wait<S::kStages - 1>();
            __syncwarp();
            const uint4* kr = sh.rows[warp][stage][0];
            const uint4* vr = sh.rows[warp][stage][1];
            Vec16 x[2], o;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                load8(x[0], c, kr, chunk0 + c * 16 / EPC, T());
                load8(o, c, kr, chunk_o[c], T());
            }
            float2 s2 = mul2(x[0].p[0], x[0].p[0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) s2 = fma2(x[0].p[i], x[0].p[i], s2);
            float ss = s2.x + s2.y;
#pragma unroll
            for (int s = LPR / 2; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
            const float ms = ss / (float)D + p.eps, rinv = inv_sqrt(ms);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 w = wc[q >> 1][(q & 1) * 34], m = wc[q >> 1][(q & 1) * 34 + kSines / 4];
                x[0].p[2 * q] = fma2(x[0].p[2 * q], make_float2(w.x, w.y), mul2(o.p[2 * q], make_float2(m.x, m.y)));
                x[0].p[2 * q + 1] = fma2(x[0].p[2 * q + 1], make_float2(w.z, w.w), mul2(o.p[2 * q + 1], make_float2(m.z, m.w)));
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) load8(x[1], c, vr, chunk0 + c * 16 / EPC, T());
            __syncwarp();
            fetch(stage);
            stage ^= 1;
            encode_store(x, rinv, ms * rinv, block, plane, row, lc, D, live);
            block += TEAM * head;
        }
    }
    copies_wait<0>();
}

// Eight stored features (their nibbles lowest first) as bf16, or four and four, eight apart, as fp32.  bf16: a nibble or-ed
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
    reinterpret_cast<float4*>(out)[2] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ uint2 load_run(const uint8_t* p, bf16) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ uint2 load_run(const uint8_t* p, float) {
    return make_uint2(reinterpret_cast<const uint32_t*>(p)[0], reinterpret_cast<const uint32_t*>(p)[2]);
}

// The same layout of work: a lane reads back 16 features of one token, head after head; fp32
// in four runs of four, so that here too each store of two neighbours fills whole sectors
// (with runs of eight, stored in halves, 6 sequences of 0-4099 tokens, 8 x 64, took 17.0 us).
template <int D, typename T>
__global__ void __launch_bounds__(32 * kWarps)
    qcache_read_kernel(const __grid_constant__ QcacheReadParams p, int passes, int heads, int team) {
    constexpr int LPR = D / 16, TPW = 32 / LPR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = (blockIdx.x * (kWarps / team) + warp / team) * TPW * passes;
    pdl_wait_prerequisites();
    constexpr int RUN = 16 / sizeof(T);  // features of a run
    const int lc = lane % LPR, e0 = first_feature(lc) - (8 - RUN) * (lc & 1);
    const int g0 = blockIdx.y * heads + warp % team, g1 = min(p.G, (int)(blockIdx.y + 1) * heads);
    if (t0 >= p.T || g0 >= g1) return;
    Place mine;  // of token t0 + lane: passes * TPW <= 32 (cut_of)
    const bool ok = report(lane < passes * TPW ? place_cached(p, t0 + lane, mine) : kSkip, p.status);
    if (!ok) mine = Place{0, -1, 0};
    const int64_t head = (int64_t)(p.page_size / kQcBlock) * qc_block_bytes(D), plane = (int64_t)p.num_pages * p.G * head;
    const uint32_t sel = (lc & 2) ? 0x7632 : 0x5410;  // the group's half of a word
    for (int pass = 0; pass < passes; ++pass) {
        const Place at = place_of(mine, pass * TPW + lane / LPR);
        if (at.page < 0) continue;  // no lane of this token goes on; the shuffles above are whole again next time
        const int64_t t = t0 + pass * TPW + lane / LPR;
        const int row = at.slot % kQcBlock;
        const int codes = (lc >> 2) * 512 + row * 32 + RUN * (lc & 1);
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
                w[i][0] = load_run(src + i * plane, T());
                w[i][1] = load_run(src + i * plane + 16, T());
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

// How a call is cut: passes a warp takes (their lookups and a lane's frequency go together),
// KV heads of a block, warps that share a token's heads.  A call too small to fill the device
// with one warp for all heads of its tokens spreads the heads, over a block's warps first.
// Passes of a write: their set-up weighs the more the fewer heads follow it, and as they
// grow the warps get few.  us with one, two, four and eight (at one KV head of 64, four is the most):
//   2 x 256  12000 tokens 10.4  9.3 11.1 16.0   40000 31.3 27.8 27.0 29.2   131072 91.1 78.0 72.1 72.1
//   1 x 256  10000         7.1  6.5  7.5 10.4   33000 17.9 15.0 14.3 14.9   120000 59.6 48.7 43.0 41.9
//   1 x 128  20000         8.9  8.5 11.1 17.1   65000 22.6 20.7 21.3 22.7   240000 78.2 68.7 64.9 65.8
//   1 x 64   40000         7.9  7.5  9.1       130000 20.5 18.2 17.8        500000 73.5 62.7 57.7
//   8 x 128  32000        36.2 37.2 41.1 53.2
// A read has little set-up and one pass is best (211k tokens of 4 x 128 86.6 us, 88.4 with two,
// 97.5 with four; in fp32 150.8, 158.0, 177.4), but for long calls whose rows are long to read and
// short to write (131072 tokens of 2 x 256 in bf16: 57.8 with one, 54.0 with two).  It has no
// factors to share between heads and is spread twice as far: 8k tokens of 8 x 128 take 8.1 us
// rather than 9.2, but their write 17.1 rather than 14.5.
struct Cut {
    int passes, heads, team;
    dim3 grid;
};
template <int D, typename E>
Cut cut_of(int T, int G, bool read) {
    constexpr int TPW = 32 / (D / 16);
    const int64_t want = 8 * (int64_t)device_sm_count(), groups = ((int64_t)T + TPW - 1) / TPW;
    Cut c{1, G, 1, dim3()};
    // A warp's tokens are looked up by one lane each, so it takes 32 at most: four passes at
    // head_dim 64.
    constexpr int kMostPasses = 32 / TPW;
    if (read) {
        if (D == 256 && sizeof(E) == 2 && groups >= 8 * want) c.passes = 2;
    } else {
        while (2 * c.passes <= kMostPasses && 2 * c.passes * G <= 8 && groups >= 3 * (int64_t)c.passes * c.passes * want)
            c.passes *= 2;
    }
    if (G > 1 && groups < want) c.team = G > 2 ? kWarps : 2;
    while (c.heads > c.team && groups * c.team * ((G + c.heads - 1) / c.heads) < (read ? 2 : 1) * want) c.heads = (c.heads + 1) / 2;
    const int tokens = kWarps / c.team * TPW * c.passes;
    c.grid = dim3((unsigned)((T + tokens - 1) / tokens), (unsigned)((G + c.heads - 1) / c.heads));
    return c;
}

template <int D, typename T, int TEAM>
cudaError_t write_team(const QcacheWriteParams& p, const Cut& c, cudaStream_t stream) {
    const auto kernel = qcache_write_kernel<D, T, TEAM>;
    constexpr int shared = (int)sizeof(WriteShared<T, TEAM>);
    if (shared > 48 * 1024) {
        const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kernel), shared);
        if (e != cudaSuccess) return e;
    }
    return launch_early(kernel, c.grid, dim3(32 * kWarps), shared, stream, p, c.passes, c.heads);
}
template <int D, typename T>
cudaError_t write_d(const QcacheWriteParams& p, cudaStream_t stream) {
    const Cut c = cut_of<D, T>(p.T, p.G, false);
    return c.team == 1 ? write_team<D, T, 1>(p, c, stream)
         : c.team == 2 ? write_team<D, T, 2>(p, c, stream)
                       : write_team<D, T, kWarps>(p, c, stream);
}

template <int D, typename T>
cudaError_t read_d(const QcacheReadParams& p, cudaStream_t stream) {
    const Cut c = cut_of<D, T>(p.T, p.G, true);
    return launch_early(qcache_read_kernel<D, T>, c.grid, dim3(32 * kWarps), 0, stream, p, c.passes, c.heads, c.team);
}

}  // namespace

cudaError_t launch_qcache_write(const QcacheWriteParams& p, bool fp32, cudaStream_t stream) {
    switch (p.d) {
        case 64: return fp32 ? write_d<64, float>(p, stream) : write_d<64, bf16>(p, stream);
        case 128: return fp32 ? write_d<128, float>(p, stream) : write_d<128, bf16>(p, stream);
        case 256: return fp32 ? write_d<256, float>(p, stream) : write_d<256, bf16>(p, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_qcache_read(const QcacheReadParams& p, bool fp32, cudaStream_t stream) {
    switch (p.d) {
        case 64: return fp32 ? read_d<64, float>(p, stream) : read_d<64, bf16>(p, stream);
        case 128: return fp32 ? read_d<128, float>(p, stream) : read_d<128, bf16>(p, stream);
        case 256: return fp32 ? read_d<256, float>(p, stream) : read_d<256, bf16>(p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gattn
