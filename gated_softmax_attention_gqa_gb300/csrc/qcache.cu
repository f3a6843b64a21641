// qcache.cu -- writing the 4-bit KV cache and reading it back (format: qcache.cuh).
//
// Both passes move every number once: the write reads 2 (bf16) or 4 (fp32) bytes a
// number and leaves 0.625, the read the reverse, so HBM bounds both as long as the
// arithmetic stays small: at 6.8 TB/s an SM has some 14 instruction slots for a written
// number.  So a lane takes 16 features (half a scale group) of one token and walks its KV
// heads: the token's place, its sines and cosines (made once per warp, in shared memory)
// and their products with the norm weights are shared by all heads, and what a group
// costs (extremes, scale, reciprocal) is shared by 32 numbers and two lanes.
#include "qcache.cuh"

namespace gattn {
namespace {

constexpr int kWarps = 8;

// Sixteen consecutive features of a row, as loaded.
template <typename T>
struct Row16;
template <>
struct Row16<bf16> {
    uint4 v[2];
    __device__ __forceinline__ void load(const bf16* p) {
        v[0] = reinterpret_cast<const uint4*>(p)[0];
        v[1] = reinterpret_cast<const uint4*>(p)[1];
    }
    // features 8 c .. 8 c + 7 only, from p
    __device__ __forceinline__ void load8(int c, const bf16* p) { v[c] = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[8 * c + 2 * i] = bf16_lo(w[i]);
                x[8 * c + 2 * i + 1] = bf16_hi(w[i]);
            }
        }
    }
};
template <>
struct Row16<float> {
    float4 v[4];
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const float4*>(p)[i];
    }
    __device__ __forceinline__ void load8(int c, const float* p) {
        v[2 * c] = reinterpret_cast<const float4*>(p)[0];
        v[2 * c + 1] = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[4 * i] = v[i].x;
            x[4 * i + 1] = v[i].y;
            x[4 * i + 2] = v[i].z;
            x[4 * i + 3] = v[i].w;
        }
    }
};

// Place of packed token t: its position, and its row of the pool.  False for padding and
// for tokens that a length or a table entry keeps out of the cache (the caller reports).
struct Place {
    int pos, page, slot;
};
enum { kSkip = 0, kLive = 1, kBadLength = 2, kBadPage = 3 };

__device__ __forceinline__ int find_page(const int32_t* table, int max_pages, int num_pages, int page_size, int b,
                                         Place& at) {
    const int k = at.pos / page_size;
    at.slot = at.pos - k * page_size;
    at.page = table[(int64_t)b * max_pages + k];
    return at.page >= 0 && at.page < num_pages ? kLive : kBadPage;
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
    return find_page(p.block_table, p.max_pages, p.num_pages, p.page_size, b, at);
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
    return find_page(p.block_table, p.max_pages, p.num_pages, p.page_size, b, at);
}

__device__ __forceinline__ bool report(int what, unsigned int* status) {
    if (what == kBadLength) atomicOr(status, GATTN_DEVICE_BAD_SEQLEN);
    if (what == kBadPage) atomicOr(status, GATTN_DEVICE_BAD_PAGE);
    return what == kLive;
}

// Quantise this lane's 16 features (two neighbouring lanes share a group of 32, four a
// slab) and store them at row `row` of `block`.  All lanes of the warp.
__device__ __forceinline__ void encode_store(const float (&x)[16], uint8_t* block, int row, int e0, int d, bool live) {
    float hi = max_nan(x[0], x[1]), lo = min_nan(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < 16; i += 2) {
        hi = max_nan(hi, x[i], x[i + 1]);
        lo = min_nan(lo, x[i], x[i + 1]);
    }
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
    const QcGroup q = qc_group(lo, hi);
    uint32_t w[2];
    const bool inside = qc_round(hi, q) <= kQcMagic + 7.f && qc_round(lo, q) >= kQcMagic - 8.f;
    if (__all_sync(0xffffffffu, inside)) {
        w[0] = qc_encode8<false>(x, q);
        w[1] = qc_encode8<false>(x + 8, q);
    } else {
        w[0] = qc_encode8<true>(x, q);
        w[1] = qc_encode8<true>(x + 8, q);
    }
    // lanes j and j + 2 of a slab hold features 16 j .. and 32 + 16 j ..: together the words
    // 4 j .. 4 j + 3, of which lane j stores the first two and lane j + 2 the others
    const int j = (e0 >> 4) & 1, upper = (e0 >> 5) & 1;
    const uint32_t o = __shfl_xor_sync(0xffffffffu, upper ? w[0] : w[1], 2);
    if (!live) return;
    const uint32_t a = upper ? o : w[0], b = upper ? w[1] : o;
    *reinterpret_cast<uint2*>(block + (e0 >> 6) * 512 + row * 32 + 16 * j + 8 * upper) =
        make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    // the group's two lanes store its scale and its centre
    reinterpret_cast<uint16_t*>(block + 8 * d)[j * (d / 2) + (e0 >> 5) * 16 + row] =
        (uint16_t)(j ? q.centre_bits : q.scale_bits);
}

// A token is spread over D / 16 lanes; a warp takes 32 / (D / 16) neighbouring tokens and
// walks heads [blockIdx.y heads, ...).
template <int D, typename T>
__global__ void __launch_bounds__(32 * kWarps) qcache_write_kernel(const __grid_constant__ QcacheWriteParams p, int heads) {
    constexpr int LPR = D / 16, TPW = 32 / LPR;
    __shared__ float2 tables[kWarps][TPW * D / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = (blockIdx.x * kWarps + warp) * TPW;
    if (t0 >= p.T) return;
    const int tl = lane / LPR, t = t0 + tl, e0 = 16 * (lane % LPR);
    const int g0 = blockIdx.y * heads, g1 = min(p.G, g0 + heads);
    const int64_t row0 = min(t, p.T - 1);
    const T* kp = static_cast<const T*>(p.k) + row0 * p.k_tok_stride + g0 * p.k_head_stride + e0;
    const T* vp = static_cast<const T*>(p.v) + row0 * p.v_tok_stride + g0 * p.v_head_stride + e0;
    // rotation partners, eight features at a time (rotary_dim / 2 is a multiple of 8)
    const int half = p.rd >> 1;
    bool rot[2];
    int mate[2];  // the partners' distance
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        rot[c] = e0 + 8 * c < p.rd;
        mate[c] = e0 + 8 * c < half ? half : -half;
    }
    Row16<T> kr, ko, vr;
    auto load_k = [&]() {
        kr.load(kp);
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (rot[c]) ko.load8(c, kp + 8 * c + mate[c]);
    };
    load_k();

    Place at;
    const bool live = report(place_new(p, t, at), p.status);

    // sines and cosines of the warp's tokens
    float2* table = tables[warp];
    for (int i0 = 0; i0 < TPW * half; i0 += 32) {
        const int i = i0 + lane, k = min(i / max(half, 1), TPW - 1);
        const int pos = __shfl_sync(0xffffffffu, at.pos, k * LPR);
        if (i < TPW * half) {
            float s, c;
            rope_turn_sincos(p.turns[i - k * half], pos, &s, &c);
            table[i] = make_float2(s, c);
        }
    }
    __syncwarp();
    // K' = (x wc + partner ws) / rms, with the norm weights in wc and ws
    float wc[16], ws[16];
    {
        Row16<T> wr;
        float w[16];
        wr.load(static_cast<const T*>(p.knorm_w) + e0);
        wr.get(w);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float m[16];
            const int e = e0 + 8 * c;
            if (rot[c]) {
                wr.load8(c, static_cast<const T*>(p.knorm_w) + e + mate[c]);
                wr.get(m);
            }
            const float2* sc = table + tl * half + (e < half ? e : e - half);
#pragma unroll
            for (int i = 8 * c; i < 8 * c + 8; ++i) {
                wc[i] = w[i];
                ws[i] = 0.f;
                if (rot[c]) {
                    const float2 v = sc[i - 8 * c];
                    wc[i] = w[i] * v.y;
                    ws[i] = m[i] * (e < half ? -v.x : v.x);
                }
            }
        }
    }
    const int64_t plane = (int64_t)p.num_pages * p.G * (p.page_size / kQcBlock) * qc_block_bytes(D);
    const int64_t head = (int64_t)(p.page_size / kQcBlock) * qc_block_bytes(D);
    uint8_t* block = p.cache + (live ? qc_block_offset(at.page, g0, at.slot, p.G, p.page_size, D) : 0);
    const int row = live ? at.slot % kQcBlock : 0;
    const bool any_rot = p.rd > 0;
    for (int g = g0; g < g1; ++g) {
        vr.load(vp);
        float x[16], o[16], ss = 0.f;
        kr.get(x);
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int s = LPR / 2; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
        const float rinv = 1.0f / sqrtf(ss / (float)D + p.eps);
        if (any_rot) {
            ko.get(o);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 8 * c; i < 8 * c + 8; ++i) x[i] = fmaf(x[i], wc[i], rot[c] ? o[i] * ws[i] : 0.f) * rinv;
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = x[i] * wc[i] * rinv;
        }
        if (g + 1 < g1) {
            kp += p.k_head_stride;
            load_k();
        }
        encode_store(x, block, row, e0, D, live);
        vr.get(x);
        encode_store(x, block + plane, row, e0, D, live);
        vp += p.v_head_stride;
        block += head;
    }
}

__device__ __forceinline__ void store8(bf16* p, const float* x) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// The same layout of work: a lane reads back 16 features of one token, head after head.
template <int D, typename T>
__global__ void __launch_bounds__(32 * kWarps) qcache_read_kernel(const __grid_constant__ QcacheReadParams p, int heads) {
    constexpr int LPR = D / 16, TPW = 32 / LPR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = (blockIdx.x * kWarps + warp) * TPW;
    if (t0 >= p.T) return;
    const int t = t0 + lane / LPR, e0 = 16 * (lane % LPR);
    Place at;
    if (!report(place_cached(p, t, at), p.status)) return;
    const int g0 = blockIdx.y * heads, n = 2 * (min(p.G, g0 + heads) - g0);
    const int64_t plane = (int64_t)p.num_pages * p.G * (p.page_size / kQcBlock) * qc_block_bytes(D);
    const int64_t head = (int64_t)(p.page_size / kQcBlock) * qc_block_bytes(D);
    const uint8_t* block = p.cache + qc_block_offset(at.page, g0, at.slot, p.G, p.page_size, D);
    const int row = at.slot % kQcBlock, j = (e0 >> 4) & 1, upper = (e0 >> 5) & 1;
    const int codes = (e0 >> 6) * 512 + row * 32 + 16 * j, par = 8 * D + ((e0 >> 5) * 16 + row) * 2;
    T* kout = static_cast<T*>(p.k) + ((int64_t)t * p.G + g0) * D + e0;
    T* vout = static_cast<T*>(p.v) + ((int64_t)t * p.G + g0) * D + e0;
    const uint32_t sel = upper ? 0x7632 : 0x5410;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {  // K and V of each head in turn
        const uint8_t* src = block + (i >> 1) * head + (i & 1) * plane;
        const uint4 w = *reinterpret_cast<const uint4*>(src + codes);
        const float s = __bfloat162float(*reinterpret_cast<const bf16*>(src + par));
        const float c = __bfloat162float(*reinterpret_cast<const bf16*>(src + par + D));
        const uint32_t n8[2] = {__byte_perm(w.x, w.y, sel), __byte_perm(w.z, w.w, sel)};
        T* out = ((i & 1) ? vout : kout) + (i >> 1) * D;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[8];
            // 2^23 + code as a float; one subtraction leaves code - 8
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = fmaf(s, __uint_as_float(((n8[h] >> (4 * k)) & 15u) | 0x4B000000u) - 8388616.f, c);
            store8(out + 8 * h, x);
        }
    }
}

// Warps walk all heads of their tokens where that gives every SM work; else the heads are
// spread over the grid's second dimension.  (64 tokens of two heads: 4.2 us in one
// dimension; 131072 tokens of two: no difference.)
int heads_per_warp(int64_t token_warps, int G) {
    int heads = G;
    while (heads > 1 && token_warps * ((G + heads - 1) / heads) < 8 * device_sm_count()) heads = (heads + 1) / 2;
    return heads;
}

template <int D>
dim3 grid_of(int T, int G, int heads) {
    constexpr int tokens = kWarps * (32 / (D / 16));
    return dim3((unsigned)((T + tokens - 1) / tokens), (unsigned)((G + heads - 1) / heads));
}

template <int D>
cudaError_t write_d(const QcacheWriteParams& p, bool fp32, cudaStream_t stream) {
    const int heads = heads_per_warp((p.T + 32 / (D / 16) - 1) / (32 / (D / 16)), p.G);
    if (fp32) qcache_write_kernel<D, float><<<grid_of<D>(p.T, p.G, heads), 32 * kWarps, 0, stream>>>(p, heads);
    else qcache_write_kernel<D, bf16><<<grid_of<D>(p.T, p.G, heads), 32 * kWarps, 0, stream>>>(p, heads);
    return cudaGetLastError();
}

template <int D>
cudaError_t read_d(const QcacheReadParams& p, bool fp32, cudaStream_t stream) {
    const int heads = heads_per_warp((p.T + 32 / (D / 16) - 1) / (32 / (D / 16)), p.G);
    if (fp32) qcache_read_kernel<D, float><<<grid_of<D>(p.T, p.G, heads), 32 * kWarps, 0, stream>>>(p, heads);
    else qcache_read_kernel<D, bf16><<<grid_of<D>(p.T, p.G, heads), 32 * kWarps, 0, stream>>>(p, heads);
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
