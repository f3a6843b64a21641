// qcache.cu -- writing the 4-bit KV cache and reading it back (format: qcache.cuh).
//
// Both passes move every number once: the write reads 2 (bf16) or 4 (fp32) bytes a
// number and leaves 0.625, the read the reverse, so both are bound by HBM as long as
// the arithmetic per number stays small.
#include "qcache.cuh"

namespace gattn {
namespace {

// Eight consecutive features of a row as floats.
__device__ __forceinline__ void load8(const bf16* p, float (&x)[8]) {
    unpack8(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(bf16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Quantise this lane's eight features (four lanes share a group of 32, eight a slab)
// and store codes, scale and centre of the row at `block`.
__device__ __forceinline__ void encode_store(const float (&x)[8], uint8_t* block, int row, int e0, int d, bool live) {
    float hi = x[0], lo = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        hi = max_nan(hi, x[i]);
        lo = min_nan(lo, x[i]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    const QcGroup q = qc_group(lo, hi);
    const uint32_t w = qc_encode8(x, q);
    // lanes j and j + 4 of a slab hold features 8j.. and 32 + 8j..; their low halves make
    // word 2j, their high halves word 2j + 1
    const uint32_t o = __shfl_xor_sync(0xffffffffu, w, 4);
    if (!live) return;
    const int j = (e0 >> 3) & 3, upper = (e0 >> 5) & 1;
    const uint32_t word = upper ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
    reinterpret_cast<uint32_t*>(block + (e0 >> 6) * 512 + row * 32)[2 * j + upper] = word;
    if (j == 0) {
        uint16_t* par = reinterpret_cast<uint16_t*>(block + 8 * d);
        par[(e0 >> 5) * 16 + row] = (uint16_t)q.scale_bits;
        par[d / 2 + (e0 >> 5) * 16 + row] = (uint16_t)q.centre_bits;
    }
}

// One row (token, KV head) is spread over D / 8 lanes.
template <int D, typename T>
__global__ void __launch_bounds__(256) qcache_write_kernel(const __grid_constant__ QcacheWriteParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31;
    const int64_t row = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * RPW + lane / LPR;
    const bool in_range = row < (int64_t)p.T * p.G;
    const int t = in_range ? (int)(row / p.G) : 0, g = in_range ? (int)(row % p.G) : 0;
    const int e0 = 8 * (lane % LPR);

    // where the token goes
    int b = t, n = 1, j = 0;
    if (p.cu_seqlens) {
        b = find_sequence(p.cu_seqlens, p.B, t);
        n = p.cu_seqlens[b + 1] - p.cu_seqlens[b];
        j = t - p.cu_seqlens[b];
    }
    const int L = p.seqlens[b];
    // a length of 0 marks an unused row of a batch that adds one token to each sequence
    bool live = in_range && j >= 0 && j < n && (p.cu_seqlens || L != 0);
    const int pos = L - n + j;
    if (live && (L > p.max_pages * p.page_size || L < n)) {
        atomicOr(p.status, GATTN_DEVICE_BAD_SEQLEN);
        live = false;
    }
    int page = 0;
    if (live) {
        page = p.block_table[(int64_t)b * p.max_pages + pos / p.page_size];
        if (page < 0 || page >= p.num_pages) {
            atomicOr(p.status, GATTN_DEVICE_BAD_PAGE);
            live = false;
        }
    }
    const int slot = live ? pos % p.page_size : 0;
    uint8_t* block = p.cache + qc_block_offset(live ? page : 0, g, slot, p.G, p.page_size, D);
    const int64_t plane = (int64_t)p.num_pages * p.G * (p.page_size / kQcBlock) * qc_block_bytes(D);

    // K: norm, rotation, codes
    float x[8], w[8], y[8], ss = 0.f;
    load8(static_cast<const T*>(p.k) + t * p.k_tok_stride + g * p.k_head_stride + e0, x);
    load8(static_cast<const T*>(p.knorm_w) + e0, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        ss = fmaf(x[i], x[i], ss);
        y[i] = x[i] * w[i];
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float rinv = 1.0f / sqrtf(ss / (float)D + p.eps);
    const int half = p.rd >> 1;
    const bool rot = e0 < p.rd, first = e0 < half;
    const int src = rot ? lane + (first ? half >> 3 : -(half >> 3)) : lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, y[i], src);
        float s = 0.f, c = 1.f;
        if (rot) rope_turn_sincos(p.turns[(first ? e0 : e0 - half) + i], pos, &s, &c);
        x[i] = fmaf(y[i], c, o * (first ? -s : s)) * rinv;
    }
    encode_store(x, block, slot % kQcBlock, e0, D, live);

    load8(static_cast<const T*>(p.v) + t * p.v_tok_stride + g * p.v_head_stride + e0, x);
    encode_store(x, block + plane, slot % kQcBlock, e0, D, live);
}

template <int D, typename T>
__global__ void __launch_bounds__(256) qcache_read_kernel(const __grid_constant__ QcacheReadParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31;
    const int64_t row = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * RPW + lane / LPR;
    if (row >= (int64_t)p.T * p.G) return;
    const int t = (int)(row / p.G), g = (int)(row % p.G), e0 = 8 * (lane % LPR);
    int b = t, n = 1, j = 0;
    if (p.cu_seqlens) {
        b = find_sequence(p.cu_seqlens, p.B, t);
        n = p.cu_seqlens[b + 1] - p.cu_seqlens[b];
        j = t - p.cu_seqlens[b];
    }
    if (j < 0 || j >= n) return;
    const int64_t start = p.starts ? p.starts[b] : 0;
    if (start < 0 || start + n > (int64_t)p.max_pages * p.page_size) {
        atomicOr(p.status, GATTN_DEVICE_BAD_SEQLEN);
        return;
    }
    const int pos = (int)start + j;
    const int page = p.block_table[(int64_t)b * p.max_pages + pos / p.page_size];
    if (page < 0 || page >= p.num_pages) {
        atomicOr(p.status, GATTN_DEVICE_BAD_PAGE);
        return;
    }
    const int slot = pos % p.page_size, r = slot % kQcBlock;
    const uint8_t* block = p.cache + qc_block_offset(page, g, slot, p.G, p.page_size, D);
    const int64_t plane = (int64_t)p.num_pages * p.G * (p.page_size / kQcBlock) * qc_block_bytes(D);
    const int q = (e0 >> 3) & 3, upper = (e0 >> 5) & 1;
    for (int pl = 0; pl < 2; ++pl, block += plane) {
        const uint2 w = *reinterpret_cast<const uint2*>(block + (e0 >> 6) * 512 + r * 32 + q * 8);
        const uint32_t codes = __byte_perm(w.x, w.y, upper ? 0x7632 : 0x5410);
        const bf16* par = reinterpret_cast<const bf16*>(block + 8 * D) + (e0 >> 5) * 16 + r;
        const float s = __bfloat162float(par[0]), c = __bfloat162float(par[D / 2]);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(s, (float)((int)((codes >> (4 * i)) & 15u) - 8), c);
        store8(static_cast<T*>(pl ? p.v : p.k) + row * D + e0, x);
    }
}

template <int D>
cudaError_t write_d(const QcacheWriteParams& p, bool fp32, cudaStream_t stream) {
    constexpr int RPB = 8 * (32 / (D / 8));
    const unsigned blocks = (unsigned)(((int64_t)p.T * p.G + RPB - 1) / RPB);
    if (fp32) qcache_write_kernel<D, float><<<blocks, 256, 0, stream>>>(p);
    else qcache_write_kernel<D, bf16><<<blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t read_d(const QcacheReadParams& p, bool fp32, cudaStream_t stream) {
    constexpr int RPB = 8 * (32 / (D / 8));
    const unsigned blocks = (unsigned)(((int64_t)p.T * p.G + RPB - 1) / RPB);
    if (fp32) qcache_read_kernel<D, float><<<blocks, 256, 0, stream>>>(p);
    else qcache_read_kernel<D, bf16><<<blocks, 256, 0, stream>>>(p);
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
