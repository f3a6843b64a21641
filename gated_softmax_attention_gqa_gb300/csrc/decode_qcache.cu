// decode_qcache.cu -- one decode step of gated GQA attention against the 4-bit KV
// cache (format: qcache.cuh).
//
// The keys of a sequence are cut into chunks of kChunk; one block per (chunk, KV head,
// sequence) computes the chunk's partial softmax state (maximum, sum, unnormalised
// output) for the head's H/G queries, and a second pass merges the chunks and applies
// the output gate.
#include "qcache.cuh"

namespace gattn {
namespace {

constexpr int kChunk = 256;

// The newest query of every head of one KV group, normed and rotated: q[h][e] (fp32).
template <int D>
__device__ void make_queries(const QcacheDecodeParams& p, int b, int g, int pos, float (*q)[D]) {
    const int r = p.H / p.G, lane = threadIdx.x & 31, nwarp = blockDim.x >> 5;
    const bf16* w = static_cast<const bf16*>(p.qnorm_w);
    for (int h = threadIdx.x >> 5; h < r; h += nwarp) {
        const bf16* row = static_cast<const bf16*>(p.q) + b * p.q_seq_stride + (int64_t)(g * r + h) * p.q_head_stride;
        float ss = 0.f;
        for (int e = lane; e < D; e += 32) {
            const float x = __bfloat162float(row[e]);
            ss = fmaf(x, x, ss);
            q[h][e] = x * __bfloat162float(w[e]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rinv = 1.0f / sqrtf(ss / (float)D + p.eps);
        __syncwarp();
        const int half = p.rd >> 1;
        for (int e = lane; e < half; e += 32) {
            float s, c;
            rope_turn_sincos(p.turns[e], pos, &s, &c);
            const float x0 = q[h][e], x1 = q[h][e + half];
            q[h][e] = (x0 * c - x1 * s) * rinv;
            q[h][e + half] = (x1 * c + x0 * s) * rinv;
        }
        for (int e = p.rd + lane; e < D; e += 32) q[h][e] *= rinv;
    }
    __syncthreads();
}

__device__ __forceinline__ const uint8_t* key_block(const QcacheDecodeParams& p, int b, int g, int key) {
    int page = p.block_table[(int64_t)b * p.max_pages + key / p.page_size];
    if (page < 0 || page >= p.num_pages) {
        atomicOr(p.status, GATTN_DEVICE_BAD_PAGE);
        page = 0;
    }
    return p.cache + qc_block_offset(page, g, key % p.page_size, p.G, p.page_size, p.d);
}

// value of feature e of row `row` of a block
__device__ __forceinline__ float qc_value(const uint8_t* block, int row, int e, int d) {
    const uint8_t byte = block[(e >> 6) * 512 + row * 32 + 4 * ((e & 31) >> 2) + 2 * ((e >> 5) & 1) + ((e & 3) >> 1)];
    const bf16* par = reinterpret_cast<const bf16*>(block + 8 * d) + (e >> 5) * 16 + row;
    const int n = (int)((byte >> (4 * (e & 1))) & 15) - 8;
    return fmaf(__bfloat162float(par[0]), (float)n, __bfloat162float(par[d / 2]));
}

template <int D>
__global__ void __launch_bounds__(kChunk) qdecode_chunk_kernel(const __grid_constant__ QcacheDecodeParams p) {
    __shared__ float q[8][D];
    __shared__ float sc[8][kChunk];
    __shared__ const uint8_t* blocks[kChunk / kQcBlock];
    const int g = blockIdx.y, b = blockIdx.z, r = p.H / p.G;
    const int L = p.seqlens[b], k0 = blockIdx.x * kChunk;
    if (L < 1 || L > p.max_pages * p.page_size || k0 >= L) return;
    const int n = min(kChunk, L - k0), tid = threadIdx.x;
    if (tid < kChunk / kQcBlock && tid * kQcBlock < n) blocks[tid] = key_block(p, b, g, k0 + tid * kQcBlock);
    make_queries<D>(p, b, g, L - 1, q);
    float acc[8] = {};
    if (tid < n) {
        for (int e = 0; e < D; ++e) {
            const float kv = qc_value(blocks[tid / kQcBlock], tid % kQcBlock, e, D);
#pragma unroll
            for (int h = 0; h < 8; ++h)
                if (h < r) acc[h] = fmaf(q[h][e], kv, acc[h]);
        }
    }
#pragma unroll
    for (int h = 0; h < 8; ++h)
        if (h < r) sc[h][tid] = tid < n ? acc[h] * p.scale_log2 : -INFINITY;
    __syncthreads();
    const int64_t nch = gridDim.x;
    const int lane = tid & 31;
    for (int h = tid >> 5; h < r; h += kChunk / 32) {
        float m = -INFINITY, l = 0.f;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, sc[h][i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        for (int i = lane; i < n; i += 32) {
            sc[h][i] = exp2f(sc[h][i] - m);
            l += sc[h][i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) {
            float* ps = p.part + (((int64_t)b * p.H + g * r + h) * nch + blockIdx.x) * (D + 2);
            ps[0] = m;
            ps[1] = l;
        }
    }
    __syncthreads();
    const int64_t plane = (int64_t)p.num_pages * p.G * (p.page_size / kQcBlock) * qc_block_bytes(D);
    for (int e = tid; e < D; e += kChunk) {
        float o[8] = {};
        for (int i = 0; i < n; ++i) {
            const float v = qc_value(blocks[i / kQcBlock] + plane, i % kQcBlock, e, D);
#pragma unroll
            for (int h = 0; h < 8; ++h)
                if (h < r) o[h] = fmaf(sc[h][i], v, o[h]);
        }
        for (int h = 0; h < r; ++h)
            p.part[(((int64_t)b * p.H + g * r + h) * nch + blockIdx.x) * (D + 2) + 2 + e] = o[h];
    }
}

// Merge the chunks of one (sequence, head) and apply the gate; one thread per feature.
__global__ void qdecode_combine_kernel(const __grid_constant__ QcacheDecodeParams p, int nch) {
    const int h = blockIdx.x, b = blockIdx.y, e = threadIdx.x, d = p.d;
    const int L = p.seqlens[b];
    if (L < 0 || L > p.max_pages * p.page_size) {
        if (e == 0 && h == 0) atomicOr(p.status, GATTN_DEVICE_BAD_SEQLEN);
        return;
    }
    const int n = (L + kChunk - 1) / kChunk;
    const float* ps = p.part + ((int64_t)b * p.H + h) * nch * (d + 2);
    float m = -INFINITY, den = 0.f, num = 0.f;
    for (int i = 0; i < n; ++i) m = fmaxf(m, ps[(int64_t)i * (d + 2)]);
    for (int i = 0; i < n; ++i) {
        const float* s = ps + (int64_t)i * (d + 2);
        const float w = exp2f(s[0] - m);
        den = fmaf(w, s[1], den);
        num = fmaf(w, s[2 + e], num);
    }
    float o = n ? num / den : 0.f;  // no key: the empty sum
    const int layout = gate_layout(p.gate_mode);
    if (layout != GATTN_GATE_NONE) {
        const bf16* gp = static_cast<const bf16*>(p.gate) + b * p.gate_seq_stride;
        const float z = __bfloat162float(layout == GATTN_GATE_ELEMENTWISE ? gp[h * p.gate_head_stride + e]
                                         : layout == GATTN_GATE_HEADWISE  ? gp[h * p.gate_head_stride]
                                                                          : gp[e]);
        const float a = gate_act(z, sigmoidf_dev(z), p.gate_mode);
        o = gate_additive(p.gate_mode) ? o + a : o * a;
    }
    static_cast<bf16*>(p.out)[((int64_t)b * p.H + h) * d + e] = __float2bfloat16_rn(o);
}

template <int D>
cudaError_t launch_d(const QcacheDecodeParams& p, cudaStream_t stream, cudaEvent_t ev_start, cudaEvent_t ev_stop) {
    const int nch = (p.max_pages * p.page_size + kChunk - 1) / kChunk;
    if (ev_start) cudaEventRecord(ev_start, stream);
    qdecode_chunk_kernel<D><<<dim3(nch, p.G, p.B), kChunk, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (ev_stop) cudaEventRecord(ev_stop, stream);
    if (e != cudaSuccess) return e;
    qdecode_combine_kernel<<<dim3(p.H, p.B), D, 0, stream>>>(p, nch);
    return cudaGetLastError();
}

}  // namespace

size_t qcache_decode_workspace(int B, int H, int G, int d, int Lmax, int n_sms) {
    (void)G, (void)n_sms;
    return (size_t)B * H * (((size_t)Lmax + kChunk - 1) / kChunk) * (d + 2) * sizeof(float);
}

cudaError_t launch_qcache_decode(const QcacheDecodeParams& p, cudaStream_t stream, cudaEvent_t ev_start,
                                 cudaEvent_t ev_stop) {
    switch (p.d) {
        case 64: return launch_d<64>(p, stream, ev_start, ev_stop);
        case 128: return launch_d<128>(p, stream, ev_start, ev_stop);
        case 256: return launch_d<256>(p, stream, ev_start, ev_stop);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gattn
