// qcache_api.cu -- C entry points of the 4-bit KV cache: argument checks and launches
// (contract: include/gattn.h).
#include <cmath>
#include <cstdint>
#include <cstring>

#include "qcache.cuh"

using namespace gattn;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Rotation of pair i per position, base^(-2i/rd) / (2 pi), modulo one turn in 2^-64 turns.
// The table of the last (rd, base) is kept per thread: rd/2 powers cost more than a launch.
void fill_turns(uint64_t* dst, int rd, double base) {
    static thread_local struct {
        int rd;
        double base;
        uint64_t turns[kMaxRotaryHalf];
    } last = {};
    if (rd != last.rd || base != last.base) {
        for (int i = 0; i < rd / 2; ++i) {
            const double turns = std::pow(base, -2.0 * i / rd) * 0.15915494309189533576888376337251436;
            const double frac = turns - std::floor(turns);
            last.turns[i] = frac >= 0.0 && frac < 1.0 ? (uint64_t)std::ldexp(frac, 64) : 0;  // exact: 53 bits
        }
        last.rd = rd;
        last.base = base;
    }
    std::memcpy(dst, last.turns, sizeof(uint64_t) * (rd / 2));
}

// floor(x / d) = floor(x m / 2^(31 + k)) for 0 <= x < 2^31, with 2^k the power of two at or
// above d >= 2 and m = floor(2^(31 + k) / d) + 1 (m d exceeds 2^(31 + k) by at most d <= 2^k).
// mul = 0 stands for d = 1.
PageDiv page_div(int d) {
    if (d == 1) return PageDiv{0, 0};
    int k = 0;
    while (((int64_t)1 << k) < d) ++k;
    return PageDiv{(uint32_t)((((uint64_t)1 << (31 + k)) / (uint64_t)d) + 1), (uint32_t)(k - 1)};
}

constexpr int kMostTokens = INT32_MAX - 1024;  // of a sequence: the kernels round lengths up to tiles in 31 bits

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

// The pool's geometry: what every entry point checks of it.
gattn_status check_pool(const void* cache, const int32_t* table, int num_pages, int page_size, int max_pages, int B,
                        int G, int d) {
    if (!cache || !table || num_pages < 1 || page_size < 1 || max_pages < 1 || B < 1 || G < 1 || d < 1)
        return GATTN_ERR_INVALID_ARG;
    if (!aligned(cache, 16) || !aligned(table, 4)) return GATTN_ERR_INVALID_ARG;
    if (!head_dim_ok(d) || page_size % kQcBlock != 0) return GATTN_ERR_UNSUPPORTED;
    if ((int64_t)max_pages * page_size > kMostTokens) return GATTN_ERR_INVALID_ARG;
    return GATTN_OK;
}

gattn_status check_rope(int d, int rotary_dim, double rope_base, float eps) {
    if (rotary_dim < 0 || rotary_dim > d || (rotary_dim & 1)) return GATTN_ERR_INVALID_ARG;
    if (rotary_dim > 0 && !(rope_base > 0.0 && std::isfinite(rope_base))) return GATTN_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return GATTN_ERR_INVALID_ARG;
    return rotary_dim % 16 ? GATTN_ERR_UNSUPPORTED : GATTN_OK;
}

// The batches a decode step takes, of heads, dimensions and lengths that are right otherwise.
bool batch_ok(int B, int H, int G, int64_t Lmax) {
    if (H / G > 8 || B > decode_max_batch()) return false;
    // the kernels count the batch's 64-key tiles (and a few per head and sequence) in 31 bits
    return (int64_t)B * G * (Lmax / 64 + 8) <= INT32_MAX;
}

// Rows are moved 16 bytes at a time.
bool row_strides_ok(const void* p, int64_t tok, int64_t head, int elt) {
    return aligned(p, 16) && tok >= 0 && head >= 0 && tok * elt % 16 == 0 && head * elt % 16 == 0;
}

// gattn_qcache_write; before_decode: a decode step's split kernel is launched next.
gattn_status write_tokens(const void* k, const void* v, void* qcache, const int32_t* block_table, int num_pages,
                          int page_size, int max_pages, const int32_t* seqlens, const int32_t* cu_seqlens,
                          const void* knorm_w, int T, int B, int G, int d, int rotary_dim, double rope_base,
                          float eps, int64_t k_tok_stride, int64_t k_head_stride, int64_t v_tok_stride,
                          int64_t v_head_stride, int dtype, void* stream, bool before_decode) {
    if (dtype != GATTN_BF16 && dtype != GATTN_FP32) return GATTN_ERR_INVALID_ARG;
    if (T < 0 || (!cu_seqlens && T != B)) return GATTN_ERR_INVALID_ARG;
    gattn_status st = check_pool(qcache, block_table, num_pages, page_size, max_pages, B, G, d);
    if (st != GATTN_OK) return st;
    if ((st = check_rope(d, rotary_dim, rope_base, eps)) != GATTN_OK) return st;
    if (!seqlens || !knorm_w || !aligned(seqlens, 4) || !aligned(cu_seqlens, 4) || !aligned(knorm_w, 16))
        return GATTN_ERR_INVALID_ARG;
    if (T == 0) return GATTN_OK;
    if (!k || !v || (int64_t)T * G > ((int64_t)1 << 30)) return GATTN_ERR_INVALID_ARG;
    if (k_tok_stride == 0) k_tok_stride = (int64_t)G * d;
    if (k_head_stride == 0) k_head_stride = d;
    if (v_tok_stride == 0) v_tok_stride = (int64_t)G * d;
    if (v_head_stride == 0) v_head_stride = d;
    const int elt = dtype == GATTN_BF16 ? 2 : 4;
    if (!row_strides_ok(k, k_tok_stride, k_head_stride, elt) || !row_strides_ok(v, v_tok_stride, v_head_stride, elt))
        return GATTN_ERR_INVALID_ARG;
    QcacheWriteParams p;
    std::memset(&p, 0, sizeof(p));
    if (!(p.status = device_status_word())) return GATTN_ERR_CUDA;
    p.k = k;
    p.v = v;
    p.cache = static_cast<uint8_t*>(qcache);
    p.block_table = block_table;
    p.seqlens = seqlens;
    p.cu_seqlens = cu_seqlens;
    p.knorm_w = knorm_w;
    p.k_tok_stride = k_tok_stride;
    p.k_head_stride = k_head_stride;
    p.v_tok_stride = v_tok_stride;
    p.v_head_stride = v_head_stride;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.by_page = page_div(page_size);
    p.T = T;
    p.B = B;
    p.G = G;
    p.d = d;
    p.rd = rotary_dim;
    p.before_decode = before_decode;
    p.eps = eps;
    fill_turns(p.turns, rotary_dim, rope_base);
    return launch_qcache_write(p, dtype == GATTN_FP32, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GATTN_OK
               : GATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t gattn_qcache_bytes(int num_pages, int G, int page_size, int d) {
    if (num_pages < 1 || G < 1 || page_size < kQcBlock || page_size % kQcBlock || !head_dim_ok(d)) return 0;
    return (size_t)2 * num_pages * G * (page_size / kQcBlock) * (size_t)qc_block_bytes(d);
}

gattn_status gattn_qcache_write(const void* k, const void* v, void* qcache, const int32_t* block_table, int num_pages,
                                int page_size, int max_pages, const int32_t* seqlens, const int32_t* cu_seqlens,
                                const void* knorm_w, int T, int B, int G, int d, int rotary_dim, double rope_base,
                                float eps, int64_t k_tok_stride, int64_t k_head_stride, int64_t v_tok_stride,
                                int64_t v_head_stride, int dtype, void* stream) {
    return write_tokens(k, v, qcache, block_table, num_pages, page_size, max_pages, seqlens, cu_seqlens, knorm_w, T, B, G,
                        d, rotary_dim, rope_base, eps, k_tok_stride, k_head_stride, v_tok_stride, v_head_stride, dtype,
                        stream, false);
}

gattn_status gattn_qcache_read(const void* qcache, const int32_t* block_table, int num_pages, int page_size,
                               int max_pages, const int32_t* starts, const int32_t* cu_seqlens, int T, int B, int G,
                               int d, int dtype, void* k, void* v, void* stream) {
    if (dtype != GATTN_BF16 && dtype != GATTN_FP32) return GATTN_ERR_INVALID_ARG;
    if (T < 0 || (!cu_seqlens && T != B)) return GATTN_ERR_INVALID_ARG;
    const gattn_status st = check_pool(qcache, block_table, num_pages, page_size, max_pages, B, G, d);
    if (st != GATTN_OK) return st;
    if (!aligned(starts, 4) || !aligned(cu_seqlens, 4)) return GATTN_ERR_INVALID_ARG;
    if (T == 0) return GATTN_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || (int64_t)T * G > ((int64_t)1 << 30))
        return GATTN_ERR_INVALID_ARG;
    QcacheReadParams p;
    std::memset(&p, 0, sizeof(p));
    if (!(p.status = device_status_word())) return GATTN_ERR_CUDA;
    p.cache = static_cast<const uint8_t*>(qcache);
    p.block_table = block_table;
    p.starts = starts;
    p.cu_seqlens = cu_seqlens;
    p.k = k;
    p.v = v;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.by_page = page_div(page_size);
    p.T = T;
    p.B = B;
    p.G = G;
    p.d = d;
    return launch_qcache_read(p, dtype == GATTN_FP32, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GATTN_OK
               : GATTN_ERR_CUDA;
}

size_t gattn_decode_qcache_workspace_size(int B, int H, int G, int d, int Lmax) {
    if (B < 1 || H < 1 || G < 1 || H % G != 0 || !head_dim_ok(d) || Lmax < 1 || Lmax > kMostTokens) return 0;
    if (!batch_ok(B, H, G, Lmax)) return 0;
    const int n = device_sm_count();
    return n > 0 ? round_up(qcache_decode_workspace(B, H, G, d, n), 256) : 0;
}

gattn_status gattn_decode_qcache(const void* q_new, const void* k_new, const void* v_new, void* qcache,
                                 const int32_t* block_table, int num_pages, int page_size, int max_pages,
                                 const int32_t* seqlens, const void* gate, const void* qnorm_w, const void* knorm_w,
                                 int B, int H, int G, int d, int rotary_dim, double rope_base, float eps,
                                 int gate_mode, int64_t q_seq_stride, int64_t q_head_stride, int64_t gate_seq_stride,
                                 int64_t gate_head_stride, void* workspace, size_t workspace_bytes, void* out,
                                 void* stream_) {
    if (!q_new || !seqlens || !qnorm_w || !out) return GATTN_ERR_INVALID_ARG;
    if (!valid_gate_mode(gate_mode) || (gate_layout(gate_mode) != GATTN_GATE_NONE && !gate))
        return GATTN_ERR_INVALID_ARG;
    if (H < 1 || G < 1 || H % G != 0) return GATTN_ERR_INVALID_ARG;
    gattn_status st = check_pool(qcache, block_table, num_pages, page_size, max_pages, B, G, d);
    if (st != GATTN_OK) return st;
    if ((st = check_rope(d, rotary_dim, rope_base, eps)) != GATTN_OK) return st;
    if (!batch_ok(B, H, G, (int64_t)max_pages * page_size)) return GATTN_ERR_UNSUPPORTED;
    if (!aligned(seqlens, 4) || !aligned(out, 16)) return GATTN_ERR_INVALID_ARG;
    const bool append = k_new || v_new;
    if (append && (!k_new || !v_new || !knorm_w)) return GATTN_ERR_INVALID_ARG;
    if (append && (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(knorm_w, 16))) return GATTN_ERR_INVALID_ARG;
    const int layout = gate_layout(gate_mode);
    const bool headwise = layout == GATTN_GATE_HEADWISE, shared = layout == GATTN_GATE_HEAD_SHARED;
    if (q_seq_stride == 0) q_seq_stride = (int64_t)H * d;
    if (q_head_stride == 0) q_head_stride = d;
    if (gate_seq_stride == 0) gate_seq_stride = headwise ? H : shared ? d : (int64_t)H * d;
    if (gate_head_stride == 0) gate_head_stride = headwise ? 1 : d;
    if (!row_strides_ok(q_new, q_seq_stride, q_head_stride, 2) || !aligned(qnorm_w, 16)) return GATTN_ERR_INVALID_ARG;
    if (layout != GATTN_GATE_NONE && (gate_seq_stride < 0 || gate_head_stride < 0 || !aligned(gate, 2)))
        return GATTN_ERR_INVALID_ARG;
    const size_t need = gattn_decode_qcache_workspace_size(B, H, G, d, max_pages * page_size);
    if (need == 0) return GATTN_ERR_CUDA;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return GATTN_ERR_WORKSPACE;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (append) {
        st = write_tokens(k_new, v_new, qcache, block_table, num_pages, page_size, max_pages, seqlens, nullptr,
                          knorm_w, B, B, G, d, rotary_dim, rope_base, eps, 0, 0, 0, 0, GATTN_BF16, stream_, true);
        if (st != GATTN_OK) return st;
    }
    QcacheDecodeParams p;
    std::memset(&p, 0, sizeof(p));
    if (!(p.status = device_status_word())) return GATTN_ERR_CUDA;
    p.q = q_new;
    p.cache = static_cast<const uint8_t*>(qcache);
    p.block_table = block_table;
    p.seqlens = seqlens;
    p.gate = gate;
    p.qnorm_w = qnorm_w;
    p.out = out;
    p.part = static_cast<float*>(workspace);
    p.q_seq_stride = q_seq_stride;
    p.q_head_stride = q_head_stride;
    p.gate_seq_stride = gate_seq_stride;
    p.gate_head_stride = gate_head_stride;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.by_page = page_div(page_size / kQcBlock);
    p.B = B;
    p.H = H;
    p.G = G;
    p.d = d;
    p.rd = rotary_dim;
    p.gate_mode = gate_mode;
    p.n_sms = device_sm_count();
    p.eps = eps;
    p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)d));
    fill_turns(p.turns, rotary_dim, rope_base);
    cudaEvent_t ev_start, ev_stop;
    profile_events(&ev_start, &ev_stop);
    return launch_qcache_decode(p, append, stream, ev_start, ev_stop) == cudaSuccess ? GATTN_OK : GATTN_ERR_CUDA;
}

}  // extern "C"
