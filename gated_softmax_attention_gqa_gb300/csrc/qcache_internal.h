// qcache_internal.h -- what the 4-bit KV cache's translation units share: launch
// parameters, launchers, and the helpers of api.cu that their entry points use.
#pragma once

#include "internal.h"

namespace gattn {

// Division of an index below 2^31 by a page's tokens or blocks: (x * mul) >> 32 >> shift, or
// x itself where mul is 0.
struct PageDiv {
    uint32_t mul, shift;
};

// 4-bit KV cache (qcache.cuh).  turns[i]: rotation of pair i per position, in 2^-64 turns.
struct QcacheWriteParams {
    const void* k;
    const void* v;
    uint8_t* cache;
    const int32_t* block_table;
    const int32_t* seqlens;
    const int32_t* cu_seqlens;  // NULL: one token per sequence
    const void* knorm_w;
    int64_t k_tok_stride, k_head_stride, v_tok_stride, v_head_stride;
    int num_pages, page_size, max_pages;
    PageDiv by_page;
    int T, B, G, d, rd;
    bool before_decode;  // the kernel launched next may be placed early
    float eps;
    unsigned int* status;
    uint64_t turns[kMaxRotaryHalf];
};
struct QcacheReadParams {
    const uint8_t* cache;
    const int32_t* block_table;
    const int32_t* starts;      // NULL: every sequence from token 0
    const int32_t* cu_seqlens;  // NULL: one token per sequence
    void* k;
    void* v;
    int num_pages, page_size, max_pages;
    PageDiv by_page;
    int T, B, G, d;
    unsigned int* status;
};
struct QcacheDecodeParams {
    const void* q;
    const uint8_t* cache;
    const int32_t* block_table;
    const int32_t* seqlens;
    const void* gate;
    const void* qnorm_w;
    void* out;
    float* part;  // partial softmax states
    int64_t q_seq_stride, q_head_stride, gate_seq_stride, gate_head_stride;
    int num_pages, page_size, max_pages;
    PageDiv by_page;  // divides a block index by the blocks of a page
    int B, H, G, d, rd, gate_mode, n_sms;
    float eps, scale_log2;
    unsigned int* status;
    uint64_t turns[kMaxRotaryHalf];
};
cudaError_t launch_qcache_write(const QcacheWriteParams& p, bool fp32, cudaStream_t stream);
cudaError_t launch_qcache_read(const QcacheReadParams& p, bool fp32, cudaStream_t stream);
size_t qcache_decode_workspace(int B, int H, int G, int d, int n_sms);
// after_write: the kernel ahead in the stream is this step's launch_qcache_write
cudaError_t launch_qcache_decode(const QcacheDecodeParams& p, bool after_write, cudaStream_t stream,
                                 cudaEvent_t ev_start, cudaEvent_t ev_stop);

// Shared by the entry points' translation units (defined in api.cu).
unsigned int* device_status_word();  // address of the status word on the current device, NULL on failure
int device_sm_count();
bool valid_gate_mode(int mode);
void profile_events(cudaEvent_t* start, cudaEvent_t* stop);

}  // namespace gattn
