// decode_qcache.cu -- one decode step of gated GQA attention against the 4-bit KV
// cache (format: qcache.cuh).
//
// The step has to read sum(L) * 2 G d * 0.625 bytes of cache, so the design goal is the
// same as for the bf16 decode -- keep every SM streaming -- but a byte now carries 1.6
// numbers instead of half a one, and the instructions that unpack them decide how much
// of the bandwidth is reached.
//
//   qdecode_split_kernel  persistent, two to four CTAs of four warps per SM.  The (sequence,
//       KV head) pairs are cut into tiles of 128 keys (192 at d = 128) and the global tile
//       list into equal contiguous ranges, one per CTA.  Each warp owns two (three) 16-token
//       blocks of every tile: it copies their K and V bytes into a ring of its own with
//       bulk copies, a few tiles ahead, and keeps its own softmax state, so the warps meet
//       only at the end of a piece, where they are merged in shared memory.  (A producer warp for the
//       four cost a fifth warp's registers, which the accumulators need: 128 a thread
//       spilled, and 64 sequences of 16k-32k tokens took 432 us.)
//         S^T = K Q^T   m16n8k16, fp16: sixteen keys by the H/G <= 8 queries.  Numbers below
//             2^-13 count in steps of 2^-24 in fp16, so a byte of two codes, zero-extended by
//             one byte permute, is an fp16 operand as it stands, and so is its lower code,
//             masked.  Upper codes are never taken apart: with byte = 16 upper + lower,
//             q_l lower + q_u upper = (q_u / 16) byte + (q_l - q_u / 16) lower, and the
//             queries are laid out as those two factors.  The accumulator starts at
//             -8 sum q.  Each group's sum is scaled once per key; the centres enter by one
//             more product, centre_k . (sum of q over the group), q's sums split into two
//             bf16 parts.  The weights turn into the next product's operand by a register
//             transpose (movmatrix).
//         O^T += V^T P^T   m16n8k16, bf16.  The rows are features, so the pairs an operand
//             register holds are two keys of one feature: two words of neighbouring keys
//             are interleaved by halves, once, and their bytes and lower codes masked.  A
//             bf16 below 2^-125 counts in steps of 2^-133; one multiply-add by 2^127 makes
//             (byte - 136) / 64 and (lower - 8) / 64, exact, which are rows 8-15 and 0-7;
//             the upper codes' sums are 4 times their difference, taken at the end.  The
//             scales multiply P instead (they are per key and group), and the centres' part,
//             sum_k p_k centre_k, is one product for all groups, in whose spare rows ones
//             sum the weights.
//       What the unpacking costs the ALU decides:
//       with every nibble shifted down and or-ed into a power of two (28 instructions for 16
//       keys of a group) 64 sequences of 16k-32k tokens, d = 256, took 181 us and 4 of
//       60k-131k, d = 128, 55 us; with bytes and lower codes (18) 168 and 49.
//       Measured: 64 sequences of 16k-32k tokens, 2 heads of 256 (1.08 GB), 166 us with the
//       combine, 6.5 TB/s, 0.96 of a copy; 4 of 60k-131k, 4 of 128 (0.25 GB), 47 us, 5.4 TB/s.
//       Of that 8 to 13 us are the call's own (lengths, search, first copies, queries, merge,
//       combine, and the more pieces the more); what lies above goes at the rate of a copy at
//       d = 256 and d = 128: 4 of 65536, 131072 and 262144 tokens, 4 heads of 128, take 34.6,
//       58.4 and 106.5 us, their bytes 24.7, 49.5 and 98.9.  At d = 64, where what a key costs
//       whatever its length (softmax, loop, copies) is shared by half the features again, instructions
//       hold it at 0.75 of a copy: 32 of 16384, 32768 and 65536, 8 heads, take 79.6, 146.4 and
//       279.2 us, their bytes 49.5, 99.0 and 197.9.
//   qdecode_combine_kernel  merges the partial states of pieces that several CTAs share
//       and applies the gate; a (sequence, KV head) that one CTA covered is finished by
//       that CTA.  1 to 2 us behind the split kernel, of which the loads of the states are most.
#include <cuda_fp16.h>

#include "qcache.cuh"

namespace gattn {
namespace {

constexpr int NW = 4;  // warps, each with its own 16-token blocks of every tile
constexpr int THREADS = 32 * NW;
// What starting and merging a (sequence, KV head) piece costs, in tiles: the work split
// counts it, so a CTA with many short sequences gets fewer tiles.  us with one, two and three:
// 256 sequences of 100-1500 tokens, 4 x 128, 45.9, 42.4, 42.5; 48 of 1-4096, 8 x 128, 37.5, 33.4,
// 34.8; 32 of 200-2000, 8 x 128, 19.8, 19.3, 20.3; 32 of 200-3000, 4 x 256, 24.1, 23.7, 22.7.
constexpr int kPieceTiles = 2;
// What a code of one is worth as an operand of the K product: the lowest fp16 bit.
constexpr float kCode = 1.f / 16777216.f;

template <int D>
struct QdCfg {
    static constexpr int NG = D / kQcGroup;             // scale groups
    // Blocks a warp takes at once, whose waits fill one another and which share the loads of
    // the query fragments, and CTAs an SM holds at the registers that takes.  d = 128: three
    // and three (4 sequences of 60k-131k tokens 47.6 us, 32 of 200-2000 20.1) rather than two
    // and four (48.9, 23.9) or four and two (47.8, 21.7); d = 64: two and four (200 of 0-300
    // 14.5 us) rather than four and three (15.9).
    static constexpr int NB = D == 128 ? 3 : 2;
    static constexpr int CTAS_PER_SM = D == 256 ? 2 : D == 128 ? 3 : 4;
    static constexpr int BT = NW * NB * kQcBlock;       // keys per tile
    static constexpr int BLOCK_BYTES = 10 * D;          // one 16-token block
    static constexpr int STAGE_BYTES = 2 * NB * BLOCK_BYTES;  // a warp's K and V blocks
    static constexpr int MAX_STAGES = 8;                // per warp
    static constexpr int OROW = D + 4;                  // floats per row of the merge buffer (banks)
    // shared memory: the warps' rings (NW * stages), then
    static constexpr int OFF_QF = 0;                         // uint4 [NG][32] B fragments of the queries
    static constexpr int OFF_CINIT = OFF_QF + NG * 512;      // float [NG][4][4] accumulator start of heads 2t, 2t+1, twice
    static constexpr int OFF_QSUM = OFF_CINIT + NG * 64;     // bf16 [2][8 heads][8 groups], high and low parts
    static constexpr int OFF_QSC = OFF_QSUM + 256;           // float [8] logit scale of a head
    static constexpr int OFF_ML = OFF_QSC + 32;              // float [NW][8][2] the warps' (max, sum)
    static constexpr int OFF_BAR = OFF_ML + NW * 64;         // mbarrier [NW][MAX_STAGES]
    static constexpr int OFF_MISC = OFF_BAR + NW * 8 * MAX_STAGES;
    static constexpr int OFF_RED = OFF_MISC + 16;            // int [NW][2] scan scratch
    static constexpr int OFF_OBUF = OFF_RED + 32;            // float [r][OROW]; the sine table (rd/2 float2) before it
};

// What a CTA keeps of the batch in shared memory.
struct Sequences {
    int* tiles;     // [B + 1] tiles of the sequences ahead of each (one KV head)
    int* lens;      // [B]
    uint16_t* live; // [B + 1] sequences with any tile ahead of each
    __host__ __device__ static int bytes(int B) { return 4 * (B + 1) + 4 * B + 2 * (B + 2); }
    __device__ Sequences(uint8_t* at, int B) {
        tiles = reinterpret_cast<int*>(at);
        lens = tiles + B + 1;
        live = reinterpret_cast<uint16_t*>(lens + B);
    }
};

// Bytes of the merge buffer / sine table, and of everything behind the rings.
template <int D>
__host__ __device__ int obuf_bytes(int r, int rd) {
    const int o = r * QdCfg<D>::OROW * 4, t = (rd / 2) * 8;
    return o > t ? o : t;
}
template <int D>
__host__ __device__ int tail_bytes(int B, int r, int rd) {
    return QdCfg<D>::OFF_OBUF + obuf_bytes<D>(r, rd) + Sequences::bytes(B);
}

template <int D>
__device__ __forceinline__ int seq_tiles(int L, int Lmax) {
    return (L >= 1 && L <= Lmax) ? (L + QdCfg<D>::BT - 1) / QdCfg<D>::BT : 0;
}

// The work split counts units: a (sequence, KV head) piece is kPieceTiles units that stand
// for starting and merging it, then one unit a tile.  CTA c of N takes the units from
// start(c) on; there are no more CTAs than units, so none between two that hold parts of a
// sequence is empty.  (The host refuses batches of 2^31 units.)
struct WorkSplit {
    int N, base, rem;
    __device__ WorkSplit(int units, int n_ctas) {
        N = units < n_ctas ? units : n_ctas;
        base = N ? units / N : 0;
        rem = units - base * N;
    }
    __device__ int start(int c) const { return c * base + min(c, rem); }
    __device__ int owner(int u) const {  // the CTA that holds unit u
        const int wide = rem * (base + 1);
        return u < wide ? u / (base + 1) : rem + (u - wide) / base;
    }
};

// Fills `q` for the whole batch; all threads.  first_len: the length of sequence threadIdx.x.
template <int D>
__device__ void scan_batch(const int32_t* seqlens, int first_len, int B, int Lmax, const Sequences& q, int* red) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) q.tiles[0] = q.live[0] = 0;
    int tiles0 = 0, live0 = 0;
    for (int first = 0; first < B; first += THREADS) {
        const int i = first + tid, L = first == 0 ? first_len : i < B ? seqlens[i] : 0;
        int v = seq_tiles<D>(L, Lmax);
        const uint32_t any = __ballot_sync(0xffffffffu, v > 0);
        const int n = __popc(any & ((2u << lane) - 1u));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += up;
        }
        if (lane == 31) {
            red[2 * warp] = v;
            red[2 * warp + 1] = n;
        }
        __syncthreads();
        int t = tiles0, l = live0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w == warp && i < B) {
                q.tiles[i + 1] = t + v;
                q.live[i + 1] = (uint16_t)(l + n);
                q.lens[i] = L;
            }
            t += red[2 * w];
            l += red[2 * w + 1];
        }
        tiles0 = t;
        live0 = l;
        __syncthreads();
    }
}

// Tile i of the nt of KV head g of sequence b.
struct TileAt {
    int b, g, i, nt;
};
// The first tile at or behind unit u, and how many lie ahead of it.
__device__ __forceinline__ TileAt first_tile(int u, const Sequences& q, int B, int G, int& ahead) {
    int lo = 0, hi = B - 1;  // largest b with G * units(b) <= u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (G * (q.tiles[mid] + kPieceTiles * q.live[mid]) <= u) lo = mid; else hi = mid - 1;
    }
    TileAt t;
    t.b = lo;
    t.nt = q.tiles[lo + 1] - q.tiles[lo];
    const int rel = u - G * (q.tiles[lo] + kPieceTiles * q.live[lo]);
    t.g = (int)((unsigned)rel / (unsigned)(t.nt + kPieceTiles));
    t.i = max(rel - t.g * (t.nt + kPieceTiles) - kPieceTiles, 0);
    ahead = G * q.tiles[lo] + (t.nt ? t.g * t.nt + t.i : 0);  // nt = 0: past the last piece
    return t;
}
// Tile x of the batch.
__device__ __forceinline__ TileAt tile_at(int x, const Sequences& q, int B, int G) {
    int lo = 0, hi = B - 1;  // largest b with G * tiles[b] <= x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (G * q.tiles[mid] <= x) lo = mid; else hi = mid - 1;
    }
    TileAt t;
    t.b = lo;
    t.nt = q.tiles[lo + 1] - q.tiles[lo];
    const int rel = x - G * q.tiles[lo];
    t.g = (int)((unsigned)rel / (unsigned)t.nt);
    t.i = rel - t.g * t.nt;
    return t;
}

// Floats of one partial state: the output rows, then the heads' maxima and sums.
__host__ __device__ __forceinline__ int state_floats(int r, int d) { return (r * d + 2 * r + 3) & ~3; }

// D[16x8] = A[16x16] * B[16x8] + C, fp16 inputs.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
// Transpose of an 8x8 matrix of 16-bit elements spread over the warp, two a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
template <typename T>
__device__ __forceinline__ T ld(const uint8_t* p) {
    return *reinterpret_cast<const T*>(p);
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float round_f16(float x) { return __half2float(__float2half_rn(x)); }

// The gate's logit for feature e of head h, and its application to an output value.
__device__ __forceinline__ float gate_logit(const QcacheDecodeParams& p, int b, int h, int e) {
    const int layout = gate_layout(p.gate_mode);
    if (layout == GATTN_GATE_NONE) return 0.f;
    const bf16* gp = static_cast<const bf16*>(p.gate) + b * p.gate_seq_stride;
    return __bfloat162float(layout == GATTN_GATE_ELEMENTWISE ? gp[h * p.gate_head_stride + e]
                            : layout == GATTN_GATE_HEADWISE  ? gp[h * p.gate_head_stride]
                                                             : gp[e]);
}
__device__ __forceinline__ float gate_apply(int mode, float z, float o) {
    if (gate_layout(mode) == GATTN_GATE_NONE) return o;
    const float a = gate_act(z, sigmoidf_dev(z), mode);
    return gate_additive(mode) ? o + a : o * a;
}
// Four neighbouring output values.
__device__ __forceinline__ void gated4(const QcacheDecodeParams& p, int b, int h, int e, float (&o)[4]) {
    const int layout = gate_layout(p.gate_mode);
    if (layout == GATTN_GATE_NONE) return;
    const bf16* gp = static_cast<const bf16*>(p.gate) + b * p.gate_seq_stride;
    if (layout != GATTN_GATE_HEAD_SHARED) gp += h * p.gate_head_stride;
    const int step = layout == GATTN_GATE_HEADWISE ? 0 : 1;
    if (step) gp += e;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = gate_apply(p.gate_mode, __bfloat162float(gp[k * step]), o[k]);
}

template <int D>
struct QueryLanes {
    static constexpr int LPH = D / 8, HPW = 32 / LPH;  // lanes per head, heads per warp and pass
};
// Brings the gate logits of heads h0 .. h0 + r - 1 into L2, a line of 64 a lane.
template <int D>
__device__ __forceinline__ void prefetch_gate(const QcacheDecodeParams& p, int b, int h0, int r, int lane) {
    const int layout = gate_layout(p.gate_mode);
    if (layout == GATTN_GATE_NONE) return;
    const int lines = layout == GATTN_GATE_HEADWISE ? 1 : D / 64, h = layout == GATTN_GATE_HEAD_SHARED ? 0 : h0 + lane / lines;
    if (lane < (layout == GATTN_GATE_HEAD_SHARED ? 1 : r) * lines)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const bf16*>(p.gate) + b * p.gate_seq_stride +
                                                      h * p.gate_head_stride + lane % lines * 64));
}

// This lane's eight features of query head h of a KV head (head 0's for one past the last).
template <int D>
__device__ __forceinline__ uint4 load_query(const QcacheDecodeParams& p, int b, int g, int h) {
    const int r = p.H / p.G;
    return *reinterpret_cast<const uint4*>(static_cast<const bf16*>(p.q) + b * p.q_seq_stride +
                                           (int64_t)(g * r + (h < r ? h : 0)) * p.q_head_stride +
                                           8 * (threadIdx.x % QueryLanes<D>::LPH));
}
template <int D>
__device__ __forceinline__ uint4 load_first_query(const QcacheDecodeParams& p, int b, int g) {
    return load_query<D>(p, b, g, (int)threadIdx.x / QueryLanes<D>::LPH);
}
// The queries of one piece as B fragments (all threads).  A thread takes eight
// neighbouring features of a head; q' is scaled by a power of two that brings the
// head's largest |q'| into [0.5, 1), so any norm weights fit fp16, and the power goes
// into the logit scale.  Two of the four operand registers of a group hold q / 16
// (the codes they meet sit one nibble higher).
template <int D>
__device__ void make_queries(const QcacheDecodeParams& p, int b, int g, int pos, uint4 qraw, uint4 wraw, uint8_t* tail) {
    using C = QdCfg<D>;
    constexpr int LPH = QueryLanes<D>::LPH, HPW = QueryLanes<D>::HPW;
    const int r = p.H / p.G, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float2* table = reinterpret_cast<float2*>(tail + C::OFF_OBUF);
    const int u = lane % LPH, e0 = 8 * u;
    __syncthreads();  // the previous piece has left the fragments and the merge buffer
    for (int i = tid; i < (p.rd >> 1); i += THREADS) {
        float s, c;
        rope_turn_sincos(p.turns[i], pos, &s, &c);
        table[i] = make_float2(s, c);
    }
    __syncthreads();
    const int half = p.rd >> 1;
    for (int h0 = warp * HPW; h0 < r; h0 += NW * HPW) {
        const int h = h0 + lane / LPH;
        const bool live = h < r;
        float x[8], w[8], ss = 0.f;
        unpack8(qraw, x);
        unpack8(wraw, w);
        if (h0 + NW * HPW < r) qraw = load_query<D>(p, b, g, h + NW * HPW);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            ss = fmaf(x[i], x[i], ss);
            w[i] *= x[i];
        }
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rinv = inv_sqrt(ss / (float)D + p.eps);
        const bool rot = e0 < p.rd, first = e0 < half;
        const int src = rot ? lane + (first ? half >> 3 : -(half >> 3)) : lane;
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(0xffffffffu, w[i], src);
            const float2 sc = rot ? table[(first ? e0 : e0 - half) + i] : make_float2(0.f, 1.f);
            x[i] = fmaf(w[i], sc.y, o * (first ? -sc.x : sc.x)) * rinv;
            big = fmaxf(big, fabsf(x[i]));
        }
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        // 2^-k with big in [2^(k-1), 2^k); 1 for a zero or non-finite row
        const int ex = (int)((__float_as_uint(big) >> 23) & 255u);
        const bool plain = ex == 0 || ex == 255;
        const float down = plain ? 1.f : __uint_as_float((uint32_t)min(max(253 - ex, 1), 254) << 23);
        const float up = plain ? 1.f : 1.f / down;
        // a byte of two codes is met as itself and as its lower code alone, so q of the upper
        // code, over 16, multiplies the byte and is taken off the lower one's
        float qsum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float upper = round_f16(x[i + 1] * down * 0.0625f), lower = round_f16(x[i] * down - upper);
            x[i] = lower;
            x[i + 1] = upper;
            qsum += lower + 17.f * upper;  // the lower code's factor and 16 upper
        }
        qsum *= kCode;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            qsum += __shfl_xor_sync(0xffffffffu, qsum, o);
        }
        if (live) {
            const int grp = u >> 2, t = u & 3;
            reinterpret_cast<uint4*>(tail + C::OFF_QF)[grp * 32 + h * 4 + t] =
                make_uint4(pack_f16x2(x[1], x[3]), pack_f16x2(x[0], x[2]), pack_f16x2(x[5], x[7]), pack_f16x2(x[4], x[6]));
            if (t == 0) {
                float* ci = reinterpret_cast<float*>(tail + C::OFF_CINIT) + (grp * 4 + (h >> 1)) * 4 + (h & 1);
                ci[0] = ci[2] = -8.f * qsum;
                bf16* qs = reinterpret_cast<bf16*>(tail + C::OFF_QSUM);
                const bf16 hi = __float2bfloat16_rn(qsum);
                qs[h * 8 + grp] = hi;
                qs[64 + h * 8 + grp] = __float2bfloat16_rn(qsum - __bfloat162float(hi));
            }
            if (u == 0) reinterpret_cast<float*>(tail + C::OFF_QSC)[h] = p.scale_log2 * (up / kCode);
        }
    }
    __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(THREADS, QdCfg<D>::CTAS_PER_SM)
    qdecode_split_kernel(const __grid_constant__ QcacheDecodeParams p, int n_stages, bool after_write) {
    using C = QdCfg<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* tail = smem + NW * n_stages * C::STAGE_BYTES;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = p.H / p.G, Lmax = p.max_pages * p.page_size;
    const Sequences seqs(tail + C::OFF_OBUF + obuf_bytes<D>(r, p.rd), p.B);
    const uint32_t ring_u32 = smem_u32(smem) + warp * n_stages * C::STAGE_BYTES;
    uint8_t* ring = smem + warp * n_stages * C::STAGE_BYTES;
    const uint32_t bars = smem_u32(tail + C::OFF_BAR) + warp * 8 * C::MAX_STAGES;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + C::OFF_MISC);
    // After a write of the appended rows everything but the cache is ready: that kernel
    // lets this one start only once those ahead of it have finished.
    bool cache_ready = !after_write;
    auto wait_for_cache = [&]() {
        pdl_wait_prerequisites();
        fence_proxy_async_global();  // plain stores of the kernel ahead, bulk copies here
        cache_ready = true;
    };
    if (cache_ready) wait_for_cache();
    else fence_proxy_async_global();  // the rows of earlier calls were plain stores too
    pdl_launch_dependents();  // the combine kernel may become resident; it waits for this grid to finish
    const int first_len = (int)threadIdx.x < p.B ? p.seqlens[threadIdx.x] : 0;

    if (lane == 0) {
        for (int s = 0; s < n_stages; ++s) mbar_init(bars + 8 * s, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) *abort_flag = 0;
    // heads and (in the sums) groups that do not exist stay zero
    for (int i = threadIdx.x + (r < 8 ? 0 : C::OFF_QSUM / 16); i < C::OFF_ML / 16; i += THREADS)
        reinterpret_cast<uint4*>(tail)[i] = make_uint4(0, 0, 0, 0);
    scan_batch<D>(p.seqlens, first_len, p.B, Lmax, seqs, reinterpret_cast<int*>(tail + C::OFF_RED));  // ends with a block barrier

    const WorkSplit split(p.G * (seqs.tiles[p.B] + kPieceTiles * seqs.live[p.B]), gridDim.x);
    if ((int)blockIdx.x >= split.N) {
        if (!cache_ready) wait_for_cache();  // this grid's end means the end of the one ahead
        return;
    }
    // this CTA's tiles: x0 .. x0 + n_tiles - 1 of the batch; `at` is the first of the piece at hand
    int x;
    TileAt at = first_tile(split.start(blockIdx.x + (lane & 1)), seqs, p.B, p.G, x);
    const int x0 = __shfl_sync(0xffffffffu, x, 0), n_tiles = __shfl_sync(0xffffffffu, x, 1) - x0;
    at = TileAt{__shfl_sync(0xffffffffu, at.b, 0), __shfl_sync(0xffffffffu, at.g, 0), __shfl_sync(0xffffffffu, at.i, 0),
                __shfl_sync(0xffffffffu, at.nt, 0)};
    const int64_t plane = (int64_t)p.num_pages * p.G * (p.page_size / kQcBlock) * C::BLOCK_BYTES;
    const int bpp = p.page_size / kQcBlock;
    // ---- the warp's copies run n_stages tiles ahead.  Lane j holds the addresses of the
    // warp's blocks of tile x0 + 32 k + j (0: past the sequence's end), 32 tiles' table
    // entries a time.  A tile without a block for this warp still completes its stage's
    // phase, so the stages' parities flip together.
    int sent = 0;
    uint64_t src[C::NB] = {};
    uint32_t newest = 0;  // bit j: tile x0 + 32 k + j's blocks of this warp hold the sequence's last token
    uint4 qraw = {}, wraw = {};  // the piece's queries and their norm weights as loaded
    auto load_queries = [&]() {
        qraw = load_first_query<D>(p, at.b, at.g);
        wraw = reinterpret_cast<const uint4*>(p.qnorm_w)[threadIdx.x % QueryLanes<D>::LPH];
        if (warp == 0) prefetch_gate<D>(p, at.b, at.g * r, r, lane);
    };
    auto send = [&](int stage) {  // all lanes; tile x0 + sent into `stage`
        if (sent >= n_tiles) return;
        if ((sent & 31) == 0) {
#pragma unroll
            for (int j = 0; j < C::NB; ++j) src[j] = 0;
            TileAt t{at.b, at.g, at.i + sent + lane, at.nt};
            if (sent > 0 || t.i >= at.nt) t = tile_at(x0 + min(sent + lane, n_tiles - 1), seqs, p.B, p.G);
            bool last = false;
            if (sent + lane < n_tiles) {
#pragma unroll
                for (int j = 0; j < C::NB; ++j) {
                    const int blk = (t.i * NW + warp) * C::NB + j;
                    if (blk * kQcBlock < seqs.lens[t.b]) {
                        last = (blk + 1) * kQcBlock >= seqs.lens[t.b];
                        const int slot = page_of(blk, p.by_page);
                        int page = p.block_table[(int64_t)t.b * p.max_pages + slot];
                        if (page < 0 || page >= p.num_pages) {
                            atomicOr(p.status, GATTN_DEVICE_BAD_PAGE);
                            page = 0;
                        }
                        src[j] = reinterpret_cast<uint64_t>(p.cache + (((int64_t)page * p.G + t.g) * bpp + (blk - slot * bpp)) * C::BLOCK_BYTES);
                    }
                }
            }
            newest = __ballot_sync(0xffffffffu, last);
        }
        // the appended rows are being written by the kernel ahead of this one; the blocks
        // that hold none of them are copied meanwhile
        if (!cache_ready && (newest >> (sent & 31) & 1u)) wait_for_cache();
        uint64_t a[C::NB];
#pragma unroll
        for (int j = 0; j < C::NB; ++j) a[j] = __shfl_sync(0xffffffffu, src[j], sent & 31);
        if (elect_one()) {
            const uint32_t bar = bars + 8 * stage, dst = ring_u32 + stage * C::STAGE_BYTES;
            bool row = true;  // the blocks lie in a row: one copy a plane
            int n = a[0] != 0;
#pragma unroll
            for (int j = 1; j < C::NB; ++j) {
                row = row && a[j] == a[0] + j * C::BLOCK_BYTES;
                n += a[j] != 0;
            }
            if (row && a[0]) {
                mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
                bulk_load(dst, reinterpret_cast<const uint8_t*>(a[0]), C::NB * C::BLOCK_BYTES, bar);
                bulk_load(dst + C::NB * C::BLOCK_BYTES, reinterpret_cast<const uint8_t*>(a[0]) + plane,
                          C::NB * C::BLOCK_BYTES, bar);
            } else {
                mbar_arrive_expect_tx(bar, 2 * n * C::BLOCK_BYTES);
#pragma unroll
                for (int j = 0; j < C::NB; ++j) {
                    if (!a[j]) continue;
                    const uint8_t* k = reinterpret_cast<const uint8_t*>(a[j]);
                    bulk_load(dst + j * C::BLOCK_BYTES, k, C::BLOCK_BYTES, bar);
                    bulk_load(dst + (C::NB + j) * C::BLOCK_BYTES, k + plane, C::BLOCK_BYTES, bar);
                }
            }
        }
        ++sent;
    };
    if (n_tiles > 0) load_queries();  // ahead of the copies, behind which they would wait 2 us
    for (int s = 0; s < n_stages; ++s) send(s);

    const int gid = lane >> 2, t = lane & 3;
    // V words are read so that the four lanes of a quad touch different banks: the upper
    // two take the pair's second key first, and the interleave undoes it
    const int kf = 2 * t + (t >> 1), ks = 2 * t + 1 - (t >> 1);
    const uint32_t sel_lo = t < 2 ? 0x5410u : 0x1054u, sel_hi = t < 2 ? 0x7632u : 0x3276u;
    constexpr uint32_t kNibble = 0x000F000Fu, kByte = 0x00FF00FFu;
    constexpr uint32_t kUp = 0x7F007F00u, kMid = 0xBE00BE00u, kMidByte = 0xC008C008u;  // 2^127, -8/64, -136/64
    int st = 0, done = 0;  // stage and number of the unit at hand
    uint32_t phase = 0;
    bool dead = false;
    // waits for the unit at hand; a wait that runs out leaves the warp walking on without data,
    // because the block's barriers need every warp
    auto receive = [&]() {
        if (!dead && !__all_sync(0xffffffffu, mbar_try_wait(bars + 8 * st, phase)))
            dead = !__all_sync(0xffffffffu, mbar_wait(bars + 8 * st, phase, abort_flag, p.status));
        done += !dead;
    };
    auto release = [&]() {  // the warp is through with the stage: the next copy goes there
        __syncwarp();
        if (!dead) send(st);
        if (++st == n_stages) {
            st = 0;
            phase ^= 1u;
        }
    };
    for (int n = 0; n < n_tiles;) {
        const int i0 = at.i, i1 = min(at.nt, i0 + (n_tiles - n));  // this CTA's tiles of the piece
        const int L = seqs.lens[at.b];
        n += i1 - i0;
        const bool alone = i0 == 0 && i1 == at.nt;
        make_queries<D>(p, at.b, at.g, L - 1, qraw, wraw, tail);
        const float2 qsc = ld<float2>(tail + C::OFF_QSC + t * 8);
        const uint32_t qhi = ld<uint32_t>(tail + C::OFF_QSUM + gid * 16 + t * 4);
        const uint32_t qlo = ld<uint32_t>(tail + C::OFF_QSUM + 128 + gid * 16 + t * 4);
        const uint8_t* qfp = tail + C::OFF_QF + lane * 16;
        const uint8_t* cip = tail + C::OFF_CINIT + t * 16;
        float oacc[2 * C::NG][4], cacc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < 2 * C::NG; ++m) oacc[m][0] = oacc[m][1] = oacc[m][2] = oacc[m][3] = 0.f;
        // the softmax reference of heads 2t and 2t + 1, the same in every lane that holds the
        // head; the sums of the weights, as they are used, are cacc[2] and cacc[3]
        float m_run[2] = {-INFINITY, -INFINITY};

        for (int i = i0; i < i1; ++i) {
            const int key0 = (i * NW + warp) * C::NB * kQcBlock;
            receive();
            if (!dead && key0 < L) {
                constexpr int NB = C::NB, BB = C::BLOCK_BYTES;
                uint8_t* kb = ring + st * C::STAGE_BYTES;
                uint8_t* vb = kb + NB * BB;
                const bool ragged = key0 + NB * kQcBlock > L;
                if (ragged) {  // rows past the end may hold anything: no scale, no centre
#pragma unroll
                    for (int n2 = 0; n2 < NB; ++n2) {
                        uint16_t* par = reinterpret_cast<uint16_t*>(vb + n2 * BB + 8 * D);
                        for (int j = lane; j < 2 * C::NG * 16; j += 32)
                            if (key0 + n2 * kQcBlock + (j & 15) >= L) par[j] = 0;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                // ---- S^T = K Q^T: lane holds keys gid and gid + 8 of each block, heads 2t and 2t + 1
                const uint8_t* kc = kb + gid * 32 + t * 8;
                const uint8_t* kp = kb + 8 * D + gid * 2;
                float s[NB][4];
#pragma unroll
                for (int n2 = 0; n2 < NB; ++n2) {
                    uint32_t ca = 0, cb = 0;  // centres of groups 2t, 2t + 1
                    if (2 * t < C::NG) {
                        const uint8_t* c = kb + n2 * BB + 9 * D + t * 64 + gid * 2;
                        ca = ld<uint16_t>(c) | ((uint32_t)ld<uint16_t>(c + 32) << 16);
                        cb = ld<uint16_t>(c + 16) | ((uint32_t)ld<uint16_t>(c + 48) << 16);
                    }
                    s[n2][0] = s[n2][1] = s[n2][2] = s[n2][3] = 0.f;
                    mma_bf16_16816(s[n2], ca, cb, ca, cb, qhi, qlo);
                }
#pragma unroll
                for (int sl = 0; sl < D / 64; ++sl) {
                    uint2 wa[NB], wb[NB];
#pragma unroll
                    for (int n2 = 0; n2 < NB; ++n2) {
                        wa[n2] = ld<uint2>(kc + n2 * BB + sl * 512);
                        wb[n2] = ld<uint2>(kc + n2 * BB + sl * 512 + 256);
                    }
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int grp = 2 * sl + hf;
                        const uint4 qf = ld<uint4>(qfp + grp * 512);
                        const float4 ci = ld<float4>(cip + grp * 64);
                        const uint32_t sel = hf ? 0x4342 : 0x4140;  // the half's two bytes, zero-extended
#pragma unroll
                        for (int n2 = 0; n2 < NB; ++n2) {
                            const uint32_t x0 = __byte_perm(wa[n2].x, 0, sel), x1 = __byte_perm(wb[n2].x, 0, sel);
                            const uint32_t y0 = __byte_perm(wa[n2].y, 0, sel), y1 = __byte_perm(wb[n2].y, 0, sel);
                            float a[4];
                            mma_f16_16816(a, x0, x1, x0 & kNibble, x1 & kNibble, qf.x, qf.y, ci.x, ci.y, ci.z, ci.w);
                            mma_f16_16816(a, y0, y1, y0 & kNibble, y1 & kNibble, qf.z, qf.w, a[0], a[1], a[2], a[3]);
                            const uint8_t* kpn = kp + n2 * BB + grp * 32;
                            const float s0 = __uint_as_float((uint32_t)ld<uint16_t>(kpn) << 16);
                            const float s1 = __uint_as_float((uint32_t)ld<uint16_t>(kpn + 16) << 16);
                            s[n2][0] = fmaf(s0, a[0], s[n2][0]);
                            s[n2][1] = fmaf(s0, a[1], s[n2][1]);
                            s[n2][2] = fmaf(s1, a[2], s[n2][2]);
                            s[n2][3] = fmaf(s1, a[3], s[n2][3]);
                        }
                    }
                }
                float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int n2 = 0; n2 < NB; ++n2) {
                    s[n2][0] *= qsc.x;
                    s[n2][1] *= qsc.y;
                    s[n2][2] *= qsc.x;
                    s[n2][3] *= qsc.y;
                    if (ragged) {
                        const int key = key0 + n2 * kQcBlock + gid;
                        if (key >= L) s[n2][0] = s[n2][1] = -INFINITY;
                        if (key + 8 >= L) s[n2][2] = s[n2][3] = -INFINITY;
                    }
                    t0 = fmaxf(t0, fmaxf(s[n2][0], s[n2][2]));
                    t1 = fmaxf(t1, fmaxf(s[n2][1], s[n2][3]));
                }
                // ---- online softmax; the reference moves only when some logit is 2^8 above it
                if (__any_sync(0xffffffffu, t0 > m_run[0] + 8.f || t1 > m_run[1] + 8.f)) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, o));
                        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, o));
                    }
                    t0 = fmaxf(t0, m_run[0]);
                    t1 = fmaxf(t1, m_run[1]);
                    const float a0 = t0 == m_run[0] ? 1.f : ex2_approx(m_run[0] - t0);
                    const float a1 = t1 == m_run[1] ? 1.f : ex2_approx(m_run[1] - t1);
                    m_run[0] = t0;
                    m_run[1] = t1;
#pragma unroll
                    for (int m = 0; m < 2 * C::NG; ++m) {
                        oacc[m][0] *= a0;
                        oacc[m][1] *= a1;
                        oacc[m][2] *= a0;
                        oacc[m][3] *= a1;
                    }
                    cacc[0] *= a0;
                    cacc[1] *= a1;
                    cacc[2] *= a0;
                    cacc[3] *= a1;
                }
                uint32_t pr[NB][2];
#pragma unroll
                for (int n2 = 0; n2 < NB; ++n2)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t w =
                            pack_bf16x2(ex2_approx(s[n2][2 * k] - m_run[0]), ex2_approx(s[n2][2 * k + 1] - m_run[1]));
                        pr[n2][k] = transpose8x8(w);  // head gid, keys 8k + 2t, 8k + 2t + 1
                    }
                // ---- centres: row g of A is group g; rows 8 and on are ones and sum the weights
#pragma unroll
                for (int n2 = 0; n2 < NB; ++n2) {
                    const uint8_t* ca = vb + n2 * BB + 9 * D + gid * 32 + t * 4;
                    uint32_t a0 = 0, a2 = 0;
                    if (gid < C::NG) {
                        a0 = ld<uint32_t>(ca);
                        a2 = ld<uint32_t>(ca + 16);
                    }
                    mma_bf16_16816(cacc, a0, 0x3F803F80u, a2, 0x3F803F80u, pr[n2][0], pr[n2][1]);
                }
                // ---- O^T += V^T P^T
                const uint8_t* vf = vb + gid * 4 + kf * 32;
                const uint8_t* vs = vb + gid * 4 + ks * 32;
                const uint8_t* vp = vb + 8 * D + t * 4;
#pragma unroll
                for (int sl = 0; sl < D / 64; ++sl) {
#pragma unroll
                    for (int n2 = 0; n2 < NB; ++n2) {
                        const int off = n2 * BB + sl * 512;
                        const uint32_t f0 = ld<uint32_t>(vf + off), s0 = ld<uint32_t>(vs + off);
                        const uint32_t f1 = ld<uint32_t>(vf + off + 256), s1 = ld<uint32_t>(vs + off + 256);
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const int grp = 2 * sl + hf;
                            const uint32_t sel = hf ? sel_hi : sel_lo;
                            const uint32_t w0 = __byte_perm(f0, s0, sel), w1 = __byte_perm(f1, s1, sel);
                            const uint32_t b0[2] = {w0 & kByte, __byte_perm(w0, 0, 0x4341)};
                            const uint32_t b1[2] = {w1 & kByte, __byte_perm(w1, 0, 0x4341)};
                            const uint8_t* vpn = vp + n2 * BB + grp * 32;
                            // the weights' second rounding to bf16 (the first made pr): each is at most
                            // half a step, 2^-8 of the value, and errors of many keys average
                            const uint32_t p0 = mul_bf16x2(pr[n2][0], ld<uint32_t>(vpn));
                            const uint32_t p1 = mul_bf16x2(pr[n2][1], ld<uint32_t>(vpn + 16));
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                // (lower - 8) / 64 in rows 0-7, (byte - 136) / 64 in rows 8-15
                                const uint32_t a0 = fma_bf16x2((m ? b0[1] : w0) & kNibble, kUp, kMid);
                                const uint32_t a1 = fma_bf16x2(b0[m], kUp, kMidByte);
                                const uint32_t a2 = fma_bf16x2((m ? b1[1] : w1) & kNibble, kUp, kMid);
                                const uint32_t a3 = fma_bf16x2(b1[m], kUp, kMidByte);
                                mma_bf16_16816(oacc[2 * grp + m], a0, a1, a2, a3, p0, p1);
                            }
                        }
                    }
                }
            }
            release();
        }

        // -------- end of the piece: merge the four warps, then finish or hand over
        float* ml = reinterpret_cast<float*>(tail + C::OFF_ML);
        if (gid == 0) reinterpret_cast<float4*>(ml)[warp * 4 + t] = make_float4(m_run[0], cacc[2], m_run[1], cacc[3]);
        // Merged maximum and sum of head h, and the weights of the warps' states.  A weight of zero
        // multiplies its state like any other: the maximum passes over NaN logits (a warp that met
        // only such has -infinity, as one without keys, whose state is zeros), so that a NaN
        // reaches the output through the sums wherever its key lies in the work split.
        auto weights = [&](int h, float (&f)[NW], float& mx, float& l) {
            float2 v[NW];
            mx = -INFINITY;
            l = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                v[w] = reinterpret_cast<const float2*>(ml)[w * 8 + h];
                mx = fmaxf(mx, v[w].x);
            }
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                f[w] = v[w].x == -INFINITY ? 0.f : ex2_approx(v[w].x - mx);
                l += f[w] * v[w].y;
            }
        };
        // features 4 gid' .. of row tile m and head 2t + e as a pair
        auto place = [&](float* rows, int m, int e) {
            return reinterpret_cast<float2*>(rows + (2 * t + e) * C::OROW + (m >> 1) * 32 + gid * 4 + (m & 1) * 2);
        };
        // the state's own pair there: rows 0-7 lower codes, 8-15 bytes, and the centres' part
        auto own = [&](int m, int e) {
            const float c0 = __shfl_sync(0xffffffffu, cacc[0], 4 * (m >> 1) + t);
            const float c1 = __shfl_sync(0xffffffffu, cacc[1], 4 * (m >> 1) + t);
            const float c = e ? c1 : c0;
            return make_float2(fmaf(64.f, oacc[m][e], c), fmaf(4.f, oacc[m][2 + e] - oacc[m][e], c));
        };
        auto finish = [&](auto merged) {  // merged(h, e): features e .. e + 3 of head h
            bf16* out = static_cast<bf16*>(p.out) + ((int64_t)at.b * p.H + at.g * r) * D;
            float* ps = p.part + ((int64_t)blockIdx.x + (int64_t)at.b * p.G + at.g) * state_floats(r, D);
            for (int j = 4 * threadIdx.x; j < r * D; j += 4 * THREADS) {
                const int h = j / D, e = j % D;
                float mx, l;
                const float4 o = merged(h, e, mx, l);
                if (alone) {
                    l = 1.f / l;
                    float v[4] = {o.x * l, o.y * l, o.z * l, o.w * l};
                    gated4(p, at.b, at.g * r + h, e, v);
                    *reinterpret_cast<uint2*>(out + j) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                } else {
                    *reinterpret_cast<float4*>(ps + j) = o;
                    if (e == 0) {
                        ps[r * D + h] = mx;
                        ps[r * D + r + h] = l;
                    }
                }
            }
        };
        if (n >= n_tiles) {
            // the CTA's last piece: each warp lays its state into its ring, which is done with
            float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
            for (int m = 0; m < 2 * C::NG; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 o = own(m, e);
                    if (2 * t + e < r) *place(mine, m, e) = o;
                }
            __syncthreads();
            finish([&](int h, int e, float& mx, float& l) {
                float f[NW];
                weights(h, f, mx, l);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float4 a = *reinterpret_cast<const float4*>(smem + w * n_stages * C::STAGE_BYTES + (h * C::OROW + e) * 4);
                    o.x = fmaf(f[w], a.x, o.x);
                    o.y = fmaf(f[w], a.y, o.y);
                    o.z = fmaf(f[w], a.z, o.z);
                    o.w = fmaf(f[w], a.w, o.w);
                }
                return o;
            });
            break;
        }
        // the rings hold the next piece's blocks: four rounds over one buffer, in each of which
        // the warps add to different quarters of the features, loads first
        float* obuf = reinterpret_cast<float*>(tail + C::OFF_OBUF);
        __syncthreads();
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float all[NW], mx, l;
            weights(2 * t + e, all, mx, l);
            f[e] = warp == 0 ? all[0] : warp == 1 ? all[1] : warp == 2 ? all[2] : all[3];
        }
        constexpr int MQ = C::NG / 2;  // row tiles a quarter
#pragma unroll 1
        for (int k = 0; k < NW; ++k) {
            const int quarter = (warp + k) & 3;
#pragma unroll
            for (int qt = 0; qt < 4; ++qt) {
                if (qt != quarter) continue;
                float2 o[MQ][2];
#pragma unroll
                for (int i = 0; i < MQ; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        o[i][e] = k && 2 * t + e < r ? *place(obuf, qt * MQ + i, e) : make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < MQ; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 a = own(qt * MQ + i, e);
                        o[i][e].x = fmaf(f[e], a.x, o[i][e].x);
                        o[i][e].y = fmaf(f[e], a.y, o[i][e].y);
                        if (2 * t + e < r) *place(obuf, qt * MQ + i, e) = o[i][e];
                    }
            }
            __syncthreads();
        }
        finish([&](int h, int e, float& mx, float& l) {
            float all[NW];
            weights(h, all, mx, l);
            return *reinterpret_cast<const float4*>(obuf + h * C::OROW + e);
        });
        // the next piece: the next KV head, or the next sequence that holds anything
        at.i = 0;
        if (++at.g == p.G) {
            at.g = 0;
            do { ++at.b; } while (seqs.tiles[at.b + 1] == seqs.tiles[at.b]);  // there is one: tiles are left
            at.nt = seqs.tiles[at.b + 1] - seqs.tiles[at.b];
        }
        load_queries();
    }
    if (!cache_ready) wait_for_cache();
    // every copy that was sent lands before the block leaves (none is left unless a wait ran out)
    for (; done < sent; ++done) mbar_wait_drain(bars + 8 * (done % n_stages), (uint32_t)(done / n_stages) & 1u, p.status);
}

// Merge the partial states of one (sequence, query head) that several CTAs share and
// apply the gate: warp w of NWC sums every NWC-th state, lane l owning D / 32 features, and
// the warps meet in shared memory.  States of weight zero take part (their NaN do).  A
// sequence of length 0 gets the gate of an empty sum.
template <int D, int NWC>
__global__ void __launch_bounds__(32 * NWC) qdecode_combine_kernel(const __grid_constant__ QcacheDecodeParams p, int n_ctas) {
    constexpr int DPL = D / 32, VEC = DPL < 4 ? DPL : 4, CH = NWC == 8 ? 8 : 4, EPT = (D + 32 * NWC - 1) / (32 * NWC);
    struct alignas(4 * VEC) Vec {
        float v[VEC];
    };
    __shared__ float sm[NWC][2];
    __shared__ __align__(16) float so[NWC][D];
    __shared__ int units[NWC][2];
    const int b = blockIdx.x / p.H, hq = blockIdx.x % p.H;
    const int r = p.H / p.G, g = hq / r, h = hq % r, Lmax = p.max_pages * p.page_size;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int L = p.seqlens[b], nt = seq_tiles<D>(L, Lmax);
    int before = 0, total = 0;  // units ahead of this sequence, and of all (one KV head)
    for (int i = threadIdx.x; i < p.B; i += 32 * NWC) {
        const int n = seq_tiles<D>(p.seqlens[i], Lmax), u = n ? n + kPieceTiles : 0;
        total += u;
        if (i < b) before += u;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) {
        units[warp][0] = before;
        units[warp][1] = total;
    }
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int w = 0; w < NWC; ++w) {
        before += units[w][0];
        total += units[w][1];
    }
    bf16* out = static_cast<bf16*>(p.out) + ((int64_t)b * p.H + hq) * D;
    float z[EPT];  // the gate of features threadIdx.x + k 32 NWC
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
        const int e = threadIdx.x + k * 32 * NWC;
        z[k] = e < D ? gate_logit(p, b, hq, e) : 0.f;
    }
    int n_slots = 0, c0 = 0;
    if (nt) {
        const WorkSplit split(p.G * total, n_ctas);
        const int u0 = p.G * before + g * (nt + kPieceTiles) + kPieceTiles;  // the first tile's unit
        c0 = split.owner(u0);
        n_slots = split.owner(u0 + nt - 1) - c0 + 1;
    }
    const int64_t stride = state_floats(r, D);
    const float* part0 = p.part + ((int64_t)c0 + (int64_t)b * p.G + g) * stride;

    // Everything above reads only the inputs.  Every block waits for the split kernel before
    // it leaves: this grid's end then means both.
    pdl_wait_prerequisites();
    if (nt == 0) {
        if (L == 0) {
#pragma unroll
            for (int k = 0; k < EPT; ++k)
                if (threadIdx.x + k * 32 * NWC < D)
                    out[threadIdx.x + k * 32 * NWC] = __float2bfloat16_rn(gate_apply(p.gate_mode, z[k], 0.f));
        } else if (threadIdx.x == 0 && hq == 0) {
            atomicOr(p.status, GATTN_DEVICE_BAD_SEQLEN);
        }
        return;
    }
    if (n_slots == 1) return;  // one CTA covered and finished it
    float m_run = -INFINITY, den = 0.f, num[DPL];
#pragma unroll
    for (int k = 0; k < DPL; ++k) num[k] = 0.f;
    for (int s0 = warp; s0 < n_slots; s0 += CH * NWC) {
        float ms[CH], ls[CH], os[CH][DPL];
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int s = s0 + j * NWC;
            const bool live = s < n_slots;
            const float* ps = part0 + (live ? s : 0) * stride;
            ms[j] = live ? ps[r * D + h] : -INFINITY;
            ls[j] = live ? ps[r * D + r + h] : 0.f;
#pragma unroll
            for (int k = 0; k < DPL / VEC; ++k) {
                Vec x = {};
                if (live) x = reinterpret_cast<const Vec*>(ps + h * D)[lane + 32 * k];
#pragma unroll
                for (int i = 0; i < VEC; ++i) os[j][k * VEC + i] = x.v[i];
            }
        }
        float mx = m_run;
#pragma unroll
        for (int j = 0; j < CH; ++j) mx = fmaxf(mx, ms[j]);
        const float keep = m_run == -INFINITY ? 0.f : ex2_approx(m_run - mx);
        den *= keep;
#pragma unroll
        for (int k = 0; k < DPL; ++k) num[k] *= keep;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const float w = ms[j] == -INFINITY ? 0.f : ex2_approx(ms[j] - mx);
            den = fmaf(w, ls[j], den);
#pragma unroll
            for (int k = 0; k < DPL; ++k) num[k] = fmaf(w, os[j][k], num[k]);
        }
        m_run = mx;
    }
    if (lane == 0) {
        sm[warp][0] = m_run;
        sm[warp][1] = den;
    }
#pragma unroll
    for (int k = 0; k < DPL / VEC; ++k) {
        Vec x;
#pragma unroll
        for (int i = 0; i < VEC; ++i) x.v[i] = num[k * VEC + i];
        reinterpret_cast<Vec*>(so[warp])[lane + 32 * k] = x;
    }
    __syncthreads();
    float mx = -INFINITY, l = 0.f, f[NWC];
#pragma unroll
    for (int w = 0; w < NWC; ++w) mx = fmaxf(mx, sm[w][0]);
#pragma unroll
    for (int w = 0; w < NWC; ++w) {
        f[w] = sm[w][0] == -INFINITY ? 0.f : ex2_approx(sm[w][0] - mx);
        l += f[w] * sm[w][1];
    }
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
        const int e = threadIdx.x + k * 32 * NWC;
        if (e >= D) break;
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < NWC; ++w) o += f[w] * so[w][e];
        out[e] = __float2bfloat16_rn(gate_apply(p.gate_mode, z[k], o / l));
    }
}

template <int D>
cudaError_t launch_d(const QcacheDecodeParams& p, bool after_write, cudaStream_t stream, cudaEvent_t ev_start,
                     cudaEvent_t ev_stop) {
    using C = QdCfg<D>;
    // no more CTAs than units the batch can have (one sequence of 500: 8.8 us with all, 8.5 with 14)
    const int64_t most = (int64_t)p.B * p.G * ((p.max_pages * p.page_size + C::BT - 1) / C::BT + kPieceTiles);
    const int n_ctas = (int)(most < C::CTAS_PER_SM * p.n_sms ? most : C::CTAS_PER_SM * p.n_sms);
    // ring depth: what an SM's 228 KB (1 KB of it reserved per CTA) leave for each warp
    const int tail = tail_bytes<D>(p.B, p.H / p.G, p.rd);
    int stages = ((228 * 1024) / C::CTAS_PER_SM - 1024 - tail) / (NW * C::STAGE_BYTES);
    stages = stages < 2 ? 2 : stages > C::MAX_STAGES ? C::MAX_STAGES : stages;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(qdecode_split_kernel<D>), 227 * 1024);
    if (e != cudaSuccess) return e;
    if (ev_start) cudaEventRecord(ev_start, stream);
    e = launch_early(qdecode_split_kernel<D>, dim3((unsigned)n_ctas), dim3(THREADS),
                     (size_t)(NW * stages * C::STAGE_BYTES + tail), stream, p, stages, after_write);
    if (ev_stop) cudaEventRecord(ev_stop, stream);
    if (e != cudaSuccess) return e;
    // Eight warps share a head's states where a sequence may be spread over many CTAs, two
    // where there are about as many (sequence, KV head) pairs as CTAs and so a state or two
    // each.  us with two and eight: one sequence of 32768 tokens, 2 x 256, 32.3, 15.6; one of 131072,
    // 4 x 128, 30.4, 23.6; 8 of 8192, 2 x 256, 17.1, 15.9; 200 of 0-300, 4 x 64, 13.8, 18.9; 32 of
    // 200-2000, 8 x 128, 19.2, 22.9.  Between, at two to five CTAs a pair, two would often do:
    // 64 of 16k-32k, 2 x 256, 163.9, 166.8; 32 of 8k-32k, 8 x 64, 89.7, 93.1; 32 of 200-3000, 4 x 256,
    // 22.5, 23.8; but 4 of 60k-131k, 4 x 128, 48.8, 46.6.
    const dim3 heads((unsigned)(p.B * p.H));
    if ((int64_t)p.B * p.G * 2 <= n_ctas)
        return launch_early(qdecode_combine_kernel<D, 8>, heads, dim3(256), 0, stream, p, n_ctas);
    return launch_early(qdecode_combine_kernel<D, 2>, heads, dim3(64), 0, stream, p, n_ctas);
}

}  // namespace

size_t qcache_decode_workspace(int B, int H, int G, int d, int n_sms) {
    const int per_sm = d == 256   ? QdCfg<256>::CTAS_PER_SM
                       : d == 128 ? QdCfg<128>::CTAS_PER_SM
                                  : QdCfg<64>::CTAS_PER_SM;
    const int r = H / G;
    return ((size_t)per_sm * n_sms + (size_t)B * G) * (size_t)state_floats(r, d) * sizeof(float);
}

cudaError_t launch_qcache_decode(const QcacheDecodeParams& p, bool after_write, cudaStream_t stream,
                                 cudaEvent_t ev_start, cudaEvent_t ev_stop) {
    switch (p.d) {
        case 64: return launch_d<64>(p, after_write, stream, ev_start, ev_stop);
        case 128: return launch_d<128>(p, after_write, stream, ev_start, ev_stop);
        case 256: return launch_d<256>(p, after_write, stream, ev_start, ev_stop);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gattn
