// Shared internals of the attention-like token mixers: linear attention with a decay per
// head and causal softmax attention, over packed sequences and for single tokens.
#pragma once

#include "common.cuh"

namespace ssd {

// Largest head dimension of the mixers' queries, keys and values.
constexpr int kMixMaxDim = 128;

// Packed linear attention (ssd_linattn_prefill); strides are elements between tokens.
struct LinattnArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const float* log_decay;       // [heads_v]
    const float* init_states;     // [nseq][heads_v][dk][dv] or null (zeros)
    const int* cu;                // device [nseq + 1]
    int nseq, total, hq, hv, dk, dv;
    float scale;
    void* out;                    // [total][heads_v][dv]
    float* final_states;          // [nseq][heads_v][dk][dv]
};

// Packed causal attention (ssd_attn_prefill); strides are elements between tokens.
struct AttnArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const int* cu;                // device [nseq + 1]
    int nseq, total, hq, hkv, dim;
    float scale;
    void* out;                    // [total][heads_q][dim]
};

// One token per sequence against a cache (ssd_attn_decode_step).
struct AttnDecodeArgs {
    void *k_cache, *v_cache;      // [batch][capacity][heads_kv][dim]
    const int* lens;              // device [batch]
    const void *q, *k, *v;        // [batch][heads][dim]
    int batch, capacity, hq, hkv, dim;
    float scale;
    void* out;                    // [batch][heads_q][dim]
};

// ---- blocks of packed sequences ----------------------------------------------------
// The rows of sequence s are cut into blocks of Q tokens.  Numbering block j of sequence s
// as cu[s] / Q + s + j needs no table: ceil(len / Q) <= cu[s+1] / Q - cu[s] / Q + 1, so the
// ranges of successive sequences do not overlap, every sequence (an empty one too) owns at
// least one number, and there are at most total / Q + nseq of them.
__host__ __device__ inline int packed_blocks(int total, int nseq, int Q) { return total / Q + nseq; }

// a / d for 0 <= a < 2^31 and a divisor 2 <= d < 2^31 that the host knows: the kernels divide
// offsets by block lengths before their first load, where a division's instructions are cold.
struct Divisor {
    int d;
    unsigned long long inv;                          // floor(2^64 / d) + 1
    explicit Divisor(int n) : d(n), inv(~0ULL / (unsigned long long)n + 1) {}
    __device__ __forceinline__ int div(int a) const { return (int)__umul64hi((unsigned long long)(unsigned)a, inv); }
};

// Sequence, block within it, first token and sequence length of block number i, found by
// whole warps (32 offsets per round of loads).  False (and SSD_ERR_SHAPE in the error word)
// when the offsets around it are not a valid partition; a true return may still name a block
// past its sequence's end (j * Q >= len).
__device__ __forceinline__ bool packed_block(const int* __restrict__ cu, int nseq, int total, const Divisor& Q, int i,
                                             int* err, int* seq, int* j, int* first, int* len)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = nseq;                            // the largest s with cu[s] / Q + s <= i is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32, s = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, lane * step < n && Q.div(max(cu[s], 0)) + s <= i);
        const int k = below ? 31 - __clz(below) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    const int a = cu[lo], b = cu[lo + 1];
    if (!valid_offsets(a, b, total)) {
        record_error(err, SSD_ERR_SHAPE);
        return false;
    }
    *seq = lo;
    *j = i - (Q.div(a) + lo);
    *first = a;
    *len = b - a;
    return *j >= 0;
}

// Every offset, checked once by the threads of one CTA: cu[0] = 0, non-decreasing, at most
// total.  Blocks check the two offsets that they use themselves (packed_block).
__device__ __forceinline__ void check_offsets(const int* __restrict__ cu, int nseq, int total, int* err)
{
    bool bad = false;
    for (int s = threadIdx.x; s < nseq; s += blockDim.x)
        bad |= !valid_offsets(cu[s], cu[s + 1], total) || (s == 0 && cu[0] != 0);
    if (bad) record_error(err, SSD_ERR_SHAPE);
}

// g^n for g = exp(log_decay): 1 at n = 0 whatever the decay (-inf forgets everything else).
__device__ __forceinline__ float decay_pow(float log_decay, int n)
{
    return n == 0 ? 1.f : expf(log_decay * (float)n);
}

// ---- launchers -----------------------------------------------------------------------
cudaError_t launch_linattn_decode(ssd_dtype_t dtype, float* state, const void* q, const void* k, const void* v,
                                  const float* log_decay, void* out, int batch, int hq, int hv, int dk, int dv,
                                  float scale, cudaStream_t s);
// Packed prefill: bf16 on the tensor cores, fp32 on the CUDA cores.
size_t linattn_tc_workspace(int nseq, int total, int hv, int dk, int dv);
cudaError_t launch_linattn_prefill_tc(const LinattnArgs& a, void* workspace, cudaStream_t s);
size_t linattn_simt_workspace(int nseq, int total, int hv, int dk, int dv);
cudaError_t launch_linattn_prefill_simt(const LinattnArgs& a, void* workspace, cudaStream_t s);

// Tensor-core attention (bf16), for up to 128 query heads per key/value head.
bool attn_tc_supported(const AttnArgs& a);
cudaError_t launch_attn_prefill_tc(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_prefill_simt(const AttnArgs& a, ssd_dtype_t dtype, cudaStream_t s);

size_t attn_decode_workspace(int batch, int capacity, int hq, int hkv, ssd_dtype_t dtype);
cudaError_t launch_attn_decode(const AttnDecodeArgs& a, ssd_dtype_t dtype, void* workspace, cudaStream_t s);

}  // namespace ssd
