// Linear attention with a decay per head on the CUDA cores: the single-token step on the
// state, and the chunked prefill of fp32 tensors (bf16: linattn_tc.cu).
//
//     S_t = g S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,   g = exp(log_decay[h])
//
// with S a dk x dv matrix per value head; value head h reads query/key head h / (hv / hq).
#include "mixers.cuh"
#include "prefill_tc.h"
#include "ptx.cuh"

namespace ssd {

namespace {

// ================================================================ single-token step
// Bound by memory: 8 bytes of state traffic per element against 4 flops.  The columns of S
// are independent, so a CTA takes one (batch row, value head, block of columns); a thread
// owns 16 rows of 4 columns, issues those 16-byte loads before using any of them, updates
// and writes them back, and the partial sums of S^T q cross the row groups through shared
// memory once.  32 heads of 128 x 128: 42.6 us for 64 rows (270 MB, 6.3 TB/s), 2.3 us for one; with 128 columns a
// CTA instead of 64, 42.3 and 3.0 us.
constexpr int kStepRows = 16;                              // rows per thread

template <typename T, int kCols>
__global__ void __launch_bounds__(kCols / 4 * (kMixMaxDim / kStepRows))
linattn_decode_kernel(float* __restrict__ state, const T* __restrict__ q, const T* __restrict__ k,
                      const T* __restrict__ v, const float* __restrict__ log_decay, T* __restrict__ out, int hq,
                      int hv, int dk, int dv, float scale)
{
    constexpr int kQuads = kCols / 4;
    constexpr int kGroups = kMixMaxDim / kStepRows;
    __shared__ float4 red[kGroups][kQuads];
    const int unit = blockIdx.x, b = unit / hv, h = unit - b * hv;
    const int cq = threadIdx.x % kQuads, rg = threadIdx.x / kQuads;
    const int c0 = blockIdx.y * kCols + 4 * cq, i0 = rg * kStepRows;
    const bool col = c0 < dv;
    float* S = state + (size_t)unit * dk * dv + c0;
    float4 s[kStepRows];
#pragma unroll
    for (int r = 0; r < kStepRows; ++r)
        s[r] = (col && i0 + r < dk) ? *reinterpret_cast<const float4*>(S + (size_t)(i0 + r) * dv)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
    const size_t qk = ((size_t)b * hq + h / (hv / hq)) * dk;
    const float g = expf(log_decay[h]);
    const float4 vv = col ? load4<T>(v + (size_t)unit * dv + c0) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r4 = 0; r4 < kStepRows; r4 += 4) {
        if (i0 + r4 < dk) {                                // dk is a multiple of 8
            const float4 k4 = load4<T>(k + qk + i0 + r4), q4 = load4<T>(q + qk + i0 + r4);
            const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float4& x = s[r4 + r];
                x.x = fmaf(kk[r], vv.x, g * x.x);
                x.y = fmaf(kk[r], vv.y, g * x.y);
                x.z = fmaf(kk[r], vv.z, g * x.z);
                x.w = fmaf(kk[r], vv.w, g * x.w);
                o.x = fmaf(qq[r], x.x, o.x);
                o.y = fmaf(qq[r], x.y, o.y);
                o.z = fmaf(qq[r], x.z, o.z);
                o.w = fmaf(qq[r], x.w, o.w);
                if (col) *reinterpret_cast<float4*>(S + (size_t)(i0 + r4 + r) * dv) = x;
            }
        }
    }
    red[rg][cq] = o;
    __syncthreads();
    if (rg == 0 && col) {
        float4 t = red[0][cq];
#pragma unroll
        for (int w = 1; w < kGroups; ++w) {
            const float4 a = red[w][cq];
            t.x += a.x; t.y += a.y; t.z += a.z; t.w += a.w;
        }
        T* p = out + (size_t)unit * dv + c0;
        Elem<T>::store(p + 0, scale * t.x);
        Elem<T>::store(p + 1, scale * t.y);
        Elem<T>::store(p + 2, scale * t.z);
        Elem<T>::store(p + 3, scale * t.w);
    }
}

template <typename T>
cudaError_t decode_t(float* state, const void* q, const void* k, const void* v, const float* log_decay, void* out,
                     int batch, int hq, int hv, int dk, int dv, float scale, cudaStream_t s)
{
    constexpr int kCols = 64;
    const dim3 grid((unsigned)(batch * hv), (unsigned)((dv + kCols - 1) / kCols));
    linattn_decode_kernel<T, kCols><<<grid, kCols / 4 * (kMixMaxDim / kStepRows), 0, s>>>(
        state, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), log_decay,
        static_cast<T*>(out), hq, hv, dk, dv, scale);
    return cudaGetLastError();
}

// ================================================================ chunked prefill, CUDA cores
// Blocks of 64 tokens in three launches: every block's own state U = sum_s g^(len-1-s) k_s v_s^T
// (all blocks in parallel), a scan that turns the U into start states and writes the final
// states, and every block's output  o_t = g^(t+1) S^T q_t + sum_{s<=t} g^(t-s) (q_t.k_s) v_s.
// Each launch is a programmatic dependent of the one before.  Products run on packed fp32 pairs.
// The kernels exist for dimensions padded to 64 and to 128: 2000 tokens, 64 heads of 64 x 64: 131 us, 168 us on
// the kernels for 128 x 64.  Bound by latency where the blocks are few: 1501 tokens, 8 heads of 64 x 64, three sequences
// (192 blocks): 27 us, of which the products would take 3.  With many blocks every block's fp32 state passes
// through memory twice: the 131 us above compare with 29 us of the recurrence's operations at 72 TFLOP/s; 16384 tokens, 32
// heads of 128 x 128: 2.1 ms, of 477.
constexpr int kTok = 64;                                   // tokens per block
constexpr int kThreads = 256;
constexpr int kLdP = kTok + 4;

// `rows` rows of `cols` elements (a multiple of 4) into padded shared rows as fp32, zeros past
// them.  (Rows of D + 4 floats: 16-byte reads of 8 rows hit 8 different bank quads.)
template <typename T, int D>
__device__ __forceinline__ void load_rows(float* dst, const T* src, long long stride, int rows, int cols)
{
#pragma unroll 4
    for (int i = threadIdx.x; i < kTok * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4));
        const float4 x = (r < rows && c < cols) ? load4<T>(src + (size_t)r * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = x;
    }
}

__device__ __forceinline__ float2 lo2(const float4& x) { return make_float2(x.x, x.y); }
__device__ __forceinline__ float2 hi2(const float4& x) { return make_float2(x.z, x.w); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kThreads)
linattn_block_state_kernel(const LinattnArgs a, const Divisor block, float* states, int* err)
{
    constexpr int kLdK = DK + 4, kLdV = DV + 4, kR = DK / 16, kC = DV / 64;   // thread: kR rows, 4 kC columns
    extern __shared__ float sm[];
    __shared__ float sw[kTok];
    float *sk = sm, *sv = sm + kTok * kLdK;
    const int h = blockIdx.y, tid = threadIdx.x;
    ptx::griddep_wait();                                   // every input may come from the kernel before
    ptx::griddep_launch_dependents();                      // (only now: the next kernels read inputs at once)
    if (blockIdx.x == 0 && h == 0) check_offsets(a.cu, a.nseq, a.total, err);
    int seq, j, first, len;
    if (!packed_block(a.cu, a.nseq, a.total, block, blockIdx.x, err, &seq, &j, &first, &len)) return;
    if ((long long)j * kTok >= len) return;
    const int n = min(kTok, len - j * kTok);
    const size_t t0 = (size_t)first + (size_t)j * kTok;
    if (tid < n) sw[tid] = decay_pow(a.log_decay[h], n - 1 - tid);
    load_rows<T, DK>(sk, static_cast<const T*>(a.k) + t0 * a.k_stride + (size_t)(h / (a.hv / a.hq)) * a.dk, a.k_stride, n, a.dk);
    load_rows<T, DV>(sv, static_cast<const T*>(a.v) + t0 * a.v_stride + (size_t)h * a.dv, a.v_stride, n, a.dv);
    __syncthreads();
    // rows kR ty .. + kR - 1, columns 4 tx .. + 3 (and 64 + 4 tx .. + 3)
    const int tx = tid & 15, ty = tid >> 4;
    float2 acc[kR][kC][2];
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
        for (int c = 0; c < kC; ++c) acc[i][c][0] = acc[i][c][1] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
        const float w = sw[s];
        float kk[kR];
#pragma unroll
        for (int i = 0; i < kR; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(sk + s * kLdK + kR * ty + i);
            kk[i] = w * x.x; kk[i + 1] = w * x.y; kk[i + 2] = w * x.z; kk[i + 3] = w * x.w;
        }
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(sv + s * kLdV + 64 * c + 4 * tx);
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                acc[i][c][0] = ptx::ffma2(both(kk[i]), lo2(v), acc[i][c][0]);
                acc[i][c][1] = ptx::ffma2(both(kk[i]), hi2(v), acc[i][c][1]);
            }
        }
    }
    float* U = states + ((size_t)blockIdx.x * a.hv + h) * a.dk * a.dv;
#pragma unroll
    for (int i = 0; i < kR; ++i) {
        const int r = kR * ty + i;
#pragma unroll
        for (int c = 0; c < kC; ++c)
            if (r < a.dk && 64 * c + 4 * tx < a.dv)
                *reinterpret_cast<float4*>(U + (size_t)r * a.dv + 64 * c + 4 * tx) =
                    make_float4(acc[i][c][0].x, acc[i][c][0].y, acc[i][c][1].x, acc[i][c][1].y);
    }
}

// Start state of every block (over its U) and the final state, four elements a thread.  The
// next blocks' U are loaded ahead of the chain.
constexpr int kScanThreads = 64, kAhead = 4;

__global__ void __launch_bounds__(kScanThreads)
linattn_scan_kernel(const LinattnArgs a, float* states)
{
    const int seq = blockIdx.x / a.hv, h = blockIdx.x - seq * a.hv;
    const int e = (blockIdx.y * kScanThreads + threadIdx.x) * 4, elems = a.dk * a.dv;
    ptx::griddep_launch_dependents();
    const int first = a.cu[seq], end = a.cu[seq + 1];
    const float ld = a.log_decay[h];
    const size_t base = (size_t)blockIdx.x * elems + e;
    float4 H = a.init_states && e < elems ? *reinterpret_cast<const float4*>(a.init_states + base) : make_float4(0.f, 0.f, 0.f, 0.f);
    ptx::griddep_wait();
    if (e >= elems || !valid_offsets(first, end, a.total)) return;      // (offsets reported by the blocks)
    const int len = end - first;
    float* U = states + ((size_t)(first / kTok + seq) * a.hv + h) * elems + e;
    const size_t step = (size_t)a.hv * elems;
    const int blocks = (len + kTok - 1) / kTok;
    const float whole = decay_pow(ld, kTok);
    float4 u[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (i < blocks) u[i] = *reinterpret_cast<const float4*>(U + i * step);
    for (int t = 0; t < blocks; t += kAhead) {
        float4 next[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (t + kAhead + i < blocks) next[i] = *reinterpret_cast<const float4*>(U + (size_t)(t + kAhead + i) * step);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (t + i >= blocks) break;
            *reinterpret_cast<float4*>(U + (size_t)(t + i) * step) = H;
            const float g = t + i + 1 < blocks ? whole : decay_pow(ld, len - (t + i) * kTok);
            H.x = fmaf(g, H.x, u[i].x); H.y = fmaf(g, H.y, u[i].y); H.z = fmaf(g, H.z, u[i].z); H.w = fmaf(g, H.w, u[i].w);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) u[i] = next[i];
    }
    *reinterpret_cast<float4*>(a.final_states + base) = H;
}

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kThreads)
linattn_block_output_kernel(const LinattnArgs a, const Divisor block, const float* states, int* err)
{
    constexpr int kLdK = DK + 4, kLdV = DV + 4, kC = DV / 64;
    extern __shared__ float sm[];
    __shared__ float sg[kTok + 1];                         // g^0 .. g^64
    float *sq = sm, *sk = sq + kTok * kLdK, *sv = sk + kTok * kLdK, *sp = sv + kTok * kLdV;
    float* ss = sk;                                        // 64 rows of the start state, in the keys' place
    const int h = blockIdx.y, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    int seq, j, first, len;
    const bool valid = packed_block(a.cu, a.nseq, a.total, block, blockIdx.x, err, &seq, &j, &first, &len);
    const int n = valid && (long long)j * kTok < len ? min(kTok, len - j * kTok) : 0;
    if (n <= 0) {
        ptx::griddep_wait();                               // (this grid ends after the one before)
        return;
    }
    const size_t t0 = (size_t)first + (size_t)j * kTok;
    const size_t hk = (size_t)(h / (a.hv / a.hq)) * a.dk;
    if (tid <= kTok) sg[tid] = decay_pow(a.log_decay[h], tid);
    load_rows<T, DK>(sq, static_cast<const T*>(a.q) + t0 * a.q_stride + hk, a.q_stride, n, a.dk);
    load_rows<T, DK>(sk, static_cast<const T*>(a.k) + t0 * a.k_stride + hk, a.k_stride, n, a.dk);
    load_rows<T, DV>(sv, static_cast<const T*>(a.v) + t0 * a.v_stride + (size_t)h * a.dv, a.v_stride, n, a.dv);
    __syncthreads();
    // scores: thread rows t = 4 ty + i, columns s = tx + 16 jj
    float2 p[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) p[i][jj] = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int d = 0; d < a.dk; d += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(sq + (4 * ty + i) * kLdK + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = *reinterpret_cast<const float4*>(sk + (tx + 16 * i) * kLdK + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
                p[i][jj] = ptx::ffma2(hi2(x[i]), hi2(y[jj]), ptx::ffma2(lo2(x[i]), lo2(y[jj]), p[i][jj]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            const int t = 4 * ty + i, s = tx + 16 * jj;
            sp[t * kLdP + s] = s <= t ? (p[i][jj].x + p[i][jj].y) * sg[t - s] : 0.f;
        }
    // the carried part: acc = S^T q, 64 rows of S at a time
    const float* S = states + ((size_t)blockIdx.x * a.hv + h) * a.dk * a.dv;
    float2 acc[4][kC][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < kC; ++c) acc[i][c][0] = acc[i][c][1] = make_float2(0.f, 0.f);
    ptx::griddep_wait();                                   // the start states come from the kernel before
    for (int d0 = 0; d0 < a.dk; d0 += kTok) {
        __syncthreads();
        load_rows<float, DV>(ss, S + (size_t)d0 * a.dv, a.dv, min(kTok, a.dk - d0), a.dv);
        __syncthreads();
#pragma unroll 2
        for (int d = 0; d < min(kTok, a.dk - d0); d += 4) {        // dk is a multiple of 8
            float4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(sq + (4 * ty + i) * kLdK + d0 + d);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const float4 v = *reinterpret_cast<const float4*>(ss + (d + e) * kLdV + 64 * c + 4 * tx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float w = e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w;
                        acc[i][c][0] = ptx::ffma2(both(w), lo2(v), acc[i][c][0]);
                        acc[i][c][1] = ptx::ffma2(both(w), hi2(v), acc[i][c][1]);
                    }
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            acc[i][c][0] = ptx::fmul2(acc[i][c][0], both(sg[4 * ty + i + 1]));
            acc[i][c][1] = ptx::fmul2(acc[i][c][1], both(sg[4 * ty + i + 1]));
        }
    // the block's own part: rows s <= t of v (those before the thread's rows for all four alike)
    int s = 0;
#pragma unroll 2
    for (; s < min(n, 4 * ty) / 4 * 4; s += 4) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(sp + (4 * ty + i) * kLdP + s);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const float4 v = *reinterpret_cast<const float4*>(sv + (s + e) * kLdV + 64 * c + 4 * tx);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w;
                    acc[i][c][0] = ptx::ffma2(both(w), lo2(v), acc[i][c][0]);
                    acc[i][c][1] = ptx::ffma2(both(w), hi2(v), acc[i][c][1]);
                }
            }
    }
    for (; s < min(n, 4 * ty + 4); ++s) {
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(sv + s * kLdV + 64 * c + 4 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (s <= 4 * ty + i) {
                    const float w = sp[(4 * ty + i) * kLdP + s];
                    acc[i][c][0] = ptx::ffma2(both(w), lo2(v), acc[i][c][0]);
                    acc[i][c][1] = ptx::ffma2(both(w), hi2(v), acc[i][c][1]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (4 * ty + i < n) {
            T* o = static_cast<T*>(a.out) + ((t0 + 4 * ty + i) * a.hv + h) * a.dv;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int col = 64 * c + 4 * tx;
                if (col < a.dv) {
                    Elem<T>::store(o + col + 0, a.scale * acc[i][c][0].x);
                    Elem<T>::store(o + col + 1, a.scale * acc[i][c][0].y);
                    Elem<T>::store(o + col + 2, a.scale * acc[i][c][1].x);
                    Elem<T>::store(o + col + 3, a.scale * acc[i][c][1].y);
                }
            }
        }
    }
}

template <typename T, int DK, int DV>
cudaError_t prefill_d(const LinattnArgs& a, float* states, cudaStream_t s)
{
    constexpr int kStateBytes = kTok * (DK + DV + 8) * 4;
    constexpr int kOutBytes = kTok * (2 * (DK + 4) + DV + 4 + kLdP) * 4;
    static_assert(DK >= DV, "the rows of the start state fit into the place of the keys");
    auto state_kernel = linattn_block_state_kernel<T, DK, DV>;
    auto output_kernel = linattn_block_output_kernel<T, DK, DV>;
    cudaError_t e = cudaFuncSetAttribute(state_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStateBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(output_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kOutBytes);
    if (e != cudaSuccess) return e;
    int* err = device_error_word();
    const dim3 grid((unsigned)packed_blocks(a.total, a.nseq, kTok), (unsigned)a.hv);
    e = launch_dependent(state_kernel, grid, dim3(kThreads), kStateBytes, s, a, Divisor(kTok), states, err);
    const dim3 scan((unsigned)(a.nseq * a.hv), (unsigned)((a.dk * a.dv + 4 * kScanThreads - 1) / (4 * kScanThreads)));
    if (e == cudaSuccess) e = launch_dependent(linattn_scan_kernel, scan, dim3(kScanThreads), 0, s, a, states);
    if (e == cudaSuccess && a.total > 0)
        e = launch_dependent(output_kernel, grid, dim3(kThreads), kOutBytes, s, a, Divisor(kTok), static_cast<const float*>(states), err);
    return e;
}

template <typename T>
cudaError_t prefill_t(const LinattnArgs& a, float* states, cudaStream_t s)
{
    if (a.dk <= 64 && a.dv <= 64) return prefill_d<T, 64, 64>(a, states, s);
    return a.dv <= 64 ? prefill_d<T, 128, 64>(a, states, s) : prefill_d<T, 128, 128>(a, states, s);
}

}  // namespace

cudaError_t launch_linattn_decode(ssd_dtype_t dtype, float* state, const void* q, const void* k, const void* v,
                                  const float* log_decay, void* out, int batch, int hq, int hv, int dk, int dv,
                                  float scale, cudaStream_t s)
{
    return dtype == SSD_F32 ? decode_t<float>(state, q, k, v, log_decay, out, batch, hq, hv, dk, dv, scale, s)
                            : decode_t<__nv_bfloat16>(state, q, k, v, log_decay, out, batch, hq, hv, dk, dv, scale, s);
}

size_t linattn_simt_workspace(int nseq, int total, int hv, int dk, int dv)
{
    return (size_t)packed_blocks(total, nseq, kTok) * hv * dk * dv * sizeof(float);
}

cudaError_t launch_linattn_prefill_simt(const LinattnArgs& a, void* workspace, cudaStream_t s)
{
    return prefill_t<float>(a, static_cast<float*>(workspace), s);
}

}  // namespace ssd
