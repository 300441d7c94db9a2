// head.cu -- operators on the LM head's logits that keep a list of columns:
//
//   k_top_rows      per row the k largest logits (ties: the lowest column) and
//                   the log-sum-exp
//   k_distill       distillation from a teacher's top logits: loss and
//                   gradient of a row
//   k_row_mean      the mean of the row losses (fixed order)
//
// A row of V logits is read in the storage type; sums, statistics and losses
// are fp32.
#include "tt_internal.h"

#include <algorithm>

namespace tt {
namespace {

template <typename T> __device__ __forceinline__ float ldf(const T* p);
template <> __device__ __forceinline__ float ldf<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float ldf<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <> __device__ __forceinline__ float ldf<__half>(const __half* p) { return __half2float(*p); }
template <typename T> __device__ __forceinline__ T stf(float v);
template <> __device__ __forceinline__ float stf<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 stf<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half stf<__half>(float v) { return __float2half_rn(v); }

// Order-preserving key of (value, column): larger values first, then lower
// columns.  -0 counts as +0 and a NaN as -inf.
__device__ __forceinline__ unsigned long long top_key(float v, int col) {
    if (v != v) v = -INFINITY;
    uint32_t u = __float_as_uint(v);
    if ((u & 0x7FFFFFFFu) == 0) u = 0;
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((unsigned long long)u << 32) | (unsigned long long)(0xFFFFFFFFu - (uint32_t)col);
}
__device__ __forceinline__ float key_value(unsigned long long key) {
    uint32_t u = (uint32_t)(key >> 32);
    u = (u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u;
    return __uint_as_float(u);
}
__device__ __forceinline__ int key_col(unsigned long long key) {
    return (int)(0xFFFFFFFFu - (uint32_t)(key & 0xFFFFFFFFull));
}

constexpr int HD_THREADS = 256;
constexpr int HD_WARPS = HD_THREADS / 32;

// block reductions in a fixed order; every thread gets the result
__device__ __forceinline__ float block_sum(float v, float* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < HD_WARPS; w++) t += s[w];
    return t;
}
__device__ __forceinline__ float block_max(float v, float* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = s[0];
    for (int w = 1; w < HD_WARPS; w++) t = fmaxf(t, s[w]);
    return t;
}

// One CTA per row.  k rounds: each round finds the largest key below the last
// one found.
template <typename T>
__global__ void __launch_bounds__(HD_THREADS)
k_top_rows(const T* __restrict__ z, long long ld, int V, int k, float inv_tau, float* __restrict__ vals,
           int32_t* __restrict__ idx, float* __restrict__ lse, double* __restrict__ lse64,
           const int32_t* __restrict__ skip) {
    pdl_enter();
    __shared__ float s_f[HD_WARPS];
    __shared__ unsigned long long s_k[HD_WARPS];
    const long long row = blockIdx.x;
    if (skip && skip[row]) return;
    const T* zr = z + row * ld;
    if (lse || lse64) {
        float m = -INFINITY;
        for (int v = threadIdx.x; v < V; v += HD_THREADS) m = fmaxf(m, ldf(zr + v));
        m = block_max(m, s_f);
        float s = 0.0f;
        for (int v = threadIdx.x; v < V; v += HD_THREADS) s += expf((ldf(zr + v) - m) * inv_tau);
        s = block_sum(s, s_f);
        // an empty row (every logit -inf) and a row with +inf have that as their value, unless a NaN is there too
        if (m == INFINITY) {
            float n = 0.0f;
            for (int v = threadIdx.x; v < V; v += HD_THREADS) n += ldf(zr + v) != ldf(zr + v) ? 1.0f : 0.0f;
            if (block_sum(n, s_f) > 0.0f) m = NAN;
        }
        if (threadIdx.x == 0) {
            const bool flat = m == -INFINITY || m == INFINITY;
            if (lse) lse[row] = flat ? m : m * inv_tau + logf(s);
            if (lse64) lse64[row] = flat ? (double)m : (double)m * (double)inv_tau + log((double)s);
        }
    }
    unsigned long long last = ~0ull;
    for (int j = 0; j < k; j++) {
        unsigned long long best = 0;
        for (int v = threadIdx.x; v < V; v += HD_THREADS) {
            const unsigned long long key = top_key(ldf(zr + v), v);
            if (key < last && key > best) best = key;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s_k[threadIdx.x >> 5] = best;
        __syncthreads();
        best = s_k[0];
        for (int w = 1; w < HD_WARPS; w++) best = max(best, s_k[w]);
        last = best;
        if (threadIdx.x == 0) {
            vals[row * k + j] = key_value(best);
            idx[row * k + j] = key_col(best);
        }
    }
}

// One CTA per row.  With q = softmax(z / tau), s = softmax(z), the list's
// probabilities p_j at columns i_j, W their sum (plus p_r, the teacher's mass
// outside the list, when it is known and the student has any there, q_r):
//   loss = alpha tau^2 (sum p_j (ln p_j - ln q_ij) + p_r (ln p_r - ln q_r)) + (1 - alpha) (lse(z) - z_y)
//   dz_i = g alpha tau (W q_i - p_i)            on the list
//        = g alpha tau q_i (W - p_r / q_r)      off it
//        + g (1 - alpha) (s_i - [i = y])
// The list's columns are marked in a bitmap, so that q_r is summed without the
// list instead of as a difference.
struct DistillArgs {
    const float* t_vals;
    const int32_t* t_idx;
    const float* t_lse;
    const int32_t* targets;
    const float* scale_dev;
    float* row_loss;
    int V, ld, k;
    float alpha, tau, dscale;
    int* flags;
};

constexpr int LIST_MAX = 128;

template <typename T>
__global__ void __launch_bounds__(HD_THREADS)
k_distill(const T* z, T* dz, const DistillArgs a) {
    pdl_enter();
    extern __shared__ uint32_t s_bits[];
    __shared__ float s_f[HD_WARPS];
    __shared__ int s_i[LIST_MAX];
    __shared__ float s_z[LIST_MAX], s_p[LIST_MAX];
    const long long row = blockIdx.x;
    const int tid = threadIdx.x, V = a.V, k = a.k;
    const T* zr = z + row * (long long)a.ld;
    T* dr = dz ? dz + row * (long long)a.ld : nullptr;
    const float it = 1.0f / a.tau;
    float g = a.dscale;
    if (a.scale_dev) g *= *a.scale_dev;
    for (int w = tid; w < (V + 31) / 32; w += HD_THREADS) s_bits[w] = 0;
    __syncthreads();
    float t = -INFINITY;
    int col = -1;
    bool bad = false;
    if (tid < k) {
        col = a.t_idx[row * k + tid];
        if (col >= 0 && col < V) {
            const uint32_t bit = 1u << (col & 31);
            if (atomicOr(&s_bits[col >> 5], bit) & bit) { bad = true; col = -1; }
            else t = a.t_vals[row * k + tid] * it;
        } else {
            bad = col != -1;
            col = -1;
        }
    }
    int y = a.targets ? a.targets[row] : -1;
    if (y < -1 || y >= V) { bad = true; y = -1; }
    if (bad) atomicOr(&a.flags[FLAG_BAD_TOKEN], 1);
    const int used = __syncthreads_count(col >= 0);
    const bool soft = used > 0 && a.alpha > 0.0f, hard = y >= 0 && a.alpha < 1.0f;
    if (!soft && !hard) {
        if (tid == 0) a.row_loss[row] = 0.0f;
        if (dr)
            for (int v = tid; v < a.ld; v += HD_THREADS) dr[v] = stf<T>(0.0f);
        return;
    }
    float m = -INFINITY;
    for (int v = tid; v < V; v += HD_THREADS) m = fmaxf(m, ldf(zr + v));
    m = block_max(m, s_f);
    float s1 = 0.0f, st = 0.0f, sr = 0.0f;
    for (int v = tid; v < V; v += HD_THREADS) {
        const float d = ldf(zr + v) - m;
        if (hard) s1 += expf(d);
        if (soft) {
            const float e = expf(d * it);
            if (s_bits[v >> 5] >> (v & 31) & 1) st += e;
            else sr += e;
        }
    }
    s1 = block_sum(s1, s_f);
    st = block_sum(st, s_f);
    sr = block_sum(sr, s_f);
    st += sr;
    float loss = 0.0f, W = 0.0f, off = 0.0f;
    if (soft) {
        const float lse = logf(st);
        const float zl = col >= 0 ? ldf(zr + col) : 0.0f;
        float lp = -INFINITY;
        if (a.t_lse) {
            if (col >= 0) lp = t - a.t_lse[row];
        } else {
            const float tm = block_max(t, s_f);
            const float sum = block_sum(col >= 0 ? expf(t - tm) : 0.0f, s_f);
            if (col >= 0) lp = t - tm - logf(sum);
        }
        const float p = col >= 0 ? expf(lp) : 0.0f;
        W = block_sum(p, s_f);
        loss = block_sum(p > 0.0f || p != p ? p * (lp - ((zl - m) * it - lse)) : 0.0f, s_f);
        off = W;
        if (a.t_lse && sr > 0.0f) {
            const float pr = fmaxf(1.0f - W, 0.0f);
            if (pr > 0.0f) loss += pr * (logf(pr) - (logf(sr) - lse));
            W += pr;
            off = W - pr * st / sr;
        }
        if (tid < k) { s_i[tid] = col; s_z[tid] = zl; s_p[tid] = p; }
        loss *= a.alpha * a.tau * a.tau;
    }
    const float zy = hard ? ldf(zr + y) : 0.0f;
    if (hard) loss += (1.0f - a.alpha) * (m + logf(s1) - zy);
    if (tid == 0) a.row_loss[row] = loss;
    if (!dr) return;
    const float ks = g * a.alpha * a.tau, kh = hard ? g * (1.0f - a.alpha) : 0.0f;
    __syncthreads();
    auto grad = [&](float zv, float w, float p, bool is_y) {
        const float d = zv - m;
        float r = 0.0f;
        if (soft) r = ks * (w * expf(d * it) / st - p);
        if (hard) r += kh * (expf(d) / s1 - (is_y ? 1.0f : 0.0f));
        return r;
    };
    for (int v = tid; v < a.ld; v += HD_THREADS) {
        float r = 0.0f;
        if (v < V) {
            if (soft && (s_bits[v >> 5] >> (v & 31) & 1)) continue;  // the list's columns: below
            r = grad(ldf(zr + v), off, 0.0f, v == y);
        }
        dr[v] = stf<T>(r);
    }
    if (soft && tid < k && s_i[tid] >= 0) dr[s_i[tid]] = stf<T>(grad(s_z[tid], W, s_p[tid], s_i[tid] == y));
}

// mean of M row losses: each thread adds rows t, t + 1024, ..., the threads'
// sums meet in a fixed tree
__global__ void __launch_bounds__(1024) k_row_mean(const float* __restrict__ row_loss, int M, float* __restrict__ out,
                                                   int* flags) {
    pdl_enter();
    __shared__ float s_w[32];
    float s = 0.0f;
    for (int i = threadIdx.x; i < M; i += 1024) s += row_loss[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = s_w[threadIdx.x];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) {
            s /= (float)M;
            out[0] = s;
            if (!isfinite(s)) atomicOr(&flags[FLAG_NONFINITE], 1);
        }
    }
}

template <typename T>
bool top_rows(const Launch& L, const void* z, long long ld, int V, int k, float inv_tau, float* vals, int32_t* idx,
              float* lse, double* lse64, const int32_t* skip, int M) {
    L.count();
    launch_k(L, k_top_rows<T>, dim3(M), dim3(HD_THREADS), 0, (const T*)z, ld, V, k, inv_tau, vals, idx, lse, lse64,
             skip);
    return true;
}

template <typename T>
bool distill(const Launch& L, const void* z, void* dz, const DistillArgs& a, int M) {
    static PerDevice attr;
    const size_t smem = (size_t)((a.V + 31) / 32) * 4;
    if (!attr.once([] {
            return cudaFuncSetAttribute(k_distill<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024) ==
                   cudaSuccess;
        }))
        return false;
    L.count();
    launch_k(L, k_distill<T>, dim3(M), dim3(HD_THREADS), smem, (const T*)z, (T*)dz, a);
    return true;
}

}  // namespace

bool head_row_ok(tt_dtype dtype, int V) { return (dtype == TT_FP32 || dtype == TT_BF16 || dtype == TT_FP16) && V < 1048576; }

bool launch_top_rows(const Launch& L, tt_dtype dtype, const void* z, long long ld, int M, int V, int k, float tau,
                     float* vals, int32_t* idx, float* lse, double* lse64, const int32_t* skip) {
    if (L.dry) return true;
    const float it = 1.0f / tau;
    if (dtype == TT_FP32) return top_rows<float>(L, z, ld, V, k, it, vals, idx, lse, lse64, skip, M);
    if (dtype == TT_FP16) return top_rows<__half>(L, z, ld, V, k, it, vals, idx, lse, lse64, skip, M);
    return top_rows<__nv_bfloat16>(L, z, ld, V, k, it, vals, idx, lse, lse64, skip, M);
}

bool launch_distill(const Launch& L, tt_dtype dtype, const void* z, void* dz, const float* t_vals,
                    const int32_t* t_idx, const float* t_lse, const int32_t* targets, float* row_loss,
                    float* mean_loss, int M, int V, int ld, int k, float alpha, float tau, float dscale,
                    const float* scale_dev) {
    if (L.dry) return true;
    DistillArgs a;
    a.t_vals = t_vals; a.t_idx = t_idx; a.t_lse = t_lse; a.targets = targets; a.scale_dev = scale_dev;
    a.row_loss = row_loss; a.V = V; a.ld = ld; a.k = k;
    a.alpha = alpha; a.tau = tau; a.dscale = dscale; a.flags = L.flags;
    bool ok;
    if (dtype == TT_FP32) ok = distill<float>(L, z, dz, a, M);
    else if (dtype == TT_FP16) ok = distill<__half>(L, z, dz, a, M);
    else ok = distill<__nv_bfloat16>(L, z, dz, a, M);
    if (!ok) return false;
    if (mean_loss) {
        L.count();
        launch_k(L, k_row_mean, dim3(1), dim3(1024), 0, row_loss, M, mean_loss, L.flags);
    }
    return true;
}

}  // namespace tt
