// answer.cu -- losses on the probabilities of given tokens:
//
//   k_answer        rows of more than 256 granules: a label's log probability, or
//                   the clipped policy loss and its gradient; a CTA a row
//   k_answer_short  the same for shorter rows, a warp or a part of one a row, in
//                   registers
//   k_pairs         the loss of pairs of answers from their labels' log
//                   probabilities, and each row's coefficient
//   k_answer_grad   coefficient times (onehot - softmax)
//
// With u = z / tau, l = log sum exp(u) and the label y of a row,
//   ln pi = u_y - l,   d ln pi / dz_i = ([i = y] - softmax(u)_i) / tau,
// so a row's gradient is one coefficient c = d loss / d ln pi times that.
//
// Policy: A the advantage, ratio r = exp(ln pi - old), x = ref - ln pi,
//   loss = w (-min(r A, clip(r, 1 - lo, 1 + hi) A) + beta (e^x - x - 1))
//   c    = w (-[not clipped] r A - beta (e^x - 1))
// The coefficient of a row is known once the row has been summed: the row is
// read from memory once, and again out of L2 for its gradient.
//
// Preference: with S the sums of (ln pi - ref) over an answer's labels (or
// their means), v = beta (S_chosen - S_rejected) - gamma,
//   loss = (1 - e) ln(1 + exp(-v)) + e ln(1 + exp(v))
//   c    = +-beta (e s(v) - (1 - e) s(-v)) (/ n),   s(v) = 1 / (1 + exp(-v))
// whose coefficient needs every row of both answers, so the logits are read
// twice: there is nowhere to keep a batch of them.
//
// Statistics, losses and coefficients are fp32, sums over an answer 64 bits.
// Rows without a label are not read: a loss of 0, and a gradient of zeros.
//
// All but the shortest rows are bound by memory.  32768 rows of 50257 in bf16, the
// lm head's logits, 54% of them labelled (rates by the bytes that have to move):
// log probabilities 267 to 271 us, 6.6 TB/s; the policy step 784 to 789 us, 6.2 TB/s,
// reads and writes in turn; the preference step 1022 us, of which the second reading
// of the logits is some 260, 6.7 TB/s with it counted.
#include "row_view.cuh"

namespace tt {
namespace {

using namespace head;

struct AnswerArgs {
    const int32_t* targets;
    const float *old, *ref, *adv, *weight;  // each may be NULL but adv
    const float* scale_dev;
    float *logp, *lse, *row_loss;  // may be NULL
    float4* stat;                  // R, sum of 2^((z - R) ct), coefficient, ln pi (or NULL)
    int* claim;                    // with stat: whether an answer has the row; [M]: pairs that are done
    int* flags;
    long long ld;
    int M, V, G;
    float it, lo, hi, llo, lhi, beta, dscale;  // it = 1 / tau, llo = ln(1 - lo), lhi = ln(1 + hi)
    bool same_phase;
};

__device__ __forceinline__ void put_stat(const AnswerArgs& a, long long row, float4 s) {
    a.stat[row] = s;
    a.claim[row] = 0;
    if (row == 0) a.claim[a.M] = 0;
}

// The label of a row, -1 for none; one that is out of range counts as none.
__device__ __forceinline__ int label_of(const int32_t* targets, long long row, int V, int* flags, bool first) {
    const int y = targets[row];
    if (y >= -1 && y < V) return y;
    if (first) atomicOr(&flags[FLAG_BAD_TOKEN], 1);
    return -1;
}

// ln pi and l from the reference and the sum.  For ln pi the difference of the
// logits comes first, so that nothing is lost where both are far from zero (a
// mask's lowest value).  In 32 bits: a warp's 64-bit instruction takes the SM 16
// cycles, and eight of them a row were 7 of the 12 us of 16384 rows of 65.
__device__ __forceinline__ float logp_of(float zy, float R, float s, float it) { return fmaf(zy - R, it, -logf(s)); }
__device__ __forceinline__ float lse_f(float R, float s, float it) { return fmaf(R, it, logf(s)); }

// e^x - x - 1, em1 = e^x - 1.  Near 0, where a policy starts out from its reference,
// the difference is an x of rounding beside x^2 / 2: up to 1/2 the series (what is
// left out, x^10 / 10! and on, is below 2^-28 of the sum).  Never below 0.
__device__ __forceinline__ float exp_minus(float x, float em1) {
    if (!(fabsf(x) < 0.5f)) return em1 - x;
    float s = 1.0f / 362880.0f;
    s = fmaf(s, x, 1.0f / 40320.0f);
    s = fmaf(s, x, 1.0f / 5040.0f);
    s = fmaf(s, x, 1.0f / 720.0f);
    s = fmaf(s, x, 1.0f / 120.0f);
    s = fmaf(s, x, 1.0f / 24.0f);
    s = fmaf(s, x, 1.0f / 6.0f);
    s = fmaf(s, x, 0.5f);
    return x * x * s;
}

// what the policy loss of a row needs beside its logits (loaded with the label,
// so that the row waits once)
struct PolicyRow {
    float old = 0.0f, ref = 0.0f, A = 0.0f, w = 1.0f;
    bool fresh;
    __device__ __forceinline__ PolicyRow(const AnswerArgs& a, long long row, bool policy) : fresh(!a.old) {
        if (!policy) return;
        if (a.old) old = a.old[row];
        if (a.beta > 0.0f) ref = a.ref[row];
        A = a.adv[row];
        if (a.weight) w = a.weight[row];
    }
    // loss, and its derivative by lp
    __device__ __forceinline__ float2 loss(const AnswerArgs& a, float lp) const {
        const float d = fresh ? lp - lp : lp - old;  // NaN where ln pi is not finite
        const bool inside = A >= 0.0f ? d <= a.lhi : d >= a.llo;
        const float r = inside || d != d ? expf(d) : A >= 0.0f ? 1.0f + a.hi : 1.0f - a.lo;
        float v = A == 0.0f && d == d ? 0.0f : -r * A, c = inside || v != v ? v : 0.0f;
        if (a.beta > 0.0f) {
            const float x = ref - lp, e = expm1f(x);
            v = fmaf(a.beta, exp_minus(x, e), v);
            c = fmaf(-a.beta, e, c);
        }
        return make_float2(w * v, w * c);
    }
};

// zeros over the ld columns of a row, by N threads
template <typename T> __device__ __forceinline__ void zero_row(T* d, long long ld, int tid, int N) {
    constexpr int EPG = Elem<T>::EPG;
    const int ph = (int)(((uintptr_t)d & 15) / sizeof(T));
    const long long first = min((long long)(ph ? EPG - ph : 0), ld), n = (ld - first) / EPG;
    for (int c = tid; c < first; c += N) d[c] = Elem<T>::put(0.0f);
    uint4* v = reinterpret_cast<uint4*>(d + first);
    for (long long i = tid; i < n; i += N) __stcs(v + i, make_uint4(0, 0, 0, 0));
    for (long long c = first + n * EPG + tid; c < ld; c += N) d[c] = Elem<T>::put(0.0f);
}

// the thread of N that writes slot i of the row
template <typename T> __device__ __forceinline__ int owner_of(const RowView<T>& view, int i, int N) {
    const Slice<T>& s = view.s;
    return s.inner(i) ? (i - s.i0) % N : s.head && i == 0 ? 0 : view.tail_tid;
}

// k (onehot - softmax) over a row, R and s its reference and sum (N threads; no
// barrier: the label's column is written by the thread that has its granule)
template <typename T>
__device__ __forceinline__ void row_gradient(const RowView<T>& view, T* drow, long long ld, int tid, int N, bool same_phase,
                                             float R, float s, float ct, float k, int y, float zy) {
    if (k == 0.0f) {
        zero_row(drow, ld, tid, N);
        return;
    }
    const float At = -__fdividef(k, s);
    view.template gradient<true, false>(tid, N, drow, same_phase, R, ct, At, 0.0f);
    if (tid == owner_of(view, view.s.at(y) >> 4, N)) drow[y] = Elem<T>::put(fmaf(At, exp_of(zy, R, ct), k));
    for (long long c = view.V + tid; c < ld; c += N) drow[c] = Elem<T>::put(0.0f);
}

constexpr int AN_THREADS = 1024;  // most threads of a CTA

// A CTA has one row, or blockDim.y rows of a warp each.
template <typename T, bool POLICY>
__global__ void __launch_bounds__(AN_THREADS, 1) k_answer(const T* z, T* dz, const AnswerArgs a) {
    pdl_wait();
    __shared__ float2 s_part[AN_THREADS / 32];
    const int N = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = a.V;
    const long long row = blockIdx.x * (long long)blockDim.y + threadIdx.y;
    if (row >= a.M) return;
    const PolicyRow pr(a, row, POLICY);
    const int y = label_of(a.targets, row, V, a.flags, tid == 0);
    T* drow = dz ? dz + row * a.ld : nullptr;
    if (y < 0) {
        if (tid == 0) {
            if (a.logp) a.logp[row] = 0.0f;
            if (a.lse) a.lse[row] = 0.0f;
            if (a.row_loss) a.row_loss[row] = 0.0f;
            if (a.stat) put_stat(a, row, make_float4(0.0f, 1.0f, 0.0f, 0.0f));
        }
        if (drow) zero_row(drow, a.ld, tid, N);
        return;
    }
    const Slice<T> s(z, row, a.ld, V, 0, a.G);
    const float zy = Elem<T>::get(z + row * a.ld + y);
    const float ct = LOG2E * a.it, lift = 20.0f / fmaxf(1.0f, a.it);
    const RowView<T> view{s, V, nullptr, N == 32 ? 1 : 32};
    float R, sum, none;
    view.template sums<false, true>(tid, N, 0.0f, ct, lift, R, none, sum);
    merge(R, sum, ct);
    if (N == 32) {
        __syncwarp();  // everything has been read (dz may be z)
    } else {
        if (lane == 0) s_part[warp] = make_float2(R, sum);
        __syncthreads();
        const float2 p = lane < N / 32 ? s_part[lane] : make_float2(-INFINITY, 0.0f);
        R = p.x, sum = p.y;
        merge(R, sum, ct);
    }
    const float lp = logp_of(zy, R, sum, a.it);
    float k = 0.0f;
    if (POLICY) {
        const float2 f = pr.loss(a, lp);
        if (tid == 0) a.row_loss[row] = f.x;
        k = f.y * a.it * a.dscale;
        if (a.scale_dev) k *= *a.scale_dev;
    }
    if (tid == 0) {
        if (a.logp) a.logp[row] = lp;
        if (a.lse) a.lse[row] = lse_f(R, sum, a.it);
        if (a.stat) put_stat(a, row, make_float4(R, sum, 0.0f, lp));
    }
    if (POLICY && dz) row_gradient(view, drow, a.ld, tid, N, a.same_phase, R, sum, ct, k, y, zy);
}

// Rows of up to LPR GL granules, LPR lanes each, lane l the granules l + LPR j:
// a row is some hundred instructions whatever its length, so the shortest share a
// warp.  16384 rows of 65 in bf16, half of them labelled, as a policy step: 6.9 us
// by eight lanes a row, 10.3 by a warp.
constexpr int AS_THREADS = 128;

template <typename T, int LPR, int GL, bool POLICY>
__global__ void __launch_bounds__(AS_THREADS) k_answer_short(const T* z, T* dz, const AnswerArgs a) {
    pdl_enter();
    using E = Elem<T>;
    constexpr int H = E::EPG / 2;
    const int lane = threadIdx.x % LPR, V = a.V;
    const uint32_t mates = (LPR == 32 ? 0xffffffffu : (1u << LPR % 32) - 1u) << (threadIdx.x & 31 & ~(LPR - 1));
    const long long row = blockIdx.x * (long long)(AS_THREADS / LPR) + threadIdx.x / LPR;
    if (row >= a.M) return;
    const PolicyRow pr(a, row, POLICY);
    const int y = label_of(a.targets, row, V, a.flags, lane == 0);
    T* drow = dz ? dz + row * a.ld : nullptr;
    if (y < 0) {
        if (lane == 0) {
            if (a.logp) a.logp[row] = 0.0f;
            if (a.lse) a.lse[row] = 0.0f;
            if (a.row_loss) a.row_loss[row] = 0.0f;
            if (a.stat) put_stat(a, row, make_float4(0.0f, 1.0f, 0.0f, 0.0f));
        }
        if (drow) zero_row(drow, a.ld, lane, LPR);
        return;
    }
    const Slice<T> s(z, row, a.ld, V, 0, a.G);
    const float zy = E::get(z + row * a.ld + y), ct = LOG2E * a.it;
    f2 e[GL][H];
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < GL; j++) {
        const int i = lane + LPR * j;
        uint4 u = make_uint4(E::NINF, E::NINF, E::NINF, E::NINF);
        if (i < s.n) u = granule(s, i, V);
        E::unpack(u, e[j]);
#pragma unroll
        for (int h = 0; h < H; h++) {
            float p, q;
            unpk(e[j][h], p, q);
            m = fmaxf(m, fmaxf(p, q));
        }
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mates, m, o));
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < GL; j++)
#pragma unroll
        for (int h = 0; h < H; h++) {
            float p, q;
            unpk(e[j][h], p, q);
            // (a difference of 0 where both are infinite; a row of -inf has no terms)
            p = m == -INFINITY && p == m ? 0.0f : p == m ? 1.0f : exp_of(p, m, ct);
            q = m == -INFINITY && q == m ? 0.0f : q == m ? 1.0f : exp_of(q, m, ct);
            sum += p + q;
            e[j][h] = pk(p, q);
        }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mates, sum, o);
    const float lp = logp_of(zy, m, sum, a.it);
    float k = 0.0f;
    if (POLICY) {
        const float2 f = pr.loss(a, lp);
        if (lane == 0) a.row_loss[row] = f.x;
        k = f.y * a.it * a.dscale;
        if (a.scale_dev) k *= *a.scale_dev;
    }
    if (lane == 0) {
        if (a.logp) a.logp[row] = lp;
        if (a.lse) a.lse[row] = lse_f(m, sum, a.it);
        if (a.stat) put_stat(a, row, make_float4(m, sum, 0.0f, lp));
    }
    if (!POLICY || !dz) return;
    __syncwarp(mates);  // everything has been read (dz may be z)
    if (k == 0.0f) {
        zero_row(drow, a.ld, lane, LPR);
        return;
    }
    const float At = -__fdividef(k, sum);
    const f2 at2 = pk(At, At);
    uint4* const d0 = reinterpret_cast<uint4*>(drow + s.col(0));
    const int iy = s.at(y) >> 4;
#pragma unroll
    for (int j = 0; j < GL; j++) {
        const int i = lane + LPR * j;
        if (i >= s.n) continue;
        f2 r[H];
#pragma unroll
        for (int h = 0; h < H; h++) r[h] = mul2(e[j][h], at2);
        if (a.same_phase && s.inner(i)) d0[i] = E::pack(r);
        else store_edge(s, i, drow, V, r);
        if (i == iy) drow[y] = E::put(fmaf(At, zy == m ? 1.0f : exp_of(zy, m, ct), k));
    }
    for (long long c = V + lane; c < a.ld; c += LPR) drow[c] = E::put(0.0f);
}

template <typename T, int LPR, int GL, bool POLICY>
void answer_short(const Launch& L, const void* z, void* dz, const AnswerArgs& a) {
    constexpr int R = AS_THREADS / LPR;
    launch_k(L, k_answer_short<T, LPR, GL, POLICY>, dim3((unsigned)((a.M - 1) / R + 1)), dim3(AS_THREADS), 0, (const T*)z,
             (T*)dz, a);
}

// rows of blockDim.y at a time, blockDim.x threads each
template <typename T>
__global__ void __launch_bounds__(AN_THREADS, 1) k_answer_grad(const T* z, T* dz, const AnswerArgs a) {
    pdl_wait();
    // from the last row on: what the sums read last is still in L2
    const long long row = a.M - 1 - (blockIdx.x * (long long)blockDim.y + threadIdx.y);
    if (row < 0) return;
    const int tid = threadIdx.x, N = blockDim.x;
    T* drow = dz + row * a.ld;
    const float4 st = a.stat[row];
    const float k = st.z;
    if (k == 0.0f) {
        zero_row(drow, a.ld, tid, N);
        return;
    }
    const int y = a.targets[row];  // in range, else there is no coefficient
    const Slice<T> s(z, row, a.ld, a.V, 0, a.G);
    const float ct = LOG2E * a.it;
    const RowView<T> view{s, a.V, nullptr, N == 32 ? 1 : 32};
    // the label's logit is its granule's owner's to read, before that thread writes
    const float zy = tid == owner_of(view, s.at(y) >> 4, N) ? Elem<T>::get(z + row * a.ld + y) : 0.0f;
    row_gradient(view, drow, a.ld, tid, N, a.same_phase, st.x, st.y, ct, k, y, zy);
}

struct PairArgs {
    const int32_t *targets, *spans;
    const float *ref, *scale_dev;
    float4* stat;
    int *claim, *flags;
    float *seq_logp, *pair_loss, *mean_loss;
    int M, V, pairs;
    float beta, gamma, smooth, k;  // k = dscale / tau
    bool mean;
};
constexpr int PAIR_THREADS = 256;  // an answer

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }

// One CTA a pair, half of it an answer: the answers' sums in a fixed order, in 64
// bits (an answer's sum is thousands, the difference of two a few), the loss, the
// rows' coefficients.  The CTA that finishes last forms the mean of the pairs'
// losses, in their order.
__global__ void __launch_bounds__(2 * PAIR_THREADS) k_pairs(const PairArgs a) {
    pdl_enter();
    constexpr int WARPS = PAIR_THREADS / 32;  // of an answer
    __shared__ double s_sum[2 * WARPS][2];
    __shared__ int s_n[2 * WARPS];
    __shared__ float s_coef[2];
    __shared__ bool s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, w = tid / PAIR_THREADS;
    const long long pair = blockIdx.x;
    // (64 bits: a row behind the last, by a thread's number, may be past 2^31)
    long long first = a.spans[(2 * pair + w) * 2], last = a.spans[(2 * pair + w) * 2 + 1];
    bool bad = false;
    if (first < 0 || first > last || last > a.M) {
        bad = true;
        first = last = 0;
    }
    first += tid % PAIR_THREADS;
    double total = 0.0, score = 0.0;
    int n = 0;
    constexpr int U = 4;  // rows in flight
    for (long long r0 = first; r0 < last; r0 += U * PAIR_THREADS) {
        float lp[U], ref[U];
        int claimed[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const long long r = r0 + u * PAIR_THREADS;
            const int y = r < last ? a.targets[r] : -1;
            on[u] = y >= 0 && y < a.V;
            lp[u] = r < last ? a.stat[r].w : 0.0f;
            ref[u] = r < last && a.ref ? a.ref[r] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; u++) claimed[u] = on[u] ? atomicExch(&a.claim[r0 + u * PAIR_THREADS], 1) : 0;
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (!on[u]) continue;
            bad |= claimed[u] != 0;  // in two answers
            total += lp[u];
            score += (double)lp[u] - (double)ref[u];
            n++;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        score += __shfl_xor_sync(0xffffffffu, score, o);
        n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if (lane == 0) {
        s_sum[warp][0] = total;
        s_sum[warp][1] = score;
        s_n[warp] = n;
    }
    if (bad) atomicOr(&a.flags[FLAG_BAD_TOKEN], 1);
    __syncthreads();
    if (warp == 0) {  // lanes 0-7 (and their copies) hold the first answer's warps, 8-15 the second's
        const int l = lane & (2 * WARPS - 1);
        total = s_sum[l][0];
        score = s_sum[l][1];
        n = s_n[l];
#pragma unroll
        for (int o = WARPS / 2; o > 0; o >>= 1) {
            total += __shfl_xor_sync(0xffffffffu, total, o);
            score += __shfl_xor_sync(0xffffffffu, score, o);
            n += __shfl_xor_sync(0xffffffffu, n, o);
        }
        if (a.seq_logp && lane < 2 * WARPS && lane % WARPS == 0) a.seq_logp[2 * pair + lane / WARPS] = (float)total;
        const float inv = a.mean && n > 1 ? 1.0f / (float)n : 1.0f;
        if (a.mean && n > 1) {  // a step of Newton's: 1 / n in 64 bits without their division
            const double x = inv;
            score *= x * (2.0 - n * x);
        }
        const double other = __shfl_sync(0xffffffffu, score, WARPS);
        const float inv1 = __shfl_sync(0xffffffffu, inv, WARPS);
        if (lane == 0) {
            const float v = fmaf(a.beta, (float)(score - other), -a.gamma), e = a.smooth;
            const float loss = (1.0f - e) * softplus(-v) + (e > 0.0f ? e * softplus(v) : 0.0f);
            const float dv = e / (1.0f + expf(-v)) - (1.0f - e) / (1.0f + expf(v));
            const float k = dv * a.beta * a.k * (a.scale_dev ? *a.scale_dev : 1.0f);
            s_coef[0] = k * inv;
            s_coef[1] = -k * inv1;
            a.pair_loss[pair] = loss;
            if (a.mean_loss && a.pairs == 1) {
                *a.mean_loss = loss;
                if (!isfinite(loss)) atomicOr(&a.flags[FLAG_NONFINITE], 1);
            } else if (a.mean_loss) {
                __threadfence();  // the pair's loss comes before the count
                s_last = atomicAdd(&a.claim[a.M], 1) == a.pairs - 1;
                __threadfence();
            }
        }
    }
    __syncthreads();
    for (long long r0 = first; r0 < last; r0 += U * PAIR_THREADS) {
        int y[U];
#pragma unroll
        for (int u = 0; u < U; u++) y[u] = r0 + u * PAIR_THREADS < last ? a.targets[r0 + u * PAIR_THREADS] : -1;
#pragma unroll
        for (int u = 0; u < U; u++)
            if (y[u] >= 0 && y[u] < a.V) a.stat[r0 + u * PAIR_THREADS].z = s_coef[w];
    }
    if (!a.mean_loss || a.pairs == 1 || !s_last) return;
    double sum = 0.0;
    for (int p = tid; p < a.pairs; p += 2 * PAIR_THREADS) sum += (double)__ldcg(a.pair_loss + p);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();  // s_sum has been read
    if (lane == 0) s_sum[warp][0] = sum;
    __syncthreads();
    if (tid == 0) {
        sum = 0.0;
        for (int i = 0; i < 2 * WARPS; i++) sum += s_sum[i][0];
        const float m = (float)(sum / a.pairs);
        *a.mean_loss = m;
        if (!isfinite(m)) atomicOr(&a.flags[FLAG_NONFINITE], 1);
    }
}

// Threads that a row of G granules gets, 32 at least, then a warp of a CTA that
// has ROWS of them.  Fewer threads a row are fewer barriers and less of a row's
// own latency, as long as there are rows enough that every SM has its 1024, and
// as long as a row is not so slow by itself (four loads in flight a thread) that
// a last round of a few rows takes long: 80 granules a thread are some 16 us.  At
// most 512, and at least eight granules each.  In bf16, log probabilities of
// 20000 rows of 2500 logits take 27 us by warps, 38 by 64 threads, 54 by 128
// (20000 of 5000 36, 40, 54; 300 of 50257 15 by 256 or 512, 19 by 1024); 32768 of
// 50257, half of them labelled, 279 by warps or 64 threads, 283 by 128, 337 by
// 256; 4000 of 150000 166 by 64, 128 by 128, 132 by 256.  (A row over a cluster of
// two to eight CTAs: 2 us less for up to 16 rows, more from 64 rows on: 150 rows
// 15 to 24.)
constexpr int ROWS = 4;

int row_threads(const Launch& L, int G, long long M) {
    int N = 32;
    while (N < 512 && ((M * N < L.num_sms * 1024LL && G >= 16 * N) || G > 80 * N)) N *= 2;
    return N;
}

// With the gradient (and without it, so that the loss has the same bits) the rows
// in flight, which are read a second time, also have to stay in L2: below 92 MB of
// them where every SM has 1024 threads.  In bf16, 32768 rows of 50257 take 848 us by
// 256 threads, 893 by 128, 982 by warps, 992 by 512 (784 by 256 once the rows' other
// inputs were loaded with the label); 4000 of 150000 339 by 512, 370 by 256 or 1024;
// 20000 of 5000 62 by warps or 64 threads, 78 by 128.
int policy_threads(const Launch& L, int G, long long M) {
    int N = row_threads(L, G, M);
    while (N < AN_THREADS && L.num_sms * 1024LL / N * G * 16 > 92000000LL) N *= 2;
    return N;
}

// The gradient alone reads and writes a row once: 20000 rows of 5000 by 64 threads,
// 32768 of 50257 by 256 (by warps 2 and 4% slower).
int grad_threads(const Launch& L, int G, long long M) {
    return G <= 256 ? 32 : std::max(row_threads(L, G, M), G <= 1280 ? 64 : G <= 2560 ? 128 : 256);
}

dim3 row_block(int N) { return dim3(N, N == 32 ? ROWS : 1); }
dim3 row_grid(int N, int M) { return dim3((unsigned)(N == 32 ? (M - 1) / ROWS + 1 : M)); }

template <typename T, bool POLICY>
void answer(const Launch& L, const void* z, void* dz, AnswerArgs a) {
    a.G = row_granules<T>(z, a.ld, a.V);
    a.same_phase = (((uintptr_t)z ^ (uintptr_t)dz) & 15) == 0;
    if (a.G <= 256) {
        L.count();
        if (a.G <= 16) answer_short<T, 8, 2, POLICY>(L, z, dz, a);
        else if (a.G <= 32) answer_short<T, 16, 2, POLICY>(L, z, dz, a);
        else if (a.G <= 64) answer_short<T, 32, 2, POLICY>(L, z, dz, a);
        else if (a.G <= 128) answer_short<T, 32, 4, POLICY>(L, z, dz, a);
        else answer_short<T, 32, 8, POLICY>(L, z, dz, a);
        return;
    }
    const int N = POLICY ? policy_threads(L, a.G, a.M) : row_threads(L, a.G, a.M);
    L.count();
    launch_k(L, k_answer<T, POLICY>, row_grid(N, a.M), row_block(N), 0, (const T*)z, (T*)dz, a);
}

template <typename T> void answer_grad(const Launch& L, const void* z, void* dz, AnswerArgs a) {
    a.G = row_granules<T>(z, a.ld, a.V);
    a.same_phase = (((uintptr_t)z ^ (uintptr_t)dz) & 15) == 0;
    const int N = grad_threads(L, a.G, a.M);
    L.count();
    launch_k(L, k_answer_grad<T>, row_grid(N, a.M), row_block(N), 0, (const T*)z, (T*)dz, a);
}

template <bool POLICY> void answer_of(const Launch& L, tt_dtype dtype, const void* z, void* dz, const AnswerArgs& a) {
    if (dtype == TT_FP32) answer<float, POLICY>(L, z, dz, a);
    else if (dtype == TT_FP16) answer<__half, POLICY>(L, z, dz, a);
    else answer<__nv_bfloat16, POLICY>(L, z, dz, a);
}

AnswerArgs rows_of(const Launch& L, const int32_t* targets, int M, int V, int ld, float tau) {
    AnswerArgs a{};
    a.targets = targets;
    a.flags = L.flags;
    a.ld = ld; a.M = M; a.V = V;
    a.it = 1.0f / tau;
    return a;
}

}  // namespace

void launch_logprobs(const Launch& L, tt_dtype dtype, const void* z, const int32_t* targets, float* logp, float* lse, int M,
                     int V, int ld, float tau) {
    if (L.dry) return;
    AnswerArgs a = rows_of(L, targets, M, V, ld, tau);
    a.logp = logp;
    a.lse = lse;
    answer_of<false>(L, dtype, z, nullptr, a);
}

void launch_policy(const Launch& L, tt_dtype dtype, const void* z, void* dz, const PolicyLoss& p, const int32_t* targets,
                   float* logp, float* row_loss, float* mean_loss, int M, int V, int ld, float tau, float dscale,
                   const float* scale_dev) {
    if (L.dry) return;
    AnswerArgs a = rows_of(L, targets, M, V, ld, tau);
    a.old = p.old_logp; a.ref = p.ref_logp; a.adv = p.adv; a.weight = p.weight;
    a.scale_dev = scale_dev;
    a.logp = logp;
    a.row_loss = row_loss;
    a.lo = p.lo; a.hi = p.hi;
    a.llo = (float)log1p(-(double)p.lo);
    a.lhi = (float)log1p((double)p.hi);
    a.beta = p.beta;
    a.dscale = dscale;
    answer_of<true>(L, dtype, z, dz, a);
    if (mean_loss) launch_row_mean(L, row_loss, M, mean_loss);
}

size_t preference_scratch_bytes(int M) { return (size_t)M * (sizeof(float4) + sizeof(int)) + sizeof(int); }

void launch_preference(const Launch& L, tt_dtype dtype, const void* z, void* dz, const PreferenceLoss& p,
                       const int32_t* targets, float* seq_logp, float* pair_loss, float* mean_loss, int M, int V, int ld,
                       float tau, float dscale, const float* scale_dev, void* scratch) {
    if (L.dry) return;
    AnswerArgs a = rows_of(L, targets, M, V, ld, tau);
    a.stat = (float4*)scratch;
    a.claim = (int*)(a.stat + M);
    answer_of<false>(L, dtype, z, nullptr, a);
    PairArgs q{};
    q.targets = targets; q.spans = p.spans; q.ref = p.ref_logp; q.scale_dev = scale_dev;
    q.stat = a.stat; q.claim = a.claim; q.flags = L.flags;
    q.seq_logp = seq_logp; q.pair_loss = pair_loss; q.mean_loss = mean_loss;
    q.M = M; q.V = V; q.pairs = p.pairs;
    q.beta = p.beta; q.gamma = p.gamma; q.smooth = p.smooth; q.k = dscale / tau; q.mean = p.mean;
    L.count();
    launch_k(L, k_pairs, dim3((unsigned)p.pairs), dim3(2 * PAIR_THREADS), 0, q);
    if (dz) {
        if (dtype == TT_FP32) answer_grad<float>(L, z, dz, a);
        else if (dtype == TT_FP16) answer_grad<__half>(L, z, dz, a);
        else answer_grad<__nv_bfloat16>(L, z, dz, a);
    }
}

}  // namespace tt
