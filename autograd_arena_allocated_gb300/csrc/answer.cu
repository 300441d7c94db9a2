// answer.cu -- losses on the probabilities of given tokens:
//
//   k_answer        rows of more than 256 granules: a label's log probability, or
//                   the clipped policy loss and its gradient; a CTA a row
//   k_answer_short  the same for shorter rows, a warp a row, in registers
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
    int* claim;                    // with stat: whether an answer has the row
    int* flags;
    long long ld;
    int M, V, G;
    float it, lo, hi, llo, lhi, beta, dscale;  // it = 1 / tau, llo = ln(1 - lo), lhi = ln(1 + hi)
    bool same_phase;
};

// The label of a row, -1 for none; one that is out of range counts as none.
__device__ __forceinline__ int label_of(const int32_t* targets, long long row, int V, int* flags, bool first) {
    const int y = targets[row];
    if (y >= -1 && y < V) return y;
    if (first) atomicOr(&flags[FLAG_BAD_TOKEN], 1);
    return -1;
}

// ln pi from the reference and the sum: the difference of the logits comes first,
// so that nothing is lost where both are far from zero (a mask's lowest value).
// The logarithm is taken of the mantissa, as in lse_of.
__device__ __forceinline__ float logp_of(float zy, float R, float s, float it) {
    int e = 0;
    const float m = frexpf(s, &e);
    return (float)(((double)zy - (double)R) * (double)it - ((double)e * 0.6931471805599453 + (double)logf(m)));
}

// what the policy loss of a row needs beside its logits
struct PolicyRow {
    float old = 0.0f, ref = 0.0f, A = 0.0f, w = 1.0f;
    bool fresh;
    __device__ __forceinline__ PolicyRow(const AnswerArgs& a, long long row) : fresh(!a.old) {
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
            v = fmaf(a.beta, e - x, v);
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

// k (onehot - softmax) over a row, R and s its reference and sum (N threads; no
// barrier: the label's column is written by the thread that has its granule)
template <typename T>
__device__ __forceinline__ void row_gradient(const RowView<T>& view, T* drow, long long ld, int tid, int N, bool same_phase,
                                             float R, float s, float ct, float k, int y, float zy) {
    if (k == 0.0f) {
        zero_row(drow, ld, tid, N);
        return;
    }
    const Slice<T>& sl = view.s;
    const float At = -__fdividef(k, s);
    view.template gradient<true, false>(tid, N, drow, same_phase, R, ct, At, 0.0f);
    const int i = sl.at(y) >> 4;
    const int owner = sl.inner(i) ? (i - sl.i0) % N : sl.head && i == 0 ? 0 : view.tail_tid;
    if (tid == owner) drow[y] = Elem<T>::put(fmaf(At, exp_of(zy, R, ct), k));
    for (long long c = view.V + tid; c < ld; c += N) drow[c] = Elem<T>::put(0.0f);
}

constexpr int AN_THREADS = 1024;  // most threads of a CTA

template <typename T, bool POLICY>
__global__ void __launch_bounds__(AN_THREADS, 1) k_answer(const T* z, T* dz, const AnswerArgs a) {
    pdl_wait();
    __shared__ float2 s_part[AN_THREADS / 32];
    const int N = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = a.V;
    const long long row = blockIdx.x;
    const int y = label_of(a.targets, row, V, a.flags, tid == 0);
    T* drow = dz ? dz + row * a.ld : nullptr;
    if (y < 0) {
        if (tid == 0) {
            if (a.logp) a.logp[row] = 0.0f;
            if (a.lse) a.lse[row] = 0.0f;
            if (a.row_loss) a.row_loss[row] = 0.0f;
            if (a.stat) a.stat[row] = make_float4(0.0f, 1.0f, 0.0f, 0.0f), a.claim[row] = 0;
        }
        if (drow) zero_row(drow, a.ld, tid, N);
        return;
    }
    const Slice<T> s(z, row, a.ld, V, 0, a.G);
    const float zy = Elem<T>::get(z + row * a.ld + y);
    const float ct = LOG2E * a.it, lift = 20.0f / fmaxf(1.0f, a.it);
    const RowView<T> view{s, V, nullptr};
    float R, sum, none;
    view.template sums<false, true>(tid, N, 0.0f, ct, lift, R, none, sum);
    merge(R, sum, ct);
    if (lane == 0) s_part[warp] = make_float2(R, sum);
    __syncthreads();  // also: everything has been read (dz may be z)
    const float2 p = lane < N / 32 ? s_part[lane] : make_float2(-INFINITY, 0.0f);
    R = p.x, sum = p.y;
    merge(R, sum, ct);
    const float lp = logp_of(zy, R, sum, a.it);
    float k = 0.0f;
    if (POLICY) {
        const PolicyRow pr(a, row);
        const float2 f = pr.loss(a, lp);
        if (tid == 0) a.row_loss[row] = f.x;
        k = f.y * a.it * a.dscale;
        if (a.scale_dev) k *= *a.scale_dev;
    }
    if (tid == 0) {
        if (a.logp) a.logp[row] = lp;
        if (a.lse) a.lse[row] = (float)lse_of(R, sum, a.it);
        if (a.stat) a.stat[row] = make_float4(R, sum, 0.0f, lp), a.claim[row] = 0;
    }
    if (POLICY && dz) row_gradient(view, drow, a.ld, tid, N, a.same_phase, R, sum, ct, k, y, zy);
}

// Rows of up to 32 GL granules, a warp each, lane l the granules l + 32 j.
constexpr int AS_WARPS = 4;

template <typename T, int GL, bool POLICY>
__global__ void __launch_bounds__(AS_WARPS * 32) k_answer_short(const T* z, T* dz, const AnswerArgs a) {
    pdl_enter();
    using E = Elem<T>;
    constexpr int H = E::EPG / 2;
    const int lane = threadIdx.x & 31, V = a.V;
    const long long row = blockIdx.x * (long long)AS_WARPS + (threadIdx.x >> 5);
    if (row >= a.M) return;
    const int y = label_of(a.targets, row, V, a.flags, lane == 0);
    T* drow = dz ? dz + row * a.ld : nullptr;
    if (y < 0) {
        if (lane == 0) {
            if (a.logp) a.logp[row] = 0.0f;
            if (a.lse) a.lse[row] = 0.0f;
            if (a.row_loss) a.row_loss[row] = 0.0f;
            if (a.stat) a.stat[row] = make_float4(0.0f, 1.0f, 0.0f, 0.0f), a.claim[row] = 0;
        }
        if (drow) zero_row(drow, a.ld, lane, 32);
        return;
    }
    const Slice<T> s(z, row, a.ld, V, 0, a.G);
    const float zy = E::get(z + row * a.ld + y), ct = LOG2E * a.it;
    f2 e[GL][H];
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < GL; j++) {
        const int i = lane + 32 * j;
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
    m = warp_max(m);
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
    sum = warp_sum(sum);
    const float lp = logp_of(zy, m, sum, a.it);
    float k = 0.0f;
    if (POLICY) {
        const PolicyRow pr(a, row);
        const float2 f = pr.loss(a, lp);
        if (lane == 0) a.row_loss[row] = f.x;
        k = f.y * a.it * a.dscale;
        if (a.scale_dev) k *= *a.scale_dev;
    }
    if (lane == 0) {
        if (a.logp) a.logp[row] = lp;
        if (a.lse) a.lse[row] = (float)lse_of(m, sum, a.it);
        if (a.stat) a.stat[row] = make_float4(m, sum, 0.0f, lp), a.claim[row] = 0;
    }
    if (!POLICY || !dz) return;
    __syncwarp();  // everything has been read (dz may be z)
    if (k == 0.0f) {
        zero_row(drow, a.ld, lane, 32);
        return;
    }
    const float At = -__fdividef(k, sum);
    const f2 at2 = pk(At, At);
    uint4* const d0 = reinterpret_cast<uint4*>(drow + s.col(0));
    const int iy = s.at(y) >> 4;
#pragma unroll
    for (int j = 0; j < GL; j++) {
        const int i = lane + 32 * j;
        if (i >= s.n) continue;
        f2 r[H];
#pragma unroll
        for (int h = 0; h < H; h++) r[h] = mul2(e[j][h], at2);
        if (a.same_phase && s.inner(i)) d0[i] = E::pack(r);
        else store_edge(s, i, drow, V, r);
        if (i == iy) drow[y] = E::put(fmaf(At, zy == m ? 1.0f : exp_of(zy, m, ct), k));
    }
    for (long long c = V + lane; c < a.ld; c += 32) drow[c] = E::put(0.0f);
}

// rows of blockDim.y at a time, blockDim.x threads each
template <typename T>
__global__ void __launch_bounds__(AN_THREADS, 1) k_answer_grad(const T* z, T* dz, const AnswerArgs a) {
    pdl_wait();
    const long long row = blockIdx.x * (long long)blockDim.y + threadIdx.y;
    if (row >= a.M) return;
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
    RowView<T> view{s, a.V, nullptr};
    if (N == 32) view.tail_tid = 1;
    // the label's logit is its granule's owner's to read, before that thread writes
    const int i = s.at(y) >> 4;
    const int owner = s.inner(i) ? (i - s.i0) % N : s.head && i == 0 ? 0 : view.tail_tid;
    const float zy = tid == owner ? Elem<T>::get(z + row * a.ld + y) : 0.0f;
    row_gradient(view, drow, a.ld, tid, N, a.same_phase, st.x, st.y, ct, k, y, zy);
}

struct PairArgs {
    const int32_t *targets, *spans;
    const float *ref, *scale_dev;
    float4* stat;
    int *claim, *flags;
    float *seq_logp, *pair_loss;
    int M, V;
    float beta, gamma, smooth, k;  // k = dscale / tau
    bool mean;
};
constexpr int PAIR_THREADS = 256;

__device__ __forceinline__ double softplus(double x) { return fmax(x, 0.0) + log1p(exp(-fabs(x))); }

// One CTA a pair: its answers' sums in a fixed order, in 64 bits (an answer's
// sum is thousands, the difference of two a few), the loss, the rows' coefficients.
__global__ void __launch_bounds__(PAIR_THREADS) k_pairs(const PairArgs a) {
    pdl_enter();
    __shared__ double s_sum[PAIR_THREADS / 32][2], s_score[2];
    __shared__ int s_n[PAIR_THREADS / 32];
    __shared__ float s_coef[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long pair = blockIdx.x;
    int first[2], last[2], n_of[2] = {0, 0};
    bool bad = false;
    for (int w = 0; w < 2; w++) {
        first[w] = a.spans[(2 * pair + w) * 2];
        last[w] = a.spans[(2 * pair + w) * 2 + 1];
        if (first[w] < 0 || first[w] > last[w] || last[w] > a.M) {
            bad = true;
            first[w] = last[w] = 0;
        }
        double total = 0.0, score = 0.0;
        int n = 0;
        for (long long r = first[w] + tid; r < last[w]; r += PAIR_THREADS) {
            const int y = a.targets[r];
            if (y < 0 || y >= a.V) continue;
            if (atomicExch(&a.claim[r], 1)) bad = true;  // in two answers
            const double lp = a.stat[r].w;
            total += lp;
            score += a.ref ? lp - (double)a.ref[r] : lp;
            n++;
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
        __syncthreads();
        if (tid == 0) {
            total = score = 0.0;
            n = 0;
            for (int i = 0; i < PAIR_THREADS / 32; i++) {
                total += s_sum[i][0];
                score += s_sum[i][1];
                n += s_n[i];
            }
            n_of[w] = a.mean ? max(n, 1) : 1;
            s_score[w] = score / n_of[w];
            if (a.seq_logp) a.seq_logp[2 * pair + w] = (float)total;
        }
        __syncthreads();
    }
    if (bad) atomicOr(&a.flags[FLAG_BAD_TOKEN], 1);
    if (tid == 0) {
        const double v = (double)a.beta * (s_score[0] - s_score[1]) - (double)a.gamma, e = a.smooth;
        a.pair_loss[pair] = (float)((1.0 - e) * softplus(-v) + (e > 0.0 ? e * softplus(v) : 0.0));
        const double dv = e / (1.0 + exp(-v)) - (1.0 - e) / (1.0 + exp(v));
        const double k = dv * (double)a.beta * (double)a.k * (a.scale_dev ? (double)*a.scale_dev : 1.0);
        s_coef[0] = (float)(k / n_of[0]);
        s_coef[1] = (float)(-k / n_of[1]);
    }
    __syncthreads();
    for (int w = 0; w < 2; w++)
        for (long long r = first[w] + tid; r < last[w]; r += PAIR_THREADS) {
            const int y = a.targets[r];
            if (y >= 0 && y < a.V) a.stat[r].z = s_coef[w];
        }
}

// threads of a CTA that a row of G granules gets: enough that a thread has a
// few granules, and more where there are fewer rows than the SMs hold
int row_threads(const Launch& L, int G, long long M) {
    int N = G <= 1280 ? 128 : G <= 8192 ? 256 : G <= 16384 ? 512 : 1024;
    while (N < AN_THREADS && M * N <= L.num_sms * 512LL && G > 4 * N) N *= 2;
    return N;
}

template <typename T, bool POLICY>
void answer(const Launch& L, const void* z, void* dz, AnswerArgs a) {
    a.G = row_granules<T>(z, a.ld, a.V);
    a.same_phase = (((uintptr_t)z ^ (uintptr_t)dz) & 15) == 0;
    L.count();
    if (a.G <= 256) {
        const dim3 grid((unsigned)((a.M - 1) / AS_WARPS + 1)), block(AS_WARPS * 32);
        if (a.G <= 32) launch_k(L, k_answer_short<T, 1, POLICY>, grid, block, 0, (const T*)z, (T*)dz, a);
        else if (a.G <= 64) launch_k(L, k_answer_short<T, 2, POLICY>, grid, block, 0, (const T*)z, (T*)dz, a);
        else if (a.G <= 128) launch_k(L, k_answer_short<T, 4, POLICY>, grid, block, 0, (const T*)z, (T*)dz, a);
        else launch_k(L, k_answer_short<T, 8, POLICY>, grid, block, 0, (const T*)z, (T*)dz, a);
        return;
    }
    launch_k(L, k_answer<T, POLICY>, dim3((unsigned)a.M), dim3(row_threads(L, a.G, a.M)), 0, (const T*)z, (T*)dz, a);
}

template <typename T> void answer_grad(const Launch& L, const void* z, void* dz, AnswerArgs a) {
    a.G = row_granules<T>(z, a.ld, a.V);
    a.same_phase = (((uintptr_t)z ^ (uintptr_t)dz) & 15) == 0;
    const int N = a.G <= 256 ? 32 : row_threads(L, a.G, a.M), rows = N == 32 ? 4 : 1;
    L.count();
    launch_k(L, k_answer_grad<T>, dim3((unsigned)((a.M - 1) / rows + 1)), dim3(N, rows), 0, (const T*)z, (T*)dz, a);
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

size_t preference_scratch_bytes(int M) { return (size_t)M * (sizeof(float4) + sizeof(int)); }

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
    q.seq_logp = seq_logp; q.pair_loss = pair_loss;
    q.M = M; q.V = V;
    q.beta = p.beta; q.gamma = p.gamma; q.smooth = p.smooth; q.k = dscale / tau; q.mean = p.mean;
    L.count();
    launch_k(L, k_pairs, dim3((unsigned)p.pairs), dim3(PAIR_THREADS), 0, q);
    if (dz) {
        if (dtype == TT_FP32) answer_grad<float>(L, z, dz, a);
        else if (dtype == TT_FP16) answer_grad<__half>(L, z, dz, a);
        else answer_grad<__nv_bfloat16>(L, z, dz, a);
    }
    if (mean_loss) launch_row_mean(L, pair_loss, p.pairs, mean_loss);
}

}  // namespace tt
