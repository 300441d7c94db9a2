// distill.cuh -- what the distillation kernels (distill.cu, distill_stream.cu)
// share: arguments, and a row's coefficients and gradient.
#pragma once

#include "head_row.cuh"

namespace tt {
namespace head {

// With q = softmax(z / tau), s = softmax(z), the list's probabilities p_j at
// columns i_j, W their sum (plus p_r, the teacher's mass outside the list,
// when it is known and the student has any there, q_r):
//   loss = alpha tau^2 (sum p_j (ln p_j - ln q_ij) + p_r (ln p_r - ln q_r)) + (1 - alpha) (lse(z) - z_y)
//   dz_i = g alpha tau (W q_i - p_i)            on the list
//        = g alpha tau q_i (W - p_r / q_r)      off it
//        + g (1 - alpha) (s_i - [i = y])
// One pass over the row sums the exponentials, a second writes the gradient as
// if no column were listed, and the list's columns are then written over.
// Where q_r is needed (t_lse) the first pass leaves the listed logits out, so
// that q_r is not a difference; their own exponentials are added from the list.
// The sum off the list, su, may be any fraction of the sum of all, sa.  At the
// common reference R a column 87 tau below it is lost; so below OFF_OWN of sa
// the sum is formed again at a reference of its own, Ro: ln q_r is then a
// difference of logarithms, and the second pass takes
//   ks ((W + p_r) e^((Ro - R) / tau) / sa - p_r / su) e^((z - Ro) / tau)
// whose coefficient does not grow with the list's lead.  Below e^-700 q_r
// counts as 0, as it nearly is in 64 bits: so low are columns that a mask of
// large negative numbers hides.
struct DistillArgs {
    const float* t_vals;
    const int32_t* t_idx;
    const float* t_lse;
    const int32_t* targets;
    const float* scale_dev;
    float* row_loss;
    int* flags;
    long long ld;
    int M, V, k, Gs, cs, nbuf;
    float alpha, tau, dscale;
    bool same_phase;  // a row of dz starts at the same place of a 16-byte line as its row of z
};

// tau as a power that one softmax's terms are of the other's: 1 to 4, else 0
__device__ __forceinline__ int power_of(float tau) {
    return tau == 1.0f ? 1 : tau == 2.0f ? 2 : tau == 3.0f ? 3 : tau == 4.0f ? 4 : 0;
}

// At 2^((z - m) ct) + A1 e^(z - m) of a granule (S, H: which of the two there
// are); both coefficients 0: zeros, whatever the logits are.
template <typename T, bool S, bool H, int PW> struct Grad {
    using E = Elem<T>;
    static constexpr int P = E::EPG / 2;
    float m, ct, At, A1;
    bool zero, slow;  // slow: the form without overflow, which also serves for zeros
    f2 c2, c1, nt2, n12, at2, a12;
    __device__ __forceinline__ Grad(float m_, float ct_, float At_, float A1_) : m(m_), ct(ct_), At(At_), A1(A1_) {
        zero = At == 0.0f && A1 == 0.0f;
        slow = zero || is_far(m);
        const float nt = -(m * ct), n1 = -(m * LOG2E);
        const float bt = S ? At * unbias(m, ct, nt) : 0.0f;
        const float b1 = H ? A1 * (PW ? powi<PW>(unbias(m, ct, nt)) : unbias(m, LOG2E, n1)) : 0.0f;
        c2 = pk(ct, ct);
        c1 = pk(LOG2E, LOG2E);
        nt2 = pk(nt, nt);
        n12 = pk(n1, n1);
        at2 = pk(bt, bt);
        a12 = pk(b1, b1);
    }
    __device__ __forceinline__ void operator()(const uint4& u, f2* r) const {
        f2 e[P];
        E::unpack(u, e);
        float x, y;
#pragma unroll
        for (int j = 0; j < P; j++) {
            if (PW) {
                unpk(fma2(e[j], c2, nt2), x, y);
                const f2 q = pk(ex2f(x), ex2f(y));
                r[j] = fma2(powi<PW>(q), a12, mul2(q, at2));
                continue;
            }
            if (S) {
                unpk(fma2(e[j], c2, nt2), x, y);
                r[j] = mul2(pk(ex2f(x), ex2f(y)), at2);
            }
            if (H) {
                unpk(fma2(e[j], c1, n12), x, y);
                r[j] = S ? fma2(pk(ex2f(x), ex2f(y)), a12, r[j]) : mul2(pk(ex2f(x), ex2f(y)), a12);
            }
        }
    }
    __device__ __forceinline__ float of(float z) const {
        return zero ? 0.0f : (S ? At * exp_of(z, m, ct) : 0.0f) + (H ? A1 * exp_of(z, m, LOG2E) : 0.0f);
    }
    __device__ __forceinline__ void slowly(const uint4& u, f2* r) const {
        f2 e[P];
        E::unpack(u, e);
        float x, y;
#pragma unroll
        for (int j = 0; j < P; j++) {
            unpk(e[j], x, y);
            r[j] = pk(of(x), of(y));
        }
    }
};

// stores slot i's gradient: as a granule, or the elements that lie in the row
template <typename T>
__device__ __forceinline__ void store_edge(const Slice<T>& s, int i, T* drow, int V, const f2* r) {
    const int c0 = s.col(i);
#pragma unroll
    for (int j = 0; j < Elem<T>::EPG / 2; j++) {
        float x, y;
        unpk(r[j], x, y);
        const int c = c0 + 2 * j;
        if (c >= 0 && c < V) drow[c] = Elem<T>::put(x);
        if (c + 1 >= 0 && c + 1 < V) drow[c + 1] = Elem<T>::put(y);
    }
}

// The teacher's normaliser and mass from its list's warps (s_lw: largest logit
// and sum of exponentials, or, where the normaliser is known, the probabilities'
// sum; whether an entry is used), and the coefficients of loss and gradient.
// su_ is off the list, sl on it, where these are apart.
constexpr float OFF_OWN = 1e-8f;    // of sa: 18 tau, which leaves 69 to the columns
constexpr float OFF_MIN = -700.0f;  // of ln q_r

// whether a sum off the list, of sums st and sl off and on it, needs that reference
__device__ __forceinline__ bool off_own(float st, float sl) { return st <= OFF_OWN * (st + sl); }

struct Coefs {
    float base = -INFINITY, W = 0.0f, pr = 0.0f, ks, kh, Al, At, A1, su, sa;  // su: the sum off the list, sa: of all
    float Rp, A1p;  // the second pass's reference, that of At, and A1 for it
    float lq = 0.0f;  // ln q_r where su has a reference of its own
    bool soft, own, used = false;
    // R, Ro: the reference of s1 and sl, and of su_
    __device__ __forceinline__ Coefs(const DistillArgs& a, const float4* s_lw, int nlw, bool rest, bool soft_on, bool hard,
                                     float tl, float g_all, float R, float Ro, float s1, float su_, float sl, float it,
                                     float ct)
        : su(su_), sa(su_), own(Ro != R) {
        if (rest) {
            base = tl;
            for (int w = 0; w < nlw; w++) {
                W += s_lw[w].y;
                used |= s_lw[w].z != 0.0f;
            }
        } else {
            for (int w = 0; w < nlw; w++) {
                base = fmaxf(base, s_lw[w].x);
                used |= s_lw[w].z != 0.0f;
            }
            float ts = 0.0f;
            for (int w = 0; w < nlw; w++) ts += s_lw[w].y * rescale(s_lw[w].x, base, LOG2E);
            W = ts != 0.0f ? 1.0f : 0.0f;  // entries of probability 0 only: nothing
            base += logf(ts);
        }
        soft = used && soft_on;
        ks = g_all * a.alpha * a.tau;
        kh = hard ? g_all * (1.0f - a.alpha) : 0.0f;
        Rp = R;
        A1 = A1p = hard ? __fdividef(kh, s1) : 0.0f;
        if (rest) {
            sa = (own ? su * rescale(Ro, R, ct) : su) + sl;
            if (su > 0.0f) pr = fmaxf(1.0f - W, 0.0f);
            if (own) {
                lq = ln_off(su, sa, Ro, R, it);
                if (!(lq >= OFF_MIN)) pr = 0.0f;
            }
        }
        const float rt = __fdividef(soft ? ks : 0.0f, sa);
        Al = (W + pr) * rt;
        At = W * rt;
        if (pr > 0.0f) {
            if (own) {
                At = Al * rescale(Ro, R, ct) - (soft ? ks * __fdividef(pr, su) : 0.0f);
                A1p = A1 * rescale(Ro, R, LOG2E);
                Rp = Ro;
            } else {
                At = rt * (W + pr - pr * __fdividef(sa, su));
            }
        }
    }
    static __device__ __forceinline__ float ln_off(float su, float sa, float Ro, float R, float it) {
        return (Ro - R) * it + logf(__fdividef(su, sa));
    }
    // an entry's part of sum p (ln p - ln q): teacher's logit t, student's z
    __device__ __forceinline__ float kl(float t, float z, float R, float it) const {
        const float lp = t - base, p = ex2f(lp * LOG2E);
        return t != -INFINITY && (p > 0.0f || p != p) ? p * (lp - ((z - R) * it - logf(sa))) : 0.0f;
    }
    __device__ __forceinline__ float loss(const DistillArgs& a, const float* s_ll, int nlw, bool hard, float R, float s1,
                                          float zy) const {
        float l = 0.0f;
        if (soft) {
            for (int w = 0; w < nlw; w++) l += s_ll[w];
            if (pr > 0.0f) l += pr * (logf(pr) - (own ? lq : logf(__fdividef(su, sa))));
            l *= a.alpha * a.tau * a.tau;
        }
        if (hard) l += (1.0f - a.alpha) * ((R - zy) + logf(s1));  // R may be far from 0
        return l;
    }
    __device__ __forceinline__ float listed(float t, float z, float R, float ct, bool hard, bool target) const {
        float r = 0.0f;
        if (soft) r = Al * exp_of(z, R, ct) - (t == -INFINITY ? 0.0f : ks * ex2f((t - base) * LOG2E));
        if (hard) r += A1 * exp_of(z, R, LOG2E) - (target ? kh : 0.0f);
        return r;
    }
    // the target's column, off the list
    __device__ __forceinline__ float target(float z, float R, float ct) const {
        return A1 * exp_of(z, R, LOG2E) - kh + (soft ? At * exp_of(z, Rp, ct) : 0.0f);
    }
};

// G: granules of a row.  N: threads of a CTA.
constexpr int DL_THREADS = 512;  // most of them
template <typename T> bool distill_stream(const Launch& L, const void* z, void* dz, DistillArgs a, int G, int N);

}  // namespace head
}  // namespace tt
