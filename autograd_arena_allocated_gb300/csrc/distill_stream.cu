// distill_stream.cu -- distillation of rows that are not held on chip.
#include "distill.cuh"

namespace tt {
namespace {

using namespace head;

// Rows that no CTA holds, and rows so short that one's own chain (barriers,
// merge, coefficients) is longer than its passes: a CTA of N threads goes over
// the row in memory twice, with no copy on chip; the second time, last granules
// first, much of it is in L2 (or, a short one, in L1): the loads and stores of
// that pass are marked as the last use, and the rows in flight (two of 512
// threads an SM, or eight of 128) stay below L2's size for 16-bit vocabularies.
// With t_lse the listed columns are known from a bit each, by which the first
// pass leaves them out.
//
// Long rows: memory, and what of the second read misses L2.  1000 rows of
// 120000 logits, 512 threads: 107 us in 16 bits (66% of the measured copy
// rate; forwards without the marks 122 us, a cluster of CTAs that hold the row
// 194 us), 214 us in 32 bits; 999 rows of 50257 in 32 bits 89 us (92 us by
// clusters).  Short rows, 128 threads: a row's fixed work, at 32 warps an SM;
// 10000 rows of 3000 16-bit logits 61 us, 4000 of 8192 40 us (149 and 73 on chip).
template <typename T> __device__ __forceinline__ uint4 drop(uint4 u, uint32_t bits) {
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
    constexpr int PER = 4 / sizeof(T);
    constexpr uint32_t LOW = PER == 2 ? 0xFFFFu : 0xFFFFFFFFu;
#pragma unroll
    for (int e = 0; e < 4 * PER; e++) {
        const uint32_t m = LOW << (e % PER * 16);
        if (bits >> e & 1u) w[e / PER] = (w[e / PER] & ~m) | (Elem<T>::NINF & m);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T> struct RowView {
    using E = Elem<T>;
    static constexpr int U = 4;
    const Slice<T>& s;
    int V;
    const uint8_t* bits;  // NULL: every column counts

    __device__ __forceinline__ uint4 masked(int i, uint4 u) const {
        if (bits) {
            const uint32_t b = E::EPG == 8 ? bits[i] : bits[i >> 1] >> ((i & 1) * 4) & 15u;
            if (b) u = drop<T>(u, b);
        }
        return u;
    }
    // f(slot) for the thread's share of the slots that are not wholly inside the row
    template <typename F> __device__ __forceinline__ void edges(int tid, F&& f) const {
        const int i = tid == 0 && s.head ? 0 : tid == 32 && s.tail ? s.n - 1 : -1;
        if (i >= 0) f(i);
    }
    // sums of exponentials (Sums) of thread tid's granules
    template <bool SA, bool SB, int PW = 0>
    __device__ __forceinline__ void sums(int tid, int N, float ca, float cb, float lift, float& R, float& sa, float& sb) const {
        Sums<T, SA, SB, PW> q(ca, cb, lift);
        const uint4* v = reinterpret_cast<const uint4*>(s.base);
        int i = s.i0 + tid;
        q.start(warp_max(i < s.i1 ? E::value(E::gmax(masked(i, v[i]))) : -INFINITY));
        for (; i + (U - 1) * N < s.i1; i += U * N) {
            uint4 u[U];
#pragma unroll
            for (int j = 0; j < U; j++) u[j] = v[i + j * N];
#pragma unroll
            for (int j = 0; j < U; j++) u[j] = masked(i + j * N, u[j]);
            q.look(E::max2(E::max2(E::gmax(u[0]), E::gmax(u[1])), E::max2(E::gmax(u[2]), E::gmax(u[3]))));
            q.take(u);
        }
        if (i < s.i1) {
            uint4 u[U - 1];
#pragma unroll
            for (int j = 0; j < U - 1; j++) u[j] = v[min(i + j * N, s.i1 - 1)];
#pragma unroll
            for (int j = 0; j < U - 1; j++)
                if (i + j * N < s.i1) {
                    const uint4 x = masked(i + j * N, u[j]);
                    q.look(E::gmax(x));
                    q.take(x);
                }
        }
        edges(tid, [&](int e) {
            const uint4 x = masked(e, granule(s, e, V));
            q.look(E::gmax(x));
            q.take(x);
        });
        float tm;
        if (q.finish(tm, sa, sb)) {
            auto far = [&](int g) {
                f2 e[E::EPG / 2];
                E::unpack(masked(g, granule(s, g, V)), e);
#pragma unroll
                for (int j = 0; j < E::EPG / 2; j++) {
                    float x, y;
                    unpk(e[j], x, y);
                    q.take_far(x, sa, sb);
                    q.take_far(y, sa, sb);
                }
            };
#pragma unroll 1
            for (int g = s.i0 + tid; g < s.i1; g += N) far(g);
            edges(tid, far);
        }
        R = q.R;
    }
    template <bool S, bool H, int PW = 0>
    __device__ __forceinline__ void gradient(int tid, int N, T* drow, bool same_phase, float m, float ct, float At, float A1) const {
        uint4* const d0 = reinterpret_cast<uint4*>(drow + s.col(0));
        const uint4* v = reinterpret_cast<const uint4*>(s.base);
        const Grad<T, S, H, PW> grad(m, ct, At, A1);
        int i = s.i0 + tid;
        if (!grad.slow && same_phase && i < s.i1) {
            const int mine = (s.i1 - 1 - i) / N + 1, last = i + mine / U * U * N;
            if (last < s.i1) {
                uint4 u[U - 1];
#pragma unroll
                for (int j = 0; j < U - 1; j++) u[j] = __ldcs(v + min(last + j * N, s.i1 - 1));
#pragma unroll
                for (int j = 0; j < U - 1; j++)
                    if (last + j * N < s.i1) {
                        f2 r[E::EPG / 2];
                        grad(u[j], r);
                        __stcs(d0 + last + j * N, E::pack(r));
                    }
            }
            for (int g = last - U * N; g >= i; g -= U * N) {
                uint4 u[U];
#pragma unroll
                for (int j = 0; j < U; j++) u[j] = __ldcs(v + g + j * N);
#pragma unroll
                for (int j = 0; j < U; j++) {
                    f2 r[E::EPG / 2];
                    grad(u[j], r);
                    __stcs(d0 + g + j * N, E::pack(r));
                }
            }
            i = s.i1;
        }
        auto one = [&](int g) {
            f2 r[E::EPG / 2];
            const uint4 x = granule(s, g, V);
            if (grad.slow) grad.slowly(x, r);
            else grad(x, r);
            store_edge(s, g, drow, V, r);
        };
#pragma unroll 1
        for (; i < s.i1; i += N) one(i);
        edges(tid, one);
    }
};

template <typename T, bool REST>
__global__ void __launch_bounds__(DL_THREADS, 2) k_distill_stream(const T* z, T* dz, const DistillArgs a) {
    pdl_wait();
    extern __shared__ __align__(16) char smem[];
    constexpr int LW = LIST_MAX / 32, PARTS = DL_THREADS / 32 + LW;
    static_assert(PARTS <= 32, "a lane a part");
    const int N = blockDim.x;
    uint32_t* s_bits = reinterpret_cast<uint32_t*>(smem);  // listed columns, by their place in the granules
    __shared__ float4 s_part[PARTS], s_lw[LW];
    __shared__ float s_ll[LW];
    __shared__ int s_flag;  // the target is on the list
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int k = a.k, V = a.V, nlw = (k + 31) / 32, pw = power_of(a.tau);
    constexpr bool rest = REST;
    const bool soft_on = a.alpha > 0.0f, hard_on = a.targets && a.alpha < 1.0f;
    const float it = 1.0f / a.tau, ct = LOG2E * it, lift = 20.0f / fmaxf(1.0f, it);
    float g_all = a.dscale;
    if (a.scale_dev) g_all *= *a.scale_dev;
    for (int w = tid; w < (a.Gs * Elem<T>::EPG + 31) / 32; w += N) s_bits[w] = 0;
    if (tid == 0) s_flag = 0;
    const long long stride = gridDim.x;
    int c_next = -1, y_next = -1;
    float t_next = -INFINITY;
    auto fetch = [&](long long r) {  // the list is known a row ahead
        if (r >= a.M) return;
        if (tid < k) {
            c_next = a.t_idx[r * k + tid];
            t_next = a.t_vals[r * k + tid];
        }
        if (a.targets) y_next = a.targets[r];
    };
    fetch(blockIdx.x);
    for (long long row = blockIdx.x; row < a.M; row += stride) {
        const Slice<T> s(z, row, a.ld, V, 0, a.Gs);
        const T* zr = z + row * a.ld;
        int c = c_next, y = y_next;
        float t = t_next * it;
        const float tl = rest ? a.t_lse[row] : 0.0f;
        bool bad = (y < -1 || y >= V) && tid == 0;
        if (y < -1 || y >= V) y = -1;
        const bool hard = hard_on && y >= 0;
        __syncthreads();  // the last row's bits are cleared
        const int at = c + s.ph / (int)sizeof(T);
        if (c < 0 || c >= V) {
            bad |= c != -1;
            c = -1;
        } else if (atomicOr(&s_bits[at >> 5], 1u << (at & 31)) >> (at & 31) & 1u) {  // listed twice
            bad = true;
            c = -1;
        }
        if (c < 0) t = -INFINITY;
        const float zc = c >= 0 ? Elem<T>::get(zr + c) : -INFINITY;
        const float zy = tid == 0 && hard ? Elem<T>::get(zr + y) : 0.0f;
        if (c >= 0 && c == y) s_flag = 1;
        if (bad) atomicOr(&a.flags[FLAG_BAD_TOKEN], 1);
        fetch(row + stride);
        if (rest) __syncthreads();  // the bits are set

        // first pass
        const RowView<T> view{s, V, rest ? reinterpret_cast<const uint8_t*>(s_bits) : nullptr};
        float R = -INFINITY, s1 = 0.0f, st = 0.0f, sl = 0.0f;
        const int p2 = hard && soft_on ? pw : 0;
        if (!soft_on) view.template sums<true, false>(tid, N, LOG2E, ct, lift, R, s1, st);
        else if (!hard || p2 == 1) view.template sums<false, true>(tid, N, LOG2E, ct, lift, R, s1, st);
        else if (p2 == 2) view.template sums<true, true, 2>(tid, N, LOG2E, ct, lift, R, s1, st);
        else if (p2 == 3) view.template sums<true, true, 3>(tid, N, LOG2E, ct, lift, R, s1, st);
        else if (p2 == 4) view.template sums<true, true, 4>(tid, N, LOG2E, ct, lift, R, s1, st);
        else view.template sums<true, true>(tid, N, LOG2E, ct, lift, R, s1, st);
        if (p2 == 1) s1 = st;
        merge(R, s1, st, sl, ct, hard, false);
        if (lane == 0) s_part[warp] = make_float4(R, s1, st, 0.0f);
        // the list: the teacher's side, and the exponentials that the pass has left out
        if (warp < nlw) {
            const float tm = rest ? tl : warp_max(t);
            const float ts = warp_sum(t != -INFINITY ? ex2f((t - tm) * LOG2E) : 0.0f);
            const bool used = __any_sync(0xffffffffu, c >= 0);
            if (lane == 0) s_lw[warp] = make_float4(tm, ts, used ? 1.0f : 0.0f, 0.0f);
            if (rest) {
                const float Rl = warp_max(zc);
                const float l1 = warp_sum(zc != -INFINITY ? exp_of(zc, Rl, LOG2E) : 0.0f);
                const float lts = warp_sum(zc != -INFINITY ? exp_of(zc, Rl, ct) : 0.0f);
                if (lane == 0) s_part[N / 32 + warp] = make_float4(Rl, l1, 0.0f, lts);
            }
        }
        __syncthreads();
        float Ro;
        {
            const float4 p = lane < N / 32 + (rest ? nlw : 0) ? s_part[lane] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
            R = p.x; s1 = p.y; st = p.z; sl = p.w;
            merge(R, s1, st, sl, ct, hard, rest);
            Ro = R;
            if (rest && off_own(st, sl)) {
                Ro = lane < N / 32 ? p.x : -INFINITY;  // the other parts are the list's
                st = lane < N / 32 ? p.z : 0.0f;
                merge(Ro, st, ct);
            }
        }
        const Coefs f(a, s_lw, nlw, rest, soft_on, hard, tl, g_all, R, Ro, s1, st, sl, it, ct);

        // second pass
        T* drow = dz ? dz + row * a.ld : nullptr;
        if (dz) {
            const float As = f.soft ? f.At : 0.0f;
            if (f.soft && hard && p2 == 2) view.template gradient<true, true, 2>(tid, N, drow, a.same_phase, f.Rp, ct, As, f.A1p);
            else if (f.soft && hard && p2 == 3) view.template gradient<true, true, 3>(tid, N, drow, a.same_phase, f.Rp, ct, As, f.A1p);
            else if (f.soft && hard && p2 == 4) view.template gradient<true, true, 4>(tid, N, drow, a.same_phase, f.Rp, ct, As, f.A1p);
            else if (f.soft && hard && p2 != 1) view.template gradient<true, true>(tid, N, drow, a.same_phase, f.Rp, ct, As, f.A1p);
            else if (f.soft || !hard) view.template gradient<true, false>(tid, N, drow, a.same_phase, f.Rp, ct, As + f.A1p, 0.0f);
            else view.template gradient<false, true>(tid, N, drow, a.same_phase, f.Rp, ct, 0.0f, f.A1p);
            for (long long p = V + tid; p < a.ld; p += N) drow[p] = Elem<T>::put(0.0f);
        }
        if (warp < nlw && f.soft) {
            const float part = warp_sum(f.kl(t, zc, R, it));
            if (lane == 0) s_ll[warp] = part;
        }
        __syncthreads();  // the second pass's stores come before those of the list
        if (tid == 0) a.row_loss[row] = f.loss(a, s_ll, nlw, hard, R, s1, zy);
        if (c >= 0) {
            s_bits[at >> 5] = 0;
            if (dz) drow[c] = Elem<T>::put(f.listed(t, zc, R, ct, hard, c == y));
        }
        if (tid == 0) {
            if (dz && hard && !s_flag) drow[y] = Elem<T>::put(f.target(zy, R, ct));
            s_flag = 0;
        }
    }
}

}  // namespace

namespace head {
template <typename T, bool REST>
static bool stream(const Launch& L, const void* z, void* dz, const DistillArgs& a, const Plan& p) {
    static PerDevice attr;
    if (!allow_smem(attr, k_distill_stream<T, REST>)) return false;
    launch_rows(L, k_distill_stream<T, REST>, p, (const T*)z, (T*)dz, a);
    return true;
}
template <typename T> bool distill_stream(const Launch& L, const void* z, void* dz, DistillArgs a, int G, int N) {
    a.Gs = G;
    Plan p;
    p.threads = N;
    p.smem = align16((a.Gs * Elem<T>::EPG + 31) / 32 * 4);
    p.ctas = (int)std::min<long long>(a.M, L.num_sms * (2 * DL_THREADS / N));
    return a.t_lse ? stream<T, true>(L, z, dz, a, p) : stream<T, false>(L, z, dz, a, p);
}
template bool distill_stream<float>(const Launch&, const void*, void*, DistillArgs, int, int);
template bool distill_stream<__nv_bfloat16>(const Launch&, const void*, void*, DistillArgs, int, int);
template bool distill_stream<__half>(const Launch&, const void*, void*, DistillArgs, int, int);
}  // namespace head

}  // namespace tt
