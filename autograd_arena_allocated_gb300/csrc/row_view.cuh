// row_view.cuh -- a row of logits gone over in memory by the threads of a CTA or
// a warp: sums of exponentials, then the gradient (distill_stream.cu, answer.cu).
#pragma once

#include "distill.cuh"

namespace tt {
namespace head {

// u with the elements of the given bits replaced by -inf
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
    int tail_tid = 32;    // the thread that looks after the last granule (the first has thread 0)

    __device__ __forceinline__ uint4 masked(int i, uint4 u) const {
        if (bits) {
            const uint32_t b = E::EPG == 8 ? bits[i] : bits[i >> 1] >> ((i & 1) * 4) & 15u;
            if (b) u = drop<T>(u, b);
        }
        return u;
    }
    // f(slot) for the thread's share of the slots that are not wholly inside the row
    template <typename F> __device__ __forceinline__ void edges(int tid, F&& f) const {
        const int i = tid == 0 && s.head ? 0 : tid == tail_tid && s.tail ? s.n - 1 : -1;
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

}  // namespace head
}  // namespace tt
