// head_row.cuh -- what the list kernels (head.cu, distill.cu, beam.cu) share: a row of
// logits in granules, its sums of exponentials, and lists of its columns.
//
// A row is cut into granules of 16 bytes on 16-byte boundaries of memory.
// Rows may start anywhere (odd ld, offset pointers): granules wholly inside
// the row are copied and read as 16 bytes; the first and the last, where they
// are not, are fetched element by element and filled up with -inf, which no
// result depends on.  Nothing outside the row is read.
//
// In distillation a granule of the row (or, in a cluster, of the CTA's slice
// of it) is in slot i of a shared-memory buffer and belongs to thread i mod NT,
// which copies it in (cp.async), reads it in every pass, and refills it with
// the next row's as soon as it has read it for the last time: the passes need
// no barrier for the row's data, and a row is read from memory once.
#pragma once

#include "tt_internal.h"

#include <algorithm>

namespace tt {
namespace head {

constexpr int LIST_MAX = TT_TOP_MAX;
__host__ __device__ constexpr int align16(int n) { return (n + 15) & ~15; }
constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// pairs of floats in one 64-bit register: one instruction for two lanes
using f2 = unsigned long long;
__device__ __forceinline__ f2 pk(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpk(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// x^N for N = 2, 3, 4 (other N: x)
template <int N> __device__ __forceinline__ f2 powi(f2 x) {
    const f2 q = mul2(x, x);
    return N == 2 ? q : N == 3 ? mul2(q, x) : N == 4 ? mul2(q, q) : x;
}
template <int N> __device__ __forceinline__ float powi(float x) {
    const float q = x * x;
    return N == 2 ? q : N == 3 ? q * x : N == 4 ? q * q : x;
}

// ------------------------------------------------------------ storage types
// A granule of EPG elements as EPG / 2 pairs of floats, and back.  Max is what
// maxima are kept in (a pair for the 16-bit types): exact, and a NaN is passed
// over.
template <typename T> struct Elem;
template <> struct Elem<float> {
    static constexpr int EPG = 4;
    using Max = float;
    static constexpr uint32_t NINF = 0xFF800000u;
    static __device__ __forceinline__ float get(const float* p) { return *p; }
    static __device__ __forceinline__ float put(float v) { return v; }
    static __device__ __forceinline__ void unpack(const uint4& u, f2* f) {
        f[0] = pk(__uint_as_float(u.x), __uint_as_float(u.y));
        f[1] = pk(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ uint4 pack(const f2* f) {
        float a, b, c, d;
        unpk(f[0], a, b);
        unpk(f[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
    static __device__ __forceinline__ Max gmax(const uint4& u) {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)),
                     fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
    static __device__ __forceinline__ Max max2(Max a, Max b) { return fmaxf(a, b); }
    static __device__ __forceinline__ Max to_max(float v) { return v; }
    static __device__ __forceinline__ Max min2(Max a, Max b) { return fminf(a, b); }
    static __device__ __forceinline__ float top(Max m) { return m; }
    static __device__ __forceinline__ float bottom(Max m) { return m; }
    static __device__ __forceinline__ float value(Max m) { return fmaxf(m, -INFINITY); }
};
template <typename T, typename P, typename Cvt> struct Elem16 {
    static constexpr int EPG = 8;
    using Max = P;
    static __device__ __forceinline__ P pair(uint32_t w) { return *reinterpret_cast<const P*>(&w); }
    static __device__ __forceinline__ uint4 pack(const f2* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float a, b;
            unpk(f[i], a, b);
            const P h = Cvt::pair(a, b);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ Max gmax(const uint4& u) {
        return __hmax2(__hmax2(pair(u.x), pair(u.y)), __hmax2(pair(u.z), pair(u.w)));
    }
    static __device__ __forceinline__ Max max2(Max a, Max b) { return __hmax2(a, b); }
    static __device__ __forceinline__ Max to_max(float v) { return Cvt::pair(v, v); }
    static __device__ __forceinline__ Max min2(Max a, Max b) { return __hmin2(a, b); }
    static __device__ __forceinline__ T top(Max m) { return __hmax(m.x, m.y); }
    static __device__ __forceinline__ T bottom(Max m) { return __hmin(m.x, m.y); }
    // (top(a), top(b))
    static __device__ __forceinline__ P fold(P a, P b) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(&a), y = *reinterpret_cast<const uint32_t*>(&b);
        return __hmax2(pair(__byte_perm(x, y, 0x5410)), pair(__byte_perm(x, y, 0x7632)));
    }
    static __device__ __forceinline__ float value(Max m) {
        return fmaxf(fmaxf(__low2float(m), __high2float(m)), -INFINITY);
    }
};
struct CvtBf {
    static __device__ __forceinline__ __nv_bfloat162 pair(float a, float b) { return __floats2bfloat162_rn(a, b); }
};
struct CvtHalf {
    static __device__ __forceinline__ __half2 pair(float a, float b) { return __floats2half2_rn(a, b); }
};
template <> struct Elem<__nv_bfloat16> : Elem16<__nv_bfloat16, __nv_bfloat162, CvtBf> {
    static constexpr uint32_t NINF = 0xFF80FF80u;
    static __device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
    static __device__ __forceinline__ void unpack(const uint4& u, f2* f) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; i++) f[i] = pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
};
template <> struct Elem<__half> : Elem16<__half, __half2, CvtHalf> {
    static constexpr uint32_t NINF = 0xFC00FC00u;
    static __device__ __forceinline__ float get(const __half* p) { return __half2float(*p); }
    static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
    static __device__ __forceinline__ void unpack(const uint4& u, f2* f) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[i] = pk(v.x, v.y);
        }
    }
};

// ------------------------------------------------------------ copies
template <int AT> __device__ __forceinline__ void cp16(uint32_t s, const void* g) {
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;" ::"r"(s), "l"(g), "n"(AT) : "memory");
}
__device__ __forceinline__ void cp4(void* s, const void* g) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(s)), "l"(g)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest (nbuf - 1) groups have arrived
__device__ __forceinline__ void cp_wait(int nbuf) {
    if (nbuf == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------ clusters
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// every CTA's writes to the others' shared memory before it are seen after it
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* s, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(s)), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_remote(uint32_t at, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t at, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

// ------------------------------------------------------------ warps
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// ------------------------------------------------------------ a row's slice
template <typename T> struct Slice {
    const char* base;  // the slice's first granule in memory
    int ph;            // byte offset of column 0 from the row's first granule
    int g0, n;         // first granule of this CTA, and how many
    int i0, i1;        // slots whose granules are wholly inside the row
    bool head, tail;   // this slice has a granule that column 0 (the last column) is inside of

    __device__ __forceinline__ Slice(const T* z, long long row, long long ld, int V, int rank, int Gs) {
        const char* p = reinterpret_cast<const char*>(z + row * ld);
        ph = (int)((uintptr_t)p & 15);
        const int end = ph + V * (int)sizeof(T), G = (end + 15) >> 4, full = end >> 4;
        g0 = min(rank * Gs, G);
        n = min(Gs, G - g0);
        base = p - ph + (long long)g0 * 16;
        i0 = ph && g0 == 0 ? 1 : 0;
        i1 = min(n, max(0, full - g0));
        head = ph && g0 == 0 && n > 0;
        tail = i1 < n && !(head && n == 1);
    }
    // column of the first element of slot i (may be negative at the head)
    __device__ __forceinline__ int col(int i) const { return ((g0 + i) * 16 - ph) / (int)sizeof(T); }
    __device__ __forceinline__ bool inner(int i) const { return i >= i0 && i < i1; }
    // byte offset in the buffer of column c, or -1 if another CTA has it
    __device__ __forceinline__ int at(int c) const {
        const int b = ph + c * (int)sizeof(T) - g0 * 16;
        return b >= 0 && b < n * 16 ? b : -1;
    }
};

// Copies worker tid's granules (of NT workers) of the slice into buf.
template <typename T, int NT>
__device__ __forceinline__ void fill(const Slice<T>& s, char* buf, int tid) {
    int i = tid < s.i0 ? tid + NT : tid;  // the head's granule comes element by element
    const char* g = s.base + (long long)i * 16;
    uint32_t b = (uint32_t)__cvta_generic_to_shared(buf) + i * 16;
    for (; i + 3 * NT < s.i1; i += 4 * NT, g += 64 * NT, b += 64 * NT) {
        cp16<0>(b, g);
        cp16<16 * NT>(b, g);
        cp16<32 * NT>(b, g);
        cp16<48 * NT>(b, g);
    }
    for (; i < s.i1; i += NT, g += 16 * NT, b += 16 * NT) cp16<0>(b, g);
}

// The slot of the edge granule that thread tid < 16 of the group looks after
// one element of: threads 0..7 the head's, 8..15 the tail's; -1: none.
template <typename T>
__device__ __forceinline__ int edge_slot(const Slice<T>& s, int tid) {
    if (tid < 0 || tid >= 16 || (tid & 7) >= Elem<T>::EPG) return -1;
    if (tid < 8) return s.head ? 0 : -1;
    return s.tail ? s.n - 1 : -1;
}
template <typename T>
__device__ __forceinline__ T edge_load(const Slice<T>& s, int V, int tid) {
    const int i = edge_slot(s, tid);
    const int c = i < 0 ? -1 : s.col(i) + (tid & 7);
    return c >= 0 && c < V ? reinterpret_cast<const T*>(s.base)[i * Elem<T>::EPG + (tid & 7)]
                           : Elem<T>::put(-INFINITY);
}
// Slot i of the slice, read from memory; what lies outside the row is -inf.
template <typename T> __device__ __noinline__ uint4 edge_granule(const T* row, int c0, int V) {
    union {
        T e[Elem<T>::EPG];
        uint4 u;
    } x;
#pragma unroll
    for (int j = 0; j < Elem<T>::EPG; j++) x.e[j] = c0 + j >= 0 && c0 + j < V ? row[c0 + j] : Elem<T>::put(-INFINITY);
    return x.u;
}

// Slot i of the slice, read from memory.
template <typename T> __device__ __forceinline__ uint4 granule(const Slice<T>& s, int i, int V) {
    return s.inner(i) ? reinterpret_cast<const uint4*>(s.base)[i]
                      : edge_granule(reinterpret_cast<const T*>(s.base) - s.col(0), s.col(i), V);
}

// ------------------------------------------------------------ sums of exponentials
// Sums of 2^((z - R) c) over a thread's granules in one pass, at one
// exponential an element, without knowing the maximum: R starts at the largest
// of the warp's first granules and moves up only when a value is more than
// `lift` above it (the sums are then scaled), which keeps every term below
// e^20.  The argument is one fused multiply-add, z c + nb with nb = -(R c)
// rounded; the rounding of nb is common to all terms and is taken out at the
// end as the factor 2^-(R c + nb), which a fused multiply-add gives exactly.
// Logits beyond 1e30 (the type's lowest value, +inf) would overflow z c: threads
// that start from one, meet a positive one or nothing else form (z - R) first.
constexpr float FAR = 1e30f;

__device__ __forceinline__ bool is_far(float v) { return !(fabsf(v) < FAR); }
__device__ __forceinline__ float exp_of(float z, float r, float c) { return ex2f((z - r) * c); }
// 2^-(R c + nb): what sums of 2^(z c + nb) are multiplied by
__device__ __forceinline__ float unbias(float R, float c, float nb) { return ex2f(-fmaf(R, c, nb)); }

// SA, SB: whether the sum with coefficient ca, cb is wanted.  PW = n (2, 3 or
// 4): ca is n cb, and the first sum's terms are the n-th powers of the second's:
// two softmaxes at one exponential an element (with two, the special-function
// unit, 32 a cycle and SM, is what a pass waits for).
// FOLD: the first sum may be put aside (fold).
template <typename T, bool SA, bool SB, int PW = 0, bool FOLD = false> struct Sums {
    using E = Elem<T>;
    static constexpr int H = E::EPG / 2;
    typename E::Max m;  // the thread's largest values
    f2 xa, xb, na2, nb2;
    float ya = 0.0f;  // what was put aside
    float la, lb;
    float R, lim, na, nb;  // a value above lim moves the reference; -inf: there is none yet
    const float ca, cb, lift;
    bool far;

    // w: a value to start the reference from (the same in all lanes), -inf for none
    __device__ __forceinline__ Sums(float ca_, float cb_, float lift_) : ca(ca_), cb(cb_), lift(lift_) {}
    __device__ __forceinline__ void start(float w) {
        m = E::to_max(-INFINITY);
        xa = xb = pk(0.0f, 0.0f);
        ya = 0.0f;
        R = na = nb = 0.0f;
        lim = -INFINITY;
        far = is_far(w) && w != -INFINITY;
        if (!is_far(w)) {
            R = w;
            lim = R + lift;
            na = -(R * ca);
            nb = -(R * cb);
        }
        na2 = pk(na, na);
        nb2 = pk(nb, nb);
    }
    // the largest values of the granules that take() will be given next
    __device__ __forceinline__ void look(typename E::Max gm) {
        m = E::max2(m, gm);
        if (!(SA || SB)) return;
        const float vm = E::value(gm);
        if (vm > lim) {
            if (is_far(vm)) {
                far |= vm > 0.0f;
                return;
            }
            R = vm;
            const float ma = -(R * ca), mb = -(R * cb);
            const float fb = lim == -INFINITY ? 0.0f : ex2f(mb - nb);
            const float fa = PW ? powi<PW>(fb) : lim == -INFINITY ? 0.0f : ex2f(ma - na);
            if (SA) xa = mul2(xa, pk(fa, fa));
            if (FOLD) ya *= fa;
            if (SB) xb = mul2(xb, pk(fb, fb));
            na = ma;
            nb = mb;
            na2 = pk(na, na);
            nb2 = pk(nb, nb);
            lim = R + lift;
        }
    }
    __device__ __forceinline__ void take(const uint4& u) {
        if (!(SA || SB)) return;
        const f2 ca2 = pk(ca, ca), cb2 = pk(cb, cb);
        f2 e[H];
        E::unpack(u, e);
        float x, y;
        if (PW) {
#pragma unroll
            for (int i = 0; i < H; i++) {
                unpk(fma2(e[i], cb2, nb2), x, y);
                const f2 q = pk(ex2f(x), ex2f(y));
                xb = add2(xb, q);
                xa = add2(xa, powi<PW>(q));
            }
            return;
        }
        if (SA) {
#pragma unroll
            for (int i = 0; i < H; i++) {
                unpk(fma2(e[i], ca2, na2), x, y);
                xa = add2(xa, pk(ex2f(x), ex2f(y)));
            }
        }
        if (SB) {
#pragma unroll
            for (int i = 0; i < H; i++) {
                unpk(fma2(e[i], cb2, nb2), x, y);
                xb = add2(xb, pk(ex2f(x), ex2f(y)));
            }
        }
    }
    // The same number of additions for N granules in a shorter chain: a granule's
    // terms meet in a tree, the granules' sums in a row, and one addition adds them
    // to the sums.  (Rows that one CTA holds are at most 28 granules a thread and
    // keep to the other form: 32768 of 50257 16-bit logits 1059 us, 1078 us by this
    // one.)  The longest chain of additions on the way of a term into a row's sum,
    // threads' and warps' sums included: 100 in k_top_stream (whose chains start
    // anew after 64 stages), 125 in k_distill, 75 in k_distill_stream.
    template <int N> __device__ __forceinline__ void take(const uint4 (&u)[N]) {
        if (!(SA || SB)) return;
        const f2 ca2 = pk(ca, ca), cb2 = pk(cb, cb);
        f2 ta = 0, tb = 0;
#pragma unroll
        for (int g = 0; g < N; g++) {
            f2 e[H], p[H];
            E::unpack(u[g], e);
            auto terms = [&](f2 c2, f2 n2) {
#pragma unroll
                for (int i = 0; i < H; i++) {
                    float x, y;
                    unpk(fma2(e[i], c2, n2), x, y);
                    p[i] = pk(ex2f(x), ex2f(y));
                }
            };
            auto tree = [&](f2& t) {
#pragma unroll
                for (int d = 1; d < H; d *= 2)
#pragma unroll
                    for (int i = 0; i < H; i += 2 * d) p[i] = add2(p[i], p[i + d]);
                t = g ? add2(t, p[0]) : p[0];
            };
            if (PW) {
                f2 q[H];
                terms(cb2, nb2);
#pragma unroll
                for (int i = 0; i < H; i++) q[i] = powi<PW>(p[i]);
                tree(tb);
#pragma unroll
                for (int i = 0; i < H; i++) p[i] = q[i];
                tree(ta);
                continue;
            }
            if (SA) {
                terms(ca2, na2);
                tree(ta);
            }
            if (SB) {
                terms(cb2, nb2);
                tree(tb);
            }
        }
        if (SA) xa = add2(xa, ta);
        if (SB) xb = add2(xb, tb);
    }
    // what has gathered so far is put aside: a chain starts anew
    __device__ __forceinline__ void fold() {
        float x, y;
        unpk(xa, x, y);
        ya += x + y;
        xa = pk(0.0f, 0.0f);
    }
    // one value of a far row, formed without overflow; R is its largest.  A
    // thread's chain is its whole share of the row, so the sums are compensated
    // (Kahan 1965: l is what the last addition lost).
    __device__ __forceinline__ void take_far(float z, float& sa, float& sb) {
        const float d = z == R ? 0.0f : z - R;  // inf - inf is a term of 1
        auto add = [&](float c, float& s, float& l) {
            const float y = (R == -INFINITY && d == 0.0f ? 0.0f : ex2f(d * c)) - l, t = s + y;
            l = (t - s) - y;
            s = t;
        };
        if (SA) add(ca, sa, la);
        if (SB) add(cb, sb, lb);
    }
    // tm: the largest value; R = -inf where there is none above -inf.  True
    // where the row has to be gone through again with take_far (R = tm then).
    __device__ __forceinline__ bool finish(float& tm, float& sa, float& sb) {
        tm = E::value(m);
        sa = sb = la = lb = 0.0f;
        if (!(SA || SB)) return false;
        // a thread that has met nothing but -inf and values below -FAR has no reference
        if (far || (lim == -INFINITY && tm > -INFINITY)) {
            R = tm;
            return true;
        }
        float x, y;
        const float ub = unbias(R, cb, nb);
        unpk(xa, x, y);
        if (SA) sa = (FOLD ? x + y + ya : x + y) * (PW ? powi<PW>(ub) : unbias(R, ca, na));
        unpk(xb, x, y);
        if (SB) sb = (x + y) * ub;
        if (tm == -INFINITY) R = -INFINITY;  // no terms, unless they are NaN
        return false;
    }
};

// Granules are taken four at a time, so that the reference is looked at once for four.
// TREE: in the form with the shorter chain.
template <typename T, int NT, bool TREE, bool SA, bool SB, int PW = 0>
__device__ __forceinline__ void sum_pass(const Slice<T>& s, const char* buf, int tid, float ca, float cb, float lift,
                                         float& tm, float& R, float& sa, float& sb) {
    using E = Elem<T>;
    constexpr int U = 4;
    const uint4* v = reinterpret_cast<const uint4*>(buf);
    Sums<T, SA, SB, PW> q(ca, cb, lift);
    q.start(SA || SB ? warp_max(tid < s.n ? E::value(E::gmax(v[tid])) : -INFINITY) : -INFINITY);
    int i = tid;
    for (; i + (U - 1) * NT < s.n; i += U * NT) {
        uint4 u[U];
#pragma unroll
        for (int j = 0; j < U; j++) u[j] = v[i + j * NT];
        q.look(E::max2(E::max2(E::gmax(u[0]), E::gmax(u[1])), E::max2(E::gmax(u[2]), E::gmax(u[3]))));
        if (TREE) {
            q.take(u);
        } else {
#pragma unroll
            for (int j = 0; j < U; j++) q.take(u[j]);
        }
    }
#pragma unroll 1
    for (; i < s.n; i += NT) {
        const uint4 u = v[i];
        q.look(E::gmax(u));
        q.take(u);
    }
    if (q.finish(tm, sa, sb)) {
#pragma unroll 1
        for (int g = tid; g < s.n; g += NT)
#pragma unroll 1
            for (int j = 0; j < E::EPG; j++) q.take_far(E::get(reinterpret_cast<const T*>(v + g) + j), sa, sb);
    }
    R = q.R;
}

// what a sum with reference `from` is multiplied by to have the larger reference `to`
__device__ __forceinline__ float rescale(float from, float to, float c) {
    if (from == to) return 1.0f;
    return from == -INFINITY ? 0.0f : ex2f((from - to) * c);
}

// Merges the sums of lanes that differ in their lowest bits (all below N); a
// lane without terms has R = -inf and 0.  The three have coefficients LOG2E, ct
// and ct.
template <int N = 32> __device__ __forceinline__ void merge(float& R, float& s, float c) {
    float m = R;
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    s *= rescale(R, m, c);
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    R = m;
}
template <int N = 32>
__device__ __forceinline__ void merge(float& R, float& s1, float& st, float& sl, float ct, bool one, bool list) {
    float m = R;
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float f = rescale(R, m, ct);
    st *= f;
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) st += __shfl_xor_sync(0xffffffffu, st, o);
    if (one) {
        s1 *= rescale(R, m, LOG2E);
#pragma unroll
        for (int o = N / 2; o > 0; o >>= 1) s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    }
    if (list) {
        sl *= f;
#pragma unroll
        for (int o = N / 2; o > 0; o >>= 1) sl += __shfl_xor_sync(0xffffffffu, sl, o);
    }
    R = m;
}

// log sum exp(z / tau) of merged sums: a row of -inf and a row with +inf have
// that as their value, unless a NaN is there too.  The logarithm is taken of
// the mantissa, so that it adds no error to speak of to the sum's.
__device__ __forceinline__ double lse_of(float R, float s, float inv_tau) {
    if (s == s && (R == -INFINITY || R == INFINITY)) return (double)R;
    int e = 0;
    const float m = frexpf(s, &e);
    return (double)R * (double)inv_tau + ((double)e * 0.6931471805599453 + (double)logf(m));
}

// ------------------------------------------------------------ lists
// Order-preserving whole number of a value: -0 counts as +0 and a NaN as -inf.
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t u = __float_as_uint(fmaxf(v, -INFINITY) + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}
// (value, column): larger values first, then lower columns.  Never 0.
__device__ __forceinline__ unsigned long long top_key(float v, int col) {
    return ((unsigned long long)order_of(v) << 32) | (unsigned long long)(0xFFFFFFFFu - (uint32_t)col);
}
__device__ __forceinline__ int key_col(unsigned long long key) {
    return (int)(0xFFFFFFFFu - (uint32_t)(key & 0xFFFFFFFFull));
}
// out(rank, key) for the kk first of cnt keys in list order, by a warp: a lane
// counts the keys above its own, two a load.  s_key is 16-byte aligned and has
// room for an even number.
template <typename F>
__device__ __forceinline__ void ranks(unsigned long long* s_key, int cnt, int kk, F&& out) {
    const int lane = threadIdx.x & 31;
    if (lane == 0 && cnt % 2) s_key[cnt] = 0;  // counts for nothing
    __syncwarp();
    for (int i0 = 0; i0 < cnt; i0 += 32) {
        const unsigned long long key = i0 + lane < cnt ? s_key[i0 + lane] : ~0ull;
        int r = 0;
#pragma unroll 4
        for (int j = 0; j < cnt; j += 2) {
            const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(s_key + j);
            r += o.x > key;
            r += o.y > key;
        }
        if (i0 + lane < cnt && r < kk) out(r, key);
    }
}

// Sorts keys over a warp, the largest first: key 32 e + lane of the list is
// x[e].  A bitonic sort, for a warp that has little beside it: 28 steps for 128
// keys.  The many warps of k_top_stream fare better with ranks(), which asks
// less of the pipe that shuffles share with shared memory (32768 rows of 50257
// 16-bit logits, k = 64: 628 us, sorted 663).
template <int E> __device__ __forceinline__ void sort_keys(unsigned long long (&x)[E]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32 * E; size *= 2) {
#pragma unroll
        for (int d = size / 2; d > 0; d /= 2) {
            if (d >= 32) {
#pragma unroll
                for (int e = 0; e < E; e++) {
                    if (e & (d / 32)) continue;
                    const int o = e | (d / 32);
                    const unsigned long long a = x[e], b = x[o];
                    const bool swap = (a < b) == ((32 * e & size) == 0);
                    x[e] = swap ? b : a;
                    x[o] = swap ? a : b;
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; e++) {
                    const unsigned long long y = __shfl_xor_sync(0xffffffffu, x[e], d);
                    const bool larger = ((lane & d) == 0) == (((32 * e + lane) & size) == 0);
                    x[e] = (x[e] > y) == larger ? x[e] : y;
                }
            }
        }
    }
}
// ranks() by sorting
template <int E, typename F>
__device__ __forceinline__ void sorted(const unsigned long long* s_key, int cnt, int kk, F&& out) {
    const int lane = threadIdx.x & 31;
    unsigned long long x[E];
#pragma unroll
    for (int e = 0; e < E; e++) x[e] = 32 * e + lane < cnt ? s_key[32 * e + lane] : 0ull;
    sort_keys(x);
#pragma unroll
    for (int e = 0; e < E; e++)
        if (32 * e + lane < min(cnt, kk)) out(32 * e + lane, x[e]);
}

// The kk first of n keys (0: no entry; at least kk are entries) by a warp: a
// bound that kk to JOIN_ROOM keys reach is found bit by bit by counting (keys
// are all different, so there is one), and those are ranked.  s_key holds
// JOIN_ROOM keys.
constexpr int JOIN_ROOM = 160;

template <typename F>
__device__ __forceinline__ void join_lists(const unsigned long long* l, int n, int kk, unsigned long long* s_key,
                                           F&& out) {
    const int lane = threadIdx.x & 31;
    unsigned long long t = 0;
    if (n > min(kk + 32, JOIN_ROOM)) {  // few enough are ranked as they are
        uint32_t hi = 0, lo = ~0u;
        for (int i = lane; i < n; i += 32) {
            const uint32_t w = (uint32_t)(l[i] >> 32);
            hi = max(hi, w);
            lo = min(lo, w);
        }
        hi = __reduce_max_sync(0xffffffffu, hi);
        lo = __reduce_min_sync(0xffffffffu, lo);
        int bit = hi == lo ? 31 : 63 - __clz(hi ^ lo);
        t = (unsigned long long)hi << 32;
        t &= ~((2ull << bit) - 1ull);
        for (; bit >= 0; bit--) {
            const unsigned long long cand = t | (1ull << bit);
            int c = 0;
#pragma unroll 4
            for (int i = lane; i < n; i += 32) c += l[i] >= cand;
            c = __reduce_add_sync(0xffffffffu, c);
            if (c >= kk) t = cand;
            if (c >= kk && c <= min(kk + 16, JOIN_ROOM)) break;
        }
    }
    int cnt = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const unsigned long long key = i0 + lane < n ? l[i0 + lane] : 0ull;
        const bool on = key != 0 && key >= t;
        const uint32_t m = __ballot_sync(0xffffffffu, on);
        if (on) s_key[cnt + __popc(m & ((1u << lane) - 1u))] = key;
        cnt += __popc(m);
    }
    __syncwarp();
    if (cnt <= 32) sorted<1>(s_key, cnt, kk, out);
    else if (cnt <= 128) sorted<4>(s_key, cnt, kk, out);
    else ranks(s_key, cnt, kk, out);
}

// A warp merges P parts' references and sums.
__device__ __forceinline__ void join_parts(const float2* parts, int P, float c, float& R, float& s) {
    const int lane = threadIdx.x & 31;
    R = -INFINITY;
    s = 0.0f;
    for (int p = lane; p < P; p += 32) {
        const float2 x = parts[p];
        const float m = fmaxf(R, x.x);
        s = s * rescale(R, m, c) + x.y * rescale(x.x, m, c);
        R = m;
    }
    merge(R, s, c);
}

// ------------------------------------------------------------ launch
// How a kernel's CTAs are laid out; for distillation also the CTAs that share
// a row, their slices, and whether two rows of a CTA are on chip at once.
struct Plan {
    int cs = 1, nbuf = 1, Gs = 0, ctas = 0, threads = 0;
    size_t smem = 0;
};

constexpr size_t SMEM_CTA = 231424;  // 226 KB, and 1 KB for what is not dynamic
constexpr size_t SMEM_SM = 233472;   // 228 KB, of which each CTA takes 1 KB more than its own
constexpr size_t SMEM_HALF = SMEM_SM / 2 - 1024;

template <typename K> bool allow_smem(PerDevice& attr, K kern) {
    return attr.once([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_CTA) == cudaSuccess;
    });
}

template <typename... KA, typename... A>
void launch_rows(const Launch& L, void (*kern)(KA...), const Plan& p, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.ctas);
    cfg.blockDim = dim3((unsigned)p.threads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = L.stream;
    cudaLaunchAttribute at[2];
    unsigned n = 0;
    if (L.pdl) {
        at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (p.cs > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim.x = (unsigned)p.cs;
        at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
        n++;
    }
    cfg.attrs = at;
    cfg.numAttrs = n;
    L.count();
    cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...);
}

// granules of a row, for the worst place of its start
template <typename T> int row_granules(const void* z, long long ld, int V) {
    const bool aligned = ((uintptr_t)z & 15) == 0 && ld * (long long)sizeof(T) % 16 == 0;
    return (int)(((aligned ? 0 : 16 - (int)sizeof(T)) + (long long)V * (int)sizeof(T) + 15) / 16);
}

}  // namespace head
}  // namespace tt
