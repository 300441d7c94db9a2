// attn_group_mma.cu -- attention over groups of answers that share a prompt
// (group.cuh) for 16-bit heads of 16 and 32.
//
// Heads this narrow fill neither a tensor-memory tile (128 rows of 64-byte or
// 32-byte operands, products of K = 16 or 32) nor the work of one: a warp's
// mma.sync m16n8k16 takes them as they are.  64 queries (keys) a CTA, 16 a warp,
// past blocks of 64 keys (queries); tiles come by cp.async into two buffers, 16-byte
// chunks XOR-swizzled by row so that ldmatrix meets no bank twice.  Rows of
// padding are zeros in shared memory.  All sums fp32; P and dS are rounded to the
// storage type for the second products.  4 groups of 1400 positions, 16 heads of 32,
// half: 46 us forward and 141 backward (143 and 118 TFLOP/s; by fp32 FMAs 298 and
// 885), where exponentials and packing, not products, are most of the work.
//
//   k_fwd    S = Q K^T, running maximum and sum, O += P V
//   k_dq     D = rowsum(dO o O), dS = P o (dO V^T - D), dQ += dS K
//   k_dkdv   dV += P^T dO, dK += dS^T Q, over a key's queries in order
#include "tt_internal.h"
#include "group.cuh"

namespace tt {
namespace {

using group::BLK;
using group::Group;

constexpr int THREADS = 128;  // 4 warps x 16 rows
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// byte offset of (row, 8-element chunk) in a 64 x D tile
template <int D> __device__ __forceinline__ uint32_t tile_off(int row, int chunk) {
    constexpr int N = D / 8;
    return (uint32_t)(row * D * 2 + ((chunk ^ (row * N / 8 & (N - 1))) << 4));
}

// 64 rows of D elements, ld apart; rows from `valid` on are zeros
template <int D>
__device__ __forceinline__ void load_tile(uint32_t s, const void* g, long long ld, int valid) {
    for (int i = threadIdx.x; i < BLK * (D / 8); i += THREADS) {
        const int r = i / (D / 8), c = i % (D / 8);
        const bool ok = r < valid;
        const char* src = (const char*)g + (ok ? (r * ld + c * 8) * 2 : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s + tile_off<D>(r, c)), "l"(src), "r"(ok ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait1() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

__device__ __forceinline__ void ldsm(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}
__device__ __forceinline__ void ldsm_t(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}

template <typename T> struct Mma;
template <> struct Mma<__nv_bfloat16> {
    static __device__ __forceinline__ void run(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    }
};
template <> struct Mma<__half> {
    static __device__ __forceinline__ void run(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
};

// A fragments (16 rows from row0, D columns) of a tile
template <int D> __device__ __forceinline__ void a_frags(uint32_t s, int row0, uint32_t (&f)[D / 16][4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < D / 16; k++)
        ldsm(s + tile_off<D>(row0 + (lane & 7) + 8 * ((lane >> 3) & 1), 2 * k + (lane >> 4)), f[k]);
}

// acc [16 x 64] = A [16 x D] B^T, B a tile
template <typename T, int D>
__device__ __forceinline__ void product(float (&acc)[8][4], const uint32_t (&a)[D / 16][4], uint32_t s) {
    const int lane = threadIdx.x & 31, i = lane >> 3, j = lane & 7;
#pragma unroll
    for (int n = 0; n < 8; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[n][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < D / 16; k++)
#pragma unroll
        for (int n = 0; n < 4; n++) {
            uint32_t b[4];
            ldsm(s + tile_off<D>(n * 16 + j + 8 * (i >> 1), 2 * k + (i & 1)), b);
            Mma<T>::run(acc[2 * n], a[k], b[0], b[1]);
            Mma<T>::run(acc[2 * n + 1], a[k], b[2], b[3]);
        }
}

// acc [16 x D] += P [16 x 64] B, P an accumulator rounded to the storage type, B a tile
template <typename T, int D>
__device__ __forceinline__ void accumulate(float (&acc)[D / 8][4], const float (&p)[8][4], uint32_t s) {
    const int lane = threadIdx.x & 31, i = lane >> 3, j = lane & 7;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const uint32_t a[4] = {Mma<T>::pack(p[2 * k][0], p[2 * k][1]), Mma<T>::pack(p[2 * k][2], p[2 * k][3]),
                               Mma<T>::pack(p[2 * k + 1][0], p[2 * k + 1][1]), Mma<T>::pack(p[2 * k + 1][2], p[2 * k + 1][3])};
#pragma unroll
        for (int d = 0; d < D / 16; d++) {
            uint32_t b[4];
            ldsm_t(s + tile_off<D>(k * 16 + j + 8 * (i & 1), 2 * d + (i >> 1)), b);
            Mma<T>::run(acc[2 * d], a, b[0], b[1]);
            Mma<T>::run(acc[2 * d + 1], a, b[2], b[3]);
        }
    }
}

struct GroupArgs {
    const int32_t* starts;
    int T, C, H, K, tiles, pairs;
    int* flags;
};

// a CTA's place, and what a thread has of a 16-row tile: rows row, row + 8, columns
// 8 n + 2 t4, + 1
struct Place : group::Place {
    int first, row, t4;
    __device__ __forceinline__ Place(const GroupArgs& a, bool last_first) : group::Place(a.tiles, a.pairs, a.H, last_first) {
        first = tile * BLK;
        const int lane = threadIdx.x & 31;
        row = first + (threadIdx.x >> 5) * 16 + (lane >> 2);
        t4 = lane & 3;
    }
};

__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// a thread's part of one row (half 0: row, 1: row + 8) of a 16 x D result
template <typename T, int D>
__device__ __forceinline__ void store_row(T* d, const float (&acc)[D / 8][4], int half, int t4, float scale, bool real) {
    uint32_t* w = reinterpret_cast<uint32_t*>(d);
#pragma unroll
    for (int n = 0; n < D / 8; n++)
        w[4 * n + t4] = real ? Mma<T>::pack(acc[n][2 * half] * scale, acc[n][2 * half + 1] * scale) : 0u;
}

template <typename T, int D> __global__ void __launch_bounds__(THREADS) k_fwd(const T* qkv, T* y, float* lse, const GroupArgs a) {
    pdl_enter();
    __shared__ __align__(128) T sQ[BLK * D], sK[2][BLK * D], sV[2][BLK * D];
    const Place at(a, true);
    const Group g(a.starts, at.b, a.K, a.T);
    const long long ld = 3LL * a.C, row0 = (long long)at.b * a.T;
    const T* base = qkv + row0 * ld + at.h * D;
    if (at.first == 0 && at.h == 0) g.check(threadIdx.x, THREADS, a.T, a.flags);
    float o[D / 8][4], m[2] = {-3e38f, -3e38f}, l[2] = {0.0f, 0.0f};  // finite: a row may see nothing of a block
    for (int n = 0; n < D / 8; n++)
        for (int e = 0; e < 4; e++) o[n][e] = 0.0f;
    if (at.first < g.end) {  // uniform over the CTA
        const group::QueryTile tile(g, at.first, BLK);
        const float sl2 = rsqrtf((float)D) * LOG2E;
        const int st[2] = {g.start_of(at.row), g.start_of(at.row + 8)};
        auto load = [&](int j) {
            const int k0 = tile.block(j) * BLK;
            load_tile<D>(smem_u32(sK[j & 1]), base + a.C + k0 * ld, ld, g.end - k0);
            load_tile<D>(smem_u32(sV[j & 1]), base + 2 * a.C + k0 * ld, ld, g.end - k0);
        };
        load_tile<D>(smem_u32(sQ), base + at.first * ld, ld, g.end - at.first);
        load(0);
        cp_commit();
        uint32_t q[D / 16][4];
        for (int j = 0; j < tile.n; j++) {
            if (j + 1 < tile.n) load(j + 1);
            cp_commit();
            cp_wait1();
            __syncthreads();
            if (j == 0) a_frags<D>(smem_u32(sQ), (threadIdx.x >> 5) * 16, q);
            float s[8][4];
            product<T, D>(s, q, smem_u32(sK[j & 1]));
            const int k0 = tile.block(j) * BLK;
            if (tile.masked(k0)) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const unsigned long long seen = g.keys(at.row + 8 * h, st[h], k0) >> (2 * at.t4);
#pragma unroll
                    for (int n = 0; n < 8; n++)
#pragma unroll
                        for (int e = 0; e < 2; e++)
                            if (!(seen >> (8 * n + e) & 1)) s[n][2 * h + e] = -INFINITY;
                }
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 8; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    s[n][e] *= sl2;
                    mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
                }
            float corr[2], rs[2] = {0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const float mn = fmaxf(m[h], quad_max(mx[h]));
                corr[h] = exp2f(m[h] - mn);
                m[h] = mn;
            }
#pragma unroll
            for (int n = 0; n < 8; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    s[n][e] = exp2f(s[n][e] - m[e >> 1]);  // of -inf: 0
                    rs[e >> 1] += s[n][e];
                }
            l[0] = l[0] * corr[0] + rs[0];
            l[1] = l[1] * corr[1] + rs[1];
#pragma unroll
            for (int n = 0; n < D / 8; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) o[n][e] *= corr[e >> 1];
            accumulate<T, D>(o, s, smem_u32(sV[j & 1]));
            __syncthreads();  // the buffer is refilled next
        }
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int q = at.row + 8 * h;
        const float sum = quad_sum(l[h]);
        if (q >= a.T) continue;
        const bool real = q < g.end;
        store_row<T, D>(y + (row0 + q) * a.C + at.h * D, o, h, at.t4, 1.0f / sum, real);
        if (at.t4 == 0) lse[((long long)at.b * a.H + at.h) * a.T + q] = real ? (m[h] + log2f(sum)) * LN2 : 0.0f;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(THREADS)
k_dq(const T* qkv, const T* y, const float* lse, const T* dy, T* dqkv, float* Dlt, const GroupArgs a) {
    pdl_enter();
    __shared__ __align__(128) T sQ[BLK * D], sO[BLK * D], sK[2][BLK * D], sV[2][BLK * D];
    const Place at(a, true);
    const Group g(a.starts, at.b, a.K, a.T);
    const long long ld = 3LL * a.C, row0 = (long long)at.b * a.T, bh = ((long long)at.b * a.H + at.h) * a.T;
    const T* base = qkv + row0 * ld + at.h * D;
    if (at.first == 0 && at.h == 0) g.check(threadIdx.x, THREADS, a.T, a.flags);
    float dq[D / 8][4];
    for (int n = 0; n < D / 8; n++)
        for (int e = 0; e < 4; e++) dq[n][e] = 0.0f;
    const float scale = rsqrtf((float)D), sl2 = scale * LOG2E;
    if (at.first < g.end) {
        const group::QueryTile tile(g, at.first, BLK);
        auto load = [&](int j) {
            const int k0 = tile.block(j) * BLK;
            load_tile<D>(smem_u32(sK[j & 1]), base + a.C + k0 * ld, ld, g.end - k0);
            load_tile<D>(smem_u32(sV[j & 1]), base + 2 * a.C + k0 * ld, ld, g.end - k0);
        };
        load_tile<D>(smem_u32(sQ), base + at.first * ld, ld, g.end - at.first);
        load_tile<D>(smem_u32(sO), dy + (row0 + at.first) * a.C + at.h * D, a.C, g.end - at.first);
        load(0);
        cp_commit();
        int st[2];
        float L[2], Dr[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int q = at.row + 8 * h;
            const bool real = q < g.end;
            st[h] = g.start_of(q);
            L[h] = real ? lse[bh + q] * LOG2E : 0.0f;
            float d = 0.0f;
            if (real) {
                const uint32_t* yr = reinterpret_cast<const uint32_t*>(y + (row0 + q) * a.C + at.h * D);
                const uint32_t* gr = reinterpret_cast<const uint32_t*>(dy + (row0 + q) * a.C + at.h * D);
#pragma unroll
                for (int n = 0; n < D / 8; n++) {
                    const float2 u = Mma<T>::unpack(yr[4 * n + at.t4]), v = Mma<T>::unpack(gr[4 * n + at.t4]);
                    d = fmaf(u.x, v.x, fmaf(u.y, v.y, d));
                }
            }
            Dr[h] = quad_sum(d);
            if (real && at.t4 == 0) Dlt[bh + q] = Dr[h];
        }
        uint32_t q[D / 16][4], o[D / 16][4];
        for (int j = 0; j < tile.n; j++) {
            if (j + 1 < tile.n) load(j + 1);
            cp_commit();
            cp_wait1();
            __syncthreads();
            if (j == 0) {
                a_frags<D>(smem_u32(sQ), (threadIdx.x >> 5) * 16, q);
                a_frags<D>(smem_u32(sO), (threadIdx.x >> 5) * 16, o);
            }
            float s[8][4], dp[8][4];
            product<T, D>(s, q, smem_u32(sK[j & 1]));
            product<T, D>(dp, o, smem_u32(sV[j & 1]));
            const int k0 = tile.block(j) * BLK;
            const bool masked = tile.masked(k0);
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const unsigned long long seen = masked ? g.keys(at.row + 8 * h, st[h], k0) >> (2 * at.t4) : ~0ull;
#pragma unroll
                for (int n = 0; n < 8; n++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int i = 2 * h + e;
                        s[n][i] = seen >> (8 * n + e) & 1 ? exp2f(fmaf(s[n][i], sl2, -L[h])) * (dp[n][i] - Dr[h]) : 0.0f;
                    }
            }
            accumulate<T, D>(dq, s, smem_u32(sK[j & 1]));
            __syncthreads();
        }
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int q = at.row + 8 * h;
        if (q < a.T) store_row<T, D>(dqkv + (row0 + q) * ld + at.h * D, dq, h, at.t4, scale, q < g.end);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(THREADS)
k_dkdv(const T* qkv, const float* lse, const T* dy, T* dqkv, const float* Dlt, const GroupArgs a) {
    pdl_enter();
    __shared__ __align__(128) T sK[BLK * D], sV[BLK * D], sQ[2][BLK * D], sO[2][BLK * D];
    __shared__ float s_L[2][BLK], s_D[2][BLK];
    const Place at(a, false);
    const Group g(a.starts, at.b, a.K, a.T);
    const long long ld = 3LL * a.C, row0 = (long long)at.b * a.T, bh = ((long long)at.b * a.H + at.h) * a.T;
    const T* base = qkv + row0 * ld + at.h * D;
    float dk[D / 8][4], dv[D / 8][4];
    for (int n = 0; n < D / 8; n++)
        for (int e = 0; e < 4; e++) dk[n][e] = dv[n][e] = 0.0f;
    const float scale = rsqrtf((float)D), sl2 = scale * LOG2E;
    if (at.first < g.end) {
        const group::KeyTile tile(g, at.first, BLK);
        const int kend[2] = {at.row < g.end ? g.end_of(at.row) : 0, at.row + 8 < g.end ? g.end_of(at.row + 8) : 0};
        auto load = [&](int j) {
            const int q0 = (tile.j0 + j) * BLK;
            load_tile<D>(smem_u32(sQ[j & 1]), base + q0 * ld, ld, g.end - q0);
            load_tile<D>(smem_u32(sO[j & 1]), dy + (row0 + q0) * a.C + at.h * D, a.C, g.end - q0);
            if (threadIdx.x < BLK) {
                const int q = q0 + threadIdx.x;
                s_L[j & 1][threadIdx.x] = q < g.end ? lse[bh + q] * LOG2E : 0.0f;
                s_D[j & 1][threadIdx.x] = q < g.end ? Dlt[bh + q] : 0.0f;
            }
        };
        load_tile<D>(smem_u32(sK), base + a.C + at.first * ld, ld, g.end - at.first);
        load_tile<D>(smem_u32(sV), base + 2 * a.C + at.first * ld, ld, g.end - at.first);
        load(0);
        cp_commit();
        uint32_t k[D / 16][4], v[D / 16][4];
        for (int j = 0; j < tile.n; j++) {
            if (j + 1 < tile.n) load(j + 1);
            cp_commit();
            cp_wait1();
            __syncthreads();
            if (j == 0) {
                a_frags<D>(smem_u32(sK), (threadIdx.x >> 5) * 16, k);
                a_frags<D>(smem_u32(sV), (threadIdx.x >> 5) * 16, v);
            }
            const int q0 = (tile.j0 + j) * BLK, buf = j & 1;
            float s[8][4], dp[8][4];
            product<T, D>(s, k, smem_u32(sQ[buf]));
            product<T, D>(dp, v, smem_u32(sO[buf]));
            const bool masked = tile.masked(q0);
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const unsigned long long seen =
                    masked ? g.queries(at.row + 8 * h, kend[h], q0) >> (2 * at.t4) : ~0ull;
#pragma unroll
                for (int n = 0; n < 8; n++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int i = 2 * h + e, q = 8 * n + 2 * at.t4 + e;
                        const bool on = seen >> (8 * n + e) & 1;
                        const float p = on ? exp2f(fmaf(s[n][i], sl2, -s_L[buf][q])) : 0.0f;
                        s[n][i] = p;
                        dp[n][i] = on ? p * (dp[n][i] - s_D[buf][q]) : 0.0f;
                    }
            }
            accumulate<T, D>(dv, s, smem_u32(sO[buf]));
            accumulate<T, D>(dk, dp, smem_u32(sQ[buf]));
            __syncthreads();
        }
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int key = at.row + 8 * h;
        if (key >= a.T) continue;
        T* d = dqkv + (row0 + key) * ld + at.h * D;
        store_row<T, D>(d + a.C, dk, h, at.t4, scale, key < g.end);
        store_row<T, D>(d + 2 * a.C, dv, h, at.t4, 1.0f, key < g.end);
    }
}

template <typename T, int D>
void fwd(const Launch& L, const void* qkv, void* y, float* lse, const GroupArgs& a, int ctas) {
    L.count();
    launch_k(L, k_fwd<T, D>, dim3(ctas), dim3(THREADS), 0, (const T*)qkv, (T*)y, lse, a);
}
template <typename T, int D>
void bwd(const Launch& L, const void* qkv, const void* y, const float* lse, const void* dy, void* dqkv, float* Dlt,
         const GroupArgs& a, int ctas) {
    L.count();
    launch_k(L, k_dq<T, D>, dim3(ctas), dim3(THREADS), 0, (const T*)qkv, (const T*)y, lse, (const T*)dy, (T*)dqkv, Dlt, a);
    L.count();
    launch_k(L, k_dkdv<T, D>, dim3(ctas), dim3(THREADS), 0, (const T*)qkv, lse, (const T*)dy, (T*)dqkv, (const float*)Dlt, a);
}

GroupArgs args_of(const Launch& L, const int32_t* starts, int B, int T, int C, int H, int K) {
    GroupArgs a{};
    a.starts = starts; a.T = T; a.C = C; a.H = H; a.K = K;
    a.tiles = (T + BLK - 1) / BLK;
    a.pairs = B * H;
    a.flags = L.flags;
    return a;
}

}  // namespace

void launch_group_fwd_mma(const Launch& L, const void* qkv, const int32_t* starts, void* y, float* lse, int B, int T, int C,
                          int H, int K) {
    const GroupArgs a = args_of(L, starts, B, T, C, H, K);
    const int ctas = a.tiles * B * H;
    if (C / H == 16 && L.f16) fwd<__half, 16>(L, qkv, y, lse, a, ctas);
    else if (C / H == 16) fwd<__nv_bfloat16, 16>(L, qkv, y, lse, a, ctas);
    else if (L.f16) fwd<__half, 32>(L, qkv, y, lse, a, ctas);
    else fwd<__nv_bfloat16, 32>(L, qkv, y, lse, a, ctas);
}

void launch_group_bwd_mma(const Launch& L, const void* qkv, const int32_t* starts, const void* y, const float* lse,
                          const void* dy, void* dqkv, int B, int T, int C, int H, int K, float* Dlt) {
    const GroupArgs a = args_of(L, starts, B, T, C, H, K);
    const int ctas = a.tiles * B * H;
    if (C / H == 16 && L.f16) bwd<__half, 16>(L, qkv, y, lse, dy, dqkv, Dlt, a, ctas);
    else if (C / H == 16) bwd<__nv_bfloat16, 16>(L, qkv, y, lse, dy, dqkv, Dlt, a, ctas);
    else if (L.f16) bwd<__half, 32>(L, qkv, y, lse, dy, dqkv, Dlt, a, ctas);
    else bwd<__nv_bfloat16, 32>(L, qkv, y, lse, dy, dqkv, Dlt, a, ctas);
}

}  // namespace tt
