// attn_group.cu -- attention over groups of answers that share a prompt
// (group.cuh) in fp32, and the choice of the kernels: 16 bits take attn_tc.cu's.
//
//   k_group_fwd   64 queries a CTA past blocks of 64 keys: S = Q K^T / sqrt(D),
//                 running maximum and sum, O += P V
//   k_group_dq    D = rowsum(dO o O), dS = P o (dO V^T - D), dQ += dS K
//   k_group_dkdv  64 keys a CTA past blocks of 64 queries: dV += P^T dO,
//                 dK += dS^T Q (a prompt's keys: every answer's queries, in order)
//
// All in fp32 FMAs, two rows an instruction.  A thread of the 8 x 16 owns rows 8 ty
// .. + 7 (heads of 16: of 16 x 16, 4 rows) and columns 4 tx .. + 3 of a 64 x 64
// product, and the same rows and D / 16 columns of a 64 x D one: 32 multiply-adds
// take three 16-byte loads from shared memory.  The tiles that a product sums over D lie transposed.  The next block is
// fetched into registers while the products run.  What bounds it is the issue of
// instructions, half of them FMAs: 8 groups of 1000 positions, 12 heads of 64, 374
// us forward and 1013 backward, 27 and 25 TFLOP/s of some 74 (one group of 1976, 16
// heads, 258 and 681; by pieces of 4 x 4 that read two rows a time, without the
// fetch ahead, 293 and 913).  Registers set how much is resident: three CTAs an SM
// forward (heads of 16: two), two backward (one), and at heads of 64 the forward
// spills 96 bytes, the keys' kernel 8.
#include "tt_internal.h"
#include "group.cuh"

namespace tt {
namespace {

using group::BLK;
using group::Group;

// Rows of a product that a thread has, and the threads of a CTA.  Heads of 16 have so
// little to do a block that a thread's own chain of instructions counts: 4 rows and
// 256 threads, one group of 7900 positions, 4 heads: 301 us forward and 1008 backward
// (8 rows and 128 threads 348 and 1016), 4 groups of 40, 4 heads: 5.6 (7.1).
template <int D> constexpr int R_OF = D == 16 ? 4 : 8;
template <int D> constexpr int NT_OF = 16 * BLK / R_OF<D>;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// places in the tiles, in floats: [64][D] by rows, [D][64] transposed, and a 64 x 64
// product transposed, [column][row].  Loads meet no bank twice; the stores of a
// row tile and of a product do four times, which costs less than the arithmetic of
// a swizzle in the loops that load.
constexpr int PS = BLK + 4;
template <int D> __device__ __forceinline__ int at_row(int row, int col) { return row * D + col; }
__device__ __forceinline__ int at_col(int d, int row) { return d * BLK + row; }
__device__ __forceinline__ int at_prod(int col, int row) { return col * PS + row; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a thread's part of 64 rows of D floats: two (four) neighbouring threads have a row
template <int D> struct Piece {
    static constexpr int TPR = NT_OF<D> / BLK, N = D / 4 / TPR;
    float4 v[N];
    static __device__ __forceinline__ int row() { return threadIdx.x / TPR; }
    static __device__ __forceinline__ int col(int i) { return 4 * (threadIdx.x % TPR + TPR * i); }
    // rows of g, ld apart; those from `valid` on are zeros
    __device__ __forceinline__ void load(const float* g, long long ld, int valid) {
#pragma unroll
        for (int i = 0; i < N; i++)
            v[i] = row() < valid ? *reinterpret_cast<const float4*>(g + row() * ld + col(i)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    __device__ __forceinline__ void rows(float* s) const {
#pragma unroll
        for (int i = 0; i < N; i++) *reinterpret_cast<float4*>(s + at_row<D>(row(), col(i))) = v[i];
    }
    __device__ __forceinline__ void cols(float* s) const {
#pragma unroll
        for (int i = 0; i < N; i++) {
            s[at_col(col(i), row())] = v[i].x;
            s[at_col(col(i) + 1, row())] = v[i].y;
            s[at_col(col(i) + 2, row())] = v[i].z;
            s[at_col(col(i) + 3, row())] = v[i].w;
        }
    }
};

// acc[i][j]: rows R ty + 2 i, + 1 of column 4 tx + j
template <int D> using Acc = float2[R_OF<D> / 2][4];

// a thread's R rows of column c of a transposed tile, as pairs
template <int R> __device__ __forceinline__ void row_pairs(const float* p, float2 (&a)[R / 2]) {
#pragma unroll
    for (int i = 0; i < R / 4; i++) {
        const float4 v = *reinterpret_cast<const float4*>(p + 4 * i);
        a[2 * i] = make_float2(v.x, v.y);
        a[2 * i + 1] = make_float2(v.z, v.w);
    }
}

// sum over d of A[row][d] B[col][d], both tiles transposed
template <int D> __device__ __forceinline__ void product(const float* A, const float* B, int tx, int ty, Acc<D>& s) {
    constexpr int R = R_OF<D>;
#pragma unroll
    for (int i = 0; i < R / 2; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) s[i][j] = make_float2(0.0f, 0.0f);
#pragma unroll 8
    for (int d = 0; d < D; d++) {
        float2 a[R / 2];
        row_pairs<R>(A + at_col(d, R * ty), a);
        const float4 b = *reinterpret_cast<const float4*>(B + at_col(d, 4 * tx));
        const float c[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < R / 2; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) s[i][j] = __ffma2_rn(a[i], make_float2(c[j], c[j]), s[i][j]);
    }
}

// o[i][e] += sum over k of P[k][rows R ty + 2 i, + 1] X[k][tx E + e], E = D / 16
template <int D>
__device__ __forceinline__ void accumulate(const float* P, const float* X, int tx, int ty, float2 (&o)[R_OF<D> / 2][D / 16]) {
    constexpr int E = D / 16, R = R_OF<D>;
#pragma unroll 8
    for (int k = 0; k < BLK; k++) {
        float2 a[R / 2];
        row_pairs<R>(P + at_prod(k, R * ty), a);
        const float* x = X + at_row<D>(k, tx * E);
        float c[4];
        if (E == 4) {
            const float4 b = *reinterpret_cast<const float4*>(x);
            c[0] = b.x; c[1] = b.y; c[2] = b.z; c[3] = b.w;
        } else if (E == 2) {
            const float2 b = *reinterpret_cast<const float2*>(x);
            c[0] = b.x; c[1] = b.y;
        } else {
            c[0] = *x;
        }
#pragma unroll
        for (int i = 0; i < R / 2; i++)
#pragma unroll
            for (int e = 0; e < E; e++) o[i][e] = __ffma2_rn(a[i], make_float2(c[e], c[e]), o[i][e]);
    }
}

// row r of a thread's
template <int N> __device__ __forceinline__ float& of(float2 (&s)[N][4], int r, int j) { return r & 1 ? s[r >> 1][j].y : s[r >> 1][j].x; }

// a product goes to shared memory for accumulate; its 16 lanes of a row group alone
// read it
template <int N> __device__ __forceinline__ void put_product(float* P, const float2 (&s)[N][4], int tx, int ty) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int i = 0; i < N; i += 2)
            *reinterpret_cast<float4*>(P + at_prod(4 * tx + j, 2 * N * ty + 2 * i)) =
                make_float4(s[i][j].x, s[i][j].y, s[i + 1][j].x, s[i + 1][j].y);
    __syncwarp();
}

struct GroupArgs {
    const int32_t* starts;
    int T, C, H, K, tiles, pairs;
    int* flags;
};

template <int N, int E> __device__ __forceinline__ void zero(float2 (&o)[N][E]) {
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int e = 0; e < E; e++) o[i][e] = make_float2(0.0f, 0.0f);
}

// row r of a thread's E columns, times scale; zeros where it is padding
template <int N, int E> __device__ __forceinline__ void store_row(float* d, const float2 (&o)[N][E], int r, float scale, bool real) {
#pragma unroll
    for (int e = 0; e < E; e++) d[e] = real ? (r & 1 ? o[r >> 1][e].y : o[r >> 1][e].x) * scale : 0.0f;
}

__device__ __forceinline__ float row_max(float v) {  // over the 16 lanes of a row
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int D> __global__ void __launch_bounds__(NT_OF<D>, D == 16 ? 2 : 3) k_group_fwd(const float* qkv, float* y, float* lse, const GroupArgs a) {
    pdl_enter();
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *sK = sQ + BLK * D, *sV = sK + BLK * D, *sP = sV + BLK * D;
    constexpr int E = D / 16, R = R_OF<D>;
    const group::Place at(a.tiles, a.pairs, a.H, true);
    const Group g(a.starts, at.b, a.K, a.T);
    const int q0 = at.tile * BLK, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long ld = 3LL * a.C, row0 = (long long)at.b * a.T;
    const float* base = qkv + row0 * ld + at.h * D;
    if (q0 == 0 && at.h == 0) g.check(threadIdx.x, NT_OF<D>, a.T, a.flags);
    float2 o[R / 2][E];
    zero(o);
    float m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        m[r] = -3e38f;  // finite: a row may see nothing of a block
        l[r] = 0.0f;
    }
    const float sl2 = rsqrtf((float)D) * LOG2E;
    if (q0 < g.end) {  // uniform over the CTA
        const group::QueryTile tile(g, q0, BLK);
        Piece<D> k, v;
        k.load(base + q0 * ld, ld, g.end - q0);
        k.cols(sQ);
        auto fetch = [&](int j) {
            const int k0 = tile.block(j) * BLK;
            k.load(base + a.C + k0 * ld, ld, g.end - k0);
            v.load(base + 2 * a.C + k0 * ld, ld, g.end - k0);
        };
        fetch(0);
        for (int j = 0; j < tile.n; j++) {
            const int k0 = tile.block(j) * BLK;
            __syncthreads();  // the block before has been used
            k.cols(sK);
            v.rows(sV);
            __syncthreads();
            if (j + 1 < tile.n) fetch(j + 1);
            Acc<D> s;
            product<D>(sQ, sK, tx, ty, s);
            if (tile.masked(k0)) {
#pragma unroll
                for (int r = 0; r < R; r++) {
                    const int q = q0 + R * ty + r;
                    const uint32_t seen = (uint32_t)(g.keys(q, g.start_of(q), k0) >> (4 * tx));
#pragma unroll
                    for (int c = 0; c < 4; c++)
                        if (!(seen >> c & 1u)) of(s, r, c) = -INFINITY;
                }
            }
#pragma unroll
            for (int r = 0; r < R; r++) {
                // m is the largest score, before the scale
                const float mx = row_max(fmaxf(fmaxf(of(s, r, 0), of(s, r, 1)), fmaxf(of(s, r, 2), of(s, r, 3))));
                const float mn = fmaxf(m[r], mx), corr = ex2((m[r] - mn) * sl2);
                float rs = 0.0f;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    of(s, r, c) = ex2((of(s, r, c) - mn) * sl2);  // of -inf: 0
                    rs += of(s, r, c);
                }
                m[r] = mn;
                l[r] = l[r] * corr + rs;  // this lane's columns; the lanes' sums meet at the end
#pragma unroll
                for (int e = 0; e < E; e++) {
                    if (r & 1) o[r >> 1][e].y *= corr;
                    else o[r >> 1][e].x *= corr;
                }
            }
            put_product(sP, s, tx, ty);
            accumulate<D>(sP, sV, tx, ty, o);
        }
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int q = q0 + R * ty + r;
        const float sum = row_sum(l[r]);
        if (q >= a.T) continue;
        store_row(y + (row0 + q) * a.C + at.h * D + tx * E, o, r, 1.0f / sum, q < g.end);
        if (tx == 0) lse[((long long)at.b * a.H + at.h) * a.T + q] = q < g.end ? (m[r] * sl2 + log2f(sum)) * LN2 : 0.0f;
    }
}

template <int D>
__global__ void __launch_bounds__(NT_OF<D>, D == 16 ? 1 : 2)
k_group_dq(const float* qkv, const float* y, const float* lse, const float* dy, float* dqkv, float* Dlt, const GroupArgs a) {
    pdl_enter();
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *sO = sQ + BLK * D, *sK = sO + BLK * D, *sV = sK + BLK * D, *sX = sV + BLK * D, *sS = sX + BLK * D;
    constexpr int E = D / 16, R = R_OF<D>;
    const group::Place at(a.tiles, a.pairs, a.H, true);
    const Group g(a.starts, at.b, a.K, a.T);
    const int q0 = at.tile * BLK, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long ld = 3LL * a.C, row0 = (long long)at.b * a.T, bh = ((long long)at.b * a.H + at.h) * a.T;
    const float* base = qkv + row0 * ld + at.h * D;
    if (q0 == 0 && at.h == 0) g.check(threadIdx.x, NT_OF<D>, a.T, a.flags);
    float2 o[R / 2][E];
    zero(o);
    const float scale = rsqrtf((float)D);
    if (q0 < g.end) {
        const group::QueryTile tile(g, q0, BLK);
        const float sl2 = scale * LOG2E;
        __shared__ float s_D[BLK];
        Piece<D> k, v;
        k.load(base + q0 * ld, ld, g.end - q0);
        k.cols(sQ);
        // D = rowsum(dO o O): the threads of a row add their parts
        k.load(dy + (row0 + q0) * a.C + at.h * D, a.C, g.end - q0);
        k.cols(sO);
        v.load(y + (row0 + q0) * a.C + at.h * D, a.C, g.end - q0);
        float d = 0.0f;
#pragma unroll
        for (int i = 0; i < Piece<D>::N; i++)
            d = fmaf(k.v[i].x, v.v[i].x, fmaf(k.v[i].y, v.v[i].y, fmaf(k.v[i].z, v.v[i].z, fmaf(k.v[i].w, v.v[i].w, d))));
#pragma unroll
        for (int x = 1; x < Piece<D>::TPR; x *= 2) d += __shfl_xor_sync(0xffffffffu, d, x);
        if (threadIdx.x % Piece<D>::TPR == 0) {
            const int r = Piece<D>::row();
            s_D[r] = d;
            if (q0 + r < g.end) Dlt[bh + q0 + r] = d;
        }
        float L[R];
#pragma unroll
        for (int r = 0; r < R; r++) L[r] = q0 + R * ty + r < g.end ? lse[bh + q0 + R * ty + r] * LOG2E : 0.0f;
        auto fetch = [&](int j) {
            const int k0 = tile.block(j) * BLK;
            k.load(base + a.C + k0 * ld, ld, g.end - k0);
            v.load(base + 2 * a.C + k0 * ld, ld, g.end - k0);
        };
        fetch(0);
        for (int j = 0; j < tile.n; j++) {
            const int k0 = tile.block(j) * BLK;
            __syncthreads();
            k.cols(sK);
            k.rows(sX);
            v.cols(sV);
            __syncthreads();
            if (j + 1 < tile.n) fetch(j + 1);
            Acc<D> s, dp;
            product<D>(sQ, sK, tx, ty, s);
            product<D>(sO, sV, tx, ty, dp);
#pragma unroll
            for (int r = 0; r < R; r++) {
                const float Dr = s_D[R * ty + r];
#pragma unroll
                for (int c = 0; c < 4; c++) of(s, r, c) = ex2(fmaf(of(s, r, c), sl2, -L[r])) * (of(dp, r, c) - Dr);
            }
            if (tile.masked(k0)) {
#pragma unroll
                for (int r = 0; r < R; r++) {
                    const int q = q0 + R * ty + r;
                    const uint32_t seen = (uint32_t)(g.keys(q, g.start_of(q), k0) >> (4 * tx));
#pragma unroll
                    for (int c = 0; c < 4; c++)
                        if (!(seen >> c & 1u)) of(s, r, c) = 0.0f;
                }
            }
            put_product(sS, s, tx, ty);
            accumulate<D>(sS, sX, tx, ty, o);
        }
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int q = q0 + R * ty + r;
        if (q < a.T) store_row(dqkv + (row0 + q) * ld + at.h * D + tx * E, o, r, scale, q < g.end);
    }
}

template <int D>
__global__ void __launch_bounds__(NT_OF<D>, D == 16 ? 1 : 2)
k_group_dkdv(const float* qkv, const float* lse, const float* dy, float* dqkv, const float* Dlt, const GroupArgs a) {
    pdl_enter();
    extern __shared__ __align__(16) float sm[];
    float *sK = sm, *sV = sK + BLK * D, *sQ = sV + BLK * D, *sO = sQ + BLK * D, *sX = sO + BLK * D, *sY = sX + BLK * D,
          *sP = sY + BLK * D;
    constexpr int E = D / 16, R = R_OF<D>;
    const group::Place at(a.tiles, a.pairs, a.H, false);
    const Group g(a.starts, at.b, a.K, a.T);
    const int k0 = at.tile * BLK, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long ld = 3LL * a.C, row0 = (long long)at.b * a.T, bh = ((long long)at.b * a.H + at.h) * a.T;
    const float* base = qkv + row0 * ld + at.h * D;
    const float scale = rsqrtf((float)D);
    float2 dk[R / 2][E], dv[R / 2][E];
    zero(dk);
    zero(dv);
    if (k0 < g.end) {
        const group::KeyTile tile(g, k0, BLK);
        const float sl2 = scale * LOG2E;
        Piece<D> q, o;
        q.load(base + a.C + k0 * ld, ld, g.end - k0);
        q.cols(sK);
        q.load(base + 2 * a.C + k0 * ld, ld, g.end - k0);
        q.cols(sV);
        auto fetch = [&](int j) {
            const int q0 = (tile.j0 + j) * BLK;
            q.load(base + q0 * ld, ld, g.end - q0);
            o.load(dy + (row0 + q0) * a.C + at.h * D, a.C, g.end - q0);
        };
        fetch(0);
        for (int j = 0; j < tile.n; j++) {
            const int q0 = (tile.j0 + j) * BLK;
            __syncthreads();
            q.cols(sQ);
            q.rows(sX);
            o.cols(sO);
            o.rows(sY);
            __syncthreads();
            if (j + 1 < tile.n) fetch(j + 1);
            float L[4], Dr[4];  // of the thread's four queries
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const int i = q0 + 4 * tx + c;
                L[c] = i < g.end ? lse[bh + i] * LOG2E : 0.0f;
                Dr[c] = i < g.end ? Dlt[bh + i] : 0.0f;
            }
            Acc<D> s, dp;
            product<D>(sK, sQ, tx, ty, s);
            product<D>(sV, sO, tx, ty, dp);
#pragma unroll
            for (int r = 0; r < R; r++)
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    of(s, r, c) = ex2(fmaf(of(s, r, c), sl2, -L[c]));
                    of(dp, r, c) = of(s, r, c) * (of(dp, r, c) - Dr[c]);
                }
            if (tile.masked(q0)) {
#pragma unroll
                for (int r = 0; r < R; r++) {
                    const int k = k0 + R * ty + r;
                    const uint32_t seen = k < g.end ? (uint32_t)(g.queries(k, g.end_of(k), q0) >> (4 * tx)) : 0u;
#pragma unroll
                    for (int c = 0; c < 4; c++)
                        if (!(seen >> c & 1u)) of(s, r, c) = of(dp, r, c) = 0.0f;
                }
            }
            put_product(sP, s, tx, ty);
            accumulate<D>(sP, sY, tx, ty, dv);
            put_product(sP, dp, tx, ty);
            accumulate<D>(sP, sX, tx, ty, dk);
        }
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int k = k0 + R * ty + r;
        if (k >= a.T) continue;
        float* d = dqkv + (row0 + k) * ld + at.h * D + tx * E;
        store_row(d + a.C, dk, r, scale, k < g.end);
        store_row(d + 2 * a.C, dv, r, 1.0f, k < g.end);
    }
}

template <typename K> bool allow(PerDevice& done, K kern, size_t smem) {
    return done.once([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess;
    });
}

// `tiles` tiles of 64 rows and one product
template <int D> constexpr size_t smem_of(int tiles) { return (size_t)(tiles * BLK * D + BLK * PS) * sizeof(float); }

template <int D> bool fwd(const Launch& L, const float* qkv, float* y, float* lse, const GroupArgs& a, int ctas) {
    static PerDevice done;
    if (!allow(done, k_group_fwd<D>, smem_of<D>(3))) return false;
    L.count();
    launch_k(L, k_group_fwd<D>, dim3(ctas), dim3(NT_OF<D>), smem_of<D>(3), qkv, y, lse, a);
    return true;
}

template <int D>
bool bwd(const Launch& L, const float* qkv, const float* y, const float* lse, const float* dy, float* dqkv, float* Dlt,
         const GroupArgs& a, int ctas) {
    static PerDevice done_q, done_k;
    if (!allow(done_q, k_group_dq<D>, smem_of<D>(5)) || !allow(done_k, k_group_dkdv<D>, smem_of<D>(6))) return false;
    L.count();
    launch_k(L, k_group_dq<D>, dim3(ctas), dim3(NT_OF<D>), smem_of<D>(5), qkv, y, lse, dy, dqkv, Dlt, a);
    L.count();
    launch_k(L, k_group_dkdv<D>, dim3(ctas), dim3(NT_OF<D>), smem_of<D>(6), qkv, lse, dy, dqkv, (const float*)Dlt, a);
    return true;
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

bool launch_group_attention_fwd(const Launch& L, bool bf16, const void* qkv, const int32_t* starts, void* y, float* lse,
                                int B, int T, int C, int H, int K) {
    if (L.dry) return true;
    const int hd = C / H;
    if (bf16) return launch_attention_fwd_tc(L, qkv, y, lse, B, T, C, H, starts, K);
    const GroupArgs a = args_of(L, starts, B, T, C, H, K);
    const int ctas = a.tiles * B * H;
    const auto *q = (const float*)qkv;
    auto* o = (float*)y;
    return hd == 16 ? fwd<16>(L, q, o, lse, a, ctas) : hd == 32 ? fwd<32>(L, q, o, lse, a, ctas) : fwd<64>(L, q, o, lse, a, ctas);
}

bool launch_group_attention_bwd(const Launch& L, bool bf16, const void* qkv, const int32_t* starts, const void* y,
                                const float* lse, const void* dy, void* dqkv, int B, int T, int C, int H, int K,
                                float* scratch, float* dbias, bool acc_bias) {
    if (L.dry) return true;
    const int hd = C / H;
    float* bpart = scratch + attention_d_floats(B, T, H);
    if (bf16 && hd == 64) {
        if (!launch_attention_bwd_tc(L, qkv, y, lse, dy, dqkv, B, T, C, H, scratch, dbias ? bpart : nullptr, starts, K))
            return false;
        if (dbias) launch_sum_rows(L, bpart, B * ((T + 127) / 128), 3 * C, 3 * C, dbias, nullptr, acc_bias);
        return true;
    }
    if (bf16) {
        if (!launch_attention_bwd_tc(L, qkv, y, lse, dy, dqkv, B, T, C, H, scratch, nullptr, starts, K)) return false;
    } else {
        const GroupArgs a = args_of(L, starts, B, T, C, H, K);
        const int ctas = a.tiles * B * H;
        auto run = [&](auto f) {
            return f(L, (const float*)qkv, (const float*)y, lse, (const float*)dy, (float*)dqkv, scratch, a, ctas);
        };
        if (!(hd == 16 ? run(bwd<16>) : hd == 32 ? run(bwd<32>) : run(bwd<64>))) return false;
    }
    if (dbias) launch_colsum(L, bf16, dqkv, B * T, 3 * C, dbias, bpart, acc_bias);
    return true;
}

}  // namespace tt
