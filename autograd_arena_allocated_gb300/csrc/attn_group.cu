// attn_group.cu -- attention over groups of answers that share a prompt
// (group.cuh) in fp32, and the choice of the kernels: 16-bit heads of 64 take
// attn_tc.cu's, of 16 and 32 attn_group_mma.cu's.
//
//   k_group_fwd   64 queries a CTA past blocks of 64 keys: S = Q K^T / sqrt(D),
//                 running maximum and sum, O += P V
//   k_group_dq    D = rowsum(dO o O), dS = P o (dO V^T - D), dQ += dS K
//   k_group_dkdv  64 keys a CTA past blocks of 64 queries: dV += P^T dO,
//                 dK += dS^T Q (a prompt's keys: every answer's queries, in order)
//
// All in fp32 FMAs, two lanes an instruction; the operands lie in shared memory
// as rows of D floats, padded by four so that the rows of eight lanes fall in
// different banks.  A thread of the 16 x 16 owns rows ty + 16 i and columns
// tx + 16 j of a 64 x 64 product, and rows ty + 16 i and D / 16 neighbouring
// columns of a 64 x D one: eight 16-byte loads for 64 multiply-adds, which is
// what bounds it.
#include "tt_internal.h"
#include "group.cuh"

#include <algorithm>

namespace tt {
namespace {

using group::BLK;
using group::Group;

constexpr int NT = 256;
constexpr int PS = BLK + 4;  // row of a 64 x 64 product
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// 64 rows of D elements, ld apart, into shared memory; rows from `valid` on are zeros
template <int D>
__device__ __forceinline__ void load_tile(float* s, const float* g, long long ld, int valid) {
    for (int i = threadIdx.x; i < BLK * (D / 4); i += NT) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        *reinterpret_cast<float4*>(s + r * (D + 4) + c) =
            r < valid ? *reinterpret_cast<const float4*>(g + (long long)r * ld + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
}

// acc[i][j] = sum_d A[ty + 16 i][d] B[tx + 16 j][d]
template <int D>
__device__ __forceinline__ void product(const float* A, const float* B, int tx, int ty, float (&acc)[4][4]) {
    float2 s[4][4];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) s[i][j] = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; i++) a[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * (D + 4) + d);
#pragma unroll
        for (int j = 0; j < 4; j++) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * (D + 4) + d);
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                s[i][j] = __ffma2_rn(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), s[i][j]);
                s[i][j] = __ffma2_rn(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), s[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = s[i][j].x + s[i][j].y;
}

// o[i][e] += sum_k P[ty + 16 i][k] X[k][tx E + e], E = D / 16
template <int D>
__device__ __forceinline__ void accumulate(const float* P, const float* X, int tx, int ty, float (&o)[4][D / 16]) {
    constexpr int E = D / 16;
#pragma unroll 4
    for (int k = 0; k < BLK; k += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; i++) p[i] = *reinterpret_cast<const float4*>(P + (ty + 16 * i) * PS + k);
        float x[4][E];
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const float* r = X + (k + u) * (D + 4) + tx * E;
            if (E == 4) {
                const float4 v = *reinterpret_cast<const float4*>(r);
                x[u][0] = v.x; x[u][E > 1 ? 1 : 0] = v.y; x[u][E > 2 ? 2 : 0] = v.z; x[u][E > 3 ? 3 : 0] = v.w;
            } else if (E == 2) {
                const float2 v = *reinterpret_cast<const float2*>(r);
                x[u][0] = v.x; x[u][E > 1 ? 1 : 0] = v.y;
            } else {
                x[u][0] = *r;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float w[4] = {p[i].x, p[i].y, p[i].z, p[i].w};
#pragma unroll
            for (int u = 0; u < 4; u++) {
                if (E == 1) o[i][0] = fmaf(w[u], x[u][0], o[i][0]);
#pragma unroll
                for (int e = 0; e + 1 < E; e += 2) {
                    const float2 r = __ffma2_rn(make_float2(w[u], w[u]), make_float2(x[u][e], x[u][e + 1]),
                                                make_float2(o[i][e], o[i][e + 1]));
                    o[i][e] = r.x;
                    o[i][e + 1] = r.y;
                }
            }
        }
    }
}

struct GroupArgs {
    const int32_t* starts;
    int T, C, H, K, tiles;
    int* flags;
};

// CTA -> (tile, head, sequence): a head's tiles side by side, so that they share
// its keys in L2; the tiles with the most work first
struct Place {
    int tile, h, b;
    __device__ __forceinline__ Place(const GroupArgs& a, bool last_first) {
        const int t = blockIdx.x % a.tiles, bh = blockIdx.x / a.tiles;
        tile = last_first ? a.tiles - 1 - t : t;
        b = bh / a.H;
        h = bh % a.H;
    }
};

template <int E> __device__ __forceinline__ void store_row(float* d, const float (&v)[E], float scale) {
#pragma unroll
    for (int e = 0; e < E; e++) d[e] = v[e] * scale;
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

template <int D> __host__ __device__ constexpr int tile_floats() { return BLK * (D + 4); }

template <int D>
__global__ void __launch_bounds__(NT, 2) k_group_fwd(const float* qkv, float* y, float* lse, const GroupArgs a) {
    pdl_enter();
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *sK = sQ + tile_floats<D>(), *sV = sK + tile_floats<D>(), *sP = sV + tile_floats<D>();
    constexpr int E = D / 16;
    const Place at(a, true);
    const Group g(a.starts, at.b, a.K, a.T);
    const int q0 = at.tile * BLK, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long ld = 3LL * a.C, row0 = (long long)at.b * a.T;
    const float* base = qkv + row0 * ld + at.h * D;
    float* yb = y + row0 * a.C + at.h * D + tx * E;
    float* lb = lse + ((long long)at.b * a.H + at.h) * a.T;
    if (at.tile == 0 && at.h == 0) g.check(threadIdx.x, NT, a.T, a.flags);
    float o[4][E], m[4], l[4];
    int st[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        m[i] = -3e38f;  // finite: a row may see nothing of a block
        l[i] = 0.0f;
        st[i] = g.start_of(q0 + ty + 16 * i);
#pragma unroll
        for (int e = 0; e < E; e++) o[i][e] = 0.0f;
    }
    if (q0 < g.end) {  // uniform over the CTA
        const group::QueryTile tile(g, q0, BLK);
        const float sl2 = rsqrtf((float)D) * LOG2E;
        load_tile<D>(sQ, base + q0 * ld, ld, g.end - q0);
        for (int j = 0; j < tile.n; j++) {
            const int k0 = tile.block(j) * BLK;
            __syncthreads();  // the block before has been used
            load_tile<D>(sK, base + a.C + k0 * ld, ld, g.end - k0);
            load_tile<D>(sV, base + 2 * a.C + k0 * ld, ld, g.end - k0);
            __syncthreads();
            float s[4][4];
            product<D>(sQ, sK, tx, ty, s);
            const bool masked = tile.masked(k0);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const unsigned long long seen = masked ? g.keys(q0 + ty + 16 * i, st[i], k0) : ~0ull;
                float mx = -3e38f;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    s[i][c] *= sl2;
                    if (seen >> (tx + 16 * c) & 1) mx = fmaxf(mx, s[i][c]);
                }
                const float mn = fmaxf(m[i], row_max(mx)), corr = exp2f(m[i] - mn);
                float rs = 0.0f;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const float p = seen >> (tx + 16 * c) & 1 ? exp2f(s[i][c] - mn) : 0.0f;
                    sP[(ty + 16 * i) * PS + tx + 16 * c] = p;
                    rs += p;
                }
                m[i] = mn;
                l[i] = l[i] * corr + row_sum(rs);
#pragma unroll
                for (int e = 0; e < E; e++) o[i][e] *= corr;
            }
            __syncwarp();  // a row of P is its 16 lanes' own
            accumulate<D>(sP, sV, tx, ty, o);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int q = q0 + ty + 16 * i;
        if (q >= a.T) continue;
        const bool on = q < g.end;
        float v[E];
#pragma unroll
        for (int e = 0; e < E; e++) v[e] = on ? o[i][e] / l[i] : 0.0f;
        store_row(yb + (long long)q * a.C, v, 1.0f);
        if (tx == 0) lb[q] = on ? (m[i] + log2f(l[i])) * LN2 : 0.0f;
    }
}

template <int D>
__global__ void __launch_bounds__(NT, 2)
k_group_dq(const float* qkv, const float* y, const float* lse, const float* dy, float* dqkv, float* Dlt, const GroupArgs a) {
    pdl_enter();
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *sO = sQ + tile_floats<D>(), *sK = sO + tile_floats<D>(), *sV = sK + tile_floats<D>(),
          *sS = sV + tile_floats<D>();
    constexpr int E = D / 16;
    const Place at(a, true);
    const Group g(a.starts, at.b, a.K, a.T);
    const int q0 = at.tile * BLK, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long ld = 3LL * a.C, row0 = (long long)at.b * a.T;
    const float* base = qkv + row0 * ld + at.h * D;
    const long long bh = ((long long)at.b * a.H + at.h) * a.T;
    if (at.tile == 0 && at.h == 0) g.check(threadIdx.x, NT, a.T, a.flags);
    float o[4][E];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int e = 0; e < E; e++) o[i][e] = 0.0f;
    const float scale = rsqrtf((float)D);
    if (q0 < g.end) {
        const group::QueryTile tile(g, q0, BLK);
        const float sl2 = scale * LOG2E;
        load_tile<D>(sQ, base + q0 * ld, ld, g.end - q0);
        load_tile<D>(sO, dy + (row0 + q0) * a.C + at.h * D, a.C, g.end - q0);
        load_tile<D>(sK, y + (row0 + q0) * a.C + at.h * D, a.C, g.end - q0);  // y, for D alone
        __syncthreads();
        float L[4], Dr[4];
        int st[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int r = ty + 16 * i, q = q0 + r;
            float d = 0.0f;
#pragma unroll
            for (int e = 0; e < E; e++) d = fmaf(sO[r * (D + 4) + tx * E + e], sK[r * (D + 4) + tx * E + e], d);
            Dr[i] = row_sum(d);
            L[i] = q < g.end ? lse[bh + q] * LOG2E : 0.0f;
            st[i] = g.start_of(q);
            if (tx == 0 && q < g.end) Dlt[bh + q] = Dr[i];
        }
        for (int j = 0; j < tile.n; j++) {
            const int k0 = tile.block(j) * BLK;
            __syncthreads();
            load_tile<D>(sK, base + a.C + k0 * ld, ld, g.end - k0);
            load_tile<D>(sV, base + 2 * a.C + k0 * ld, ld, g.end - k0);
            __syncthreads();
            float s[4][4], dp[4][4];
            product<D>(sQ, sK, tx, ty, s);
            product<D>(sO, sV, tx, ty, dp);
            const bool masked = tile.masked(k0);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const unsigned long long seen =
                    masked ? g.keys(q0 + ty + 16 * i, st[i], k0) : q0 + ty + 16 * i < g.end ? ~0ull : 0ull;
#pragma unroll
                for (int c = 0; c < 4; c++)
                    sS[(ty + 16 * i) * PS + tx + 16 * c] =
                        seen >> (tx + 16 * c) & 1 ? exp2f(fmaf(s[i][c], sl2, -L[i])) * (dp[i][c] - Dr[i]) : 0.0f;
            }
            __syncwarp();
            accumulate<D>(sS, sK, tx, ty, o);
        }
    }
    float* ob = dqkv + row0 * ld + at.h * D + tx * E;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int q = q0 + ty + 16 * i;
        if (q < a.T) store_row(ob + (long long)q * ld, o[i], q < g.end ? scale : 0.0f);
    }
}

template <int D>
__global__ void __launch_bounds__(NT, 2)
k_group_dkdv(const float* qkv, const float* lse, const float* dy, float* dqkv, const float* Dlt, const GroupArgs a) {
    pdl_enter();
    extern __shared__ __align__(16) float sm[];
    float *sK = sm, *sV = sK + tile_floats<D>(), *sQ = sV + tile_floats<D>(), *sO = sQ + tile_floats<D>(),
          *sP = sO + tile_floats<D>(), *sS = sP + BLK * PS;
    __shared__ float s_L[BLK], s_D[BLK];
    constexpr int E = D / 16;
    const Place at(a, false);
    const Group g(a.starts, at.b, a.K, a.T);
    const int k0 = at.tile * BLK, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long ld = 3LL * a.C, row0 = (long long)at.b * a.T;
    const float* base = qkv + row0 * ld + at.h * D;
    const long long bh = ((long long)at.b * a.H + at.h) * a.T;
    const float scale = rsqrtf((float)D);
    float dk[4][E], dv[4][E];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int e = 0; e < E; e++) dk[i][e] = dv[i][e] = 0.0f;
    if (k0 < g.end) {
        const group::KeyTile tile(g, k0, BLK);
        const float sl2 = scale * LOG2E;
        load_tile<D>(sK, base + a.C + k0 * ld, ld, g.end - k0);
        load_tile<D>(sV, base + 2 * a.C + k0 * ld, ld, g.end - k0);
        int kend[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int k = k0 + ty + 16 * i;
            kend[i] = k < g.end ? g.end_of(k) : 0;
        }
        for (int j = 0; j < tile.n; j++) {
            const int q0 = (tile.j0 + j) * BLK;
            __syncthreads();
            load_tile<D>(sQ, base + q0 * ld, ld, g.end - q0);
            load_tile<D>(sO, dy + (row0 + q0) * a.C + at.h * D, a.C, g.end - q0);
            if (threadIdx.x < BLK) {
                const int q = q0 + threadIdx.x;
                s_L[threadIdx.x] = q < g.end ? lse[bh + q] * LOG2E : 0.0f;
                s_D[threadIdx.x] = q < g.end ? Dlt[bh + q] : 0.0f;
            }
            __syncthreads();
            float s[4][4], dp[4][4];
            product<D>(sK, sQ, tx, ty, s);
            product<D>(sV, sO, tx, ty, dp);
            const bool masked = tile.masked(q0);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int k = k0 + ty + 16 * i;
                const unsigned long long seen = masked ? g.queries(k, kend[i], q0) : k < g.end ? ~0ull : 0ull;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const int q = tx + 16 * c;
                    const bool on = seen >> q & 1;
                    const float p = on ? exp2f(fmaf(s[i][c], sl2, -s_L[q])) : 0.0f;
                    sP[(ty + 16 * i) * PS + q] = p;
                    sS[(ty + 16 * i) * PS + q] = on ? p * (dp[i][c] - s_D[q]) : 0.0f;
                }
            }
            __syncwarp();
            accumulate<D>(sP, sO, tx, ty, dv);
            accumulate<D>(sS, sQ, tx, ty, dk);
        }
    }
    float* ob = dqkv + row0 * ld + at.h * D + tx * E;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int k = k0 + ty + 16 * i;
        if (k >= a.T) continue;
        store_row(ob + (long long)k * ld + a.C, dk[i], k < g.end ? scale : 0.0f);
        store_row(ob + (long long)k * ld + 2 * a.C, dv[i], k < g.end ? 1.0f : 0.0f);
    }
}

template <typename K> bool allow(PerDevice& done, K kern, size_t smem) {
    return done.once([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess;
    });
}

template <int D> bool fwd(const Launch& L, const float* qkv, float* y, float* lse, const GroupArgs& a, int ctas) {
    static PerDevice done;
    constexpr size_t smem = (3 * tile_floats<D>() + BLK * PS) * 4;
    if (!allow(done, k_group_fwd<D>, smem)) return false;
    L.count();
    launch_k(L, k_group_fwd<D>, dim3(ctas), dim3(NT), smem, qkv, y, lse, a);
    return true;
}

template <int D>
bool bwd(const Launch& L, const float* qkv, const float* y, const float* lse, const float* dy, float* dqkv, float* Dlt,
         const GroupArgs& a, int ctas) {
    static PerDevice done_q, done_k;
    constexpr size_t sq = (4 * tile_floats<D>() + BLK * PS) * 4, sk = (4 * tile_floats<D>() + 2 * BLK * PS) * 4;
    if (!allow(done_q, k_group_dq<D>, sq) || !allow(done_k, k_group_dkdv<D>, sk)) return false;
    L.count();
    launch_k(L, k_group_dq<D>, dim3(ctas), dim3(NT), sq, qkv, y, lse, dy, dqkv, Dlt, a);
    L.count();
    launch_k(L, k_group_dkdv<D>, dim3(ctas), dim3(NT), sk, qkv, lse, dy, dqkv, (const float*)Dlt, a);
    return true;
}

GroupArgs args_of(const Launch& L, const int32_t* starts, int T, int C, int H, int K) {
    GroupArgs a{};
    a.starts = starts; a.T = T; a.C = C; a.H = H; a.K = K;
    a.tiles = (T + BLK - 1) / BLK;
    a.flags = L.flags;
    return a;
}

}  // namespace

bool launch_group_attention_fwd(const Launch& L, bool bf16, const void* qkv, const int32_t* starts, void* y, float* lse,
                                int B, int T, int C, int H, int K) {
    if (L.dry) return true;
    const int hd = C / H;
    if (bf16 && hd == 64) return launch_attention_fwd_tc(L, qkv, y, lse, B, T, C, H, starts, K);
    if (bf16) {
        launch_group_fwd_mma(L, qkv, starts, y, lse, B, T, C, H, K);
        return true;
    }
    const GroupArgs a = args_of(L, starts, T, C, H, K);
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
        launch_group_bwd_mma(L, qkv, starts, y, lse, dy, dqkv, B, T, C, H, K, scratch);
    } else {
        const GroupArgs a = args_of(L, starts, T, C, H, K);
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
