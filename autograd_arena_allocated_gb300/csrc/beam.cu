// beam.cu -- beam search: the choice of the next hypotheses among the beams'
// best continuations, the reordering of per-beam state, the prompt's cache
// copied to every beam, and the walk back along the chosen parents.
//
//   k_beam_merge    per sequence the n best of its K beams' lists
//   k_beam_reorder  state rows of K slots moved in place along parents[K]
//   k_kv_fill_beams keys and values of a prompt into the K cache rows of its beams
//   k_beam_walk     the K token sequences, from the last step's back to the first
#include "head_row.cuh"

#include <algorithm>

namespace tt {
namespace {

using namespace head;

// One CTA per sequence: it joins the parts' lists of each beam, then ranks the
// beams' candidates.  Candidate (j, v) of beam j has the score
//   s_j + (z_v - lse_j)          for a live beam
//   s_j for v = eos, else -inf   for a finished one (done_j != 0)
// in 64 bits: the cumulative scores of long hypotheses are hundreds, where a
// 32-bit sum would tie or swap candidates that differ by less than 1e-5.
// A beam without a distribution (its log-sum-exp is not finite) or without a
// finite score offers -inf only.  Order: score, then the lowest j V + v.
//
// Beams with the same score and the same list are the same hypothesis as far
// as this step goes, and their candidates have to tie; but a row's
// log-sum-exp depends in its last bits on how the row lies in memory.  Such a
// beam takes the log-sum-exp of the first one it equals, where the two are
// within LSE_EPS: the rounding of arguments of up to 20 log2(e) by half a step
// (1.3e-6) and of 100 additions in a row (6e-6), whatever the logits' own size is.
//
// A step's time is the two kernels' latency: the lists of 4 rows in 32 parts
// and this merge take 12 us, those of 256 fp32 rows (51 MB) in 14 parts 28 us.
constexpr int BM_THREADS = 256;
constexpr double LSE_EPS = 1e-5;

// Scores are compared as whole numbers: the 64-bit float unit is so narrow that
// 128 candidates' comparisons took longer than all the rest.
__device__ __forceinline__ unsigned long long order_of(double v) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
    return u >> 63 ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ double value_of(unsigned long long u) {
    return __longlong_as_double((long long)(u >> 63 ? u & ~(1ull << 63) : ~u));
}

constexpr int BM_ENTRIES = 4096;  // of a sequence's lists: K * parts * n

__global__ void __launch_bounds__(BM_THREADS)
k_beam_merge(const unsigned long long* __restrict__ keys, const float2* __restrict__ parts, const float* scores,
             const int32_t* done, int K, int P, int V, int kk, int n, int eos, int32_t* parent, int32_t* token,
             float* out_scores, int32_t* out_done, int32_t* __restrict__ tok_hist, int32_t* __restrict__ par_hist,
             int ld_hist, const int* __restrict__ pos_dev, int* flags) {
    pdl_enter();
    extern __shared__ __align__(16) char smem[];
    const int N = K * kk, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto* s_in = reinterpret_cast<unsigned long long*>(smem);  // [K][P][kk]
    auto* s_j = s_in + (P > 1 ? N * P : 0);                    // [K][kk]
    auto* s_s = s_j + N;                                       // [K][kk] scores, as whole numbers in order
    int* s_f = reinterpret_cast<int*>(s_s + N);                // [K][kk] j V + v
    __shared__ __align__(16) unsigned long long s_key[BM_THREADS / 32][JOIN_ROOM];
    __shared__ double s_lse[TT_BEAM_MAX];
    __shared__ float s_sc[TT_BEAM_MAX];
    __shared__ int s_as[TT_BEAM_MAX];  // the beam whose log-sum-exp counts; -1: a finished one
    const int b = blockIdx.x;
    const long long row0 = (long long)b * K;
    for (int i = tid; i < N * P; i += BM_THREADS) s_in[i] = keys[row0 * P * kk + i];
    for (int j = warp; j < K; j += BM_THREADS / 32) {
        const bool over = done && done[row0 + j] != 0;
        double l = 0.0;
        if (!over) {
            float R, s;
            join_parts(parts + (row0 + j) * P, P, LOG2E, R, s);
            l = lse_of(R, s, 1.0f);
        }
        if (lane == 0) {
            s_sc[j] = scores[row0 + j];
            s_lse[j] = l;
            s_as[j] = over ? -1 : j;
            if (l != l || l == INFINITY) atomicOr(&flags[FLAG_NONFINITE], 1);
        }
    }
    __syncthreads();
    if (P > 1) {
        for (int j = warp; j < K; j += BM_THREADS / 32)
            if (s_as[j] >= 0)  // a finished beam's lists were not made
                join_lists(s_in + j * P * kk, P * kk, kk, s_key[warp],
                           [&](int r, unsigned long long key) { s_j[j * kk + r] = key; });
        __syncthreads();
    }
    if (tid > 0 && tid < K && s_as[tid] >= 0) {
        for (int j = 0; j < tid; j++) {
            if (s_sc[j] != s_sc[tid] || s_as[j] < 0 || !(fabs(s_lse[j] - s_lse[tid]) <= LSE_EPS)) continue;
            int same = 0;
            while (same < kk && s_j[j * kk + same] == s_j[tid * kk + same]) same++;
            if (same == kk) {
                s_as[tid] = j;  // the first such: it stands for itself
                break;
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < N; i += BM_THREADS) {
        const int j = i / kk, r = i % kk;
        const float s = s_sc[j];
        double c = -INFINITY;
        int v = r;
        if (s_as[j] < 0) {
            if (isfinite(s)) {
                v = r == 0 ? eos : (r - 1 < eos ? r - 1 : r);
                if (r == 0) c = (double)s;
            }
        } else {
            const double l = s_lse[s_as[j]];
            if (isfinite(l) && isfinite(s)) {
                v = key_col(s_j[i]);
                c = (double)s + ((double)head::value_of((uint32_t)(s_j[i] >> 32)) - l);
            }
        }
        s_s[i] = order_of(c != c ? -INFINITY : c);
        s_f[i] = j * V + v;
    }
    // everything of the inputs is read before an output is written: they may be the same arrays
    uint32_t over_mask = 0;
    if (done)
        for (int j = 0; j < K; j++) over_mask |= (s_as[j] < 0 ? 1u : 0u) << j;
    __syncthreads();
    // a candidate's rank, by four lanes
    for (int i0 = 0; i0 < N; i0 += BM_THREADS / 4) {
        const int i = i0 + tid / 4;
        const unsigned long long c = i < N ? s_s[i] : 0ull;
        const int f = i < N ? s_f[i] : 0;
        int rank = 0;
        if (i < N)
            for (int o = tid & 3; o < N; o += 4) rank += s_s[o] > c || (s_s[o] == c && s_f[o] < f);
        rank += __shfl_xor_sync(0xffffffffu, rank, 1);
        rank += __shfl_xor_sync(0xffffffffu, rank, 2);
        if ((tid & 3) || i >= N || rank >= n) continue;
        const int j = f / V, v = f % V;
        const long long at = (long long)b * n + rank;
        parent[at] = j;
        token[at] = v;
        out_scores[at] = (float)value_of(c);
        if (out_done) out_done[at] = ((over_mask >> j) & 1u) || v == eos;
        if (tok_hist) {
            tok_hist[at * ld_hist + *pos_dev] = v;
            par_hist[at * ld_hist + *pos_dev] = j;
        }
    }
}

// Slot j of sequence b takes the bytes of slot parents[b, j].  A thread owns
// one unit (1 to 16 bytes) of the row across all K slots: it reads every
// moved slot's source before it writes any slot, so the move is in place
// whatever the parents are (cycles, several children of one parent).  Blocks
// whose sequence moves nothing end at once.  The traffic is the distinct
// sources in and the moved slots out; the 124M model's cache at 500 positions,
// B = 8, K = 4 (737 MB): 116 to 123 us, 88 to 94% of the measured copy rate;
// 4.4 GB of the 350M model's in fp32: 699 to 790 us, 82 to 93%.
template <typename U, int KM>
__global__ void __launch_bounds__(256)
k_beam_reorder(char* state, const int32_t* __restrict__ parents, int B, int K, long long row_bytes, long long first,
               long long count, const int* __restrict__ pos_dev, long long pos_bytes, long long blocks_per_row,
               int* flags) {
    pdl_enter();
    __shared__ int s_p[KM];
    __shared__ int s_any;
    const long long nb = blockIdx.x / blocks_per_row, blk = blockIdx.x % blocks_per_row;
    if (pos_dev) count = (long long)*pos_dev * pos_bytes - first;
    const long long u = (blk * 256 + threadIdx.x) * (long long)sizeof(U);
    if (threadIdx.x == 0) s_any = 0;
    __syncthreads();
    if (threadIdx.x < KM) {
        int p = threadIdx.x;
        if (p < K) {
            p = parents[(nb % B) * K + threadIdx.x];
            if (p < 0 || p >= K) {
                atomicOr(&flags[FLAG_BAD_TOKEN], 1);
                p = threadIdx.x;
            }
        }
        s_p[threadIdx.x] = p;
        if (p != (int)threadIdx.x) s_any = 1;
    }
    __syncthreads();
    if (!s_any || u >= count) return;
    char* base = state + nb * K * row_bytes + first + u;
    U v[KM];
#pragma unroll
    for (int j = 0; j < KM; j++)
        if (s_p[j] != j) v[j] = *reinterpret_cast<const U*>(base + s_p[j] * row_bytes);
#pragma unroll
    for (int j = 0; j < KM; j++)
        if (s_p[j] != j) *reinterpret_cast<U*>(base + j * row_bytes) = v[j];
}

// cache[b K + j][t][0 : 2C] = qkv[b T + t][C : 3C] for every beam j
template <typename T>
__global__ void k_kv_fill_beams(const T* __restrict__ qkv, T* __restrict__ cache, int B, int K, int Tn, int C,
                                int maxT) {
    const long long n = (long long)B * Tn * 2 * C;
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        const int c = (int)(i % (2 * C));
        const long long r = i / (2 * C);
        const int t = (int)(r % Tn), b = (int)(r / Tn);
        const T v = qkv[r * 3 * C + C + c];
        for (int j = 0; j < K; j++) cache[(((long long)b * K + j) * maxT + t) * 2 * C + c] = v;
    }
}

// out[b, k, 0 : Tp] = prompt[b], then the tokens of hypothesis k of the last
// step, found from its end: at position t slot j held tok[j][t], whose parent
// slot at t - 1 is par[j][t].
__global__ void k_beam_walk(const int32_t* __restrict__ prompt, const int32_t* __restrict__ tok,
                            const int32_t* __restrict__ par, int32_t* __restrict__ out, int R, int K, int Tp, int T) {
    const int r = blockIdx.x * blockDim.x + threadIdx.x;
    if (r >= R) return;
    const int b = r / K;
    int j = r % K;
    for (int t = T - 1; t >= Tp; t--) {
        const long long at = ((long long)b * K + j) * T + t;
        out[(long long)r * T + t] = tok[at];
        j = par[at];
    }
    for (int t = 0; t < Tp; t++) out[(long long)r * T + t] = prompt[(long long)b * Tp + t];
}

template <typename U>
bool reorder(const Launch& L, void* state, const int32_t* parents, int N, int B, int K, long long row_bytes,
             long long first, long long count, const int* pos_dev, long long pos_bytes) {
    const long long per = ((count + (long long)sizeof(U) - 1) / (long long)sizeof(U) + 255) / 256;
    const long long grid = per * N * B;
    if (grid > 0x7fffffffLL) return false;
    L.count();
#define RO(KM_)                                                                                                  \
    launch_k(L, k_beam_reorder<U, KM_>, dim3((unsigned)grid), dim3(256), 0, (char*)state, parents, B, K, row_bytes, \
             first, count, pos_dev, pos_bytes, per, L.flags)
    if (K <= 4) RO(4);
    else if (K <= 8) RO(8);
    else if (K <= 16) RO(16);
    else RO(32);
#undef RO
    return true;
}

}  // namespace

size_t beam_select_scratch_bytes(tt_dtype dtype, int B, int K, int V, int n) {
    const int kk = std::min(n, V);
    return (size_t)B * K * top_parts(dtype, B * K, V, kk, BM_ENTRIES / K, TOP_TASKS) * 8 * ((size_t)kk + 1);
}

bool launch_beam_select(const Launch& L, tt_dtype dtype, const void* z, long long ld, const float* scores,
                        const int32_t* done, int32_t* parent, int32_t* token, float* out_scores, int32_t* out_done,
                        int B, int K, int V, int n, int eos, void* scratch, int32_t* tok_hist, int32_t* par_hist,
                        int ld_hist, const int* pos_dev) {
    if (L.dry) return true;
    const int R = B * K, kk = std::min(n, V), P = top_parts(dtype, R, V, kk, BM_ENTRIES / K, TOP_TASKS), N = K * kk;
    const size_t smem = (size_t)(P > 1 ? N * P : 0) * 8 + (size_t)N * (8 + 8 + 4);
    static PerDevice attr;
    if (!attr.once([] {
            return cudaFuncSetAttribute(k_beam_merge, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        BM_ENTRIES * 8 + 2 * TT_BEAM_MAX * TT_BEAM_MAX * 20) == cudaSuccess;
        }))
        return false;
    auto* keys = (unsigned long long*)scratch;
    float2* parts = (float2*)(keys + (size_t)R * P * kk);
    if (!launch_top_parts(L, dtype, z, ld, R, V, kk, P, keys, parts, done)) return false;
    L.count();
    launch_k(L, k_beam_merge, dim3(B), dim3(BM_THREADS), smem, keys, parts, scores, done, K, P, V, kk, n, eos, parent,
             token, out_scores, out_done, tok_hist, par_hist, ld_hist, pos_dev, L.flags);
    return true;
}

bool launch_beam_reorder(const Launch& L, void* state, const int32_t* parents, int N, int B, int K,
                         long long row_bytes, long long first, long long count, const int* pos_dev,
                         long long pos_bytes) {
    if (L.dry || count <= 0) return true;
    const unsigned long long all =
        (unsigned long long)(uintptr_t)state | row_bytes | first | (pos_dev ? pos_bytes : count);
    if (all % 16 == 0) return reorder<uint4>(L, state, parents, N, B, K, row_bytes, first, count, pos_dev, pos_bytes);
    if (all % 4 == 0) return reorder<uint32_t>(L, state, parents, N, B, K, row_bytes, first, count, pos_dev, pos_bytes);
    return reorder<uint8_t>(L, state, parents, N, B, K, row_bytes, first, count, pos_dev, pos_bytes);
}

void launch_kv_fill_beams(const Launch& L, bool bf16, const void* qkv, void* cache, int B, int K, int Tn, int C,
                          int maxT) {
    if (L.dry) return;
    L.count();
    const long long n = (long long)B * Tn * 2 * C;
    const unsigned g = (unsigned)std::min<long long>((n + 255) / 256, 65535);
    if (bf16)
        k_kv_fill_beams<__nv_bfloat16><<<g, 256, 0, L.stream>>>((const __nv_bfloat16*)qkv, (__nv_bfloat16*)cache, B, K,
                                                                Tn, C, maxT);
    else
        k_kv_fill_beams<float><<<g, 256, 0, L.stream>>>((const float*)qkv, (float*)cache, B, K, Tn, C, maxT);
}

void launch_beam_walk(const Launch& L, const int32_t* prompt, const int32_t* tok, const int32_t* par, int32_t* out,
                      int B, int K, int Tp, int T) {
    if (L.dry) return;
    L.count();
    k_beam_walk<<<(B * K + 63) / 64, 64, 0, L.stream>>>(prompt, tok, par, out, B * K, K, Tp, T);
}

}  // namespace tt
