// head.cu -- operators on the LM head's logits that deal in lists of columns:
//
//   k_top_rows      per row the k largest logits (ties: the lowest column) and
//                   the log-sum-exp
//   k_distill       distillation from a teacher's top logits: loss and
//                   gradient of a row
//   k_row_mean      the mean of the row losses (fixed order)
//
// Both row kernels read a row of V logits from memory once, in the storage
// type, and hold it on chip (head_row.cuh); sums, statistics and losses are
// fp32.
#include "head_row.cuh"

#include <algorithm>

namespace tt {
namespace {

using namespace head;

constexpr int LIST_MAX = TT_TOP_MAX;
constexpr int LIST_PER_LANE = LIST_MAX / 32;
constexpr int CS_MAX = 8;      // CTAs of a cluster (the portable limit)
constexpr int CAND_MAX = 512;  // candidates of a row's (or slice's) list, and granules that hold them
constexpr int THR_MAX = 256;   // thread maxima that a threshold is chosen from

constexpr int LIST_CTA = 64;  // threads of a CTA that look after the list

__host__ __device__ constexpr int cta_threads(int NT) { return NT == 32 ? 256 : NT; }
__host__ __device__ constexpr int cta_per_sm(int NT) { return NT == 32 ? 3 : 2; }
__host__ __device__ constexpr int cta_groups(int NT) { return NT == 32 ? 8 : 1; }
__host__ __device__ constexpr int align16(int n) { return (n + 15) & ~15; }

// ------------------------------------------------------------ top logits
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
// bits of order_of that tell two values of a storage type apart
template <typename T> struct OrderBits { static constexpr int N = 32; };
template <> struct OrderBits<__nv_bfloat16> { static constexpr int N = 16; };
template <> struct OrderBits<__half> { static constexpr int N = 19; };  // sign, 8 exponent bits of fp32, 10 of mantissa

struct TopArgs {
    float* vals;
    int32_t* idx;
    float* lse;
    double* lse64;
    const int32_t* skip;
    long long ld;
    int M, V, k, Gs, cs, nbuf;
    float inv_tau;
};

// shared memory of a group, in bytes from its start
struct TopLayout {
    int cand, thr, gl, part, red, lists, x, cnt, total;
    __host__ __device__ TopLayout(int nt, int Gs, int nbuf, int k, bool cl) {
        int at = nbuf * Gs * 16;
        cand = at; at += (nt > 32 ? CAND_MAX : LIST_MAX) * 8;  // a warp's candidates are exact ones
        thr = at; at += nt > 32 ? 4 * THR_MAX + 16 : 0;
        gl = at; at += nt > 32 ? 4 * CAND_MAX : 0;
        part = at; at += nt > 32 ? 256 : 0;
        red = at; at += nt > 32 ? 256 : 0;
        lists = at; at += cl ? align16(2 * CS_MAX * k * 8) : 0;
        x = at; at += cl ? 2 * CS_MAX * 8 : 0;
        cnt = at; at += 16;
        total = at;
    }
};

// sum of c over the group; `turn` alternates between two rows of s_red, so
// that one barrier a call is enough
template <int NT> __device__ __forceinline__ int group_count(int c, int* s_red, int& turn) {
    c = __reduce_add_sync(0xffffffffu, c);
    if (NT == 32) return c;
    const int lane = threadIdx.x & 31;
    int* r = s_red + (turn & 1) * 32;
    turn++;
    if (lane == 0) r[threadIdx.x >> 5] = c;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < NT / 32 ? r[lane] : 0);
}

// where a thread's granules are read from: the on-chip copy, or memory
struct OnChip {
    const char* buf;
    template <typename T> __device__ __forceinline__ uint4 get(const Slice<T>&, int i, int) const {
        return reinterpret_cast<const uint4*>(buf)[i];
    }
};
struct InMemory {
    template <typename T> __device__ __forceinline__ uint4 get(const Slice<T>& s, int i, int V) const {
        return s.inner(i) ? reinterpret_cast<const uint4*>(s.base)[i]
                          : edge_granule(reinterpret_cast<const T*>(s.base) - s.col(0), s.col(i), V);
    }
};

// f(value, column) for every element of the thread's granules
template <typename T, int NT, typename S, typename F>
__device__ __forceinline__ void each_element(const Slice<T>& s, const S& src, int V, int tid, F&& f) {
    for (int g = tid; g < s.n; g += NT) {
        const uint4 u = src.get(s, g, V);
        f2 e[Elem<T>::EPG / 2];
        Elem<T>::unpack(u, e);
        const int c0 = s.col(g);
#pragma unroll
        for (int i = 0; i < Elem<T>::EPG / 2; i++) {
            float a, b;
            unpk(e[i], a, b);
            if (c0 + 2 * i >= 0 && c0 + 2 * i < V) f(a, c0 + 2 * i);
            if (c0 + 2 * i + 1 >= 0 && c0 + 2 * i + 1 < V) f(b, c0 + 2 * i + 1);
        }
    }
}

// The kk first elements of the slice in list order, exactly, as candidates:
// the kk-th largest value is found bit by bit by counting, then, where equal
// values are more than are needed, the last column that is taken.  Used where
// the threads' maxima say too little: rows of a warp, rows with most columns
// masked, rows of few different values.
template <typename T, int NT, typename S>
__device__ __noinline__ void exact_candidates(const Slice<T>& s, const S& buf, int V, int kk, int n_el,
                                 unsigned long long* s_cand, int* s_cnt, int* s_red, int tid) {
    int turn = 0;
    if (tid == 0) *s_cnt = 0;
    group_sync<NT>();
    if (n_el <= (NT == 32 ? LIST_MAX : CAND_MAX / 2)) {
        // few enough to rank them all
        each_element<T, NT>(s, buf, V, tid, [&](float v, int c) { s_cand[atomicAdd(s_cnt, 1)] = top_key(v, c); });
        group_sync<NT>();
        return;
    }
    constexpr int LOW = 32 - OrderBits<T>::N;
    uint32_t t = 0;
    for (int bit = 31; bit >= LOW; bit--) {
        const uint32_t cand = t | (1u << bit);
        int c = 0;
        each_element<T, NT>(s, buf, V, tid, [&](float v, int) { c += order_of(v) >= cand; });
        if (group_count<NT>(c, s_red, turn) >= kk) t = cand;
    }
    const uint32_t above = t + (1u << LOW);  // no value's order is so large that this wraps
    int c = 0, e = 0;
    each_element<T, NT>(s, buf, V, tid, [&](float v, int) {
        const uint32_t o = order_of(v);
        c += o >= above;
        e += o >= t && o < above;
    });
    const int need = kk - group_count<NT>(c, s_red, turn);
    int last = V;  // equal values are taken up to this column
    if (group_count<NT>(e, s_red, turn) > need) {
        last = 0;
        for (int bit = 20; bit >= 0; bit--) {  // V < 2^20
            const int x = last | (1 << bit);
            int n = 0;
            each_element<T, NT>(s, buf, V, tid, [&](float v, int col) {
                const uint32_t o = order_of(v);
                n += o >= t && o < above && col < x;
            });
            if (group_count<NT>(n, s_red, turn) < need) last = x;
        }
    }
    each_element<T, NT>(s, buf, V, tid, [&](float v, int col) {
        const uint32_t o = order_of(v);
        if (o >= above || (o >= t && col <= last)) s_cand[atomicAdd(s_cnt, 1)] = top_key(v, col);
    });
    group_sync<NT>();
}

// out(rank, key) for the kk first of cnt candidates in list order; four lanes count for a candidate
template <int NT, typename F>
__device__ __forceinline__ void ranks(const unsigned long long* s_cand, int cnt, int kk, int tid, F&& out) {
    for (int i0 = 0; i0 < cnt; i0 += NT / 4) {
        const int i = i0 + tid / 4;
        if (__all_sync(0xffffffffu, i >= cnt)) break;
        const unsigned long long key = i < cnt ? s_cand[i] : ~0ull;
        int r = 0;
#pragma unroll 4
        for (int j = tid & 3; j < cnt; j += 4) r += s_cand[j] > key;
        r += __shfl_xor_sync(0xffffffffu, r, 1);
        r += __shfl_xor_sync(0xffffffffu, r, 2);
        if ((tid & 3) == 0 && i < cnt && r < kk) out(r, key);
    }
}

// A row's list in four stages:
//   1. one pass over the granules: each thread's largest value and its sum of
//      exponentials;
//   2. a threshold: each of the fw warps that have work in every lane gives its
//      Q largest thread maxima, Q = ceil(k / fw) + 2, and the k-th largest of
//      these fw Q values is the threshold.  At least k elements are at or
//      above it;
//   3. threads whose largest value is at or above it name their granules that
//      are, and all threads look through those for the elements: the
//      candidates, on unordered data a few more than k;
//   4. each candidate's rank among them by counting.
// With more than CAND_MAX candidates, or too few threads for a threshold, the
// candidates are found exactly instead.  Clusters: each CTA lists its slice
// and sends the list to CTA 0, which ranks every entry by binary searches in
// the other lists.
template <typename T, int NT, bool CL>
__global__ void __launch_bounds__(cta_threads(NT), cta_per_sm(NT))
k_top_rows(const T* __restrict__ z, const TopArgs a) {
    pdl_enter();
    extern __shared__ __align__(16) char smem[];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int lane = threadIdx.x & 31, warp = tid >> 5;
    const TopLayout lay(NT, a.Gs, a.nbuf, a.k, CL);
    char* sm = smem + (NT == 32 ? threadIdx.x >> 5 : 0) * lay.total;
    auto* s_cand = reinterpret_cast<unsigned long long*>(sm + lay.cand);
    uint32_t* s_thr = reinterpret_cast<uint32_t*>(sm + lay.thr);
    int* s_gl = reinterpret_cast<int*>(sm + lay.gl);
    float2* s_part = reinterpret_cast<float2*>(sm + lay.part);
    int* s_red = reinterpret_cast<int*>(sm + lay.red);
    auto* s_lists = reinterpret_cast<unsigned long long*>(sm + lay.lists);  // [2][cs][k]
    float2* s_x = reinterpret_cast<float2*>(sm + lay.x);                    // [2][cs]
    int* s_cnt = reinterpret_cast<int*>(sm + lay.cnt);
    const int rank = CL ? (int)cluster_rank() : 0, cs = CL ? a.cs : 1;
    const long long first = CL ? blockIdx.x / cs : blockIdx.x * (long long)cta_groups(NT) + (NT == 32 ? threadIdx.x >> 5 : 0);
    const long long stride = CL ? gridDim.x / cs : gridDim.x * (long long)cta_groups(NT);
    const bool want = a.lse || a.lse64;
    const float ct = LOG2E * a.inv_tau, lift = 20.0f / fmaxf(1.0f, a.inv_tau);
    const int k = a.k, V = a.V;
    using E = Elem<T>;
    auto slice = [&](long long r) { return Slice<T>(z, r, a.ld, V, rank, a.Gs); };
    auto here = [&](long long r) { return r < a.M && !(a.skip && a.skip[r]); };

    for (int i = 0; i < a.nbuf; i++) {
        const long long r = first + i * stride;
        if (here(r)) fill<T, NT>(slice(r), sm + i * a.Gs * 16, tid);
        cp_commit();
    }
    T edge = Elem<T>::put(0.0f);
    if (here(first)) edge_store(slice(first), sm, edge_load(slice(first), V, tid), tid);
    if (here(first + stride)) edge = edge_load(slice(first + stride), V, tid);
    if (tid == 0) s_cnt[0] = s_cnt[1] = 0;  // candidates, granules
    if (CL) cluster_sync();  // the others run: their shared memory may be written

    int it = 0;
    for (long long row = first; row < a.M; row += stride, it++) {
        const int par = it & 1;
        char* buf = sm + (a.nbuf == 2 ? par : 0) * a.Gs * 16;
        const Slice<T> s = slice(row);
        cp_wait(a.nbuf);
        group_sync<NT>();
        const bool run = here(row);
        const long long next = row + a.nbuf * stride;
        if (run) {
            // stage 1
            float tmax, R, sum, none;
            if (want) {
                sum_pass<T, NT, true, false>(s, buf, tid, ct, ct, lift, tmax, R, sum, none);
                merge(R, sum, ct);
            } else {
                sum_pass<T, NT, false, false>(s, buf, tid, ct, ct, lift, tmax, R, sum, none);
            }
            // stage 2
            const int n_slots = s.n;
            const int n_el = max(0, min(V, s.col(s.n)) - max(0, s.col(0)));
            const int kk = min(k, n_el);
            const int fw = NT == 32 ? 0 : min(NT, n_slots) / 32;
            const int Q = fw ? min(32, (k + fw - 1) / fw + 2) : 0;
            bool exact = fw * Q < k || fw * Q > THR_MAX;
            int cnt = 0;
            if (NT > 32) {
                if (!exact && warp < fw) {
                    uint32_t cur = order_of(tmax), mine = 0;
                    for (int i = 0; i < Q; i++) {
                        const uint32_t m = __reduce_max_sync(0xffffffffu, cur);
                        if (lane == i) mine = m;
                        if (lane == __ffs(__ballot_sync(0xffffffffu, cur == m)) - 1) cur = 0;
                    }
                    if (lane < Q) s_thr[warp * Q + lane] = mine;
                }
                if (lane == 0) s_part[warp] = make_float2(R, sum);
                __syncthreads();
                if (!exact) {
                    // the k-th largest of the fw Q values, by one warp bit by bit
                    // from the first bit that differs
                    if (warp == 0) {
                        const int nv = fw * Q;
                        uint32_t v[THR_MAX / 32], hi = 0, lo = ~0u;
#pragma unroll
                        for (int j = 0; j < THR_MAX / 32; j++) {
                            v[j] = 0;
                            if (j * 32 + lane < nv) {
                                v[j] = s_thr[j * 32 + lane];
                                lo = min(lo, v[j]);
                                hi = max(hi, v[j]);
                            }
                        }
                        hi = __reduce_max_sync(0xffffffffu, hi);
                        lo = __reduce_min_sync(0xffffffffu, lo);
                        int bit = 31 - __clz(hi ^ lo);  // -1: all are equal
                        uint32_t t = bit < 0 ? hi : hi & ~((2u << bit) - 1u);
                        for (; bit >= 32 - OrderBits<T>::N; bit--) {
                            const uint32_t cand = t | (1u << bit);
                            int c = 0;
#pragma unroll
                            for (int j = 0; j < THR_MAX / 32; j++)
                                if (j * 32 < nv) c += v[j] >= cand;
                            c = __reduce_add_sync(0xffffffffu, c);
                            if (c >= k) t = cand;
                            if (c == k) break;
                        }
                        if (lane == 0) s_thr[THR_MAX] = t;
                    }
                    __syncthreads();
                    // stage 3
                    const uint32_t thr = s_thr[THR_MAX];
                    if (order_of(tmax) >= thr) {
                        const typename E::Max thr2 = E::to_max(fmaxf(value_of(thr), -INFINITY));
#pragma unroll 2
                        for (int i = tid; i < n_slots; i += NT)
                            if (E::at_least(E::gmax(reinterpret_cast<const uint4*>(buf)[i]), thr2)) {
                                const int p = atomicAdd(s_cnt + 1, 1);
                                if (p < CAND_MAX) s_gl[p] = i;
                            }
                    }
                    __syncthreads();
                    const int ng = s_cnt[1];
                    exact = ng > CAND_MAX;
                    if (!exact) {
                        for (int i = tid; i < ng * E::EPG; i += NT) {
                            const int slot = s_gl[i / E::EPG], e = i % E::EPG;
                            const float w = E::get(reinterpret_cast<const T*>(buf + slot * 16) + e);
                            const int c = s.col(slot) + e;
                            if (order_of(w) >= thr && c >= 0 && c < V) {
                                const int p = atomicAdd(s_cnt, 1);
                                if (p < CAND_MAX) s_cand[p] = top_key(w, c);
                            }
                        }
                        __syncthreads();
                        cnt = s_cnt[0];
                        exact = cnt > CAND_MAX;
                        if (exact) __syncthreads();  // every thread has read the count
                    }
                }
            }
            if (exact) {
                exact_candidates<T, NT>(s, OnChip{buf}, V, kk, n_el, s_cand, s_cnt, s_red, tid);
                cnt = *s_cnt;
            }
            if (here(next)) fill<T, NT>(slice(next), buf, tid);
            cp_commit();
            // stage 4
            ranks<NT>(s_cand, cnt, kk, tid, [&](int r, unsigned long long key) {
                if (CL) {
                    st_remote(remote(s_lists + (par * cs + rank) * k + r, 0), key);
                } else {
                    a.vals[row * k + r] = value_of((uint32_t)(key >> 32));
                    a.idx[row * k + r] = key_col(key);
                }
            });
            if (CL)
                for (int r = kk + tid; r < k; r += NT) st_remote(remote(s_lists + (par * cs + rank) * k + r, 0), 0ull);
            if (want && warp == 0) {
                if (NT > 32) {
                    const float2 p = lane < NT / 32 ? s_part[lane] : make_float2(-INFINITY, 0.0f);
                    R = p.x;
                    sum = p.y;
                    merge(R, sum, ct);
                }
                if (CL && lane == 0) {
                    const uint32_t at = remote(s_x + par * cs + rank, 0);
                    st_remote(at, R);
                    st_remote(at + 4, sum);
                }
            }
            if (CL) {
                cluster_sync();
                if (rank == 0) {
                    const unsigned long long* l = s_lists + par * cs * k;
                    for (int i = tid; i < cs * k; i += NT) {
                        const unsigned long long key = l[i];
                        int r = i % k;
                        if (key == 0) continue;
                        for (int o = 0; o < cs; o++) {
                            if (o == i / k) continue;
                            int lo = 0, hi = k;  // entries of list o above key
                            while (lo < hi) {
                                const int mid = (lo + hi) >> 1;
                                if (l[o * k + mid] > key) lo = mid + 1;
                                else hi = mid;
                            }
                            r += lo;
                        }
                        if (r < k) {
                            a.vals[row * k + r] = value_of((uint32_t)(key >> 32));
                            a.idx[row * k + r] = key_col(key);
                        }
                    }
                    if (want && warp == 0) {
                        const float2 p = lane < cs ? s_x[par * cs + lane] : make_float2(-INFINITY, 0.0f);
                        R = p.x;
                        sum = p.y;
                        merge<CS_MAX>(R, sum, ct);
                    }
                }
            }
            if (want && tid == 0 && rank == 0) {
                // a row of -inf and a row with +inf have that as their value, unless a NaN is there too
                const bool flat = sum == sum && (R == -INFINITY || R == INFINITY);
                if (a.lse) a.lse[row] = flat ? R : R * a.inv_tau + logf(sum);
                if (a.lse64) a.lse64[row] = flat ? (double)R : (double)R * (double)a.inv_tau + log((double)sum);
            }
        } else {
            if (here(next)) fill<T, NT>(slice(next), buf, tid);
            cp_commit();
            if (CL) cluster_sync();
        }
        group_sync<NT>();
        if (tid == 0) s_cnt[0] = s_cnt[1] = 0;
        const long long n1 = row + stride, n2 = n1 + stride;
        if (tid < 16) {
            if (here(n1)) edge_store(slice(n1), sm + (a.nbuf == 2 ? par ^ 1 : 0) * a.Gs * 16, edge, tid);
            if (here(n2)) edge = edge_load(slice(n2), V, tid);
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------ top logits of many rows
// A warp a row, for calls with more rows than the SMs hold warps: the row
// streams through a ring of the warp's own, without a barrier, and what stays
// of it is the largest value of every block of UB granules of a lane.  The
// k-th largest of those is the threshold; the few blocks at or above it (k,
// and those that tie) are read again from memory, and their elements at or
// above it are ranked.  A lane's four granules of a stage are neighbours in
// memory (64 bytes; in shared memory they are permuted so that eight lanes'
// reads fall into different banks): reading 64 blocks again then is 4% of a
// row of 50257 16-bit logits, where blocks of four granules 512 bytes apart
// cost 26% more DRAM traffic.  A whole row on chip (k_top_rows) needs no
// second read but waits at its barriers: 940 us for 32768 such rows.
// A row with more candidates than there is room for (ties, masks) is gone
// through bit by bit from memory.
constexpr int TS_WARPS = 8;                 // of a CTA
constexpr int TS_BLOCKS = 64;               // most blocks of a lane
constexpr int TS_U = 4;                     // granules of a lane in a stage of the ring
constexpr int TS_RING = 2 * TS_U * 32 * 16;  // two stages

// candidates, and blocks that hold them: 24 warps of an SM have room for their
// rings with the smaller number, 20 with the larger
__host__ __device__ constexpr int stream_cand(int k) { return k <= 64 ? 160 : 256; }
__host__ __device__ constexpr int stream_warp_smem(int words, int k) {
    return TS_RING + words * 128 + stream_cand(k) * (8 + 2) + 16;
}

// A lane's block maxima, as the counting below reads them: pairs for the 16-bit types.
template <typename T> struct Blocks {
    static constexpr int PER = sizeof(T) == 2 ? 2 : 1;  // blocks of a word
    uint32_t* w;                                        // [word][lane]
    __device__ __forceinline__ void put(int b, int lane, T v) {
        reinterpret_cast<T*>(w + ((unsigned)b / PER) * 32 + lane)[(unsigned)b % PER] = v;
    }
    // how many of the lane's n words' blocks are at least t
    __device__ __forceinline__ int count(int n, int lane, T t) const;
    // blocks b (even) and b + 1
    __device__ __forceinline__ void put2(int b, int lane, typename Elem<T>::Max x, typename Elem<T>::Max y) {
        if constexpr (PER == 2) {
            *reinterpret_cast<typename Elem<T>::Max*>(w + b * 16 + lane) = Elem<T>::fold(x, y);
        } else {
            put(b, lane, x);
            put(b + 1, lane, y);
        }
    }
    __device__ __forceinline__ typename Elem<T>::Max word(int i, int lane) const {
        return *reinterpret_cast<const typename Elem<T>::Max*>(w + i * 32 + lane);
    }
};
template <> __device__ __forceinline__ int Blocks<float>::count(int n, int lane, float t) const {
    int c = 0;
#pragma unroll 4
    for (int i = 0; i < n; i++) c += __uint_as_float(w[i * 32 + lane]) >= t;
    return c;
}
template <> __device__ __forceinline__ int Blocks<__nv_bfloat16>::count(int n, int lane, __nv_bfloat16 t) const {
    const __nv_bfloat162 t2 = __halves2bfloat162(t, t);
    __nv_bfloat162 c = __floats2bfloat162_rn(0.0f, 0.0f);  // whole numbers up to 32: exact
#pragma unroll 4
    for (int i = 0; i < n; i++) c = __hadd2(c, __hge2(*reinterpret_cast<const __nv_bfloat162*>(w + i * 32 + lane), t2));
    return (int)(__low2float(c) + __high2float(c));
}
template <> __device__ __forceinline__ int Blocks<__half>::count(int n, int lane, __half t) const {
    const __half2 t2 = __halves2half2(t, t);
    __half2 c = __floats2half2_rn(0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < n; i++) c = __hadd2(c, __hge2(*reinterpret_cast<const __half2*>(w + i * 32 + lane), t2));
    return (int)(__low2float(c) + __high2float(c));
}

// a storage type's values in order as whole numbers
template <typename T> struct Ordered {
    static constexpr int N = 8 * sizeof(T);
    static __device__ __forceinline__ uint32_t of(T v) {
        uint32_t u = 0;
        memcpy(&u, &v, sizeof(T));
        return (u >> (N - 1)) & 1 ? ~u & (0xFFFFFFFFu >> (32 - N)) : u | (1u << (N - 1));
    }
    static __device__ __forceinline__ T value(uint32_t o) {
        const uint32_t u = (o >> (N - 1)) & 1 ? o ^ (1u << (N - 1)) : ~o;
        T v;
        memcpy(&v, &u, sizeof(T));
        return v;
    }
};

// element l of N pairs
template <int N> __device__ __forceinline__ float pick(const f2 (&e)[N], int l) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
        float x, y;
        unpk(e[i], x, y);
        v = l == 2 * i ? x : l == 2 * i + 1 ? y : v;
    }
    return v;
}

template <typename T>
__global__ void __launch_bounds__(TS_WARPS * 32, 3)
k_top_stream(const T* __restrict__ z, const TopArgs a, int ub_log, int words) {
    pdl_enter();
    extern __shared__ __align__(16) char smem[];
    using E = Elem<T>;
    constexpr int PER = Blocks<T>::PER;
    const int lane = threadIdx.x & 31;
    const int TS_CAND = stream_cand(a.k);
    char* sm = smem + (threadIdx.x >> 5) * stream_warp_smem(words, a.k);
    Blocks<T> blocks{reinterpret_cast<uint32_t*>(sm + TS_RING)};
    auto* s_cand = reinterpret_cast<unsigned long long*>(sm + TS_RING + words * 128);
    auto* s_hit = reinterpret_cast<uint16_t*>(s_cand + TS_CAND);
    int* s_cnt = reinterpret_cast<int*>(s_hit + TS_CAND);
    const long long first = blockIdx.x * (long long)TS_WARPS + (threadIdx.x >> 5), stride = gridDim.x * (long long)TS_WARPS;
    const bool want = a.lse || a.lse64;
    const float ct = LOG2E * a.inv_tau, lift = 20.0f / fmaxf(1.0f, a.inv_tau);
    const int k = a.k, V = a.V;
    auto slice = [&](long long r) { return Slice<T>(z, r, a.ld, V, 0, a.Gs); };
    // Granule g of a stage (128 of them) is in slot (g & ~7) | (g ^ (g >> 3 & 3)) & 7:
    // a lane copies granules lane + 32 j and reads 4 lane + j.
    const uint32_t ring_at =
        (uint32_t)__cvta_generic_to_shared(sm) + ((lane & ~7) | ((lane ^ ((lane >> 3) & 3)) & 7)) * 16;
    const uint4* own[TS_U];
#pragma unroll
    for (int j = 0; j < TS_U; j++) own[j] = reinterpret_cast<const uint4*>(sm) + 4 * lane + (j ^ ((lane >> 1) & 3));
    auto whole = [&](const Slice<T>& s, int st) { return (st > 0 || s.i0 == 0) && (st + 1) * 128 <= s.i1; };
    auto copy = [&](const Slice<T>& s, int st) {  // stage st of a row
        const char* g = s.base + (long long)(st * 128 + lane) * 16;
        const uint32_t b = ring_at + (st & 1) * 2048;
        if (whole(s, st)) {
            cp16<0>(b, g);
            cp16<512>(b, g);
            cp16<1024>(b, g);
            cp16<1536>(b, g);
        } else {
            const int i = st * 128 + lane;
#pragma unroll
            for (int j = 0; j < TS_U; j++)
                if (i + j * 32 >= s.i0 && i + j * 32 < s.i1) cp16<0>(b + j * 512, g + j * 512);
        }
        cp_commit();
    };
    // stages are counted in pairs, so that a row always starts in the ring's first half
    const int SX = (a.Gs + 127) / 128, S = (SX + 1) & ~1;
    const int ub = 1 << ub_log, nb = (4 * SX + ub - 1) >> ub_log, nw = words;
    for (long long row = first; row < a.M; row += stride) {
        const Slice<T> s = slice(row);
        const bool more = row + stride < a.M;
        const Slice<T> nx = slice(more ? row + stride : row);
        if (row == first) {
            copy(s, 0);
            copy(s, 1);
        }
        if (lane == 0) *s_cnt = 0;
        if (PER == 2 && nb % 2) blocks.put(nb, lane, E::put(-INFINITY));
        Sums<T, true, false> q(ct, ct, lift);
        typename E::Max bm = E::to_max(-INFINITY);
        // two stages at a time: the usual form, where both and the two after
        // them are wholly inside the row, and the form that looks at every granule
        auto block = [&](int st, typename E::Max g4, const typename E::Max* g) {
            if (st >= SX) return;
            if (ub == 1) {
#pragma unroll
                for (int j = 0; j < TS_U; j++) blocks.put(st * 4 + j, lane, E::top(g[j]));
            } else {
                bm = E::max2(bm, g4);
                if (((st + 1) * 4 & (ub - 1)) == 0 || st == SX - 1) {
                    blocks.put((st * 4) >> ub_log, lane, E::top(bm));
                    bm = E::to_max(-INFINITY);
                }
            }
        };
        const int whole0 = s.i0 == 0 ? 0 : 2, whole1 = s.i1 / 128 - 4;  // st in [whole0, whole1]: the usual form
        for (int st = 0; st < S; st += 2) {
            if (st >= whole0 && st <= whole1) {
                typename E::Max g4[2];
                const char* src = s.base + (long long)((st + 2) * 128 + lane) * 16;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                    __syncwarp();
                    uint4 u[TS_U];
                    typename E::Max g[TS_U];
#pragma unroll
                    for (int j = 0; j < TS_U; j++) u[j] = own[j][h * 128];
#pragma unroll
                    for (int j = 0; j < TS_U; j++) g[j] = E::gmax(u[j]);
                    if (h == 0 && st == 0) q.start(want ? warp_max(E::value(g[0])) : -INFINITY);
                    g4[h] = E::max2(E::max2(g[0], g[1]), E::max2(g[2], g[3]));
                    if (want) q.look(g4[h]);
                    __syncwarp();  // the stage has been read
                    if (h == 0) {
                        cp16<0>(ring_at, src);
                        cp16<512>(ring_at, src);
                        cp16<1024>(ring_at, src);
                        cp16<1536>(ring_at, src);
                    } else {
                        cp16<2048>(ring_at, src);
                        cp16<2560>(ring_at, src);
                        cp16<3072>(ring_at, src);
                        cp16<3584>(ring_at, src);
                    }
                    cp_commit();
                    if (want) {
#pragma unroll
                        for (int j = 0; j < TS_U; j++) q.take(u[j]);
                    }
                    if (ub != 4) block(st + h, g4[h], g);
                }
                if (ub == 4) blocks.put2(st, lane, g4[0], g4[1]);
            } else {
#pragma unroll 1
                for (int h = 0; h < 2; h++) {
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                    __syncwarp();
                    uint4 u[TS_U];
                    typename E::Max g[TS_U];
#pragma unroll
                    for (int j = 0; j < TS_U; j++) {
                        const int i = (st + h) * 128 + 4 * lane + j;
                        if (i >= s.i0 && i < s.i1) u[j] = own[j][h * 128];
                        else if (i < s.n) u[j] = InMemory().get(s, i, V);
                        else u[j] = make_uint4(E::NINF, E::NINF, E::NINF, E::NINF);
                    }
#pragma unroll
                    for (int j = 0; j < TS_U; j++) g[j] = E::gmax(u[j]);
                    if (h == 0 && st == 0) q.start(want ? warp_max(E::value(g[0])) : -INFINITY);
                    const typename E::Max g4 = E::max2(E::max2(g[0], g[1]), E::max2(g[2], g[3]));
                    if (want) q.look(g4);
                    __syncwarp();
                    if (st + 2 < S) copy(s, st + 2 + h);
                    else if (more) copy(nx, h);
                    else cp_commit();
                    if (want) {
#pragma unroll
                        for (int j = 0; j < TS_U; j++) q.take(u[j]);
                    }
                    block(st + h, g4, g);
                }
            }
        }
        float tmax, sum, none;
        if (q.finish(tmax, sum, none) && want)
            each_element<T, 32>(s, InMemory(), V, lane, [&](float v, int) { q.take_far(v, sum, none); });
        float R = q.R;
        if (want) merge(R, sum, ct);

        // the threshold: the k-th largest of the blocks' maxima
        typename E::Max mx = E::to_max(-INFINITY), mn = E::to_max(INFINITY);
#pragma unroll 4
        for (int i = 0; i < nw; i++) {
            const typename E::Max v = blocks.word(i, lane);
            mx = E::max2(mx, v);
            mn = E::min2(mn, v);
        }
        uint32_t hi = Ordered<T>::of(E::top(mx)), low = Ordered<T>::of(E::bottom(mn));
        hi = __reduce_max_sync(0xffffffffu, hi);
        low = __reduce_min_sync(0xffffffffu, low);
        int bit = 31 - __clz(hi ^ low);
        uint32_t t = bit < 0 ? hi : hi & ~((2u << bit) - 1u);
        for (; bit >= 0; bit--) {
            const uint32_t cand = t | (1u << bit);
            const int c = __reduce_add_sync(0xffffffffu, blocks.count(nw, lane, Ordered<T>::value(cand)));
            if (c >= k) t = cand;
            if (c >= k && c <= k + 16) break;  // a few blocks more cost less than another bit
        }
        const T tv = Ordered<T>::value(t);
        const float thr = E::get(&tv);
        bool exact = !(thr > -INFINITY);  // or no number
        __syncwarp();
        if (!exact) {
            unsigned long long mine = 0;  // the lane's blocks at or above it
#pragma unroll 4
            for (int i = 0; i < nw; i++) {
                const typename E::Max v = blocks.word(i, lane);
#pragma unroll
                for (int j = 0; j < PER; j++)
                    if (E::get(reinterpret_cast<const T*>(&v) + j) >= thr) mine |= 1ull << (i * PER + j);
            }
            const int n_mine = __popcll(mine);
            int at = n_mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, at, o);
                if (lane >= o) at += x;
            }
            const int nh = __shfl_sync(0xffffffffu, at, 31);
            at -= n_mine;
            exact = nh > TS_CAND;
            if (!exact) {
                while (mine) {
                    s_hit[at++] = (uint16_t)((__ffsll(mine) - 1) * 32 + lane);
                    mine &= mine - 1;
                }
                __syncwarp();
                const int items = nh << ub_log;
#pragma unroll 1
                for (int i0 = 0; i0 < items; i0 += 32 * TS_U) {
                    uint4 u[TS_U];
                    int col[TS_U];
#pragma unroll
                    for (int j = 0; j < TS_U; j++) {
                        const int it = min(i0 + j * 32 + lane, items - 1);
                        const int h = s_hit[it >> ub_log], t = ub == 1 ? h >> 5 : ((h >> 5) << ub_log) + (it & (ub - 1));
                        const int slot = (t >> 2) * 128 + 4 * (h & 31) + (t & 3);
                        const bool on = slot < s.n && i0 + j * 32 + lane < items;
                        u[j] = on ? InMemory().get(s, slot, V) : make_uint4(E::NINF, E::NINF, E::NINF, E::NINF);
                        col[j] = s.col(slot);
                    }
#pragma unroll
                    for (int j = 0; j < TS_U; j++) {
                        f2 e[E::EPG / 2];
                        E::unpack(u[j], e);
                        uint32_t mask = 0;  // what lies outside the row is -inf: not at or above the threshold
#pragma unroll
                        for (int l = 0; l < E::EPG / 2; l++) {
                            float x, y;
                            unpk(e[l], x, y);
                            mask |= (x >= thr ? 1u << (2 * l) : 0u) | (y >= thr ? 2u << (2 * l) : 0u);
                        }
                        while (mask) {
                            const int l = __ffs(mask) - 1;
                            mask &= mask - 1;
                            const int p = atomicAdd(s_cnt, 1);
                            if (p < TS_CAND) s_cand[p] = top_key(pick(e, l), col[j] + l);
                        }
                    }
                }
                __syncwarp();
                exact = s_cnt[0] > TS_CAND;
                __syncwarp();
            }
        }
        if (exact) exact_candidates<T, 32>(s, InMemory(), V, k, V, s_cand, s_cnt, (int*)nullptr, lane);
        __syncwarp();
        ranks<32>(s_cand, s_cnt[0], k, lane, [&](int r, unsigned long long key) {
            a.vals[row * k + r] = value_of((uint32_t)(key >> 32));
            a.idx[row * k + r] = key_col(key);
        });
        if (want && lane == 0) {
            const bool flat = sum == sum && (R == -INFINITY || R == INFINITY);
            if (a.lse) a.lse[row] = flat ? R : R * a.inv_tau + logf(sum);
            if (a.lse64) a.lse64[row] = flat ? (double)R : (double)R * (double)a.inv_tau + log((double)sum);
        }
        __syncwarp();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------ distillation
// With q = softmax(z / tau), s = softmax(z), the list's probabilities p_j at
// columns i_j, W their sum (plus p_r, the teacher's mass outside the list,
// when it is known and the student has any there, q_r):
//   loss = alpha tau^2 (sum p_j (ln p_j - ln q_ij) + p_r (ln p_r - ln q_r)) + (1 - alpha) (lse(z) - z_y)
//   dz_i = g alpha tau (W q_i - p_i)            on the list
//        = g alpha tau q_i (W - p_r / q_r)      off it
//        + g (1 - alpha) (s_i - [i = y])
// One pass over the row's granules sums the exponentials, a second writes the
// gradient as if no column were listed, and the list's columns are then
// written over.  Where q_r is needed (t_lse) the listed logits are first
// replaced by -inf in the on-chip copy, so that q_r is summed without them and
// not as a difference; their own exponentials are added from the list.
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

__host__ __device__ constexpr int distill_threads(int NT) { return NT == 32 ? 256 : NT + LIST_CTA; }

// tau as a power that one softmax's terms are of the other's: 1 to 4, else 0
__device__ __forceinline__ int power_of(float tau) {
    return tau == 1.0f ? 1 : tau == 2.0f ? 2 : tau == 3.0f ? 3 : tau == 4.0f ? 4 : 0;
}

struct DistillLayout {
    int bits, ti, tv, yl, zl, zo, t, off, part, lw, ll, x, flag, total;
    __host__ __device__ DistillLayout(int nt, int Gs, int nbuf, int k, int epg, bool cl) {
        const int k4 = align16(4 * (k + 1));
        int at = nbuf * Gs * 16;
        bits = at; at += align16((Gs * epg + 31) / 32 * 4);
        ti = at; at += nbuf * k4;
        tv = at; at += nbuf * k4;
        yl = at; at += 16;      // [nbuf] targets, [nbuf] t_lse
        zl = at; at += 2 * k4;  // student logits of the list, and of the target
        zo = at; at += k4;      // those of this CTA's slice
        t = at; at += k4;       // t_j / tau
        off = at; at += k4;     // where this CTA holds the column, or -1
        part = at; at += nt > 32 ? (nt + LIST_CTA) / 32 * 16 : 0;
        lw = at; at += LIST_CTA / 32 * 16;
        ll = at; at += 16;
        x = at; at += cl ? 2 * CS_MAX * 16 : 0;
        flag = at; at += 16;
        total = at;
    }
};

// At 2^((z - m) ct) + A1 e^(z - m) for every column of the slice (S, H: which
// of the two there are); both coefficients 0: zeros, whatever the logits are.
// Each slot is refilled from the next row nx (if there is one) once it has been read.
template <typename T, int NT, bool S, bool H, int PW = 0>
__device__ __forceinline__ void grad_pass(const Slice<T>& s, char* buf, T* drow, int V, int tid, bool same_phase,
                                          float m, float ct, float At, float A1, const Slice<T>& nx, bool more) {
    using E = Elem<T>;
    constexpr int P = E::EPG / 2, U = 4;
    const bool zero = At == 0.0f && A1 == 0.0f, far = is_far(m);
    uint4* const d0 = reinterpret_cast<uint4*>(drow + s.col(0));  // where slot 0 goes
    const uint4* v = reinterpret_cast<const uint4*>(buf);
    auto store_edge = [&](int i, const f2* r) {
        const int c0 = s.col(i);
#pragma unroll
        for (int j = 0; j < P; j++) {
            float x, y;
            unpk(r[j], x, y);
            const int c = c0 + 2 * j;
            if (c >= 0 && c < V) drow[c] = E::put(x);
            if (c + 1 >= 0 && c + 1 < V) drow[c + 1] = E::put(y);
        }
    };
    if (zero || far) {
#pragma unroll 1
        for (int i = tid; i < s.n; i += NT) {
            f2 r[P];
#pragma unroll
            for (int j = 0; j < P; j++) {
                const T* p = reinterpret_cast<const T*>(v + i) + 2 * j;
                float w[2];
#pragma unroll
                for (int l = 0; l < 2; l++) {
                    const float z = E::get(p + l);
                    w[l] = zero ? 0.0f : (S ? At * exp_of(z, m, ct) : 0.0f) + (H ? A1 * exp_of(z, m, LOG2E) : 0.0f);
                }
                r[j] = pk(w[0], w[1]);
            }
            if (same_phase && s.inner(i)) d0[i] = E::pack(r);
            else store_edge(i, r);
        }
        if (more) fill<T, NT>(nx, buf, tid);
        return;
    }
    const float nt = -(m * ct), n1 = -(m * LOG2E);
    const float bt = S ? At * unbias(m, ct, nt) : 0.0f, b1 = H ? A1 * (PW ? powi<PW>(unbias(m, ct, nt)) : unbias(m, LOG2E, n1)) : 0.0f;
    const f2 c2 = pk(ct, ct), c1 = pk(LOG2E, LOG2E), nt2 = pk(nt, nt), n12 = pk(n1, n1), at2 = pk(bt, bt), a12 = pk(b1, b1);
    auto grad = [&](const uint4& u, f2* r) {
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
    };
    const int nx0 = more ? nx.i0 : 0, nx1 = more ? nx.i1 : 0;
    const char* g = nx.base + (long long)tid * 16;
    uint32_t b = (uint32_t)__cvta_generic_to_shared(buf) + tid * 16;
    int i = tid;
    // blocks of four slots that are wholly inside the row
    for (; same_phase && i + (U - 1) * NT < s.i1; i += U * NT, g += 16 * U * NT, b += 16 * U * NT) {
        uint4 u[U];
#pragma unroll
        for (int j = 0; j < U; j++) u[j] = v[i + j * NT];
#pragma unroll
        for (int j = 0; j < U; j++) {
            f2 r[P];
            grad(u[j], r);
            if (i >= s.i0) d0[i + j * NT] = E::pack(r);
            else if (j > 0) d0[i + j * NT] = E::pack(r);
            else store_edge(i, r);
        }
        if (i >= nx0 && i + (U - 1) * NT < nx1) {
            cp16<0>(b, g);
            cp16<16 * NT>(b, g);
            cp16<32 * NT>(b, g);
            cp16<48 * NT>(b, g);
        } else {
#pragma unroll
            for (int j = 0; j < U; j++)
                if (i + j * NT >= nx0 && i + j * NT < nx1) cp16<0>(b + j * 16 * NT, g + j * 16 * NT);
        }
    }
#pragma unroll 1
    for (; i < max(s.n, nx1); i += NT, g += 16 * NT, b += 16 * NT) {
        if (i < s.n) {
            f2 r[P];
            grad(v[i], r);
            if (same_phase && s.inner(i)) d0[i] = E::pack(r);
            else store_edge(i, r);
        }
        if (i >= nx0 && i < nx1) cp16<0>(b, g);
    }
}

// In a CTA, LIST_CTA threads of their own look after the list, beside the NT
// threads' passes over the row (as a part of one of those warps' work it held
// the others up at every barrier: 1422 us for the 32768 rows of 50257).  Every
// warp merges the warps' sums and forms the coefficients for itself, which
// saves a barrier.
template <typename T, int NT, bool CL>
__global__ void __launch_bounds__(distill_threads(NT), cta_per_sm(NT))
k_distill(const T* z, T* dz, const DistillArgs a) {
    pdl_enter();
    extern __shared__ __align__(16) char smem[];
    constexpr int EPG = Elem<T>::EPG;
    constexpr int LT = NT == 32 ? 32 : LIST_CTA;
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int lane = threadIdx.x & 31, warp = tid >> 5;
    const int lt = NT == 32 ? tid : tid - NT;  // >= 0: a thread of the list
    const bool worker = NT == 32 || tid < NT, lister = lt >= 0;
    const DistillLayout lay(NT, a.Gs, a.nbuf, a.k, EPG, CL);
    char* sm = smem + (NT == 32 ? threadIdx.x >> 5 : 0) * lay.total;
    const int k = a.k, V = a.V, k4 = align16(4 * (k + 1)) / 4, nlw = (min(k, LT) + 31) / 32, pw = power_of(a.tau);
    uint32_t* s_bits = reinterpret_cast<uint32_t*>(sm + lay.bits);
    int* s_y = reinterpret_cast<int*>(sm + lay.yl);
    float* s_tl = reinterpret_cast<float*>(sm + lay.yl) + 2;
    float* s_t = reinterpret_cast<float*>(sm + lay.t);
    int* s_off = reinterpret_cast<int*>(sm + lay.off);
    float* s_zo = reinterpret_cast<float*>(sm + lay.zo);
    float4* s_part = reinterpret_cast<float4*>(sm + lay.part);
    float4* s_lw = reinterpret_cast<float4*>(sm + lay.lw);
    float* s_ll = reinterpret_cast<float*>(sm + lay.ll);
    float4* s_x = reinterpret_cast<float4*>(sm + lay.x);  // [2][cs]
    int* s_flag = reinterpret_cast<int*>(sm + lay.flag);  // the target is on the list
    const int rank = CL ? (int)cluster_rank() : 0, cs = CL ? a.cs : 1;
    const long long first = CL ? blockIdx.x / cs : blockIdx.x * (long long)cta_groups(NT) + (NT == 32 ? threadIdx.x >> 5 : 0);
    const long long stride = CL ? gridDim.x / cs : gridDim.x * (long long)cta_groups(NT);
    const bool rest = a.t_lse != nullptr, soft_on = a.alpha > 0.0f, hard_on = a.targets && a.alpha < 1.0f;
    const float it = 1.0f / a.tau, ct = LOG2E * it, lift = 20.0f / fmaxf(1.0f, it);
    float g_all = a.dscale;
    if (a.scale_dev) g_all *= *a.scale_dev;
    auto slice = [&](long long r) { return Slice<T>(z, r, a.ld, V, rank, a.Gs); };
    auto copy_lists = [&](long long r, int b) {
        if (lister)
            for (int j = lt; j < k; j += LT) {
                cp4(sm + lay.ti + (b * k4 + j) * 4, a.t_idx + r * k + j);
                cp4(sm + lay.tv + (b * k4 + j) * 4, a.t_vals + r * k + j);
            }
        if (lt == 0 && a.targets) cp4(s_y + b, a.targets + r);
        if (lt == 1 && rest) cp4(s_tl + b, a.t_lse + r);
    };

    if (worker)
        for (int w = tid; w < (a.Gs * EPG + 31) / 32; w += NT) s_bits[w] = 0;
    if (tid < 2) s_y[tid] = -1;
    if (tid == 0) *s_flag = 0;
    group_sync<NT>();
    for (int i = 0; i < a.nbuf; i++) {
        const long long r = first + i * stride;
        if (r < a.M) {
            if (worker) fill<T, NT>(slice(r), sm + i * a.Gs * 16, tid);
            copy_lists(r, i);
        }
        cp_commit();
    }
    T edge = Elem<T>::put(0.0f);
    if (lt >= 0 && lt < 16) {
        if (first < a.M) edge_store(slice(first), sm, edge_load(slice(first), V, lt), lt);
        if (first + stride < a.M) edge = edge_load(slice(first + stride), V, lt);
    }
    if (CL) cluster_sync();  // the others run: their shared memory may be written

    int itn = 0;
    for (long long row = first; row < a.M; row += stride, itn++) {
        const int par = itn & 1, b = a.nbuf == 2 ? par : 0;
        char* buf = sm + b * a.Gs * 16;
        int* s_ti = reinterpret_cast<int*>(sm + lay.ti) + b * k4;
        const float* s_tv = reinterpret_cast<const float*>(sm + lay.tv) + b * k4;
        float* s_zl = reinterpret_cast<float*>(sm + lay.zl) + par * k4;
        const Slice<T> s = slice(row);
        cp_wait(a.nbuf);
        group_sync<NT>();
        int y = s_y[b];
        const bool y_bad = y < -1 || y >= V;
        if (y_bad) y = -1;
        const bool hard = hard_on && y >= 0;

        // the list: the student's logits at its columns (in a cluster the
        // column's CTA sends them to all), duplicates, the replacement by -inf
        auto keep = [&](int j, float v) {
            if (CL)
                for (int r = 0; r < cs; r++) st_remote(remote(s_zl + j, r), v);
            else s_zl[j] = v;
        };
        float Rl = -INFINITY, l1 = 0.0f, lts = 0.0f;  // sums of listed exponentials
        const bool list_warp = lister && lt < nlw * 32;
        if (list_warp) {
            bool bad = y_bad && lt == 0;
            for (int j = lt; j < k; j += LT) {
                int c = s_ti[j], o = -1;
                if (c < 0 || c >= V) {
                    bad |= c != -1;
                    c = -1;
                } else {
                    o = s.at(c);
                }
                if (o >= 0) {
                    const int at = o / (int)sizeof(T);
                    const uint32_t bit = 1u << (at & 31);
                    if (atomicOr(&s_bits[at >> 5], bit) & bit) {  // listed twice
                        bad = true;
                        c = o = -1;
                    } else {
                        T* p = reinterpret_cast<T*>(buf + o);
                        const float v = Elem<T>::get(p);
                        keep(j, v);
                        s_zo[j] = v;
                        if (rest) {
                            *p = Elem<T>::put(-INFINITY);
                            Rl = fmaxf(Rl, v);
                        }
                        if (c == y) {
                            *s_flag = 1;
                            if (rest) keep(k, v);
                        }
                    }
                }
                s_ti[j] = c;
                s_off[j] = o;
                s_t[j] = c < 0 ? -INFINITY : s_tv[j] * it;
            }
            if (bad) atomicOr(&a.flags[FLAG_BAD_TOKEN], 1);
        }
        // (a listed target may read as -inf here; its entry then gives the value)
        const int oy = lt == 0 && hard ? s.at(y) : -1;
        const float vy = oy >= 0 ? Elem<T>::get(reinterpret_cast<const T*>(buf + oy)) : 0.0f;
        if (rest || !dz) group_sync<NT>();  // the list has been read (and replaced)
        if (oy >= 0 && !(rest && *s_flag)) keep(k, vy);
        // the teacher's side of a warp's entries: the largest and the sum of
        // exponentials, or, where the normaliser is known, the probabilities' sum
        if (list_warp) {
            float tm = -INFINITY, ts = 0.0f;
            bool used = false;
            for (int j = lt; j < k; j += LT) {
                tm = fmaxf(tm, s_t[j]);
                used |= s_ti[j] >= 0;
            }
            tm = rest ? s_tl[b] : warp_max(tm);
            for (int j = lt; j < k; j += LT)
                if (s_t[j] != -INFINITY) ts += ex2f((s_t[j] - tm) * LOG2E);
            ts = warp_sum(ts);
            used = __any_sync(0xffffffffu, used);
            if (lane == 0) s_lw[lt >> 5] = make_float4(tm, ts, used ? 1.0f : 0.0f, 0.0f);
            if (rest) {
                Rl = warp_max(Rl);
                for (int j = lt; j < k; j += LT)
                    if (s_off[j] >= 0) {
                        const float v = s_zo[j];
                        if (v != -INFINITY) {
                            l1 += exp_of(v, Rl, LOG2E);
                            lts += exp_of(v, Rl, ct);
                        }
                    }
                l1 = warp_sum(l1);
                lts = warp_sum(lts);
            }
        }

        // first pass: sums of exponentials, s1 and st, and sl of the listed ones
        float R = -INFINITY, s1 = 0.0f, st = 0.0f, sl = 0.0f, none;
        const long long next = row + a.nbuf * stride;
        const bool more = next < a.M;
        const Slice<T> nx = slice(more ? next : row);
        const int p2 = hard && soft_on ? pw : 0;
        if (worker) {
            if (!soft_on) sum_pass<T, NT, true, false>(s, buf, tid, LOG2E, ct, lift, none, R, s1, st);
            else if (!hard || p2 == 1) sum_pass<T, NT, false, true>(s, buf, tid, LOG2E, ct, lift, none, R, s1, st);
            else if (p2 == 2) sum_pass<T, NT, true, true, 2>(s, buf, tid, LOG2E, ct, lift, none, R, s1, st);
            else if (p2 == 3) sum_pass<T, NT, true, true, 3>(s, buf, tid, LOG2E, ct, lift, none, R, s1, st);
            else if (p2 == 4) sum_pass<T, NT, true, true, 4>(s, buf, tid, LOG2E, ct, lift, none, R, s1, st);
            else sum_pass<T, NT, true, true>(s, buf, tid, LOG2E, ct, lift, none, R, s1, st);
            if (p2 == 1) s1 = st;
            if (!dz && more) fill<T, NT>(nx, buf, tid);
            merge(R, s1, st, sl, ct, hard, false);
        }
        if (rest && list_warp) {
            if (NT == 32) {
                const float m = fmaxf(R, Rl);
                s1 = s1 * rescale(R, m, LOG2E) + l1 * rescale(Rl, m, LOG2E);
                st *= rescale(R, m, ct);
                sl = lts * rescale(Rl, m, ct);
                R = m;
            } else {
                R = Rl;
                s1 = l1;
                sl = lts;
            }
        }
        if (NT > 32) {
            constexpr int W = (NT + LIST_CTA) / 32;
            static_assert(W <= 16, "the merge below is over 16 lanes");
            if (lane == 0) s_part[warp] = make_float4(R, s1, st, sl);
            __syncthreads();
            if (!CL || warp == 0) {
                const int l = lane & 15;
                const float4 p = l < W ? s_part[l] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
                R = p.x; s1 = p.y; st = p.z; sl = p.w;
                merge<16>(R, s1, st, sl, ct, hard, rest);
            }
        }
        if (CL) {
            if (warp == 0 && lane < cs) {
                const uint32_t at = remote(s_x + par * cs + rank, lane);
                st_remote(at, R);
                st_remote(at + 4, s1);
                st_remote(at + 8, st);
                st_remote(at + 12, sl);
            }
            cluster_sync();
            const int l = lane & (CS_MAX - 1);
            const float4 p = l < cs ? s_x[par * cs + l] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
            R = p.x; s1 = p.y; st = p.z; sl = p.w;
            merge<CS_MAX>(R, s1, st, sl, ct, hard, rest);
        }

        // the teacher's normaliser and mass, and the coefficients of the gradient
        if (NT == 32) __syncwarp();
        float base = -INFINITY, W = 0.0f;
        bool used = false;
        if (rest) {
            base = s_tl[b];
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
        const bool soft = used && soft_on;
        const float ks = g_all * a.alpha * a.tau, kh = hard ? g_all * (1.0f - a.alpha) : 0.0f;
        const float su = st;  // off the list
        float pr = 0.0f;
        if (rest) {
            st += sl;
            if (su > 0.0f) pr = fmaxf(1.0f - W, 0.0f);
        }
        const float rt = __fdividef(soft ? ks : 0.0f, st), A1 = hard ? __fdividef(kh, s1) : 0.0f;
        const float Al = (W + pr) * rt, At = pr > 0.0f ? rt * (W + pr - pr * __fdividef(st, su)) : W * rt;
        T* drow = dz ? dz + row * a.ld : nullptr;
        if (dz && worker) {
            // second pass: the gradient
            const float As = soft ? At : 0.0f;
            if (soft && hard && p2 == 2)
                grad_pass<T, NT, true, true, 2>(s, buf, drow, V, tid, a.same_phase, R, ct, As, A1, nx, more);
            else if (soft && hard && p2 == 3)
                grad_pass<T, NT, true, true, 3>(s, buf, drow, V, tid, a.same_phase, R, ct, As, A1, nx, more);
            else if (soft && hard && p2 == 4)
                grad_pass<T, NT, true, true, 4>(s, buf, drow, V, tid, a.same_phase, R, ct, As, A1, nx, more);
            else if (soft && hard && p2 != 1)
                grad_pass<T, NT, true, true>(s, buf, drow, V, tid, a.same_phase, R, ct, As, A1, nx, more);
            else if (soft || !hard)
                grad_pass<T, NT, true, false>(s, buf, drow, V, tid, a.same_phase, R, ct, As + A1, 0.0f, nx, more);
            else
                grad_pass<T, NT, false, true>(s, buf, drow, V, tid, a.same_phase, R, ct, 0.0f, A1, nx, more);
            if (rank == cs - 1)
                for (long long c = V + tid; c < a.ld; c += NT) drow[c] = Elem<T>::put(0.0f);
        }
        if (list_warp && soft && rank == 0) {
            const float ls = logf(st);
            float part = 0.0f;
            for (int j = lt; j < k; j += LT) {
                const float lp = s_t[j] - base, p = ex2f(lp * LOG2E);
                if (s_t[j] != -INFINITY && (p > 0.0f || p != p)) part += p * (lp - ((s_zl[j] - R) * it - ls));
            }
            part = warp_sum(part);
            if (lane == 0) s_ll[lt >> 5] = part;
        }
        group_sync<NT>();  // the second pass's stores come before those of the list
        if (lt == 0 && rank == 0) {
            float loss = 0.0f;
            if (soft) {
                for (int w = 0; w < nlw; w++) loss += s_ll[w];
                if (pr > 0.0f) loss += pr * (logf(pr) - logf(__fdividef(su, st)));
                loss *= a.alpha * a.tau * a.tau;
            }
            if (hard) loss += (1.0f - a.alpha) * (R + logf(s1) - s_zl[k]);
            a.row_loss[row] = loss;
        }
        if (list_warp) {
            for (int j = lt; j < k; j += LT) {
                const int o = s_off[j], c = s_ti[j];
                if (o < 0) continue;
                s_bits[o / (int)sizeof(T) >> 5] = 0;
                if (!dz) continue;
                float r = 0.0f;
                if (soft) r = Al * exp_of(s_zl[j], R, ct) - (s_t[j] == -INFINITY ? 0.0f : ks * ex2f((s_t[j] - base) * LOG2E));
                if (hard) r += A1 * exp_of(s_zl[j], R, LOG2E) - (c == y ? kh : 0.0f);
                drow[c] = Elem<T>::put(r);
            }
        }
        if (lt == 0) {
            if (dz && hard && !*s_flag && s.at(y) >= 0) {
                float r = A1 * exp_of(s_zl[k], R, LOG2E) - kh;
                if (soft) r += At * exp_of(s_zl[k], R, ct);
                drow[y] = Elem<T>::put(r);
            }
            *s_flag = 0;
        }
        if (more) copy_lists(next, b);
        cp_commit();
        const long long n1 = row + stride, n2 = n1 + stride;
        if (lt >= 0 && lt < 16) {
            if (n1 < a.M) edge_store(slice(n1), sm + (a.nbuf == 2 ? par ^ 1 : 0) * a.Gs * 16, edge, lt);
            if (n2 < a.M) edge = edge_load(slice(n2), V, lt);
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// mean of M row losses: each thread adds rows t, t + 1024, ..., the threads'
// sums meet in a fixed tree
__global__ void __launch_bounds__(1024) k_row_mean(const float* __restrict__ row_loss, int M, float* __restrict__ out,
                                                   int* flags) {
    pdl_enter();
    __shared__ float s_w[32];
    float s = 0.0f;
    for (int i = threadIdx.x; i < M; i += 1024) s += row_loss[i];
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = warp_sum(s_w[threadIdx.x]);
        if (threadIdx.x == 0) {
            s /= (float)M;
            out[0] = s;
            if (!isfinite(s)) atomicOr(&flags[FLAG_NONFINITE], 1);
        }
    }
}

// ------------------------------------------------------------ launch
// How M rows of G granules are spread: the group size, the CTAs a row is
// shared by, and whether two rows of a group are on chip at once.
struct Plan {
    int nt = 0, cs = 1, nbuf = 2, Gs = 0, ctas = 0, threads = 0;
    size_t smem = 0;
};

constexpr size_t SMEM_CTA = 232448;  // 227 KB
constexpr size_t SMEM_SM = 233472;   // 228 KB, of which each CTA takes 1 KB more than its own
constexpr size_t SMEM_HALF = SMEM_SM / 2 - 1024;

template <typename Bytes> bool make_plan(Plan& p, int sms, long long M, int G, int big, Bytes&& bytes) {
    p.cs = 1;
    p.nbuf = 1;
    // two CTAs of an SM, each with a row (or slice) of its own: a larger row is cut
    auto need = [&](int cs) { return bytes(512, (G + cs - 1) / cs, 1, cs > 1); };
    while (p.cs < CS_MAX && need(p.cs) > SMEM_HALF) p.cs *= 2;
    if (need(p.cs) > SMEM_CTA) return false;
    // few rows are cut so that every SM has a part
    while (p.cs < CS_MAX && M * p.cs * 2 <= sms && G / (p.cs * 2) >= 256) p.cs *= 2;
    p.Gs = (G + p.cs - 1) / p.cs;
    p.nt = p.cs == 1 && G <= 128 ? 32 : p.Gs <= 2048 ? 256 : big;
    if (p.Gs <= 2048) p.nbuf = 2;
    p.smem = (size_t)bytes(p.nt, p.Gs, p.nbuf, p.cs > 1) * cta_groups(p.nt);
    const long long groups = (M + cta_groups(p.nt) - 1) / cta_groups(p.nt);
    const int per_sm = std::max<int>(1, std::min<int>(cta_per_sm(p.nt), (int)(SMEM_SM / (p.smem + 1024))));
    const long long room = std::max<long long>(1, (long long)sms * per_sm / p.cs);
    p.ctas = (int)(std::min(groups, room) * p.cs);
    p.threads = cta_threads(p.nt);
    return true;
}

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

#define ROW_KERNEL(NAME, NT_, CL_, ...)                            \
    do {                                                           \
        static PerDevice attr;                                     \
        if (!allow_smem(attr, NAME<T, NT_, CL_>)) return false;    \
        launch_rows(L, NAME<T, NT_, CL_>, p, __VA_ARGS__);         \
        return true;                                               \
    } while (0)

// granules of a row, for the worst place of its start
template <typename T> int row_granules(const void* z, long long ld, int V) {
    const bool aligned = ((uintptr_t)z & 15) == 0 && ld * (long long)sizeof(T) % 16 == 0;
    return (int)(((aligned ? 0 : 16 - (int)sizeof(T)) + (long long)V * (int)sizeof(T) + 15) / 16);
}

template <typename T> bool top_rows(const Launch& L, const void* z, TopArgs a) {
    Plan p;
    const int k = a.k, G = row_granules<T>(z, a.ld, a.V);
    // many rows: a warp each
    if (G > 128 && a.M >= L.num_sms * 12 && !a.skip) {
        const int granules = (G + 127) / 128 * 4;  // of a lane, whole stages
        int ub_log = granules <= TS_BLOCKS ? 0 : 2;
        while ((granules + (1 << ub_log) - 1) >> ub_log > TS_BLOCKS) ub_log++;
        const int nb = (granules + (1 << ub_log) - 1) >> ub_log;
        const int words = (nb + Blocks<T>::PER - 1) / Blocks<T>::PER;
        static PerDevice attr;
        if (!allow_smem(attr, k_top_stream<T>)) return false;
        a.Gs = G;
        p.smem = TS_WARPS * stream_warp_smem(words, k);
        p.threads = TS_WARPS * 32;
        const int per_sm = std::min(3, (int)(SMEM_SM / (p.smem + 1024)));
        p.ctas = std::min((a.M + TS_WARPS - 1) / TS_WARPS, L.num_sms * per_sm);
        launch_rows(L, k_top_stream<T>, p, (const T*)z, a, ub_log, words);
        return true;
    }
    if (!make_plan(p, L.num_sms, a.M, G, 512, [k](int nt, int Gs, int nbuf, bool cl) {
            return (size_t)TopLayout(nt, Gs, nbuf, k, cl).total;
        }))
        return false;
    a.Gs = p.Gs; a.cs = p.cs; a.nbuf = p.nbuf;
    if (p.nt == 32) ROW_KERNEL(k_top_rows, 32, false, (const T*)z, a);
    if (p.nt == 256 && p.cs == 1) ROW_KERNEL(k_top_rows, 256, false, (const T*)z, a);
    if (p.nt == 256) ROW_KERNEL(k_top_rows, 256, true, (const T*)z, a);
    if (p.cs == 1) ROW_KERNEL(k_top_rows, 512, false, (const T*)z, a);
    ROW_KERNEL(k_top_rows, 512, true, (const T*)z, a);
}

template <typename T> bool distill(const Launch& L, const void* z, void* dz, DistillArgs a) {
    Plan p;
    const int k = a.k;
    if (!make_plan(p, L.num_sms, a.M, row_granules<T>(z, a.ld, a.V), 256, [k](int nt, int Gs, int nbuf, bool cl) {
            return (size_t)DistillLayout(nt, Gs, nbuf, k, Elem<T>::EPG, cl).total;
        }))
        return false;
    a.Gs = p.Gs; a.cs = p.cs; a.nbuf = p.nbuf;
    p.threads = distill_threads(p.nt);
    a.same_phase = (((uintptr_t)z ^ (uintptr_t)dz) & 15) == 0;
    if (p.nt == 32) ROW_KERNEL(k_distill, 32, false, (const T*)z, (T*)dz, a);
    if (p.cs == 1) ROW_KERNEL(k_distill, 256, false, (const T*)z, (T*)dz, a);
    ROW_KERNEL(k_distill, 256, true, (const T*)z, (T*)dz, a);
}

}  // namespace

// a row is held by at most CS_MAX CTAs, which also need room for the lists
bool head_row_ok(tt_dtype dtype, int V) {
    if (dtype != TT_FP32 && dtype != TT_BF16 && dtype != TT_FP16) return false;
    return (long long)V * (dtype == TT_FP32 ? 4 : 2) <= TT_ROW_BYTES_MAX;
}

bool launch_top_rows(const Launch& L, tt_dtype dtype, const void* z, long long ld, int M, int V, int k, float tau,
                     float* vals, int32_t* idx, float* lse, double* lse64, const int32_t* skip) {
    if (L.dry) return true;
    TopArgs a{};
    a.vals = vals; a.idx = idx; a.lse = lse; a.lse64 = lse64; a.skip = skip;
    a.ld = ld; a.M = M; a.V = V; a.k = k; a.inv_tau = 1.0f / tau;
    if (dtype == TT_FP32) return top_rows<float>(L, z, a);
    if (dtype == TT_FP16) return top_rows<__half>(L, z, a);
    return top_rows<__nv_bfloat16>(L, z, a);
}

bool launch_distill(const Launch& L, tt_dtype dtype, const void* z, void* dz, const float* t_vals,
                    const int32_t* t_idx, const float* t_lse, const int32_t* targets, float* row_loss,
                    float* mean_loss, int M, int V, int ld, int k, float alpha, float tau, float dscale,
                    const float* scale_dev) {
    if (L.dry) return true;
    DistillArgs a{};
    a.t_vals = t_vals; a.t_idx = t_idx; a.t_lse = t_lse; a.targets = targets; a.scale_dev = scale_dev;
    a.row_loss = row_loss; a.flags = L.flags; a.ld = ld; a.M = M; a.V = V; a.k = k;
    a.alpha = alpha; a.tau = tau; a.dscale = dscale;
    bool ok;
    if (dtype == TT_FP32) ok = distill<float>(L, z, dz, a);
    else if (dtype == TT_FP16) ok = distill<__half>(L, z, dz, a);
    else ok = distill<__nv_bfloat16>(L, z, dz, a);
    if (!ok) return false;
    if (mean_loss) {
        L.count();
        launch_k(L, k_row_mean, dim3(1), dim3(1024), 0, row_loss, M, mean_loss, L.flags);
    }
    return true;
}

}  // namespace tt
