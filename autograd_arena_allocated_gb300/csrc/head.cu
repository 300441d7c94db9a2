// head.cu -- operators on the LM head's logits that deal in lists of columns:
//
//   k_top_stream    per row (or part of one) the k largest logits (ties: the
//                   lowest column) and the log-sum-exp
//   k_top_join      the parts' lists of a row as one
//   k_distill       distillation from a teacher's top logits: loss and
//                   gradient of a row
//   k_distill_short the same for rows of up to 2048 logits
//   k_row_mean      the mean of the row losses (fixed order)
//
// The kernels read a row of V logits from memory once, in the storage type
// (head_row.cuh); sums, statistics and losses are fp32.
#include "head_row.cuh"

#include <algorithm>
#include <cfloat>

namespace tt {
namespace {

using namespace head;

constexpr int LIST_MAX = TT_TOP_MAX;
constexpr int CS_MAX = 8;      // CTAs of a cluster (the portable limit)

constexpr int NT = 256;        // threads of a CTA that pass over a row
constexpr int LIST_CTA = 64;   // and those that look after its list

__host__ __device__ constexpr int align16(int n) { return (n + 15) & ~15; }

// ------------------------------------------------------------ top logits
// bits of order_of that tell two values of a storage type apart
template <typename T> struct OrderBits { static constexpr int N = 32; };
template <> struct OrderBits<__nv_bfloat16> { static constexpr int N = 16; };
template <> struct OrderBits<__half> { static constexpr int N = 19; };  // sign, 8 exponent bits of fp32, 10 of mantissa

struct TopArgs {
    float* vals;  // the lists, where a row is one part
    int32_t* idx;
    float* lse;
    unsigned long long* keys;  // [M][P][k] the parts' lists (NULL: one part), 0 where a part has fewer
    float2* parts;             // [M][P] the parts' references and sums of exponentials
    const int32_t* skip;
    long long ld;
    int M, V, k, Gs, P;
    bool want;  // the sums
    float inv_tau;
};

// Slot i of the slice, read from memory.
template <typename T> __device__ __forceinline__ uint4 granule(const Slice<T>& s, int i, int V) {
    return s.inner(i) ? reinterpret_cast<const uint4*>(s.base)[i]
                      : edge_granule(reinterpret_cast<const T*>(s.base) - s.col(0), s.col(i), V);
}

// f(value, column) for every element of the lane's granules, read from memory
template <typename T, typename F>
__device__ __forceinline__ void each_element(const Slice<T>& s, int V, int lane, F&& f) {
    for (int g = lane; g < s.n; g += 32) {
        f2 e[Elem<T>::EPG / 2];
        Elem<T>::unpack(granule(s, g, V), e);
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
// the blocks' maxima say too little: few different values.
template <typename T>
__device__ __noinline__ void exact_candidates(const Slice<T>& s, int V, int kk, int n_el, unsigned long long* s_cand,
                                              int* s_cnt, int lane) {
    __syncwarp();
    if (lane == 0) *s_cnt = 0;
    __syncwarp();
    auto sum = [](int c) { return __reduce_add_sync(0xffffffffu, c); };
    if (n_el <= LIST_MAX) {  // few enough to rank them all
        each_element(s, V, lane, [&](float v, int c) { s_cand[atomicAdd(s_cnt, 1)] = top_key(v, c); });
        __syncwarp();
        return;
    }
    constexpr int LOW = 32 - OrderBits<T>::N;
    uint32_t t = 0;
    for (int bit = 31; bit >= LOW; bit--) {
        const uint32_t cand = t | (1u << bit);
        int c = 0;
        each_element(s, V, lane, [&](float v, int) { c += order_of(v) >= cand; });
        if (sum(c) >= kk) t = cand;
    }
    const uint32_t above = t + (1u << LOW);  // no value's order is so large that this wraps
    int c = 0, e = 0;
    each_element(s, V, lane, [&](float v, int) {
        const uint32_t o = order_of(v);
        c += o >= above;
        e += o >= t && o < above;
    });
    const int need = kk - sum(c);
    int last = V;  // equal values are taken up to this column
    if (sum(e) > need) {
        last = 0;
        for (int bit = 20; bit >= 0; bit--) {  // V < 2^20
            const int x = last | (1 << bit);
            int n = 0;
            each_element(s, V, lane, [&](float v, int col) {
                const uint32_t o = order_of(v);
                n += o >= t && o < above && col < x;
            });
            if (sum(n) < need) last = x;
        }
    }
    each_element(s, V, lane, [&](float v, int col) {
        const uint32_t o = order_of(v);
        if (o >= above || (o >= t && col <= last)) s_cand[atomicAdd(s_cnt, 1)] = top_key(v, col);
    });
    __syncwarp();
}

// A warp takes a row, or a part of one where there are fewer rows than the SMs
// hold warps (the parts' lists are then joined, by k_top_join or by the beams'
// merge).  The row streams through a ring of the warp's own, without a barrier,
// and what stays of it is the largest value of every block of UB granules of a
// lane.  The
// k-th largest of those is the threshold; the few blocks at or above it (k,
// and those that tie) are read again from memory, and their elements at or
// above it are ranked.  A lane's four granules of a stage are neighbours in
// memory (64 bytes; in shared memory they are permuted so that eight lanes'
// reads fall into different banks): reading 64 blocks again then is 4% of a
// row of 50257 16-bit logits, where blocks of four granules 512 bytes apart
// cost 26% more DRAM traffic.  A CTA a row, the row held on chip, needs no
// second read but waits at its barriers: 940 us for 32768 such rows, and 75 us
// for a selection step of 256 fp32 rows.
// A row with more candidates than there is room for (ties: few different
// values) is gone through bit by bit from memory.
// 32768 rows of 50257 16-bit logits, k = 64: 624 us, 5.3 TB/s, 78% of the
// measured copy rate; what is left is instructions (15 thousand a row, 5
// thousand of them for the exponentials' sum).
constexpr int TS_WARPS = 8;                 // most warps of a CTA
// (28 warps of an SM at 72 registers: 642 us; 18 with a ring twice as deep: 686 us)
constexpr int TS_CTAS = 3;                  // CTAs of an SM
constexpr int TS_TASKS = 152 * TS_CTAS * TS_WARPS;  // rows, or parts, that are worked on at once
constexpr int TS_PARTS = 64;                // most parts of a row
constexpr int TS_JOIN = 2048;               // most entries of a row's parts' lists
constexpr int TS_BLOCKS = 64;               // most blocks of a lane
constexpr int TS_U = 4;                     // granules of a lane in a stage of the ring
constexpr int TS_RING = 2 * TS_U * 32 * 16;  // two stages

// room for candidates, and for blocks that hold them
__host__ __device__ constexpr int stream_cand(int k) { return k <= 64 ? 160 : 256; }
// the candidates take the place of the blocks' maxima once these are done with
__host__ __device__ constexpr int stream_blocks(int words, int k) {
    return words * 128 > stream_cand(k) * 8 ? words * 128 : stream_cand(k) * 8;
}
__host__ __device__ constexpr int stream_warp_smem(int words, int k) {
    return TS_RING + stream_blocks(words, k) + align16(stream_cand(k) * 2) + 16;
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
__global__ void __launch_bounds__(TS_WARPS * 32, TS_CTAS)
k_top_stream(const T* __restrict__ z, const TopArgs a, int ub_log, int words) {
    // no early trigger: the next kernel's CTAs, resident and waiting, take the room of this grid's last ones
    // (a selection step of 256 fp32 rows 93 us with it, 34 us without)
    pdl_wait();
    extern __shared__ __align__(16) char smem[];
    using E = Elem<T>;
    constexpr int PER = Blocks<T>::PER;
    const int lane = threadIdx.x & 31;
    const int TS_CAND = stream_cand(a.k);
    char* sm = smem + (threadIdx.x >> 5) * stream_warp_smem(words, a.k);
    Blocks<T> blocks{reinterpret_cast<uint32_t*>(sm + TS_RING)};
    auto* s_cand = reinterpret_cast<unsigned long long*>(sm + TS_RING);
    auto* s_hit = reinterpret_cast<uint16_t*>(sm + TS_RING + stream_blocks(words, a.k));
    int* s_cnt = reinterpret_cast<int*>(sm + stream_warp_smem(words, a.k) - 16);
    const int warps = blockDim.x >> 5, P = a.P;
    const long long tasks = (long long)a.M * P, stride = (long long)gridDim.x * warps;
    const bool want = a.want;
    const float ct = LOG2E * a.inv_tau, lift = 20.0f / fmaxf(1.0f, a.inv_tau);
    const int k = a.k, V = a.V;
    auto slice = [&](long long q) { return Slice<T>(z, q / P, a.ld, V, (int)(q % P), a.Gs); };
    auto from = [&](long long q) {  // the first task of this warp at or after q
        while (a.skip && q < tasks && a.skip[q / P]) q += stride;
        return q;
    };
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
    const long long first = from(blockIdx.x * (long long)warps + (threadIdx.x >> 5));
    for (long long task = first, next; task < tasks; task = next) {
        const Slice<T> s = slice(task);
        next = from(task + stride);
        const bool more = next < tasks;
        const Slice<T> nx = slice(more ? next : task);
        if (task == first) {
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
                        else if (i < s.n) u[j] = granule(s, i, V);
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
        const bool far = q.finish(tmax, sum, none);
        if (want && __any_sync(0xffffffffu, far)) {
            // (the lanes take other elements than they did above, so all have one reference)
            q.R = warp_max(tmax);
            sum = 0.0f;
            each_element(s, V, lane, [&](float v, int) { q.take_far(v, sum, none); });
        }
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
        // fewer than k blocks hold anything above -inf: then all that they hold is taken
        const bool few = !(E::get(&tv) > -INFINITY);
        const float thr = few ? -FLT_MAX : E::get(&tv);
        const int n_el = max(0, min(V, s.col(s.n)) - max(0, s.col(0))), kk = min(k, n_el);
        bool exact = false;
        __syncwarp();
        {
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
                        u[j] = on ? granule(s, slot, V) : make_uint4(E::NINF, E::NINF, E::NINF, E::NINF);
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
                const int cnt = *s_cnt;
                exact = cnt > TS_CAND;
                __syncwarp();
                if (few && cnt < kk) {
                    // the list ends with the first columns of -inf (or NaN), found among the first cnt + kk
                    const int c0 = max(0, s.col(0)), need = kk - cnt;
                    for (int i0 = 0, got = 0; i0 < n_el && got < need; i0 += 32) {
                        const T* zr = reinterpret_cast<const T*>(s.base) - s.col(0);
                        const bool on = i0 + lane < n_el && !(E::get(zr + c0 + min(i0 + lane, n_el - 1)) > -INFINITY);
                        const uint32_t m = __ballot_sync(0xffffffffu, on);
                        const int p = got + __popc(m & ((1u << lane) - 1u));
                        if (on && p < need) s_cand[cnt + p] = top_key(-INFINITY, c0 + i0 + lane);
                        got += __popc(m);
                    }
                    __syncwarp();
                    if (lane == 0) *s_cnt = kk;
                }
            }
        }
        if (exact) exact_candidates(s, V, kk, n_el, s_cand, s_cnt, lane);
        __syncwarp();
        if (a.keys) {
            unsigned long long* out = a.keys + task * k;
            ranks(s_cand, *s_cnt, kk, [&](int r, unsigned long long key) { out[r] = key; });
            for (int r = kk + lane; r < k; r += 32) out[r] = 0;
            if (want && lane == 0) a.parts[task] = make_float2(R, sum);
        } else {
            ranks(s_cand, *s_cnt, kk, [&](int r, unsigned long long key) {
                a.vals[task * k + r] = value_of((uint32_t)(key >> 32));
                a.idx[task * k + r] = key_col(key);
            });
            if (want && lane == 0) a.lse[task] = (float)lse_of(R, sum, a.inv_tau);
        }
        __syncwarp();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The lists of a row's parts as one, a warp a row (300 rows of 12 parts, k = 10: under 8 us).
constexpr int TJ_WARPS = 2;

__global__ void __launch_bounds__(TJ_WARPS * 32) k_top_join(const TopArgs a) {
    pdl_enter();
    __shared__ unsigned long long s_l[TJ_WARPS][TS_JOIN], s_key[TJ_WARPS][JOIN_ROOM];
    const int P = a.P, k = a.k, N = P * k, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = blockIdx.x * (long long)TJ_WARPS + warp;
    if (row >= a.M) return;
    for (int i = lane; i < N; i += 32) s_l[warp][i] = a.keys[row * N + i];
    float R = -INFINITY, s = 0.0f;
    if (a.want) join_parts(a.parts + row * P, P, LOG2E * a.inv_tau, R, s);
    __syncwarp();
    join_lists(s_l[warp], N, k, s_key[warp], [&](int r, unsigned long long key) {
        a.vals[row * k + r] = value_of((uint32_t)(key >> 32));
        a.idx[row * k + r] = key_col(key);
    });
    if (a.want && lane == 0) a.lse[row] = (float)lse_of(R, s, a.inv_tau);
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
//
// What has to be moved is the row in and the gradient out.  A row of 50257
// 16-bit logits (100 KB) is held by one CTA, two CTAs an SM, so that one's
// passes run beside the other's loads; a longer one is cut over a cluster.  At
// two exponentials an element and pass the special-function unit (32 a cycle
// and SM) would take 3.1 of the 4.5 us that such a row's traffic takes an SM,
// hence the powers (Sums).  32768 rows, k = 64, tau = 2, with hard labels:
// 1116 us, 5.9 TB/s, 87% of the measured copy rate (75% with t_lse, whose
// replacement holds up the first pass); then the rows' own chains (barrier,
// merge, coefficients: about 4 us of a row's 10) are what is left.  999 rows of
// 50257 fp32 logits, two CTAs a row: 92 us, 64%, of which 6% are the last
// round's empty places.
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

struct DistillLayout {
    int bits, ti, tv, tl, edge, zl, zo, t, off, part, lw, ll, x, flag, total;
    __host__ __device__ DistillLayout(int Gs, int nbuf, int k, int epg, bool cl) {
        const int k4 = align16(4 * (k + 1));
        int at = nbuf * Gs * 16;
        bits = at; at += align16((Gs * epg + 31) / 32 * 4);
        ti = at; at += nbuf * k4;
        tv = at; at += nbuf * k4;
        tl = at; at += 16;      // [nbuf] t_lse
        edge = at; at += 64;
        zl = at; at += 2 * k4;  // student logits of the list, and of the target
        zo = at; at += k4;      // those of this CTA's slice
        t = at; at += k4;       // t_j / tau
        off = at; at += k4;     // where this CTA holds the column, or -1
        part = at; at += 2 * (NT + LIST_CTA) / 32 * 16;
        lw = at; at += LIST_CTA / 32 * 16;
        ll = at; at += 16;
        x = at; at += cl ? 2 * CS_MAX * 16 : 0;
        flag = at; at += 16;
        total = at;
    }
};

// A CTA's threads meet at barrier ID, or arrive there without waiting.
template <int ID> __device__ __forceinline__ void meet() {
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(NT + LIST_CTA) : "memory");
}
template <int ID> __device__ __forceinline__ void arrive() {
    __threadfence_block();
    asm volatile("bar.arrive %0, %1;" ::"n"(ID), "n"(NT + LIST_CTA) : "memory");
}

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
// the others up at every barrier: 1422 us for the 32768 rows of 50257).  They
// wait for the others at the start of a row (its copies have arrived) and at
// its end (its gradient is written), the others do not wait for them there; all
// meet where the sums do.  Every warp merges the warps' sums and forms the
// coefficients for itself, which saves a barrier.
template <typename T, bool CL>
__global__ void __launch_bounds__(NT + LIST_CTA, 2)
k_distill(const T* z, T* dz, const DistillArgs a) {
    pdl_wait();
    extern __shared__ __align__(16) char smem[];
    constexpr int EPG = Elem<T>::EPG;
    constexpr int LT = LIST_CTA;
    const int tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    const int lt = tid - NT;  // >= 0: a thread of the list
    const bool worker = tid < NT, lister = lt >= 0;
    const DistillLayout lay(a.Gs, a.nbuf, a.k, EPG, CL);
    char* sm = smem;
    const int k = a.k, V = a.V, k4 = align16(4 * (k + 1)) / 4, nlw = (min(k, LT) + 31) / 32, pw = power_of(a.tau);
    uint32_t* s_bits = reinterpret_cast<uint32_t*>(sm + lay.bits);
    float* s_tl = reinterpret_cast<float*>(sm + lay.tl);
    T* s_edge = reinterpret_cast<T*>(sm + lay.edge);  // [2][head, tail] granules
    float* s_t = reinterpret_cast<float*>(sm + lay.t);
    int* s_off = reinterpret_cast<int*>(sm + lay.off);
    float* s_zo = reinterpret_cast<float*>(sm + lay.zo);
    float4* s_part = reinterpret_cast<float4*>(sm + lay.part);
    float4* s_lw = reinterpret_cast<float4*>(sm + lay.lw);
    float* s_ll = reinterpret_cast<float*>(sm + lay.ll);
    float4* s_x = reinterpret_cast<float4*>(sm + lay.x);  // [2][cs]
    int* s_flag = reinterpret_cast<int*>(sm + lay.flag);  // the target is on the list
    const int rank = CL ? (int)cluster_rank() : 0, cs = CL ? a.cs : 1;
    const long long first = blockIdx.x / cs, stride = gridDim.x / cs;
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
        if (lt == 0 && rest) cp4(s_tl + b, a.t_lse + r);
    };

    if (worker)
        for (int w = tid; w < (a.Gs * EPG + 31) / 32; w += NT) s_bits[w] = 0;
    if (tid == 0) *s_flag = 0;
    for (int i = 0; i < a.nbuf; i++) {
        const long long r = first + i * stride;
        if (r < a.M) {
            if (worker) fill<T, NT>(slice(r), sm + i * a.Gs * 16, tid);
            copy_lists(r, i);
        }
        cp_commit();
    }
    // edge granules: this row's are put beside the buffers a row ahead, by the
    // list's threads; their slots' threads move them in
    auto put_edge = [&](const Slice<T>& e, int q, T v) {
        if (edge_slot(e, lt) >= 0) s_edge[(q * 2 + (lt >> 3)) * EPG + (lt & 7)] = v;
    };
    T edge = Elem<T>::put(0.0f);
    if (lister && lt < 16) {
        if (first < a.M) put_edge(slice(first), 0, edge_load(slice(first), V, lt));
        if (first + stride < a.M) edge = edge_load(slice(first + stride), V, lt);
    }
    int y_next = a.targets && first < a.M ? a.targets[first] : -1;
    __syncthreads();
    if (CL) cluster_sync();  // the others run: their shared memory may be written

    int itn = 0;
    for (long long row = first; row < a.M; row += stride, itn++) {
        const int par = itn & 1, b = a.nbuf == 2 ? par : 0;
        char* buf = sm + b * a.Gs * 16;
        int* s_ti = reinterpret_cast<int*>(sm + lay.ti) + b * k4;
        const float* s_tv = reinterpret_cast<const float*>(sm + lay.tv) + b * k4;
        float* s_zl = reinterpret_cast<float*>(sm + lay.zl) + par * k4;
        const Slice<T> s = slice(row);
        int y = y_next;
        if (a.targets && row + stride < a.M) y_next = a.targets[row + stride];
        const bool y_bad = y < -1 || y >= V;
        if (y_bad) y = -1;
        const bool hard = hard_on && y >= 0;
        cp_wait(a.nbuf);
        if (worker) {
            const uint4* e = reinterpret_cast<const uint4*>(s_edge) + par * 2;
            if (s.head && tid == 0) reinterpret_cast<uint4*>(buf)[0] = e[0];
            if (s.tail && tid == (s.n - 1) % NT) reinterpret_cast<uint4*>(buf)[s.n - 1] = e[1];
            arrive<1>();
        } else {
            meet<1>();
        }

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
            for (int j = lt; j < k; j += LT) {
                const int c = s_ti[j], o = c >= 0 && c < V ? s.at(c) : -1;
                s_off[j] = o;
                if (o < 0) continue;
                T* p = reinterpret_cast<T*>(buf + o);
                s_zo[j] = Elem<T>::get(p);
                if (rest) *p = Elem<T>::put(-INFINITY);
            }
        }
        // the target's logit; listed, it is the entry's to give (here it may read as -inf)
        const int oy = lt == 0 && hard ? s.at(y) : -1;
        const float vy = oy >= 0 ? Elem<T>::get(reinterpret_cast<const T*>(buf + oy)) : 0.0f;
        if (list_warp && hard)
            for (int j = lt; j < k; j += LT)
                if (s_ti[j] == y && s_off[j] >= 0) {
                    *s_flag = 1;
                    if (rest) keep(k, s_zo[j]);
                }
        if (rest || !dz) __syncthreads();  // the list has been read (and replaced)
        if (oy >= 0 && !(rest && *s_flag)) keep(k, vy);
        if (lister && lt < 16) {
            const long long n1 = row + stride, n2 = n1 + stride;
            if (n1 < a.M) put_edge(slice(n1), par ^ 1, edge);
            if (n2 < a.M) edge = edge_load(slice(n2), V, lt);
        }
        if (list_warp) {
            bool bad = y_bad && lt == 0;
            for (int j = lt; j < k; j += LT) {
                int c = s_ti[j];
                const int o = s_off[j];
                if (c < 0 || c >= V) {
                    bad |= c != -1;
                    c = -1;
                } else if (o >= 0) {
                    const int at = o / (int)sizeof(T);
                    const uint32_t bit = 1u << (at & 31);
                    if (atomicOr(&s_bits[at >> 5], bit) & bit) {  // listed twice
                        bad = true;
                        c = s_off[j] = -1;
                    } else {
                        keep(j, s_zo[j]);
                        Rl = fmaxf(Rl, s_zo[j]);
                    }
                }
                s_ti[j] = c;
                s_t[j] = c < 0 ? -INFINITY : s_tv[j] * it;
            }
            if (bad) atomicOr(&a.flags[FLAG_BAD_TOKEN], 1);
        }
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
            R = Rl;
            s1 = l1;
            sl = lts;
        }
        constexpr int WARPS = (NT + LIST_CTA) / 32;
        static_assert(WARPS <= 16, "the merge below is over 16 lanes");
        if (lane == 0) s_part[par * WARPS + warp] = make_float4(R, s1, st, sl);
        __syncthreads();
        if (!CL || warp == 0) {
            const int l = lane & 15;
            const float4 p = l < WARPS ? s_part[par * WARPS + l] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
            R = p.x; s1 = p.y; st = p.z; sl = p.w;
            merge<16>(R, s1, st, sl, ct, hard, rest);
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
        if (worker) {
            cp_commit();
            arrive<2>();  // the second pass's stores come before those of the list
            continue;
        }
        meet<2>();
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
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Short rows (a warp holds one in its registers, lane l the columns l + 32 e):
// the same sums, with the list spread over the columns, ln p_j at column i_j in
// shared memory, so that every column knows whether it is listed and nothing
// is written twice.  A row takes a few hundred instructions whatever its
// length, which is what bounds the shortest: 16384 rows of 65 with k = 8 take
// 15.5 us (38 us as a warp's form of the kernel above, whose list handling is
// made for long rows), 30400 rows of 1024 102 us (401 us a CTA a row).
constexpr int DS_WARPS = 4;
constexpr uint32_t DS_UNLISTED = 0x7FC0DEADu;  // a NaN that no arithmetic makes

template <typename T, int E>
__global__ void __launch_bounds__(DS_WARPS * 32, E <= 4 ? 8 : E <= 16 ? 6 : E <= 32 ? 5 : 3)
k_distill_short(const T* z, T* dz, const DistillArgs a) {
    pdl_enter();
    __shared__ uint32_t s_all[DS_WARPS][32 * E];
    using El = Elem<T>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = a.k, V = a.V;
    uint32_t* s_lp = s_all[warp] + lane;  // the lane's columns at steps of 32
    const bool rest = a.t_lse != nullptr, soft_on = a.alpha > 0.0f, hard_on = a.targets && a.alpha < 1.0f;
    const float it = 1.0f / a.tau, ct = LOG2E * it;
    float g_all = a.dscale;
    if (a.scale_dev) g_all *= *a.scale_dev;
    for (long long row = blockIdx.x * (long long)DS_WARPS + warp; row < a.M; row += gridDim.x * (long long)DS_WARPS) {
        const T* zr = z + row * a.ld;
        float x[E];
        float m = -INFINITY;
#pragma unroll
        for (int e = 0; e < E; e++) {
            const int c = lane + 32 * e;
            x[e] = c < V ? El::get(zr + c) : -INFINITY;
        }
        int col[LIST_MAX / 32];
        float t[LIST_MAX / 32];
#pragma unroll
        for (int i = 0; i < LIST_MAX / 32; i++) {
            const int j = lane + 32 * i;
            col[i] = j < k ? a.t_idx[row * k + j] : -1;
            t[i] = j < k ? a.t_vals[row * k + j] * it : -INFINITY;
        }
        int y = a.targets ? a.targets[row] : -1;
        const float tl = rest ? a.t_lse[row] : 0.0f;
        bool bad = y < -1 || y >= V;
        if (bad) y = -1;
        const bool hard = hard_on && y >= 0;
#pragma unroll
        for (int e = 0; e < E; e++) {
            s_lp[32 * e] = DS_UNLISTED;
            m = fmaxf(m, x[e]);
        }
        m = warp_max(m);
        // the teacher's normaliser
        float base = tl;
        bool used = false;
        float tm = -INFINITY, ts = 0.0f;
#pragma unroll
        for (int i = 0; i < LIST_MAX / 32; i++) {
            if (col[i] < 0 || col[i] >= V) {
                bad |= col[i] != -1;
                col[i] = -1;
                t[i] = -INFINITY;
            }
            used |= col[i] >= 0;
            tm = fmaxf(tm, t[i]);
        }
        used = __any_sync(0xffffffffu, used);
        if (!rest) {
            tm = warp_max(tm);
#pragma unroll
            for (int i = 0; i < LIST_MAX / 32; i++)
                if (t[i] != -INFINITY) ts += ex2f((t[i] - tm) * LOG2E);
            ts = warp_sum(ts);
            base = tm + logf(ts);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < LIST_MAX / 32; i++)
            if (col[i] >= 0) {
                const float lp = t[i] == -INFINITY ? -INFINITY : t[i] - base;
                bad |= atomicCAS(s_all[warp] + col[i], DS_UNLISTED, __float_as_uint(lp)) != DS_UNLISTED;  // listed twice
            }
        if (bad) atomicOr(&a.flags[FLAG_BAD_TOKEN], 1);
        __syncwarp();
        const bool soft = used && soft_on;
        float s1 = 0.0f, su = 0.0f, sl = 0.0f, W = 0.0f, part = 0.0f, zy = 0.0f;
#pragma unroll
        for (int e = 0; e < E; e++) {
            const int c = lane + 32 * e;
            if (c >= V) continue;
            const float d = x[e] - m;
            if (hard) s1 += ex2f(d * LOG2E);
            if (c == y) zy = x[e];
            if (soft) {
                const float et = ex2f(d * ct);
                const uint32_t u = s_lp[32 * e];
                if (u == DS_UNLISTED) {
                    su += et;
                } else {
                    const float lp = __uint_as_float(u), p = ex2f(lp * LOG2E);
                    sl += et;
                    W += p;
                    if (p > 0.0f || p != p) part += p * (lp - d * it);
                }
            }
        }
        if (hard) {
            s1 = warp_sum(s1);
            zy = __shfl_sync(0xffffffffu, zy, y & 31);
        }
        float st = 0.0f, pr = 0.0f;
        if (soft) {
            su = warp_sum(su);
            sl = warp_sum(sl);
            W = warp_sum(W);
            part = warp_sum(part);
            st = su + sl;
            if (rest && su > 0.0f) pr = fmaxf(1.0f - W, 0.0f);
        }
        if (lane == 0) {
            float loss = 0.0f;
            if (soft) {
                loss = part + W * logf(st);
                if (pr > 0.0f) loss += pr * (logf(pr) - logf(__fdividef(su, st)));
                loss *= a.alpha * a.tau * a.tau;
            }
            if (hard) loss += (1.0f - a.alpha) * (m + logf(s1) - zy);
            a.row_loss[row] = loss;
        }
        if (dz) {
            T* dr = dz + row * a.ld;
            const float ks = g_all * a.alpha * a.tau, kh = hard ? g_all * (1.0f - a.alpha) : 0.0f;
            const float rt = soft ? __fdividef(ks, st) : 0.0f, A1 = hard ? __fdividef(kh, s1) : 0.0f;
            const float Al = (W + pr) * rt, At = pr > 0.0f ? rt * (W + pr - pr * __fdividef(st, su)) : W * rt;
#pragma unroll
            for (int e = 0; e < E; e++) {
                const int c = lane + 32 * e;
                const float d = x[e] - m;
                float r = 0.0f;
                if (soft) {
                    const uint32_t u = s_lp[32 * e];
                    const float et = ex2f(d * ct);
                    r = u == DS_UNLISTED ? At * et : Al * et - ks * ex2f(__uint_as_float(u) * LOG2E);
                }
                if (hard) r += A1 * ex2f(d * LOG2E) - (c == y ? kh : 0.0f);
                if (c < a.ld) dr[c] = El::put(c < V ? r : 0.0f);
            }
            for (long long c = 32 * E + lane; c < a.ld; c += 32) dr[c] = El::put(0.0f);
        }
        __syncwarp();
    }
}

// mean of M row losses: each thread adds rows t, t + 1024, ..., the threads'
// sums meet in a fixed tree (3 us for 32768)
__global__ void __launch_bounds__(1024) k_row_mean(const float* __restrict__ row_loss, int M, float* __restrict__ out,
                                                   int* flags) {
    pdl_enter();
    __shared__ float s_w[32];
    float s = 0.0f;
    for (long long i = threadIdx.x; i < M; i += 1024) s += row_loss[i];
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
// How a kernel's CTAs are laid out; for distillation also the CTAs that share
// a row, their slices, and whether two rows of a CTA are on chip at once.
struct Plan {
    int cs = 1, nbuf = 1, Gs = 0, ctas = 0, threads = 0;
    size_t smem = 0;
};

constexpr size_t SMEM_CTA = 232448;  // 227 KB
constexpr size_t SMEM_SM = 233472;   // 228 KB, of which each CTA takes 1 KB more than its own
constexpr size_t SMEM_HALF = SMEM_SM / 2 - 1024;

template <typename Bytes> bool make_plan(Plan& p, int sms, long long M, int G, Bytes&& bytes) {
    // two CTAs of an SM, each with a row (or slice) of its own: a larger row is cut
    auto need = [&](int cs, int nbuf) { return bytes((G + cs - 1) / cs, nbuf, cs > 1); };
    while (p.cs < CS_MAX && need(p.cs, 1) > SMEM_HALF) p.cs *= 2;
    if (need(p.cs, 1) > SMEM_CTA) return false;
    // few rows are cut so that every SM has a part
    while (p.cs < CS_MAX && M * p.cs <= sms && G / (p.cs * 2) >= 256) p.cs *= 2;
    p.Gs = (G + p.cs - 1) / p.cs;
    p.nbuf = need(p.cs, 2) <= SMEM_HALF ? 2 : 1;
    p.smem = need(p.cs, p.nbuf);
    const long long per_sm = p.smem <= SMEM_HALF ? 2 : 1;
    p.ctas = (int)(std::min(M, std::max<long long>(1, sms * per_sm / p.cs)) * p.cs);
    p.threads = NT + LIST_CTA;
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

#define ROW_KERNEL(NAME, CL_, ...)                            \
    do {                                                      \
        static PerDevice attr;                                \
        if (!allow_smem(attr, NAME<T, CL_>)) return false;    \
        launch_rows(L, NAME<T, CL_>, p, __VA_ARGS__);         \
        return true;                                          \
    } while (0)

// granules of a row, for the worst place of its start
template <typename T> int row_granules(const void* z, long long ld, int V) {
    const bool aligned = ((uintptr_t)z & 15) == 0 && ld * (long long)sizeof(T) % 16 == 0;
    return (int)(((aligned ? 0 : 16 - (int)sizeof(T)) + (long long)V * (int)sizeof(T) + 15) / 16);
}

template <typename T> bool top_rows(const Launch& L, const void* z, TopArgs a) {
    Plan p;
    const int G = row_granules<T>(z, a.ld, a.V);
    a.Gs = (G + a.P - 1) / a.P;
    const int granules = (a.Gs + 127) / 128 * 4;  // of a lane, whole stages
    // blocks of four granules where they are enough to tell k of them from the rest
    int ub_log = granules <= TS_BLOCKS && granules * 8 < 4 * a.k ? 0 : 2;
    while ((granules + (1 << ub_log) - 1) >> ub_log > TS_BLOCKS) ub_log++;
    const int nb = (granules + (1 << ub_log) - 1) >> ub_log;
    const int words = (nb + Blocks<T>::PER - 1) / Blocks<T>::PER;
    static PerDevice attr;
    if (!allow_smem(attr, k_top_stream<T>)) return false;
    // few tasks are spread over the SMs
    const long long tasks = (long long)a.M * a.P;
    const int warps = (int)std::min<long long>(TS_WARPS, std::max<long long>(1, tasks / L.num_sms));
    p.smem = (size_t)warps * stream_warp_smem(words, a.k);
    p.threads = warps * 32;
    const long long per_sm = std::min<long long>(TS_CTAS * TS_WARPS / warps, (long long)(SMEM_SM / (p.smem + 1024)));
    p.ctas = (int)std::min((tasks + warps - 1) / warps, L.num_sms * per_sm);
    launch_rows(L, k_top_stream<T>, p, (const T*)z, a, ub_log, words);
    return true;
}

template <typename T, int E> bool distill_short(const Launch& L, const void* z, void* dz, const DistillArgs& a) {
    L.count();
    const unsigned ctas = (unsigned)std::min((a.M - 1) / DS_WARPS + 1, L.num_sms * 12);
    launch_k(L, k_distill_short<T, E>, dim3(ctas), dim3(DS_WARPS * 32), 0, (const T*)z, (T*)dz, a);
    return true;
}

template <typename T> bool distill(const Launch& L, const void* z, void* dz, DistillArgs a) {
    Plan p;
    const int k = a.k;
    if (a.V <= 128) return distill_short<T, 4>(L, z, dz, a);
    if (a.V <= 512) return distill_short<T, 16>(L, z, dz, a);
    if (a.V <= 1024) return distill_short<T, 32>(L, z, dz, a);
    // (64 registers of a row a lane: 30400 rows of 2048 215 us, 20 rows 14 us; a CTA a row 450 and 9 us)
    if (a.V <= 2048 && a.M >= 2 * L.num_sms) return distill_short<T, 64>(L, z, dz, a);
    if (!make_plan(p, L.num_sms, a.M, row_granules<T>(z, a.ld, a.V), [k](int Gs, int nbuf, bool cl) {
            return (size_t)DistillLayout(Gs, nbuf, k, Elem<T>::EPG, cl).total;
        }))
        return false;
    a.Gs = p.Gs; a.cs = p.cs; a.nbuf = p.nbuf;
    a.same_phase = (((uintptr_t)z ^ (uintptr_t)dz) & 15) == 0;
    if (p.cs == 1) ROW_KERNEL(k_distill, false, (const T*)z, (T*)dz, a);
    ROW_KERNEL(k_distill, true, (const T*)z, (T*)dz, a);
}

}  // namespace

// distillation: a row is held by at most CS_MAX CTAs, which also need room for the list
bool head_row_ok(tt_dtype dtype, int V) {
    if (dtype != TT_FP32 && dtype != TT_BF16 && dtype != TT_FP16) return false;
    return (long long)V * (dtype == TT_FP32 ? 4 : 2) <= TT_ROW_BYTES_MAX;
}

int top_parts(tt_dtype dtype, int M, int V, int k, int entries) {
    const long long G = ((long long)V * (dtype == TT_FP32 ? 4 : 2) + 15) / 16;
    const long long p = std::min<long long>(std::min<long long>(TS_TASKS / M, G / 192),
                                            std::min<long long>(entries / k, TS_PARTS));
    return (int)std::max<long long>(p, 1);
}

size_t top_rows_scratch_bytes(tt_dtype dtype, int M, int V, int k) {
    const size_t P = (size_t)top_parts(dtype, M, V, k, TS_JOIN);
    return P == 1 ? 0 : (size_t)M * P * 8 * ((size_t)k + 1);
}

bool launch_top_rows(const Launch& L, tt_dtype dtype, const void* z, long long ld, int M, int V, int k, float tau,
                     float* vals, int32_t* idx, float* lse, void* scratch) {
    if (L.dry) return true;
    TopArgs a{};
    a.vals = vals; a.idx = idx; a.lse = lse; a.want = lse != nullptr;
    a.ld = ld; a.M = M; a.V = V; a.k = k; a.inv_tau = 1.0f / tau;
    a.P = top_parts(dtype, M, V, k, TS_JOIN);
    if (a.P > 1) {
        a.keys = (unsigned long long*)scratch;
        a.parts = (float2*)(a.keys + (size_t)M * a.P * k);
    }
    const bool ok = dtype == TT_FP32   ? top_rows<float>(L, z, a)
                    : dtype == TT_FP16 ? top_rows<__half>(L, z, a)
                                       : top_rows<__nv_bfloat16>(L, z, a);
    if (!ok) return false;
    if (a.P > 1) {
        L.count();
        launch_k(L, k_top_join, dim3((M + TJ_WARPS - 1) / TJ_WARPS), dim3(TJ_WARPS * 32), 0, a);
    }
    return true;
}

bool launch_top_parts(const Launch& L, tt_dtype dtype, const void* z, long long ld, int M, int V, int k, int P,
                      unsigned long long* keys, float2* parts, const int32_t* skip) {
    if (L.dry) return true;
    TopArgs a{};
    a.keys = keys; a.parts = parts; a.skip = skip; a.want = true;
    a.ld = ld; a.M = M; a.V = V; a.k = k; a.P = P; a.inv_tau = 1.0f;
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
