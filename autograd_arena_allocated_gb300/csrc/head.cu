// head.cu -- the top logits of rows of the LM head's logits:
//
//   k_top_stream    per row (or part of one) the k largest logits (ties: the
//                   lowest column) and the log-sum-exp
//   k_top_join      the parts' lists of a row as one
//   k_top_short     the same of rows of up to 128 logits
//
// A row of V logits is read from memory once, in the storage type, but for the
// few blocks that hold its largest (head_row.cuh); sums are fp32.
#include "head_row.cuh"

#include <cfloat>

namespace tt {
namespace {

using namespace head;

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
// 32768 rows of 50257 16-bit logits, k = 64: 628 us, 5.3 TB/s, 78% of the
// measured copy rate; what is left is instructions (14 thousand a row, 5
// thousand of them for the exponentials' sum).
constexpr int TS_WARPS = 8;                 // most warps of a CTA
// (28 warps of an SM at 72 registers: 642 us; 18 with a ring twice as deep: 686 us)
constexpr int TS_CTAS = 3;                  // CTAs of an SM
constexpr int TS_TASKS = TOP_TASKS;           // rows, or parts, that are worked on at once
static_assert(TS_TASKS == 152 * TS_CTAS * TS_WARPS, "a warp a task");
constexpr int TS_PARTS = 64;                // most parts of a row
constexpr int TS_JOIN = 1024;               // most entries of a row's parts' lists
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
        Sums<T, true, false, 0, true> q(ct, ct, lift);
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
                        cp16<4 * 512>(ring_at, src);
                        cp16<5 * 512>(ring_at, src);
                        cp16<6 * 512>(ring_at, src);
                        cp16<7 * 512>(ring_at, src);
                    }
                    cp_commit();
                    if (want) q.take(u);
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
                    if (want) q.take(u);
                    block(st + h, g4, g);
                }
            }
            // a chain of additions is 64 stages at most, and a few granules at the row's ends
            if (want && (st & 62) == 62) q.fold();
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
        unsigned long long* const part = a.keys ? a.keys + task * k : nullptr;
        ranks(s_cand, *s_cnt, kk, [&](int r, unsigned long long key) {
            if (part) {
                part[r] = key;
            } else {
                a.vals[task * k + r] = value_of((uint32_t)(key >> 32));
                a.idx[task * k + r] = key_col(key);
            }
        });
        if (part)
            for (int r = kk + lane; r < k; r += 32) part[r] = 0;
        if (want && lane == 0) {
            if (part) a.parts[task] = make_float2(R, sum);
            else a.lse[task] = (float)lse_of(R, sum, a.inv_tau);
        }
        __syncwarp();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Rows of up to 32 E logits: a warp holds one, lane l the columns l + 32 e, and
// sorts it.  What a row takes is the sort's instructions (E = 4: about 800):
// 30000 rows of 100 37 us; 91 and 166 us (k = 10, 64) by the kernel above, whose
// ring, threshold and second read are made for long rows.
constexpr int TH_WARPS = 4;

template <typename T, int E>
__global__ void __launch_bounds__(TH_WARPS * 32) k_top_short(const T* __restrict__ z, const TopArgs a) {
    pdl_enter();
    const int lane = threadIdx.x & 31, k = a.k, V = a.V;
    const float ct = LOG2E * a.inv_tau;
    for (long long row = blockIdx.x * (long long)TH_WARPS + (threadIdx.x >> 5); row < a.M;
         row += gridDim.x * (long long)TH_WARPS) {
        const T* zr = z + row * a.ld;
        float v[E];
        unsigned long long x[E];
        float R = -INFINITY;
#pragma unroll
        for (int e = 0; e < E; e++) {
            const int c = lane + 32 * e;
            v[e] = c < V ? Elem<T>::get(zr + c) : -INFINITY;
            x[e] = c < V ? top_key(v[e], c) : 0ull;
            R = fmaxf(R, v[e]);
        }
        if (a.want) {
            R = warp_max(R);
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < E; e++)
                if (lane + 32 * e < V) s += v[e] == R ? 1.0f : exp_of(v[e], R, ct);  // (inf - inf is a term of 1)
            s = warp_sum(s);
            if (lane == 0) a.lse[row] = (float)lse_of(R, s, a.inv_tau);
        }
        sort_keys(x);
#pragma unroll
        for (int e = 0; e < E; e++) {
            const int r = 32 * e + lane;
            if (r < k) {
                a.vals[row * k + r] = value_of((uint32_t)(x[e] >> 32));
                a.idx[row * k + r] = key_col(x[e]);
            }
        }
    }
}

// The lists of a row's parts as one, a warp a row (300 rows of 12 parts, k = 10: under 8 us).
constexpr int TJ_WARPS = 2;

__global__ void __launch_bounds__(TJ_WARPS * 32) k_top_join(const TopArgs a) {
    pdl_enter();
    __shared__ __align__(16) unsigned long long s_l[TJ_WARPS][TS_JOIN], s_key[TJ_WARPS][JOIN_ROOM];
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

template <typename T, int E> bool top_short(const Launch& L, const void* z, const TopArgs& a) {
    L.count();
    const unsigned ctas = (unsigned)std::min((a.M - 1) / TH_WARPS + 1, L.num_sms * 16);
    launch_k(L, k_top_short<T, E>, dim3(ctas), dim3(TH_WARPS * 32), 0, (const T*)z, a);
    return true;
}

template <typename T> bool top_rows(const Launch& L, const void* z, TopArgs a) {
    if (!a.keys && a.V <= 32) return top_short<T, 1>(L, z, a);
    if (!a.keys && a.V <= 64) return top_short<T, 2>(L, z, a);
    if (!a.keys && a.V <= 128) return top_short<T, 4>(L, z, a);
    Plan p;
    const int G = row_granules<T>(z, a.ld, a.V);
    a.Gs = (G + a.P - 1) / a.P;
    const int granules = (a.Gs + 127) / 128 * 4;  // of a lane, whole stages
    // blocks of four granules where they are enough (8 k) to tell k of them from
    // the rest: fewer make the second read long (100 rows of 120000 16-bit
    // logits, k = 64: 34 us from 4 k blocks on, 26 us so)
    int ub_log = granules <= TS_BLOCKS && granules < a.k ? 0 : 2;
    while ((granules + (1 << ub_log) - 1) >> ub_log > TS_BLOCKS) ub_log++;
    const int nb = (granules + (1 << ub_log) - 1) >> ub_log;
    const int words = (nb + Blocks<T>::PER - 1) / Blocks<T>::PER;
    static PerDevice attr;
    if (!allow_smem(attr, k_top_stream<T>)) return false;
    // tasks that are all worked on at once are spread evenly over the SMs by
    // small CTAs (100 rows of 120000 16-bit logits in 16 parts: 38 us as 200
    // CTAs of 8 warps, which are 16 warps on some SMs and 8 on others; 34 us so)
    const long long tasks = (long long)a.M * a.P;
    const int warps = tasks > TS_CTAS * TS_WARPS * L.num_sms ? TS_WARPS : tasks > L.num_sms ? 2 : 1;
    p.smem = (size_t)warps * stream_warp_smem(words, a.k);
    p.threads = warps * 32;
    const long long per_sm = std::min<long long>(TS_CTAS * TS_WARPS / warps, (long long)(SMEM_SM / (p.smem + 1024)));
    p.ctas = (int)std::min((tasks + warps - 1) / warps, L.num_sms * per_sm);
    launch_rows(L, k_top_stream<T>, p, (const T*)z, a, ub_log, words);
    return true;
}

}  // namespace

// A part has 192 granules at least, and 8 more for each entry of its list: what
// the list takes of a part's time does not shrink with the part (300 rows of
// 20000 16-bit logits, k = 64: 12 parts 26.6 us, 3 to 8 parts 22 to 25).
int top_parts(tt_dtype dtype, int M, int V, int k, int entries, int tasks) {
    const long long G = ((long long)V * (dtype == TT_FP32 ? 4 : 2) + 15) / 16;
    const long long p = std::min<long long>(std::min<long long>(tasks / M, G / (192 + 8 * k)),
                                            std::min<long long>(entries / k, TS_PARTS));
    return (int)std::max<long long>(p, 1);
}

// Two thirds of the SMs' warps (1000 rows of 50257 16-bit logits, k = 64, in 2
// parts 40 us, in 3 parts 48; 300 rows in 8 parts 26 us, in 12 parts 30), but
// two parts rather than one.
static int row_parts(tt_dtype dtype, int M, int V, int k) {
    const int p = top_parts(dtype, M, V, k, TS_JOIN, TS_TASKS * 2 / 3);
    return p > 1 ? p : top_parts(dtype, M, V, k, TS_JOIN, TS_TASKS);
}

size_t top_rows_scratch_bytes(tt_dtype dtype, int M, int V, int k) {
    const size_t P = (size_t)row_parts(dtype, M, V, k);
    return P == 1 ? 0 : (size_t)M * P * 8 * ((size_t)k + 1);
}

bool launch_top_rows(const Launch& L, tt_dtype dtype, const void* z, long long ld, int M, int V, int k, float tau,
                     float* vals, int32_t* idx, float* lse, void* scratch) {
    if (L.dry) return true;
    TopArgs a{};
    a.vals = vals; a.idx = idx; a.lse = lse; a.want = lse != nullptr;
    a.ld = ld; a.M = M; a.V = V; a.k = k; a.inv_tau = 1.0f / tau;
    a.P = row_parts(dtype, M, V, k);
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

}  // namespace tt
