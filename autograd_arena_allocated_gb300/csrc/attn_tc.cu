// attn_tc.cu -- causal self-attention on the 5th-generation tensor cores
// (tcgen05, bf16 or half in, fp32 accumulate in tensor memory), heads of 64, and the
// same over groups of answers, heads of 16, 32 and 64 (GRP, HD below).
//
// Every kernel streams 64-wide blocks of the other sequence past a
// 128-row tile, so that the score block (128 x 64 fp32) needs only 64 TMEM
// columns and several CTAs fit on one SM:
//   warp 0      TMA (128-byte-swizzled tiles straight from the packed
//               [B*T, 3C] qkv buffer and the [B*T, C] output gradient)
//   warp 1      TMEM allocation and the MMAs (one elected lane)
//   the others  one or two threads per tile row: a row of the score block from
//               TMEM, the elementwise work in fp32, and the 16-bit operand of the
//               next MMA back into TMEM.
//
// The MMA warp issues what does not wait for the rows' present work behind what
// does, so that the tensor pipe and the elementwise work overlap.
//
// Forward (one CTA per 128 queries, 4 CTAs/SM): S = Q K_j^T; online softmax
//   in base 2; P_j over S; O += P_j V_j accumulates in TMEM (V read as an
//   MN-major operand), rescaled in place only when the row max grows by more
//   than 2^8; finally y = O / l and the row's log-sum-exp.
// Backward, deterministic (no atomics):
//   dQ kernel (one CTA per 128 queries, 2 CTAs/SM): D = rowsum(dO o O);
//     S = Q K_j^T, dP = dO V_j^T; dS = P o (dP - D) with P from the saved
//     log-sum-exp (two dS buffers); dQ += dS K_j accumulates in TMEM.
//   dK/dV kernel (one CTA per 128 keys, 2 CTAs/SM): S^T = K Q_j^T,
//     dP^T = V dO_j^T; P^T and dS^T; dV += P^T dO_j, dK += dS^T Q_j in TMEM
//     (Q_j and dO_j, loaded K-major, are read again as MN-major operands).
//
// P and dS are rounded to the storage type, as operands of the second products (tf32
// operands would run at half the rate and take twice the tensor memory); the row sum
// takes P before that.  Against 64 bits y and dqkv are off by 1.3 to 1.4 times what
// their own rounding alone leaves.
//
// What bounds them: the row warps' chains of dependent steps (issue 43 to 47%, special
// functions below a third, no unit of the SM saturated); the MMAs take 34, 76 and 60%
// of the time at the rates below.
// Every wait is bounded (FLAG_TIMEOUT), as in the GEMM.
//
// GRP: the same kernels over groups of answers that share a prompt (group.cuh).
// The tile goes past the blocks that it needs only, blocks that are not seen
// whole take a 64-bit mask a row, and tiles of padding write zeros.  Padding may
// hold anything: a masked probability is 0, and 0 times a NaN is a NaN, so the
// block in which the padding begins has its rows of the operand whose rows the
// product sums over (V; K; Q and dO) cleared in shared memory.  Eight groups of 2048
// positions (half of them the prompt, four answers), 12 heads: 80 us forward (482
// TFLOP/s) and 236 backward (407); 16% of the blocks' pairs are masked, and by block
// they run as the causal ones do (85 and 255 us for as many causal positions).
// HD (groups only): heads of 32 and 16 load the 64 columns that theirs are among.
// Scores take the K steps of their own columns, the products into O, dQ, dK and dV
// all 64, of which theirs are stored: an MMA costs the same at N = 16 and at 64, and
// what bounds the kernels, the exponentials and their hand-overs, does not change.
// Four groups of 1400, 16 heads of 32, half: 28 us forward and 75 backward (by
// mma.sync, scores in registers, 57 and 173).
#include "tt_internal.h"
#include "group.cuh"
#include "tc_ptx.cuh"

#include <math.h>

#include <type_traits>

namespace tt {
namespace fa5 {

using namespace tc;
typedef __nv_bfloat16 bf16;

constexpr int D = 64;
constexpr int BQ = 128;  // rows of the CTA's tile
constexpr int BN = 64;   // width of the streamed blocks
constexpr int THREADS = 192;
constexpr int T128 = 128 * 128;  // 128 rows x 128 bytes
constexpr int T64 = 64 * 128;    // 64 rows x 128 bytes
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
// 1 / sqrt(head dim), and in base-2 units
template <int HD> constexpr float SCALE = HD == 64 ? 0.125f : HD == 32 ? 0.17677669529663687f : 0.25f;
template <int HD> constexpr float SCALE2 = SCALE<HD> * LOG2E;

// Grid (band, tiles, bands): blockIdx.x is a (batch, head) pair within a band
// of BAND pairs, y the tile (heaviest first), z the band.  The hardware hands
// CTAs out x fastest, so a band's pairs go out together, every pair's heaviest
// tile first: the short tiles fill the gaps at the band's end while the next
// band starts, and the operands of a band's pairs (256 KB a pair, read by all
// its tiles) stay in L2 while it runs, so each kernel reads them from DRAM
// about once.  Slots past the last pair return at once.
constexpr int BAND = 64;

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
    return (uint8_t*)(((uintptr_t)p + 1023) & ~(uintptr_t)1023);
}

// 2^x by the single hardware instruction (relative error ~2^-22)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The next kernel may start once every CTA of this one has its tensor memory: a CTA
// of the next that takes tensor memory and then waits for this kernel's end would
// otherwise hold what this one still needs.  Causal, the set-up overlaps the previous
// kernel's end, and global memory is touched only from here on; groups have waited at
// the top, for their lists.
template <bool GRP> __device__ __forceinline__ void enter_after_setup() {
    if (GRP) pdl_trigger();
    else pdl_enter();
}

__device__ __forceinline__ void init_done() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// One lane of a converged warp, and a value that all its lanes have.  A branch on
// elect.sync, over operands the compiler knows as the warp's, lets a tcgen05.mma take
// them from uniform registers: alone on the SM, 64 x 16 from tensor memory 33 cycles
// each, by `lane == 0` 47 (from shared memory, 48 cycles of reading, 50 and 53).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}\n" : "=r"(p));
    return p != 0;
}
template <typename T> __device__ __forceinline__ T uniform(T v) { return __shfl_sync(0xffffffffu, v, 0); }

// Descriptors of the tiles' first K step, formed once; the next K step of a K-major
// tile is 32 bytes on, of an MN-major one 16 rows, the next stage T64 bytes.
__device__ __forceinline__ uint64_t kmajor(uint32_t saddr) { return sdesc(saddr, 16, 1024); }
__device__ __forceinline__ uint64_t mnmajor(uint32_t saddr) { return sdesc(saddr, T64, 1024); }
constexpr uint32_t DESC_T64 = T64 >> 4;

// The 64-wide blocks that a 128-row tile of queries (keys) goes past, and which
// of them are masked: causal attention over T positions, or a group.
template <bool GRP> struct Tile;
template <> struct Tile<false> {
    int qt, end, n;
    __device__ __forceinline__ Tile(const int32_t*, int, int, int T, int qt_)
        : qt(qt_), end(T), n(min(2 * qt_ + 2, (T + BN - 1) / BN)) {}
    __device__ __forceinline__ int block(int j) const { return j; }
    __device__ __forceinline__ bool masked(int j, int) const { return j >= 2 * qt; }
    __device__ __forceinline__ void check(int, int, int, int*) const {}
    __device__ __forceinline__ int start_of(int) const { return 0; }
    __device__ __forceinline__ unsigned long long keys(int, int, int) const { return 0; }
};
template <> struct Tile<true> : group::Group {
    group::QueryTile t;  // unused where the tile is padding
    int n;
    __device__ __forceinline__ Tile(const int32_t* starts, int b, int K, int T, int qt) : group::Group(starts, b, K, T) {
        if (qt * BQ >= end) return;
        t = group::QueryTile(*this, qt * BQ, BQ);
        n = t.n;
    }
    __device__ __forceinline__ int block(int j) const { return t.block(j); }
    __device__ __forceinline__ bool masked(int, int k0) const { return t.masked(k0); }
};
template <bool GRP> struct KTile;
template <> struct KTile<false> {
    int end, n;
    __device__ __forceinline__ KTile(const int32_t*, int, int, int T, int kt) : end(T), n((T + BN - 1) / BN - 2 * kt) {}
    __device__ __forceinline__ bool masked(int i, int) const { return i < 2; }
    __device__ __forceinline__ int end_of(int) const { return 0; }
    __device__ __forceinline__ unsigned long long queries(int, int, int) const { return 0; }
};
template <> struct KTile<true> : group::Group {
    group::KeyTile t;  // unused where the tile is padding
    int n;
    __device__ __forceinline__ KTile(const int32_t* starts, int b, int K, int T, int kt) : group::Group(starts, b, K, T) {
        if (kt * BQ >= end) return;
        t = group::KeyTile(*this, kt * BQ, BQ);
        n = t.n;
    }
    __device__ __forceinline__ bool masked(int, int q0) const { return t.masked(q0); }
};

// A head's columns at `col` of the rows first..last - 1 of a tile of padding, and
// their column sums, where they are wanted (bpart: the tile's row of 3C)
template <int HD>
__device__ __forceinline__ void clear_padding(bf16* dqkv, int row0, int first, int last, int C, int col, float* bpart) {
    constexpr int G = HD / 8;
    for (int i = first * G + (int)threadIdx.x; i < last * G; i += blockDim.x)
        reinterpret_cast<uint4*>(dqkv + (long long)(row0 + i / G) * 3 * C + col)[i % G] = make_uint4(0, 0, 0, 0);
    if (bpart && threadIdx.x < HD) bpart[col + threadIdx.x] = 0.0f;
}

// the rows from `from` on of a 64-row tile are cleared by `threads` threads
__device__ __forceinline__ void clear_rows(uint8_t* tile, int from, int tid, int threads) {
    for (int i = from * 8 + tid; i < BN * 8; i += threads) reinterpret_cast<uint4*>(tile)[i] = make_uint4(0, 0, 0, 0);
}

// tensor-memory column of the A operand for K step k (16 elements) of a
// 64-wide bf16 operand written as two 16-column halves 32 columns apart
__device__ __forceinline__ uint32_t split_a_col(int k) { return (uint32_t)(8 * k + (k >= 2 ? 16 : 0)); }

// N columns of an output row
template <bool F16, int N>
__device__ __forceinline__ void store_out(bf16* dst, const uint32_t (&w)[N], float scale) {
    uint4* o = reinterpret_cast<uint4*>(dst);
#pragma unroll
    for (int i = 0; i < N / 8; i++)
        o[i] = make_uint4(pack2<F16>(__uint_as_float(w[8 * i]) * scale, __uint_as_float(w[8 * i + 1]) * scale),
                          pack2<F16>(__uint_as_float(w[8 * i + 2]) * scale, __uint_as_float(w[8 * i + 3]) * scale),
                          pack2<F16>(__uint_as_float(w[8 * i + 4]) * scale, __uint_as_float(w[8 * i + 5]) * scale),
                          pack2<F16>(__uint_as_float(w[8 * i + 6]) * scale, __uint_as_float(w[8 * i + 7]) * scale));
}
template <int N> __device__ __forceinline__ void zero_out(bf16* dst) {
#pragma unroll
    for (int i = 0; i < N / 8; i++) reinterpret_cast<uint4*>(dst)[i] = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// One arrival per warp: every lane has passed its own fences (the caller's
// tcgen05.fence / fence.proxy.async) before lane 0 arrives for the warp.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// ================================================================== forward
// Four CTAs an SM, whose phases fill each other's gaps.  P_j, bf16, replaces S_j in
// tensor memory (its halves 32 columns apart), the A operand of O += P_j V_j; S_{j+1}
// is issued behind that product, so that a row that sees it knows O to be whole, and
// may rescale it in place.  A row keeps 32 of its 64 scores in registers and reads the
// other half again from tensor memory.  Four CTAs leave a thread 80 registers, too
// few for all forms: 68 bytes are spilled in the causal one, 80 over groups with heads
// of 64, 84 with narrower ones (140, 164 and 172 bytes of loads).  It is the faster
// form all the same: three CTAs with P in shared memory took 88 us, this 79.
constexpr int F_Q = 0;
constexpr int F_K = F_Q + T128;     // 2 stages
constexpr int F_V = F_K + 2 * T64;  // 1 stage
constexpr int F_BAR = F_V + T64;
constexpr int F_SMEM = F_BAR + 256 + 1024;
constexpr uint32_t F_TMEM = 128;    // S, P: cols 0..63, O: 64..127

template <bool F16, bool GRP, int HD>
__global__ void __launch_bounds__(THREADS, 4)
k_attn_fwd_tc(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
              bf16* __restrict__ y, float* __restrict__ lse, int T, int C, int H, int nbh, int* flags,
              long long wl, const int32_t* __restrict__ starts, int K) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = align1024(smem_raw);
    uint64_t* bars = (uint64_t*)(sm + F_BAR);
    uint64_t* q_full = bars + 0;
    uint64_t* k_full = bars + 1;   // [2]
    uint64_t* k_empty = bars + 3;  // [2]
    uint64_t* v_full = bars + 5;
    uint64_t* v_empty = bars + 6;
    uint64_t* s_full = bars + 7;
    uint64_t* p_full = bars + 8;   // S_j read, P_j in tensor memory
    uint64_t* o_full = bars + 9;   // the last product done
    uint64_t* drain = bars + 10;   // MMAs issued before an abort are done
    uint32_t* tmem_holder = (uint32_t*)(bars + 11);
    volatile int* abort_flag = (volatile int*)(tmem_holder + 1);

    const int bh = (int)(blockIdx.z * gridDim.x + blockIdx.x);
    if (bh >= nbh) return;  // the last band's unused slots (uniform over the CTA, before any setup)
    const int nqt = gridDim.y;
    const int qt = nqt - 1 - (int)blockIdx.y;  // longest rows first within the band
    const int b = bh / H, h = bh % H;
    const int row0 = b * T;
    // the head's columns, the 64 that are loaded, its place among them
    const int hc = h * HD, hx = hc & ~63, co = HD == 64 ? 0 : hc & 63;
    constexpr float SL2 = SCALE2<HD>;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (GRP) pdl_wait();  // the lists of starts are read from here on
    const Tile<GRP> tile(starts, b, K, T, qt);
    if (GRP) {
        if (qt == 0 && h == 0) tile.check(threadIdx.x, THREADS, T, flags);
        if (tile.end <= qt * BQ) {  // padding only (uniform over the CTA)
            const int last = min(qt * BQ + BQ, T);
            constexpr int G = HD / 8;
            for (int i = qt * BQ * G + threadIdx.x; i < last * G; i += THREADS)
                reinterpret_cast<uint4*>(y + (long long)(row0 + i / G) * C + hc)[i % G] = make_uint4(0, 0, 0, 0);
            for (int q = qt * BQ + threadIdx.x; q < last; q += THREADS) lse[((long long)b * H + h) * T + q] = 0.0f;
            return;
        }
    }
    const int nkv = tile.n;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(&k_full[0], 1);
        mbar_init(&k_full[1], 1);
        mbar_init(&k_empty[0], 1);
        mbar_init(&k_empty[1], 1);
        mbar_init(v_full, 1);
        mbar_init(v_empty, 1);
        mbar_init(s_full, 1);
        mbar_init(p_full, 4);
        mbar_init(o_full, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        init_done();
    }
    if (warp == 1) tmem_alloc(tmem_holder, F_TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_holder);
    enter_after_setup<GRP>();

    if (warp == 0) {
        if (elect_one()) {
            const int xq = hx, xk = C + hx, xv = 2 * C + hx;
            mbar_expect_tx(q_full, T128);
            tma_load_2d(smem_u32(sm + F_Q), &tq, q_full, xq, row0 + qt * BQ);
            // K runs two blocks ahead of V: K_{j+2} needs only S_j done, while
            // V_{j+1} has to wait for P_j V_j (V has one buffer)
            int issued_k = 0, issued_v = 0;
            bool ok = true;
            auto load_k = [&](int j) -> bool {
                const int st = j & 1;
                if (!mbar_wait(&k_empty[st], ((j >> 1) & 1) ^ 1, abort_flag, flags, 0x100 + 1, wl)) return false;
                mbar_expect_tx(&k_full[st], T64);
                tma_load_2d(smem_u32(sm + F_K + st * T64), &tk, &k_full[st], xk, row0 + tile.block(j) * BN);
                ++issued_k;
                return true;
            };
            ok = load_k(0) && (nkv < 2 || load_k(1));
            for (int j = 0; j < nkv && ok; j++) {
                if (!mbar_wait(v_empty, (j & 1) ^ 1, abort_flag, flags, 0x100 + 2, wl)) { ok = false; break; }
                mbar_expect_tx(v_full, T64);
                tma_load_2d(smem_u32(sm + F_V), &tk, v_full, xv, row0 + tile.block(j) * BN);
                ++issued_v;
                if (j + 2 < nkv && !load_k(j + 2)) { ok = false; break; }
            }
            if (!ok) {  // let issued copies land before the CTA exits
                mbar_drain(q_full, 0);
                for (int j = (issued_k > 2 ? issued_k - 2 : 0); j < issued_k; j++)
                    mbar_drain(&k_full[j & 1], (j >> 1) & 1);
                if (issued_v > 0) mbar_drain(v_full, (issued_v - 1) & 1);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t ID = idesc16<F16>(BQ, BN, false, false);
            constexpr uint32_t ID_O = idesc16<F16>(BQ, D, false, true);
            const uint64_t dq = kmajor(smem_u32(sm + F_Q) + 2 * co), dv = mnmajor(smem_u32(sm + F_V)),
                           dk = kmajor(smem_u32(sm + F_K) + 2 * co);
            bool ok = mbar_wait(q_full, 0, abort_flag, flags, 0x100 + 3, wl);
            bool issued = false;
            auto issue_s = [&](int j) -> bool {  // overwrites P_{j-1}, read by MMAs issued before
                const int st = j & 1;
                if (!mbar_wait(&k_full[st], (j >> 1) & 1, abort_flag, flags, 0x100 + 4, wl)) return false;
                tc_fence_after();
                const uint64_t dks = dk + st * DESC_T64;
#pragma unroll
                for (int k = 0; k < HD / 16; k++) umma_bf16(tmem, dq + 2 * k, dks + 2 * k, ID, k > 0);
                issued = true;
                umma_commit(s_full);
                umma_commit(&k_empty[st]);
                return true;
            };
            if (ok) ok = issue_s(0);
            for (int j = 0; j < nkv && ok; j++) {
                if (!mbar_wait(v_full, j & 1, abort_flag, flags, 0x100 + 7, wl)) { ok = false; break; }
                if (!mbar_wait(p_full, j & 1, abort_flag, flags, 0x100 + 6, wl)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < BN / 16; k++)
                    umma_bf16_ts(tmem + BN, tmem + split_a_col(k), dv + 128 * k, ID_O, (j > 0 || k > 0) ? 1u : 0u);
                umma_commit(v_empty);
                if (j + 1 < nkv && !issue_s(j + 1)) { ok = false; break; }
            }
            if (ok) umma_commit(o_full);
            if (!ok && issued) {  // the MMAs already issued finish before tensor memory is freed
                umma_commit(drain);
                mbar_drain(drain, 0);
            }
        }
    } else {
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const int q = qt * BQ + r;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
        // P is taken relative to a reference max m that is raised -- and O, l
        // rescaled in place -- only when some row of the warp exceeds it by
        // more than 8 (P <= 2^8 otherwise); the decision is a warp vote since
        // the TMEM loads and stores of O are warp-collective.  Rows that are no
        // result (padding, and the next sequence's rows in a tile that runs past
        // its own) have no vote: the rows beside them would be rounded otherwise
        // (GRP: a row may see nothing of its first blocks; m then starts below
        // any score, but finite, so that no difference is infinity minus infinity)
        float m = GRP ? -3e38f : -INFINITY, l = 0.0f;
        bool ok = true;
        const int st0 = GRP ? tile.start_of(q) : 0;
        for (int j = 0; j < nkv; j++) {
            if (!mbar_wait_warp(s_full, j & 1, abort_flag, flags, 0x100 + 8, wl)) { ok = false; break; }
            tc_fence_after();
            const int kb = tile.block(j) * BN;
            const bool diag = tile.masked(j, kb);
            const int kq = q - kb;  // on the diagonal, key columns > kq are masked
            const unsigned long long seen = GRP && diag ? tile.keys(q, st0, kb) : 0ull;
            const uint32_t seen0 = (uint32_t)seen, seen1 = (uint32_t)(seen >> 32);
            uint32_t w[32];
            // row max over four independent chains (max is exact in any order), the
            // second half of the columns first
            float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 1; c >= 0; c--) {
                tmem_ld32(tl + 32 * c, w);
                if (!diag) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)  // two values an instruction
#pragma unroll
                        for (int u = 0; u < 4; u++)
                            mq[u] = fmaxf(fmaxf(mq[u], __uint_as_float(w[e + 2 * u])), __uint_as_float(w[e + 2 * u + 1]));
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e++)
                        if (GRP ? (c ? seen1 : seen0) >> e & 1u : 32 * c + e <= kq) mq[e & 3] = fmaxf(mq[e & 3], __uint_as_float(w[e]));
                }
            }
            const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
            const float mn = fmaxf(m, mx * SL2);
            const bool rescale = j > 0 && __any_sync(0xffffffffu, q < tile.end && mn > m + 8.0f);
            const float m_old = m;
            if (j == 0 || rescale) m = mn;
            // P = 2^(s*scale - m) as bf16, each 32-column half over its scores
            // (packed fp32x2 scale-and-subtract and sums: two lanes per instruction;
            // the sums in two independent packed chains)
            float2 rsa = make_float2(0.0f, 0.0f), rsb = make_float2(0.0f, 0.0f);
            const float2 sl2 = make_float2(SL2, SL2), nm = make_float2(-m, -m);
            auto probabilities = [&](auto masked) {
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    if (c) tmem_ld32(tl + 32, w);
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 x = __ffma2_rn(make_float2(__uint_as_float(w[e]), __uint_as_float(w[e + 1])), sl2, nm);
                        float2 p = make_float2(ex2(x.x), ex2(x.y));
                        if (GRP && masked.value) {
                            if (!((c ? seen1 : seen0) >> e & 1u)) p.x = 0.0f;
                            if (!((c ? seen1 : seen0) >> (e + 1) & 1u)) p.y = 0.0f;
                        } else if (masked.value) {
                            if (32 * c + e > kq) p.x = 0.0f;
                            if (32 * c + e + 1 > kq) p.y = 0.0f;
                        }
                        if (e & 2) rsb = __fadd2_rn(rsb, p);
                        else rsa = __fadd2_rn(rsa, p);
                        pk[e >> 1] = pack2<F16>(p.x, p.y);
                    }
                    tmem_st16(tl + 32 * c, pk);
                }
            };
            if (diag) probabilities(std::true_type{});
            else probabilities(std::false_type{});
            const float rs = (rsa.x + rsb.x) + (rsa.y + rsb.y);
            if (rescale) {  // O holds P_{j-1} V_{j-1}, which S_j was issued behind
                const float corr = ex2(m_old - m);
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    tmem_ld32(tl + BN + 32 * c, w);
#pragma unroll
                    for (int d = 0; d < 32; d++) w[d] = __float_as_uint(__uint_as_float(w[d]) * corr);
                    tmem_st32(tl + BN + 32 * c, w);
                }
                l *= corr;
            }
            l += rs;
            if (GRP && j == nkv - 1 && kb + BN > tile.end) {
                // V_j has arrived once its barrier's phase is over; the phase before
                // it is: S_j was issued behind P_{j-1} V_{j-1}
                if (!mbar_wait_warp(v_full, j & 1, abort_flag, flags, 0x100 + 13, wl)) {
                    ok = false;
                    break;
                }
                clear_rows(sm + F_V, tile.end - kb, threadIdx.x - 64, 128);
                fence_proxy_async_smem();
            }
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(p_full, lane);
        }
        if (ok && mbar_wait_warp(o_full, 0, abort_flag, flags, 0x100 + 11, wl)) {
            tc_fence_after();
            const bool none = GRP && q >= tile.end;
            if (none) m = 0.0f, l = 1.0f;
            bf16* out = y + (long long)(row0 + q) * C + hc;
            constexpr int N = HD < 32 ? HD : 32;
#pragma unroll
            for (int c = 0; c < HD; c += N) {
                uint32_t v[N];
                tmem_ld_cols(tl + BN + co + c, v);
                if (none && q < T) zero_out<N>(out + c);
                else if (q < T) store_out<F16, N>(out + c, v, 1.0f / l);
            }
            if (q < T) {
                lse[((long long)b * H + h) * T + q] = (m + log2f(l)) * LN2;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, F_TMEM);
}

// ================================================================== backward
// Both backward kernels run 320 threads: warp 0 loads by TMA, warp 1 owns the
// tensor memory and issues the MMAs, and warps 2..9 are the row warps.  Two
// row warps share each 32-lane quarter of tensor memory (quarter = warp & 3)
// and split the streamed block's 64 columns: half (warp - 2) >> 2 takes
// columns [32 half, 32 half + 32).  Each thread therefore owns one row and
// 32 columns of the score block.
//
// The 16-bit operand that the row threads produce is written into tensor memory
// and the next MMAs read it from there as their A operand, so the N = 64 products
// read only their B operand from shared memory.  P^T and dS^T of the dK/dV kernel
// go over the scores they were computed from -- half h writes the 16 columns
// [32 h, 32 h + 16) of its own 32.  The next block's score MMAs overwrite those
// columns; they are issued after the MMAs that read them, and one thread's
// tcgen05.mma operations run in issue order.  dS of the dQ kernel has two buffers
// of its own (Q_TDS).
constexpr int BW_THREADS = 320;
constexpr int BW_ROWS = 256;  // row threads

// Named barrier for the 256 row threads only.
__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The tile's column sums of one 32-column output half: each warp's 32 rows by
// warp_colsum32, then the four quarter warps of the half in quarter order
// (cs: [2 halves][4 quarters][32] floats of shared memory).  Reached by all
// 256 row threads; `v` holds zeros for rows that are not valid.
__device__ __forceinline__ void tile_colsum(float (&v)[32], float* cs, float* dst, int half, int quarter, int lane) {
    cs[(half * 4 + quarter) * 32 + lane] = warp_colsum32(v, lane);
    rows_sync();
    if (quarter == 0 && dst)
        dst[lane] = cs[(half * 4) * 32 + lane] + cs[(half * 4 + 1) * 32 + lane] + cs[(half * 4 + 2) * 32 + lane] +
                    cs[(half * 4 + 3) * 32 + lane];
    rows_sync();
}

// ------------------------------------------------------------------ dQ
// One CTA per 128 queries (2 CTAs per SM).  S = Q K_j^T and dP = dO V_j^T
// (Q and dO are A operands read from shared memory); the row threads form
// dS = P o (dP - D), P from the saved log-sum-exp, into one of two bf16
// buffers in tensor memory; dQ += dS K_j accumulates in tensor memory.
// D = rowsum(dO o O) is computed here and saved for the dK/dV kernel.
//
// S_{j+1} and dP_{j+1} are issued once the row threads have block j's in
// registers, ahead of dQ_j, and run while those work on it; dS is double-buffered so
// that block j's dS never overwrites the operand of block j - 1's dQ MMAs (done when
// S_{j+1}, issued after them, is).
constexpr int Q_Q = 0;
constexpr int Q_O = Q_Q + T128;          // dO tile
constexpr int Q_KST = 3;                 // K stages: K_j is read by S_j and by dQ_j
constexpr int Q_K = Q_O + T128;
constexpr int Q_V = Q_K + Q_KST * T64;   // 2 stages: V_j is free once dP_j is done
constexpr int Q_DP = Q_V + 2 * T64;      // D partials [2 halves][128 rows]
constexpr int Q_CS = Q_DP + 2 * 128 * 4; // column sums [2 halves][4 quarters][32]
constexpr int Q_BAR = Q_CS + 2 * 4 * 32 * 4;
constexpr int Q_SMEM = Q_BAR + 256 + 1024;
constexpr uint32_t Q_TMEM = 256;         // S 0..63, dP 64..127, dS[2] 128..191, dQ 192..255
constexpr uint32_t Q_TS = 0, Q_TP = 64, Q_TDS = 128, Q_TACC = 192;

template <bool F16, bool GRP, int HD>
__global__ void __launch_bounds__(BW_THREADS, 2)
k_attn_bwd_dq_tc(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const __grid_constant__ CUtensorMap to, const bf16* __restrict__ y,
                 const float* __restrict__ lse, float* __restrict__ Dlt, bf16* __restrict__ dqkv,
                 float* __restrict__ bpart, int T, int C, int H, int nbh, int* flags, long long wl,
                 const int32_t* __restrict__ starts, int K) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = align1024(smem_raw);
    uint64_t* bars = (uint64_t*)(sm + Q_BAR);
    uint64_t* qo_full = bars + 0;
    uint64_t* k_full = bars + 1;    // [3]
    uint64_t* k_empty = bars + 4;   // [3]
    uint64_t* v_full = bars + 7;    // [2]
    uint64_t* v_empty = bars + 9;   // [2]
    uint64_t* s_full = bars + 11;   // S_j, dP_j (and every earlier MMA) done
    uint64_t* ds_full = bars + 12;  // [2] block j's dS written: the rows may be a block ahead of the MMA thread's wait
    uint64_t* acc_full = bars + 14;
    uint64_t* drain = bars + 15;    // MMAs issued before an abort are done
    uint64_t* s_free = bars + 16;   // S_j and dP_j are in registers
    uint32_t* tmem_holder = (uint32_t*)(bars + 17);
    volatile int* abort_flag = (volatile int*)(tmem_holder + 1);

    const int bh = (int)(blockIdx.z * gridDim.x + blockIdx.x);
    if (bh >= nbh) return;
    const int nqt = gridDim.y;
    const int qt = nqt - 1 - (int)blockIdx.y;  // longest rows first within the band
    const int b = bh / H, h = bh % H;
    const int row0 = b * T;
    // the head's columns, the 64 that are loaded, its place among them
    const int hc = h * HD, hx = hc & ~63, co = HD == 64 ? 0 : hc & 63;
    constexpr float SL2 = SCALE2<HD>;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (GRP) pdl_wait();
    const Tile<GRP> tile(starts, b, K, T, qt);
    if (GRP) {
        if (qt == 0 && h == 0) tile.check(threadIdx.x, BW_THREADS, T, flags);
        if (tile.end <= qt * BQ) {
            clear_padding<HD>(dqkv, row0, qt * BQ, min(qt * BQ + BQ, T), C, hc,
                          bpart ? bpart + ((long long)b * nqt + qt) * 3 * C : nullptr);
            return;
        }
    }
    const int nkv = tile.n;

    if (threadIdx.x == 0) {
        mbar_init(qo_full, 1);
        for (int i = 0; i < Q_KST; i++) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(s_full, 1);
        for (int i = 0; i < 2; i++) mbar_init(&ds_full[i], BW_ROWS / 32);
        mbar_init(s_free, BW_ROWS / 32);
        mbar_init(acc_full, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        init_done();
    }
    if (warp == 1) tmem_alloc(tmem_holder, Q_TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_holder);
    enter_after_setup<GRP>();

    if (warp == 0) {
        if (elect_one()) {
            const int xq = hx, xk = C + hx, xv = 2 * C + hx;
            mbar_expect_tx(qo_full, 2 * T128);
            tma_load_2d(smem_u32(sm + Q_Q), &tq, qo_full, xq, row0 + qt * BQ);
            tma_load_2d(smem_u32(sm + Q_O), &to, qo_full, hx, row0 + qt * BQ);
            int issued_k = 0, issued_v = 0;
            bool ok = true;
            for (int j = 0; j < nkv; j++) {
                const int ks = j % Q_KST, kr = j / Q_KST;
                if (!mbar_wait(&k_empty[ks], (kr & 1) ^ 1, abort_flag, flags, 0x200 + 1, wl)) { ok = false; break; }
                mbar_expect_tx(&k_full[ks], T64);
                tma_load_2d(smem_u32(sm + Q_K + ks * T64), &tk, &k_full[ks], xk, row0 + tile.block(j) * BN);
                ++issued_k;
                const int vs = j & 1;
                if (!mbar_wait(&v_empty[vs], ((j >> 1) & 1) ^ 1, abort_flag, flags, 0x200 + 10, wl)) { ok = false; break; }
                mbar_expect_tx(&v_full[vs], T64);
                tma_load_2d(smem_u32(sm + Q_V + vs * T64), &tk, &v_full[vs], xv, row0 + tile.block(j) * BN);
                ++issued_v;
            }
            if (!ok) {  // let issued copies land before the CTA exits
                mbar_drain(qo_full, 0);
                for (int j = (issued_k > Q_KST ? issued_k - Q_KST : 0); j < issued_k; j++)
                    mbar_drain(&k_full[j % Q_KST], (j / Q_KST) & 1);
                for (int j = (issued_v > 2 ? issued_v - 2 : 0); j < issued_v; j++)
                    mbar_drain(&v_full[j & 1], (j >> 1) & 1);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t ID = idesc16<F16>(BQ, BN, false, false);
            constexpr uint32_t ID_Q = idesc16<F16>(BQ, D, false, true);
            const uint64_t dq = kmajor(smem_u32(sm + Q_Q) + 2 * co), dout = kmajor(smem_u32(sm + Q_O) + 2 * co),
                           dk = kmajor(smem_u32(sm + Q_K) + 2 * co), dkt = mnmajor(smem_u32(sm + Q_K)),
                           dv = kmajor(smem_u32(sm + Q_V) + 2 * co);
            bool ok = mbar_wait(qo_full, 0, abort_flag, flags, 0x200 + 2, wl);
            bool issued = false;
            // dQ += dS_j K_j: dS from tensor-memory buffer j & 1, K_j read MN-major
            auto issue_dq = [&](int j) {
                const uint64_t dks = dkt + (j % Q_KST) * DESC_T64;
                const uint32_t ta = tmem + Q_TDS + 32 * (j & 1);
#pragma unroll
                for (int k = 0; k < BN / 16; k++)
                    umma_bf16_ts(tmem + Q_TACC, ta + 8 * k, dks + 128 * k, ID_Q, (j > 0 || k > 0) ? 1u : 0u);
                umma_commit(&k_empty[j % Q_KST]);
            };
            // S_j and dP_j: two independent chains, interleaved
            auto issue_s = [&](int j) {
                const int ks = j % Q_KST, vs = j & 1;
                if (!mbar_wait(&k_full[ks], (j / Q_KST) & 1, abort_flag, flags, 0x200 + 3, wl)) return false;
                if (!mbar_wait(&v_full[vs], (j >> 1) & 1, abort_flag, flags, 0x200 + 11, wl)) return false;
                if (j > 0 && !mbar_wait(s_free, (j - 1) & 1, abort_flag, flags, 0x200 + 4, wl)) return false;
                tc_fence_after();
                const uint64_t dks = dk + ks * DESC_T64, dvs = dv + vs * DESC_T64;
#pragma unroll
                for (int k = 0; k < HD / 16; k++) {
                    umma_bf16(tmem + Q_TS, dq + 2 * k, dks + 2 * k, ID, k > 0);
                    umma_bf16(tmem + Q_TP, dout + 2 * k, dvs + 2 * k, ID, k > 0);
                }
                issued = true;
                umma_commit(s_full);
                umma_commit(&v_empty[vs]);  // V_j is no longer needed
                return true;
            };
            ok = ok && issue_s(0);
            for (int j = 0; j < nkv && ok; j++) {
                // the next block's scores while the row threads work on this one's
                if (j + 1 < nkv && !issue_s(j + 1)) { ok = false; break; }
                if (!mbar_wait(&ds_full[j & 1], (j >> 1) & 1, abort_flag, flags, 0x200 + 5, wl)) { ok = false; break; }
                tc_fence_after();
                issue_dq(j);
            }
            if (ok) {
                umma_commit(acc_full);
            } else if (issued) {  // the MMAs already issued finish before tensor memory is freed
                umma_commit(drain);
                mbar_drain(drain, 0);
            }
        }
    } else {
        const int quarter = warp & 3;
        const int half = (warp - 2) >> 2;
        const int r = quarter * 32 + lane;
        const int q = qt * BQ + r;
        const bool qv = q < tile.end;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
        const long long bhl = (long long)b * H + h;
        float* dpart = reinterpret_cast<float*>(sm + Q_DP);
        bool ok = mbar_wait_warp(qo_full, 0, abort_flag, flags, 0x200 + 6, wl);
        // This thread's half of D = rowsum(dO o O) (half of the head's 16-byte
        // chunks of the swizzled dO row); the two halves meet in shared memory.
        float Dq = 0.0f;
        if (ok) {
            const uint8_t* orow = sm + Q_O + r * 128;
            float part = 0.0f;
            if (qv) {
                const uint4* yr = reinterpret_cast<const uint4*>(y + (long long)(row0 + q) * C + hc + HD / 2 * half);
#pragma unroll
                for (int c = 0; c < HD / 16; c++) {
                    const uint4 a = *reinterpret_cast<const uint4*>(orow + (((co / 8 + HD / 16 * half + c) ^ (r & 7)) << 4));
                    const uint4 bb = yr[c];
                    const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
                    const uint32_t bw[4] = {bb.x, bb.y, bb.z, bb.w};
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        part = fmaf(lo16<F16>(aw[i]), lo16<F16>(bw[i]), part);
                        part = fmaf(hi16<F16>(aw[i]), hi16<F16>(bw[i]), part);
                    }
                }
            }
            dpart[half * 128 + r] = part;
        }
        rows_sync();
        if (ok) {
            Dq = dpart[r] + dpart[128 + r];  // the two halves in a fixed order
            if (qv && half == 0) Dlt[bhl * T + q] = Dq;
        }
        const float Lq = qv ? lse[bhl * T + q] * LOG2E : 0.0f;
        const int st0 = GRP ? tile.start_of(q) : 0;
        for (int j = 0; j < nkv && ok; j++) {
            if (!mbar_wait_warp(s_full, j & 1, abort_flag, flags, 0x200 + 7, wl)) { ok = false; break; }
            tc_fence_after();
            const int kb = tile.block(j) * BN;
            const bool diag = tile.masked(j, kb);
            const int kq = q - kb - 32 * half;  // on the diagonal, this half's columns > kq are masked
            const uint32_t seen = GRP && diag ? (uint32_t)(tile.keys(q, st0, kb) >> (32 * half)) : 0u;
            uint32_t sw[32], pw[32];
            tmem_ld32x2(tl + Q_TS + 32 * half, sw, tl + Q_TP + 32 * half, pw);
            tc_fence_before();
            warp_arrive(s_free, lane);  // the next block's scores may be computed
            // dS = P o (dP - D), packed bf16
            // (packed fp32x2: the same roundings as the scalar fma, sub and mul)
            uint32_t pk[16];
            const float2 sl2 = make_float2(SL2, SL2), nl = make_float2(-Lq, -Lq), nd = make_float2(-Dq, -Dq);
            auto slopes = [&](auto masked) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(sw[e]), __uint_as_float(sw[e + 1])), sl2, nl);
                    const float2 dd = __fadd2_rn(make_float2(__uint_as_float(pw[e]), __uint_as_float(pw[e + 1])), nd);
                    float2 d = __fmul2_rn(make_float2(ex2(x.x), ex2(x.y)), dd);
                    if (GRP && masked.value) {
                        if (!(seen >> e & 1u)) d.x = 0.0f;
                        if (!(seen >> (e + 1) & 1u)) d.y = 0.0f;
                    } else if (masked.value) {
                        if (e > kq) d.x = 0.0f;
                        if (e + 1 > kq) d.y = 0.0f;
                    }
                    pk[e >> 1] = pack2<F16>(d.x, d.y);
                }
            };
            if (diag) slopes(std::true_type{});
            else slopes(std::false_type{});
            tmem_st16(tl + Q_TDS + 32 * (j & 1) + 16 * half, pk);
            tmem_st_wait();
            if (GRP && j == nkv - 1 && kb + BN > tile.end) {  // S_j is done, dS_j K_j is to come
                clear_rows(sm + Q_K + (j % Q_KST) * T64, tile.end - kb, threadIdx.x - 64, BW_ROWS);
                fence_proxy_async_smem();
            }
            tc_fence_before();
            warp_arrive(&ds_full[j & 1], lane);
        }
        float cv[32];
#pragma unroll
        for (int d = 0; d < 32; d++) cv[d] = 0.0f;
        if (ok && mbar_wait_warp(acc_full, 0, abort_flag, flags, 0x200 + 9, wl)) {
            tc_fence_after();
            // half the head's columns a thread, or, narrow heads, all of them by the first half
            constexpr int N = HD < 32 ? HD : 32;
            uint32_t w[N];
            if (HD == 64 || half == 0) {
                tmem_ld_cols(tl + Q_TACC + co + 32 * half, w);
                bf16* out = dqkv + (long long)(row0 + q) * 3 * C + hc + 32 * half;
                if (qv) {
                    store_out<F16, N>(out, w, SCALE<HD>);
#pragma unroll
                    for (int d = 0; d < N; d++) cv[d] = __uint_as_float(w[d]) * SCALE<HD>;
                } else if (GRP && q < T) {
                    zero_out<N>(out);
                }
            }
        }
        if (bpart)  // the qkv bias gradient's partial: this tile's column sums of dQ
            tile_colsum(cv, reinterpret_cast<float*>(sm + Q_CS),
                        bpart + ((long long)b * nqt + qt) * 3 * C + hc + 32 * half, half, quarter, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, Q_TMEM);
}

// ------------------------------------------------------------------ dK, dV
// One CTA per 128 keys (2 CTAs per SM), streaming the query blocks at and
// after the diagonal: S^T = K Q_j^T and dP^T = V dO_j^T (K and V as A operands
// from shared memory), then P^T and dS^T into tensor memory, and
// dV += P^T dO_j, dK += dS^T Q_j (Q_j and dO_j read again as MN-major
// operands) accumulate in tensor memory.  P^T and dS^T are handed over one after the
// other: dV's products and the next block's S^T run while the rows form dS^T, dK's
// and the next dP^T while they take the next block's exponentials.
constexpr int K_K = 0;
constexpr int K_V = K_K + T128;
constexpr int K_ST = 3;                  // Q / dO block stages
constexpr int K_Q = K_V + T128;
constexpr int K_O = K_Q + K_ST * T64;
constexpr int K_LD = K_O + K_ST * T64;   // per stage: -log-sum-exp (base 2) [64], -D [64]
constexpr int K_CS = K_LD + K_ST * 128 * 4;  // column sums [2 halves][4 quarters][32]
constexpr int K_BAR = K_CS + 2 * 4 * 32 * 4;
constexpr int K_SMEM = K_BAR + 256 + 1024;
constexpr uint32_t K_TMEM = 256;         // S^T 0..63, dP^T 64..127, dV 128..191, dK 192..255
constexpr uint32_t K_TS = 0, K_TP = 64, K_TV = 128, K_TK = 192;

template <bool F16, bool GRP, int HD>
__global__ void __launch_bounds__(BW_THREADS, 2)
k_attn_bwd_dkdv_tc(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap to, const float* __restrict__ lse,
                   const float* __restrict__ Dlt, bf16* __restrict__ dqkv, float* __restrict__ bpart, int T,
                   int C, int H, int nbh, int* flags, long long wl, const int32_t* __restrict__ starts, int K) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = align1024(smem_raw);
    uint64_t* bars = (uint64_t*)(sm + K_BAR);
    uint64_t* kv_full = bars + 0;
    uint64_t* qo_full = bars + 1;   // [3]
    uint64_t* qo_empty = bars + 4;  // [3]
    uint64_t* s_full = bars + 7;    // S^T_i (and every earlier MMA) done
    uint64_t* dp_full = bars + 8;   // dP^T_i likewise
    uint64_t* p_full = bars + 9;    // P^T_i written to tensor memory
    uint64_t* ds_full = bars + 10;  // dS^T_i likewise
    uint64_t* acc_full = bars + 11;
    uint64_t* drain = bars + 12;
    uint32_t* tmem_holder = (uint32_t*)(bars + 13);
    volatile int* abort_flag = (volatile int*)(tmem_holder + 1);

    const int bh = (int)(blockIdx.z * gridDim.x + blockIdx.x);
    if (bh >= nbh) return;
    const int kt = (int)blockIdx.y;  // key tile; low tiles see the most query blocks
    const int b = bh / H, h = bh % H;
    const int row0 = b * T;
    // the head's columns, the 64 that are loaded, its place among them
    const int hc = h * HD, hx = hc & ~63, co = HD == 64 ? 0 : hc & 63;
    constexpr float SL2 = SCALE2<HD>;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (GRP) pdl_wait();
    const KTile<GRP> tile(starts, b, K, T, kt);
    if (GRP && tile.end <= kt * BQ) {
        float* brow = bpart ? bpart + ((long long)b * gridDim.y + kt) * 3 * C : nullptr;
        clear_padding<HD>(dqkv, row0, kt * BQ, min(kt * BQ + BQ, T), C, C + hc, brow);
        clear_padding<HD>(dqkv, row0, kt * BQ, min(kt * BQ + BQ, T), C, 2 * C + hc, brow);
        return;
    }
    const int j0 = 2 * kt;
    const int nq = tile.n;

    if (threadIdx.x == 0) {
        mbar_init(kv_full, 1);
        for (int i = 0; i < K_ST; i++) {
            mbar_init(&qo_full[i], 2);  // the copies' and the log-sum-exps'
            mbar_init(&qo_empty[i], 1);
        }
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(p_full, BW_ROWS / 32);
        mbar_init(ds_full, BW_ROWS / 32);
        mbar_init(acc_full, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        init_done();
    }
    if (warp == 1) tmem_alloc(tmem_holder, K_TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_holder);
    enter_after_setup<GRP>();

    if (warp == 0) {
        // The whole warp: one lane starts the copies, all of them bring the block's
        // log-sum-exps and Ds, negated (the rows' packed fma and add take them as
        // addends), so that the row warps, which everything waits for, do not.
        const int xq = hx, xk = C + hx, xv = 2 * C + hx;
        const long long bhl = (long long)b * H + h;
        if (elect_one()) {
            mbar_expect_tx(kv_full, 2 * T128);
            tma_load_2d(smem_u32(sm + K_K), &tq, kv_full, xk, row0 + kt * BQ);
            tma_load_2d(smem_u32(sm + K_V), &tq, kv_full, xv, row0 + kt * BQ);
        }
        int issued = 0;
        bool ok = true;
        for (int i = 0, st = 0; i < nq; i++) {
            const int j = j0 + i;
            float L[2], Dq[2];
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int qq = j * BN + 32 * u + lane;
                L[u] = qq < tile.end ? __ldg(lse + bhl * T + qq) : INFINITY;
                Dq[u] = qq < tile.end ? __ldg(Dlt + bhl * T + qq) : 0.0f;
            }
            if (!mbar_wait_warp(&qo_empty[st], ((i / K_ST) & 1) ^ 1, abort_flag, flags, 0x300 + 1, wl)) { ok = false; break; }
            if (elect_one()) {
                mbar_expect_tx(&qo_full[st], 2 * T64);
                tma_load_2d(smem_u32(sm + K_Q + st * T64), &tk, &qo_full[st], xq, row0 + j * BN);
                tma_load_2d(smem_u32(sm + K_O + st * T64), &to, &qo_full[st], hx, row0 + j * BN);
            }
            ++issued;
            float* ld = reinterpret_cast<float*>(sm + K_LD) + st * 128;
#pragma unroll
            for (int u = 0; u < 2; u++) {
                ld[32 * u + lane] = -(L[u] * LOG2E);
                ld[64 + 32 * u + lane] = -Dq[u];
            }
            warp_arrive(&qo_full[st], lane);
            st = st + 1 == K_ST ? 0 : st + 1;
        }
        if (!ok && lane == 0) {  // let issued copies land before the CTA exits
            mbar_drain(kv_full, 0);
            for (int i = (issued > K_ST ? issued - K_ST : 0); i < issued; i++)
                mbar_drain(&qo_full[i % K_ST], (i / K_ST) & 1);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t ID = idesc16<F16>(BQ, BN, false, false);
            constexpr uint32_t ID_A = idesc16<F16>(BQ, D, false, true);
            const uint64_t dk = kmajor(smem_u32(sm + K_K) + 2 * co), dv = kmajor(smem_u32(sm + K_V) + 2 * co);
            const uint64_t dq = kmajor(smem_u32(sm + K_Q) + 2 * co), dqt = mnmajor(smem_u32(sm + K_Q));
            const uint64_t dout = kmajor(smem_u32(sm + K_O) + 2 * co), doutt = mnmajor(smem_u32(sm + K_O));
            bool ok = mbar_wait(kv_full, 0, abort_flag, flags, 0x300 + 2, wl);
            bool issued = false;
            auto issue_s = [&](int i, int st) {  // overwrites P^T_{i-1}, read by MMAs issued before
                if (!mbar_wait(&qo_full[st], (i / K_ST) & 1, abort_flag, flags, 0x300 + 3, wl)) return false;
                tc_fence_after();
                const uint64_t ds = dq + st * DESC_T64;
#pragma unroll
                for (int k = 0; k < HD / 16; k++) umma_bf16(tmem + K_TS, dk + 2 * k, ds + 2 * k, ID, k > 0);
                issued = true;
                umma_commit(s_full);
                return true;
            };
            auto issue_dp = [&](int st) {  // overwrites dS^T_{i-1} likewise
                const uint64_t ds = dout + st * DESC_T64;
#pragma unroll
                for (int k = 0; k < HD / 16; k++) umma_bf16(tmem + K_TP, dv + 2 * k, ds + 2 * k, ID, k > 0);
                umma_commit(dp_full);
            };
            ok = ok && issue_s(0, 0);
            if (ok) issue_dp(0);
            for (int i = 0, st = 0; i < nq && ok; i++) {
                const int next = st + 1 == K_ST ? 0 : st + 1;
                const uint64_t dos = doutt + st * DESC_T64, dqs = dqt + st * DESC_T64;
                if (!mbar_wait(p_full, i & 1, abort_flag, flags, 0x300 + 4, wl)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < BN / 16; k++)
                    umma_bf16_ts(tmem + K_TV, tmem + K_TS + split_a_col(k), dos + 128 * k, ID_A, (i > 0 || k > 0) ? 1u : 0u);
                if (i + 1 < nq && !issue_s(i + 1, next)) { ok = false; break; }
                if (!mbar_wait(ds_full, i & 1, abort_flag, flags, 0x300 + 5, wl)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < BN / 16; k++)
                    umma_bf16_ts(tmem + K_TK, tmem + K_TP + split_a_col(k), dqs + 128 * k, ID_A, (i > 0 || k > 0) ? 1u : 0u);
                umma_commit(&qo_empty[st]);
                if (i + 1 < nq) issue_dp(next);
                st = next;
            }
            if (ok) umma_commit(acc_full);
            else if (issued) {
                umma_commit(drain);
                mbar_drain(drain, 0);
            }
        }
    } else {
        const int quarter = warp & 3;
        const int half = (warp - 2) >> 2;
        const int r = quarter * 32 + lane;
        const int key = kt * BQ + r;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
        bool ok = true;
        const int kend = GRP && key < tile.end ? tile.end_of(key) : 0;
        for (int i = 0, st = 0; i < nq; i++, st = st + 1 == K_ST ? 0 : st + 1) {
            const int j = j0 + i;
            // -L and -D of this half's queries, read as broadcasts
            const float* sl = reinterpret_cast<const float*>(sm + K_LD) + st * 128 + 32 * half;
            if (!mbar_wait_warp(&qo_full[st], (i / K_ST) & 1, abort_flag, flags, 0x300 + 10, wl)) { ok = false; break; }
            if (!mbar_wait_warp(s_full, i & 1, abort_flag, flags, 0x300 + 6, wl)) { ok = false; break; }
            tc_fence_after();
            const bool diag = tile.masked(i, j * BN);  // else all keys are seen by the whole block
            const int q0 = j * BN + 32 * half;
            const uint32_t seen = GRP && diag ? (uint32_t)(tile.queries(key, kend, j * BN) >> (32 * half)) : 0u;
            // P^T, packed fp32x2 with the scalar operations' roundings; -L and -D
            // from the slice
            float2 p[16];
            {
                uint32_t w[32], pk[16];
                tmem_ld32(tl + K_TS + 32 * half, w);
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 l = *reinterpret_cast<const float4*>(sl + e);
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(w[e]), __uint_as_float(w[e + 1])),
                                                make_float2(SL2, SL2), make_float2(l.x, l.y));
                    const float2 x2 = __ffma2_rn(make_float2(__uint_as_float(w[e + 2]), __uint_as_float(w[e + 3])),
                                                 make_float2(SL2, SL2), make_float2(l.z, l.w));
                    p[e >> 1] = make_float2(ex2(x.x), ex2(x.y));
                    p[(e >> 1) + 1] = make_float2(ex2(x2.x), ex2(x2.y));
                }
                if (diag) {
#pragma unroll
                    for (int e = 0; e < 32; e++)
                        if (GRP ? !(seen >> e & 1u) : q0 + e < key) (e & 1 ? p[e >> 1].y : p[e >> 1].x) = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 16; e++) pk[e] = pack2<F16>(p[e].x, p[e].y);
                tmem_st16(tl + K_TS + 32 * half, pk);
                tmem_st_wait();
            }
            if (GRP && j * BN + BN > tile.end) {  // S^T_i and dP^T_i are done, the products with Q_i and dO_i to come
                if (!mbar_wait_warp(dp_full, i & 1, abort_flag, flags, 0x300 + 7, wl)) { ok = false; break; }
                clear_rows(sm + K_Q + st * T64, tile.end - j * BN, threadIdx.x - 64, BW_ROWS);
                clear_rows(sm + K_O + st * T64, tile.end - j * BN, threadIdx.x - 64, BW_ROWS);
                fence_proxy_async_smem();
            }
            tc_fence_before();
            warp_arrive(p_full, lane);
            // dS^T
            if (!mbar_wait_warp(dp_full, i & 1, abort_flag, flags, 0x300 + 9, wl)) { ok = false; break; }
            tc_fence_after();
            {
                uint32_t w[32], pk[16];
                tmem_ld32(tl + K_TP + 32 * half, w);
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 d = *reinterpret_cast<const float4*>(sl + 64 + e);
                    p[e >> 1] = __fmul2_rn(p[e >> 1], __fadd2_rn(make_float2(__uint_as_float(w[e]), __uint_as_float(w[e + 1])),
                                                                 make_float2(d.x, d.y)));
                    p[(e >> 1) + 1] = __fmul2_rn(p[(e >> 1) + 1], __fadd2_rn(make_float2(__uint_as_float(w[e + 2]), __uint_as_float(w[e + 3])),
                                                                             make_float2(d.z, d.w)));
                }
                if (GRP && diag) {  // dP may be NaN where dO is padding
#pragma unroll
                    for (int e = 0; e < 32; e++)
                        if (!(seen >> e & 1u)) (e & 1 ? p[e >> 1].y : p[e >> 1].x) = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 16; e++) pk[e] = pack2<F16>(p[e].x, p[e].y);
                tmem_st16(tl + K_TP + 32 * half, pk);
                tmem_st_wait();
            }
            tc_fence_before();
            warp_arrive(ds_full, lane);
        }
        const bool got = ok && mbar_wait_warp(acc_full, 0, abort_flag, flags, 0x300 + 8, wl);
        if (got) tc_fence_after();
        bf16* base = dqkv + (long long)(row0 + key) * 3 * C + hc + 32 * half;
        // the qkv bias gradient's partials: this tile's column sums of dV, then dK
        float* brow = bpart ? bpart + ((long long)b * gridDim.y + kt) * 3 * C + hc + 32 * half : nullptr;
#pragma unroll 1
        for (int which = 0; which < 2; which++) {  // 0: dV, 1: dK (times 1/sqrt(HD))
            const float scale = which ? SCALE<HD> : 1.0f;
            float v[32];
#pragma unroll
            for (int d = 0; d < 32; d++) v[d] = 0.0f;
            if (got && (HD == 64 || half == 0)) {
                constexpr int N = HD < 32 ? HD : 32;
                uint32_t w[N];
                tmem_ld_cols(tl + (which ? K_TK : K_TV) + co + 32 * half, w);
                if (key < tile.end) {
                    store_out<F16, N>(base + (which ? C : 2 * C), w, scale);
#pragma unroll
                    for (int d = 0; d < N; d++) v[d] = __uint_as_float(w[d]) * scale;
                } else if (GRP && key < T) {
                    zero_out<N>(base + (which ? C : 2 * C));
                }
            }
            if (brow) tile_colsum(v, reinterpret_cast<float*>(sm + K_CS), brow + (which ? C : 2 * C), half, quarter, lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, K_TMEM);
}

}  // namespace fa5

// bf16 or IEEE-half storage (the caller says which through Launch::f16)
bool attention_tc_eligible(bool bf16, int C, int H) {
    return bf16 && H > 0 && C % H == 0 && C / H == fa5::D && C % 8 == 0;
}

template <bool F16, bool GRP, int HD>
static bool attn_set_smem() {
    static PerDevice done;
    return done.once([] {
        return cudaFuncSetAttribute(fa5::k_attn_fwd_tc<F16, GRP, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    fa5::F_SMEM) == cudaSuccess &&
               cudaFuncSetAttribute(fa5::k_attn_bwd_dq_tc<F16, GRP, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    fa5::Q_SMEM) == cudaSuccess &&
               cudaFuncSetAttribute(fa5::k_attn_bwd_dkdv_tc<F16, GRP, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    fa5::K_SMEM) == cudaSuccess;
    });
}

static dim3 attn_grid(int bh, int tiles) {
    const int band = bh < fa5::BAND ? bh : fa5::BAND;
    return dim3((unsigned)band, (unsigned)tiles, (unsigned)((bh + band - 1) / band));
}

// starts [B, K + 1] (GRP): the groups
template <bool F16, bool GRP, int HD>
static bool attn_fwd_tc(const Launch& L, const void* qkv, void* y, float* lse, int B, int T, int C, int H,
                        const int32_t* starts, int K) {
    CUtensorMap tq, tk;
    if (!tc::make_tmap_bf16(&tq, qkv, 3LL * C, (long long)B * T, 3LL * C, fa5::D, fa5::BQ)) return false;
    if (!tc::make_tmap_bf16(&tk, qkv, 3LL * C, (long long)B * T, 3LL * C, fa5::D, fa5::BN)) return false;
    if (!attn_set_smem<F16, GRP, HD>()) return false;
    const dim3 grid = attn_grid(B * H, (T + fa5::BQ - 1) / fa5::BQ);
    L.count();
    launch_k(L, fa5::k_attn_fwd_tc<F16, GRP, HD>, dim3(grid), dim3(fa5::THREADS), fa5::F_SMEM, tq, tk, (fa5::bf16*)y, lse, T,
             C, H, B * H, L.flags, L.wait_cycles, starts, K);
    return true;
}

template <bool F16, bool GRP, int HD>
static bool attn_bwd_tc(const Launch& L, const void* qkv, const void* y, const float* lse, const void* dy,
                        void* dqkv, int B, int T, int C, int H, float* Dlt, float* bpart, const int32_t* starts, int K) {
    // the maps only move 16-bit elements (no conversion), for bf16 and half alike
    CUtensorMap tq, tk, to128, to64;
    if (!tc::make_tmap_bf16(&tq, qkv, 3LL * C, (long long)B * T, 3LL * C, fa5::D, fa5::BQ)) return false;
    if (!tc::make_tmap_bf16(&tk, qkv, 3LL * C, (long long)B * T, 3LL * C, fa5::D, fa5::BN)) return false;
    if (!tc::make_tmap_bf16(&to128, dy, (long long)C, (long long)B * T, (long long)C, fa5::D, fa5::BQ))
        return false;
    if (!tc::make_tmap_bf16(&to64, dy, (long long)C, (long long)B * T, (long long)C, fa5::D, fa5::BN))
        return false;
    if (!attn_set_smem<F16, GRP, HD>()) return false;
    const dim3 grid = attn_grid(B * H, (T + fa5::BQ - 1) / fa5::BQ);
    L.count();
    launch_k(L, fa5::k_attn_bwd_dq_tc<F16, GRP, HD>, dim3(grid), dim3(fa5::BW_THREADS), fa5::Q_SMEM, tq, tk, to128,
             (const fa5::bf16*)y, lse, Dlt, (fa5::bf16*)dqkv, bpart, T, C, H, B * H, L.flags, L.wait_cycles, starts, K);
    L.count();
    launch_k(L, fa5::k_attn_bwd_dkdv_tc<F16, GRP, HD>, dim3(grid), dim3(fa5::BW_THREADS), fa5::K_SMEM, tq, tk, to64, lse,
             Dlt, (fa5::bf16*)dqkv, bpart, T, C, H, B * H, L.flags, L.wait_cycles, starts, K);
    return true;
}

// the form by storage, by groups and, over those, by the head's width
template <typename F>
static bool attn_form(const Launch& L, bool groups, int hd, F&& f) {
    using std::integral_constant;
    auto by_type = [&](auto grp, auto width) { return L.f16 ? f(std::true_type{}, grp, width) : f(std::false_type{}, grp, width); };
    if (!groups) return by_type(std::false_type{}, integral_constant<int, 64>{});
    if (hd == 64) return by_type(std::true_type{}, integral_constant<int, 64>{});
    if (hd == 32) return by_type(std::true_type{}, integral_constant<int, 32>{});
    return by_type(std::true_type{}, integral_constant<int, 16>{});
}

bool launch_attention_fwd_tc(const Launch& L, const void* qkv, void* y, float* lse, int B, int T, int C, int H,
                             const int32_t* starts, int K) {
    if (L.dry) return true;
    return attn_form(L, starts != nullptr, C / H, [&](auto f16, auto grp, auto hd) {
        return attn_fwd_tc<f16.value, grp.value, hd.value>(L, qkv, y, lse, B, T, C, H, starts, K);
    });
}

bool launch_attention_bwd_tc(const Launch& L, const void* qkv, const void* y, const float* lse, const void* dy, void* dqkv,
                             int B, int T, int C, int H, float* Dlt, float* bpart, const int32_t* starts, int K) {
    if (L.dry) return true;
    return attn_form(L, starts != nullptr, C / H, [&](auto f16, auto grp, auto hd) {
        return attn_bwd_tc<f16.value, grp.value, hd.value>(L, qkv, y, lse, dy, dqkv, B, T, C, H, Dlt, bpart, starts, K);
    });
}

}  // namespace tt
