// distill.cu -- distillation from a teacher's top logits, loss and gradient:
//
//   k_distill       a row (or a cluster's slices of one) held on chip
//   k_distill_short rows of up to 1024 logits in a warp's registers
//   k_row_mean      the mean of the row losses (fixed order)
//
// Statistics, sums and losses are fp32.  (distill_stream.cu: the other rows.)
#include "distill.cuh"

namespace tt {
namespace {

using namespace head;

constexpr int CS_MAX = 8;      // CTAs of a cluster (the portable limit)

constexpr int NT = 256;        // threads of a CTA that pass over a row
constexpr int LIST_CTA = 64;   // and those that look after its list

// A row is held on chip, where both passes find it (distill.cuh); listed logits
// that the first must leave out are replaced by -inf there.
//
// What has to be moved is the row in and the gradient out.  A row of 50257
// 16-bit logits (100 KB) is held by one CTA, two CTAs an SM, so that one's
// passes run beside the other's loads.  At
// two exponentials an element and pass the special-function unit (32 a cycle
// and SM) would take 3.1 of the 4.5 us that such a row's traffic takes an SM,
// hence the powers (Sums).  32768 rows, k = 64, tau = 2, with hard labels:
// 1069 us, 6.2 TB/s, 91% of the measured copy rate (8192 half rows with t_lse,
// whose replacement holds up the first pass, 75%); then the rows' own chains
// (barrier, merge, coefficients: about 4 us of a row's 10) are what is left.
// REST: with t_lse, in a kernel of its own (as a flag of one kernel it cost the
// others 5%: 1121 us).  Longer rows
// are cut over a cluster only where there are few of them.

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
        x = at; at += cl ? 2 * CS_MAX * (16 + 8) : 0;
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

// The gradient of every column of the slice.  Each slot is refilled from the
// next row nx (if there is one) once it has been read.
template <typename T, int NT, bool S, bool H, int PW = 0>
__device__ __forceinline__ void grad_pass(const Slice<T>& s, char* buf, T* drow, int V, int tid, bool same_phase,
                                          float m, float ct, float At, float A1, const Slice<T>& nx, bool more) {
    using E = Elem<T>;
    constexpr int P = E::EPG / 2, U = 4;
    uint4* const d0 = reinterpret_cast<uint4*>(drow + s.col(0));  // where slot 0 goes
    const uint4* v = reinterpret_cast<const uint4*>(buf);
    const Grad<T, S, H, PW> grad(m, ct, At, A1);
    if (grad.slow) {
#pragma unroll 1
        for (int i = tid; i < s.n; i += NT) {
            f2 r[P];
            grad.slowly(v[i], r);
            if (same_phase && s.inner(i)) d0[i] = E::pack(r);
            else store_edge(s, i, drow, V, r);
        }
        if (more) fill<T, NT>(nx, buf, tid);
        return;
    }
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
            else store_edge(s, i, drow, V, r);
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
            else store_edge(s, i, drow, V, r);
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
template <typename T, bool CL, bool REST>
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
    float2* s_xo = reinterpret_cast<float2*>(s_x + 2 * CS_MAX);  // [2][cs] off the list, at its own reference
    int* s_flag = reinterpret_cast<int*>(sm + lay.flag);  // the target is on the list
    const int rank = CL ? (int)cluster_rank() : 0, cs = CL ? a.cs : 1;
    const long long first = blockIdx.x / cs, stride = gridDim.x / cs;
    constexpr bool rest = REST;
    const bool soft_on = a.alpha > 0.0f, hard_on = a.targets && a.alpha < 1.0f;
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
            if (!soft_on) sum_pass<T, NT, CL, true, false>(s, buf, tid, LOG2E, ct, lift, none, R, s1, st);
            else if (!hard || p2 == 1) sum_pass<T, NT, CL, false, true>(s, buf, tid, LOG2E, ct, lift, none, R, s1, st);
            else if (p2 == 2) sum_pass<T, NT, CL, true, true, 2>(s, buf, tid, LOG2E, ct, lift, none, R, s1, st);
            else if (p2 == 3) sum_pass<T, NT, CL, true, true, 3>(s, buf, tid, LOG2E, ct, lift, none, R, s1, st);
            else if (p2 == 4) sum_pass<T, NT, CL, true, true, 4>(s, buf, tid, LOG2E, ct, lift, none, R, s1, st);
            else sum_pass<T, NT, CL, true, true>(s, buf, tid, LOG2E, ct, lift, none, R, s1, st);
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
        float Ro = -INFINITY, so = 0.0f;  // the sum off the list at a reference of its own
        if (!CL || warp == 0) {
            const int l = lane & 15;
            const float4 p = l < WARPS ? s_part[par * WARPS + l] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
            R = p.x; s1 = p.y; st = p.z; sl = p.w;
            merge<16>(R, s1, st, sl, ct, hard, rest);
            if (rest && (CL || off_own(st, sl))) {
                if (l < NT / 32) Ro = p.x, so = p.z;  // the other warps have none
                merge<16>(Ro, so, ct);
                if (!CL) st = so;
            } else {
                Ro = R;
            }
        }
        if (CL) {
            if (warp == 0 && lane < cs) {
                const uint32_t at = remote(s_x + par * cs + rank, lane);
                st_remote(at, R);
                st_remote(at + 4, s1);
                st_remote(at + 8, st);
                st_remote(at + 12, sl);
                if (rest) {
                    const uint32_t off = remote(s_xo + par * cs + rank, lane);
                    st_remote(off, Ro);
                    st_remote(off + 4, so);
                }
            }
            cluster_sync();
            const int l = lane & (CS_MAX - 1);
            const float4 p = l < cs ? s_x[par * cs + l] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
            R = p.x; s1 = p.y; st = p.z; sl = p.w;
            merge<CS_MAX>(R, s1, st, sl, ct, hard, rest);
            Ro = R;
            if (rest && off_own(st, sl)) {
                const float2 o = l < cs ? s_xo[par * cs + l] : make_float2(-INFINITY, 0.0f);
                Ro = o.x; st = o.y;
                merge<CS_MAX>(Ro, st, ct);
            }
        }

        const Coefs f(a, s_lw, nlw, rest, soft_on, hard, rest ? s_tl[b] : 0.0f, g_all, R, Ro, s1, st, sl, it,
                      ct);
        const bool soft = f.soft;
        const float m = f.Rp, A1 = f.A1p;
        T* drow = dz ? dz + row * a.ld : nullptr;
        if (dz && worker) {
            // second pass: the gradient
            const float As = soft ? f.At : 0.0f;
            if (soft && hard && p2 == 2)
                grad_pass<T, NT, true, true, 2>(s, buf, drow, V, tid, a.same_phase, m, ct, As, A1, nx, more);
            else if (soft && hard && p2 == 3)
                grad_pass<T, NT, true, true, 3>(s, buf, drow, V, tid, a.same_phase, m, ct, As, A1, nx, more);
            else if (soft && hard && p2 == 4)
                grad_pass<T, NT, true, true, 4>(s, buf, drow, V, tid, a.same_phase, m, ct, As, A1, nx, more);
            else if (soft && hard && p2 != 1)
                grad_pass<T, NT, true, true>(s, buf, drow, V, tid, a.same_phase, m, ct, As, A1, nx, more);
            else if (soft || !hard)
                grad_pass<T, NT, true, false>(s, buf, drow, V, tid, a.same_phase, m, ct, As + A1, 0.0f, nx, more);
            else
                grad_pass<T, NT, false, true>(s, buf, drow, V, tid, a.same_phase, m, ct, 0.0f, A1, nx, more);
            if (rank == cs - 1)
                for (long long c = V + tid; c < a.ld; c += NT) drow[c] = Elem<T>::put(0.0f);
        }
        if (list_warp && soft && rank == 0) {
            float part = 0.0f;
            for (int j = lt; j < k; j += LT) part += f.kl(s_t[j], s_zl[j], R, it);
            part = warp_sum(part);
            if (lane == 0) s_ll[lt >> 5] = part;
        }
        if (worker) {
            cp_commit();
            arrive<2>();  // the second pass's stores come before those of the list
            continue;
        }
        meet<2>();
        if (lt == 0 && rank == 0) a.row_loss[row] = f.loss(a, s_ll, nlw, hard, R, s1, s_zl[k]);
        if (list_warp) {
            for (int j = lt; j < k; j += LT) {
                const int o = s_off[j], c = s_ti[j];
                if (o < 0) continue;
                s_bits[o / (int)sizeof(T) >> 5] = 0;
                if (!dz) continue;
                drow[c] = Elem<T>::put(f.listed(s_t[j], s_zl[j], R, ct, hard, c == y));
            }
        }
        if (lt == 0) {
            if (dz && hard && !*s_flag && s.at(y) >= 0) drow[y] = Elem<T>::put(f.target(s_zl[k], R, ct));
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
// made for long rows), 30400 rows of 1024 102 us (401 us a CTA a row; with t_lse
// at five CTAs an SM and 96 registers 105 us, at four and 122 102 us; 30000 of
// 500 with t_lse at six CTAs 48.8 us, at seven and 72 registers 47.6 us).
constexpr int DS_WARPS = 4;
constexpr uint32_t DS_UNLISTED = 0x7FC0DEADu;  // a NaN that no arithmetic makes

// Columns off the list that need a reference of their own (Coefs; rare): their
// largest logit and their sum, then the gradient, from memory.
template <typename T>
__device__ __noinline__ float2 short_off_sum(const T* zr, const uint32_t* s_lp, int V, float ct) {
    float mo = -INFINITY, su = 0.0f;
    for (int c = threadIdx.x & 31; c < V; c += 32)
        if (s_lp[c] == DS_UNLISTED) mo = fmaxf(mo, Elem<T>::get(zr + c));
    mo = warp_max(mo);
    for (int c = threadIdx.x & 31; c < V; c += 32)
        if (mo != -INFINITY && s_lp[c] == DS_UNLISTED) su += exp_of(Elem<T>::get(zr + c), mo, ct);
    return make_float2(mo, warp_sum(su));
}
template <typename T>
__device__ __noinline__ void short_gradient(const T* zr, T* dr, const uint32_t* s_lp, int V, float m, float mo, float ct,
                                            float Al, float Ao, float ks, float A1, float A1o, int y, float kh) {
    for (int c = threadIdx.x & 31; c < V; c += 32) {
        const uint32_t u = s_lp[c];
        const bool off = u == DS_UNLISTED;
        const float v = Elem<T>::get(zr + c), et = exp_of(v, off ? mo : m, ct);
        float r = off ? Ao * et : Al * et - ks * ex2f(__uint_as_float(u) * LOG2E);
        if (kh != 0.0f) r += (off ? A1o : A1) * exp_of(v, off ? mo : m, LOG2E) - (c == y ? kh : 0.0f);
        dr[c] = Elem<T>::put(r);
    }
}

template <typename T, int E, bool REST>
__global__ void __launch_bounds__(DS_WARPS * 32, E <= 4 ? 8 : E <= 16 ? (REST ? 7 : 6) : REST ? 4 : 5)
k_distill_short(const T* z, T* dz, const DistillArgs a) {
    pdl_enter();
    __shared__ uint32_t s_all[DS_WARPS][32 * E];
    using El = Elem<T>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = a.k, V = a.V;
    uint32_t* s_lp = s_all[warp] + lane;  // the lane's columns at steps of 32
    constexpr bool rest = REST;
    const bool soft_on = a.alpha > 0.0f, hard_on = a.targets && a.alpha < 1.0f;
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
        float st = 0.0f, pr = 0.0f, mo = m;  // mo: the reference of su
        if (soft) {
            su = warp_sum(su);
            sl = warp_sum(sl);
            W = warp_sum(W);
            part = warp_sum(part);
            st = su + sl;
            if (rest && off_own(su, sl)) {
                const float2 o = short_off_sum(zr, s_all[warp], V, ct);
                if (Coefs::ln_off(o.y, st, o.x, m, it) >= OFF_MIN) mo = o.x;
                su = mo == o.x ? o.y : 0.0f;
            }
            if (rest && su > 0.0f) pr = fmaxf(1.0f - W, 0.0f);
        }
        if (lane == 0) {
            float loss = 0.0f;
            if (soft) {
                loss = part + W * logf(st);
                if (pr > 0.0f) loss += pr * (logf(pr) - Coefs::ln_off(su, st, mo, m, it));
                loss *= a.alpha * a.tau * a.tau;
            }
            if (hard) loss += (1.0f - a.alpha) * ((m - zy) + logf(s1));
            a.row_loss[row] = loss;
        }
        if (dz) {
            T* dr = dz + row * a.ld;
            const float ks = g_all * a.alpha * a.tau, kh = hard ? g_all * (1.0f - a.alpha) : 0.0f;
            const float rt = soft ? __fdividef(ks, st) : 0.0f, A1 = hard ? __fdividef(kh, s1) : 0.0f;
            const float Al = (W + pr) * rt, At = pr > 0.0f ? rt * (W + pr - pr * __fdividef(st, su)) : W * rt;
            if (rest && mo < m) {
                short_gradient(zr, dr, s_all[warp], V, m, mo, ct, Al, Al * rescale(mo, m, ct) - ks * __fdividef(pr, su),
                               ks, A1, A1 * rescale(mo, m, LOG2E), hard ? y : -1, kh);
                for (long long c = V + lane; c < a.ld; c += 32) dr[c] = El::put(0.0f);
                __syncwarp();
                continue;
            }
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

// mean of M row losses: each thread adds rows t, t + 1024, ... by compensated
// summation (Kahan 1965: c is what the last addition lost; there may be 2^21 of
// them), the threads' sums meet in a fixed tree (3 us for 32768)
__global__ void __launch_bounds__(1024) k_row_mean(const float* __restrict__ row_loss, int M, float* __restrict__ out,
                                                   int* flags) {
    pdl_enter();
    __shared__ float s_w[32];
    float s = 0.0f, c = 0.0f;
    for (long long i = threadIdx.x; i < M; i += 1024) {
        const float y = row_loss[i] - c, t = s + y;
        c = isfinite(t) ? (t - s) - y : 0.0f;
        s = t;
    }
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

// cs: how many CTAs of two to an SM a row takes at least
template <typename Bytes> bool make_plan(Plan& p, int sms, long long M, int G, int cs, Bytes&& bytes) {
    auto need = [&](int cs, int nbuf) { return bytes((G + cs - 1) / cs, nbuf, cs > 1); };
    p.cs = cs;
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

#define ROW_KERNEL(NAME, CL_, REST_, ...)                            \
    do {                                                      \
        static PerDevice attr;                                \
        if (!allow_smem(attr, NAME<T, CL_, REST_>)) return false;    \
        launch_rows(L, NAME<T, CL_, REST_>, p, __VA_ARGS__);         \
        return true;                                          \
    } while (0)

template <typename T, int E> bool distill_short(const Launch& L, const void* z, void* dz, const DistillArgs& a) {
    L.count();
    const unsigned ctas = (unsigned)std::min((a.M - 1) / DS_WARPS + 1, L.num_sms * 12);
    if (a.t_lse) launch_k(L, k_distill_short<T, E, true>, dim3(ctas), dim3(DS_WARPS * 32), 0, (const T*)z, (T*)dz, a);
    else launch_k(L, k_distill_short<T, E, false>, dim3(ctas), dim3(DS_WARPS * 32), 0, (const T*)z, (T*)dz, a);
    return true;
}

template <typename T> bool distill(const Launch& L, const void* z, void* dz, DistillArgs a) {
    Plan p;
    const int k = a.k;
    if (a.V <= 128) return distill_short<T, 4>(L, z, dz, a);
    if (a.V <= 512) return distill_short<T, 16>(L, z, dz, a);
    if (a.V <= 1024) return distill_short<T, 32>(L, z, dz, a);
    // (64 registers of a row a lane: 2000 rows of 1500 logits 23 us, 20000 rows of 2000 142 us; streamed 17 and 122)
    const int G = row_granules<T>(z, a.ld, a.V);
    a.same_phase = (((uintptr_t)z ^ (uintptr_t)dz) & 15) == 0;
    auto bytes = [k](int Gs, int nbuf, bool cl) { return (size_t)DistillLayout(Gs, nbuf, k, Elem<T>::EPG, cl).total; };
    int cs = 1;  // CTAs of two to an SM that a row takes
    while (cs < CS_MAX && bytes((G + cs - 1) / cs, 1, cs > 1) > SMEM_HALF) cs *= 2;
    // a row of more than one, where there are more than the SMs hold at once
    // (1000 rows of 120000 16-bit logits 194 us by clusters, 107 us streamed;
    // 40 such rows 13 us by clusters, 17 us streamed)
    if (cs > 1 && 2LL * a.M * cs > 3LL * L.num_sms) return distill_stream<T>(L, z, dz, a, G, DL_THREADS);
    // a row of at most 40 KB, where there are more than two to an SM (10000 rows
    // of 3000 16-bit logits 149 us on chip, 61 us streamed; 4000 rows of 20000
    // 93 and 74; from 52 KB on, and with fewer rows, no difference or a loss)
    if (G <= 2560 && a.M > 2 * L.num_sms) return distill_stream<T>(L, z, dz, a, G, 128);
    if (!make_plan(p, L.num_sms, a.M, G, cs, bytes)) return false;
    a.Gs = p.Gs; a.cs = p.cs; a.nbuf = p.nbuf;
    if (p.cs == 1 && a.t_lse) ROW_KERNEL(k_distill, false, true, (const T*)z, (T*)dz, a);
    if (p.cs == 1) ROW_KERNEL(k_distill, false, false, (const T*)z, (T*)dz, a);
    if (a.t_lse) ROW_KERNEL(k_distill, true, true, (const T*)z, (T*)dz, a);
    ROW_KERNEL(k_distill, true, false, (const T*)z, (T*)dz, a);
}

}  // namespace

// distillation: a row is held by at most CS_MAX CTAs, which also need room for the list
bool head_row_ok(tt_dtype dtype, int V) {
    if (dtype != TT_FP32 && dtype != TT_BF16 && dtype != TT_FP16) return false;
    return (long long)V * (dtype == TT_FP32 ? 4 : 2) <= TT_ROW_BYTES_MAX;
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
