// group.cuh -- which positions of a group see each other (attn_tc.cu,
// attn_group.cu).  A group is a prompt of P positions, answers that follow it
// independently of each other, and padding from `end` on: position q of the
// answer that begins at a sees keys [0, P) and [a, q], one of the prompt [0, q].
// Seen from a key, the queries are one range: from the key itself to the end of
// its answer, or, for a key of the prompt, to the group's end.
//
// Keys and queries go past a tile in blocks of 64.  A query tile needs the
// prompt's blocks and those from the first answer that it touches to its last
// row; a key tile the blocks up to the end of its last row's answer.  Blocks
// that all rows of the tile see whole are not masked.
#pragma once

#include "tt_internal.h"

namespace tt {
namespace group {

constexpr int BLK = 64;  // width of the streamed blocks

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return max(lo, min(v, hi)); }
// n ones (n <= 0: none, n >= 64: all)
__device__ __forceinline__ unsigned long long ones(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// Every value is clamped into its range, so that a list that does not ascend
// leads to no access outside the group.
struct Group {
    const int32_t* s;
    int K, P, end;
    __device__ __forceinline__ Group(const int32_t* starts, int b, int K_, int T) : s(starts + (long long)b * (K_ + 1)), K(K_) {
        P = clampi(s[0], 0, T);
        end = clampi(s[K], P, T);
    }
    // the last answer that begins at or before position q >= P
    __device__ __forceinline__ int answer_of(int q) const {
        int lo = 0, hi = K;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s[mid] <= q) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
    // where the part that position q belongs to begins
    __device__ __forceinline__ int start_of(int q) const { return q < P ? 0 : clampi(s[answer_of(q)], P, q); }
    // the position behind the last one that sees key k < end
    __device__ __forceinline__ int end_of(int k) const {
        return k < P ? end : clampi(s[min(answer_of(k) + 1, K)], k + 1, end);
    }
    // by the threads of one CTA of the group
    __device__ __forceinline__ void check(int tid, int N, int T, int* flags) const {
        bool bad = tid == 0 && (s[0] < 0 || s[K] > T);
        for (int i = tid; i < K; i += N) bad |= s[i] > s[i + 1];
        if (bad) atomicOr(&flags[FLAG_BAD_TOKEN], 1);
    }
    // the keys of block k0.. that query q, whose part begins at st, sees
    __device__ __forceinline__ unsigned long long keys(int q, int st, int k0) const {
        if (q >= end) return 0ull;
        return ones(min(P, q + 1) - k0) | (ones(q + 1 - k0) & ~ones(st - k0));
    }
    // the queries of block q0.. that see key k, kend = end_of(k)
    __device__ __forceinline__ unsigned long long queries(int k, int kend, int q0) const {
        return k >= end ? 0ull : ones(kend - q0) & ~ones(k - q0);
    }
};

// the key blocks of the query tile [q0, q0 + rows), q0 < end
struct QueryTile {
    int q0, P, npre, skip, n, last_start;
    QueryTile() = default;
    __device__ __forceinline__ QueryTile(const Group& g, int q0_, int rows) : q0(q0_), P(g.P) {
        const int last = min(q0 + rows, g.end) - 1, first_block = g.start_of(q0) / BLK;
        npre = (P + BLK - 1) / BLK;
        skip = max(first_block - npre, 0);
        n = last / BLK + 1 - skip;
        last_start = g.start_of(last);
    }
    __device__ __forceinline__ int block(int j) const { return j < npre ? j : j + skip; }
    __device__ __forceinline__ bool masked(int k0) const {
        return !((k0 + BLK <= P || k0 >= last_start) && k0 + BLK - 1 <= q0);
    }
};

// the query blocks j0, j0 + 1, .. of the key tile [k0, k0 + rows), k0 < end
struct KeyTile {
    int j0, n, last, min_end;
    KeyTile() = default;
    __device__ __forceinline__ KeyTile(const Group& g, int k0, int rows) : j0(k0 / BLK) {
        last = min(k0 + rows, g.end) - 1;
        n = ((k0 < g.P ? g.end : g.end_of(last)) - 1) / BLK + 1 - j0;
        min_end = last < g.P ? g.end : g.end_of(max(k0, g.P));
    }
    __device__ __forceinline__ bool masked(int q0) const { return !(q0 >= last && q0 + BLK <= min_end); }
};

// CTA -> (tile, head, sequence) in a grid of one dimension: bands of 64 (sequence,
// head) pairs, whose keys L2 holds together, and in a band every pair's tile with
// the most work first (the last for queries, the first for keys), so that short
// tiles fill the band's end.
struct Place {
    int tile, h, b;
    __device__ __forceinline__ Place(int tiles, int pairs, int H, bool last_first) {
        constexpr int BAND = 64;
        const int band = blockIdx.x / (tiles * BAND), width = min(BAND, pairs - band * BAND);
        const int i = blockIdx.x - band * tiles * BAND, t = i / width, pair = band * BAND + i % width;
        tile = last_first ? tiles - 1 - t : t;
        b = pair / H;
        h = pair % H;
    }
};

}  // namespace group
}  // namespace tt
