// Work split of the paged attention kernels, computed on the device from the
// sequence lengths (the host never sees them).
//
// The keys that the items of a call have to read are numbered as one list of
// units (an item: a kv head and a tile of query rows of one sequence; a unit:
// a fixed number of its keys), of which each of P CTAs takes an equal run.  So
// every CTA has the same amount to read however the lengths differ, and an item
// is cut only at a CTA's ends; a cut that would fall near the item's own ends
// is moved there, as joining costs more than the imbalance.  An item may count
// for `over` units more than it reads, for what it costs besides (its query
// rows, its output).  A CTA has at most two cut items, one that it continues
// (partial slot 0) and one that it begins (slot 1).  The CTAs of a cut item are
// consecutive; each stores its
// unnormalised output, maximum and sum, and the last one to arrive (a counter
// that belongs to the first of them, reset by the last) joins them in CTA
// order, so results do not depend on timing.  No CTA waits for another.
#pragma once
#include "common.cuh"
#include "paged.h"

namespace q3 {

// A sequence as the kernels may use it: rows inside [0, n_tokens), lengths
// inside the table; anything else sets the bounds bit and has no rows (or a
// clamped context).
struct PagedSeq { int row0, n_new, ctx; };

__device__ __forceinline__ PagedSeq paged_seq(const PagedAttn& a, int s, bool report) {
    PagedSeq q;
    q.row0 = a.q_off[s];
    const int end = a.q_off[s + 1], cap = a.c.max_pages << a.c.page_shift;
    q.ctx = a.ctx[s];
    // (the order matters: the difference is formed of offsets in range only, as that of any two may wrap around)
    bool bad = q.row0 < 0 || end < q.row0 || end > a.n_tokens || end - q.row0 > a.max_q;
    q.n_new = bad ? 0 : end - q.row0;
    if (q.n_new > 0 && (q.ctx < 0 || q.ctx > cap)) { bad = true; q.ctx = min(max(q.ctx, 0), cap); }
    if (bad && report && a.err) atomicOr(a.err, ERRB_BOUNDS);
    return q;
}

struct PagedRange {
    int W;              // units of the call (0: nothing to do)
    int P;              // CTAs that share them: the first `extra` take quota + 1, the others quota
    int quota, extra;
    int u0, u1;         // this CTA's
    int snap;           // cuts so near to an item's end move to it
    int start;          // first unit of the sequence of u0
    int s;              // that sequence
    PagedSeq q;
};

// first unit of CTA c, and the CTA that owns unit u
__device__ __forceinline__ int paged_first(const PagedRange& r, int c) { return c * r.quota + min(c, r.extra); }
__device__ __forceinline__ int paged_owner(const PagedRange& r, int u) {
    const int big = r.extra * (r.quota + 1);
    return u < big ? u / (r.quota + 1) : r.extra + (u - big) / r.quota;
}

// The part of item [a, b) that a CTA takes, having come to unit `from` of it;
// false: none, its share ends in front of the item.
__device__ __forceinline__ bool paged_cut(const PagedRange& r, int a, int b, int* end) {
    if (r.u1 <= a) return false;
    *end = b;
    if (r.u1 >= b) return true;
    if (r.u1 - a <= r.snap) return false;
    if (b - r.u1 > r.snap) *end = r.u1;
    return true;
}
// Where a CTA whose share begins inside item [a, b) starts: a, u0, or b (the next item).
__device__ __forceinline__ int paged_begin(const PagedRange& r, int a, int b) {
    return r.u0 - a <= r.snap ? a : b - r.u0 <= r.snap ? b : r.u0;
}
// first and last CTA of a cut item
__device__ __forceinline__ int paged_cut_first(const PagedRange& r, int a) { return paged_owner(r, a + r.snap); }
__device__ __forceinline__ int paged_cut_last(const PagedRange& r, int b) { return paged_owner(r, b - r.snap - 1); }

// This CTA's range.  units(q): units of a sequence, all kv heads.  NT threads
// call it; min_units: units that a CTA gets at least (fewer CTAs then work).
template <int NT, class F>
__device__ __forceinline__ PagedRange paged_range(const PagedAttn& a, int P, int min_units, int over, F units) {
    __shared__ long long warp_sum_s[NT / 32];
    __shared__ int found_start, found_s;
    __shared__ PagedSeq found_q;
    const int n_seqs = a.c.n_seqs;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (n_seqs + NT - 1) / NT;
    const int s0 = min(tid * per, n_seqs), s1 = min(s0 + per, n_seqs);
    long long mine = 0;
    PagedSeq q;
    for (int s = s0; s < s1; ++s) {
        q = paged_seq(a, s, blockIdx.x == 0);
        mine += units(q);
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum_s[warp] = incl;
    __syncthreads();
    long long before = 0, W = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += warp_sum_s[w];
        W += warp_sum_s[w];
    }
    PagedRange r;
    if (W > 0x7fff0000LL) {   // more than 2^31 units (tens of terabytes of keys): not served
        if (tid == 0 && blockIdx.x == 0 && a.err) atomicOr(a.err, ERRB_BOUNDS);
        W = 0;
    }
    r.W = (int)W;
    r.P = min(P, max(1, r.W / min_units));
    r.quota = r.W / r.P;
    r.extra = r.W - r.quota * r.P;
    r.snap = over + min(r.quota / 2, 2);   // (a cut never falls into the `over` units; a quarter was slower at 4 a CTA)
    const int c = blockIdx.x;
    r.u0 = c < r.P ? paged_first(r, c) : r.W;
    r.u1 = c < r.P ? paged_first(r, c + 1) : r.W;
    int start = (int)(before + incl - mine);
    if (r.u0 < r.u1 && start <= r.u0 && r.u0 < start + mine) {
        int s = s0;
        if (s1 - s0 > 1) {
            for (;; ++s) {
                q = paged_seq(a, s, false);
                const int n = (int)units(q);
                if (r.u0 < start + n) break;
                start += n;
            }
        }
        found_s = s;
        found_start = start;
        found_q = q;
    }
    __syncthreads();
    r.s = found_s;
    r.start = found_start;
    r.q = found_q;
    return r;
}

// Items of tpi tokens (of one kv head), units of KEYS keys that their last token
// sees at most, and OVER more; in the order sequence, head, item.
struct Walk {
    PagedSeq q;
    int u, item0;         // unit to begin at, first unit of the item
    int s, h, item, nu;   // nu: units of the item
    bool more;
};

// tokens of an item (tpi) and the key tiles that item i of a sequence reads
template <int KEYS, int OVER>
__device__ __forceinline__ int item_units(const PagedSeq& q, int tpi, int i) {
    const int last = min(q.n_new, (i + 1) * tpi);
    const int vis = min(q.ctx - q.n_new + last, q.ctx);
    return max(1, (vis + KEYS - 1) / KEYS) + OVER;
}
template <int KEYS, int OVER>
__device__ __forceinline__ long long seq_units(const PagedSeq& q, int tpi) {
    long long n = 0;
    for (int i = 0; i * tpi < q.n_new; ++i) n += item_units<KEYS, OVER>(q, tpi, i);
    return n;
}

// on to the next item
template <int KEYS, int OVER>
__device__ __forceinline__ void walk_step(Walk& w, const PagedAttn& a, const PagedRange& R, int tpi) {
    w.item0 += w.nu;
    w.u = w.item0;
    if (w.item0 >= R.u1) { w.more = false; return; }
    if (++w.item * tpi >= w.q.n_new) {
        w.item = 0;
        if (++w.h == a.c.nkv) {
            w.h = 0;
            do { w.q = paged_seq(a, ++w.s, false); } while (w.q.n_new <= 0);
        }
    }
    w.nu = item_units<KEYS, OVER>(w.q, tpi, w.item);
}
template <int KEYS, int OVER>
__device__ __forceinline__ void walk_begin(Walk& w, const PagedAttn& a, const PagedRange& R, int tpi) {
    w.s = R.s;
    w.q = R.q;
    w.more = true;
    const int per = (int)seq_units<KEYS, OVER>(w.q, tpi);
    int rel = R.u0 - R.start;
    w.h = rel / per;
    rel -= w.h * per;
    w.item0 = R.start + w.h * per;
    w.item = 0;
    for (;;) {
        w.nu = item_units<KEYS, OVER>(w.q, tpi, w.item);
        if (rel < w.nu) break;
        rel -= w.nu;
        w.item0 += w.nu;
        ++w.item;
    }
    w.u = paged_begin(R, w.item0, w.item0 + w.nu);
    if (w.u == w.item0 + w.nu) walk_step<KEYS, OVER>(w, a, R, tpi);
}
// Workspace of the paged attention: counters, then two partial slots a CTA.
constexpr int PAGED_MAX_CTAS = 1024;
constexpr size_t PAGED_COUNTER_BYTES = Q3PAGED_COUNTER_BYTES;
static_assert(PAGED_MAX_CTAS * sizeof(int) <= PAGED_COUNTER_BYTES, "a counter for each CTA");

}  // namespace q3
