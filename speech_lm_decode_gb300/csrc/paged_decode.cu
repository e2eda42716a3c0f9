// Paged attention for few query rows (single tokens, a handful of tokens of a
// sequence): q3paged_attention's kernel while the new tokens times the q heads
// of a kv head fit a tile or two of tensor-core columns.
//
// Bound by reading K and V once (512 bytes a key and kv head).  A CTA of four
// warps walks its keys in blocks of 16, a warp to a block; K and V go from
// global memory straight into the fragments of mma.m16n8k16, without shared
// memory.  Scores are K q^T and outputs V^T p^T, the keys and the head dimension
// on the 16-row side and the few query rows on the 8-column side.  With the head
// dimension of K and q permuted alike, a lane's 16 bytes of a K row are two
// k-steps of its A fragment; a lane's 16 bytes of two V rows are, after a byte
// permute of each pair, A fragments of 16 output values at a time.  The next
// block's K is requested when the scores are done with this one's and the next V
// when the outputs are, so that loads are always in flight without a second set
// of registers.
//
// fp32 activations take four columns a row: the bf16 parts of q (24 bits,
// exact), whose scores are added up across lanes; the weights enter the second
// product as their three parts the same way, so that fp32 needs no further
// tensor-core work.  bf16 activations multiply the weights in two parts one after
// the other (17 bits), as one part would cost the output as much again as its own
// rounding does; the tensor cores are idle enough (256 tokens: 1 us of 180, 64
// sequences of eight: 84 -> 87).
//
// fp32 pages are multiplied on the CUDA cores, eight lanes a key.
//
// Measured (16 q and 8 kv heads): 256 tokens over 1025..1280 positions, bf16,
// 1.2 GB in 180 us (98 % of the copy rate), fp32 pages 2.4 GB in 345 us; three
// tokens over 30000..65537 (32 and 4 heads) 56 us for 42 us of reading, the
// rest being the join of what 456 CTAs hold of 12 items; 32 fp32 tokens over
// 65..768, 17 us, and one over 228, 8 us, are latencies.  Five to eight rows of
// fp32 activations are two groups that each read the keys (four tokens of 64
// sequences over 2000: 183 us, bf16 86).
#include "common.cuh"
#include "kernels.h"
#include "paged.h"
#include "paged_sched.cuh"
#include "pdl.cuh"

namespace q3 {

namespace {

constexpr int DW = 4;             // warps of a CTA
constexpr int DU = 64;            // keys of a unit
constexpr int d_ctas(int nt) { return nt == 1 ? 3 : 2; }   // resident CTAs of an SM (registers)
constexpr int D_OVER = 0;         // units that an item costs besides its keys (1 was slower on ragged batches)
constexpr int D_MIN_UNITS = D_OVER + 1;

__device__ __forceinline__ uint4 ldg16(const void* p, bool ok) {
    uint4 r;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
        "mov.b32 %3, 0;\n\t@p ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w) : "l"(p), "r"((int)ok));
    return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t*)&v;
}
// transposes an 8 x 8 matrix of bf16 (lane (g, t): row g, columns 2t and 2t+1)
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// part `p` of two values, packed: bf16 parts with x = part 0 + part 1 + part 2 (24 bits); part 3 is zero
__device__ __forceinline__ uint32_t part2(float x0, float x1, int p) {
    const uint32_t h = pack2(x0, x1);
    x0 -= __uint_as_float(h << 16);
    x1 -= __uint_as_float(h & 0xffff0000u);
    const uint32_t m = pack2(x0, x1);
    const uint32_t l = pack2(x0 - __uint_as_float(m << 16), x1 - __uint_as_float(m & 0xffff0000u));
    return p < 2 ? (p == 0 ? h : m) : (p == 2 ? l : 0u);
}

// NT: column tiles of eight; a query row takes one column (bf16 activations) or
// four (the parts of fp32 ones; columns 8 n + 2 p + e hold part p of row 2 n + e).
template <typename TA, typename TK, int NT>
__global__ void __launch_bounds__(DW * 32, d_ctas(NT)) paged_decode_kernel(const PagedAttn a, int grid_max) {
    pdl_wait();
    pdl_trigger();
    constexpr bool F32 = sizeof(TA) == 4, KV32 = sizeof(TK) == 4;
    constexpr int RG = F32 ? 2 * NT : 8 * NT;   // query rows of an item
    const PagedView& c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    __shared__ __align__(16) float so[DW][8 * NT][HD + 4];   // stored two values at a time
    __shared__ float sm_m[DW][RG], sm_l[DW][RG];
    __shared__ int s_last;

    auto units_of = [&](const PagedSeq& q) -> long long {
        if (q.n_new <= 0) return 0;
        const int groups = (q.n_new * c.G + RG - 1) / RG;
        return (long long)c.nkv * groups * (max(1, (q.ctx + DU - 1) / DU) + D_OVER);
    };
    const PagedRange R = paged_range<DW * 32>(a, grid_max, D_MIN_UNITS, D_OVER, units_of);
    if (R.u0 >= R.u1) return;
    const float sl2 = a.scale * 1.4426950408889634f;   // scores in powers of two
    const float slack = fminf(8.f / sl2, 3e38f);       // finite: added to -inf, it has to stay -inf
    int* counters = (int*)a.ws;
    constexpr size_t SLOT = (size_t)RG * (HD + 4);   // outputs, maxima, sums (16-byte rows)
    float* parts = (float*)((char*)a.ws + PAGED_COUNTER_BYTES);
    static_assert(sizeof(so) / sizeof(float) >= (size_t)160 * d_ctas(NT) * RG, "weights of the parts fit");

    int s = R.s;
    PagedSeq q = R.q;
    int nu = max(1, (q.ctx + DU - 1) / DU) + D_OVER, groups = (q.n_new * c.G + RG - 1) / RG;   // units and row groups of a head
    int item = (R.u0 - R.start) / nu;       // head * groups + row group
    int item0 = R.start + item * nu;        // the item's units [item0, item0 + nu)
    auto next_item = [&]() -> bool {
        item0 += nu;
        if (++item < c.nkv * groups) return true;
        if (item0 >= R.u1) return false;
        do { q = paged_seq(a, ++s, false); } while (q.n_new <= 0);
        nu = max(1, (q.ctx + DU - 1) / DU) + D_OVER;
        groups = (q.n_new * c.G + RG - 1) / RG;
        item = 0;
        return true;
    };
    int u = paged_begin(R, item0, item0 + nu), seg_end;
    if (u == item0 + nu && !next_item()) return;
    while (paged_cut(R, item0, item0 + nu, &seg_end)) {
        const int h = item / groups, rg = item - h * groups;
        const int key0 = u == item0 ? 0 : (u - item0 - D_OVER) * DU;
        const int key1 = (int)min((long long)q.ctx, (long long)(seg_end - item0 - D_OVER) * DU);
        const int rows = min(RG, q.n_new * c.G - rg * RG);

        const int nb = (key1 - key0 + 15) >> 4;
        const int32_t* table = c.table + (int64_t)s * c.max_pages;
        const int pmask = (1 << c.page_shift) - 1;
        const int64_t head_off = (int64_t)h * c.head_stride;
        auto page_at = [&](int b) -> int {   // page of block b; < 0: none
            if (b >= nb) return -1;
            const int pg = __ldg(table + ((key0 + b * 16) >> c.page_shift));
            return (unsigned)pg < (unsigned)c.n_pages ? pg : -1;
        };
        if constexpr (KV32) {
            // ---- fp32 pages: eight lanes a key (four of its values out of every 32), four keys a step, the next
            // step's K and V on their way; each group of eight lanes keeps its own maximum, sum and output
            const int grp = lane >> 3, sub = lane & 7;
            const float* kbase = (const float*)c.k + head_off + sub * 4;
            const float* vbase = (const float*)c.v + head_off + sub * 4;
            const int steps = warp < nb ? 4 * ((nb - warp + DW - 1) / DW) : 0;
            uint4 kr[2][4], vr[2][4];
            int pg = -1, pgn = page_at(warp);
            bool lost = false;
            auto load = [&](int buf, int i) {
                const int b = warp + DW * (i >> 2), key = key0 + b * 16 + (i & 3) * 4 + grp;
                if ((i & 3) == 0) { pg = pgn; pgn = page_at(b + DW); lost |= pg < 0; }
                const bool ok = pg >= 0 && key < key1;
                const int64_t off = (int64_t)max(pg, 0) * c.page_stride + (int64_t)(key & pmask) * c.token_stride;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    kr[buf][j] = ldg16(kbase + off + 32 * j, ok);
                    vr[buf][j] = ldg16(vbase + off + 32 * j, ok);
                }
                return pg >= 0;
            };
            bool there[2] = {true, true};
            if (steps > 0) there[0] = load(0, 0);
            float qf[RG][16], o[RG][16], mx[RG], l[RG];
            int lim[RG];
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                const bool row = r < rows;
                const int rr = rg * RG + r, tok = rr / c.G;
                const float* src = (const float*)a.q + (int64_t)(q.row0 + (row ? tok : 0)) * a.q_stride +
                                   (int64_t)(h * c.G + (row ? rr - tok * c.G : 0)) * HD + sub * 4;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 f = row ? *(const float4*)(src + 32 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
                    qf[r][4 * j] = f.x; qf[r][4 * j + 1] = f.y; qf[r][4 * j + 2] = f.z; qf[r][4 * j + 3] = f.w;
                }
                lim[r] = row ? min(q.ctx - q.n_new + tok + 1, key1) : 0;
                mx[r] = -INFINITY;
                l[r] = 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) o[r][j] = 0.f;
            }
            auto compute = [&](int buf, int i) {
                const int key = key0 + (warp + DW * (i >> 2)) * 16 + (i & 3) * 4 + grp;
                float x[RG];
                bool grew = false;
#pragma unroll
                for (int r = 0; r < RG; ++r) {
                    float v = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v = fmaf(qf[r][4 * j], __uint_as_float(kr[buf][j].x), v);
                        v = fmaf(qf[r][4 * j + 1], __uint_as_float(kr[buf][j].y), v);
                        v = fmaf(qf[r][4 * j + 2], __uint_as_float(kr[buf][j].z), v);
                        v = fmaf(qf[r][4 * j + 3], __uint_as_float(kr[buf][j].w), v);
                    }
                    v += __shfl_xor_sync(0xffffffffu, v, 1);
                    v += __shfl_xor_sync(0xffffffffu, v, 2);
                    v += __shfl_xor_sync(0xffffffffu, v, 4);
                    x[r] = there[buf] && key < lim[r] ? v : -INFINITY;
                    grew |= x[r] > mx[r] + slack;
                }
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int r = 0; r < RG; ++r) {
                        const float m = fmaxf(mx[r], x[r]), f = m == -INFINITY ? 1.f : ex2((mx[r] - m) * sl2);
                        mx[r] = m;
                        l[r] *= f;
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[r][j] *= f;
                    }
                }
#pragma unroll
                for (int r = 0; r < RG; ++r) {
                    const float p = ex2(fmaf(x[r], sl2, mx[r] == -INFINITY ? 0.f : -mx[r] * sl2));
                    l[r] += p;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        o[r][4 * j] = fmaf(p, __uint_as_float(vr[buf][j].x), o[r][4 * j]);
                        o[r][4 * j + 1] = fmaf(p, __uint_as_float(vr[buf][j].y), o[r][4 * j + 1]);
                        o[r][4 * j + 2] = fmaf(p, __uint_as_float(vr[buf][j].z), o[r][4 * j + 2]);
                        o[r][4 * j + 3] = fmaf(p, __uint_as_float(vr[buf][j].w), o[r][4 * j + 3]);
                    }
                }
            };
            for (int i = 0; i < steps; i += 2) {      // (a multiple of four)
                there[1] = load(1, i + 1);
                compute(0, i);
                if (i + 2 < steps) there[0] = load(0, i + 2);
                compute(1, i + 1);
            }
            if (lost && lane == 0 && a.err) atomicOr(a.err, ERRB_BOUNDS);
            __syncthreads();   // the previous segment's readers are done
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                float m = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 8));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                const float f = ex2((mx[r] - (m == -INFINITY ? 0.f : m)) * sl2);
                l[r] *= f;
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 8);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 16);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    o[r][j] *= f;
                    o[r][j] += __shfl_xor_sync(0xffffffffu, o[r][j], 8);
                    o[r][j] += __shfl_xor_sync(0xffffffffu, o[r][j], 16);
                }
                if (grp == 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *(float4*)&so[warp][r][32 * j + sub * 4] =
                            make_float4(o[r][4 * j], o[r][4 * j + 1], o[r][4 * j + 2], o[r][4 * j + 3]);
                }
                if (lane == 0) { sm_m[warp][r] = m; sm_l[warp][r] = l[r]; }
            }
        } else {
        // ---- bf16 pages: blocks of 16 keys, lane (g, t) holds K rows g, g + 8 and V rows 2t, 2t+1, 2t+8, 2t+9
        const bf16* kbase = (const bf16*)c.k + head_off + g * c.token_stride + t * 8;
        const bf16* vbase = (const bf16*)c.v + head_off + 2 * t * c.token_stride + g * 8;
        uint4 kr[2][4], vr[4][2];
        auto load_k = [&](int b, int pg) {
            const int kb = key0 + b * 16;
            const bf16* p = kbase + (int64_t)max(pg, 0) * c.page_stride + (int64_t)(kb & pmask) * c.token_stride;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool ok = pg >= 0 && kb + g + 8 * i < key1;
#pragma unroll
                for (int j = 0; j < 4; ++j) kr[i][j] = ldg16(p + j * 32, ok);
                p += 8 * c.token_stride;
            }
        };
        auto load_v = [&](int b, int pg) {
            const int kb = key0 + b * 16;
            const bf16* p = vbase + (int64_t)max(pg, 0) * c.page_stride + (int64_t)(kb & pmask) * c.token_stride;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool ok = pg >= 0 && kb + 2 * t + (i & 1) + 8 * (i >> 1) < key1;
                vr[i][0] = ldg16(p, ok);
                vr[i][1] = ldg16(p + 64, ok);
                p += (i == 1 ? 7 : 1) * c.token_stride;
            }
        };
        int b = warp;
        int pg = page_at(b), pgn = page_at(b + DW);
        if (b < nb) { load_k(b, pg); load_v(b, pg); }

        // ---- query rows into B fragments
        uint32_t qb[NT][8][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = F32 ? 2 * n + (g & 1) : 8 * n + g;
            const bool there = r < rows;
            const int rr = rg * RG + r, tok = rr / c.G;
            const TA* src = (const TA*)a.q + (int64_t)(q.row0 + (there ? tok : 0)) * a.q_stride +
                            (int64_t)(h * c.G + (there ? rr - tok * c.G : 0)) * HD + t * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (F32) {
                    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                    const float4 f0 = there ? *(const float4*)(src + j * 32) : z;
                    const float4 f1 = there ? *(const float4*)(src + j * 32 + 4) : z;
                    const int p = g >> 1;
                    qb[n][2 * j][0] = part2(f0.x, f0.y, p);
                    qb[n][2 * j][1] = part2(f0.z, f0.w, p);
                    qb[n][2 * j + 1][0] = part2(f1.x, f1.y, p);
                    qb[n][2 * j + 1][1] = part2(f1.z, f1.w, p);
                } else {
                    const uint4 w = there ? *(const uint4*)(src + j * 32) : make_uint4(0, 0, 0, 0);
                    qb[n][2 * j][0] = w.x; qb[n][2 * j][1] = w.y;
                    qb[n][2 * j + 1][0] = w.z; qb[n][2 * j + 1][1] = w.w;
                }
            }
        }
        // rows whose softmax the lane follows (columns 2t, 2t+1 of each tile) and the keys they see
        int lim[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = F32 ? 2 * n + e : 8 * n + 2 * t + e;
                lim[n][e] = r < rows ? min(q.ctx - q.n_new + (rg * RG + r) / c.G + 1, key1) : 0;
            }
        const int lim_all = min(q.ctx - q.n_new + rg * RG / c.G + 1, key1);   // keys that every row sees

        float o[NT][2][4][4], mx[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[n][i >> 4][(i >> 2) & 3][i & 3] = 0.f;
            mx[n][0] = mx[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }
        for (; b < nb; b += DW) {
            const int pgnn = page_at(b + 2 * DW);
            const int kb = key0 + b * 16;
            float x[NT][4];   // scores: [key g: rows 2t, 2t+1; key g + 8: rows 2t, 2t+1]
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mma16816(x[n], kr[0][j].x, kr[1][j].x, kr[0][j].y, kr[1][j].y, qb[n][2 * j][0], qb[n][2 * j][1]);
                    mma16816(x[n], kr[0][j].z, kr[1][j].z, kr[0][j].w, kr[1][j].w, qb[n][2 * j + 1][0], qb[n][2 * j + 1][1]);
                }
            }
            if (b + DW < nb) load_k(b + DW, pgn);
            if constexpr (F32) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[n][i] += __shfl_xor_sync(0xffffffffu, x[n][i], 1);
                        x[n][i] += __shfl_xor_sync(0xffffffffu, x[n][i], 2);
                    }
            }
            if (kb + 16 > lim_all || pg < 0) {
                if (pg < 0 && lane == 0 && a.err) atomicOr(a.err, ERRB_BOUNDS);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (pg < 0 || kb + g + 8 * (i >> 1) >= lim[n][i & 1]) x[n][i] = -INFINITY;
            }
            // The maximum that the weights refer to moves only when a score passes it by 2^8, which fp32 sums
            // and the parts of the weights take without loss.
            bool grew = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) grew |= fmaxf(x[n][e], x[n][e + 2]) > mx[n][e] + slack;
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(x[n][e], x[n][e + 2]);
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        m = fmaxf(m, mx[n][e]);
                        f[e] = m == -INFINITY ? 1.f : ex2((mx[n][e] - m) * sl2);   // first keys: 0
                        mx[n][e] = m;
                        l[n][e] *= f[e];
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int z = 0; z < 4; ++z) o[n][i >> 2][i & 3][z] *= f[z & 1];
                }
            }
            // (fp32 activations: the weights' parts are columns of their own; bf16: a second part, what the first leaves)
            uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float m = mx[n][i & 1];
                    p[i] = ex2(fmaf(x[n][i], sl2, m == -INFINITY ? 0.f : -m * sl2));
                    l[n][i & 1] += p[i];
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t h = F32 ? part2(p[2 * i], p[2 * i + 1], t) : pack2(p[2 * i], p[2 * i + 1]);
                    if constexpr (!F32)
                        pl[n][i] = transpose8(pack2(p[2 * i] - __uint_as_float(h << 16), p[2 * i + 1] - __uint_as_float(h & 0xffff0000u)));
                    pb[n][i] = transpose8(h);
                }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint32_t v0[4] = {vr[0][y].x, vr[0][y].y, vr[0][y].z, vr[0][y].w};
                const uint32_t v1[4] = {vr[1][y].x, vr[1][y].y, vr[1][y].z, vr[1][y].w};
                const uint32_t v2[4] = {vr[2][y].x, vr[2][y].y, vr[2][y].z, vr[2][y].w};
                const uint32_t v3[4] = {vr[3][y].x, vr[3][y].y, vr[3][y].z, vr[3][y].w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t a0 = __byte_perm(v0[w], v1[w], 0x5410), a1 = __byte_perm(v0[w], v1[w], 0x7632);
                    const uint32_t a2 = __byte_perm(v2[w], v3[w], 0x5410), a3 = __byte_perm(v2[w], v3[w], 0x7632);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if constexpr (!F32) mma16816(o[n][y][w], a0, a1, a2, a3, pl[n][0], pl[n][1]);
                        mma16816(o[n][y][w], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                    }
                }
            }
            if (b + DW < nb) load_v(b + DW, pgn);
            pg = pgn;
            pgn = pgnn;
        }

        // ---- the four warps' outputs, joined
        __syncthreads();   // the previous segment's readers are done
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[n][e];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                const int r = F32 ? 2 * n + e : 8 * n + 2 * t + e;
                if (g == 0 && (!F32 || t == 0)) { sm_m[warp][r] = mx[n][e]; sm_l[warp][r] = v; }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *(float2*)&so[warp][8 * n + 2 * t + e][64 * (i >> 2) + 8 * g + 2 * (i & 3)] =
                        make_float2(o[n][i >> 2][i & 3][e], o[n][i >> 2][i & 3][e + 2]);
        }
        }
        __syncthreads();
        const bool whole = u == item0 && seg_end == item0 + nu;
        const int ca = paged_cut_first(R, item0), cb = paged_cut_last(R, item0 + nu);   // where it is cut
        float* slot = parts + (size_t)(blockIdx.x * 2 + (blockIdx.x == ca ? 1 : 0)) * SLOT;
        TA* out = (TA*)a.out;
        auto store = [&](int r, float v) {
            const int rr = rg * RG + r, tok = rr / c.G;
            out[(int64_t)(q.row0 + tok) * a.out_stride + (int64_t)(h * c.G + rr - tok * c.G) * HD + tid] = from_f<TA>(v);
        };
        for (int r = 0; r < rows; ++r) {
            float m = sm_m[0][r];
#pragma unroll
            for (int w = 1; w < DW; ++w) m = fmaxf(m, sm_m[w][r]);
            const float ms = m == -INFINITY ? 0.f : m;
            float acc = 0.f, sum = 0.f;
#pragma unroll
            for (int w = 0; w < DW; ++w) {
                const float f = ex2((sm_m[w][r] - ms) * sl2);
                float v;
                if constexpr (F32 && !KV32) {
                    const int col = 8 * (r >> 1) + (r & 1);
                    v = so[w][col][tid] + so[w][col + 2][tid] + so[w][col + 4][tid];
                } else {
                    v = so[w][r][tid];
                }
                acc += f * v;
                sum += f * sm_l[w][r];
            }
            if (whole) {
                store(r, sum != 0.f ? acc / sum : 0.f);
            } else {
                slot[r * HD + tid] = acc;
                if (tid == 0) { slot[RG * HD + r] = m; slot[RG * HD + RG + r] = sum; }
            }
        }
        if (!whole) {
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                s_last = atomicAdd(&counters[ca], 1) == cb - ca;
                if (s_last) counters[ca] = 0;
                __threadfence();
            }
            __syncthreads();
            if (s_last) {
                // weights of the parts (so is free: every thread is past the barriers above), then each warp
                // adds up every fourth part
                const int n = cb - ca + 1;
                float* wt = &so[0][0][0];
                auto part = [&](int i) { return parts + (size_t)((ca + i) * 2 + (i == 0 ? 1 : 0)) * SLOT; };
                const int sub = lane & 15;
                for (int r = warp * 2 + (lane >> 4); r < (rows + 1) / 2 * 2; r += 2 * DW) {   // sixteen lanes a row
                    float m = -INFINITY, sum = 0.f;
                    if (r < rows)
#pragma unroll 3
                        for (int i = sub; i < n; i += 16) {
                            const float v = __ldcg(part(i) + RG * HD + r), l = __ldcg(part(i) + RG * HD + RG + r);
                            const float nm = fmaxf(m, v), ms = nm == -INFINITY ? 0.f : nm;
                            sum = sum * ex2((m - ms) * sl2) + l * ex2((v - ms) * sl2);
                            m = nm;
                            wt[i * RG + r] = v;
                        }
#pragma unroll
                    for (int z = 1; z < 16; z <<= 1) {
                        const float v = __shfl_xor_sync(0xffffffffu, m, z), l = __shfl_xor_sync(0xffffffffu, sum, z);
                        const float nm = fmaxf(m, v), ms = nm == -INFINITY ? 0.f : nm;
                        sum = sum * ex2((m - ms) * sl2) + l * ex2((v - ms) * sl2);
                        m = nm;
                    }
                    if (r < rows) {
                        const float ms = m == -INFINITY ? 0.f : m;
                        for (int i = sub; i < n; i += 16) wt[i * RG + r] = ex2((wt[i * RG + r] - ms) * sl2);
                        if (sub == 0) sm_l[0][r] = sum;
                    }
                }
                __syncthreads();
                float4 acc[RG];
#pragma unroll
                for (int r = 0; r < RG; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                for (int i = warp; i < n; i += DW) {
                    const float* p = part(i) + lane * 4;
#pragma unroll
                    for (int r = 0; r < RG; ++r)
                        if (r < rows) {
                            const float4 v = __ldcg((const float4*)(p + r * HD));
                            const float f = wt[i * RG + r];
                            acc[r].x = fmaf(v.x, f, acc[r].x); acc[r].y = fmaf(v.y, f, acc[r].y);
                            acc[r].z = fmaf(v.z, f, acc[r].z); acc[r].w = fmaf(v.w, f, acc[r].w);
                        }
                }
                __syncthreads();
#pragma unroll
                for (int r = 0; r < RG; ++r)
                    if (r < rows) *(float4*)&so[warp][r][lane * 4] = acc[r];
                __syncthreads();
                for (int r = 0; r < rows; ++r) {
                    const float sum = sm_l[0][r];
                    const float v = so[0][r][tid] + so[1][r][tid] + so[2][r][tid] + so[3][r][tid];
                    store(r, sum != 0.f ? v / sum : 0.f);
                }
            }
        }
        if (seg_end < item0 + nu || !next_item()) return;
        u = item0;
    }
}

template <typename TA, typename TK, int NT>
cudaError_t launch_t(const PagedAttn& a, cudaStream_t st) {
    const int grid = min(device_sm_count(), 160) * d_ctas(NT);
    return launch_pdl(paged_decode_kernel<TA, TK, NT>, grid, DW * 32, 0, st, a, grid);
}

}  // namespace

size_t paged_decode_ws() { return (size_t)PAGED_MAX_CTAS * 2 * 16 * (HD + 4) * sizeof(float); }

// rows of a kv head that one sequence may have: one tile of columns (bf16), two (fp32: the keys are read twice, by
// neighbours of the same L2)
bool paged_decode_takes(const PagedAttn& a) { return (int64_t)a.max_q * a.c.G <= (a.act == Q3_BF16 ? 16 : 8); }

cudaError_t launch_paged_decode(const PagedAttn& a, cudaStream_t st) {
    const int rows = a.max_q * a.c.G;
    if (a.act == Q3_BF16) return rows <= 8 ? launch_t<bf16, bf16, 1>(a, st) : launch_t<bf16, bf16, 2>(a, st);
    if (a.kv == Q3_BF16) return rows <= 2 ? launch_t<float, bf16, 1>(a, st) : launch_t<float, bf16, 2>(a, st);
    return rows <= 2 ? launch_t<float, float, 1>(a, st) : launch_t<float, float, 2>(a, st);
}

}  // namespace q3
