// Paged attention over 8-bit codes for many query rows (chunks of prompts, mixed
// batches), on the fifth-generation tensor cores.
//
// The items, the two slots and the softmax are those of the kernel over bf16
// pages (paged_chunk.cu): an item is up to 256 query rows of one sequence and kv
// head (fp32 activations: 128), its units are tiles of 128 keys, one persistent
// CTA per SM takes an equal share of all units.  Inside a CTA
//   warp 0       copies tiles of codes into a ring of 16 KB places (TMA, a box a
//                page), and their blocks' scales beside them;
//   warp 1       issues S = Q K^T and O += P V (tcgen05.mma, f16, M = N = 128);
//   warp 2       goes through the pages and scales of the next cut: its largest
//                scales, and whether pages are out of range;
//   warps 4-11   softmax, a warpgroup a slot, a thread a row;
//   warps 12-15  turn codes into f16 tiles in the layout of the products.
// Codes are taken into f16 times their block's scale over the cut's largest one,
// which is exact to a ratio of 2^15 (f16 has steps of 2^-24, codes of 2^-9); the
// largest scale itself multiplies the scores' factor and the outputs, in fp32.
// The conversion runs beside the softmax, and a tile is converted once for 256
// query rows.
// q enters in f16 relative to the power of two above its row's largest value, one
// part (bf16 activations: exact) or two (fp32: 22 bits); weights relative to 2^-7
// of the running maximum, one part (11 bits) or two, each with an output of its own
// as over bf16 pages.
//
// Measured (16 q and 8 kv heads): 4096 tokens over 12288, bf16, 422 us = 1.14
// PFLOP/s (58 % of the measured rate; without the conversion 391, without the
// exponentials no less: what is left is a slot's chain score -> softmax -> output),
// fp32 830; 24 prompts of 1..512 over 0..255, fp32, 83 us; 64 tokens over 32k, bf16,
// 58 us.  Errors against 64 bits: bf16 1.67e-3 of the result (the output's rounding
// is 1.66e-3 of it), fp32 4.5e-7 at those prompts, 1.3e-6 to 1.6e-6 over 1000 to
// 32000 keys (the plain form in fp32: 6.1e-7, 1.0e-6 to 3.5e-6).
//
// Every wait is bounded: one that runs out sets the timeout bit, after which the
// CTA goes through its remaining steps without waiting or issuing, drains its
// copies and products, frees its tensor memory and returns.
#include "common.cuh"
#include "kernels.h"
#include "paged8.h"
#include "paged_sched.cuh"
#include "paged_tc.cuh"

namespace q3 {

namespace {

constexpr int CONV = 4;                    // warps that convert
constexpr int C8_THREADS = 384 + 32 * CONV;
// registers a thread: at launch (the launcher checks it), and of warps 0-3, the softmax and the conversion after they
// have divided them; more than there are would be waited for for ever (128 each: 849 us at 4096 tokens over 12288, as the
// softmax has too few; eight converting warps and 136 registers of the softmax: 482)
constexpr int REGS = 128, REGS_0 = 48, REGS_SOFT = 176, REGS_CONV = 112;
static_assert(128 * REGS_0 + 256 * REGS_SOFT + 32 * CONV * REGS_CONV <= REGS * C8_THREADS, "registers of the CTA");
static_assert(REGS_0 <= REGS && REGS_CONV <= REGS && REGS_SOFT >= REGS, "the former give registers up, the latter take them");
constexpr int ST = 3;                      // f16 tiles (32 KB)
constexpr int RS = 3;                      // tiles of codes (16 KB)
constexpr int RAW = CT * HD;
constexpr int C8_QBYTES = 2 * STAGE;       // Q: of two tiles of rows, or the two parts of one
// fp32 activations: key tiles after which the output leaves the tensor memory for a total in fp32.  Products add to it
// cut off, not rounded, so that it falls behind by as much again with every tile: 1.1e-5 of the result after 120 tiles,
// 2.7e-6 so after every sixteen, 1.6e-6 after every eight (the plain form in fp32: 2.6e-6); 4096 tokens over 12288 take
// 750, 785 and 830 us.
constexpr int FLUSH = 8;
constexpr float P_SHIFT = 7.f;             // weights are 2^7 times exp2 of score - reference (f16 holds 2^-21 of it in full)

struct Chunk8Smem {
    uint64_t full[ST], empty[ST], raw_full[RS], raw_empty[RS], s_full[2], p_full[2], r_full[2], pv_full, q_full, o_full, drain;
    uint64_t mail_full[2], mail_empty[2];
    uint32_t tmem;
    int dead, last;
    // of a cut: its keys have a page out of range among them; bytes of the largest scales of keys and of values
    struct { int lost, kmax, vmax; } mail[2];
    uint8_t scale[RS][8];    // of 16 keys each
    float ref[CT];           // one tile of rows: the maxima that both slots' weights refer to
    float row[2 * CT];       // by which a row's q was divided
    float stats[4][CT];      // one tile of rows: the slots' maxima and sums
    PagedRange range;        // the softmax warps' walk, kept here to save them the registers
    Walk walk;
    Seg seg;
    int more;
};

// of the softmax warps
__device__ __forceinline__ void wg_sync(int id) { asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void expect_tx(uint64_t* b, unsigned bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *(const uint32_t*)&v;
}
// what the f16 part h of two values leaves of them, as f16
__device__ __forceinline__ uint32_t rest2(float x0, float x1, uint32_t h) {
    const float2 f = __half22float2(*(const __half2*)&h);
    return half2_bits(x0 - f.x, x1 - f.y);
}
// f16 of 2^-d, zero from 2^-25 on
__device__ __forceinline__ uint32_t half_two(int d) { return d <= 14 ? (uint32_t)(15 - d) << 10 : d <= 24 ? 1u << (24 - d) : 0u; }

// fp32 D, f16 A and B, M = N = 128; bit 16: B is MN-major
constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(CT >> 3) << 17) | ((uint32_t)(CT >> 4) << 24);
constexpr uint32_t IDESC_V = IDESC | (1u << 16);

template <typename TA>
__global__ void __launch_bounds__(C8_THREADS, 1)
paged8_chunk_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                   const __grid_constant__ Paged8Attn a) {
    constexpr bool F32 = sizeof(TA) == 4;
    constexpr int QP = F32 ? 2 : 1, PP = F32 ? 2 : 1, NX = F32 ? 1 : 2;   // NX: 32 scores of a thread at a time
    // tensor memory: the slots' scores (the weights over them), then outputs: of the two tiles, or (fp32) of the
    // weights' two parts
    constexpr int SLOT = CT, OUT = 2 * SLOT;
    extern __shared__ __align__(1024) unsigned char raw[];
    __shared__ Chunk8Smem sm;
    unsigned char* base = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    unsigned char* qs = base;                       // Q tiles (bf16: per slot; fp32: per part)
    unsigned char* ring = base + C8_QBYTES;
    unsigned char* codes = ring + ST * STAGE;
    const PagedView& c = a.c;
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int tpt = CT / c.G, tpi = F32 ? tpt : 2 * tpt;   // tokens of a tile, of an item
    const uint32_t ginv = 65536u / c.G + 1;                // row / G for rows below 256 and G <= 16: row * ginv >> 16

    const PagedRange R = paged_range<C8_THREADS>(a, gridDim.x, C_MIN_UNITS, C_OVER,
                                                [&](const PagedSeq& q) { return c.nkv * seq_units<CT, C_OVER>(q, tpi); });
    if (R.u0 >= R.u1) return;

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) { bar_init(&sm.full[i], CONV); bar_init(&sm.empty[i], 1); }   // (a warp each)
        for (int i = 0; i < RS; ++i) { bar_init(&sm.raw_full[i], 1); bar_init(&sm.raw_empty[i], CONV); }
        for (int i = 0; i < 2; ++i) { bar_init(&sm.mail_full[i], 1); bar_init(&sm.mail_empty[i], 8 + CONV); }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sm.s_full[i], 1);
            bar_init(&sm.p_full[i], CT / 32);   // a warp each
            bar_init(&sm.r_full[i], CT / 32);
        }
        bar_init(&sm.q_full, 2 * CT);
        bar_init(&sm.o_full, 1);
        bar_init(&sm.pv_full, 1);
        bar_init(&sm.drain, 1);
        sm.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&sm.tmem)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sm.tmem;

    Walk w;
    walk_begin<CT, C_OVER>(w, a, R, tpi);
    if (threadIdx.x == 128) { sm.range = R; sm.walk = w; }

    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_0));
    Seg g;
    if (warp == 0) {
        // ---------------------------------------------------------- tiles of codes
        int cnt = 0, issued = 0;
        bool ok = true;
        const int box = min(1 << c.page_shift, CT), pmask = (1 << c.page_shift) - 1;
        uint32_t byte = 0;      // of lanes 0-7: scales of the last tile, which are put down when the next one's are asked for
        auto put_scales = [&] {
            if (issued == 0) return;
            const int st = (issued - 1) % RS;
            if (lane < 8) sm.scale[st][lane] = (uint8_t)byte;
            __syncwarp();
            if (lane == 0) bar_arrive(&sm.raw_full[st]);
        };
        auto load = [&](const CUtensorMap* map, const uint8_t* scales, int kt) {
            const int st = cnt % RS;
            if (cnt >= RS) ok = ok && bar_wait(&sm.raw_empty[st], (cnt / RS - 1) & 1, sm, a.err);
            if (cnt + 1 == a.inject) {
                give_up(sm, a.err);
                ok = false;
            }
            ok = __all_sync(0xffffffffu, ok);
            ++cnt;
            if (!ok) return;
            const int rows = min(CT, w.q.ctx - kt * CT), nbox = (rows + box - 1) / box;
            // a box a lane (a page has 16 positions at least); a page out of range is not followed: its box lies past the
            // last page, where copies read zeros
            const int key = kt * CT + min(lane, nbox - 1) * box;
            int page = 0;
            bool bad = false;
            if (lane < nbox) {
                page = c.table[(int64_t)g.s * c.max_pages + (key >> c.page_shift)];
                bad = (unsigned)page >= (unsigned)c.n_pages;
            }
            if (bad) {
                if (a.err) atomicOr(a.err, ERRB_BOUNDS);
                page = c.n_pages;
            }
            __syncwarp();
            if (lane == 0) expect_tx(&sm.raw_full[st], (unsigned)(nbox * box * HD));
            __syncwarp();
            if (lane < nbox) tma_4d(su32(codes + (size_t)st * RAW) + lane * box * HD, map, 0, key & pmask, g.h, page, &sm.raw_full[st]);
            put_scales();
            issued = cnt;
            const int from = kt * CT + 16 * (lane & 7), of = __shfl_sync(0xffffffffu, page, 16 * (lane & 7) / box);
            byte = 0;
            if (16 * (lane & 7) < rows && of < c.n_pages)
                byte = __ldg(scales + (((of * c.nkv + g.h) << (c.page_shift - a.block_shift)) + ((from & pmask) >> a.block_shift)));
        };
        while (walk_seg(w, R, tpt, tpi, g)) {
            const int lead = g.two ? 1 : 2;
            for (int i = 0; i < min(lead, g.n); ++i) load(&mapK, a.ks, g.kt0 + i);
            for (int i = 0; i < g.n; ++i) {
                load(&mapV, a.vs, g.kt0 + i);
                if (i + lead < g.n) load(&mapK, a.ks, g.kt0 + i + lead);
            }
            if (w.more) walk_step<CT, C_OVER>(w, a, R, tpi);
        }
        put_scales();
        // nothing may still be writing this CTA's shared memory when it leaves (given up, its last copies are not
        // waited for elsewhere)
        for (int i = max(0, issued - RS); i < issued; ++i) bar_wait(&sm.raw_full[i % RS], (i / RS) & 1, sm, a.err, false);
    } else if (warp == 1) {
        // ---------------------------------------------------------- products
        int cnt = 0, pc[2] = {0, 0}, qc = 0;
        bool ok = true;
        const uint32_t ring0 = su32(ring), q0 = su32(qs);
        auto full = [&](int i) {
            ok = ok && bar_wait(&sm.full[i % ST], (i / ST) & 1, sm, a.err);
            ok = __all_sync(0xffffffffu, ok);
            fence_after();
        };
        auto p_ready = [&](int t) {
            ok = ok && bar_wait(&sm.p_full[t], pc[t] & 1, sm, a.err);
            ++pc[t];
            ok = __all_sync(0xffffffffu, ok);
            fence_after();
        };
        auto release = [&](int i) {
            if (ok && elect_one()) commit(&sm.empty[i % ST]);
            __syncwarp();
        };
        // S of slot t from the K tile of ring entry i
        auto scores = [&](int t, int i) {
            const uint32_t kd = uniform(tile_desc(ring0 + (i % ST) * STAGE, 16));
            const uint32_t qd = uniform(tile_desc(q0 + (!F32 && g.two ? t : 0) * STAGE, 16)), d = uniform(tmem + t * SLOT);
            if (ok && elect_one()) {
#pragma unroll
                for (int p = QP - 1; p >= 0; --p)     // the smallest part first: sums are cut to the bits of the largest term
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t off = ((ks >> 2) * (STAGE / 2) + (ks & 3) * 32) >> 4;
                        umma_ss(d, qd + p * (STAGE >> 4) + off, kd + off, IDESC, p != QP - 1 || ks != 0);
                    }
                commit(&sm.s_full[t]);
            }
            __syncwarp();
        };
        // O of slot t += P V, once P is there
        auto outputs = [&](int t, int i, bool acc) {
            const uint32_t vd = uniform(tile_desc(ring0 + (i % ST) * STAGE, STAGE / 2));
            const uint32_t pa = uniform(tmem + t * SLOT), d = uniform(tmem + OUT + (g.two ? t * CT : 0)), first = uniform(acc);
            p_ready(t);
            if (ok && elect_one()) {
#pragma unroll
                for (int p = 0; p < PP; ++p)
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_ts(d + p * CT, pa + 32 * (ks >> 1) + 16 * p + 8 * (ks & 1), vd + ks * (2048 >> 4), IDESC_V, ks != 0 ? 1u : first);
            }
            __syncwarp();
        };
        while (walk_seg(w, R, tpt, tpi, g)) {
            if (g.n > 0) {
                ok = ok && bar_wait(&sm.q_full, qc & 1, sm, a.err);
                ++qc;
                ok = __all_sync(0xffffffffu, ok);
                fence_after();
                const int lead = g.two ? 1 : 2;
                const int first = min(lead, g.n);
                for (int i = 0; i < first; ++i) {
                    full(cnt);
                    scores(g.two ? 0 : i, cnt);
                    if (g.two) scores(1, cnt);
                    release(cnt);
                    ++cnt;
                }
                for (int i = 0; i < g.n; ++i) {
                    const int v = cnt, k = cnt + 1;
                    const bool more = i + lead < g.n;
                    full(v);
                    if (g.two) {
                        outputs(0, v, i > 0);
                        if (more) { full(k); scores(0, k); }
                        outputs(1, v, i > 0);
                        release(v);
                        if (more) { scores(1, k); release(k); }
                    } else {
                        const int t = i & 1;
                        outputs(t, v, F32 ? i % FLUSH != 0 : i > 0);
                        if (ok && elect_one()) commit(&sm.pv_full);
                        __syncwarp();
                        release(v);
                        if (more) { full(k); scores(t, k); release(k); }
                    }
                    cnt += more ? 2 : 1;
                }
                if (ok && elect_one()) commit(&sm.o_full);
                __syncwarp();
            }
            if (w.more) walk_step<CT, C_OVER>(w, a, R, tpi);
        }
        // products in flight end before the tensor memory goes (they have, unless the softmax warps gave up on them)
        if (elect_one()) {
            commit(&sm.drain);
            bar_wait(&sm.drain, 0, sm, a.err, false);
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------- pages and scales of a cut, ahead of the others
        bool ok = true;
        for (int k = 0; walk_seg(w, R, tpt, tpi, g); ++k) {
            if (k >= 2) ok = ok && bar_wait(&sm.mail_empty[k & 1], (k / 2 - 1) & 1, sm, a.err);
            ok = __all_sync(0xffffffffu, ok);
            const int32_t* row = c.table + (int64_t)g.s * c.max_pages;
            const int k0 = g.kt0 * CT, k1 = g.n > 0 ? min((g.kt0 + g.n) * CT, w.q.ctx) : k0, bs = a.block_shift;
            bool bad = false;
            int kmax = 0, vmax = 0;
            if (k0 < k1)
#pragma unroll 4
                for (int i = (k0 >> bs) + lane; i <= (k1 - 1) >> bs; i += 32) {
                    const int page = row[i << bs >> c.page_shift];
                    if ((unsigned)page >= (unsigned)c.n_pages) { bad = true; continue; }
                    const int at = ((page * c.nkv + g.h) << (c.page_shift - bs)) + (i & ((1 << (c.page_shift - bs)) - 1));
                    const int kb = __ldg(a.ks + at), vb = __ldg(a.vs + at);
                    if (kb != 255) kmax = max(kmax, kb);
                    if (vb != 255) vmax = max(vmax, vb);
                }
            bad = __any_sync(0xffffffffu, bad);
            kmax = __reduce_max_sync(0xffffffffu, kmax);
            vmax = __reduce_max_sync(0xffffffffu, vmax);
            if (lane == 0) {
                sm.mail[k & 1] = {bad, kmax, vmax};
                bar_arrive(&sm.mail_full[k & 1]);
            }
            __syncwarp();
            if (w.more) walk_step<CT, C_OVER>(w, a, R, tpi);
        }
    }
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_CONV));
        // ---------------------------------------------------------- codes to f16 tiles
        Seg g;
        bool ok = true;
        int cnt = 0;
        // Eight lanes take half a row each of two rows, so that neither their loads nor their stores meet a bank twice.
        const int half = lane >> 2 & 1, row0 = (warp - 12) * (CT / CONV) + (lane >> 3) * 2 + half;
        int src[2], dst[2];      // places of the lane's two pieces of row0 (eight rows on: 1024 bytes, in either tile)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int piece = (lane & 3) + 4 * (half ^ z);
            src[z] = row0 * HD + piece * 16;
            dst[z] = (piece >> 2) * (STAGE / 2) + row0 * 128 + (((piece & 3) * 2 ^ (row0 & 7)) << 4);    // (the second half: ^ 16)
        }
        for (int k = 0; walk_seg(w, R, tpt, tpi, g); ++k) {
            ok = ok && bar_wait(&sm.mail_full[k & 1], (k >> 1) & 1, sm, a.err);
            ok = __all_sync(0xffffffffu, ok);
            const int kmax = sm.mail[k & 1].kmax, vmax = sm.mail[k & 1].vmax;
            __syncwarp();
            if (lane == 0) bar_arrive(&sm.mail_empty[k & 1]);
            for (int i = 0; i < 2 * g.n; ++i) {
                // the order of the products: K0 V0 K1 V1 .. or, with one tile of rows, K0 K1 V0 K2 V1 .. V(n-1)
                const bool is_v = g.two ? i & 1 : i == 2 * g.n - 1 || (i > 0 && !(i & 1));
                const int most = is_v ? vmax : kmax, live = w.q.ctx - (g.kt0 + (i == 2 * g.n - 1 ? g.n - 1 : g.two ? i / 2 : i / 2 - 1)) * CT;
                const int rs = cnt % RS, st = cnt % ST;
                ok = ok && bar_wait(&sm.raw_full[rs], (cnt / RS) & 1, sm, a.err);
                if (cnt >= ST) ok = ok && bar_wait(&sm.empty[st], (cnt / ST - 1) & 1, sm, a.err);
                ok = __all_sync(0xffffffffu, ok);
                ++cnt;
                if (!ok) continue;
                const unsigned char* from = codes + (size_t)rs * RAW;
                unsigned char* to = ring + (size_t)st * STAGE;
                const bool tail = is_v && live < CT;      // values of keys that do not exist become zeros
                // (a short loop: long straight code of one warp per scheduler starves on instruction fetches)
#pragma unroll 1
                for (int j = 0; j < CT / CONV; j += 16) {
                    const int e = sm.scale[rs][((warp - 12) * (CT / CONV) + j) >> 4];
                    const uint32_t f = e == 255 ? 0x7fffu : half_two(most - e), f2 = f | f << 16;
                    uint4 v[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) v[z] = *(const uint4*)(from + src[z & 1] + (j + 8 * (z >> 1)) * 128);
                    if (tail) {
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            if (row0 + j + 8 * (z >> 1) >= live) v[z] = make_uint4(0, 0, 0, 0);
                    }
                    uint32_t d[4][8];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        half4_of(v[z].x, d[z][0], d[z][1]);
                        half4_of(v[z].y, d[z][2], d[z][3]);
                        half4_of(v[z].z, d[z][4], d[z][5]);
                        half4_of(v[z].w, d[z][6], d[z][7]);
                    }
                    if (f != 0x3c00u) {
#pragma unroll
                        for (int z = 0; z < 32; ++z) {
                            const __half2 p = __hmul2(*(const __half2*)&d[z >> 3][z & 7], *(const __half2*)&f2);
                            d[z >> 3][z & 7] = *(const uint32_t*)&p;
                        }
                    }
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        unsigned char* at = to + (j + 8 * (z >> 1)) * 128;
                        *(uint4*)(at + dst[z & 1]) = make_uint4(d[z][0], d[z][1], d[z][2], d[z][3]);
                        *(uint4*)(at + (dst[z & 1] ^ 16)) = make_uint4(d[z][4], d[z][5], d[z][6], d[z][7]);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(&sm.full[st]);
                    bar_arrive(&sm.raw_empty[rs]);
                }
            }
            if (w.more) walk_step<CT, C_OVER>(w, a, R, tpi);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFT));
        // ---------------------------------------------------------- softmax
        const int t = warp >= 8 ? 1 : 0;
        const int r = (threadIdx.x & 127);                 // this thread's row of a tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + t * SLOT;
        const float sl2 = a.scale * 1.4426950408889634f;
        int* counters = (int*)a.ws;
        float* parts = (float*)((char*)a.ws + PAGED_COUNTER_BYTES);
        int sc = 0, oc = 0, rc = 0, pvc = 0;   // steps of this slot, items; of the other slot and products (one tile)
        bool ok = true;
        for (int k = 0;; ++k) {
            // both slots are done with Q and with the tensor memory of the item before
            wg_sync(1);
            if (threadIdx.x == 128) sm.more = walk_seg(sm.walk, sm.range, tpt, tpi, sm.seg);
            wg_sync(1);
            if (!sm.more) break;
            const Seg& g = sm.seg;
            const PagedSeq& wq = sm.walk.q;
            const int tile = g.two ? t : 0;
            const uint32_t tO = tmem + lanes + OUT + tile * CT;
            const int rg = (int)(r * ginv >> 16), tok = g.tok0 + tile * tpt + rg, head = g.h * c.G + r - rg * c.G;
            const bool live = r < tpt * c.G && tok < g.tok0 + g.ntok;
            auto lim = [&] { return live ? min(wq.ctx - wq.n_new + tok + 1, wq.ctx) : 0; };   // keys that the row sees
            float mx = -INFINITY, l = 0.f;
            // the place of the cut's part, whose upper 128 rows have the output that left the tensor memory (one tile of
            // rows alone), at the maximum mt
            float* slot = parts + (size_t)(blockIdx.x * 2 + (blockIdx.x == g.ca ? 1 : 0)) * C_SLOT;
            auto total = [&](int group) { return (float4*)(slot + ((size_t)group * 2 * CT + CT + r) * 4); };
            float mt = -INFINITY;
            if (g.n > 0) {
                // ---- query rows: 16 threads a row, 8 values each, loads of a batch in flight together
                constexpr int NB = 8, V4 = F32 ? 2 : 1;
                const int first = g.two ? 0 : t * 64, count = g.two ? CT : 64, ch = r & 15;
                for (int b0 = 0; b0 < count / 8; b0 += NB) {
                    uint4 raw[NB][V4];
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const int row = first + (r >> 4) + 8 * (b0 + b), rg = (int)(row * ginv >> 16);
                        const int rt = g.tok0 + tile * tpt + rg;
                        const bool there = row < tpt * c.G && rt < g.tok0 + g.ntok;
                        const uint4* src = (const uint4*)((const TA*)a.q + (int64_t)(wq.row0 + (there ? rt : 0)) * a.q_stride +
                                                          (int64_t)(g.h * c.G + (there ? row - rg * c.G : 0)) * HD + ch * 8);
#pragma unroll
                        for (int j = 0; j < V4; ++j) raw[b][j] = there ? src[j] : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const int row = first + (r >> 4) + 8 * (b0 + b);
                        const uint32_t off = (uint32_t)((ch >> 3) * (STAGE / 2) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
                        float x[8], top = 0.f;
                        if constexpr (F32) {
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                x[4 * j] = __uint_as_float(raw[b][j].x); x[4 * j + 1] = __uint_as_float(raw[b][j].y);
                                x[4 * j + 2] = __uint_as_float(raw[b][j].z); x[4 * j + 3] = __uint_as_float(raw[b][j].w);
                            }
                        } else {
                            unpack_bf16x8(raw[b][0], x);
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
#pragma unroll
                        for (int z = 1; z < 16; z <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, z));
                        // the largest value comes to 2^14..2^15
                        const int ex = min((int)(__float_as_uint(top) >> 23), 254), fe = min(268 - ex, 253);
                        const float f = __uint_as_float((uint32_t)fe << 23);
                        if (ch == 0) sm.row[tile * CT + row] = __uint_as_float((uint32_t)(254 - fe) << 23);
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] *= f;
#pragma unroll
                        for (int p = 0; p < QP; ++p) {
                            uint32_t d[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                d[j] = half2_bits(x[2 * j], x[2 * j + 1]);
                                const float2 was = __half22float2(*(const __half2*)&d[j]);
                                x[2 * j] -= was.x;
                                x[2 * j + 1] -= was.y;
                            }
                            *(uint4*)(qs + (size_t)(F32 ? p : tile) * STAGE + off) = make_uint4(d[0], d[1], d[2], d[3]);
                        }
                    }
                }
                fence_async_smem();
                bar_arrive(&sm.q_full);
            }
            ok = ok && bar_wait(&sm.mail_full[k & 1], (k >> 1) & 1, sm, a.err);
            ok = __all_sync(0xffffffffu, ok);
            const bool lost = sm.mail[k & 1].lost;
            const float vf = e8m0(sm.mail[k & 1].vmax), kf = e8m0(sm.mail[k & 1].kmax);
            __syncwarp();
            if (lane == 0) bar_arrive(&sm.mail_empty[k & 1]);
            wg_sync(4);
            // factor of the row's scores (positive and finite: -inf times it stays -inf)
            const float sl = fminf(fmaxf(sl2 * sm.row[tile * CT + r] * kf, 1e-37f), 3e38f), slack = fminf(8.f / sl, 3e38f);
            const int plain = lost ? 0 : lim();        // tiles up to here are taken as they are
            const int n = g.two ? g.n : (g.n + 1 - t) / 2;
            for (int j = 0; j < n; ++j) {
                const int k0 = (g.kt0 + (g.two ? j : 2 * j + t)) * CT;
                ok = ok && bar_wait(&sm.s_full[t], sc & 1, sm, a.err);
                ++sc;
                ok = __all_sync(0xffffffffu, ok);
                fence_after();
                const bool masked = __any_sync(0xffffffffu, plain - k0 < CT);
                const int seen = masked ? lim() - k0 : CT;          // columns that the row sees
                if (masked && lost) {   // keys of pages out of range do not count: their scores become -inf
                    const int key = k0 + 16 * (lane & 7);
                    const unsigned gone = __ballot_sync(0xffffffffu, key < wq.ctx &&    // bit i: keys 16 i .. 16 i + 15
                        (unsigned)c.table[(int64_t)g.s * c.max_pages + (key >> c.page_shift)] >= (unsigned)c.n_pages);
                    uint32_t none[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) none[i] = 0xff800000u;
#pragma unroll 1
                    for (int i = 0; i < 8; ++i)
                        if (gone >> i & 1) tmem_st16(tS + 16 * i, none);
                    tmem_wait_st();
                }
                // The scores are read twice, for their maximum and for the weights, whose place is over the scores that
                // they come from: short loops and few registers, as instruction fetches of the softmax and of the
                // conversion go to one cache (once, from registers: 499 us instead of 422 at 4096 tokens over 12288).  64
                // columns at a time, or 32 of fp32's longer code (prompts: 89 and 82 us; bf16 as above: 422 and 441).
                uint32_t x[NX][32];
                auto scores = [&](int col) {         // of the columns from col on
#pragma unroll
                    for (int e = 0; e < NX; ++e) tmem_ld32(tS + col + 32 * e, x[e]);
#pragma unroll
                    for (int e = 0; e < NX; ++e) tmem_wait_ld(x[e]);
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 32 * NX; ++i)
                            if (i >= seen - col) x[i >> 5][i & 31] = 0xff800000u;
                    }
                };
                float top = -INFINITY;
#pragma unroll 1
                for (int col = 0; col < CT; col += 32 * NX) {
                    scores(col);
                    float m[2 * NX];         // of 16 columns each
#pragma unroll
                    for (int e = 0; e < 2 * NX; ++e) {
                        const uint32_t* y = &x[e >> 1][e & 1 ? 16 : 0];
                        m[e] = __uint_as_float(y[0]);
#pragma unroll
                        for (int i = 1; i < 15; i += 2) m[e] = fmaxf(fmaxf(m[e], __uint_as_float(y[i])), __uint_as_float(y[i + 1]));
                        m[e] = fmaxf(m[e], __uint_as_float(y[15]));
                    }
#pragma unroll
                    for (int e = 0; e < 2 * NX; ++e) top = fmaxf(top, m[e]);
                }
                // The maximum that the weights refer to moves only when a score passes it by 2^8.  Two slots with one
                // tile share it: a step takes it over from the step before, which is the other slot's.
                const int step = g.two ? j : 2 * j + t;
                if (!g.two && step > 0) {
                    ok = ok && bar_wait(&sm.r_full[1 - t], (rc + ((step - 1) >> 1)) & 1, sm, a.err);
                    ok = __all_sync(0xffffffffu, ok);
                    const float now = sm.ref[r];
                    if (now != mx) l *= ex2f((mx - now) * sl);    // (never back to -inf)
                    mx = now;
                }
                const bool grew = top > mx + slack, flush = F32 && step > 0 && step % FLUSH == 0;
                if (flush || __any_sync(0xffffffffu, grew)) {
                    const float nm = fmaxf(mx, top);
                    const float f = nm == -INFINITY ? 1.f : ex2f((mx - nm) * sl);
                    mx = nm;
                    l *= f;
                    if (flush) {       // (the first slot's, as FLUSH is even; the next product does not add)
                        ok = ok && bar_wait(&sm.pv_full, (pvc + step - 1) & 1, sm, a.err);
                        ok = __all_sync(0xffffffffu, ok);
                        fence_after();
                        const float h = step == FLUSH ? 0.f : mx == -INFINITY ? 1.f : ex2f((mt - mx) * sl);
                        mt = mx;
#pragma unroll 1
                        for (int cc = 0; cc < 8; ++cc) {
                            uint32_t y[16], z[16];
                            tmem_ld16(tO + 16 * cc, y);
                            tmem_ld16(tO + CT + 16 * cc, z);
                            float4 was[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) was[i] = step == FLUSH ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldcg(total(4 * cc + i));
                            auto sum = [&](int i, float w) { return fmaf(__uint_as_float(y[i]) + __uint_as_float(z[i]), f, w * h); };
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                __stcg(total(4 * cc + i), make_float4(sum(4 * i, was[i].x), sum(4 * i + 1, was[i].y),
                                                                      sum(4 * i + 2, was[i].z), sum(4 * i + 3, was[i].w)));
                        }
                        fence_before();
                    } else if (step > 0) {
                        if (!g.two) {      // the products of the step before are in
                            ok = ok && bar_wait(&sm.pv_full, (pvc + step - 1) & 1, sm, a.err);
                            ok = __all_sync(0xffffffffu, ok);
                            fence_after();
                        }
#pragma unroll 1
                        for (int cc = 0; cc < 8 * PP; ++cc) {
                            uint32_t y[16];
                            tmem_ld16(tO + 16 * cc, y);
#pragma unroll
                            for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                            tmem_st16(tO + 16 * cc, y);
                        }
                        tmem_wait_st();
                        fence_before();
                    }
                }
                if (!g.two) {
                    sm.ref[r] = mx;
                    __syncwarp();
                    if (lane == 0) bar_arrive(&sm.r_full[t]);
                }
                const float ref = mx == -INFINITY ? 0.f : P_SHIFT - mx * sl;
                const f2c sf = pair(sl, sl), rf = pair(ref, ref);
                f2c sums = pair(0.f, 0.f);
#pragma unroll 1
                for (int col = 0; col < CT; col += 32 * NX) {
                    scores(col);
#pragma unroll
                    for (int e = 0; e < NX; ++e) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float p0, p1;
                            unpair(fma_pair(pair(__uint_as_float(x[e][2 * i]), __uint_as_float(x[e][2 * i + 1])), sf, rf), p0, p1);
                            p0 = ex2f(p0);
                            p1 = ex2f(p1);
                            sums = add_pair(sums, pair(p0, p1));
                            hi[i] = half2_bits(p0, p1);
                            if constexpr (F32) lo[i] = rest2(p0, p1, hi[i]);
                        }
                        tmem_st16(tS + col + 32 * e, hi);
                        if constexpr (F32) tmem_st16(tS + col + 32 * e + 16, lo);
                    }
                }
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&sm.p_full[t]);
                {
                    float s0, s1;
                    unpair(sums, s0, s1);
                    l += s0 + s1;
                }
            }
            // ---- the item's (or the cut's) output
            if (g.n > 0) {
                ok = ok && bar_wait(&sm.o_full, oc & 1, sm, a.err);
                ++oc;
                ok = __all_sync(0xffffffffu, ok);
                fence_after();
            }
            if (!g.two) {
                rc += (g.n + t) / 2;      // the other slot's steps
                pvc += g.n;
                // both slots' sums, at the last maximum
                sm.stats[t][r] = mx;
                sm.stats[2 + t][r] = l;
                if (t == 0) sm.row[CT + r] = mt;      // (free with one tile of rows)
                wg_sync(2);
                mt = sm.row[CT + r];
                l = 0.f;
                if (g.n > 0) {
                    mx = sm.ref[r];
                    const float ms = mx == -INFINITY ? 0.f : mx;
                    l = sm.stats[2][r] * ex2f((sm.stats[0][r] - ms) * sl) + sm.stats[3][r] * ex2f((sm.stats[1][r] - ms) * sl);
                }
            }
            // blocks of 32 values that this thread puts out: of its own row, or (one tile) half of the row's
            const int blk0 = g.two ? 0 : 2 * t, blk1 = g.two ? 4 : blk0 + 2;
            TA* dst = (TA*)a.out + (int64_t)(wq.row0 + tok) * a.out_stride + (int64_t)head * HD;
            const float inv = l != 0.f ? 1.f / l : 0.f;   // (NaN stays NaN)
            // the output leaves through the tile's place for Q, whose products are done
            const RowOut<TA> row_out = {qs + (size_t)(F32 ? 0 : tile) * STAGE, r, dst, live};
            // partials: [32 groups of 4 values][256 rows], then maxima and sums
            const int prow = tile * CT + r;
            {
                // what left the tensor memory before, at the last maximum
                const bool more = F32 && g.n > FLUSH;
                const float h = more && mt != -INFINITY ? ex2f((mt - mx) * sl) : 0.f;
                const float w0 = g.whole ? inv * vf : vf;
#pragma unroll 1
                for (int c2 = blk0; c2 < blk1; c2 += 2) {
                    uint32_t x[2][32];
                    if (g.n > 0) {
                        tmem_ld32(tO + 32 * c2, x[0]);
                        tmem_ld32(tO + 32 * c2 + 32, x[1]);
                        tmem_wait_ld(x[0]);
                        tmem_wait_ld(x[1]);
                        if constexpr (F32) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t y[32];
                                tmem_ld32(tO + CT + 32 * (c2 + e), y);
                                tmem_wait_ld(y);
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    x[e][i] = __float_as_uint(__uint_as_float(x[e][i]) + __uint_as_float(y[i]));
                                if (more) {
#pragma unroll
                                    for (int i = 0; i < 8; ++i) {
                                        const float4 z = __ldcg(total(8 * (c2 + e) + i));
                                        x[e][4 * i] = __float_as_uint(fmaf(z.x, h, __uint_as_float(x[e][4 * i])));
                                        x[e][4 * i + 1] = __float_as_uint(fmaf(z.y, h, __uint_as_float(x[e][4 * i + 1])));
                                        x[e][4 * i + 2] = __float_as_uint(fmaf(z.z, h, __uint_as_float(x[e][4 * i + 2])));
                                        x[e][4 * i + 3] = __float_as_uint(fmaf(z.w, h, __uint_as_float(x[e][4 * i + 3])));
                                    }
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int cc = c2 + e;
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = l != 0.f ? __uint_as_float(x[e][i]) * w0 : 0.f;
                        if (g.whole) {
                            row_out.put(cc, v);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *(float4*)(slot + ((size_t)(8 * cc + i / 4) * 2 * CT + prow) * 4) =
                                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                        }
                    }
                }
                if (g.whole) {
                    row_out.flush(blk0, blk1);
                } else if (blk0 == 0) {
                    slot[2 * CT * HD + prow] = mx * sl;     // in powers of two, as cuts have factors of their own
                    slot[2 * CT * HD + 2 * CT + prow] = l;
                }
            }
            fence_before();
            if (!g.whole) {
                wg_sync(3);
                if (threadIdx.x == 128) {
                    __threadfence();
                    sm.last = atomicAdd(&counters[g.ca], 1) == g.cb - g.ca;
                    if (sm.last) counters[g.ca] = 0;
                    __threadfence();
                }
                wg_sync(3);
                if (sm.last) {
                    chunk_join(parts, g.ca, g.cb, tile * CT + r, 1.f, blk0, blk1, row_out);
                    row_out.flush(blk0, blk1);
                }
            }
            wg_sync(1);
            if (threadIdx.x == 128 && sm.walk.more) walk_step<CT, C_OVER>(sm.walk, a, sm.range, tpi);
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// pages as [page][head][position][128] bytes, boxes of min(page, 128) positions
bool page_map(CUtensorMap* m, const PagedView& c, void* base) {
    auto fn = encoder();
    if (!fn) return false;
    const int P = 1 << c.page_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)HD, (cuuint64_t)P, (cuuint64_t)c.nkv, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride, (cuuint64_t)c.head_stride, (cuuint64_t)c.page_stride};
    const cuuint32_t box[4] = {HD, (cuuint32_t)min(P, CT), 1, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <typename TA>
cudaError_t launch_t(const Paged8Attn& a, cudaStream_t st) {
    CUtensorMap mk, mv;
    if (!page_map(&mk, a.c, a.c.k) || !page_map(&mv, a.c, a.c.v)) return cudaErrorInvalidValue;
    constexpr int smem = C8_QBYTES + ST * STAGE + RS * RAW + 1024;
    // a per-device attribute: set on every call (a host-side table lookup)
    cudaError_t e = cudaFuncSetAttribute(paged8_chunk_kernel<TA>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // the kernel's warps redistribute exactly this many registers; with fewer they would wait for ever
    static const bool regs_ok = [] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, paged8_chunk_kernel<TA>) == cudaSuccess && at.numRegs == REGS;
    }();
    if (!regs_ok) return cudaErrorInvalidConfiguration;
    const int grid = min(device_sm_count(), C_MAX_CTAS);
    paged8_chunk_kernel<TA><<<grid, C8_THREADS, smem, st>>>(mk, mv, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged8_chunk(const Paged8Attn& a, cudaStream_t st) {
    return a.act == Q3_BF16 ? launch_t<bf16>(a, st) : launch_t<float>(a, st);
}

}  // namespace q3
