// Paged attention for many query rows (chunks of prompts, mixed batches) over
// bf16 pages, on the fifth-generation tensor cores.
//
// An item is up to 256 query rows (tokens x q heads of one kv head; two tiles
// of 128) of one sequence, its units are tiles of 128 keys; one persistent CTA
// per SM takes an equal share of all units (paged_sched.cuh).  Inside a CTA
//   warp 0      copies K and V tiles into a ring of 32 KB stages (TMA, one box
//               per page and 64 values of the head, 128-byte swizzle);
//   warp 1      issues S = Q K^T and O += P V (tcgen05.mma, M = N = 128); P is
//               the A operand in tensor memory, V the transposed B operand;
//   warp 2      looks for page ids out of range among a cut's: their keys get -inf
//               as their score (the copies read zeros past the last page);
//   warps 4-7   softmax of slot 0, warps 8-11 of slot 1: a thread owns a row,
//               reads its 128 scores from tensor memory, keeps the running
//               maximum and sum, and writes P back over the scores.
// The two slots alternate on the tensor cores, so that one's softmax runs while
// the other's products do.  With two tiles of rows, a slot is a tile and both
// read the same keys; with one tile (few rows, or fp32 activations), the slots
// take the tile's even and odd key tiles, with one output and one reference
// maximum that is handed on from step to step.
//
// bf16 activations: the weights enter the second product rounded to bf16 (their
// sum is that of the fp32 ones), which adds 1.6e-3 of the result to the 1.7e-3
// of the output's own rounding; a second part would be half as many products again.
//
// fp32 activations enter as three bf16 parts of q (24 bits: exact) and two of p
// (17 bits), 5 products for 2.  The parts of p have an output each, as the
// tensor cores cut the terms of a sum to the bits of its largest one: with one
// output and three parts of p the error was no smaller (2e-6 to 7e-6 of the
// result, growing with the context) and the call a fifth slower.
//
// Measured (16 q and 8 kv heads): 4096 tokens over 12288, bf16, 355 us = 1.36
// PFLOP/s (72 % of the measured rate; what is left is a slot's softmax between
// two of its products), fp32 782 us; 24 prompts of 1..512 over 0..255, fp32, 85
// us, five items a CTA of two or three steps, of which loading the query rows
// and the output are the larger part; 64 tokens over 32k, bf16, 53 us.
//
// Every wait is bounded: one that runs out sets the timeout bit, after which
// the CTA goes through its remaining steps without waiting or issuing, drains
// its copies and products, frees its tensor memory and returns.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "kernels.h"
#include "paged.h"
#include "paged_sched.cuh"

namespace q3 {

namespace {

constexpr int CT = 128;                    // rows of a tile, keys of a unit
constexpr int STAGE = CT * HD * 2;         // bytes of a K or V tile
constexpr int C_THREADS = 384;
constexpr int C_MAX_CTAS = 192;
constexpr int C_OVER = 4;                  // units that an item costs besides its keys
constexpr int C_MIN_UNITS = C_OVER + 2;
constexpr long long C_WAIT_LIMIT = 2000000000LL;
constexpr int c_stages(bool f32) { return f32 ? 4 : 5; }
constexpr int c_qbytes(bool f32) { return f32 ? 3 * STAGE : 2 * STAGE; }
constexpr size_t C_SLOT = (size_t)2 * CT * (HD + 2);   // floats of a partial

// One cut of an item that a CTA works on.
struct Seg {
    int s, h;             // sequence, kv head
    int tok0, ntok;       // first token (of the sequence's new ones) and tokens of the item
    int n;                // key tiles of this cut (0: the item sees no key)
    int kt0;              // first of them
    bool two;             // two tiles of rows
    bool whole;           // the cut is the item
    int ca, cb;           // CTAs of the item
};

struct ChunkSmem {
    uint64_t full[5], empty[5], s_full[2], p_full[2], r_full[2], pv_full, q_full, o_full, drain;
    uint32_t tmem;
    int dead, last;
    int lost;                // the cut's keys have a page out of range among them
    float ref[CT];           // one tile of rows: the maxima that both slots' weights refer to
    PagedRange range;        // the softmax warps' walk, kept here to save them the registers
    Walk walk;
    Seg seg;
    int more;
};

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* b, unsigned n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, unsigned bytes) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}"
                 ::"r"(su32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, unsigned parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(su32(b)), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ void give_up(ChunkSmem& s, int* err) {
    *(volatile int*)&s.dead = 1;
    if (err) atomicOr(err, ERRB_TIMEOUT);
}
// bounded wait; false once the CTA has given up (heed: not even looked at then)
__device__ __forceinline__ bool bar_wait(uint64_t* b, unsigned parity, ChunkSmem& s, int* err, bool heed = true) {
    if (bar_try(b, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(b, parity)) {
        if (heed && *(volatile int*)&s.dead) return false;
        if (clock64() - t0 > C_WAIT_LIMIT) {
            give_up(s, err);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(su32(bar)) : "memory");
}
// One product of the chain; a, b: low words of the operands' descriptors (a of
// umma_ts: an address in tensor memory).  The upper words are constants, so
// that an instruction's operands are one uniform add away from the last one's.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(DESC_HI) : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(DESC_HI) : "memory");
}
// one thread of the warp, always the same
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
// a value that all lanes have, made known as such
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// of the softmax warps, or of those and warp 2
__device__ __forceinline__ void wg_sync(int id) { asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void seg_sync(int id) { asm volatile("bar.sync %0, 288;" ::"r"(id) : "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {   // and waits for it
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
          "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr) : "memory");
}
// waits for the loads; the registers pass through it, so that no use of them can move in front
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :: "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Low word of the descriptor of a tile in shared memory, rows of 128 bytes,
// 128-byte swizzle.  K-major (Q, K): eight-row groups 1024 bytes apart.
// MN-major (V: the 128 bytes run along the head): eight-key groups 1024 bytes
// apart, the second half of the head `lead` bytes on.
__device__ __forceinline__ uint32_t tile_desc(uint32_t saddr, uint32_t lead) { return (saddr >> 4) | (lead >> 4) << 16; }
// fp32 D, bf16 A and B, M = N = 128; bit 16: B is MN-major
constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(CT >> 3) << 17) | ((uint32_t)(CT >> 4) << 24);
constexpr uint32_t IDESC_V = IDESC | (1u << 16);

__device__ __forceinline__ float ex2f(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// two fp32 values side by side: one instruction works on both
using f2c = unsigned long long;
__device__ __forceinline__ f2c pair(float a, float b) {
    f2c r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(f2c v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2c fma_pair(f2c a, f2c b, f2c c) {
    f2c r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2c add_pair(f2c a, f2c b) {
    f2c r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t*)&v;
}

// ------------------------------------------------------------------ items
// the part of the walk's item that this CTA takes
__device__ __forceinline__ bool walk_seg(Walk& w, const PagedRange& R, int tpt, int tpi, Seg& g) {
    int end;
    if (!w.more || !paged_cut(R, w.item0, w.item0 + w.nu, &end)) return false;
    g.s = w.s;
    g.h = w.h;
    g.tok0 = w.item * tpi;
    g.ntok = min(tpi, w.q.n_new - g.tok0);
    g.two = g.ntok > tpt;
    g.kt0 = w.u == w.item0 ? 0 : w.u - w.item0 - C_OVER;
    g.n = end - w.item0 - C_OVER - g.kt0;
    if (w.q.ctx - w.q.n_new + g.tok0 + g.ntok <= 0 || w.q.ctx <= 0) g.n = 0;
    g.whole = w.u == w.item0 && end == w.item0 + w.nu;
    g.ca = paged_cut_first(R, w.item0);
    g.cb = paged_cut_last(R, w.item0 + w.nu);
    w.more = end == w.item0 + w.nu;   // a cut end is this CTA's last
    return true;
}

template <typename TA>
__global__ void __launch_bounds__(C_THREADS, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                   const __grid_constant__ PagedAttn a) {
    constexpr bool F32 = sizeof(TA) == 4;
    constexpr int ST = c_stages(F32), QP = F32 ? 3 : 1, PP = F32 ? 2 : 1;
    // tensor memory: the slots' scores (the weights over them), then outputs: of the two tiles, or (fp32) of the
    // weights' two parts
    constexpr int SLOT = CT, OUT = 2 * SLOT;
    extern __shared__ __align__(1024) unsigned char raw[];
    __shared__ ChunkSmem sm;
    unsigned char* base = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    unsigned char* qs = base;                       // Q tiles (bf16: per slot; fp32: per part)
    unsigned char* ring = base + c_qbytes(F32);
    const PagedView& c = a.c;
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int tpt = CT / c.G, tpi = F32 ? tpt : 2 * tpt;   // tokens of a tile, of an item
    const uint32_t ginv = 65536u / c.G + 1;                // row / G for rows below 256 and G <= 16: row * ginv >> 16

    const PagedRange R = paged_range<C_THREADS>(a, gridDim.x, C_MIN_UNITS, C_OVER,
                                                [&](const PagedSeq& q) { return c.nkv * seq_units<CT, C_OVER>(q, tpi); });
    if (R.u0 >= R.u1) return;

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) { bar_init(&sm.full[i], 1); bar_init(&sm.empty[i], 1); }
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

    // registers: 384 threads x 168 at launch = 128 x 72 + 256 x 216 (the launcher checks the 168)
    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    Seg g;
    if (warp == 0) {
        // ---------------------------------------------------------- K and V tiles
        int cnt = 0, issued = 0;
        bool ok = true;
        const int box = min(1 << c.page_shift, CT), pmask = (1 << c.page_shift) - 1;
        auto load = [&](const CUtensorMap* map, int kt) {
            const int st = cnt % ST;
            if (cnt >= ST) ok = ok && bar_wait(&sm.empty[st], (cnt / ST - 1) & 1, sm, a.err);
            if (cnt + 1 == a.inject) {
                give_up(sm, a.err);
                ok = false;
            }
            ok = __all_sync(0xffffffffu, ok);
            ++cnt;
            if (!ok) return;
            issued = cnt;
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
            if (lane == 0) bar_expect(&sm.full[st], (unsigned)(nbox * box * HD * 2));
            __syncwarp();
            if (lane < nbox) {
                const uint32_t dst = su32(ring + (size_t)st * STAGE) + lane * box * 128;
                tma_4d(dst, map, 0, key & pmask, g.h, page, &sm.full[st]);
                tma_4d(dst + STAGE / 2, map, 64, key & pmask, g.h, page, &sm.full[st]);
            }
        };
        while (walk_seg(w, R, tpt, tpi, g)) {
            const int lead = g.two ? 1 : 2;
            for (int i = 0; i < min(lead, g.n); ++i) load(&mapK, g.kt0 + i);
            for (int i = 0; i < g.n; ++i) {
                load(&mapV, g.kt0 + i);
                if (i + lead < g.n) load(&mapK, g.kt0 + i + lead);
            }
            if (w.more) walk_step<CT, C_OVER>(w, a, R, tpi);
        }
        // nothing may still be writing this CTA's shared memory when it leaves (given up, its last copies are not
        // waited for elsewhere)
        for (int i = max(0, issued - ST); i < issued; ++i) bar_wait(&sm.full[i % ST], (i / ST) & 1, sm, a.err, false);
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
                        umma_ts(d + p * CT, pa + 64 * p + 8 * ks, vd + ks * (2048 >> 4), IDESC_V, ks != 0 ? 1u : first);
            }
            __syncwarp();
        };
        // V rows of keys that do not exist become zeros (their weights are zero, what the pages hold may be NaN)
        auto clear_tail = [&](int kt, int i) {
            const int rows = w.q.ctx - kt * CT;
            if (rows >= CT || !ok) return;
            uint4* v = (uint4*)(ring + (size_t)(i % ST) * STAGE);
            for (int r = rows * 8 + lane; r < CT * 8; r += 32) {
                v[r] = make_uint4(0, 0, 0, 0);
                v[r + STAGE / 32] = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
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
                    clear_tail(g.kt0 + i, v);
                    if (g.two) {
                        outputs(0, v, i > 0);
                        if (more) { full(k); scores(0, k); }
                        outputs(1, v, i > 0);
                        release(v);
                        if (more) { scores(1, k); release(k); }
                    } else {
                        const int t = i & 1;
                        outputs(t, v, i > 0);
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
        // ---------------------------------------------------------- pages out of range among a cut's, beside the query rows
        for (;;) {
            seg_sync(1);
            seg_sync(1);
            if (!sm.more) break;
            const Seg& g = sm.seg;
            const int32_t* row = c.table + (int64_t)g.s * c.max_pages;
            const int p0 = g.kt0 * CT >> c.page_shift;
            const int p1 = g.n > 0 ? (min((g.kt0 + g.n) * CT, sm.walk.q.ctx) - 1 >> c.page_shift) + 1 : p0;
            bool bad = false;
#pragma unroll 8
            for (int i = p0 + lane; i < p1; i += 32) bad |= (unsigned)row[i] >= (unsigned)c.n_pages;
            bad = __any_sync(0xffffffffu, bad);
            if (lane == 0) sm.lost = bad;
            seg_sync(4);
            seg_sync(1);
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ---------------------------------------------------------- softmax
        const int t = warp >= 8 ? 1 : 0;
        const int r = (threadIdx.x & 127);                 // this thread's row of a tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + t * SLOT;
        const float sl2 = a.scale * 1.4426950408889634f, slack = fminf(8.f / sl2, 3e38f);   // (finite: -inf stays -inf)
        int* counters = (int*)a.ws;
        float* parts = (float*)((char*)a.ws + PAGED_COUNTER_BYTES);
        int sc = 0, oc = 0, rc = 0, pvc = 0;   // steps of this slot, items; of the other slot and products (one tile)
        bool ok = true;
        for (;;) {
            // both slots are done with Q and with the tensor memory of the item before
            seg_sync(1);
            if (threadIdx.x == 128) sm.more = walk_seg(sm.walk, sm.range, tpt, tpi, sm.seg);
            seg_sync(1);
            if (!sm.more) break;
            const Seg& g = sm.seg;
            const PagedSeq& wq = sm.walk.q;
            const int tile = g.two ? t : 0;
            const uint32_t tO = tmem + lanes + OUT + tile * CT;
            const int rg = (int)(r * ginv >> 16), tok = g.tok0 + tile * tpt + rg, head = g.h * c.G + r - rg * c.G;
            const bool live = r < tpt * c.G && tok < g.tok0 + g.ntok;
            auto lim = [&] { return live ? min(wq.ctx - wq.n_new + tok + 1, wq.ctx) : 0; };   // keys that the row sees
            float mx = -INFINITY, l = 0.f;
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
                        if constexpr (F32) {
                            float x[8];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                x[4 * j] = __uint_as_float(raw[b][j].x); x[4 * j + 1] = __uint_as_float(raw[b][j].y);
                                x[4 * j + 2] = __uint_as_float(raw[b][j].z); x[4 * j + 3] = __uint_as_float(raw[b][j].w);
                            }
#pragma unroll
                            for (int p = 0; p < 3; ++p) {
                                uint32_t d[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    d[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
                                    x[2 * j] -= __uint_as_float(d[j] << 16);
                                    x[2 * j + 1] -= __uint_as_float(d[j] & 0xffff0000u);
                                }
                                *(uint4*)(qs + (size_t)p * STAGE + off) = make_uint4(d[0], d[1], d[2], d[3]);
                            }
                        } else {
                            *(uint4*)(qs + (size_t)tile * STAGE + off) = raw[b][0];
                        }
                    }
                }
                fence_async_smem();
                bar_arrive(&sm.q_full);
            }
            seg_sync(4);
            const int plain = sm.lost ? 0 : lim();     // tiles up to here are taken as they are
            const int n = g.two ? g.n : (g.n + 1 - t) / 2;
            for (int j = 0; j < n; ++j) {
                const int k0 = (g.kt0 + (g.two ? j : 2 * j + t)) * CT;
                ok = ok && bar_wait(&sm.s_full[t], sc & 1, sm, a.err);
                ++sc;
                ok = __all_sync(0xffffffffu, ok);
                fence_after();
                uint32_t x[4][32];
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) tmem_ld32(tS + 32 * cc, x[cc]);
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) tmem_wait_ld(x[cc]);
                if (__any_sync(0xffffffffu, plain - k0 < CT)) {
                    if (sm.lost) {   // keys of pages out of range do not count: their scores become -inf, all are read again
                        const int key = k0 + 16 * (lane & 7);
                        const unsigned gone = __ballot_sync(0xffffffffu, key < wq.ctx &&    // bit i: keys 16 i .. 16 i + 15
                            (unsigned)c.table[(int64_t)g.s * c.max_pages + (key >> c.page_shift)] >= (unsigned)c.n_pages);
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[0][i] = 0xff800000u;
                        uint32_t (&none)[16] = *reinterpret_cast<uint32_t (*)[16]>(&x[0][0]);
#pragma unroll 1
                        for (int i = 0; i < 8; ++i)
                            if (gone >> i & 1) tmem_st16(tS + 16 * i, none);
                        tmem_wait_st();
#pragma unroll
                        for (int cc = 0; cc < 4; ++cc) tmem_ld32(tS + 32 * cc, x[cc]);
#pragma unroll
                        for (int cc = 0; cc < 4; ++cc) tmem_wait_ld(x[cc]);
                    }
                    const int seen = lim() - k0;                   // columns that the row sees
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * cc + i >= seen) x[cc][i] = 0xff800000u;
                }
                float tops[4];
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    tops[cc] = __uint_as_float(x[cc][0]);
#pragma unroll
                    for (int i = 1; i < 31; i += 2)
                        tops[cc] = fmaxf(fmaxf(tops[cc], __uint_as_float(x[cc][i])), __uint_as_float(x[cc][i + 1]));
                    tops[cc] = fmaxf(tops[cc], __uint_as_float(x[cc][31]));
                }
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                // The maximum that the weights refer to moves only when a score passes it by 2^8.  Two slots with one
                // tile share it: a step takes it over from the step before, which is the other slot's.
                const int step = g.two ? j : 2 * j + t;
                if (!g.two && step > 0) {
                    ok = ok && bar_wait(&sm.r_full[1 - t], (rc + ((step - 1) >> 1)) & 1, sm, a.err);
                    ok = __all_sync(0xffffffffu, ok);
                    const float now = sm.ref[r];
                    if (now != mx) l *= ex2f((mx - now) * sl2);    // (never back to -inf)
                    mx = now;
                }
                const bool grew = top > mx + slack;
                if (__any_sync(0xffffffffu, grew)) {
                    const float nm = fmaxf(mx, top);
                    const float f = nm == -INFINITY ? 1.f : ex2f((mx - nm) * sl2);
                    mx = nm;
                    l *= f;
                    if (step > 0) {
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
                const float ref = mx == -INFINITY ? 0.f : -mx * sl2;
                const f2c sl = pair(sl2, sl2), rf = pair(ref, ref);
                f2c sums = pair(0.f, 0.f);
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float p0, p1;
                        unpair(fma_pair(pair(__uint_as_float(x[cc][2 * i]), __uint_as_float(x[cc][2 * i + 1])), sl, rf), p0, p1);
                        p0 = ex2f(p0);
                        p1 = ex2f(p1);
                        sums = add_pair(sums, pair(p0, p1));
                        hi[i] = pack_bf16(p0, p1);
                        if constexpr (F32)
                            lo[i] = pack_bf16(p0 - __uint_as_float(hi[i] << 16), p1 - __uint_as_float(hi[i] & 0xffff0000u));
                    }
                    tmem_st16(tS + 16 * cc, hi);
                    if constexpr (F32) tmem_st16(tS + 64 + 16 * cc, lo);
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
                float* stats = (float*)(qs + (F32 ? 2 : 1) * STAGE);   // [maxima, sums][slot][row], where Q is not needed
                stats[t * CT + r] = mx;
                stats[(2 + t) * CT + r] = l;
                wg_sync(2);
                l = 0.f;
                if (g.n > 0) {
                    mx = sm.ref[r];
                    const float ms = mx == -INFINITY ? 0.f : mx;
                    l = stats[2 * CT + r] * ex2f((stats[r] - ms) * sl2) + stats[3 * CT + r] * ex2f((stats[CT + r] - ms) * sl2);
                }
            }
            // blocks of 32 values that this thread puts out: of its own row, or (one tile) half of the row's
            const int blk0 = g.two ? 0 : 2 * t, blk1 = g.two ? 4 : blk0 + 2;
            TA* dst = (TA*)a.out + (int64_t)(wq.row0 + tok) * a.out_stride + (int64_t)head * HD;
            const float inv = l != 0.f ? 1.f / l : 0.f;   // (NaN stays NaN)
            // The output leaves through the tile's place for Q, whose products are done: a thread puts 32 values of its
            // row, then the warp stores its rows side by side (16-byte pieces at places that depend on the row).
            constexpr int PR = HD * (int)sizeof(TA) / 16, PB = PR / 4;   // pieces of a row, of 32 values
            unsigned char* stage = qs + (size_t)(F32 ? 0 : tile) * STAGE;
            auto put = [&](int blk, const float (&v)[32]) {
#pragma unroll
                for (int i = 0; i < PB; ++i) {
                    uint4 d;
                    if constexpr (F32)
                        d = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                                       __float_as_uint(v[4 * i + 3]));
                    else
                        d = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                       pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
                    *(uint4*)(stage + (size_t)(r * PR + ((blk * PB + i) ^ (r & (PR - 1)))) * 16) = d;
                }
            };
            auto flush = [&](int blk0, int blk1) {     // blocks [blk0, blk1) of the warp's 32 rows
                __syncwarp();
                const int n = (blk1 - blk0) * PB, per = 32 / n, piece = blk0 * PB + lane % n;
#pragma unroll 4
                for (int i0 = 0; i0 < 32; i0 += per) {
                    const int i = i0 + lane / n;
                    TA* to = (TA*)__shfl_sync(0xffffffffu, (unsigned long long)dst, i);
                    const bool there = __shfl_sync(0xffffffffu, (int)live, i);
                    const int row = (r & ~31) + i;
                    const uint4 d = *(const uint4*)(stage + (size_t)(row * PR + (piece ^ (row & (PR - 1)))) * 16);
                    if (there) *((uint4*)to + piece) = d;
                }
                __syncwarp();
            };
            // partials: [32 groups of 4 values][256 rows], then maxima and sums
            const int prow = tile * CT + r;
            float* slot = parts + (size_t)(blockIdx.x * 2 + (blockIdx.x == g.ca ? 1 : 0)) * C_SLOT;
            {
                const float w0 = g.whole ? inv : 1.f;
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
                            put(cc, v);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *(float4*)(slot + ((size_t)(8 * cc + i / 4) * 2 * CT + prow) * 4) =
                                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                        }
                    }
                }
                if (g.whole) {
                    flush(blk0, blk1);
                } else if (blk0 == 0) {
                    slot[2 * CT * HD + prow] = mx;
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
                    const int mrow = tile * CT + r;
                    auto part = [&](int cc) { return parts + (size_t)(cc * 2 + (cc == g.ca)) * C_SLOT; };
                    float m = -INFINITY, sum = 0.f;
#pragma unroll 1
                    for (int c0 = g.ca; c0 <= g.cb; c0 += 8) {
                        float pm[8], pl[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float* p = part(min(c0 + j, g.cb)) + 2 * CT * HD + mrow;
                            pm[j] = __ldcg(p);
                            pl[j] = __ldcg(p + 2 * CT);
                        }
                        const float was = m;
#pragma unroll
                        for (int j = 0; j < 8; ++j) m = fmaxf(m, pm[j]);
                        const float ms = m == -INFINITY ? 0.f : m;
                        sum *= ex2f((was - ms) * sl2);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (c0 + j <= g.cb) sum = fmaf(ex2f((pm[j] - ms) * sl2), pl[j], sum);
                    }
                    const float ms = m == -INFINITY ? 0.f : m, rs = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll 1
                    for (int b = blk0; b < blk1; ++b) {
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 1
                        for (int c0 = g.ca; c0 <= g.cb; c0 += 2) {
                            float4 z[2][8];
                            float f[2];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float* p = part(min(c0 + j, g.cb));
                                f[j] = __ldcg(p + 2 * CT * HD + mrow);
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    z[j][i] = __ldcg((const float4*)(p + ((size_t)(8 * b + i) * 2 * CT + mrow) * 4));
                            }
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float wj = c0 + j <= g.cb ? ex2f((f[j] - ms) * sl2) : 0.f;
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    v[4 * i] = fmaf(z[j][i].x, wj, v[4 * i]);
                                    v[4 * i + 1] = fmaf(z[j][i].y, wj, v[4 * i + 1]);
                                    v[4 * i + 2] = fmaf(z[j][i].z, wj, v[4 * i + 2]);
                                    v[4 * i + 3] = fmaf(z[j][i].w, wj, v[4 * i + 3]);
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= rs;
                        put(b, v);
                    }
                    flush(blk0, blk1);
                }
            }
            seg_sync(1);
            if (threadIdx.x == 128 && sm.walk.more) walk_step<CT, C_OVER>(sm.walk, a, sm.range, tpi);
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* p = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)p;
    }();
    return fn;
}

// pages as [page][head][position][128], boxes of min(page, 128) positions x 64 values
bool page_map(CUtensorMap* m, const PagedView& c, void* base) {
    auto fn = encoder();
    if (!fn) return false;
    const int P = 1 << c.page_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)HD, (cuuint64_t)P, (cuuint64_t)c.nkv, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride * 2, (cuuint64_t)c.head_stride * 2,
                                   (cuuint64_t)c.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)min(P, CT), 1, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <typename TA>
cudaError_t launch_t(const PagedAttn& a, cudaStream_t st) {
    constexpr bool F32 = sizeof(TA) == 4;
    CUtensorMap mk, mv;
    if (!page_map(&mk, a.c, a.c.k) || !page_map(&mv, a.c, a.c.v)) return cudaErrorInvalidValue;
    constexpr int smem = c_qbytes(F32) + c_stages(F32) * STAGE + 1024;
    // a per-device attribute: set on every call (a host-side table lookup)
    cudaError_t e = cudaFuncSetAttribute(paged_chunk_kernel<TA>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // the kernel's warps redistribute exactly this many registers; with fewer they would wait for ever
    static const bool regs_ok = [] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, paged_chunk_kernel<TA>) == cudaSuccess && at.numRegs == 168;
    }();
    if (!regs_ok) return cudaErrorInvalidConfiguration;
    const int grid = min(device_sm_count(), C_MAX_CTAS);
    paged_chunk_kernel<TA><<<grid, C_THREADS, smem, st>>>(mk, mv, a);
    return cudaGetLastError();
}

}  // namespace

size_t paged_chunk_ws() { return (size_t)C_MAX_CTAS * 2 * C_SLOT * sizeof(float); }

cudaError_t launch_paged_chunk(const PagedAttn& a, cudaStream_t st) {
    return a.act == Q3_BF16 ? launch_t<bf16>(a, st) : launch_t<float>(a, st);
}

}  // namespace q3
