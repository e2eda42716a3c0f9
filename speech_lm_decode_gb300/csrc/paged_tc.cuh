// What the chunk kernels of paged attention share: mbarriers, TMA, tcgen05 and
// packed fp32 arithmetic (sm_103a); their items, their outputs and the join of
// the parts of a cut item.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "paged_sched.cuh"

namespace q3 {

constexpr int CT = 128;                    // rows of a tile, keys of a unit
constexpr int STAGE = CT * HD * 2;         // bytes of a K or V tile of 16-bit values
constexpr int C_MAX_CTAS = 192;
constexpr int C_OVER = 4;                  // units that an item costs besides its keys
constexpr int C_MIN_UNITS = C_OVER + 2;
constexpr size_t C_SLOT = (size_t)2 * CT * (HD + 2);   // floats of a partial
constexpr long long C_WAIT_LIMIT = 2000000000LL;   // cycles

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
// Waits are bounded: `dead` of the CTA's shared state is set by the first that runs out.
template <class S> __device__ __forceinline__ void give_up(S& s, int* err) {
    *(volatile int*)&s.dead = 1;
    if (err) atomicOr(err, ERRB_TIMEOUT);
}
// bounded wait; false once the CTA has given up (heed: not even looked at then)
template <class S>
__device__ __forceinline__ bool bar_wait(uint64_t* b, unsigned parity, S& s, int* err, bool heed = true) {
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

// ------------------------------------------------------------------ outputs
// 32 values at a time of a thread's row (row r of a tile of 128) through shared
// memory: 16-byte pieces at places that depend on the row, so that the warp then
// stores its rows side by side.
template <typename TA> struct RowOut {
    static constexpr int PR = HD * (int)sizeof(TA) / 16, PB = PR / 4;   // pieces of a row, of 32 values
    unsigned char* stage;
    int r;
    TA* dst;
    bool live;
    __device__ __forceinline__ void put(int blk, const float (&v)[32]) const {
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            uint4 d;
            if constexpr (sizeof(TA) == 4)
                d = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                               __float_as_uint(v[4 * i + 3]));
            else
                d = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                               pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
            *(uint4*)(stage + (size_t)(r * PR + ((blk * PB + i) ^ (r & (PR - 1)))) * 16) = d;
        }
    }
    __device__ __forceinline__ void flush(int blk0, int blk1) const {     // blocks [blk0, blk1) of the warp's 32 rows
        const int lane = threadIdx.x & 31;
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
    }
};

// Row mrow of an item cut over CTAs ca .. cb: the blocks [blk0, blk1) of their
// parts, which hold maxima in units of 1 / sl2, put out.
template <typename TA>
__device__ __forceinline__ void chunk_join(const float* parts, int ca, int cb, int mrow, float sl2, int blk0, int blk1,
                                           const RowOut<TA>& out) {
    auto part = [&](int cc) { return parts + (size_t)(cc * 2 + (cc == ca)) * C_SLOT; };
    float m = -INFINITY, sum = 0.f;
#pragma unroll 1
    for (int c0 = ca; c0 <= cb; c0 += 8) {
        float pm[8], pl[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float* p = part(min(c0 + j, cb)) + 2 * CT * HD + mrow;
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
            if (c0 + j <= cb) sum = fmaf(ex2f((pm[j] - ms) * sl2), pl[j], sum);
    }
    const float ms = m == -INFINITY ? 0.f : m, rs = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll 1
    for (int b = blk0; b < blk1; ++b) {
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 1
        for (int c0 = ca; c0 <= cb; c0 += 2) {
            float4 z[2][8];
            float f[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float* p = part(min(c0 + j, cb));
                f[j] = __ldcg(p + 2 * CT * HD + mrow);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[j][i] = __ldcg((const float4*)(p + ((size_t)(8 * b + i) * 2 * CT + mrow) * 4));
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float wj = c0 + j <= cb ? ex2f((f[j] - ms) * sl2) : 0.f;
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
        out.put(b, v);
    }
}

// the driver's encoder of tensor maps (null: none)
inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
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

}  // namespace q3
