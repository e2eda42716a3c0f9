// Paged attention over 8-bit codes for few query rows (single tokens, a handful
// of tokens of a sequence): q3paged8_attention's kernel while the new tokens
// times the q heads of a kv head fit a tile or two of tensor-core columns.
//
// Bound by reading K and V once (256 bytes a key and kv head).  As over bf16
// pages (paged_decode.cu), a CTA of four warps walks its keys in blocks of 16, a
// warp to a block; scores are K q^T and outputs V^T p^T of mma.m16n8k16.  A block
// comes through the warp's own ring in shared memory: with fragments straight from
// global memory the registers hold half the bytes that they hold of bf16, too few
// to hide the latency behind (116 us instead of 100 below).  Codes become f16 as
// fragments, which holds each exactly: a lane's 16 bytes of a K row are four k-steps
// of its A fragment with the head dimension of K and q permuted alike, its 16 bytes
// of two V rows, bytes interleaved, fragments of two output values at a time.
//
// Scales stay out of the tensor cores, so that they may be any: the 16 keys of a
// block have one scale, the keys' multiplies the scores, and outputs are summed in
// units of the largest scale of values so far, in fp32.  q enters relative to the
// power of two above its row's largest value, the weights relative to 2^-7 of the
// running maximum (f16 then holds a weight of 2^-21 of it with all its bits, and
// as the maximum moves only when a score passes it by 2^8, none passes 2^15).
//
// bf16 activations are exact in one f16 part, their weights take one (11 bits;
// the output's rounding keeps 8: 1.67e-3 of the result, the plain form's 1.66e-3).
// fp32 activations take two columns a row, f16 parts of 22 bits together, and so do
// their weights; their products with V are added up in fp32 (2.9e-7, 8.3e-7).
//
// Measured (16 q and 8 kv heads, GPU alone): 256 tokens over 1025..1280, bf16, 605
// MB in 100 us (89 % of the copy rate), fp32 102; 64 sequences of 4 / 8 tokens over
// 2000, bf16, 52 / 70 us; three tokens over 30000..65537 (32 and 4 heads) 38 us for
// 21 of reading, the rest being the join of what 456 CTAs hold of 12 items; 32 fp32
// tokens over 65..768, 14 us, and one over 228, 8 us, are latencies.
#include "common.cuh"
#include "kernels.h"
#include "paged8.h"
#include "paged_sched.cuh"
#include "pdl.cuh"

namespace q3 {

namespace {

constexpr int DW = 4;             // warps of a CTA
constexpr int DU = 16 * DW;       // keys of a unit
// Resident CTAs of an SM.  256 tokens: 100 us with three, 107 with four, whose warps have 128 registers, 126 with two;
// with two of eight warps 106.
constexpr int d8_ctas(int nt) { return nt == 1 ? 3 : 2; }
constexpr int D8_RING = 3;                                  // blocks of a warp's ring (two: 107 us, four: as three)
constexpr int D8_STAGE = 2 * 16 * HD;                       // bytes of one: K and V of 16 keys
constexpr float P_SHIFT = 7.f;    // weights are 2^7 times exp2 of score - maximum

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// without a sum to add to
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 16 bytes into shared memory, or zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
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
// 2^e, e <= 0; below 2^-126: zero
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)max(127 + e, 0) << 23); }
// transposes an 8 x 8 matrix of 16-bit values (lane (g, t): row g, columns 2t and 2t+1)
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// NT: column tiles of eight; a query row takes one column (bf16 activations) or two (fp32: columns 8 n + r and
// 8 n + 4 + r hold the parts of row 4 n + r).
template <typename TA, int NT>
__global__ void __launch_bounds__(DW * 32, d8_ctas(NT)) paged8_decode_kernel(const Paged8Attn a, int grid_max) {
    pdl_wait();
    pdl_trigger();
    constexpr bool F32 = sizeof(TA) == 4;
    constexpr int RG = F32 ? 4 * NT : 8 * NT;   // query rows of an item
    const PagedView& c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    constexpr int S = D8_RING;
    // The warps' rings; between two segments the outputs and the weights of an item's parts.  A row of 16 keys' codes is 128
    // bytes; its 16-byte pieces are moved about so that a warp's reads of fragments meet no bank twice.
    extern __shared__ __align__(128) unsigned char raw[];
    static_assert(8 * NT * (HD + 4) * 4 <= S * D8_STAGE && 160 * d8_ctas(NT) * RG * 4 <= DW * S * D8_STAGE, "what lies over the rings");
    float* so_all = (float*)raw;
    float (*so)[8 * NT][HD + 4] = (float (*)[8 * NT][HD + 4])raw;
    unsigned char* ring = raw + warp * S * D8_STAGE;
    const uint32_t ring32 = (uint32_t)__cvta_generic_to_shared(ring);
    const uint32_t kdst = ring32 + (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3 & 1) << 2) << 4);
    const uint32_t vdst = ring32 + 2048 + (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 4) << 1) << 4);
    const int kread = g * 128 + (t << 4), kflip = (g & 1) << 6, vread = 2048 + 2 * t * 128 + ((g ^ t << 1) << 4);
    __shared__ float sm_m[DW][RG], sm_l[DW][RG];
    __shared__ int s_last;

    auto units_of = [&](const PagedSeq& q) -> long long {
        if (q.n_new <= 0) return 0;
        const int groups = (q.n_new * c.G + RG - 1) / RG;
        return (long long)c.nkv * groups * max(1, (q.ctx + DU - 1) / DU);
    };
    const PagedRange R = paged_range<DW * 32>(a, grid_max, 1, 0, units_of);
    if (R.u0 >= R.u1) return;
    const float sl2 = a.scale * 1.4426950408889634f;   // scores in powers of two
    int* counters = (int*)a.ws;
    constexpr size_t SLOT = (size_t)RG * (HD + 4);   // outputs, maxima, sums (16-byte rows)
    float* parts = (float*)((char*)a.ws + PAGED_COUNTER_BYTES);

    int s = R.s;
    PagedSeq q = R.q;
    int nu = max(1, (q.ctx + DU - 1) / DU), groups = (q.n_new * c.G + RG - 1) / RG;   // units and row groups of a head
    int item = (R.u0 - R.start) / nu;       // head * groups + row group
    int item0 = R.start + item * nu;        // the item's units [item0, item0 + nu)
    auto next_item = [&]() -> bool {
        item0 += nu;
        if (++item < c.nkv * groups) return true;
        if (item0 >= R.u1) return false;
        do { q = paged_seq(a, ++s, false); } while (q.n_new <= 0);
        nu = max(1, (q.ctx + DU - 1) / DU);
        groups = (q.n_new * c.G + RG - 1) / RG;
        item = 0;
        return true;
    };
    int u = paged_begin(R, item0, item0 + nu), seg_end;
    if (u == item0 + nu && !next_item()) return;
    while (paged_cut(R, item0, item0 + nu, &seg_end)) {
        const int h = item / groups, rg = item - h * groups;
        const int key0 = (u - item0) * DU;
        const int key1 = (int)min((long long)q.ctx, (long long)(seg_end - item0) * DU);
        const int rows = min(RG, q.n_new * c.G - rg * RG);

        const int nb = (key1 - key0 + 15) >> 4;
        const int32_t* table = c.table + (int64_t)s * c.max_pages;
        const int pmask = (1 << c.page_shift) - 1;
        const int64_t head_off = (int64_t)h * c.head_stride;
        // A warp takes every DW-th block of 16 keys.  Their codes come through its own ring in shared memory, S - 1 blocks
        // ahead; keys past the last one read as zeros (a weight of zero times a value of zero).
        auto page_at = [&](int b) -> int { return b < nb ? __ldg(table + ((key0 + b * 16) >> c.page_shift)) : 0; };
        // (a page's positions lie within 2^31 bytes, the caller checks, and its scales within 2^31 of the pool's first)
        const int ts = (int)c.token_stride, lr = lane >> 3, per_shift = c.page_shift - a.block_shift;
        const int64_t lane_off = head_off + lr * ts + (lane & 7) * 16;
        const uint8_t *kbase = (const uint8_t*)c.k + lane_off, *vbase = (const uint8_t*)c.v + lane_off;
        // place i of the ring: the page of its block (-1: out of range), its scales, and the page of its next block
        int pg[S], ahead[S] = {};
        uint32_t ks[S], vs[S];
        auto issue = [&](int i, int b) {
            if (b < nb) {
                const bool there = (unsigned)ahead[i] < (unsigned)c.n_pages;
                const int kb = key0 + b * 16, slot = kb & pmask, page = there ? ahead[i] : 0, left = there ? key1 - kb - lr : 0;
                pg[i] = there ? page : -1;
                ahead[i] = page_at(b + DW * S);
                const int64_t off = page * c.page_stride + slot * ts;
                const uint32_t kd = kdst + i * D8_STAGE, vd = vdst + i * D8_STAGE;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    copy16(kd + j * 512, kbase + off + 4 * j * ts, left > 4 * j);
                    copy16((vd ^ (j & 1) << 6) + j * 512, vbase + off + 4 * j * ts, left > 4 * j);
                }
                const int sc = ((page * c.nkv + h) << per_shift) + (slot >> a.block_shift);
                ks[i] = vs[i] = 0;
                if (there) { ks[i] = __ldg(a.ks + sc); vs[i] = __ldg(a.vs + sc); }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < S; ++i) ahead[i] = page_at(warp + DW * i);
#pragma unroll
        for (int i = 0; i < S - 1; ++i) issue(i, warp + DW * i);

        // ---- query rows into B fragments, and the factors of the rows whose softmax the lane follows (columns 2t, 2t+1)
        uint32_t qb[NT][8][2];
        float qs[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = F32 ? 4 * n + (g & 3) : 8 * n + g;
            const bool there = r < rows;
            const int rr = rg * RG + r, tok = rr / c.G;
            const TA* src = (const TA*)a.q + (int64_t)(q.row0 + (there ? tok : 0)) * a.q_stride +
                            (int64_t)(h * c.G + (there ? rr - tok * c.G : 0)) * HD + t * 16;
            float x[32], top = 0.f;
#pragma unroll
            for (int j = 0; j < 32; j += 16 / (int)sizeof(TA)) {
                const uint4 w = there ? *(const uint4*)(src + (j >> 4) * 64 + (j & 15)) : make_uint4(0, 0, 0, 0);
                if constexpr (F32) {
                    x[j] = __uint_as_float(w.x); x[j + 1] = __uint_as_float(w.y);
                    x[j + 2] = __uint_as_float(w.z); x[j + 3] = __uint_as_float(w.w);
                } else {
                    float v[8];
                    unpack_bf16x8(w, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[j + i] = v[i];
                }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) top = fmaxf(top, fabsf(x[j]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = min((int)(__float_as_uint(top) >> 23), 254), fe = min(268 - ex, 253);   // largest value to 2^14..2^15
            const float f = __uint_as_float((uint32_t)fe << 23);
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x0 = x[4 * j + 2 * e] * f, x1 = x[4 * j + 2 * e + 1] * f;
                    const uint32_t hi = half2_bits(x0, x1);
                    qb[n][j][e] = F32 && g >= 4 ? rest2(x0, x1, hi) : hi;
                }
            const float inv = sl2 * __uint_as_float((uint32_t)(254 - fe) << 23);
            qs[n][0] = __shfl_sync(0xffffffffu, inv, 8 * t);
            qs[n][1] = __shfl_sync(0xffffffffu, inv, 8 * t + 4);
        }
        int lim[NT][2];   // keys that those rows see
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = F32 ? 4 * n + 2 * (t & 1) + e : 8 * n + 2 * t + e;
                lim[n][e] = r < rows ? min(q.ctx - q.n_new + (rg * RG + r) / c.G + 1, key1) : 0;
            }
        const int lim_all = min(q.ctx - q.n_new + rg * RG / c.G + 1, key1);   // keys that every row sees

        float o[NT][8][4], mx[NT][2], l[NT][2];   // o: in units of the largest scale of values so far, 2^(vcur - 127)
        int vcur = 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[n][i >> 2][i & 3] = 0.f;
            mx[n][0] = mx[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }
        for (int b0 = warp; b0 < nb; b0 += DW * S) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int b = b0 + DW * i, kb = key0 + b * 16;
            if (b >= nb) break;
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            __syncwarp();      // the block is there, and every lane is done with the one before it
            issue((i + S - 1) % S, b + DW * (S - 1));
            const unsigned char* st = ring + i * D8_STAGE;
            float x[NT][4];   // scores: [key g: columns 2t, 2t+1; key g + 8: the same]
            {
                float y[NT][4];   // of every other step, so that a product does not wait for the one before it
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 r0 = *(const uint4*)(st + kread + (j << 6 ^ kflip)), r1 = *(const uint4*)(st + kread + 1024 + (j << 6 ^ kflip));
                    const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t a0, a1, a2, a3;
                        half4_of(w0[w], a0, a2);
                        half4_of(w1[w], a1, a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float (&z)[4] = w & 1 ? y[n] : x[n];
                            if (j == 0 && w < 2) mma16816_first(z, a0, a1, a2, a3, qb[n][4 * j + w][0], qb[n][4 * j + w][1]);
                            else mma16816(z, a0, a1, a2, a3, qb[n][4 * j + w][0], qb[n][4 * j + w][1]);
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int z = 0; z < 4; ++z) x[n][z] += y[n][z];
            }
            const float kf = e8m0(ks[i]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    if constexpr (F32) x[n][z] += __shfl_xor_sync(0xffffffffu, x[n][z], 2);
                    x[n][z] = x[n][z] * qs[n][z & 1] * kf;
                }
            if (kb + 16 > lim_all || pg[i] < 0) {
                if (pg[i] < 0 && lane == 0 && a.err) atomicOr(a.err, ERRB_BOUNDS);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        if (pg[i] < 0 || kb + g + 8 * (z >> 1) >= lim[n][z & 1]) x[n][z] = -INFINITY;
            }
            bool grew = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) grew |= fmaxf(x[n][e], x[n][e + 2]) > mx[n][e] + 8.f;
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
                        f[e] = m == -INFINITY ? 1.f : ex2(mx[n][e] - m);   // first keys: 0
                        mx[n][e] = m;
                        l[n][e] *= f[e];
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int z = 0; z < 4; ++z) o[n][k][z] *= f[z & 1];
                }
            }
            uint32_t pb[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float p[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const float m = mx[n][z & 1];
                    p[z] = ex2(x[n][z] - (m == -INFINITY ? 0.f : m - P_SHIFT));
                    l[n][z & 1] += p[z];
                }
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    uint32_t v = half2_bits(p[2 * z], p[2 * z + 1]);
                    if (F32 && t >= 2) v = rest2(p[2 * z], p[2 * z + 1], v);
                    pb[n][z] = transpose8(v);
                }
            }
            const uint4 r0 = *(const uint4*)(st + vread), r1 = *(const uint4*)(st + vread + 128);
            const uint4 r2 = *(const uint4*)(st + vread + 1024), r3 = *(const uint4*)(st + vread + 1152);
            const uint32_t v0[4] = {r0.x, r0.y, r0.z, r0.w}, v1[4] = {r1.x, r1.y, r1.z, r1.w};
            const uint32_t v2[4] = {r2.x, r2.y, r2.z, r2.w}, v3[4] = {r3.x, r3.y, r3.z, r3.w};
            auto outputs = [&](auto f) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int w = k >> 1, sel = k & 1 ? 0x7362 : 0x5140;
                    uint32_t a0, a1, a2, a3;
                    half4_of(__byte_perm(v0[w], v1[w], sel), a0, a1);
                    half4_of(__byte_perm(v2[w], v3[w], sel), a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n) f(o[n][k], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                }
            };
            const int vb = (int)vs[i];
            if (vb > vcur) {
                const float f = two_to(vcur - vb);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[n][k >> 2][k & 3] *= f;
                vcur = vb;
            }
            if (!F32 && vb == vcur) {
                outputs(mma16816);
            } else {
                const float f = two_to(vb - vcur);
                outputs([&](float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
                    float z[4];
                    mma16816_first(z, a0, a1, a2, a3, b0, b1);
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[e] = fmaf(z[e], f, d[e]);
                });
            }
        }
        }
        const float of = e8m0(vcur);

        // ---- the four warps' outputs, joined
        __syncthreads();   // every warp is done with its ring
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[n][e];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                const int r = F32 ? 4 * n + 2 * t + e : 8 * n + 2 * t + e;
                if (g == 0 && (!F32 || t < 2)) { sm_m[warp][r] = mx[n][e]; sm_l[warp][r] = v; }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *(float2*)&so[warp][8 * n + 2 * t + e][16 * g + 2 * i] = make_float2(o[n][i][e] * of, o[n][i][e + 2] * of);
        }
        __syncthreads();
        const bool whole = u == item0 && seg_end == item0 + nu;
        const int ca = paged_cut_first(R, item0), cb = paged_cut_last(R, item0 + nu);   // where it is cut
        float* mine = parts + (size_t)(blockIdx.x * 2 + (blockIdx.x == ca ? 1 : 0)) * SLOT;
        TA* out = (TA*)a.out;
        const int dim = tid & (HD - 1), r0 = tid / HD;     // value and first row that the thread puts out
        auto store = [&](int r, float v) {
            const int rr = rg * RG + r, tok = rr / c.G;
            out[(int64_t)(q.row0 + tok) * a.out_stride + (int64_t)(h * c.G + rr - tok * c.G) * HD + dim] = from_f<TA>(v);
        };
        for (int r = r0; r < rows; r += DW / 4) {
            float m = sm_m[0][r];
#pragma unroll
            for (int w = 1; w < DW; ++w) m = fmaxf(m, sm_m[w][r]);
            const float ms = m == -INFINITY ? 0.f : m;
            float acc = 0.f, sum = 0.f;
#pragma unroll
            for (int w = 0; w < DW; ++w) {
                const float f = ex2(sm_m[w][r] - ms);
                const int col = F32 ? 8 * (r >> 2) + (r & 3) : r;
                acc += f * (F32 ? so[w][col][dim] + so[w][col + 4][dim] : so[w][col][dim]);
                sum += f * sm_l[w][r];
            }
            if (whole) {
                store(r, sum != 0.f ? acc / sum : 0.f);
            } else {
                mine[r * HD + dim] = acc;
                if (dim == 0) { mine[RG * HD + r] = m; mine[RG * HD + RG + r] = sum; }
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
                // weights of the parts (the outputs' place is free: every thread is past the barriers above), then each
                // warp adds up every DW-th part
                const int n = cb - ca + 1;
                float* wt = so_all;
                auto part = [&](int i) { return parts + (size_t)((ca + i) * 2 + (i == 0 ? 1 : 0)) * SLOT; };
                const int sub = lane & 15;
                for (int r = warp * 2 + (lane >> 4); r < (rows + 1) / 2 * 2; r += 2 * DW) {   // sixteen lanes a row
                    float m = -INFINITY, sum = 0.f;
                    if (r < rows)
#pragma unroll 3
                        for (int i = sub; i < n; i += 16) {
                            const float v = __ldcg(part(i) + RG * HD + r), l = __ldcg(part(i) + RG * HD + RG + r);
                            const float nm = fmaxf(m, v), ms = nm == -INFINITY ? 0.f : nm;
                            sum = sum * ex2(m - ms) + l * ex2(v - ms);
                            m = nm;
                            wt[i * RG + r] = v;
                        }
#pragma unroll
                    for (int z = 1; z < 16; z <<= 1) {
                        const float v = __shfl_xor_sync(0xffffffffu, m, z), l = __shfl_xor_sync(0xffffffffu, sum, z);
                        const float nm = fmaxf(m, v), ms = nm == -INFINITY ? 0.f : nm;
                        sum = sum * ex2(m - ms) + l * ex2(v - ms);
                        m = nm;
                    }
                    if (r < rows) {
                        const float ms = m == -INFINITY ? 0.f : m;
                        for (int i = sub; i < n; i += 16) wt[i * RG + r] = ex2(wt[i * RG + r] - ms);
                        if (sub == 0) sm_l[0][r] = sum;
                    }
                }
                __syncthreads();
                float4 acc[RG];
#pragma unroll
                for (int r = 0; r < RG; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
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
                for (int r = r0; r < rows; r += DW / 4) {
                    const float sum = sm_l[0][r];
                    float v = 0.f;
#pragma unroll
                    for (int w = 0; w < DW; ++w) v += so[w][r][dim];
                    store(r, sum != 0.f ? v / sum : 0.f);
                }
            }
        }
        if (seg_end < item0 + nu || !next_item()) return;
        u = item0;
        __syncthreads();   // the rings are free
    }
}

template <typename TA, int NT>
cudaError_t launch_t(const Paged8Attn& a, cudaStream_t st) {
    const int grid = min(device_sm_count(), 160) * d8_ctas(NT);
    constexpr int smem = DW * D8_RING * D8_STAGE;
    // a per-device attribute: set on every call (a host-side table lookup)
    const cudaError_t e = cudaFuncSetAttribute(paged8_decode_kernel<TA, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged8_decode_kernel<TA, NT>, grid, DW * 32, smem, st, a, grid);
}

}  // namespace

// Rows of a kv head that one sequence may have: 16, of two tiles of columns (bf16) or two groups of two (fp32: the keys
// are read twice, by neighbours of the same L2).  Sequences of eight tokens and two heads over 2000 keys, 64 of them: 70
// us here and 148 by the chunk kernel (bf16), 120 and 169 (fp32).
bool paged8_decode_takes(const Paged8Attn& a) { return (int64_t)a.max_q * a.c.G <= 16; }

cudaError_t launch_paged8_decode(const Paged8Attn& a, cudaStream_t st) {
    const int rows = a.max_q * a.c.G;
    if (a.act == Q3_BF16) return rows <= 8 ? launch_t<bf16, 1>(a, st) : launch_t<bf16, 2>(a, st);
    return rows <= 4 ? launch_t<float, 1>(a, st) : launch_t<float, 2>(a, st);
}

}  // namespace q3
