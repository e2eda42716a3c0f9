// Paged attention (q3paged.h): the choice of kernel, and the one for fp32 pages.
//
// fp32 keys and values would take six products of bf16 parts on the tensor cores
// (a tenth of this kernel's time, with the parts formed as K and V are brought in:
// not built), so this kernel multiplies on the CUDA cores.  A CTA
// of 256 threads takes ROWS query rows of one kv head and walks tiles of 64
// keys in shared memory: V(t) is on its way (cp.async) while the scores of t
// are formed, K(t+1) while its outputs are.  A thread forms ROWS/16 x 4 scores
// and ROWS/16 x 8 outputs, so that a 16-byte shared load serves 8 (ROWS = 64)
// multiply-adds; two CTAs fit an SM, as the places in shared memory are mixed
// against bank conflicts instead of padded.  ROWS =
// 16 serves a few tokens of many heads.  Bound by the multiply-adds and the
// shared loads beside them: a prompt of 2048 tokens (16 q, 8 kv heads) 519 us,
// 33 TFLOP/s (padded, with one CTA an SM, 604; packed products: the same).
#include "common.cuh"
#include "kernels.h"
#include "paged.h"
#include "paged_sched.cuh"
#include "pdl.cuh"

namespace q3 {

namespace {

constexpr int FT = 256;            // threads
constexpr int FK = 64;             // keys of a tile and of a unit
constexpr int F_OVER = 0;          // units that an item costs besides its keys (1 and 2 were slower)
constexpr int F_CTAS = 2;          // resident CTAs of an SM
constexpr int f_smem(int rows) { return (rows * HD + 2 * FK * HD + rows * FK) * 4; }
static_assert(F_CTAS * (f_smem(64) + 2048) <= 228 * 1024, "both fit an SM's shared memory");
constexpr size_t f_slot(int rows) { return (size_t)rows * (HD + 4); }   // outputs, maxima, sums

__device__ __forceinline__ void cp16(float* dst, const float* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ float fex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int ROWS>
__global__ void __launch_bounds__(FT, F_CTAS) paged_f32_kernel(const PagedAttn a, int grid_max) {
    pdl_wait();
    pdl_trigger();
    constexpr int RT = ROWS / 16;      // rows of a thread
    extern __shared__ __align__(16) float fs[];
    float* Qs = fs;                    // [ROWS][128]
    float* Ks = Qs + ROWS * HD;        // [64][128], 16-byte pieces of a row in the order piece ^ (row & 7)
    float* Vs = Ks + FK * HD;          // [64][128]
    float* Ps = Vs + FK * HD;          // [ROWS][64], the halves of 16 swapped for every other thread row
    __shared__ int s_last, s_lost;     // s_lost: a page out of range has been met
    const PagedView& c = a.c;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    if (tid == 0) s_lost = 0;

    const int tpi = ROWS / c.G;        // tokens of an item
    const PagedRange R = paged_range<FT>(a, grid_max, F_OVER + 1, F_OVER, [&](const PagedSeq& q) { return c.nkv * seq_units<FK, F_OVER>(q, tpi); });
    if (R.u0 >= R.u1) return;
    const float sl2 = a.scale * 1.4426950408889634f;
    int* counters = (int*)a.ws;
    float* parts = (float*)((char*)a.ws + PAGED_COUNTER_BYTES);

    Walk w;
    walk_begin<FK, F_OVER>(w, a, R, tpi);
    int end;
    while (w.more && paged_cut(R, w.item0, w.item0 + w.nu, &end)) {
        const PagedSeq q = w.q;
        const int s = w.s, h = w.h, tok0 = w.item * tpi, ntok = min(tpi, q.n_new - tok0), rows = ntok * c.G;
        const int vis = max(0, min(q.ctx, q.ctx - q.n_new + tok0 + ntok));   // keys that the last token sees
        const int key0 = w.u == w.item0 ? 0 : (w.u - w.item0 - F_OVER) * FK;
        const int key1 = (int)min((long long)vis, (long long)(end - w.item0 - F_OVER) * FK);
        const int nt = key1 > key0 ? (key1 - key0 + FK - 1) / FK : 0;
        const int32_t* table = c.table + (int64_t)s * c.max_pages;
        const int pmask = (1 << c.page_shift) - 1;
        auto load = [&](float* dst, int mix, const void* pool, int t) {
#pragma unroll
            for (int i = 0; i < FK * 32 / FT; ++i) {
                const int row = (tid + i * FT) >> 5, ch = tid & 31, key = key0 + t * FK + row;
                const float* src = (const float*)pool;
                bool ok = key < key1;
                if (ok) {
                    const int page = __ldg(table + (key >> c.page_shift));
                    if ((unsigned)page < (unsigned)c.n_pages)
                        src += page * c.page_stride + (int64_t)h * c.head_stride + (int64_t)(key & pmask) * c.token_stride + ch * 4;
                    else {
                        ok = false;
                        *(volatile int*)&s_lost = 1;
                        if (a.err) atomicOr(a.err, ERRB_BOUNDS);
                    }
                }
                cp16(dst + row * HD + (ch ^ (row & mix)) * 4, src, ok);
            }
            cp_commit();
        };
        __syncthreads();   // the segment before is done with the buffers
        if (nt > 0) load(Ks, 7, c.k, 0);
        for (int i = tid; i < ROWS * 32; i += FT) {
            const int r = i >> 5, tok = tok0 + r / c.G;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows)
                v = *(const float4*)((const float*)a.q + (int64_t)(q.row0 + tok) * a.q_stride +
                                     (int64_t)(h * c.G + r % c.G) * HD + (i & 31) * 4);
            *(float4*)(Qs + r * HD + (i & 31) * 4) = v;
        }
        int lim[RT];
        float m[RT], l[RT], o[RT][8];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = ty * RT + i;
            lim[i] = r < rows ? min(q.ctx - q.n_new + tok0 + r / c.G + 1, key1) : 0;
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int d = 0; d < 8; ++d) o[i][d] = 0.f;
        }
        for (int t = 0; t < nt; ++t) {
            load(Vs, 0, c.v, t);
            cp_wait<1>();
            __syncthreads();
            float x[RT][4];
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
#pragma unroll 4
            for (int d = 0; d < HD; d += 4) {
                float4 qv[RT], kv[4];
#pragma unroll
                for (int i = 0; i < RT; ++i) qv[i] = *(const float4*)(Qs + (ty * RT + i) * HD + d);
#pragma unroll
                for (int j = 0; j < 4; ++j) kv[j] = *(const float4*)(Ks + (tx + 16 * j) * HD + (d ^ (tx & 7) * 4));
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[i][j] = fmaf(qv[i].x, kv[j].x, x[i][j]);
                        x[i][j] = fmaf(qv[i].y, kv[j].y, x[i][j]);
                        x[i][j] = fmaf(qv[i].z, kv[j].z, x[i][j]);
                        x[i][j] = fmaf(qv[i].w, kv[j].w, x[i][j]);
                    }
            }
            const int kb = key0 + t * FK + tx;
            int gone = 0;      // of the four keys: those of pages out of range, which do not count
            if (*(volatile int*)&s_lost)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (kb + 16 * j < key1 && (unsigned)__ldg(table + ((kb + 16 * j) >> c.page_shift)) >= (unsigned)c.n_pages)
                        gone |= 1 << j;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                float top = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (kb + 16 * j >= lim[i] || (gone >> j & 1)) x[i][j] = -INFINITY;
                    top = fmaxf(top, x[i][j]);
                }
#pragma unroll
                for (int z = 1; z < 16; z <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, z));
                const float ref = top == -INFINITY ? 0.f : top * sl2;
                const float f = fex2(m[i] * sl2 - ref);      // nothing seen before: 0
                m[i] = top;
                l[i] *= f;
#pragma unroll
                for (int d = 0; d < 8; ++d) o[i][d] *= f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = fex2(fmaf(x[i][j], sl2, -ref));
                    l[i] += p;
                    Ps[(ty * RT + i) * FK + ((tx + 16 * j) ^ (ty & 1) * 16)] = p;
                }
            }
            __syncthreads();   // weights are there, K is free
            if (t + 1 < nt) {
                load(Ks, 7, c.k, t + 1);
                cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            __syncthreads();
#pragma unroll 2
            for (int k = 0; k < FK; k += 4) {
                float4 p[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i) p[i] = *(const float4*)(Ps + (ty * RT + i) * FK + (k ^ (ty & 1) * 16));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const float4 v0 = *(const float4*)(Vs + (k + kk) * HD + tx * 4);
                    const float4 v1 = *(const float4*)(Vs + (k + kk) * HD + 64 + tx * 4);
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const float pw = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                        o[i][0] = fmaf(pw, v0.x, o[i][0]); o[i][1] = fmaf(pw, v0.y, o[i][1]);
                        o[i][2] = fmaf(pw, v0.z, o[i][2]); o[i][3] = fmaf(pw, v0.w, o[i][3]);
                        o[i][4] = fmaf(pw, v1.x, o[i][4]); o[i][5] = fmaf(pw, v1.y, o[i][5]);
                        o[i][6] = fmaf(pw, v1.z, o[i][6]); o[i][7] = fmaf(pw, v1.w, o[i][7]);
                    }
                }
            }
            __syncthreads();   // V and the weights are free
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int z = 1; z < 16; z <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], z);
        auto store = [&](int r, const float (&v)[8], float sum) {
            const int tok = tok0 + r / c.G;
            const float f = sum != 0.f ? 1.f / sum : 0.f;   // (NaN stays NaN)
            float* dst = (float*)a.out + (int64_t)(q.row0 + tok) * a.out_stride + (int64_t)(h * c.G + r % c.G) * HD + tx * 4;
            *(float4*)dst = make_float4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
            *(float4*)(dst + 64) = make_float4(v[4] * f, v[5] * f, v[6] * f, v[7] * f);
        };
        if (w.u == w.item0 && end == w.item0 + w.nu) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
                if (ty * RT + i < rows) store(ty * RT + i, o[i], l[i]);
        } else {
            const int ca = paged_cut_first(R, w.item0), cb = paged_cut_last(R, w.item0 + w.nu);
            auto part = [&](int cc) { return parts + (size_t)(cc * 2 + (cc == ca ? 1 : 0)) * f_slot(ROWS); };
            float* slot = part(blockIdx.x);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int r = ty * RT + i;
                if (r >= rows) continue;
                *(float4*)(slot + r * HD + tx * 4) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
                *(float4*)(slot + r * HD + 64 + tx * 4) = make_float4(o[i][4], o[i][5], o[i][6], o[i][7]);
                if (tx == 0) { slot[ROWS * HD + r] = m[i]; slot[ROWS * HD + ROWS + r] = l[i]; }
            }
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                s_last = atomicAdd(&counters[ca], 1) == cb - ca;
                if (s_last) counters[ca] = 0;
                __threadfence();
            }
            __syncthreads();
            if (s_last) {
#pragma unroll 1
                for (int i = 0; i < RT; ++i) {
                    const int r = ty * RT + i;
                    if (r >= rows) continue;
                    float top = -INFINITY, sum = 0.f, v[8] = {};
#pragma unroll 4
                    for (int cc = ca; cc <= cb; ++cc) {
                        const float* p = part(cc);
                        const float pm = __ldcg(p + ROWS * HD + r), pl = __ldcg(p + ROWS * HD + ROWS + r);
                        const float4 v0 = __ldcg((const float4*)(p + r * HD + tx * 4));
                        const float4 v1 = __ldcg((const float4*)(p + r * HD + 64 + tx * 4));
                        const float nm = fmaxf(top, pm), ref = nm == -INFINITY ? 0.f : nm;
                        const float f0 = fex2((top - ref) * sl2), f1 = fex2((pm - ref) * sl2);
                        top = nm;
                        sum = sum * f0 + pl * f1;
                        v[0] = v[0] * f0 + v0.x * f1; v[1] = v[1] * f0 + v0.y * f1;
                        v[2] = v[2] * f0 + v0.z * f1; v[3] = v[3] * f0 + v0.w * f1;
                        v[4] = v[4] * f0 + v1.x * f1; v[5] = v[5] * f0 + v1.y * f1;
                        v[6] = v[6] * f0 + v1.z * f1; v[7] = v[7] * f0 + v1.w * f1;
                    }
                    store(r, v, sum);
                }
            }
        }
        if (end < w.item0 + w.nu) return;
        walk_step<FK, F_OVER>(w, a, R, tpi);
    }
}

template <int ROWS>
cudaError_t launch_f32(const PagedAttn& a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(paged_f32_kernel<ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, f_smem(ROWS));
    if (e != cudaSuccess) return e;
    const int grid = min(device_sm_count(), 160) * F_CTAS;
    return launch_pdl(paged_f32_kernel<ROWS>, grid, FT, f_smem(ROWS), st, a, grid);
}

}  // namespace

size_t paged_workspace_bytes() {
    return PAGED_COUNTER_BYTES + max(max(paged_decode_ws(), paged_chunk_ws()), (size_t)160 * F_CTAS * 2 * f_slot(64) * sizeof(float));
}

cudaError_t launch_paged_attention(const PagedAttn& a, cudaStream_t st) {
    if (paged_decode_takes(a)) return launch_paged_decode(a, st);
    if (a.kv == Q3_BF16) return launch_paged_chunk(a, st);
    return (int64_t)a.max_q * a.c.G <= 16 ? launch_f32<16>(a, st) : launch_f32<64>(a, st);
}

}  // namespace q3
