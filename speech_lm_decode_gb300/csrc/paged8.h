// Shared by the operators over a paged cache of 8-bit codes (q3paged8.h).
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "paged.h"
#include "q3paged8.h"

namespace q3 {

// PagedView's strides are in codes (bytes); scales: [page][kv head][block]
struct Paged8Attn : PagedAttn {
    int block_shift;             // positions of a block: 1 << block_shift
    const uint8_t *ks, *vs;
};

struct Paged8Append {
    PagedView c;
    int block_shift;
    uint8_t *ks, *vs;
    int n_tokens, max_q;
    const void* qkv;
    int64_t ldq;
    const int32_t *q_off, *ctx;
    const float *qn, *kn;
    float eps;
    const float2* rope;
    int rope_rows;
    void* q_out;
    int64_t ldo;
    int* err;
};

// few query rows (paged8_decode.cu)
bool paged8_decode_takes(const Paged8Attn& a);
cudaError_t launch_paged8_decode(const Paged8Attn& a, cudaStream_t st);
// many query rows (paged8_chunk.cu)
cudaError_t launch_paged8_chunk(const Paged8Attn& a, cudaStream_t st);

constexpr int E8_MIN = 127 - 100, E8_MAX = 127 + 119;   // scales that append writes

// 2^(b - 127); 255: NaN
__device__ __forceinline__ float e8m0(uint32_t b) { return __uint_as_float(max((b << 23) + ((b + 1) >> 8), 0x00400000u)); }
// codes as f16 values (exact), the lower byte first
__device__ __forceinline__ void half4_of(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(codes));
}
__device__ __forceinline__ void float4_of(uint32_t codes, float (&v)[4]) {
    uint32_t lo, hi;
    half4_of(codes, lo, hi);
    const float2 a = __half22float2(*(const __half2*)&lo), b = __half22float2(*(const __half2*)&hi);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
// two values as codes, the first in the lower byte: nearest, ties to even, at most 448 (NaN stays, infinities do not)
__device__ __forceinline__ uint32_t codes_of(float a, float b) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace q3
