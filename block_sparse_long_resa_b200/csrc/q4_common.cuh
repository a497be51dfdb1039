// The 4-bit cache format (resa_cache_q4_t): 16 channels of a token and kv head
// share an e4m3 scale s, a channel is an e2m1 code c, and c * s is exact in
// fp16 (2 + 4 significant bits, magnitudes 2^-10 .. 2688), which is what the
// attention kernels feed their MMAs with.  The head's fp32 scale g is folded
// into the softmax scale (keys) and into the output (values).
#pragma once

#include <cuda_fp16.h>

#include "resa_common.cuh"

namespace resa {

constexpr int kQ4Group = 16;  // channels a group scale covers

// The pointers of a resa_cache_q4_t the kernels take.
struct Q4Cache {
    uint8_t *k, *v, *k_sf, *v_sf;
    const float *k_scale, *v_scale;
};

// ceil(a / b) of counts; a + b may pass 2^31.
__device__ __forceinline__ int ceil_div(int a, int b) {
    return (int)(((unsigned)a + (unsigned)b - 1u) / (unsigned)b);
}

__device__ __forceinline__ float head_scale(const float *g, int h) { return g ? g[h] : 1.f; }

// Eight codes (channels c .. c+7, low nibble first) to four fp16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
// Two e4m3 bytes (low byte first) to an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
// Nearest e4m3 (ties to even, saturating at 448) of a non-negative value.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) {
    const uint32_t h = e4m3x2_to_f16(byte);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float f16_lo(uint32_t p) {
    return __half2float(__ushort_as_half((unsigned short)(p & 0xffffu)));
}
__device__ __forceinline__ float f16_hi(uint32_t p) {
    return __half2float(__ushort_as_half((unsigned short)(p >> 16)));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float pow2i(int k) {  // 2^k, k in [-126, 127]
    return __int_as_float((127 + k) << 23);
}
__device__ __forceinline__ void cp_async16_s(uint32_t smem_dst, const void *gsrc) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(gsrc) : "memory");
}

// Quantise one group of 16 bf16 values (pairs, channel 0 low) with 1/g = rg: codes
// (channel i in nibble i) and the e4m3 scale byte.  A code is the nearest e2m1 of
// y / s with the quotient correctly rounded (a reciprocal, and one residual step
// after Markstein, 1990): ties, y = t * s for a decision point t of at most 3 bits,
// then stay ties, and no y beside one is rounded onto it, since y and the quotient
// have 24 bits both.  (Counting the seven decision points that |y| passes took five
// times the instructions.)  NaN counts as 0 and infinity saturates; returns
// whether either occurred.
__device__ __forceinline__ bool q4_quantise(const uint32_t (&w)[8], float rg, uint2 &codes,
                                            uint32_t &sf) {
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & 0x7fff7fffu);
    const uint32_t mag = max(m2 & 0xffffu, m2 >> 16);
    float amax = bf16_bits_to_f32((uint16_t)mag) * rg;  // rounding keeps the order
    float y[kQ4Group];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[2 * i] = bf_lo(w[i]) * rg;
        y[2 * i + 1] = bf_hi(w[i]) * rg;
    }
    const bool finite = amax < INFINITY;
    if (!finite) {
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < kQ4Group; ++i) {
            y[i] = y[i] == y[i] ? fminf(fmaxf(y[i], -3e38f), 3e38f) : 0.f;
            amax = fmaxf(amax, fabsf(y[i]));
        }
    }
    sf = f32_to_e4m3(__fdiv_rn(amax, 6.f));
    const float s = e4m3_to_f32(sf);
    const float rs = s > 0.f ? __frcp_rn(s) : 0.f;
#pragma unroll
    for (int i = 0; i < kQ4Group; ++i) {
        const float q = y[i] * rs;
        y[i] = fmaf(fmaf(-q, s, y[i]), rs, q);
    }
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(c[i])
            : "f"(y[8 * i]), "f"(y[8 * i + 1]), "f"(y[8 * i + 2]), "f"(y[8 * i + 3]), "f"(y[8 * i + 4]),
              "f"(y[8 * i + 5]), "f"(y[8 * i + 6]), "f"(y[8 * i + 7]));
    codes = s > 0.f ? make_uint2(c[0], c[1]) : make_uint2(0u, 0u);
    return !finite;
}

// Eight channels as bf16: c * s * g in fp32, then rounded to bf16.  (Two roundings: within
// 1/2 + 2^-17 of a bf16 step.  One would take three more instructions a channel.)
__device__ __forceinline__ uint4 q4_values_bf16(uint32_t word, uint32_t sf, float g) {
    uint32_t e[4];
    e2m1x8_to_f16(word, e);
    const float s = e4m3_to_f32(sf);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // c * s is exact in fp32
        o[i] = pack_bf16(f16_lo(e[i]) * s * g, f16_hi(e[i]) * s * g);
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Arguments of the rotary append kernels.
struct AppendArgs {
    void *k, *v, *k_sf, *v_sf, *desc;   // k_sf, v_sf: 4-bit cache only
    const float *k_scale, *v_scale;
    const void *q, *kn, *vn;
    void *q_out;
    long long q_stride, k_stride, v_stride;  // elements
    const int32_t *page_table, *seq_len, *n_new, *positions;
    const float *inv_freq;
    double mscale;
    int f, rot, interleaved;
};
cudaError_t launch_append_rope(const Shape &s, const AppendArgs &a, bool q4, uint32_t *err,
                               cudaStream_t st);
cudaError_t launch_expand_q4(const Shape &s, const Q4Cache &c, const int32_t *page_table,
                             const int32_t *seq_len, void *k_out, void *v_out, uint32_t *err,
                             cudaStream_t st);
// Split-KV attention over a 4-bit cache.  block_idx == nullptr: every position
// (query rows f, row r of n sees positions 0 .. L - n + r); else the listed
// blocks (f = 1).  At most kMaxGroup rows f * g.
cudaError_t launch_decode_q4(const Shape &s, const Q4Cache &c, const int32_t *page_table,
                             const int32_t *seq_len, const void *q, int f, const int32_t *n_new,
                             const int32_t *block_idx, const int32_t *block_cnt,
                             int max_topk, int sms, float *part_o, float *part_ml,
                             uint32_t *grid_bar, float *out, float *lse, uint32_t *err,
                             cudaStream_t st);
// The chunk attention's partial row groups: one a CTA for the first unit of its share, and for a
// unit that begins further on in a share one by its number (by the CTA's where there are more
// units than CTAs).  A slot a unit and not a second one a CTA: with few units the partials are
// then no larger than the bf16 rectification's, whose place in the workspace they take.
__host__ __device__ inline int chunk_q4_later_slot(int units, int u, int cta) {
    return kNumSms + (units < kNumSms ? u : cta);
}
inline size_t chunk_q4_slots(int units) { return kNumSms + (units < kNumSms ? units : kNumSms); }
inline size_t chunk_q4_partial_floats(int units, int d) {  // of O; (max, sum) pairs follow
    return chunk_q4_slots(units) * kRectRowsPerCta * d;
}
inline size_t chunk_q4_bytes(int units, int d) {
    return (chunk_q4_partial_floats(units, d) + chunk_q4_slots(units) * kRectRowsPerCta * 2) * 4;
}
// The same for chunks of more than kMaxGroup rows, on tcgen05 (part_o and part_ml: chunk_q4_slots
// row groups; grid_bar: a 64-bit barrier word).
cudaError_t launch_chunk_q4(const Shape &s, const Q4Cache &c, const int32_t *page_table,
                            const int32_t *seq_len, const void *q, int f, const int32_t *n_new,
                            int sms, float *part_o, float *part_ml, uint32_t *grid_bar, float *out,
                            float *lse, uint32_t *err, cudaStream_t st);

}  // namespace resa
