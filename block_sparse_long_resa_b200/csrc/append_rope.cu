// Append of fresh tokens to a paged cache with the rotary embedding applied on
// the way, to bf16 pages or to the 4-bit format, and the 4-bit cache's
// expansion to bf16 pages (ReSA summary §3.2 "Block Key Cache", Eq. 3;
// Algorithm 1 incremental updates, for any number of tokens).
//
// Grid (CTAs of keys and values, then CTAs of queries; batch).  A key CTA owns
// one block of the cache that holds fresh tokens and a range of kv heads, so it
// alone writes that block's slots and its descriptor: 16 tokens at a time it
// brings the keys as stored (rotated, or read back from the cache below the
// first fresh slot) into shared memory and folds their min / max per channel.
// A query CTA rotates up to kQueryTokens tokens of every query head.  The
// angles of a CTA's tokens are worked out once, in a shared table, and used by
// all its heads.
//
// An angle is pos * inv_freq in turns in fp64, reduced to [-1/2, 1/2] before
// the sine, so that a position of 2^20 has as good an angle as position 1.  Keys
// are rotated in fp64: their 4-bit codes are decisions, and an fp32 rotation
// would move about one key in 10^4 to the neighbouring bf16 value.
#include "q4_common.cuh"

namespace resa {
namespace {

constexpr int kThreads = 256;
constexpr int kQueryTokens = 16;  // tokens a query CTA rotates
constexpr double kInvTwoPi = 0.15915494309189533577;

struct AppendGeom {
    int hq, hkv, heads;  // heads: kv heads a key CTA takes
    int max_pages, num_pages, bs;
    int key_ctas;        // CTAs of keys and values along x
    RowMap rm;
};

// Position of token r of sequence b (cache position pos), as a turn count of
// frequency i reduced to [-1/2, 1/2].
__device__ __forceinline__ double turns(const AppendArgs &a, int b, int r, int pos, int i) {
    const int p = a.positions ? a.positions[(size_t)b * a.f + r] : pos;
    const double t = (double)p * ((double)a.inv_freq[i] * kInvTwoPi);
    return t - rint(t);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(double x) { return __double2float_rn(x); }

// Rotate eight pairs: x1, x2 hold the pairs' channels as bf16, cs their
// (cos, sin) in T; results in place, rounded to bf16.
template <typename T, typename T2>
__device__ __forceinline__ void rotate8(uint4 &x1, uint4 &x2, const T2 *cs) {
    uint32_t *w1 = &x1.x, *w2 = &x2.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const T2 p = cs[2 * i], q = cs[2 * i + 1];
        const T a0 = bf_lo(w1[i]), a1 = bf_hi(w1[i]), b0 = bf_lo(w2[i]), b1 = bf_hi(w2[i]);
        w1[i] = pack_bf16(to_f32(a0 * p.x - b0 * p.y), to_f32(a1 * q.x - b1 * q.y));
        w2[i] = pack_bf16(to_f32(b0 * p.x + a0 * p.y), to_f32(b1 * q.x + a1 * q.y));
    }
}
// The same for four pairs of adjacent channels in one 16-byte vector.
template <typename T, typename T2>
__device__ __forceinline__ void rotate4_adjacent(uint4 &x, const T2 *cs) {
    uint32_t *w = &x.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const T2 p = cs[i];
        const T a = bf_lo(w[i]), b = bf_hi(w[i]);
        w[i] = pack_bf16(to_f32(a * p.x - b * p.y), to_f32(b * p.x + a * p.y));
    }
}

// Fold a pair of keys into a running (min, max), as fold8 does.
__device__ __forceinline__ void fold2(uint32_t &mn, uint32_t &mx, uint32_t x) {
    mn = (bf_lo(x) < bf_lo(mn) ? x & 0xffffu : mn & 0xffffu) |
         (bf_hi(x) < bf_hi(mn) ? x & 0xffff0000u : mn & 0xffff0000u);
    mx = (bf_lo(x) > bf_lo(mx) ? x & 0xffffu : mx & 0xffffu) |
         (bf_hi(x) > bf_hi(mx) ? x & 0xffff0000u : mx & 0xffff0000u);
}

// Work items of one head row of D channels: rotated items first (a pair of
// 16-byte vectors half a rotation apart, or one vector of adjacent pairs), then
// the vectors that are copied.
template <int D>
struct RowItems {
    int rotated, all;
    __device__ __forceinline__ RowItems(int rot, int interleaved)
        : rotated(interleaved ? rot / 8 : rot / 16), all(rotated + (D - rot) / 8) {}
};

// Apply item `it` of a row: src and dst in 16-byte vectors of the row.
template <int D, typename T, typename T2>
__device__ __forceinline__ void rotate_item(const uint4 *src, uint4 *dst, uint4 *dst2, int it,
                                            const RowItems<D> &ri, int rot, int interleaved,
                                            const T2 *cs) {
    if (it >= ri.rotated) {
        const int c = rot / 8 + it - ri.rotated;
        const uint4 x = src[c];
        dst[c] = x;
        if (dst2) dst2[c] = x;
    } else if (interleaved) {
        uint4 x = src[it];
        rotate4_adjacent<T>(x, cs + 4 * it);
        dst[it] = x;
        if (dst2) dst2[it] = x;
    } else {
        uint4 x1 = src[it], x2 = src[it + rot / 16];
        rotate8<T>(x1, x2, cs + 8 * it);
        dst[it] = x1;
        dst[it + rot / 16] = x2;
        if (dst2) {
            dst2[it] = x1;
            dst2[it + rot / 16] = x2;
        }
    }
}

template <int D, bool Q4>
__global__ void __launch_bounds__(kThreads)
    append_rope_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ AppendGeom gm,
                       uint32_t *err) {
    constexpr int CPR = D / 8;  // 16-byte vectors a row
    extern __shared__ __align__(16) uint8_t smem[];
    pdl_wait();
    const int b = blockIdx.y, tid = threadIdx.x;
    const bool first = blockIdx.x == 0 && tid == 0;
    const int n = a.n_new ? a.n_new[b] : a.f;
    if (n == 0) return;
    const int row = cache_row(gm.rm, b, first ? err : nullptr);
    const int L = row_seq_len(a.seq_len, row);
    if (L < 0 || (long long)L > (long long)gm.max_pages * gm.bs || row < 0) {
        if (first) set_error(err, RESA_DEVERR_SEQ_LEN);
        return;
    }
    if (n < 0 || n > a.f || n > L) {
        if (first) set_error(err, RESA_DEVERR_CHUNK);
        return;
    }
    const int start = L - n;  // cache position of the first fresh token
    const int half = a.rot / 2;
    const RowItems<D> ri(a.rot, a.interleaved);

    if ((int)blockIdx.x >= gm.key_ctas) {  // ------------------------------- queries
        const int r0 = ((int)blockIdx.x - gm.key_ctas) * kQueryTokens;
        const int nt = min(kQueryTokens, n - r0);
        if (nt <= 0) return;
        float2 *tab = reinterpret_cast<float2 *>(smem);  // [kQueryTokens][half]
        for (int e = tid; e < nt * half; e += kThreads) {
            const int t = e / half, i = e - t * half;
            float s, c;
            sincospif(2.f * (float)turns(a, b, r0 + t, start + r0 + t, i), &s, &c);
            const float m = (float)a.mscale;
            tab[t * half + i] = make_float2(c * m, s * m);
        }
        __syncthreads();
        const uint16_t *q = static_cast<const uint16_t *>(a.q);
        uint16_t *qo = static_cast<uint16_t *>(a.q_out);
        for (int e = tid; e < nt * gm.hq * ri.all; e += kThreads) {
            const int th = e / ri.all, it = e - th * ri.all;
            const int t = th / gm.hq, h = th - t * gm.hq;
            const size_t tok = (size_t)b * a.f + r0 + t;
            rotate_item<D, float>(
                reinterpret_cast<const uint4 *>(q + tok * a.q_stride + (size_t)h * D),
                reinterpret_cast<uint4 *>(qo + (tok * gm.hq + h) * D), nullptr, it, ri, a.rot,
                a.interleaved, tab + t * half);
        }
        return;
    }

    // ------------------------------------------------------------ keys and values
    const int groups = gm.hkv / gm.heads;
    const int blk = start / gm.bs + (int)blockIdx.x / groups;
    const int h0 = ((int)blockIdx.x % groups) * gm.heads;
    if (blk > (L - 1) / gm.bs) return;
    const int page = a.page_table[(size_t)row * gm.max_pages + blk];
    if (page < 0 || page >= gm.num_pages) {
        if (tid == 0) set_error(err, RESA_DEVERR_PAGE);
        return;
    }
    double2 *tab = reinterpret_cast<double2 *>(smem);                       // [16][half]
    uint4 *keys = reinterpret_cast<uint4 *>(smem + kTileRows * half * 16);  // [16][heads][CPR]
    const int valid = min(gm.bs, L - blk * gm.bs);  // slots of the block below seq_len
    const int pos0 = blk * gm.bs;
    const size_t prow = (size_t)page * gm.hkv;  // (page, head) row base
    constexpr int kFold = kMaxKvHeads * (D / 2) / kThreads;  // channel pairs a thread folds
    uint32_t mn[kFold], mx[kFold];  // bf16 pairs
#pragma unroll
    for (int j = 0; j < kFold; ++j) mn[j] = mx[j] = 0u;
    bool bad = false;

    for (int t0 = 0; t0 < valid; t0 += kTileRows) {
        const int nt = min(kTileRows, valid - t0);
        const int fresh0 = max(0, min(nt, start - pos0 - t0));  // first fresh slot of these
        const int nf = nt - fresh0;
        const int r0 = pos0 + t0 + fresh0 - start;  // its row in the call's arrays
        if (t0) __syncthreads();
        for (int e = tid; e < nf * half; e += kThreads) {
            const int t = e / half, i = e - t * half;
            double s, c;
            sincospi(2.0 * turns(a, b, r0 + t, start + r0 + t, i), &s, &c);
            tab[t * half + i] = make_double2(c * a.mscale, s * a.mscale);
        }
        // keys below the first fresh slot, as stored
        for (int e = tid; e < fresh0 * gm.heads * CPR; e += kThreads) {
            const int th = e / CPR, c = e - th * CPR;
            const int t = th / gm.heads, h = th - t * gm.heads;
            const size_t slot = (prow + h0 + h) * gm.bs + t0 + t;
            if (Q4) {
                const uint32_t w = static_cast<const uint32_t *>(a.k)[slot * CPR + c];
                const uint32_t sf = static_cast<const uint8_t *>(a.k_sf)[slot * (D / 16) + c / 2];
                keys[e] = q4_values_bf16(w, sf, head_scale(a.k_scale, h0 + h));
            } else {
                keys[e] = static_cast<const uint4 *>(a.k)[slot * CPR + c];
            }
        }
        // values
        if (Q4) {
            for (int e = tid; e < nf * gm.heads * (D / 16); e += kThreads) {
                const int th = e / (D / 16), gi = e - th * (D / 16);
                const int t = th / gm.heads, h = th - t * gm.heads;
                const size_t tok = (size_t)b * a.f + r0 + t;
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    static_cast<const uint16_t *>(a.vn) + tok * a.v_stride + (size_t)(h0 + h) * D +
                    gi * 16);
                const uint4 x0 = src[0], x1 = src[1];
                const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                float x[kQ4Group];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[2 * i] = bf_lo(w[i]);
                    x[2 * i + 1] = bf_hi(w[i]);
                }
                uint2 codes;
                uint32_t sf;
                bad |= q4_quantise(x, 1.f / head_scale(a.v_scale, h0 + h), codes, sf);
                const size_t slot = (prow + h0 + h) * gm.bs + t0 + fresh0 + t;
                static_cast<uint2 *>(a.v)[slot * (D / 16) + gi] = codes;
                static_cast<uint8_t *>(a.v_sf)[slot * (D / 16) + gi] = (uint8_t)sf;
            }
        } else {
            for (int e = tid; e < nf * gm.heads * CPR; e += kThreads) {
                const int th = e / CPR, c = e - th * CPR;
                const int t = th / gm.heads, h = th - t * gm.heads;
                const size_t tok = (size_t)b * a.f + r0 + t;
                const size_t slot = (prow + h0 + h) * gm.bs + t0 + fresh0 + t;
                static_cast<uint4 *>(a.v)[slot * CPR + c] = reinterpret_cast<const uint4 *>(
                    static_cast<const uint16_t *>(a.vn) + tok * a.v_stride + (size_t)(h0 + h) * D)[c];
            }
        }
        __syncthreads();
        // fresh keys, rotated, into shared memory (and the bf16 cache)
        for (int e = tid; e < nf * gm.heads * ri.all; e += kThreads) {
            const int th = e / ri.all, it = e - th * ri.all;
            const int t = th / gm.heads, h = th - t * gm.heads;
            const size_t tok = (size_t)b * a.f + r0 + t;
            const size_t slot = (prow + h0 + h) * gm.bs + t0 + fresh0 + t;
            rotate_item<D, double>(
                reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.kn) +
                                                tok * a.k_stride + (size_t)(h0 + h) * D),
                keys + ((fresh0 + t) * gm.heads + h) * CPR,
                Q4 ? nullptr : static_cast<uint4 *>(a.k) + slot * CPR, it, ri, a.rot, a.interleaved,
                tab + t * half);
        }
        __syncthreads();
        if (Q4) {
            // 4-bit codes of the fresh keys; shared memory then holds what they stand for
            for (int e = tid; e < nf * gm.heads * (D / 16); e += kThreads) {
                const int th = e / (D / 16), gi = e - th * (D / 16);
                const int t = th / gm.heads, h = th - t * gm.heads;
                uint4 *kp = keys + ((fresh0 + t) * gm.heads + h) * CPR + 2 * gi;
                const uint32_t w[8] = {kp[0].x, kp[0].y, kp[0].z, kp[0].w,
                                       kp[1].x, kp[1].y, kp[1].z, kp[1].w};
                float x[kQ4Group];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[2 * i] = bf_lo(w[i]);
                    x[2 * i + 1] = bf_hi(w[i]);
                }
                const float g = head_scale(a.k_scale, h0 + h);
                uint2 codes;
                uint32_t sf;
                bad |= q4_quantise(x, 1.f / g, codes, sf);
                const size_t slot = (prow + h0 + h) * gm.bs + t0 + fresh0 + t;
                static_cast<uint2 *>(a.k)[slot * (D / 16) + gi] = codes;
                static_cast<uint8_t *>(a.k_sf)[slot * (D / 16) + gi] = (uint8_t)sf;
                kp[0] = q4_values_bf16(codes.x, sf, g);
                kp[1] = q4_values_bf16(codes.y, sf, g);
            }
            __syncthreads();
        }
        const uint32_t *kw = reinterpret_cast<const uint32_t *>(keys);
#pragma unroll
        for (int j = 0; j < kFold; ++j) {
            const int e = tid + j * kThreads;  // (head, channel pair)
            if (e < gm.heads * (D / 2)) {
                for (int t = 0; t < nt; ++t) {
                    const uint32_t w = kw[t * gm.heads * (D / 2) + e];
                    if (t0 + t == 0)
                        mn[j] = mx[j] = w;
                    else
                        fold2(mn[j], mx[j], w);
                }
            }
        }
    }
    uint32_t *desc = static_cast<uint32_t *>(a.desc);
#pragma unroll
    for (int j = 0; j < kFold; ++j) {
        const int e = tid + j * kThreads;
        if (e < gm.heads * (D / 2)) {
            const int h = e / (D / 2), c = e - h * (D / 2);
            uint32_t *d = desc + (prow + h0 + h) * D + c;  // [2][D / 2] words a (page, head)
            d[0] = mn[j];
            d[D / 2] = mx[j];
        }
    }
    if (Q4 && bad) set_error(err, RESA_DEVERR_NONFINITE);
}

// ---------------------------------------------------------------------------
// 4-bit pages to bf16 pages
// ---------------------------------------------------------------------------
constexpr int kExpandTokens = 64;  // positions a CTA expands

// Grid (ceil(max positions / kExpandTokens), batch).  A thread turns eight
// channels (4 bytes of codes) into one 16-byte vector, so reads and writes of a
// warp are contiguous runs.
template <int D>
__global__ void __launch_bounds__(kThreads)
    expand_q4_kernel(const Q4Cache c, const int32_t *__restrict__ page_table,
                     const int32_t *__restrict__ seq_len, uint4 *__restrict__ k_out,
                     uint4 *__restrict__ v_out, int hkv, int max_pages, int num_pages, int bs,
                     const RowMap rm, uint32_t *err) {
    constexpr int CPR = D / 8;
    pdl_wait();
    const int b = blockIdx.y, tid = threadIdx.x;
    const bool first = blockIdx.x == 0 && tid == 0;
    const int row = cache_row(rm, b, first ? err : nullptr);
    const int L = row_seq_len(seq_len, row);
    if (L < 0 || (long long)L > (long long)max_pages * bs || row < 0) {
        if (first) set_error(err, RESA_DEVERR_SEQ_LEN);
        return;
    }
    const long long p0 = (long long)blockIdx.x * kExpandTokens;
    const int per_page = hkv * bs * CPR;
    for (long long p = p0; p < p0 + kExpandTokens && p < L; p += bs) {
        const int blk = (int)(p / bs), valid = min(bs, L - (int)p);
        const int page = page_table[(size_t)row * max_pages + blk];
        if (page < 0 || page >= num_pages) {
            if (tid == 0) set_error(err, RESA_DEVERR_PAGE);
            continue;
        }
        const size_t base = (size_t)page * per_page;
        for (int e = tid; e < 2 * per_page; e += kThreads) {
            const bool is_v = e >= per_page;
            const int i = is_v ? e - per_page : e;
            const int hs = i / CPR, h = hs / bs, t = hs - h * bs;
            if (t >= valid) continue;
            const uint32_t w = reinterpret_cast<const uint32_t *>(is_v ? c.v : c.k)[base + i];
            const uint32_t sf = (is_v ? c.v_sf : c.k_sf)[(base + i) / 2];
            const float g = head_scale(is_v ? c.v_scale : c.k_scale, h);
            (is_v ? v_out : k_out)[base + i] = q4_values_bf16(w, sf, g);
        }
    }
}

template <int D, bool Q4>
cudaError_t launch_append_t(const Shape &s, const AppendArgs &a, uint32_t *err, cudaStream_t st) {
    AppendGeom gm{};
    gm.hq = s.hq;
    gm.hkv = s.hkv;
    gm.heads = s.hkv;
    gm.max_pages = s.max_pages;
    gm.num_pages = s.num_pages;
    gm.bs = s.bs;
    gm.rm = s.rows;
    const int blocks = a.f / s.bs + 2;  // blocks f tokens can touch
    gm.key_ctas = (blocks < s.max_pages ? blocks : s.max_pages) * (s.hkv / gm.heads);
    const int query_ctas = a.q ? (a.f - 1) / kQueryTokens + 1 : 0;
    const size_t keys = (size_t)kTileRows * (a.rot / 2) * 16 + (size_t)kTileRows * gm.heads * D * 2;
    const size_t queries = (size_t)kQueryTokens * (a.rot / 2) * 8;
    return launch_pdl(append_rope_kernel<D, Q4>, dim3(gm.key_ctas + query_ctas, s.batch),
                      dim3(kThreads), keys > queries ? keys : queries, st, a, gm, err);
}

}  // namespace

cudaError_t launch_append_rope(const Shape &s, const AppendArgs &a, bool q4, uint32_t *err,
                               cudaStream_t st) {
    if (s.d == 128)
        return q4 ? launch_append_t<128, true>(s, a, err, st)
                  : launch_append_t<128, false>(s, a, err, st);
    return q4 ? launch_append_t<64, true>(s, a, err, st) : launch_append_t<64, false>(s, a, err, st);
}

cudaError_t launch_expand_q4(const Shape &s, const Q4Cache &c, const int32_t *page_table,
                             const int32_t *seq_len, void *k_out, void *v_out, uint32_t *err,
                             cudaStream_t st) {
    const dim3 grid((unsigned)(((long long)s.max_pages * s.bs + kExpandTokens - 1) / kExpandTokens),
                    s.batch);
    auto kernel = s.d == 128 ? expand_q4_kernel<128> : expand_q4_kernel<64>;
    return launch_pdl(kernel, grid, dim3(kThreads), 0, st, c, page_table, seq_len, (uint4 *)k_out,
                      (uint4 *)v_out, s.hkv, s.max_pages, s.num_pages, s.bs, s.rows, err);
}

}  // namespace resa
