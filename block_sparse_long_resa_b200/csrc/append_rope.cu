// Append of fresh tokens to a paged cache with the rotary embedding applied on
// the way, to bf16 pages or to the 4-bit format, and the 4-bit cache's
// expansion to bf16 pages (ReSA summary §3.2 "Block Key Cache", Eq. 3;
// Algorithm 1 incremental updates, for any number of tokens).
//
// Grid (key and token clusters in turns; batch).  A key cluster owns one block of the
// cache that holds fresh tokens and a range of kv heads, so it alone writes that
// block's keys and its descriptor.  Each of its CTAs brings 16 tokens' keys as stored
// (rotated, or read back from the cache below the first fresh slot) into shared
// memory and folds their min / max per channel, and through the cluster's shared memory
// they fold the block's (with one CTA for the four tiles of a 64-token block five prompts
// took 55 us, not 48).  Of a token CTA a warp, or several where there are few tokens,
// takes a token: its queries and its values.
//
// An angle is pos * inv_freq in turns in fp64, reduced to [-1/2, 1/2] before
// the sine, so that the angle of a position of 2^20 is off by 2^-31 at most.  Keys
// are rotated in fp64: their 4-bit codes are decisions, and an fp32 rotation
// would move about one key in 10^4 to the neighbouring bf16 value.  (The fp64 result
// is rounded to fp32 and then to bf16, which moves one in 10^5 that lies by a halfway
// point: within 1/2 + 2^-17 of a step.)
//
// Measured (28 q / 4 kv heads, d 128): 8192 tokens, 152 MB, 32 us, 4.7 TB/s, bound by
// the latency of 24 warps an SM (80 registers) more than by a unit (issue 57 %, exp and
// sine unit 22 %, fp64 5 %); one token of each of 32 sequences 5.2 us, the host's side of a
// call.
// Five ragged prompts of up to 2777 tokens into 4-bit pages (32 / 8 heads, d 128) and the
// pages' expansion, 189 MB together, take 58 us: the groups' maxima, scales and codes
// are added to each key and value.
#include <cooperative_groups.h>

#include "q4_common.cuh"

namespace cg = cooperative_groups;

namespace resa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr double kInvTwoPi = 0.15915494309189533577;

struct AppendGeom {
    int hq, hkv, lg_heads;  // 2^lg_heads kv heads a key CTA takes
    int max_pages, num_pages, bs;
    int key_clusters;    // clusters of keys along x
    int q_tokens;        // tokens a token CTA takes: 1, 2, 4 or 8
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
// (cos, sin) in T; results in place, rounded to fp32 and then to bf16.
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

// A head row of D channels is D / 16 slots of two 16-byte vectors each, such that
// neighbouring slots' vectors are neighbours: a pair of vectors half a rotation
// apart, two vectors of adjacent pairs half a row apart, or two that are copied.
struct Slot {
    int c1, c2;    // the vectors
    int f1, f2;    // first of the four frequencies of each half of the slot
    bool r1, r2;   // rotated
};
template <int D>
__device__ __forceinline__ Slot slot_of(int it, int rot, int interleaved) {
    Slot s;
    if (interleaved) {
        s.c1 = it;
        s.c2 = it + D / 16;
        s.f1 = 4 * s.c1;
        s.f2 = 4 * s.c2;
    } else if (it < rot / 16) {
        s.c1 = it;
        s.c2 = it + rot / 16;
        s.f1 = 8 * it;
        s.f2 = 8 * it + 4;
    } else {
        s.c1 = rot / 16 + it;
        s.c2 = it + D / 16;
        s.f1 = s.f2 = 0;
    }
    s.r1 = s.c1 < rot / 8;
    s.r2 = s.c2 < rot / 8;
    return s;
}
// Rotate them; cs: (cos, sin) of the slot's eight frequencies.
template <typename T, typename T2>
__device__ __forceinline__ void rotate_slot(uint4 &x1, uint4 &x2, const Slot &s, int interleaved,
                                            const T2 (&cs)[8]) {
    if (interleaved) {
        if (s.r1) rotate4_adjacent<T>(x1, cs);
        if (s.r2) rotate4_adjacent<T>(x2, cs + 4);
    } else if (s.r1) {
        rotate8<T>(x1, x2, cs);
    }
}

template <int D, bool Q4>
__global__ void __launch_bounds__(kThreads, 3)
    append_rope_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ AppendGeom gm,
                       uint32_t *err) {
    constexpr int CPR = D / 8;     // 16-byte vectors a row
    constexpr int SPR = D / 16;    // slots a row, and groups of 16 channels
    extern __shared__ __align__(16) uint8_t smem[];
    pdl_launch_next();
    pdl_wait();
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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

    // Key and token clusters, of a CTA for each tile of a block, take turns along x, so that
    // they share the SMs.
    const int tiles = gm.bs / kTileRows, clusters = gridDim.x / tiles;
    const int cluster = blockIdx.x / tiles, rank = blockIdx.x % tiles;
    const int ki = (int)((long long)cluster * gm.key_clusters / clusters);
    bool bad = false;
    if ((int)(((long long)cluster + 1) * gm.key_clusters / clusters) == ki) {  // ---- a token's queries and values
        // warps per token: 8 / q_tokens, each a share of the vectors
        const int wpt = kWarps / gm.q_tokens, step = 32 * wpt;
        const int r = ((cluster - ki) * tiles + rank) * gm.q_tokens + warp / wpt;
        if (r >= n) return;
        const size_t tok = (size_t)b * a.f + r;
        const int pos = start + r;
        const int page = a.page_table[(size_t)row * gm.max_pages + pos / gm.bs];
        if (page >= 0 && page < gm.num_pages) {  // (the key CTA reports it)
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.vn) + tok * a.v_stride);
            const size_t slot0 = (size_t)page * gm.hkv * gm.bs + pos % gm.bs;
#pragma unroll 2
            for (int e = (warp % wpt) * 32 + lane; e < gm.hkv * (Q4 ? SPR : CPR); e += step) {
                if (Q4) {
                    const int h = e / SPR;
                    const uint4 x0 = src[2 * e], x1 = src[2 * e + 1];
                    const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                    uint2 codes;
                    uint32_t sf;
                    bad |= q4_quantise(w, 1.f / head_scale(a.v_scale, h), codes, sf);
                    const size_t at = (slot0 + (size_t)h * gm.bs) * SPR + e % SPR;
                    static_cast<uint2 *>(a.v)[at] = codes;
                    static_cast<uint8_t *>(a.v_sf)[at] = (uint8_t)sf;
                } else {
                    static_cast<uint4 *>(a.v)[(slot0 + (size_t)(e / CPR) * gm.bs) * CPR + e % CPR] = src[e];
                }
            }
        }
        if (Q4 && bad) set_error(err, RESA_DEVERR_NONFINITE);
        if (!a.q) return;
        float2 *tab = reinterpret_cast<float2 *>(smem) + warp * (D / 2);
        for (int i = lane; i < half; i += 32) {
            float s, c;
            sincospif(2.f * (float)turns(a, b, r, start + r, i), &s, &c);
            const float m = (float)a.mscale;
            tab[i] = make_float2(c * m, s * m);
        }
        __syncwarp();
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + tok * a.q_stride);
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.q_out) + tok * gm.hq * D);
        const int slots = gm.hq * SPR;
        // a lane's slots are all slot `it` of a head: its angles stay in registers (read from
        // shared memory for each head they took most of the time)
        const Slot sl = slot_of<D>(lane % SPR, a.rot, a.interleaved);
        float2 cs[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = tab[(i < 4 ? sl.f1 : sl.f2 - 4) + i];
        constexpr int kAhead = 4;
        for (int e0 = (warp % wpt) * 32 + lane; e0 < slots; e0 += kAhead * step) {
            uint4 x1[kAhead], x2[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int e = e0 + k * step;
                if (e < slots) {
                    x1[k] = src[e / SPR * CPR + sl.c1];
                    x2[k] = src[e / SPR * CPR + sl.c2];
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int e = e0 + k * step;
                if (e < slots) {
                    rotate_slot<float>(x1[k], x2[k], sl, a.interleaved, cs);
                    dst[e / SPR * CPR + sl.c1] = x1[k];
                    dst[e / SPR * CPR + sl.c2] = x2[k];
                }
            }
        }
        return;
    }

    // ----------------------------------------------------------------------- keys
    const int heads = 1 << gm.lg_heads, groups = gm.hkv >> gm.lg_heads;
    const int blk = start / gm.bs + ki / groups;
    const int h0 = (ki % groups) * heads;
    if (blk > (L - 1) / gm.bs) return;
    const int page = a.page_table[(size_t)row * gm.max_pages + blk];
    if (page < 0 || page >= gm.num_pages) {
        if (tid == 0) set_error(err, RESA_DEVERR_PAGE);
        return;
    }
    uint4 *keys = reinterpret_cast<uint4 *>(smem);  // [16][head][CPR]
    // Angle i of a token lies at i ^ (i / 8 % 8), so that eight lanes with eight slots
    // meet all banks.
    double2 *tab = reinterpret_cast<double2 *>(smem + (kTileRows * D * 2 << gm.lg_heads));  // [16][D / 2]
    const int pos0 = blk * gm.bs;
    const int valid = min(gm.bs, L - pos0);          // slots of the block below seq_len
    const int fresh0 = max(0, start - pos0);         // the first fresh one
    const size_t prow = (size_t)page * gm.hkv + h0;  // (page, head) row base
    const int lg_row = gm.lg_heads + (D == 128 ? 3 : 2);  // slots of a token: 2^lg_row
    const Slot sl = slot_of<D>(tid % SPR, a.rot, a.interleaved);
    const int t0 = rank * kTileRows;                 // the first of this CTA's tile
    const int nt = max(0, min(kTileRows, valid - t0));
    const int old = max(0, min(nt, fresh0 - t0));                   // keys that are there already
    const int nf = nt - old;
    const int r0 = pos0 + t0 + old - start;                         // the first fresh one's row
    const int slots = nf << lg_row;
    auto src_of = [&](int e) -> const uint4 * {
        return reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.kn) +
                                               ((size_t)b * a.f + r0 + (e >> lg_row)) * a.k_stride +
                                               (size_t)(h0 + (e / SPR & (heads - 1))) * D);
    };
    // a thread's first vectors are on their way while the angles are worked out
    constexpr int kAhead = 2;
    uint4 x1[kAhead], x2[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (tid + k * kThreads < slots) {
            const uint4 *src = src_of(tid + k * kThreads);
            x1[k] = src[sl.c1];
            x2[k] = src[sl.c2];
        }
#pragma unroll 2
    for (int e = tid; e < nf * half; e += kThreads) {
        const int t = e / half, i = e - t * half;
        double s, c;
        sincospi(2.0 * turns(a, b, r0 + t, start + r0 + t, i), &s, &c);
        tab[t * (D / 2) + (i ^ (i / 8 % 8))] = make_double2(c * a.mscale, s * a.mscale);
    }
    for (int e = tid; e < old * heads * CPR; e += kThreads) {
        const int c = e % CPR, th = e / CPR;
        const int h = th & (heads - 1), t = t0 + (th >> gm.lg_heads);
        const size_t slot = (prow + h) * gm.bs + t;
        if (Q4) {
            const uint32_t w = static_cast<const uint32_t *>(a.k)[slot * CPR + c];
            const uint32_t sf = static_cast<const uint8_t *>(a.k_sf)[slot * SPR + c / 2];
            keys[e] = q4_values_bf16(w, sf, head_scale(a.k_scale, h0 + h));
        } else {
            keys[e] = static_cast<const uint4 *>(a.k)[slot * CPR + c];
        }
    }
    __syncthreads();
    for (int e0 = tid; e0 < slots; e0 += kAhead * kThreads) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int e = e0 + k * kThreads;
            if (e >= slots) break;
            if (e0 != tid) {
                const uint4 *src = src_of(e);
                x1[k] = src[sl.c1];
                x2[k] = src[sl.c2];
            }
            const int t = e >> lg_row, h = e / SPR & (heads - 1);
            double2 cs[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int f = (i < 4 ? sl.f1 : sl.f2 - 4) + i;
                cs[i] = tab[t * (D / 2) + (f ^ (f / 8 % 8))];
            }
            rotate_slot<double>(x1[k], x2[k], sl, a.interleaved, cs);
            uint4 *dst = keys + ((old + t) * heads + h) * CPR;
            dst[sl.c1] = x1[k];
            dst[sl.c2] = x2[k];
            if (!Q4) {
                uint4 *out = static_cast<uint4 *>(a.k) + ((prow + h) * gm.bs + t0 + old + t) * CPR;
                out[sl.c1] = x1[k];
                out[sl.c2] = x2[k];
            }
        }
    }
    __syncthreads();
    if (Q4) {
        // 4-bit codes of the fresh keys; shared memory then holds what they stand for
        for (int e = tid; e < slots; e += kThreads) {
            const int gi = e % SPR, h = e / SPR & (heads - 1), t = old + (e >> lg_row);
            uint4 *kp = keys + (t * heads + h) * CPR + 2 * gi;
            const uint4 y0 = kp[0], y1 = kp[1];
            const uint32_t w[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
            const float g = head_scale(a.k_scale, h0 + h);
            uint2 codes;
            uint32_t sf;
            bad |= q4_quantise(w, 1.f / g, codes, sf);
            const size_t at = ((prow + h) * gm.bs + t0 + t) * SPR + gi;
            static_cast<uint2 *>(a.k)[at] = codes;
            static_cast<uint8_t *>(a.k_sf)[at] = (uint8_t)sf;
            kp[0] = q4_values_bf16(codes.x, sf, g);
            kp[1] = q4_values_bf16(codes.y, sf, g);
        }
        __syncthreads();
    }
    // Descriptors: a thread two channels of a head, from the neutral values in all tiles but the
    // block's first; then each CTA a share of the channels over the tiles, in order.
    const uint32_t *kw = reinterpret_cast<const uint32_t *>(keys);
    uint2 *fold = reinterpret_cast<uint2 *>(tab);  // (the angles are used up)
    const int width = heads * (D / 2);
    for (int e = tid; e < width; e += kThreads) {
        uint32_t mn = rank == 0 ? kw[e] : 0x7f807f80u, mx = rank == 0 ? kw[e] : 0xff80ff80u;
#pragma unroll 4
        for (int t = rank == 0; t < nt; ++t) fold2(mn, mx, kw[t * width + e]);
        fold[e] = make_uint2(mn, mx);
    }
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    for (int e = width * rank / tiles + tid; e < width * (rank + 1) / tiles; e += kThreads) {
        uint2 m = *cl.map_shared_rank(fold + e, 0);
        for (int q = 1; q < tiles; ++q) {
            const uint2 x = *cl.map_shared_rank(fold + e, q);
            uint32_t other = 0u;
            fold2(m.x, other, x.x);
            fold2(other, m.y, x.y);
        }
        uint32_t *d = static_cast<uint32_t *>(a.desc) + (prow + e / (D / 2)) * D + e % (D / 2);  // [2][D / 2] words
        d[0] = m.x;
        d[D / 2] = m.y;
    }
    if (tiles > 1) cl.sync();  // no CTA leaves while another reads its shared memory
    if (Q4 && bad) set_error(err, RESA_DEVERR_NONFINITE);
}

// ---------------------------------------------------------------------------
// 4-bit pages to bf16 pages
// ---------------------------------------------------------------------------
constexpr int kExpandTokens = 64;  // positions a CTA expands, or some of their groups
constexpr int kExpandAhead = 4;

// Grid (ceil(max positions / kExpandTokens), batch, parts of their groups).  A thread turns a group of 16
// channels (8 bytes of codes and a scale) into one 32-byte store, kAhead groups in
// flight; a warp's reads and writes are contiguous runs.  Measured: 4 x 65536 tokens of 4
// heads, d 128, 685 MB, 114 us, 6.0 TB/s (16-byte stores, one group in flight: 179 us).
template <int D>
__global__ void __launch_bounds__(kThreads)
    expand_q4_kernel(const __grid_constant__ Q4Cache c, const int32_t *__restrict__ page_table,
                     const int32_t *__restrict__ seq_len, uint16_t *__restrict__ k_out,
                     uint16_t *__restrict__ v_out, int lg_hkv, int max_pages, int num_pages, int lg_bs,
                     const RowMap rm, bool wide, uint32_t *err) {
    constexpr int kAhead = kExpandAhead, LG = D == 128 ? 3 : 2;  // 2^LG groups a row
    __shared__ int pages[kExpandTokens / 16];
    pdl_launch_next();
    pdl_wait();
    const int b = blockIdx.y, tid = threadIdx.x;
    const bool first = blockIdx.x == 0 && tid == 0;
    const int row = cache_row(rm, b, first ? err : nullptr);
    const int L = row_seq_len(seq_len, row);
    if (L < 0 || (long long)L > ((long long)max_pages << lg_bs) || row < 0) {
        if (first) set_error(err, RESA_DEVERR_SEQ_LEN);
        return;
    }
    const long long p0 = (long long)blockIdx.x * kExpandTokens;
    if (p0 >= L) return;
    const int left = min(kExpandTokens, L - (int)p0);  // positions of this CTA
    const int np = (left + (1 << lg_bs) - 1) >> lg_bs;  // pages of this CTA
    if (tid < np) {
        int page = page_table[(size_t)row * max_pages + (int)(p0 >> lg_bs) + tid];
        if (page < 0 || page >= num_pages) {
            set_error(err, RESA_DEVERR_PAGE);
            page = -1;
        }
        pages[tid] = page;
    }
    __syncthreads();
    const int lg_page = lg_hkv + lg_bs + LG;  // groups of a page, of K or V
    const int all = np << (lg_page + 1);
    // group e: its place in the cache, or false where there is none
    auto place = [&](int e, size_t &at, bool &is_v, int &h) -> bool {
        const int pi = e >> (lg_page + 1), i = e & ((1 << lg_page) - 1);
        const int t = (i >> LG) & ((1 << lg_bs) - 1);
        is_v = (e >> lg_page) & 1;
        h = i >> (LG + lg_bs);
        if (e >= all || (pi << lg_bs) + t >= left || pages[pi] < 0) return false;
        at = ((size_t)pages[pi] << lg_page) + i;
        return true;
    };
    for (int e0 = blockIdx.z * kAhead * kThreads + tid; e0 < all; e0 += gridDim.z * kAhead * kThreads) {
        uint2 w[kAhead];
        uint32_t sf[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            size_t at;
            bool is_v;
            int h;
            if (place(e0 + k * kThreads, at, is_v, h)) {
                w[k] = __ldcs(reinterpret_cast<const uint2 *>(is_v ? c.v : c.k) + at);
                sf[k] = (is_v ? c.v_sf : c.k_sf)[at];
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            size_t at;
            bool is_v;
            int h;
            if (place(e0 + k * kThreads, at, is_v, h)) {
                const float g = head_scale(is_v ? c.v_scale : c.k_scale, h);
                const uint4 x = q4_values_bf16(w[k].x, sf[k], g), y = q4_values_bf16(w[k].y, sf[k], g);
                uint16_t *dst = (is_v ? v_out : k_out) + at * 16;
                if (wide) {
                    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(x.x),
                                 "r"(x.y), "r"(x.z), "r"(x.w), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
                                 : "memory");
                } else {  // pages aligned to 16 bytes only
                    reinterpret_cast<uint4 *>(dst)[0] = x;
                    reinterpret_cast<uint4 *>(dst)[1] = y;
                }
            }
        }
    }
}

template <int D, bool Q4>
cudaError_t launch_append_t(const Shape &s, const AppendArgs &a, uint32_t *err, cudaStream_t st) {
    AppendGeom gm{};
    gm.hq = s.hq;
    gm.hkv = s.hkv;
    gm.max_pages = s.max_pages;
    gm.num_pages = s.num_pages;
    gm.bs = s.bs;
    gm.rm = s.rows;
    long long blocks = ((long long)a.f + s.bs - 2) / s.bs + 1;  // blocks f tokens can touch
    if (blocks > s.max_pages) blocks = s.max_pages;
    // All heads a CTA, so that the angles are worked out once, unless that leaves too few CTAs.
    int lg_heads = s.hkv == 8 ? 3 : s.hkv == 4 ? 2 : s.hkv == 2 ? 1 : 0;
    const int tiles = s.bs / kTileRows;
    while (lg_heads > 0 && blocks * tiles * s.batch * (s.hkv >> lg_heads) < 2 * kNumSms) --lg_heads;
    gm.lg_heads = lg_heads;
    gm.key_clusters = (int)blocks * (s.hkv >> lg_heads);
    gm.q_tokens = a.f >= kWarps ? kWarps : a.f >= 4 ? 4 : a.f >= 2 ? 2 : 1;
    const int token_clusters = ((a.f - 1) / gm.q_tokens + tiles) / tiles;
    const int smem = (kTileRows * D * 2 << lg_heads) + kTileRows * (D / 2) * 16;  // at most 48 KB
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((gm.key_clusters + token_clusters) * tiles, s.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = tiles;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = tiles > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, append_rope_kernel<D, Q4>, a, gm, err);
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
    // Eight CTAs an SM (five run at once) where there are the groups for it: five sequences of up
    // to 2888 tokens, 8 heads, d 128, 21.7 us with a CTA for all groups of 64 tokens, 8.6 so.
    const long long pieces = ((long long)s.max_pages * s.bs + kExpandTokens - 1) / kExpandTokens;
    const long long lack = (8 * kNumSms - 1) / (pieces * s.batch) + 1;
    const int rounds = kExpandTokens * s.hkv * (s.d / 16) * 2 / (kExpandAhead * kThreads);
    const dim3 grid((unsigned)pieces, s.batch, rounds < 1 ? 1 : lack < rounds ? (unsigned)lack : rounds);
    auto kernel = s.d == 128 ? expand_q4_kernel<128> : expand_q4_kernel<64>;
    const bool wide = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31u) == 0;
    auto lg = [](int x) { return x == 1 ? 0 : x == 2 ? 1 : x == 4 ? 2 : x == 8 ? 3 : x == 16 ? 4 : x == 32 ? 5 : 6; };
    return launch_pdl(kernel, grid, dim3(kThreads), 0, st, c, page_table, seq_len, (uint16_t *)k_out,
                      (uint16_t *)v_out, lg(s.hkv), s.max_pages, s.num_pages, lg(s.bs), s.rows, wide, err);
}

}  // namespace resa
