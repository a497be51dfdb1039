// Causal attention of a chunk of query rows over a 4-bit cache on the
// 5th-generation tensor cores (ReSA summary §3.4.2; prompt chunks): more than 16
// query rows of one (sequence, kv head).
//
// Rows of one (sequence, kv head) are rho = r * g + j (chunk row r, group head j),
// taken 256 at a time (a row group: two M = 128 tiles, m = 0 and 1).  A unit is
// (sequence, kv head, row group) with its tiles of 128 keys.  The tiles of all
// units form one line of W entries; CTA c of G takes [cW/G, (c+1)W/G), a run of
// pieces, each one unit's.  A unit inside one CTA is written directly; of a
// unit that spans several, each stores its partial (o, max, sum), and after a
// bounded grid barrier (cooperative launch, one CTA per SM) those CTAs merge an
// equal share of its rows, in CTA order.
//
// Warp roles (768 threads; registers moved from the others to the softmax warps):
//   warps 0-3    expand the 4-bit tiles, c * s in fp16 (exact), into 128-byte
//                swizzled operand tiles: a ring of three 32 KB slots K0 V0 K1 V1 ..;
//   warps 4-19   softmax: eight warps an M tile, two threads a row, each with 64 of
//                the tile's keys and half of O's channels; they tell each other
//                the maximum;
//   warp 20      TMEM owner and MMA issuer;
//   warps 21-22  bring the 4-bit tiles in (cp.async), two tiles ahead.
// Per M tile the chain is QK^T(i) -> softmax -> P V(i) -> QK^T(i+1); the two M
// tiles run half a period apart, so one's MMAs fill the other's softmax.
//
// Precision.  q enters as fp16 scaled per row by a power of two (its 8 bits stay
// exact), so Q K^T has exact products.  P enters as fp16 hi + lo (22 bits), both
// over the tile's S in tensor memory, 16 keys (8 + 8 columns) at a time.  The
// matrix unit truncates when it adds to its fp32 accumulator, which over a long
// sequence would be a bias of 10^-5, so O starts from zero every kChain tiles and
// is added to the row in memory, where additions round to nearest.
#include "q4_common.cuh"
#include "tc_common.cuh"

namespace resa {
namespace {

constexpr int kThreads = 768;
constexpr int kRows = kRectRowsPerCta;  // 256
constexpr int kKeys = 128;              // keys per tile
constexpr int kSlots = 3;               // fp16 operand tiles
constexpr int kRaw = 3;                 // 4-bit tiles in flight
constexpr int kConvWarps = 4, kSoftmaxWarp = 4, kMmaWarp = 20, kLoadWarp = 21, kLoadWarps = 2;
constexpr int kLaunchRegs = 80;         // 768 threads: the whole file
constexpr int kConvRegs = 72, kSoftmaxRegs = 88, kOtherRegs = 56;
static_assert(kConvRegs + 4 * kSoftmaxRegs + kOtherRegs <= 6 * kLaunchRegs, "registers of the launch");
constexpr int kChain = 16;              // tiles whose P V add up in tensor memory
constexpr int kMinTiles = 2;            // tiles a CTA takes at least, when there are few
constexpr float kShift = 12.f;          // P is stored as 2^kShift * exp2(x - m)
constexpr float kSlack = 3.f;           // growth of the maximum tolerated before rescaling

template <int D>
struct ChunkSmem {
    static constexpr int kHalves = D / 64;
    static constexpr int kHalf = 128 * 128;          // 128 rows of 64 channels
    static constexpr int kTile = kHalves * kHalf;    // one M tile of Q, or K or V
    static constexpr int kCodes = kKeys * D / 2;
    static constexpr int kScales = kKeys * D / 16;
    static constexpr int kRawStage = 2 * (kCodes + kScales);  // K codes, V codes, K and V scales
    static constexpr int kSlotOff = 2 * kTile;
    static constexpr int kRawOff = kSlotOff + kSlots * kTile;
    static constexpr int kBytes = kRawOff + kRaw * kRawStage + 1024;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 operations at a time.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float pow2i(int k) { return __int_as_float((127 + k) << 23); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void cp_async16_s(uint32_t smem_dst, const void *gsrc) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(gsrc) : "memory");
}

// Registers a thread of this warpgroup has from here on (every warp of it runs this).
template <int N, bool Up>
__device__ __forceinline__ void set_regs() {
    if constexpr (Up)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct ChunkArgs {
    Q4Cache c;
    const int32_t *page_table, *seq_len, *n_new;
    const uint16_t *q;
    float *part_o, *out, *lse;
    float2 *part_ml;
    unsigned long long *grid_bar;
    uint32_t *err;
    RowMap rm;
    int f, batch, hkv, g, groups, max_pages, num_pages, bs;
    float scale_log2;
};

// One CTA's run through the line of tiles.
struct Piece {
    int b, h, row, L, n;
    int row0, rows;   // first query row of the unit's group, rows of it
    int cnt, t0, t1;  // the unit's tiles, this piece's
    int ustart;       // the unit's first entry
    int slot;         // partial slot of the CTA: 0 for its first piece
};

struct UnitInfo {
    int b, h, row, L, n, row0, rows, cnt;
};
__device__ __forceinline__ UnitInfo chunk_unit(const ChunkArgs &a, int u, uint32_t *err) {
    UnitInfo x;
    const int rg = u % a.groups, bh = u / a.groups;
    x.b = bh / a.hkv;
    x.h = bh - x.b * a.hkv;
    x.n = a.n_new ? a.n_new[x.b] : a.f;
    x.cnt = x.rows = x.L = 0;
    x.row = -1;
    x.row0 = rg * kRows;
    if (x.n == 0) return x;
    if (x.h != 0 || rg != 0) err = nullptr;
    x.row = cache_row(a.rm, x.b, err);
    x.L = row_seq_len(a.seq_len, x.row);
    if (x.row < 0 || x.L < 0 || (long long)x.L > (long long)a.max_pages * a.bs) {
        set_error(err, RESA_DEVERR_SEQ_LEN);
        return x;
    }
    if (x.n < 0 || x.n > a.f || x.n > x.L) {
        set_error(err, RESA_DEVERR_CHUNK);
        return x;
    }
    x.rows = min(kRows, x.n * a.g - x.row0);
    if (x.rows <= 0) {
        x.rows = 0;
        return x;
    }
    const int lim = x.L - x.n + (x.row0 + x.rows - 1) / a.g + 1;  // keys the last row sees
    x.cnt = (lim + kKeys - 1) / kKeys;
    return x;
}

// First entry of CTA q's share.
__device__ __forceinline__ int entry_of(int q, int W, int G) {
    return q < G ? (int)((long long)W * q / G) : W;
}

struct Walk {
    int x, x1, ustart, u, slot;
    __device__ __forceinline__ bool next(const ChunkArgs &a, Piece &p) {
        while (x < x1) {
            const UnitInfo i = chunk_unit(a, u++, nullptr);
            if (i.cnt > 0) {
                p.b = i.b;
                p.h = i.h;
                p.row = i.row;
                p.L = i.L;
                p.n = i.n;
                p.row0 = i.row0;
                p.rows = i.rows;
                p.cnt = i.cnt;
                p.ustart = ustart;
                p.slot = slot;
                slot = 1;
                p.t0 = x - ustart;
                ustart += i.cnt;
                x = min(x1, ustart);
                p.t1 = x - p.ustart;
                return true;
            }
        }
        return false;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_q4_kernel(const __grid_constant__ ChunkArgs a) {
    using SM = ChunkSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    __shared__ uint64_t q_ready[2], slot_full[kSlots], slot_free[kSlots], s_full[2], p_full[2];
    __shared__ uint32_t tmem_base_s, sh_ok;
    __shared__ uint64_t raw_full[kRaw], raw_free[kRaw];
    __shared__ uint32_t raw_mask[kRaw];  // a raw tile's valid blocks
    __shared__ uint32_t tile_mask[4];    // a tile's valid runs of 16 keys
    __shared__ uint64_t pair_bar[8];     // the two warps of 32 rows
    __shared__ float sh_x[2][2][2][128]; // what they tell each other, two messages deep
    __shared__ int sh_sum[kThreads / 32], sh_w, sh_ctas, sh_first, sh_unit;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = a.batch * a.hkv * a.groups;
    const int cta = blockIdx.x;

    // This CTA's share of the line: prefix sums of the units' tiles.
    const int per = (units + kThreads - 1) / kThreads;
    const int u_lo = min(units, tid * per), u_hi = min(units, u_lo + per);
    int mine = 0;
    for (int u = u_lo; u < u_hi; ++u) mine += chunk_unit(a, u, nullptr).cnt;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sh_sum[warp] = incl;
    if (tid == 0) {
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(&raw_full[s], 32 * kLoadWarps + 1);
            mbar_init(&raw_free[s], kConvWarps);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&slot_full[s], 32 * kConvWarps);
            mbar_init(&slot_free[s], 1);
        }
        for (int m = 0; m < 2; ++m) {
            mbar_init(&q_ready[m], 256);
            mbar_init(&s_full[m], 1);
            mbar_init(&p_full[m], 256);
        }
        for (int x = 0; x < 8; ++x) mbar_init(&pair_bar[x], 64);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tc::tmem_alloc(&tmem_base_s, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_base_s;
    {
        int W = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) incl += sh_sum[w];
            W += sh_sum[w];
        }
        const int G = max(1, min((int)gridDim.x, (W + kMinTiles - 1) / kMinTiles));
        if (tid == 0) {
            sh_w = W;
            sh_ctas = G;
        }
        const int x0 = entry_of(cta, W, G);
        if (x0 < entry_of(cta + 1, W, G) && incl - mine <= x0 && x0 < incl) {
            int s = incl - mine;
            for (int u = u_lo; u < u_hi; ++u) {
                const int k = chunk_unit(a, u, nullptr).cnt;
                if (x0 < s + k) {
                    sh_unit = u;
                    sh_first = s;
                    break;
                }
                s += k;
            }
        }
    }
    __syncthreads();
    auto start = [&]() -> Walk {
        Walk w;
        w.x = entry_of(cta, sh_w, sh_ctas);
        w.x1 = entry_of(cta + 1, sh_w, sh_ctas);
        w.u = w.x < w.x1 ? sh_unit : 0;
        w.ustart = w.x < w.x1 ? sh_first : 0;
        w.slot = 0;
        return w;
    };

    uint8_t *slots = smem + SM::kSlotOff;
    const int hq = a.hkv * a.g;
    Piece p;

    // Registers move from the other warps to the softmax warps and back at the end.
    if (warp < 4) {  // ----------------------------------------------------- converters
        set_regs<kConvRegs, false>();
        const int bs_shift = a.bs == 64 ? 6 : a.bs == 32 ? 5 : 4;
        const uint32_t raw_s = smem_u32(smem + SM::kRawOff), slots_s = smem_u32(slots);
        // A lane converts the 16-byte chunk c (32 channels) of row r1 of every step of
        // 32 chunks.  Lanes of the upper channel half take their words in the order
        // 2 3 0 1, so that the eight lanes of a store phase meet all banks.
        constexpr int kPerRow = D / 32, kStepRows = 32 / kPerRow;
        const int r1 = lane / kPerRow, c = lane % kPerRow;
        const bool swap = c >= 2;
        const uint32_t x0 = (uint32_t)((((c & 1) * 4) ^ (swap ? 2 : 0) ^ (r1 & 7)) << 4);
        uint32_t j = 0, tiles = 0;
        bool ok = true;
        for (Walk w = start(); ok && w.next(a, p);) {
            for (int t = p.t0; t < p.t1; ++t, ++tiles) {
                const uint32_t st = tiles % kRaw;
                ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(&raw_full[st], (tiles / kRaw) & 1));
                if (!ok) break;
                const uint32_t mask = raw_mask[st];
                const int left = p.L - t * kKeys;  // rows of the tile below the length
                const bool whole_tile = left >= kKeys && mask == (1u << (kKeys >> bs_shift)) - 1u;
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++j) {
                    const uint32_t code_at = raw_s + st * SM::kRawStage + kv * SM::kCodes + lane * 16;
                    const uint32_t scale_at = raw_s + st * SM::kRawStage + 2 * SM::kCodes + kv * SM::kScales +
                                              lane * 2;
                    const uint32_t dst = slots_s + (j % kSlots) * SM::kTile + (c / 2) * SM::kHalf + r1 * 128 + x0;
                    constexpr int kSteps = kKeys / kStepRows / kConvWarps;
                    uint32_t xs[kSteps][4];
                    uint16_t sf[kSteps];
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        const int step = warp + kConvWarps * k;
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(xs[k][0]), "=r"(xs[k][1]), "=r"(xs[k][2]), "=r"(xs[k][3])
                                     : "r"(code_at + step * 512));
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(sf[k]) : "r"(scale_at + step * 64));
                    }
                    if (j >= kSlots)
                        ok = ok && mbar_wait_bounded(&slot_free[j % kSlots], ((j / kSlots) - 1) & 1);
                    if (kv == 0 && tid == 0) {
                        uint32_t m16 = 0;
                        for (int x = 0; x < kKeys / 16; ++x)
                            m16 |= ((mask >> ((x * 16) >> bs_shift)) & 1u) << x;
                        tile_mask[tiles & 3] = m16;
                    }
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        const int step = warp + kConvWarps * k;
                        if (!whole_tile) {
                            const int r = step * kStepRows + r1;
                            if (r >= left || !((mask >> (r >> bs_shift)) & 1u)) sf[k] = 0;  // counts as 0
                        }
                        const uint32_t s2 = e4m3x2_to_f16(sf[k]);
                        const uint32_t sw[2] = {__byte_perm(s2, s2, swap ? 0x3232 : 0x1010),
                                                __byte_perm(s2, s2, swap ? 0x1010 : 0x3232)};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t y[4];
                            e2m1x8_to_f16(swap ? xs[k][i ^ 2] : xs[k][i], y);
#pragma unroll
                            for (int z = 0; z < 4; ++z) y[z] = mul_f16x2(y[z], sw[i / 2]);
                            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                                             (dst + step * (kStepRows * 128)) ^ (i << 4)),
                                         "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                                         : "memory");
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&slot_full[j % kSlots]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&raw_free[st]);
            }
        }
        if (!ok && lane == 0) set_error(a.err, RESA_DEVERR_TIMEOUT);
        __syncwarp();
        set_regs<kLaunchRegs, true>();
    } else if (warp < kMmaWarp) {  // ------------------------------------------ softmax
        set_regs<kSoftmaxRegs, true>();
        const int m = (warp - kSoftmaxWarp) >> 3, hf = ((warp - kSoftmaxWarp) >> 2) & 1;
        const int r = 32 * (warp & 3) + lane;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t scol = tmem + lane_base + m * kKeys;
        constexpr int kCh = D / 2;  // channels of O a thread keeps
        const uint32_t ocol = tmem + lane_base + 2 * kKeys + m * D + hf * kCh;
        uint32_t ns = 0, nx = 0, tiles = 0;  // S tiles (and last P V) seen, messages, key tiles so far
        bool ok = true;
        // This thread's x to the other thread of its row, and that one's.
        auto exchange = [&](float x) -> float {
            sh_x[nx & 1][m][hf][r] = x;
            uint64_t *bar = &pair_bar[m * 4 + (warp & 3)];
            mbar_arrive(bar);
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, nx & 1));
            return sh_x[nx++ & 1][m][hf ^ 1][r];
        };
        for (Walk w = start(); w.next(a, p); tiles += (uint32_t)(p.t1 - p.t0)) {
            const int T = p.t1 - p.t0, nm = p.rows > 128 ? 2 : 1;
            if (m >= nm) continue;
            const int lrow = m * 128 + r, rho = p.row0 + lrow;
            const bool row_ok = lrow < p.rows;
            const int lim = row_ok ? p.L - p.n + rho / a.g + 1 : 0;     // keys the row sees
            const int lim_warp = p.L - p.n + (rho - lane) / a.g + 1;     // keys every row of the warp sees
            // Q row, scaled to [2^8, 2^9) at its largest, into the swizzled tile
            int e = 0;
            {
                const size_t orow = ((size_t)p.b * a.f + rho / a.g) * hq + (size_t)p.h * a.g + rho % a.g;
                const uint4 *src = reinterpret_cast<const uint4 *>(a.q + orow * D);
                uint32_t mag = 0;
                if (row_ok) {
#pragma unroll 4
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 x = src[c];
                        mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                                     __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
                    }
                    mag = max(mag & 0xffffu, mag >> 16);
                    // zero and non-finite rows keep factor 1
                    if (mag != 0 && mag < 0x7f80u) e = max(-110, min(119, (int)(mag >> 7) - 127 - 8));
                }
                const float f2 = pow2i(-e);
#pragma unroll 4
                for (int c = hf * (D / 16); c < (hf + 1) * (D / 16); ++c) {
                    const uint4 x = row_ok ? src[c] : make_uint4(0u, 0u, 0u, 0u);
                    const uint4 y = make_uint4(pack_f16(bf_lo(x.x) * f2, bf_hi(x.x) * f2),
                                               pack_f16(bf_lo(x.y) * f2, bf_hi(x.y) * f2),
                                               pack_f16(bf_lo(x.z) * f2, bf_hi(x.z) * f2),
                                               pack_f16(bf_lo(x.w) * f2, bf_hi(x.w) * f2));
                    *reinterpret_cast<uint4 *>(smem + m * SM::kTile + (c / 8) * SM::kHalf +
                                               swz128(r, c % 8)) = y;
                }
                fence_proxy_async_smem();
                mbar_arrive(&q_ready[m]);
            }
            const float rs = a.scale_log2 * head_scale(a.c.k_scale, p.h) * pow2i(e);
            float mx = -INFINITY, l = 0.f;
            // The row's O outside tensor memory, relative to 2^mo: in the CTA's partial slot,
            // [32-row group][channel / 4][row in group][4], so that a warp's accesses are runs.
            float4 *row_o = reinterpret_cast<float4 *>(a.part_o + (size_t)(2 * cta + p.slot) * kRows * D) +
                            ((size_t)(lrow / 32) * (D / 4) + hf * (kCh / 4)) * 32 + lane;
            float mo = -INFINITY;
            // Add the kChain tiles' O to it (relative to 2^mx).
            auto flush = [&](bool fresh) {
                const float f2 = mo == mx || mo == -INFINITY ? 1.f : ex2(mo - mx);
#pragma unroll 1
                for (int c = 0; c < kCh; c += 16) {
                    uint32_t ov[16];
                    tc::tmem_ld16(ocol + c, ov);
                    tc::tmem_wait_ld();
                    if (!row_ok) continue;
#pragma unroll
                    for (int x = 0; x < 16; x += 4) {
                        float4 v = make_float4(__uint_as_float(ov[x]), __uint_as_float(ov[x + 1]),
                                               __uint_as_float(ov[x + 2]), __uint_as_float(ov[x + 3]));
                        float4 *dst = row_o + (c + x) / 4 * 32;
                        if (fresh) {
                            __stcg(dst, v);
                        } else if (f2 == 1.f) {
                            asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst),
                                         "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                                         : "memory");
                        } else {
                            const float4 u = __ldcg(dst);
                            __stcg(dst, make_float4(fmaf(u.x, f2, v.x), fmaf(u.y, f2, v.y),
                                                    fmaf(u.z, f2, v.z), fmaf(u.w, f2, v.w)));
                        }
                    }
                }
                mo = mx;
            };
            for (int i = 0; i < T; ++i) {
                const int t0 = (p.t0 + i) * kKeys;
                ok = ok && mbar_wait_bounded(&s_full[m], ns++ & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t tm = tile_mask[(tiles + i) & 3];
                const bool full = tm == (1u << (kKeys / 16)) - 1u && t0 + kKeys <= lim_warp;
                // the row's largest logit
                float mt = -INFINITY, mt2 = -INFINITY;
                if (full) {
                    uint32_t sv[2][32];
                    tc::tmem_ld32(scol + 64 * hf, sv[0]);
                    tc::tmem_wait_ld();
                    tc::tmem_ld32(scol + 64 * hf + 32, sv[1]);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (c == 1) tc::tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; x += 4) {
                            mt = max3(mt, __uint_as_float(sv[c][x]), __uint_as_float(sv[c][x + 1]));
                            mt2 = max3(mt2, __uint_as_float(sv[c][x + 2]), __uint_as_float(sv[c][x + 3]));
                        }
                    }
                    mt = fmaxf(mt, mt2);
                } else {
#pragma unroll 1
                    for (int c = 4 * hf; c < 4 * hf + 4; ++c) {
                        uint32_t sv[16];
                        tc::tmem_ld16(scol + 16 * c, sv);
                        tc::tmem_wait_ld();
                        const int left = ((tm >> c) & 1u) ? lim - t0 - 16 * c : 0;
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            if (x < left) mt = fmaxf(mt, __uint_as_float(sv[x]));
                    }
                }
                mt = fmaxf(mt, exchange(mt)) * rs;
                if (!ok) break;
                // O of the last kChain tiles leaves tensor memory before P V overwrites it
                if (i > 0 && i % kChain == 0) flush(i == kChain);
                // The maximum moves (to a whole number, so that every factor 2^(m - m') is
                // exact) only when it grows by more than kSlack; rarely after the first tiles.
                const bool grow = mt > mx + kSlack;
                if (__any_sync(0xffffffffu, grow)) {
                    const float mn = grow ? ceilf(mt) : mx;
                    const float al = mx == -INFINITY ? 0.f : ex2(mx - mn);
                    mx = mn;
                    l *= al;
                    if (i % kChain != 0) {
#pragma unroll 1
                        for (int c = 0; c < kCh; c += 16) {
                            uint32_t ov[16];
                            tc::tmem_ld16(ocol + c, ov);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 16; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * al);
                            tc::tmem_st16(ocol + c, ov);
                        }
                    }
                }
                const float nb = mx == -INFINITY ? 0.f : kShift - mx;
                const uint64_t rs2 = pack2(rs, rs), nb2 = pack2(nb, nb), minus = pack2(-1.f, -1.f);
                uint64_t ls[2] = {0ull, 0ull};
                uint32_t sv[2][16];
                tc::tmem_ld16(scol + 64 * hf, sv[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t col = scol + 64 * hf + 16 * c;
                    uint32_t (&x)[16] = sv[c & 1];
                    tc::tmem_wait_ld();
                    if (c < 3) tc::tmem_ld16(col + 16, sv[(c + 1) & 1]);
                    if (!full) {
                        const int left = ((tm >> (4 * hf + c)) & 1u) ? lim - t0 - 64 * hf - 16 * c : 0;
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (k >= left) x[k] = 0xff800000u;
                    }
                    uint32_t pw[16];  // 8 columns of hi, 8 of lo
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float p0, p1, l0, l1;
                        unpack2(fma2(pack2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), rs2, nb2),
                                p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        const uint64_t pp = pack2(p0, p1);
                        ls[k & 1] = add2(ls[k & 1], pp);
                        // hi: the leading 11 bits, so that lo = p - hi is exact
                        const float h0 = __uint_as_float(__float_as_uint(p0) & 0xffffe000u);
                        const float h1 = __uint_as_float(__float_as_uint(p1) & 0xffffe000u);
                        unpack2(fma2(pack2(h0, h1), minus, pp), l0, l1);
                        pw[k] = pack_f16(h0, h1);
                        pw[8 + k] = pack_f16(l0, l1);
                    }
                    tc::tmem_st16(col, pw);
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                mbar_arrive(&p_full[m]);
                {
                    float l0, l1;
                    unpack2(add2(ls[0], ls[1]), l0, l1);
                    l += l0 + l1;
                }
            }
            ok = ok && mbar_wait_bounded(&s_full[m], ns++ & 1);  // the last P V
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc::fence_after_sync();
            // the row's sum over both halves of the keys, in one order
            const float lx = exchange(l);
            if (!ok) break;
            l = hf == 0 ? l + lx : lx + l;
            const bool whole = p.t0 == 0 && p.t1 == p.cnt, kept = T > kChain;
            const float inv = !whole ? 1.f : l == 0.f ? 0.f : head_scale(a.c.v_scale, p.h) / l;
            const float f2 = !kept || mo == -INFINITY ? 0.f : ex2(mo - mx);
            const size_t orow = ((size_t)p.b * a.f + rho / a.g) * hq + (size_t)p.h * a.g + rho % a.g;
            float4 *dst = whole ? reinterpret_cast<float4 *>(a.out + orow * D + hf * kCh) : row_o;
            const int step = whole ? 1 : 32;
#pragma unroll 1
            for (int c = 0; c < kCh; c += 16) {
                uint32_t ov[16];
                tc::tmem_ld16(ocol + c, ov);
                tc::tmem_wait_ld();
                if (!row_ok) continue;
#pragma unroll
                for (int x = 0; x < 16; x += 4) {
                    float4 v = make_float4(__uint_as_float(ov[x]), __uint_as_float(ov[x + 1]),
                                           __uint_as_float(ov[x + 2]), __uint_as_float(ov[x + 3]));
                    if (kept) {
                        const float4 u = __ldcg(row_o + (c + x) / 4 * 32);
                        v = make_float4(fmaf(u.x, f2, v.x), fmaf(u.y, f2, v.y), fmaf(u.z, f2, v.z),
                                        fmaf(u.w, f2, v.w));
                    }
                    dst[(c + x) / 4 * step] = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                }
            }
            if (row_ok && hf == 0) {
                if (!whole)
                    a.part_ml[(size_t)(2 * cta + p.slot) * kRows + lrow] = make_float2(mx, l);
                else if (a.lse)
                    a.lse[orow] = l > 0.f ? (mx - kShift + log2f(l)) * 0.6931471805599453f
                                  : l == 0.f ? -INFINITY : l;
            }
        }
        if (!ok && lane == 0) set_error(a.err, RESA_DEVERR_TIMEOUT);
        __syncwarp();
        set_regs<kLaunchRegs, false>();
    } else {
        set_regs<kOtherRegs, false>();
        if (warp == kMmaWarp) {  // ----------------------------------------------- MMA issuer
            // The whole warp runs the loop and one elected thread issues: with the
            // addresses uniform over the warp an MMA issues in its 64 cycles, from
            // a branch of one thread it took 120.
            constexpr uint32_t idesc_qk = tc::idesc_f16(0, 0, 0, 0, 128, kKeys);
            constexpr uint32_t idesc_pv = tc::idesc_f16(0, 0, 0, 1, 128, D);
            const bool el = tc::elect_one();
            uint32_t j = 0, np[2] = {0, 0}, nq[2] = {0, 0};  // operand tiles, P and Q tiles used
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(bar, parity));
                tc::fence_after_sync();
            };
            auto wait_slot = [&](uint32_t jj) { wait(&slot_full[jj % kSlots], (jj / kSlots) & 1); };
            // S of M tile m against operand tile jj
            auto qk = [&](int m, uint32_t jj) {
                const uint64_t qd = tc::smem_desc(smem_u32(smem), 16, 1024) + m * (SM::kTile >> 4);
                const uint64_t kd = tc::smem_desc(smem_u32(slots) + (jj % kSlots) * SM::kTile, 16, 1024);
                if (el) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = ((ks / 4) * SM::kHalf + (ks % 4) * 32) >> 4;
                        tc::mma_f16_ss(tmem + m * kKeys, qd + off, kd + off, idesc_qk, ks > 0 ? 1u : 0u);
                    }
                }
            };
            // O of M tile m from its P and operand tile jj; fresh: the first of kChain tiles
            auto pv = [&](int m, uint32_t jj, bool fresh) {
                const uint64_t vd = tc::smem_desc(smem_u32(slots) + (jj % kSlots) * SM::kTile, SM::kHalf, 1024);
                if (el) {
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk) {
                        const uint64_t bd = vd + kk * (16 * 128 >> 4);
                        const uint32_t pt = tmem + m * kKeys + kk * 16;
                        tc::mma_f16_ts(tmem + 2 * kKeys + m * D, pt, bd, idesc_pv, kk > 0 || !fresh ? 1u : 0u);
                        tc::mma_f16_ts(tmem + 2 * kKeys + m * D, pt + 8, bd, idesc_pv, 1u);
                    }
                }
            };
            auto commit = [&](uint64_t *bar) {
                if (el) tc::commit(bar);
            };
            for (Walk w = start(); ok && w.next(a, p);) {
                const int T = p.t1 - p.t0, nm = p.rows > 128 ? 2 : 1;
                wait_slot(j);
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    if (m < nm) {
                        wait(&q_ready[m], nq[m]++ & 1);
                        if (!ok) break;
                        qk(m, j);
                        commit(&s_full[m]);
                    }
                if (!ok) break;
                commit(&slot_free[j % kSlots]);
                for (int i = 0; i < T && ok; ++i, j += 2) {
                    const uint32_t jv = j + 1, jk = j + 2;
                    const bool more = i + 1 < T;
                    wait_slot(jv);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        if (m >= nm || !ok) break;
                        wait(&p_full[m], np[m]++ & 1);
                        if (!ok) break;
                        pv(m, jv, i % kChain == 0);
                        if (m == nm - 1) commit(&slot_free[jv % kSlots]);
                        if (more) {
                            if (m == 0) wait_slot(jk);
                            if (!ok) break;
                            qk(m, jk);
                        }
                        commit(&s_full[m]);  // the next S, or the last P V of the piece
                        if (more && m == nm - 1) commit(&slot_free[jk % kSlots]);
                    }
                }
            }
            if (!ok && lane == 0) set_error(a.err, RESA_DEVERR_TIMEOUT);
            __syncwarp();
        } else {  // -------------------------------------------------------- loaders
            // Runs of 16 keys are contiguous in the cache: one warp takes the even and one the
            // odd ones of a tile, a lane 16 bytes at a time.  (Bulk copies, one a run
            // and array, took 80 cycles each to issue.)
            const int lw = warp - kLoadWarp;
            const int bs_shift = a.bs == 64 ? 6 : a.bs == 32 ? 5 : 4;
            const int bpt = kKeys >> bs_shift;  // blocks a tile
            const uint32_t raw_s = smem_u32(smem + SM::kRawOff);
            uint32_t tiles = 0;
            bool ok = lw < kLoadWarps;
            for (Walk w = start(); ok && w.next(a, p);) {
                const int nblk = (p.L + a.bs - 1) >> bs_shift;
                const int32_t *pages = a.page_table + (size_t)p.row * a.max_pages;
                // Page ids 32 blocks at a time, one a lane, the next window in flight.
                const int blk0 = p.t0 * bpt, blk1 = min(nblk, p.t1 * bpt);
                auto load_win = [&](int first) -> int {
                    const int blk = blk0 + first + lane;
                    return blk < blk1 ? pages[blk] : -1;
                };
                int win_cur = load_win(0), win_next = load_win(32);
                for (int t = 0; t < p.t1 - p.t0; ++t, ++tiles) {
                    const uint32_t st = tiles % kRaw;
                    const int first = t * bpt;
                    if (first > 0 && first % 32 == 0) {
                        win_cur = win_next;
                        win_next = load_win(first + 32);
                    }
                    int page = __shfl_sync(0xffffffffu, win_cur, (first + lane) & 31);
                    const bool there = lane < bpt && blk0 + first + lane < blk1;
                    if (there && (page < 0 || page >= a.num_pages)) {
                        set_error(a.err, RESA_DEVERR_PAGE);
                        page = -1;
                    }
                    if (!there) page = -1;
                    const uint32_t mask = __ballot_sync(0xffffffffu, page >= 0);
                    if (tiles >= kRaw) ok = mbar_wait_bounded(&raw_free[st], ((tiles / kRaw) - 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    constexpr int kRunCodes = 16 * D / 2, kRunScales = 16 * D / 16;
                    const uint32_t base = raw_s + st * SM::kRawStage + lane * 16;
#pragma unroll
                    for (int k = 0; k < kKeys / 16 / kLoadWarps; ++k) {
                        const int run = lw + kLoadWarps * k;
                        const int pg = __shfl_sync(0xffffffffu, page, (run << 4) >> bs_shift);
                        if (pg >= 0) {
                            const size_t at16 = ((((size_t)pg * a.hkv + p.h) << bs_shift) >> 4) +
                                                (run & ((a.bs >> 4) - 1));  // run of 16 keys in the cache
                            const uint8_t *gk = a.c.k + at16 * kRunCodes + lane * 16;
                            const uint8_t *gv = a.c.v + at16 * kRunCodes + lane * 16;
                            const uint32_t dst = base + run * kRunCodes;
#pragma unroll
                            for (int x = 0; x < kRunCodes; x += 512) {
                                cp_async16_s(dst + x, gk + x);
                                cp_async16_s(dst + SM::kCodes + x, gv + x);
                            }
                            constexpr int kSc = kRunScales / 16;  // chunks of scales
                            if (lane < 2 * kSc) {
                                const bool is_v = lane >= kSc;
                                cp_async16_s(base + 2 * SM::kCodes + run * kRunScales +
                                                 (is_v ? SM::kScales - kRunScales : 0),
                                             (is_v ? a.c.v_sf - kRunScales : a.c.k_sf) + at16 * kRunScales + lane * 16);
                            }
                        }
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&raw_full[st]))
                                 : "memory");
                    if (lw == 0 && lane == 0) {
                        raw_mask[st] = mask;
                        mbar_arrive(&raw_full[st]);
                    }
                }
            }
            cp_async_wait<0>();
            if (!ok && lw < kLoadWarps && lane == 0) set_error(a.err, RESA_DEVERR_TIMEOUT);
        }
        __syncwarp();
        set_regs<kLaunchRegs, true>();
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);

    // The errors of every sequence.
    for (int u = cta * kThreads + tid; u < units; u += gridDim.x * kThreads) chunk_unit(a, u, a.err);
    if (gridDim.x == 1) return;

    // Merge the units that span CTAs: their CTAs take an equal share of the rows.
    __threadfence();
    __syncthreads();
    if (tid == 0) sh_ok = grid_barrier_bounded(a.grid_bar, gridDim.x) ? 1u : 0u;
    __syncthreads();
    if (!sh_ok) {
        if (tid == 0) set_error(a.err, RESA_DEVERR_TIMEOUT);
        return;
    }
    __threadfence();
    for (Walk w = start(); w.next(a, p);) {
        if (p.t0 == 0 && p.t1 == p.cnt) continue;
        const int W = sh_w, G = sh_ctas;
        const int q0 = (int)((((long long)p.ustart + 1) * G - 1) / W);
        const int q1 = (int)((((long long)p.ustart + p.cnt) * G - 1) / W);
        const int odd = entry_of(q0, W, G) < p.ustart ? 1 : 0;  // only q0's share can begin before the unit
        // a warp 32 rows and four channels of them at a time, a lane a row
        const int k = q1 - q0 + 1, items = (p.rows + 31) / 32 * (D / 4);
        const int i0 = items * (cta - q0) / k, i1 = items * (cta - q0 + 1) / k;
        const float vg = head_scale(a.c.v_scale, p.h);
        for (int it = i0 + warp; it < i1; it += kThreads / 32) {
            const int lrow = it / (D / 4) * 32 + lane, c4 = it % (D / 4);
            const float2 *mls = a.part_ml + lrow;
            const float4 *os = reinterpret_cast<const float4 *>(a.part_o) + (size_t)it * 32 + lane;
            float ms = -INFINITY, ls = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int q = q0; q <= q1; ++q) {
                const size_t sl = (size_t)(2 * q + (q == q0 ? odd : 0)) * kRows;
                const float2 ml = __ldcg(mls + sl);
                const float4 v = __ldcg(os + sl * (D / 4));
                const float mn = fmaxf(ms, ml.x);
                const float f1 = mn == -INFINITY ? 0.f : ex2(ms - mn), f2 = mn == -INFINITY ? 0.f : ex2(ml.x - mn);
                ms = mn;
                ls = ls * f1 + ml.y * f2;
                o.x = o.x * f1 + v.x * f2;
                o.y = o.y * f1 + v.y * f2;
                o.z = o.z * f1 + v.z * f2;
                o.w = o.w * f1 + v.w * f2;
            }
            if (lrow < p.rows) {
                const int rho = p.row0 + lrow;
                const size_t orow = ((size_t)p.b * a.f + rho / a.g) * hq + (size_t)p.h * a.g + rho % a.g;
                const float inv = ls == 0.f ? 0.f : vg / ls;
                reinterpret_cast<float4 *>(a.out + orow * D)[c4] =
                    make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                if (a.lse && c4 == 0)
                    a.lse[orow] = ls > 0.f ? (ms - kShift + log2f(ls)) * 0.6931471805599453f
                                  : ls == 0.f ? -INFINITY : ls;
            }
        }
    }
}

template <int D>
cudaError_t launch_t(const ChunkArgs &a, int ctas, cudaStream_t st) {
    constexpr int smem = ChunkSmem<D>::kBytes;
    static std::atomic<int> done[64];
    cudaError_t e = ensure_smem(chunk_q4_kernel<D>, smem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // the CTAs meet at a grid barrier
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, chunk_q4_kernel<D>, a);
}

}  // namespace

cudaError_t launch_chunk_q4(const Shape &s, const Q4Cache &c, const int32_t *page_table,
                            const int32_t *seq_len, const void *q, int f, const int32_t *n_new,
                            int sms, float *part_o, float *part_ml, uint32_t *grid_bar, float *out,
                            float *lse, uint32_t *err, cudaStream_t st) {
    ChunkArgs a{};
    a.c = c;
    a.page_table = page_table;
    a.seq_len = seq_len;
    a.n_new = n_new;
    a.q = static_cast<const uint16_t *>(q);
    a.part_o = part_o;
    a.out = out;
    a.lse = lse;
    a.part_ml = reinterpret_cast<float2 *>(part_ml);
    a.grid_bar = reinterpret_cast<unsigned long long *>(grid_bar);
    a.err = err;
    a.rm = s.rows;
    a.f = f;
    a.batch = s.batch;
    a.hkv = s.hkv;
    a.g = s.g;
    a.groups = rect_row_groups(f, s.g);
    a.max_pages = s.max_pages;
    a.num_pages = s.num_pages;
    a.bs = s.bs;
    a.scale_log2 = s.sm_scale * 1.4426950408889634f;
    // one CTA per SM, no more than the longest sequences could use
    const long long most = (long long)s.batch * s.hkv * a.groups *
                           (((long long)s.max_pages * s.bs + kKeys - 1) / kKeys);
    long long ctas = sms < kNumSms ? sms : kNumSms;
    const long long need = (most + kMinTiles - 1) / kMinTiles;
    if (need < ctas) ctas = need;
    return s.d == 128 ? launch_t<128>(a, (int)ctas, st) : launch_t<64>(a, (int)ctas, st);
}

}  // namespace resa
