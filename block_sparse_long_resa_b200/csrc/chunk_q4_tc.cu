// Causal attention of a chunk of query rows over a 4-bit cache on the
// 5th-generation tensor cores (ReSA summary §3.4.2; prompt chunks): more than 16
// query rows of one (sequence, kv head).
//
// Rows of one (sequence, kv head) are rho = r * g + j (chunk row r, group head j),
// taken 256 at a time (a row group: two M = 128 tiles, m = 0 and 1).  A unit is
// (sequence, kv head, row group) with its tiles of 128 keys.  Every unit is cut
// into even shares, one a CTA, or, where that would give some CTAs much more than
// others, the tiles of all units form one line of W entries and CTA c of G takes
// [cW/G, (c+1)W/G), a run of pieces, each one unit's.  A unit inside one CTA is
// written directly; of a unit that spans several, each stores its partial (o, max,
// sum), and after a bounded grid barrier (cooperative launch, one CTA per SM)
// those CTAs merge an equal share of its rows, in CTA order.
//
// Warp roles (384 threads; registers moved from warpgroup 0 to the others):
//   warp 0      TMEM owner and MMA issuer;
//   warps 1-3   bring the 4-bit tiles in (cp.async, three raw stages) and expand
//               them, c * s in fp16 (exact), into 128-byte swizzled operand tiles:
//               a ring of three 32 KB slots K0 V0 K1 V1 ..;
//   warps 4-7, 8-11   softmax of M tile 0 and 1, one thread a row.
// Per M tile the chain is QK^T(i) -> softmax -> P V(i) -> QK^T(i+1); the two M
// tiles run half a period apart, so one's MMAs fill the other's softmax, and P V
// of a tile's first 64 keys runs while the softmax makes the others' weights.
//
// Precision.  q enters as fp16 scaled per row by a power of two (its 8 bits stay
// exact down to 2^-25 of the row's largest channel), so Q K^T has exact products.  P
// enters as fp16 hi + lo (22 bits, or 2^-36 of the row's largest weight where that is
// coarser; fp16 alone would be 1.4e-4 off), both over the tile's S in tensor memory, 16 keys
// (8 + 8 columns) at a time: P V takes twice the MMAs.  The matrix unit truncates
// when it adds to its fp32 accumulator: 1.1e-5 off after 1024 additions.  So O
// starts from zero every kChain tiles and is then added to its row in registers,
// where additions round to nearest: 7e-7 off for 2 tiles, 1.2e-6 for 4, 2.4e-6
// for 8, and 2 takes 1.2 % and 1.6 % longer than 4 and 8.
//
// Measured (28 q / 4 kv heads, d 128, 32 rows against 4 x 65536 tokens: 120 GFLOP,
// 1.5 times that in MMAs, 153 MB): 204 us, 0.59 PFLOP/s, 0.88 PFLOP/s in MMAs (185 us on
// machines that hold a higher clock under this load).
// Of a tile's 4900 cycles the chain of one M tile takes all: maximum 500, weights
// 2600 (128 exponentials a thread at 4 a cycle and SM quarter are 1024), P V of the
// second half 490, Q K^T 780.  An MMA with A in shared memory takes 97 cycles
// whatever its N up to 128, so 64-key tiles with S double-buffered, which hide
// the chain, double Q K^T and measured 250 us; two threads a row (O added up in
// memory, 4.5e-6 off) 212 us; four converter and two loader warps beside the MMA
// warp, with fewer registers for the rows, 191 us.
#include "q4_common.cuh"
#include "tc_common.cuh"

namespace resa {
namespace {

constexpr int kThreads = 384;
constexpr int kRows = kRectRowsPerCta;  // 256
constexpr int kKeys = 128;              // keys per tile
constexpr int kSlots = 3;               // fp16 operand tiles
constexpr int kRaw = 3;                 // 4-bit tiles in flight
constexpr int kConv = 96;               // converter threads
constexpr int kLaunchRegs = 168;        // 384 threads: 64512 of the file's 65536
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "registers of the launch");
constexpr int kPieceTiles = 8;          // tiles a CTA takes in the time that a second piece adds
constexpr int kMinTiles = 2;            // tiles a CTA takes at least, when there are few
constexpr int kChain = 2;               // tiles whose P V add up in tensor memory
// P is stored as 2^kShift * exp2(x - m), at most 2^(kShift + kSlack).  hi is cut off, not
// rounded, to 11 bits, so a P below fp16's normal numbers is off by half a smallest step in hi
// and another in lo, 2^-24: 2^-36 of the row's largest, which is at least 2^(kShift - 1).
constexpr float kShift = 13.f;
constexpr float kSlack = 2.f;           // growth of the maximum tolerated before rescaling

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
    int u;            // its number
    bool later;       // not the CTA's first piece
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
    x.cnt = ceil_div(lim, kKeys);
    return x;
}

// First entry of CTA q's share.
__device__ __forceinline__ int entry_of(int q, int W, int G) {
    return q < G ? (int)((long long)W * q / G) : W;
}

struct Walk {
    int x, x1, ustart, u;
    bool later;
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
                p.u = u - 1;
                p.later = later;
                later = true;
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
    __shared__ uint64_t q_ready[2], slot_full[kSlots], slot_free[kSlots], s_full[2], p_full[2][2];
    __shared__ uint32_t tmem_base_s, sh_ok;
    __shared__ uint64_t raw_full[kRaw], raw_free[kRaw];
    __shared__ uint32_t tile_mask[4];    // a tile's valid runs of 16 keys
    __shared__ int sh_sum[kThreads / 32], sh_w, sh_ctas, sh_first, sh_unit, sh_x[2], sh_most;
    __shared__ int2 sh_own;  // even shares: the CTAs of this one's unit, the first of them

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = a.batch * a.hkv * a.groups;
    const int cta = blockIdx.x;

    // This CTA's share of the units' tiles (as in the split-KV kernel): an even share of one
    // unit, so that every CTA has one piece, or, where that would give some CTAs kPieceTiles
    // more than others, a share of the line of all tiles.
    const int per = (units + kThreads - 1) / kThreads;
    const int u_lo = min(units, tid * per), u_hi = min(units, u_lo + per);
    int mine = 0;
    for (int u = u_lo; u < u_hi; ++u) mine += chunk_unit(a, u, nullptr).cnt;
    if (tid == 0) {
        sh_most = 0;
        sh_own = make_int2(0, 0);
        sh_x[0] = sh_x[1] = 0;
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(&raw_full[s], kConv);
            mbar_init(&raw_free[s], 3);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&slot_full[s], kConv);
            mbar_init(&slot_free[s], 1);
        }
        for (int m = 0; m < 2; ++m) {
            mbar_init(&q_ready[m], 128);
            mbar_init(&s_full[m], 1);
            mbar_init(&p_full[m][0], 128);
            mbar_init(&p_full[m][1], 128);
        }
        fence_mbar_init();
    }
    if (warp == 0) tc::tmem_alloc(&tmem_base_s, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_base_s;
    {
        // sums over the threads before this one and over all
        auto scan = [&](int x, int &all) -> int {
            int incl = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            __syncthreads();
            if (lane == 31) sh_sum[warp] = incl;
            __syncthreads();
            all = 0;
            int before = incl - x;
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) before += sh_sum[w];
                all += sh_sum[w];
            }
            return before;
        };
        int W;
        const int before = scan(mine, W), grid = gridDim.x;
        int share = 0;
        if (per == 1 && units < grid && W > 0) {
            if (mine > 0) atomicMax(&sh_most, mine);
            const int even = ceil_div(W, grid), last = ceil_div(W, grid - units);
#pragma unroll 1
            for (int k = 0; k < 5; ++k) {  // the smallest of five shares that keep to the grid
                share = max(kMinTiles, even + (int)((long long)(last - even) * k / 4));
                int ctas;
                const int mine_ctas = ceil_div(mine, share), first = scan(mine_ctas, ctas);
                if (ctas > grid) continue;
                if (min(share, sh_most) - max(kMinTiles, even) > kPieceTiles) share = 0;
                if (share > 0 && first <= cta && cta < first + mine_ctas) {
                    sh_unit = tid;
                    sh_first = before;
                    sh_own = make_int2(mine_ctas, first);
                    sh_x[0] = before + (cta - first) * share;
                    sh_x[1] = sh_x[0] + min(share, before + mine - sh_x[0]);
                }
                break;
            }
        }
        const int G = max(1, min(grid, ceil_div(W, kMinTiles)));
        if (tid == 0) {
            sh_w = W;
            sh_ctas = G;
        }
        if (share == 0) {
            const int x0 = entry_of(cta, W, G), x1 = entry_of(cta + 1, W, G);
            if (x0 < x1 && before <= x0 && x0 < before + mine) {  // one thread: the unit that x0 lies in
                int s = before;
                for (int u = u_lo; u < u_hi; ++u) {
                    const int k = chunk_unit(a, u, nullptr).cnt;
                    if (x0 < s + k) {
                        sh_unit = u;
                        sh_first = s;
                        sh_x[0] = x0;
                        sh_x[1] = x1;
                        break;
                    }
                    s += k;
                }
            }
        }
    }
    __syncthreads();
    auto start = [&]() -> Walk {
        Walk w;
        w.x = sh_x[0];
        w.x1 = sh_x[1];
        w.u = w.x < w.x1 ? sh_unit : 0;
        w.ustart = w.x < w.x1 ? sh_first : 0;
        w.later = false;
        return w;
    };

    uint8_t *slots = smem + SM::kSlotOff;
    const int hq = a.hkv * a.g;
    Piece p;

    // Registers move from the other warps to the softmax warps and back at the end.
    if (warp >= 4) {  // ------------------------------------------------------- softmax
        set_regs<kSoftmaxRegs, true>();
        const int m = (warp - 4) >> 2, r = (tid - 128) & 127;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t scol = tmem + lane_base + m * kKeys;
        const uint32_t ocol = tmem + lane_base + 2 * kKeys + m * D;
        uint32_t ns = 0, tiles = 0;  // S tiles (and last P V) seen, key tiles so far
        bool ok = true;
        for (Walk w = start(); w.next(a, p); tiles += (uint32_t)(p.t1 - p.t0)) {
            const int T = p.t1 - p.t0, nm = p.rows > 128 ? 2 : 1;
            const int lrow = m * 128 + r, rho = p.row0 + lrow;
            const bool row_ok = lrow < p.rows;
            const int pos_first = p.L - p.n;
            const int lim = row_ok ? pos_first + rho / a.g + 1 : 0;  // keys the row sees
            const int lim_warp = pos_first + min((rho - lane) / a.g, p.n - 1) + 1;  // keys every row of the warp sees
            const size_t orow = ((size_t)p.b * a.f + rho / a.g) * hq + (size_t)p.h * a.g + rho % a.g;
            // The warp's 32 Q rows, each scaled to [2^8, 2^9) at its largest, into the swizzled
            // tile: D / 8 lanes a row, so that its loads are runs.
            int e = 0;
            if (m < nm) {
                constexpr int kLanes = D / 8, kRowsAt = 32 / kLanes;
                const int sub = lane / kLanes, c = lane % kLanes;
                uint4 xs[kLanes];  // all loads before the first use: one trip to memory
#pragma unroll
                for (int it = 0; it < kLanes; ++it) {
                    const int qrow = m * 128 + (r - lane) + it * kRowsAt + sub, qrho = p.row0 + qrow;
                    xs[it] = make_uint4(0u, 0u, 0u, 0u);
                    if (qrow < p.rows)
                        xs[it] = reinterpret_cast<const uint4 *>(
                            a.q + (((size_t)p.b * a.f + qrho / a.g) * hq + (size_t)p.h * a.g + qrho % a.g) * D)[c];
                }
#pragma unroll
                for (int it = 0; it < kLanes; ++it) {
                    const uint4 x = xs[it];
                    const int qr = (r - lane) + it * kRowsAt + sub;
                    uint32_t mag = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                            __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
                    mag = max(mag & 0xffffu, mag >> 16);
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, o));
                    // zero and non-finite rows keep factor 1
                    int ee = 0;
                    if (mag != 0 && mag < 0x7f80u) ee = max(-110, min(119, (int)(mag >> 7) - 127 - 8));
                    const float f2 = pow2i(-ee);
                    const uint4 y = make_uint4(pack_f16(bf_lo(x.x) * f2, bf_hi(x.x) * f2),
                                               pack_f16(bf_lo(x.y) * f2, bf_hi(x.y) * f2),
                                               pack_f16(bf_lo(x.z) * f2, bf_hi(x.z) * f2),
                                               pack_f16(bf_lo(x.w) * f2, bf_hi(x.w) * f2));
                    *reinterpret_cast<uint4 *>(smem + m * SM::kTile + (c / 8) * SM::kHalf + swz128(qr, c % 8)) = y;
                    const int mine = __shfl_sync(0xffffffffu, ee, lane % kRowsAt * kLanes);
                    if (lane / kRowsAt == it) e = mine;
                }
                fence_proxy_async_smem();
                mbar_arrive(&q_ready[m]);
            }
            if (m >= nm) continue;
            const float rs = a.scale_log2 * head_scale(a.c.k_scale, p.h) * pow2i(e);
            float mx = -INFINITY, l = 0.f, mo = -INFINITY;  // acc is relative to 2^mo
            uint64_t acc[D / 2];  // pairs of channels
#pragma unroll
            for (int c = 0; c < D / 2; ++c) acc[c] = 0ull;
            // Add the O in tensor memory (relative to 2^mx).
            auto drain = [&]() {
                const float f = mo == mx || mo == -INFINITY ? 1.f : ex2(mo - mx);
                const uint64_t f2 = pack2(f, f);
                uint32_t ov[2][16];
                tc::tmem_ld16(ocol, ov[0]);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    tc::tmem_wait_ld();
                    if (c + 1 < D / 16) tc::tmem_ld16(ocol + 16 * (c + 1), ov[(c + 1) & 1]);
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        acc[8 * c + x] = fma2(acc[8 * c + x], f2,
                                              pack2(__uint_as_float(ov[c & 1][2 * x]),
                                                    __uint_as_float(ov[c & 1][2 * x + 1])));
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
                const bool full = tm == (1u << (kKeys / 16)) - 1u && t0 <= lim_warp - kKeys;
                // the row's largest logit
                float mt = -INFINITY, mt2 = -INFINITY;
                if (full) {
                    uint32_t sv[2][16];
                    tc::tmem_ld16(scol, sv[0]);
#pragma unroll
                    for (int c = 0; c < kKeys / 16; ++c) {
                        tc::tmem_wait_ld();
                        if (c + 1 < kKeys / 16) tc::tmem_ld16(scol + 16 * (c + 1), sv[(c + 1) & 1]);
#pragma unroll
                        for (int x = 0; x < 16; x += 4) {
                            mt = max3(mt, __uint_as_float(sv[c & 1][x]), __uint_as_float(sv[c & 1][x + 1]));
                            mt2 = max3(mt2, __uint_as_float(sv[c & 1][x + 2]), __uint_as_float(sv[c & 1][x + 3]));
                        }
                    }
                    mt = fmaxf(mt, mt2);
                } else {
#pragma unroll 1
                    for (int c = 0; c < kKeys / 16; ++c) {
                        uint32_t sv[16];
                        tc::tmem_ld16(scol + 16 * c, sv);
                        tc::tmem_wait_ld();
                        const int left = ((tm >> c) & 1u) ? lim - t0 - 16 * c : 0;
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            if (x < left) mt = fmaxf(mt, __uint_as_float(sv[x]));
                    }
                }
                mt *= rs;
                // O of the last kChain tiles joins the row before P V overwrites it
                if (i > 0 && i % kChain == 0) drain();
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
                        for (int c = 0; c < D; c += 16) {
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
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int k0 = 64 * hf + 32 * c;
                        uint32_t x[32];
                        tc::tmem_ld32(scol + k0, x);
                        tc::tmem_wait_ld();
                        if (!full) {
                            const int left0 = ((tm >> (k0 / 16)) & 1u) ? lim - t0 - k0 : 0;
                            const int left1 = ((tm >> (k0 / 16 + 1)) & 1u) ? lim - t0 - k0 : 0;
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (k >= (k < 16 ? left0 : left1)) x[k] = 0xff800000u;
                        }
                        uint32_t pw[32];  // of 16 keys 8 columns of hi, 8 of lo
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
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
                            pw[k / 8 * 16 + k % 8] = pack_f16(h0, h1);
                            pw[k / 8 * 16 + 8 + k % 8] = pack_f16(l0, l1);
                        }
                        tc::tmem_st32(scol + k0, pw);
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    mbar_arrive(&p_full[m][hf]);
                }
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
            drain();
            const bool whole = p.t0 == 0 && p.t1 == p.cnt;
            const float inv = l > 0.f ? head_scale(a.c.v_scale, p.h) / l : (l == 0.f ? 0.f : l);
            const size_t slot = p.later ? chunk_q4_later_slot(units, p.u, cta) : cta;
            // a partial lies as [32-row group][channel / 4][row in group][4], so that a warp's
            // stores are runs
            float4 *dst = whole ? reinterpret_cast<float4 *>(a.out + orow * D)
                                : reinterpret_cast<float4 *>(a.part_o + slot * kRows * D) +
                                      (size_t)(lrow / 32) * (D / 4) * 32 + lane;
            const int step = whole ? 1 : 32;
            if (row_ok) {
                const uint64_t f2 = whole ? pack2(inv, inv) : pack2(1.f, 1.f);
#pragma unroll
                for (int c = 0; c < D / 4; ++c) {
                    float4 v;
                    unpack2(fma2(acc[2 * c], f2, 0ull), v.x, v.y);
                    unpack2(fma2(acc[2 * c + 1], f2, 0ull), v.z, v.w);
                    dst[c * step] = v;
                }
            }
            if (row_ok) {
                if (!whole)
                    a.part_ml[slot * kRows + lrow] = make_float2(mx, l);
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
        if (warp == 0) {  // -------------------------------------------- MMA issuer
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
            // O of M tile m from the P and V of keys 64 hf ..; fresh: the first of kChain tiles
            auto pv = [&](int m, uint32_t jj, int hf, bool fresh) {
                const uint64_t vd = tc::smem_desc(smem_u32(slots) + (jj % kSlots) * SM::kTile, SM::kHalf, 1024) +
                                    hf * (SM::kHalf >> 5);
                if (el) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t bd = vd + kk * (16 * 128 >> 4);
                        const uint32_t pt = tmem + m * kKeys + hf * 64 + kk * 16;
                        tc::mma_f16_ts(tmem + 2 * kKeys + m * D, pt, bd, idesc_pv,
                                       hf > 0 || kk > 0 || !fresh ? 1u : 0u);
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
                        // half a tile at a time, while the softmax makes the other half
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            wait(&p_full[m][hf], np[m] & 1);
                            if (ok) pv(m, jv, hf, i % kChain == 0);
                        }
                        if (!ok) break;
                        ++np[m];
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
        } else {  // ------------------------------------------------------ converters
            // The 4-bit tiles come in two tiles ahead, by runs of 16 keys (contiguous in the
            // cache): warp w takes runs w - 1, w + 2, .., a lane 16 bytes at a time.  (Bulk
            // copies, one a run and array, took 80 cycles each to issue.)
            const int bs_shift = a.bs == 64 ? 6 : a.bs == 32 ? 5 : 4;
            const int bpt = kKeys >> bs_shift;  // blocks a tile
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
            for (Walk w = start(); w.next(a, p);) {
                const int T = p.t1 - p.t0;
                const int nblk = ceil_div(p.L, a.bs);
                const int32_t *pages = a.page_table + (size_t)p.row * a.max_pages;
                // Page ids 32 blocks at a time, one a lane, the next window in flight.
                const int blk0 = p.t0 * bpt, blk1 = min(nblk, p.t1 * bpt);
                auto load_win = [&](int w32) -> int {
                    const int blk = blk0 + w32 * 32 + lane;
                    return blk < blk1 ? pages[blk] : -1;
                };
                int win_cur = load_win(0), win_next = load_win(1), win = 0;
                auto issue = [&](int t) -> uint32_t {  // tile t of the piece; its valid blocks
                    const uint32_t at = tiles + (uint32_t)t, st = at % kRaw;
                    if (at >= kRaw) ok = ok && mbar_wait_bounded(&raw_free[st], ((at / kRaw) - 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) return 0u;
                    const int first = t * bpt;
                    if (first >> 5 != win) {
                        win_cur = win_next;
                        ++win;
                        win_next = load_win(win + 1);
                    }
                    int page = __shfl_sync(0xffffffffu, win_cur, (first + lane) & 31);
                    const bool there = lane < bpt && blk0 + first + lane < blk1;
                    if (there && (page < 0 || page >= a.num_pages)) {
                        set_error(a.err, RESA_DEVERR_PAGE);
                        page = -1;
                    }
                    if (!there) page = -1;
                    const uint32_t mask = __ballot_sync(0xffffffffu, page >= 0);
                    constexpr int kRunCodes = 16 * D / 2, kRunScales = 16 * D / 16;
                    const uint32_t base = raw_s + st * SM::kRawStage + lane * 16;
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const int run = warp - 1 + 3 * k;
                        const int pg = __shfl_sync(0xffffffffu, page, (run << 4) >> bs_shift);
                        if (run < kKeys / 16 && pg >= 0) {
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
                    return mask;
                };
                uint32_t masks[3];  // of this tile and the next two
                masks[0] = issue(0);
                masks[1] = T > 1 ? issue(1) : 0u;
                for (int t = 0; t < T; ++t) {
                    masks[2] = t + 2 < T ? issue(t + 2) : 0u;
                    const uint32_t at = tiles + (uint32_t)t, st = at % kRaw;
                    ok = ok && mbar_wait_bounded(&raw_full[st], (at / kRaw) & 1);
                    const uint32_t mask = masks[0];
                    masks[0] = masks[1];
                    masks[1] = masks[2];
                    const int left = p.L - (p.t0 + t) * kKeys;  // rows of the tile below the length
                    const bool whole_tile = left >= kKeys && mask == (1u << bpt) - 1u;
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv, ++j) {
                        if (j >= kSlots)
                            ok = ok && mbar_wait_bounded(&slot_free[j % kSlots], ((j / kSlots) - 1) & 1);
                        if (kv == 0 && tid == 32) {
                            uint32_t m16 = 0;
                            for (int x = 0; x < kKeys / 16; ++x)
                                m16 |= ((mask >> ((x * 16) >> bs_shift)) & 1u) << x;
                            tile_mask[at & 3] = m16;
                        }
                        const uint32_t code_at = raw_s + st * SM::kRawStage + kv * SM::kCodes + lane * 16;
                        const uint32_t scale_at = raw_s + st * SM::kRawStage + 2 * SM::kCodes + kv * SM::kScales +
                                                  lane * 2;
                        const uint32_t dst = slots_s + (j % kSlots) * SM::kTile + (c / 2) * SM::kHalf + r1 * 128 + x0;
                        constexpr int kSteps = (kKeys / kStepRows + 2) / 3;
                        uint32_t xs[kSteps][4];
                        uint16_t sf[kSteps];
#pragma unroll
                        for (int k = 0; k < kSteps; ++k) {
                            const int step = warp - 1 + 3 * k;
                            if (step < kKeys / kStepRows) {
                                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                             : "=r"(xs[k][0]), "=r"(xs[k][1]), "=r"(xs[k][2]), "=r"(xs[k][3])
                                             : "r"(code_at + step * 512));
                                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(sf[k]) : "r"(scale_at + step * 64));
                            }
                        }
#pragma unroll
                        for (int k = 0; k < kSteps; ++k) {
                            const int step = warp - 1 + 3 * k;
                            if (step >= kKeys / kStepRows) break;
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
                tiles += (uint32_t)T;
            }
            cp_async_wait<0>();
            if (!ok && lane == 0) set_error(a.err, RESA_DEVERR_TIMEOUT);
        }
        __syncwarp();
        set_regs<kLaunchRegs, true>();
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);

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
        // CTAs q0 .. q1 whose shares meet the unit; only q0's can begin before it
        const int W = sh_w, G = sh_ctas, own = sh_own.x;
        const int q0 = own > 0 ? sh_own.y : (int)((((long long)p.ustart + 1) * G - 1) / W);
        const int q1 = own > 0 ? q0 + own - 1 : (int)((((long long)p.ustart + p.cnt) * G - 1) / W);
        const bool odd = own == 0 && entry_of(q0, W, G) < p.ustart;
        const int slot0 = odd ? chunk_q4_later_slot(units, p.u, q0) : q0;
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
                const size_t sl = (size_t)(q == q0 ? slot0 : q) * kRows;
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
