// Split-KV attention over a 4-bit cache for few query rows (GBSA, ReSA summary
// §3.4.1 Eq. 2 over a block list, or Eq. 1 over every position): up to 16 query
// rows of one kv head (a group's heads, or the heads of a few chunk rows) read
// each 4-bit key and value once.
//
// Work.  A unit is a (sequence, kv head) with its list of blocks.  Short units go
// to a CTA each, longer ones to a thread-block cluster each, whose CTAs take even
// shares and merge them through its shared memory.  Else every unit is cut into even shares, one a CTA, or, where
// that would leave some CTAs with much more than others (many unequal units), the
// blocks of all units form one line of W entries, and CTA c of G takes entries
// [cW/G, (c+1)W/G), a run of pieces, each one unit's.  A unit inside one CTA is
// written directly; of a unit that spans several, each CTA stores a partial (o,
// max, sum), and behind a grid barrier they add them up, each an equal share of
// the rows, in CTA order, so the result does not depend on the arrival order.
//
// Inside a piece, warp w of kWarps takes every kWarps-th step of 32 positions (two
// tiles of 16) through a private cp.async ring of kStages steps and keeps its own
// online softmax; the warps' states are merged at the end of the piece.
//
// The MMAs are m16n8k16 fp16 with the operands swapped, S^T = K Q^T and
// O^T = V^T P^T, so the query rows sit on the N = 8 side.  The contraction index
// may be permuted freely as long as both operands agree, and so may O's
// channels, so that a lane's MMA fragments are the codes of one contiguous run:
//   K: lane (r, c) = (lane / 4, lane % 4) takes channels c * D/4 .. of tokens r
//      and r + 8; MMA k-step s uses its channels 4s .. 4s+3;
//   V: lane (r, c) takes channels r * D/8 .. of tokens 2c, 2c+1, 2c+8, 2c+9, and
//      pairs up the two tokens of a register with byte permutes.
// c * s is exact in fp16.  q is scaled by a power of two per row into fp16's range,
// the row's largest channel to [2^8, 2^9): its 8 bits stay exact down to 2^-25 of the
// largest, and a smaller channel is off by 2^-33 of that at most.  P enters as fp16
// hi + lo scaled by 2^kShift: 22 bits, or 2^-36 of the row's largest weight where that is
// coarser.  So the products lose nothing that fp32 accumulation keeps.  A step's
// products start from zero and join the row in fp32 registers (see below).
//
// Measured (28 q / 4 kv heads, d 128): every position of one 262144-token sequence,
// 151 MB, 51 us, 2.9 TB/s.  Instructions bound it, by their latency more than by a unit:
// a warp's step of 32 tokens is 722 of them, issued at 2.3 of 4 a cycle and SM in the
// loop's 36 us (over the whole kernel, 26.6 M in 51 us, at 1.8); the rest is the share-out
// and the first loads, 5.4 us, and the warps' merge, the barrier and the parts' merge, 8 us.
// 16 warps for 12 and two accumulator chains for one changed nothing.  A list of 10 % of the same sequence's blocks, 15 MB: 16 us, nearly
// all of it latency (list, page, tile, barrier, partials).
#include <cooperative_groups.h>

#include "q4_common.cuh"

namespace cg = cooperative_groups;

namespace resa {
namespace {

template <int D, int NT>
struct Q4Warps {
    static constexpr int kWarps = NT == 1 ? 12 : 8, kStages = 4;
};
// Units of at most so many keys are not split, by the width of the query tile, where a
// cluster is no choice and where it is.  Measured (28 q / 4 kv heads, d 128, batch 16): 1024
// keys 11.4 us whole, 11.4 by clusters of 2, 2048 keys 17 and 14 and, over the grid, 16-24;
// batch 1: 512 keys 8.6 whole and 9.7 by clusters of 8, 1024 keys 11.0 and 10.1; with 16
// heads a group 512 keys 11.1 and 11.5, 1024 keys 15 and 12.0.  These and the next constants
// go by the width of the page table, which is all that the host knows, and were found with
// tables as wide as the sequences.  In a table of 131072 keys the grid takes them all, for 2 to
// 3 us more: one sequence of 2048 keys 11.1 us for 9.2, 8 of 1024 11.1 for 9.4, 16 of 2048
// 15.4 for 12.5; d 64, where the same constants stand, 10.2 for 8.1, 10.3 for 8.3 and 13.0
// for 10.1.
constexpr int kWholeKeys[2] = {2048, 768}, kWholeNear[2] = {768, 512};
// With units for most of the SMs: 128 units of 8192 keys 50 us whole and 54 split, 256 units of
// 1 .. 2500 keys 30 and 57.
constexpr int kWholeKeysMany = 8192;
// Clusters, which leave out the grid barrier and the partials' way through L2, but share by
// the unit where the grid shares by all units' keys: a CTA takes at most kClusterKeys, and at
// most kClusterMore more than over the grid.  Measured, clusters and grid: batch 1, 4096 keys
// 11.3 and 12.1 us, 8192 keys 13.7 and 12.4; batch 2, 8192 keys 13.8 and 14.7, 16384 keys 19.3
// and 17.3; batch 8 (clusters of 4), 4096 keys 14.1 and 16.9; 16 heads a group, batch 1, 2048
// keys 12.5 and 13.7, 4096 keys 14.5 and 13.8.  Unequal lengths favour the grid (16 sequences
// of 17 .. 9001 keys, 16 heads a group: 26.7 and 24.6), hence the first bound.
constexpr int kClusterKeys[2] = {1024, 512}, kClusterMore[2] = {600, 400};
// Units whose clusters run at once (74, 33 and 15 clusters of 2, 4 and 8 CTAs fit; 16 units by
// 8, a second wave, 17 us where 14 units take 10).  Clusters of 16 gained 0.1 to 0.7 us.
constexpr int cluster_units(int cl) { return cl == 8 ? 14 : cl == 4 ? 32 : 72; }
constexpr int kPieceKeys = 2048;   // keys a CTA takes in the time that a second piece adds
constexpr float kShift = 13.f;     // P is stored as 2^kShift * exp2(x - m)
constexpr float kSlack = 2.f;      // growth of the maximum tolerated before rescaling

template <int D, int NT>
struct Q4Smem {
    static constexpr int kWarps = Q4Warps<D, NT>::kWarps, kStages = Q4Warps<D, NT>::kStages;
    static constexpr int kCodes = kTileRows * D / 2;   // one tile's K or V codes
    static constexpr int kScales = kTileRows * D / 16; // and group scales
    static constexpr int kV = 2 * kCodes;              // offsets inside a stage (two tiles)
    static constexpr int kKs = 4 * kCodes;
    static constexpr int kVs = kKs + 2 * kScales;
    static constexpr int kStage = kVs + 2 * kScales;
    static constexpr int kRing = kWarps * kStages * kStage;
};

__device__ __forceinline__ void split_f16(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_f16(a, b);
    lo = pack_f16(a - f16_lo(hi), b - f16_hi(hi));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Byte offset of (token t, 8-byte piece p) of a V code tile: the 16-byte chunks
// of a 128-byte line are XORed with its index, so that the eight lanes of a
// quarter-warp phase (four token pairs, two neighbouring pieces) meet all banks.
template <int D>
__device__ __forceinline__ uint32_t v_chunk(int t, int chunk) {
    constexpr int kPerRow = D / 32;         // 16-byte chunks a row
    constexpr int kRowsPerLine = 8 / kPerRow;
    const int line = t / kRowsPerLine, slot = (t % kRowsPerLine) * kPerRow + chunk;
    return (uint32_t)(line * 128 + ((slot ^ ((line & 3) * 2)) << 4));
}

// A load that stays where it is among the asynchronous copies.
__device__ __forceinline__ uint4 ld_now(const uint4 *p) {
    uint4 x;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p) : "memory");
    return x;
}
// Shared-memory loads of 1, 2 or 4 consecutive words, and of a byte or two.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], uint32_t addr) {
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
    uint16_t x;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(addr));
    return x;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t x;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(addr));
    return x;
}

struct Unit {
    int b, h, row, L, n, cnt;  // cnt: blocks to take, 0 when there is nothing to do
    bool live;                 // outputs are written (else they stay as they were)
};

struct Part {  // rows 0: none
    int b, h, rows;
    int q0, parts, odd;  // CTAs q0 .. whose shares meet the unit; odd: q0's is its later piece
    int i0, i1;          // the items this CTA merges
    float vg;
};

struct DecodeQ4Args {
    Q4Cache c;
    const int32_t *page_table, *seq_len, *n_new, *block_idx, *block_cnt;
    const uint16_t *q;
    float *part_o, *out, *lse;
    float2 *part_ml;
    unsigned long long *grid_bar;
    uint32_t *err;
    RowMap rm;
    int f, max_topk, batch, hq, hkv, g, max_pages, num_pages, bs;
    int cluster;  // CTAs a unit takes (a thread-block cluster), without a grid barrier
    float scale_log2;
};

template <int D, int NT>
__global__ void __launch_bounds__(32 * Q4Warps<D, NT>::kWarps, 1)
    decode_q4_kernel(const __grid_constant__ DecodeQ4Args a) {
    using SM = Q4Smem<D, NT>;
    constexpr int kWarps = SM::kWarps, kStages = SM::kStages, kThreads = 32 * kWarps;
    constexpr int kWords = D / 32;   // 32-bit words of codes a lane takes per K row
    constexpr int kRows = NT * 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int sh_sum[kWarps], sh_unit, sh_first;
    __shared__ int2 sh_own;
    __shared__ int sh_most;  // blocks of the longest unit
    __shared__ int4 sh_units[kThreads];  // (blocks, length, fresh tokens, row) when they fit
    __shared__ float2 sh_ml[kRows];  // a row's maximum and sum
    __shared__ Part sh_part[2];      // this CTA's partial pieces: the first one, a later one
    __shared__ uint32_t sh_ok;

    pdl_launch_next();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int units = a.batch * a.hkv;
    const int cta = blockIdx.x;

    // Unit u: its row, length, fresh tokens and number of blocks.
    auto unit_of = [&](int u, bool report) -> Unit {
        Unit x;
        x.b = u / a.hkv;
        x.h = u - x.b * a.hkv;
        const bool dense = a.block_idx == nullptr;
        const int listed = dense ? 0 : a.block_cnt[u];
        x.n = a.n_new ? a.n_new[x.b] : a.f;
        x.cnt = 0;
        x.L = 0;
        x.row = -1;
        x.live = !a.n_new || x.n != 0;
        if (!x.live) return x;
        uint32_t *err = report && x.h == 0 ? a.err : nullptr;
        x.row = cache_row(a.rm, x.b, err);
        x.L = row_seq_len(a.seq_len, x.row);
        if (x.row < 0 || x.L < (dense ? 0 : 1) || (long long)x.L > (long long)a.max_pages * a.bs) {
            set_error(err, RESA_DEVERR_SEQ_LEN);
            x.live = !dense;
            return x;
        }
        if (dense) {
            if (x.n < 0 || x.n > a.f || x.n > x.L) {
                set_error(err, RESA_DEVERR_CHUNK);
                x.live = false;
                return x;
            }
            x.cnt = ceil_div(x.L, a.bs);
        } else {
            x.cnt = max(0, min(listed, a.max_topk + 1));
        }
        return x;
    };

    if (tid < 2) sh_part[tid].rows = 0;
    if (tid == 0) sh_most = 0;
    // Without a grid barrier a unit has a CTA or a cluster of them, in even shares.  Else
    // prefix sums of the units' blocks: thread t sums units [t * per, ...).
    const bool split = a.grid_bar != nullptr;
    const int per = (units + kThreads - 1) / kThreads;
    const bool kept = per == 1 && split;  // the units' data are in sh_units
    int W = 0, G = 1, x0 = 0, x1 = 0;
    int own = 0, own_first = 0;  // even shares of each unit: the CTAs of this one's unit, the first of them
    auto entry_of = [&](int q) -> int { return q < G ? (int)((long long)W * q / G) : W; };
    // Sums over the threads before this one (exclusive) and over all.
    auto scan = [&](int mine, int &all) -> int {
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        __syncthreads();
        if (lane == 31) sh_sum[warp] = incl;
        __syncthreads();
        all = 0;
        int before = incl - mine;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sh_sum[w];
            all += sh_sum[w];
        }
        return before;
    };
    if (split) {
        const int u_lo = min(units, tid * per), u_hi = min(units, u_lo + per);
        int mine = 0;
        for (int u = u_lo; u < u_hi; ++u) {
            const Unit x = unit_of(u, false);
            mine += x.cnt;
            if (kept) sh_units[u] = make_int4(x.cnt, x.L, x.n, x.row);
        }
        const int before = scan(mine, W);
        if (kept && mine > 0) atomicMax(&sh_most, mine);
        const int grid = gridDim.x;
        const int least = max(1, 32 * kWarps / a.bs);  // a step of every warp
        int share = 0;
        if (kept && units < grid && W > 0) {
            // Shares of `share` entries of one unit each, so that every CTA has one piece: the
            // smallest of five that keeps to the grid (the last one does), unless it is more
            // than kPieceKeys above the even share, which is what a second piece costs.
            const int even = ceil_div(W, grid), last = ceil_div(W, grid - units);
#pragma unroll 1
            for (int k = 0; k < 5; ++k) {
                share = max(least, even + (int)((long long)(last - even) * k / 4));
                int ctas;
                const int mine_ctas = ceil_div(mine, share), first = scan(mine_ctas, ctas);
                if (ctas > grid) continue;
                if ((long long)(min(share, sh_most) - max(least, even)) * a.bs > kPieceKeys) share = 0;
                if (share > 0 && first <= cta && cta < first + mine_ctas) {
                    sh_unit = tid;
                    sh_first = before;
                    sh_own = make_int2(mine_ctas, first);
                }
                if (share > 0 && cta >= ctas && tid == 0) sh_own = make_int2(0, 0);
                break;
            }
        }
        if (share > 0) {
            __syncthreads();
            own = sh_own.x;
            own_first = sh_own.y;
            if (own > 0) {
                x0 = sh_first + (cta - own_first) * share;
                x1 = x0 + min(share, sh_first + sh_units[sh_unit].x - x0);
            }
        } else {
            // the line of entries in even shares
            G = max(1, min(min(grid, W), max(units, ceil_div(W, least))));
            x0 = entry_of(cta);
            x1 = entry_of(cta + 1);
            if (x0 < x1 && before <= x0 && x0 < before + mine) {  // one thread: the unit entry x0 lies in
                int s = before;
                for (int u = u_lo; u < u_hi; ++u) {
                    const int k = kept ? mine : unit_of(u, false).cnt;
                    if (x0 < s + k) {
                        sh_unit = u;
                        sh_first = s;
                        break;
                    }
                    s += k;
                }
            }
            __syncthreads();
        }
    } else {
        const int cnt = unit_of(cta / a.cluster, false).cnt, rank = cta % a.cluster;
        const int share = max(max(1, 32 * kWarps / a.bs), ceil_div(cnt, a.cluster));
        x0 = min(cnt, rank * share);
        x1 = min(cnt, x0 + share);
        own = ceil_div(cnt, share);
        own_first = cta - rank;
    }

    auto orow_of = [&](int b, int h, int rho) -> size_t {
        return ((size_t)b * a.f + rho / a.g) * a.hq + (size_t)h * a.g + rho % a.g;
    };
    // four places of a row: channels ch, ch + 1 and ch + D/8, ch + D/8 + 1
    auto store_out = [&](int b, int h, int rho, int p4, float4 v) {
        float *dst = a.out + orow_of(b, h, rho) * D + (p4 % 4) * (D / 4) + (p4 / 4) * 2;
        *reinterpret_cast<float2 *>(dst) = make_float2(v.x, v.y);
        *reinterpret_cast<float2 *>(dst + D / 8) = make_float2(v.z, v.w);
    };
    auto lse_of = [&](float ms, float ls) -> float {
        return ls > 0.f ? (ms - kShift + log2f(ls)) * 0.6931471805599453f : ls == 0.f ? -INFINITY : ls;
    };
    int u = !split ? cta / a.cluster : x0 < x1 ? sh_unit : 0;
    int ustart = split && x0 < x1 ? sh_first : 0;
    const int sub_shift = a.bs == 64 ? 2 : a.bs == 32 ? 1 : 0;  // tiles a block
    uint8_t *ring = smem + (size_t)warp * kStages * SM::kStage;
    const uint32_t ring_s = smem_u32(ring);
    // The warps' merge, over the rings.  A row's channels lie there (and in the partials) in
    // the order of the lanes, channel r * D/8 + 2 t2 + z at place 16 t2 + 2 r + z, and rows
    // are padded by 4, so that a store's lanes meet all banks.
    constexpr int kRow = D + 4;
    float *wm = reinterpret_cast<float *>(smem);
    float *wl = wm + kWarps * kRows, *wf = wl + kWarps * kRows;
    float *wo = wf + kWarps * kRows;

    for (int x = x0; x < x1; ++u) {
        Unit un;
        if (kept) {
            const int4 x4 = sh_units[u];
            un.b = u / a.hkv;
            un.h = u - un.b * a.hkv;
            un.cnt = x4.x;
            un.L = x4.y;
            un.n = x4.z;
            un.row = x4.w;
        } else {
            un = unit_of(u, false);
        }
        if (un.cnt == 0) continue;
        const int uend = ustart + un.cnt;
        const int j0 = x - ustart, j1 = min(x1, uend) - ustart;  // entries of this piece
        const int b = un.b, h = un.h, L = un.L;
        const int rows_all = a.block_idx ? a.g : un.n * a.g;
        const int base_pos = a.block_idx ? 0 : L - un.n;  // row rho sees positions <= base_pos + rho / g
        const int nblk_seq = ceil_div(L, a.bs);
        const int32_t *list =
            a.block_idx ? a.block_idx + (size_t)u * (a.max_topk + 1) : nullptr;
        const int32_t *pages = a.page_table + (size_t)un.row * a.max_pages;

        // This warp's steps: tiles 2p, 2p + 1 of the piece for p = warp + kWarps t.
        const int ntiles = (j1 - j0) << sub_shift;
        const int npairs = (ntiles + 1) >> 1;
        const int nsteps = warp < npairs ? (npairs - warp + kWarps - 1) / kWarps : 0;
        // Tiles' places 16 steps at a time, one a lane (lane 2i + k: tile k of
        // step 16 w + i), with the next window already in flight: byte-tile
        // index of the cache (page, head, tile in block), position, validity.
        auto load_win = [&](int w, int &tile, int &pos) {
            const int t = w * 16 + (lane >> 1);
            const int e = 2 * (warp + kWarps * t) + (lane & 1);
            tile = -1;
            pos = 0;
            if (t >= nsteps || e >= ntiles) return;
            const int j = j0 + (e >> sub_shift), sub = e & ((1 << sub_shift) - 1);
            const int blk = list ? list[j] : j;
            if (blk < 0 || blk >= nblk_seq) {
                set_error(a.err, RESA_DEVERR_BLOCK);
                return;
            }
            pos = blk * a.bs + sub * kTileRows;
            if (pos >= L) return;
            const int page = pages[blk];
            if (page < 0 || page >= a.num_pages) {
                set_error(a.err, RESA_DEVERR_PAGE);
                return;
            }
            tile = ((page * a.hkv + h) << sub_shift) | sub;
        };
        int win_tile[2], win_pos[2];
        load_win(0, win_tile[0], win_pos[0]);
        load_win(1, win_tile[1], win_pos[1]);
        // Tile k of step t (its window is 0 or 1 ahead of the consumer's).  A branch, so
        // that the next window's loads are not waited for before they are used.
        int win_base = 0;  // window held in slot 0
        auto tile_at = [&](int t, int k) -> int {
            const int src = 2 * (t & 15) + k;
            if ((t >> 4) == win_base) return __shfl_sync(0xffffffffu, win_tile[0], src);
            return __shfl_sync(0xffffffffu, win_tile[1], src);
        };
        auto issue = [&](int t) {
            if (t < nsteps) {
                const uint32_t st = ring_s + (uint32_t)(t % kStages) * SM::kStage;
                constexpr int kChunks = SM::kCodes / 16;  // 16-byte chunks of a code tile
                constexpr int kPerRow = D / 32;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int tile = tile_at(t, k);
                    if (tile < 0) continue;
                    const uint8_t *gk = a.c.k + (size_t)tile * SM::kCodes;
                    const uint8_t *gv = a.c.v + (size_t)tile * SM::kCodes;
#pragma unroll
                    for (int i = 0; i < kChunks / 32; ++i) {
                        const int q = lane + 32 * i;
                        cp_async16_s(st + k * SM::kCodes + q * 16, gk + q * 16);
                        cp_async16_s(st + SM::kV + k * SM::kCodes + v_chunk<D>(q / kPerRow, q % kPerRow),
                                     gv + q * 16);
                    }
                    constexpr int kSc = SM::kScales / 16;  // chunks of a scale tile
                    if (lane < 2 * kSc) {
                        const bool is_v = lane >= kSc;
                        const int q = is_v ? lane - kSc : lane;
                        cp_async16_s(st + (is_v ? SM::kVs : SM::kKs) + k * SM::kScales + q * 16,
                                     (is_v ? a.c.v_sf : a.c.k_sf) + (size_t)tile * SM::kScales + q * 16);
                    }
                }
            }
            cp_async_commit();
        };
        // The queries and the head's scales are asked for first: behind the rings' first copies
        // they took 3 us.
        const float kg = head_scale(a.c.k_scale, h), vg = head_scale(a.c.v_scale, h);
        uint4 qx[NT][D / 32];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int rho = n * 8 + r;
            const bool ok = rho < rows_all;
            const int qr = ok ? rho : 0;
            const size_t qrow = ((size_t)b * a.f + qr / a.g) * a.hq + (size_t)h * a.g + qr % a.g;
            const uint4 *src = reinterpret_cast<const uint4 *>(a.q + qrow * D + c * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) qx[n][i] = ok ? ld_now(src + i) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int t = 0; t < kStages - 1; ++t) issue(t);

        // Q^T fragments and each row's factors.
        uint32_t qb[D / 16][NT][2];
        float row_scale[NT][2];
        int lim[NT][2];  // positions row 2c + k of n-tile n sees (0: no such row)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4(&x)[D / 32] = qx[n];
            uint32_t mag = 0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                             __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
            }
            mag = max(mag & 0xffffu, mag >> 16);
            mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
            mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
            // largest |q| to [2^8, 2^9); zero and non-finite rows keep factor 1
            int e = 0;
            if (mag != 0 && mag < 0x7f80u) e = max(-110, min(119, (int)(mag >> 7) - 127 - 8));
            const float f2 = pow2i(-e);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    qb[2 * i + k][n][0] = pack_f16(bf_lo(w[2 * k]) * f2, bf_hi(w[2 * k]) * f2);
                    qb[2 * i + k][n][1] = pack_f16(bf_lo(w[2 * k + 1]) * f2, bf_hi(w[2 * k + 1]) * f2);
                }
            }
            const float sc = a.scale_log2 * kg * pow2i(e);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int row = n * 8 + 2 * c + k;
                row_scale[n][k] = __shfl_sync(0xffffffffu, sc, (2 * c + k) * 4);
                lim[n][k] = row >= rows_all ? 0
                            : a.block_idx   ? L
                                            : base_pos + row / a.g + 1;
            }
        }
        const int lim_all = a.block_idx ? L : base_pos + 1;  // every row sees these

        float m[NT][2], l[NT][2], o[D / 16][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
        }

        for (int t = 0; t < nsteps; ++t) {
            int tp[2];
            bool there[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // of the window in slot 0
                there[k] = __shfl_sync(0xffffffffu, win_tile[0], 2 * (t & 15) + k) >= 0;
                tp[k] = __shfl_sync(0xffffffffu, win_pos[0], 2 * (t & 15) + k);
            }
            issue(t + kStages - 1);
            cp_async_wait<kStages - 1>();
            __syncwarp();
            const uint32_t st = ring_s + (uint32_t)(t % kStages) * SM::kStage;
            // positions of the tiles that any row sees (0 .. 16), and whether all rows see all
            int ntok[2];
            bool masked = false;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ntok[k] = there[k] ? min(kTileRows, L - tp[k]) : 0;
                masked |= !there[k] || tp[k] + kTileRows > lim_all;
            }
            float s[2][NT][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int n = 0; n < NT; ++n) s[k][n][0] = s[k][n][1] = s[k][n][2] = s[k][n][3] = 0.f;
                const uint32_t kt = st + k * SM::kCodes;
                uint32_t w[2][kWords];
#pragma unroll
                for (int i = 0; i < 2; ++i) lds_words<kWords>(w[i], kt + (r + 8 * i) * (D / 2) + c * (D / 8));
                uint32_t sc[2][D / 64];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t at = st + SM::kKs + k * SM::kScales + (r + 8 * i) * (D / 16) + c * (D / 64);
                    if (D == 128) {
                        const uint32_t p = e4m3x2_to_f16(lds_u16(at));
                        sc[i][0] = __byte_perm(p, p, 0x1010);
                        sc[i][D / 64 - 1] = __byte_perm(p, p, 0x3232);
                    } else {
                        const uint32_t p = e4m3x2_to_f16(lds_u8(at));
                        sc[i][0] = __byte_perm(p, p, 0x1010);
                    }
                }
#pragma unroll
                for (int wi = 0; wi < kWords; ++wi) {
                    uint32_t e0[4], e1[4];
                    e2m1x8_to_f16(w[0][wi], e0);
                    e2m1x8_to_f16(w[1][wi], e1);
                    const int gi = wi / 2;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        e0[j] = mul_f16x2(e0[j], sc[0][gi]);
                        e1[j] = mul_f16x2(e1[j], sc[1][gi]);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma_f16(s[k][n], e0[2 * j], e1[2 * j], e0[2 * j + 1], e1[2 * j + 1],
                                    qb[2 * wi + j][n][0], qb[2 * wi + j][n][1]);
                }
            }
            // Softmax over the step's 32 positions, per query row (column).
            uint32_t bh[2][NT][2], bl[2][NT][2];
            bool grow = false;
            float mt[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k2 = 0; k2 < 2; ++k2) {
                    if (masked) {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int hh = 0; hh < 2; ++hh) {
                                const int pos = tp[k] + r + 8 * hh;
                                if (!there[k] || pos >= lim[n][k2]) s[k][n][2 * hh + k2] = -INFINITY;
                            }
                    }
                    mt[n][k2] = fmaxf(fmaxf(s[0][n][k2], s[0][n][2 + k2]), fmaxf(s[1][n][k2], s[1][n][2 + k2]));
                    grow |= mt[n][k2] * row_scale[n][k2] > m[n][k2] + kSlack;
                }
            if (__any_sync(0xffffffffu, grow)) {  // the columns' maxima only when one may grow
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float alpha[2];
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        float x = mt[n][k2];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        // a whole number, so that every factor 2^(m - m') is exact
                        const float mn = ceilf(fmaxf(m[n][k2], x * row_scale[n][k2]));
                        alpha[k2] = m[n][k2] == -INFINITY ? 0.f : ex2(m[n][k2] - mn);
                        m[n][k2] = mn;
                        l[n][k2] *= alpha[k2];
                    }
#pragma unroll
                    for (int t2 = 0; t2 < D / 16; ++t2) {
                        o[t2][n][0] *= alpha[0];
                        o[t2][n][1] *= alpha[1];
                        o[t2][n][2] *= alpha[0];
                        o[t2][n][3] *= alpha[1];
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float nb[2];
#pragma unroll
                for (int k2 = 0; k2 < 2; ++k2) nb[k2] = m[n][k2] == -INFINITY ? 0.f : kShift - m[n][k2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = ex2(fmaf(s[k][n][e], row_scale[n][e & 1], nb[e & 1]));
                    l[n][0] += p[0] + p[2];
                    l[n][1] += p[1] + p[3];
                    uint32_t h0, l0, h1, l1;
                    split_f16(p[0], p[1], h0, l0);
                    split_f16(p[2], p[3], h1, l1);
                    bh[k][n][0] = movmatrix_trans(h0);
                    bh[k][n][1] = movmatrix_trans(h1);
                    bl[k][n][0] = movmatrix_trans(l0);
                    bl[k][n][1] = movmatrix_trans(l1);
                }
            }
            // O^T += V^T P^T.  The matrix unit truncates when it adds to its
            // accumulator; over a long sequence that would be a bias, so a step's
            // products start from zero and are added to the row in fp32 here.
            uint32_t sv[2][2];  // scales of the token pairs (2c, 2c+1), (2c+8, 2c+9)
            uint32_t w[2][4][D / 64];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t vt = st + SM::kV + k * SM::kCodes;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t0 = 2 * c + 8 * i;
                    const uint32_t at = st + SM::kVs + k * SM::kScales + t0 * (D / 16) + r * D / 128;
                    uint32_t s0 = lds_u8(at), s1 = lds_u8(at + D / 16);
                    if (masked) {  // whatever the slots past the end hold, their values count as 0
                        s0 = t0 < ntok[k] ? s0 : 0u;
                        s1 = t0 + 1 < ntok[k] ? s1 : 0u;
                    }
                    sv[k][i] = e4m3x2_to_f16(s0 | (s1 << 8));
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int t1 = t0 + j;
                        if (D == 128)
                            lds_words<D / 64>(w[k][2 * i + j], vt + v_chunk<D>(t1, r >> 1) + (r & 1) * 8);
                        else
                            lds_words<D / 64>(w[k][2 * i + j], vt + v_chunk<D>(t1, r >> 2) + (r & 3) * 4);
                    }
                }
            }
#pragma unroll
            for (int wi = 0; wi < D / 64; ++wi) {
                // codes of two tokens side by side: even channels in e0, odd ones in e1
                uint32_t e0[2][2][4], e1[2][2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t t0 = w[k][2 * i][wi], t1 = w[k][2 * i + 1][wi];
                        e2m1x8_to_f16((t0 & 0x0f0f0f0fu) | ((t1 << 4) & 0xf0f0f0f0u), e0[k][i]);
                        e2m1x8_to_f16(((t0 >> 4) & 0x0f0f0f0fu) | (t1 & 0xf0f0f0f0u), e1[k][i]);
                    }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float part[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n) part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0.f;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t a0 = mul_f16x2(e0[k][0][j], sv[k][0]), a1 = mul_f16x2(e1[k][0][j], sv[k][0]);
                        const uint32_t a2 = mul_f16x2(e0[k][1][j], sv[k][1]), a3 = mul_f16x2(e1[k][1][j], sv[k][1]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_f16(part[n], a0, a1, a2, a3, bh[k][n][0], bh[k][n][1]);
                            mma_f16(part[n], a0, a1, a2, a3, bl[k][n][0], bl[k][n][1]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[4 * wi + j][n][x] += part[n][x];
                }
            }
            __syncwarp();
            if ((t & 15) == 15) {  // window 0 is used up
                win_tile[0] = win_tile[1];
                win_pos[0] = win_pos[1];
                ++win_base;
                load_win(win_base + 1, win_tile[1], win_pos[1]);
            }
        }
        cp_async_wait<0>();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
                l[n][k2] += __shfl_xor_sync(0xffffffffu, l[n][k2], 4);
                l[n][k2] += __shfl_xor_sync(0xffffffffu, l[n][k2], 8);
                l[n][k2] += __shfl_xor_sync(0xffffffffu, l[n][k2], 16);
            }
        __syncthreads();  // every ring is drained
        // Merge the warps.
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
                const int rho = n * 8 + 2 * c + k2;
                if (r == 0) {
                    wm[warp * kRows + rho] = m[n][k2];
                    wl[warp * kRows + rho] = l[n][k2];
                }
                float *dst = wo + (warp * kRows + rho) * kRow + 2 * r;
#pragma unroll
                for (int t2 = 0; t2 < D / 16; ++t2)
                    *reinterpret_cast<float2 *>(dst + 16 * t2) = make_float2(o[t2][n][k2], o[t2][n][2 + k2]);
            }
        __syncthreads();
        // Each row's maximum and sum, and the warps' factors: a warp a row, a lane a warp.
        // (From here on the code runs once, from a cold instruction cache: loops are kept
        // short rather than unrolled.)
        for (int rho = warp; rho < rows_all; rho += kWarps) {
            const int at = lane * kRows + rho;
            const float mw = lane < kWarps ? wm[at] : -INFINITY;
            float ms = mw;
#pragma unroll
            for (int o2 = 8; o2 > 0; o2 >>= 1) ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, o2));
            const float f2 = ms == -INFINITY ? 0.f : ex2(mw - ms);
            float ls = lane < kWarps ? wl[at] * f2 : 0.f;
#pragma unroll
            for (int o2 = 8; o2 > 0; o2 >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o2);
            if (lane < kWarps) wf[at] = f2;
            if (lane == 0) sh_ml[rho] = make_float2(ms, ls);
        }
        __syncthreads();
        const bool whole = j0 == 0 && j1 == un.cnt;
        // Partial slot of this CTA: 2 cta for its first piece, 2 cta + 1 for a later one.
        const int slot = 2 * cta + (x == x0 ? 0 : 1);
        for (int e = tid; e < rows_all * (D / 4); e += kThreads) {
            const int rho = e / (D / 4), p4 = e % (D / 4);
            float4 os = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int w = 0; w < kWarps; ++w) {
                const float f2 = wf[w * kRows + rho];
                const float4 v = *reinterpret_cast<const float4 *>(wo + (w * kRows + rho) * kRow + 4 * p4);
                os.x += v.x * f2;
                os.y += v.y * f2;
                os.z += v.z * f2;
                os.w += v.w * f2;
            }
            const float2 ml = sh_ml[rho];
            if (whole) {
                const float f2 = ml.y == 0.f ? 0.f : vg / ml.y;
                store_out(b, h, rho, p4, make_float4(os.x * f2, os.y * f2, os.z * f2, os.w * f2));
                if (a.lse && p4 == 0) a.lse[orow_of(b, h, rho)] = lse_of(ml.x, ml.y);
            } else if (!split) {  // over the first warp's own, which this thread alone reads
                *reinterpret_cast<float4 *>(wo + rho * kRow + 4 * p4) = os;
            } else {
                reinterpret_cast<float4 *>(a.part_o + ((size_t)slot * kMaxGroup + rho) * D)[p4] = os;
                if (p4 == 0) a.part_ml[slot * kMaxGroup + rho] = ml;
            }
        }
        if (!whole && tid == 32) {  // what the merge wants to know, worked out before the barrier
            Part pt{b, h, rows_all, own_first, own, 0, 0, 0, vg};
            if (own == 0) {  // only q0's share can begin before the unit
                pt.q0 = (int)((((long long)ustart + 1) * G - 1) / W);
                pt.parts = (int)(((long long)uend * G - 1) / W) - pt.q0 + 1;
                pt.odd = entry_of(pt.q0) < ustart ? 1 : 0;
            }
            const int items = rows_all * (D / 4);
            pt.i0 = items * (cta - pt.q0) / pt.parts;
            pt.i1 = items * (cta - pt.q0 + 1) / pt.parts;
            sh_part[x == x0 ? 0 : 1] = pt;
        }
        __syncthreads();  // the merge area is the ring again
        x = min(x1, uend);
        ustart = uend;
    }

    // Merge the units that span CTAs: behind a barrier of the grid, or of the cluster, whose
    // partials are in its shared memory, each of a unit's CTAs takes an equal share of its
    // (row, four channels) items, with gl lanes an item, a lane a part.
    if (split ? gridDim.x > 1 : a.cluster > 1) {
        if (split) {
            __threadfence();
            __syncthreads();
            if (tid == 0) sh_ok = grid_barrier_bounded(a.grid_bar, gridDim.x) ? 1u : 0u;
            __syncthreads();
            if (!sh_ok && tid == 0) set_error(a.err, RESA_DEVERR_TIMEOUT);
            __threadfence();
        } else {
            if (tid == 0) sh_ok = 1u;
            cg::this_cluster().sync();
        }
#pragma unroll 1
        for (int w2 = 0; w2 < 2 && sh_ok; ++w2) {
            const Part pt = sh_part[w2];
            if (pt.rows == 0) continue;
            const int q0 = pt.q0, parts = pt.parts, odd = pt.odd, i0 = pt.i0, i1 = pt.i1;
            const int lg = parts > 16 ? 5 : parts > 8 ? 4 : parts > 4 ? 3 : parts > 2 ? 2 : 1;
            const int gl = 1 << lg, me = tid & (gl - 1);
#pragma unroll 1
            for (int base = i0; base < i1; base += kThreads >> lg) {
                const int e = base + (tid >> lg);
                const int rho = min(e, i1 - 1) / (D / 4), p4 = min(e, i1 - 1) % (D / 4);
                float ms = -INFINITY, ls = 0.f;
                float4 os = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                for (int q = me; q < parts; q += gl) {
                    float2 ml;
                    float4 v;
                    if (split) {
                        const size_t at = (size_t)(2 * (q0 + q) + (q == 0 ? odd : 0)) * kMaxGroup + rho;
                        ml = __ldcg(a.part_ml + at);
                        v = __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * D) + p4);
                    } else {
                        ml = *cg::this_cluster().map_shared_rank(sh_ml + rho, q);
                        v = *reinterpret_cast<const float4 *>(
                            cg::this_cluster().map_shared_rank(wo + rho * kRow + 4 * p4, q));
                    }
                    const float mn = fmaxf(ms, ml.x);
                    const float f1 = mn == -INFINITY ? 0.f : ex2(ms - mn), f2 = mn == -INFINITY ? 0.f : ex2(ml.x - mn);
                    ms = mn;
                    ls = ls * f1 + ml.y * f2;
                    os.x = os.x * f1 + v.x * f2;
                    os.y = os.y * f1 + v.y * f2;
                    os.z = os.z * f1 + v.z * f2;
                    os.w = os.w * f1 + v.w * f2;
                }
                float mt = ms;
                for (int o2 = gl >> 1; o2 > 0; o2 >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o2));
                const float f1 = mt == -INFINITY ? 0.f : ex2(ms - mt);
                ls *= f1;
                os.x *= f1;
                os.y *= f1;
                os.z *= f1;
                os.w *= f1;
                for (int o2 = gl >> 1; o2 > 0; o2 >>= 1) {
                    ls += __shfl_xor_sync(0xffffffffu, ls, o2);
                    os.x += __shfl_xor_sync(0xffffffffu, os.x, o2);
                    os.y += __shfl_xor_sync(0xffffffffu, os.y, o2);
                    os.z += __shfl_xor_sync(0xffffffffu, os.z, o2);
                    os.w += __shfl_xor_sync(0xffffffffu, os.w, o2);
                }
                if (me == 0 && e < i1) {
                    const float f2 = ls == 0.f ? 0.f : pt.vg / ls;
                    store_out(pt.b, pt.h, rho, p4, make_float4(os.x * f2, os.y * f2, os.z * f2, os.w * f2));
                    if (a.lse && p4 == 0) a.lse[orow_of(pt.b, pt.h, rho)] = lse_of(mt, ls);
                }
            }
        }
    }

    // no CTA leaves while another reads its shared memory
    if (!split && a.cluster > 1) cg::this_cluster().sync();

    // Units without any block: zeros and -inf, and the errors of every unit.  (A unit's loads again
    // only where it may be one: they would take 1 us after the merge.)
    const int u0 = split ? cta : own == 0 && own_first == cta ? cta / a.cluster : units;
    for (int u = u0; u < units; u += split ? gridDim.x : units) {
        if (kept && sh_units[u].x > 0) continue;
        const Unit x = unit_of(u, tid == 0);
        if (x.cnt > 0 || !x.live) continue;
        const size_t o = (size_t)x.b * a.f * a.hq + (size_t)x.h * a.g;  // sparse: f = 1
        for (int e = tid; e < a.g * D; e += kThreads) a.out[o * D + e] = 0.f;
        if (a.lse && tid < a.g) a.lse[o + tid] = -INFINITY;
    }
}

template <int D, int NT>
cudaError_t launch_t(const DecodeQ4Args &a, int ctas, cudaStream_t st) {
    using SM = Q4Smem<D, NT>;
    constexpr int merge = SM::kWarps * NT * 8 * (D + 4 + 3) * 4;
    constexpr int smem = SM::kRing > merge ? SM::kRing : merge;
    static std::atomic<int> done[64];
    cudaError_t e = ensure_smem(decode_q4_kernel<D, NT>, smem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32 * SM::kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    if (a.grid_bar != nullptr) {
        attr[1].id = cudaLaunchAttributeCooperative;  // the CTAs meet at a grid barrier
        attr[1].val.cooperative = 1;
    } else {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = a.cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = (a.grid_bar != nullptr ? ctas : a.cluster) > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, decode_q4_kernel<D, NT>, a);
}

}  // namespace

cudaError_t launch_decode_q4(const Shape &s, const Q4Cache &c, const int32_t *page_table,
                             const int32_t *seq_len, const void *q, int f, const int32_t *n_new,
                             const int32_t *block_idx, const int32_t *block_cnt,
                             int max_topk, int sms, float *part_o, float *part_ml,
                             uint32_t *grid_bar, float *out, float *lse, uint32_t *err,
                             cudaStream_t st) {
    DecodeQ4Args a{};
    a.c = c;
    a.page_table = page_table;
    a.seq_len = seq_len;
    a.n_new = n_new;
    a.block_idx = block_idx;
    a.block_cnt = block_cnt;
    a.q = static_cast<const uint16_t *>(q);
    a.part_o = part_o;
    a.out = out;
    a.lse = lse;
    a.part_ml = reinterpret_cast<float2 *>(part_ml);
    a.grid_bar = reinterpret_cast<unsigned long long *>(grid_bar);
    a.err = err;
    a.rm = s.rows;
    a.f = f;
    a.max_topk = max_topk;
    a.batch = s.batch;
    a.hq = s.hq;
    a.hkv = s.hkv;
    a.g = s.g;
    a.max_pages = s.max_pages;
    a.num_pages = s.num_pages;
    a.bs = s.bs;
    a.scale_log2 = s.sm_scale * 1.4426950408889634f;
    const int rows = block_idx ? s.g : f * s.g;
    // one CTA per SM (two partial slots a CTA in the decode partials), no more than the
    // longest lists could use
    const long long most = (long long)s.batch * s.hkv * (block_idx ? (long long)max_topk + 1 : s.max_pages);
    const long long ctas_most = (most * s.bs + 255) / 256;
    const int all = sms < kNumSms ? sms : kNumSms;
    int ctas = ctas_most < all ? (int)ctas_most : all;
    // Units short enough for one CTA each, or for a cluster: no grid barrier, no cooperative
    // launch.
    const long long longest = (block_idx ? (long long)max_topk + 1 : s.max_pages) * s.bs;
    const int units = s.batch * s.hkv;
    a.cluster = 1;
    const int wide = rows > 8;
    int cl = 8;
    while (cl > 1 && units > cluster_units(cl)) cl /= 2;
    if (longest <= (cl > 1 ? kWholeNear : kWholeKeys)[wide] || (longest <= kWholeKeysMany && units * 5 >= all * 4)) {
        a.grid_bar = nullptr;
        ctas = units;
    } else if (cl > 1 && longest <= (long long)kClusterKeys[wide] * cl &&
               longest * (all - units * cl) <= (long long)kClusterMore[wide] * cl * all) {
        a.grid_bar = nullptr;
        a.cluster = cl;
        ctas = units * cl;
    }
    if (s.d == 128) return rows <= 8 ? launch_t<128, 1>(a, ctas, st) : launch_t<128, 2>(a, ctas, st);
    return rows <= 8 ? launch_t<64, 1>(a, ctas, st) : launch_t<64, 2>(a, ctas, st);
}

}  // namespace resa
