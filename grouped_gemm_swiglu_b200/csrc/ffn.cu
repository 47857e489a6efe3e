// ffn.cu -- the experts' gated feed-forward block for training, forward and backward, each
// one persistent launch on the 5th-generation tensor cores (bf16 operands, fp32 sums).
//
// Rows are grouped by expert (group g: rows off[g] .. off[g+1]); one group is the dense
// block. With [g|u] = x W1^T scaled per group, a(g) = gc sigmoid(alpha gc), gc = min(g, L)
// and keep = mask / (1 - p) drawn from philox.cuh (element row * I + column):
//   forward   gu = [g|u] (bf16, saved),  h = keep a(g) (clamp(u,-L,L) + beta),  y = h W2^T
//   backward  dh = keep (dy W2)
//             dg = dh (clamp(u) + beta) a'(g) [g <= L] s_g,  du = dh a(g) [|u| <= L] s_u
//             dx = [dg|du] W1,  dW1 = [dg|du]^T x,  dW2 = dy^T h     per group
// with a'(g) = s (1 + alpha gc (1 - s)), s = sigmoid(alpha gc). h, [dg|du] and the outputs
// are rounded once to bf16 from fp32: they are operands of the next product, or results in
// the type of what they are the gradient of.
//
// Products. Every product is a tile D[256][<=256] = sum_k A[m][k] B[n][k] of a CTA pair
// (tcgen05.mma.cta_group::2): each CTA holds 128 rows of A, half of B's rows and, in TMEM,
// its 128 rows of D, so a 64-deep step moves 32 KB from L2 to each SM where one CTA's
// 128 x 256 tile would move 48 KB. The forward pass and dh, dx take the weight rows (the
// features) as M and up to 256 token rows of a group as N, so a ragged group costs
// ceil(n/32)*32 columns; the weight gradients take output rows as M, output columns as N
// and the group's rows as K. Operands whose contracted index is not the contiguous one (W2
// in dh, W1 in dx, all four of the weight gradients) are read as they lie: TMA boxes of 64
// contiguous elements x 64 k rows, and the MMA's MN-major descriptors.
//   phase   A (M)              B (N)          K          output
//   UP      W1, 16 gate and    x rows         H          gu, h
//           16 up rows by turns
//   DOWN    W2 rows            h rows         I          y
//   DH      W2 columns         dy rows        H          [dg|du] (workspace)
//   DX      W1 columns         [dg|du] rows   2I         dx
//   DW1     [dg|du] columns    x columns      rows of g  dW1
//   DW2     dy columns         h columns      rows of g  dW2
// UP interleaves gate and up rows by 16 (one five-dimensional TMA box), so that the 16-lane
// TMEM loads give a thread the gate and the up of the same element.
//
// The last step of a weight gradient reaches into the next group's rows: the MMA runs over
// ceil(rem/16) 16-row parts of it only, and a warp of each CTA zeroes the rows past the
// group within the last of them in shared memory before the MMA reads it (a factor 0 on one
// side would not do: the rows may hold infinities or NaN).
//
// Scheduling: tiles are claimed in order from a global counter by a warp of rank 1 and
// handed, decoded, to both CTAs' warps through a ring in shared memory: forward UP then DOWN,
// backward DH, DW2, DX, DW1 (DW2 does not depend on DH and runs while its last tiles
// finish). A DOWN, DX or DW1 tile waits until every UP (DH) tile of the token blocks it
// reads has published its rows (a counter per block); it waits only for tiles claimed
// before it, which wait for nothing, so the schedule cannot deadlock.
//
// Few tiles: token blocks are 64, 128 or 256 rows (ffn_block), and weight gradients of fewer
// tiles than pairs are split along the rows (SPLIT, ffn_split): each part of a group stores
// fp32 sums in the workspace, and JOIN tasks behind all other tiles, one for each part's
// tile, wait for a tile's parts and add them up in their order, each a share of the tile.
// One group of 24396 rows, H 640, I 128, whose six tiles took 163 us, takes 75; 8000 rows,
// H 1024, I 512 (24 tiles) 85 and 71. Parts of half as many rows cost 91 there: a part's
// sums are written and read once each, 256 KB.
//
// Roles: warps 0 and 2 TMA producers (operands A and B), warp 1 MMA issuer (rank 0) and
// scheduler (rank 1), warp 3 zeroes rows past a group and publishes stored rows, warps 4-11
// epilogue (warp w reads TMEM lanes 32 (w % 4).., and every second 16-column chunk), two
// 256-column TMEM accumulators. Every wait is bounded (ptx.cuh).
//
// Measured (one B200; the upper figures at the power cap, where the clock falls from 1.9 to
// 1.05-1.3 GHz): a dense block of 8191 rows, H 4096, I 1536, in 220-264 us forward and 480-548 us
// backward (1.2 PFLOP/s, tensor cores 83-87 % active: 530 cycles a 64-deep step where the MMAs
// take 512); 32768 rows over 128 experts, H 2048, I 768, in 357-429 and 876-933 us (of the
// backward pass dx alone 446, dW1 alone 483, each with dh, dW2 alone 161-202); 1024 rows over 32
// experts in 57-60 and 131-138 us (302 MB of weights read, and as much of gradients written).
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <mutex>
#include <type_traits>

#include "ptx.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr int kFfnRing = 8;      // decoded tiles in flight, 32 bytes each
constexpr int kFfnAhead = 3;     // long tiles in flight
constexpr int kFfnEpi = 8;       // epilogue warps: two per TMEM lane quarter
constexpr int kEpiG = kFfnEpi / 4;
constexpr int kFfnThreads = 32 * (4 + kFfnEpi);  // 384: up to 168 registers a thread
constexpr int kFfnXpose = 2048;  // staging per epilogue warp: three 16 x 16 tiles, 16 x 32 or 16 x 64
constexpr int kFfnPanel = 8;     // rows of tiles walked together (tile order within a group)
constexpr int kFfnMaxG = 1024 + 32;
constexpr int kFfnPairs = 74;      // CTA pairs of 148 SMs: what the choices of sizes reckon with
constexpr int kFfnSplitMin = 2048; // rows of a part at least, if the group's rows divide so
constexpr int kFfnSlot = 65536;    // fp32 sums of a 256 x 256 tile
constexpr int kFfnJoined = 4 * kFfnPairs;  // slots at most
constexpr int kFfnSmallRows = 32;    // average rows a group up to which the SMALL sizes are used
constexpr int kFfnManyRows = 1024;   // and above which dx comes after dW1

// Block and stage sizes. With few columns a step takes the tensor cores less than it takes the
// threads that issue its copies and MMAs: 490 cycles with 64 k, 740 with 128 k (32 columns;
// with half the rows of weights and so half the bytes the same), so tiles of few columns go
// 128 k a step.
//   LARGE  256 token rows a block, 64 k a step in six 32 KB stages. With 128 k in three 64 KB ones
//          the 128-expert forward pass gained 1.5 %, its backward pass lost 6 %.
//   MID    128 rows, 128 k in four 48 KB stages (weight gradients 64 rows a step, and never split):
//          2000 rows, H 1024, I 512 forward 24.6 us LARGE, 22.2 MID. Backward, 128-row blocks both
//          times, 300 rows, H 2048, I 1024 took 38.7 and 34.6 (they run SMALL now: 32.3).
//   SMALL  64 rows, 128 k in five 40 KB stages (weight gradients 64 rows a step): two experts of
//          30 rows, H 2048, I 1024, forward 24.8 us with 64 k in ten 20 KB stages, 21.9 so.
//          Chosen where groups average at most 32 rows, and where there are few tiles (ffn_block).
//          32 experts, H 2048, I 768, us LARGE and SMALL, uneven groups (beyond 64 rows a group
//          reads its weights twice): forward, average 32 rows 58.9, 57.2; 40 rows 59.1, 57.6;
//          48 rows 60.7, 60.9; 64 rows 61.8, 66.8; backward 136.5, 130.9; 137, 131.7; 140.5, 139.9;
//          147, 146. So it would gain 3 % up to about 40 rows, which the bound leaves to LARGE.
enum { LARGE, MID, SMALL };
template <int SIZE>
struct FfnCfg {
    static constexpr int TB = SIZE == LARGE ? 256 : (SIZE == MID ? 128 : 64);  // token rows per block at most
    static constexpr int KT = SIZE == LARGE ? 64 : 128;                        // token tiles: k per step
    static constexpr int STAGES = SIZE == LARGE ? 6 : (SIZE == MID ? 4 : 5);
    static constexpr int A_CHUNK = 16384;                             // token tiles: 128 x 64 of A (or two chunks of KT k rows)
    static constexpr int B_TOK = KT / 64 * A_CHUNK;                   // B within a stage
    static constexpr int STAGE = B_TOK + KT / 64 * (TB / 2 * 128);
    static constexpr int KW = 64;                                     // weight gradients: k rows per step
    static constexpr int LONG = 512 / KT;            // steps of a long tile at least
    static constexpr int CHUNK = KW * 128;          // and bytes of a 64-column chunk: two of A, two of B
    static constexpr int B_W = 2 * CHUNK;
    static constexpr int BARS = 4 * STAGES + 4 + 3 * kFfnRing + 1;
    static constexpr size_t CTRL = 8 * BARS + 16 + 32 * kFfnRing + 32;
    static constexpr size_t smem(int G) {
        return 1024 + (size_t)STAGES * STAGE + kFfnEpi * kFfnXpose + CTRL + 8 * (size_t)(G + 1) + 16;
    }
    static_assert(smem(kFfnMaxG) <= 232448, "shared memory of the largest group table");
    static_assert(STAGE % 1024 == 0 && CHUNK % 1024 == 0, "swizzle atoms");
    static_assert(4 * CHUNK <= STAGE, "operands of a weight-gradient step");
};

enum { kUp, kDown, kDh, kDx, kDw1, kDw2, kJoin1, kJoin2 };

// Division by a number known on the host: floor(n / d) for 0 <= n < 2^31 by a product with
// m = floor((2^32 - 1) / d), which is at most one too small.
struct FastDiv {
    int d;
    uint32_t m;
    __device__ __forceinline__ int div(int n) const {
        const int q = (int)__umulhi((uint32_t)n, m);
        return n - q * d >= d ? q + 1 : q;
    }
};
inline FastDiv fast_div(int64_t d) { return FastDiv{(int)d, (uint32_t)(0xFFFFFFFFull / (uint64_t)d)}; }

struct FfnPhase {
    int kind;
    int rt, ct;  // token phases: ct feature tiles per block; weight gradients: rt x ct tiles per group
    int nkb;     // token phases: steps, FfnCfg::KT deep
    FastDiv per, panel;  // tiles per part of a group (weight gradients) or block (token phases), per panel
    int base;            // weight gradients: the phase's first tile among the split_tiles of a part
};

constexpr int kFfnPhases = 6;  // DH, DW2, DX, DW1, two joins

struct FfnMaps {
    CUtensorMap a[4];     // per phase: operand A
    CUtensorMap b[4][3];  // operand B: boxes of 128, 64 and 32 token rows (weight gradients use the first)
};

struct FfnDev {
    const int32_t* offsets;
    int G, A, H, I;
    int nphase;
    FfnPhase ph[kFfnPhases];
    int nmaps;      // the first phases have operands
    int tb_log2;    // token rows per block: 64 (SMALL), 128 or 256
    int max_blk;    // token blocks at most (`done` has a flag for each, and more)
    int dep_total;  // arrivals that complete a token block's UP (DH) tiles
    const float* gate_scale;
    const float* up_scale;
    float alpha, beta, limit;
    const float* limits;
    DropArgs drop;
    const uint16_t* gu_in;  // backward
    uint16_t *gu, *h, *y;   // forward outputs
    uint16_t *dgu, *dx, *dw1, *dw2;
    unsigned int *tile_ctr, *exit_ctr;
    int* done;  // per token block (zero when idle)
    // Weight gradients of groups of more than split_blk blocks (0: none is split):
    int split_blk;    // token blocks per part of a group
    int split_tiles;  // tiles of both weight gradients
    int* joined;      // per tile: epilogue warps that have stored their partial sums (zero when idle)
    float* part;      // partial sums, 256 x 256 per part and tile
    int* status;
};

struct FTile {
    int ph;  // -1: no more tiles
    int g, blk;
    int r, c;  // token phases: c = feature tile; weight gradients: output row and column tile
    int row0, nrows, nkb;
    int kind;  // from ph; not part of a ring entry
};
constexpr int kTileWords = 8;

// Tile l of an R x C grid walked in panels of kFfnPanel rows (columns in order, the panel's
// rows within a column), so the tiles that run at one time share both operands in L2.
__device__ __forceinline__ void raster(int l, int R, const FastDiv& panel, int& r, int& c) {
    const int p = panel.div(l);
    const int w = min(kFfnPanel, R - p * kFfnPanel);
    l -= p * panel.d;
    // l / w, l below 2^31 / 8: by 2^32 / w rounded up (w <= 8), at most one too large
    const uint32_t m = w == 8 ? 1u << 29 : (w == 7 ? 613566757u : (w == 6 ? 715827883u : (w == 5 ? 858993460u :
                       (w == 4 ? 1u << 30 : (w == 3 ? 1431655766u : (w == 2 ? 1u << 31 : 0xFFFFFFFFu))))));
    c = (int)__umulhi((uint32_t)l, m);
    if (l - c * w >= w) ++c;
    else if (l - c * w < 0) --c;
    r = p * kFfnPanel + l - c * w;
}

// The last g with start[g] <= want, G >= 1 entries: first the 32nd part of them, then its members.
__device__ __forceinline__ int last_start(const int* start, int G, int want, int lane) {
    const int part = (G + 31) >> 5;
    const int first = min(lane * part, G);
    const int q = 31 - __clz(__ballot_sync(0xffffffffu, first < G && start[first] <= want));
    int g = q * part;
    for (int i = 0; i < part; i += 32) {
        const int m = q * part + i + lane;
        const uint32_t le = __ballot_sync(0xffffffffu, i + lane < part && m < G && start[m] <= want);
        if (le) g = q * part + i + 31 - __clz(le);
    }
    return g;
}

// Tiles of a phase. part_start (SPLIT): running number of the groups' parts.
template <bool SPLIT>
__device__ __forceinline__ int phase_tiles(const FfnPhase& f, int nblk, const int* part_start, int G) {
    if (f.kind < kDw1) return nblk * f.ct;
    const int parts = SPLIT ? part_start[G] : G;
    return SPLIT && f.kind >= kJoin1 && parts == G ? 0 : parts * f.rt * f.ct;
}

// The first block of part s of a group of n blocks, none of whose parts is empty (parts <= n);
// and the part that starts at block b.
__device__ __forceinline__ int part_first(int s, int n, int parts) { return (int)((int64_t)s * n / parts); }
__device__ __forceinline__ int part_of(int b, int n, int parts) { return (int)(((int64_t)b * parts + n - 1) / n); }

// Tile L, decoded by a whole warp.
template <class C, bool SPLIT>
__device__ __forceinline__ FTile ffn_tile(int L, const int* blk_start, const int* s_off, const int* part_start,
                                          const FfnDev& p, int lane) {
    FTile t;
    const int nblk = blk_start[p.G];
    t.ph = 0;
#pragma unroll
    for (int i = 0; i < (SPLIT ? kFfnPhases : 4) - 1; ++i) {
        if (t.ph == i && i + 1 < p.nphase) {
            const int n = phase_tiles<SPLIT>(p.ph[i], nblk, part_start, p.G);
            if (L >= n) {
                L -= n;
                t.ph = i + 1;
            }
        }
    }
    const FfnPhase& f = p.ph[t.ph];
    t.kind = f.kind;
    if (t.kind >= kDw1) {
        const int part = f.per.div(L);
        raster(L - part * f.per.d, f.rt, f.panel, t.r, t.c);
        t.g = part;
        int b0 = 0, b1 = INT_MAX / 256;  // the part's first block within the group, the next part's
        if constexpr (SPLIT) {
            t.g = last_start(part_start, p.G, part, lane);
            const int s = part - part_start[t.g], parts = part_start[t.g + 1] - part_start[t.g];
            if (t.kind >= kJoin1) {  // no operands: row0 is the number of the part
                t.blk = blk_start[t.g], t.row0 = s, t.nrows = 0, t.nkb = 0;
                return t;
            }
            if (parts > 1) {
                const int n = blk_start[t.g + 1] - blk_start[t.g];
                b0 = part_first(s, n, parts);
                if (s + 1 < parts) b1 = part_first(s + 1, n, parts);
            }
        }
        t.blk = blk_start[t.g] + b0;
        t.row0 = s_off[t.g] + (b0 << p.tb_log2);
        t.nrows = min(max(s_off[t.g + 1] - t.row0, 0), (b1 - b0) << p.tb_log2);
        t.nkb = (t.nrows + C::KW - 1) / C::KW;
        return t;
    }
    t.g = last_start(blk_start, p.G, f.per.div(L), lane);  // empty groups have no block
    raster(L - blk_start[t.g] * f.ct, blk_start[t.g + 1] - blk_start[t.g], f.panel, t.r, t.c);
    t.blk = blk_start[t.g] + t.r;
    t.row0 = s_off[t.g] + (t.r << p.tb_log2);
    t.nrows = min(1 << p.tb_log2, s_off[t.g + 1] - t.row0);
    t.nkb = f.nkb;
    return t;
}

__device__ __forceinline__ FTile ring_tile(const int* ring, int slot, const FfnDev& p) {
    const int4 a = *reinterpret_cast<const int4*>(ring + slot * kTileWords);
    const int4 b = *reinterpret_cast<const int4*>(ring + slot * kTileWords + 4);
    FTile t;
    t.ph = a.x, t.g = a.y, t.blk = a.z, t.r = a.w, t.c = b.x, t.row0 = b.y, t.nrows = b.z, t.nkb = b.w;
    t.kind = t.ph >= 0 ? p.ph[t.ph].kind : -1;
    return t;
}

// MMA columns of a token tile: the pair's N is a multiple of 32 (each CTA brings half).
__device__ __forceinline__ int tok_cols(int nrows) { return (nrows + 31) & ~31; }

// Token rows of B's box in each CTA: half of those, rounded up to 32, 64 or 128.
template <int MOST>
__device__ __forceinline__ int box_rows(int nrows) {
    const int half = tok_cols(nrows) >> 1;
    return MOST <= 32 || half <= 32 ? 32 : (MOST <= 64 || half <= 64 ? 64 : 128);
}

// ---- PTX used only here
// 16 bytes into shared memory of a cluster CTA, counted as transaction bytes by a barrier there.
__device__ __forceinline__ void st_async_v4(uint32_t dst, uint32_t bar, int a, int b, int c, int d) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                     dst),
                 "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void arrive_expect_tx_cluster(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

__device__ __forceinline__ void tma_load_5d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                                 int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}

__device__ __forceinline__ float ex2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// min and max that give NaN where either side is NaN (fminf and fmaxf give the other side): a
// NaN gate clamped to the limit would leave the pass as an ordinary number.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 16 lanes x 16 fp32 columns from each of two addresses, in the matrix-fragment layout:
// thread t holds rows t/4 and t/4 + 8, columns 2 (t % 4) + {0, 1} and those + 8:
// v[4j + 2i + e] = row t/4 + 8i, column 8j + 2 (t % 4) + e.
__device__ __forceinline__ void tmem_ld_frag2(uint32_t ta, uint32_t tb, float* a, float* b) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(ta), "r"(tb)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = __uint_as_float(r[i]);
        b[i] = __uint_as_float(r[8 + i]);
    }
}

// 16 lanes x 64 fp32 columns in the same layout: v[4j + 2i + e] = row t/4 + 8i, column
// 8j + 2 (t % 4) + e.
__device__ __forceinline__ void tmem_ld_frag64(uint32_t ta, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(ta)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Four 8x8 b16 matrices into shared memory: lane i gives the address of row i % 8 of matrix
// i / 8. stmatrix_t, ldmatrix_t: transposed on the way.
__device__ __forceinline__ void stmatrix(uint32_t addr, const uint32_t* v) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3])
                 : "memory");
}

__device__ __forceinline__ void stmatrix_t(uint32_t addr, const uint32_t* v) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_t(uint32_t addr, uint32_t* v) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
// Two values rounded to bf16 on the side of the limit on which they lie: the backward pass
// reads its clamp masks off the saved values, and a gate just above the limit that was saved
// as one just below would take part in a gradient in which it has none (at a limit of half a
// standard deviation that made 5 % of dx). Where rounding to nearest crosses the limit,
// which is positive, the magnitude takes one step back.
__device__ __forceinline__ uint32_t pack2_side(float lo, float hi, float lim) {
    uint32_t w = pack2(lo, hi);
    const float rl = __uint_as_float(w << 16), rh = __uint_as_float(w & 0xFFFF0000u);
    if ((lo > lim) != (rl > lim)) w += lo > lim ? 1u : 0xFFFFFFFFu;
    if ((hi > lim) != (rh > lim)) w += hi > lim ? 0x10000u : 0xFFFF0000u;
    return w;
}
// The same for a limit on the magnitude.
__device__ __forceinline__ uint32_t pack2_side_abs(float lo, float hi, float lim) {
    uint32_t w = pack2(lo, hi);
    const float rl = fabsf(__uint_as_float(w << 16)), rh = fabsf(__uint_as_float(w & 0xFFFF0000u));
    if ((fabsf(lo) > lim) != (rl > lim)) w += fabsf(lo) > lim ? 1u : 0xFFFFFFFFu;
    if ((fabsf(hi) > lim) != (rh > lim)) w += fabsf(hi) > lim ? 0x10000u : 0xFFFF0000u;
    return w;
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Operand descriptors (128B swizzle). K-major: rows of 64 k, 8-row atoms 1024 bytes apart
// (stride offset), leading offset unused; 16 k further is 32 bytes on. MN-major: rows of 64
// elements of M or N, one per k; 8-row atoms 1024 bytes apart along k (stride offset), the
// two 64-element chunks `chunk` bytes apart (leading offset); 16 k further is 2048 bytes on.
// The upper word is the same for both: stride offset, version 1, layout type 2.
constexpr uint32_t kKLead = 1u << 16;
constexpr uint32_t mn_lead(uint32_t chunk) { return (chunk >> 4) << 16; }
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;

__device__ __forceinline__ void mma_pair_lo(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)acc), "r"(kDescHi)
        : "memory");
}

// Whether the phase with the given parity has completed; never blocks.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// One thread polls, the warp goes on together. Barriers between the two CTAs are waited for
// and arrived on at the default (CTA) scope: what they order travels through the
// asynchronous proxy (copies, st.async, operands), through tensor memory, or is a read
// that has returned its value. With cluster-scope release and acquire in the tile ring, and
// the publishing fence in the epilogue, the 128-expert forward pass took 358 us, 340 without.
// The exception is `fix`, which orders rank 1's ordinary stores of zeros before the MMAs that
// rank 0 issues over both CTAs' operands: release and acquire at cluster scope.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, PipeAbort* ab, int* status) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, ab, status);
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    __syncwarp();
    return ok;
}

__device__ __forceinline__ bool warp_wait_cl(uint64_t* bar, uint32_t parity, PipeAbort* ab, int* status) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) ok = mbar_wait_cl(bar, parity, ab, status);
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    __syncwarp();
    return ok;
}

// Two fp32 values in a register pair, and their arithmetic in one instruction each.
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
    __device__ __forceinline__ explicit F2(float both) : F2(both, both) {}
    __device__ __forceinline__ void get(float& lo, float& hi) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// The kept elements of a 16 feature x 16 token fragment whose thread holds features
// f0 + t/4 and + 8, tokens row + 2 (t % 4) + {0, 1} and those + 8 (the order of
// tmem_ld_frag2): bit 4j + 2i + e. A generator block covers four consecutive features, that
// is the same register of four lanes; each of the four draws the blocks of one of their
// four tokens and the keep bits go round by shuffles, so no block is drawn twice.
__device__ __forceinline__ uint32_t frag_keep(const PhiloxKey& key, uint32_t thr, int64_t row, int I, int f0, int lane) {
    const int j = (lane >> 2) & 3;               // this lane's feature within its blocks
    const int fb = f0 + 4 * (lane >> 4);         // first feature of the lower block
    const int64_t tok = row + 2 * (lane & 3) + (j & 1) + 8 * (j >> 1);
    const uint64_t ctr = (uint64_t)(tok * I + fb) >> 2;
    const uint32_t mine = philox_keep4(key, ctr, thr) | philox_keep4(key, ctr + 2, thr) << 4;
    uint32_t keep = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // token q of the four
        const uint32_t o = __shfl_sync(0xffffffffu, mine, (lane & ~12) | (q << 2));
        const int e = q & 1, jj = q >> 1;
        keep |= ((o >> j) & 1u) << (4 * jj + e);
        keep |= ((o >> (4 + j)) & 1u) << (4 * jj + 2 + e);
    }
    return keep;
}

// Zeroes rows [r0, r1) of this CTA's A and B of a weight-gradient step (two chunks of
// 128-byte rows each).
template <class C>
__device__ __forceinline__ void zero_k_rows(uint8_t* st, int r0, int r1, int lane) {
    uint8_t* at = st + (lane >> 3) * C::CHUNK + (lane & 7) * 16;  // chunk of A or B, 16-byte piece of its row
    for (int r = r0; r < r1; ++r) *reinterpret_cast<uint4*>(at + r * 128) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
}

template <bool BWD, int SIZE, bool SPLIT>
__global__ void __launch_bounds__(kFfnThreads, 1)
    ffn_kernel(const __grid_constant__ FfnMaps maps, const __grid_constant__ FfnDev p) {
    static_assert(!SPLIT || (BWD && SIZE == LARGE));
    using C = FfnCfg<SIZE>;
    constexpr int kStages = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* xpose = smem + kStages * C::STAGE;
    uint64_t* full = reinterpret_cast<uint64_t*>(xpose + kFfnEpi * kFfnXpose);
    uint64_t* empty = full + kStages;
    uint64_t* tail = empty + kStages;  // this CTA's copies of a stage whose rows are to be zeroed
    uint64_t* fix = tail + kStages;    // rank 0: rank 1 has zeroed its rows of the stage
    uint64_t* tfull = fix + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* ring_full = tempty + 2;
    uint64_t* ring_empty = ring_full + kFfnRing;
    uint64_t* pub = ring_empty + kFfnRing;  // per ring slot: an UP (DH) tile's rows are stored
    uint64_t* drain = pub + kFfnRing;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    PipeAbort* ab = reinterpret_cast<PipeAbort*>(tmem_slot + 1);
    int* s_last = reinterpret_cast<int*>(tmem_slot + 2);
    int* ring = reinterpret_cast<int*>((reinterpret_cast<uintptr_t>(tmem_slot + 4) + 15) & ~uintptr_t(15));
    int* blk_start = ring + kTileWords * kFfnRing;
    int* s_off = blk_start + (p.G + 1);
    int* part_start = s_off + (p.G + 1);  // used where groups may be split

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.G;
    const uint32_t rank = cluster_ctarank();
    // `lead`/`peer`: a barrier's (or word's) copy in rank 0 / rank 1
    auto lead = [&](const void* b) -> uint32_t { return mapa_shared(smem_u32(b), 0); };
    auto peer = [&](const void* b) -> uint32_t { return mapa_shared(smem_u32(b), 1); };
    auto smem_cluster = [&](const void* b) -> uint32_t { return mapa_shared(smem_u32(b), rank); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&tail[s], 1);
            mbar_init(&fix[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * kFfnEpi);
        }
        for (int r = 0; r < kFfnRing; ++r) {
            mbar_init(&ring_full[r], 1);
            mbar_init(&pub[r], kFfnEpi);
            mbar_init(&ring_empty[r], 2 * (3 + kFfnEpi) + 1);  // producers, zeroing, epilogues; rank 0's MMA
        }
        mbar_init(drain, 1);
        ab->flag = 0;
        fence_barrier_init();
    }
    // The first copies would wait a microsecond for their descriptors.
    if (warp == 0 && lane < 4 * p.nmaps) {
        const int i = lane >> 2, j = lane & 3;
        tma_prefetch_desc(j == 3 ? &maps.a[i] : &maps.b[i][j]);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    pdl_wait();
    int next_L = 0;  // the scheduler's first claim, under way while the group table is made
    if (warp == 1 && lane == 0 && rank == 1) next_L = (int)atomicAdd(p.tile_ctr, 1u);
    // Token blocks per group and their running start; group bounds clamped into [0, A], so
    // that no tile reads or writes a row outside the matrices whatever the offsets hold.
    for (int g = threadIdx.x; g < G; g += blockDim.x) {
        const int o0 = __ldg(p.offsets + g), o1 = __ldg(p.offsets + g + 1);
        const int lo = min(max(o0, 0), p.A), hi = min(max(o1, lo), p.A);
        if (o0 != lo || o1 != hi) set_status(p.status, MOE_ERR_EXPERT_ID);
        const int blocks = (hi - lo + (1 << p.tb_log2) - 1) >> p.tb_log2;
        blk_start[g + 1] = blocks;
        if (SPLIT) part_start[g + 1] = max((blocks + p.split_blk - 1) / p.split_blk, 1);
        s_off[g] = lo;
        if (g == G - 1) s_off[G] = hi;
    }
    __syncthreads();
    if (warp == 0 || (SPLIT && warp == 2)) {
        int* start = warp == 0 ? blk_start : part_start;
        int carry = 0;
        for (int b0 = 1; b0 <= G; b0 += 32) {
            const int g = b0 + lane;
            int incl = g <= G ? start[g] : 0;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int n = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += n;
            }
            if (g <= G) start[g] = carry + incl;
            carry += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) start[0] = 0;
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers are initialised
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // Offsets that are not in order make groups overlap; more blocks than rows can fill are
    // refused as a whole (the sum is below 2^32: a wrapped one is negative).
    int nblk = blk_start[G], total = 0;
    if (nblk < 0 || nblk > p.max_blk) nblk = 0;
    else for (int i = 0; i < p.nphase; ++i)
        total += phase_tiles<SPLIT>(p.ph[i], nblk, part_start, G);

    if (warp == 0 || warp == 2) {
        // ---------------------------------------------------------------- TMA producers
        // One thread per operand: a copy's issue and the wait for a free stage cost a thread
        // a few hundred cycles, and a step has 512. A's producer arms the stage for both.
        if (lane == 0) {
            const bool op_a = warp == 0, arms = op_a && rank == 0;
            const uint32_t full0 = lead(full), tail0 = smem_cluster(tail);
            const uint32_t empty0 = smem_u32(empty), smem0 = smem_u32(smem);
            uint32_t stage = 0, phase = 0, fills = 0, tails = 0, tail_parity = 0;
            bool ready = false;  // the next stage is known to be free
            bool ok = true;
            for (int i = 0; ok; ++i) {
                const int slot = i % kFfnRing;
                if (!mbar_wait(&ring_full[slot], (i / kFfnRing) & 1, ab, p.status)) break;
                const FTile t = ring_tile(ring, slot, p);
                mbar_arrive_remote(peer(&ring_empty[slot]));
                if (t.ph < 0) break;
                const bool wgrad = t.kind >= kDw1;
                const int half = tok_cols(t.nrows) >> 1;  // token rows of B in each CTA
                const int rows_b = box_rows<C::TB / 2>(t.nrows), sel = wgrad || rows_b == 128 ? 0 : (rows_b == 64 ? 1 : 2);
                const CUtensorMap* map = op_a ? &maps.a[t.ph] : &maps.b[t.ph][sel];
                const uint32_t bytes = wgrad ? 4 * C::CHUNK : (16384u + (16384u >> sel)) * (C::KT / 64);  // of both operands in one CTA
                const uint32_t dst0 = smem0 + (op_a ? 0 : (wgrad ? C::B_W : C::B_TOK));
                // The box of step kb is at row y + kb * dy, 64-column chunk c + kb * dc.
                const int m0 = (wgrad ? t.r : t.c) * 256 + (int)rank * 128, n0 = t.c * 256 + (int)rank * 128;
                int y = t.row0, c = 0, dy = wgrad ? C::KW : C::KT, dc = 0;
                if (op_a ? t.kind == kDown : !wgrad) {  // K-major
                    y = op_a ? t.g * p.H + m0 : t.row0 + (int)rank * half;
                    dy = 0;
                    dc = C::KT / 64;
                } else {
                    c = (op_a ? m0 : n0) >> 6;
                    if (t.kind == kDh) y = t.g * p.H;
                    if (t.kind == kDx) y = t.g * 2 * p.I;
                }
                const bool up = op_a && t.kind == kUp;
                if (up) y = t.c * 8 + (int)rank * 4, dy = 0, c = 0, dc = C::KT / 64;  // 16-row block, 64-deep chunk
                // Rows that this launch computes: wait until the UP (DH) tiles have published them.
                const bool dep_row = !op_a && (t.kind == kDown || t.kind == kDx), dep_k = op_a && t.kind == kDw1;
                const bool zero = wgrad && (t.nrows & 15);  // the last step goes through the zeroing warp
                const int n_main = t.nkb - (zero ? 1 : 0);
                // One step: what follows the wait takes as few instructions as possible, and the
                // next stage is looked at (without blocking) before this one's copy is issued.
                auto step = [&](auto is_up, uint32_t bar) {
                    if (!ready && !mbar_wait(&empty[stage], phase ^ 1, ab, p.status)) return false;
                    const uint32_t dst = dst0 + stage * C::STAGE;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                    ready = mbar_test_wait(empty0 + stage * 8, phase ^ 1);
                    if constexpr (is_up.value) tma_load_5d_pair(dst, map, bar, 0, 0, 2 * t.g, y, c);
                    else tma_load_3d_pair(dst, map, bar, 0, y, c);
                    y += dy;
                    c += dc;
                    ++fills;
                    return true;
                };
                auto run = [&](auto is_up, int n) {
                    for (int kb = 0; kb < n; ++kb) {
                        if (arms) {  // rank 0 arms its barrier for both CTAs' copies
                            if (!ready && !mbar_wait(&empty[stage], phase ^ 1, ab, p.status)) return false;
                            ready = true;
                            mbar_arrive_expect_tx(&full[stage], 2 * bytes);
                        }
                        if (!step(is_up, full0 + stage * 8)) return false;
                    }
                    return true;
                };
                if (dep_row) ok = wait_counter_geq(p.done + t.blk, p.dep_total, ab, p.status);
                if (up) {
                    ok = ok && run(std::true_type{}, n_main);
                } else if (dep_k) {
                    const int per = (1 << p.tb_log2) / C::KW;  // steps of a block: a power of two
                    for (int k0 = 0, b = t.blk; k0 < t.nkb && ok; k0 += per, ++b) {
                        ok = wait_counter_geq(p.done + b, p.dep_total, ab, p.status) &&
                             run(std::false_type{}, min(per, n_main - k0));
                    }
                } else {
                    ok = ok && run(std::false_type{}, n_main);
                }
                if (zero && ok) {  // each CTA's copies go to a barrier of its own first
                    ok = ready || mbar_wait(&empty[stage], phase ^ 1, ab, p.status);
                    if (!ok) break;
                    ready = true;
                    if (op_a) {
                        mbar_arrive_expect_tx(&tail[stage], bytes);
                        tails |= 1u << stage;
                        tail_parity ^= 1u << stage;
                    }
                    ok = step(std::false_type{}, tail0 + stage * 8);
                }
            }
            // Never leave with a copy in flight: the last fill of every stage. Rank 0's full
            // barriers count all copies but those of zeroed stages, which each CTA awaits
            // itself. (Everything has landed long ago unless a wait gave up.)
            // One limit for all of them: after a wait that gave up, stages may be armed for copies
            // that the other producer never issued.
            if (op_a) {
                const long long t0 = clock64();
                auto drained = [&](uint64_t* bar, uint32_t parity) {
                    while (!mbar_test_wait(smem_u32(bar), parity))
                        if (clock64() - t0 > kWaitLimitCycles) return false;
                    return true;
                };
                bool landed = true;
                for (int s = 0; s < kStages && landed; ++s)
                    if ((tails >> s) & 1u) landed = drained(&tail[s], ((tail_parity >> s) & 1u) ^ 1u);
                if (rank == 0)
                    for (uint32_t j = fills < kStages ? 0 : fills - kStages; j < fills && landed; ++j)
                        landed = drained(&full[j % kStages], (j / kStages) & 1u);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- scheduler (rank 1), MMA issuer (rank 0)
        // The scheduler claims and decodes tiles ahead of everyone, for both CTAs: a tile of a
        // weight gradient may have a single step, less than a claim's latency.
        if (rank == 1) {
            for (int i = 0;; ++i) {
                const int slot = i % kFfnRing;
                const int L = __shfl_sync(0xffffffffu, next_L, 0);
                FTile t{};
                t.ph = -1;
                if (L < total) {
                    if (lane == 0) next_L = (int)atomicAdd(p.tile_ctr, 1u);  // one ahead
                    t = ffn_tile<C, SPLIT>(L, blk_start, s_off, part_start, p, lane);
                }
                // Long tiles are handed out kFfnAhead ahead only, so that the last ones are claimed
                // by the pairs that get to them first.
                const int behind = t.nkb >= C::LONG ? kFfnAhead : kFfnRing;
                if (i >= behind && !warp_wait(&ring_empty[(i - behind) % kFfnRing], ((i - behind) / kFfnRing) & 1, ab, p.status))
                    break;
                if (lane == 0) {
#pragma unroll
                    for (uint32_t r = 0; r < 2; ++r) {
                        const uint32_t bar = mapa_shared(smem_u32(&ring_full[slot]), r);
                        const uint32_t e = mapa_shared(smem_u32(ring + slot * kTileWords), r);
                        arrive_expect_tx_cluster(bar, 4 * kTileWords);
                        st_async_v4(e, bar, t.ph, t.g, t.blk, t.r);
                        st_async_v4(e + 16, bar, t.c, t.row0, t.nrows, t.nkb);
                    }
                }
                if (t.ph < 0) break;
            }
        }
        // One thread of rank 0 issues for both CTAs. Everything a step needs is ready before
        // the loop: four MMAs of 256 columns take the tensor core 512 cycles, and building descriptors
        // (or the whole warp waiting) in the loop took 1100.
        if (rank == 0 && lane == 0) {
            uint32_t stage = 0, phase = 0;
            const uint32_t lo = (smem_u32(smem) >> 4) & 0x3FFF;  // no carry: shared memory ends below 2^18
            bool ok = true;
            for (int i = 0; ok; ++i) {
                const int slot = i % kFfnRing;
                if (!mbar_wait(&ring_full[slot], (i / kFfnRing) & 1, ab, p.status)) break;
                const FTile t = ring_tile(ring, slot, p);
                mbar_arrive_remote(peer(&ring_empty[slot]));
                if (t.ph < 0) break;
                const bool wgrad = t.kind >= kDw1, a_mn = t.kind >= kDh;
                const int full_steps = wgrad ? C::KW / 16 : C::KT / 16;  // 16-deep MMAs of a step
                const int last_steps = wgrad ? (t.nrows - C::KW * (t.nkb - 1) + 15) >> 4 : C::KT / 16;
                const uint32_t idesc = idesc_m256(wgrad ? 256 : tok_cols(t.nrows), false) | (a_mn ? 1u << 15 : 0u) |
                                       (wgrad ? 1u << 16 : 0u);
                const uint32_t buf = i & 1, bph = (i >> 1) & 1;
                const uint32_t d = tmem_base + buf * 256;
                const uint32_t lo_a = lo | (wgrad ? mn_lead(C::CHUNK) : (a_mn ? mn_lead(C::KT * 128) : kKLead));
                const uint32_t lo_b = wgrad ? (lo + (C::B_W >> 4)) | mn_lead(C::CHUNK) : (lo + (C::B_TOK >> 4)) | kKLead;
                const uint32_t step_a = a_mn ? 128 : 2, step_b = wgrad ? 128 : 2;  // 16 k further, in 16 bytes
                // The second 64 k of a step.
                const uint32_t next_a = a_mn ? 512 : C::A_CHUNK >> 4, next_b = (uint32_t)box_rows<C::TB / 2>(t.nrows) * 8;
                if (!mbar_wait(&tempty[buf], bph ^ 1, ab, p.status)) break;
                tc_fence_after();
                for (int kb = 0; kb < t.nkb; ++kb) {
                    if (!mbar_wait(&full[stage], phase, ab, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = lo_a + stage * (C::STAGE >> 4), b = lo_b + stage * (C::STAGE >> 4);
                    const int steps = kb + 1 < t.nkb ? full_steps : last_steps;
                    if (steps == 4 && !(C::KT > 64 && !wgrad)) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_pair_lo(d, a + kk * step_a, b + kk * step_b, idesc, kb > 0 || kk > 0);
                    } else if (C::KT > 64 && !wgrad) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_pair_lo(d, a + (kk & 3) * step_a + (kk >> 2) * next_a,
                                        b + (kk & 3) * 2 + (kk >> 2) * next_b, idesc, kb > 0 || kk > 0);
                    } else {
                        for (int kk = 0; kk < steps; ++kk)
                            mma_pair_lo(d, a + kk * step_a, b + kk * step_b, idesc, kb > 0 || kk > 0);
                    }
                    tc_commit_pair_both(&empty[stage]);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                tc_commit_pair_both(&tfull[buf]);
            }
            tc_commit_pair(drain);  // every MMA completes before TMEM is freed
            mbar_wait_drain(drain, 0);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ---------------------------------------------------------------- zeroing, publishing
        // The last step of a weight gradient: this CTA's copies land on `tail`; the rows
        // past the group within its last 16-row step are zeroed; rank 1 tells rank 0, which
        // completes the stage.
        // UP and DH: once every epilogue warp has stored its rows, the fence that makes them
        // visible to the whole GPU, and the count. It takes a microsecond under load, which
        // the epilogue does not wait for.
        uint32_t stage = 0, parity = 0, pub_parity = 0;
        for (int i = 0;; ++i) {
            const int slot = i % kFfnRing;
            if (!warp_wait(&ring_full[slot], (i / kFfnRing) & 1, ab, p.status)) break;
            const FTile t = ring_tile(ring, slot, p);
            __syncwarp();
            if (t.ph < 0) break;
            stage = (stage + t.nkb) % kStages;
            if (t.kind == kUp || t.kind == kDh) {
                if (!warp_wait(&pub[slot], (pub_parity >> slot) & 1u, ab, p.status)) break;
                pub_parity ^= 1u << slot;
                if (lane == 0) {
                    __threadfence();
                    fence_proxy_async_global();
                    red_release_add_gpu(p.done + t.blk, 1);
                }
            } else if (t.kind >= kDw1 && (t.nrows & 15)) {
                const uint32_t s = stage ? stage - 1 : kStages - 1;
                const int rows = t.nrows - C::KW * (t.nkb - 1);
                if (!warp_wait(&tail[s], (parity >> s) & 1u, ab, p.status)) break;
                zero_k_rows<C>(smem + s * C::STAGE, rows, (rows + 15) & ~15, lane);
                if (rank == 0) {
                    if (!warp_wait_cl(&fix[s], (parity >> s) & 1u, ab, p.status)) break;
                    if (lane == 0) mbar_arrive(&full[s]);
                } else if (lane == 0) {
                    mbar_arrive_cluster(lead(&fix[s]));
                }
                parity ^= 1u << s;
            }
            // only now: `pub` of this slot is used again by the tile that gets the slot next
            if (lane == 0) mbar_arrive_remote(peer(&ring_empty[slot]));
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- epilogue
        const int ew = warp - 4, q = warp & 3, eg = ew >> 2;
        uint8_t* xb = xpose + ew * kFfnXpose;
        const uint32_t xs = smem_u32(xb);
        const uint32_t lane_off = (uint32_t)(32 * q) << 16;
        // stmatrix / ldmatrix row of this lane: token (lane & 7) + 8 * (lane >> 4), 8-feature
        // half (lane >> 3) & 1
        const int mt_tok = (lane & 7) + 8 * (lane >> 4), mt_seg = (lane >> 3) & 1;
        // Staged rows of 16 (32) features are 32 (64) bytes; their 16-byte pieces are permuted
        // by the token so that eight rows of a matrix lie in different banks.
        auto at16 = [](int tok, int seg) { return tok * 32 + ((seg ^ (tok >> 2)) & 1) * 16; };
        auto at32 = [](int tok, int seg) { return tok * 64 + ((seg ^ (tok >> 1)) & 3) * 16; };
        const int m16 = at16(mt_tok, mt_seg), m32a = at32(mt_tok, mt_seg), m32b = at32(mt_tok, mt_seg + 2);
        const int r16 = at16(lane >> 1, lane & 1);  // this lane's 16 bytes of a 16 x 16 tile, row by row
        const bool drop = p.drop.on != 0;
        const float nal2 = -1.44269504f * p.alpha;  // sigmoid(alpha g) = 1 / (1 + 2^(nal2 g)); 1/inf = 0 for huge -g
        PhiloxKey key{};
        if (drop) key = philox_key(p.drop.rng);
        bool ok = true;
        for (int i = 0; ok; ++i) {
            const int slot = i % kFfnRing;
            if (!warp_wait(&ring_full[slot], (i / kFfnRing) & 1, ab, p.status)) break;
            const FTile t = ring_tile(ring, slot, p);
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(peer(&ring_empty[slot]));
            if (t.ph < 0) break;
            const uint32_t buf = i & 1, bph = (i >> 1) & 1;
            const uint32_t d = tmem_base + buf * 256 + lane_off;
            const int nch = (t.nrows + 15) >> 4;  // 16-token chunks
            if (!(BWD && t.kind == kDh && t.c * 256 + (int)rank * 128 < p.I)) {  // which waits after its first loads
                if (!warp_wait(&tfull[buf], bph, ab, p.status)) break;
                tc_fence_after();
            }
            if (!BWD && t.kind == kUp) {
                const float sg = p.gate_scale ? __ldg(p.gate_scale + t.g) : 1.f;
                const float su = p.up_scale ? __ldg(p.up_scale + t.g) : 1.f;
                const float lim = p.limits ? __ldg(p.limits + t.g) : p.limit;
                const int f0 = t.c * 128 + (int)rank * 64 + q * 16;
                const F2 one(1.f), sg2(sg), su2(su), n2(nal2), beta2(p.beta), scale2(p.drop.scale);  // two elements at once
                auto rows = [&](auto clamps) {  // two loops, no branch within an element
                for (int ch = eg; ch < nch; ch += kEpiG) {
                    float gv[8], uv[8];
                    tmem_ld_frag2(d + ch * 16, d + (16u << 16) + ch * 16, gv, uv);
                    const int64_t row = t.row0 + ch * 16;
                    uint32_t keep = 0xFFu;
                    if (drop) keep = frag_keep(key, p.drop.thr, row, p.I, f0, lane);
                    uint32_t pg[4], pu[4], phh[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float &g0 = gv[2 * e], &g1 = gv[2 * e + 1], &u0 = uv[2 * e], &u1 = uv[2 * e + 1];
                        (F2(g0, g1) * sg2).get(g0, g1);
                        (F2(u0, u1) * su2).get(u0, u1);
                        F2 g(g0, g1), u(u0, u1);
                        if constexpr (clamps.value) {
                            g = F2(min_nan(g0, lim), min_nan(g1, lim));
                            u = F2(min_nan(max_nan(u0, -lim), lim), min_nan(max_nan(u1, -lim), lim));
                        }
                        float e0, e1, hv[2];
                        (g * n2).get(e0, e1);
                        fma2(F2(ex2_fast(e0), ex2_fast(e1)), one, one).get(e0, e1);
                        (g * fma2(u, one, beta2) * F2(rcp_fast(e0), rcp_fast(e1)) * scale2).get(hv[0], hv[1]);
                        hv[0] = (keep >> (2 * e)) & 1u ? hv[0] : 0.f;
                        hv[1] = (keep >> (2 * e + 1)) & 1u ? hv[1] : 0.f;
                        if constexpr (clamps.value) {
                            pg[e] = pack2_side(gv[2 * e], gv[2 * e + 1], lim);
                            pu[e] = pack2_side_abs(uv[2 * e], uv[2 * e + 1], lim);
                        } else {
                            pg[e] = pack2(gv[2 * e], gv[2 * e + 1]);
                            pu[e] = pack2(uv[2 * e], uv[2 * e + 1]);
                        }
                        phh[e] = pack2(hv[0], hv[1]);
                    }
                    stmatrix_t(xs + m16, pg);
                    stmatrix_t(xs + m16 + 512, pu);
                    stmatrix_t(xs + m16 + 1024, phh);
                    __syncwarp();
                    const int tok = lane >> 1, f = f0 + (lane & 1) * 8;
                    if (ch * 16 + tok < t.nrows) {
                        const size_t r = (size_t)(row + tok);
                        *reinterpret_cast<uint4*>(p.gu + r * 2 * p.I + f) = *reinterpret_cast<uint4*>(xb + r16);
                        *reinterpret_cast<uint4*>(p.gu + r * 2 * p.I + p.I + f) =
                            *reinterpret_cast<uint4*>(xb + 512 + r16);
                        *reinterpret_cast<uint4*>(p.h + r * p.I + f) = *reinterpret_cast<uint4*>(xb + 1024 + r16);
                    }
                    __syncwarp();
                }
                };
                if (lim < INFINITY) rows(std::true_type{});
                else rows(std::false_type{});
            } else if (t.kind == kDown || t.kind == kDx) {
                uint16_t* out = BWD ? p.dx : p.y;
                const int f0 = t.c * 256 + (int)rank * 128 + q * 32;
                if (f0 < p.H) {
                    for (int ch = eg; ch < nch; ch += kEpiG) {
                        float va[8], vb[8];
                        tmem_ld_frag2(d + ch * 16, d + (16u << 16) + ch * 16, va, vb);
                        uint32_t pa[4], pb[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            pa[e] = pack2(va[2 * e], va[2 * e + 1]);
                            pb[e] = pack2(vb[2 * e], vb[2 * e + 1]);
                        }
                        stmatrix_t(xs + m32a, pa);
                        stmatrix_t(xs + m32b, pb);
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int tok = (lane >> 2) + 8 * j;
                            if (ch * 16 + tok < t.nrows)
                                *reinterpret_cast<uint4*>(out + (size_t)(t.row0 + ch * 16 + tok) * p.H + f0 +
                                                          (lane & 3) * 8) =
                                    *reinterpret_cast<uint4*>(xb + at32(tok, lane & 3));
                        }
                        __syncwarp();
                    }
                }
            } else if (BWD && t.kind == kDh) {
                const float sg = p.gate_scale ? __ldg(p.gate_scale + t.g) : 1.f;
                const float su = p.up_scale ? __ldg(p.up_scale + t.g) : 1.f;
                const float lim = p.limits ? __ldg(p.limits + t.g) : p.limit;
                const int f0 = t.c * 256 + (int)rank * 128 + q * 32;
                if (f0 < p.I) {
                    // The saved gate and up are fetched two chunks ahead, the first two while the
                    // products finish.
                    uint4 pre[2][4];
                    const int f = f0 + (lane & 1) * 8;
                    auto fetch = [&](uint4* dst, int ch) {
                        const int tok = ch * 16 + (lane >> 1);
                        const uint16_t* s = p.gu_in + (size_t)(t.row0 + tok) * 2 * p.I + f;
#pragma unroll
                        for (int j = 0; j < 4; ++j)  // gate and up of features f0.., then of f0 + 16..
                            dst[j] = tok < t.nrows ? __ldg(reinterpret_cast<const uint4*>(s + (j & 1) * p.I + 8 * (j & 2)))
                                                   : make_uint4(0, 0, 0, 0);
                    };
                    fetch(pre[0], eg);
                    fetch(pre[1], eg + kEpiG);
                    if (!warp_wait(&tfull[buf], bph, ab, p.status)) break;
                    tc_fence_after();
                    const float cg = p.drop.scale * sg, cu = p.drop.scale * su, bcg = p.beta * cg;
                    // dg = dh (uc + beta) s (1 + alpha gc (1 - s)), du = dh gc s, of two elements at once
                    // (24000 rows, H 128, I 1152, dx alone: 114 us one by one, 110 so).
                    const F2 one(1.f), minus(-1.f), n2(nal2), al(p.alpha), cg2(cg), cu2(cu), bcg2(bcg);
                    auto grad = [&](auto clamps, uint32_t& gw, uint32_t& uw, float dh0, float dh1) {
                        float g0 = lo_f(gw), g1 = hi_f(gw), u0 = lo_f(uw), u1 = hi_f(uw);
                        const float r0 = g0, r1 = g1, w0 = u0, w1 = u1;
                        if (clamps.value) {
                            g0 = min_nan(g0, lim), g1 = min_nan(g1, lim);
                            u0 = min_nan(max_nan(u0, -lim), lim), u1 = min_nan(max_nan(u1, -lim), lim);
                        }
                        const F2 g(g0, g1), dh(dh0, dh1);
                        float e0, e1;
                        (g * n2).get(e0, e1);
                        fma2(F2(ex2_fast(e0), ex2_fast(e1)), one, one).get(e0, e1);
                        const F2 s(rcp_fast(e0), rcp_fast(e1)), gs = g * s;
                        const F2 slope = fma2(al * gs, fma2(s, minus, one), s);
                        float dg0, dg1, du0, du1;
                        (dh * slope * fma2(F2(u0, u1), cg2, bcg2)).get(dg0, dg1);
                        (dh * gs * cu2).get(du0, du1);
                        // NaN: of a gate, dg and du are NaN; of an up value, dg is, and du, taken only
                        // where |u| <= L, is 0 (without a limit, too).
                        if constexpr (clamps.value) {
                            dg0 = r0 > lim ? 0.f : dg0, dg1 = r1 > lim ? 0.f : dg1;
                            du0 = fabsf(w0) <= lim ? du0 : 0.f, du1 = fabsf(w1) <= lim ? du1 : 0.f;
                        } else {
                            du0 = w0 == w0 ? du0 : 0.f, du1 = w1 == w1 ? du1 : 0.f;
                        }
                        gw = pack2(dg0, dg1);
                        uw = pack2(du0, du1);
                    };
                    auto chunk = [&](auto clamps, uint4* in, int ch) {
                        const int64_t row = t.row0 + ch * 16;
                        float v[2][8];
                        tmem_ld_frag2(d + ch * 16, d + (16u << 16) + ch * 16, v[0], v[1]);
                        if (drop) {
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const uint32_t keep = frag_keep(key, p.drop.thr, row, p.I, f0 + 16 * hf, lane);
#pragma unroll
                                for (int n = 0; n < 8; ++n) v[hf][n] = (keep >> n) & 1u ? v[hf][n] : 0.f;
                            }
                        }
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {  // features f0.. and f0 + 16..
                            *reinterpret_cast<uint4*>(xb + r16) = in[2 * hf];
                            *reinterpret_cast<uint4*>(xb + 512 + r16) = in[2 * hf + 1];
                            __syncwarp();
                            if (hf == 1) fetch(in, ch + 2 * kEpiG);
                            uint32_t gw[4], uw[4];
                            ldmatrix_t(xs + m16, gw);
                            ldmatrix_t(xs + m16 + 512, uw);
#pragma unroll
                            for (int e = 0; e < 4; ++e) grad(clamps, gw[e], uw[e], v[hf][2 * e], v[hf][2 * e + 1]);
                            __syncwarp();  // every lane has read its matrices
                            stmatrix_t(xs + m16, gw);
                            stmatrix_t(xs + m16 + 512, uw);
                            __syncwarp();
                            const int tok = lane >> 1;
                            if (ch * 16 + tok < t.nrows) {
                                uint16_t* o = p.dgu + (size_t)(row + tok) * 2 * p.I + f + 16 * hf;
                                *reinterpret_cast<uint4*>(o) = *reinterpret_cast<uint4*>(xb + r16);
                                *reinterpret_cast<uint4*>(o + p.I) = *reinterpret_cast<uint4*>(xb + 512 + r16);
                            }
                            __syncwarp();
                        }
                    };
                    auto rows = [&](auto clamps) {  // two loops: the clamps are a third of the instructions
                        for (int ch = eg; ch < nch; ch += 2 * kEpiG) {
                            chunk(clamps, pre[0], ch);
                            if (ch + kEpiG < nch) chunk(clamps, pre[1], ch + kEpiG);
                        }
                    };
                    if (lim < INFINITY) rows(std::true_type{});
                    else rows(std::false_type{});
                }
            } else if (BWD) {  // weight gradients: row-major, 16 rows x 64 columns at a time
                const bool first = t.kind == kDw1 || t.kind == kJoin1;
                const int M = first ? 2 * p.I : p.H, N = first ? p.H : p.I;
                const int m0 = t.r * 256 + (int)rank * 128 + q * 32, n0 = t.c * 256 + eg * (256 / kEpiG);
                const int nparts = SPLIT ? part_start[t.g + 1] - part_start[t.g] : 1;
                if (SPLIT && nparts > 1) {
                    // Slots of a group's parts start at ceil(2 b / split_blk), b its first block: a
                    // group of n > split_blk blocks has ceil(n / split_blk) <= floor(2 n / split_blk) parts.
                    const int b0 = blk_start[t.g], per = p.split_tiles;
                    const int slot0 = ((2 * b0 + p.split_blk - 1) / p.split_blk) * per + p.ph[t.ph].base +
                                      t.r * p.ph[t.ph].ct + t.c;
                    // A slot: 16 warps x 4 pieces of 16 x 64 x 8 column octets x 32 lanes x 4 sums, as
                    // tmem_ld_frag64 gives them.
                    if (t.kind < kJoin1) {
                        if (m0 < M && n0 < N) {
                            const int slot = slot0 + part_of(t.blk - b0, blk_start[t.g + 1] - b0, nparts) * per;
                            float4* o = reinterpret_cast<float4*>(p.part + (size_t)slot * kFfnSlot) +
                                        (rank * kFfnEpi + ew) * 1024 + lane;
#pragma unroll 1
                            for (int blk = 0; blk < 2 * (256 / kEpiG / 64); ++blk) {
                                float v[32];
                                tmem_ld_frag64(d + ((uint32_t)(16 * (blk & 1)) << 16) + eg * (256 / kEpiG) + 64 * (blk >> 1), v);
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    o[blk * 256 + j * 32] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                            }
                        }
                        __syncwarp();
                        if (lane == 0) {
                            __threadfence();
                            red_release_add_gpu(p.joined + slot0, 1);
                        }
                    } else {
                        // Each part's join task adds up, in the order of the parts, every nparts-th
                        // piece of 16 rows of this CTA's half of the tile. 16 loads are under way
                        // in a thread: of 8 parts and 16 columns, or of 4 parts and 32 columns.
                        bool there = true;
                        if (lane == 0) there = wait_counter_geq(p.joined + slot0, 2 * kFfnEpi * nparts, ab, p.status);
                        ok = __shfl_sync(0xffffffffu, there ? 1 : 0, 0) != 0;
                        __syncwarp();
                        if (!ok) break;
                        const size_t stride = (size_t)per * (kFfnSlot / 4);
                        const float4* tile = reinterpret_cast<const float4*>(p.part + (size_t)slot0 * kFfnSlot) + lane;
                        uint16_t* out = (first ? p.dw1 : p.dw2) + (size_t)t.g * M * N;
                        auto join = [&](auto octets) {
                            constexpr int J = octets.value, PB = 16 / J, U = 8 / J;  // octets of columns, parts; pieces of 64 columns
                            for (int u = t.row0 + nparts * ew; u < 32 * U; u += nparts * kFfnEpi) {
                                const int w = u / (4 * U), blk = u / U & 3, cc = u % U;
                                const int um = t.r * 256 + (int)rank * 128 + (w & 3) * 32 + 16 * (blk & 1);
                                const int un = t.c * 256 + (w >> 2) * 128 + 64 * (blk >> 1) + 8 * J * cc;
                                if (um >= M || un >= N) continue;
                                const float4* src = tile + (rank * kFfnEpi + w) * 1024 + blk * 256 + cc * (32 * J);
                                float4 v[J] = {};
                                for (int n0 = 0; n0 < nparts; n0 += PB) {
                                    float4 x[PB][J];
#pragma unroll
                                    for (int n = 0; n < PB; ++n)
#pragma unroll
                                        for (int j = 0; j < J; ++j)
                                            x[n][j] = n0 + n < nparts ? __ldcg(src + (n0 + n) * stride + j * 32) : float4{};
#pragma unroll
                                    for (int n = 0; n < PB; ++n)
#pragma unroll
                                        for (int j = 0; j < J; ++j)
                                            v[j].x += x[n][j].x, v[j].y += x[n][j].y, v[j].z += x[n][j].z, v[j].w += x[n][j].w;
                                }
                                const int srow = (lane & 7) + 8 * ((lane >> 3) & 1), spiece = lane >> 4;
#pragma unroll
                                for (int j = 0; j < J; j += 2) {
                                    const uint32_t w4[4] = {pack2(v[j].x, v[j].y), pack2(v[j].z, v[j].w),
                                                            pack2(v[j + 1].x, v[j + 1].y), pack2(v[j + 1].z, v[j + 1].w)};
                                    stmatrix(xs + srow * (16 * J) + (j + spiece) * 16, w4);
                                }
                                __syncwarp();
#pragma unroll
                                for (int i = lane; i < 16 * J; i += 32)
                                    *reinterpret_cast<uint4*>(out + (size_t)(um + i / J) * N + un + i % J * 8) =
                                        *reinterpret_cast<uint4*>(xb + i * 16);
                                __syncwarp();
                            }
                        };
                        if (nparts > 4) join(std::integral_constant<int, 2>{});
                        else join(std::integral_constant<int, 4>{});
                    }
                } else if (t.kind < kJoin1 && m0 < M && n0 < N) {
                    // Through shared memory, so that a store covers whole 128-byte lines of four
                    // rows: from the registers it would cover one sector of each of 32 rows, and
                    // with few rows a group the stores, not the products, are what these tiles
                    // cost (128-expert backward pass: 992 us with 32-byte stores, 859 so).
                    uint16_t* o = (t.kind == kDw1 ? p.dw1 : p.dw2) + ((size_t)t.g * M + m0 + (lane >> 3)) * N + n0 +
                                  (lane & 7) * 8;
                    const int srow = (lane & 7) + 8 * ((lane >> 3) & 1), spiece = lane >> 4;  // stmatrix row, piece of two
#pragma unroll 1
                    for (int blk = 0; blk < 2 * (256 / kEpiG / 64); ++blk) {
                        const int rh = 16 * (blk & 1), c0 = 64 * (blk >> 1);
                        if (t.nkb > 0) {
                            float v[32];
                            tmem_ld_frag64(d + ((uint32_t)rh << 16) + eg * (256 / kEpiG) + c0, v);
#pragma unroll
                            for (int j = 0; j < 8; j += 2) {
                                const uint32_t w[4] = {pack2(v[4 * j], v[4 * j + 1]), pack2(v[4 * j + 2], v[4 * j + 3]),
                                                       pack2(v[4 * j + 4], v[4 * j + 5]), pack2(v[4 * j + 6], v[4 * j + 7])};
                                stmatrix(xs + srow * 128 + ((j + spiece) ^ (srow & 7)) * 16, w);
                            }
                            __syncwarp();
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = 4 * j + (lane >> 3);
                            uint4 w = make_uint4(0, 0, 0, 0);  // a group without rows
                            if (t.nkb > 0) w = *reinterpret_cast<uint4*>(xb + r * 128 + (((lane & 7) ^ (r & 7)) * 16));
                            *reinterpret_cast<uint4*>(o + (size_t)(rh + 4 * j) * N + c0) = w;
                        }
                        __syncwarp();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(lead(&tempty[buf]));
            if ((t.kind == kUp || t.kind == kDh) && lane == 0) mbar_arrive(&pub[slot]);
        }
    }

    pdl_trigger();
    __syncthreads();
    cluster_sync_all();  // rank 0's MMAs and copies are done before either CTA frees TMEM or exits
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
    // The last CTA leaves the counters at zero for the next launch.
    if (threadIdx.x == 0) {
        __threadfence();
        *s_last = atomicAdd(p.exit_ctr, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (*s_last) {
        for (int b = threadIdx.x; b < nblk; b += blockDim.x) p.done[b] = 0;
        if (SPLIT)
            for (int b = threadIdx.x; b < kFfnJoined; b += blockDim.x) p.joined[b] = 0;
        if (threadIdx.x == 0) {
            atomicExch(p.tile_ctr, 0u);
            atomicExch(p.exit_ctr, 0u);
        }
    }
}

// ---------------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 ffn_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// rows x cols bf16 as (64, rows, cols / 64): a box is box_rows rows of `chunks` neighbouring
// 64-column chunks, one chunk after the other, 128B swizzle.
bool make_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows, uint32_t chunks) {
    auto enc = ffn_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {64, rows, cols / 64};
    cuuint64_t strides[2] = {cols * 2, 128};
    cuuint32_t box[3] = {64, box_rows, chunks};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand whose rows are token rows (K-major): boxes of 128, 64 and 32 rows, those that a
// block of this many rows can ask for (each CTA takes half of a block).
bool make_map_tokens(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t block, uint32_t chunks) {
    const uint64_t most = std::min(rows, block);
    for (int i = most <= 64 ? 2 : (most <= 128 ? 1 : 0); i < 3; ++i)
        if (!make_map(&map[i], base, rows, cols, 128u >> i, chunks)) return false;
    return true;
}

// An MN-major operand: k rows of two 64-element chunks.
bool make_map_mn(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t k_rows) {
    return make_map(map, base, rows, cols, k_rows, 2);
}

// W1 [G][2][I/16][16][H/64][64] as (64, 16, G x gate|up, I/16, H/64): a box is `chunks` times
// 64 columns of 16 gate rows, then the same 16 up rows, four times.
bool make_map_w1(CUtensorMap* map, const void* base, uint64_t G, uint64_t I, uint64_t H, uint32_t chunks) {
    auto enc = ffn_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[5] = {64, 16, 2 * G, I / 16, H / 64};
    cuuint64_t strides[4] = {H * 2, I * H * 2, 16 * H * 2, 128};
    cuuint32_t box[5] = {64, 16, 2, 4, chunks};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs of a launch: two per cluster that can be resident at once.
template <bool BWD, int SIZE, bool SPLIT = false>
cudaError_t ffn_grid(int* grid) {
    static std::mutex mu;
    static int cache[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && cache[dev]) {
        *grid = cache[dev];
        return cudaSuccess;
    }
    const size_t smem = FfnCfg<SIZE>::smem(kFfnMaxG);
    e = cudaFuncSetAttribute(ffn_kernel<BWD, SIZE, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (num_sms() / 2));
    cfg.blockDim = dim3(kFfnThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, ffn_kernel<BWD, SIZE, SPLIT>, &cfg);
    if (e != cudaSuccess) return e;
    const int g = std::min(2 * n, 2 * (num_sms() / 2));
    if (g < 2) return cudaErrorInvalidConfiguration;
    if (dev < 64) cache[dev] = g;
    *grid = g;
    return cudaSuccess;
}

template <bool BWD, int SIZE, bool SPLIT = false>
cudaError_t ffn_launch(const FfnMaps& maps, const FfnDev& p, int64_t tiles, cudaStream_t stream) {
    int grid = 0;
    cudaError_t e = ffn_grid<BWD, SIZE, SPLIT>(&grid);
    if (e != cudaSuccess) return e;
    if (tiles < grid / 2) grid = 2 * (int)std::max<int64_t>(tiles, 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kFfnThreads);
    cfg.dynamicSmemBytes = FfnCfg<SIZE>::smem(p.G) + (SPLIT ? 4 * (size_t)(p.G + 1) : 0);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, ffn_kernel<BWD, SIZE, SPLIT>, maps, p);
}

}  // namespace

// Token rows per block: 64 where groups average at most kFfnSmallRows rows (see FfnCfg). Else 256,
// whose blocks read the weights least often, unless few tiles leave CTA pairs without work or
// waiting for the longest: with smaller blocks the products and epilogues are shared among
// more of them. Bounds on the tiles of gate and up (rows / 128 x I / 128): with 64 rows one a CTA
// pair, with 128 rows three forward, one and a half backward, where weight gradients wait
// for more blocks. Microseconds with 256 and 128 rows: forward 1570 rows of 9 groups, H 768,
// I 1024 (168 tiles) 29.4, 24.7; backward 1200 rows, H 2048, I 1024 (80) 50.2, 45.2; 2199 of 16
// groups, H 1024, I 512 (132) 44.3, 50.4. With 256, 128 and 64: forward 695 rows of 2 groups,
// H 1280, I 640 (60 tiles of 64) 25.1, 21.5, 21.0; backward 300 rows, H 2048, I 1024 (40) 43.7,
// 34.8, 32.3. One group of 1000 rows, H 256, I 128, backward 27.4, 23.9 and 27.9: weight
// gradients of long groups are slower SMALL.
static int ffn_block(int64_t A, int G, int I, bool bwd) {
    if (A <= (int64_t)kFfnSmallRows * G) return 64;
    auto tiles = [&](int tb) { return (std::min<int64_t>(A, G) + A / tb) * (I / 128); };
    if (tiles(64) <= kFfnPairs && (!bwd || A <= 512 * (int64_t)G)) return 64;
    return tiles(128) <= (bwd ? kFfnPairs * 3 / 2 : kFfnPairs * 3) ? 128 : 256;
}

// Token blocks at most: every group that has rows ends in one that may be part.
static int64_t max_blocks(int64_t A, int G, int tb) { return std::min<int64_t>(A, G) + A / tb; }

// Completion flags of a workspace: enough for every block size, and never fewer for more rows,
// so that a workspace serves every smaller call. Then those of split weight gradients.
static int64_t block_flags(int64_t A, int G) { return std::min<int64_t>(A, G) + A / FfnCfg<SMALL>::TB; }
int64_t ffn_flags(int64_t A, int G, bool bwd) { return block_flags(A, G) + (bwd ? kFfnJoined : 0); }

// How the weight gradients' contraction over a group's rows is split: into parts of `blocks`
// token blocks (0: not at all), so that the parts' slots (256 x 256 sums each) stay within
// kFfnJoined. `parts`: slots of one tile, never fewer for more rows.
struct FfnSplit {
    int blocks, tiles, parts;
};
static FfnSplit ffn_split(int64_t A, int G, int H, int I) {
    const int64_t th = (H + 255) / 256, tiles = th * (I / 128) + th * ((I + 255) / 256);
    FfnSplit s{0, 0, 0};
    const int tb = ffn_block(A, G, I, true);
    if (tb == 64 || A < 2 * kFfnSplitMin || G * tiles > kFfnPairs) return s;
    // Slots are numbered by twice the block (one group: by the part), see the epilogue.
    const int64_t twice = G == 1 ? 1 : 2, limit = kFfnPairs * 2 * twice / tiles;
    const int64_t n = twice * max_blocks(A, G, tb);
    s.blocks = (int)std::max<int64_t>(kFfnSplitMin / tb, (n + limit - 1) / limit);
    s.tiles = (int)tiles;
    // n / blocks rounded up, or more: n tb <= twice (256 min(A, G) + A)
    s.parts = (int)std::min<int64_t>(limit, (twice * (256 * std::min<int64_t>(A, G) + A) + kFfnSplitMin - 1) / kFfnSplitMin);
    return s;
}

size_t ffn_part_bytes(int64_t A, int G, int H, int I) {
    const FfnSplit s = ffn_split(A, G, H, I);
    return (size_t)s.parts * s.tiles * kFfnSlot * sizeof(float);
}

int64_t ffn_max_tiles(int64_t A, int G, int H, int I, bool bwd) {
    const int64_t nb = max_blocks(A, G, ffn_block(A, G, I, bwd)), h = (H + 255) / 256, i = (I + 255) / 256, i1 = I / 128;
    const int64_t parts = G + ffn_split(A, G, H, I).parts;
    return bwd ? nb * (i + h) + 2 * parts * (h * i + i1 * h) : nb * (i1 + h);
}

cudaError_t launch_ffn(const FfnArgs& a, cudaStream_t stream) {
    FfnMaps maps{};
    FfnDev p{};
    p.offsets = a.offsets;
    p.G = a.G;
    p.A = (int)a.A;
    p.H = a.H;
    p.I = a.I;
    p.gate_scale = a.gate_scale;
    p.up_scale = a.up_scale;
    p.alpha = a.alpha;
    p.beta = a.beta;
    p.limit = a.limit;
    p.limits = a.limits;
    p.drop = a.drop;
    p.tile_ctr = a.tile_ctr;
    p.exit_ctr = a.exit_ctr;
    p.done = a.done;
    p.status = a.status;
    const int tb = ffn_block(a.A, a.G, a.I, a.bwd);
    const FfnSplit split = a.bwd ? ffn_split(a.A, a.G, a.H, a.I) : FfnSplit{0, 0, 0};
    const int size = tb == FfnCfg<SMALL>::TB ? SMALL : (tb == FfnCfg<MID>::TB && !split.blocks ? MID : LARGE);
    const uint32_t kt = size == LARGE ? FfnCfg<LARGE>::KT : FfnCfg<MID>::KT, kw = FfnCfg<LARGE>::KW;
    static_assert(FfnCfg<MID>::KT == FfnCfg<SMALL>::KT && FfnCfg<LARGE>::KW == FfnCfg<SMALL>::KW);
    const int th = (a.H + 255) / 256, ti = (a.I + 255) / 256, ti1 = a.I / 128;
    const uint64_t A = (uint64_t)a.A, GH = (uint64_t)a.G * a.H, G2I = (uint64_t)a.G * 2 * a.I;
    bool ok = true;
    int64_t tiles = 0;
    const int64_t nb = max_blocks(a.A, a.G, tb);
    p.tb_log2 = tb == 64 ? 6 : (tb == 128 ? 7 : 8);
    p.max_blk = (int)nb;
    auto add = [&](int kind, int rt, int ct, int nkb) {
        p.ph[p.nphase] = FfnPhase{kind, rt, ct, nkb, fast_div(kind >= kDw1 ? (int64_t)rt * ct : ct),
                                  fast_div((int64_t)kFfnPanel * ct), kind == kDw1 || kind == kJoin1 ? th * ti : 0};
        if (kind < kJoin1) p.nmaps = p.nphase + 1;
        tiles += kind >= kDw1 ? (int64_t)(a.G + split.parts) * rt * ct : nb * ct;
        return p.nphase++;
    };
    if (!a.bwd) {
        p.gu = static_cast<uint16_t*>(a.gu);
        p.h = static_cast<uint16_t*>(a.h);
        p.y = static_cast<uint16_t*>(a.y);
        p.dep_total = ti1 * 2;
        int i = add(kUp, 0, ti1, a.H / kt);
        ok &= make_map_w1(&maps.a[i], a.w1, a.G, a.I, a.H, kt / 64) && make_map_tokens(maps.b[i], a.x, A, a.H, tb, kt / 64);
        i = add(kDown, 0, th, a.I / kt);
        ok &= make_map(&maps.a[i], a.w2, GH, a.I, 128, kt / 64) && make_map_tokens(maps.b[i], a.h, A, a.I, tb, kt / 64);
        if (!ok) return cudaErrorInvalidValue;
        if (size == SMALL) return ffn_launch<false, SMALL>(maps, p, tiles, stream);
        if (size == MID) return ffn_launch<false, MID>(maps, p, tiles, stream);
        return ffn_launch<false, LARGE>(maps, p, tiles, stream);
    }
    p.gu_in = static_cast<const uint16_t*>(a.gu);
    p.dgu = static_cast<uint16_t*>(a.dgu);
    p.dx = static_cast<uint16_t*>(a.dx);
    p.dw1 = static_cast<uint16_t*>(a.dw1);
    p.dw2 = static_cast<uint16_t*>(a.dw2);
    p.dep_total = ti * 2;
    if (a.A > 0 && (a.dx || a.dw1)) {
        const int i = add(kDh, 0, ti, a.H / kt);
        ok &= make_map_mn(&maps.a[i], a.w2, GH, a.I, kt) && make_map_tokens(maps.b[i], a.dy, A, a.H, tb, kt / 64);
    }
    // Without rows the weight gradients are zero and no operand is read.
    const void* any = a.w1;
    const uint64_t rows = A > 0 ? A : 1;
    if (a.dw2) {
        const int i = add(kDw2, th, ti, 0);
        ok &= make_map_mn(&maps.a[i], A ? a.dy : any, rows, a.H, kw) &&
              make_map_mn(&maps.b[i][0], A ? a.h : any, rows, a.I, kw);
    }
    // DW1 last: what it stores at the end leaves L2 after the launch (32 experts of 32 rows: 138
    // us, 148 with DX last). Groups of many rows make its tiles the longest, which would leave
    // pairs idle at the end (one group of 8191 rows: 541 us, 517 with DX last). In between (us with
    // DW1 last, DX last; H 2048, I 768): 8 groups of 512 rows 79.5, 82.5; of 1024 131.8, 132.7; of
    // 2048 241-266, 236-253; 4 of 4096 295-308, 278-289.
    const bool dx_last = a.A > (int64_t)kFfnManyRows * a.G;
    for (int pass = 0; pass < 2; ++pass) {
        if (a.A > 0 && a.dx && dx_last == (pass == 1)) {
            const int i = add(kDx, 0, th, 2 * a.I / kt);
            ok &= make_map_mn(&maps.a[i], a.w1, G2I, a.H, kt) && make_map_tokens(maps.b[i], a.dgu, A, 2 * a.I, tb, kt / 64);
        }
        if (a.dw1 && dx_last == (pass == 0)) {
            const int i = add(kDw1, ti1, th, 0);
            ok &= make_map_mn(&maps.a[i], A ? a.dgu : any, rows, 2 * a.I, kw) &&
                  make_map_mn(&maps.b[i][0], A ? a.x : any, rows, a.H, kw);
        }
    }
    if (split.blocks) {
        if (a.dw2) add(kJoin2, th, ti, 0);
        if (a.dw1) add(kJoin1, ti1, th, 0);
        p.split_blk = split.blocks;
        p.split_tiles = split.tiles;
        p.joined = a.done + block_flags(a.A, a.G);
        p.part = a.part;
    }
    if (!ok) return cudaErrorInvalidValue;
    if (p.nphase == 0) return cudaSuccess;
    if (split.blocks) return ffn_launch<true, LARGE, true>(maps, p, tiles, stream);
    if (size == SMALL) return ffn_launch<true, SMALL>(maps, p, tiles, stream);
    if (size == MID) return ffn_launch<true, MID>(maps, p, tiles, stream);
    return ffn_launch<true, LARGE>(maps, p, tiles, stream);
}

}  // namespace moe
