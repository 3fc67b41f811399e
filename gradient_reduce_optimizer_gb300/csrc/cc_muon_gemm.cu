// The tensor-core products of the Newton-Schulz iteration (cc_muon.cu):
//   A = X X^T - t I          (X^T X - t I for matrices taller than wide)
//   P = b A + c A A
//   Y = rho (a X + P X)      (X P when tall)
// for a batch of matrices, fp16 operands with fp32 accumulation.
//
// No matrix is ever transposed in memory.  Every operand is a row-major
// matrix read either along its rows (K-major) or across them (MN-major), and
// since A and P are symmetric each product has such a form:
//   wide  X X^T  both K-major     P X    P K-major, X MN-major
//   tall  X^T X  both MN-major    X P    both K-major
// A and P are symmetric, so only the tiles on and above the diagonal are
// computed; the epilogue writes each of them twice, the second time
// transposed.
//
// One persistent kernel runs the whole iteration of the whole batch, in
// clusters of two CTAs that share one MMA over two SMs
// (tcgen05.mma.cta_group::2, M = 256: each CTA loads its own 128 rows of A
// and half of the B tile).  All output tiles of all products form one list:
// groups of matrices, in each group step by step and product by product
// matrix after matrix, and the clusters take its tiles in turn.  A matrix's
// product starts when its last one is complete, which a counter per matrix
// says; the tiles in between are other matrices', so that with enough of them
// nobody waits, no product ends in a half-empty wave, and a group's matrices
// stay in L2 from one product to the next.  With few matrices the counter
// takes the place of a launch between dependent products.  The launch is
// cooperative: every cluster is resident, and the earliest unfinished tile
// never waits for a later one, so each wait ends.
//
// In each CTA
//   * a producer warp streams 64-wide k-blocks with TMA into a ring of
//     shared-memory stages, and the leader's MMA warp accumulates them into
//     one of two TMEM accumulators, so that a tile's epilogue overlaps the
//     next one's products;
//   * eight epilogue warps each own 32 rows and every other 64 columns,
//     independently of one another.  The elements of X (and its low part, or
//     of A) come by TMA into the warp's own boxes; accumulators, boxes and
//     results meet as 8 x 8 matrix fragments (tcgen05.ld 16x256b, ldmatrix,
//     stmatrix), so that a transposed copy costs no more than a plain one;
//   * results leave by TMA, issued by two more warps for four epilogue warps
//     each, which also wait until they are in memory and then count the tile.
// What bounds it.  A k-block costs about 2.7 cycles for each 128-byte row of
// operands that the SM's copy engine takes in: 256 rows of a 256 x 256 tile 690
// cycles, where the tensor cores take 512 (and cuBLAS's 8192^3 product, at 1,706
// TFLOP/s and 1,455 MHz, about 545).  One product of a single 1024^2 matrix takes
// 9 us: 3.6 for the k-blocks, the rest from the last one through epilogue, store,
// counter and the first loads of the next.
// A tile's epilogue has to stay below its products (16 k-blocks for K = 1024).
// What it costs is latency, not instructions: a copy instruction queues behind the
// operands' (about 450 cycles), so it moves 4 KiB; and waiting for stores in flight
// (1500 to 4000 cycles) is not the epilogue warps' business.
//
// Ragged sizes: TMA fills what lies outside a matrix with zeros and clips what is
// stored there.  It does so at whole 16 bytes, so the workspace's matrices have
// their rows filled up with zeros to there, and maps that end there.

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "cc_dp_internal.h"
#include "cc_muon_internal.h"
#include "cc_tc_device.cuh"

namespace ccdp {

// Codes or-ed in by a wait of these kernels that ran out.
__device__ unsigned int g_muon_status = 0;

namespace muon {
namespace {

using namespace tc;

constexpr unsigned kStatusProducer = 256u;
constexpr unsigned kStatusMma = 512u;
constexpr unsigned kStatusEpilogue = 1024u;
constexpr unsigned kStatusDrain = 2048u;

constexpr int kBM = 128;                 // output rows of one CTA of the pair
constexpr int kBK = 64;                  // K per stage
constexpr int kUmmaK = 16;
constexpr int kTileA = kBM * kBK * 2;
constexpr int kAccCols = 256;            // TMEM columns per accumulator
constexpr int kTmemCols = 2 * kAccCols;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr int kBox = 32 * 64 * 2;        // an epilogue box: 32 rows x 64 of 16 bits
constexpr int kWarpBytes = 8 * 1024;     // an epilogue warp's boxes
constexpr int kRing = 226 * 1024 - 2048 - kEpiWarps * kWarpBytes;   // operand stages
constexpr int kSmem = kRing + kEpiWarps * kWarpBytes + 1024;
constexpr int kMostStages = 8;
constexpr int kAhead = 8;                // tiles the producer may be ahead of the rest

// An epilogue warp's two boxes, each of 32 rows x 64 columns.  Results: a tile's
// at 0, its transpose (64 x 32) or Y's 8-bit low part at 4 KiB, or the last
// step's fp32 updates at 0 to 8 KiB.  Input, read before they are written: X or A
// at 4 KiB, its low part at 0.  (Boxes of the input's own would let it come one
// unit earlier, and cost a stage of operands.)
constexpr uint32_t kOutAt = 0, kOut2At = 4096, kLoAt = 0, kInAt = 4096;

// What a tile is of.
enum Kind { kGram, kPoly, kUpdate, kFinal };

// The tensor maps of a 16-bit batch: as an operand read along its rows (boxes
// of 64 k x 128 rows as A; half a tile's columns as B, for symmetric results
// and for Y) or across them (64 x 64), and the epilogues' boxes (64 columns x 32
// rows, and transposed).
struct Maps {
    CUtensorMap a, b_sym, b_x, across, box, box_t;
};

// Which tiles of a symmetric product are cut into `pieces` along K (1: none): those
// from `whole` on; and the tiles and pieces of a matrix.
struct Cut {
    int whole, pieces, list;
    float inv_list;
};

struct Params {
    Maps g, x[2], gram, poly;
    CUtensorMap g_lo, lo;                // boxes of low parts: 16-bit of G, 8-bit of X
    int count, rows, cols, small, tall, bf16, has_lo;
    int steps;
    int group, rest;                     // matrices a group; the first `rest` one more
    int bn_sym, bn_x;                    // columns of a tile of A and P, of Y
    int tiles_sym, tiles_x, tiles_xn;    // tiles of A and P, of Y; Y's column tiles
    int tiles_sn;                        // A's column tiles
    float inv_tiles_x, inv_tiles_xn;
    unsigned counts_sym, counts_x;       // what A (or P) and what Y adds to a counter
    int stages, stage_bytes;
    int jobs;
    float shift[CC_MUON_MAX_STEPS], ca[CC_MUON_MAX_STEPS], cb[CC_MUON_MAX_STEPS],
        cc[CC_MUON_MAX_STEPS];
    const float *partial;
    int parts;
    float eps;
    unsigned *done;
    // One large matrix: of A and P, the tiles from `whole` on are cut into
    // `pieces` along K each (1: none), fp32 sums of all but the last in `split`.
    Cut cut_a, cut_p;
    int cut_tiles;                       // of a matrix and product
    float *split;
    unsigned *split_done;                // of each matrix
    unsigned split_counts;               // what a product's pieces add to it
    int stall;                           // a matrix whose counter never gets there, or -1
    unsigned long long limit_ns;         // of a wait for a counter
};

// ---- building blocks ----------------------------------------------------------

// An operand tile across its rows: boxes of 64 k-rows x 64 contiguous MN
// elements (128 bytes, 128-byte swizzle), box after box along MN.  Leading
// offset: from one 64-element block to the next; stride offset: from 8 k to
// the next 8.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((kBK * 128) >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, int x, int y, int z,
                                             uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}
// A TMA load that signals an mbarrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, int x,
                                                 int y, int z, uint32_t bar_cluster) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z),
          "r"(bar_cluster)
        : "memory");
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// Sixteen TMEM lanes (from the address's) x 32 fp32 columns in the layout of
// 8 x 8 matrix fragments: of column block q (8 columns), r[4 q + 2 h + e] is
// row 8 h + lane / 4, column 2 (lane % 4) + e.
__device__ __forceinline__ void tmem_ld_fragments(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// Four 8 x 8 matrices of 16-bit elements, fragment by fragment; lane i gives
// the address of row i % 8 of matrix i / 8 (stored transposed: of column i % 8).
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                          uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                                uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// One thread of a converged warp.  A branch on this, unlike one on the lane's
// number, is known to run a single thread, so that the copies and products in
// it take their operands straight from uniform registers (about 300 cycles less
// for each copy).
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Arrive on an mbarrier given by its cluster address, ordering nothing: the
// accumulator's reads are complete (tcgen05.wait::ld), and a releasing arrive
// would wait for the global stores in flight (measured: 1500 to 4000 cycles).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];"
                 ::"r"(bar_cluster) : "memory");
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 half2_floats(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 bf16x2_floats(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// 16-byte chunk j of row i of a box with 128-byte rows, as the 128-byte swizzle
// lays it, and of one with 64-byte rows, 64-byte swizzle (conflict-free for
// eight rows of one matrix fragment).
__device__ __forceinline__ uint32_t box_at(uint32_t box, int i, int j) {
    return box + static_cast<uint32_t>(i * 128 + ((j ^ (i & 7)) * 16));
}
__device__ __forceinline__ uint32_t box64_at(uint32_t box, int i, int j) {
    return box + static_cast<uint32_t>(i * 64 + ((j ^ ((i >> 1) & 3)) * 16));
}
// 16-byte chunk j of row i of a box of 32 rows x 64 floats.
__device__ __forceinline__ uint32_t wide_at(uint32_t box, int i, int j) {
    return box + static_cast<uint32_t>(i * 256 + ((j ^ (2 * (i & 3))) * 16));
}

// One output tile: 256 rows from m0, bn columns from n0 of matrix b in step k.
// Symmetric results are walked from the diagonal block rightwards; `mirror`:
// the tile lies above the diagonal block of its rows.  `ready`: the matrix's
// counter once what the tile reads is complete.  A cut tile's last piece adds
// the others' sums and makes the result.
struct Tile {
    int kind, k, b, m0, n0, bn;
    int piece, pieces, cut;              // of its K; the cut tile's number
    bool mirror;
    unsigned ready;
};
// q = a / d, r = the rest, by 1 / d: a and d positive.
__device__ __forceinline__ int divide(int a, int d, float inv, int &r) {
    int q = static_cast<int>(static_cast<float>(a) * inv);
    r = a - q * d;
    while (r < 0) {
        r += d;
        --q;
    }
    while (r >= d) {
        r -= d;
        ++q;
    }
    return q;
}
// A place in the list of tiles: product `product` (three a step) of the group of
// `size` matrices from `first` on, `r` tiles into it.
struct Place {
    int first, size, product, r;
    unsigned before;                     // what the group's products so far added
};
__device__ __forceinline__ int tiles_of(const Params &p, int product) {
    const int kind = product % 3;
    return kind == 2 ? p.tiles_x : kind == 1 ? p.cut_p.list : p.cut_a.list;
}
__device__ __forceinline__ Place start_of(const Params &p) {
    return {0, p.group + (p.rest > 0 ? 1 : 0), 0, 0, 0u};
}
// `tiles` further on; whether the list goes on that far.
__device__ __forceinline__ bool advance(const Params &p, Place &a, int tiles) {
    a.r += tiles;
    for (int all; a.r >= (all = a.size * tiles_of(p, a.product));) {
        a.r -= all;
        a.before += a.product % 3 == 2 ? p.counts_x : p.counts_sym;
        if (++a.product == 3 * p.steps) {
            a.first += a.size;
            if (a.first >= p.count) return false;
            a.size = p.group + (a.first < p.rest * (p.group + 1) ? 1 : 0);
            a.product = 0;
            a.before = 0;
        }
    }
    return true;
}
__device__ __forceinline__ Tile tile_at(const Params &p, const Place &a) {
    Tile t;
    t.k = a.product / 3;
    const int kind = a.product - 3 * t.k;
    t.kind = kind == 2 ? (t.k == p.steps - 1 ? kFinal : kUpdate) : kind;
    t.ready = a.before;
    t.piece = t.cut = 0;
    t.pieces = 1;
    int r;
    if (t.kind <= kPoly) {
        const Cut &c = t.kind == kGram ? p.cut_a : p.cut_p;
        t.b = a.first + divide(a.r, c.list, c.inv_list, r);
        if (c.pieces > 1 && r >= c.whole) {
            t.cut = (r - c.whole) / c.pieces;
            t.piece = r - c.whole - t.cut * c.pieces;
            t.pieces = c.pieces;
            r = c.whole + t.cut;
        }
        t.bn = p.bn_sym;
        const int step = 256 / t.bn;
        int i = 0;
        for (int left = p.tiles_sn; r >= left; r -= left, left -= step) ++i;
        t.mirror = r >= step;
        t.m0 = i * 256;
        t.n0 = (i * step + r) * t.bn;
    } else {
        int j;
        t.b = a.first + divide(a.r, p.tiles_x, p.inv_tiles_x, r);
        t.bn = p.bn_x;
        t.mirror = false;
        t.m0 = divide(r, p.tiles_xn, p.inv_tiles_xn, j) * 256;
        t.n0 = j * t.bn;
    }
    if (t.b == p.stall && t.ready > 0) t.ready = 0xFFFFFFFFu;      // failure injection
    return t;
}

// A tile as the producer hands it to the other warps.
struct Job {
    Tile t;
    int kb;
    unsigned idesc;                      // the MMA's instruction descriptor
    bool a_mn, b_mn, once;
};

// Rows and columns of a tile's result.
__device__ __forceinline__ int rows_of(const Params &p, const Tile &t) {
    return t.kind <= kPoly ? p.small : p.rows;
}
__device__ __forceinline__ int cols_of(const Params &p, const Tile &t) {
    return t.kind <= kPoly ? p.small : p.cols;
}
// The batch that is X in step k, and whether a X takes its low part.
__device__ __forceinline__ const Maps &x_maps(const Params &p, int k) {
    return k == 0 ? p.g : p.x[k & 1];
}
__device__ __forceinline__ bool takes_lo(const Params &p, int k) {
    return k == 0 ? p.has_lo != 0 : k <= p.steps - 3;
}

// The operands of a tile and how they are read.
struct Operands {
    const CUtensorMap *a, *b;
    bool a_mn, b_mn;
    bool once;                           // on the diagonal both are the same rows
    int from, kb;                        // the tile's k-blocks: the first, how many
};
__device__ __forceinline__ Operands operands(const Params &p, const Tile &t) {
    Operands o;
    const Maps &x = x_maps(p, t.k);
    int k;
    if (t.kind == kGram) {               // X X^T, or X^T X
        o.a_mn = o.b_mn = p.tall;
        o.a = p.tall ? &x.across : &x.a;
        o.b = p.tall ? &x.across : &x.b_sym;
        k = p.tall ? p.rows : p.cols;
    } else if (t.kind == kPoly) {        // A A
        o.a_mn = o.b_mn = false;
        o.a = &p.gram.a;
        o.b = &p.gram.b_sym;
        k = p.small;
    } else if (p.tall) {                 // X P
        o.a_mn = o.b_mn = false;
        o.a = &x.a;
        o.b = &p.poly.b_x;
        k = p.cols;
    } else {                             // P X
        o.a_mn = false;
        o.b_mn = true;
        o.a = &p.poly.a;
        o.b = &x.across;
        k = p.rows;
    }
    o.once = t.bn == 256 && t.kind <= kPoly && t.m0 == t.n0;
    o.kb = (k + kBK - 1) / kBK;
    o.from = 0;
    if (t.pieces > 1) {
        const int all = o.kb;
        o.from = all * t.piece / t.pieces;
        o.kb = all * (t.piece + 1) / t.pieces - o.from;
    }
    return o;
}

// tcgen05.mma kind::f16: fp16 A and B (or, bits 7 and 10, both bf16), fp32
// accumulator, M = 256 (the pair), N = bn; bits 15 and 16 mark operands read
// across their rows.
__device__ __forceinline__ uint32_t instruction(const Params &p, const Tile &t,
                                                const Operands &o) {
    const bool bf16 = p.bf16 && t.k == 0 && t.kind != kPoly;
    return (1u << 4) | (static_cast<uint32_t>(t.bn >> 3) << 17) |
           (static_cast<uint32_t>(256 >> 4) << 24) | (bf16 ? (1u << 7) | (1u << 10) : 0u) |
           (o.a_mn ? 1u << 15 : 0u) | (o.b_mn ? 1u << 16 : 0u);
}

// A matrix's counter, and the wait until it reaches `target` (at most about
// limit_ns).
__device__ __forceinline__ unsigned progress(const unsigned *done) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(done) : "memory");
    return v;
}
__device__ __forceinline__ bool wait_progress(const unsigned *done, unsigned target,
                                              unsigned long long limit_ns) {
    if (progress(done) >= target) return true;
    const unsigned long long t0 = global_ns();
    while (progress(done) < target) {
        if (global_ns() - t0 > limit_ns) return false;
        __nanosleep(32);
    }
    return true;
}

// A wait that can last as long as several others in turn.
__device__ __forceinline__ bool long_wait(const Params &p, uint32_t bar, uint32_t parity) {
    return mbar_wait(bar, parity, 4 * p.limit_ns);
}

// ---- operands -------------------------------------------------------------------

// The ring of stages as the producer walks it.  parity: of the wait for the
// stage's "empty" barrier; a barrier never used yet passes for parity 1.
struct Ring {
    uint32_t base, empty, full, full_leader, stages, stage_bytes;
    bool leader;
    uint32_t stage, parity;
};
// One tile's operands: where, and the bytes of a k-block in both CTAs.
struct Loads {
    const CUtensorMap *a, *b;
    int m0, n0, matrix, bn;
    uint32_t bytes;
};

// K-blocks [from, to) into the ring.  One thread does this at a few cycles an
// instruction, so what the tile decides is decided outside of the loop.
template <bool A_MN, bool B_MN, bool ONCE>
__device__ __forceinline__ bool load_blocks(Ring &r, const Loads &l, int from, int to) {
#pragma unroll 1
    for (int kb = from; kb < to; ++kb) {
        const uint32_t bar = r.full_leader + 8u * r.stage;
        if (!mbar_wait(r.empty + 8u * r.stage, r.parity)) return false;
        if (r.leader)         // both CTAs' bytes land before the stage is full
            mbar_arrive_expect_tx(r.full + 8u * r.stage, l.bytes);
        const uint32_t sa = r.base + r.stage * r.stage_bytes;
        const int k0 = kb * kBK;
        if constexpr (A_MN) {
            tma_load_3d_pair(sa, l.a, l.m0, k0, l.matrix, bar);
            tma_load_3d_pair(sa + kBK * 128, l.a, l.m0 + 64, k0, l.matrix, bar);
        } else {
            tma_load_3d_pair(sa, l.a, k0, l.m0, l.matrix, bar);
        }
        if constexpr (!ONCE) {
            const uint32_t sb = sa + kTileA;
            if constexpr (B_MN) {
                tma_load_3d_pair(sb, l.b, l.n0, k0, l.matrix, bar);
                if (l.bn == 256)
                    tma_load_3d_pair(sb + kBK * 128, l.b, l.n0 + 64, k0, l.matrix, bar);
            } else {
                tma_load_3d_pair(sb, l.b, k0, l.n0, l.matrix, bar);
            }
        }
        if (++r.stage == r.stages) {
            r.stage = 0;
            r.parity ^= 1u;
        }
    }
    return true;
}

// ---- the epilogue of one chunk --------------------------------------------------
//
// A chunk is 32 rows x 32 columns (half a box), in registers as matrix
// fragments: word 4 q + r (r = 0..3) holds row 8 r + lane / 4, columns 8 q +
// 2 (lane % 4) and the next one.  v[2 w], v[2 w + 1] are word w's fp32 values.

// Start loading a chunk's accumulators: raw[16 h + ...] of rows 16 h ..
__device__ __forceinline__ void load_chunk(uint32_t taddr, uint32_t (&raw)[32]) {
    tmem_ld_fragments(taddr, raw);
    tmem_ld_fragments(taddr + (16u << 16), raw + 16);
}
// In the words' order, once loaded.
__device__ __forceinline__ void ordered(const uint32_t (&raw)[32], float (&v)[32]) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                v[2 * (4 * q + r) + e] =
                    __uint_as_float(raw[16 * (r / 2) + 4 * q + 2 * (r & 1) + e]);
}

// A = c rho^2 acc - shift on the diagonal.
__device__ __forceinline__ void gram_results(float (&v)[32], float c, float rho, float shift,
                                             int lane, bool diagonal) {
    const float f = c * rho;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = v[i] * f * rho;
    if (diagonal) {
        // row 8 r + lane / 4 meets its column in column block q = r
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (lane / 4 == 2 * (lane % 4) + e) v[2 * (4 * r + r) + e] -= shift;
    }
}

// c0 x + c1 acc with x from half `half` of a box of X or of A.
template <bool BF16>
__device__ __forceinline__ void poly_results(float (&v)[32], uint32_t box, int half, float c0,
                                             float c1, int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t h[4];
        ldmatrix4(box_at(box, lane, 4 * half + q), h);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float2 x = BF16 ? bf16x2_floats(h[r]) : half2_floats(h[r]);
            const int w = 4 * q + r;
            v[2 * w] = __fmaf_rn(c0, x.x, c1 * v[2 * w]);
            v[2 * w + 1] = __fmaf_rn(c0, x.y, c1 * v[2 * w + 1]);
        }
    }
}
// + c times X's low part: G's, bf16.
__device__ __forceinline__ void add_lo16(float (&v)[32], uint32_t box, int half, float c,
                                         int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t l[4];
        ldmatrix4(box_at(box, lane, 4 * half + q), l);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float2 x = bf16x2_floats(l[r]);
            const int w = 4 * q + r;
            v[2 * w] = __fmaf_rn(c, x.x, v[2 * w]);
            v[2 * w + 1] = __fmaf_rn(c, x.y, v[2 * w + 1]);
        }
    }
}
// The same of 8 bits (e5m2, the upper byte of an fp16 value): word 4 q + r's two
// values are bytes of fragment word (q / 2, r), the lower two for even q.  The
// chunk's columns lie in the order that gives, for reader and writer alike.
__device__ __forceinline__ void add_lo8(float (&v)[32], uint32_t box, int half, float c, int lane) {
#pragma unroll
    for (int qq = 0; qq < 2; ++qq) {
        uint32_t l[4];
        ldmatrix4(box64_at(box, lane, 2 * half + qq), l);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 x = half2_floats(__byte_perm(l[r], 0, e ? 0x3424 : 0x1404));
                const int w = 4 * (2 * qq + e) + r;
                v[2 * w] = __fmaf_rn(c, x.x, v[2 * w]);
                v[2 * w + 1] = __fmaf_rn(c, x.y, v[2 * w + 1]);
            }
    }
}
// e5m2 of a (lower byte) and b.
__device__ __forceinline__ uint32_t e5m2x2_bits(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// The chunk's low part: v - its fp16 words, times kScaleLo.
__device__ __forceinline__ void store_lo8(uint32_t box, int half, const float (&v)[32],
                                          const uint32_t (&w)[16], int lane) {
#pragma unroll
    for (int qq = 0; qq < 2; ++qq) {
        uint32_t l[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            uint32_t two[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 4 * (2 * qq + e) + r;
                const float2 h = half2_floats(w[i]);
                two[e] = e5m2x2_bits((v[2 * i] - h.x) * kScaleLo, (v[2 * i + 1] - h.y) * kScaleLo);
            }
            l[r] = two[0] | two[1] << 16;
        }
        stmatrix4(box64_at(box, lane, 2 * half + qq), l[0], l[1], l[2], l[3]);
    }
}

// The chunk's 16 words into half `half` of a box, or transposed into rows
// 32 half .. of one.
__device__ __forceinline__ void store_words(uint32_t box, int half, const uint32_t (&w)[16],
                                            int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        stmatrix4(box_at(box, lane, 4 * half + q), w[4 * q], w[4 * q + 1], w[4 * q + 2],
                  w[4 * q + 3]);
}
__device__ __forceinline__ void store_words_transposed(uint32_t box, int half,
                                                       const uint32_t (&w)[16], int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        stmatrix4_trans(box64_at(box, 32 * half + 8 * q + lane % 8, lane / 8), w[4 * q],
                        w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
}

// ---- tiles cut along K ------------------------------------------------------------

// Where a piece's sums of 32 rows (`quarter` of a CTA's) x 64 columns (unit u)
// lie: 64 accumulator words a lane, word by word.
constexpr size_t kPieceFloats = 2 * 4 * 4 * 64 * 32;
__device__ __forceinline__ float *split_at(const Params &p, const Tile &t, int piece, int rank,
                                           int quarter, int u) {
    return p.split +
           static_cast<size_t>((t.b * p.cut_tiles + t.cut) * (t.pieces - 1) + piece) * kPieceFloats +
           static_cast<size_t>((rank * 4 + quarter) * 4 + u) * (64 * 32);
}
// The pieces of this product (their last warp's count).
__device__ __forceinline__ bool pieces_there(const Params &p, const Tile &t, int lane) {
    bool there = true;
    if (lane == 0)
        there = wait_progress(
            p.split_done + t.b,
            static_cast<unsigned>(p.cut_p.pieces > 1 ? 2 * t.k + t.kind + 1 : t.k + 1) *
                p.split_counts,
            p.limit_ns);
    there = __all_sync(0xFFFFFFFFu, there) != 0;
    __syncwarp();                        // orders the other lanes' reads behind lane 0's acquire
    return there;
}
__device__ __forceinline__ void add_sums(uint32_t (&raw)[2][32], const float *from) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __ldcg(from + 32 * (32 * h + i));
#pragma unroll
        for (int i = 0; i < 32; ++i)
            raw[h][i] = __float_as_uint(__fadd_rn(__uint_as_float(raw[h][i]), v[i]));
    }
}

// 1 / (|G|_F + eps) of matrix b, from its partial sums of squares; one warp,
// the same on every lane.
__device__ __forceinline__ float normalisation(const Params &p, int b, int lane) {
    const float *q = p.partial + static_cast<size_t>(b) * kMaxParts;
    float v = 0.0f;
#pragma unroll 4
    for (int i = lane; i < p.parts; i += 32) v += q[i];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return __fdiv_rn(1.0f, __fadd_rn(__fsqrt_rn(v), p.eps));
}

// A master weight after its decay and its update.
__device__ __forceinline__ float updated(const StepOut &o, float w, float y) {
    return __fsub_rn(__fmul_rn(w, o.decay), __fmul_rn(o.lr_scale, y));
}
// Eight of them from element `at` on, a multiple of 8, and their bf16 to every replica.
__device__ __forceinline__ void store_parameters(const StepOut &o, size_t at, const float (&v)[8]) {
    float4 *dst = reinterpret_cast<float4 *>(o.master + at);
    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    const uint4 bits = make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]),
                                  bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
    for (int r = 0; r < o.R; ++r)
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(o.out[r]) + at) = bits;
}

// The parameters of rows row0.. x 64 columns col0.. of matrix b from the box of
// updates: p' = p (1 - lr wd) - lr scale y, its bf16 to every replica.  Eight
// lanes a row, so that each slab is written in whole 128-byte lines.
__device__ __forceinline__ void step_chunk(const Params &p, const StepOut &o, int b, int row0,
                                           int col0, uint32_t box, int lane) {
    const size_t base = o.offset[b];
    if (p.cols % 8 == 0) {
        const int q = lane % 8, col = col0 + 8 * q;
        if (col >= p.cols) return;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float4 w[4][2];
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int row = row0 + 16 * half + 4 * it + lane / 8;
                if (row < p.rows) {
                    const float4 *src = reinterpret_cast<const float4 *>(
                        o.master + base + static_cast<size_t>(row) * p.cols + col);
                    w[it][0] = src[0];
                    w[it][1] = src[1];
                }
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int i = 16 * half + 4 * it + lane / 8, row = row0 + i;
                if (row >= p.rows) continue;
                uint32_t y[8];
                lds128(wide_at(box, i, 2 * q), *reinterpret_cast<uint32_t(*)[4]>(y));
                lds128(wide_at(box, i, 2 * q + 1), *reinterpret_cast<uint32_t(*)[4]>(y + 4));
                float v[8] = {w[it][0].x, w[it][0].y, w[it][0].z, w[it][0].w,
                              w[it][1].x, w[it][1].y, w[it][1].z, w[it][1].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = updated(o, v[e], __uint_as_float(y[e]));
                store_parameters(o, base + static_cast<size_t>(row) * p.cols + col, v);
            }
        }
    } else {
        // Rows off 16-byte boundaries: the vectors that lie whole in the row's 64
        // columns, and before and after them what shares a vector with a neighbour,
        // element by element.  (All of it element by element: 190 us for 12 x 3254 x
        // 355 and four replicas, this 91; of 352 columns, all in vectors, 65.)
        const int q = lane % 8, n = min(64, p.cols - col0);
        if (n <= 0) return;
        auto from_box = [&](int i, int c) {
            float y;
            asm volatile("ld.shared.f32 %0, [%1];"
                         : "=f"(y) : "r"(wide_at(box, i, c / 4) + (c % 4) * 4) : "memory");
            return y;
        };
        constexpr int kDeep = 2;
#pragma unroll 1
        for (int it0 = 0; it0 < 8; it0 += kDeep) {
            size_t at[kDeep];
            int c[kDeep], single[kDeep][2];              // a vector's column, elements'
            float4 w[kDeep][2];
            float w1[kDeep][2];
#pragma unroll
            for (int d = 0; d < kDeep; ++d) {
                const int row = row0 + 4 * (it0 + d) + lane / 8;
                at[d] = base + static_cast<size_t>(row) * p.cols + col0;
                const int head = min(n, static_cast<int>((8 - at[d] % 8) % 8));
                const int whole = (n - head) / 8;
                const bool in = row < p.rows;
                c[d] = in && q < whole ? head + 8 * q : -1;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = q + 8 * h, one = e < head ? e : e + 8 * whole;
                    single[d][h] = in && one < n ? one : -1;
                    if (single[d][h] >= 0) w1[d][h] = o.master[at[d] + one];
                }
                if (c[d] >= 0) {
                    const float4 *src = reinterpret_cast<const float4 *>(o.master + at[d] + c[d]);
                    w[d][0] = src[0];
                    w[d][1] = src[1];
                }
            }
#pragma unroll
            for (int d = 0; d < kDeep; ++d) {
                const int i = 4 * (it0 + d) + lane / 8;
                if (c[d] >= 0) {
                    float v[8] = {w[d][0].x, w[d][0].y, w[d][0].z, w[d][0].w,
                                  w[d][1].x, w[d][1].y, w[d][1].z, w[d][1].w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = updated(o, v[e], from_box(i, c[d] + e));
                    store_parameters(o, at[d] + c[d], v);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (single[d][h] >= 0) {
                        const size_t to = at[d] + single[d][h];
                        const float v = updated(o, w1[d][h], from_box(i, single[d][h]));
                        o.master[to] = v;
                        const __nv_bfloat16 bits = __float2bfloat16_rn(v);
                        for (int r = 0; r < o.R; ++r)
                            static_cast<__nv_bfloat16 *>(o.out[r])[to] = bits;
                    }
            }
        }
    }
}

// bf16 results of rows row0.. x 64 columns col0.. from a box, eight lanes a row.
__device__ __forceinline__ void out_chunk(const Params &p, const PlainOut &o, int b, int row0,
                                          int col0, uint32_t box, int lane) {
    __nv_bfloat16 *base = o.p + static_cast<size_t>(b) * o.stride;
    const bool vec = reinterpret_cast<uintptr_t>(o.p) % 16 == 0 && o.ld % 8 == 0 &&
                     (p.count == 1 || o.stride % 8 == 0) && col0 + 64 <= p.cols;
    if (vec) {
#pragma unroll
        for (int it = 0; it < 8; ++it) {
            const int i = 4 * it + lane / 8, row = row0 + i;
            uint4 w;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(box_at(box, i, lane % 8)) : "memory");
            if (row < p.rows)
                *reinterpret_cast<uint4 *>(base + static_cast<size_t>(row) * o.ld + col0 +
                                           8 * (lane % 8)) = w;
        }
    } else {
        uint16_t *to = reinterpret_cast<uint16_t *>(base) + static_cast<size_t>(row0) * o.ld + col0;
#pragma unroll 8
        for (int i = 0; i < 32; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = lane + 32 * h;
                uint16_t v;
                asm volatile("ld.shared.b16 %0, [%1];"
                             : "=h"(v) : "r"(box_at(box, i, c / 8) + (c % 8) * 2) : "memory");
                if (row0 + i < p.rows && col0 + c < p.cols) to[static_cast<size_t>(i) * o.ld + c] = v;
            }
    }
}

// ---- the kernel -----------------------------------------------------------------

// FINAL: StepOut (the parameter update) or PlainOut (bf16 matrices).
template <typename FINAL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
ns_kernel(const __grid_constant__ Params p, const __grid_constant__ FINAL final_out) {
    constexpr bool kStep = sizeof(FINAL) == sizeof(StepOut);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[kMostStages];     // the leader's is used
    __shared__ __align__(8) uint64_t empty_bar[kMostStages];
    __shared__ __align__(8) uint64_t acc_full[2];
    __shared__ __align__(8) uint64_t acc_empty[2];              // the leader's is used
    __shared__ __align__(8) uint64_t mma_done;
    __shared__ __align__(8) uint64_t input_ready[kAhead];       // the tile's input is complete
    __shared__ __align__(8) uint64_t input_seen[kAhead];        // everybody knows
    __shared__ __align__(8) uint64_t in_full[kEpiWarps];        // input boxes
    __shared__ __align__(8) uint64_t out_full[kEpiWarps];       // result boxes
    __shared__ __align__(8) uint64_t out_free[kEpiWarps];       // stored from
    __shared__ Job ring[kAhead];
    __shared__ uint32_t tmem_base_slot;

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    const uint32_t crank = cluster_ctarank();               // 0: the leader
    const bool leader = crank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMostStages; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&empty_bar[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&acc_full[a]), 1);
            mbar_init(smem_u32(&acc_empty[a]), 2 * kEpiWarps);
        }
        mbar_init(smem_u32(&mma_done), 1);
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(smem_u32(&input_ready[i]), 1);
            mbar_init(smem_u32(&input_seen[i]), 2 + kEpiWarps + (leader ? 1 : 0));
        }
        for (int w = 0; w < kEpiWarps; ++w) {
            mbar_init(smem_u32(&in_full[w]), 1);
            mbar_init(smem_u32(&out_full[w]), 1);
            mbar_init(smem_u32(&out_free[w]), 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    cluster_sync();                                          // the pair's barriers exist
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&tmem_base_slot)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_slot;
    const int first = static_cast<int>(blockIdx.x) / 2;
    const int stride = static_cast<int>(gridDim.x) / 2;
    const uint32_t boxes = base + static_cast<uint32_t>(kRing);

    if (warp == 0) {
        // ---------------- producer (both CTAs) --------------------------
        if (elect_one()) {
            Ring r{base, smem_u32(&empty_bar[0]), smem_u32(&full_bar[0]),
                   map_to_cta(smem_u32(&full_bar[0]), 0), static_cast<uint32_t>(p.stages),
                   static_cast<uint32_t>(p.stage_bytes), leader, 0u, 1u};
            uint32_t n_tile = 0;
            bool ok = true;
            Place place = start_of(p);
            advance(p, place, first);
            Tile t = tile_at(p, place);
            Operands o = operands(p, t);
            bool known = false;                               // the tile's input is complete
            // Put tile n_tile into the ring for the other warps.
            auto publish = [&]() {
                const uint32_t slot = n_tile % kAhead, lap = n_tile / kAhead;
                if (lap > 0 && !long_wait(p, smem_u32(&input_seen[slot]), (lap - 1) & 1)) return false;
                ring[slot] = Job{t, o.kb, instruction(p, t, o), o.a_mn, o.b_mn, o.once};
                return true;
            };
            if (first < p.jobs) ok = publish();
            for (int job = first; ok && job < p.jobs; job += stride) {
                if (!known && !wait_progress(p.done + t.b, t.ready, p.limit_ns)) {
                    ok = false;
                    break;
                }
                mbar_arrive(smem_u32(&input_ready[n_tile % kAhead]));
                // what the counter announces, before copies through the async proxy
                asm volatile("fence.proxy.async.global;" ::: "memory");
                ++n_tile;
                const Operands now = o;
                const Loads l{now.a, now.b, t.m0 + static_cast<int>(crank) * kBM,
                              t.n0 + static_cast<int>(crank) * (t.bn / 2), t.b, t.bn,
                              static_cast<uint32_t>(2 * (kTileA + (now.once ? 0 : t.bn * kBK)))};
                auto stream = [&](int from, int to) {
                    from += now.from;
                    to += now.from;
                    if (now.a_mn)
                        return now.once ? load_blocks<true, true, true>(r, l, from, to)
                                        : load_blocks<true, true, false>(r, l, from, to);
                    if (now.b_mn) return load_blocks<false, true, false>(r, l, from, to);
                    return now.once ? load_blocks<false, false, true>(r, l, from, to)
                                    : load_blocks<false, false, false>(r, l, from, to);
                };
                // the next tile is made out while the stages are full
                const int look = min(now.kb, p.stages + 1);
                ok = stream(0, look);
                if (ok && job + stride < p.jobs) {
                    advance(p, place, stride);
                    t = tile_at(p, place);
                    o = operands(p, t);
                    ok = publish();
                    // complete by now, it need not be asked for again
                    known = progress(p.done + t.b) >= t.ready;
                }
                ok = ok && stream(look, now.kb);
            }
            if (!ok) atomicOr(&g_muon_status, kStatusProducer);
            // The leader's MMAs have read every stage this CTA filled (and so
            // every copy into it has landed) before the CTA may exit.
            for (uint32_t i = 0; i < r.stages; ++i)
                if (!mbar_wait(r.empty + 8u * i, i < r.stage ? r.parity ^ 1u : r.parity))
                    atomicOr(&g_muon_status, kStatusDrain);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer (the leader only) ------------------
        if (leader && elect_one()) {
            const uint32_t stage_units = static_cast<uint32_t>(p.stage_bytes) / 16;
            const uint32_t stages = static_cast<uint32_t>(p.stages);
            uint32_t s = 0, turn = 0, n_tile = 0;
            bool ok = true;
            for (int job = first; ok && job < p.jobs; job += stride, ++n_tile) {
                const uint32_t acc = n_tile & 1u, acc_use = n_tile >> 1;
                const uint32_t slot = n_tile % kAhead;
                if (!long_wait(p, smem_u32(&input_ready[slot]), (n_tile / kAhead) & 1)) {
                    atomicOr(&g_muon_status, kStatusMma);
                    break;
                }
                const int kbs = ring[slot].kb;
                const uint32_t idesc = ring[slot].idesc;
                const bool a_mn = ring[slot].a_mn, b_mn = ring[slot].b_mn;
                const uint32_t b_at = ring[slot].once ? 0u : static_cast<uint32_t>(kTileA);
                mbar_arrive(smem_u32(&input_seen[slot]));
                if (acc_use > 0 && !mbar_wait(smem_u32(&acc_empty[acc]), (acc_use - 1) & 1)) {
                    atomicOr(&g_muon_status, kStatusMma);
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + acc * kAccCols;
                // 16 k further: 32 bytes along a row, or 16 rows of 128 bytes
                const uint64_t step_a = a_mn ? 128u : 2u, step_b = b_mn ? 128u : 2u;
                const uint64_t da0 = a_mn ? smem_desc_mn(base) : smem_desc_sw128(base);
                const uint64_t db0 =
                    b_mn ? smem_desc_mn(base + b_at) : smem_desc_sw128(base + b_at);
                for (int kb = 0; kb < kbs; ++kb) {
                    const bool there = mbar_wait(smem_u32(&full_bar[s]), turn & 1);
                    if (!there) {
                        atomicOr(&g_muon_status, kStatusMma);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t at = static_cast<uint64_t>(s * stage_units);
                    const uint64_t da = da0 + at, db = db0 + at;
#pragma unroll
                    for (int j = 0; j < kBK / kUmmaK; ++j)
                        mma_bf16_pair(d, da + step_a * j, db + step_b * j, idesc,
                                      (kb > 0 || j > 0) ? 1u : 0u);
                    mma_commit_pair(smem_u32(&empty_bar[s]));
                    if (++s == stages) {
                        s = 0;
                        ++turn;
                    }
                }
                if (ok) mma_commit_pair(smem_u32(&acc_full[acc]));
            }
            // Every MMA issued completes before the TMEM is freed.
            mma_commit_pair_local(smem_u32(&mma_done));
            if (!mbar_wait(smem_u32(&mma_done), 0)) atomicOr(&g_muon_status, kStatusDrain);
        }
        __syncwarp();
    } else if (warp < 4) {
        // ---------------- stores of epilogue warps 4 h .. 4 h + 3 ----------
        if (elect_one()) {
            const int h = warp - 2;
            uint32_t parity = 0;                             // of out_full, a bit a warp
            uint32_t n_tile = 0;
            bool ok = true;
            for (int job = first; ok && job < p.jobs; job += stride, ++n_tile) {
                // No tile is counted before all it depends on is: a counter never
                // runs ahead.
                const uint32_t slot = n_tile % kAhead;
                ok = long_wait(p, smem_u32(&input_ready[slot]), (n_tile / kAhead) & 1);
                const Tile t = ring[slot].t;
                if (ok) mbar_arrive(smem_u32(&input_seen[slot]));
                // the last step's results leave otherwise, and nobody waits for them;
                // pieces' sums too
                if (ok && (t.kind == kFinal || t.piece + 1 < t.pieces)) continue;
                const int m = rows_of(p, t), n = cols_of(p, t);
                const int row0 = t.m0 + static_cast<int>(crank) * kBM;
                const CUtensorMap *map = t.kind == kGram   ? &p.gram.box
                                         : t.kind == kPoly ? &p.poly.box
                                                           : &p.x[(t.k + 1) & 1].box;
                const CUtensorMap *map_t = t.kind == kGram ? &p.gram.box_t : &p.poly.box_t;
                const bool lo_out = t.kind == kUpdate && takes_lo(p, t.k + 1);
                for (int u = h; ok && u < t.bn / 64; u += 2) {
                    const int col0 = t.n0 + 64 * u;
                    if (col0 >= n) break;
                    int q = 0;
                    for (; ok && q < 4 && row0 + 32 * q < m; ++q) {
                        const int e = 4 * h + q;
                        ok = long_wait(p, smem_u32(&out_full[e]), (parity >> q) & 1);
                        if (!ok) break;
                        parity ^= 1u << q;
                        const uint32_t mine = boxes + static_cast<uint32_t>(e * kWarpBytes);
                        tma_store_3d(map, col0, row0 + 32 * q, t.b, mine + kOutAt);
                        if (t.mirror) tma_store_3d(map_t, row0 + 32 * q, col0, t.b, mine + kOut2At);
                        if (lo_out) tma_store_3d(&p.lo, col0, row0 + 32 * q, t.b, mine + kOut2At);
                        bulk_commit_group();
                    }
                    bulk_wait_read_all();
                    for (int i = 0; i < q; ++i) mbar_arrive(smem_u32(&out_free[4 * h + i]));
                }
                if (!ok) atomicOr(&g_muon_status, kStatusEpilogue);
                else if (h < t.bn / 64) {
                    // this half of the CTA's tile is in memory
                    bulk_wait_all();
                    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.done + t.b)
                                 : "memory");
                }
            }
            bulk_wait_all();
        }
        __syncwarp();
    } else {
        // ---------------- epilogue ---------------------------------------
        const int e = warp - 4;
        const int quarter = warp % 4;                        // TMEM lanes 32 * quarter ..
        const uint32_t mine = boxes + static_cast<uint32_t>(e * kWarpBytes);
        const uint32_t lane_addr = static_cast<uint32_t>(32 * quarter) << 16;
        const uint32_t leader_empty[2] = {map_to_cta(smem_u32(&acc_empty[0]), 0),
                                          map_to_cta(smem_u32(&acc_empty[1]), 0)};
        uint32_t in_parity = 0, free_parity = 0;
        bool stored = false;                                 // the result boxes may be in use
        uint32_t n_tile = 0;
        bool ok = true;
        auto boxes_free = [&]() {
            if (!stored) return true;
            stored = false;
            const bool free = mbar_wait(smem_u32(&out_free[e]), free_parity);
            free_parity ^= 1u;
            return __all_sync(0xFFFFFFFFu, free) != 0;
        };
        for (int job = first; ok && job < p.jobs; job += stride, ++n_tile) {
            const uint32_t slot = n_tile % kAhead;
            ok = __all_sync(0xFFFFFFFFu,
                            long_wait(p, smem_u32(&input_ready[slot]), (n_tile / kAhead) & 1));
            if (!ok) break;
            const Tile t = ring[slot].t;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&input_seen[slot]));
            const int m = rows_of(p, t), n = cols_of(p, t);
            const int row0 = t.m0 + static_cast<int>(crank) * kBM + 32 * quarter;
            const int units = t.bn / 64;                     // of 64 columns: e / 4, e / 4 + 2
            const uint32_t acc = n_tile & 1u;
            const bool first_x = t.k == 0;                   // X is G as it came
            const bool lo = t.kind >= kUpdate && takes_lo(p, t.k);
            const bool lo16 = lo && first_x;
            const CUtensorMap *in = t.kind == kPoly ? &p.gram.box : &x_maps(p, t.k).box;
            const bool sums = t.piece + 1 < t.pieces;        // only the sums of a piece
            // a unit outside the matrix moves nothing
            auto inside = [&](int u) { return u < units && row0 < m && t.n0 + 64 * u < n; };
            auto load = [&](int u) {
                if (t.kind != kGram && !sums && inside(u) && elect_one()) {
                    // what the counter announced, before this thread's copies through
                    // the async proxy (once a tile)
                    if (u < 2) asm volatile("fence.proxy.async.global;" ::: "memory");
                    const uint32_t bar = smem_u32(&in_full[e]);
                    const int col0 = t.n0 + 64 * u;
                    mbar_arrive_expect_tx(bar, kBox + (lo16 ? kBox : lo ? kBox / 2 : 0));
                    tma_load_3d(mine + kInAt, in, col0, row0, t.b, bar);
                    if (lo16) tma_load_3d(mine + kLoAt, &p.g_lo, col0, row0, t.b, bar);
                    else if (lo) tma_load_3d(mine + kLoAt, &p.lo, col0, row0, t.b, bar);
                }
            };
            ok = boxes_free();
            if (ok) {
                load(e / 4);
                ok = __all_sync(0xFFFFFFFFu,
                                long_wait(p, smem_u32(&acc_full[acc]), (n_tile >> 1) & 1));
            }
            if (!ok) break;
            tc_fence_after();
            // X / scale + its low part / (scale lo_scale), normalised by rho
            const float scale = first_x ? 1.0f : kScaleX;
            const float rho = first_x && t.kind != kPoly ? normalisation(p, t.b, lane) : 1.0f;
            const bool bf16 = p.bf16 && first_x;
            float c0, c1;
            if (t.kind == kGram) {
                c0 = kScaleA / (scale * scale);
                c1 = kScaleA * p.shift[t.k];
            } else if (t.kind == kPoly) {
                c0 = p.cb[t.k] * (kScaleP / kScaleA);
                c1 = p.cc[t.k] * (kScaleP / (kScaleA * kScaleA));
            } else {
                const float out = t.kind == kUpdate ? kScaleX * rho : rho;   // Y as it is kept
                c0 = p.ca[t.k] / scale * out;
                c1 = 1.0f / (kScaleP * scale) * out;
            }
            bool held = true;                                // the accumulator
#pragma unroll 1
            for (int u = e / 4; u < units; u += 2) {
                uint32_t raw[2][32];
                const uint32_t addr = tmem + lane_addr + acc * kAccCols + 64 * u;
                load_chunk(addr, raw[0]);
                load_chunk(addr + 32, raw[1]);
                if (u >= 2) {                                // the next unit's input
                    if (!boxes_free()) {
                        tmem_wait_ld();
                        ok = false;
                        break;
                    }
                    load(u);
                }
                tmem_wait_ld();
                if (u + 2 >= units) {                        // the accumulator has been read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(leader_empty[acc]);
                    held = false;
                }
                if (!inside(u)) continue;
                if (sums) {
                    float *to = split_at(p, t, t.piece, static_cast<int>(crank), quarter, u) + lane;
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        __stcg(to + 32 * i, __uint_as_float(raw[i / 32][i % 32]));
                    continue;
                }
                if (t.pieces > 1) {
                    if (!pieces_there(p, t, lane)) {
                        ok = false;
                        break;
                    }
                    for (int i = 0; i + 1 < t.pieces; ++i)
                        add_sums(raw, split_at(p, t, i, static_cast<int>(crank), quarter, u) + lane);
                }
                const int col0 = t.n0 + 64 * u;
                float v[2][32];
                ordered(raw[0], v[0]);
                ordered(raw[1], v[1]);
                if (t.kind == kGram) {
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        gram_results(v[half], c0, rho, c1, lane, col0 + 32 * half == row0);
                } else {
                    const bool there = mbar_wait(smem_u32(&in_full[e]), in_parity);
                    in_parity ^= 1u;
                    if (!__all_sync(0xFFFFFFFFu, there)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (bf16 && t.kind != kPoly)
                            poly_results<true>(v[half], mine + kInAt, half, c0, c1, lane);
                        else poly_results<false>(v[half], mine + kInAt, half, c0, c1, lane);
                        if (lo16) add_lo16(v[half], mine + kLoAt, half, c0, lane);
                        else if (lo)
                            add_lo8(v[half], mine + kLoAt, half, c0 * (1.0f / kScaleLo), lane);
                    }
                    __syncwarp();                            // the input has been read
                }
                if (t.kind <= kUpdate) {
                    const bool lo_out = t.kind == kUpdate && takes_lo(p, t.k + 1);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t w[16];
                        if (t.kind == kPoly && bf16) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = bf16x2_bits(v[half][2 * i], v[half][2 * i + 1]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = half2_bits(v[half][2 * i], v[half][2 * i + 1]);
                        }
                        store_words(mine + kOutAt, half, w, lane);
                        if (t.mirror) store_words_transposed(mine + kOut2At, half, w, lane);
                        if (lo_out)
                            store_lo8(mine + kOut2At, half, v[half], w, lane);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&out_full[e]));
                    stored = true;
                } else if constexpr (kStep) {
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int row = 8 * (i % 4) + lane / 4;
                            const int chunk = 8 * half + 2 * (i / 4) + (lane % 4) / 2;
                            asm volatile("st.shared.v2.f32 [%0], {%1, %2};"
                                         ::"r"(wide_at(mine, row, chunk) + 8 * (lane & 1)),
                                           "f"(v[half][2 * i]), "f"(v[half][2 * i + 1])
                                         : "memory");
                        }
                    __syncwarp();
                    step_chunk(p, final_out, t.b, row0, col0, mine, lane);
                    fence_proxy_async_smem();                // the box has been read: the
                    __syncwarp();                            // next input may come
                } else {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = bf16x2_bits(v[half][2 * i], v[half][2 * i + 1]);
                        store_words(mine + kOutAt, half, w, lane);
                    }
                    __syncwarp();
                    out_chunk(p, final_out, t.b, row0, col0, mine + kOutAt, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }
            if (sums) {                                      // this warp's part is in memory
                __threadfence();
                __syncwarp();
                if (lane == 0)
                    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.split_done + t.b)
                                 : "memory");
            }
            if (held) {                                      // no unit for this warp
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(leader_empty[acc]);
            }
        }
        if (!ok && lane == 0) {
            atomicOr(&g_muon_status, kStatusEpilogue);
            // a wait ran out: give the copies in flight time to land
            if (!mbar_wait(smem_u32(&in_full[e]), in_parity, p.limit_ns))
                atomicOr(&g_muon_status, kStatusDrain);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();                                          // the peer is done with us
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                     ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ---- host side ------------------------------------------------------------------

int encode_map(CUtensorMap *map, const Batch &x, int box_cols, int box_rows, bool bytes = false) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return fail(CC_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled unavailable");
    const size_t elem_bytes = bytes ? 1 : 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(x.cols), static_cast<cuuint64_t>(x.rows),
                                static_cast<cuuint64_t>(x.count)};
    const cuuint64_t strides[2] = {x.ld * elem_bytes, x.stride * elem_bytes};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows),
                               1};
    const cuuint32_t elem[3] = {1, 1, 1};
    const size_t row = box_cols * elem_bytes;
    const CUresult res =
        fn(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
           const_cast<void *>(x.p), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
           row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (res != CUDA_SUCCESS)
        return fail(CC_ERR_INVALID, "tensor map rejected (CUresult %d)", static_cast<int>(res));
    return CC_OK;
}

int encode(const Batch &x, const Params &p, Maps *maps) {
    int st;
    if ((st = encode_map(&maps->a, x, 64, 128)) != CC_OK) return st;
    if ((st = encode_map(&maps->b_sym, x, 64, p.bn_sym / 2)) != CC_OK) return st;
    if ((st = encode_map(&maps->b_x, x, 64, p.bn_x / 2)) != CC_OK) return st;
    if ((st = encode_map(&maps->across, x, 64, 64)) != CC_OK) return st;
    if ((st = encode_map(&maps->box, x, 64, 32)) != CC_OK) return st;
    return encode_map(&maps->box_t, x, 32, 64);
}

// Tiles of a symmetric m x m result in blocks of 256 x bn, from the diagonal
// block rightwards.
int symmetric_tiles(int m, int bn) {
    const int across = (m + bn - 1) / bn;
    int tiles = 0;
    for (int i = 0; i < (m + 255) / 256; ++i) tiles += across - i * (256 / bn);
    return tiles;
}

constexpr double kBlockCycles[3] = {690.0, 430.0, 375.0};    // of 256, 128, 64 columns

// Pieces of each of the `left` tiles that a large product has over after whole
// rounds: they are spread over all clusters, but four at most, since the last one
// reads the others' sums (about two microseconds a piece), within kMostPieces.
int pieces_of(int left, int clusters) {
    int pieces = left > 0 ? std::min(4, clusters / left) : 1;
    while (pieces > 1 && left * (pieces - 1) > kMostPieces) --pieces;
    return std::max(1, pieces);
}

// Pieces of every tile of A where there are few (`tiles` in all) and K is long: the
// fewest cycles of a piece's k-blocks and of adding the sums up (us, whole and in
// the pieces taken: 2 x 3328 x 200 151 and 130, 1 x 300 x 4000 141 and 128, 2 x 500 x
// 4000 168 and 158; 1 x 700 x 1400, where none are taken, 128 and 135 with two).
int pieces_of_long(int tiles, int kbs, double cycles, int clusters) {
    int best = 1;
    double least = kbs * cycles;
    for (int s = 2; s <= 8 && tiles * s <= clusters && tiles * (s - 1) <= kMostPieces; ++s) {
        const double cost = (kbs + s - 1) / s * cycles + 3000.0 + 2000.0 * s;
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

// Whether tiles are cut: one matrix, with more tiles of A than clusters.  (With
// several matrices others' tiles fill a round; with fewer tiles narrower ones do.)
bool cuts(int count, int small, int clusters) {
    return count == 1 && symmetric_tiles(small, 256) > clusters;
}

// The columns of the tiles of A and P and of those of Y.  Narrower tiles spread
// a product over more clusters and leave a shorter epilogue after it, but take
// in more operand bytes for their size.  The width with the least estimate is
// taken: a tile costs its k-blocks or, where that is more, its epilogue (a
// 64-column tile's no less than 128's, since half of its warps are idle); from one
// product to the next a matrix waits for an epilogue and the way through memory,
// which other matrices' tiles hide when there are several to a cluster; and rounds
// are whole where nothing follows up.  The constants, in cycles, are fitted to
// all widths' times of 109 batches (1 to 64 matrices of 66 to 4100 a side): the
// choice is 0.2 % slower than the best one in the mean and 3.5 % at most.  (A second
// operand read across its rows comes in boxes of 64 columns a CTA: X^T X and
// P X have 128 at least.)
void choose_widths(Params &p, int clusters) {
    const int widths[3] = {256, 128, 64};
    const double(&cycles)[3] = kBlockCycles;
    const double epilogue[3] = {6800.0, 4300.0, 4250.0};
    const int matrices = p.group + (p.rest ? 1 : 0);
    double best_sym = 0.0, best_x = 0.0;
    p.bn_sym = p.bn_x = 0;
    for (int i = 0; i < 3; ++i) {
        const int bn = widths[i];
        auto cost = [&](int tiles, int k, bool cut = false) {
            const int kbs = (k + kBK - 1) / kBK;
            const double tile = std::max(kbs * cycles[i], epilogue[i]);
            double latency = 2000.0 + epilogue[i];
            const int pieces = cut ? pieces_of(tiles % clusters, clusters) : 1;
            if (pieces > 1)
                return (tiles / clusters + 1.0 / pieces) * tile + latency +
                       2000.0 * (tiles / clusters) + 4000.0 * pieces;
            const double r = static_cast<double>(tiles) * matrices / clusters;
            const double rounds = r <= 1.0 || matrices == 1 ? std::ceil(r) : r;
            if (matrices > 1) latency *= std::max(0.25, 1.0 - 0.75 * std::max(0.0, r - 1.0));
            return rounds * tile + latency + 2000.0 * (rounds - 1.0);
        };
        const int sym = symmetric_tiles(p.small, bn);
        const bool cut = bn == 256 && cuts(p.count, p.small, clusters);
        const double c_sym =
            cost(sym, std::max(p.rows, p.cols), cut) + cost(sym, p.small, cut);
        if ((bn >= 128 || !p.tall) && (p.bn_sym == 0 || c_sym < best_sym)) {
            p.bn_sym = bn;
            best_sym = c_sym;
        }
        const double c_x = cost((p.rows + 255) / 256 * ((p.cols + bn - 1) / bn), p.small);
        if ((bn >= 128 || p.tall) && (p.bn_x == 0 || c_x < best_x)) {
            p.bn_x = bn;
            best_x = c_x;
        }
    }
}

// One-shot injected stall of this thread's next launch (cc_inject_muon_stall): the
// matrix whose second product never starts, or -1, and the limit of the waits.
thread_local int g_stall_matrix = -1;
thread_local unsigned long long g_stall_ns = 0;

template <typename FINAL>
int iterate(const Iteration &it, const FINAL &out, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return fail_cuda(e, "SM count");
    Params p{};
    p.count = it.x[0].count;
    p.rows = it.rows;
    p.cols = it.cols;
    p.small = std::min(p.rows, p.cols);
    p.tall = p.rows > p.cols;
    p.bf16 = it.bf16;
    p.has_lo = it.g_lo.p != nullptr;
    p.steps = it.steps;
    p.partial = it.partial;
    p.parts = it.parts;
    p.eps = it.eps;
    p.done = it.done;
    p.stall = g_stall_matrix;
    p.limit_ns = g_stall_matrix >= 0 ? g_stall_ns : kTimeoutNs;
    g_stall_matrix = -1;
    for (int k = 0; k < it.steps; ++k) {
        const float *c = it.coeffs + 3 * k;
        // near the end, but not before the singular values have grown (k = 2)
        const double t = 0.25 * std::max(0, std::min(3 - (it.steps - 1 - k), k - 1));
        // a + b l + c l^2 around l = t
        p.shift[k] = static_cast<float>(t);
        p.ca[k] = static_cast<float>(c[0] + t * (c[1] + t * c[2]));
        p.cb[k] = static_cast<float>(c[1] + 2.0 * t * c[2]);
        p.cc[k] = c[2];
    }
    // Groups of matrices with about three tiles a cluster in each product, so
    // that a matrix's next product finds its last one complete (96 x 1024^2, a
    // step of R = 8: one tile a cluster 3.10 ms, two 2.56, three 2.49, four 2.54;
    // larger groups leave L2).
    const int group = std::max(1, 240 / symmetric_tiles(p.small, 256));
    const int groups = std::max(1, p.count / group);
    p.group = p.count / groups;
    p.rest = p.count % groups;

    auto kernel = ns_kernel<FINAL>;
    e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return fail_cuda(e, "shared memory attribute");
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
    int clusters = 0;               // that are resident at once
    e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    if (e != cudaSuccess) return fail_cuda(e, "cluster occupancy");
    clusters = std::min(clusters, sms / 2);
    if (clusters < 1) return fail(CC_ERR_UNSUPPORTED, "no CTA pair fits the device");
    choose_widths(p, clusters);
    p.stage_bytes = kTileA + std::max(p.bn_sym, p.bn_x) / 2 * kBK * 2;
    p.stages = std::min(kRing / p.stage_bytes, kMostStages);
    p.tiles_sym = symmetric_tiles(p.small, p.bn_sym);
    p.cut_a = p.cut_p = Cut{p.tiles_sym, 1, p.tiles_sym, 0.0f};
    p.split = it.split;
    p.split_done = it.done + p.count;
    if (p.bn_sym == 256 && it.split && cuts(p.count, p.small, clusters)) {
        const int left = p.tiles_sym % clusters;
        const int pieces = pieces_of(left, clusters);
        if (pieces > 1) {
            const int whole = p.tiles_sym - left;
            p.cut_a = p.cut_p = Cut{whole, pieces, whole + left * pieces, 0.0f};
            p.cut_tiles = left;
            // every epilogue warp of both CTAs counts
            p.split_counts = static_cast<unsigned>(left * (pieces - 1) * 2 * kEpiWarps);
        }
    } else if (it.split && groups == 1) {
        const int pieces = pieces_of_long(
            p.count * p.tiles_sym, (std::max(p.rows, p.cols) + kBK - 1) / kBK,
            p.bn_sym == 256 ? kBlockCycles[0] : p.bn_sym == 128 ? kBlockCycles[1] : kBlockCycles[2],
            clusters);
        if (pieces > 1) {
            p.cut_a = Cut{0, pieces, p.tiles_sym * pieces, 0.0f};
            p.cut_tiles = p.tiles_sym;
            p.split_counts = static_cast<unsigned>(p.tiles_sym * (pieces - 1) * 2 * kEpiWarps);
        }
    }
    p.cut_a.inv_list = 1.0f / static_cast<float>(p.cut_a.list);
    p.cut_p.inv_list = 1.0f / static_cast<float>(p.cut_p.list);
    p.tiles_sn = (p.small + p.bn_sym - 1) / p.bn_sym;
    p.tiles_xn = (p.cols + p.bn_x - 1) / p.bn_x;
    p.tiles_x = (p.rows + 255) / 256 * p.tiles_xn;
    // two CTAs report each tile, for each half of its columns if it has two
    p.counts_sym = static_cast<unsigned>(p.tiles_sym) * (p.bn_sym >= 128 ? 4u : 2u);
    p.counts_x = static_cast<unsigned>(p.tiles_x) * (p.bn_x >= 128 ? 4u : 2u);
    p.inv_tiles_x = 1.0f / static_cast<float>(p.tiles_x);
    p.inv_tiles_xn = 1.0f / static_cast<float>(p.tiles_xn);
    const size_t jobs =
        static_cast<size_t>(p.cut_a.list + p.cut_p.list + p.tiles_x) * p.steps * static_cast<size_t>(p.count);
    if (jobs > 0x3FFFFFFFu) return fail(CC_ERR_INVALID, "%zu tiles: too many", jobs);
    p.jobs = static_cast<int>(jobs);
    int st;
    if ((st = encode(it.g, p, &p.g)) != CC_OK || (st = encode(it.x[0], p, &p.x[0])) != CC_OK ||
        (st = encode(it.x[1], p, &p.x[1])) != CC_OK || (st = encode(it.a, p, &p.gram)) != CC_OK ||
        (st = encode(it.p, p, &p.poly)) != CC_OK ||
        (p.has_lo && (st = encode_map(&p.g_lo, it.g_lo, 64, 32)) != CC_OK) ||
        (st = encode_map(&p.lo, it.lo, 64, 32, true)) != CC_OK)
        return st;

    cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min(clusters, p.jobs)));
    e = cudaLaunchKernelEx(&cfg, kernel, p, out);
    return e == cudaSuccess ? CC_OK : fail_cuda(e, "orthogonalisation launch");
}

}  // namespace

int iterate_out(const Iteration &it, const PlainOut &out, cudaStream_t stream) {
    return iterate(it, out, stream);
}
int iterate_step(const Iteration &it, const StepOut &out, cudaStream_t stream) {
    return iterate(it, out, stream);
}

}  // namespace muon

void arm_muon_stall(int matrix, unsigned long long limit_ns) {
    muon::g_stall_matrix = matrix;
    muon::g_stall_ns = limit_ns;
}

cudaError_t read_muon_status(unsigned *status, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(status, g_muon_status, sizeof(unsigned));
    if (e == cudaSuccess && clear) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_muon_status, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace ccdp
