// Attention of one new token per sequence over the paged cache:
//
//     o[b, h] = sum_j p_j v_j,  p = softmax over lo <= j < n of s_j = cap(scale q[b, h] . k_j),
//
// n = lengths[b], lo = max(0, n - window) (0 without a window), cap(s) =
// c tanh(s / c) when c > 0.  Heads share the keys of head h / group.  n = 0
// gives zeros.  With weights, weights[b, g, j] grows by the sum of p_j over the
// group's heads.
//
// Every key and value row is read once and used for `group` heads: 4 group
// operations per 16-bit element pair, so the reading bounds it (6.8 TB/s), and
// the design is about keeping enough bytes in flight on every SM whatever the
// batch looks like.
//
// Work.  An item is one sequence, key head and block of up to 8 * NT query
// heads; its positions come in tiles of kWarps * kKeys.  The tiles of all
// sequences in a row are cut into equal runs, and each run is given to one CTA
// per (key head, block), as many as fit the GPU at once: a ragged batch, or a
// single long sequence, loads every SM alike, and the heads of a position are
// read at about the same time, which is what DRAM wants where they lie side by
// side (with every CTA on its own, 64-byte rows of 8 heads come at 2.7 TB/s
// instead of 5.2, and blocks of one head read its rows twice).  Each CTA finds
// its run from the lengths, which only the device knows.  With so many heads
// that a run each would leave places empty, runs go through the heads instead.
// A run that ends inside an item leaves (maximum, sum, output) of its part in
// the workspace, and the CTA that arrives last joins the parts in order of
// position (the result does not depend on the order of arrival).
//
// A CTA.  Each warp owns kKeys positions of a tile and a ring of kStages
// stages in shared memory that it fills with its own asynchronous 16-byte
// copies and drains alone: no barrier between warps until an item ends.  A row
// is found through the page list, so any page size and layout will do; page
// numbers are fetched one step before the copies that need them.
//
// Arithmetic.  Positions are the rows (M = 16) and heads the columns (N = 8) of
// both products: S^T = K Q^T and O^T += V^T P^T with mma.sync m16n8k16, K as it
// lies and V transposed by ldmatrix.  Eight heads fill a tile, where heads as
// rows would leave half of sixteen empty, and P^T turns from accumulator to
// operand by one 8 x 8 transpose per eight positions.  (tcgen05 needs 64 or 128
// rows of one operand: with 8 heads at most 1/8 of it would be used, and P would
// have to go through shared or tensor memory, to speed up what is not the bound.)
// The softmax keeps a running reference m (at first the maximum; moved when
// that grows by a factor 2^8, so that the output is rarely rescaled) and the sum
// of the weights in fp32.  The tensor core takes no wider operand than 16 bits at
// this rate, so P goes in as two of them (split16).  fp16 rounds what is below
// 2^-25 to zero: there the reference stays 2^7 below the maximum, so that P
// uses the range up to 2^15 and only weights below 2^-32 of the largest that the
// warp has met are lost (the same times for every case measured).
//
// e4m3 rows are widened to fp16 exactly.  The row's key scale multiplies its
// score.  Its value scale vs_j = f 2^e, 1 <= f < 2, joins the weight that
// multiplies the row, f 2^(t_j + e - mu), with a reference mu of its own that
// follows the largest t_j + e of the rows that are not all zeros: P stays in
// fp16's range whatever the scales are (any that fp32 holds), what is lost is
// below 2^-31 of the largest weight times scale of these rows that the warp has
// met, and the sum, 2^(t_j - m), does not know of the scales.  The outputs change
// to the reference m when the warps are joined.  bf16 queries enter the first
// product as fp16 after a power of two per head has been taken out.
//
// Weights.  p_j is known only when the item is joined, so the scores (fp32) go
// to the workspace and a second kernel adds 2^(t_j - m) / sum over the group.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv_cache.cuh"

namespace tgemm {

constexpr int kAttendMaxCtas = 320;       // CTAs at most (workspace slots)
constexpr int kAttendFanIn = 18;          // parts joined at once, at most
constexpr int kAttendOneLevel = 16;       // parts of an item joined at once (more: in two levels)
static_assert(kAttendMaxCtas <= kAttendFanIn * kAttendFanIn, "two levels join every CTA's part");
constexpr int kAttendDirect = 8;          // parts that threads join on their own
constexpr float kAttendGrow = 8.0f;       // log2 of the factor that moves the reference
constexpr float kAttendBelow = 7.0f;      // log2 of the maximum over the reference that it sets, where P is fp16
constexpr float kAttendScaledBelow = kAttendBelow - 1.0f;     // where a factor f < 2 multiplies P
static_assert(kAttendGrow + kAttendBelow <= 15.0f, "P in fp16's range");

// The workspace: arrival counters (zero between calls), the parts' outputs
// and their (m, l), then, with weights, each head's (m, l) and scores.
struct AttendSpace {
    unsigned *parts;        // [2 * kAttendMaxCtas]: arrivals at a group of parts, by its first part's slot
    unsigned *groups;       // [2 * kAttendMaxCtas]: arrivals of an item's groups, by its first part's slot
    float *out;             // [2 * kAttendMaxCtas][heads of a block][padded dim]
    float2 *ml;             // [2 * kAttendMaxCtas][heads of a block]
    float2 *stats;          // [batch, q_heads]
    float *scores;          // [batch, heads, positions, scored]: in log2 units, before the reference is taken off
};

struct AttendParams {
    KvView cache;
    KvTable table;
    KvWeights weights;
    AttendSpace space;
    const unsigned char *q;
    unsigned char *o;
    long long q_batch_stride, q_head_stride, o_batch_stride, o_head_stride;   // bytes
    long long positions;                  // what the page lists can hold
    int scored;                           // query heads of a key head, rounded up to an even number
    int group, blocks;                    // query heads of a key head; blocks that they make
    int lanes;                            // CTAs that share a run: heads * blocks, or 1
    int window;
    int page_shift;                       // log2 of the page size, -1: not a power of two
    // A score in log2 units is first * (q . k); capped, last * tanh(first * (q . k)).
    float first, last;
    bool capped;
    unsigned int *status;
    long long dbg_o_bytes, dbg_scores;    // debug builds: O's bytes, the workspace's scores
};

// Shapes.  A step is a chain (copy, product, softmax, product) with a fixed cost
// of some hundred instructions, and a warp has no more than one on the way, so
// the SM wants many warps, each with as much in a step as the ring allows: 96
// KiB per CTA, steps of 16 positions, 32 where a row has 128 bytes or less (e4m3
// 128 wide, 8 warps with steps of 16: 2.1 TB/s, 6 with 32: 6.2).  Six warps of two
// stages beat four of three for 16-bit rows of 256 dims, whose CTA is alone on its
// SM (6.5 against 6.3 TB/s); two or three eights of heads need 255 registers, and
// spill even so where they are three of 128 dims (428 bytes stored; two of 64,
// with 168 registers: 84).
template <bool kE4m3, int DP, int NT>
struct AttendShape {
    static constexpr int kRow = DP * (kE4m3 ? 1 : 2);                     // bytes of a row in shared memory
    static constexpr int kKeys = kRow >= 256 ? 16 : 32;                   // positions of a warp's step
    static constexpr int kWarps = (DP * NT >= 192 && kRow < 512) || (kE4m3 && NT == 2) ? 4 : 6;   // 255 registers a thread, or 168
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kTile = kWarps * kKeys;
    static constexpr int kHeads = 8 * NT;
    static constexpr int kStage = 2 * kKeys * kRow;                       // keys, values
    static constexpr int kStages = kRow >= 512 || DP * NT > 256 ? 2 : 98304 / (kWarps * kStage);
    static constexpr int kSide = kE4m3 ? 2 * kKeys * 4 + 16 : 16;         // a stage's scales and mask
    static constexpr int kSides = kWarps * kStages * kStage;              // where the sides begin
    static constexpr int kOffsets = kSides + kWarps * kStages * kSide;    // a step's rows in the pools
    static constexpr int kMerge = kOffsets + kWarps * kKeys * 8;
    static constexpr int kPitch = DP + 4;                                 // floats: heads 2t, dims g fall into different banks
    static constexpr int kBytes = kMerge + kHeads * kPitch * 4;
    static constexpr int kCtas = kBytes + 4096 <= 115712 ? 2 : 1;         // per SM: 228 KiB, of which each CTA also takes 1 KiB and its statics
    static_assert(kBytes + 4096 <= 232448, "a CTA's shared memory");
    static_assert(kStage % 128 == 0 && kOffsets % 16 == 0 && kMerge % 16 == 0, "alignment");
};

// ---------------------------------------------------------------- primitives
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool ok) {
    const int bytes = ok ? 16 : 0;          // 0: the destination is filled with zeros, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool ok) {
    const int bytes = ok ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// The bits that any of four words in shared memory has.
__device__ __forceinline__ uint32_t lds_or(uint32_t addr) {
    uint32_t a, b, c, d;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
    return a | b | c | d;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kBf16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four e4m3 values as fp16: the lower two and the upper two.
__device__ __forceinline__ void widen4(uint32_t x, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}

// Counts up to `last` and from there back to 0; returns the count before.  The
// block's writes before it (through a barrier) are visible to the blocks that
// count after it, and theirs before to this one.
__device__ __forceinline__ unsigned count_acq_rel(unsigned *counter, unsigned last) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(counter), "r"(last) : "memory");
    return old;
}

// 2^x, results below 2^-126 flushed to zero (relative error about 2^-22).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x = f * 2^e, 1 <= |f| < 2; e = -infinity for 0; an infinity or NaN is its own f.
__device__ __forceinline__ void split_scale(float x, float &e, float &f) {
    const bool small = fabsf(x) < 0x1p-126f;
    const float y = small ? x * 0x1p32f : x;
    const uint32_t bits = __float_as_uint(y);
    const int field = static_cast<int>((bits >> 23) & 255u);
    e = field == 0 ? -INFINITY : static_cast<float>(field - (small ? 159 : 127));
    f = field == 255 ? x : __uint_as_float((bits & 0x807FFFFFu) | 0x3F800000u);
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pair16(float lo, float hi) {
    if (kBf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Two weights w >= 0 as sums of 16-bit values: `high` towards zero, and what that
// leaves, rounded: off by at most 2^-16 of w (bf16), 2^-21 or 2^-25 absolutely
// (fp16).  Neither is 0 where w is not tiny, nor negative, so that an infinity
// among the values stays one: for bf16 w's last bit is set before (2^-23 of it),
// for fp16 `high` is taken of a little less.  (32 contexts of 9000, 128 wide, 8
// heads on each of 8: 178.6 us, with w rounded once 178.8; 24 heads 228.9 and
// 215.5; e4m3, 8 heads 107.0 and 105.6, 16 heads 138.7 and 123.6.)
template <bool kBf16>
__device__ __forceinline__ void split16(float w0, float w1, uint32_t &high, uint32_t &rest) {
    if (kBf16) {
        const uint32_t a = __float_as_uint(w0) | 1u, b = __float_as_uint(w1) | 1u;
        high = __byte_perm(a, b, 0x7632);
        rest = pair16<true>(__uint_as_float(a) - __uint_as_float(a & 0xFFFF0000u),
                            __uint_as_float(b) - __uint_as_float(b & 0xFFFF0000u));
    } else {
        constexpr float kLess = 1.0f - 0x1p-12f, kStep = 0x1.fffffep-25f;      // just below fp16's smallest step
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(high) : "f"(fmaf(w1, kLess, -kStep)), "f"(fmaf(w0, kLess, -kStep)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&high));
        rest = pair16<false>(w0 - f.x, w1 - f.y);
    }
}

// ---------------------------------------------------------------- the runs
// Where a run is: the item (sequence b, key head, block of query heads) and the
// tile in it.
struct AttendCursor {
    int b, head, block, tile, tiles, n, lo;
};

// Positions and tiles of a sequence; `pad`: tiles come in multiples of it.
__host__ __device__ inline int attend_tiles(int n, int window, int tile, int pad, int *lo) {
    *lo = window > 0 && n > window ? n - window : 0;
    int t = (n - *lo + tile - 1) / tile;
    if (t < 1) t = 1;                       // an empty sequence still has its zeros to write
    return (t + pad - 1) / pad * pad;
}

// How many of the positions of a warp's step, which begin `in_tile` into tile `tile`, the workspace has scores for: all
// of those that the step has rows of, unless the lengths change while the kernel runs.
__host__ __device__ inline long long attend_scored(int lo, int tile, int tile_size, int in_tile, long long positions) {
    const long long at = lo + static_cast<long long>(tile) * tile_size + in_tile;
    return at < positions ? positions - at : 0;
}

// With up to 32 sequences and few tiles, runs of one length that end with their item (its
// tiles padded to a multiple) join faster than equal ones that begin and end
// anywhere.  The shortest of these lengths is taken that makes at most `runs`
// of them, unless that would cost more than four tiles over an equal share.
// units[k]: runs of length attend_length(k) that the items make; 0: equal runs.
constexpr int kAttendLengths = 8;
__host__ __device__ inline int attend_length(int k) {
    constexpr int kLength[kAttendLengths] = {1, 2, 3, 4, 6, 8, 12, 16};
    return kLength[k];
}
__host__ __device__ inline int attend_pad(const long long *units, long long total, int runs) {
    for (int k = 0; k < kAttendLengths; ++k)
        if (units[k] <= runs && static_cast<long long>(attend_length(k)) * runs <= total + 4ll * runs) return attend_length(k);
    return 0;
}

// Run c of `ctas` has the tiles [attend_first(c), attend_first(c + 1)) of `total`;
// attend_owner() is the inverse.
__host__ __device__ inline long long attend_div(long long a, long long b) {     // a >= 0, b > 0
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}
__host__ __device__ inline long long attend_first(long long c, long long ctas, long long total) {
    return attend_div(c * total, ctas);
}
__host__ __device__ inline int attend_owner(long long t, long long ctas, long long total) {
    // The bounds hold by themselves; lengths that another stream changes meanwhile must not lead out of the slots.
    const long long c = t < 0 ? 0 : attend_div((t + 1) * ctas - 1, total);
    return static_cast<int>(c < ctas ? c : ctas - 1);
}

// Of more than kAttendOneLevel parts, about as many are joined at once as there
// are groups of them.  262143 positions, 8 key heads of 8: 161.8 us, 163.0 with 32
// at once; 7 contexts of 8192, 8 heads on one: 15.6, 17.1; 200000 e4m3 positions,
// 2 key heads: 32.1, 32.3; 2 contexts of 32768: 51.1, 51.8; 4096 positions alone:
// 13.5, 13.1.  (With this from 8 parts on, 1000 positions alone took 11.6
// instead of 10.5.)
__host__ __device__ inline int attend_fan(int parts) {
    int fan = 1;
    while (fan * fan < parts) ++fan;
    return fan;
}

// The slot of run c's part of an item whose first part is run `first`'s, for the
// run's CTA `lane` of `lanes`: a CTA has at most one part that it begins and one
// that it continues.
__host__ __device__ inline int attend_slot(int c, int first, int lane, int lanes) {
    return 2 * (c * lanes + lane) + (c == first ? 1 : 0);
}

__device__ __forceinline__ void cursor_load(AttendCursor &u, const AttendParams &p, int tile, int pad) {
    bool bad = false;
    u.n = kv_length(p.table.lengths[u.b], p.table.width, p.cache.page_size, &bad);
    u.tiles = attend_tiles(u.n, p.window, tile, pad, &u.lo);
}

// To the next item; true when that is another sequence's (whose n, lo and tiles
// are still to be set).
__device__ __forceinline__ bool cursor_item(AttendCursor &u, const AttendParams &p) {
    u.tile = 0;
    if (p.lanes == 1) {
        if (++u.block < p.blocks) return false;
        u.block = 0;
        if (++u.head < p.cache.heads) return false;
        u.head = 0;
    }
    if (u.b + 1 >= p.table.batch) return false;
    ++u.b;
    return true;
}

__device__ __forceinline__ void cursor_next(AttendCursor &u, const AttendParams &p, int tile, int pad) {
    if (++u.tile < u.tiles) return;
    if (cursor_item(u, p)) cursor_load(u, p, tile, pad);
}

// A block's run, found by its first warp or by all: every warp goes by the same
// numbers, also by the same lengths, so that all meet at the same barriers
// whatever another stream does to the lengths meanwhile.
struct AttendRun {
    long long all, first, last;
    int ctas, pad, b, h, tile, n;
};

template <bool kBf16, bool kE4m3, int DP, int NT>
__global__ void __launch_bounds__(AttendShape<kE4m3, DP, NT>::kThreads, AttendShape<kE4m3, DP, NT>::kCtas)
    kv_attend_kernel(const AttendParams p) {
    using S = AttendShape<kE4m3, DP, NT>;
    constexpr bool kMmaBf16 = kBf16 && !kE4m3;      // e4m3 is widened to fp16
    constexpr float kBelow = kBf16 || kE4m3 ? 0.0f : kAttendBelow;
    constexpr int kChunks = S::kRow / 16;           // 16-byte pieces of a row
    constexpr int kRowsPerCopy = 32 / kChunks;      // rows that a warp's copy instruction covers
    constexpr int kBlocks = S::kKeys / 16;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long s_sum[S::kWarps];
    __shared__ AttendRun s_run;
    __shared__ int s_next;                          // length of the sequence after the one at hand
    __shared__ float s_m[S::kWarps][S::kHeads], s_l[S::kWarps][S::kHeads];
    __shared__ float s_w[kAttendFanIn][S::kHeads];
    __shared__ float s_inv[S::kHeads], s_ref[S::kHeads];
    __shared__ unsigned s_last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    float *merge = reinterpret_cast<float *>(smem + S::kMerge);
    const uint32_t ring = smem_u32(smem) + warp * S::kStages * S::kStage;
    unsigned char *const sides = smem + S::kSides + warp * S::kStages * S::kSide;
    long long *const offsets = reinterpret_cast<long long *>(smem + S::kOffsets) + warp * S::kKeys;
    griddep_wait();
    griddep_launch_dependents();

    // ---- this CTA's run, from all lengths
    const int heads_all = p.lanes > 1 ? 1 : p.cache.heads * p.blocks;    // that a run goes through
    const int runs = static_cast<int>(gridDim.x) / p.lanes, lane_cta = static_cast<int>(blockIdx.x) % p.lanes;
    const int cta = static_cast<int>(blockIdx.x) / p.lanes;
    if (p.table.batch <= 32) {
        // One sequence a lane of the first warp.
        if (warp == 0) {
            bool bad = false;
            int lo, n = 0, tiles = 0;
            if (lane < p.table.batch) {
                n = kv_length(p.table.lengths[lane], p.table.width, p.cache.page_size, &bad);
                if (bad && blockIdx.x == 0) record_status(p.status, kStatusCache);
                tiles = attend_tiles(n, p.window, S::kTile, 1, &lo);
            }
            AttendRun r;
            int length = 0;
            if (static_cast<long long>(p.table.batch) * heads_all <= runs) {
                long long units[kAttendLengths];
#pragma unroll
                for (int k = 0; k < kAttendLengths; ++k)
                    units[k] = static_cast<long long>(__reduce_add_sync(0xffffffffu, (tiles + attend_length(k) - 1) / attend_length(k))) * heads_all;
                length = attend_pad(units, static_cast<long long>(__reduce_add_sync(0xffffffffu, tiles)) * heads_all, runs);
            }
            r.pad = max(length, 1);
            tiles = (tiles + r.pad - 1) / r.pad * r.pad;
            const int upto = warp_scan(tiles);
            r.all = static_cast<long long>(__shfl_sync(0xffffffffu, upto, 31)) * heads_all;
            r.ctas = static_cast<int>(length > 0 ? attend_div(r.all, length) : min(static_cast<long long>(runs), r.all));
            const int c = min(cta, r.ctas - 1);
            r.first = attend_first(c, r.ctas, r.all);
            r.last = attend_first(c + 1, r.ctas, r.all);
            const long long at = static_cast<long long>(upto - tiles) * heads_all;
            const unsigned found = __ballot_sync(0xffffffffu, r.first >= at && r.first < at + static_cast<long long>(tiles) * heads_all);
            r.b = max(__ffs(found) - 1, 0);
            const int its = __shfl_sync(0xffffffffu, tiles, r.b);
            const long long in = r.first - static_cast<long long>(__shfl_sync(0xffffffffu, upto, r.b) - its) * heads_all;
            r.h = static_cast<int>(attend_div(in, its));
            r.tile = static_cast<int>(in - static_cast<long long>(r.h) * its);
            r.n = __shfl_sync(0xffffffffu, n, r.b);
            if (lane == 0) s_run = r;
        }
    } else {
        const int each = (p.table.batch + S::kThreads - 1) / S::kThreads;
        const int b_lo = min(p.table.batch, static_cast<int>(threadIdx.x) * each), b_hi = min(p.table.batch, b_lo + each);
        bool bad = false;
        int lo;
        long long mine = 0;
        for (int b = b_lo; b < b_hi; ++b)
            mine += attend_tiles(kv_length(p.table.lengths[b], p.table.width, p.cache.page_size, &bad), p.window, S::kTile, 1, &lo);
        if (bad && blockIdx.x == 0) record_status(p.status, kStatusCache);
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
        }
        if (lane == 31) s_sum[warp] = upto;
        __syncthreads();
        AttendRun r;
        r.all = 0;
#pragma unroll
        for (int w = 0; w < S::kWarps; ++w) {
            if (w < warp) upto += s_sum[w];
            r.all += s_sum[w];
        }
        r.all *= heads_all;
        r.pad = 1;
        r.ctas = static_cast<int>(min(static_cast<long long>(runs), r.all));
        const int c = min(cta, r.ctas - 1);
        r.first = attend_first(c, r.ctas, r.all);
        r.last = attend_first(c + 1, r.ctas, r.all);
        r.b = r.h = r.tile = r.n = 0;
        if (threadIdx.x == 0) s_run = r;
        __syncthreads();
        long long at = (upto - mine) * heads_all;
        if (r.first >= at && r.first < upto * heads_all)
            for (int b = b_lo; b < b_hi; ++b) {
                const int n = kv_length(p.table.lengths[b], p.table.width, p.cache.page_size, &bad);
                const int tiles = attend_tiles(n, p.window, S::kTile, 1, &lo);
                if (r.first < at + static_cast<long long>(tiles) * heads_all) {
                    const long long in = r.first - at;
                    s_run.b = b;
                    s_run.h = static_cast<int>(attend_div(in, tiles));
                    s_run.tile = static_cast<int>(in - static_cast<long long>(s_run.h) * tiles);
                    s_run.n = n;
                    break;
                }
                at += static_cast<long long>(tiles) * heads_all;
            }
    }
    __syncthreads();
    const int ctas = s_run.ctas, pad = s_run.pad;
    if (cta >= ctas) return;
    const long long all = s_run.all, first = s_run.first;
    const int steps = static_cast<int>(s_run.last - first);

    // ---- loading: the places of the next step's rows are looked up, then copied
    AttendCursor load;
    load.b = s_run.b;
    const int h_first = min(p.lanes > 1 ? lane_cta : s_run.h, p.cache.heads * p.blocks - 1);
    load.head = h_first / p.blocks;
    load.block = h_first - load.head * p.blocks;
    load.tile = s_run.tile;
    load.n = s_run.n;
    load.tiles = attend_tiles(load.n, p.window, S::kTile, pad, &load.lo);
    AttendCursor use = load;
    int page = -1, slot = 0, load_head = 0;    // lane i: of the step's position i
    unsigned want = 0;                         // positions that there are
    int looked = 0;
    auto lookup = [&]() {
        load_head = load.head;
        const int pos = load.lo + load.tile * S::kTile + warp * S::kKeys + lane;
        const bool in = lane < S::kKeys && pos < load.n && looked < steps;
        int i = 0;
        if (in)
            i = p.page_shift >= 0 ? pos >> p.page_shift
                                  : static_cast<int>(static_cast<unsigned>(pos) / static_cast<unsigned>(p.cache.page_size));
        slot = pos - i * p.cache.page_size;
        page = in ? p.table.pages[load.b * p.table.stride + i] : -1;
        want = __ballot_sync(0xffffffffu, in);
        if (++looked < steps) cursor_next(load, p, S::kTile, pad);
    };
    // A lane copies piece `piece` of rows in_copy, in_copy + kRowsPerCopy, ...; the pieces of a row are
    // exchanged by its low bits (xor), so that ldmatrix finds eight rows in different banks.
    const int piece = lane % kChunks, in_copy = lane / kChunks;
    const bool inside = piece * 16 < p.cache.row_bytes, whole_row = p.cache.row_bytes == S::kRow;     // past dim: zeros
    const unsigned char *const kpool = p.cache.k + (inside ? piece * 16 : 0);
    const unsigned char *const vpool = p.cache.v + (inside ? piece * 16 : 0);
    auto swizzle = [](int row) { return kChunks >= 8 ? (row & 7) : ((row >> 1) & (kChunks - 1)); };
    const uint32_t copy_to = in_copy * S::kRow + ((piece ^ swizzle(in_copy)) << 4);
    constexpr unsigned kAll = S::kKeys == 32 ? 0xffffffffu : (1u << (S::kKeys & 31)) - 1u;
    // Starts the copies of the rows that lookup() found.
    auto issue = [&](int stage, int page, int slot, unsigned want, int load_head) {
        const uint32_t dst = ring + stage * S::kStage;
        unsigned char *const side = sides + stage * S::kSide;
        const bool in = page >= 0 && page < p.cache.pages;
        const unsigned ok = __ballot_sync(0xffffffffu, in);
        if (ok != want && lane == 0) record_status(p.status, kStatusCache);
        if (lane < S::kKeys) {
            offsets[lane] = in ? kv_offset(p.cache, page, slot, load_head) : -1;
            if (kE4m3) {
                const long long so = in ? kv_scale_offset(p.cache, page, slot, load_head) : 0;
                cp_async4(smem_u32(side) + 16 + 4 * lane, p.cache.k_scale + so, in);
                cp_async4(smem_u32(side) + 16 + 4 * (S::kKeys + lane), p.cache.v_scale + so, in);
            }
        }
        if (lane == 0) *reinterpret_cast<unsigned *>(side) = ok;
        __syncwarp();
        if (want) {
            // swizzle(row) of row i * kRowsPerCopy + in_copy is swizzle(in_copy) ^ swizzle(i * kRowsPerCopy)
            if (ok == kAll && whole_row) {
#pragma unroll
                for (int i = 0; i < S::kKeys / kRowsPerCopy; ++i) {
                    const long long o = offsets[i * kRowsPerCopy + in_copy];
                    const uint32_t to = dst + i * kRowsPerCopy * S::kRow + (copy_to ^ (swizzle(i * kRowsPerCopy) << 4));
                    cp_async16(to, kpool + o);
                    cp_async16(to + S::kKeys * S::kRow, vpool + o);
                }
            } else {
#pragma unroll
                for (int i = 0; i < S::kKeys / kRowsPerCopy; ++i) {
                    const long long o = offsets[i * kRowsPerCopy + in_copy];
                    const uint32_t to = dst + i * kRowsPerCopy * S::kRow + (copy_to ^ (swizzle(i * kRowsPerCopy) << 4));
                    const bool good = inside && o >= 0;
                    cp_async16(to, kpool + (good ? o : 0), good);
                    cp_async16(to + S::kKeys * S::kRow, vpool + (good ? o : 0), good);
                }
            }
        }
        cp_async_commit();
    };

    {
        // The first two steps' pages are requested together.
        lookup();
        const int page0 = page, slot0 = slot, head0 = load_head;
        const unsigned want0 = want;
        lookup();
        issue(0, page0, slot0, want0, head0);
#pragma unroll
        for (int s = 1; s < S::kStages - 1; ++s) {
            __syncwarp();
            issue(s, page, slot, want, load_head);
            lookup();
        }
    }

    // ---- the item at hand
    uint32_t qf[NT][DP / 16][2];
    float qscale[NT][2];                   // to log2 units, for heads 2 t4 and 2 t4 + 1
    float o[NT][DP / 16][4], m[NT][2], l[NT][2];
    float mu[NT][2];                       // e4m3: the outputs' own reference
    int begun = use.tile;                  // first tile of this CTA's part
    // The item's queries are requested (request_q) as soon as the previous item's last product is done,
    // and made ready (begin) after it is joined.
    auto request_q = [&](const AttendCursor &u) {
        const int h0 = u.block * S::kHeads, hn = min(S::kHeads, p.group - h0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const bool is = 8 * nt + g < hn;
            const unsigned char *row = p.q + u.b * p.q_batch_stride +
                                       (static_cast<long long>(u.head) * p.group + h0 + (is ? 8 * nt + g : 0)) * p.q_head_stride;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int d = kE4m3 ? 16 * kk + 4 * t4 + 2 * i : 16 * kk + 2 * t4 + 8 * i;
                    qf[nt][kk][i] = is && d < p.cache.dim ? *reinterpret_cast<const uint32_t *>(row + 2 * d) : 0u;
                }
        }
    };
    auto begin = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float unit = 1.0f;
            if (kE4m3 && kBf16) {
                // Largest element to [2^14, 2^15): fp16 then keeps bf16's eight bits down to 2^-29 of it.
                float top = 0.0f;
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t x = qf[nt][kk][i];
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x << 16)), fabsf(__uint_as_float(x & 0xFFFF0000u))));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;      // -127 for zero
                const int shift = min(max(14 - e, -126), 126);
                const float up = __uint_as_float(static_cast<uint32_t>(shift + 127) << 23);
                unit = __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t x = qf[nt][kk][i];
                        qf[nt][kk][i] = pair16<false>(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xFFFF0000u) * up);
                    }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                qscale[nt][i] = p.first * __shfl_sync(0xffffffffu, unit, (2 * t4 + i) * 4);
                m[nt][i] = mu[nt][i] = -INFINITY;
                l[nt][i] = 0.0f;
            }
#pragma unroll
            for (int mt = 0; mt < DP / 16; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][mt][i] = 0.0f;
        }
    };
    request_q(use);
    begin();
    // The first thread has the next sequence's length for all warps.
    auto next_length = [&]() {
        bool bad = false;
        return kv_length(p.table.lengths[min(use.b + 1, p.table.batch - 1)], p.table.width, p.cache.page_size, &bad);
    };
    int next = threadIdx.x == 0 ? next_length() : 0;
    int stage = 0;
    for (int step = 0; step < steps; ++step) {
        const int head = use.head, h0 = use.block * S::kHeads, hn = min(S::kHeads, p.group - h0);    // the block's heads
        cp_async_wait<S::kStages - 2>();
        __syncwarp();
        // the stage that the previous step has read takes the step that comes kStages - 1 after this one
        issue(stage == 0 ? S::kStages - 1 : stage - 1, page, slot, want, load_head);
        lookup();
        const uint32_t src = ring + stage * S::kStage;
        const unsigned char *const side = sides + stage * S::kSide;
        const unsigned mask = *reinterpret_cast<const unsigned *>(side);
        if (mask) {
            // S^T = K Q^T.  16-bit: matrices (rows 0-7 | 8-15) x (pieces 2c | 2c + 1), one k step; e4m3: the
            // same bytes are two.  A lone block's k steps go to two accumulators in turn: half the chain.
            constexpr int kChains = NT * kBlocks == 1 ? 2 : 1;
            float s[NT][kBlocks][4];
            const int krow = (lane & 7) + ((lane >> 3) & 1) * 8;
            const uint32_t ka = src + krow * S::kRow, kx = ((lane >> 4) ^ swizzle(krow)) << 4;
#pragma unroll
            for (int kb = 0; kb < kBlocks; ++kb) {
                float acc[kChains][NT][4] = {};
#pragma unroll
                for (int c = 0; c < kChunks / 2; ++c) {
                    uint32_t a[4];
                    ldmatrix4(a, ka + (kx ^ (c << 5)) + kb * 16 * S::kRow);
                    if (!kE4m3) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<kMmaBf16>(acc[c % kChains][nt], a, qf[nt][c][0], qf[nt][c][1]);
                    } else {
                        // a[0] / a[1]: rows g / g + 8 of dims 32 c + 4 t4 .. + 3; a[2] / a[3]: of the next 16 dims
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t w[4];
                            widen4(a[2 * i], w[0], w[2]);
                            widen4(a[2 * i + 1], w[1], w[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<false>(acc[i % kChains][nt], w, qf[nt][2 * c + i][0], qf[nt][2 * c + i][1]);
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[nt][kb][i] = kChains == 2 ? acc[0][nt][i] + acc[kChains - 1][nt][i] : acc[0][nt][i];
            }
            // scores in log2 units; the value scales
            float ve[kBlocks][2], vf[kBlocks][2];
            const float *scales = reinterpret_cast<const float *>(side + 16);
#pragma unroll
            for (int kb = 0; kb < kBlocks; ++kb)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float ks = 1.0f;
                    if (kE4m3) {                 // (rows left out have scales of 0)
                        ks = scales[16 * kb + g + 8 * r];
                        split_scale(scales[S::kKeys + 16 * kb + g + 8 * r], ve[kb][r], vf[kb][r]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float &x = s[nt][kb][2 * r + i];
                            x *= kE4m3 ? qscale[nt][i] * ks : qscale[nt][i];
                            if (p.capped) x = p.last * tanhf(x);
                        }
                }
            if (p.space.scores) {
                float *const scores = p.space.scores +
                                      ((static_cast<long long>(use.b) * p.cache.heads + head) * p.positions + use.lo +
                                       use.tile * S::kTile + warp * S::kKeys) * p.scored + h0 + 2 * t4;
                const int room = static_cast<int>(min(attend_scored(use.lo, use.tile, S::kTile, warp * S::kKeys, p.positions),
                                                      static_cast<long long>(S::kKeys)));
#pragma unroll
                for (int kb = 0; kb < kBlocks; ++kb)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int row = 16 * kb + g + 8 * r;
                            if (((mask >> row) & 1u) && row < room && 8 * nt + 2 * t4 < hn &&
                                TGEMM_CHECK(scores - p.space.scores + row * p.scored + 8 * nt + 2 <= p.dbg_scores, kChkKvSpace, p.status))
                                *reinterpret_cast<float2 *>(scores + row * p.scored + 8 * nt) =
                                    make_float2(s[nt][kb][2 * r], s[nt][kb][2 * r + 1]);
                        }
            }
            if (mask != kAll) {
#pragma unroll
                for (int kb = 0; kb < kBlocks; ++kb)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (!((mask >> (16 * kb + g + 8 * r)) & 1u)) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) s[nt][kb][2 * r] = s[nt][kb][2 * r + 1] = -INFINITY;
                        }
            }
            // a reference moves when some score exceeds the maximum that set it by more than 2^kAttendGrow
            bool grow = false;
            float top[NT][2], top_u[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = -INFINITY, u = -INFINITY;
#pragma unroll
                    for (int kb = 0; kb < kBlocks; ++kb) {
                        x = fmaxf(x, fmaxf(s[nt][kb][i], s[nt][kb][2 + i]));
                        if (kE4m3) u = fmaxf(u, fmaxf(s[nt][kb][i] + ve[kb][0], s[nt][kb][2 + i] + ve[kb][1]));
                    }
                    top[nt][i] = x;
                    top_u[nt][i] = u;
                    grow |= x > m[nt][i] + (kAttendGrow + kBelow);
                    if (kE4m3) grow |= u > mu[nt][i] + (kAttendGrow + kAttendScaledBelow);
                }
            if (__any_sync(0xffffffffu, grow)) {
                if constexpr (kE4m3) {
                    // A row of zeros (kv_append gives it a scale of 1) adds nothing whatever its weight, so it sets no
                    // reference: it counts as one with a scale of 0.  Its four lanes look at a quarter each.
#pragma unroll
                    for (int kb = 0; kb < kBlocks; ++kb)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const uint32_t at = src + (S::kKeys + 16 * kb + g + 8 * r) * S::kRow + t4 * (S::kRow / 4);
                            uint32_t any = 0;
#pragma unroll
                            for (int c = 0; c < S::kRow / 64; ++c) any |= lds_or(at + 16 * c);
                            any |= __shfl_xor_sync(0xffffffffu, any, 1);
                            any |= __shfl_xor_sync(0xffffffffu, any, 2);
                            if ((any & 0x7F7F7F7Fu) == 0u) ve[kb][r] = -INFINITY;
                        }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float u = -INFINITY;
#pragma unroll
                            for (int kb = 0; kb < kBlocks; ++kb)
                                u = fmaxf(u, fmaxf(s[nt][kb][i] + ve[kb][0], s[nt][kb][2 + i] + ve[kb][1]));
                            top_u[nt][i] = u;
                        }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float a[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = top[nt][i], u = top_u[nt][i];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                            if (kE4m3) u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, d));
                        }
                        const float next = fmaxf(m[nt][i], x - kBelow);
                        a[i] = next == -INFINITY ? 1.0f : exp2_fast(m[nt][i] - next);
                        m[nt][i] = next;
                        l[nt][i] *= a[i];
                        if (kE4m3) {
                            const float next_u = fmaxf(mu[nt][i], u - kAttendScaledBelow);
                            a[i] = next_u == -INFINITY ? 1.0f : exp2_fast(mu[nt][i] - next_u);
                            mu[nt][i] = next_u;
                        }
                    }
#pragma unroll
                    for (int mt = 0; mt < DP / 16; ++mt) {
                        o[nt][mt][0] *= a[0];
                        o[nt][mt][1] *= a[1];
                        o[nt][mt][2] *= a[0];
                        o[nt][mt][3] *= a[1];
                    }
                }
            }
            // weights, their sum, and O^T += V^T P^T
            float ref[NT][2], ref_u[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ref[nt][i] = m[nt][i] == -INFINITY ? 0.0f : m[nt][i];
                    ref_u[nt][i] = mu[nt][i] == -INFINITY ? 0.0f : mu[nt][i];
                }
#pragma unroll
            for (int kb = 0; kb < kBlocks; ++kb) {
                uint32_t pf[NT][2], pr[NT][2];           // high parts, and the rest
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float w[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float t = s[nt][kb][2 * r + i];
                            w[i] = exp2_fast(t - ref[nt][i]);
                            l[nt][i] += w[i];
                            if (kE4m3) w[i] = exp2_fast((t + ve[kb][r]) - ref_u[nt][i]) * vf[kb][r];
                        }
                        uint32_t high, rest;
                        split16<kMmaBf16>(w[0], w[1], high, rest);
                        pf[nt][r] = movmatrix_trans(high);
                        pr[nt][r] = movmatrix_trans(rest);
                    }
                }
                if (!kE4m3) {
                    // matrices: (positions 0-7 | 8-15: bit 4 of the lane) x (dims 0-7 | 8-15: bit 3)
                    const int row = (lane & 7) + (lane >> 4) * 8;
                    const uint32_t va = src + (S::kKeys + 16 * kb + row) * S::kRow, vx = (((lane >> 3) & 1) ^ swizzle(row)) << 4;
#pragma unroll
                    for (int mt = 0; mt < DP / 16; mt += 2) {
                        uint32_t a[4], b[4];
                        ldmatrix4_trans(a, va + (vx ^ (mt << 5)));
                        ldmatrix4_trans(b, va + (vx ^ ((mt + 1) << 5)));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816<kMmaBf16>(o[nt][mt], a, pf[nt][0], pf[nt][1]);
                            mma16816<kMmaBf16>(o[nt][mt + 1], b, pf[nt][0], pf[nt][1]);
                            mma16816<kMmaBf16>(o[nt][mt], a, pr[nt][0], pr[nt][1]);
                            mma16816<kMmaBf16>(o[nt][mt + 1], b, pr[nt][0], pr[nt][1]);
                        }
                    }
                } else {
                    // matrices of byte pairs: (positions 0-7 | 8-15: bit 3) x (dims 0-15 | 16-31: bit 4); a
                    // register holds two positions of dims 2 g and 2 g + 1, which become rows g and g + 8
                    const int row = (lane & 7) + ((lane >> 3) & 1) * 8;
                    const uint32_t va = src + (S::kKeys + 16 * kb + row) * S::kRow, vx = ((lane >> 4) ^ swizzle(row)) << 4;
#pragma unroll
                    for (int c = 0; c < DP / 32; ++c) {
                        uint32_t a[4];
                        ldmatrix4_trans(a, va + (vx ^ (c << 5)));
                        uint32_t w[2][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            widen4(__byte_perm(a[2 * i], 0, 0x3120), w[i][0], w[i][1]);
                            widen4(__byte_perm(a[2 * i + 1], 0, 0x3120), w[i][2], w[i][3]);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma16816<false>(o[nt][2 * c + (i & 1)], w[i & 1], i < 2 ? pf[nt][0] : pr[nt][0],
                                                i < 2 ? pf[nt][1] : pr[nt][1]);
                    }
                }
            }
        }
        stage = stage + 1 == S::kStages ? 0 : stage + 1;

        const bool ends = use.tile + 1 == use.tiles, more = step + 1 < steps;
        if (!ends && more) {
            ++use.tile;
            continue;
        }
        {
            const int b = use.b;
            const long long item = first + step - use.tile;      // the item's first tile among all
            const long long item_end = item + use.tiles;
            const bool whole = begun == 0 && ends;
            bool other = false;                                  // the next item is another sequence's
            if (more) {
                other = cursor_item(use, p);
                request_q(use);
                begun = 0;
            }
            if (threadIdx.x == 0) s_next = next;
            // ---- join the warps: one reference, then the outputs one warp after the other
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], d);
                    if (g == 0) {
                        s_m[warp][8 * nt + 2 * t4 + i] = m[nt][i];
                        s_l[warp][8 * nt + 2 * t4 + i] = l[nt][i];
                    }
                }
            __syncthreads();
            if (other) {
                use.n = s_next;
                use.tiles = attend_tiles(use.n, p.window, S::kTile, pad, &use.lo);
                if (threadIdx.x == 0) next = next_length();
            }
            float a[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int h = 8 * nt + 2 * t4 + i;
                    float ref = s_m[0][h], sum = 0.0f;
#pragma unroll
                    for (int w = 1; w < S::kWarps; ++w) ref = fmaxf(ref, s_m[w][h]);
                    const float base = ref == -INFINITY ? 0.0f : ref;
#pragma unroll
                    for (int w = 0; w < S::kWarps; ++w) sum += s_l[w][h] * exp2_fast(s_m[w][h] - base);
                    // (e4m3: the root of the factor, which fp32 holds whatever the scales are)
                    a[nt][i] = kE4m3 ? exp2_fast(0.5f * (mu[nt][i] - base)) : exp2_fast(m[nt][i] - base);
                    if (warp == 0 && g == 0) {
                        s_ref[h] = ref;
                        s_inv[h] = sum;
                    }
                }
            // Each round every warp adds a part of the dims of its own, so that all work at once and every part
            // meets the warps in a fixed order.
#pragma unroll 1
            for (int round = 0; round < S::kWarps; ++round) {
                const int part = warp + round < S::kWarps ? warp + round : warp + round - S::kWarps;
#pragma unroll
                for (int mt = 0; mt < DP / 16; ++mt) {
                    if (mt * S::kWarps / (DP / 16) == part) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int d = 16 * mt + (kE4m3 ? 2 * g + (i >> 1) : g + 8 * (i >> 1));
                                float *at = merge + (8 * nt + 2 * t4 + (i & 1)) * S::kPitch + d;
                                float x = o[nt][mt][i] * a[nt][i & 1];
                                if (kE4m3) x *= a[nt][i & 1];
                                *at = round == 0 ? x : *at + x;
                            }
                    }
                }
                __syncthreads();
            }
            // ---- whole: the answer; a part: to the workspace, and the last to arrive joins
            bool answer = whole;
            if (!whole) {
                const int c0 = attend_owner(item, ctas, all), c1 = attend_owner(item_end - 1, ctas, all);
                const int parts = max(c1 - c0 + 1, 1), mine_at = min(max(cta - c0, 0), parts - 1);
                int fan = kAttendFanIn, group = 0, groups = 1;
                if (parts > kAttendOneLevel) {
                    fan = attend_fan(parts);
                    group = mine_at / fan;
                    groups = (parts + fan - 1) / fan;
                }
                auto slot_of = [&](int part) { return attend_slot(c0 + part, c0, lane_cta, p.lanes); };
                auto put = [&](int to) {
                    if (!TGEMM_CHECK(to >= 0 && to < 2 * kAttendMaxCtas, kChkKvSpace, p.status)) return;
                    float *dst = p.space.out + static_cast<long long>(to) * S::kHeads * DP;
                    for (int i = threadIdx.x; i < hn * DP / 4; i += S::kThreads) {
                        const int h = i / (DP / 4), d = i % (DP / 4) * 4;
                        __stcg(reinterpret_cast<float4 *>(dst) + i, *reinterpret_cast<const float4 *>(merge + h * S::kPitch + d));
                    }
                    if (threadIdx.x < S::kHeads)
                        __stcg(p.space.ml + to * S::kHeads + threadIdx.x, make_float2(s_ref[threadIdx.x], s_inv[threadIdx.x]));
                };
                // Whether this CTA is the last of `n` to count at `counter` (which then is 0 again).
                auto arrive = [&](unsigned *counter, int n) {
                    __syncthreads();
                    if (threadIdx.x == 0) s_last = count_acq_rel(counter, static_cast<unsigned>(n - 1)) == static_cast<unsigned>(n - 1);
                    __syncthreads();
                    return s_last != 0u;
                };
                // Joins `n` parts (the first at part0, `stride` apart) into merge, s_ref and s_inv.
                auto join = [&](int part0, int stride, int n) {
                    for (int i = threadIdx.x; i < n * S::kHeads; i += S::kThreads) {
                        const int e = i / S::kHeads, h = i % S::kHeads;
                        const float2 ml = __ldcg(p.space.ml + slot_of(part0 + e * stride) * S::kHeads + h);
                        s_w[e][h] = ml.x;
                        merge[i] = ml.y;
                    }
                    __syncthreads();
                    if (threadIdx.x < S::kHeads) {
                        const int h = threadIdx.x;
                        float ref = -INFINITY, sum = 0.0f;
                        for (int e = 0; e < n; ++e) ref = fmaxf(ref, s_w[e][h]);
                        const float base = ref == -INFINITY ? 0.0f : ref;
                        for (int e = 0; e < n; ++e) {
                            const float w = exp2_fast(s_w[e][h] - base);
                            s_w[e][h] = w;
                            sum += w * merge[e * S::kHeads + h];
                        }
                        s_ref[h] = ref;
                        s_inv[h] = sum;
                    }
                    __syncthreads();
                    if (n <= kAttendDirect) {
                        // Few parts: a thread's outputs one after the other, all parts requested together.
#pragma unroll 1
                        for (int i = threadIdx.x; i < hn * DP / 4; i += S::kThreads) {
                            const int h = i / (DP / 4);
                            float4 x[kAttendDirect], sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                            for (int e = 0; e < kAttendDirect; ++e)
                                x[e] = e < n ? __ldcg(reinterpret_cast<const float4 *>(p.space.out) +
                                                      static_cast<long long>(slot_of(part0 + e * stride)) * (S::kHeads * DP / 4) + i)
                                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                            for (int e = 0; e < kAttendDirect; ++e) {
                                if (e >= n) break;
                                const float w = s_w[e][h];
                                sum.x += w * x[e].x;
                                sum.y += w * x[e].y;
                                sum.z += w * x[e].z;
                                sum.w += w * x[e].w;
                            }
                            *reinterpret_cast<float4 *>(merge + h * S::kPitch + i % (DP / 4) * 4) = sum;
                        }
                        __syncthreads();
                        return;
                    }
                    // Each warp sums every kWarps-th part, two parts' loads in flight, then the warps' sums are
                    // added in a fixed order as above; up to eight float4s of a lane at a time (a divisor of all:
                    // merge ends with the last).
                    constexpr int kAllOfLane = S::kHeads * DP / 4 / 32;
                    constexpr int kEach = kAllOfLane < 8 ? kAllOfLane : kAllOfLane % 8 == 0 ? 8 : 6;
                    static_assert(kAllOfLane * 128 == S::kHeads * DP && kAllOfLane % kEach == 0, "whole turns");
#pragma unroll 1
                    for (int c0 = 0; c0 < kAllOfLane && c0 * 128 < hn * DP; c0 += kEach) {
                        float4 sum[kEach] = {};
#pragma unroll 1
                        for (int e = warp; e < n; e += 2 * S::kWarps) {
                            const int e2 = e + S::kWarps < n ? e + S::kWarps : e;
                            const float4 *const from = reinterpret_cast<const float4 *>(p.space.out) + c0 * 32 + lane;
                            const float4 *const a = from + static_cast<long long>(slot_of(part0 + e * stride)) * (S::kHeads * DP / 4);
                            const float4 *const b = from + static_cast<long long>(slot_of(part0 + e2 * stride)) * (S::kHeads * DP / 4);
                            float4 x[kEach], y[kEach];
#pragma unroll
                            for (int c = 0; c < kEach; ++c) x[c] = __ldcg(a + c * 32);
#pragma unroll
                            for (int c = 0; c < kEach; ++c) y[c] = __ldcg(b + c * 32);
#pragma unroll
                            for (int c = 0; c < kEach; ++c) {
                                const int h = ((c0 + c) * 32 + lane) / (DP / 4);
                                const float w = s_w[e][h];
                                sum[c].x += w * x[c].x;
                                sum[c].y += w * x[c].y;
                                sum[c].z += w * x[c].z;
                                sum[c].w += w * x[c].w;
                            }
                            if (e2 == e) break;
#pragma unroll
                            for (int c = 0; c < kEach; ++c) {
                                const int h = ((c0 + c) * 32 + lane) / (DP / 4);
                                const float w = s_w[e2][h];
                                sum[c].x += w * y[c].x;
                                sum[c].y += w * y[c].y;
                                sum[c].z += w * y[c].z;
                                sum[c].w += w * y[c].w;
                            }
                        }
#pragma unroll 1
                        for (int round = 0; round < S::kWarps; ++round) {
                            const int part = warp + round < S::kWarps ? warp + round : warp + round - S::kWarps;
#pragma unroll
                            for (int c = 0; c < kEach; ++c)
                                if (c * S::kWarps / kEach == part) {
                                    const int i = (c0 + c) * 32 + lane;
                                    float4 *const at = reinterpret_cast<float4 *>(merge + i / (DP / 4) * S::kPitch + i % (DP / 4) * 4);
                                    float4 v = sum[c];
                                    if (round > 0) {
                                        const float4 old = *at;
                                        v.x += old.x;
                                        v.y += old.y;
                                        v.z += old.z;
                                        v.w += old.w;
                                    }
                                    *at = v;
                                }
                            if (round + 1 < S::kWarps) __syncthreads();
                        }
                    }
                    __syncthreads();
                };
                put(slot_of(mine_at));
                const int part0 = group * fan, count = min(fan, parts - part0);
                bool here = arrive(p.space.parts + slot_of(part0), count);
                if (here) {
                    join(part0, 1, count);
                    if (groups > 1) {
                        put(slot_of(part0));
                        here = arrive(p.space.groups + slot_of(0), groups);
                        if (here) join(0, fan, groups);
                    }
                }
                answer = here;
            }
            if (answer) {
                const int h_all = p.cache.heads * p.group;
                if (threadIdx.x < hn && p.space.scores)
                    p.space.stats[static_cast<long long>(b) * h_all + head * p.group + h0 + threadIdx.x] =
                        make_float2(s_ref[threadIdx.x], s_inv[threadIdx.x]);
                for (int i = threadIdx.x; i < hn * (DP / 8); i += S::kThreads) {
                    const int h = i / (DP / 8), d = i % (DP / 8) * 8;
                    if (d >= p.cache.dim) continue;
                    const float sum = s_inv[h];
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = sum == 0.0f ? 0.0f : merge[h * S::kPitch + d + e] / sum;
                    const uint4 v = make_uint4(pair16<kBf16>(x[0], x[1]), pair16<kBf16>(x[2], x[3]),
                                               pair16<kBf16>(x[4], x[5]), pair16<kBf16>(x[6], x[7]));
                    const long long at = b * p.o_batch_stride +
                                         (static_cast<long long>(head) * p.group + h0 + h) * p.o_head_stride + 2 * d;
                    if (TGEMM_CHECK(at >= 0 && at + 16 <= p.dbg_o_bytes, kChkKvOutput, p.status))
                        *reinterpret_cast<uint4 *>(p.o + at) = v;
                }
            }
            __syncthreads();               // merge and the statistics are free again
            if (more) begin();
        }
    }
    cp_async_wait<0>();
}

// weights[b, head, j] += sum over the group of 2^(t_j - m) / l.  A position's
// scores lie together; a thread adds for kSpreadEach positions, kSpreadThreads
// apart, whose first eight heads it requests together.
constexpr int kSpreadThreads = 128, kSpreadEach = 4;

__global__ void __launch_bounds__(kSpreadThreads) kv_spread_kernel(const AttendParams p) {
    constexpr int kPairs = 4;             // of heads, per request
    const int head = blockIdx.y, b = blockIdx.z;
    griddep_wait();
    bool bad = false;
    int n = kv_length(p.table.lengths[b], p.table.width, p.cache.page_size, &bad);
    int lo;
    attend_tiles(n, p.window, 1, 1, &lo);
    if (n > p.weights.width) {
        if (blockIdx.x == 0 && threadIdx.x == 0) record_status(p.status, kStatusCache);
        n = p.weights.width;
    }
    const int *list = p.table.pages + b * p.table.stride;
    float *w = p.weights.base + b * p.weights.batch_stride + head * p.weights.head_stride;
    const long long row0 = static_cast<long long>(b) * p.cache.heads + head;
    const float *const scores = p.space.scores + row0 * p.positions * p.scored;
    const float2 *const stats = p.space.stats + row0 * p.group;
    for (long long base = lo + static_cast<long long>(blockIdx.x) * kSpreadThreads * kSpreadEach; base < n;
         base += static_cast<long long>(gridDim.x) * kSpreadThreads * kSpreadEach) {
        int at[kSpreadEach];
        bool is[kSpreadEach];
        float old[kSpreadEach], sum[kSpreadEach];
#pragma unroll
        for (int e = 0; e < kSpreadEach; ++e) {
            const long long j = base + e * kSpreadThreads + threadIdx.x;
            is[e] = j < n;
            at[e] = is[e] ? static_cast<int>(j) : lo;
            old[e] = w[at[e]];
            sum[e] = 0.0f;
            int page, slot;
            is[e] = kv_row(list, at[e], p.cache.page_size, p.cache.pages, &page, &slot) && is[e];   // else it has no score
        }
        for (int h0 = 0; h0 < p.group; h0 += 2 * kPairs) {
            float2 t[kSpreadEach][kPairs], ml[2 * kPairs];
#pragma unroll
            for (int i = 0; i < 2 * kPairs; ++i) ml[i] = stats[min(h0 + i, p.group - 1)];
#pragma unroll
            for (int e = 0; e < kSpreadEach; ++e) {
                const float *const row = scores + static_cast<long long>(at[e]) * p.scored + h0;
                if (p.scored % 8 == 0) {
#pragma unroll
                    for (int i = 0; i < kPairs; i += 2) {
                        const float4 x = *reinterpret_cast<const float4 *>(row + 2 * i);
                        t[e][i] = make_float2(x.x, x.y);
                        t[e][i + 1] = make_float2(x.z, x.w);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kPairs; ++i)
                        t[e][i] = *reinterpret_cast<const float2 *>(row + min(2 * i, p.scored - 2 - h0));
                }
            }
#pragma unroll
            for (int i = 0; i < 2 * kPairs; ++i) {
                const float inv = h0 + i < p.group ? __fdividef(1.0f, ml[i].y) : 0.0f;
#pragma unroll
                for (int e = 0; e < kSpreadEach; ++e) {
                    const float x = i & 1 ? t[e][i / 2].y : t[e][i / 2].x;
                    sum[e] += h0 + i < p.group ? exp2_fast(x - ml[i].x) * inv : 0.0f;
                }
            }
        }
#pragma unroll
        for (int e = 0; e < kSpreadEach; ++e)
            if (is[e]) w[at[e]] = old[e] + sum[e];
    }
}

}  // namespace tgemm
