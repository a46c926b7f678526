// Attention of one new token per sequence over a paged bf16 key-value cache (sm_100a).
//
// Per sequence and query head: o = sum_j p_j v_j / sum_j p_j with
// p_j = 2^(x_j - m), x_j = (q . k_j) scale log2 e and m the largest x_j, in one
// pass over the keys with a running m, sum and o (rescaled when m grows).
//
// Bound: HBM.  Every key and value is read once and used for the query heads
// that share it, up to 16 of them (8 above 128 features), a handful of
// operations per byte; more heads read it once for each 16 (8 x 16384 keys of one
// head of 128: 16 query heads 31 us, 40 of them 47).  So:
//  * The work of a call, in units of 128 keys of one key-value head, is cut into
//    one equal contiguous range per CTA (whatever the lengths are; the end of a
//    head counts as half a unit where there are many), and a CTA
//    writes an unnormalised partial (m, sum, o) for a head whose keys it holds
//    only a part of; a second small launch joins those.  The cut depends only
//    on the lengths, so results repeat bit for bit.
//  * Each of a CTA's four warps takes 32 keys of a unit (16 at 256 features).  They
//    go through a ring of its own in shared memory (cp.async, two or three
//    pieces of 8 KB per warp in flight), so warps wait for nobody but
//    themselves.  Eight lanes copy 128 consecutive bytes: with each lane
//    copying just what it will use (32- and 64-byte runs), L2 delivered every
//    byte twice.
//  * Products on mma.sync m16n8k16 with 16 keys (or 16 features of the values)
//    as rows and 8 query heads as columns: S^T = K Q^T, then O^T += V^T P^T.
//    The contraction index may be permuted at will, so K's fragments are the 16
//    bytes a lane loaded, and V^T's are byte permutes of two rows' words.  S^T
//    becomes the P^T operand by an 8 x 8 transpose per warp (movmatrix).  p is
//    split into bf16 parts, one MMA each: with a single one its rounding alone
//    would be as large as that of a bf16 output.  For an fp32 output three parts
//    hold all its 24 bits; for bf16 two parts keep it within 2^-17, 1/256 of the
//    output's own rounding (the third costs 2 to 5% where heads are short, 300
//    sequences of up to 40 keys 28.7 against 29.8 us, and 6% with 16 query heads
//    per key-value head).
//  * The tensor core cuts its sums off: over a long chain of products that
//    loses up to 2^-23 of the sum each time, always towards zero (6.8e-6 of the
//    output at 3300 keys per warp).  So its accumulators hold the keys of one
//    step only, the smallest parts first, and the running sums are rounded fp32
//    additions (7.6e-8 there; no cost but 3 to 4% with 16 query heads per
//    key-value head).
//
// Measured on the device: 8 contexts of 65536 to 131072 keys, 20 heads on 5 of
// 128 features, 312 us (6.7 TB/s); 24 ragged sequences of up to 4096 keys x 32
// heads of 100, 100 us (5.6 TB/s); 128 sequences of up to 500 keys, 32 heads on
// 8, 34 us (4.2 TB/s: the ends of heads); one sequence of 4001 keys 9.7 us.
#include "common.cuh"
#include "kernels.h"

#include <atomic>
#include <limits>

namespace bitnet {

namespace {

constexpr int kWarps = 4;

struct AttnParams {
    const __nv_bfloat16 *q;
    int64_t ldq;
    const __nv_bfloat16 *k, *v;
    int64_t page_stride, head_stride, row_stride;
    const int32_t *pages;
    int64_t max_pages, n_pages;
    int page_shift;
    const int32_t *lens;
    int n_seqs, n_heads, group;       // group: query heads per key-value head
    int n_kv, vheads, vper, per_vhead;   // virtual key-value heads: vheads = n_kv x vper, each with up to per_vhead query heads
    int head_dim;
    float scale_log2;                 // scale log2 e, not zero
    float none;                       // the infinity that scale_log2 turns into minus infinity: a key that is left out
    void *o;
    int64_t ldo;
    int o_bf16;
    int o_vec;                        // four features of O at once: head_dim and ldo multiples of 4, O on their bytes
    float *lse;                       // or NULL
    float *part;                      // [grid, 2] partials
    uint32_t *status;
    int unit_shift;                   // log2 of the keys per unit
    int shift;                        // rows of the ring have a chunk to spare, and pages hold whole sectors (see the kernel)
    int q_vec;                        // bytes on which Q's rows and heads lie: 16, 8 or 2
    int grid;                         // CTAs of the first launch (those behind the number of units stay idle)
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// zeros where `in` is false (nothing is read then)
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
    return r;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the same without an accumulator before it
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A pair of weights as PARTS bf16 parts each, packed.  Cutting keeps the leading 8 bits and leaves an exact rest of 16, then
// of 8: three parts add up to all 24 bits of the weight.  Two parts, the second rounded, keep it within 2^-17.  A rest of
// zero becomes 2^-126, which no sum here feels: zero times a value of Inf would be NaN, where the weight itself gives Inf.
template <int PARTS>
__device__ __forceinline__ void split(float a, float b, uint32_t (&part)[PARTS]) {
    constexpr float kLeast = 1.17549435e-38f;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        if (PARTS == 2 && i == 1) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            part[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            part[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
        }
        a = fmaxf(a - __uint_as_float(__float_as_uint(a) & 0xffff0000u), kLeast);
        b = fmaxf(b - __uint_as_float(__float_as_uint(b) & 0xffff0000u), kLeast);
    }
}

// a sequence's length, held to what its page list can hold; EARLY: read before the launch's own wait, so from L2 (what
// this SM's L1 holds may be older than the wait of the launch before)
template <bool EARLY = false>
__device__ __forceinline__ int length_of(const AttnParams &p, int b) {
    int64_t n = EARLY ? __ldcg(p.lens + b) : __ldg(p.lens + b);
    const int64_t cap = p.max_pages << p.page_shift;
    return static_cast<int>(n < 0 ? 0 : n > cap ? cap : n);
}
template <bool EARLY>
__device__ __forceinline__ int units_of(const AttnParams &p, int b) {
    return (length_of<EARLY>(p, b) + (1 << p.unit_shift) - 1) >> p.unit_shift;
}

// a / b of non-negative values; 32-bit where they fit (a 64-bit division takes a few hundred cycles)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The cut: all units in a row, sequence by sequence and head by head, each at a place; CTA i works on the units whose
// place lies in [i places / ctas, (i + 1) places / ctas).  Few units lie at consecutive places.  With four and more per
// CTA a unit takes two places and the end of a head one more: that costs about half a unit (1.0 of 1.6 us), and ranges
// of many short heads would take longer than the others.
struct Cut {
    int64_t places;   // in all
    int ctas, many;   // CTAs that work; 1: two places per unit and one per head's end
    __device__ __forceinline__ int64_t start(int i) const { return quotient(places * i, ctas); }   // of CTA i's range
    __device__ __forceinline__ int64_t of(int64_t units, int64_t heads) const { return (units << many) + (many ? heads : 0); }
    __device__ __forceinline__ int step() const { return 1 << many; }
};
// Where range `index` begins (for index < cut.ctas): its first place, the sequence there, and the places before that.
struct Share {
    Cut cut;
    int64_t start, first;
    int b;
};

// Sums over the CTA's 128 threads of n (at most 2^24), low word, and of n > 0, high word: in all, and up to this thread.
__device__ __forceinline__ uint64_t scan_units(uint32_t n, uint64_t &upto, int64_t *s_scan) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
    uint32_t s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += x;
    }
    upto = static_cast<uint64_t>(__popc(some & (0xffffffffu >> (31 - lane)))) << 32 | s;
    if (lane == 31) s_scan[warp] = static_cast<int64_t>(upto);
    __syncthreads();
    uint64_t all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) upto += static_cast<uint64_t>(s_scan[i]);
        all += static_cast<uint64_t>(s_scan[i]);
    }
    return all;
}

__device__ __forceinline__ Cut make_cut(const AttnParams &p, int64_t units, int64_t heads) {
    Cut c;
    units *= p.vheads;
    c.many = units >= 4ll * p.grid ? 1 : 0;
    c.places = c.of(units, heads * p.vheads);
    c.ctas = static_cast<int>(units < p.grid ? units : p.grid);
    return c;
}

// more than 128 sequences: two passes over them
template <bool EARLY>
__device__ __forceinline__ Share find_range_of_many(const AttnParams &p, int index, int64_t *s_scan, int *s_at) {
    Share r;
    int64_t units = 0, heads = 0;
    uint64_t upto;
    for (int b0 = 0; b0 < p.n_seqs; b0 += kWarps * 32) {
        const int b = b0 + threadIdx.x;
        const uint64_t all = scan_units(b < p.n_seqs ? units_of<EARLY>(p, b) : 0, upto, s_scan);
        units += static_cast<uint32_t>(all);
        heads += static_cast<int64_t>(all >> 32);
        __syncthreads();
    }
    r.cut = make_cut(p, units, heads);
    if (index >= r.cut.ctas) return r;   // the same for the whole CTA
    r.start = r.cut.start(index);
    int64_t before = 0;
    for (int b0 = 0; b0 < p.n_seqs; b0 += kWarps * 32) {
        const int b = b0 + threadIdx.x;
        const int n = b < p.n_seqs ? units_of<EARLY>(p, b) : 0;
        if (threadIdx.x == 0) *s_at = -1;
        const uint64_t all = scan_units(n, upto, s_scan);
        const int64_t end = before + r.cut.of(static_cast<uint32_t>(upto), upto >> 32) * p.vheads;
        const int64_t first = end - (n > 0 ? r.cut.of(n, 1) * p.vheads : 0);
        if (first <= r.start && r.start < end) {
            *s_at = b;
            s_scan[kWarps] = first;
        }
        __syncthreads();
        if (*s_at >= 0) break;
        before += r.cut.of(static_cast<uint32_t>(all), all >> 32) * p.vheads;
        __syncthreads();
    }
    r.first = s_scan[kWarps];
    r.b = *s_at;
    return r;
}

// s_scan: kWarps + 1 values
template <bool EARLY>
__device__ __forceinline__ Share find_range(const AttnParams &p, int index, int64_t *s_scan, int *s_at) {
    if (p.n_seqs > kWarps * 32) return find_range_of_many<EARLY>(p, index, s_scan, s_at);
    Share r;
    const int n = static_cast<int>(threadIdx.x) < p.n_seqs ? units_of<EARLY>(p, threadIdx.x) : 0;
    uint64_t upto;
    const uint64_t all = scan_units(n, upto, s_scan);
    r.cut = make_cut(p, static_cast<uint32_t>(all), all >> 32);
    if (index >= r.cut.ctas) return r;   // the same for the whole CTA
    r.start = r.cut.start(index);
    const int64_t end = r.cut.of(static_cast<uint32_t>(upto), upto >> 32) * p.vheads;
    const int64_t first = end - (n > 0 ? r.cut.of(n, 1) * p.vheads : 0);
    if (first <= r.start && r.start < end) {
        *s_at = threadIdx.x;
        s_scan[kWarps] = first;
    }
    __syncthreads();
    r.first = s_scan[kWarps];
    r.b = *s_at;
    return r;
}

// four features of the output from element `at` on, the first `left` of them
__device__ __forceinline__ void store4(const AttnParams &p, int64_t at, int left, const float (&x)[4]) {
    if (p.o_vec) {   // rows and heads of whole fours on their alignment
        if (p.o_bf16) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.o) + at) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + at) = make_float4(x[0], x[1], x[2], x[3]);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (e >= left) break;
        if (p.o_bf16) static_cast<__nv_bfloat16 *>(p.o)[at + e] = __float2bfloat16_rn(x[e]);
        else static_cast<float *>(p.o)[at + e] = x[e];
    }
}

// floats of one partial: per query head o in a row of head_dim rounded up to 4, then m and the sum of each
__host__ __device__ __forceinline__ int part_row(int head_dim) { return (head_dim + 3) & ~3; }
__host__ __device__ __forceinline__ int part_floats(int per_vhead, int head_dim) {
    return (per_vhead * (part_row(head_dim) + 2) + 3) & ~3;
}

// shared memory behind the ring: the four warps' results of 8 heads x up to 128 features at a time
template <int DB>
struct AttnShared {
    static constexpr int kFeatures = DB < 2 ? 64 : 128;
    float o[kWarps][8][kFeatures];
    float m[kWarps][8], l[kWarps][8];
    int64_t scan[kWarps + 1];
    int at;
};

// A unit: sequence b (len keys, n units per head), part `sub` of the query heads of key-value head kv, unit j of it, and
// its place counted from the first of this CTA's range.
struct Walker {
    int b, len, n, kv, sub, j, place;
    __device__ __forceinline__ void next(const AttnParams &p, const Cut &cut) {
        place += cut.step();
        if (++j < n) return;
        j = 0;
        place += cut.many;
        if (++sub < p.vper) return;
        sub = 0;
        if (++kv < p.n_kv) return;
        kv = 0;
        do {   // sequences without keys have no units
            ++b;
            len = b < p.n_seqs ? length_of(p, b) : 0;
            n = (len + (1 << p.unit_shift) - 1) >> p.unit_shift;
        } while (n == 0 && b < p.n_seqs);
    }
    __device__ __forceinline__ int head0(const AttnParams &p) const { return kv * p.group + sub * p.per_vhead; }
    __device__ __forceinline__ int heads(const AttnParams &p) const { return min(p.per_vhead, p.group - sub * p.per_vhead); }
};

// DB: 64-feature blocks (head_dim <= 64 DB), NT: tiles of 8 query heads, KT: keys a warp takes at once (16 or 32),
// ST: pieces (K or V of KT keys) in a warp's ring, FULL: head_dim is 64 DB, PARTS: bf16 parts of a softmax weight
template <int DB, int NT, int KT, int ST, bool FULL, int PARTS>
__global__ void __launch_bounds__(kWarps * 32, 2) k_paged_attn(const AttnParams p) {
    constexpr int D = 64 * DB;
    constexpr int R = KT / 8;                       // groups of 8 keys: a page holds whole groups
    constexpr int M = KT / 16;                      // MMA row tiles
    constexpr int kUnit = KT * kWarps;
    constexpr uint32_t kPiece = KT * D * 2;         // bytes
    constexpr uint32_t kAll = (1u << R) - 1;
    // The ring comes first, on 128 bytes: a copy whose 32-byte sector straddles two of shared memory's is split, and
    // L2 then delivers the sector twice (measured: 671 MB for 336, 5.4 instead of 6.9 TB/s).
    extern __shared__ __align__(128) uint8_t smem[];
    AttnShared<DB> &sh = *reinterpret_cast<AttnShared<DB> *>(smem + kWarps * ST * kPiece);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // sequences without keys: zeros, and a log-sum of minus infinity
    for (int b = blockIdx.x; b < p.n_seqs; b += gridDim.x) {
        const int n = __ldg(p.lens + b);
        if (threadIdx.x == 0 && (n < 0 || n > (p.max_pages << p.page_shift))) atomicOr(p.status, kStatusBadIndex);
        if (n > 0) continue;
        for (int i = threadIdx.x; i < p.n_heads * p.head_dim; i += kWarps * 32) {
            if (p.o_bf16) static_cast<__nv_bfloat16 *>(p.o)[b * p.ldo + i] = __float2bfloat16_rn(0.0f);
            else static_cast<float *>(p.o)[b * p.ldo + i] = 0.0f;
        }
        if (p.lse)
            for (int i = threadIdx.x; i < p.n_heads; i += kWarps * 32)
                p.lse[static_cast<int64_t>(b) * p.n_heads + i] = -INFINITY;
    }

    const Share share = find_range<false>(p, blockIdx.x, sh.scan, &sh.at);
    const Cut &cut = share.cut;
    if (static_cast<int>(blockIdx.x) >= cut.ctas) return;   // every CTA that works gets a unit
    const int todo = static_cast<int>(cut.start(blockIdx.x + 1) - share.start);   // places
    Walker at;   // the unit being worked on
    at.b = share.b;
    at.len = length_of(p, at.b);
    at.n = (at.len + kUnit - 1) / kUnit;
    const int vhead = static_cast<int>(quotient(share.start - share.first, cut.of(at.n, 1)));
    at.kv = vhead / p.vper;
    at.sub = vhead % p.vper;
    at.j = 0;
    at.place = 0;
    const int inside = static_cast<int>(share.start - share.first - vhead * cut.of(at.n, 1));   // places of the head before the range
    if (inside > 0) {   // the first unit at or behind the range's start: in this head, or the next head's first
        at.j = ((inside + cut.many) >> cut.many) - 1;
        at.place = (at.j << cut.many) - inside;
        at.next(p, cut);
    }

    // A piece in the ring: rows of 128-byte segments (segment d of row r at (r DB + d) 128).  Copies: eight lanes take
    // a segment, 16 bytes each.  The 16-byte chunk k of a segment lies at k ^ 4 (r & 1) for K, k ^ (r & 6) for V, so
    // that the eight lanes of a read phase (below) meet eight different chunks.  Where rows may start in the middle of
    // a 32-byte sector (p.shift: the ring's rows have a chunk to spare then), those rows are copied from 16 bytes before
    // their start, a place that is not read, and so lie one chunk further on: sectors stay whole.  Which rows depends on
    // the head, and for strides of an odd number of chunks on the row.
    const uint32_t ring = smem_u32(smem) + warp * (ST * kPiece);
    const int cq = lane >> 3, cj = lane & 7;   // copies: row of four, chunk
    const uint32_t turn = FULL ? 0u : static_cast<uint32_t>(p.shift) & static_cast<uint32_t>(p.row_stride >> 3);   // odd rows differ from even ones
    auto odd_of = [&](const __nv_bfloat16 *head) { return FULL ? 0u : static_cast<uint32_t>(p.shift) & static_cast<uint32_t>(reinterpret_cast<uintptr_t>(head) >> 4); };
    const int last_piece = (p.head_dim - 1) >> 3;   // the last 16-byte piece of a row that holds features
    const int row_mask = (1 << p.page_shift) - 1;
    const int64_t row4 = 4 * p.row_stride, lane_at = cq * p.row_stride + 8 * cj;
    const bool one_page = ((KT - 1) >> p.page_shift) == 0;   // a tile lies in one page
    // segments of which this lane's chunk holds features, in a row that lies where it should and in one a chunk further on
    uint32_t have0 = 0, have1 = 0;
#pragma unroll
    for (int d = 0; d < DB; ++d) {
        have0 |= 8 * d + cj <= last_piece ? 1u << d : 0u;
        have1 |= 8 * d + cj >= 1 && 8 * d + cj - 1 <= last_piece ? 1u << d : 0u;
    }
    // words of K's pieces 4 (last_piece / 4) + t that hold features: what lies behind head_dim may be anything
    uint32_t keep[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int left = p.head_dim - 8 * ((last_piece & ~3) + t) - 2 * e;
        keep[e] = left >= 2 ? 0xffffffffu : left == 1 ? 0xffffu : 0u;
    }

    // ---- copies, ahead of the work: unit `ahead` is the next whose K goes into the ring
    Walker ahead = at;
    int copied = 0, slot = 0;          // units whose K and V have been begun, ring slot for the next piece
    const int32_t *list = nullptr;     // ahead's page list
    const __nv_bfloat16 *kh = nullptr, *vh = nullptr;   // its head's keys and values
    int next[R];                       // pages of its groups of 8 keys (loaded one unit before their use)
    int64_t off[R];                    // offset of each group's first row
    uint32_t bits = 0;                 // 8 bits per unit in flight: a group's page is valid
    bool plain = false;                // every row of the tile is there
    auto enter = [&]() {
        const int64_t head = ahead.kv * p.head_stride;
        kh = p.k + head;
        vh = p.v + head;
        list = p.pages + ahead.b * p.max_pages;
    };
    auto look_up = [&]() {
        const int key = ahead.j * kUnit + KT * warp;
        next[0] = key < ahead.len ? __ldg(list + (key >> p.page_shift)) : -1;
        if (!one_page) {
#pragma unroll
            for (int r = 1; r < R; ++r) next[r] = key + 8 * r < ahead.len ? __ldg(list + ((key + 8 * r) >> p.page_shift)) : -1;
        }
    };
    // copies one piece: rows 4 h + cq of the groups
    auto copy = [&](const __nv_bfloat16 *head, bool values, int key, uint32_t ok) {
        const uint32_t on = FULL ? 0u : (odd_of(head) ^ (cq & turn)) & 1u, have = on ? have1 : have0;
        const __nv_bfloat16 *from = head + lane_at - (FULL ? 0 : 8 * static_cast<int>(on));
        const uint32_t to0 = ring + slot * kPiece + cq * DB * 128 + ((cj ^ (values ? cq & 2 : 4 * (cq & 1))) << 4);
        const uint32_t to1 = values ? to0 ^ 64u : to0;   // rows 4 to 7 of a group
        if (plain) {   // the common case without a test per row
#pragma unroll
            for (int h = 0; h < 2 * R; ++h) {
                const uint32_t to = (h & 1 ? to1 : to0) + 4 * h * DB * 128;
                const __nv_bfloat16 *src = from + off[h >> 1] + (h & 1 ? row4 : 0);
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    if (FULL || (have >> d & 1u)) cp16(to + d * 128, src + 64 * d);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2 * R; ++h) {
                const uint32_t to = (h & 1 ? to1 : to0) + 4 * h * DB * 128;
                const __nv_bfloat16 *src = from + off[h >> 1] + (h & 1 ? row4 : 0);
                const bool in = (ok >> (h >> 1) & 1u) && key + 4 * h + cq < ahead.len;
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    if (FULL || (have >> d & 1u)) cp16_or_zero(to + d * 128, in ? src + 64 * d : p.k, in);
            }
        }
    };
    auto issue_k = [&]() {
        if (ahead.place < todo) {
            const int key = ahead.j * kUnit + KT * warp;
            uint32_t ok = 0;
            if (one_page) {
                const bool fine = next[0] >= 0 && next[0] < p.n_pages;
                off[0] = fine ? next[0] * p.page_stride + (key & row_mask) * p.row_stride : 0;
#pragma unroll
                for (int r = 1; r < R; ++r) off[r] = off[r - 1] + 2 * row4;
                ok = fine ? kAll : 0u;
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const bool fine = next[r] >= 0 && next[r] < p.n_pages;
                    off[r] = fine ? next[r] * p.page_stride + ((key + 8 * r) & row_mask) * p.row_stride : 0;
                    ok |= fine ? 1u << r : 0u;
                }
            }
            plain = ok == kAll && key + KT <= ahead.len;
            if (!plain && lane == 0) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (!(ok >> r & 1u) && key + 8 * r < ahead.len) atomicOr(p.status, kStatusBadIndex);
            }
            bits = (bits & ~(0xffu << (8 * (copied & 3)))) | ok << (8 * (copied & 3));
            if (key < ahead.len) copy(kh, false, key, ok);
            slot = slot + 1 == ST ? 0 : slot + 1;
        }
        cp_commit();
    };
    auto issue_v = [&]() {
        if (ahead.place < todo) {
            const int key = ahead.j * kUnit + KT * warp;
            if (key < ahead.len) copy(vh, true, key, bits >> (8 * (copied & 3)));
            slot = slot + 1 == ST ? 0 : slot + 1;
            ++copied;
            ahead.next(p, cut);
            if (ahead.place < todo) {
                if (ahead.j == 0) enter();
                look_up();
            }
        }
        cp_commit();
    };

    // Q fragments: column g of tile n is query head 8 n + g of the virtual head; piece i of lane (g, t) is
    // features 32 i + 8 t .. + 7, the same that the lane holds of a key.  With rows on 16 bytes the loads are
    // unconditional, so that nothing waits for them before their use: a column behind the last head repeats it (what
    // becomes of it is not written), and a piece behind head_dim repeats the last (it meets zeros of the keys).
    uint4 qf[NT][D / 32];
    auto load_q = [&](const Walker &w) {
        const int head0 = w.head0(p), heads = w.heads(p);
        const uint16_t *row = reinterpret_cast<const uint16_t *>(p.q) + w.b * p.ldq + static_cast<int64_t>(head0) * p.head_dim;
        if (p.q_vec == 16) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 *src = reinterpret_cast<const uint4 *>(row + min(8 * n + g, heads - 1) * p.head_dim);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) qf[n][i] = __ldg(src + (FULL ? 4 * i + t : min(4 * i + t, last_piece)));
            }
            return;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int h = 8 * n + g, f = 32 * i + 8 * t;
                uint32_t x[4] = {0u, 0u, 0u, 0u};
                const uint16_t *src = row + h * p.head_dim + f;
                if (h < heads) {
                    if (p.q_vec == 8) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (f + 4 * e < p.head_dim) {
                                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src) + e);
                                x[2 * e] = v.x;
                                x[2 * e + 1] = v.y;
                            }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (f + e < p.head_dim) x[e >> 1] |= static_cast<uint32_t>(__ldg(src + e)) << (16 * (e & 1));
                    }
                }
                qf[n][i] = make_uint4(x[0], x[1], x[2], x[3]);
            }
    };

    enter();
    look_up();
    load_q(at);
    issue_k();
    issue_v();
    if (ST == 4) issue_k();

    float o[NT][DB][4][4];
    float m[NT][2], l[NT][2];
    int use = 0, seg_from = 0;   // ring slot of the next piece to be used; unit that began this head
    for (int done = 0;; ++done) {
        if (done == seg_from) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                m[n][0] = m[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.0f;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int w = 0; w < 4; ++w)
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[n][d][w][c] = 0.0f;
            }
        }
        const int key = at.j * kUnit + KT * warp;
        const uint32_t now = bits >> (8 * (done & 3));
        const bool live = key < at.len;   // the same for the whole warp

        // S^T = K Q^T: rows g and g + 8 of row tile k are keys 16 k + g and 16 k + 8 + g, columns the heads 2 t
        // and 2 t + 1 of each tile of 8.  (The barrier also ends every lane's reads of the piece before, whose slot
        // is filled next.)
        cp_wait<ST - 2>();
        __syncwarp();
        float s[NT][M][4];
        if (live) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < M; ++k) s[n][k][0] = s[n][k][1] = s[n][k][2] = s[n][k][3] = 0.0f;
            // places of pieces t (even i) and 4 + t (odd i) in row g
            const uint32_t on = FULL ? 0u : (odd_of(p.k + at.kv * p.head_stride) ^ (g & turn)) & 1u;
            const uint32_t src = ring + use * kPiece + g * DB * 128, swz = 4 * (g & 1);
            const uint32_t even = src + (((t + on) ^ swz) << 4);
            const uint32_t odd = src + ((4 + t + on) >> 3) * 128 + ((((4 + t + on) & 7) ^ swz) << 4);
#pragma unroll
            for (int k = 0; k < M; ++k) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    if (!FULL && 4 * i > last_piece) break;
                    const uint32_t piece = (i & 1 ? odd : even) + (16 * k * DB + (i >> 1)) * 128;
                    uint4 a = lds16(piece), c = lds16(piece + 8 * DB * 128);
                    if (!FULL && 4 * i + 3 >= last_piece) {
                        a = make_uint4(a.x & keep[0], a.y & keep[1], a.z & keep[2], a.w & keep[3]);
                        c = make_uint4(c.x & keep[0], c.y & keep[1], c.z & keep[2], c.w & keep[3]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma(s[n][k], a.x, c.x, a.y, c.y, qf[n][i].x, qf[n][i].y);
                        mma(s[n][k], a.z, c.z, a.w, c.w, qf[n][i].z, qf[n][i].w);
                    }
                }
            }
        }
        use = use + 1 == ST ? 0 : use + 1;
        if (ST == 4) issue_v(); else issue_k();

        // mask, running maximum, p = 2^(s scale - maximum) with the product not rounded on its own
        uint32_t ps[PARTS][NT][M][2];
        if (live) {
            if ((now & kAll) != kAll || key + KT > at.len) {   // the same for the whole warp
#pragma unroll
                for (int k = 0; k < M; ++k) {
                    const bool in0 = (now >> (2 * k) & 1u) && key + 16 * k + g < at.len;
                    const bool in1 = (now >> (2 * k + 1) & 1u) && key + 16 * k + 8 + g < at.len;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[n][k][c] = (c < 2 ? in0 : in1) ? s[n][k][c] : p.none;
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
                for (int k = 0; k < M; ++k) {
                    x0 = fmaxf(x0, fmaxf(s[n][k][0] * p.scale_log2, s[n][k][2] * p.scale_log2));
                    x1 = fmaxf(x1, fmaxf(s[n][k][1] * p.scale_log2, s[n][k][3] * p.scale_log2));
                }
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, w));
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, w));
                }
                const float m0 = fmaxf(m[n][0], x0), m1 = fmaxf(m[n][1], x1);
                if (__any_sync(0xffffffffu, m0 > m[n][0] || m1 > m[n][1])) {
                    // factors 2^(old - new); an old maximum of minus infinity gives 0
                    const float f0 = m0 == m[n][0] ? 1.0f : exp2_fast(m[n][0] - m0);
                    const float f1 = m1 == m[n][1] ? 1.0f : exp2_fast(m[n][1] - m1);
                    l[n][0] *= f0;
                    l[n][1] *= f1;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            o[n][d][w][0] *= f0;
                            o[n][d][w][1] *= f1;
                            o[n][d][w][2] *= f0;
                            o[n][d][w][3] *= f1;
                        }
                    m[n][0] = m0;
                    m[n][1] = m1;
                }
                const float z0 = m0 == -INFINITY ? 0.0f : m0, z1 = m1 == -INFINITY ? 0.0f : m1;
#pragma unroll
                for (int k = 0; k < M; ++k) {
                    float w[2][2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        w[r][0] = exp2_fast(fmaf(s[n][k][2 * r], p.scale_log2, -z0));
                        w[r][1] = exp2_fast(fmaf(s[n][k][2 * r + 1], p.scale_log2, -z1));
                    }
                    l[n][0] += w[0][0] + w[1][0];
                    l[n][1] += w[0][1] + w[1][1];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        uint32_t part[PARTS];
                        split<PARTS>(w[r][0], w[r][1], part);
#pragma unroll
                        for (int i = 0; i < PARTS; ++i) ps[i][n][k][r] = transpose8x8(part[i]);
                    }
                }
            }
        }

        // O^T += V^T P^T: of row tile k, lane (g, t) holds features 64 d + 8 g .. + 7 of keys 16 k + 2t, 2t + 1,
        // 2t + 8 and 2t + 9
        cp_wait<ST - 2>();
        __syncwarp();
        if (live) {
            // places of piece g in rows 2 t and 2 t + 1
            const uint32_t on = odd_of(p.v + at.kv * p.head_stride) & 1u, c0 = g + on, c1 = g + (on ^ (turn & 1u));
            const uint32_t src = ring + use * kPiece + 2 * t * DB * 128;
            const uint32_t row0 = src + (c0 >> 3) * 128 + (((c0 & 7) ^ (2 * t)) << 4);
            const uint32_t row1 = src + DB * 128 + (c1 >> 3) * 128 + (((c1 & 7) ^ (2 * t)) << 4);
            // in accumulators of this step's own (of 16 keys where two tiles of heads and three parts fill the registers)
            constexpr int KC = NT == 1 || PARTS == 2 ? M : 1;
#pragma unroll
            for (int k0 = 0; k0 < M; k0 += KC) {
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    if (!FULL && 8 * d > last_piece) break;
                    uint32_t v[KC][4][4];   // rows 2 t, 2 t + 1, 2 t + 8 and 2 t + 9
#pragma unroll
                    for (int k = 0; k < KC; ++k)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint4 x = lds16((r & 1 ? row1 : row0) + (16 * (k0 + k) * DB + d) * 128 + (r >> 1) * (8 * DB * 128));
                            v[k][r][0] = x.x;
                            v[k][r][1] = x.y;
                            v[k][r][2] = x.z;
                            v[k][r][3] = x.w;
                        }
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        // rows g and g + 8 of the MMA are features 64 d + 8 g + 2 w and + 1
                        uint32_t a[KC][4];
#pragma unroll
                        for (int k = 0; k < KC; ++k)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                a[k][c] = __byte_perm(v[k][c & 2][w], v[k][(c & 2) + 1][w], c & 1 ? 0x7632 : 0x5410);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float x[4];
#pragma unroll
                            for (int i = PARTS - 1; i >= 0; --i)
#pragma unroll
                                for (int k = 0; k < KC; ++k) {
                                    const uint32_t(&pk)[2] = ps[i][n][k0 + k];
                                    if (i == PARTS - 1 && k == 0) mma_first(x, a[k][0], a[k][1], a[k][2], a[k][3], pk[0], pk[1]);
                                    else mma(x, a[k][0], a[k][1], a[k][2], a[k][3], pk[0], pk[1]);
                                }
#pragma unroll
                            for (int c = 0; c < 4; ++c) o[n][d][w][c] += x[c];
                        }
                    }
                }
            }
        }
        use = use + 1 == ST ? 0 : use + 1;
        if (ST == 4) issue_k(); else issue_v();

        const bool ends = at.j + 1 == at.n;
        const bool more = at.place + cut.step() + (ends ? cut.many : 0) < todo;   // a unit is left in the range
        if (!ends && more) {
            ++at.j;
            at.place += cut.step();
            continue;
        }
        // The head ends here, or this CTA's range does: join the four warps through shared memory, while the copies
        // for the next head are on their way.
        const int head0 = at.head0(p), heads = at.heads(p);
        const bool whole = ends && at.j == done - seg_from;
        const int b = at.b;
        float *part = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (seg_from == 0 ? 0 : 1)) * part_floats(p.per_vhead, p.head_dim);
        const int row = part_row(p.head_dim);
        if (more) {
            at.next(p, cut);
            load_q(at);
        }
        seg_from = done + 1;
        constexpr int kF = AttnShared<DB>::kFeatures;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) {
                l[n][0] += __shfl_xor_sync(0xffffffffu, l[n][0], w);
                l[n][1] += __shfl_xor_sync(0xffffffffu, l[n][1], w);
            }
            const int mine = min(8, heads - 8 * n);   // heads of this tile
#pragma unroll
            for (int f0 = 0; f0 < D; f0 += kF) {
                __syncthreads();   // the buffer is free
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int h = 2 * t + c;
                    if (h >= mine) continue;
                    if (g == 0) {
                        sh.m[warp][h] = m[n][c];
                        sh.l[warp][h] = l[n][c];
                    }
#pragma unroll
                    for (int d = f0 / 64; d < (f0 + kF) / 64; ++d) {
                        float4 *dst = reinterpret_cast<float4 *>(&sh.o[warp][h][64 * d - f0 + 8 * g]);
                        dst[0] = make_float4(o[n][d][0][c], o[n][d][0][2 + c], o[n][d][1][c], o[n][d][1][2 + c]);
                        dst[1] = make_float4(o[n][d][2][c], o[n][d][2][2 + c], o[n][d][3][c], o[n][d][3][2 + c]);
                    }
                }
                __syncthreads();
                // four features of a head per thread and step
                for (int i = threadIdx.x; i < mine * (kF / 4); i += kWarps * 32) {
                    const int h = i / (kF / 4), at4 = 4 * (i % (kF / 4)), d = f0 + at4;
                    if (d >= row) continue;
                    float mw[kWarps];
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) mw[w] = sh.m[w][h];
                    const float top = fmaxf(fmaxf(mw[0], mw[1]), fmaxf(mw[2], mw[3]));
                    const float z = top == -INFINITY ? 0.0f : top;
                    float sum = 0.0f, x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float4 v = *reinterpret_cast<const float4 *>(&sh.o[w][h][at4]);
                        const float f = exp2_fast(mw[w] - z);
                        sum = fmaf(f, sh.l[w][h], sum);
                        x[0] = fmaf(f, v.x, x[0]);
                        x[1] = fmaf(f, v.y, x[1]);
                        x[2] = fmaf(f, v.z, x[2]);
                        x[3] = fmaf(f, v.w, x[3]);
                    }
                    const int64_t head = head0 + 8 * n + h;
                    if (!whole) {
                        *reinterpret_cast<float4 *>(part + (8 * n + h) * row + d) = make_float4(x[0], x[1], x[2], x[3]);
                        if (d == 0) {
                            part[p.per_vhead * row + 2 * (8 * n + h)] = top;
                            part[p.per_vhead * row + 2 * (8 * n + h) + 1] = sum;
                        }
                        continue;
                    }
                    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] *= inv;
                    store4(p, b * p.ldo + head * p.head_dim + d, p.head_dim - d, x);
                    if (d == 0 && p.lse) p.lse[static_cast<int64_t>(b) * p.n_heads + head] = (top + log2f(sum)) * 0.6931471805599453f;
                }
            }
        }
        if (!more) break;
    }
    cp_wait<0>();
}

// Joins the partials of the heads that more than one CTA of the first launch worked on.  CTA (i, h) joins query head h
// of the virtual head that CTA i of the first launch began and did not finish.  It finds that out before it waits for
// the first launch: the lengths were complete before that one's CTAs let this launch begin.  A warp takes every fourth
// partial, 32 of them at a time: lane j holds the j-th one's maximum and sum.
__global__ void __launch_bounds__(kWarps * 32) k_paged_attn_join(const AttnParams p) {
    __shared__ int64_t s_scan[kWarps + 1];
    __shared__ int s_at;
    __shared__ float s_top[kWarps], s_sum[kWarps];
    __shared__ float4 s_o[kWarps][64];
    const int i0 = blockIdx.x, h = blockIdx.y;
    const Share next = find_range<true>(p, i0 + 1, s_scan, &s_at);   // behind CTA i0's range
    const Cut &cut = next.cut;
    bool mine = i0 + 1 < cut.ctas, late = false;
    int b = 0, head = 0, i1 = 0;
    if (mine) {
        b = next.b;
        const int n = units_of<true>(p, b);
        const int vh = static_cast<int>(quotient(next.start - next.first, cut.of(n, 1))), sub = vh % p.vper;
        const int64_t first = next.first + vh * cut.of(n, 1), begin = cut.start(i0);
        const int64_t last = first + (static_cast<int64_t>(n - 1) << cut.many);   // places of the head's first and last unit
        head = vh / p.vper * p.group + sub * p.per_vhead + h;
        mine = next.start > first && begin <= first && next.start <= last && h < p.group - sub * p.per_vhead;
        late = begin <= first - cut.many - cut.step();   // a unit of i0's range lies before the head: its partial is in slot 1
        // the CTA of the head's last unit: the largest i whose range starts at its place or before
        i1 = static_cast<int>(quotient((last + 1) * cut.ctas - 1, cut.places));
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!mine) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t size = part_floats(p.per_vhead, p.head_dim);
    const int row = part_row(p.head_dim);
    auto partial = [&](int i) { return p.part + (2 * static_cast<int64_t>(i) + (i == i0 && late ? 1 : 0)) * size; };
    float top = -INFINITY, sum = 0.0f;
    float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int j0 = i0 + warp; j0 <= i1; j0 += kWarps * 32) {
        const int ij = j0 + kWarps * lane;
        float mi = -INFINITY, li = 0.0f;
        if (ij <= i1) {
            const float *ml = partial(ij) + p.per_vhead * row + 2 * h;
            mi = ml[0];
            li = ml[1];
        }
        float x = fmaxf(top, mi);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
        const float z = x == -INFINITY ? 0.0f : x;
        const float f = exp2_fast(top - z), fi = exp2_fast(mi - z);
        float si = li * fi;
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) si += __shfl_xor_sync(0xffffffffu, si, w);
        sum = sum * f + si;
        top = x;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            o[c].x *= f; o[c].y *= f; o[c].z *= f; o[c].w *= f;
        }
        const int n = min(32, (i1 - j0) / kWarps + 1);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (c == 1 && row <= 128) break;
            const int at = 4 * (lane + 32 * c) < row ? 4 * (lane + 32 * c) : 0;   // lanes without features repeat the first
            for (int j = 0; j < n; j += 8) {
                // eight loads with no condition, so that they are in flight together; those behind the last one are not used
                float4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = *reinterpret_cast<const float4 *>(partial(j0 + kWarps * min(j + k, n - 1)) + h * row + at);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const bool used = j + k < n;   // (0 times an Inf behind the last one would be NaN)
                    const float fj = __shfl_sync(0xffffffffu, fi, j + k);
                    o[c].x = used ? fmaf(v[k].x, fj, o[c].x) : o[c].x;
                    o[c].y = used ? fmaf(v[k].y, fj, o[c].y) : o[c].y;
                    o[c].z = used ? fmaf(v[k].z, fj, o[c].z) : o[c].z;
                    o[c].w = used ? fmaf(v[k].w, fj, o[c].w) : o[c].w;
                }
            }
        }
    }
    if (lane == 0) {
        s_top[warp] = top;
        s_sum[warp] = sum;
    }
    s_o[warp][lane] = o[0];
    s_o[warp][lane + 32] = o[1];
    __syncthreads();
    float x = s_top[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) x = fmaxf(x, s_top[i]);
    const float z = x == -INFINITY ? 0.0f : x;
    float f[kWarps], all = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        f[i] = exp2_fast(s_top[i] - z);
        all += f[i] * s_sum[i];
    }
    const float inv = all > 0.0f ? 1.0f / all : (all == 0.0f ? 0.0f : all);
    for (int d = threadIdx.x; d < p.head_dim; d += kWarps * 32) {
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) y += f[i] * reinterpret_cast<const float *>(s_o[i])[d];
        y *= inv;
        const int64_t at = b * p.ldo + static_cast<int64_t>(head) * p.head_dim + d;
        if (p.o_bf16) static_cast<__nv_bfloat16 *>(p.o)[at] = __float2bfloat16_rn(y);
        else static_cast<float *>(p.o)[at] = y;
    }
    if (p.lse && threadIdx.x == 0) p.lse[static_cast<int64_t>(b) * p.n_heads + head] = (x + log2f(all)) * 0.6931471805599453f;
}

int per_vhead_of(int64_t group, int64_t head_dim) {
    const int most = head_dim <= 128 ? 16 : 8;   // accumulators of 16 heads x 256 features do not fit the registers
    return static_cast<int>(group < most ? group : most);
}

template <int DB, int NT, int KT, int ST, bool FULL, int PARTS>
cudaError_t go_parts(AttnParams p, cudaStream_t s) {
    constexpr int smem = kWarps * ST * KT * 64 * DB * 2 + static_cast<int>(sizeof(AttnShared<DB>));
    static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs per SM");
    p.shift = !FULL && (p.head_dim + 7) / 8 < 8 * DB && p.page_stride % 16 == 0 ? 1 : 0;
    const void *f = reinterpret_cast<const void *>(k_paged_attn<DB, NT, KT, ST, FULL, PARTS>);
    cudaError_t e = smem_attr(f, smem);
    if (e != cudaSuccess) return e;
    static std::atomic<int> occupancy{0};   // the same on every device of this architecture
    int occ = occupancy.load(std::memory_order_relaxed);
    if (occ == 0) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, k_paged_attn<DB, NT, KT, ST, FULL, PARTS>, kWarps * 32, smem);
        if (e != cudaSuccess) return e;
        if (occ < 1) occ = 1;
        if (occ > kAttnMaxCtas) occ = kAttnMaxCtas;
        occupancy.store(occ, std::memory_order_relaxed);
    }
    constexpr int unit = KT * kWarps;
    p.unit_shift = unit == 128 ? 7 : 6;
    static_assert(unit == 128 || unit == 64, "the shift above");
    const int64_t most = (((p.max_pages << p.page_shift) + unit - 1) / unit) * p.n_seqs * p.vheads;
    const int64_t room = static_cast<int64_t>(num_sms()) * occ;
    p.grid = static_cast<int>(most < room ? most : room);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.grid));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_paged_attn<DB, NT, KT, ST, FULL, PARTS>, p);
    if (e != cudaSuccess) return e;
    if (p.grid < 2 || (p.max_pages << p.page_shift) <= unit) return cudaSuccess;   // one CTA, or one unit per head at most: nothing to join
    cfg.gridDim = dim3(static_cast<unsigned>(p.grid - 1), static_cast<unsigned>(p.per_vhead));
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, k_paged_attn_join, p);
}

template <int DB, int NT, int KT, int ST, bool FULL>
cudaError_t go(const AttnParams &p, cudaStream_t s) {
    return p.o_bf16 ? go_parts<DB, NT, KT, ST, FULL, 2>(p, s) : go_parts<DB, NT, KT, ST, FULL, 3>(p, s);
}

template <int DB, int KT, int ST>
cudaError_t by_heads(const AttnParams &p, cudaStream_t s) {
    const bool full = p.head_dim == 64 * DB;
    if constexpr (DB < 4) {
        if (p.per_vhead > 8) return full ? go<DB, 2, KT, ST, true>(p, s) : go<DB, 2, KT, ST, false>(p, s);
    }
    return full ? go<DB, 1, KT, ST, true>(p, s) : go<DB, 1, KT, ST, false>(p, s);
}

}  // namespace

size_t paged_attn_ws_bytes(int64_t n_seqs, int64_t n_heads, int64_t n_kv_heads, int64_t head_dim) {
    if (n_seqs <= 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0) return 256;
    const int64_t ctas = static_cast<int64_t>(num_sms()) * kAttnMaxCtas;
    return 256 + static_cast<size_t>(2 * ctas) * static_cast<size_t>(part_floats(per_vhead_of(n_heads / n_kv_heads, head_dim), static_cast<int>(head_dim))) * 4;
}

cudaError_t launch_paged_attn(const void *Q, int64_t ldq, int64_t n_seqs, int64_t n_heads, const KvCacheHost &c,
                              const int32_t *pages, int64_t max_pages, const int32_t *lens, float scale, void *O, bool o_bf16,
                              int64_t ldo, float *lse, void *ws, cudaStream_t s) {
    AttnParams p = {};
    p.q = static_cast<const __nv_bfloat16 *>(Q); p.ldq = ldq;
    p.k = static_cast<const __nv_bfloat16 *>(c.k); p.v = static_cast<const __nv_bfloat16 *>(c.v);
    p.page_stride = c.page_stride; p.head_stride = c.head_stride; p.row_stride = c.row_stride;
    p.pages = pages; p.max_pages = max_pages; p.n_pages = c.n_pages; p.page_shift = c.page_shift; p.lens = lens;
    p.n_seqs = static_cast<int>(n_seqs); p.n_heads = static_cast<int>(n_heads);
    p.group = static_cast<int>(n_heads / c.n_kv_heads);
    p.per_vhead = per_vhead_of(p.group, c.head_dim);
    p.vper = (p.group + p.per_vhead - 1) / p.per_vhead;
    p.n_kv = c.n_kv_heads;
    p.vheads = p.n_kv * p.vper;
    p.head_dim = c.head_dim;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    if (p.scale_log2 == 0.0f) p.scale_log2 = std::numeric_limits<float>::denorm_min();   // weights of 1 all the same
    p.none = p.scale_log2 < 0.0f ? INFINITY : -INFINITY;
    p.o = O; p.o_bf16 = o_bf16 ? 1 : 0; p.ldo = ldo; p.lse = lse;
    p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + 256);
    p.status = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(ws) + kStatusOffset);
    p.q_vec = c.head_dim % 8 == 0 && ldq % 8 == 0 && (reinterpret_cast<uintptr_t>(Q) & 15) == 0   ? 16
              : c.head_dim % 4 == 0 && ldq % 4 == 0 && (reinterpret_cast<uintptr_t>(Q) & 7) == 0 ? 8
                                                                                                 : 2;
    p.o_vec = c.head_dim % 4 == 0 && ldo % 4 == 0 && (reinterpret_cast<uintptr_t>(O) & (o_bf16 ? 7 : 15)) == 0 ? 1 : 0;
    // 32 keys at once and two CTAs per SM; at 256 features 16 keys, so that two CTAs fit
    if (c.head_dim <= 64) return by_heads<1, 32, 4>(p, s);
    if (c.head_dim <= 128) return by_heads<2, 32, 3>(p, s);
    return by_heads<4, 16, 3>(p, s);
}

}  // namespace bitnet
