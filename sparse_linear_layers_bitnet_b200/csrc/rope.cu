// Rotary positions, and the write of keys and values into a paged cache (sm_100a).
//
// A pair (a, b) of a head's features is turned by the angle of its position
// and frequency, with (c, s) = (cos, sin) read from an fp32 table:
//   a' = fp32(fp32(a c) - fp32(b s)),   b' = fp32(fp32(b c) + fp32(a s)),
// each step one rounded fp32 operation, then one rounding to the output's
// type, so the result is the same bit for bit everywhere.  The inverse (the
// backward pass: the rotation is orthogonal) takes -s.
//
// Memory-bound: every head is read once and written once.  A thread owns one
// place of the head (the vectors of up to 16 bytes that hold its pairs) in
// several heads of a row, so it reads its (c, s) once per row, and has all its
// loads in flight before it looks at the row's position and page.  Measured: 4095
// fp32 rows of 64 heads of 128 41 us (6.5 TB/s), 4096 bf16 rows 25.4 us (5.3 TB/s).
#include "common.cuh"
#include "kernels.h"

namespace bitnet {

namespace {

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC <= 16 ? sizeof(T) * VEC : 16) Vec {
    T v[VEC];
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// a feature that is not turned: as it is, or rounded to the narrower type
template <typename TO, typename TI>
__device__ __forceinline__ TO copied(TI x) {
    if constexpr (sizeof(TI) == sizeof(TO)) return x;
    else return narrow<TO>(widen(x));
}

struct RopeParams {
    const void *x;            // input rows
    int64_t ldx;
    void *y;                  // rotated heads (rope) or the query heads (append)
    int64_t ldy;
    const int32_t *pos;
    const float2 *table;      // [n_pos, rot / 2] (cos, sin); NULL with rot = 0
    int64_t n_pos;
    int64_t T;
    int heads;                // heads per row that are rotated and go to y
    int kv_heads;             // append: key heads, then value heads behind them
    int head_dim, rot, inverse;
    int table_vec;            // table rows lie on 16 bytes
    int places;               // threads per head
    int slots;                // heads a CTA holds at once
    uint32_t row_bytes, slot_bytes;   // of the ring: a row's features, a slot
    // append
    void *k, *v;
    int64_t page_stride, head_stride, row_stride;
    const int32_t *pages;     // [n_seqs, max_pages]
    const int32_t *seq;       // [T] or NULL (row t is sequence t)
    int64_t n_seqs, max_pages, n_pages;
    int page_shift;
    uint32_t *status;
};

// vectors of a head that one thread holds: both halves of its pairs, or (interleaved) one vector of whole pairs
template <int VEC, bool INTERLEAVED>
constexpr int kVectors = INTERLEAVED && VEC > 1 ? 1 : 2;
// heads per thread: 64 bytes of a row, at most 4 heads (32 to 128 bytes with 3 to 8 CTAs per SM measured)
template <typename TI, int VEC, bool INTERLEAVED>
constexpr int kHeads = 64 / (kVectors<VEC, INTERLEAVED> * VEC * static_cast<int>(sizeof(TI))) < 4
                           ? 64 / (kVectors<VEC, INTERLEAVED> * VEC * static_cast<int>(sizeof(TI))) : 4;

// two neighbouring features of a vector, rounded together
template <int VEC>
__device__ __forceinline__ void put2(Vec<float, VEC> &w, int i, float x, float y) {
    w.v[i] = x;
    w.v[i + 1] = y;
}
template <int VEC>
__device__ __forceinline__ void put2(Vec<__nv_bfloat16, VEC> &w, int i, float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    w.v[i] = h.x;
    w.v[i + 1] = h.y;
}

// Turns the pairs of one place: the halves of pair i lie in the two vectors (halves layout) or side by side
// (interleaved).  Scalar operations: the paired ones (f32x2) are joined into a fused multiply-add by the compiler, in
// PTX with .rn too, which rounds once less.
template <typename TI, typename TO, int VEC, bool INTERLEAVED, int NV, int PAIRS>
__device__ __forceinline__ void turn_place(const Vec<TI, VEC> (&v)[NV], Vec<TO, VEC> (&w)[NV], const float (&c)[PAIRS], const float (&s)[PAIRS]) {
    float x[2 * PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        const int ea = INTERLEAVED ? 2 * i : i, eb = INTERLEAVED ? 2 * i + 1 : i + VEC;
        const float a = widen(v[ea / VEC].v[ea % VEC]), b = widen(v[eb / VEC].v[eb % VEC]);
        x[ea] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
        x[eb] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
    }
    if constexpr (VEC == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) w[i].v[0] = narrow<TO>(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < NV * VEC; i += 2) put2(w[i / VEC], i % VEC, x[i], x[i + 1]);
    }
}

template <typename TI, typename TO, int VEC, bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(256, 4) k_rope(const RopeParams p) {
    constexpr int NV = kVectors<VEC, INTERLEAVED>, HEADS = kHeads<TI, VEC, INTERLEAVED>;
    constexpr int PAIRS = NV * VEC / 2;
    using VI = Vec<TI, VEC>;
    using VO = Vec<TO, VEC>;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t t = blockIdx.x;
    const int place = threadIdx.x % p.places, slot = threadIdx.x / p.places;
    if (slot >= p.slots) return;
    // this place's vectors: pairs below `turned`, copied features behind them
    const int half = p.rot >> 1;
    const int turned = half / PAIRS;   // places that rotate
    const bool turns = place < turned;
    int off[2];
    if (turns) {
        off[0] = INTERLEAVED ? NV * VEC * place : VEC * place;
        off[1] = INTERLEAVED ? off[0] + VEC : half + off[0];
    } else {
        off[0] = p.rot + NV * VEC * (place - turned);
        off[1] = off[0] + VEC;
    }
    const bool has1 = NV == 2 && off[1] < p.head_dim;   // an odd count of copied vectors leaves the last one alone

    // the heads' features first: they wait for nothing else
    const int all = p.heads + 2 * p.kv_heads;
    const int h0 = blockIdx.y * p.slots * HEADS + slot;
    const TI *x = static_cast<const TI *>(p.x) + t * p.ldx;
    VI v[HEADS][NV];
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
        const int h = h0 + j * p.slots;
        if (h < all) {
            const TI *src = x + static_cast<int64_t>(h) * p.head_dim;
            v[j][0] = *reinterpret_cast<const VI *>(src + off[0]);
            if (has1) v[j][NV - 1] = *reinterpret_cast<const VI *>(src + off[1]);
        }
    }

    // the row's position, and for the cache its sequence, page and row in the page
    const int pos = __ldg(p.pos + t);
    int64_t seq = t;
    if (APPEND && p.seq) seq = __ldg(p.seq + t);
    if (pos < 0 || (APPEND && seq < 0)) return;   // a padding row
    int64_t cache_row = 0;
    bool bad = p.rot > 0 && pos >= p.n_pos;
    float c[PAIRS], s[PAIRS];
    if (turns && !bad) {
        const float2 *row = p.table + static_cast<int64_t>(pos) * half + PAIRS * place;
        if (PAIRS % 2 == 0 && p.table_vec) {
#pragma unroll
            for (int i = 0; i < PAIRS / 2; ++i) {
                const float4 cs = __ldg(reinterpret_cast<const float4 *>(row) + i);
                c[(2 * i) % PAIRS] = cs.x;
                s[(2 * i) % PAIRS] = cs.y;
                c[(2 * i + 1) % PAIRS] = cs.z;
                s[(2 * i + 1) % PAIRS] = cs.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const float2 cs = __ldg(row + i);
                c[i] = cs.x;
                s[i] = cs.y;
            }
        }
    }
    if (APPEND) {
        const int64_t in_table = pos >> p.page_shift;
        bad = bad || seq >= p.n_seqs || in_table >= p.max_pages;
        if (!bad) {
            const int64_t page = __ldg(p.pages + seq * p.max_pages + in_table);
            bad = page < 0 || page >= p.n_pages;
            cache_row = page * p.page_stride + static_cast<int64_t>(pos & ((1 << p.page_shift) - 1)) * p.row_stride;
        }
    }
    if (bad) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
        return;
    }
    if (p.inverse) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) s[i] = -s[i];
    }
    TO *y = static_cast<TO *>(p.y) + t * p.ldy;
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
        const int h = h0 + j * p.slots;
        if (h >= all) continue;
        TO *dst = y + static_cast<int64_t>(h) * p.head_dim;
        if (APPEND && h >= p.heads) {
            const int kh = h - p.heads;
            dst = kh < p.kv_heads ? static_cast<TO *>(p.k) + cache_row + kh * p.head_stride
                                  : static_cast<TO *>(p.v) + cache_row + (kh - p.kv_heads) * p.head_stride;
        }
        VO u[NV];
        if (turns && !(APPEND && h >= p.heads + p.kv_heads)) {
            turn_place<TI, TO, VEC, INTERLEAVED>(v[j], u, c, s);
        } else {
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int i = 0; i < VEC; ++i) u[n].v[i] = copied<TO>(v[j][n].v[i]);
        }
        *reinterpret_cast<VO *>(dst + off[0]) = u[0];
        if (has1) *reinterpret_cast<VO *>(dst + off[1]) = u[NV - 1];
    }
}

// ---------------------------------------------------------------- many rows
//
// A persistent CTA takes rows blockIdx.x, + gridDim.x, ...: one producer warp brings whole rows and their rows of the
// table into a ring in shared memory (bulk copies counted on an mbarrier) and looks up their places in the cache,
// eight warps turn them and write them out.  What a CTA per row waits for one after the other (its start, the
// position, the page, the features) then lies behind the rows before it: 4096 rows of 96 heads of 128 into the
// cache take 39.7 us (5.1 TB/s) here and 50.6 in the direct form above, whatever its share of registers and loads in
// flight; of 100, whose rows of 200 bytes leave a sector in seven partly written, 45.9 and 66.5.
constexpr int kRowWarps = 8;
constexpr int kRowSlots = 3;

struct RowInfo {
    int64_t at;   // place in the cache
    int pos;      // or -1: nothing is written for this row
};
struct RowShared {
    uint64_t full[kRowSlots], empty[kRowSlots];
    RowInfo info[kRowSlots];
    int abort;
};

template <typename TI, typename TO, int VEC, bool INTERLEAVED, bool APPEND, int CTAS>
__global__ void __launch_bounds__((kRowWarps + 1) * 32, CTAS) k_rope_rows(const RopeParams p) {
    constexpr int NV = kVectors<VEC, INTERLEAVED>;
    constexpr int PAIRS = NV * VEC / 2;
    using VI = Vec<TI, VEC>;
    using VO = Vec<TO, VEC>;
    extern __shared__ __align__(128) uint8_t smem[];
    RowShared &sh = *reinterpret_cast<RowShared *>(smem + kRowSlots * static_cast<size_t>(p.slot_bytes));
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRowSlots; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kRowWarps);
        }
        fence_mbar_init();
        sh.abort = 0;
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = p.rot >> 1, table_bytes = half * 8;

    if (warp == kRowWarps) {   // producer: its lanes look up 32 rows at a time, lane 0 copies them in turn
        int slot = 0, round = 0;
        // no copy may outlive the CTA, after a wait that ran out least of all: wait for the last one into each slot
        auto drain = [&]() {
            if (lane == 0) {
                for (int i = 0; i < kRowSlots; ++i) {
                    const int last = i < slot ? round : round - 1;
                    int own = 0;
                    if (last >= 0) mbar_wait_bounded(&sh.full[i], last & 1, &own, p.status);
                }
            }
            __syncwarp();
        };
        for (int64_t t0 = blockIdx.x; t0 < p.T; t0 += 32ll * gridDim.x) {
            const int64_t mine = t0 + static_cast<int64_t>(lane) * gridDim.x;
            int pos = -1;
            int64_t at = 0;
            if (mine < p.T) {
                pos = __ldg(p.pos + mine);
                int64_t seq = mine;
                if (APPEND && p.seq) seq = __ldg(p.seq + mine);
                if (APPEND && seq < 0) pos = -1;   // a padding row, like one of a negative position
                if (pos >= 0) {
                    bool bad = p.rot > 0 && pos >= p.n_pos;
                    if (APPEND) {
                        const int64_t in_table = pos >> p.page_shift;
                        bad = bad || seq >= p.n_seqs || in_table >= p.max_pages;
                        if (!bad) {
                            const int64_t page = __ldg(p.pages + seq * p.max_pages + in_table);
                            bad = page < 0 || page >= p.n_pages;
                            at = page * p.page_stride + static_cast<int64_t>(pos & ((1 << p.page_shift) - 1)) * p.row_stride;
                        }
                    }
                    if (bad) {
                        atomicOr(p.status, kStatusBadIndex);
                        pos = -1;
                    }
                }
            }
            for (int k = 0; k < 32; ++k) {
                const int64_t t = t0 + static_cast<int64_t>(k) * gridDim.x;
                if (t >= p.T) break;
                const int row_pos = __shfl_sync(0xffffffffu, pos, k);
                const int64_t row_at = __shfl_sync(0xffffffffu, at, k);
                bool ok = true;
                if (lane == 0) {
                    if (round > 0) ok = mbar_wait_bounded(&sh.empty[slot], (round - 1) & 1, &sh.abort, p.status);
                    if (ok) {
                        uint8_t *to = smem + slot * static_cast<size_t>(p.slot_bytes);
                        sh.info[slot].at = row_at;
                        sh.info[slot].pos = row_pos;
                        const uint32_t bytes = row_pos >= 0 ? p.row_bytes + table_bytes : 0;
                        mbar_arrive_expect_tx(&sh.full[slot], bytes);   // also releases the row's info
                        if (row_pos >= 0) {
                            bulk_load(to, static_cast<const uint8_t *>(p.x) + t * p.ldx * static_cast<int64_t>(sizeof(TI)), p.row_bytes, &sh.full[slot]);
                            if (table_bytes) bulk_load(to + p.row_bytes, p.table + static_cast<int64_t>(row_pos) * half, table_bytes, &sh.full[slot]);
                        }
                    }
                }
                if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) {
                    drain();
                    return;
                }
                if (++slot == kRowSlots) {
                    slot = 0;
                    ++round;
                }
            }
        }
        drain();
        return;
    }

    const int place = threadIdx.x % p.places, first = threadIdx.x / p.places;
    const bool works = first < p.slots;
    const int turned = half / PAIRS;   // places that rotate
    const bool turns = place < turned;
    int off[2];
    if (turns) {
        off[0] = INTERLEAVED ? NV * VEC * place : VEC * place;
        off[1] = INTERLEAVED ? off[0] + VEC : half + off[0];
    } else {
        off[0] = p.rot + NV * VEC * (place - turned);
        off[1] = off[0] + VEC;
    }
    const bool has1 = NV == 2 && off[1] < p.head_dim;   // an odd count of copied vectors leaves the last one alone
    int slot = 0, round = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        if (!mbar_wait_bounded(&sh.full[slot], round & 1, &sh.abort, p.status)) return;
        const uint8_t *from = smem + slot * static_cast<size_t>(p.slot_bytes);
        const RowInfo info = sh.info[slot];
        if (info.pos >= 0 && works) {
            float c[PAIRS], s[PAIRS];
            if (turns) {
                const float2 *cs = reinterpret_cast<const float2 *>(from + p.row_bytes) + PAIRS * place;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    c[i] = cs[i].x;
                    s[i] = p.inverse ? -cs[i].y : cs[i].y;
                }
            }
            const TI *row = reinterpret_cast<const TI *>(from);
            // heads first, + slots, ... of n heads from `src` on, to dst + head * stride
            auto heads = [&](const TI *src, int n, TO *dst, int64_t stride, bool turn) {
                src += first * p.head_dim;
                dst += first * stride;
                const int src_step = p.slots * p.head_dim;
                const int64_t dst_step = p.slots * stride;
#pragma unroll 4
                for (int h = first; h < n; h += p.slots) {
                    VI v[NV];
                    VO w[NV];
                    v[0] = *reinterpret_cast<const VI *>(src + off[0]);
                    if (has1) v[NV - 1] = *reinterpret_cast<const VI *>(src + off[1]);
                    if (turn) {
                        turn_place<TI, TO, VEC, INTERLEAVED>(v, w, c, s);
                    } else {
#pragma unroll
                        for (int i = 0; i < NV; ++i)
#pragma unroll
                            for (int e = 0; e < VEC; ++e) w[i].v[e] = copied<TO>(v[i].v[e]);
                    }
                    *reinterpret_cast<VO *>(dst + off[0]) = w[0];
                    if (has1) *reinterpret_cast<VO *>(dst + off[1]) = w[NV - 1];
                    src += src_step;
                    dst += dst_step;
                }
            };
            heads(row, p.heads, static_cast<TO *>(p.y) + t * p.ldy, p.head_dim, turns);
            if (APPEND) {
                const TI *k = row + static_cast<int64_t>(p.heads) * p.head_dim;
                heads(k, p.kv_heads, static_cast<TO *>(p.k) + info.at, p.head_stride, turns);
                heads(k + static_cast<int64_t>(p.kv_heads) * p.head_dim, p.kv_heads, static_cast<TO *>(p.v) + info.at, p.head_stride, false);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[slot]);
        if (++slot == kRowSlots) {
            slot = 0;
            ++round;
        }
    }
}

// whether every vector access of VEC features is aligned
bool fits(const RopeParams &p, int vec, int in_size, int out_size, bool interleaved, bool append) {
    auto on = [&](const void *q, int size) {
        const int n = size * vec < 16 ? size * vec : 16;
        return (reinterpret_cast<uintptr_t>(q) & static_cast<uintptr_t>(n - 1)) == 0;
    };
    if (p.head_dim % vec || p.rot % vec || p.ldx % vec || p.ldy % vec) return false;
    if (!interleaved && (p.rot / 2) % vec) return false;
    if (!on(p.x, in_size) || !on(p.y, out_size)) return false;
    if (append && (p.page_stride % vec || p.head_stride % vec || p.row_stride % vec || !on(p.k, out_size) || !on(p.v, out_size)))
        return false;
    return true;
}

// by the ring: one CTA for every place on the device, CTAS per SM
template <typename TI, typename TO, int VEC, bool INTERLEAVED, bool APPEND, int CTAS>
cudaError_t go_rows(const RopeParams &p, int64_t smem, cudaStream_t s) {
    auto kernel = k_rope_rows<TI, TO, VEC, INTERLEAVED, APPEND, CTAS>;
    const cudaError_t e = smem_attr(reinterpret_cast<const void *>(kernel), 113 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int64_t grid = static_cast<int64_t>(CTAS) * num_sms();
    cfg.gridDim = dim3(static_cast<unsigned>(grid < p.T ? grid : p.T));
    cfg.blockDim = dim3((kRowWarps + 1) * 32);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename TI, typename TO, int VEC, bool INTERLEAVED, bool APPEND>
cudaError_t go(RopeParams p, cudaStream_t s) {
    constexpr int NV = kVectors<VEC, INTERLEAVED>, HEADS = kHeads<TI, VEC, INTERLEAVED>;
    const int all = p.heads + 2 * p.kv_heads;
    p.places = p.rot / (NV * VEC) + (p.head_dim - p.rot + NV * VEC - 1) / (NV * VEC);
    p.table_vec = p.rot % 4 == 0 && (reinterpret_cast<uintptr_t>(p.table) & 15) == 0;
    // many rows: each thread takes as many heads as it can hold; few rows: one head per thread where that fits a CTA
    int slots = p.T >= 2 * num_sms() ? (all + HEADS - 1) / HEADS : all;
    if (slots > 256 / p.places) slots = 256 / p.places;
    p.slots = slots;
    // Rows by the ring: enough of them for every CTA to have several, and whole 16-byte pieces in a row and in the
    // table's; three rows have to leave room for two CTAs.
    const int64_t row_bytes = static_cast<int64_t>(all) * p.head_dim * static_cast<int64_t>(sizeof(TI));
    const int64_t slot_bytes = (row_bytes + p.rot * 4 + 127) / 128 * 128;
    const int64_t smem = kRowSlots * slot_bytes + static_cast<int64_t>(sizeof(RowShared));
    // Measured (direct / ring, us).  Long rows: 4096 of 96 heads of 128 into the cache 50.6 / 39.7, 1200 of them 16.2 / 13.3,
    // 4096 of 64 heads of 128 turned only 31.3 / 25.3; but 12 KB (4096 of 48 heads of 128) 26.0 / 26.1, 8 KB (30 heads)
    // 17.4 / 24.2, 3 KB 7.2 / 18.6: a row's hand-over costs more than it hides.  Pieces narrower than 16 bytes, whatever the
    // row: 4096 of 96 heads of 100 66.5 / 45.9, of 30 24.1 / 14.1, 600 of 64 5.0 / 4.9.  fp32 that stays fp32 has half the
    // features per byte to turn and gains nothing: 4096 of 32 heads of 128 22.0 / 23.7, of 64 of 100 35.4 / 37.7.
    const bool narrow = VEC * sizeof(TI) < 16;
    if ((APPEND || sizeof(TI) == 2) && (narrow || row_bytes >= 16 * 1024) && p.T >= 8 * num_sms() && smem <= 113 * 1024 &&
        row_bytes % 16 == 0 && p.ldx * sizeof(TI) % 16 == 0 && (reinterpret_cast<uintptr_t>(p.x) & 15) == 0 && p.rot % 4 == 0 &&
        (reinterpret_cast<uintptr_t>(p.table) & 15) == 0) {
        p.row_bytes = static_cast<uint32_t>(row_bytes);
        p.slot_bytes = static_cast<uint32_t>(slot_bytes);
        p.slots = 32 * kRowWarps / p.places;
        // Two CTAs per SM with the registers for four heads in flight per thread, or three with fewer, so that the waits of
        // shorter rows overlap.  Measured (two / three, us): 4084 rows of 96 heads of 96 (18 KB) 29.4 / 33.8, 8192 of 64 heads
        // of 100 (13 KB) 39.8 / 38.1.
        return row_bytes > 16 * 1024 || smem > 74 * 1024 ? go_rows<TI, TO, VEC, INTERLEAVED, APPEND, 2>(p, smem, s)
                                                         : go_rows<TI, TO, VEC, INTERLEAVED, APPEND, 3>(p, smem, s);
    }
    const int rounds = (all + slots * HEADS - 1) / (slots * HEADS);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.T), static_cast<unsigned>(rounds));
    cfg.blockDim = dim3(static_cast<unsigned>((p.places * slots + 31) / 32 * 32));
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_rope<TI, TO, VEC, INTERLEAVED, APPEND>, p);
}

template <typename TI, typename TO, bool INTERLEAVED, bool APPEND>
cudaError_t by_vec(const RopeParams &p, cudaStream_t s) {
    const int in = sizeof(TI), out = sizeof(TO);
    if constexpr (sizeof(TI) == 2) {   // 16 bytes of a row at most
        if (fits(p, 8, in, out, INTERLEAVED, APPEND)) return go<TI, TO, 8, INTERLEAVED, APPEND>(p, s);
    }
    if (fits(p, 4, in, out, INTERLEAVED, APPEND)) return go<TI, TO, 4, INTERLEAVED, APPEND>(p, s);
    if (fits(p, 2, in, out, INTERLEAVED, APPEND)) return go<TI, TO, 2, INTERLEAVED, APPEND>(p, s);
    return go<TI, TO, 1, INTERLEAVED, APPEND>(p, s);
}

template <typename TI, typename TO, bool APPEND>
cudaError_t by_layout(const RopeParams &p, bool interleaved, cudaStream_t s) {
    return interleaved ? by_vec<TI, TO, true, APPEND>(p, s) : by_vec<TI, TO, false, APPEND>(p, s);
}

}  // namespace

cudaError_t launch_rope(const void *X, bool bf16, int64_t ldx, const int32_t *pos, const float *table, int64_t n_pos,
                        int64_t T, int64_t heads, int64_t head_dim, int64_t rot_dim, bool interleaved, bool inverse, void *Y,
                        int64_t ldy, uint32_t *status, cudaStream_t s) {
    RopeParams p = {};
    p.x = X; p.ldx = ldx; p.y = Y; p.ldy = ldy;
    p.pos = pos; p.table = reinterpret_cast<const float2 *>(table); p.n_pos = n_pos;
    p.T = T; p.heads = static_cast<int>(heads); p.kv_heads = 0;
    p.head_dim = static_cast<int>(head_dim); p.rot = static_cast<int>(rot_dim); p.inverse = inverse ? 1 : 0;
    p.status = status;
    return bf16 ? by_layout<__nv_bfloat16, __nv_bfloat16, false>(p, interleaved, s)
                : by_layout<float, float, false>(p, interleaved, s);
}

cudaError_t launch_rope_append(const void *QKV, bool bf16, int64_t ld, const int32_t *pos, const int32_t *seq,
                               const float *table, int64_t n_pos, int64_t T, int64_t n_heads, int64_t rot_dim,
                               bool interleaved, const KvCacheHost &c, const int32_t *pages, int64_t n_seqs,
                               int64_t max_pages, void *Q, uint32_t *status, cudaStream_t s) {
    RopeParams p = {};
    p.x = QKV; p.ldx = ld; p.y = Q; p.ldy = n_heads * c.head_dim;
    p.pos = pos; p.table = reinterpret_cast<const float2 *>(table); p.n_pos = n_pos;
    p.T = T; p.heads = static_cast<int>(n_heads); p.kv_heads = c.n_kv_heads;
    p.head_dim = c.head_dim; p.rot = static_cast<int>(rot_dim);
    p.k = c.k; p.v = c.v;
    p.page_stride = c.page_stride; p.head_stride = c.head_stride; p.row_stride = c.row_stride;
    p.pages = pages; p.seq = seq; p.n_seqs = n_seqs; p.max_pages = max_pages; p.n_pages = c.n_pages;
    p.page_shift = c.page_shift; p.status = status;
    return bf16 ? by_layout<__nv_bfloat16, __nv_bfloat16, true>(p, interleaved, s)
                : by_layout<float, __nv_bfloat16, true>(p, interleaved, s);
}

}  // namespace bitnet
