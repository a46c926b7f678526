// Gradient of RMSNorm with a residual branch (sm_100a).
//
// Forward, per token: y_k = h_k r w_k with r = (mean_j h_j^2 + eps)^(-1/2),
// quantised to int8 with a straight-through gradient; h also runs on as the
// residual stream.  With g = dL/dy, e_k = g_k w_k and u_k = h_k r:
//   dh_k = r (e_k - u_k (1/K) sum_j e_j u_j) + dR_k,   dw_k = sum_t g_k u_k.
// r is the forward's (rinv).  All sums are fp32; dh is rounded once.
//
// Rows of up to 12288 are touched once: a CTA takes whole rows (its threads hold the
// row's 16-byte chunks in registers between the dot product and the result)
// and walks over rows blockIdx.x, + gridDim.x, ..., keeping its columns' dw in
// registers.  A second launch adds the CTAs' dw rows in a fixed order, so dw
// does not depend on timing.  Bound: HBM for many rows (8191 x 4096 with an fp32
// dY 47 us, 5.7 TB/s); 2048 x 3200 with a residual branch takes 15.3 us, about 3
// of them the second launch.  Longer rows are read twice, and a third time for
// dw: 4096 x 16384 with a residual branch 173 us, a floor of 82 (4096 x 12288: 86, 62).
#include "common.cuh"
#include "kernels.h"

namespace bitnet {

namespace {

// eight values of a row at chunk c, widened to fp32
__device__ __forceinline__ void load8(const __nv_bfloat16 *row, int c, float *f) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(row) + c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *row, int c, float *f) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(row) + 2 * c);
    const float4 b = __ldg(reinterpret_cast<const float4 *>(row) + 2 * c + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
// the same in two steps: eight values as they lie in memory (plain loads: dH may be dR), and their fp32 values
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *row, int c) { u = reinterpret_cast<const uint4 *>(row)[c]; }
    __device__ __forceinline__ void widen(float *f) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *row, int c) {
        a = reinterpret_cast<const float4 *>(row)[2 * c];
        b = reinterpret_cast<const float4 *>(row)[2 * c + 1];
    }
    __device__ __forceinline__ void widen(float *f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *row, int c, const float *f) {
    reinterpret_cast<uint4 *>(row)[c] =
        make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ void store8(float *row, int c, const float *f) {
    reinterpret_cast<float4 *>(row)[2 * c] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(row)[2 * c + 1] = make_float4(f[4], f[5], f[6], f[7]);
}

// CPT chunks of 8 columns per thread; the row's K / 8 chunks lie at threadIdx.x
// + j blockDim.x.  dwp: [gridDim.x, K] partial dw rows, or NULL.
template <typename TY, typename TG, int CPT, int THREADS>
__global__ void __launch_bounds__(THREADS) k_rmsnorm_grad(const TY *__restrict__ dY, const __nv_bfloat16 *__restrict__ H,
                                                      const float *__restrict__ w, const float *__restrict__ rinv,
                                                      const TG *dR, TG *dH, float *__restrict__ dwp, int T, int K) {
    __shared__ float s_red[2][32];
    const int nchunk = K >> 3;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const float inv_k = 1.0f / static_cast<float>(K);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    float dw[CPT][8];
#pragma unroll
    for (int j = 0; j < CPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
    // The next row is on its way while this one is worked on, where its words leave the registers room: two chunks with a
    // 16-bit side spill up to 60 bytes and gain all the same, with both sides in fp32 they spill 128 and lose, three chunks
    // lose throughout (4096 rows, without / with, us: 8640 bf16 72.7 / 55.9, fp32 dY 70.8 / 65.8, both fp32 117 / 129;
    // 12288 86 / 114, both fp32 155 / 207).
    constexpr bool kAhead = CPT * (sizeof(TY) + sizeof(TG) + 2) <= 16;
    Raw8<TY> ny[CPT];
    Raw8<__nv_bfloat16> nh[CPT];
    Raw8<TG> nr[CPT];
    float next_r = 0.0f;
    // rows are counted without a sign: T < 2^31 and a step further does not overflow
    const unsigned rows = T;
    auto fetch = [&](unsigned t) {
        const int64_t base = static_cast<int64_t>(t) * K;
        next_r = __ldg(rinv + t);
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < nchunk) {
                ny[j].load(dY + base, c);
                nh[j].load(H + base, c);
                if (dR) nr[j].load(dR + base, c);
            }
        }
    };
    if (kAhead && blockIdx.x < rows) fetch(blockIdx.x);
    int flip = 0;
    for (unsigned t = blockIdx.x; t < rows; t += gridDim.x) {
        const int64_t base = static_cast<int64_t>(t) * K;
        if (!kAhead) fetch(t);
        const float r = next_r;
        float e[CPT][8], u[CPT][8];
        Raw8<TG> res[CPT];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            if (static_cast<int>(threadIdx.x + j * blockDim.x) < nchunk) {
                ny[j].widen(e[j]);
                nh[j].widen(u[j]);
                res[j] = nr[j];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) e[j][i] = u[j][i] = 0.0f;
            }
        }
        if (kAhead && t + gridDim.x < rows) fetch(t + gridDim.x);
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            float wv[8];
            if (w && c < nchunk) {
                load8(w, c, wv);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) wv[i] = 1.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                u[j][i] *= r;
                dw[j][i] = fmaf(e[j][i], u[j][i], dw[j][i]);
                e[j][i] *= wv[i];
                dot = fmaf(e[j][i], u[j][i], dot);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) s_red[flip][warp] = dot;
        __syncthreads();   // two buffers: a warp reaches the next row's write only after all have passed this row's barrier
        float sum = lane < nw ? s_red[flip][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum *= inv_k;
        flip ^= 1;
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < nchunk) {
                float d[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] = r * fmaf(-u[j][i], sum, e[j][i]);
                if (dR) {
                    float q[8];
                    res[j].widen(q);
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] += q[i];
                }
                store8(dH + base, c, d);
            }
        }
    }
    if (dwp) {
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            if (c < nchunk) store8(dwp + static_cast<int64_t>(blockIdx.x) * K, c, dw[j]);
        }
    }
}

// Rows longer than the register form holds: one CTA per row, the row read twice
// (the second time from L2).
template <typename TY, typename TG>
__global__ void __launch_bounds__(512) k_rmsnorm_grad_long(const TY *__restrict__ dY, const __nv_bfloat16 *__restrict__ H,
                                                           const float *__restrict__ w, const float *__restrict__ rinv,
                                                           const TG *dR, TG *dH, int K) {
    __shared__ float s_red[16];
    const int nchunk = K >> 3;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t base = static_cast<int64_t>(blockIdx.x) * K;
    const float r = __ldg(rinv + blockIdx.x);
    float dot = 0.0f;
    for (int c = threadIdx.x; c < nchunk; c += blockDim.x) {
        float e[8], u[8], wv[8];
        load8(dY + base, c, e);
        load8(H + base, c, u);
        if (w) load8(w, c, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(w ? e[i] * wv[i] : e[i], u[i] * r, dot);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) s_red[warp] = dot;
    __syncthreads();
    float sum = lane < static_cast<int>(blockDim.x >> 5) ? s_red[lane] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sum = __shfl_sync(0xffffffffu, sum, 0) / static_cast<float>(K);
    for (int c = threadIdx.x; c < nchunk; c += blockDim.x) {
        float e[8], u[8], wv[8], d[8];
        load8(dY + base, c, e);
        load8(H + base, c, u);
        if (w) load8(w, c, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = r * fmaf(-(u[i] * r), sum, w ? e[i] * wv[i] : e[i]);
        if (dR) {
            float q[8];
            Raw8<TG> raw;
            raw.load(dR + base, c);
            raw.widen(q);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] += q[i];
        }
        store8(dH + base, c, d);
    }
}

// dw partial rows of long rows: CTA (x, y) sums rows y, y + gridDim.y, ... of its 8 blockDim.x columns.
template <typename TY>
__global__ void __launch_bounds__(256) k_rmsnorm_dw(const TY *__restrict__ dY, const __nv_bfloat16 *__restrict__ H,
                                                    const float *__restrict__ rinv, float *__restrict__ dwp, int T, int K) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= (K >> 3)) return;
    float dw[8] = {};
    for (unsigned t = blockIdx.y; t < static_cast<unsigned>(T); t += gridDim.y) {
        const int64_t base = static_cast<int64_t>(t) * K;
        const float r = __ldg(rinv + t);
        float e[8], u[8];
        load8(dY + base, c, e);
        load8(H + base, c, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] = fmaf(e[i], u[i] * r, dw[i]);
    }
    store8(dwp + static_cast<int64_t>(blockIdx.y) * K, c, dw);
}

// dw[k] (+)= sum over n partial rows, in order: 32 columns per CTA, warp y adds
// rows y, y + 32, ..., then the 32 warp sums are added in order.
__global__ void __launch_bounds__(1024) k_rmsnorm_dw_sum(const float *__restrict__ dwp, int n, int K, float *dw,
                                                         int accumulate) {
    __shared__ float s_sum[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int k = blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (k < K)
        for (int i = threadIdx.y; i < n; i += 32) s += dwp[static_cast<int64_t>(i) * K + k];
    s_sum[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && k < K) {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) a += s_sum[i][threadIdx.x];
        dw[k] = accumulate ? dw[k] + a : a;
    }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t s, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Chunks per thread and threads of the row kernel (0 chunks: rows too long for it).
int chunks_per_thread(int64_t nchunk, int *threads) {
    const int cpt = nchunk <= 1024 ? 1 : nchunk <= 1152 ? 2 : nchunk <= 1536 ? 3 : 0;
    *threads = cpt ? static_cast<int>((nchunk + cpt - 1) / cpt + 31) / 32 * 32 : 512;
    return cpt;
}

// CTAs of the row kernel, each with a partial dw row: as many as fit an SM's registers with about 1024 threads, eight at
// most (more of them cost more in partial rows than they hide: 4 instead of 2 per SM at K = 4096 53.1 against 48.8 us).
int partial_rows(int64_t T, int64_t K) {
    int threads;
    const int cpt = chunks_per_thread(K / 8, &threads);
    int per_sm = cpt > 1 ? 1 : 1024 / threads;
    per_sm = per_sm < 1 ? 1 : per_sm > 8 ? 8 : per_sm;
    const int64_t most = static_cast<int64_t>(per_sm) * num_sms();
    return static_cast<int>(T < most ? T : most);
}

template <typename TY, typename TG>
cudaError_t grad_launch(const TY *dY, const __nv_bfloat16 *H, const float *w, const float *rinv, const TG *dR, int T, int K,
                        TG *dH, float *dwp, cudaStream_t s) {
    const int nchunk = K / 8, rows = partial_rows(T, K);
    int threads;
    switch (chunks_per_thread(nchunk, &threads)) {
        case 1:   // 65536 / 512 registers a thread measured better than 65536 / 1024 wherever they do: 47.2 / 49.6 us at 8191 x 4096
            if (threads <= 512) return launch_pdl(k_rmsnorm_grad<TY, TG, 1, 512>, dim3(rows), dim3(threads), s, dY, H, w, rinv, dR, dH, dwp, T, K);
            return launch_pdl(k_rmsnorm_grad<TY, TG, 1, 1024>, dim3(rows), dim3(threads), s, dY, H, w, rinv, dR, dH, dwp, T, K);
        case 2: return launch_pdl(k_rmsnorm_grad<TY, TG, 2, 576>, dim3(rows), dim3(threads), s, dY, H, w, rinv, dR, dH, dwp, T, K);
        case 3: return launch_pdl(k_rmsnorm_grad<TY, TG, 3, 512>, dim3(rows), dim3(threads), s, dY, H, w, rinv, dR, dH, dwp, T, K);
    }
    cudaError_t e = launch_pdl(k_rmsnorm_grad_long<TY, TG>, dim3(T), dim3(512), s, dY, H, w, rinv, dR, dH, K);
    if (e != cudaSuccess || !dwp) return e;
    return launch_pdl(k_rmsnorm_dw<TY>, dim3((nchunk + 255) / 256, rows), dim3(256), s, dY, H, rinv, dwp, T, K);
}

}  // namespace

// status word, then one partial dw row per CTA of the row kernel
size_t rmsnorm_grad_ws_bytes(int64_t T, int64_t K) {
    if (T <= 0 || K <= 0) return 256;
    return static_cast<size_t>(partial_rows(T, K)) * static_cast<size_t>(K) * 4 + 256;
}

cudaError_t launch_rmsnorm_grad(const void *dY, bool dy_bf16, const void *H, const float *w, const float *rinv,
                                const void *dR, bool g_bf16, int64_t T, int64_t K, void *dH, float *dw, bool accumulate,
                                void *ws, cudaStream_t s) {
    float *dwp = dw ? reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + 256) : nullptr;
    const auto *h = static_cast<const __nv_bfloat16 *>(H);
    const int t = static_cast<int>(T), k = static_cast<int>(K);
    cudaError_t e;
    if (dy_bf16) {
        const auto *g = static_cast<const __nv_bfloat16 *>(dY);
        e = g_bf16 ? grad_launch(g, h, w, rinv, static_cast<const __nv_bfloat16 *>(dR), t, k, static_cast<__nv_bfloat16 *>(dH), dwp, s)
                   : grad_launch(g, h, w, rinv, static_cast<const float *>(dR), t, k, static_cast<float *>(dH), dwp, s);
    } else {
        const auto *g = static_cast<const float *>(dY);
        e = g_bf16 ? grad_launch(g, h, w, rinv, static_cast<const __nv_bfloat16 *>(dR), t, k, static_cast<__nv_bfloat16 *>(dH), dwp, s)
                   : grad_launch(g, h, w, rinv, static_cast<const float *>(dR), t, k, static_cast<float *>(dH), dwp, s);
    }
    if (e != cudaSuccess || !dw) return e;
    return launch_pdl(k_rmsnorm_dw_sum, dim3((k + 31) / 32), dim3(32, 32), s, dwp, partial_rows(T, K), k, dw, accumulate ? 1 : 0);
}

}  // namespace bitnet
