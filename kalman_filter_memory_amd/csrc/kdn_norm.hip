// kdn_norm.hip -- RMS norm with the residual's addition, its output in the
// input's type or in 8 bits with a scale per 128 columns, and its backward.
//
//   s = round(x + residual)          (the residual stream, in its own type)
//   rstd = (mean_j s_j^2 + eps)^(-1/2),   y = s rstd w
//   8 bits: per 128 columns scale = max(max |y| (1 / 448), 2^-126), q = e4m3(y / scale)
// The norm is taken of s as stored, so that the backward, which reads the
// stored s, differentiates exactly what was computed; y is rounded once, from
// float32, also on its way to 8 bits.
//
// Backward, with xhat = s rstd and dn = dy w:
//   dx = rstd (dn - xhat mean_j(dn xhat)) + ds      (x's and the residual's gradient)
//   dw = sum over rows of dy xhat
//
// Everything here is bound by HBM: one pass, each row held in registers between
// its sum and its use.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kdn.h"
#include "kdn_norm.h"
#include "kdn_quant.h"

namespace {

using kdn::bf16_t;

constexpr int kThreads = 256;
constexpr int kMaxD = 16384;  // 256 threads x 8 vectors of 8 columns
constexpr int kMaxGroups = (1 << 24) - 1;  // a grid holds fewer than 2^32 threads

// sum over the TPR threads that share a row, returned to each of them.  A row
// of one wave needs no barrier; a row of the whole workgroup meets in LDS
// (red: two sets of four floats used in turn, so one barrier per call is enough).
template <int TPR> __device__ __forceinline__ float row_sum(float x, float* red) {
    x = kdn::group_sum<32>(x);
    x += __shfl_xor(x, 32, 64);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
        __syncthreads();
        x = (red[0] + red[1]) + (red[2] + red[3]);
    }
    return x;
}

// One row per TPR threads; thread t holds columns 8 (t + TPR v) .. + 7 of it.
// 16 neighbouring threads hold one block of 128 columns, so its maximum is four
// DPP steps.  A wave per row, up to 1024 columns, meets no barrier; wider rows
// would leave too few waves to hide the loads.
// 32768 x 2048 bfloat16 with residual to 8 bits: 83 us, 5.7 TB/s (above what a copy
// reaches, which writes more of its bytes); 1537 x 2056 float32 10.2 us (5.0 TB/s).  Bound
// by latency where there are few rows (256 of them: 3.1 us, a launch and the loads of x, of
// the residual and, behind the sum, of w, one after the other), and by lanes without a
// column where they are narrow (500000 x 64 without residual to 8 bits: 129 us, 0.8 TB/s,
// 8 of 64 lanes at work; 500000 x 128 129 us).
template <typename Ex, typename Er, bool RES, bool QUANT, int TPR, int NV>
__global__ __launch_bounds__(kThreads) void rms_norm_kernel(
    int rows, int d, float eps, const Ex* __restrict__ x, const Er* residual,
    const float* __restrict__ w, Ex* __restrict__ y, uint8_t* __restrict__ q,
    float* __restrict__ scale, Er* s_out, float* __restrict__ rstd_out) {
    __shared__ float red[4];
    const int t = threadIdx.x % TPR;
    const int row = int(blockIdx.x) * (kThreads / TPR) + int(threadIdx.x / TPR);
    if (TPR < kThreads && row >= rows) return;  // (whole waves; TPR == kThreads has exact grids)
    const size_t base = size_t(row) * d;
    float s[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = 8 * (t + TPR * v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[v][i] = 0.f;
        if (c < d) {
            kdn::load_vec<Ex, 8>(x + base + c, s[v]);
            if constexpr (RES) {
                float r[8];
                kdn::load_vec<Er, 8>(residual + base + c, r);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s[v][i] = kdn::to_f<Er>(kdn::from_f<Er>(s[v][i] + r[i]));
            }
        }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = 8 * (t + TPR * v);
        if constexpr (RES) {
            if (c < d) kdn::store8<Er>(s_out + base + c, s[v]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(s[v][i], s[v][i], ss);
    }
    ss = row_sum<TPR>(ss, red);
    const float rstd = 1.f / sqrtf(ss / float(d) + eps);
    if (rstd_out != nullptr && t == 0) rstd_out[row] = rstd;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = 8 * (t + TPR * v);
        const bool in = c < d;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.f;
        if (in) kdn::load_vec<float, 8>(w + c, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= s[v][i] * rstd;
        if constexpr (!QUANT) {
            if (in) kdn::store8<Ex>(y + base + c, f);
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = kdn::umax(m, kdn::abs_bits(f[i]));
            m = kdn::row_umax(in ? m : 0u);
            const float sc = kdn::quant_scale(m);
            if (in) {
                *reinterpret_cast<kdn::u32x2*>(q + base + c) = kdn::quant8(f, 1.0 / sc);
                if ((t & 15) == 0)
                    scale[size_t(row) * ((d + kdn::kQuantBlock - 1) / kdn::kQuantBlock) +
                          c / kdn::kQuantBlock] = sc;
            }
        }
    }
}

// Backward.  Each workgroup takes rows blockIdx.x RPB + (threads' row), then
// gridDim.x RPB further on; a thread keeps its columns' dw in registers over all
// of them and the workgroup writes one partial row of dw, which dw_kernel adds
// up in a fixed order (no atomics: the same inputs give the same bits).  1024
// workgroups leave 8 MB of partial rows at 2048 columns.
// 32768 x 2048 bfloat16: 152 us, 5 of them for dw, 5.3 TB/s.  Up to 4096 columns four waves
// or more share a SIMD; up to 8192 two (174 registers; 8192 x 8192 180 us, 4.5 TB/s), beyond
// that xh, dn and dw leave room for one, and the loads' latency shows (256 and 62 registers;
// 4096 x 16384 287 us, 2.8 TB/s).  500000 x 64, 8 of 64 lanes at work: 260 us, 1.5 TB/s.
template <typename Ex, typename Er, int TPR, int NV>
__global__ __launch_bounds__(kThreads) void rms_norm_bwd_kernel(
    int rows, int d, const Ex* __restrict__ dy, const Er* __restrict__ s,
    const float* __restrict__ w, const float* __restrict__ rstd, const float* ds, float* dx,
    float* __restrict__ part) {
    constexpr int RPB = kThreads / TPR;
    __shared__ float red[2][4];
    __shared__ float comb[RPB > 1 ? (RPB - 1) * TPR * 8 : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    float dw[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.f;
    int flip = 0;
    // every thread of the workgroup runs the same number of rounds when a row
    // spans it (RPB == 1), so the barrier in row_sum is met by all
    for (int64_t row = int64_t(blockIdx.x) * RPB + sub; row < rows;
         row += int64_t(gridDim.x) * RPB) {
        const size_t base = size_t(row) * d;
        const float r = rstd[row];
        float xh[NV][8], dn[NV][8];
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = 8 * (t + TPR * v);
#pragma unroll
            for (int i = 0; i < 8; ++i) xh[v][i] = dn[v][i] = 0.f;
            if (c < d) {
                kdn::load_vec<Er, 8>(s + base + c, xh[v]);
                kdn::load_vec<Ex, 8>(dy + base + c, dn[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = 8 * (t + TPR * v);
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = 0.f;
            if (c < d) kdn::load_vec<float, 8>(w + c, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xh[v][i] *= r;
                dw[v][i] = fmaf(dn[v][i], xh[v][i], dw[v][i]);
                dn[v][i] *= f[i];
                dot = fmaf(dn[v][i], xh[v][i], dot);
            }
        }
        const float mean = row_sum<TPR>(dot, red[flip]) / float(d);
        flip ^= 1;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = 8 * (t + TPR * v);
            if (c < d) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = 0.f;
                if (ds != nullptr) kdn::load_vec<float, 8>(ds + base + c, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] += r * (dn[v][i] - xh[v][i] * mean);
                kdn::store8<float>(dx + base + c, f);
            }
        }
    }
    // the workgroup's rows, in the order of its waves
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = 8 * (t + TPR * v);
        if constexpr (RPB > 1) {
            if (sub > 0)
#pragma unroll
                for (int i = 0; i < 8; ++i) comb[((sub - 1) * 8 + i) * TPR + t] = dw[v][i];
            __syncthreads();
            if (sub == 0)
                for (int o = 0; o < RPB - 1; ++o)
#pragma unroll
                    for (int i = 0; i < 8; ++i) dw[v][i] += comb[(o * 8 + i) * TPR + t];
            __syncthreads();
        }
        if (sub == 0 && c < d) kdn::store8<float>(part + size_t(blockIdx.x) * d + c, dw[v]);
    }
}

// dw = sum of n partial rows.  1024 threads over 32 columns: 128 groups of 8
// lanes (4 columns each) add every 128th row, then the groups meet in LDS.
__global__ __launch_bounds__(1024) void dw_kernel(int n, int d, const float* __restrict__ part,
                                                  float* __restrict__ dw) {
    __shared__ float acc[128][33];
    const int lane = threadIdx.x & 7, grp = threadIdx.x >> 3;
    const int c = blockIdx.x * 32 + 4 * lane;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < d) {
#pragma unroll 8
        for (int r = grp; r < n; r += 128) {
            const kdn::floatx4 p = *reinterpret_cast<const kdn::floatx4*>(part + size_t(r) * d + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] += p[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[grp][4 * lane + i] = a[i];
    __syncthreads();
    for (int h = 64; h > 0; h >>= 1) {  // 32 columns x h group pairs
        for (int k = threadIdx.x; k < 32 * h; k += 1024) acc[k >> 5][k & 31] += acc[(k >> 5) + h][k & 31];
        __syncthreads();
    }
    const int col = blockIdx.x * 32 + threadIdx.x;
    if (threadIdx.x < 32 && col < d) dw[col] = acc[0][threadIdx.x];
}

// x in 8 bits with a scale per 128 columns of one row: 16 lanes per block, one block
// per lane group, so that many workgroups hide the loads.  4099 x 2056 bfloat16:
// 6.1 us (4.2 TB/s).
template <typename E>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(
    size_t nblocks, int nb, int d, const E* __restrict__ x, uint8_t* __restrict__ q,
    float* __restrict__ scale) {
    const int l16 = threadIdx.x & 15;
    const size_t blk = size_t(blockIdx.x) * (kThreads / 16) + (threadIdx.x >> 4);
    const bool live = blk < nblocks;
    const size_t row = live ? blk / nb : 0;
    const int b = live ? int(blk - row * nb) : 0, c = kdn::kQuantBlock * b + 8 * l16;
    const bool in = live && c < d;
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.f;
    if (in) kdn::load_vec<E, 8>(x + row * d + c, f);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = kdn::umax(m, kdn::abs_bits(f[i]));
    const float sc = kdn::quant_scale(kdn::row_umax(m));
    if (in) *reinterpret_cast<kdn::u32x2*>(q + row * d + c) = kdn::quant8(f, 1.0 / sc);
    if (live && l16 == 0) scale[blk] = sc;
}

// the same with a scale per 128 x 128 block: one workgroup per block, the
// block's 8 vectors per thread held in registers between maximum and rounding.
// 6192 x 2048 bfloat16: 8.0 us (4.8 TB/s) in 784 workgroups.
template <typename E>
__global__ __launch_bounds__(kThreads) void quantize_block_kernel(
    int rows, int nb, int d, const E* __restrict__ x, uint8_t* __restrict__ q,
    float* __restrict__ scale) {
    __shared__ uint32_t red[4];
    const int l16 = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    const int br = blockIdx.x / nb, b = blockIdx.x % nb, c = kdn::kQuantBlock * b + 8 * l16;
    float f[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int64_t row = int64_t(br) * kdn::kQuantBlock + r0 + 16 * k;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[k][i] = 0.f;
        if (row < rows && c < d) kdn::load_vec<E, 8>(x + size_t(row) * d + c, f[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = kdn::umax(m, kdn::abs_bits(f[k][i]));
    m = kdn::row_umax(m);
    m = kdn::umax(m, __shfl_xor(m, 16, 64));
    m = kdn::umax(m, __shfl_xor(m, 32, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = kdn::umax(kdn::umax(red[0], red[1]), kdn::umax(red[2], red[3]));
    const float sc = kdn::quant_scale(m);
    const double inv = 1.0 / sc;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int64_t row = int64_t(br) * kdn::kQuantBlock + r0 + 16 * k;
        if (row < rows && c < d)
            *reinterpret_cast<kdn::u32x2*>(q + size_t(row) * d + c) = kdn::quant8(f[k], inv);
    }
    if (threadIdx.x == 0) scale[blockIdx.x] = sc;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool type_ok(int t) { return t == KDN_F32 || t == KDN_BF16; }

kdn_status check_norm(const kdn_norm_desc* n) {
    if (!n) return KDN_ERR_NULL;
    if (n->rows < 0 || n->d < 0 || !(n->eps >= 0.f)) return KDN_ERR_SHAPE;
    if (!type_ok(n->dtype) || !type_ok(n->residual_dtype)) return KDN_ERR_UNSUPPORTED;
    if (n->dtype == KDN_F32 && n->residual_dtype != KDN_F32) return KDN_ERR_UNSUPPORTED;
    if (n->d == 0 || n->d % 8 != 0 || n->d > kMaxD) return KDN_ERR_UNSUPPORTED;
    if (n->rows > kMaxGroups) return KDN_ERR_UNSUPPORTED;
    return KDN_OK;
}

// Threads per row: a wave, while the row fits a wave's registers; more for wide rows.
// (the rule by both sides, bfloat16, to 8 bits and backward: 32768 x 2048 94 and 163 us with
// a wave, 83 and 152 with four; 32768 x 1024 37 and 80 against 42 and 97)
bool wave_rows(int d) { return d <= 1024; }

struct NormArgs {
    int rows, d;
    float eps;
    const void *x, *residual;
    const float* w;
    void* y;
    uint8_t* q;
    float* scale;
    void* s;
    float* rstd;
};

template <typename Ex, typename Er, bool RES, bool QUANT, int TPR, int NV>
void norm_launch(const NormArgs& a, hipStream_t st) {
    constexpr int RPB = kThreads / TPR;
    rms_norm_kernel<Ex, Er, RES, QUANT, TPR, NV>
        <<<unsigned((int64_t(a.rows) + RPB - 1) / RPB), kThreads, 0, st>>>(
            a.rows, a.d, a.eps, static_cast<const Ex*>(a.x), static_cast<const Er*>(a.residual),
            a.w, static_cast<Ex*>(a.y), a.q, a.scale, static_cast<Er*>(a.s), a.rstd);
}

template <typename Ex, typename Er, bool RES, bool QUANT>
void norm_width(const NormArgs& a, hipStream_t st) {
    if (wave_rows(a.d)) {
        if (a.d <= 512) return norm_launch<Ex, Er, RES, QUANT, 64, 1>(a, st);
        return norm_launch<Ex, Er, RES, QUANT, 64, 2>(a, st);
    }
    if (a.d <= 2048) return norm_launch<Ex, Er, RES, QUANT, 256, 1>(a, st);
    if (a.d <= 4096) return norm_launch<Ex, Er, RES, QUANT, 256, 2>(a, st);
    if (a.d <= 8192) return norm_launch<Ex, Er, RES, QUANT, 256, 4>(a, st);
    return norm_launch<Ex, Er, RES, QUANT, 256, 8>(a, st);
}

template <bool QUANT> hipError_t norm_types(const kdn_norm_desc* n, const NormArgs& a, hipStream_t st) {
    const bool res = a.residual != nullptr;
    if (n->dtype == KDN_F32) {
        if (res) norm_width<float, float, true, QUANT>(a, st);
        else norm_width<float, float, false, QUANT>(a, st);
    } else if (!res) {
        norm_width<bf16_t, bf16_t, false, QUANT>(a, st);
    } else if (n->residual_dtype == KDN_BF16) {
        norm_width<bf16_t, bf16_t, true, QUANT>(a, st);
    } else {
        norm_width<bf16_t, float, true, QUANT>(a, st);
    }
    return hipGetLastError();
}

kdn_status norm_call(const kdn_norm_desc* n, const void* x, const void* residual, const float* w,
                     void* y, uint8_t* q, float* scale, void* s, float* rstd, bool quant,
                     void* stream) {
    const kdn_status st = check_norm(n);
    if (st != KDN_OK) return st;
    if (n->rows == 0) return KDN_OK;
    if (!x || !w || (quant ? !q || !scale : !y)) return KDN_ERR_NULL;
    if ((residual != nullptr) != (s != nullptr)) return KDN_ERR_NULL;
    for (const void* p : {x, residual, (const void*)w, (const void*)y, (const void*)q, (const void*)s})
        if (!aligned16(p)) return KDN_ERR_ALIGN;
    const NormArgs a{int(n->rows), n->d, n->eps, x, residual, w, y, q, scale, s, rstd};
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    const hipError_t e = quant ? norm_types<true>(n, a, hs) : norm_types<false>(n, a, hs);
    return e == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

// workgroups of the backward: enough to fill the GPU, few enough that their
// partial dw rows stay small beside the rows themselves (us, bfloat16, 512 and 1024: 1000 x
// 8192 25.3, 31.5; 2048 x 8192 39.5, 44.6; 4096 x 4096 36.8, 38.2; 16384 x 2048 97, 81;
// 32768 x 2048 186, 151)
int bwd_groups(const kdn_norm_desc* n) {
    const int rpb = wave_rows(n->d) ? 4 : 1;
    const int64_t units = (n->rows + rpb - 1) / rpb;
    return int(std::min<int64_t>(units, units < 4096 ? 512 : 1024));
}

struct BwdNormArgs {
    int rows, d, groups;
    const void *dy, *s;
    const float *w, *rstd, *ds;
    float *dx, *part;
};

template <typename Ex, typename Er, int TPR, int NV>
void bwd_launch(const BwdNormArgs& a, hipStream_t st) {
    rms_norm_bwd_kernel<Ex, Er, TPR, NV><<<a.groups, kThreads, 0, st>>>(
        a.rows, a.d, static_cast<const Ex*>(a.dy), static_cast<const Er*>(a.s), a.w, a.rstd, a.ds,
        a.dx, a.part);
}

template <typename Ex, typename Er> void bwd_width(const BwdNormArgs& a, hipStream_t st) {
    if (wave_rows(a.d)) {
        if (a.d <= 512) return bwd_launch<Ex, Er, 64, 1>(a, st);
        return bwd_launch<Ex, Er, 64, 2>(a, st);
    }
    if (a.d <= 2048) return bwd_launch<Ex, Er, 256, 1>(a, st);
    if (a.d <= 4096) return bwd_launch<Ex, Er, 256, 2>(a, st);
    if (a.d <= 8192) return bwd_launch<Ex, Er, 256, 4>(a, st);
    return bwd_launch<Ex, Er, 256, 8>(a, st);
}

}  // namespace

namespace kdn {
hipError_t launch_column_sums(int n, int d, const float* rows, float* out, hipStream_t st) {
    dw_kernel<<<(d + 31) / 32, 1024, 0, st>>>(n, d, rows, out);
    return hipGetLastError();
}
}  // namespace kdn

extern "C" {

kdn_status kdn_rms_norm(const kdn_norm_desc* n, const void* x, const void* residual,
                        const float* weight, void* y, void* s, float* rstd, void* stream) {
    return norm_call(n, x, residual, weight, y, nullptr, nullptr, s, rstd, false, stream);
}

kdn_status kdn_rms_norm_quant(const kdn_norm_desc* n, const void* x, const void* residual,
                              const float* weight, void* q, float* scale, void* s, float* rstd,
                              void* stream) {
    return norm_call(n, x, residual, weight, nullptr, static_cast<uint8_t*>(q), scale, s, rstd,
                     true, stream);
}

size_t kdn_rms_norm_backward_workspace_bytes(const kdn_norm_desc* n) {
    if (check_norm(n) != KDN_OK) return 0;
    return std::max<size_t>(size_t(bwd_groups(n)) * n->d * 4, 16);
}

kdn_status kdn_rms_norm_backward(const kdn_norm_desc* n, const void* dy, const void* s,
                                 const float* weight, const float* rstd, const float* ds,
                                 float* dx, float* dweight, void* ws, size_t ws_bytes,
                                 void* stream) {
    const kdn_status st = check_norm(n);
    if (st != KDN_OK) return st;
    if (!dweight || !ws) return KDN_ERR_NULL;
    if (n->rows > 0 && (!dy || !s || !weight || !rstd || !dx)) return KDN_ERR_NULL;
    if (ws_bytes < kdn_rms_norm_backward_workspace_bytes(n)) return KDN_ERR_WORKSPACE;
    for (const void* p : {dy, s, (const void*)weight, (const void*)ds, (const void*)dx, (const void*)ws})
        if (!aligned16(p)) return KDN_ERR_ALIGN;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    const BwdNormArgs a{int(n->rows), n->d, bwd_groups(n), dy, s, weight, rstd, ds,
                        dx, static_cast<float*>(ws)};
    if (n->rows > 0) {
        if (n->dtype == KDN_F32) bwd_width<float, float>(a, hs);
        else if (n->residual_dtype == KDN_BF16) bwd_width<bf16_t, bf16_t>(a, hs);
        else bwd_width<bf16_t, float>(a, hs);
        if (hipGetLastError() != hipSuccess) return KDN_ERR_HIP;
    }
    // (no rows: no partial rows, and dw is zero)
    dw_kernel<<<(n->d + 31) / 32, 1024, 0, hs>>>(a.groups, n->d, a.part, dweight);
    return hipGetLastError() == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

kdn_status kdn_quantize(const kdn_quant_desc* n, const void* x, void* q, float* scale,
                        void* stream) {
    if (!n) return KDN_ERR_NULL;
    if (n->rows < 0 || n->d < 0) return KDN_ERR_SHAPE;
    if (!type_ok(n->dtype) || (n->block_rows != 1 && n->block_rows != kdn::kQuantBlock))
        return KDN_ERR_UNSUPPORTED;
    if (n->d % 8 != 0 || n->rows > INT32_MAX) return KDN_ERR_UNSUPPORTED;
    const int nb = int((int64_t(n->d) + kdn::kQuantBlock - 1) / kdn::kQuantBlock);
    const int64_t br = (n->rows + n->block_rows - 1) / n->block_rows;
    const int64_t groups = n->block_rows == 1 ? (n->rows * nb + 15) / 16 : br * nb;
    if (groups > kMaxGroups) return KDN_ERR_UNSUPPORTED;
    if (n->rows == 0 || n->d == 0) return KDN_OK;
    if (!x || !q || !scale) return KDN_ERR_NULL;
    if (!aligned16(x) || !aligned16(q)) return KDN_ERR_ALIGN;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    const unsigned g = unsigned(groups);
    uint8_t* q8 = static_cast<uint8_t*>(q);
    const bool bf = n->dtype == KDN_BF16;
    const float* xf = static_cast<const float*>(x);
    const bf16_t* xb = static_cast<const bf16_t*>(x);
    if (n->block_rows == 1) {
        const size_t blocks = size_t(n->rows) * nb;
        if (bf) quantize_rows_kernel<bf16_t><<<g, kThreads, 0, hs>>>(blocks, nb, n->d, xb, q8, scale);
        else quantize_rows_kernel<float><<<g, kThreads, 0, hs>>>(blocks, nb, n->d, xf, q8, scale);
    } else {
        const int rows = int(n->rows);
        if (bf) quantize_block_kernel<bf16_t><<<g, kThreads, 0, hs>>>(rows, nb, n->d, xb, q8, scale);
        else quantize_block_kernel<float><<<g, kThreads, 0, hs>>>(rows, nb, n->d, xf, q8, scale);
    }
    return hipGetLastError() == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

}  // extern "C"
