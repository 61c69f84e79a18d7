// ssm_norm.cu -- layer norm over rows, optionally of a residual sum: forward and backward
// (include/ssm_scan.h, ssm_layer_norm_*).
//
//   s = x + residual;  mean, var over the row;  rstd = 1 / sqrt(var + eps)
//   y = (s - mean) rstd weight + bias
//
// A row lives in the registers of NT threads, CH vectors of VEC neighbouring columns each,
// from its one read to its one write; mean and variance take two passes over those
// registers (the squares are of centred values, so a row far from zero loses nothing).
#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/ssm_scan.h"
#include "ssm_device.cuh"

using namespace ssm;

namespace {

constexpr int kMaxDim = 16384;
constexpr int kBwdBlocksPerSm = 2;

// VEC neighbouring values of type T, as floats.
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float *f) {
    if constexpr (VEC == 1) {
        f[0] = Tok<T>::load(p);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < VEC; k += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + k);
            f[k] = v.x, f[k + 1] = v.y, f[k + 2] = v.z, f[k + 3] = v.w;
        }
    } else {
        static_assert(VEC == 8, "");
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) f[2 * k] = __uint_as_float(w[k] << 16), f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float *f) {
    if constexpr (VEC == 1) {
        *p = Tok<T>::from_f(f[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < VEC; k += 4) *reinterpret_cast<float4 *>(p + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
    } else {
        __nv_bfloat162 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(w);
    }
}

// Sums of N values over the NT threads of a row; the result is the same in every thread.
template <int NT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float *buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (NT > 32) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0)
            for (int k = 0; k < N; ++k) buf[k * 32 + warp] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            v[k] = 0.0f;
#pragma unroll
            for (int w = 0; w < NT / 32; ++w) v[k] += buf[k * 32 + w];
        }
    }
}

template <typename T>
struct NormFwd {
    int64_t rows;
    int dim;
    float eps;
    const T *x;
    const float *weight, *bias, *residual;
    T *y;
    float *s, *mean, *rstd;
};

template <typename T, int VEC, int CH, int NT>
__global__ void __launch_bounds__(NT < 128 ? 128 : NT) norm_fwd_kernel(const NormFwd<T> p) {
    constexpr int RPB = NT < 128 ? 128 / NT : 1;
    __shared__ float buf[2][32];
    const int tid = threadIdx.x % NT;
    const int64_t row = int64_t(blockIdx.x) * RPB + threadIdx.x / NT;
    if (row >= p.rows) return;  // whole warps; with NT > 32 whole blocks
    const int64_t o = row * p.dim;
    float f[CH][VEC];
    float sum[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * NT + tid) * VEC;
        if (col < p.dim) {
            load_vec<T, VEC>(p.x + o + col, f[c]);
            if (p.residual) {
                float r[VEC];
                load_vec<float, VEC>(p.residual + o + col, r);
#pragma unroll
                for (int k = 0; k < VEC; ++k) f[c][k] += r[k];
                store_vec<float, VEC>(p.s + o + col, f[c]);
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) sum[0] += f[c][k];
        }
    }
    row_sum<NT>(sum, buf[0]);
    const float mean = sum[0] / float(p.dim);
    float sq[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if ((c * NT + tid) * VEC < p.dim)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                f[c][k] -= mean;
                sq[0] = fmaf(f[c][k], f[c][k], sq[0]);
            }
    row_sum<NT>(sq, buf[1]);
    const float rstd = rsqrtf(sq[0] / float(p.dim) + p.eps);
    if (tid == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * NT + tid) * VEC;
        if (col < p.dim) {
            float w[VEC], b[VEC];
            load_vec<float, VEC>(p.weight + col, w);
            if (p.bias) load_vec<float, VEC>(p.bias + col, b);
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[c][k] = fmaf(f[c][k] * rstd, w[k], p.bias ? b[k] : 0.0f);
            store_vec<T, VEC>(p.y + o + col, f[c]);
        }
    }
}

// The input of the norm is of type S: the tokens' own without a residual, float32 with one.
template <typename T, typename S>
struct NormBwd {
    int64_t rows;
    int dim, groups;
    const S *s;
    const T *dy;
    const float *weight, *mean, *rstd, *ds_out;
    T *dx;
    float *dres, *part_w, *part_b;
};

// ds = rstd (g - mean(g) - xh mean(g xh)) + ds_out with g = dy weight, xh = (s - mean) rstd.
// Each group of NT threads walks rows group, group + groups, ... and keeps the columns'
// sums of dy xh and dy in registers; it leaves them as one row of the parts.
template <typename T, typename S, int VEC, int CH, int NT>
__global__ void __launch_bounds__(NT < 128 ? 128 : NT) norm_bwd_kernel(const NormBwd<T, S> p) {
    constexpr int RPB = NT < 128 ? 128 / NT : 1;
    __shared__ float buf[2][64];
    const int tid = threadIdx.x % NT;
    const int64_t group = int64_t(blockIdx.x) * RPB + threadIdx.x / NT;
    float aw[CH][VEC] = {}, ab[CH][VEC] = {};
    int flip = 0;
    for (int64_t row = group < p.groups ? group : p.rows; row < p.rows; row += p.groups) {
        const int64_t o = row * p.dim;
        const float mean = p.mean[row], rstd = p.rstd[row];
        float xh[CH][VEC], g[CH][VEC];
        float sums[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * NT + tid) * VEC;
            if (col < p.dim) {
                float w[VEC];
                load_vec<S, VEC>(p.s + o + col, xh[c]);
                load_vec<T, VEC>(p.dy + o + col, g[c]);
                load_vec<float, VEC>(p.weight + col, w);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    xh[c][k] = (xh[c][k] - mean) * rstd;
                    aw[c][k] = fmaf(g[c][k], xh[c][k], aw[c][k]);
                    ab[c][k] += g[c][k];
                    g[c][k] *= w[k];
                    sums[0] += g[c][k];
                    sums[1] = fmaf(g[c][k], xh[c][k], sums[1]);
                }
            }
        }
        row_sum<NT>(sums, buf[flip]);
        flip ^= 1;
        const float m0 = sums[0] / float(p.dim), m1 = sums[1] / float(p.dim);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * NT + tid) * VEC;
            if (col < p.dim) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) g[c][k] = rstd * (g[c][k] - m0 - xh[c][k] * m1);
                if (p.ds_out) {
                    float r[VEC];
                    load_vec<float, VEC>(p.ds_out + o + col, r);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) g[c][k] += r[k];
                }
                store_vec<T, VEC>(p.dx + o + col, g[c]);
                if (p.dres) store_vec<float, VEC>(p.dres + o + col, g[c]);
            }
        }
    }
    if (group < p.groups)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * NT + tid) * VEC;
            if (col < p.dim) {
                store_vec<float, VEC>(p.part_w + group * p.dim + col, aw[c]);
                if (p.part_b) store_vec<float, VEC>(p.part_b + group * p.dim + col, ab[c]);
            }
        }
}

// Column sums of the parts, in a fixed order (blockIdx.y: weight, bias).
__global__ void __launch_bounds__(256)
    norm_parts_kernel(int groups, int dim, const float *__restrict__ part_w, const float *__restrict__ part_b,
                      float *__restrict__ dweight, float *__restrict__ dbias) {
    __shared__ float s[8][32];
    const float *part = blockIdx.y ? part_b : part_w;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    float t = 0.0f;
    if (col < dim)
#pragma unroll 8
        for (int k = warp; k < groups; k += 8) t += part[int64_t(k) * dim + col];
    s[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && col < dim) {
        t = 0.0f;
        for (int w = 0; w < 8; ++w) t += s[w][lane];
        (blockIdx.y ? dbias : dweight)[col] = t;
    }
}

// ---------------------------------------------------------------------- host
inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }
ssm_status launched() { return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA; }

// The smallest of these splits of a row that holds its vectors.
#define SSM_ROW_SPLIT(vectors, F)          \
    if ((vectors) <= 32) F(1, 32);         \
    else if ((vectors) <= 128) F(4, 32);   \
    else if ((vectors) <= 256) F(2, 128);  \
    else if ((vectors) <= 512) F(2, 256);  \
    else if ((vectors) <= 1024) F(4, 256); \
    else if ((vectors) <= 2048) F(4, 512); \
    else if ((vectors) <= 4096) F(4, 1024);\
    else F(16, 1024)

// Groups of threads the backward's rows are dealt to.
int64_t bwd_groups(int64_t rows, int64_t sms) { return std::max<int64_t>(1, std::min<int64_t>(rows, sms * kBwdBlocksPerSm * 4)); }

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return n;
}

template <typename T, int VEC>
ssm_status run_fwd(const NormFwd<T> &p, cudaStream_t st) {
#define SSM_GO(CH, NT) norm_fwd_kernel<T, VEC, CH, NT><<<unsigned(ceil_div(p.rows, NT < 128 ? 128 / NT : 1)), NT < 128 ? 128 : NT, 0, st>>>(p)
    const int nv = p.dim / VEC;
    SSM_ROW_SPLIT(nv, SSM_GO);
#undef SSM_GO
    return launched();
}

template <typename T, typename S, int VEC>
ssm_status run_bwd(NormBwd<T, S> p, float *dweight, float *dbias, cudaStream_t st) {
#define SSM_GO(CH, NT) norm_bwd_kernel<T, S, VEC, CH, NT><<<unsigned(ceil_div(p.groups, NT < 128 ? 128 / NT : 1)), NT < 128 ? 128 : NT, 0, st>>>(p)
    const int nv = p.dim / VEC;
    SSM_ROW_SPLIT(nv, SSM_GO);
#undef SSM_GO
    norm_parts_kernel<<<dim3(unsigned(ceil_div(p.dim, 32)), dbias ? 2 : 1), 256, 0, st>>>(p.groups, p.dim, p.part_w, p.part_b, dweight, dbias);
    return launched();
}

ssm_status check_sizes(int64_t rows, int64_t dim, ssm_dtype dtype) {
    if (rows < 0 || dim < 0 || (dtype != SSM_F32 && dtype != SSM_BF16)) return SSM_ERR_INVALID;
    return (dim > kMaxDim || rows > INT_MAX) ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

}  // namespace

extern "C" {

ssm_status ssm_layer_norm_fwd(const ssm_norm_args *a, void *stream) {
    if (!a) return SSM_ERR_INVALID;
    const ssm_status ok = check_sizes(a->rows, a->dim, a->dtype);
    if (ok != SSM_OK) return ok;
    if (!(a->eps >= 0.0f) || a->eps > FLT_MAX) return SSM_ERR_INVALID;
    if (a->rows == 0 || a->dim == 0) return SSM_OK;
    if (!a->x || !a->weight || !a->y || (a->residual == nullptr) != (a->residual_out == nullptr)) return SSM_ERR_INVALID;
    const size_t es = a->dtype == SSM_BF16 ? 2 : 4;
    if (!aligned(a->x, es) || !aligned(a->y, es)) return SSM_ERR_UNSUPPORTED;
    const int vec = a->dtype == SSM_BF16 ? 8 : 4;
    bool wide = a->dim % vec == 0 && aligned(a->x, 16) && aligned(a->y, 16);
    for (const float *q : {a->weight, a->bias, a->residual, static_cast<const float *>(a->residual_out)}) {
        if (!aligned(q, 4)) return SSM_ERR_UNSUPPORTED;
        wide = wide && aligned(q, 16);
    }
    if (!aligned(a->mean, 4) || !aligned(a->rstd, 4)) return SSM_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
#define SSM_RUN(T, VEC)                                                                                          \
    run_fwd<T, VEC>({a->rows, int(a->dim), a->eps, static_cast<const T *>(a->x), a->weight, a->bias, a->residual, \
                     static_cast<T *>(a->y), a->residual_out, a->mean, a->rstd}, st)
    if (a->dtype == SSM_BF16) return wide ? SSM_RUN(__nv_bfloat16, 8) : SSM_RUN(__nv_bfloat16, 1);
    return wide ? SSM_RUN(float, 4) : SSM_RUN(float, 1);
#undef SSM_RUN
}

size_t ssm_layer_norm_bwd_workspace_size(const ssm_norm_bwd_args *a) {
    if (!a || check_sizes(a->rows, a->dim, a->dtype) != SSM_OK || a->rows == 0 || a->dim == 0) return 0;
    // for the largest grid any GPU of this architecture takes (148 SMs here)
    return 2 * up256(size_t(bwd_groups(a->rows, 160)) * size_t(a->dim) * 4);
}

ssm_status ssm_layer_norm_bwd(const ssm_norm_bwd_args *a, void *stream) {
    if (!a) return SSM_ERR_INVALID;
    const ssm_status ok = check_sizes(a->rows, a->dim, a->dtype);
    if (ok != SSM_OK) return ok;
    if (a->dim == 0) return SSM_OK;
    if (!a->dweight) return SSM_ERR_INVALID;
    if (a->rows > 0 && (!a->s || !a->dy || !a->weight || !a->mean || !a->rstd || !a->dx)) return SSM_ERR_INVALID;
    const size_t es = a->dtype == SSM_BF16 ? 2 : 4;
    const int vec = a->dtype == SSM_BF16 ? 8 : 4;
    if (!aligned(a->dy, es) || !aligned(a->dx, es) || !aligned(a->s, a->has_residual ? 4 : es)) return SSM_ERR_UNSUPPORTED;
    bool wide = a->dim % vec == 0 && aligned(a->dy, 16) && aligned(a->dx, 16) && aligned(a->s, 16);
    for (const float *q : {a->weight, a->dresidual_out, static_cast<const float *>(a->dresidual)}) {
        if (!aligned(q, 4)) return SSM_ERR_UNSUPPORTED;
        wide = wide && aligned(q, 16);
    }
    for (const float *q : {a->mean, a->rstd, static_cast<const float *>(a->dweight), static_cast<const float *>(a->dbias)})
        if (!aligned(q, 4)) return SSM_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->rows == 0) {
        if (cudaMemsetAsync(a->dweight, 0, size_t(a->dim) * 4, st) != cudaSuccess) return SSM_ERR_CUDA;
        if (a->dbias && cudaMemsetAsync(a->dbias, 0, size_t(a->dim) * 4, st) != cudaSuccess) return SSM_ERR_CUDA;
        return SSM_OK;
    }
    if (!a->workspace || a->workspace_bytes < ssm_layer_norm_bwd_workspace_size(a)) return SSM_ERR_INVALID;
    if (!aligned(a->workspace, 16)) return SSM_ERR_UNSUPPORTED;
    const int sms = sm_count();
    if (sms <= 0) return SSM_ERR_CUDA;
    const int groups = int(bwd_groups(a->rows, std::min(sms, 160)));
    float *pw = static_cast<float *>(a->workspace);
    float *pb = a->dbias ? reinterpret_cast<float *>(static_cast<unsigned char *>(a->workspace) + up256(size_t(groups) * size_t(a->dim) * 4)) : nullptr;
#define SSM_RUN(T, S, VEC)                                                                                         \
    run_bwd<T, S, VEC>({a->rows, int(a->dim), groups, static_cast<const S *>(a->s), static_cast<const T *>(a->dy), \
                        a->weight, a->mean, a->rstd, a->dresidual_out, static_cast<T *>(a->dx), a->dresidual, pw, pb}, \
                       a->dweight, a->dbias, st)
    if (a->dtype == SSM_F32) return wide ? SSM_RUN(float, float, 4) : SSM_RUN(float, float, 1);
    if (a->has_residual) return wide ? SSM_RUN(__nv_bfloat16, float, 8) : SSM_RUN(__nv_bfloat16, float, 1);
    return wide ? SSM_RUN(__nv_bfloat16, __nv_bfloat16, 8) : SSM_RUN(__nv_bfloat16, __nv_bfloat16, 1);
#undef SSM_RUN
}

}  // extern "C"
