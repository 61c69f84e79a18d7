// ssm_norm.cu -- layer norm over rows, optionally of a residual sum: forward and backward
// (include/ssm_scan.h, ssm_layer_norm_*).
//
//   s = x + residual;  mean, var over the row;  rstd = 1 / sqrt(var + eps)
//   y = (s - mean) rstd weight + bias
//
// A row lives in the registers of a group of warps, CH vectors of VEC neighbouring columns in
// each thread, from its one read to its one write; mean and variance take two passes over
// those registers (the squares are of centred values, so a row far from zero keeps its variance).
// Bound by memory: 32768 x 2048 bfloat16 with a residual forward in 127 us (6.3 TB/s), backward in 184 us (5.8
// TB/s), float32 165 and 178 us (6.5 and 6.0 TB/s), without one 88 and 133 us (6.1 and 6.1 TB/s). bfloat16 without a residual
// takes 66 us (4.1 TB/s) and 82 us (4.9 TB/s): two bytes a column, and only the rows in registers are on their way.
#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "../../include/ssm_scan.h"
#include "ssm_device.cuh"

using namespace ssm;

namespace {

constexpr int kMaxDim = 16384;
constexpr int kOneWarpGroups = 4;   // groups of a block whose rows take one warp each
constexpr int kMostWarps = 16;      // of a row that takes more than one
constexpr int kMostGroups = 2560;   // of the backward: rows of partial sums

// The widest access for a piece of so many bytes (16 at most).
template <int BYTES>
struct Word;
template <>
struct Word<2> { using type = unsigned short; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<16> { using type = uint4; };

// VEC neighbouring values of type T as they lie in memory, and as floats.
template <typename T, int VEC>
struct Raw {
    static constexpr int BYTES = VEC * int(sizeof(T)), PIECE = BYTES < 16 ? BYTES : 16, N = BYTES / PIECE;
    using W = typename Word<PIECE>::type;
    W w[N];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int n = 0; n < N; ++n) w[n] = reinterpret_cast<const W *>(p)[n];
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int n = 0; n < N; ++n) reinterpret_cast<W *>(p)[n] = w[n];
    }
    // 32 bits: two bfloat16 or a float
    static __device__ __forceinline__ void split(uint32_t v, float *f) {
        if constexpr (sizeof(T) == 2)
            f[0] = __uint_as_float(v << 16), f[1] = __uint_as_float(v & 0xffff0000u);
        else
            f[0] = __uint_as_float(v);
    }
    static __device__ __forceinline__ uint32_t join(const float *f) {
        if constexpr (sizeof(T) == 2) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[0], f[1]);
            return *reinterpret_cast<const uint32_t *>(&v);
        } else {
            return __float_as_uint(f[0]);
        }
    }
    __device__ __forceinline__ void get(float (&f)[VEC]) const {
        constexpr int S = 4 / sizeof(T);  // values in 32 bits
        if constexpr (PIECE == 2) {
            f[0] = __uint_as_float(uint32_t(w[0]) << 16);
        } else {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float *q = f + n * (PIECE / int(sizeof(T)));
                if constexpr (PIECE == 4) {
                    split(w[n], q);
                } else if constexpr (PIECE == 8) {
                    split(w[n].x, q), split(w[n].y, q + S);
                } else {
                    split(w[n].x, q), split(w[n].y, q + S), split(w[n].z, q + 2 * S), split(w[n].w, q + 3 * S);
                }
            }
        }
    }
    __device__ __forceinline__ void set(const float (&f)[VEC]) {
        constexpr int S = 4 / sizeof(T);
        if constexpr (PIECE == 2) {
            w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
        } else {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const float *q = f + n * (PIECE / int(sizeof(T)));
                if constexpr (PIECE == 4)
                    w[n] = join(q);
                else if constexpr (PIECE == 8)
                    w[n] = make_uint2(join(q), join(q + S));
                else
                    w[n] = make_uint4(join(q), join(q + S), join(q + 2 * S), join(q + 3 * S));
            }
        }
    }
};

// Sums of N values over the group's warps, the same in every thread; buf holds the warps' sums and
// is free again after the group's next sum.
template <bool ONE, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*buf)[32], const int warps) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (!ONE) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) buf[k][warp] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = 0.0f;
#pragma unroll 4
        for (int w = 0; w < warps; ++w)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += buf[k][w];
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

// ONE: a group is a warp, kOneWarpGroups of them to a block; else a block is a group. RES: with a residual; then a
// group takes one row (ten bytes a column in flight are enough, and many small blocks keep more rows
// in flight than fewer that stay: 127 against 134 us for 32768 x 2048). Tokens alone are two bytes a column: there the groups
// stay and walk the rows, weight and bias in registers and two rows on their way.
template <typename T, int VEC, int CH, bool ONE, bool RES>
__global__ void __launch_bounds__(32 * (ONE ? kOneWarpGroups : kMostWarps)) norm_fwd_kernel(const NormFwd<T> p) {
    constexpr bool KEEP = !RES && CH * VEC <= 16;  // weight and bias in registers
    constexpr int SLOTS = KEEP ? 2 : 1;
    __shared__ float buf[2][1][32];
    const int threads = ONE ? 32 : blockDim.x, tid = ONE ? threadIdx.x & 31 : threadIdx.x;
    const int64_t groups = ONE ? int64_t(gridDim.x) * kOneWarpGroups : gridDim.x;
    int64_t row = ONE ? int64_t(blockIdx.x) * kOneWarpGroups + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= p.rows) return;  // whole groups
    Raw<T, VEC> x[SLOTS][CH];
    Raw<float, VEC> r[RES ? CH : 1];
    const auto fetch = [&](const int64_t k, Raw<T, VEC>(&to)[CH]) {
        if (k >= p.rows) return;
        const int64_t o = k * p.dim;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * threads + tid) * VEC;
            if (col < p.dim) {
                to[c].load(p.x + o + col);
                if constexpr (RES) r[c].load(p.residual + o + col);
            }
        }
    };
#pragma unroll
    for (int q = 0; q < SLOTS; ++q) fetch(row + q * groups, x[q]);
    float w[KEEP ? CH : 1][VEC], b[KEEP ? CH : 1][VEC];
    const auto params = [&](const int col, float (&wv)[VEC], float (&bv)[VEC]) {
        Raw<float, VEC> v;
        v.load(p.weight + col);
        v.get(wv);
        if (p.bias) {
            v.load(p.bias + col);
            v.get(bv);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) bv[k] = 0.0f;
        }
    };
    if constexpr (KEEP) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if ((c * threads + tid) * VEC < p.dim) params((c * threads + tid) * VEC, w[c], b[c]);
    }
    const float inv = 1.0f / float(p.dim);
    for (;;) {
#pragma unroll
        for (int q = 0; q < SLOTS; ++q, row += groups) {
            if (row >= p.rows) return;
            const int64_t o = row * p.dim;
            float f[CH][VEC], sum[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int col = (c * threads + tid) * VEC;
                if (col < p.dim) {
                    x[q][c].get(f[c]);
                    if constexpr (RES) {
                        float rv[VEC];
                        r[c].get(rv);
#pragma unroll
                        for (int k = 0; k < VEC; ++k) f[c][k] += rv[k];
                        r[c].set(f[c]);
                        r[c].store(p.s + o + col);
                    }
#pragma unroll
                    for (int k = 0; k < VEC; ++k) sum[0] += f[c][k];
                }
            }
            fetch(row + SLOTS * groups, x[q]);
            row_sum<ONE>(sum, buf[0], threads / 32);
            const float mean = sum[0] * inv;
            float sq[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if ((c * threads + tid) * VEC < p.dim)
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        f[c][k] -= mean;
                        sq[0] = fmaf(f[c][k], f[c][k], sq[0]);
                    }
            row_sum<ONE>(sq, buf[1], threads / 32);
            const float rstd = rsqrtf(sq[0] * inv + p.eps);
            if (tid == 0) {
                if (p.mean) p.mean[row] = mean;
                if (p.rstd) p.rstd[row] = rstd;
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int col = (c * threads + tid) * VEC;
                if (col < p.dim) {
                    if constexpr (!KEEP) params(col, w[0], b[0]);
                    Raw<T, VEC> y;
#pragma unroll
                    for (int k = 0; k < VEC; ++k) f[c][k] = fmaf(f[c][k] * rstd, w[KEEP ? c : 0][k], b[KEEP ? c : 0][k]);
                    y.set(f[c]);
                    y.store(p.y + o + col);
                }
            }
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
// A group walks rows group, group + groups, ... and keeps its columns' sums of dy xh and dy in
// registers (in shared memory, each thread its own columns, where a thread has 32 of them); it leaves them as one
// row of the parts.
template <typename T, typename S, int VEC, int CH, bool ONE>
__global__ void __launch_bounds__(32 * (ONE ? kOneWarpGroups : kMostWarps)) norm_bwd_kernel(const NormBwd<T, S> p) {
    constexpr bool KEEP = CH * VEC <= 16, SHARED = CH * VEC >= 32;
    // rows on their way: two take 121 against 104 us for 32768 x 2048 bfloat16, their registers spilled. (One spills as well, with
    // 128 registers: 44 bytes stored and 56 loaded a thread in the form of this size with a residual, 16 and 12 without.)
    constexpr int SLOTS = 1;
    __shared__ float buf[2][2][32];
    extern __shared__ __align__(16) float acc[];  // SHARED: [2][dim]
    const int threads = ONE ? 32 : blockDim.x, tid = ONE ? threadIdx.x & 31 : threadIdx.x;
    const int group = ONE ? blockIdx.x * kOneWarpGroups + (threadIdx.x >> 5) : blockIdx.x;
    if (group >= p.groups) return;  // whole groups; groups <= rows
    int64_t row = group;
    Raw<S, VEC> s[SLOTS][CH];
    Raw<T, VEC> d[SLOTS][CH];
    float mean[SLOTS], rstd[SLOTS];
    const auto fetch = [&](const int64_t k, const int q) {
        if (k >= p.rows) return;
        const int64_t o = k * p.dim;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * threads + tid) * VEC;
            if (col < p.dim) {
                s[q][c].load(p.s + o + col);
                d[q][c].load(p.dy + o + col);
            }
        }
        mean[q] = p.mean[k], rstd[q] = p.rstd[k];
    };
#pragma unroll
    for (int q = 0; q < SLOTS; ++q) fetch(row + q * int64_t(p.groups), q);
    Raw<float, VEC> w[KEEP ? CH : 1];
    if constexpr (KEEP) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if ((c * threads + tid) * VEC < p.dim) w[c].load(p.weight + (c * threads + tid) * VEC);
    }
    float aw[SHARED ? 1 : CH][VEC], ab[SHARED ? 1 : CH][VEC];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            if constexpr (SHARED) {
                const int col = (c * threads + tid) * VEC + v;
                if (col < p.dim) acc[col] = acc[p.dim + col] = 0.0f;
            } else {
                aw[c][v] = ab[c][v] = 0.0f;
            }
        }
    const float inv = 1.0f / float(p.dim);
    for (int flip = 0; row < p.rows;) {
#pragma unroll
        for (int q = 0; q < SLOTS; ++q, row += p.groups, flip ^= 1) {
            if (row >= p.rows) break;
            const int64_t o = row * p.dim;
            const float k = rstd[q];
            float xh[CH][VEC], g[CH][VEC], sums[2] = {0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int col = (c * threads + tid) * VEC;
                if (col < p.dim) {
                    if constexpr (!KEEP) w[0].load(p.weight + col);
                    Raw<float, VEC> tw, tb;
                    if constexpr (SHARED) {
                        tw.load(acc + col);
                        tb.load(acc + p.dim + col);
                        tw.get(aw[0]);
                        tb.get(ab[0]);
                    }
                    float(&sw)[VEC] = aw[SHARED ? 0 : c], (&sb)[VEC] = ab[SHARED ? 0 : c];
                    float wv[VEC];
                    w[KEEP ? c : 0].get(wv);
                    s[q][c].get(xh[c]);
                    d[q][c].get(g[c]);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        xh[c][v] = (xh[c][v] - mean[q]) * k;
                        sw[v] = fmaf(g[c][v], xh[c][v], sw[v]);
                        sb[v] += g[c][v];
                        g[c][v] *= wv[v];
                        sums[0] += g[c][v];
                        sums[1] = fmaf(g[c][v], xh[c][v], sums[1]);
                    }
                    if constexpr (SHARED) {
                        tw.set(sw);
                        tb.set(sb);
                        tw.store(acc + col);
                        tb.store(acc + p.dim + col);
                    }
                }
            }
            Raw<float, VEC> r[SHARED ? 1 : CH];
            if constexpr (!SHARED) {
                if (p.ds_out) {
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        if ((c * threads + tid) * VEC < p.dim) r[c].load(p.ds_out + o + (c * threads + tid) * VEC);
                }
            }
            fetch(row + SLOTS * int64_t(p.groups), q);
            row_sum<ONE>(sums, buf[flip], threads / 32);
            const float m0 = sums[0] * inv, m1 = sums[1] * inv;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int col = (c * threads + tid) * VEC;
                if (col < p.dim) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) g[c][v] = k * (g[c][v] - m0 - xh[c][v] * m1);
                    if (p.ds_out) {
                        if constexpr (SHARED) r[0].load(p.ds_out + o + col);
                        float rv[VEC];
                        r[SHARED ? 0 : c].get(rv);
#pragma unroll
                        for (int v = 0; v < VEC; ++v) g[c][v] += rv[v];
                    }
                    Raw<T, VEC> dx;
                    dx.set(g[c]);
                    dx.store(p.dx + o + col);
                    if (p.dres) {
                        Raw<float, VEC> f;
                        f.set(g[c]);
                        f.store(p.dres + o + col);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * threads + tid) * VEC;
        if (col < p.dim) {
            Raw<float, VEC> v;
            if constexpr (SHARED)
                v.load(acc + col);
            else
                v.set(aw[c]);
            v.store(p.part_w + int64_t(group) * p.dim + col);
            if (p.part_b) {
                if constexpr (SHARED)
                    v.load(acc + p.dim + col);
                else
                    v.set(ab[c]);
                v.store(p.part_b + int64_t(group) * p.dim + col);
            }
        }
    }
}

// Column sums of the parts, in a fixed order (blockIdx.y: weight, bias).
__global__ void __launch_bounds__(1024)
    norm_parts_kernel(int groups, int dim, const float *__restrict__ part_w, const float *__restrict__ part_b,
                      float *__restrict__ dweight, float *__restrict__ dbias) {
    __shared__ float s[32][32];
    const float *part = blockIdx.y ? part_b : part_w;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    float t = 0.0f;
    if (col < dim)
#pragma unroll 8
        for (int k = warp; k < groups; k += 32) t += part[int64_t(k) * dim + col];
    s[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && col < dim) {
        t = 0.0f;
#pragma unroll
        for (int w = 0; w < 32; ++w) t += s[w][lane];
        (blockIdx.y ? dbias : dweight)[col] = t;
    }
}

// ---------------------------------------------------------------------- host
inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }
ssm_status launched() { return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA; }

// How a row of nv vectors of VEC columns is split, as go.run<CH, ONE>(warps): one warp for short rows, then two
// vectors a thread and as many warps as that needs, up to two_up_to vectors (the forward with a residual is
// better off with smaller blocks of four vectors beyond 512: 165 against 189 us for 16384 x 5120; the
// backward, which has sums to keep, is not: 252 against 625); more vectors where 16 warps would not
// do. Narrower vectors take more of them from the start.
template <int VEC, typename Go>
ssm_status split_row(int nv, int two_up_to, const Go &go) {
    const auto warps = [&](int ch) { return int(ceil_div(nv, 32 * ch)); };
    constexpr int W = 32 * kMostWarps;
    if constexpr (VEC >= 4) {
        if (nv <= 32) return go.template run<1, true>(1);
        if (nv <= 64) return go.template run<2, true>(1);
        if (nv <= two_up_to) return go.template run<2, false>(warps(2));
        if (VEC == 8 || nv <= 4 * W) return go.template run<4, false>(warps(4));
        if constexpr (VEC == 4) return go.template run<8, false>(warps(8));
    } else {
        if (nv <= 64) return go.template run<2, true>(1);
        if (nv <= 4 * W) return go.template run<4, false>(warps(4));
        if constexpr (VEC == 1)
            if (nv <= 8 * W) return go.template run<8, false>(warps(8));
        return go.template run<32 / VEC, false>(warps(32 / VEC));
    }
    return SSM_ERR_UNSUPPORTED;
}
static_assert(kMaxDim / 8 <= 4 * 32 * kMostWarps && kMaxDim / 4 <= 8 * 32 * kMostWarps && kMaxDim <= 32 * 32 * kMostWarps, "");

// Blocks of each number of warps that an SM holds at once, and the device's SMs (0: not asked yet), by device.
struct Residency {
    std::atomic<int> blocks[64][kMostWarps + 1], sms[64];
};
int resident_blocks(Residency &r, const void *kernel, int warps, int threads, size_t smem) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = r.blocks[dev][warps].load(std::memory_order_relaxed), sms = r.sms[dev].load(std::memory_order_relaxed);
    if (n == 0 || sms == 0) {
        if ((smem > 0 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kMaxDim * 4) != cudaSuccess) ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n <= 0 ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
            return 0;
        r.sms[dev].store(sms, std::memory_order_relaxed);
        r.blocks[dev][warps].store(n, std::memory_order_relaxed);
    }
    return n * sms;
}

template <typename T, int VEC, int CH, bool ONE, bool RES>
ssm_status launch_fwd(const NormFwd<T> &p, int warps, cudaStream_t st) {
    static Residency resident;
    const int threads = ONE ? 32 * kOneWarpGroups : 32 * warps;
    const auto kernel = norm_fwd_kernel<T, VEC, CH, ONE, RES>;
    int64_t blocks = INT_MAX;
    if (!RES) {
        blocks = resident_blocks(resident, reinterpret_cast<const void *>(kernel), warps, threads, 0);
        if (blocks <= 0) return SSM_ERR_CUDA;
    }
    kernel<<<unsigned(std::min<int64_t>(blocks, ceil_div(p.rows, ONE ? kOneWarpGroups : 1))), threads, 0, st>>>(p);
    return launched();
}

template <typename T, int VEC>
struct GoFwd {
    const NormFwd<T> &p;
    cudaStream_t st;
    template <int CH, bool ONE>
    ssm_status run(int warps) const {
        return p.residual ? launch_fwd<T, VEC, CH, ONE, true>(p, warps, st) : launch_fwd<T, VEC, CH, ONE, false>(p, warps, st);
    }
};
template <typename T, int VEC>
ssm_status run_fwd(const NormFwd<T> &p, cudaStream_t st) {
    return split_row<VEC>(p.dim / VEC, p.residual ? 512 : 1024, GoFwd<T, VEC>{p, st});
}

template <typename T, typename S, int VEC, int CH, bool ONE>
ssm_status launch_bwd(NormBwd<T, S> p, int warps, float *dweight, float *dbias, cudaStream_t st) {
    static Residency resident;
    const int threads = ONE ? 32 * kOneWarpGroups : 32 * warps;
    const auto kernel = norm_bwd_kernel<T, S, VEC, CH, ONE>;
    const size_t smem = CH * VEC >= 32 ? size_t(p.dim) * 8 : 0;
    // asked with the longest row of so many warps, which is what `resident` is kept by (8192 x 4099 bfloat16, five warps
    // a block: 427 us; with one block an SM, as the longest row of all would allow, 960)
    const int longest = std::min(kMaxDim, warps * 32 * CH * VEC);
    const int blocks = resident_blocks(resident, reinterpret_cast<const void *>(kernel), warps, threads, smem ? size_t(longest) * 8 : 0);
    if (blocks <= 0) return SSM_ERR_CUDA;
    // at least four rows to a group: fewer rows of partial sums where there is little to do
    p.groups = int(std::min<int64_t>(std::min(blocks * (ONE ? kOneWarpGroups : 1), p.groups), ceil_div(p.rows, 4)));
    kernel<<<unsigned(ceil_div(p.groups, ONE ? kOneWarpGroups : 1)), threads, smem, st>>>(p);
    norm_parts_kernel<<<dim3(unsigned(ceil_div(p.dim, 32)), dbias ? 2 : 1), 1024, 0, st>>>(p.groups, p.dim, p.part_w, p.part_b, dweight, dbias);
    return launched();
}

template <typename T, typename S, int VEC>
struct GoBwd {
    const NormBwd<T, S> &p;
    float *dweight, *dbias;
    cudaStream_t st;
    template <int CH, bool ONE>
    ssm_status run(int warps) const { return launch_bwd<T, S, VEC, CH, ONE>(p, warps, dweight, dbias, st); }
};
template <typename T, typename S, int VEC>
ssm_status run_bwd(const NormBwd<T, S> &p, float *dweight, float *dbias, cudaStream_t st) {
    return split_row<VEC>(p.dim / VEC, 1024, GoBwd<T, S, VEC>{p, dweight, dbias, st});
}

// Rows of partial sums a backward may leave.
int64_t most_groups(int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(ceil_div(rows, 4), kMostGroups)); }

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
    bool two = a->dim % 2 == 0 && aligned(a->x, 2 * es) && aligned(a->y, 2 * es);
    for (const float *q : {a->weight, a->bias, a->residual, static_cast<const float *>(a->residual_out)}) {
        if (!aligned(q, 4)) return SSM_ERR_UNSUPPORTED;
        wide = wide && aligned(q, 16);
        two = two && aligned(q, 8);
    }
    if (!aligned(a->mean, 4) || !aligned(a->rstd, 4)) return SSM_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
#define SSM_RUN(T, VEC)                                                                                          \
    run_fwd<T, VEC>({a->rows, int(a->dim), a->eps, static_cast<const T *>(a->x), a->weight, a->bias, a->residual, \
                     static_cast<T *>(a->y), a->residual_out, a->mean, a->rstd}, st)
    if (a->dtype == SSM_BF16) return wide ? SSM_RUN(__nv_bfloat16, 8) : two ? SSM_RUN(__nv_bfloat16, 2) : SSM_RUN(__nv_bfloat16, 1);
    return wide ? SSM_RUN(float, 4) : two ? SSM_RUN(float, 2) : SSM_RUN(float, 1);
#undef SSM_RUN
}

size_t ssm_layer_norm_bwd_workspace_size(const ssm_norm_bwd_args *a) {
    if (!a || check_sizes(a->rows, a->dim, a->dtype) != SSM_OK || a->rows == 0 || a->dim == 0) return 0;
    return 2 * up256(size_t(most_groups(a->rows)) * size_t(a->dim) * 4);
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
    bool two = a->dim % 2 == 0 && aligned(a->dy, 2 * es) && aligned(a->dx, 2 * es) && aligned(a->s, a->has_residual ? 8 : 2 * es);
    for (const float *q : {a->weight, a->dresidual_out, static_cast<const float *>(a->dresidual)}) {
        if (!aligned(q, 4)) return SSM_ERR_UNSUPPORTED;
        wide = wide && aligned(q, 16);
        two = two && aligned(q, 8);
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
    const int groups = int(most_groups(a->rows));
    float *pw = static_cast<float *>(a->workspace);
    float *pb = a->dbias ? reinterpret_cast<float *>(static_cast<unsigned char *>(a->workspace) + up256(size_t(groups) * size_t(a->dim) * 4)) : nullptr;
#define SSM_RUN(T, S, VEC)                                                                                         \
    run_bwd<T, S, VEC>({a->rows, int(a->dim), groups, static_cast<const S *>(a->s), static_cast<const T *>(a->dy), \
                        a->weight, a->mean, a->rstd, a->dresidual_out, static_cast<T *>(a->dx), a->dresidual, pw, pb}, \
                       a->dweight, a->dbias, st)
#define SSM_WIDTH(T, S, VEC) (wide ? SSM_RUN(T, S, VEC) : two ? SSM_RUN(T, S, 2) : SSM_RUN(T, S, 1))
    if (a->dtype == SSM_F32) return SSM_WIDTH(float, float, 4);
    return a->has_residual ? SSM_WIDTH(__nv_bfloat16, float, 8) : SSM_WIDTH(__nv_bfloat16, __nv_bfloat16, 8);
#undef SSM_WIDTH
#undef SSM_RUN
}

}  // extern "C"
