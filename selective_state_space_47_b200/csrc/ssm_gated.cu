// ssm_gated.cu -- the gated linear recurrence: forward over whole sequences, backward
// and the one-token step (include/ssm_scan.h, ssm_gated_*).
//
//   w_t = p sigmoid(r_t), p = c softplus(lam);  a_t = exp(-w_t);  beta_t = sqrt(1 - a_t^2)
//   h_t = a_t h_{t-1} + beta_t sigmoid(i_t) x_t,  y_t = h_t;  at a reset a_t = 0, beta_t = 1
//
// A tile is 32 V channels by W K steps: lane = V neighbouring channels, warp = K
// consecutive steps, held in registers. A piece of time acts on the state entering it as
// h -> P h + H, and two such maps compose, so each thread forms the map of its K steps,
// the warps of a block chain theirs through shared memory, and the tiles chain theirs
// through the workspace.
#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/ssm_scan.h"
#include "ssm_device.cuh"

using namespace ssm;

namespace {

constexpr int kChunk = SSM_GATED_CHUNK;  // steps between the states kept for the backward
constexpr int kW = 8;                    // warps of a block
constexpr int kKF = 16;                  // steps per thread, forward
constexpr int kKB = 8;                   // steps per thread, backward
static_assert((kW * kKF) % kChunk == 0 && kW * kKB == kChunk, "tiles are made of whole chunks");

// ------------------------------------------------------------- element math
__device__ __forceinline__ float sigmoid_f(float v) { return rcp_approx(1.0f + ex2_approx(-v * kLog2e)); }

// a = e^-w and e = 1 - a for w >= 0, each to float32's relative precision: below 1/2,
// e = w (1 + w Q(w)) with Q the Chebyshev interpolation of ((1 - e^-w)/w - 1)/w of degree 4
// on [0, 1/2] (6e-9 relative before rounding, 1e-7 in float32), and a = 1 - e; above, a from
// the exponential and e = 1 - a. Decays near 1 are the rule, and their distance from 1
// sets both how long the state remembers and the input's weight.
__device__ __forceinline__ float small_e(float w) {
    const float q = fmaf(w, fmaf(w, fmaf(w, fmaf(w, -0.0011642870f, 0.0082382215f), -0.041649930f), 0.16666563f), -0.5f);
    return w * fmaf(w, q, 1.0f);
}
__device__ __forceinline__ float decay(float w, float &e) {
    e = small_e(w);
    float a = 1.0f - e;
    if (!(w < 0.5f)) {
        a = ex2_approx(-w * kLog2e);
        e = 1.0f - a;
    }
    return a;
}

// 1 / beta, beta^2 = 1 - a^2 = e (2 - e) with e = 1 - a; 0 where beta itself (below 3e-19) counts as 0.
__device__ __forceinline__ float inv_beta(float sq) {
    float q;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(sq));
    return sq > 1e-37f ? q : 0.0f;
}

__device__ __forceinline__ float rate(float lam, float c) { return c * (fmaxf(lam, 0.0f) + log1pf(expf(-fabsf(lam)))); }

// The map h -> P h + H of a piece of time. P is 0 exactly where the piece holds a reset:
// what came before is then dropped, whatever it was (an infinity or NaN too). A product
// of decays that underflows is kept at the smallest normal number for the same reason.
struct Map {
    float P, H;
};
__device__ __forceinline__ float apply(const Map m, float h) { return m.P == 0.0f ? m.H : fmaf(m.P, h, m.H); }
__device__ __forceinline__ float keep(float P) { return P < FLT_MIN ? FLT_MIN : P; }  // (a NaN stays)
__device__ __forceinline__ Map then(const Map first, const Map second) {
    Map m;
    m.P = (first.P == 0.0f || second.P == 0.0f) ? 0.0f : keep(first.P * second.P);
    m.H = apply(second, first.H);
    return m;
}

// ----------------------------------------------------------- vector accesses
template <typename T, int V>
struct Vec;
template <typename T>
struct Vec<T, 1> {
    T v;
    __device__ __forceinline__ float get(int) const { return Tok<T>::to_f(v); }
    __device__ __forceinline__ void set(int, float f) { v = Tok<T>::from_f(f); }
};
template <>
struct Vec<float, 2> {
    float2 v;
    __device__ __forceinline__ float get(int k) const { return k ? v.y : v.x; }
    __device__ __forceinline__ void set(int k, float f) { (k ? v.y : v.x) = f; }
};
template <>
struct Vec<__nv_bfloat16, 2> {
    __nv_bfloat162 v;
    __device__ __forceinline__ float get(int k) const { return k ? __high2float(v) : __low2float(v); }
    __device__ __forceinline__ void set(int k, float f) { (k ? v.y : v.x) = __float2bfloat16_rn(f); }
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> ldv(const T *p) {
    return *reinterpret_cast<const Vec<T, V> *>(p);
}
template <typename T, int V>
__device__ __forceinline__ void stv(T *p, const Vec<T, V> v) {
    *reinterpret_cast<Vec<T, V> *>(p) = v;
}

struct Shape {
    int64_t B, L, D;
    int64_t groups, tiles;  // channel groups of 32 V, tiles of time
    float c;
};

// ------------------------------------------------------------------- forward
template <typename T>
struct FwdArgs {
    Shape s;
    const T *x, *r, *i;
    int64_t xb, xt, rb, rt, ib, it;
    const uint8_t *reset;
    const float *lam, *h0;
    T *y;
    float *h_last, *states, *starts;
    Map *maps;
};

// MAIN false: the map of every tile into maps; true: outputs, from the state before every tile in starts.
template <typename T, int V, bool MAIN>
__global__ void __launch_bounds__(kW * 32) gated_fwd_kernel(const FwdArgs<T> p) {
    constexpr int K = kKF;
    __shared__ Map sm[kW][V][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t g = blockIdx.x % p.s.groups, jb = blockIdx.x / p.s.groups;
    const int64_t b = jb % p.s.B, j = jb / p.s.B;
    const int64_t d = (g * 32 + lane) * V;
    const int64_t t0 = (j * kW + warp) * K;
    const bool on = d < p.s.D;
    const int n = int(max(int64_t(0), min(int64_t(K), p.s.L - t0)));

    float a[K][V], h[K][V];
    float rt[V];
#pragma unroll
    for (int v = 0; v < V; ++v) rt[v] = on ? rate(p.lam[d + v], p.s.c) : 0.0f;
    bool cut = false;
    {
        Vec<T, V> xv[K], rv[K], iv[K];
        const T *xp = p.x + b * p.xb + t0 * p.xt + d, *rp = p.r + b * p.rb + t0 * p.rt + d,
                *ip = p.i + b * p.ib + t0 * p.it + d;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (on && k < n) {
                xv[k] = ldv<T, V>(xp + k * p.xt);
                rv[k] = ldv<T, V>(rp + k * p.rt);
                iv[k] = ldv<T, V>(ip + k * p.it);
            } else {
                for (int v = 0; v < V; ++v) xv[k].set(v, 0.0f), rv[k].set(v, 0.0f), iv[k].set(v, 0.0f);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool fresh = p.reset && k < n && p.reset[b * p.s.L + t0 + k];
            cut |= fresh;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float e;
                const float dec = decay(rt[v] * sigmoid_f(rv[k].get(v)), e);
                const float sq = e * (2.0f - e), u = sigmoid_f(iv[k].get(v)) * xv[k].get(v);
                a[k][v] = k < n ? (fresh ? 0.0f : dec) : 1.0f;
                h[k][v] = k < n ? (fresh ? u : sq * inv_beta(sq) * u) : 0.0f;
            }
        }
    }
    // the thread's map, and the maps of the block's warps
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Map m{1.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            m.P *= a[k][v];
            m.H = (p.reset && a[k][v] == 0.0f) ? h[k][v] : fmaf(a[k][v], m.H, h[k][v]);
        }
        m.P = cut ? 0.0f : keep(m.P);
        sm[warp][v][lane] = m;
    }
    __syncthreads();
    if (!MAIN) {
        if (warp == 0 && on) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                Map m = sm[0][v][lane];
                for (int w = 1; w < kW; ++w) m = then(m, sm[w][v][lane]);
                p.maps[(j * p.s.B + b) * p.s.D + d + v] = m;
            }
        }
        return;
    }
    if (!on || n == 0) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float hs = p.starts[(j * p.s.B + b) * p.s.D + d + v];
        for (int w = 0; w < warp; ++w) hs = apply(sm[w][v][lane], hs);
        if (p.states && t0 % kChunk == 0) p.states[(b * ((p.s.L + kChunk - 1) / kChunk) + t0 / kChunk) * p.s.D + d + v] = hs;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            hs = (p.reset && a[k][v] == 0.0f) ? h[k][v] : fmaf(a[k][v], hs, h[k][v]);
            h[k][v] = hs;
        }
        if (p.h_last && t0 + n == p.s.L) p.h_last[b * p.s.D + d + v] = hs;
    }
    if (p.y) {
        T *yp = p.y + (b * p.s.L + t0) * p.s.D + d;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (k < n) {
                Vec<T, V> o;
                for (int v = 0; v < V; ++v) o.set(v, h[k][v]);
                stv<T, V>(yp + k * p.s.D, o);
            }
        }
    }
}

// Chains the tiles' maps of every channel: starts[j] is the state entering tile j; for the
// backward (from the last tile to the first) the adjoint entering it from its right end.
__global__ void gated_chain_kernel(int64_t n, int64_t tiles, bool backward, const float *__restrict__ first,
                                   const Map *__restrict__ maps, float *__restrict__ starts) {
    const int64_t k = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (k >= n) return;
    float h = first ? first[k] : 0.0f;
#pragma unroll 8
    for (int64_t j = 0; j < tiles; ++j) {
        const int64_t o = (backward ? tiles - 1 - j : j) * n + k;
        const Map m = maps[o];
        starts[o] = h;
        h = apply(m, h);
    }
    if (backward) starts[tiles * n + k] = h;
}

// ------------------------------------------------------------------ backward
template <typename T>
struct BwdArgs {
    Shape s;
    const T *x, *r, *i, *dy;
    int64_t xb, xt, rb, rt, ib, it;
    const uint8_t *reset;
    const float *lam, *states;
    T *dx, *dr, *di;
    float *dh0, *starts, *parts;
    Map *maps;
};

// v_t = dL/dh_t follows v_t = dy_t + a_{t+1} v_{t+1}; with g_t = a_t v_t, what a step hands
// to the one before it, a piece of time acts on the g entering from its right as
// g -> P g + G with the forward's P.
template <typename T, int V, bool MAIN>
__global__ void __launch_bounds__(kW * 32) gated_bwd_kernel(const BwdArgs<T> p) {
    constexpr int K = kKB;
    __shared__ Map sf[kW][V][32], sb[kW][V][32];
    __shared__ float sl[kW][V][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t g = blockIdx.x % p.s.groups, jb = blockIdx.x / p.s.groups;
    const int64_t b = jb % p.s.B, j = jb / p.s.B;
    const int64_t d = (g * 32 + lane) * V;
    const int64_t t0 = (j * kW + warp) * K;
    const bool on = d < p.s.D;
    const int n = int(max(int64_t(0), min(int64_t(K), p.s.L - t0)));

    float rt[V];
#pragma unroll
    for (int v = 0; v < V; ++v) rt[v] = on ? rate(p.lam[d + v], p.s.c) : 0.0f;
    Vec<T, V> xv[K], rv[K], iv[K], dv[K];
    const T *xp = p.x + b * p.xb + t0 * p.xt + d, *rp = p.r + b * p.rb + t0 * p.rt + d,
            *ip = p.i + b * p.ib + t0 * p.it + d, *dp = p.dy + (b * p.s.L + t0) * p.s.D + d;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (on && k < n) {
            xv[k] = ldv<T, V>(xp + k * p.xt);
            rv[k] = ldv<T, V>(rp + k * p.rt);
            iv[k] = ldv<T, V>(ip + k * p.it);
            dv[k] = ldv<T, V>(dp + k * p.s.D);
        } else {
            for (int v = 0; v < V; ++v) xv[k].set(v, 0.0f), rv[k].set(v, 0.0f), iv[k].set(v, 0.0f), dv[k].set(v, 0.0f);
        }
    }
    unsigned fresh = 0;
    if (p.reset)
        for (int k = 0; k < K; ++k)
            if (k < n && p.reset[b * p.s.L + t0 + k]) fresh |= 1u << k;

    float a[K][V], h[K][V];  // the decay, and the input; then the state before the step
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float e;
            const float dec = decay(rt[v] * sigmoid_f(rv[k].get(v)), e);
            const float sq = e * (2.0f - e), u = sigmoid_f(iv[k].get(v)) * xv[k].get(v);
            a[k][v] = k < n ? dec : 1.0f;
            h[k][v] = (fresh >> k & 1) ? u : sq * inv_beta(sq) * u;
        }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Map f{1.0f, 0.0f}, r{1.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            f.P *= a[k][v];
            f.H = (fresh >> k & 1) ? h[k][v] : fmaf(a[k][v], f.H, h[k][v]);
        }
#pragma unroll
        for (int k = K - 1; k >= 0; --k) r.H = (fresh >> k & 1) ? 0.0f : a[k][v] * (dv[k].get(v) + r.H);
        f.P = r.P = fresh ? 0.0f : keep(f.P);
        sf[warp][v][lane] = f;
        sb[warp][v][lane] = r;
    }
    __syncthreads();
    if (!MAIN) {
        if (warp == 0 && on) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                Map m = sb[kW - 1][v][lane];
                for (int w = kW - 2; w >= 0; --w) m = then(m, sb[w][v][lane]);
                p.maps[(j * p.s.B + b) * p.s.D + d + v] = m;
            }
        }
        return;
    }
    float gr[V], dl[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float hs = on ? p.states[(b * p.s.tiles + j) * p.s.D + d + v] : 0.0f;
        for (int w = 0; w < warp; ++w) hs = apply(sf[w][v][lane], hs);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float next = (fresh >> k & 1) ? h[k][v] : fmaf(a[k][v], hs, h[k][v]);
            h[k][v] = hs;
            hs = next;
        }
        gr[v] = on ? p.starts[(j * p.s.B + b) * p.s.D + d + v] : 0.0f;
        for (int w = kW - 1; w > warp; --w) gr[v] = apply(sb[w][v][lane], gr[v]);
        dl[v] = 0.0f;
    }
    T *dxp = p.dx + (b * p.s.L + t0) * p.s.D + d, *drp = p.dr + (b * p.s.L + t0) * p.s.D + d,
      *dip = p.di + (b * p.s.L + t0) * p.s.D + d;
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
        if (k < n) {
            const bool fr = fresh >> k & 1;
            Vec<T, V> ox, orr, oi;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float sr = sigmoid_f(rv[k].get(v)), si = sigmoid_f(iv[k].get(v));
                const float w = rt[v] * sr, at = a[k][v], e = w < 0.5f ? small_e(w) : 1.0f - at;
                const float sq = e * (2.0f - e), q = inv_beta(sq);
                const float u = si * xv[k].get(v), vt = dv[k].get(v) + gr[v];
                const float vb = fr ? vt : vt * sq * q;
                // dL/dw = a v (a u / beta - h_{t-1}); beta -> 0 only as w -> 0, where w / beta -> 0
                const float dw = fr ? 0.0f : at * vt * fmaf(at * q, u, -h[k][v]);
                ox.set(v, vb * si);
                oi.set(v, vb * u * (1.0f - si));
                orr.set(v, dw * w * (1.0f - sr));
                dl[v] = fmaf(dw, sr, dl[v]);
                gr[v] = fr ? 0.0f : at * vt;
            }
            if (on) {
                stv<T, V>(dxp + k * p.s.D, ox);
                stv<T, V>(drp + k * p.s.D, orr);
                stv<T, V>(dip + k * p.s.D, oi);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sl[warp][v][lane] = dl[v];
        if (p.dh0 && t0 == 0 && on) p.dh0[b * p.s.D + d + v] = gr[v];
    }
    __syncthreads();
    if (warp == 0 && on) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float t = 0.0f;
            for (int w = 0; w < kW; ++w) t += sl[w][v][lane];
            p.parts[(j * p.s.B + b) * p.s.D + d + v] = t;
        }
    }
}

// dlam[d] = c sigmoid(lam[d]) * the sum of the tiles' parts, in a fixed order.
__global__ void __launch_bounds__(256)
    gated_dlam_kernel(int64_t rows, int64_t D, float c, const float *__restrict__ parts, const float *__restrict__ lam,
                      float *__restrict__ dlam) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t d = int64_t(blockIdx.x) * 32 + lane;
    float t = 0.0f;
    if (d < D)
        for (int64_t k = warp; k < rows; k += 8) t += parts[k * D + d];
    s[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && d < D) {
        t = 0.0f;
        for (int w = 0; w < 8; ++w) t += s[w][lane];
        dlam[d] = t * c / (1.0f + expf(-lam[d]));
    }
}

// ---------------------------------------------------------------------- step
template <typename T, int V>
__global__ void __launch_bounds__(256)
    gated_step_kernel(int64_t B, int64_t D, float c, const T *__restrict__ x, const T *__restrict__ r,
                      const T *__restrict__ i, int64_t xs, int64_t rs, int64_t is, const float *__restrict__ lam,
                      const float *h, float *h_out, T *__restrict__ y) {
    const int64_t k = int64_t(blockIdx.x) * blockDim.x + threadIdx.x, per = D / V;
    if (k >= B * per) return;
    const int64_t b = k / per, d = (k - b * per) * V;
    const Vec<T, V> xv = ldv<T, V>(x + b * xs + d), rv = ldv<T, V>(r + b * rs + d), iv = ldv<T, V>(i + b * is + d);
    const Vec<float, V> lv = ldv<float, V>(lam + d), hv = ldv<float, V>(h + b * D + d);
    Vec<float, V> ho;
    Vec<T, V> o;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float e;
        const float a = decay(rate(lv.get(v), c) * sigmoid_f(rv.get(v)), e), sq = e * (2.0f - e);
        const float hn = fmaf(a, hv.get(v), sq * inv_beta(sq) * (sigmoid_f(iv.get(v)) * xv.get(v)));
        ho.set(v, hn);
        o.set(v, hn);
    }
    stv<float, V>(h_out + b * D + d, ho);
    stv<T, V>(y + b * D + d, o);
}

// ---------------------------------------------------------------------- host
inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Sizes whose products leave 62 bits, or more tiles than a grid holds, are refused.
bool sizes_fit(int64_t B, int64_t L, int64_t D, int64_t t) {
    int64_t n;
    if (__builtin_mul_overflow(B, std::max<int64_t>(L, 1), &n) || __builtin_mul_overflow(n, D, &n)) return false;
    if (n > (int64_t(1) << 56)) return false;
    return B * ceil_div(L, t) * ceil_div(D, 32) <= INT_MAX;
}

struct Strides {
    int64_t b, t;
};
bool even(const int64_t *s) { return s[0] % 2 == 0 && s[1] % 2 == 0; }

ssm_status launched() { return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA; }

template <typename T, int V>
ssm_status run_fwd(const ssm_gated_args *a, cudaStream_t st) {
    FwdArgs<T> p;
    p.s = {a->batch, a->seqlen, a->dim, ceil_div(a->dim, 32 * V), ceil_div(a->seqlen, kW * kKF), a->c};
    p.x = static_cast<const T *>(a->x), p.r = static_cast<const T *>(a->r), p.i = static_cast<const T *>(a->i);
    p.xb = a->x_stride[0], p.xt = a->x_stride[1], p.rb = a->r_stride[0], p.rt = a->r_stride[1];
    p.ib = a->i_stride[0], p.it = a->i_stride[1];
    p.reset = a->reset, p.lam = a->lam, p.h0 = a->h0;
    p.y = static_cast<T *>(a->y), p.h_last = a->h_last, p.states = a->states;
    const int64_t n = a->batch * a->dim;
    p.maps = static_cast<Map *>(a->workspace);
    p.starts = reinterpret_cast<float *>(static_cast<unsigned char *>(a->workspace) + up256(size_t(n) * size_t(p.s.tiles) * sizeof(Map)));
    const unsigned grid = unsigned(a->batch * p.s.groups * p.s.tiles);
    gated_fwd_kernel<T, V, false><<<grid, kW * 32, 0, st>>>(p);
    gated_chain_kernel<<<unsigned(ceil_div(n, 128)), 128, 0, st>>>(n, p.s.tiles, false, a->h0, p.maps, p.starts);
    gated_fwd_kernel<T, V, true><<<grid, kW * 32, 0, st>>>(p);
    return launched();
}

template <typename T, int V>
ssm_status run_bwd(const ssm_gated_bwd_args *a, cudaStream_t st) {
    BwdArgs<T> p;
    p.s = {a->batch, a->seqlen, a->dim, ceil_div(a->dim, 32 * V), ceil_div(a->seqlen, kW * kKB), a->c};
    p.x = static_cast<const T *>(a->x), p.r = static_cast<const T *>(a->r), p.i = static_cast<const T *>(a->i);
    p.dy = static_cast<const T *>(a->dy);
    p.xb = a->x_stride[0], p.xt = a->x_stride[1], p.rb = a->r_stride[0], p.rt = a->r_stride[1];
    p.ib = a->i_stride[0], p.it = a->i_stride[1];
    p.reset = a->reset, p.lam = a->lam, p.states = a->states;
    p.dx = static_cast<T *>(a->dx), p.dr = static_cast<T *>(a->dr), p.di = static_cast<T *>(a->di), p.dh0 = a->dh0;
    const int64_t n = a->batch * a->dim;
    unsigned char *ws = static_cast<unsigned char *>(a->workspace);
    p.maps = reinterpret_cast<Map *>(ws);
    ws += up256(size_t(n) * size_t(p.s.tiles) * sizeof(Map));
    p.starts = reinterpret_cast<float *>(ws);
    ws += up256(size_t(n) * size_t(p.s.tiles + 1) * 4);
    p.parts = reinterpret_cast<float *>(ws);
    const unsigned grid = unsigned(a->batch * p.s.groups * p.s.tiles);
    gated_bwd_kernel<T, V, false><<<grid, kW * 32, 0, st>>>(p);
    gated_chain_kernel<<<unsigned(ceil_div(n, 128)), 128, 0, st>>>(n, p.s.tiles, true, a->dh_last, p.maps, p.starts);
    gated_bwd_kernel<T, V, true><<<grid, kW * 32, 0, st>>>(p);
    gated_dlam_kernel<<<unsigned(ceil_div(a->dim, 32)), 256, 0, st>>>(a->batch * p.s.tiles, a->dim, a->c, p.parts, a->lam, a->dlam);
    return launched();
}

__global__ void gated_dlam_zero_kernel(int64_t D, float *dlam) {
    const int64_t d = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (d < D) dlam[d] = 0.0f;
}

// What the forward and the backward check alike.
template <typename A>
ssm_status check_common(const A *a) {
    if (!a || a->batch < 0 || a->seqlen < 0 || a->dim < 0 || a->flags != 0 || !(a->c > 0.0f) || a->c > FLT_MAX ||
        (a->dtype != SSM_F32 && a->dtype != SSM_BF16))
        return SSM_ERR_INVALID;
    if (!sizes_fit(a->batch, a->seqlen, a->dim, kChunk)) return SSM_ERR_UNSUPPORTED;
    const int64_t *const strides[] = {a->x_stride, a->r_stride, a->i_stride};
    for (const int64_t *s : strides)
        if (s[0] < 0 || s[1] < 0) return SSM_ERR_INVALID;
    return SSM_OK;
}

template <typename A>
bool strides_fit(const A *a) {
    const int64_t *const strides[] = {a->x_stride, a->r_stride, a->i_stride};
    for (const int64_t *s : strides) {
        int64_t m, n;
        if (__builtin_mul_overflow(a->batch, s[0], &m) || __builtin_mul_overflow(a->seqlen, s[1], &n) ||
            m > (int64_t(1) << 56) || n > (int64_t(1) << 56))
            return false;
    }
    return true;
}

}  // namespace

extern "C" {

size_t ssm_gated_states_size(int64_t batch, int64_t seqlen, int64_t dim) {
    if (batch < 0 || seqlen < 0 || dim < 0 || !sizes_fit(batch, seqlen, dim, kChunk)) return 0;
    return size_t(batch) * size_t(ceil_div(seqlen, kChunk)) * size_t(dim) * 4;
}

size_t ssm_gated_scan_workspace_size(const ssm_gated_args *a) {
    if (check_common(a) != SSM_OK) return 0;
    const size_t n = size_t(a->batch) * size_t(a->dim) * size_t(ceil_div(a->seqlen, kW * kKF));
    return up256(n * sizeof(Map)) + up256(n * 4);
}

ssm_status ssm_gated_scan_fwd(const ssm_gated_args *a, void *stream) {
    const ssm_status ok = check_common(a);
    if (ok != SSM_OK) return ok;
    if (a->batch == 0 || a->dim == 0) return SSM_OK;
    const size_t es = a->dtype == SSM_BF16 ? 2 : 4;
    if (!a->lam || (a->seqlen > 0 && (!a->x || !a->r || !a->i || (!a->y && !a->states && !a->h_last))))
        return SSM_ERR_INVALID;
    if (!strides_fit(a)) return SSM_ERR_UNSUPPORTED;
    for (const void *q : {a->x, a->r, a->i, static_cast<const void *>(a->y)})
        if (!aligned(q, es)) return SSM_ERR_UNSUPPORTED;
    for (const void *q : {static_cast<const void *>(a->lam), static_cast<const void *>(a->h0),
                          static_cast<const void *>(a->h_last), static_cast<const void *>(a->states)})
        if (!aligned(q, 4)) return SSM_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->seqlen == 0) {
        if (!a->h_last) return SSM_OK;
        const size_t nb = size_t(a->batch) * size_t(a->dim) * 4;
        const cudaError_t e = a->h0 ? cudaMemcpyAsync(a->h_last, a->h0, nb, cudaMemcpyDeviceToDevice, st)
                                    : cudaMemsetAsync(a->h_last, 0, nb, st);
        return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
    }
    if (!a->workspace || a->workspace_bytes < ssm_gated_scan_workspace_size(a)) return SSM_ERR_INVALID;
    if (!aligned(a->workspace, 16)) return SSM_ERR_UNSUPPORTED;
    // two channels per lane where every access to a pair is aligned
    const bool two = a->dim % 2 == 0 && even(a->x_stride) && even(a->r_stride) && even(a->i_stride) &&
                     aligned(a->x, 2 * es) && aligned(a->r, 2 * es) && aligned(a->i, 2 * es) && aligned(a->y, 2 * es);
    if (a->dtype == SSM_BF16) return two ? run_fwd<__nv_bfloat16, 2>(a, st) : run_fwd<__nv_bfloat16, 1>(a, st);
    return two ? run_fwd<float, 2>(a, st) : run_fwd<float, 1>(a, st);
}

size_t ssm_gated_scan_bwd_workspace_size(const ssm_gated_bwd_args *a) {
    if (check_common(a) != SSM_OK) return 0;
    const size_t n = size_t(a->batch) * size_t(a->dim), t = size_t(ceil_div(a->seqlen, kChunk));
    return up256(n * t * sizeof(Map)) + up256(n * (t + 1) * 4) + up256(n * t * 4);
}

ssm_status ssm_gated_scan_bwd(const ssm_gated_bwd_args *a, void *stream) {
    const ssm_status ok = check_common(a);
    if (ok != SSM_OK) return ok;
    if (a->dim == 0) return SSM_OK;
    const size_t es = a->dtype == SSM_BF16 ? 2 : 4;
    const bool empty = a->batch == 0 || a->seqlen == 0;
    if (!a->lam || !a->dlam ||
        (!empty && (!a->x || !a->r || !a->i || !a->dy || !a->states || !a->dx || !a->dr || !a->di)))
        return SSM_ERR_INVALID;
    if (!strides_fit(a)) return SSM_ERR_UNSUPPORTED;
    for (const void *q : {a->x, a->r, a->i, a->dy, static_cast<const void *>(a->dx), static_cast<const void *>(a->dr),
                          static_cast<const void *>(a->di)})
        if (!aligned(q, es)) return SSM_ERR_UNSUPPORTED;
    for (const void *q : {static_cast<const void *>(a->lam), static_cast<const void *>(a->states),
                          static_cast<const void *>(a->dh_last), static_cast<const void *>(a->dlam),
                          static_cast<const void *>(a->dh0)})
        if (!aligned(q, 4)) return SSM_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (empty) {
        gated_dlam_zero_kernel<<<unsigned(ceil_div(a->dim, 256)), 256, 0, st>>>(a->dim, a->dlam);
        if (a->dh0 && a->batch > 0) {
            const size_t nb = size_t(a->batch) * size_t(a->dim) * 4;
            const cudaError_t e = a->dh_last ? cudaMemcpyAsync(a->dh0, a->dh_last, nb, cudaMemcpyDeviceToDevice, st)
                                             : cudaMemsetAsync(a->dh0, 0, nb, st);
            if (e != cudaSuccess) return SSM_ERR_CUDA;
        }
        return launched();
    }
    if (!a->workspace || a->workspace_bytes < ssm_gated_scan_bwd_workspace_size(a)) return SSM_ERR_INVALID;
    if (!aligned(a->workspace, 16)) return SSM_ERR_UNSUPPORTED;
    bool two = a->dim % 2 == 0 && even(a->x_stride) && even(a->r_stride) && even(a->i_stride);
    for (const void *q : {a->x, a->r, a->i, a->dy, static_cast<const void *>(a->dx), static_cast<const void *>(a->dr),
                          static_cast<const void *>(a->di)})
        two = two && aligned(q, 2 * es);
    if (a->dtype == SSM_BF16) return two ? run_bwd<__nv_bfloat16, 2>(a, st) : run_bwd<__nv_bfloat16, 1>(a, st);
    return two ? run_bwd<float, 2>(a, st) : run_bwd<float, 1>(a, st);
}

ssm_status ssm_gated_step(int64_t batch, int64_t dim, ssm_dtype dtype, float c, const void *x, int64_t x_stride,
                          const void *r, int64_t r_stride, const void *i, int64_t i_stride, const float *lam,
                          const float *h, float *h_out, void *y, void *stream) {
    if (batch < 0 || dim < 0 || x_stride < 0 || r_stride < 0 || i_stride < 0 || !(c > 0.0f) || c > FLT_MAX ||
        (dtype != SSM_F32 && dtype != SSM_BF16))
        return SSM_ERR_INVALID;
    if (!sizes_fit(batch, 1, dim, 1)) return SSM_ERR_UNSUPPORTED;
    if (batch == 0 || dim == 0) return SSM_OK;
    if (!x || !r || !i || !lam || !h || !h_out || !y) return SSM_ERR_INVALID;
    const size_t es = dtype == SSM_BF16 ? 2 : 4;
    bool two = dim % 2 == 0 && x_stride % 2 == 0 && r_stride % 2 == 0 && i_stride % 2 == 0;
    for (const void *q : {x, r, i, static_cast<const void *>(y)}) {
        if (!aligned(q, es)) return SSM_ERR_UNSUPPORTED;
        two = two && aligned(q, 2 * es);
    }
    for (const void *q : {static_cast<const void *>(lam), static_cast<const void *>(h), static_cast<const void *>(h_out)}) {
        if (!aligned(q, 4)) return SSM_ERR_UNSUPPORTED;
        two = two && aligned(q, 8);
    }
    for (const int64_t s : {x_stride, r_stride, i_stride}) {
        int64_t m;
        if (__builtin_mul_overflow(batch, s, &m) || m > (int64_t(1) << 56)) return SSM_ERR_UNSUPPORTED;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned grid = unsigned(ceil_div(batch * (two ? dim / 2 : dim), 256));
#define SSM_STEP(T, V)                                                                                        \
    gated_step_kernel<T, V><<<grid, 256, 0, st>>>(batch, dim, c, static_cast<const T *>(x),                    \
                                                  static_cast<const T *>(r), static_cast<const T *>(i), x_stride, \
                                                  r_stride, i_stride, lam, h, h_out, static_cast<T *>(y))
    if (dtype == SSM_BF16) {
        if (two) SSM_STEP(__nv_bfloat16, 2); else SSM_STEP(__nv_bfloat16, 1);
    } else {
        if (two) SSM_STEP(float, 2); else SSM_STEP(float, 1);
    }
#undef SSM_STEP
    return launched();
}

}  // extern "C"
