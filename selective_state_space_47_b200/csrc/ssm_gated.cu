// ssm_gated.cu -- the gated linear recurrence: forward over whole sequences, backward
// and the one-token step (include/ssm_scan.h, ssm_gated_*).
//
//   w_t = p sigmoid(r_t), p = c softplus(lam);  a_t = exp(-w_t);  beta_t = sqrt(1 - a_t^2)
//   h_t = a_t h_{t-1} + beta_t sigmoid(i_t) x_t,  y_t = h_t;  at a reset a_t = 0, beta_t = 1
//
// A piece of time acts on the state entering it as h -> P h + H, and two such maps compose. A
// column is 64 channels of one sequence, a tile 8 K steps of it: lane = two neighbouring
// channels, warp = K steps, in registers from the one read of the tokens to the one write of
// the results. Each warp forms the map of its steps, a block composes its tile's, and a
// cluster of blocks, which walks the column, exchanges its tiles' maps through shared memory. So time is
// passed over once, the state between rounds never leaves the chip, and the order in which pieces are
// joined depends on the shape alone.
//
// What bounds it: latency. The forward of B=1 L=262144 D=5120 bfloat16 takes 2.21 ms alone and 2.36 ms call after call, 4.9 and
// 4.5 TB/s of 6.5; a computing warp waits once a tile for the way to the carrying warp, the cluster and back, and 16 such
// warps an SM fill 53% of the issue slots and 57% of the special-function unit (four operations an element, 16 a clock)
// meanwhile. With the sigmoids and the root left out it takes 1.9 ms. The backward of B=8 L=4096 D=2048 takes 254 us, 3.7
// TB/s, at 68 instructions an element on 51% of the issue slots. float32, with twice the bytes to the same arithmetic, moves
// 6.2 TB/s forward and 5.4 TB/s backward there.
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <mutex>

#include "../../include/ssm_scan.h"
#include "ssm_device.cuh"

using namespace ssm;

namespace {

constexpr int kChunk = SSM_GATED_CHUNK;  // steps between the states kept for the backward
constexpr int kW = 8;                    // computing warps of a block
constexpr size_t kWsHeader = 256;
constexpr int kMostBlocks = 16;          // of a cluster

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
// V neighbouring values of type T, loaded and stored as one piece of 2 to 16 bytes.
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
    T v[V];
    __device__ __forceinline__ float get(int k) const { return Tok<T>::to_f(v[k]); }
    __device__ __forceinline__ void set(int k, float f) { v[k] = Tok<T>::from_f(f); }
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> ldv(const T *p) {
    Vec<T, V> r;
    if constexpr (sizeof(r) == 16)
        *reinterpret_cast<uint4 *>(&r) = *reinterpret_cast<const uint4 *>(p);
    else if constexpr (sizeof(r) == 8)
        *reinterpret_cast<uint2 *>(&r) = *reinterpret_cast<const uint2 *>(p);
    else if constexpr (sizeof(r) == 4)
        *reinterpret_cast<uint32_t *>(&r) = *reinterpret_cast<const uint32_t *>(p);
    else
        r.v[0] = p[0];
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void stv(T *p, const Vec<T, V> r) {
    if constexpr (sizeof(r) == 16)
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(&r);
    else if constexpr (sizeof(r) == 8)
        *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(&r);
    else if constexpr (sizeof(r) == 4)
        *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<const uint32_t *>(&r);
    else
        p[0] = r.v[0];
}

struct Shape {
    int64_t B, L, D;
    int64_t groups;  // of 64 channels
    float c;
};

// ------------------------------------------------- states between blocks
// A state handed from one block to another is a single 64-bit word beside a tag, zero until
// written: data and flag are one access.
__device__ __forceinline__ unsigned long long ld_word(const unsigned long long *p) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_word(unsigned long long *p, unsigned long long v) {
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long pack(float h) { return (1ull << 32) | __float_as_uint(h); }

// What a wait that gives up leaves behind: the call's status word, which may be in scratch that nobody reads, and a
// word of the device, which outlives the call (ssm_gated_status takes it).
__device__ unsigned int gave_up, gave_up_taken;
__device__ __forceinline__ void give_up(unsigned int *status) {
    atomicExch(status, unsigned(SSM_ERR_TIMEOUT));
    atomicExch(&gave_up, unsigned(SSM_ERR_TIMEOUT));
}
__global__ void gave_up_take_kernel() { gave_up_taken = atomicExch(&gave_up, 0u); }

// Waits for a word to be written. After 2 s, or once another wait has given up, it sets the
// status and returns the zero word (the call's outputs are then not valid).
__device__ __noinline__ unsigned long long wait_slow(const unsigned long long *p, unsigned int *status) {
    const uint64_t t = globaltimer_ns();
    for (;;) {
        for (int k = 0; k < 64; ++k) {
            const unsigned long long v = ld_word(p);
            if (v != 0) return v;
        }
        if (globaltimer_ns() - t > 2000000000ull || *reinterpret_cast<volatile unsigned int *>(status) != 0) {
            give_up(status);
            return 0;
        }
    }
}
__device__ __forceinline__ unsigned long long wait_word(const unsigned long long *p, unsigned int *status) {
    const unsigned long long v = ld_word(p);
    return v != 0 ? v : wait_slow(p, status);
}

// Pairs of neighbouring channels go through the packed float32 instructions: one issue
// slot for both, each rounded as the scalar instruction rounds.
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 sigmoid2(float2 v) {
    const float2 t = mul2(v, two(-kLog2e));
    const float2 f = add2(two(1.0f), make_float2(ex2_approx(t.x), ex2_approx(t.y)));
    return make_float2(rcp_approx(f.x), rcp_approx(f.y));
}
__device__ __forceinline__ float2 small_e2(float2 w) {
    float2 q = fma2(w, two(-0.0011642870f), two(0.0082382215f));
    q = fma2(w, q, two(-0.041649930f));
    q = fma2(w, q, two(0.16666563f));
    q = fma2(w, q, two(-0.5f));
    return mul2(w, fma2(w, q, two(1.0f)));
}
// SMALL: w < 1/2 is known (the rate itself is below 1/2).
template <bool SMALL>
__device__ __forceinline__ float2 decay2(float2 w, float2 &e) {
    if constexpr (SMALL) {
        e = small_e2(w);
        return fma2(e, two(-1.0f), two(1.0f));
    } else {
        float2 a;
        a.x = decay(w.x, e.x);
        a.y = decay(w.y, e.y);
        return a;
    }
}
__device__ __forceinline__ float sqrt_approx(float v) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rsqrt_approx(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// The largest of three. NAN_WINS: a NaN among them is the result; else it is passed over.
template <bool NAN_WINS>
__device__ __forceinline__ float max3(float a, float b, float c) {
    if constexpr (NAN_WINS) {
        float r;
        asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
        return r;
    } else {
        return fmaxf(fmaxf(a, b), c);
    }
}
__device__ __forceinline__ float2 load2(const float *p) { return *reinterpret_cast<const float2 *>(p); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16 *p) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void store2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float2 v) { *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y); }

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Bounded wait for a phase of an mbarrier; false once any wait of the block has given up. A
// try sleeps until the phase completes, 20 us at most: a spinning warp would take issue slots
// from those that compute.
__device__ __forceinline__ bool mbar_sleep(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000)
        : "memory");
    return ok != 0;
}
__device__ __noinline__ bool wait_phase_slow(uint64_t *bar, uint32_t parity, volatile int *abort, unsigned int *status) {
    const uint64_t t = globaltimer_ns();
    while (!mbar_sleep(bar, parity)) {
        if (*abort) return false;
        if (globaltimer_ns() - t > 4000000000ull) {
            *abort = 1;
            give_up(status);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, volatile int *abort, unsigned int *status) {
    return mbar_sleep(bar, parity) || wait_phase_slow(bar, parity, abort, status);
}
// The same for copies in flight when the block gives up.
__device__ __noinline__ void wait_landed(uint64_t *bar, uint32_t parity) {
    const uint64_t t = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t < 1000000000ull) {
    }
}

// ------------------------------------------------------------------- forward
constexpr int kItemSlots = 16;  // of items told of, and of tiles' particulars: more than any warp of a
constexpr int kInfos = 8;       // cluster is ahead of another

// How a call's time is dealt out. A column (64 channels of one sequence) is walked by a cluster
// of `cluster` blocks, which take neighbouring tiles of W K steps at a time; an item is a
// segment of `iters` such rounds of one column.
struct Plan {
    int64_t columns, rounds;  // rounds of a column: ceil(tiles / cluster)
    int cluster, iters, segs;
    unsigned int items;
    bool local;               // one pass for the segments' maps before the pass that writes
    bool drop_handoff;        // test hook, seen by the host only
    int grid;
};

template <typename T>
struct FwdArgs {
    Shape s;
    Plan pl;
    unsigned int *counter, *status;
    unsigned long long *starts;  // [segs][B D] states entering the segments
    Map *maps;                   // [segs][B D] the segments' maps (local pass)
    const T *x, *r, *i;
    int64_t xb, xt, rb, rt, ib, it;
    const uint8_t *reset;
    const float *lam, *h0;
    T *y;
    float *h_last, *states;
};

struct alignas(16) TileInfo {
    unsigned int b, g;  // sequence, group of channels
    int tile;           // of the column; -1: no more
    unsigned int more;  // steps of the sequence in the tile, flags, segment
    static constexpr unsigned int kFirst = 1u << 8, kLast = 1u << 9;  // of its item
    __device__ __forceinline__ int rows() const { return int(more & 255u); }
    __device__ __forceinline__ unsigned int seg() const { return more >> 10; }
};

template <typename T, int K, bool LAG>
struct FwdShared {
    static constexpr int kStages = LAG ? 3 : 2;
    static constexpr int kMaxCluster = LAG || sizeof(T) * K <= 16 ? kMostBlocks : 8;  // (two blocks fit an SM without LAG)
    T stage[kStages][3][kW * K][64];       // x, r, i of a tile
    float4 maps[2][kW][32];                // a warp's map (P, H of a lane's two channels), then its start
    float4 inbox[2][kMaxCluster][32];      // the blocks' maps of a round, from the whole cluster
    float rate[kStages][64];
    unsigned int fresh[kStages][(kW * K + 31) / 32];
    TileInfo tile[kInfos];
    uint64_t full[kStages], empty[kStages], posted[2], mail[2], ready[2], told[kItemSlots];
    unsigned int item[kItemSlots];
    int abort;
};

struct Maps3 {
    CUtensorMap x, r, i;
};

constexpr int kFewColumns = 24;  // up to here LAG: 1536 channels of one sequence (575 against 496 us at L=131072)

constexpr int kShortBack = 16;  // tokens that the few-token backward takes at most

enum Load { kTma, kAsync, kPlain };  // 16-byte rows; pieces of 4 or 8 bytes; elements of 2 bytes

// Decays and inputs of a thread's steps, and their map. RESETS: there may be some among them. FAST: every rate
// between 1e-18 and 1/2 (neither the decay's exponential nor a case for beta = 0 is
// needed), and one reciprocal serves both sigmoids: 1/(1+E) = (1+F)/((1+E)(1+F)); `big`
// tells of gates below -41, whose exponentials' product could overflow and w underflow, and (a NaN itself) of a NaN
// among them where there are resets: r is not used at a reset, and the reciprocal would carry its NaN to the input.
// (B=8 L=4096 D=2048 bfloat16: forward 123 us, backward 263 us; 137 and 312 us with rates that send every warp the other way.)
template <typename T, int K, bool FAST, bool RESETS>
__device__ __forceinline__ float4 fwd_steps_of(const T *x, const T *r, const T *i, const float2 rt, const unsigned int fresh,
                                               float2 (&a)[K], float2 (&h)[K], float &big) {
    float2 P = two(1.0f), H = two(0.0f);
    float top = -1.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float2 sr, si, e;
        if constexpr (FAST) {
            const float2 tr = mul2(load2(r + k * 64), two(-kLog2e)), ti = mul2(load2(i + k * 64), two(-kLog2e));
            top = max3<RESETS>(max3<RESETS>(top, tr.x, tr.y), ti.x, ti.y);
            const float2 fr = add2(two(1.0f), make_float2(ex2_approx(tr.x), ex2_approx(tr.y)));
            const float2 fi = add2(two(1.0f), make_float2(ex2_approx(ti.x), ex2_approx(ti.y)));
            const float2 pr = mul2(fr, fi), rc = make_float2(rcp_approx(pr.x), rcp_approx(pr.y));
            sr = mul2(rc, fi);
            si = mul2(rc, fr);
        } else {
            sr = sigmoid2(load2(r + k * 64));
            si = sigmoid2(load2(i + k * 64));
        }
        a[k] = decay2<FAST>(mul2(rt, sr), e);
        const float2 sq = mul2(e, fma2(e, two(-1.0f), two(2.0f)));
        const float2 u = mul2(si, load2(x + k * 64));
        if constexpr (FAST)
            h[k] = mul2(mul2(sq, make_float2(rsqrt_approx(sq.x), rsqrt_approx(sq.y))), u);
        else
            h[k] = mul2(make_float2(sqrt_approx(sq.x), sqrt_approx(sq.y)), u);
        const bool fr = RESETS && (fresh >> k & 1);
        if (fr) h[k] = u;
        P = mul2(P, a[k]);
        H = fr ? h[k] : fma2(a[k], H, h[k]);
    }
    big = top;
    return make_float4(fresh ? 0.0f : keep(P.x), H.x, fresh ? 0.0f : keep(P.y), H.y);
}
__device__ __forceinline__ float2 apply2(const float4 m, const float2 h) {
    return make_float2(apply(Map{m.x, m.y}, h.x), apply(Map{m.z, m.w}, h.y));
}
__device__ __forceinline__ float4 then2(const float4 f, const float4 g) {
    const Map a = then(Map{f.x, f.y}, Map{g.x, g.y}), b = then(Map{f.z, f.w}, Map{g.z, g.w});
    return make_float4(a.P, a.H, b.P, b.H);
}

// Eight maps in a row, joined two by two: three maps deep instead of seven. The same joints
// give what enters each of them.
struct Eight {
    float4 m[8], two[4], four[2];
    __device__ __forceinline__ void join() {
#pragma unroll
        for (int k = 0; k < 4; ++k) two[k] = then2(m[2 * k], m[2 * k + 1]);
        four[0] = then2(two[0], two[1]), four[1] = then2(two[2], two[3]);
    }
    __device__ __forceinline__ float4 all() const { return then2(four[0], four[1]); }
    __device__ __forceinline__ void enter(const float2 h, float2 (&e)[8]) const {
        e[0] = h, e[4] = apply2(four[0], h);
        e[2] = apply2(two[0], h), e[6] = apply2(two[2], e[4]);
#pragma unroll
        for (int k = 0; k < 8; k += 2) e[k + 1] = apply2(m[k], e[k]);
    }
};
static_assert(kW == 8, "");

// ---------------------------------------------------------- cluster plumbing
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
// Stores into a block of the cluster that complete a transaction on that block's barrier.
__device__ __forceinline__ void send16(uint32_t dst, float4 v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                 "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)), "r"(__float_as_uint(v.w)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void send4(uint32_t dst, uint32_t v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(dst), "r"(v), "r"(bar) : "memory");
}
// N bytes, or N zeros (nothing is read).
template <int N>
__device__ __forceinline__ void copy_async(void *dst, const void *src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(N), "r"(there ? N : 0) : "memory");
}
// The thread's arrival on `bar`, once its cp.async copies so far have landed.
__device__ __forceinline__ void copy_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Loading warps. Three keep up with tiles that are fetched in small pieces; the backward in bfloat16 has one where rows come in
// pairs, for the registers of its other warps (96 instead of 80: B=4 L=4096 D=2054 282 -> 205 us). Odd rows, which pass
// through the loading warps' registers, keep three and 80, and spill most: 472 bytes stored and 784 loaded a thread.
template <Load LOAD, bool BWD = false, int SIZE = 0>
constexpr int kLoaders = LOAD == kTma || (LOAD == kAsync && BWD && SIZE == 2) ? 1 : 3;

// A tensor's tokens, from the first step and channel of a tile on.
template <typename T>
struct Source {
    const T *base;
    int64_t at, stride;
};

// Rows w, w + NL, ... of a tile of one tensor, by one of the loading warps, as asynchronous copies; zeros
// past the last step and the last channel, as TMA fills them. pairs: a lane's two channels
// lie on their own size; else channels lane and lane + 32 come one by one (float32).
template <typename T, int ROWS, int NL>
__device__ __forceinline__ void copy_rows(T (*dst)[64], const Source<T> src, const int steps, const int64_t width, const bool pairs, const int w,
                                          const int lane) {
    if (pairs && steps >= ROWS && width >= 64) {  // a whole tile: nothing to ask
        const T *q = src.base + src.at + w * src.stride + lane * 2;
        const uint32_t to = smem_u32(&dst[w][lane * 2]);
#pragma unroll 8
        for (int k = 0; k < ROWS / NL; ++k, q += NL * src.stride)
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + k * NL * 64 * int(sizeof(T))), "l"(q), "n"(2 * sizeof(T)) : "memory");
        if (w < ROWS % NL)
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + ROWS / NL * NL * 64 * int(sizeof(T))), "l"(q), "n"(2 * sizeof(T)) : "memory");
    } else if (pairs) {
        const bool on = lane * 2 < width;
        const T *q = src.base + src.at + w * src.stride + lane * 2;
#pragma unroll 4
        for (int k = w; k < ROWS; k += NL, q += NL * src.stride)
            copy_async<2 * sizeof(T)>(&dst[k][lane * 2], on && k < steps ? q : src.base, on && k < steps);
    } else if constexpr (sizeof(T) == 4) {
        const bool on0 = lane < width, on1 = lane + 32 < width;
        const T *q = src.base + src.at + w * src.stride + lane;
#pragma unroll 4
        for (int k = w; k < ROWS; k += NL, q += NL * src.stride) {
            copy_async<4>(&dst[k][lane], on0 && k < steps ? q : src.base, on0 && k < steps);
            copy_async<4>(&dst[k][lane + 32], on1 && k < steps ? q + 32 : src.base, on1 && k < steps);
        }
    }
}

// The same element by element, through registers: N rows of all the tensors at a time, since what is on its way
// at once sets the rate (three tensors one after the other: 148 us for B=2 L=8191 D=1001 forward).
template <typename T, int ROWS, int NL, int NT>
__device__ __forceinline__ void move_rows(T (*dst)[ROWS][64], const Source<T> (&src)[NT], const int steps, const int64_t width, const int w,
                                          const int lane) {
    constexpr int N = 8;
    const bool on0 = lane < width, on1 = lane + 32 < width;
    for (int k0 = w; k0 < ROWS; k0 += NL * N) {
        T v[NT][N][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const T *q = src[t].base + src[t].at + k0 * src[t].stride + lane;
#pragma unroll
            for (int n = 0; n < N; ++n, q += NL * src[t].stride) {
                const bool in = k0 + NL * n < min(ROWS, steps);
                v[t][n][0] = on0 && in ? q[0] : Tok<T>::from_f(0.0f);
                v[t][n][1] = on1 && in ? q[32] : Tok<T>::from_f(0.0f);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (k0 + NL * n < ROWS) {
                    dst[t][k0 + NL * n][lane] = v[t][n][0];
                    dst[t][k0 + NL * n][lane + 32] = v[t][n][1];
                }
    }
}

// What the loading warps do, in both directions: take items, and bring their rounds' tiles into the stages
// through `issue`; tile_of gives the tile of a round.
template <Load LOAD, bool RESETS, int ROWS, typename Args, typename Shared, typename TileOf, typename Issue>
__device__ __forceinline__ void load_tiles(const Args &p, Shared &s, const int w, const int lane, const uint32_t rank, const unsigned int C,
                                           const unsigned int columns, const unsigned int groups, const bool counted, const TileOf &tile_of, const Issue &issue) {
    constexpr int kStages = Shared::kStages;
    unsigned int it = 0;
    for (unsigned int q = 0;; ++q) {
        const int slot = q % kItemSlots;
        if (w == 0 && lane == 0) {
            mbar_arrive_expect_tx(&s.told[slot], 4);
            if (rank == 0) {
                const unsigned int item = counted ? atomicAdd(p.counter, 1u) : blockIdx.x / C + q * (gridDim.x / C);
                for (unsigned int k = 0; k < C; ++k) send4(peer_addr(&s.item[slot], k), item, peer_addr(&s.told[slot], k));
            }
        }
        bool ok = __all_sync(0xffffffffu, wait_phase(&s.told[slot], (q / kItemSlots) & 1, &s.abort, p.status));
        const unsigned int item = s.item[slot];
        const bool done = !ok || item >= p.pl.items;
        const unsigned int seg = done ? 0 : item / columns, col = done ? 0 : item % columns;
        const int r0 = int(seg) * p.pl.iters, r1 = done ? r0 + 1 : int(min(int64_t(r0 + p.pl.iters), p.pl.rounds));
        const unsigned int g = col % groups, b = col / groups;
        // once an item: the rates; a round ahead: the tile's resets, a lane holding every 32nd step's
        float rates[2] = {0.25f, 0.25f};
        unsigned char mark[ROWS / 32] = {};
        const bool marks = RESETS && w == 0 && !done;
        const auto look = [&](const int tile) {
#pragma unroll
            for (int k = 0; k < ROWS / 32; ++k) {
                const int64_t t = int64_t(tile) * ROWS + k * 32 + lane;
                mark[k] = t < p.s.L ? p.reset[int64_t(b) * p.s.L + t] : 0;
            }
        };
        if (w == 0 && !done) {
            if (marks) look(tile_of(r0));
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int64_t d = int64_t(g) * 64 + lane * 2 + v;
                if (d < p.s.D) rates[v] = rate(p.lam[d], p.s.c);
            }
        }
        for (int round = r0; round < r1; ++round, ++it) {
            const int st = it % kStages;
            ok = ok && (it < kStages || wait_phase(&s.empty[st], (it / kStages - 1) & 1, &s.abort, p.status));
            if (!__all_sync(0xffffffffu, ok)) {  // given up: not before the copies under way have landed
                if (LOAD == kTma)
                    for (unsigned int k = it < kStages ? 0 : it - kStages; k < it; ++k) wait_landed(&s.full[k % kStages], (k / kStages) & 1);
                else
                    asm volatile("cp.async.wait_all;" ::: "memory");
                return;
            }
            const int tile = done ? -1 : tile_of(round);
            if (!done)
                issue(st, g, b, tile);
            else if (LOAD == kTma && lane == 0)
                mbar_arrive(&s.full[st]);
            if (w == 0) *reinterpret_cast<float2 *>(&s.rate[st][lane * 2]) = make_float2(rates[0], rates[1]);
            if (marks) {  // the tile's resets, 32 steps to a word
#pragma unroll
                for (int k = 0; k < ROWS / 32; ++k) {
                    const unsigned int word = __ballot_sync(0xffffffffu, mark[k] != 0);
                    if (lane == 0) s.fresh[st][k] = word;
                }
                if (round + 1 < r1) look(tile_of(round + 1));
            }
            if (w == 0 && lane == 0) {
                const unsigned int rows = unsigned(max(int64_t(0), min(int64_t(ROWS), p.s.L - int64_t(tile) * ROWS)));
                s.tile[it % kInfos] = {b, g, tile, rows | (round == r0 ? TileInfo::kFirst : 0u) | (round == r1 - 1 ? TileInfo::kLast : 0u) | seg << 10};
            }
            __syncwarp();
            if (w == 0 && lane == 0) mbar_arrive(&s.full[st]);
            if (LOAD == kAsync)
                copy_async_arrive(&s.full[st]);
            else if (LOAD == kPlain)
                mbar_arrive(&s.full[st]);
        }
        if (done) return;
    }
}

// Warps 0..7 compute; warp 8 carries the state along; the others load.
//  - A computing warp turns its K steps of a tile into decays and inputs in registers and posts
//    their map in shared memory.
//  - Warp 8 composes the block's map, sends it to every block of the cluster, and has from the
//    round's maps the state entering its block's tile, each of the tile's warps and the next
//    round. The same sums in every block: nothing comes back.
//  - Then every computing warp knows the state entering its steps, and writes them.
// No barrier joins the computing warps: they meet warp 8 on mbarriers only.
// Segments of a column are handed out in the order of time by a counter; a segment starts from
// the state that its predecessor leaves in the workspace, which with more columns than clusters is
// there long before (and after a local pass is always there).
// LAG: a tile's outputs are written one round late, once the next tile's steps are in registers too; by then its
// start is there, and no warp waits for the way to the cluster and back. That takes the registers of a whole SM per
// block. It pays where there are too few columns for two blocks an SM anyway (B=1 L=131072 D=1024: 481 -> 340 us, D=512 263 -> 189 us);
// with enough of them the other block fills the wait (D=2048: 587 us without, 707 with).
// RESETS: there is a reset array (its selections in a kernel that never uses them cost registers: 583 against 615 us for
// L=65536 D=5120).
template <typename T, int K, Load LOAD, bool LAG, bool RESETS>
__global__ void __launch_bounds__((kW + 1 + kLoaders<LOAD>) * 32, LAG ? 1 : 2)
    gated_fwd_kernel(const FwdArgs<T> p, const __grid_constant__ Maps3 tm, const bool pairs) {
    static_assert(kChunk % K == 0, "a chunk starts at a warp's first step");
    static_assert(32 % K == 0 && kW * K % 32 == 0, "a warp's resets lie in one word");
    static_assert(kW * K < 256, "a tile's steps take eight bits");
    static_assert(LAG || sizeof(FwdShared<T, K, LAG>) <= 228 * 1024 / 2 - 1024, "two blocks share an SM");
    constexpr int NL = kLoaders<LOAD>, ROWS = kW * K, kStages = FwdShared<T, K, LAG>::kStages;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    FwdShared<T, K, LAG> &s = *reinterpret_cast<FwdShared<T, K, LAG> *>(smem_raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned int groups = unsigned(p.s.groups), columns = unsigned(p.pl.columns), C = unsigned(p.pl.cluster);
    const uint32_t rank = cluster_rank();
    const bool counted = p.pl.segs > 1 && !p.pl.local;
    const int64_t n = p.s.B * p.s.D;
    if (threadIdx.x == 0) {
        for (int k = 0; k < kStages; ++k) mbar_init(&s.full[k], LOAD == kTma ? 2 : NL * 32 + 1), mbar_init(&s.empty[k], kW + 1);
        for (int k = 0; k < 2; ++k) mbar_init(&s.posted[k], kW), mbar_init(&s.mail[k], 1), mbar_init(&s.ready[k], 1);
        for (int k = 0; k < kItemSlots; ++k) mbar_init(&s.told[k], 1);
        s.abort = 0;
        fence_mbar_init();
        if (blockIdx.x == 0 && (p.pl.segs == 1 || p.maps)) *p.status = 0;  // (else cleared with the states)
    }
    cluster_sync_all();

    if (warp > kW) {
        // ------------------------------------------------------------ loading
        load_tiles<LOAD, RESETS, ROWS>(p, s, warp - kW - 1, lane, rank, C, columns, groups, counted, [&](const int round) { return round * int(C) + int(rank); },
                         [&](const int st, const unsigned int g, const unsigned int b, const int tile) {
            const int64_t t0 = int64_t(tile) * ROWS;
            if constexpr (LOAD == kTma) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(&s.full[st], sizeof(s.stage[0]));
                    tma_load_3d(s.stage[st][0], &tm.x, &s.full[st], int(g * 64), int(t0), int(b));
                    tma_load_3d(s.stage[st][1], &tm.r, &s.full[st], int(g * 64), int(t0), int(b));
                    tma_load_3d(s.stage[st][2], &tm.i, &s.full[st], int(g * 64), int(t0), int(b));
                }
            } else {
                const int w = warp - kW - 1, steps = int(max(int64_t(0), min(int64_t(ROWS), p.s.L - t0)));
                const int64_t d = int64_t(g) * 64, width = p.s.D - d;
                const Source<T> src[3] = {{p.x, b * p.xb + t0 * p.xt + d, p.xt}, {p.r, b * p.rb + t0 * p.rt + d, p.rt}, {p.i, b * p.ib + t0 * p.it + d, p.it}};
                if constexpr (LOAD == kPlain) {
                    move_rows<T, ROWS, NL>(s.stage[st], src, steps, width, w, lane);
                } else {
#pragma unroll
                    for (int t = 0; t < 3; ++t) copy_rows<T, ROWS, NL>(s.stage[st][t], src[t], steps, width, pairs, w, lane);
                }
            }
        });
    } else if (warp == kW) {
        // ---------------------------------------------------------- the carry
        float2 S = two(0.0f);
        float4 M = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
        for (unsigned int it = 0;; ++it) {
            const bool ok = wait_phase(&s.full[it % kStages], (it / kStages) & 1, &s.abort, p.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            const TileInfo t = s.tile[it % kInfos];
            if (t.tile < 0) break;
            __syncwarp();
            // (a stage is refilled once this warp has seen it too: a phase it misses would look like one to come)
            if (lane == 0) mbar_arrive(&s.empty[it % kStages]);
            const int64_t d = int64_t(t.g) * 64 + lane * 2, o = int64_t(t.b) * p.s.D + d;
            const int have = int(min(int64_t(2), p.s.D - d));  // channels of this lane (at most 2)
            const int buf = it & 1;
            const uint32_t phase = (it >> 1) & 1;
            if (lane == 0 && C > 1) mbar_arrive_expect_tx(&s.mail[buf], C * sizeof(s.inbox[0][0]));
            wait_phase(&s.posted[buf], phase, &s.abort, p.status);
            Eight f;
#pragma unroll
            for (int w = 0; w < kW; ++w) f.m[w] = s.maps[buf][w][lane];
            f.join();
            const float4 own = f.all();
            if (C > 1)
                for (unsigned int k = 0; k < C; ++k)
                    send16(peer_addr(&s.inbox[buf][rank][lane], k), own, peer_addr(&s.mail[buf], k));
            if (t.more & TileInfo::kFirst) {
                S = two(0.0f);
                M = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
                if (!p.maps) {
                    const unsigned long long *q = p.starts + int64_t(t.seg()) * n + o;
                    if (t.seg() == 0) {
                        if (p.h0 && have > 0) S.x = p.h0[o];
                        if (p.h0 && have > 1) S.y = p.h0[o + 1];
                    } else {
                        if (have > 0) S.x = __uint_as_float(unsigned(wait_word(q, p.status)));
                        if (have > 1) S.y = __uint_as_float(unsigned(wait_word(q + 1, p.status)));
                    }
                }
            }
            float2 mine = S;
            if (C > 1) {
                wait_phase(&s.mail[buf], phase, &s.abort, p.status);
                for (unsigned int k = 0; k < C; ++k) {
                    const float4 g = s.inbox[buf][k][lane];
                    if (k == rank) mine = S;
                    S = apply2(g, S);
                    if (p.maps) M = then2(M, g);
                }
            } else {
                S = apply2(own, S);
                if (p.maps) M = then2(M, own);
            }
            float2 e[kW];
            f.enter(mine, e);
#pragma unroll
            for (int w = 0; w < kW; ++w) *reinterpret_cast<float2 *>(&s.maps[buf][w][lane]) = e[w];
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.ready[buf]);
            if ((t.more & TileInfo::kLast) && rank == 0) {
                if (p.maps) {
                    if (have > 0) p.maps[int64_t(t.seg()) * n + o] = Map{M.x, M.y};
                    if (have > 1) p.maps[int64_t(t.seg()) * n + o + 1] = Map{M.z, M.w};
                } else if (counted && int(t.seg()) + 1 < p.pl.segs) {
                    unsigned long long *q = p.starts + int64_t(t.seg() + 1) * n + o;
                    if (have > 0) st_word(q, pack(S.x));
                    if (have > 1) st_word(q + 1, pack(S.y));
                }
            }
        }
    } else {
        // ---------------------------------------------------------- computing
        // read: tile `it` into decays, inputs and resets, and its map posted; write: its outputs.
        const auto read = [&](const unsigned int it, float2(&a)[K], float2(&h)[K], unsigned int &fresh) -> bool {
            const int st = it % kStages;
            const bool ok = wait_phase(&s.full[st], (it / kStages) & 1, &s.abort, p.status);
            if (!__all_sync(0xffffffffu, ok)) return false;
            const TileInfo t = s.tile[it % kInfos];
            if (t.tile < 0) return false;
            fresh = RESETS ? s.fresh[st][warp * K / 32] >> (warp * K % 32) & ((1u << K) - 1u) : 0u;
            const float2 rt = *reinterpret_cast<const float2 *>(&s.rate[st][lane * 2]);
            const T *x = &s.stage[st][0][warp * K][lane * 2], *r = &s.stage[st][1][warp * K][lane * 2],
                    *i = &s.stage[st][2][warp * K][lane * 2];
            float4 m;
            float big = 1e30f;
            if (__all_sync(0xffffffffu, fmaxf(rt.x, rt.y) < 0.5f && fminf(rt.x, rt.y) > 1e-18f))
                m = !RESETS || fresh == 0 ? fwd_steps_of<T, K, true, false>(x, r, i, rt, 0u, a, h, big)
                                          : fwd_steps_of<T, K, true, RESETS>(x, r, i, rt, fresh, a, h, big);
            if (__any_sync(0xffffffffu, !(big <= 60.0f))) m = fwd_steps_of<T, K, false, RESETS>(x, r, i, rt, fresh, a, h, big);
            s.maps[it & 1][warp][lane] = m;
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s.posted[it & 1]);
                mbar_arrive(&s.empty[st]);
            }
            return true;
        };
        const auto write = [&](const unsigned int it, const float2(&a)[K], const float2(&h)[K], const unsigned int fresh) {
            wait_phase(&s.ready[it & 1], (it >> 1) & 1, &s.abort, p.status);
            const TileInfo t = s.tile[it % kInfos];
            const unsigned int b = t.b;
            const int64_t d = int64_t(t.g) * 64 + lane * 2;
            const int64_t t0 = int64_t(t.tile) * ROWS + warp * K;
            const int steps = max(0, min(K, t.rows() - warp * K));
            if (!p.maps && d < p.s.D && steps > 0) {
                float2 hs = *reinterpret_cast<const float2 *>(&s.maps[it & 1][warp][lane]);
                const bool both = d + 1 < p.s.D;
                if (p.states && t0 % kChunk == 0) {
                    float *q = p.states + (int64_t(b) * ((p.s.L + kChunk - 1) / kChunk) + t0 / kChunk) * p.s.D + d;
                    q[0] = hs.x;
                    if (both) q[1] = hs.y;
                }
                T *yp = p.y + (int64_t(b) * p.s.L + t0) * p.s.D + d;
                if (steps == K && (!RESETS || fresh == 0) && p.y && pairs) {
#pragma unroll
                    for (int k = 0; k < K; ++k, yp += p.s.D) {
                        hs = fma2(a[k], hs, h[k]);
                        store2(yp, hs);
                    }
                } else if (RESETS && steps == K && p.y && pairs) {
#pragma unroll
                    for (int k = 0; k < K; ++k, yp += p.s.D) {
                        hs = (fresh >> k & 1) ? h[k] : fma2(a[k], hs, h[k]);
                        store2(yp, hs);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < K; ++k, yp += p.s.D)
                        if (k < steps) {
                            hs = RESETS && (fresh >> k & 1) ? h[k] : fma2(a[k], hs, h[k]);
                            if (p.y && pairs) {
                                store2(yp, hs);
                            } else if (p.y) {
                                yp[0] = Tok<T>::from_f(hs.x);
                                if (both) yp[1] = Tok<T>::from_f(hs.y);
                            }
                        }
                }
                if (p.h_last && t0 + steps == p.s.L) {
                    p.h_last[int64_t(b) * p.s.D + d] = hs.x;
                    if (both) p.h_last[int64_t(b) * p.s.D + d + 1] = hs.y;
                }
            }
            __syncwarp();
        };
        float2 a0[K], h0[K];
        unsigned int f0 = 0;
        if constexpr (LAG) {
            float2 a1[K], h1[K];
            unsigned int f1 = 0;
            bool more = read(0, a0, h0, f0);
            for (unsigned int it = 0; more; it += 2) {
                const bool next = read(it + 1, a1, h1, f1);
                write(it, a0, h0, f0);
                if (!next) break;
                more = read(it + 2, a0, h0, f0);
                write(it + 1, a1, h1, f1);
            }
        } else {
            for (unsigned int it = 0; read(it, a0, h0, f0); ++it) write(it, a0, h0, f0);
        }
    }
    __syncwarp();
    cluster_sync_all();  // no block leaves while another may still write to it
}

// The states entering the segments, from their maps.
__global__ void __launch_bounds__(128)
    gated_starts_kernel(int64_t n, int segs, const float *__restrict__ h0, const Map *__restrict__ maps, unsigned long long *__restrict__ starts) {
    const int64_t k = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (k >= n) return;
    float h = h0 ? h0[k] : 0.0f;
#pragma unroll 8
    for (int s = 0; s + 1 < segs; ++s) {
        h = apply(maps[s * n + k], h);
        starts[(s + 1) * n + k] = pack(h);
    }
}

// ------------------------------------------------------------------ backward
template <typename T>
struct BwdArgs {
    Shape s;
    Plan pl;
    unsigned int *counter, *status;
    unsigned long long *starts;  // [segs][B D] adjoints entering the segments from their right
    Map *maps;                   // [segs][B D] the segments' maps (local pass)
    const T *x, *r, *i, *dy;
    int64_t xb, xt, rb, rt, ib, it;
    const uint8_t *reset;
    const float *lam, *states, *dh_last;
    T *dx, *dr, *di;
    float *dh0, *parts;          // parts: [segs][cluster][warps][B][D] sums of dw sigmoid(r)
};

template <typename T, int K>
struct BwdShared {
    static constexpr int kStages = 2;
    static constexpr int kMaxCluster = kMostBlocks;
    T stage[kStages][4][kW * K][64];  // x, r, i, dy of a tile; then dx, dr, di in the first three
    float4 maps[2][kW][32];           // a warp's map of the state, then its start: h and g of a lane's two channels
    float2 adj[2][kW][32];            // H of its map of the adjoint (P is the same)
    float4 inbox[2][kMaxCluster][32];
    float rate[kStages][64];
    unsigned int fresh[kStages][(kW * K + 31) / 32];
    TileInfo tile[kInfos];
    uint64_t full[kStages], empty[kStages], posted[2], mail[2], ready[2], told[kItemSlots];
    unsigned int item[kItemSlots];
    int abort;
};

struct Maps7 {
    CUtensorMap x, r, i, dy, dx, dr, di;
};

// v_t = dL/dh_t follows v_t = dy_t + a_{t+1} v_{t+1}; with g_t = a_t v_t, what a step hands to
// the one before it, a piece of time acts on the g entering from its right as g -> P g + G
// with the forward's P. Steps past the end are the identity. `big` tells of a NaN gate in any case: the adjoint goes by
// r alone, and the shared reciprocal would carry a NaN of i to it.
template <typename T, int K, bool FAST, bool RESETS>
__device__ __forceinline__ void bwd_steps_of(const T *x, const T *r, const T *i, const T *dy, const float2 rt, const unsigned int fresh,
                                             const int steps, float2 (&a)[K], float2 (&h)[K], float2 (&sr)[K], float2 (&si)[K],
                                             float4 &f, float2 &g, float &big) {
    float2 P = two(1.0f), H = two(0.0f), G = two(0.0f);
    float top = -1.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float2 e;
        if constexpr (FAST) {
            const float2 tr = mul2(load2(r + k * 64), two(-kLog2e)), ti = mul2(load2(i + k * 64), two(-kLog2e));
            top = max3<true>(max3<true>(top, tr.x, tr.y), ti.x, ti.y);
            const float2 fr = add2(two(1.0f), make_float2(ex2_approx(tr.x), ex2_approx(tr.y)));
            const float2 fi = add2(two(1.0f), make_float2(ex2_approx(ti.x), ex2_approx(ti.y)));
            const float2 pr = mul2(fr, fi), rc = make_float2(rcp_approx(pr.x), rcp_approx(pr.y));
            sr[k] = mul2(rc, fi);
            si[k] = mul2(rc, fr);
        } else {
            sr[k] = sigmoid2(load2(r + k * 64));
            si[k] = sigmoid2(load2(i + k * 64));
        }
        a[k] = decay2<FAST>(mul2(rt, sr[k]), e);
        const float2 sq = mul2(e, fma2(e, two(-1.0f), two(2.0f)));
        const float2 u = mul2(si[k], load2(x + k * 64));
        if constexpr (FAST)
            h[k] = mul2(mul2(sq, make_float2(rsqrt_approx(sq.x), rsqrt_approx(sq.y))), u);
        else
            h[k] = mul2(make_float2(sqrt_approx(sq.x), sqrt_approx(sq.y)), u);
        const bool fr = RESETS && (fresh >> k & 1);
        if (fr) h[k] = u;
        if (!FAST && fr) sr[k] = two(0.0f);  // (a NaN there reaches no gradient)
        if (!FAST && k >= steps) a[k] = two(1.0f);
        P = mul2(P, a[k]);
        H = fr ? h[k] : fma2(a[k], H, h[k]);
    }
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
        if (FAST || k < steps) G = RESETS && (fresh >> k & 1) ? two(0.0f) : mul2(a[k], add2(load2(dy + k * 64), G));
    }
    big = top;
    f = make_float4(fresh ? 0.0f : keep(P.x), H.x, fresh ? 0.0f : keep(P.y), H.y);
    g = G;
}

// The gradients of a thread's steps, from the state entering them on the left and the adjoint on the right, given
// to out(k, dx, dr, di) from the last step to the first; the sum of dw sigmoid(r).
template <typename T, int K, bool FAST, bool RESETS, typename Out>
__device__ __forceinline__ float2 bwd_grads_of(const T *x, const T *dy, const float2 rt, const unsigned int fresh, const int steps,
                                               const float2 (&a)[K], float2 (&h)[K], const float2 (&sr)[K], const float2 (&si)[K],
                                               float2 hs, float2 gs, const Out &out) {
#pragma unroll
    for (int k = 0; k < K; ++k) {  // h[k]: the state before the step
        const float2 next = RESETS && (fresh >> k & 1) ? h[k] : fma2(a[k], hs, h[k]);
        h[k] = hs;
        hs = next;
    }
    float2 dl = two(0.0f);
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
        if (!FAST && k >= steps) continue;
        const bool fr = RESETS && (fresh >> k & 1);
        const float2 v = add2(load2(dy + k * 64), gs), w = mul2(rt, sr[k]), u = mul2(si[k], load2(x + k * 64));
        float2 e = small_e2(w);
        if (!FAST) e = make_float2(w.x < 0.5f ? e.x : 1.0f - a[k].x, w.y < 0.5f ? e.y : 1.0f - a[k].y);
        const float2 sq = mul2(e, fma2(e, two(-1.0f), two(2.0f)));
        const float2 q = FAST ? make_float2(rsqrt_approx(sq.x), rsqrt_approx(sq.y)) : make_float2(inv_beta(sq.x), inv_beta(sq.y));
        const float2 vb = fr ? v : mul2(v, mul2(sq, q)), av = mul2(a[k], v);
        // dL/dw = a v (a u / beta - h_{t-1}); beta -> 0 only as w -> 0, where w / beta -> 0
        float2 dw = mul2(av, fma2(mul2(a[k], q), u, mul2(h[k], two(-1.0f))));
        if (fr) dw = two(0.0f);
        const float2 ws = mul2(w, fma2(sr[k], two(-1.0f), two(1.0f))), vu = mul2(vb, u);
        out(k, mul2(vb, si[k]), mul2(dw, ws), mul2(vu, fma2(si[k], two(-1.0f), two(1.0f))));
        dl = fma2(dw, sr[k], dl);
        gs = fr ? two(0.0f) : av;
    }
    return dl;
}

// The forward's scheme from the end of time to its beginning: a tile is a chunk, whose state
// is known, so only the adjoint passes from block to block. The decays, inputs and sigmoids of a thread's
// steps stay in registers between the two passes over them; a tile's tokens stay in
// its stage until its gradients, written over them, have left.
template <typename T, int K, Load LOAD, bool RESETS>
__global__ void __launch_bounds__((kW + 1 + kLoaders<LOAD, true, sizeof(T)>) * 32, sizeof(T) == 2 ? 2 : 1)
    gated_bwd_kernel(const BwdArgs<T> p, const __grid_constant__ Maps7 tm, const bool pairs) {
    constexpr int NL = kLoaders<LOAD, true, sizeof(T)>, ROWS = kW * K, kStages = BwdShared<T, K>::kStages;
    static_assert(ROWS == kChunk, "a tile is a chunk");
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    BwdShared<T, K> &s = *reinterpret_cast<BwdShared<T, K> *>(smem_raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned int groups = unsigned(p.s.groups), columns = unsigned(p.pl.columns), C = unsigned(p.pl.cluster);
    const uint32_t rank = cluster_rank();
    const bool counted = p.pl.segs > 1 && !p.pl.local;
    const int64_t n = p.s.B * p.s.D, chunks = (p.s.L + kChunk - 1) / kChunk;
    if (threadIdx.x == 0) {
        for (int k = 0; k < kStages; ++k) mbar_init(&s.full[k], LOAD == kTma ? 2 : NL * 32 + 1), mbar_init(&s.empty[k], kW + 1);
        for (int k = 0; k < 2; ++k) mbar_init(&s.posted[k], kW), mbar_init(&s.mail[k], 1), mbar_init(&s.ready[k], 1);
        for (int k = 0; k < kItemSlots; ++k) mbar_init(&s.told[k], 1);
        s.abort = 0;
        fence_mbar_init();
        if (blockIdx.x == 0 && (p.pl.segs == 1 || p.maps)) *p.status = 0;  // (else cleared with the states)
    }
    cluster_sync_all();

    if (warp > kW) {
        // ------------------------------------------------------------ loading
        load_tiles<LOAD, RESETS, ROWS>(p, s, warp - kW - 1, lane, rank, C, columns, groups, counted, [&](const int round) { return int(p.pl.rounds * C) - 1 - (round * int(C) + int(rank)); },
                         [&](const int st, const unsigned int g, const unsigned int b, const int tile) {
            const int64_t t0 = int64_t(tile) * ROWS;
            if constexpr (LOAD == kTma) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(&s.full[st], sizeof(s.stage[0]));
                    tma_load_3d(s.stage[st][0], &tm.x, &s.full[st], int(g * 64), int(t0), int(b));
                    tma_load_3d(s.stage[st][1], &tm.r, &s.full[st], int(g * 64), int(t0), int(b));
                    tma_load_3d(s.stage[st][2], &tm.i, &s.full[st], int(g * 64), int(t0), int(b));
                    tma_load_3d(s.stage[st][3], &tm.dy, &s.full[st], int(g * 64), int(t0), int(b));
                }
            } else {
                const int w = warp - kW - 1, steps = int(max(int64_t(0), min(int64_t(ROWS), p.s.L - t0)));
                const int64_t d = int64_t(g) * 64, width = p.s.D - d;
                const Source<T> src[4] = {{p.x, b * p.xb + t0 * p.xt + d, p.xt}, {p.r, b * p.rb + t0 * p.rt + d, p.rt}, {p.i, b * p.ib + t0 * p.it + d, p.it},
                                          {p.dy, (int64_t(b) * p.s.L + t0) * p.s.D + d, p.s.D}};
                if constexpr (LOAD == kPlain) {
                    move_rows<T, ROWS, NL>(s.stage[st], src, steps, width, w, lane);
                } else {
#pragma unroll
                    for (int t = 0; t < 4; ++t) copy_rows<T, ROWS, NL>(s.stage[st][t], src[t], steps, width, pairs, w, lane);
                }
            }
        });
    } else if (warp == kW) {
        // ---------------------------------------------------------- the carry
        float2 S = two(0.0f);
        float4 M = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
        for (unsigned int it = 0;; ++it) {
            const bool ok = wait_phase(&s.full[it % kStages], (it / kStages) & 1, &s.abort, p.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            const TileInfo t = s.tile[it % kInfos];
            if (t.tile < 0) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.empty[it % kStages]);
            const unsigned int b = t.b;
            const int64_t d = int64_t(t.g) * 64 + lane * 2, o = int64_t(b) * p.s.D + d;
            const int have = int(min(int64_t(2), p.s.D - d));  // channels of this lane (at most 2)
            const int buf = it & 1;
            const uint32_t phase = (it >> 1) & 1;
            if (lane == 0 && C > 1) mbar_arrive_expect_tx(&s.mail[buf], C * sizeof(s.inbox[0][0]));
            float2 hs = two(0.0f);
            if (t.tile < chunks && !p.maps) {
                const float *q = p.states + (int64_t(b) * chunks + t.tile) * p.s.D + d;
                if (have > 0) hs.x = q[0];
                if (have > 1) hs.y = q[1];
            }
            wait_phase(&s.posted[buf], phase, &s.abort, p.status);
            Eight r;  // the adjoint's maps, from the last warp to the first
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const float4 m = s.maps[buf][w][lane];
                const float2 g = s.adj[buf][w][lane];
                r.m[kW - 1 - w] = make_float4(m.x, g.x, m.z, g.y);
            }
            r.join();
            const float4 own = r.all();
            if (C > 1)
                for (unsigned int k = 0; k < C; ++k)
                    send16(peer_addr(&s.inbox[buf][rank][lane], k), own, peer_addr(&s.mail[buf], k));
            if (t.more & TileInfo::kFirst) {
                S = two(0.0f);
                M = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
                if (!p.maps) {
                    const unsigned long long *q = p.starts + int64_t(t.seg()) * n + o;
                    if (t.seg() == 0) {
                        if (p.dh_last && have > 0) S.x = p.dh_last[o];
                        if (p.dh_last && have > 1) S.y = p.dh_last[o + 1];
                    } else {
                        if (have > 0) S.x = __uint_as_float(unsigned(wait_word(q, p.status)));
                        if (have > 1) S.y = __uint_as_float(unsigned(wait_word(q + 1, p.status)));
                    }
                }
            }
            // the states entering the warps' steps, while the mail is under way
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const float4 m = s.maps[buf][w][lane];
                *reinterpret_cast<float2 *>(&s.maps[buf][w][lane]) = hs;
                hs = apply2(m, hs);
            }
            float2 mine = S;
            if (C > 1) {
                wait_phase(&s.mail[buf], phase, &s.abort, p.status);
                for (unsigned int k = 0; k < C; ++k) {
                    const float4 g = s.inbox[buf][k][lane];
                    if (k == rank) mine = S;
                    S = apply2(g, S);
                    if (p.maps) M = then2(M, g);
                }
            } else {
                S = apply2(own, S);
                if (p.maps) M = then2(M, own);
            }
            float2 e[kW];
            r.enter(mine, e);
#pragma unroll
            for (int w = 0; w < kW; ++w) reinterpret_cast<float2 *>(&s.maps[buf][w][lane])[1] = e[kW - 1 - w];
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.ready[buf]);
            if ((t.more & TileInfo::kLast) && rank == 0) {
                if (p.maps) {
                    if (have > 0) p.maps[int64_t(t.seg()) * n + o] = Map{M.x, M.y};
                    if (have > 1) p.maps[int64_t(t.seg()) * n + o + 1] = Map{M.z, M.w};
                } else if (int(t.seg()) + 1 == p.pl.segs) {
                    if (p.dh0 && have > 0) p.dh0[o] = S.x;
                    if (p.dh0 && have > 1) p.dh0[o + 1] = S.y;
                } else if (counted) {
                    unsigned long long *q = p.starts + int64_t(t.seg() + 1) * n + o;
                    if (have > 0) st_word(q, pack(S.x));
                    if (have > 1) st_word(q + 1, pack(S.y));
                }
            }
        }
    } else {
        // ---------------------------------------------------------- computing
        float2 dl = two(0.0f);
        for (unsigned int it = 0;; ++it) {
            const int st = it % kStages, buf = it & 1;
            const bool ok = wait_phase(&s.full[st], (it / kStages) & 1, &s.abort, p.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            const TileInfo t = s.tile[it % kInfos];
            if (t.tile < 0) break;
            const unsigned int b = t.b;
            const int64_t d = int64_t(t.g) * 64 + lane * 2;
            const int64_t t0 = int64_t(t.tile) * ROWS + warp * K;
            const int steps = max(0, min(K, t.rows() - warp * K));
            const unsigned int fresh = RESETS ? s.fresh[st][warp * K / 32] >> (warp * K % 32) & ((1u << K) - 1u) : 0u;
            const float2 rt = *reinterpret_cast<const float2 *>(&s.rate[st][lane * 2]);
            T *x = &s.stage[st][0][warp * K][lane * 2], *r = &s.stage[st][1][warp * K][lane * 2], *i = &s.stage[st][2][warp * K][lane * 2];
            const T *dy = &s.stage[st][3][warp * K][lane * 2];
            float2 a[K], h[K], sr[K], si[K], g;
            float4 m;
            float big = 1e30f;
            if (steps == K && __all_sync(0xffffffffu, fmaxf(rt.x, rt.y) < 0.5f && fminf(rt.x, rt.y) > 1e-18f))
                bwd_steps_of<T, K, true, RESETS>(x, r, i, dy, rt, fresh, steps, a, h, sr, si, m, g, big);
            const bool slow = __any_sync(0xffffffffu, !(big <= 60.0f));
            if (slow) bwd_steps_of<T, K, false, RESETS>(x, r, i, dy, rt, fresh, steps, a, h, sr, si, m, g, big);
            s.maps[buf][warp][lane] = m;
            s.adj[buf][warp][lane] = g;
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.posted[buf]);
            if (LOAD == kTma && it > 0 && lane == 0) {  // the last tile's gradients have left its stage
                bulk_wait_read<0>();
                mbar_arrive(&s.empty[(it - 1) % kStages]);
            }
            wait_phase(&s.ready[buf], (it >> 1) & 1, &s.abort, p.status);
            if (!p.maps) {
                const float4 begin = s.maps[buf][warp][lane];
                const float2 hs = make_float2(begin.x, begin.y), gs = make_float2(begin.z, begin.w);
                if (t.more & TileInfo::kFirst) dl = two(0.0f);
                if constexpr (LOAD == kTma) {
                    const auto out = [&](const int k, const float2 gx, const float2 gr, const float2 gi) {
                        store2(x + k * 64, gx);
                        store2(r + k * 64, gr);
                        store2(i + k * 64, gi);
                    };
                    dl = add2(dl, slow ? bwd_grads_of<T, K, false, RESETS>(x, dy, rt, fresh, steps, a, h, sr, si, hs, gs, out)
                                       : bwd_grads_of<T, K, true, RESETS>(x, dy, rt, fresh, steps, a, h, sr, si, hs, gs, out));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && steps > 0) {
                        tma_store_3d(&tm.dx, x, int(d), int(t0), int(b));
                        tma_store_3d(&tm.dr, r, int(d), int(t0), int(b));
                        tma_store_3d(&tm.di, i, int(d), int(t0), int(b));
                    }
                    if (lane == 0) bulk_commit();
                } else {
                    const int64_t o = (int64_t(b) * p.s.L + t0) * p.s.D + d;
                    const bool on = d < p.s.D, both = d + 1 < p.s.D;
                    const auto out = [&](const int k, const float2 gx, const float2 gr, const float2 gi) {
                        const int64_t q = o + k * p.s.D;
                        if (pairs) {
                            if (on) store2(p.dx + q, gx), store2(p.dr + q, gr), store2(p.di + q, gi);
                        } else {
                            if (on) p.dx[q] = Tok<T>::from_f(gx.x), p.dr[q] = Tok<T>::from_f(gr.x), p.di[q] = Tok<T>::from_f(gi.x);
                            if (both) p.dx[q + 1] = Tok<T>::from_f(gx.y), p.dr[q + 1] = Tok<T>::from_f(gr.y), p.di[q + 1] = Tok<T>::from_f(gi.y);
                        }
                    };
                    dl = add2(dl, slow ? bwd_grads_of<T, K, false, RESETS>(x, dy, rt, fresh, steps, a, h, sr, si, hs, gs, out)
                                       : bwd_grads_of<T, K, true, RESETS>(x, dy, rt, fresh, steps, a, h, sr, si, hs, gs, out));
                }
                if (t.more & TileInfo::kLast) {
                    float *q = p.parts + (((int64_t(t.seg()) * C + rank) * kW + warp) * p.s.B + b) * p.s.D + d;
                    if (d < p.s.D) q[0] = dl.x;
                    if (d + 1 < p.s.D) q[1] = dl.y;
                }
            }
            __syncwarp();
            if (LOAD != kTma && lane == 0) mbar_arrive(&s.empty[st]);
        }
        if (LOAD == kTma && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    cluster_sync_all();  // no block leaves while another may still write to it
}

// dlam[d] = c sigmoid(lam[d]) * the sum of the tiles' parts, in a fixed order.
__global__ void __launch_bounds__(1024)
    gated_dlam_kernel(int64_t rows, int64_t D, float c, const float *__restrict__ parts, const float *__restrict__ lam,
                      float *__restrict__ dlam) {
    __shared__ float s[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t d = int64_t(blockIdx.x) * 32 + lane;
    float t = 0.0f;
    if (d < D)
#pragma unroll 4
        for (int64_t k = warp; k < rows; k += 32) t += parts[k * D + d];
    s[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && d < D) {
        t = 0.0f;
        for (int w = 0; w < 32; ++w) t += s[w][lane];
        dlam[d] = t * c / (1.0f + expf(-lam[d]));
    }
}

// ---------------------------------------------------------------------- step
// A thread has V neighbouring channels of `rows` sequences: the rate, two exponential functions of which make
// half a channel's arithmetic, is formed once for all of them (256 x 5120 bfloat16: 4.8 us, floor 3.2;
// 2048 x 5120: 29 us, floor 25.7; one sequence a thread 6.3 and 42 us).
template <typename T, int V>
__global__ void __launch_bounds__(128)
    gated_step_kernel(int64_t B, int64_t D, int rows, float c, const T *__restrict__ x, const T *__restrict__ r,
                      const T *__restrict__ i, int64_t xs, int64_t rs, int64_t is, const float *__restrict__ lam,
                      const float *h, float *h_out, T *__restrict__ y) {
    const int64_t d = (int64_t(blockIdx.x) * 128 + threadIdx.x) * V;
    if (d >= D) return;
    const Vec<float, V> lv = ldv<float, V>(lam + d);
    float p[V];
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = rate(lv.get(v), c);
    for (int64_t b0 = int64_t(blockIdx.y) * rows; b0 < B; b0 += int64_t(gridDim.y) * rows) {
        const int64_t b1 = min(B, b0 + rows);
#pragma unroll 2
        for (int64_t b = b0; b < b1; ++b) {
            const Vec<T, V> xv = ldv<T, V>(x + b * xs + d), rv = ldv<T, V>(r + b * rs + d), iv = ldv<T, V>(i + b * is + d);
            const Vec<float, V> hv = ldv<float, V>(h + b * D + d);
            Vec<float, V> ho;
            Vec<T, V> o;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float e;
                const float a = decay(p[v] * sigmoid_f(rv.get(v)), e), sq = e * (2.0f - e);
                const float hn = fmaf(a, hv.get(v), sq * inv_beta(sq) * (sigmoid_f(iv.get(v)) * xv.get(v)));
                ho.set(v, hn);
                o.set(v, hn);
            }
            stv<float, V>(h_out + b * D + d, ho);
            stv<T, V>(y + b * D + d, o);
        }
    }
}

// A few tokens of many sequences (a chunk of a decoding batch): a thread walks V neighbouring channels of one
// sequence through all of them, where tiles would be mostly empty (few_tokens_fwd says when). B=256 D=5120 bfloat16: 4 tokens 23 us,
// 32 tokens 109 us, 2.0 and 4.9 TB/s; a thread's arithmetic is scalar, with two reciprocals and two exponentials an element.
template <typename T, int V>
__global__ void __launch_bounds__(128) gated_short_kernel(const FwdArgs<T> p) {
    const int64_t d = (int64_t(blockIdx.x) * 128 + threadIdx.x) * V;
    if (d >= p.s.D) return;
    const int L = int(p.s.L);
    float rt[V];
#pragma unroll
    for (int v = 0; v < V; ++v) rt[v] = rate(p.lam[d + v], p.s.c);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = 0;
    for (int64_t b = blockIdx.y; b < p.s.B; b += gridDim.y) {
        const int64_t o = b * p.s.D + d;
        const T *x = p.x + b * p.xb + d, *r = p.r + b * p.rb + d, *i = p.i + b * p.ib + d;
        T *y = p.y + b * p.s.L * p.s.D + d;
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = p.h0 ? p.h0[o + v] : 0.0f;
            if (p.states) p.states[o + v] = h[v];  // of the only chunk
        }
#pragma unroll 4
        for (int t = 0; t < L; ++t) {
            const Vec<T, V> xv = ldv<T, V>(x + t * p.xt), rv = ldv<T, V>(r + t * p.rt), iv = ldv<T, V>(i + t * p.it);
            const bool fresh = p.reset && p.reset[b * p.s.L + t];
            Vec<T, V> out;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float e;
                const float a = decay(rt[v] * sigmoid_f(rv.get(v)), e), sq = e * (2.0f - e), u = sigmoid_f(iv.get(v)) * xv.get(v);
                h[v] = fresh ? u : fmaf(a, h[v], sq * inv_beta(sq) * u);
                out.set(v, h[v]);
            }
            if (p.y) stv<T, V>(y + t * p.s.D, out);
        }
        if (p.h_last)
#pragma unroll
            for (int v = 0; v < V; ++v) p.h_last[o + v] = h[v];
    }
}

// Its backward: the states before the steps in registers, the tokens read a second time (from the caches) on the way back.
// A thread's sums of dlam over its sequences are one value of the parts. B=256 D=5120 bfloat16: 4 tokens 59 us, 16 tokens 162 us,
// both sweeps forming every gate. (With an array for 32 tokens those 16 cost 275, and 32 tokens 558 against 302 by tiles.)
template <typename T, int V>
__global__ void __launch_bounds__(128) gated_short_bwd_kernel(const BwdArgs<T> p) {
    const int64_t d = (int64_t(blockIdx.x) * 128 + threadIdx.x) * V;
    if (d >= p.s.D) return;
    const int L = int(p.s.L);
    float rt[V], dl[V];
#pragma unroll
    for (int v = 0; v < V; ++v) rt[v] = rate(p.lam[d + v], p.s.c), dl[v] = 0.0f;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = 0;
    for (int64_t b = blockIdx.y; b < p.s.B; b += gridDim.y) {
        const int64_t o = b * p.s.D + d, first = b * p.s.L * p.s.D + d;
        const T *x = p.x + b * p.xb + d, *r = p.r + b * p.rb + d, *i = p.i + b * p.ib + d;
        float h[V], g[V], before[kShortBack][V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = p.states[o + v], g[v] = p.dh_last ? p.dh_last[o + v] : 0.0f;
#pragma unroll
        for (int t = 0; t < kShortBack; ++t)
            if (t < L) {
                const Vec<T, V> xv = ldv<T, V>(x + t * p.xt), rv = ldv<T, V>(r + t * p.rt), iv = ldv<T, V>(i + t * p.it);
                const bool fresh = p.reset && p.reset[b * p.s.L + t];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float e;
                    const float a = decay(rt[v] * sigmoid_f(rv.get(v)), e), sq = e * (2.0f - e), u = sigmoid_f(iv.get(v)) * xv.get(v);
                    before[t][v] = h[v];
                    h[v] = fresh ? u : fmaf(a, h[v], sq * inv_beta(sq) * u);
                }
            }
#pragma unroll
        for (int t = kShortBack - 1; t >= 0; --t)
            if (t < L) {
                const Vec<T, V> xv = ldv<T, V>(x + t * p.xt), rv = ldv<T, V>(r + t * p.rt), iv = ldv<T, V>(i + t * p.it),
                                dv = ldv<T, V>(p.dy + first + t * p.s.D);
                const bool fresh = p.reset && p.reset[b * p.s.L + t];
                Vec<T, V> gx, gr, gi;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float sr = sigmoid_f(rv.get(v)), si = sigmoid_f(iv.get(v)), w = rt[v] * sr, u = si * xv.get(v);
                    float e;
                    const float a = decay(w, e), sq = e * (2.0f - e), q = inv_beta(sq), vt = dv.get(v) + g[v];
                    const float vb = fresh ? vt : vt * (sq * q), dw = fresh ? 0.0f : a * vt * fmaf(a * q, u, -before[t][v]);
                    gx.set(v, vb * si);
                    gi.set(v, vb * u * (1.0f - si));
                    gr.set(v, fresh ? 0.0f : dw * w * (1.0f - sr));  // (r, not used at a reset, may be NaN)
                    if (!fresh) dl[v] = fmaf(dw, sr, dl[v]);
                    g[v] = fresh ? 0.0f : a * vt;
                }
                stv<T, V>(p.dx + first + t * p.s.D, gx);
                stv<T, V>(p.dr + first + t * p.s.D, gr);
                stv<T, V>(p.di + first + t * p.s.D, gi);
            }
        if (p.dh0)
#pragma unroll
            for (int v = 0; v < V; ++v) p.dh0[o + v] = g[v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) p.parts[int64_t(blockIdx.y) * p.s.D + d + v] = dl[v];
}

// ---------------------------------------------------------------------- host
inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Sizes whose products leave 56 bits, or with more tiles than 31 bits count, are refused.
bool sizes_fit(int64_t B, int64_t L, int64_t D, int64_t t) {
    int64_t n;
    if (__builtin_mul_overflow(B, std::max<int64_t>(L, 1), &n) || __builtin_mul_overflow(n, D, &n)) return false;
    if (n > (int64_t(1) << 56)) return false;
    return B * ceil_div(L, t) * ceil_div(D, 32) <= INT_MAX;
}

bool even(const int64_t *s) { return s[0] % 2 == 0 && s[1] % 2 == 0; }

ssm_status launched() { return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA; }

// Segments a column's time may be cut into: enough to deal the columns out evenly.
int max_segs(int64_t columns, int64_t chunks) { return int(std::max<int64_t>(1, std::min<int64_t>(chunks, std::max<int64_t>(8, std::min<int64_t>(256, 4096 / columns))))); }

// Segments times blocks of a cluster: what each column's sums of dlam are spread over at most. No plan has a
// cluster with twice as many blocks as there are tiles, nor more segments than rounds.
int most_parts(int64_t columns, int64_t tiles) {
    int64_t n = 1;
    for (int64_t c = 1; c <= kMostBlocks && (c == 1 || c / 2 < tiles); c *= 2) n = std::max(n, c * ceil_div(tiles, c));
    return int(std::min(n, std::max<int64_t>(kMostBlocks, std::min<int64_t>(256, 4096 / columns))));
}

// The header, and what segments hand on: nothing where the time is one segment.
size_t carry_bytes(int64_t B, int64_t L, int64_t D) {
    const int64_t segs = max_segs(B * ceil_div(D, 64), ceil_div(L, kChunk));
    return kWsHeader + (segs > 1 ? 2 * up256(size_t(B) * size_t(D) * size_t(segs) * 8) : 0);
}

// Whether a call takes the few-token kernels, where a thread walks its channels through all tokens, rather than tiles, which
// are then mostly empty. A thread's walk is a chain (0.9 us a token forward, 1.2 backward, beside 6 and 10 us) as long as the
// GPU has room for all of them; the tiles' time goes by the columns (11 us for 64 bfloat16 ones forward, 22 for 1024, 221 for
// 20480) and not by the tokens. So the border is a number of tokens that grows with the columns, up to where both are
// bound by memory. Threads / tiles in us, in a graph: bfloat16 forward 16x16x1024 20/14, 32x8x1024 14/16, 64x16x1024 20/23,
// 16x32x5120 35/25, 32x32x5120 37/40, 256x32x5120 109/228, 256x64x5120 199/238 but 256x64x1030 102/59; float32 forward 64x8x1024 16/16,
// 64x32x1024 39/18, 64x24x5120 41/45, 256x32x5120 139/141. Rows below 256 channels leave lanes of a block idle: bfloat16
// 4096x16x64 45/55, 4096x32x64 88/57, float32 4096x12x64 41/37, 4096x32x64 96/39.
bool few_tokens_fwd(int64_t B, int64_t L, int64_t D, ssm_dtype dtype) {
    const int64_t columns = B * ceil_div(D, 64);
    if (dtype == SSM_BF16) return L <= std::min<int64_t>(D < 256 ? 24 : 32, 5 + columns / 92);
    return L <= std::min<int64_t>(D < 256 ? 12 : 24, 4 + columns / 200);
}
// The same for the backward, either type: 32x6x1024 18/20, 32x16x1024 31/20, 64x12x1024 27/31, 256x16x5120 162/291; tiles of rows that TMA does
// not take, or that are short, cost about twice as much a column: bfloat16 32x12x1001 22/30, 512x16x128 32/38, 1024x16x16 35/49.
bool few_tokens_bwd(int64_t B, int64_t L, int64_t D, ssm_dtype dtype) {
    const bool slow = D < 256 || D * (dtype == SSM_BF16 ? 2 : 4) % 16 != 0;
    return L <= std::min<int64_t>(kShortBack, 2 + B * ceil_div(D, 64) / (slow ? 48 : 96));
}
int64_t short_rows(int64_t B) { return std::min<int64_t>(B, 2048); }  // of their backward's blocks, each a row of the parts

// Clusters of each size that the GPU holds at once (0: not asked yet), by device.
struct Residency {
    std::atomic<int> n[64][5];
};
int clusters_resident(Residency &r, const void *kernel, int threads, size_t smem, int log2c) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = r.n[dev][log2c].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(1u << log2c), cfg.blockDim = dim3(unsigned(threads)), cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = 1u << log2c, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
        cfg.attrs = &at, cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess ||
            cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
            cudaGetLastError();  // not left for the next call to find
            return 0;
        }
        r.n[dev][log2c].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Chooses the cluster size and the segments. One unit of cost is a round (a tile in every resident
// block). With more columns than clusters the columns' segments are dealt out in turn,
// in as many pieces as even out the last turn; with fewer, larger clusters share a column
// (each doubling costs a little for the slowest of more blocks), and with very few the segments
// run side by side in two passes (twice the rounds, three launches).
bool make_plan(Plan &pl, Residency &r, const void *kernel, int threads, size_t smem, int most_blocks, int64_t columns, int64_t tiles,
               int most_segs) {
    double best = 1e300;
    pl.columns = columns;
    for (int k = 0; (1 << k) <= most_blocks; ++k) {
        const int c = 1 << k;
        if (c > 1 && c / 2 >= tiles) break;
        const int n = clusters_resident(r, kernel, threads, smem, k);
        if (n <= 0 && k == 0) return false;
        if (n <= 0) break;  // a size this GPU does not take
        const int64_t rounds = ceil_div(tiles, c);
        const auto consider = [&](int64_t iters, bool local, double cost) {
            if (cost >= best) return;
            best = cost;
            pl.cluster = c, pl.rounds = rounds, pl.iters = int(iters), pl.segs = int(ceil_div(rounds, iters)), pl.local = local;
            pl.items = unsigned(columns * pl.segs);
            pl.grid = int(std::min<int64_t>(n, pl.items)) * c;
        };
        const double per = 1.0 + 0.03 * k;
        consider(rounds, false, double(ceil_div(columns, n)) * double(rounds) * per);
        for (int64_t segs = 2; segs <= std::min<int64_t>(most_segs, rounds); segs += std::max<int64_t>(1, segs / 4)) {
            if (segs * c > most_parts(columns, tiles)) break;
            const int64_t iters = ceil_div(rounds, segs), items = columns * ceil_div(rounds, iters);
            if (columns >= n) consider(iters, false, double(ceil_div(items, n)) * double(iters) * per + 1.0);
            if (c == 1) consider(iters, true, 2.0 * double(ceil_div(items, n)) * double(iters) + 6.0);
        }
    }
    return true;
}

// Counter, status and hand-off words of a plan whose segments are handed on in turn. Test hook: the counter starts
// behind the first segment of the first column, so that nobody hands its state on.
bool clear_words(const Plan &pl, unsigned char *ws, int64_t n, cudaStream_t st) {
    if (pl.segs == 1 || pl.local) return true;
    return cudaMemsetAsync(ws, 0, kWsHeader + size_t(n) * size_t(pl.segs) * 8, st) == cudaSuccess &&
           (!pl.drop_handoff || cudaMemsetAsync(ws, 1, 1, st) == cudaSuccess);
}

template <typename T, int K, Load LOAD, bool LAG, bool RESETS>
ssm_status launch_fwd_as(FwdArgs<T> p, const Maps3 &tm, bool pairs, cudaStream_t st) {
    static Residency resident;
    constexpr size_t smem = sizeof(FwdShared<T, K, LAG>);
    constexpr int threads = (kW + 1 + kLoaders<LOAD>) * 32;
    const auto kernel = gated_fwd_kernel<T, K, LOAD, LAG, RESETS>;
    const int64_t columns = p.s.B * p.s.groups, n = p.s.B * p.s.D;
    const int segs = max_segs(columns, ceil_div(p.s.L, kChunk));
    if (!make_plan(p.pl, resident, reinterpret_cast<const void *>(kernel), threads, smem, FwdShared<T, K, LAG>::kMaxCluster, columns,
                   ceil_div(p.s.L, kW * K), segs))
        return SSM_ERR_CUDA;
    unsigned char *ws = reinterpret_cast<unsigned char *>(p.counter);
    p.status = p.counter + 1;
    p.starts = reinterpret_cast<unsigned long long *>(ws + kWsHeader);
    Map *maps = reinterpret_cast<Map *>(ws + kWsHeader + up256(size_t(n) * size_t(segs) * 8));
    if (!clear_words(p.pl, ws, n, st)) return SSM_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.pl.grid)), cfg.blockDim = dim3(unsigned(threads)), cfg.dynamicSmemBytes = smem, cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = unsigned(p.pl.cluster), at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
    cfg.attrs = &at, cfg.numAttrs = 1;
    if (p.pl.local) {
        p.maps = maps;
        if (cudaLaunchKernelEx(&cfg, kernel, p, tm, pairs) != cudaSuccess) return launched();
        p.maps = nullptr;
        gated_starts_kernel<<<unsigned(ceil_div(n, 128)), 128, 0, st>>>(n, p.pl.segs, p.h0, maps, p.starts);
    }
    cudaLaunchKernelEx(&cfg, kernel, p, tm, pairs);
    return launched();
}

template <typename T, int K, Load LOAD, bool LAG>
ssm_status launch_fwd(const FwdArgs<T> &p, const Maps3 &tm, bool pairs, cudaStream_t st) {
    return p.reset ? launch_fwd_as<T, K, LOAD, LAG, true>(p, tm, pairs, st) : launch_fwd_as<T, K, LOAD, LAG, false>(p, tm, pairs, st);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }
    return fn;
}

// Tokens [B, L, D] with the strides of the call, in boxes of 64 channels by `rows` steps. False where TMA cannot
// take them: a base off 16 bytes, a stride that is not a multiple of 16 bytes or makes rows overlap.
bool token_map(CUtensorMap *m, const void *ptr, ssm_dtype dt, int64_t B, int64_t L, int64_t D, const int64_t *stride, int rows) {
    const int64_t es = dt == SSM_BF16 ? 2 : 4;
    const int64_t st = L > 1 ? stride[1] * es : (D * es + 15) / 16 * 16;
    const int64_t sb = B > 1 ? stride[0] * es : st;
    if ((reinterpret_cast<uintptr_t>(ptr) & 15) || st % 16 || sb % 16 || st < D * es || sb < st || st >= (int64_t(1) << 40) ||
        sb >= (int64_t(1) << 40) || B > INT_MAX || L > INT_MAX - 1024 || D > INT_MAX - 1024)
        return false;
    auto enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(L), cuuint64_t(B)};
    cuuint64_t strides[2] = {cuuint64_t(st), cuuint64_t(sb)};
    cuuint32_t box[3] = {64, cuuint32_t(rows), 1}, ones[3] = {1, 1, 1};
    return enc(m, dt == SSM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(ptr),
               dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
ssm_status run_fwd(const ssm_gated_args *a, cudaStream_t st) {
    constexpr size_t es = sizeof(T);
    FwdArgs<T> p = {};
    p.s = {a->batch, a->seqlen, a->dim, ceil_div(a->dim, 64), a->c};
    p.pl.drop_handoff = (a->flags & SSM_TEST_DROP_HANDOFF) != 0;
    p.counter = static_cast<unsigned int *>(a->workspace);
    p.x = static_cast<const T *>(a->x), p.r = static_cast<const T *>(a->r), p.i = static_cast<const T *>(a->i);
    p.xb = a->x_stride[0], p.xt = a->x_stride[1], p.rb = a->r_stride[0], p.rt = a->r_stride[1];
    p.ib = a->i_stride[0], p.it = a->i_stride[1];
    p.reset = a->reset, p.lam = a->lam, p.h0 = a->h0;
    p.y = static_cast<T *>(a->y), p.h_last = a->h_last, p.states = a->states;
    const bool pairs = a->dim % 2 == 0 && even(a->x_stride) && even(a->r_stride) && even(a->i_stride) && aligned(a->x, 2 * es) &&
                       aligned(a->r, 2 * es) && aligned(a->i, 2 * es) && aligned(a->y, 2 * es);
    if (few_tokens_fwd(a->batch, a->seqlen, a->dim, a->dtype)) {
        p.status = p.counter + 1;
        const bool four = (a->dim | p.xb | p.xt | p.rb | p.rt | p.ib | p.it) % 4 == 0 && aligned(a->x, 4 * es) && aligned(a->r, 4 * es) &&
                          aligned(a->i, 4 * es) && aligned(a->y, 4 * es);
        const dim3 grid(unsigned(ceil_div(a->dim, four ? 512 : pairs ? 256 : 128)), unsigned(std::min<int64_t>(a->batch, 65535)));
        if (four)
            gated_short_kernel<T, 4><<<grid, 128, 0, st>>>(p);
        else if (pairs)
            gated_short_kernel<T, 2><<<grid, 128, 0, st>>>(p);
        else
            gated_short_kernel<T, 1><<<grid, 128, 0, st>>>(p);
        return launched();
    }
    const auto maps_of = [&](Maps3 &tm, int rows) {
        return pairs && token_map(&tm.x, a->x, a->dtype, a->batch, a->seqlen, a->dim, a->x_stride, rows) &&
               token_map(&tm.r, a->r, a->dtype, a->batch, a->seqlen, a->dim, a->r_stride, rows) &&
               token_map(&tm.i, a->i, a->dtype, a->batch, a->seqlen, a->dim, a->i_stride, rows);
    };
    // Stages of 48 KB, of 24 KB where the loading warps are what counts.
    constexpr int K = es == 2 ? 16 : 8;
    const bool few = p.s.B * p.s.groups <= kFewColumns;
    Maps3 tm = {};
    if (maps_of(tm, kW * K)) return few ? launch_fwd<T, K, kTma, true>(p, tm, pairs, st) : launch_fwd<T, K, kTma, false>(p, tm, pairs, st);
    if (pairs || es == 4) return few ? launch_fwd<T, K, kAsync, true>(p, tm, pairs, st) : launch_fwd<T, K / 2, kAsync, false>(p, tm, pairs, st);
    if constexpr (es == 2) return launch_fwd<T, K / 2, kPlain, false>(p, tm, pairs, st);
    return SSM_ERR_UNSUPPORTED;
}

template <typename T, int K, Load LOAD, bool RESETS>
ssm_status launch_bwd_as(BwdArgs<T> p, const Maps7 &tm, bool pairs, float *dlam, cudaStream_t st) {
    static Residency resident;
    constexpr size_t smem = sizeof(BwdShared<T, K>);
    constexpr int threads = (kW + 1 + kLoaders<LOAD, true, sizeof(T)>) * 32;
    const auto kernel = gated_bwd_kernel<T, K, LOAD, RESETS>;
    const int64_t columns = p.s.B * p.s.groups, n = p.s.B * p.s.D;
    const int segs = max_segs(columns, ceil_div(p.s.L, kChunk));
    if (!make_plan(p.pl, resident, reinterpret_cast<const void *>(kernel), threads, smem, BwdShared<T, K>::kMaxCluster, columns,
                   ceil_div(p.s.L, kW * K), segs))
        return SSM_ERR_CUDA;
    unsigned char *ws = reinterpret_cast<unsigned char *>(p.counter);
    p.status = p.counter + 1;
    p.starts = reinterpret_cast<unsigned long long *>(ws + kWsHeader);
    Map *maps = reinterpret_cast<Map *>(ws + kWsHeader + up256(size_t(n) * size_t(segs) * 8));
    p.parts = reinterpret_cast<float *>(ws + carry_bytes(p.s.B, p.s.L, p.s.D));
    if (!clear_words(p.pl, ws, n, st)) return SSM_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.pl.grid)), cfg.blockDim = dim3(unsigned(threads)), cfg.dynamicSmemBytes = smem, cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = unsigned(p.pl.cluster), at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
    cfg.attrs = &at, cfg.numAttrs = 1;
    if (p.pl.local) {
        p.maps = maps;
        if (cudaLaunchKernelEx(&cfg, kernel, p, tm, pairs) != cudaSuccess) return launched();
        p.maps = nullptr;
        gated_starts_kernel<<<unsigned(ceil_div(n, 128)), 128, 0, st>>>(n, p.pl.segs, p.dh_last, maps, p.starts);
    }
    if (cudaLaunchKernelEx(&cfg, kernel, p, tm, pairs) != cudaSuccess) return launched();
    gated_dlam_kernel<<<unsigned(ceil_div(p.s.D, 32)), 1024, 0, st>>>(int64_t(p.pl.segs) * p.pl.cluster * kW * p.s.B, p.s.D, p.s.c, p.parts,
                                                                      p.lam, dlam);
    return launched();
}

template <typename T, int K, Load LOAD>
ssm_status launch_bwd(const BwdArgs<T> &p, const Maps7 &tm, bool pairs, float *dlam, cudaStream_t st) {
    return p.reset ? launch_bwd_as<T, K, LOAD, true>(p, tm, pairs, dlam, st) : launch_bwd_as<T, K, LOAD, false>(p, tm, pairs, dlam, st);
}

template <typename T>
ssm_status run_bwd(const ssm_gated_bwd_args *a, cudaStream_t st) {
    constexpr size_t es = sizeof(T);
    BwdArgs<T> p = {};
    p.s = {a->batch, a->seqlen, a->dim, ceil_div(a->dim, 64), a->c};
    p.pl.drop_handoff = (a->flags & SSM_TEST_DROP_HANDOFF) != 0;
    p.counter = static_cast<unsigned int *>(a->workspace);
    p.x = static_cast<const T *>(a->x), p.r = static_cast<const T *>(a->r), p.i = static_cast<const T *>(a->i);
    p.dy = static_cast<const T *>(a->dy);
    p.xb = a->x_stride[0], p.xt = a->x_stride[1], p.rb = a->r_stride[0], p.rt = a->r_stride[1];
    p.ib = a->i_stride[0], p.it = a->i_stride[1];
    p.reset = a->reset, p.lam = a->lam, p.states = a->states, p.dh_last = a->dh_last;
    p.dx = static_cast<T *>(a->dx), p.dr = static_cast<T *>(a->dr), p.di = static_cast<T *>(a->di), p.dh0 = a->dh0;
    bool pairs = a->dim % 2 == 0 && even(a->x_stride) && even(a->r_stride) && even(a->i_stride);
    for (const void *q : {a->x, a->r, a->i, a->dy, static_cast<const void *>(a->dx), static_cast<const void *>(a->dr),
                          static_cast<const void *>(a->di)})
        pairs = pairs && aligned(q, 2 * es);
    if (few_tokens_bwd(a->batch, a->seqlen, a->dim, a->dtype)) {
        p.status = p.counter + 1;
        p.parts = reinterpret_cast<float *>(static_cast<unsigned char *>(a->workspace) + kWsHeader);
        const dim3 grid(unsigned(ceil_div(a->dim, pairs ? 256 : 128)), unsigned(short_rows(a->batch)));
        if (pairs)
            gated_short_bwd_kernel<T, 2><<<grid, 128, 0, st>>>(p);
        else
            gated_short_bwd_kernel<T, 1><<<grid, 128, 0, st>>>(p);
        gated_dlam_kernel<<<unsigned(ceil_div(p.s.D, 32)), 1024, 0, st>>>(grid.y, p.s.D, p.s.c, p.parts, p.lam, a->dlam);
        return launched();
    }
    constexpr int K = kChunk / kW;
    const int64_t whole[2] = {a->seqlen * a->dim, a->dim};
    const auto map = [&](CUtensorMap &m, const void *q, const int64_t *stride, int rows) {
        return token_map(&m, q, a->dtype, a->batch, a->seqlen, a->dim, stride, rows);
    };
    Maps7 tm = {};
    if (pairs && map(tm.x, a->x, a->x_stride, kChunk) && map(tm.r, a->r, a->r_stride, kChunk) && map(tm.i, a->i, a->i_stride, kChunk) &&
        map(tm.dy, a->dy, whole, kChunk) && map(tm.dx, a->dx, whole, K) && map(tm.dr, a->dr, whole, K) && map(tm.di, a->di, whole, K))
        return launch_bwd<T, K, kTma>(p, tm, pairs, a->dlam, st);
    if (pairs || es == 4) return launch_bwd<T, K, kAsync>(p, tm, pairs, a->dlam, st);
    if constexpr (es == 2) return launch_bwd<T, K, kPlain>(p, tm, pairs, a->dlam, st);
    return SSM_ERR_UNSUPPORTED;
}

__global__ void gated_dlam_zero_kernel(int64_t D, float *dlam) {
    const int64_t d = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (d < D) dlam[d] = 0.0f;
}

// What the forward and the backward check alike.
template <typename A>
ssm_status check_common(const A *a) {
    if (!a || a->batch < 0 || a->seqlen < 0 || a->dim < 0 || (a->flags & ~uint32_t(SSM_TEST_DROP_HANDOFF)) || !(a->c > 0.0f) || a->c > FLT_MAX ||
        (a->dtype != SSM_F32 && a->dtype != SSM_BF16))
        return SSM_ERR_INVALID;
    if (!sizes_fit(a->batch, a->seqlen, a->dim, kChunk)) return SSM_ERR_UNSUPPORTED;
    const int64_t *const strides[] = {a->x_stride, a->r_stride, a->i_stride};
    for (const int64_t *s : strides)
        if (s[0] < 0 || s[1] < 0) return SSM_ERR_INVALID;
    return SSM_OK;
}

// A stride over a single sequence or step is never walked: it counts as 0.
template <typename A>
A walked(const A &args) {
    A a = args;
    int64_t *const strides[] = {a.x_stride, a.r_stride, a.i_stride};
    for (int64_t *s : strides) {
        if (a.batch <= 1) s[0] = 0;
        if (a.seqlen <= 1) s[1] = 0;
    }
    return a;
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

// A piece of memory that a call reads or writes.
struct Span {
    const void *at;
    size_t bytes;
};
template <typename A>
Span tokens_of(const A *a, const void *q, const int64_t *stride) {  // (strides_fit holds)
    return {q, size_t((a->batch - 1) * stride[0] + (a->seqlen - 1) * stride[1] + a->dim) * (a->dtype == SSM_BF16 ? 2 : 4)};
}
// True where no output overlaps an input. (A block of a cluster may still read the state or adjoint that a sequence
// starts from when another has written its last.)
bool apart(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
    for (const Span &o : outputs)
        for (const Span &i : inputs) {
            const uintptr_t p = reinterpret_cast<uintptr_t>(o.at), q = reinterpret_cast<uintptr_t>(i.at);
            if (p && q && p < q + i.bytes && q < p + o.bytes) return false;
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
    if (a->batch == 0 || a->dim == 0) return 0;
    return few_tokens_fwd(a->batch, a->seqlen, a->dim, a->dtype) ? kWsHeader : carry_bytes(a->batch, a->seqlen, a->dim);
}

ssm_status ssm_gated_scan_fwd(const ssm_gated_args *args, void *stream) {
    const ssm_status ok = check_common(args);
    if (ok != SSM_OK) return ok;
    const ssm_gated_args walk = walked(*args), *a = &walk;
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
    const size_t row = size_t(a->dim) * 4, state = size_t(a->batch) * row, steps = size_t(a->batch) * size_t(a->seqlen);
    if (!apart({{a->y, steps * size_t(a->dim) * es}, {a->h_last, state}, {a->states, ssm_gated_states_size(a->batch, a->seqlen, a->dim)}},
               {tokens_of(a, a->x, a->x_stride), tokens_of(a, a->r, a->r_stride), tokens_of(a, a->i, a->i_stride), {a->reset, steps},
                {a->lam, row}, {a->h0, state}}))
        return SSM_ERR_INVALID;
    if (!a->workspace || a->workspace_bytes < ssm_gated_scan_workspace_size(a)) return SSM_ERR_INVALID;
    if (!aligned(a->workspace, 16)) return SSM_ERR_UNSUPPORTED;
    return a->dtype == SSM_BF16 ? run_fwd<__nv_bfloat16>(a, st) : run_fwd<float>(a, st);
}

size_t ssm_gated_scan_bwd_workspace_size(const ssm_gated_bwd_args *a) {
    if (check_common(a) != SSM_OK) return 0;
    if (a->batch == 0 || a->dim == 0) return 0;
    if (few_tokens_bwd(a->batch, a->seqlen, a->dim, a->dtype)) return kWsHeader + size_t(short_rows(a->batch)) * size_t(a->dim) * 4;
    const int parts = most_parts(a->batch * ceil_div(a->dim, 64), ceil_div(a->seqlen, kChunk));
    return carry_bytes(a->batch, a->seqlen, a->dim) + size_t(a->batch) * size_t(a->dim) * size_t(parts) * kW * 4;
}

ssm_status ssm_gated_scan_bwd(const ssm_gated_bwd_args *args, void *stream) {
    const ssm_status ok = check_common(args);
    if (ok != SSM_OK) return ok;
    const ssm_gated_bwd_args walk = walked(*args), *a = &walk;
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
    const size_t row = size_t(a->dim) * 4, state = size_t(a->batch) * row, steps = size_t(a->batch) * size_t(a->seqlen);
    const size_t tokens = steps * size_t(a->dim) * es;
    if (!apart({{a->dx, tokens}, {a->dr, tokens}, {a->di, tokens}, {a->dlam, row}, {a->dh0, state}},
               {tokens_of(a, a->x, a->x_stride), tokens_of(a, a->r, a->r_stride), tokens_of(a, a->i, a->i_stride), {a->reset, steps},
                {a->lam, row}, {a->states, ssm_gated_states_size(a->batch, a->seqlen, a->dim)}, {a->dy, tokens}, {a->dh_last, state}}))
        return SSM_ERR_INVALID;
    if (!a->workspace || a->workspace_bytes < ssm_gated_scan_bwd_workspace_size(a)) return SSM_ERR_INVALID;
    if (!aligned(a->workspace, 16)) return SSM_ERR_UNSUPPORTED;
    return a->dtype == SSM_BF16 ? run_bwd<__nv_bfloat16>(a, st) : run_bwd<float>(a, st);
}

ssm_status ssm_gated_status(void *stream) {
    static std::mutex one;  // gave_up_taken serves one query at a time
    const std::lock_guard<std::mutex> hold(one);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    gave_up_take_kernel<<<1, 1, 0, st>>>();
    unsigned int v = 0;
    if (launched() != SSM_OK || cudaMemcpyFromSymbolAsync(&v, gave_up_taken, sizeof(v), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return SSM_ERR_CUDA;
    return static_cast<ssm_status>(v);
}

ssm_status ssm_gated_step(int64_t batch, int64_t dim, ssm_dtype dtype, float c, const void *x, int64_t x_stride,
                          const void *r, int64_t r_stride, const void *i, int64_t i_stride, const float *lam,
                          const float *h, float *h_out, void *y, void *stream) {
    if (batch < 0 || dim < 0 || x_stride < 0 || r_stride < 0 || i_stride < 0 || !(c > 0.0f) || c > FLT_MAX ||
        (dtype != SSM_F32 && dtype != SSM_BF16))
        return SSM_ERR_INVALID;
    if (!sizes_fit(batch, 1, dim, 1)) return SSM_ERR_UNSUPPORTED;
    if (batch == 0 || dim == 0) return SSM_OK;
    if (batch == 1) x_stride = r_stride = i_stride = 0;  // never walked
    if (!x || !r || !i || !lam || !h || !h_out || !y) return SSM_ERR_INVALID;
    const size_t es = dtype == SSM_BF16 ? 2 : 4;
    int64_t together = dim | x_stride | r_stride | i_stride;  // channels a thread may move as one piece
    int v = together % 4 == 0 ? 4 : together % 2 == 0 ? 2 : 1;
    for (const void *q : {x, r, i, static_cast<const void *>(y)}) {
        if (!aligned(q, es)) return SSM_ERR_UNSUPPORTED;
        while (!aligned(q, v * es)) v /= 2;
    }
    for (const void *q : {static_cast<const void *>(lam), static_cast<const void *>(h), static_cast<const void *>(h_out)}) {
        if (!aligned(q, 4)) return SSM_ERR_UNSUPPORTED;
        while (!aligned(q, size_t(v) * 4)) v /= 2;
    }
    for (const int64_t s : {x_stride, r_stride, i_stride}) {
        int64_t m;
        if (__builtin_mul_overflow(batch, s, &m) || m > (int64_t(1) << 56)) return SSM_ERR_UNSUPPORTED;
    }
    const size_t state = size_t(batch) * size_t(dim) * 4;
    if (h_out != h && !apart({{h_out, state}}, {{h, state}})) return SSM_ERR_INVALID;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // as many sequences a thread as leave about a thousand threads to each of 148 SMs
    const int64_t across = ceil_div(dim, v);
    const int rows = int(std::max<int64_t>(1, std::min<int64_t>(16, batch * across / (148 * 1024))));
    const dim3 grid(unsigned(ceil_div(across, 128)), unsigned(std::min<int64_t>(ceil_div(batch, rows), 65535)));
#define SSM_STEP(T, V)                                                                                                  \
    gated_step_kernel<T, V><<<grid, 128, 0, st>>>(batch, dim, rows, c, static_cast<const T *>(x), static_cast<const T *>(r), \
                                                  static_cast<const T *>(i), x_stride, r_stride, i_stride, lam, h, h_out,    \
                                                  static_cast<T *>(y))
#define SSM_STEP_BY(T) (v == 4 ? SSM_STEP(T, 4) : v == 2 ? SSM_STEP(T, 2) : SSM_STEP(T, 1))
    if (dtype == SSM_BF16)
        SSM_STEP_BY(__nv_bfloat16);
    else
        SSM_STEP_BY(float);
#undef SSM_STEP_BY
#undef SSM_STEP
    return launched();
}

}  // extern "C"
