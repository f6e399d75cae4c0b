// gdr_scan.cuh -- what the kernels of the gated scan share: the gate, the cursor over the
// sequences of a token axis, a block's tiles of raw inputs, and the chaining of runs.
//
// Per (sequence, channel):
//     alpha_t = exp(g(a_t)),   h_t = alpha_t h_{t-1} + w(alpha_t) x_t
// with g the library's gates and w = 1, 1 - alpha or sqrt(1 - alpha^2).
//
// The token axis (all sequences behind each other) is cut into tiles of 128 tokens x 32
// channels; a block takes a tile at a time.  16 lanes hold the 32 channels of one token, a lane
// two neighbouring channels of a run of L tokens: the run becomes the pair (A, B),
// h_out = A h_in + B, the pairs are chained -- the two runs of a warp by shuffles, the warps
// through shared memory, the blocks of a cluster, which take tiles next to each other, through
// their peers' shared memory -- and each lane goes over its run once more from the state that
// enters it.  Every input is read once, and no block waits for one outside its cluster.
//
// A sequence's first token cuts the chain: nothing in front of it may be seen through it, not
// even as 0 * NaN.  alpha is never negative, so a run with such a token carries A = -1, and
// chaining looks at the sign (where there can be cuts at all) instead of multiplying.
#pragma once

#include <type_traits>

#include "gdr_internal.cuh"

namespace gdr {

constexpr int kScanTile = 128;      // tokens of a tile; the interval of the states kept for the backward pass
constexpr int kScanChannels = 32;   // channels of a tile
constexpr int kScanMaxCluster = 8;
constexpr int64_t kScanMaxTokens = 0x7fffffff - 2 * kScanTile * kScanMaxCluster;   // positions are 32-bit

struct ScanShape {
    const int32_t *cu;   // offsets of packed sequences, or null: N sequences of T_per tokens
    int N, T_per, total, D;
    float b;
    int per_part;        // sequences of a part (a chain of tiles of its own)
    int parts, tiles, cluster;
};

// What is passed beside the shape; null where absent.
struct ScanFwd {
    const void *x, *a;
    const float *h0;
    void *out;
    float *hT, *states;
};
struct ScanBwd {
    const void *x, *a, *dout;
    const float *h0, *dhT, *states;
    void *dx, *da;
    float *dh0;
};

#ifdef __CUDACC__
namespace scan {

constexpr unsigned kFull = 0xffffffffu;

// ---- the gate ---------------------------------------------------------------------------
// FINE (fp32 tensors): the library functions' accuracy.  Else the special-function unit's, within
// a few 2^-23 of the value; what a long memory hangs on, 1 - alpha for alpha near 1, keeps its
// relative accuracy in both (1 - e^g from a polynomial, and alpha from that).
template <bool FINE> __device__ __forceinline__ float exp_of(float x) {
    if constexpr (FINE) return expf(x);
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504088896341f));
    return y;
}
template <bool FINE> __device__ __forceinline__ float inverse(float x) {
    if constexpr (FINE) return __frcp_rn(x);
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct Gate {
    float alpha, w;     // the decay and the input's weight
    float slope, dw;    // dg/da, and dw/dg dg/da
};

// e^g = alpha = 1 - left for g <= 0.  (e^g - 1) / g on [-1/2, 0] by a polynomial fitted to it
// (relative error 1e-8 with these coefficients).
template <bool FINE> __device__ __forceinline__ void decay_of(float g, float &alpha, float &left) {
    const float e = exp_of<FINE>(g);
    float p = 0.0011259226594120264f;
    p = fmaf(p, g, 0.008193295449018478f);
    p = fmaf(p, g, 0.04163204878568649f);
    p = fmaf(p, g, 0.16666288673877716f);
    p = fmaf(p, g, 0.49999985098838806f);
    p = fmaf(p, g, 1.f);
    const float near = -g * p;
    const bool small = g > -0.5f;
    left = small ? near : 1.f - e;
    alpha = small ? 1.f - near : e;
}

template <bool FINE, int GATE, int SRC, bool GRAD> __device__ __forceinline__ Gate gate_of(float a, float b) {
    Gate o;
    float left;
    if constexpr (GATE == GDR_GATE_BOUNDED) {
        const float c = a < -87.f ? -87.f : a;   // e^87 is finite; sigmoid is 0 below; a NaN stays
        const float e = exp_of<FINE>(-c), s = inverse<FINE>(1.f + e);
        const float g = -b * s;
        decay_of<FINE>(g, o.alpha, left);
        o.slope = g * (e * s);
    } else {
        // e^{-softplus(a)} = 1 / (1 + e^a)
        const float e = exp_of<FINE>(-fabsf(a)), lo = e * inverse<FINE>(1.f + e), hi = 1.f - lo;
        o.alpha = a > 0.f ? lo : hi;
        left = a > 0.f ? hi : lo;
        o.slope = -left;
    }
    if constexpr (SRC == GDR_SOURCE_PLAIN) {
        o.w = 1.f;
        o.dw = 0.f;
    } else if constexpr (SRC == GDR_SOURCE_CONVEX) {
        o.w = left;
        o.dw = -o.alpha * o.slope;
    } else {
        const float z = left * (1.f + o.alpha);   // 1 - alpha^2
        // at z = 0 the weight is 0 and so is its gradient (slope / w goes with sqrt(left)); NaN stays
        float r;
        if constexpr (FINE) {
            o.w = sqrtf(z);
            r = z > 0.f ? 1.f / o.w : 0.f;
        } else {
            r = z > 0.f ? rsqrtf(z) : 0.f;
            o.w = z * r;
        }
        if constexpr (GRAD) o.dw = -(o.alpha * o.alpha) * (o.slope * r);
    }
    return o;
}

// ---- sequences --------------------------------------------------------------------------
__device__ __forceinline__ int seq_start(const ScanShape &s, int n) { return s.cu ? s.cu[n] : n * s.T_per; }

// The sequence that holds a token, among those of a part (numbers first .. last - 1, last's
// start being the part's end).
struct Cursor {
    int n, from, to;
    __device__ __forceinline__ void seek(const ScanShape &s, int first, int last, int token) {
        if (token >= from && token < to) return;
        int lo = first, hi = last - 1;   // the largest n that starts at or before the token is not empty
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq_start(s, mid) <= token) lo = mid; else hi = mid - 1;
        }
        n = lo;
        from = seq_start(s, n);
        to = seq_start(s, n + 1);
    }
};

// First and last tokens of sequences among the L tokens from p, as bits; [lo, hi) are those
// of them that belong to the part.
struct Marks {
    unsigned first, last;
};
__device__ __forceinline__ Marks marks_of(const ScanShape &s, Cursor &c, int from, int upto, int p, int lo, int hi) {
    Marks m{0, 0};
    if (lo >= hi) return m;
    c.seek(s, from, upto, lo);
    if (lo == c.from) m.first = 1u << (lo - p);
    int n = c.n + 1, q = c.to;
    while (q <= hi) {
        m.last |= 1u << (q - 1 - p);
        if (q == hi) break;
        m.first |= 1u << (q - p);
        const int at = q;
        do q = seq_start(s, ++n);   // past empty sequences; the part's end is beyond `at`
        while (q <= at);
    }
    return m;
}
// The sequence of token t, going up from n.
__device__ __forceinline__ int seq_from(const ScanShape &s, int n, int t) {
    while (seq_start(s, n + 1) <= t) ++n;
    return n;
}

// Whether the offsets are 0 = c0 <= c1 <= .. <= cN = total; the whole block calls.
__device__ __forceinline__ bool offsets_ok(const ScanShape &s) {
    if (!s.cu) return true;
    int bad = threadIdx.x == 0 && (s.cu[0] != 0 || s.cu[s.N] != s.total);
    for (int i = threadIdx.x; i < s.N; i += blockDim.x) bad |= s.cu[i] > s.cu[i + 1];
    return !__syncthreads_or(bad);
}

// ---- chaining ---------------------------------------------------------------------------
// out = A h + B, or B past a cut.
__device__ __forceinline__ float through(float A, float B, float h, bool cuts) {
    return fmaf(A, cuts && __float_as_int(A) < 0 ? 0.f : h, B);
}
// (A, B) := (A, B) followed by (a, b).
__device__ __forceinline__ void follow(float &A, float &B, float a, float b, bool cuts) {
    const bool cut = cuts && __float_as_int(a) < 0;
    B = fmaf(a, cut ? 0.f : B, b);
    A = cut ? a : cuts && __float_as_int(A) < 0 ? A : A * a;
}
// A := A alpha; a cut stays one, also in front of a NaN.
__device__ __forceinline__ void decay_past_cut(float &A, float alpha) {
    if (__float_as_int(A) >= 0) A *= alpha;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void put_to_peer(const float4 *at, unsigned rank, float4 v) {
    unsigned addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"((unsigned)__cvta_generic_to_shared(at)), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// ---- tiles of raw inputs ------------------------------------------------------------------
// A warp copies the rows that its own lanes work on: 2 runs of L tokens, interleaved so that
// both halves of the warp read the same token number without bank conflicts.
template <typename T, int L> constexpr int kWarpTile = 2 * L * kScanChannels;   // elements

// WIDE: 16 bytes a copy (rows and bases on 16-byte boundaries).  PAIR: what a lane reads itself,
// where a lane's two channels can be copied asynchronously.  SINGLE: plain loads, element by element.
enum CopyMode { kWide, kPair, kSingle };

template <typename T> __host__ __device__ constexpr int wide_elems() { return 16 / (int)sizeof(T); }

__device__ __forceinline__ void copy16(unsigned dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(unsigned dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Asks for the warp's part of NT tensors' tile; `row0` is the warp's first token, [lo, hi) the
// part's.  Zeros take the place of what lies outside.
template <typename T, int L, int NT>
__device__ __forceinline__ void ask_tile(T *dst, const T *const (&src)[NT], int mode, int row0, int lo, int hi, int c0,
                                         int D) {
    const int lane = threadIdx.x & 31;
    if (mode == kWide) {
        constexpr int kPer = kScanChannels / wide_elems<T>();   // pieces of a row
        constexpr int kStep = 32 / kPer;                        // rows of one round of the warp
        const int r0 = lane / kPer, part = lane % kPer, c = c0 + part * wide_elems<T>();
#pragma unroll
        for (int k = 0; k < 2 * L / kStep; ++k) {
            const int r = r0 + k * kStep, t = row0 + (r & 1) * L + (r >> 1);
            const bool on = t >= lo && t < hi && c < D;
            const int64_t off = on ? (int64_t)t * D + c : 0;
            const unsigned d = (unsigned)__cvta_generic_to_shared(dst + r * kScanChannels + part * wide_elems<T>());
#pragma unroll
            for (int i = 0; i < NT; ++i) copy16(d + i * kWarpTile<T, L> * (int)sizeof(T), src[i] + off, on ? 16 : 0);
        }
        return;
    }
    const int half = lane >> 4, c = c0 + 2 * (lane & 15);
#pragma unroll 2
    for (int j = 0; j < L; ++j) {
        const int t = row0 + half * L + j;
        const bool on = t >= lo && t < hi;
        const bool on0 = on && c < D, on1 = on && c + 1 < D;
        const int64_t off = on0 ? (int64_t)t * D + c : 0;
        T *d = dst + (2 * j + half) * kScanChannels + 2 * (lane & 15);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            T *di = d + i * kWarpTile<T, L>;
            if (mode == kPair) {
                const unsigned da = (unsigned)__cvta_generic_to_shared(di);
                copy4(da, src[i] + off, on0 ? 4 : 0);
                if constexpr (sizeof(T) == 4) copy4(da + 4, src[i] + (on1 ? off + 1 : 0), on1 ? 4 : 0);
            } else {
                di[0] = on0 ? src[i][off] : from_f32<T>(0.f);
                di[1] = on1 ? src[i][off + 1] : from_f32<T>(0.f);
            }
        }
    }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A lane's two channels of token j.
template <typename T> __device__ __forceinline__ float2 read2(const T *tile, int j, int lane) {
    const T *p = tile + (2 * j + (lane >> 4)) * kScanChannels + 2 * (lane & 15);
    if constexpr (sizeof(T) == 4) {
        return *(const float2 *)p;
    } else {
        const uint32_t u = *(const uint32_t *)p;
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
}
template <typename T> __device__ __forceinline__ void write2(T *p, float a, float b) {
    if constexpr (sizeof(T) == 4) {
        *(float2 *)p = make_float2(a, b);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        *(uint32_t *)p = *(const uint32_t *)&v;
    }
}

// Calls f with the gate and the source as compile-time constants.
template <typename F> cudaError_t with_form(gdr_gate_t gate, gdr_source_t source, F &&f) {
    using std::integral_constant;
    auto by_source = [&](auto g) {
        switch (source) {
            case GDR_SOURCE_PLAIN: return f(g, integral_constant<int, GDR_SOURCE_PLAIN>{});
            case GDR_SOURCE_CONVEX: return f(g, integral_constant<int, GDR_SOURCE_CONVEX>{});
            default: return f(g, integral_constant<int, GDR_SOURCE_VARIANCE>{});
        }
    };
    return gate == GDR_GATE_BOUNDED ? by_source(integral_constant<int, GDR_GATE_BOUNDED>{})
                                    : by_source(integral_constant<int, GDR_GATE_SOFTPLUS>{});
}

}  // namespace scan
#endif  // __CUDACC__

// Launchers.  The shape holds the sizes; the launch fills in the division into parts and clusters.
cudaError_t launch_scan_fwd(const ScanFwd &t, ScanShape s, gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source,
                            int sms, int *status, cudaStream_t stream);
cudaError_t launch_scan_bwd(const ScanBwd &t, ScanShape s, gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source,
                            int sms, int *status, cudaStream_t stream);
cudaError_t launch_scan_step(const void *x, const void *a, float *state, void *out, int N, int T, int D, float b,
                             gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source, cudaStream_t stream);

// Division of the work: `slots` blocks run at a time.  Sequences of one length are chains of
// their own while there is room for all of them, else several follow each other in a part; then
// the tiles along a part go to the blocks of a cluster, as many as there is room for.
inline void scan_divide(ScanShape &s, int64_t slots) {
    s.tiles = (s.D + kScanChannels - 1) / kScanChannels;
    const int64_t room = slots / s.tiles > 1 ? slots / s.tiles : 1;
    s.per_part = s.cu ? s.N : (int)((s.N + room - 1) / room);
    s.parts = (s.N + s.per_part - 1) / s.per_part;
    const int64_t tokens = s.cu ? s.total : (int64_t)s.per_part * s.T_per;
    const int64_t most = room / s.parts, along = (tokens + kScanTile - 1) / kScanTile;
    int64_t c = most < along ? most : along;
    s.cluster = (int)(c > kScanMaxCluster ? kScanMaxCluster : c < 1 ? 1 : c);
}

}  // namespace gdr
