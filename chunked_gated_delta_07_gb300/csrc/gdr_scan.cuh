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

#include <atomic>
#include <cstdlib>
#include <type_traits>

#include "gdr_internal.cuh"
#include "gdr_pairs.cuh"
#include "gdr_sm100.cuh"
#include "gdr_tc.cuh"

namespace gdr {

constexpr int kScanTile = 128;      // tokens of a tile; the interval of the states kept for the backward pass
constexpr int kScanChannels = 32;   // channels of a tile
constexpr int kScanMaxCluster = 16;
constexpr int kScanMaxD = 1 << 22;  // a tile's offsets are 32-bit
constexpr int64_t kScanMaxTokens = 0x7fffffff - 2 * kScanTile * kScanMaxCluster;   // positions are 32-bit

// The gates as the kernels tell them apart.  With a bound of at most 2, alpha >= e^-2, bf16 tensors take
// 1 - alpha from one polynomial (8 x 4096 tokens of 2048 channels forward 95 us, with an exponential beside
// it 107).  What 1 - alpha is off by counts 1 / alpha times in alpha: up to 21 * 2^-24 of it at b = 2 and s = 1,
// where a memory is of a token, 4 * 2^-24 at b = 1 (emulated with an exact sigmoid s).  fp32 tensors take the
// exponential at any bound (8 x 2048 tokens forward 74 us, by that polynomial 70).
enum ScanGate { kBounded = GDR_GATE_BOUNDED, kSoftplus = GDR_GATE_SOFTPLUS, kBoundedBy2 };
constexpr int kScanPoly = 8;

struct ScanShape {
    const int32_t *cu;   // offsets of packed sequences, or null: N sequences of T_per tokens
    int N, T_per, total, D;
    float b;
    float poly[kScanPoly];   // of kBoundedBy2: 1 - alpha = s sum_k poly[k] s^k, s the sigmoid
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
// The special-function unit's accuracy, also for fp32 tensors (FINE), whose exponentials' arguments keep
// the rounding error of the product with log2 e, which is |a| 2^-24 of the exponential (8 x 2048 fp32
// tokens of 2048 channels, bound 8, forward 76 us; bound 2 with the library's exponentials, reciprocals and
// roots 175).  alpha of fp32 tensors is off by at most (n (1.25 (1 - s) + 1) + 1.75) 2^-22 of itself, n = b s; with
// bounds of at most 2 that holds without the argument's error, which is n 2^-23.  What a long memory hangs on,
// 1 - alpha for alpha near 1, keeps its relative accuracy: 1 - e^-n comes from a polynomial, and alpha from that.
constexpr float kLog2e = 1.44269504088896341f, kLog2eRest = 1.925963033500e-8f, kLn2 = 0.693147180559945f;
// 2^x
__device__ __forceinline__ float2 exp2_fast(float2 x) {
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x.y));
    return x;
}
// e^-x
template <bool FINE> __device__ __forceinline__ float2 exp_minus(float2 x) {
    const float2 hi = mul2(x, both(-kLog2e)), e = exp2_fast(hi);
    if constexpr (!FINE) return e;
    // x log2 e = -(hi + lo): 2^(hi + lo) = 2^hi (1 + lo ln 2); 2^hi is infinite from x = -88 on, and takes none
    const float2 lo = fma2(x, both(-kLog2eRest), make_float2(fmaf(x.x, -kLog2e, -hi.x), fmaf(x.y, -kLog2e, -hi.y)));
    const float2 c = mul2(lo, both(kLn2));
    return make_float2(fabsf(x.x) < 87.f ? fmaf(e.x, c.x, e.x) : e.x, fabsf(x.y) < 87.f ? fmaf(e.y, c.y, e.y) : e.y);
}
__device__ __forceinline__ float2 inverse(float2 x) {
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x.y));
    return x;
}
// max and min that keep a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
    return a;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
    return a;
}

struct Gate {
    float2 alpha, w;     // the decay and the input's weight
    float2 slope, dw;    // dg/da, and dw/dg dg/da
};

template <bool FINE, int GATE, int SRC, bool GRAD>
__device__ __forceinline__ Gate gate_of(float2 a, const ScanShape &shape) {
    Gate o;
    float2 left;   // 1 - alpha
    const float2 one = both(1.f), minus = both(-1.f);
    const float b = shape.b;
    if constexpr (GATE == kBoundedBy2 && !FINE) {
        const float2 e = exp_minus<FINE>(a), s = inverse(add2(e, one));
        if constexpr (GRAD) {
            const float2 c = make_float2(min_nan(e.x, 1e38f), min_nan(e.y, 1e38f));
            o.slope = mul2(mul2(s, both(-b)), mul2(c, s));
        }
        float2 p = both(shape.poly[kScanPoly - 1]);
#pragma unroll
        for (int k = kScanPoly - 2; k >= 0; --k)
            p = make_float2(fmaf(p.x, s.x, shape.poly[k]), fmaf(p.y, s.y, shape.poly[k]));
        left = mul2(s, p);
        o.alpha = fma2(left, minus, one);
    } else if constexpr (GATE != kSoftplus) {
        // e^-a may be inf: the sigmoid is 0 then
        const float2 e = exp_minus<FINE>(a), s = inverse(add2(e, one));
        const float2 n = mul2(s, both(b));   // -g
        if constexpr (GRAD) {
            // g' = -b s (1 - s), 1 - s = e^-a s
            const float2 c = make_float2(min_nan(e.x, 1e38f), min_nan(e.y, 1e38f));
            o.slope = mul2(mul2(n, minus), mul2(c, s));
        }
        // (1 - e^-n) / n on [0, 1/2] by a polynomial fitted to it (relative error 1e-8 with these
        // coefficients)
        float2 p = both(-0.0011259226594120264f);
        p = fma2(p, n, both(0.008193295449018478f));
        p = fma2(p, n, both(-0.04163204878568649f));
        p = fma2(p, n, both(0.16666288673877716f));
        p = fma2(p, n, both(-0.49999985098838806f));
        p = fma2(p, n, one);
        const float2 near = mul2(n, p), above = fma2(near, minus, one);
        const float2 far = FINE && GATE == kBounded ? exp_minus<FINE>(n) : exp2_fast(mul2(s, both(-b * kLog2e)));
        const float2 below = fma2(far, minus, one);
        const bool s0 = n.x < 0.5f, s1 = n.y < 0.5f;
        left = make_float2(s0 ? near.x : below.x, s1 ? near.y : below.y);
        o.alpha = make_float2(s0 ? above.x : far.x, s1 ? above.y : far.y);
    } else {
        // e^{-softplus(a)} = 1 / (1 + e^a)
        const float2 e = exp_minus<FINE>(make_float2(fabsf(a.x), fabsf(a.y)));
        const float2 lo = mul2(e, inverse(add2(e, one))), hi = fma2(lo, minus, one);
        const bool s0 = a.x > 0.f, s1 = a.y > 0.f;
        o.alpha = make_float2(s0 ? lo.x : hi.x, s1 ? lo.y : hi.y);
        left = make_float2(s0 ? hi.x : lo.x, s1 ? hi.y : lo.y);
        if constexpr (GRAD) o.slope = mul2(left, minus);
    }
    if constexpr (SRC == GDR_SOURCE_PLAIN) {
        o.w = one;
        o.dw = both(0.f);
    } else if constexpr (SRC == GDR_SOURCE_CONVEX) {
        o.w = left;
        if constexpr (GRAD) o.dw = mul2(mul2(o.alpha, o.slope), minus);
    } else {
        // w = sqrt(1 - alpha^2), w' = -alpha^2 / w g'.  At w = 0 g' is 0 too, and goes to it faster.
        const float2 z = fma2(left, o.alpha, left);
        float2 r = z;
        if constexpr (GRAD) r = make_float2(max_nan(z.x, 1.2e-38f), max_nan(z.y, 1.2e-38f));
        if constexpr (GRAD) {
            asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(r.x));
            asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(r.y));
            o.w = mul2(z, r);
        } else {
            asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(o.w.x) : "f"(z.x));
            asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(o.w.y) : "f"(z.y));
        }
        if constexpr (GRAD) o.dw = mul2(mul2(mul2(o.alpha, o.alpha), minus), mul2(o.slope, r));
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
        if (token >= to && to > 0 && n + 1 < last) {   // going up, mostly the next one
            const int next = seq_start(s, n + 2);
            if (token < next) {
                ++n;
                from = to;
                to = next;
                return;
            }
            lo = n + 1;
        } else if (token < from && n > first) {   // going down, mostly the one before
            const int prev = seq_start(s, n - 1);
            if (token >= prev) {
                --n;
                to = from;
                from = prev;
                return;
            }
            hi = n - 1;
        }
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq_start(s, mid) <= token) lo = mid; else hi = mid - 1;
        }
        n = lo;
        from = seq_start(s, n);
        to = seq_start(s, n + 1);
    }
};

// The sequence of token t, going up from n, or down: steps that double while they stay on n's side of
// it and halve where they would not, so that any number of sequences without tokens in between costs
// its logarithm in loads (four sequences with three times 20000 empty ones between them: 435 us forward
// and 263 backward; with steps of one 3109 and 4948).
__device__ __forceinline__ int seq_from(const ScanShape &s, int n, int t) {
    int step = 1;
    while (seq_start(s, n + 1) <= t) {
        const int m = n + min(step, s.N - n);
        if (seq_start(s, m) <= t) {
            n = m;
            step += step;
        } else {
            step = (step + 1) >> 1;
        }
    }
    return n;
}
__device__ __forceinline__ int seq_back(const ScanShape &s, int n, int t) {
    int step = 1;
    while (seq_start(s, n) > t) {
        const int m = n - min(step, n);
        if (step == 1 || seq_start(s, m) > t) {
            n = m;
            step += step;
        } else {
            step >>= 1;
        }
    }
    return n;
}

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
        n = seq_from(s, n, q) + 1;   // past empty sequences; the part's end is beyond q
        q = seq_start(s, n);
    }
    return m;
}
// Whether the offsets are 0 = c0 <= c1 <= .. <= cN = total; the whole block calls.
__device__ __forceinline__ bool offsets_ok(const ScanShape &s) {
    if (!s.cu) return true;
    int bad = threadIdx.x == 0 && (s.cu[0] != 0 || s.cu[s.N] != s.total);
    for (int i = threadIdx.x; i < s.N; i += blockDim.x) bad |= s.cu[i] > s.cu[i + 1];
    return !__syncthreads_or(bad);
}

// ---- chaining ---------------------------------------------------------------------------
// A run of both channels: h_out = A h + B.
struct Run {
    float2 A, B;
};
__device__ __forceinline__ bool is_cut(float A) { return __float_as_int(A) < 0; }
__device__ __forceinline__ float4 pack(const Run &r) { return make_float4(r.A.x, r.A.y, r.B.x, r.B.y); }
__device__ __forceinline__ Run unpack(float4 v) { return Run{make_float2(v.x, v.y), make_float2(v.z, v.w)}; }
// What comes out of a run for h going in; past a cut that is B.
__device__ __forceinline__ float2 through(const Run &r, float2 h, bool cuts) {
    if (cuts) h = make_float2(is_cut(r.A.x) ? 0.f : h.x, is_cut(r.A.y) ? 0.f : h.y);
    return fma2(r.A, h, r.B);
}
// The run f followed by the run r; a cut in either stays one.
__device__ __forceinline__ Run follow(Run f, const Run &r, bool cuts) {
    if (!cuts) return Run{mul2(f.A, r.A), fma2(r.A, f.B, r.B)};
    const bool c0 = is_cut(r.A.x), c1 = is_cut(r.A.y);
    Run o;
    o.B = fma2(r.A, make_float2(c0 ? 0.f : f.B.x, c1 ? 0.f : f.B.y), r.B);
    o.A.x = c0 ? r.A.x : is_cut(f.A.x) ? f.A.x : f.A.x * r.A.x;
    o.A.y = c1 ? r.A.y : is_cut(f.A.y) ? f.A.y : f.A.y * r.A.y;
    return o;
}
// A := A alpha; a cut stays one, also in front of a NaN.
__device__ __forceinline__ void decay_past_cut(float2 &A, float2 alpha) {
    if (!is_cut(A.x)) A.x *= alpha.x;
    if (!is_cut(A.y)) A.y *= alpha.y;
}
__device__ __forceinline__ float2 other_half(float2 v) {
    return make_float2(__shfl_xor_sync(kFull, v.x, 16), __shfl_xor_sync(kFull, v.y, 16));
}

// ---- clusters ------------------------------------------------------------------------------
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// The blocks of a cluster tell each other their tile's run, every step (with the cluster's barrier
// instead, whose release waits for the outputs' stores too, 262144 tokens took 932 us against 860 at
// the time): a row of 16 lanes' pairs
// into every peer's memory, each counted by the peer's barrier for the step (two of them taken in
// turn; nobody can be two steps ahead, since a step needs everyone's).
struct Peers {
    float4 (*slot)[kScanMaxCluster][16];   // [2] steps
    uint64_t *bar;                         // [2]
    uint64_t limit_ns;

    __device__ __forceinline__ static unsigned peer(const void *at, unsigned rank) {
        unsigned a;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(sm100::smem_u32(at)), "r"(rank));
        return a;
    }
    // Thread 0, once a step: what this block waits for.
    __device__ __forceinline__ void expect(int step, int cluster) {
        sm100::mbar_arrive_expect_tx(&bar[step & 1], cluster * 16 * (unsigned)sizeof(float4));
    }
    __device__ __forceinline__ void tell(int step, unsigned to, int rank, int l, float4 v) {
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                         peer(&slot[step & 1][rank][l], to)),
                     "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(peer(&bar[step & 1], to))
                     : "memory");
    }
    // Every thread; false when the wait ran out.
    __device__ __forceinline__ bool wait(int step) {
        const unsigned at = sm100::smem_u32(&bar[step & 1]), parity = step >> 1 & 1;
        auto done = [&] {
            unsigned ok;
            asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                         : "=r"(ok)
                         : "r"(at), "r"(parity)
                         : "memory");
            return ok != 0;
        };
        if (limit_ns == 0) return false;
        if (done()) return true;
        const uint64_t since = sm100::globaltimer_ns();
        while (sm100::globaltimer_ns() - since < limit_ns)
            if (done()) return true;
        return false;
    }
    // The block's end; every thread calls, none with a copy under way.  Nobody leaves while a peer may
    // still write to its memory: behind the cluster's barrier every peer has sent its last run.  With no wait
    // run out all of them have been counted, by the last step's wait.  Where one has (a lost block), what
    // was sent is not all counted, and the barrier does not wait for such stores: the block stays a
    // millisecond longer, a thousand times their way.
    __device__ __forceinline__ static void leave(bool lost, int cluster, int *status) {
        lost = __syncthreads_or(lost);
        if (lost && threadIdx.x == 0) set_status(status, GDR_ERR_TIMEOUT);
        if (cluster == 1) return;
        cluster_sync();
        if (lost && threadIdx.x == 0) settle();
    }
    __device__ __forceinline__ static void settle() {
        const uint64_t since = sm100::globaltimer_ns();
        while (sm100::globaltimer_ns() - since < 1000000) {}
    }
};

// ---- tiles of raw inputs ------------------------------------------------------------------
// BOXES: a TMA box of each tensor (rows and bases on 16-byte boundaries).  ROWS (bf16): the 16-byte pieces
// of each row that hold one of its channels, each by a lane's asynchronous copy; the lanes then move their
// run's channels to where a box would have them.  PAIRS (fp32): a lane copies its own two channels.
//
// 8 x 4096 bf16 tokens, forward and backward: 2048 channels in boxes 95 and 204 us, 2046 and 2047 in
// rows 184 and 340, 236 and 448 (with bulk copies of whole rows 226 and 450, 277 and 545: the copy
// unit takes some 16 cycles a row; element by element 2047 channels 690 and 1200).  8 x 2048 fp32
// tokens of 2047 channels: pairs 206 and 287, rows, at the time, 179 and 388 (fewer blocks fit).
enum CopyMode { kBoxes, kRows, kPairs };
template <typename T, bool BOXES> constexpr CopyMode copy_mode() { return BOXES ? kBoxes : sizeof(T) == 2 ? kRows : kPairs; }
__device__ __forceinline__ void copy4(unsigned dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(unsigned dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A block's ring of DEPTH tiles of NT tensors, TOK tokens each; a lane's run is L of them.
// Boxes have kernels of their own (BOXES).
template <typename T, int L, int TOK, int NT, int DEPTH, bool BOXES> struct Ring {
    static constexpr CopyMode kMode = copy_mode<T, BOXES>();
    static constexpr int kRow = kScanChannels * (int)sizeof(T);   // bytes of a row as it is read
    static constexpr int kRawRow = kRow + 16;                     // and of its pieces
    static constexpr int kPitch = kMode == kRows ? kRawRow : kRow;   // from row to row, before rows are moved
    static constexpr int kBytes = DEPTH * NT * TOK * kPitch;
    char *at;          // [DEPTH][NT] tiles of TOK rows, 128-byte aligned
    uint64_t *full;    // [DEPTH]: the slot's copies are there
    int issued;        // tiles asked for by boxes

    __device__ __forceinline__ Ring(char *smem, uint64_t *bars) : at(smem), full(bars), issued(0) {}
    // Thread 0, before the first use.
    __device__ __forceinline__ void init() {
        for (int i = 0; i < DEPTH; ++i) sm100::mbar_init(&full[i], 1);
    }
    __device__ __forceinline__ char *tile(int slot, int tensor) const { return at + (slot * NT + tensor) * TOK * kPitch; }
    // A lane's two channels of its run's first token; the others follow, kScanChannels elements apart.
    __device__ __forceinline__ T *run(int slot, int tensor, int first, int l) const {
        return (T *)(tile(slot, tensor) + first * kPitch) + 2 * l;
    }

    // Every thread: asks for the tile from token `row` on, after the whole block is done with what
    // was in the slot.  The boxes are issued by a lane of one warp, which costs that warp some 400
    // cycles; the warps take turns.
    __device__ __forceinline__ void ask(int slot, int turn, const CUtensorMap *const (&maps)[NT], const T *const (&src)[NT],
                                        int row, int lo, int hi, int c0, int D) {
        if constexpr (kMode == kBoxes) {
            if (threadIdx.x == 32 * (turn % (TOK / (2 * L)))) {
                sm100::mbar_arrive_expect_tx(&full[slot], NT * TOK * kRow);
#pragma unroll
                for (int i = 0; i < NT; ++i) sm100::tma_load_2d(tile(slot, i), maps[i], c0, row, &full[slot]);
            }
            ++issued;
        } else if constexpr (kMode == kRows) {
            ask_rows(tile(slot, 0), src[0], src[1], src[NT - 1], row, lo, hi, c0, D);
        } else {
            ask_pairs(tile(slot, 0), src[0], src[1], src[NT - 1], row, lo, hi, c0, D);
        }
    }
    // The warp's own rows, as many of them at once as have pieces for its lanes.  A piece of 16 bytes
    // that holds one of the row's elements lies within the allocation that holds that element.
    // (These are functions apart that take values: they are called once a step at most, and would
    // cost the steps' code registers.)
    __device__ __noinline__ static void ask_rows(char *to, const T *s0, const T *s1, const T *s2, int row, int lo, int hi,
                                                 int c0, int D) {
        static_assert(sizeof(T) == 2);
        const T *const src[3] = {s0, s1, s2};
        constexpr int kPieces = kRawRow / 16, kAtOnce = 32 / kPieces;
        const int lane = threadIdx.x & 31, mine = lane / kPieces, piece = lane % kPieces;
        const int first = (threadIdx.x >> 5) * 2 * L, width = min(kScanChannels, D - c0) * (int)sizeof(T);
        if (mine >= kAtOnce) return;
#pragma unroll 2
        for (int r = mine; r < 2 * L; r += kAtOnce) {
            const int t = row + first + r;
            if (t < lo || t >= hi) continue;
            const int64_t off = (int64_t)t * D + c0;
#pragma unroll
            for (int k = 0; k < NT; ++k) {
                const uintptr_t p = (uintptr_t)(src[k] + off), q = (p & ~(uintptr_t)15) + 16 * piece;
                if (q < p + width)
                    copy16(sm100::smem_u32(to + (k * TOK + first + r) * kRawRow + 16 * piece), (const void *)q);
            }
        }
    }
    __device__ __noinline__ static void ask_pairs(char *to, const T *s0, const T *s1, const T *s2, int row, int lo, int hi,
                                                  int c0, int D) {
        static_assert(sizeof(T) == 4);   // the copies' 4 bytes
        const T *const src[3] = {s0, s1, s2};
        const int lane = threadIdx.x & 31, c = c0 + 2 * (lane & 15);
        const int first = ((threadIdx.x >> 5) * 2 + (lane >> 4)) * L;
#pragma unroll 4
        for (int j = first; j < first + L; ++j) {
            const int t = row + j;
            const bool on0 = t >= lo && t < hi && c < D, on1 = on0 && c + 1 < D;
            const int64_t off = on0 ? (int64_t)t * D + c : 0;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const unsigned d = sm100::smem_u32(to + (i * TOK + j) * kRow) + 2 * (lane & 15) * (unsigned)sizeof(T);
                copy4(d, src[i] + off, on0 ? 4 : 0);
                copy4(d + 4, src[i] + (on1 ? off + 1 : 0), on1 ? 4 : 0);
            }
        }
    }
    // Closes a step's asking (also one that asked for nothing): every step, once.
    __device__ __forceinline__ void close() {
        if constexpr (!BOXES) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // Every thread: the slot's tile of `use` (its use'th) is there, or false where the wait ran out.
    __device__ __forceinline__ bool wait(int slot, int use, uint64_t limit_ns) {
        if constexpr (BOXES)
            return limit_ns && sm100::mbar_try_wait(&full[slot], use & 1) ? true : wait_long(&full[slot], use & 1, limit_ns);
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        __syncwarp();
        return true;
    }
    __device__ __noinline__ static bool wait_long(uint64_t *bar, int parity, uint64_t limit_ns) {
        return sm100::mbar_wait(bar, parity, limit_ns);
    }
    // The whole warp: moves the channels of its runs from where the rows' copies put them; rows
    // come to lie 16 bytes closer, so a row is read before anything is written over it.
    __device__ __forceinline__ void move(int slot, const T *const (&src)[NT], int token, int c0, int D) const {
        move_rows(tile(slot, 0), src[0], src[1], src[NT - 1], token, c0, D);
    }
    __device__ __noinline__ static void move_rows(char *at, const T *s0, const T *s1, const T *s2, int token, int c0, int D) {
        const T *const src[3] = {s0, s1, s2};
        const int lane = threadIdx.x & 31, l = lane & 15, first = ((threadIdx.x >> 5) * 2 + (lane >> 4)) * L;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const char *raw = at + (i * TOK + first) * kRawRow;
            T *to = (T *)raw + 2 * l;
            const T *p = src[i] + (int64_t)(token + first) * D + c0;
#pragma unroll 1
            for (int j = 0; j < L; j += 4) {
                T v[4][2];
#pragma unroll
                for (int k = 0; k < 4; ++k, raw += kRawRow, p += D) {
                    const T *q = (const T *)(raw + ((uintptr_t)p & 15)) + 2 * l;
                    v[k][0] = q[0];
                    v[k][1] = q[1];
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k, to += kScanChannels) {
                    to[0] = v[k][0];
                    to[1] = v[k][1];
                }
            }
            __syncwarp();
        }
    }
    // No copy of this block's is under way any more, also after a wait that ran out.
    __device__ __forceinline__ void drain(bool lost) {
        if constexpr (!BOXES)
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        else if (lost)
            for (int k = max(0, issued - DEPTH); k < issued; ++k)
                sm100::mbar_wait(&full[k % DEPTH], k / DEPTH & 1, 2000000000ull);
    }
};

template <typename T> __device__ __forceinline__ float2 read2(const T *run, int j) {
    const T *p = run + j * kScanChannels;
    if constexpr (sizeof(T) == 4) {
        return *(const float2 *)p;
    } else {
        const uint32_t u = *(const uint32_t *)p;
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
}
template <typename T> __device__ __forceinline__ void write2(T *p, float2 x) {
    if constexpr (sizeof(T) == 4) {
        *(float2 *)p = x;
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x.x, x.y);
        *(uint32_t *)p = *(const uint32_t *)&v;
    }
}
// What a lane's L tokens from p outside [lo, hi) hold: gates of -inf, which keep the state and take
// no input, and zeros in the other tensors.
template <typename T, int L> __device__ __forceinline__ void blank(T *run, float value, int p, int lo, int hi) {
#pragma unroll 1
    for (int j = 0; j < L; ++j)
        if (p + j < lo || p + j >= hi) run[j * kScanChannels] = run[j * kScanChannels + 1] = from_f32<T>(value);
}
// Two channels of a row of fp32 states, those that exist.
__device__ __forceinline__ float2 load_state(const float *p, int64_t row, int D, int c) {
    if (!p) return make_float2(0.f, 0.f);
    p += row * D + c;
    return make_float2(c < D ? p[0] : 0.f, c + 1 < D ? p[1] : 0.f);
}
__device__ __forceinline__ void store_state(float *p, int64_t row, int D, int c, float2 v) {
    p += row * D + c;
    if (c < D) p[0] = v.x;
    if (c + 1 < D) p[1] = v.y;
}

// Calls f with the type, the gate and the source as compile-time constants; completes the shape.
template <typename F>
cudaError_t with_form(ScanShape &s, gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source, F &&f) {
    using std::integral_constant;
    auto by_source = [&](auto t, auto g) {
        switch (source) {
            case GDR_SOURCE_PLAIN: return f(t, g, integral_constant<int, GDR_SOURCE_PLAIN>{});
            case GDR_SOURCE_CONVEX: return f(t, g, integral_constant<int, GDR_SOURCE_CONVEX>{});
            default: return f(t, g, integral_constant<int, GDR_SOURCE_VARIANCE>{});
        }
    };
    auto by_gate = [&](auto t) {
        if (gate == GDR_GATE_SOFTPLUS) return by_source(t, integral_constant<int, kSoftplus>{});
        if (s.b <= 2.f) {
            // (1 - e^-n) / n on [0, 2] by a polynomial fitted to it, within 1.8e-8 (4.1e-8 of itself at n = 2)
            static const double fit[kScanPoly] = {0.99999998631057,       -0.4999991992693423,  0.16665864060437813,
                                                  -0.04163556673545308,   0.008272895784878453, -0.0013234571801574847,
                                                  0.00015753673867873683, -1.0291639928970174e-05};
            double n = s.b;
            for (int k = 0; k < kScanPoly; ++k, n *= s.b) s.poly[k] = (float)(fit[k] * n);
            return by_source(t, integral_constant<int, kBoundedBy2>{});
        }
        return by_source(t, integral_constant<int, kBounded>{});
    };
    return dtype == GDR_BF16 ? by_gate(__nv_bfloat16{}) : by_gate(float{});
}

}  // namespace scan
#endif  // __CUDACC__

// Launchers.  The shape holds the sizes; the launch fills in the division into parts and clusters.
cudaError_t launch_scan_fwd(const ScanFwd &t, ScanShape s, gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source,
                            int sms, int *status, cudaStream_t stream);
cudaError_t launch_scan_bwd(const ScanBwd &t, ScanShape s, gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source,
                            int sms, int *status, cudaStream_t stream);
cudaError_t launch_scan_step(const void *x, const void *a, float *state, void *out, ScanShape s, gdr_dtype_t dtype,
                             gdr_gate_t gate, gdr_source_t source, cudaStream_t stream);

// The limit of a wait for the peers of a cluster: 2 s, or GDR_TC_WAIT_NS (the tests make waits
// run out with it).
inline uint64_t scan_wait_ns() {
    const char *w = std::getenv("GDR_TC_WAIT_NS");
    return w ? (uint64_t)std::strtoull(w, nullptr, 10) : 2000000000ull;
}

// Division of the work: `slots` blocks run at a time, and clusters of 2^k blocks as many as room[k]
// says.  Sequences of one length are chains of their own while there is room for all of them, else
// several follow each other in a part; then the tiles along a part go to the blocks of a cluster, as
// many as leave all clusters running at once.  More of them, in turns, would wait for each other:
// 262144 tokens of 2048 channels 820 us with clusters of 8 (one round), 920 with 16 (two); 65536
// packed tokens of 1000 channels 235 with 8, 179 with 16 (one round both).
constexpr int kScanSizes = 5;   // 1, 2, 4, 8, 16 blocks
inline void scan_divide(ScanShape &s, const int (&room)[kScanSizes], int tok) {
    s.tiles = (s.D + kScanChannels - 1) / kScanChannels;
    const int64_t fit = room[0] / s.tiles > 1 ? room[0] / s.tiles : 1;
    s.per_part = s.cu ? s.N : (int)((s.N + fit - 1) / fit);
    s.parts = (s.N + s.per_part - 1) / s.per_part;
    const int64_t tokens = s.cu ? s.total : (int64_t)s.per_part * s.T_per;
    const int64_t units = (int64_t)s.parts * s.tiles, along = (tokens + tok - 1) / tok;
    s.cluster = 1;
    for (int k = 1; k < kScanSizes; ++k)
        if ((1 << k) < 2 * along && units <= room[k]) s.cluster = 1 << k;
}

using ScanRoom = std::atomic<int>[16][kScanSizes];   // by device

#ifdef __CUDACC__
// How many blocks, and clusters of 2, 4, 8 and 16 blocks, of a kernel run at a time on the current
// device; the kernel's attributes are set, and this is asked for, once per kernel and device.
template <typename K>
cudaError_t scan_room(K kern, int threads, int smem, int sms, ScanRoom &known, int (&room)[kScanSizes]) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const bool keep = dev < 16;
    if (keep && known[dev][0].load(std::memory_order_acquire) > 0) {
        for (int k = 0; k < kScanSizes; ++k) room[k] = known[dev][k].load(std::memory_order_relaxed);
        return cudaSuccess;
    }
    if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return err;
    if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return err;
    int per_sm = 0;
    if ((err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem)) != cudaSuccess) return err;
    room[0] = per_sm * sms;
    for (int k = 1; k < kScanSizes; ++k) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(1u << k);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 1u << k;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if ((err = cudaOccupancyMaxActiveClusters(&room[k], kern, &cfg)) != cudaSuccess) return err;
    }
    if (keep)
        for (int k = kScanSizes - 1; k >= 0; --k) known[dev][k].store(room[k], std::memory_order_release);
    return cudaSuccess;
}

// One launch: the attributes, the division, the clusters.
template <typename K, typename... A>
cudaError_t scan_launch(K kern, ScanShape &s, int threads, int smem, int tok, int sms,
                        ScanRoom &known, const char *name, cudaStream_t stream, A... args) {
    int room[kScanSizes];
    cudaError_t err = scan_room(kern, threads, smem, sms, known, room);
    if (err != cudaSuccess) return err;
    scan_divide(s, room, tok);
    const int64_t blocks = (int64_t)s.tiles * s.parts * s.cluster;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)s.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = s.cluster > 1 ? 1 : 0;
    ProfScope prof(stream, name);
    err = cudaLaunchKernelEx(&cfg, kern, s, args...);
    count_launch();
    return err;
}
#endif

}  // namespace gdr
