// gdr_scan_bwd.cu -- gradients of the gated scan.
//
// With l_t the gradient of h_t and r_t that of h_{t-1} through alpha_t:
//     l_t = dout_t + r_{t+1} (the last token's holds dhT too),   r_t = alpha_t l_t,  dh0 = r_1
//     dx_t = w l_t,   da_t = l_t (alpha_t h_{t-1} + w'(g_t) x_t) g'(a_t)
// One pass over the tiles from the last to the first: the gradient is chained backwards as the
// forward pass chains its states (gdr_scan.cuh), and the states within a tile are chained
// forwards again from the one that the forward pass kept in front of it.  Three tensors are
// read and two written, each once.  The runs of both directions share their A.
//
// A lane goes over its run once.  Of what enters the run, h and r, everything in it depends
// linearly: alpha_t h_{t-1} g' + w' x g' = c1 h + c0 and l_t = S r + l0 are kept as such, so that
// after the chaining one multiplication and addition each gives what was missing, and the tile
// in shared memory is read once.
//
// Measured (bf16): 8 x 4096 tokens of 2048 channels 201 to 204 us, 3.3 TB/s, 50% of a copy's rate; fp32, 8 x
// 2048: 136 us, 74%.  Bound like the forward pass by its arithmetic in its order (57 instructions an
// element, 52% of the issue slots), on 256 blocks for 304 places: with two sequences to a block the
// SMs that have one block end early, with one sequence to a block there are two rounds.
#include <algorithm>

#include "gdr_scan.cuh"

namespace gdr {
namespace {

using namespace scan;

constexpr int kL = 8;
constexpr int kWarps = kScanTile / (2 * kL);
constexpr int kThreads = 32 * kWarps;
constexpr int kBlocksPerSm = 2;
constexpr int kDepth = 2;
template <typename T, bool BOXES> using BwdRing = Ring<T, kL, kScanTile, 3, kDepth, BOXES>;

// Sequences that start with a run or end with it, and none within it.
__device__ __forceinline__ bool plain_marks(const Marks &m) {
    return !(m.first & ~1u) && !(m.last & ~(1u << (kL - 1)));
}

struct BwdMaps {
    CUtensorMap x, a, dout;
};

template <typename T, int GATE, int SRC, bool BOXES>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
scan_bwd_kernel(const __grid_constant__ ScanShape s, const __grid_constant__ BwdMaps maps, const T *x, const T *a, const T *dout, const float *__restrict__ h0,
                const float *__restrict__ dhT, const float *__restrict__ states, T *dx, T *da, float *dh0,
                int pairs, uint64_t limit_ns, int *status) {
    constexpr bool kFine = sizeof(T) == 4;
    extern __shared__ char smem[];
    __shared__ __align__(16) float4 agg[2][2][kWarps][16];   // the states' runs, and the gradients', last warp first
    __shared__ __align__(16) float4 told[2][kScanMaxCluster][16];
    __shared__ uint64_t bars[2], full[kDepth];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = lane >> 4, l = lane & 15;
    const int run_at0 = (warp * 2 + half) * kL;   // the lane's run in a tile
    const int CS = s.cluster, rank = blockIdx.x % CS, unit = blockIdx.x / CS;
    const int c0 = unit % s.tiles * kScanChannels, c = c0 + 2 * l, D = s.D;
    const int first = unit / s.tiles * s.per_part, last = min(s.N, first + s.per_part);
    if (!offsets_ok(s)) {
        if (threadIdx.x == 0) set_status(status, GDR_ERR_BAD_SEQLENS);
        return;
    }
    const int p0 = seq_start(s, first), p1 = seq_start(s, last);
    if (s.cu && dh0 && c0 + lane < D)   // sequences of no tokens
        for (int n = first + warp + rank * kWarps; n < last; n += kWarps * CS)
            if (seq_start(s, n) == seq_start(s, n + 1))
                dh0[(int64_t)n * D + c0 + lane] = dhT ? dhT[(int64_t)n * D + c0 + lane] : 0.f;
    const int t0 = p0 / kScanTile, t1 = (p1 + kScanTile - 1) / kScanTile, steps = (t1 - t0 + CS - 1) / CS;
    const bool many = last - first > 1;
    BwdRing<T, BOXES> ring((char *)(((uintptr_t)smem + 127) & ~(uintptr_t)127), full);
    if (threadIdx.x == 0) {
        ring.init();
        sm100::mbar_init(&bars[0], 1);
        sm100::mbar_init(&bars[1], 1);
        sm100::fence_mbar_init();
    }
    if (CS > 1)
        cluster_sync();   // every peer runs, and its barriers are set up, before its memory is written to
    else
        __syncthreads();
    const CUtensorMap *const map[3] = {&maps.x, &maps.a, &maps.dout};
    const T *const src[3] = {x, a, dout};
    // step i of this block: tile t1 - 1 - (i CS + rank), none below t0
    auto ask = [&](int i, int slot) {
        const int tile = t1 - 1 - (i * CS + rank);
        if (tile >= t0) ring.ask(slot, i, map, src, tile * kScanTile, p0, p1, c0, D);
        ring.close();
    };
    for (int i = 0; i < kDepth; ++i) ask(i, i);
    Peers peers{told, bars, limit_ns};
    Cursor cur{first, 0, -1};
    float2 carry = both(0.f);
    bool lost = false;   // a wait ran out: the results are lost, but every block goes through its steps
    // of the lane's run in the outputs' tile, in bytes
    const unsigned lane_out = ((unsigned)run_at0 * (unsigned)D + (unsigned)c) * (unsigned)sizeof(T);
    for (int i = 0, slot = 0, use = 0; i < steps; ++i) {
        if (CS > 1 && threadIdx.x == 0 && !lost) peers.expect(i, CS);
        const int tile_no = t1 - 1 - (i * CS + rank);
        const bool there = tile_no >= t0;
        const int base = there ? tile_no * kScanTile : p0 - kScanTile;
        // a tile that one sequence fills, and goes beyond on both sides
        bool inner = false;
        float2 h = both(0.f);
        if (there) {
            // the state in front of the tile: kept by the forward pass behind the tile before
            if (base > p0) h = load_state(states, tile_no - 1, D, c);
            cur.seek(s, first, last, max(base, p0));
            inner = cur.from < base && cur.to > base + kScanTile;
            if (!lost) lost = !__all_sync(kFull, ring.wait(slot, use, limit_ns));
            if constexpr (ring.kMode == kRows) ring.move(slot, src, base, c0, D);
        }
        const bool cuts = CS == 1 ? there && !inner : many || i == steps - 1;   // a part's first token is in the last step
        T *tx = ring.run(slot, 0, run_at0, l), *ta = ring.run(slot, 1, run_at0, l);
        T *td = ring.run(slot, 2, run_at0, l);
        const int p = base + run_at0, lo = max(p, p0), hi = min(p + kL, p1);
        // l_t = S r + l0,  alpha h_{t-1} g' + w' x g' = c1 h + c0
        float2 w[kL], S[kL], l0[kL], k1[kL], k0[kL];
        float2 A = both(1.f), B = both(0.f), R = both(0.f);
        if (there) {
            Cursor mine = cur;
            Marks m{0, 0};
            if (!inner) {
                m = marks_of(s, mine, first, last, p, lo, hi);
                if (hi - lo < kL) {
                    blank<T, kL>(tx, 0.f, p, lo, hi);
                    blank<T, kL>(ta, -INFINITY, p, lo, hi);
                    blank<T, kL>(td, 0.f, p, lo, hi);
                    sm100::fence_proxy_async_smem();   // before the slot is filled again
                }
            }
            auto pass = [&](auto marked) {
                float2 al[kL];
                int n = mine.n;
#pragma unroll
                for (int j = 0; j < kL; ++j) {
                    const float2 xv = read2(tx, j);
                    const Gate g = gate_of<kFine, GATE, SRC, true>(read2(ta, j), s);
                    al[j] = g.alpha;
                    w[j] = g.w;
                    const float2 q = mul2(g.slope, al[j]);
                    if (marked && (m.first >> j & 1)) {
                        n = seq_from(s, n, p + j);
                        B = load_state(h0, n, D, c);
                        A = both(-1.f);
                    }
                    k0[j] = SRC == GDR_SOURCE_PLAIN ? mul2(q, B) : fma2(q, B, mul2(g.dw, xv));
                    k1[j] = mul2(q, A);
                    B = fma2(al[j], B, SRC == GDR_SOURCE_PLAIN ? xv : mul2(w[j], xv));
                    if (marked)
                        decay_past_cut(A, al[j]);
                    else
                        A = mul2(A, al[j]);
                }
                if (marked && m.last) n = seq_from(s, mine.n, hi - 1);
                float2 P = both(1.f);
#pragma unroll
                for (int j = kL - 1; j >= 0; --j) {
                    float2 d = read2(td, j);
                    if (marked && (m.last >> j & 1)) {
                        n = seq_back(s, n, p + j);
                        d = add2(d, load_state(dhT, n, D, c));
                        R = both(0.f);
                    }
                    l0[j] = add2(d, R);
                    S[j] = P;
                    P = mul2(P, al[j]);
                    R = mul2(al[j], l0[j]);
                    if (marked && (m.first >> j & 1)) R = both(0.f);
                }
            };
            // a sequence that starts with the run or ends with it: what enters there is known
            if (plain_marks(m)) {
                if (m.first) B = load_state(h0, mine.n, D, c);
                if (m.last) R = load_state(dhT, seq_from(s, mine.n, p + kL - 1), D, c);
                pass(std::false_type{});
                if (m.first) {
                    A = both(-1.f);
                    R = both(0.f);
                }
            } else {
                pass(std::true_type{});
            }
        }
        float2 r;
        auto chain = [&](auto cuts) {
            const Run oh{other_half(A), other_half(B)}, og{oh.A, other_half(R)};
            // states: the first half's run, then the second's; gradients: the other way round, from the
            // last warp on.  The first half's lanes chain the states, the second half's the gradients.
            {
                const Run f = half ? follow(Run{A, R}, og, cuts) : follow(Run{A, B}, oh, cuts);
                agg[i & 1][half][half ? kWarps - 1 - warp : warp][l] = pack(f);
            }
            __syncthreads();
            if (!lost && inner) ask(i + kDepth, slot);
            const int my_place = half ? kWarps - 1 - warp : warp;
            if (CS == 1) {
                float2 e = half ? carry : h, at = e;
    #pragma unroll
                for (int v = 0; v < kWarps; ++v) {
                    if (v == my_place) at = e;
                    e = through(unpack(agg[i & 1][half][v][l]), e, cuts);
                }
                carry = e;   // (of the second half's lanes)
                const float2 theirs = other_half(at);
                h = half ? theirs : at;
                r = half ? at : theirs;
            } else {
                Run front{both(1.f), both(0.f)}, all = front;   // what comes before the warp, and all
    #pragma unroll
                for (int v = 0; v < kWarps; ++v) {
                    if (v == my_place) front = all;
                    all = follow(all, unpack(agg[i & 1][half][v][l]), cuts);
                }
                if (!lost && half)
                    for (int k = warp; k < CS; k += kWarps) peers.tell(i, k, rank, l, pack(all));
                if (!lost) lost = !__all_sync(kFull, peers.wait(i));
                float2 e = carry, in = e;
                for (int k = 0; k < CS; ++k) {
                    if (k == rank) in = e;
                    e = through(unpack(told[i & 1][k][l]), e, cuts);
                }
                carry = e;
                const float2 at = through(front, half ? in : h, cuts), theirs = other_half(at);
                h = half ? theirs : at;
                r = half ? at : theirs;
            }
            if (half)
                h = through(oh, h, cuts);
            else
                r = through(og, r, cuts);
        };
        if (cuts)
            chain(std::true_type{});
        else
            chain(std::false_type{});
        auto put = [&] {   // a run of tokens that are all the part's, with pairs of channels
            char *ox = (char *)(dx + (int64_t)base * D) + lane_out, *oa = (char *)(da + (int64_t)base * D) + lane_out;
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                const float2 lam = fma2(S[j], r, l0[j]);
                write2((T *)ox, SRC == GDR_SOURCE_PLAIN ? lam : mul2(w[j], lam));
                write2((T *)oa, mul2(lam, fma2(k1[j], h, k0[j])));
                ox += D * (int)sizeof(T);
                oa += D * (int)sizeof(T);
            }
        };
        if (inner && pairs) {
            if (c < D) put();
        } else if (there && c < D) {
            // (looked up again: what the steps above need not keep costs them no registers)
            Cursor mine = cur;
            const Marks m = inner ? Marks{0, 0} : marks_of(s, mine, first, last, p, lo, hi);
            if (pairs && hi - lo == kL && plain_marks(m)) {
                // nothing enters past a first token (k0 has what was there), nor in front of a last one
                if (m.first) h = both(0.f);
                if (m.last) r = both(0.f);
                put();
                if (dh0 && m.first) {
                    const Gate g = gate_of<kFine, GATE, SRC, false>(read2(ta, 0), s);
                    store_state(dh0, mine.n, D, c, mul2(g.alpha, fma2(S[0], r, l0[0])));
                }
            } else {
                const int from = m.first ? __ffs(m.first) - 1 : kL, upto = 31 - __clz(m.last);
                int n = mine.n;
    #pragma unroll
                for (int j = 0; j < kL; ++j) {
                    const int t = p + j;
                    if (t < lo || t >= hi) continue;
                    const float2 lam = j <= upto ? l0[j] : fma2(S[j], r, l0[j]);
                    const float2 gx = mul2(w[j], lam), ga = mul2(lam, j >= from ? k0[j] : fma2(k1[j], h, k0[j]));
                    T *ox = dx + (int64_t)t * D + c, *oa = da + (int64_t)t * D + c;
                    if (pairs) {
                        write2(ox, gx);
                        write2(oa, ga);
                    } else {
                        ox[0] = from_f32<T>(gx.x);
                        oa[0] = from_f32<T>(ga.x);
                        if (c + 1 < D) {
                            ox[1] = from_f32<T>(gx.y);
                            oa[1] = from_f32<T>(ga.y);
                        }
                    }
                    if (dh0 && (m.first >> j & 1)) {
                        n = seq_from(s, n, t);
                        const Gate g = gate_of<kFine, GATE, SRC, false>(read2(ta, j), s);
                        store_state(dh0, n, D, c, mul2(g.alpha, lam));
                    }
                }
            }
        }
        if (!inner) {
            __syncthreads();   // the gates have been read again
            if (!lost) ask(i + kDepth, slot);
        }
        if (++slot == kDepth) {
            slot = 0;
            ++use;
        }
    }
    ring.drain(lost);
    peers.leave(lost, CS, status);
}

template <typename T, int GATE, int SRC>
cudaError_t launch_bwd_t(const ScanBwd &t, ScanShape s, int sms, int *status, cudaStream_t stream) {
    BwdMaps maps{};
    constexpr gdr_dtype_t kType = sizeof(T) == 2 ? GDR_BF16 : GDR_F32;
    auto plane = [&](CUtensorMap *m, const void *p) {
        return tc_make_plane_map(m, p, kType, s.D, s.total, kScanChannels, kScanTile);
    };
    const bool boxes = s.total > 0 && plane(&maps.x, t.x) && plane(&maps.a, t.a) && plane(&maps.dout, t.dout);
    const uintptr_t outs = (uintptr_t)t.dx | (uintptr_t)t.da;
    const int pairs = s.D % 2 == 0 && outs % (2 * sizeof(T)) == 0;
    auto run = [&](auto by_boxes, ScanRoom &known) {
        constexpr bool kB = by_boxes();
        const int smem = BwdRing<T, kB>::kBytes + 128;
        return scan_launch(scan_bwd_kernel<T, GATE, SRC, kB>, s, kThreads, smem, kScanTile, sms, known, "scan_bwd_kernel", stream,
                       maps, (const T *)t.x, (const T *)t.a, (const T *)t.dout, t.h0, t.dhT, t.states, (T *)t.dx, (T *)t.da,
                       t.dh0, pairs, scan_wait_ns(), status);
    };
    static ScanRoom boxed, other;
    return boxes ? run(std::true_type{}, boxed) : run(std::false_type{}, other);
}

}  // namespace

cudaError_t launch_scan_bwd(const ScanBwd &t, ScanShape s, gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source,
                            int sms, int *status, cudaStream_t stream) {
    return with_form(s, dtype, gate, source, [&](auto type, auto g, auto w) {
        return launch_bwd_t<decltype(type), g(), w()>(t, s, sms, status, stream);
    });
}

}  // namespace gdr
