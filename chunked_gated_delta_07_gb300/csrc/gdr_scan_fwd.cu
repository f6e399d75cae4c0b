// gdr_scan_fwd.cu -- the gated scan forward over prompts, and token by token.
//
// Per (sequence, channel) h_t = alpha_t h_{t-1} + w(alpha_t) x_t (gdr_scan.cuh).  Two tensors are
// read and one is written, each once: the floor is HBM's.  A block's tile is 128 tokens x 32
// channels: copies bring the tiles ahead into shared memory while a lane keeps the decays and
// inputs of its run in registers, from the run's own pair to the second pass over it.
//
// Measured (2048 channels, bf16): 8 x 4096 tokens 93 to 95 us, 4.3 TB/s, 64% of a copy's rate; one
// sequence of 262144 tokens 777 us, 62%.  fp32, 8 x 2048: 74 us, 82%.  What bounds the bf16 calls is
// the arithmetic in its order: 29 instructions an element (14 of them the gate's), four warps to a
// scheduler since 16 tokens' decays and inputs of two channels take 64 registers, and the steps
// of a tile (its copy, the gates, two exchanges, the second pass) one after the other; issue slots
// 61% taken.  Runs of 8 tokens with more blocks on an SM: 128 to 150 us (the exchanges weigh twice).
#include <algorithm>

#include "gdr_scan.cuh"

namespace gdr {
namespace {

using namespace scan;

constexpr int kL = 16;                           // tokens of a lane's run
constexpr int kWarps = 4;
constexpr int kTok = 2 * kL * kWarps;            // of a block's tile; divides 128, or 128 it
constexpr int kThreads = 32 * kWarps;
template <typename T> constexpr int kBlocksPerSm = sizeof(T) == 2 ? 4 : 3;
constexpr int kDepth = 2;   // tiles in shared memory (three: the same time)
template <typename T, bool BOXES> using FwdRing = Ring<T, kL, kTok, 2, kDepth, BOXES>;

struct FwdMaps {
    CUtensorMap x, a;
};

template <typename T, int GATE, int SRC, bool BOXES>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<T>)
scan_fwd_kernel(const __grid_constant__ ScanShape s, const __grid_constant__ FwdMaps maps, const T *x, const T *a, const float *h0, T *out, float *hT,
                float *states, int pairs, uint64_t limit_ns, int *status) {
    constexpr bool kFine = sizeof(T) == 4;
    extern __shared__ char smem[];
    __shared__ __align__(16) float4 agg[2][kWarps][16];
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
    if (s.cu && hT && hT != h0 && c0 + lane < D)   // sequences of no tokens
        for (int n = first + warp + rank * kWarps; n < last; n += kWarps * CS)
            if (seq_start(s, n) == seq_start(s, n + 1))
                hT[(int64_t)n * D + c0 + lane] = h0 ? h0[(int64_t)n * D + c0 + lane] : 0.f;
    const int t0 = p0 / kTok, t1 = (p1 + kTok - 1) / kTok, steps = (t1 - t0 + CS - 1) / CS;
    const bool many = last - first > 1;
    FwdRing<T, BOXES> ring((char *)(((uintptr_t)smem + 127) & ~(uintptr_t)127), full);
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
    const CUtensorMap *const map[2] = {&maps.x, &maps.a};
    const T *const src[2] = {x, a};
    auto ask = [&](int i, int slot) {   // the tile of step i
        const int tile = t0 + i * CS + rank;
        if (tile < t1) ring.ask(slot, i, map, src, tile * kTok, p0, p1, c0, D);
        ring.close();
    };
    for (int i = 0; i < kDepth; ++i) ask(i, i);
    Peers peers{told, bars, limit_ns};
    Cursor cur{first, 0, -1};
    float2 carry = both(0.f);
    bool lost = false;   // a wait ran out: the results are lost, but every block goes through its steps
    // of the lane's run in the output's tile, in bytes
    const unsigned lane_out = ((unsigned)run_at0 * (unsigned)D + (unsigned)c) * (unsigned)sizeof(T);
    for (int i = 0, slot = 0, use = 0; i < steps; ++i) {
        if (CS > 1 && threadIdx.x == 0 && !lost) peers.expect(i, CS);
        const int base = (t0 + i * CS + rank) * kTok;   // may lie behind the part
        const bool there = base < p1;
        // a tile that one sequence fills, and goes beyond on both sides
        bool inner = false;
        if (there) {
            cur.seek(s, first, last, max(base, p0));
            inner = cur.from < base && cur.to > base + kTok;
            if (!lost) lost = !__all_sync(kFull, ring.wait(slot, use, limit_ns));
            if constexpr (ring.kMode == kRows) ring.move(slot, src, base, c0, D);
        }
        const bool cuts = CS == 1 ? there && !inner : many || i == 0;
        T *tx = ring.run(slot, 0, run_at0, l), *ta = ring.run(slot, 1, run_at0, l);
        const int p = min(base, p1) + run_at0, lo = max(p, p0), hi = min(p + kL, p1);
        float2 al[kL], u[kL];
        Run run{both(1.f), both(0.f)};
        Cursor mine = cur;
        Marks m{0, 0};
        bool at_start = false;   // a sequence starts with the run, and none within it
        float2 start = both(0.f);
        if (there) {
            if (!inner) {
                m = marks_of(s, mine, first, last, p, lo, hi);
                at_start = m.first == 1;
                if (hi - lo < kL) {
                    blank<T, kL>(tx, 0.f, p, lo, hi);
                    blank<T, kL>(ta, -INFINITY, p, lo, hi);
                    sm100::fence_proxy_async_smem();   // before the slot is filled again
                }
            }
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                const Gate g = gate_of<kFine, GATE, SRC, false>(read2(ta, j), s);
                const float2 xv = read2(tx, j);
                al[j] = g.alpha;
                u[j] = SRC == GDR_SOURCE_PLAIN ? xv : mul2(g.w, xv);
            }
            if (at_start) run.B = start = load_state(h0, mine.n, D, c);
            if (!(m.first & ~1u)) {
#pragma unroll
                for (int j = 0; j < kL; ++j) {
                    run.B = fma2(al[j], run.B, u[j]);
                    run.A = mul2(run.A, al[j]);
                }
                if (at_start) run.A = both(-1.f);
            } else {
                int n = mine.n;
#pragma unroll
                for (int j = 0; j < kL; ++j)
                    if (m.first >> j & 1) {
                        n = seq_from(s, n, p + j);
                        u[j] = fma2(al[j], load_state(h0, n, D, c), u[j]);
                        run = Run{both(-1.f), u[j]};
                    } else {
                        run.B = fma2(al[j], run.B, u[j]);
                        decay_past_cut(run.A, al[j]);
                    }
            }
        }
        float2 h;   // the state that enters the run
        auto chain = [&](auto cuts) {
            // the other half's run: the second half's lanes go through the first half's
            const Run other{other_half(run.A), other_half(run.B)};
            if (half == 0) agg[i & 1][warp][l] = pack(follow(run, other, cuts));
            __syncthreads();
            if (!lost) ask(i + kDepth, slot);
            if (CS == 1) {
                float2 e = carry;
                h = e;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    if (w == warp) h = e;
                    e = through(unpack(agg[i & 1][w][l]), e, cuts);
                }
                carry = e;
            } else {
                Run front{both(1.f), both(0.f)}, all = front;   // the warps in front, and all
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    if (w == warp) front = all;
                    all = follow(all, unpack(agg[i & 1][w][l]), cuts);
                }
                if (!lost)
                    for (int r = 2 * warp + half; r < CS; r += 2 * kWarps) peers.tell(i, r, rank, l, pack(all));
                if (!lost) lost = !__all_sync(kFull, peers.wait(i));
                float2 e = carry;
                h = e;
                for (int r = 0; r < CS; ++r) {
                    if (r == rank) h = e;
                    e = through(unpack(told[i & 1][r][l]), e, cuts);
                }
                carry = e;
                h = through(front, h, cuts);
            }
            if (half) h = through(other, h, cuts);
        };
        if (cuts)
            chain(std::true_type{});
        else
            chain(std::false_type{});
        if (at_start) h = start;
        if (there && c < D && pairs && hi - lo == kL && !(m.first & ~1u) && !(hT && (m.last & ~(1u << (kL - 1))))) {
            if (out) {
                char *o = (char *)(out + (int64_t)base * D) + lane_out;
#pragma unroll
                for (int j = 0; j < kL; ++j) {
                    h = fma2(al[j], h, u[j]);
                    write2((T *)o, h);
                    o += D * (int)sizeof(T);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kL; ++j) h = fma2(al[j], h, u[j]);
            }
            if (hT && m.last) store_state(hT, seq_from(s, mine.n, p + kL - 1), D, c, h);
        } else if (there && c < D) {
            int n = mine.n;
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                h = !at_start && (m.first >> j & 1) ? u[j] : fma2(al[j], h, u[j]);
                const int t = p + j;
                if (t < lo || t >= hi) continue;
                if (out) {
                    T *o = out + (int64_t)t * D + c;
                    if (pairs) {
                        write2(o, h);
                    } else {
                        o[0] = from_f32<T>(h.x);
                        if (c + 1 < D) o[1] = from_f32<T>(h.y);
                    }
                }
                if (hT && (m.last >> j & 1)) {
                    n = seq_from(s, n, t);
                    store_state(hT, n, D, c, h);
                }
            }
        }
        // the state behind 128 tokens
        if (states && there && hi == p + kL && hi % kScanTile == 0)
            store_state(states, hi / kScanTile - 1, D, c, h);
        if (++slot == kDepth) {
            slot = 0;
            ++use;
        }
    }
    ring.drain(lost);
    peers.leave(lost, CS, status);
}

template <typename T, int GATE, int SRC>
cudaError_t launch_fwd_t(const ScanFwd &t, ScanShape s, int sms, int *status, cudaStream_t stream) {
    FwdMaps maps{};
    constexpr gdr_dtype_t kType = sizeof(T) == 2 ? GDR_BF16 : GDR_F32;
    auto plane = [&](CUtensorMap *m, const void *p) {
        return tc_make_plane_map(m, p, kType, s.D, s.total, kScanChannels, kTok);
    };
    const bool boxes = s.total > 0 && plane(&maps.x, t.x) && plane(&maps.a, t.a);
    const int pairs = s.D % 2 == 0 && (uintptr_t)t.out % (2 * sizeof(T)) == 0;
    auto run = [&](auto by_boxes, ScanRoom &known) {
        constexpr bool kB = by_boxes();
        const int smem = FwdRing<T, kB>::kBytes + 128;
        return scan_launch(scan_fwd_kernel<T, GATE, SRC, kB>, s, kThreads, smem, kTok, sms, known, "scan_fwd_kernel", stream, maps,
                       (const T *)t.x, (const T *)t.a, t.h0, (T *)t.out, t.hT, t.states, pairs, scan_wait_ns(), status);
    };
    static ScanRoom boxed, other;
    return boxes ? run(std::true_type{}, boxed) : run(std::false_type{}, other);
}

// One (sequence, channel) to a thread, the next token's inputs on their way while a token is
// computed.  Bound by the launch for a few sequences, by HBM beyond: the states, then the tokens.
template <typename T, int GATE, int SRC>
__global__ void __launch_bounds__(256)
scan_step_kernel(const T *__restrict__ x, const T *__restrict__ a, float *__restrict__ state, T *__restrict__ out,
                 int64_t units, const ScanShape s) {
    const int T_ = s.T_per, D = s.D;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= units) return;
    const int64_t n = i / D, at = n * T_ * D + (i - n * D);
    float h = state[i];
    T xv = x[at], av = a[at];
    for (int t = 0; t < T_; ++t) {
        const int64_t next = at + (int64_t)(t + 1 < T_ ? t + 1 : t) * D;
        const T xn = x[next], an = a[next];
        const Gate g = gate_of<sizeof(T) == 4, GATE, SRC, false>(both(to_f32(av)), s);
        h = fmaf(g.alpha.x, h, g.w.x * to_f32(xv));
        out[at + (int64_t)t * D] = from_f32<T>(h);
        xv = xn;
        av = an;
    }
    state[i] = h;
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanFwd &t, ScanShape s, gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source,
                            int sms, int *status, cudaStream_t stream) {
    return with_form(s, dtype, gate, source, [&](auto type, auto g, auto w) {
        return launch_fwd_t<decltype(type), g(), w()>(t, s, sms, status, stream);
    });
}

cudaError_t launch_scan_step(const void *x, const void *a, float *state, void *out, ScanShape s, gdr_dtype_t dtype,
                             gdr_gate_t gate, gdr_source_t source, cudaStream_t stream) {
    return with_form(s, dtype, gate, source, [&](auto type, auto g, auto w) {
        using T = decltype(type);
        const int64_t units = (int64_t)s.N * s.D;
        ProfScope prof(stream, "scan_step_kernel");
        scan_step_kernel<T, g(), w()><<<(unsigned)((units + 255) / 256), 256, 0, stream>>>((const T *)x, (const T *)a, state,
                                                                                         (T *)out, units, s);
        count_launch();
        return cudaGetLastError();
    });
}

}  // namespace gdr
