// gdr_decay_tc.cu -- linear attention with one constant decay per head on the
// 5th-generation tensor cores (tcgen05): bf16 tensors, widths 64 and 128.
//
// A pass (gdr_decay.cuh) takes tiles of C = 128 tokens of one (segment, head) in order.
// With rows a_i, b_i, c_i of the tile, S the state that enters it, lam = exp(log_decay) and
// n tokens in the tile (n = C but at a sequence's end):
//     f_i   = max(lam^{i+1}, 2^-64)
//     P_ij  = s_upd lam^{i-j} / f_i (a_i . b_j)  for j <= i, else 0
//     out_i = s_out f_i (S^T a_i + sum_j P_ij c_j)
//     S    <- lam^n S + sum_j (s_upd lam^{n-1-j} c_j) b_j^T  (transposed)
// and for a reversed pass i - j -> j - i, j <= i -> j >= i, lam^{i+1} -> lam^{n-1-i} and
// lam^{n-1-j} -> lam^{j+1}.  Dividing P by the factor of the state's part lets both parts sum in
// one accumulator; the floor of f keeps P in range for any decay, and what it adds is the
// state's part taken at 2^-64 where lam^{i+1} is below that.  All four products run on the tensor cores with fp32 accumulators in the tensor
// memory (TMEM), 128 x 128 each:
//     Sc = A B^T                     lanes = query tokens i
//     S^T <- lam^n S^T + C'^T B      lanes = value index e: the resident state
//     O  = A S                       lanes = query tokens i; S from shared memory in bf16
//     O  += P C                      P in TMEM in bf16
// in this order.  A tile of one head is 128 KB of HBM traffic (3 loads, 1 store; 2.9 us of an
// SM's share of the measured bandwidth) and 25 MFLOP (2.0 us of an SM's share of the bf16
// rate), so the pass can be bound by HBM if its other work stays out of the way.  The stages
// of a tile run in different warps and overlap those of its neighbours:
//   warps 0-3    Sc -> P (bf16, over Sc in TMEM); O -> out
//   warps 4-7    S^T -> bf16 (shared memory) and lam^n S^T (TMEM)
//   warps 8-11   C' = weighted C -> TMEM, 32 tokens at a time
//   warp 12      TMA loads of A, B, C, two stages of 96 KB
//   warp 13      issues every MMA (their order in the tensor pipe is the issue order)
//
// Rounding.  The state is fp32 and so are its updates: C' = s_upd lam^{..} C has 24
// significant bits, so it goes in as the sum of three bf16 numbers that represent it exactly
// (three products instead of one; two would leave 2^-17 in hT and dh0).  P and the state
// as a factor of O are rounded to bf16: each adds an error of at most 2^-9 of its part of
// an output that is itself rounded to bf16.
//
// A block is persistent: it walks the units (segment, head, pass) with a stride of the grid
// and its pipeline runs on across them.  The three passes of a backward call are
// neighbouring units, so that what they share is read from the L2 by all but the first.
// Every wait is bounded; one that runs out sets the status word and the block unwinds.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdlib>

#include "gdr_decay.cuh"
#include "gdr_sm100.cuh"
#include "gdr_tc.cuh"

namespace gdr {

GDR_DEBUG_TU()

namespace {

using namespace sm100;

constexpr int kC = kDecayTile;
constexpr int kMaxPasses = 3;
constexpr uint32_t kBox = kC * 128;        // 64 columns x 128 tokens, 128-byte rows, swizzled
constexpr uint32_t kTile = 2 * kBox;       // one tensor's tile: up to two boxes
constexpr unsigned kFull = 0xffffffffu;
constexpr uint64_t kWaitNs = 2000000000ull;   // pipeline wait limit: 2 s
constexpr uint64_t kDrainNs = 2000000000ull;  // drains before exit

struct TcMaps {
    CUtensorMap a[kMaxPasses], b[kMaxPasses], c[kMaxPasses];
};
struct TcArgs {
    DecayGeom g;
    DecayPass pass[kMaxPasses];
    int npass;
    int64_t units;      // max_segs * H * npass
    int *status;
    uint64_t wait_ns;
};

// One unit of a block's walk.
struct Unit {
    int pass, h;
    DecaySeg seg;
    int64_t t0, t1;   // tokens it runs (a local pass: those that reach the segment's end)
    int tiles;
};

// False where unit u has nothing to do.
__device__ __forceinline__ bool unit_of(const TcArgs &A, int64_t u, bool local, Unit &o) {
    o.pass = (int)(u % A.npass);
    const int64_t sh = u / A.npass;
    o.h = (int)(sh % A.g.H);
    if (!decay_segment(A.g, sh / A.g.H, o.seg)) return false;
    const bool rev = A.pass[o.pass].rev;
    o.t0 = o.seg.t0;
    o.t1 = o.seg.t1;
    if (local) {
        if (rev ? o.seg.first : o.seg.last) return false;   // no boundary behind it
        // whole tiles: the segment is one (reversed: but for its sequence's last tile)
        const int64_t reach = (decay_reach(decay_log(A.g.log_decay, o.h), o.t1 - o.t0) + kC - 1) / kC * kC;
        if (rev) o.t1 = min(o.t1, o.t0 + reach); else o.t0 = max(o.t0, o.t1 - reach);
    }
    o.tiles = (int)((o.t1 - o.t0 + kC - 1) / kC);
    return GDR_INBOUNDS(o.seg.t0 >= 0 && o.seg.t1 <= A.g.T_total && o.seg.slot <= A.g.max_slots);
}
// Tile i of a unit in the order of its pass: first token and number of tokens.
__device__ __forceinline__ void tile_of(const Unit &u, bool rev, int i, int64_t &t, int &n) {
    const int64_t at = rev ? u.tiles - 1 - i : i;
    t = u.t0 + at * kC;
    n = (int)min((int64_t)kC, u.t1 - t);
}

__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *map, int width, int h, int64_t t,
                                          uint64_t *bar) {
    tma_load_3d(dst, map, 0, h, (int)t, bar);
    if (width > 64) tma_load_3d(dst + kBox, map, 64, h, (int)t, bar);
}

// Zeroes the rows from n on of a tile in shared memory: tokens past the sequence's end,
// which are another sequence's (one warp; made visible to the tensor cores).
__device__ __forceinline__ void zero_rows(uint8_t *tile, int width, int n, int lane) {
    for (int box = 0; box < width / 64; ++box)
        for (int i = lane; i < (kC - n) * 8; i += 32)
            *(uint4 *)(tile + box * kBox + sw128_off(n + i / 8, (i & 7) * 16)) = make_uint4(0, 0, 0, 0);
}

// The weights of a tile's tokens in the update of the state, for one warp: token i has
// s_upd lam^{len - 1 - i + past} (forward) or s_upd lam^{i + 1 + past}; rows from len on are
// not the sequence's and have 0.
__device__ __forceinline__ void tile_weights(float *w, int len, bool rev, float gd, float s_upd, int64_t past,
                                             int lane) {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kC / 32; ++k) {
        const int i = lane + 32 * k;
        w[i] = i < len ? s_upd * expf(gd * (float)(past + (rev ? i + 1 : len - 1 - i))) : 0.f;
    }
    __syncwarp();
}

// Zeroes the rows from n on of the 32 columns from e0 (one warp) of a tile: what a weight
// of 0 would not silence.
__device__ __forceinline__ void zero_columns(uint8_t *tile, int e0, int n, int lane) {
    for (int i = lane; i < (kC - n) * 4; i += 32)
        *(uint4 *)(tile + (e0 >> 6) * kBox + sw128_off(n + i / 4, (e0 & 63) * 2 + (i & 3) * 16)) =
            make_uint4(0, 0, 0, 0);
}

// Quarter q (32 tokens) of a tile's C'^T, row e, into three times 16 TMEM columns at `at`
// (a whole warp): the weighted values x w as the bf16 terms hi + mid + lo = x w exactly, cut
// off the top of the fp32 product 8 significant bits at a time; a column holds two tokens.
__device__ __forceinline__ void write_terms(uint32_t at, const uint8_t *tile, int e, bool any, int q,
                                            const float *w) {
    uint32_t hi[16], mid[16], lo[16];
    if (any) {
        const uint8_t *col = tile + (e >> 6) * kBox + (e & 7) * 2 + q * 4096;
        const uint32_t chunk = (e & 63) >> 3;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float4 w4 = *(const float4 *)&w[32 * q + 2 * i];
            const float wv[4] = {w4.x, w4.y, w4.z, w4.w};
            float y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = 2 * i + k;
                const uint32_t x = *(const uint16_t *)(col + (r >> 3) * 1024 + (r & 7) * 128 + ((chunk ^ (r & 7)) << 4));
                y[k] = __uint_as_float(x << 16) * wv[k];
            }
            hi[i] = __byte_perm(__float_as_uint(y[0]), __float_as_uint(y[1]), 0x7632);
            hi[i + 1] = __byte_perm(__float_as_uint(y[2]), __float_as_uint(y[3]), 0x7632);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] -= __uint_as_float(__float_as_uint(y[k]) & 0xffff0000u);
            mid[i] = __byte_perm(__float_as_uint(y[0]), __float_as_uint(y[1]), 0x7632);
            mid[i + 1] = __byte_perm(__float_as_uint(y[2]), __float_as_uint(y[3]), 0x7632);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] -= __uint_as_float(__float_as_uint(y[k]) & 0xffff0000u);
            lo[i] = __byte_perm(__float_as_uint(y[0]), __float_as_uint(y[1]), 0x7632);
            lo[i + 1] = __byte_perm(__float_as_uint(y[2]), __float_as_uint(y[3]), 0x7632);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) hi[j] = mid[j] = lo[j] = 0;
    }
    __syncwarp();
    tmem_st16(at, hi);
    tmem_st16(at + 16, mid);
    tmem_st16(at + 32, lo);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t *)&v;
}

// 16 columns (d0 ..) of row e of a state in memory.
__device__ __forceinline__ void state_load(const DecayPass &p, const float *in, int d0, int e, uint32_t (&r)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) r[j] = 0;
    if (!in || e >= p.vd || d0 >= p.kd) return;
    if (p.transposed) {
#pragma unroll
        for (int j = 0; j < 16; j += 4) *(uint4 *)&r[j] = *(const uint4 *)&in[(int64_t)e * p.kd + d0 + j];
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(in[(int64_t)(d0 + j) * p.vd + e]);
    }
}
__device__ __forceinline__ void state_store(const DecayPass &p, float *to, int d0, int e, const uint32_t (&r)[16]) {
    if (!to || e >= p.vd || d0 >= p.kd) return;
    if (p.transposed) {
#pragma unroll
        for (int j = 0; j < 16; j += 4) *(uint4 *)&to[(int64_t)e * p.kd + d0 + j] = *(const uint4 *)&r[j];
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) to[(int64_t)(d0 + j) * p.vd + e] = __uint_as_float(r[j]);
    }
}

// Waits for the warp's TMEM loads; names the registers of one of them, so that no use of
// those moves above the wait.
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
// f(m, r) for 16 columns at a time from `at`, the next ones on their way meanwhile (an even
// number of pieces).  Rolled up: the warps of a block run five different programs, and
// their loops have to stay in the instruction caches together.
template <typename F> __device__ __forceinline__ void tmem_columns(uint32_t at, int pieces, F &&f) {
    uint32_t r0[16], r1[16];
    tmem_ld16(at, r0);
#pragma unroll 1
    for (int m = 0; m < pieces; m += 2) {
        tmem_arrived(r0);
        tmem_ld16(at + 16 * (m + 1), r1);
        f(m, r0);
        tmem_arrived(r1);
        if (m + 2 < pieces) tmem_ld16(at + 16 * (m + 2), r0);
        f(m + 1, r1);
    }
}

// ---------------------------------------------------------------------------
// the output pass
// ---------------------------------------------------------------------------
constexpr int kOutThreads = 32 * 14, kOutProducer = 12, kOutIssuer = 13;   // warps
// TMEM columns
constexpr uint32_t kColS = 0;      // Sc, then P in its first 64 columns
constexpr uint32_t kColO = 128;
constexpr uint32_t kColH = 256;    // S^T
constexpr uint32_t kColV = 384;    // C'^T: two slots of 32 tokens x 3 terms
constexpr uint32_t kSlotCols = 48;
constexpr uint32_t kTmemCols = 512;
// shared memory
constexpr uint32_t kStage = 3 * kTile;               // A, B, C
constexpr uint32_t kOffH = 2 * kStage;               // the state in bf16, [e][d], K-major
constexpr uint32_t kOffBar = kOffH + kTile;
constexpr uint32_t kOffW = kOffBar + 256;            // weights of a tile's tokens, a copy per warp
constexpr uint32_t kSmemOut = kOffW + 4 * kC * 4;
static_assert(kSmemOut <= 232448, "shared memory");

struct OutBars {
    uint64_t full[2];      // a stage's tiles have arrived
    uint64_t free_a[2];    // the stage's A is read
    uint64_t free_bc[2];   // ... its B and C
    uint64_t s_full;       // Sc complete
    uint64_t p_ready;      // P written, O scaled (4 warps)
    uint64_t o1_full;      // O = A S complete (the bf16 state is read)
    uint64_t o_full;       // O complete
    uint64_t o_free;       // O read (4 warps)
    uint64_t h_ready;      // the bf16 state written, S^T scaled (4 warps)
    uint64_t v_ready[2];   // a slot of C' written (4 warps)
    uint64_t v_free[2];    // ... read
    uint64_t kv_full;      // the tile's update of S^T complete
    uint64_t fin;          // every MMA of the block complete
    uint32_t tmem;
    int stop;
};
static_assert(sizeof(OutBars) <= 256, "barriers");

__global__ void __launch_bounds__(kOutThreads, 1)
decay_out_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs A) {
    extern __shared__ __align__(1024) uint8_t smem[];
    OutBars &bar = *(OutBars *)(smem + kOffBar);
    volatile int *stop = &bar.stop;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = A.g.H;
    if (!GDR_INBOUNDS((smem_u32(smem) & 1023u) == 0)) return;   // swizzled tiles start on 1 KB

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.free_a[i], 1);
            mbar_init(&bar.free_bc[i], 1);
            mbar_init(&bar.v_ready[i], 4);
            mbar_init(&bar.v_free[i], 1);
        }
        mbar_init(&bar.s_full, 1);
        mbar_init(&bar.p_ready, 4);
        mbar_init(&bar.o1_full, 1);
        mbar_init(&bar.o_full, 1);
        mbar_init(&bar.o_free, 4);
        mbar_init(&bar.h_ready, 4);
        mbar_init(&bar.kv_full, 1);
        mbar_init(&bar.fin, 1);
        *stop = 0;
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == 0) {
        tmem_alloc(&bar.tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = bar.tmem;

    // Waits (whole warp) until `b` has completed its use number `use` (from 0); false once
    // any wait of the block has run out.
    auto wait = [&](uint64_t *b, uint32_t use) {
        if (__all_sync(kFull, mbar_wait(b, use & 1u, A.wait_ns)) && !*stop) return true;
        if (lane == 0 && !*stop) set_status(A.status, GDR_ERR_TIMEOUT);
        *stop = 1;
        return false;
    };
    uint32_t it = 0;   // tiles so far: the use number of every once-a-tile barrier
    Unit u;

    if (warp == kOutProducer) {
        bool ok = true;
        for (int64_t n = blockIdx.x; n < A.units && ok; n += gridDim.x) {
            if (!unit_of(A, n, false, u)) continue;
            const DecayPass &p = A.pass[u.pass];
            for (int i = 0; i < u.tiles; ++i, ++it) {
                const uint32_t st = it & 1;
                if (it >= 2 && !((ok = wait(&bar.free_a[st], (it >> 1) - 1)) && (ok = wait(&bar.free_bc[st], (it >> 1) - 1))))
                    break;
                if (lane == 0) {
                    int64_t t;
                    int len;
                    tile_of(u, p.rev, i, t, len);
                    uint8_t *s = smem + st * kStage;
                    mbar_arrive_expect_tx(&bar.full[st], (2 * p.kd + p.vd) / 64 * kBox);
                    load_tile(s, &maps.a[u.pass], p.kd, u.h, t, &bar.full[st]);
                    load_tile(s + kTile, &maps.b[u.pass], p.kd, u.h, t, &bar.full[st]);
                    load_tile(s + 2 * kTile, &maps.c[u.pass], p.vd, u.h, t, &bar.full[st]);
                }
                __syncwarp();
            }
        }
        // never leave with a copy in flight
        for (uint32_t k = it >= 2 ? it - 2 : 0; k < it; ++k)
            __all_sync(kFull, mbar_wait(&bar.full[k & 1], (k >> 1) & 1u, kDrainNs));
    } else if (warp == kOutIssuer) {
        const uint32_t s0 = smem_u32(smem);
        bool ok = true;
        for (int64_t n = blockIdx.x; n < A.units && ok; n += gridDim.x) {
            if (!unit_of(A, n, false, u)) continue;
            const DecayPass &p = A.pass[u.pass];
            const uint32_t id_s = instr_desc(kC, kC, 1, false, false);
            const uint32_t id_o1 = instr_desc(kC, p.vd, 1, false, false);
            const uint32_t id_o2 = instr_desc(kC, p.vd, 1, false, true);
            const uint32_t id_h = instr_desc(kC, p.kd, 1, false, true);
            for (int i = 0; i < u.tiles; ++i, ++it) {
                const uint32_t st = it & 1;
                int64_t t;
                int len;
                tile_of(u, p.rev, i, t, len);
                uint8_t *sp = smem + st * kStage;
                const uint32_t sa = s0 + st * kStage, sb = sa + kTile, sc = sb + kTile;
                if (!(ok = wait(&bar.full[st], it >> 1))) break;
                if (len < kC) {
                    zero_rows(sp + kTile, p.kd, len, lane);   // of C: by the warps that weigh it
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                tc_fence_after();
                const uint64_t dA = smem_desc(sa, 16, 1024, kSw128), dB = smem_desc(sb, 16, 1024, kSw128);
                const uint64_t dBt = smem_desc(sb, kBox, 1024, kSw128), dCt = smem_desc(sc, kBox, 1024, kSw128);
                const uint64_t dH = smem_desc(s0 + kOffH, 16, 1024, kSw128);
                // the previous tile's P is read: its product precedes this one in the pipe
                if (elect_one()) {
                    for (int k = 0; k < p.kd / 16; ++k) {
                        const uint64_t o = ((k >> 2) * kBox + (k & 3) * 32) >> 4;
                        mma_f16_ss(tm + kColS, dA + o, dB + o, id_s, k > 0);
                    }
                    mma_commit(&bar.s_full);
                }
                __syncwarp();
                if (!(ok = wait(&bar.h_ready, it))) break;
                for (int q = 0; q < 4 && ok; ++q) {
                    const uint32_t slot = q & 1;
                    if (!(ok = wait(&bar.v_ready[slot], 2 * it + (q >> 1)))) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int term = 0; term < 3; ++term)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                mma_f16_ts(tm + kColH, tm + kColV + slot * kSlotCols + term * 16 + k * 8,
                                           dBt + (((q * 2 + k) * 2048) >> 4), id_h, 1);
                        mma_commit(&bar.v_free[slot]);
                        if (q == 3) mma_commit(&bar.kv_full);
                    }
                    __syncwarp();
                }
                if (!ok || (it && !(ok = wait(&bar.o_free, it - 1)))) break;
                tc_fence_after();
                if (elect_one()) {
                    for (int k = 0; k < p.kd / 16; ++k) {
                        const uint64_t o = ((k >> 2) * kBox + (k & 3) * 32) >> 4;
                        mma_f16_ss(tm + kColO, dA + o, dH + o, id_o1, k > 0);
                    }
                    mma_commit(&bar.o1_full);
                    mma_commit(&bar.free_a[st]);
                }
                __syncwarp();
                if (!(ok = wait(&bar.p_ready, it))) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k)
                        mma_f16_ts(tm + kColO, tm + kColS + k * 8, dCt + ((k * 2048) >> 4), id_o2, 1);
                    mma_commit(&bar.o_full);
                    mma_commit(&bar.free_bc[st]);
                }
                __syncwarp();
            }
        }
        // no tensor-core operation may still run when the TMEM is released
        if (elect_one()) mma_commit(&bar.fin);
        __syncwarp();
        __all_sync(kFull, mbar_wait(&bar.fin, 0, kDrainNs));
    } else if (warp < 4) {
        // ---- weights and outputs: thread = token row of the tile
        const int row = tid;
        const uint32_t lanes = tm + ((uint32_t)(warp * 32) << 16);
        bool ok = true;
        for (int64_t n = blockIdx.x; n < A.units && ok; n += gridDim.x) {
            if (!unit_of(A, n, false, u)) continue;
            const DecayPass &p = A.pass[u.pass];
            const bool rev = p.rev;
            // log2 lam; below -200 (lam / f < 2^-136) a weight is 0 whatever lam is, and the
            // differences of its multiples below stay exact enough
            const float g2 = fmaxf(decay_log(A.g.log_decay, u.h) * 1.4426950408889634f, -200.f);
            const float l_upd = p.s_upd;
            for (int i = 0; i < u.tiles; ++i, ++it) {
                int64_t t;
                int len;
                tile_of(u, rev, i, t, len);
                // log2 of the row's f
                const float lf = fmaxf(g2 * (float)(rev ? max(len - 1 - row, 0) : row + 1), -64.f);
                if (!(ok = wait(&bar.s_full, it))) break;
                tc_fence_after();
                tmem_columns(lanes + kColS, 8, [&](int m, const uint32_t (&x)[16]) {
                    uint32_t o[8];
                    if (rev ? 16 * m + 15 < 32 * warp : 16 * m > 32 * warp + 31) {   // no pair of the warp's rows
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] = 0;
                    } else {
                        // distance of column 16 m + j: d + j step
                        const int d = rev ? 16 * m - row : row - 16 * m, step = rev ? 1 : -1;
                        const float l0 = fmaf(g2, (float)d, -lf), l1 = rev ? g2 : -g2;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float y[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                y[k] = d + (2 * j + k) * step >= 0
                                           ? l_upd * __uint_as_float(x[2 * j + k]) * exp2_approx(fmaf((float)(2 * j + k), l1, l0))
                                           : 0.f;
                            o[j] = pack2(y[0], y[1]);
                        }
                    }
                    tmem_st8(lanes + kColS + 8 * m, o);
                });
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_ready);
                if (!(ok = wait(&bar.o_full, it))) break;
                tc_fence_after();
                const float f = p.s_out * exp2f(lf);
                __nv_bfloat16 *dst = (__nv_bfloat16 *)p.out + ((t + row) * H + u.h) * (int64_t)p.vd;
                tmem_columns(lanes + kColO, p.vd / 16, [&](int m, const uint32_t (&x)[16]) {
                    if (row < len) {
#pragma unroll
                        for (int j = 0; j < 16; j += 8) {
                            uint32_t o[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                o[k] = pack2(f * __uint_as_float(x[j + 2 * k]), f * __uint_as_float(x[j + 2 * k + 1]));
                            *(uint4 *)(dst + 16 * m + j) = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                    __syncwarp();
                });
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.o_free);
            }
        }
    } else if (warp < 8) {
        // ---- state: thread = value index (TMEM lane)
        const int e = tid - 128;
        const uint32_t lanes = tm + ((uint32_t)((warp - 4) * 32) << 16);
        bool ok = true;
        for (int64_t n = blockIdx.x; n < A.units && ok; n += gridDim.x) {
            if (!unit_of(A, n, false, u)) continue;
            const DecayPass &p = A.pass[u.pass];
            const float gd = decay_log(A.g.log_decay, u.h);
            const float *in = decay_state_in(p, u.seg, H, u.h);
            float *to = decay_state_out(p, u.seg, H, u.h);
            if (u.tiles == 0) {   // an empty sequence: the state goes through
                for (int d0 = 0; d0 < p.kd; d0 += 16) {
                    uint32_t r[16];
                    state_load(p, in, d0, e, r);
                    state_store(p, to, d0, e, r);
                }
                continue;
            }
            for (int i = 0; i < u.tiles; ++i, ++it) {
                int64_t t;
                int len;
                tile_of(u, p.rev, i, t, len);
                const DecayFactor decay(gd * (float)len);
                // 16 columns of the entering state: to shared memory in bf16, and decayed
                auto take = [&](int m, uint32_t (&r)[16]) {
#pragma unroll
                    for (int j = 0; j < 16; j += 8) {
                        uint32_t o[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            o[k] = pack2(__uint_as_float(r[j + 2 * k]), __uint_as_float(r[j + 2 * k + 1]));
                        *(uint4 *)(smem + kOffH + (m >> 2) * kBox + sw128_off(e, (16 * (m & 3) + j) * 2)) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(decay(__uint_as_float(r[j])));
                    tmem_st16(lanes + kColH + 16 * m, r);
                };
                // the update of S^T is complete, and the bf16 state read
                if (it && !((ok = wait(&bar.kv_full, it - 1)) && (ok = wait(&bar.o1_full, it - 1)))) break;
                tc_fence_after();
                if (i == 0) {
#pragma unroll 1
                    for (int m = 0; m < p.kd / 16; ++m) {
                        uint32_t r[16];
                        state_load(p, in, 16 * m, e, r);
                        __syncwarp();
                        take(m, r);
                    }
                } else {
                    tmem_columns(lanes + kColH, p.kd / 16, take);
                }
                fence_proxy_async_smem();
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.h_ready);
            }
            if (ok && to) {
                if (!(ok = wait(&bar.kv_full, it - 1))) break;
                tc_fence_after();
                tmem_columns(lanes + kColH, p.kd / 16, [&](int m, const uint32_t (&r)[16]) {
                    state_store(p, to, 16 * m, e, r);
                    __syncwarp();
                });
            }
        }
    } else {
        // ---- weighted values: thread = value index (TMEM lane)
        const int e = tid - 256;
        const uint32_t lanes = tm + ((uint32_t)((warp - 8) * 32) << 16);
        float *w = (float *)(smem + kOffW) + (warp - 8) * kC;
        bool ok = true;
        for (int64_t n = blockIdx.x; n < A.units && ok; n += gridDim.x) {
            if (!unit_of(A, n, false, u)) continue;
            const DecayPass &p = A.pass[u.pass];
            const float gd = decay_log(A.g.log_decay, u.h);
            int wlen = -1;   // tokens of the tile that w is for
            for (int i = 0; i < u.tiles; ++i, ++it) {
                const uint32_t st = it & 1;
                int64_t t;
                int len;
                tile_of(u, p.rev, i, t, len);
                if (len != wlen) tile_weights(w, len, p.rev, gd, p.s_upd, 0, lane);
                wlen = len;
                if (!(ok = wait(&bar.full[st], it >> 1))) break;
                uint8_t *ct = smem + st * kStage + 2 * kTile;
                if (len < kC && e < p.vd) {
                    zero_columns(ct, e & ~31, len, lane);
                    fence_proxy_async_smem();   // the product with P reads them too
                    __syncwarp();
                }
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    const uint32_t slot = q & 1, use = 2 * it + (q >> 1);
                    if (use && !(ok = wait(&bar.v_free[slot], use - 1))) break;
                    tc_fence_after();
                    write_terms(lanes + kColV + slot * kSlotCols, ct, e, e < p.vd, q, w);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.v_ready[slot]);
                }
                if (!ok) break;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// the local pass: each segment's own writes, decayed to its end
// ---------------------------------------------------------------------------
// Every write's weight is its distance to the segment's end, so the accumulator needs no
// decay on the way: the tensor cores sum C'^T B over all tiles.  The two groups of four
// warps take the tiles in turn, each with its own buffer of C' in TMEM.
constexpr int kLocThreads = 32 * 10, kLocProducer = 8, kLocIssuer = 9;     // warps
constexpr int kLocStages = 3;
constexpr uint32_t kLocStage = 2 * kTile;                    // B, C
constexpr uint32_t kLocOffBar = kLocStages * kLocStage;
constexpr uint32_t kLocOffW = kLocOffBar + 256;              // weights, a copy per warp
constexpr uint32_t kSmemLocal = kLocOffW + 8 * kC * 4;
constexpr uint32_t kLocColV = 128;                           // two buffers of 4 x 48 columns
static_assert(kLocColV + 2 * 4 * kSlotCols <= kTmemCols, "TMEM");

struct LocalBars {
    uint64_t full[kLocStages], free[kLocStages];
    uint64_t v_ready[2], v_free[2];
    uint64_t h_full, h_free;   // a unit's sum complete / read
    uint64_t fin;
    uint32_t tmem;
    int stop;
};
static_assert(sizeof(LocalBars) <= 256, "barriers");

__global__ void __launch_bounds__(kLocThreads, 1)
decay_local_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs A) {
    extern __shared__ __align__(1024) uint8_t smem[];
    LocalBars &bar = *(LocalBars *)(smem + kLocOffBar);
    volatile int *stop = &bar.stop;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = A.g.H;
    if (!GDR_INBOUNDS((smem_u32(smem) & 1023u) == 0)) return;   // swizzled tiles start on 1 KB
    if (tid == 0) {
        for (int i = 0; i < kLocStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.v_ready[i], 4);
            mbar_init(&bar.v_free[i], 1);
        }
        mbar_init(&bar.h_full, 1);
        mbar_init(&bar.h_free, 4);
        mbar_init(&bar.fin, 1);
        *stop = 0;
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == 0) {
        tmem_alloc(&bar.tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = bar.tmem;
    auto wait = [&](uint64_t *b, uint32_t use) {
        if (__all_sync(kFull, mbar_wait(b, use & 1u, A.wait_ns)) && !*stop) return true;
        if (lane == 0 && !*stop) set_status(A.status, GDR_ERR_TIMEOUT);
        *stop = 1;
        return false;
    };
    uint32_t it = 0, nu = 0;   // tiles and units so far
    Unit u;

    if (warp == kLocProducer) {
        bool ok = true;
        for (int64_t n = blockIdx.x; n < A.units && ok; n += gridDim.x) {
            if (!unit_of(A, n, true, u) || u.tiles == 0) continue;
            const DecayPass &p = A.pass[u.pass];
            for (int i = 0; i < u.tiles; ++i, ++it) {
                const uint32_t st = it % kLocStages, use = it / kLocStages;
                if (use && !(ok = wait(&bar.free[st], use - 1))) break;
                if (lane == 0) {
                    int64_t t;
                    int len;
                    tile_of(u, p.rev, i, t, len);
                    uint8_t *s = smem + st * kLocStage;
                    mbar_arrive_expect_tx(&bar.full[st], (p.kd + p.vd) / 64 * kBox);
                    load_tile(s, &maps.b[u.pass], p.kd, u.h, t, &bar.full[st]);
                    load_tile(s + kTile, &maps.c[u.pass], p.vd, u.h, t, &bar.full[st]);
                }
                __syncwarp();
            }
        }
        for (uint32_t k = it >= kLocStages ? it - kLocStages : 0; k < it; ++k)
            __all_sync(kFull, mbar_wait(&bar.full[k % kLocStages], (k / kLocStages) & 1u, kDrainNs));
    } else if (warp == kLocIssuer) {
        const uint32_t s0 = smem_u32(smem);
        bool ok = true;
        for (int64_t n = blockIdx.x; n < A.units && ok; n += gridDim.x) {
            if (!unit_of(A, n, true, u) || u.tiles == 0) continue;
            const DecayPass &p = A.pass[u.pass];
            const uint32_t id_h = instr_desc(kC, p.kd, 1, false, true);
            if (nu && !(ok = wait(&bar.h_free, nu - 1))) break;
            for (int i = 0; i < u.tiles; ++i, ++it) {
                const uint32_t st = it % kLocStages, buf = it & 1;
                int64_t t;
                int len;
                tile_of(u, p.rev, i, t, len);
                if (!(ok = wait(&bar.full[st], it / kLocStages))) break;
                if (len < kC) {
                    zero_rows(smem + st * kLocStage, p.kd, len, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (!(ok = wait(&bar.v_ready[buf], it >> 1))) break;
                tc_fence_after();
                const uint64_t dBt = smem_desc(s0 + st * kLocStage, kBox, 1024, kSw128);
                if (elect_one()) {
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int term = 0; term < 3; ++term)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                mma_f16_ts(tm, tm + kLocColV + (buf * 4 + q) * kSlotCols + term * 16 + k * 8,
                                           dBt + (((q * 2 + k) * 2048) >> 4), id_h, i + q + term + k > 0);
                    mma_commit(&bar.v_free[buf]);
                    mma_commit(&bar.free[st]);
                    if (i == u.tiles - 1) mma_commit(&bar.h_full);
                }
                __syncwarp();
            }
            ++nu;
        }
        if (elect_one()) mma_commit(&bar.fin);
        __syncwarp();
        __all_sync(kFull, mbar_wait(&bar.fin, 0, kDrainNs));
    } else {
        const int grp = warp >> 2, e = tid & 127;
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
        float *w = (float *)(smem + kLocOffW) + warp * kC;
        bool ok = true;
        for (int64_t n = blockIdx.x; n < A.units && ok; n += gridDim.x) {
            if (!unit_of(A, n, true, u)) continue;
            const DecayPass &p = A.pass[u.pass];
            const bool rev = p.rev;
            const float gd = decay_log(A.g.log_decay, u.h);
            float *to = decay_state_out(p, u.seg, H, u.h);
            if (u.tiles == 0) {
                if (grp == 0)
                    for (int d0 = 0; d0 < p.kd; d0 += 16) {
                        uint32_t r[16];
                        state_load(p, nullptr, d0, e, r);
                        state_store(p, to, d0, e, r);
                    }
                continue;
            }
            for (int i = 0; i < u.tiles; ++i, ++it) {
                const uint32_t st = it % kLocStages, buf = it & 1;
                if (buf != (uint32_t)grp) continue;
                int64_t t;
                int len;
                tile_of(u, rev, i, t, len);
                const uint32_t use = it >> 1;
                // past the tile: its distance to the segment's end (its start, reversed)
                tile_weights(w, len, rev, gd, p.s_upd, rev ? t - u.t0 : u.t1 - t - len, lane);
                if (!(ok = wait(&bar.full[st], it / kLocStages))) break;
                if (use && !(ok = wait(&bar.v_free[buf], use - 1))) break;
                tc_fence_after();
                uint8_t *ct = smem + st * kLocStage + kTile;
                if (len < kC && e < p.vd) {
                    zero_columns(ct, e & ~31, len, lane);
                    __syncwarp();
                }
#pragma unroll 1
                for (int q = 0; q < 4; ++q)
                    write_terms(lanes + kLocColV + (buf * 4 + q) * kSlotCols, ct, e, e < p.vd, q, w);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.v_ready[buf]);
            }
            if (ok && grp == 0) {
                if (!(ok = wait(&bar.h_full, nu))) break;
                tc_fence_after();
                tmem_columns(lanes, p.kd / 16, [&](int m, const uint32_t (&r)[16]) {
                    state_store(p, to, 16 * m, e, r);
                    __syncwarp();
                });
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.h_free);
            }
            ++nu;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, kTmemCols);
    }
}

// [rows][H][width] bf16 viewed as (d, h, row), box (64, 1, 128), 128-byte swizzle.
bool tile_map(CUtensorMap *map, const void *base, int width, int H, int64_t rows) {
    return base && tc_make_tile_map(map, base, width, H, rows, kC);
}

}  // namespace

cudaError_t launch_decay_tc(const DecayGeom &g, const DecayPass *passes, int n, int sms, int *status,
                            cudaStream_t stream) {
    if (n < 1 || n > kMaxPasses) return cudaErrorInvalidValue;
    const bool local = passes[0].local;
    TcMaps maps{};
    TcArgs args{};
    for (int i = 0; i < n; ++i) {
        const DecayPass &p = passes[i];
        if (!tile_map(&maps.b[i], p.b, p.kd, g.H, g.T_total) || !tile_map(&maps.c[i], p.c, p.vd, g.H, g.T_total) ||
            (!local && !tile_map(&maps.a[i], p.a, p.kd, g.H, g.T_total)))
            return cudaErrorNotSupported;
        args.pass[i] = p;
    }
    args.g = g;
    args.npass = n;
    args.units = g.max_segs * g.H * n;
    args.status = status;
    args.wait_ns = kWaitNs;
    if (const char *w = std::getenv("GDR_TC_WAIT_NS")) {   // test hook: shorter pipeline waits
        const long long x = std::atoll(w);
        if (x >= 0 && (uint64_t)x < kWaitNs) args.wait_ns = (uint64_t)x;
    }
    if (args.units == 0) return cudaSuccess;
    auto kern = local ? decay_local_kernel : decay_out_kernel;
    const int bytes = (int)(local ? kSmemLocal : kSmemOut);
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != cudaSuccess) return err;
    ProfScope prof(stream, local ? "decay_local_kernel" : "decay_out_kernel");
    kern<<<(unsigned)std::min<int64_t>(args.units, sms), local ? kLocThreads : kOutThreads, bytes, stream>>>(maps, args);
    count_launch();
    return cudaGetLastError();
}

}  // namespace gdr
