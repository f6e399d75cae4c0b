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
// state's part taken at 2^-64 where lam^{i+1} is below that.
//
// Four warps keep the state, 128 fp32 numbers a thread, and add each tile's part to it, which
// the tensor cores leave in the tensor memory (TMEM).  (A state that stayed there as the
// accumulator of every tile lost up to 1e-5 of itself where the decay is weak: the tensor cores
// cut a sum off where it leaves fp32 instead of rounding it, 24 times a tile and always
// towards zero.  Registers: 4e-7 and no more over 65536 tokens.)
//
// All four products run on the tensor cores with fp32 accumulators in TMEM, 128 x 128 each:
//     Sc = A B^T                     lanes = query tokens i
//     U  = C'^T B                    lanes = value index e: the tile's part of the new S^T
//     O  = A S                       lanes = query tokens i; S from shared memory in bf16
//     O += P C                       P in TMEM in bf16
// in this order, O = A S in the middle of U's parts.  A tile of one head is 128 KB of HBM traffic
// (3 loads, 1 store; 2.9 us of an SM's share of the measured bandwidth) and 25 MFLOP (2.0 us of
// an SM's share of the bf16 rate), so the pass can be bound by HBM if its other work stays out
// of the way.  The stages of a tile run in different warps and overlap those of its neighbours:
//   warps 0-7    Sc -> P (bf16, over Sc in TMEM); O -> out; half of the columns each group
//   warps 8-11   S <- lam^n S + U, in bf16 to shared memory
//   warps 12-19  C' = weighted C -> TMEM, 32 tokens at a time, half of them each group
//   warp 20      TMA loads of A, B, C, two stages of 96 KB
//   warp 21      issues every MMA (their order in the tensor pipe is the issue order)
//   warp 22      TMA stores of the outputs, out of their tile's A
// Where both widths are 64 (kNarrow) there is room for more: four stages of 48 KB, a whole tile's
// C' in TMEM, and, as the state takes half the registers, four warps of their own (20-23) for
// O -> out (65536 tokens of 32 heads x 64 in 37 sequences: 391 us against 400).
// What is left of the bound (8 x 4096 tokens of 16 heads, 128 units on 152 SMs: 116 us, 3.6 us a
// tile; 262144 tokens: 84% of the measured bandwidth): a tile's chain through its A -- load, Sc,
// P, O, store -- takes some 14000 cycles, with two tiles in flight.
//
// Rounding.  The state is fp32 and so are its updates: C' has 24 significant bits, so it goes
// in as the sum of three bf16 numbers that represent it exactly (three products instead of
// one; two would leave 2^-17 in hT and dh0).  Small terms go first and the tile's tokens in the
// order of growing weights, so that little is cut off.  P and the state as a factor of O are
// rounded to bf16: each adds an error of at most 2^-8 of its part of an output that is itself
// rounded to bf16 (2.3e-3 in the mean square over the outputs against 1.7e-3 for their rounding
// alone).
//
// A block is persistent: it walks the units (segment, head, pass) with a stride of the grid
// (equal sequences) or takes the next one from a counter (packed ones), and its pipeline
// runs on across them.  The three passes of a backward call are
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
constexpr int kMaxPasses = kDecayMaxPasses;
constexpr uint32_t kBox = kC * 128;        // 64 columns x 128 tokens, 128-byte rows, swizzled
constexpr uint32_t kTile = 2 * kBox;       // one tensor's tile: up to two boxes
constexpr uint32_t kBarBytes = 384;        // of a block's barriers
constexpr unsigned kFull = 0xffffffffu;
constexpr uint64_t kWaitNs = 2000000000ull;   // pipeline wait limit: 2 s
constexpr uint64_t kDrainNs = 2000000000ull;  // drains before exit

struct TcMaps {
    CUtensorMap a[kMaxPasses], b[kMaxPasses], c[kMaxPasses], o[kMaxPasses];
};
struct TcArgs {
    DecayGeom g;
    DecayPass pass[kMaxPasses];
    int npass;
    int64_t units;      // max_segs * H * npass, and times the parts in a local pass
    unsigned long long *next;   // the next unit to take, or null: units by stride
    bool long_first;            // the counter runs over all units twice
    int *status;
    uint64_t wait_ns;
};

// The rest of a wait that its first look did not end.  The warp sleeps meanwhile, in pieces
// of up to 0.1 ms.  (Inline: a call would have the callers save the state's registers.)
__device__ __forceinline__ bool wait_long(uint64_t *b, uint32_t parity, uint64_t limit_ns, volatile int *stop,
                                          int *status) {
    const uint64_t t0 = globaltimer_ns();
    while (__all_sync(kFull, !*stop && globaltimer_ns() - t0 < limit_ns))
        if (__all_sync(kFull, mbar_try_wait_for(b, parity, 100000))) return true;
    if (!*stop) set_status(status, GDR_ERR_TIMEOUT);
    *stop = 1;
    return false;
}
// Waits (a whole warp) until `b` has completed its use number `use` (from 0).  False if that
// takes longer than the limit (0: look once), or once another wait of the block has run
// out, which sets the status word.
__device__ __forceinline__ bool wait_use(uint64_t *b, uint32_t use, uint64_t limit_ns, volatile int *stop,
                                         int *status) {
    if (__all_sync(kFull, limit_ns ? mbar_try_wait(b, use & 1u) : mbar_test_wait(b, use & 1u))) return true;
    return wait_long(b, use & 1u, limit_ns, stop, status);
}

// One unit of a block's walk, put into shared memory by the producer for all warps.
struct Unit {
    int64_t t0, t1;    // tokens it runs (a local pass: those that reach the segment's end)
    union {
        const float *in;   // entering state (null: zero)
        int64_t past;      // a local pass's: tokens between it and where its sum ends
    };
    float *to;         // where to leave the last state (or null)
    float gd;          // the head's log-decay
    int pass, h, tiles;   // tiles < 0: no more units
};
constexpr uint32_t kRing = 4;   // units announced ahead

// The output pass, its second run of the sequences that need one, and the local pass.
enum Kind { kOut, kAgain, kLocal };

// Whether outputs of sequence n in unit o's head and pass show a value that is not finite and that
// a local sum may have skipped; if so the sequence as one segment (one warp).  Such a value is in the
// state before the last tile of the segment that it is in, so the outputs of the segment's last
// token, all of them or those of a column, are not finite either.
__device__ __forceinline__ bool whole_sequence(const TcArgs &A, int64_t n, const Unit &o, DecaySeg &seg) {
    const DecayGeom &g = A.g;
    if (n >= g.N) return false;
    const DecayPass &p = A.pass[o.pass];
    const int64_t cuts = (g.dense ? g.segs_per_seq : g.p.seg_base[n + 1] - g.p.seg_base[n]) - 1;
    if (cuts < 1 || decay_reach(decay_log(g.log_decay, o.h), g.seg_tokens) > g.seg_tokens - kC) return false;
    seg.t0 = g.dense ? n * g.T_per : g.p.seq_start[n];
    seg.t1 = g.dense ? seg.t0 + g.T_per : g.p.seq_start[n + 1];
    const int lanes = p.vd / 8, per = 32 / lanes, lane = threadIdx.x & 31;   // of a row; rows at a time
    bool bad = false;
#pragma unroll 4
    for (int64_t i = lane / lanes; i < cuts; i += per) {
        const int64_t t = seg.t0 + (i + 1) * g.seg_tokens - (p.rev ? 0 : 1);
        const uint4 x = *(const uint4 *)((const __nv_bfloat16 *)p.out + (t * g.H + o.h) * p.vd + 8 * (lane % lanes));
        for (uint32_t w : {x.x, x.y, x.z, x.w}) bad |= (~w & 0x7f80u) == 0 || (~w & 0x7f800000u) == 0;
    }
    seg.n = (int)n;
    seg.slot = 0;
    seg.first = seg.last = true;
    return __any_sync(kFull, bad);
}

// False where unit u has nothing to do.
template <Kind kKind> __device__ __forceinline__ bool unit_of(const TcArgs &A, int64_t u, Unit &o) {
    constexpr bool local = kKind == kLocal;
    uint32_t sh = (uint32_t)u, part = 0;   // fewer than 2^31 units
    o.pass = (int)(sh % (uint32_t)A.npass);
    sh /= (uint32_t)A.npass;
    if (local) {
        part = sh % (uint32_t)A.g.parts;
        sh /= (uint32_t)A.g.parts;
    }
    const uint32_t sg = sh / (uint32_t)A.g.H;
    o.h = (int)(sh - sg * (uint32_t)A.g.H);
    DecaySeg seg;
    if (!(kKind == kAgain ? whole_sequence(A, sg, o, seg) : decay_segment(A.g, sg, seg))) return false;
    const DecayPass &p = A.pass[o.pass];
    o.gd = decay_log(A.g.log_decay, o.h);
    o.t0 = seg.t0;
    o.t1 = seg.t1;
    if (local) {
        if (p.rev ? seg.first : seg.last) return false;   // no boundary behind it
        if ((int)part >= decay_parts(A.g, o.gd)) return false;
        // whole tiles: the segment is one (reversed: but for its sequence's last tile)
        const int64_t reach = (decay_reach(o.gd, o.t1 - o.t0) + kC - 1) / kC * kC;
        const int64_t past = part * A.g.part_tokens, end = min(reach, past + A.g.part_tokens);
        if (p.rev) {
            o.t1 = min(o.t1, o.t0 + end);
            o.t0 = min(o.t1, o.t0 + past);
        } else {
            o.t0 = max(o.t0, o.t1 - end);
            o.t1 = max(o.t0, o.t1 - past);
        }
    }
    o.tiles = (int)((o.t1 - o.t0 + kC - 1) / kC);
    if (local) o.past = part * A.g.part_tokens;
    else o.in = decay_state_in(p, seg, A.g.H, o.h);
    o.to = decay_state_out(p, seg, A.g.H, o.h);
    if (local) o.to += (int64_t)part * A.g.max_slots * A.g.H * p.kd * p.vd;
    return GDR_INBOUNDS(seg.t0 >= 0 && seg.t1 <= A.g.T_total && seg.slot <= A.g.max_slots);
}
// The block's next unit (one warp): those of its stride, or from the counter.  Where there are
// not very many the counter runs over all twice -- those of more than half the most tiles
// first, then the others, so that the blocks end together.  False at the end.  `n`: the last one (blockIdx.x -
// gridDim.x at the start).
template <Kind kKind> __device__ __forceinline__ bool take_unit(const TcArgs &A, int64_t &n, Unit &u) {
    constexpr bool local = kKind == kLocal;
    while (true) {
        bool want_long = false;
        int64_t i;
        if (A.next) {
            unsigned long long x = 0;
            if ((threadIdx.x & 31) == 0) x = atomicAdd(A.next, 1ull);
            i = (int64_t)__shfl_sync(kFull, x, 0);
            want_long = A.long_first && i < A.units;
            if (A.long_first && !want_long) i -= A.units;
        } else {
            i = n += gridDim.x;
        }
        if (i >= A.units) return false;
        if (unit_of<kKind>(A, i, u) &&
            (!A.long_first || (2 * (int64_t)u.tiles * kC > (local ? A.g.part_tokens : A.g.seg_tokens)) == want_long))
            return true;
    }
}
// The tiles of a unit in the order of its pass, in registers: a role's loop reads neither
// shared memory nor parameters for its bookkeeping.
struct Walk {
    int tiles, short_at, short_len;   // one tile (the last of the tokens) may be short
    bool rev;
    __device__ __forceinline__ Walk(const Unit &u, bool rev)
        : tiles(u.tiles), short_at(rev ? 0 : u.tiles - 1),
          short_len((int)(u.t1 - u.t0 - (int64_t)(u.tiles - 1) * kC)), rev(rev) {}
    __device__ __forceinline__ int len(int i) const { return i == short_at ? short_len : kC; }
    __device__ __forceinline__ int64_t first(const Unit &u, int i) const {   // token
        return u.t0 + (int64_t)(rev ? tiles - 1 - i : i) * kC;
    }
};

// Descriptor offset of K-step k (16 of up to 128 elements) of a K-major tile.
__device__ constexpr uint64_t k_major(uint32_t k) { return ((k >> 2) * kBox + (k & 3) * 32) >> 4; }

__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *map, int width, int h, int64_t t,
                                          uint64_t *bar) {
    tma_load_3d(dst, map, 0, h, (int)t, bar);
    if (width > 64) tma_load_3d(dst + kBox, map, 64, h, (int)t, bar);
}

// Zeroes the rows from n on of a tile in shared memory -- tokens past the sequence's end,
// which are another sequence's -- as warp `part` of `parts`.  (A weight of 0 would not
// silence a NaN.)
__device__ __forceinline__ void zero_rows(uint8_t *tile, int width, int n, int part, int parts, int lane) {
    for (int i = 32 * part + lane; i < (kC - n) * (width / 8); i += 32 * parts) {
        const int r = n + i / (width / 8), c = i % (width / 8);
        *(uint4 *)(tile + (c >> 3) * kBox + sw128_off(r, (c & 7) * 16)) = make_uint4(0, 0, 0, 0);
    }
}

// log2 lam; below -200 every power but the zeroth is out of the range of fp32 and its
// reciprocals, whatever lam is, and differences of multiples stay exact enough.  A NaN stays one.
__device__ __forceinline__ float decay_log2(float gd) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(gd * 1.4426950408889634f), "f"(-200.f));
    return y;
}

// A token's weight in the update of the state: s_upd lam^{len - 1 - i + past} (forward) or
// s_upd lam^{i + 1 + past}; rows from len on are not the sequence's and have 0.
__device__ __forceinline__ float token_weight(int i, int len, bool rev, float gd, float s_upd, int64_t past) {
    return i < len ? s_upd * expf(gd * (float)(past + (rev ? i + 1 : len - 1 - i))) : 0.f;
}

// Zeroes the rows from n on of the 32 columns from e0 (one warp) of a tile.
__device__ __forceinline__ void zero_columns(uint8_t *tile, int e0, int n, int lane) {
    for (int i = lane; i < (kC - n) * 4; i += 32)
        *(uint4 *)(tile + (e0 >> 6) * kBox + sw128_off(n + i / 4, (e0 & 63) * 2 + (i & 3) * 16)) =
            make_uint4(0, 0, 0, 0);
}

// Two fp32 numbers in a 64-bit register (the first in the low half) and their products and
// sums, one instruction for both.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
    return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint32_t tops(uint64_t y) {   // the upper 16 bits of both
    return __byte_perm((uint32_t)y, (uint32_t)(y >> 32), 0x7632);
}
// What is left of both after their upper 16 bits (exact).
__device__ __forceinline__ uint64_t rest(uint64_t y) {
    return add2(y, (y & 0xffff0000ffff0000ull) ^ 0x8000000080000000ull);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t *)&v;
}
__device__ __forceinline__ uint32_t pack2(uint64_t y) {
    return pack2(__uint_as_float((uint32_t)y), __uint_as_float((uint32_t)(y >> 32)));
}

// 16 tokens (from 16 k) of a tile's C'^T, row e, into 8 TMEM columns at `at`, at + 16 and
// at + 32 (a whole warp): the weighted values x w as the bf16 terms hi + mid + lo = x w exactly, cut
// off the top of the fp32 product 8 significant bits at a time; a column holds two tokens.
// w: the 16 weights.
__device__ __forceinline__ void write_terms(uint32_t at, const uint8_t *tile, int e, int k, const float *w) {
    uint32_t hi[8], mid[8], lo[8];
    const uint8_t *col = tile + (e >> 6) * kBox + (e & 7) * 2 + k * 2048;
    const uint32_t chunk = (e & 63) >> 3;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const ulonglong2 w4 = *(const ulonglong2 *)&w[2 * i];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t x[2];
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                const int r = 2 * (i + j) + l;
                const uint32_t at16 = (r >> 3) * 1024 + (r & 7) * 128 + ((chunk ^ (r & 7)) << 4);
                x[l] = (uint32_t)*(const uint16_t *)(col + at16) << 16;
            }
            uint64_t y = mul2((uint64_t)x[1] << 32 | x[0], j ? w4.y : w4.x);
            hi[i + j] = tops(y);
            y = rest(y);
            mid[i + j] = tops(y);
            lo[i + j] = tops(rest(y));
        }
    }
    tmem_st8(at, hi);
    tmem_st8(at + 16, mid);
    tmem_st8(at + 32, lo);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A thread's registers from here on (all warps of a warpgroup).
template <int kRegs, bool kMore> __device__ __forceinline__ void set_registers() {
    if (kMore) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
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
// Row e of S^T in registers, s[j] = (S[2j][e], S[2j+1][e]): from memory (zeros past the
// widths and for a null `in`), back, and in bf16 to shared memory as a K-major tile's row.
template <int kKd> using StateRow = uint64_t[kKd / 2];   // kKd: the widest kd
template <int kVd, int kKd>
__device__ __forceinline__ void state_load_from(const DecayPass &p, const float *in, int e, StateRow<kKd> &s) {
#pragma unroll
    for (int h = 0; h < kKd / 64; ++h) {
        if (64 * h >= p.kd) break;
        if (p.transposed) {
            const ulonglong2 *row = (const ulonglong2 *)(in + e * p.kd + 64 * h);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const ulonglong2 x = row[j];
                s[32 * h + 2 * j] = x.x;
                s[32 * h + 2 * j + 1] = x.y;
            }
        } else {
            const float *col = in + 64 * h * kVd + e;
#pragma unroll
            for (int j = 0; j < 32; ++j) s[32 * h + j] = two(col[2 * j * kVd], col[(2 * j + 1) * kVd]);
        }
    }
}
template <int kKd>
__device__ __forceinline__ void state_load(const DecayPass &p, const float *in, int e, StateRow<kKd> &s) {
#pragma unroll
    for (int j = 0; j < kKd / 2; ++j) s[j] = 0;
    if (!in || e >= p.vd) return;
    if (p.vd == 64) state_load_from<64, kKd>(p, in, e, s);
    else state_load_from<128, kKd>(p, in, e, s);
}
template <int kVd, int kKd>
__device__ __forceinline__ void state_store_to(const DecayPass &p, float *to, int e, const StateRow<kKd> &s) {
#pragma unroll
    for (int h = 0; h < kKd / 64; ++h) {
        if (64 * h >= p.kd) break;
        if (p.transposed) {
            ulonglong2 *row = (ulonglong2 *)(to + e * p.kd + 64 * h);
#pragma unroll
            for (int j = 0; j < 16; ++j) row[j] = make_ulonglong2(s[32 * h + 2 * j], s[32 * h + 2 * j + 1]);
        } else {
            float *col = to + 64 * h * kVd + e;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                col[2 * j * kVd] = __uint_as_float((uint32_t)s[32 * h + j]);
                col[(2 * j + 1) * kVd] = __uint_as_float((uint32_t)(s[32 * h + j] >> 32));
            }
        }
    }
}
template <int kKd>
__device__ __forceinline__ void state_store(const DecayPass &p, float *to, int e, const StateRow<kKd> &s) {
    if (e >= p.vd) return;
    if (p.vd == 64) state_store_to<64, kKd>(p, to, e, s);
    else state_store_to<128, kKd>(p, to, e, s);
}
template <int kKd>
__device__ __forceinline__ void state_to_bf16(const StateRow<kKd> &s, uint8_t *tile, int e, int kd) {
#pragma unroll
    for (int j = 0; j < kKd / 8; ++j) {
        if (8 * j == 64 && kd == 64) break;
        *(uint4 *)(tile + (j >> 3) * kBox + sw128_off(e, (j & 7) * 16)) =
            make_uint4(pack2(s[4 * j]), pack2(s[4 * j + 1]), pack2(s[4 * j + 2]), pack2(s[4 * j + 3]));
    }
}
// s <- s fa + s fb + the kd TMEM columns from `at` on, in fp32 (a whole warp); the factors, in
// pairs, are (1, lam^n - 1) near 1 and (lam^n, 0) otherwise.  Without kDecay s is only added to.
template <bool kDecay, int kKd>
__device__ __forceinline__ void state_add(StateRow<kKd> &s, uint32_t at, int kd, uint64_t fa, uint64_t fb) {
#pragma unroll
    for (int m = 0; m < kKd / 16; ++m) {
        if (m == 4 && kd == 64) break;
        uint32_t r[16];
        tmem_ld16(at + 16 * m, r);
        tmem_arrived(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint64_t &x = s[8 * m + j];
            const uint64_t u = (uint64_t)r[2 * j + 1] << 32 | r[2 * j];
            x = kDecay ? fma2(x, fa, fma2(x, fb, u)) : add2(x, u);
        }
    }
}

// f(m, r) for 16 columns at a time from `at`, the next ones on their way meanwhile.  One
// copy of f: the warps of a block run six different programs, which have to stay in the
// instruction caches together.
template <typename F> __device__ __forceinline__ void tmem_columns(uint32_t at, int pieces, F &&f) {
    uint32_t next[16], r[16];
    tmem_ld16(at, next);
#pragma unroll 1
    for (int m = 0; m < pieces; ++m) {
        tmem_arrived(next);
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = next[j];
        if (m + 1 < pieces) tmem_ld16(at + 16 * (m + 1), next);
        f(m, r);
    }
}

// ---------------------------------------------------------------------------
// the output pass
// ---------------------------------------------------------------------------
// (one warp, the last, fills up its warpgroup and has nothing to do)
constexpr int kOutWarps = 24, kOutWarpsNarrow = 28;
// TMEM columns
constexpr uint32_t kColS = 0;      // Sc; P in the first 32 columns of each of its halves
constexpr uint32_t kColO = 128;
// then U, the tile's part of the new S^T, and slots of C'^T, 32 tokens x 3 terms each: 2 of them,
// or a tile's 4 where both widths are 64 (kNarrow)
constexpr uint32_t kSlotCols = 48, kMaxSlots = 4, kParts = kC / 32;   // kParts uses of slots per tile
constexpr uint32_t kTmemCols = 512;
// shared memory
constexpr uint32_t kMaxStages = 4;                   // tiles in flight: 2 of 96 KB, or 4 of 48 (kNarrow)
constexpr uint32_t kOffH = 2 * 3 * kTile;            // the state in bf16, [e][d], K-major
constexpr uint32_t kOffBar = kOffH + kTile;
constexpr uint32_t kOffW = kOffBar + kBarBytes;            // weights of a group's 64 tokens, a copy per warp
constexpr uint32_t kOffRing = kOffW + 8 * (kC / 2) * 4;
constexpr uint32_t kSmemOut = kOffRing + kRing * sizeof(Unit);
static_assert(kSmemOut <= 232448, "shared memory");
// Registers of a thread at launch (what 768, or narrow 896, threads may have); by role from then
// on, where the increase draws on the registers that the block was launched with.
constexpr int kRegsLaunch = 80, kRegsLaunchNarrow = 72;

struct OutBars {
    uint64_t u_full[kRing], u_free[kRing];   // a unit announced / done with (every warp that takes units)
    uint64_t full_a[kMaxStages];    // a stage's A has arrived
    uint64_t full_bc[kMaxStages];   // ... its B and C
    uint64_t free_a[kMaxStages];    // the stage's A is read, and the outputs that went through it
    uint64_t free_bc[kMaxStages];   // ... its B and C
    uint64_t s_full;       // Sc complete
    uint64_t p_ready;      // P written (8 warps)
    uint64_t o_full;       // O complete
    uint64_t o_free;       // O read (8 warps; narrow: 4)
    // ... and in shared memory.  One per stage: the stores, which wait for every one, may be a
    // tile late, and a barrier that had moved on twice would look as if it had not moved.
    uint64_t staged[kMaxStages];
    uint64_t s_free;       // U read (4 warps)
    uint64_t h_ready;      // the bf16 state written (4 warps)
    uint64_t v_ready[kMaxSlots];   // a slot of C' written (8 warps)
    uint64_t v_free[kMaxSlots];    // ... read
    uint64_t kv_full;      // U complete, and the bf16 state read
    uint64_t fin;          // every MMA of the block complete
    uint32_t tmem;
    int stop;
};
static_assert(sizeof(OutBars) <= kBarBytes, "barriers");

template <bool kNarrow, Kind kKind>
__global__ void __launch_bounds__(32 * (kNarrow ? kOutWarpsNarrow : kOutWarps), 1)
decay_out_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs A) {
    constexpr uint32_t kColU = kColO + (kNarrow ? 64 : kC), kColV = kColU + (kNarrow ? 64 : kC);
    constexpr int kOutProducer = (kNarrow ? kOutWarpsNarrow : kOutWarps) - 4, kOutIssuer = kOutProducer + 1;
    constexpr int kOutStore = kOutProducer + 2;
    constexpr uint32_t kSlots = kNarrow ? 4 : 2;
    constexpr uint32_t kTileBytes = kNarrow ? kBox : kTile, kStageBytes = 3 * kTileBytes;   // A, B, C
    constexpr uint32_t kStages = kNarrow ? kMaxStages : 2;
    static_assert(kStages * kStageBytes <= kOffH, "stages");
    constexpr int kKd = kNarrow ? 64 : kC;
    constexpr int kRegsOut = 64, kRegsState = kNarrow ? 136 : 168, kRegsV = 64;
    constexpr int kRegsO = kNarrow ? 48 : 0, kRegsOther = kNarrow ? 64 : 56;
    static_assert(2 * kRegsOut + kRegsState + 2 * kRegsV + kRegsO + kRegsOther <=
                      (kNarrow ? 7 * kRegsLaunchNarrow : 6 * kRegsLaunch), "registers");
    extern __shared__ __align__(1024) uint8_t smem[];
    OutBars &bar = *(OutBars *)(smem + kOffBar);
    Unit *ring = (Unit *)(smem + kOffRing);
    volatile int *stop = &bar.stop;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = A.g.H;
    if (!GDR_INBOUNDS((smem_u32(smem) & 1023u) == 0)) return;   // swizzled tiles start on 1 KB

    let_next_start();
    if constexpr (kKind == kAgain) {   // only if the block has a unit
        after_previous();
        bool any = false;
        for (int64_t u = blockIdx.x + (int64_t)warp * gridDim.x; u < A.units; u += (int64_t)(blockDim.x / 32) * gridDim.x) {
            Unit o;
            any |= unit_of<kAgain>(A, u, o);
        }
        if (!__syncthreads_or(any)) return;
    }
    if (tid == 0) {
        for (uint32_t i = 0; i < kRing; ++i) {
            mbar_init(&bar.u_full[i], 1);
            mbar_init(&bar.u_free[i], kNarrow ? 26 : 22);
        }
        for (uint32_t i = 0; i < kStages; ++i) {
            mbar_init(&bar.full_a[i], 1);
            mbar_init(&bar.full_bc[i], 1);
            mbar_init(&bar.free_a[i], 1);
            mbar_init(&bar.staged[i], kNarrow ? 4 : 8);
            mbar_init(&bar.free_bc[i], 1);
        }
        for (uint32_t i = 0; i < kSlots; ++i) {
            mbar_init(&bar.v_ready[i], 8);
            mbar_init(&bar.v_free[i], 1);
        }
        mbar_init(&bar.s_full, 1);
        mbar_init(&bar.p_ready, 8);
        mbar_init(&bar.o_full, 1);
        mbar_init(&bar.o_free, kNarrow ? 4 : 8);
        mbar_init(&bar.s_free, 4);
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
    after_previous();
    const uint32_t tm = bar.tmem;

    auto wait = [&](uint64_t *b, uint32_t use) { return wait_use(b, use, A.wait_ns, stop, A.status); };
    uint32_t it = 0;   // tiles so far: the use number of every once-a-tile barrier
    // Walks the announced units (every warp but the producer): f(unit) until the end or until
    // it returns false.
    auto each_unit = [&](auto &&f) {
        for (uint32_t k = 0;; ++k) {
            if (!wait(&bar.u_full[k % kRing], k / kRing)) return;
            const Unit &u = ring[k % kRing];
            if (u.tiles < 0 || !f(u)) return;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.u_free[k % kRing]);
        }
    };

    // O of tile n out through its A (whose products are complete), in bf16 in the layout of the
    // store's boxes: 16 m columns from c0 of the thread's row, times f.
    auto take_o = [&](uint32_t n, int row, int c0, int pieces, uint32_t lanes, float f) {
        if (!wait(&bar.o_full, n)) return false;
        tc_fence_after();
        const uint64_t f2 = two(f, f);
        uint8_t *buf = smem + (n % kStages) * kStageBytes;
        tmem_columns(lanes + kColO + c0, pieces, [&](int m, const uint32_t (&x)[16]) {
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = pack2(mul2((uint64_t)x[2 * j + 1] << 32 | x[2 * j], f2));
            const int col = c0 + 16 * m;
            uint8_t *to = buf + (col >> 6) * kBox;
            *(uint4 *)(to + sw128_off(row, (col & 63) * 2)) = make_uint4(o[0], o[1], o[2], o[3]);
            *(uint4 *)(to + sw128_off(row, (col & 63) * 2 + 16)) = make_uint4(o[4], o[5], o[6], o[7]);
        });
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bar.o_free);
            mbar_arrive(&bar.staged[n % kStages]);
        }
        return true;
    };

    if (warp >= kOutProducer) {
        set_registers<kRegsOther, false>();
        if (warp == kOutProducer) {
            bool ok = true;
            int64_t n = (int64_t)blockIdx.x - gridDim.x;
            uint32_t nbc = 0;   // tiles whose B and C are on their way (`it`: whose A is too)
            for (uint32_t k = 0; ok; ++k) {
                Unit u;
                if (!take_unit<kKind>(A, n, u)) u.tiles = -1;
                if (k >= kRing && !(ok = wait(&bar.u_free[k % kRing], k / kRing - 1))) break;
                if (lane == 0) {
                    ring[k % kRing] = u;
                    mbar_arrive(&bar.u_full[k % kRing]);
                }
                __syncwarp();
                if (u.tiles < 0) break;
                const DecayPass &p = A.pass[u.pass];
                const Walk walk(u, p.rev);
                const int kd = p.kd, vd = p.vd;
                // the entering state on its way into the L2, ahead of the warps that take it
                if (u.in)
                    for (int i = 32 * lane; i < kd * vd; i += 1024)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(u.in + i));
                for (int i = 0; i < walk.tiles; ++i, ++it) {
                    const uint32_t st = it % kStages;
                    const int64_t t = walk.first(u, i);
                    uint8_t *s = smem + st * kStageBytes;
                    if (it >= kStages && !(ok = wait(&bar.free_bc[st], (it / kStages) - 1))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar.full_bc[st], (kd + vd) / 64 * kBox);
                        load_tile(s + kTileBytes, &maps.b[u.pass], kd, u.h, t, &bar.full_bc[st]);
                        load_tile(s + 2 * kTileBytes, &maps.c[u.pass], vd, u.h, t, &bar.full_bc[st]);
                    }
                    __syncwarp();
                    ++nbc;
                    if (it >= kStages && !(ok = wait(&bar.free_a[st], (it / kStages) - 1))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar.full_a[st], kd / 64 * kBox);
                        load_tile(s, &maps.a[u.pass], kd, u.h, t, &bar.full_a[st]);
                    }
                    __syncwarp();
                }
            }
            // never leave with a copy in flight
            for (uint32_t k = it >= kStages ? it - kStages : 0; k < it; ++k)
                __all_sync(kFull, mbar_wait(&bar.full_a[k % kStages], (k / kStages) & 1u, kDrainNs));
            for (uint32_t k = nbc >= kStages ? nbc - kStages : 0; k < nbc; ++k)
                __all_sync(kFull, mbar_wait(&bar.full_bc[k % kStages], (k / kStages) & 1u, kDrainNs));
        } else if (warp == kOutIssuer) {
            const uint32_t s0 = smem_u32(smem);
            const bool lead = elect_one();
            each_unit([&](const Unit &u) {
                bool ok = true;
                const DecayPass &p = A.pass[u.pass];
                const Walk walk(u, p.rev);
                const int kd = p.kd;
                const uint32_t kd16 = (uint32_t)kd / 16;
                const uint32_t id_s = instr_desc(kC, kC, 1, false, false);
                const uint32_t id_o1 = instr_desc(kC, p.vd, 1, false, false);
                const uint32_t id_o2 = instr_desc(kC, p.vd, 1, false, true);
                const uint32_t id_h = instr_desc(kC, kd, 1, false, true);
                for (int i = 0; i < walk.tiles; ++i, ++it) {
                    const uint32_t st = it % kStages;
                    const uint32_t sa = s0 + st * kStageBytes, sb = sa + kTileBytes, sc = sb + kTileBytes;
                    if (!(ok = wait(&bar.full_bc[st], it / kStages)) || !(ok = wait(&bar.full_a[st], it / kStages))) break;
                    tc_fence_after();
                    const uint64_t dA = smem_desc(sa, 16, 1024, kSw128), dB = smem_desc(sb, 16, 1024, kSw128);
                    const uint64_t dBt = smem_desc(sb, kBox, 1024, kSw128), dCt = smem_desc(sc, kBox, 1024, kSw128);
                    const uint64_t dH = smem_desc(s0 + kOffH, 16, 1024, kSw128);
                    // the previous tile's P is read: its product precedes this one in the pipe
#pragma unroll
                    for (uint32_t k = 0; k < 8; ++k)
                        if (k < kd16) mma_f16_ss_if(lead, tm + kColS, dA + k_major(k), dB + k_major(k), id_s, k > 0);
                    mma_commit_if(lead, &bar.s_full);
                    if (!(ok = wait(&bar.s_free, it))) break;
#pragma unroll
                    for (uint32_t k = 0; k < kParts; ++k) {
                        const uint32_t slot = k % kSlots, av = tm + kColV + slot * kSlotCols;
                        if (k == kParts / 2) {   // while the slots are filled again
                            if (!(ok = wait(&bar.h_ready, it)) || (it && !(ok = wait(&bar.o_free, it - 1)))) break;
                            tc_fence_after();
#pragma unroll
                            for (uint32_t j = 0; j < 8; ++j)
                                if (j < kd16)
                                    mma_f16_ss_if(lead, tm + kColO, dA + k_major(j), dH + k_major(j), id_o1, j > 0);
                        }
                        if (!(ok = wait(&bar.v_ready[slot], (it * kParts + k) / kSlots))) break;
                        tc_fence_after();
                        const uint64_t dPart = dBt + (((p.rev ? kParts - 1 - k : k) * 4096) >> 4);
#pragma unroll
                        for (uint32_t term = 0; term < 3; ++term)
#pragma unroll
                            for (uint32_t j = 0; j < 2; ++j)
                                mma_f16_ts_if(lead, tm + kColU, av + (2 - term) * 16 + j * 8, dPart + ((j * 2048) >> 4),
                                              id_h, k + term + j > 0);
                        mma_commit_if(lead, &bar.v_free[slot]);
                    }
                    mma_commit_if(lead, &bar.kv_full);
                    if (!ok || !(ok = wait(&bar.p_ready, it))) break;
                    tc_fence_after();
#pragma unroll
                    for (uint32_t k = 0; k < kC / 16; ++k)
                        mma_f16_ts_if(lead, tm + kColO, tm + kColS + (k >> 2) * 64 + (k & 3) * 8, dCt + ((k * 2048) >> 4), id_o2, 1);
                    mma_commit_if(lead, &bar.o_full);
                    mma_commit_if(lead, &bar.free_bc[st]);
                }
                return ok;
            });
            // no tensor-core operation may still run when the TMEM is released
            mma_commit_if(lead, &bar.fin);
            __all_sync(kFull, mbar_wait(&bar.fin, 0, kDrainNs));
        } else if (warp == kOutStore) {
            // ---- outputs: a tile's as boxes of 64 columns, or row by row at a sequence's end
            each_unit([&](const Unit &u) {
                bool ok = true;
                const DecayPass &p = A.pass[u.pass];
                const Walk walk(u, p.rev);
                const int vd = p.vd;
                for (int i = 0; i < walk.tiles; ++i, ++it) {
                    const int len = walk.len(i);
                    const int64_t t = walk.first(u, i);
                    const uint8_t *buf = smem + (it % kStages) * kStageBytes;
                    if (!(ok = wait(&bar.staged[it % kStages], it / kStages))) break;
                    if (len == kC) {
                        if (lane == 0) {
                            for (int b = 0; b < vd; b += 64)
                                tma_store_3d(&maps.o[u.pass], b, u.h, (int)t, buf + (b >> 6) * kBox);
                            bulk_commit();
                            bulk_wait_read();
                        }
                    } else {
#pragma unroll 4
                        for (int k = lane; k < len * (vd / 8); k += 32) {
                            const int r = k / (vd / 8), c = 8 * (k % (vd / 8));
                            *(uint4 *)((__nv_bfloat16 *)p.out + ((t + r) * H + u.h) * (int64_t)vd + c) =
                                *(const uint4 *)(buf + (c >> 6) * kBox + sw128_off(r, (c & 63) * 2));
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.free_a[it % kStages]);
                }
                return ok;
            });
            bulk_wait();   // the block's shared memory goes with it
        }
    } else if (warp < 8) {
        // ---- weights and outputs: thread = token row of the tile, and half of the columns
        set_registers<kRegsOut, false>();
        const int rw = warp & 3, half = warp >> 2, row = tid & 127;
        const uint32_t lanes = tm + ((uint32_t)(rw * 32) << 16);
        each_unit([&](const Unit &u) {
            bool ok = true;
            const DecayPass &p = A.pass[u.pass];
            const bool rev = p.rev;
            const Walk walk(u, rev);
            const float g2 = decay_log2(u.gd), s_upd = p.s_upd, s_out = p.s_out;
            const int vd = p.vd;
            // 7 steps of the decay on top of 1 / f stay in range
            const bool gentle = g2 > -6.f;
            // lam^{|i-j|} over 8 columns before (after, reversed) the row = (its distance to the
            // near end of them) x (a column's distance to it); the latter here, in pairs
            uint64_t near[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                near[j] = rev ? two(exp2f(g2 * (float)(2 * j)), exp2f(g2 * (float)(2 * j + 1)))
                              : two(exp2f(g2 * (float)(7 - 2 * j)), exp2f(g2 * (float)(6 - 2 * j)));
            for (int i = 0; i < walk.tiles; ++i, ++it) {
                const int len = walk.len(i);
                // log2 of the row's f
                const float lf = fmaxf(g2 * (float)(rev ? max(len - 1 - row, 0) : row + 1), -64.f);
                if (!(ok = wait(&bar.s_full, it))) break;
                tc_fence_after();
                tmem_columns(lanes + kColS + 64 * half, 4, [&](int m, const uint32_t (&x)[16]) {
                    const int c0 = 64 * half + 16 * m;
                    const int d = rev ? c0 - row : row - c0;   // distance of column c0
                    uint32_t o[8];
                    // the row's pairs among the block's columns: from lo to hi - 1
                    const int lo = rev ? -d : 0, hi = rev ? len - c0 : d + 1;
                    if (rev ? c0 + 15 < 32 * rw || hi <= 0 : c0 > 32 * rw + 31) {   // none of the warp's rows has any
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] = 0;
                    } else if (gentle) {
                        // the distance to the near end may be negative: then so is the column's
                        // to what it is taken from, and their product is still a power >= 0
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float far = s_upd * exp2_approx(fmaf(g2, (float)(rev ? d + 8 * k : d - 7 - 8 * k), -lf));
                            const uint64_t far2 = two(far, far);
#pragma unroll
                            for (int j = 4 * k; j < 4 * k + 4; ++j)
                                o[j] = pack2(mul2((uint64_t)x[2 * j + 1] << 32 | x[2 * j], mul2(near[j & 3], far2)));
                        }
                        if (!__all_sync(kFull, lo <= 0 && hi >= 16))
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                o[j] &= (2 * j >= lo && 2 * j < hi ? 0xffffu : 0u) |
                                        (2 * j + 1 >= lo && 2 * j + 1 < hi ? 0xffff0000u : 0u);
                    } else {
                        const float l0 = fmaf(g2, (float)d, -lf), l1 = rev ? g2 : -g2;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float v[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                v[k] = s_upd * __uint_as_float(x[2 * j + k]) *
                                       exp2_approx(fmaf((float)(2 * j + k), l1, l0));
                            o[j] = pack2(v[0], v[1]) & ((2 * j >= lo && 2 * j < hi ? 0xffffu : 0u) |
                                                        (2 * j + 1 >= lo && 2 * j + 1 < hi ? 0xffff0000u : 0u));
                        }
                    }
                    tmem_st8(lanes + kColS + 64 * half + 8 * m, o);
                });
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_ready);
                if constexpr (!kNarrow) {
                    const float f = s_out * exp2_approx(lf);
                    if (!(ok = take_o(it, row, half * (vd / 2), vd / 32, lanes, f))) break;
                }
            }
            return ok;
        });
    } else if (kNarrow && warp >= 20) {
        // ---- outputs: thread = token row of the tile
        set_registers<kNarrow ? kRegsO : kRegsOther, false>();
        const int row = tid & 127;
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
        each_unit([&](const Unit &u) {
            const DecayPass &p = A.pass[u.pass];
            const Walk walk(u, p.rev);
            const float g2 = decay_log2(u.gd);
            for (int i = 0; i < walk.tiles; ++i, ++it) {
                const float lf = fmaxf(g2 * (float)(walk.rev ? max(walk.len(i) - 1 - row, 0) : row + 1), -64.f);
                if (!take_o(it, row, 0, 4, lanes, p.s_out * exp2_approx(lf))) return false;
            }
            return true;
        });
    } else if (warp < 12) {
        // ---- state: thread = value index (TMEM lane), whose row of S^T it keeps in registers
        set_registers<kRegsState, true>();
        const int e = tid & 127;
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
        each_unit([&](const Unit &u) {
            bool ok = true;
            const DecayPass &p = A.pass[u.pass];
            const Walk walk(u, p.rev);
            const float gd = u.gd;
            const int kd = p.kd;
            const bool any = e < p.vd;   // (by warps; the other lanes' sums are nobody's)
            if (u.tiles == 0) {   // an empty sequence: the state goes through
                if (u.to)
                    for (int d = e; d < kd * p.vd; d += 128) u.to[d] = u.in ? u.in[d] : 0.f;
                return true;
            }
            StateRow<kKd> s;
            state_load<kKd>(p, u.in, e, s);
            uint64_t fa = 0, fb = 0;   // factors of s over flen tokens: s fa + s fb
            int flen = -1;
            // the update of tile i (whose number is n): kv_full says it is complete
            auto update = [&](int i) {
                if (walk.len(i) != flen) {
                    flen = walk.len(i);
                    const DecayFactor f(gd * (float)flen);
                    fa = f.near1 ? two(1.f, 1.f) : two(f.f, f.f);
                    fb = f.near1 ? two(f.f, f.f) : 0;
                }
                if (any) state_add<true, kKd>(s, lanes + kColU, kd, fa, fb);
            };
            for (int i = 0; i < walk.tiles; ++i, ++it) {
                if (it && !(ok = wait(&bar.kv_full, it - 1))) break;
                tc_fence_after();
                if (i) update(i - 1);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.s_free);
                if (any) state_to_bf16<kKd>(s, smem + kOffH, e, kd);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.h_ready);
            }
            if (ok && u.to) {
                if (!(ok = wait(&bar.kv_full, it - 1))) return false;
                tc_fence_after();
                update(walk.tiles - 1);
                state_store<kKd>(p, u.to, e, s);
            }
            return ok;
        });
    } else {
        // ---- weighted values: thread = value index (TMEM lane); group grp takes every other
        // 16 tokens, its token l = 16 k + j being the tile's 16 (2 k + grp) + j
        set_registers<kRegsV, false>();
        const int grp = (warp - 12) >> 2, e = tid & 127;
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
        float *w = (float *)(smem + kOffW) + (warp - 12) * (kC / 2);
        each_unit([&](const Unit &u) {
            bool ok = true;
            const DecayPass &p = A.pass[u.pass];
            const Walk walk(u, p.rev);
            const float gd = u.gd, s_upd = p.s_upd;
            const bool any = e < p.vd;   // (by warps; the other lanes' sums are nobody's)
            int wlen = -1;   // tokens of the tile that the weights are for
            for (int i = 0; i < walk.tiles; ++i, ++it) {
                const uint32_t st = it % kStages;
                const int len = walk.len(i);
                if (len != wlen) {
                    __syncwarp();   // the last tile's weights are read
                    const int tok = 16 * (2 * (lane >> 4) + grp) + (lane & 15);
                    w[lane] = token_weight(tok, len, walk.rev, gd, s_upd, 0);
                    w[lane + 32] = token_weight(tok + 64, len, walk.rev, gd, s_upd, 0);
                    __syncwarp();
                    wlen = len;
                }
                if (!(ok = wait(&bar.full_bc[st], it / kStages))) break;
                uint8_t *ct = smem + st * kStageBytes + 2 * kTileBytes;
                if (len < kC) {   // the products with P and with S^ read these rows too
                    if (any) zero_columns(ct, e & ~31, len, lane);   // both groups the same zeros
                    zero_rows(ct - kTileBytes, p.kd, len, warp - 12, 8, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
#pragma unroll 1
                for (uint32_t k = 0; k < kParts; ++k) {
                    const uint32_t slot = k % kSlots, use = (it * kParts + k) / kSlots;
                    const uint32_t part = walk.rev ? kParts - 1 - k : k;
                    if (use && !(ok = wait(&bar.v_free[slot], use - 1))) break;
                    tc_fence_after();
                    if (any) {
                        write_terms(lanes + kColV + slot * kSlotCols + 8 * grp, ct, e, 2 * part + grp, w + 16 * part);
                        tmem_st_wait();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.v_ready[slot]);
                }
                if (!ok) break;
            }
            return ok;
        });
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
// Every write's weight is its distance to the segment's end, so the sum of C'^T B over the tiles
// needs no decay on the way.  Four groups of four warps take 32 tokens of a tile each, through
// slots of C' in TMEM of their own, one each or two (kNarrow); four more add a tile's product to the sum, which they keep in
// registers, while the next one's runs in the other accumulator.  262144 tokens of 16 heads, 19
// segments in up to 3 parts: 142 us, 4.4 TB/s.  A tile takes an SM 1.8 us, near the 1.6 that its
// copies need for 64 KB; the rest is units that do not come out even.
constexpr int kLocThreads = 32 * 24, kLocProducer = 20, kLocIssuer = 21;   // warps
constexpr int kLocMaxStages = 6;                             // 3 of 64 KB, or 6 of 32 (kNarrow)
constexpr uint32_t kLocOffBar = 3 * 2 * kTile;
constexpr uint32_t kLocOffW = kLocOffBar + kBarBytes;              // weights, a copy per warp
constexpr uint32_t kLocOffRing = kLocOffW + 16 * 32 * 4;
constexpr uint32_t kSmemLocal = kLocOffRing + kRing * sizeof(Unit);
constexpr uint32_t kLocMaxSlots = 8;
struct LocalBars {
    uint64_t u_full[kRing], u_free[kRing];   // a unit announced / done with (21 warps)
    uint64_t full[kLocMaxStages], free[kLocMaxStages];
    uint64_t v_ready[kLocMaxSlots], v_free[kLocMaxSlots];
    uint64_t sum_full[2], sum_free[2];   // a tile's sum complete / read (4 warps)
    uint64_t fin;
    uint32_t tmem;
    int stop;
};
static_assert(sizeof(LocalBars) <= kBarBytes, "barriers");

template <bool kNarrow>
__global__ void __launch_bounds__(kLocThreads, 1)
decay_local_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs A) {
    // TMEM columns: two accumulators, and slots of C'^T
    constexpr uint32_t kAcc = kNarrow ? 64 : kC, kLocColV = 2 * kAcc, kLocSlots = kNarrow ? 8 : 4;
    constexpr uint32_t kTileBytes = kNarrow ? kBox : kTile, kStageBytes = 2 * kTileBytes;   // B, C
    constexpr int kLocStages = kNarrow ? kLocMaxStages : 3;
    static_assert(kLocStages * kStageBytes <= kLocOffBar, "stages");
    constexpr int kKd = kNarrow ? 64 : kC;
    constexpr int kLocRegsV = kNarrow ? 72 : 64, kLocRegsState = kNarrow ? 120 : 176, kLocRegsOther = kNarrow ? 72 : 48;
    static_assert(4 * kLocRegsV + kLocRegsState + kLocRegsOther <= 6 * kRegsLaunch, "registers");
    // a group waits for every use of its slots: a parity tells one use from the one before, no further
    // (five slots between them were no faster)
    static_assert(kLocSlots % kParts == 0, "slots of one group each");
    static_assert(kLocSlots <= kLocMaxSlots && kLocColV + kLocSlots * kSlotCols <= kTmemCols, "TMEM");
    extern __shared__ __align__(1024) uint8_t smem[];
    LocalBars &bar = *(LocalBars *)(smem + kLocOffBar);
    Unit *ring = (Unit *)(smem + kLocOffRing);
    volatile int *stop = &bar.stop;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (!GDR_INBOUNDS((smem_u32(smem) & 1023u) == 0)) return;   // swizzled tiles start on 1 KB
    let_next_start();
    if (tid == 0) {
        for (uint32_t i = 0; i < kRing; ++i) {
            mbar_init(&bar.u_full[i], 1);
            mbar_init(&bar.u_free[i], 21);
        }
        for (int i = 0; i < kLocStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.free[i], 1);
        }
        for (uint32_t i = 0; i < kLocSlots; ++i) {
            mbar_init(&bar.v_ready[i], 4);
            mbar_init(&bar.v_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.sum_full[i], 1);
            mbar_init(&bar.sum_free[i], 4);
        }
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
    after_previous();
    const uint32_t tm = bar.tmem;
    auto wait = [&](uint64_t *b, uint32_t use) { return wait_use(b, use, A.wait_ns, stop, A.status); };
    uint32_t it = 0;   // tiles so far
    // Walks the announced units (every warp but the producer): f(unit) until the end or until
    // it returns false.
    auto each_unit = [&](auto &&f) {
        for (uint32_t k = 0;; ++k) {
            if (!wait(&bar.u_full[k % kRing], k / kRing)) return;
            const Unit &u = ring[k % kRing];
            if (u.tiles < 0 || !f(u)) return;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.u_free[k % kRing]);
        }
    };

    if (warp >= kLocProducer) {
        set_registers<kLocRegsOther, false>();
        if (warp == kLocProducer) {
            bool ok = true;
            int64_t n = (int64_t)blockIdx.x - gridDim.x;
            for (uint32_t k = 0; ok; ++k) {
                Unit u;
                if (!take_unit<kLocal>(A, n, u)) u.tiles = -1;
                if (k >= kRing && !(ok = wait(&bar.u_free[k % kRing], k / kRing - 1))) break;
                if (lane == 0) {
                    ring[k % kRing] = u;
                    mbar_arrive(&bar.u_full[k % kRing]);
                }
                __syncwarp();
                if (u.tiles < 0) break;
                const DecayPass &p = A.pass[u.pass];
                const Walk walk(u, p.rev);
                const int kd = p.kd, vd = p.vd;
                for (int i = 0; i < walk.tiles; ++i, ++it) {
                    const uint32_t st = it % kLocStages, use = it / kLocStages;
                    if (use && !(ok = wait(&bar.free[st], use - 1))) break;
                    if (lane == 0) {
                        const int64_t t = walk.first(u, i);
                        uint8_t *s = smem + st * kStageBytes;
                        mbar_arrive_expect_tx(&bar.full[st], (kd + vd) / 64 * kBox);
                        load_tile(s, &maps.b[u.pass], kd, u.h, t, &bar.full[st]);
                        load_tile(s + kTileBytes, &maps.c[u.pass], vd, u.h, t, &bar.full[st]);
                    }
                    __syncwarp();
                }
            }
            for (uint32_t k = it >= kLocStages ? it - kLocStages : 0; k < it; ++k)
                __all_sync(kFull, mbar_wait(&bar.full[k % kLocStages], (k / kLocStages) & 1u, kDrainNs));
        } else if (warp == kLocIssuer) {
            const uint32_t s0 = smem_u32(smem);
            const bool lead = elect_one();
            each_unit([&](const Unit &u) {
                bool ok = true;
                if (u.tiles == 0) return true;
                const DecayPass &p = A.pass[u.pass];
                const Walk walk(u, p.rev);
                const int kd = p.kd;
                const uint32_t id_h = instr_desc(kC, kd, 1, false, true);
                for (int i = 0; i < walk.tiles; ++i, ++it) {
                    const uint32_t st = it % kLocStages, buf = it & 1;
                    const int len = walk.len(i);
                    if (!(ok = wait(&bar.full[st], it / kLocStages))) break;
                    if (len < kC) {
                        zero_rows(smem + st * kStageBytes, kd, len, 0, 1, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (it >= 2 && !(ok = wait(&bar.sum_free[buf], (it >> 1) - 1))) break;
                    tc_fence_after();
                    const uint64_t dBt = smem_desc(s0 + st * kStageBytes, kBox, 1024, kSw128);
#pragma unroll
                    for (uint32_t k = 0; k < kParts; ++k) {
                        const uint32_t n = it * kParts + k, slot = n % kLocSlots, av = tm + kLocColV + slot * kSlotCols;
                        const uint64_t dPart = dBt + (((p.rev ? kParts - 1 - k : k) * 4096) >> 4);
                        if (!(ok = wait(&bar.v_ready[slot], n / kLocSlots))) break;
                        tc_fence_after();
#pragma unroll
                        for (uint32_t term = 0; term < 3; ++term)
#pragma unroll
                            for (uint32_t j = 0; j < 2; ++j)
                                mma_f16_ts_if(lead, tm + buf * kAcc, av + (2 - term) * 16 + j * 8, dPart + ((j * 2048) >> 4),
                                              id_h, k + term + j > 0);
                        mma_commit_if(lead, &bar.v_free[slot]);
                    }
                    if (!ok) break;
                    mma_commit_if(lead, &bar.free[st]);
                    mma_commit_if(lead, &bar.sum_full[buf]);
                }
                return ok;
            });
            mma_commit_if(lead, &bar.fin);
            __all_sync(kFull, mbar_wait(&bar.fin, 0, kDrainNs));
        }
    } else if (warp < 16) {
        // ---- weighted values: thread = value index (TMEM lane), group grp the tile's 32 tokens that
        // the issuer takes as its grp-th part: forward and reversed units alike, so that its slots
        // stay its own
        set_registers<kLocRegsV, false>();
        const int grp = warp >> 2, e = tid & 127;
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
        float *w = (float *)(smem + kLocOffW) + warp * 32;
        each_unit([&](const Unit &u) {
            bool ok = true;
            const DecayPass &p = A.pass[u.pass];
            const bool rev = p.rev;
            const Walk walk(u, rev);
            const int part = rev ? (int)kParts - 1 - grp : grp;   // from token 32 part on
            const float gd = u.gd, s_upd = p.s_upd;
            const int64_t tokens = u.t1 - u.t0;
            const bool any = e < p.vd;   // (by warps; the other lanes' sums are nobody's)
            for (int i = 0; i < walk.tiles; ++i, ++it) {
                const uint32_t st = it % kLocStages;
                const uint32_t n = it * kParts + grp;   // in the issuer's order
                const uint32_t slot = n % kLocSlots, use = n / kLocSlots;
                const int len = walk.len(i);
                // past the tile: its distance to the segment's end (its start, reversed)
                const int64_t past = u.past + (rev ? (int64_t)(walk.tiles - 1 - i) * kC : tokens - (int64_t)i * kC - len);
                __syncwarp();   // the last tile's weights are read
                w[lane] = token_weight(32 * part + lane, len, rev, gd, s_upd, past);
                __syncwarp();
                if (!(ok = wait(&bar.full[st], it / kLocStages))) break;
                if (use && !(ok = wait(&bar.v_free[slot], use - 1))) break;
                tc_fence_after();
                uint8_t *ct = smem + st * kStageBytes + kTileBytes;
                if (len < kC && any) {   // all groups the same zeros
                    zero_columns(ct, e & ~31, len, lane);
                    fence_proxy_async_smem();   // before the stage's next tile is copied over them
                    __syncwarp();
                }
#pragma unroll 1
                for (uint32_t k = 0; k < 2; ++k)
                    if (any) write_terms(lanes + kLocColV + slot * kSlotCols + 8 * k, ct, e, 2 * part + k, w + 16 * k);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.v_ready[slot]);
            }
            return ok;
        });
    } else {
        // ---- sums: thread = value index (TMEM lane), whose row it keeps in registers
        set_registers<kLocRegsState, true>();
        const int e = tid & 127;
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
        each_unit([&](const Unit &u) {
            const DecayPass &p = A.pass[u.pass];
            const bool any = e < p.vd;   // (by warps; the other lanes' sums are nobody's)
            StateRow<kKd> s;
#pragma unroll
            for (int j = 0; j < kKd / 2; ++j) s[j] = 0;
            for (int i = 0; i < u.tiles; ++i, ++it) {
                const uint32_t buf = it & 1;
                if (!wait(&bar.sum_full[buf], it >> 1)) return false;
                tc_fence_after();
                if (any) state_add<false, kKd>(s, lanes + buf * kAcc, p.kd, 0, 0);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.sum_free[buf]);
            }
            state_store<kKd>(p, u.to, e, s);
            return true;
        });
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, kTmemCols);
    }
}

}  // namespace

cudaError_t launch_decay_tc(const DecayGeom &g, const DecayPass *passes, int n, int sms, unsigned long long *next,
                            bool early, int *status, cudaStream_t stream, bool again) {
    if (n < 1 || n > kMaxPasses) return cudaErrorInvalidValue;
    const bool local = passes[0].local;
    TcMaps maps{};
    TcArgs args{};
    for (int i = 0; i < n; ++i) {
        const DecayPass &p = passes[i];
        const bool ok = tc_make_tile_map(&maps.b[i], p.b, p.kd, g.H, g.T_total, kC) &&
                        tc_make_tile_map(&maps.c[i], p.c, p.vd, g.H, g.T_total, kC) &&
                        (local || (tc_make_tile_map(&maps.a[i], p.a, p.kd, g.H, g.T_total, kC) &&
                                   tc_make_tile_map(&maps.o[i], p.out, p.vd, g.H, g.T_total, kC)));
        if (!ok) return cudaErrorNotSupported;
        args.pass[i] = p;
    }
    args.g = g;
    args.npass = n;
    args.units = (again ? g.N : g.max_segs) * g.H * n * (local ? g.parts : 1);
    args.next = next;
    args.long_first = next && args.units <= 64 * (int64_t)sms;   // a look at a unit costs some 0.3 us
    args.status = status;
    args.wait_ns = kWaitNs;
    if (const char *w = std::getenv("GDR_TC_WAIT_NS")) {   // test hook: shorter pipeline waits
        const long long x = std::atoll(w);
        if (x >= 0 && (uint64_t)x < kWaitNs) args.wait_ns = (uint64_t)x;
    }
    if (args.units == 0) return cudaSuccess;
    if (args.units > 0x7fffffff) return cudaErrorInvalidValue;
    bool narrow = true;
    for (int i = 0; i < n; ++i) narrow &= passes[i].kd == 64 && passes[i].vd == 64;
    using Kernel = void (*)(TcMaps, TcArgs);
    static constexpr Kernel kernels[2][3] = {
        {decay_out_kernel<false, kOut>, decay_out_kernel<false, kAgain>, decay_local_kernel<false>},
        {decay_out_kernel<true, kOut>, decay_out_kernel<true, kAgain>, decay_local_kernel<true>}};
    const Kernel kern = kernels[narrow][local ? kLocal : again ? kAgain : kOut];
    const int bytes = (int)(local ? kSmemLocal : kSmemOut);
    // the kernels' split of the registers is made for this many a thread
    static const bool split = [] {
        bool all = true;
        for (int n = 0; n < 2; ++n)
            for (int k = 0; k < 3; ++k) {
                cudaFuncAttributes a{};
                all &= cudaFuncGetAttributes(&a, kernels[n][k]) == cudaSuccess &&
                       a.numRegs >= (n && k != kLocal ? kRegsLaunchNarrow : kRegsLaunch);
            }
        return all;
    }();
    if (!split) return cudaErrorInvalidConfiguration;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != cudaSuccess) return err;
    ProfScope prof(stream, local ? "decay_local_kernel" : again ? "decay_out_kernel (again)" : "decay_out_kernel");
    const cudaError_t run = launch_early(early, kern, dim3((unsigned)std::min<int64_t>(args.units, sms)),
                                         local ? kLocThreads : 32 * (narrow ? kOutWarpsNarrow : kOutWarps), (size_t)bytes, stream, maps, args);
    count_launch();
    return run;
}

}  // namespace gdr
