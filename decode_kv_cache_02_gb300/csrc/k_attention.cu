// k_attention.cu -- attention of a few new tokens over a paged cache, bf16,
// fp32 or held in 4 or 8 bits: out = softmax(scale * q K^T) V for each KV head's
// group of query heads.
//
// One pass over the cache with a running maximum and sum.  The rows of all
// sequences and KV heads form one line of units (64 or 128 rows), cut into
// equal runs, one per block, as many blocks as the SMs hold at once: ragged
// batches are balanced whatever their lengths, and at most two pieces a block
// are parts of a sequence that attn_combine_kernel joins.  A few short sequences
// take a cluster of blocks per problem instead, which join through their shared
// memory: one launch.  Within a piece every
// warp is on its own: it takes every fourth stage, copies it into its own ring
// of shared memory (cp.async through the block table, rows past the sequence
// filled with zeros), and keeps the maxima, sums and the output of up to 32
// queries in registers; the warps meet at the piece's end.
//
// The cache is read once, so the kernel is bound by HBM; the two products run
// on mma.sync m16n8k16 with the keys (values: the head's dimensions) as the
// 16 rows and the queries as the 8 columns, S^T = K Q^T and O^T = V^T P^T: a
// group of up to 8 queries then wastes nothing, the operands come from shared
// memory in the order the fragments want (the order of the contracted index is
// free as long as both sides share it), and P^T turns from an accumulator into
// an operand with one movmatrix per 8 x 8.  (tcgen05 would need 64 or 128
// keys a step and the probabilities through tensor memory, between warps; at 8
// to 32 queries a row the tensor pipe is a seventh to a third busy as it is.)
//
// 4 bits: codes become fp16 numbers exactly: K as they lie, c * 2^-24 or c *
// 2^-20 (half a shift and a logic op for two), against queries brought to fp16 by
// a power of two a row; V c - 8 (an FMA more).  A group's scale applies to its
// own accumulator (K) or to the probabilities (V), in fp32.  The groups' low
// values enter through one more product each: (scale, low) as stored against (0,
// 1) times the queries' sums over the group, those in three bf16 parts (K); low
// and scale against the probabilities (V).  So the products are exact up to the
// rounding of p * scale to fp16 and, for the lows, of p (kTwoQueries); a query's
// elements below 2^-27 of its row's largest are off by up to 2^-35 of that.  What
// the fp16 steps are relative to is the query's own (kSpread).
//
// 8 bits: codes become bf16 numbers exactly (bytes_as_bf16), K's scale meets the logit and
// V's the probability in fp32; the rest is the bf16 cache's.
//
// The running maximum moves only when a logit passes it by more than 8 (log2):
// p stays below 2^8 and the rescaling almost never runs.  (4 bits: by more than 4.)
//
// Measured (one GB300, KV heads 8): 64 ragged sequences to 4224 rows, G = 5,
// head_dim 128: 91.8 us, 6.2 TB/s; 256 of 1152, G = 4: 183 us, 6.6 TB/s; 16 ragged
// to 16389 with 8 new tokens, head_dim 64: 61.0 us, 5.1 TB/s (copies alone, before
// its launch overlapped what was there: 55); one of 1152: 6.1 us.  4 bits: one
// of 131071, G = 5: 47.0 us, 3.6 TB/s.  In steady state a warp spends 379 instructions
// and an SM quarter 592 cycles on 16 rows, where HBM's rate would allow 435: no pipe is
// above 55 in a hundred of them (logic; issue slots 64), the twelve warps of an SM
// wait for their own last instructions.  8 bits: the same 64 sequences 59.0 us, 5.0 TB/s;
// one of 131071, G = 8: 53.8 us, 5.2 TB/s: 432 instructions for 16 rows, some 240 of them, counted by hand,
// codes to bf16 and both operands' order, where HBM's rate would allow 720 cycles: logic 54
// in a hundred, issue slots 52 (three stages at two blocks an SM: 62.6 and 53.3).
#include <cuda_fp16.h>
#include <float.h>

#include "rkv_common.cuh"
#include "rkv_internal.h"

namespace rkv {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -FLT_MAX, kUnset = 1e30f;  // no maximum yet
constexpr float kHuge = 0x1p20f;

// Bytes and rows of one stage of a warp's ring.
template <int D, int BITS>
struct Stage {
    static constexpr bool Q4 = BITS == 4, Q8 = BITS == 8;
    static constexpr int W = D / 32;
    static constexpr int KEYS = BITS ? 32 : (D == 128 ? 16 : 32);
    // one stage in flight is enough where a stage is 5 KB of long arithmetic (4
    // bits, head_dim 128: 48.5 us against 49.7 with two, one of 131071; 84.8
    // against 86.5, 64 of 4224), not for bf16 (256 of 1152: 184 us with two, 189)
    static constexpr int DEPTH = BITS ? 2 : 3;
    static constexpr int ROW = Q4 ? D / 2 : (Q8 ? D : D * 2);
    static constexpr int SROW = Q4 ? W * 4 : (Q8 ? 4 : 0);
    static constexpr int V = KEYS * ROW;
    static constexpr int ks() { return 2 * KEYS * ROW; }
    static constexpr int vs() { return ks() + KEYS * SROW; }
    static constexpr int BYTES = 2 * KEYS * (ROW + SROW);
};
template <int D>
struct Stage32 {
    static constexpr int KEYS = 16, DEPTH = 2, ROW = D * 4, V = KEYS * ROW, BYTES = 2 * V;
};

// 4 bits: a probability times a scale goes to fp16, which holds 2^-14 .. 2^15 with
// eleven bits.  So each query's sums are relative to its largest probability times
// 2^e, e the exponent of the row's V (its largest |scale| or |low| is below 2^e), which
// kAbove and kSlack keep between 2^11 and 2^15: what a row holds that the query
// gives no weight, or does not see, counts nothing.  Where a row's groups are
// no further apart than 2^kSpread (in bf16 bits), every group then has its largest
// product above 2^2, and what fp16 cuts off below 2^-25 is 2^-24 of the group's
// numbers a row, as much as an fp32 sum loses.  From a row on whose groups
// are further apart (zeros, say), or whose exponent is not within kLeast ..
// kMost, the queries that see it take the products in two bf16 parts, at any size.
// (kMost - kLeast leaves the exponentials that join the warps' sums 2^-30 above what
// they flush.)
constexpr float kSlack = 4.f, kAbove = 11.f;
constexpr uint32_t kSpread = 8 << 7;
constexpr int kLeast = -40, kMost = 56;

// The probabilities meet a bf16 V, and the lows of a 4-bit one, as two bf16 parts
// (TWO), 2^-16 of them off (one part: 2^-8), where a KV head has up to 16 queries, so
// that the rows are read once and waited for: that costs hardly anything (us, one
// part against two: 64 ragged of 4224 92.5 / 92.6, 256 of 1152 182.4 / 183.6, 16
// queries at head_dim 128 91.3 / 93.2, 4 bits 46.6 / 47.2).  With more queries the
// products count: 8 new tokens at head_dim 64 58.5 / 65.7, at 128 99.7 / 120.7, 64 of
// them 2550 / 3197, and one part stays.
constexpr int kTwoQueries = 16;

struct Params {
    const uint8_t* k;
    const uint8_t* v;
    const uint8_t* ks;
    const uint8_t* vs;
    const int32_t* table;
    const int32_t* lens;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    int num_seqs;
    int64_t q_seq, q_tok, q_head, o_seq, o_tok, o_head;
    float* lse;
    float* raw;         // (see AttnArgs)
    float* raw_ml;
    float* partial;     // [slot][rows][D]
    float* partial_ml;  // [slot][rows][2]
    int4* joins;        // [run][group]: (sequence, head, parts) of the problem to join, if parts
    int H, G, T, R, groups, runs, max_rows;
    uint32_t lead;
    int cluster;  // blocks of a cluster that share a problem (0: runs of the line)
    int max_blocks, log2bs, num_blocks;
    float scale, slack;  // of base-2 logits, positive; how far they may pass the maximum
    uint32_t flip;       // scale < 0: sign bits for the queries
    DeviceStatus* status;
};

RKV_DEV uint32_t smem_at(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
RKV_DEV void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
RKV_DEV void cp16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
}
RKV_DEV void cp4(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 4 : 0)
                 : "memory");
}
RKV_DEV void cp8(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 8 : 0)
                 : "memory");
}
// Shared loads by 32-bit address, in program order with the waits and copies.
RKV_DEV uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}
RKV_DEV uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
RKV_DEV uint32_t lds4(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
RKV_DEV uint32_t lds2(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
// Two 8 x 8 matrices of 16-bit values, rows of 16 bytes at the addresses of lanes
// 0 .. 7 and 8 .. 15, as a fragment; transposed.
RKV_DEV void ldm2(uint32_t (&r)[2], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(a));
}
RKV_DEV void ldm2t(uint32_t (&r)[2], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(a));
}
RKV_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
RKV_DEV void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
RKV_DEV void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                 uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
RKV_DEV void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                     uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
RKV_DEV uint32_t pack_f16(float lo, float hi) {
    const __half2 b = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
RKV_DEV uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
RKV_DEV uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
RKV_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The constants of the unpacking, held in registers: an instruction takes one
// immediate, and each of these steps wants two.  (up: a bf16 becomes fp32 by a
// product with 2^16, which leaves the shifting pipe, the busiest, to others: 64
// sequences of 4224 82.3 -> 81.3 us.)
struct Unpack {
    uint32_t even, odd, half, less, sixteenth, less16;  // V's codes
    uint32_t up;                                        // scales
};
RKV_DEV Unpack unpack_constants() {
    Unpack k;
    asm volatile("mov.b32 %0, 0x000f000f;" : "=r"(k.even));
    asm volatile("mov.b32 %0, 0x00010000;" : "=r"(k.up));
    asm volatile("mov.b32 %0, 0x00f000f0;" : "=r"(k.odd));
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(k.half));       // fp16 1024, 1024
    asm volatile("mov.b32 %0, 0xe408e408;" : "=r"(k.less));       // -1032, -1032
    asm volatile("mov.b32 %0, 0x2c002c00;" : "=r"(k.sixteenth));  // 1/16, 1/16
    asm volatile("mov.b32 %0, 0xd480d480;" : "=r"(k.less16));     // -72, -72
    return k;
}
RKV_DEV uint32_t and_or(uint32_t x, uint32_t mask, uint32_t magic) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "r"(mask), "r"(magic));
    return y;
}
// A word's eight codes as fp16 numbers, exactly, as they lie: bits 0..3 of a half
// are c * 2^-24 (subnormal), bits 4..7 c * 2^-20.  The kernel is bound by such
// logic (against bf16 128 + c, three shifts a word and a constant to subtract:
// one sequence of 131071 49.2 -> 47.5 us, 256 of 1152 102.8 -> 99.3).
RKV_DEV void codes_of(uint32_t w, uint32_t (&c)[4]) {
    const uint32_t x = w >> 8;
    c[0] = w & 0x000f000fu;
    c[1] = w & 0x00f000f0u;
    c[2] = x & 0x000f000fu;
    c[3] = x & 0x00f000f0u;
}
RKV_DEV float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 .. 127
RKV_DEV __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
// Codes i and i + 4 less 8 as fp16, exactly: 1024 + c, or, four bits higher,
// 1024 + 16 c, so that a word takes one shift.  The values' product wants codes
// around zero (long sums carry no constant that the tensor core's accumulator
// would cut digits for) and fp16 for the probabilities' eleven bits.
RKV_DEV void centred(const Unpack& k, uint32_t w, uint32_t (&c)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t x = i ? w >> 8 : w;
        const __half2 lo = __hadd2(as_half2(and_or(x, k.even, k.half)), as_half2(k.less));
        const __half2 hi = __hfma2(as_half2(and_or(x, k.odd, k.half)), as_half2(k.sixteenth),
                                   as_half2(k.less16));
        c[2 * i] = *reinterpret_cast<const uint32_t*>(&lo);
        c[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&hi);
    }
}

// Small whole numbers in fp16 as bf16.
RKV_DEV uint32_t f16_as_bf16(uint32_t x) {
    const float2 f = __half22float2(as_half2(x));
    return pack(f.x, f.y);
}
// What bf16 leaves of two numbers, as bf16: h is pack(lo, hi).
RKV_DEV uint32_t pack_rest(float lo, float hi, uint32_t h) {
    return pack(lo - __uint_as_float(h << 16), hi - __uint_as_float(h & 0xffff0000u));
}

// Physical row (within 16) of row r of a key fragment.  Quarter-warp reads of
// K (two rows) and half-warp reads of V (four rows) then meet no bank twice,
// with the 16-byte units of a row permuted by unit_xor.
template <int BITS>
RKV_DEV int phys(int r) {
    if constexpr (BITS != 0) return r ^ ((r >> 1) & 1);
    return (r & 8) | ((r & 7) >> 1) | ((r & 1) << 2);
}
template <int D, int BITS>
RKV_DEV int unit_xor(int row) {
    if constexpr (BITS == 4) return D == 128 ? ((row >> 2) & 1) << 1 : 0;
    if constexpr (BITS == 8)
        return D == 128 ? (row & 6) ^ ((row & 1) << 2) : ((row >> 2) & 1) << 1;
    return ((row & 3) << 1) ^ (((row >> 2) & 1) << 2);
}

constexpr uint32_t kNoRow = 0xffffffffu;

// Copies the rows of a stage; lane i holds the pool row of row i (kNoRow:
// zeros; full: there are none).
template <int D, int BITS>
RKV_DEV void copy_stage(const Params& p, uint32_t dst, uint32_t mine, bool full) {
    using S = Stage<D, BITS>;
    const int lane = threadIdx.x & 31;
    constexpr int UPR = S::ROW / 16;  // units per row
    const int u = lane % UPR;
    const uint8_t* k = p.k + u * 16;
    const uint8_t* v = p.v + u * 16;
    if (full) {
#pragma unroll
        for (int i = 0; i < S::KEYS * UPR / 32; ++i) {
            const int r = i * (32 / UPR) + lane / UPR;
            const uint64_t at = (uint64_t)__shfl_sync(0xffffffffu, mine, r) * S::ROW;
            const uint32_t to = dst + r * S::ROW + ((u ^ unit_xor<D, BITS>(r)) << 4);
            cp16(to, k + at);
            cp16(to + S::V, v + at);
        }
    } else {
#pragma unroll
        for (int i = 0; i < S::KEYS * UPR / 32; ++i) {
            const int r = i * (32 / UPR) + lane / UPR;
            const uint32_t row = __shfl_sync(0xffffffffu, mine, r);
            const bool ok = row != kNoRow;
            const uint64_t at = (uint64_t)(ok ? row : 0u) * S::ROW;
            const uint32_t to = dst + r * S::ROW + ((u ^ unit_xor<D, BITS>(r)) << 4);
            cp16(to, k + at, ok);
            cp16(to + S::V, v + at, ok);
        }
    }
    if constexpr (BITS != 0) {
        static_assert(S::KEYS == 32, "one lane per row");
        const bool ok = mine != kNoRow;
        const uint64_t at = (uint64_t)(ok ? mine : 0u) * S::SROW;
        const uint32_t to = dst + lane * S::SROW;
        if constexpr (S::SROW == 16) {
            cp16(to + S::ks(), p.ks + at, ok);
            cp16(to + S::vs(), p.vs + at, ok);
        } else if constexpr (S::SROW == 4) {
            cp4(to + S::ks(), p.ks + at, ok);
            cp4(to + S::vs(), p.vs + at, ok);
        } else {
            cp8(to + S::ks(), p.ks + at, ok);
            cp8(to + S::vs(), p.vs + at, ok);
        }
    }
}

// q . k of 16 keys of a bf16 stage.
template <int D, int NT>
RKV_DEV void logits_bf16(uint32_t st, int base, const uint32_t (&qf)[NT][D / 8],
                         float (&c)[NT][4]) {
    using S = Stage<D, 0>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int pr = base + phys<0>(g), f = unit_xor<D, 0>(pr);
    const uint32_t row = st + pr * S::ROW;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] = 0.f;
#pragma unroll
    for (int ch = 0; ch < S::W; ++ch) {
        const int at = ((4 * ch + t) ^ f) << 4;
        const uint4 a = lds16(row + at);
        const uint4 b = lds16(row + 8 * S::ROW + at);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mma(c[n], a.x, b.x, a.y, b.y, qf[n][4 * ch], qf[n][4 * ch + 1]);
            mma(c[n], a.z, b.z, a.w, b.w, qf[n][4 * ch + 2], qf[n][4 * ch + 3]);
        }
    }
}

// An 8-bit cache's codes as bf16 numbers, exactly: bytes 0 and 2 of a word.  128 + c's
// low seven bits lie in the mantissa as they are, and the sign (-128) is in the 128
// or 256 that is taken away: two logic operations and a subtraction for two codes,
// where a conversion through integers takes six.  Constants in registers, as below.
struct Bytes {
    uint32_t low, sign, base;
};
RKV_DEV Bytes byte_constants() {
    Bytes k;
    asm volatile("mov.b32 %0, 0x007f007f;" : "=r"(k.low));
    asm volatile("mov.b32 %0, 0x00800080;" : "=r"(k.sign));
    asm volatile("mov.b32 %0, 0x43004300;" : "=r"(k.base));  // bf16 128, 128
    return k;
}
RKV_DEV uint32_t bytes_as_bf16(const Bytes& k, uint32_t w) {
    const uint32_t a = and_or(w, k.low, k.base), b = and_or(w, k.sign, k.base);
    const __nv_bfloat162 c = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&c);
}

// q . k of 16 keys of an 8-bit stage; lane (g, t) holds values 64 ch + 16 t .. of its
// keys, byte pairs (0, 2) and (1, 3) of a word as neighbours.
template <int D, int NT>
RKV_DEV void logits_q8(const Bytes& bk, uint32_t st, int base, const uint32_t (&qf)[NT][D / 8],
                       float (&c)[NT][4]) {
    using S = Stage<D, 8>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int pr = base + phys<8>(g), f = unit_xor<D, 8>(pr);
    const uint32_t row = st + pr * S::ROW;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] = 0.f;
#pragma unroll
    for (int ch = 0; ch < D / 64; ++ch) {
        const int at = ((4 * ch + t) ^ f) << 4;
        const uint4 a = lds16(row + at);
        const uint4 b = lds16(row + 8 * S::ROW + at);
        const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = bytes_as_bf16(bk, x[w]), a2 = bytes_as_bf16(bk, x[w] >> 8);
            const uint32_t a1 = bytes_as_bf16(bk, y[w]), a3 = bytes_as_bf16(bk, y[w] >> 8);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                mma(c[n], a0, a1, a2, a3, qf[n][8 * ch + 2 * w], qf[n][8 * ch + 2 * w + 1]);
        }
    }
    const float s0 = __uint_as_float(lds4(st + S::ks() + pr * 4));
    const float s1 = __uint_as_float(lds4(st + S::ks() + (pr + 8) * 4));
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] *= i < 2 ? s0 : s1;
}

// O^T += V^T P^T for 16 keys of an 8-bit stage (the scales are in P).  Lane (g, t)
// holds values D / 8 * g .. of its keys; accumulator e stands for values 2 e and
// 2 e + 1 of them.
template <int D, int NT, bool TWO>
RKV_DEV void values_q8(const Bytes& bk, uint32_t st, int base, const uint32_t (&pb)[NT][2],
                       const uint32_t (&pr)[NT][2], float (&o)[D / 16][NT][4]) {
    using S = Stage<D, 8>;
    constexpr int WORDS = D / 32;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint32_t x[4][WORDS];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = base + phys<8>(2 * t + (k & 1) + 8 * (k >> 1));
        const uint32_t row = st + S::V + r * S::ROW;
        if constexpr (D == 128) {
            const uint4 y = lds16(row + ((g ^ unit_xor<D, 8>(r)) << 4));
            x[k][0] = y.x; x[k][1] = y.y; x[k][2] = y.z; x[k][3] = y.w;
        } else {
            const uint2 y = lds8(row + (((g >> 1) ^ unit_xor<D, 8>(r)) << 4) + ((g & 1) << 3));
            x[k][0] = y.x; x[k][1] = y.y;
        }
    }
#pragma unroll
    for (int e = 0; e < D / 16; ++e) {
        const uint32_t sel = (e & 1) ? 0x7632 : 0x5410;
        const uint32_t u = __byte_perm(x[0][e >> 1], x[1][e >> 1], sel);
        const uint32_t v = __byte_perm(x[2][e >> 1], x[3][e >> 1], sel);
        const uint32_t a0 = bytes_as_bf16(bk, u), a1 = bytes_as_bf16(bk, u >> 8);
        const uint32_t a2 = bytes_as_bf16(bk, v), a3 = bytes_as_bf16(bk, v >> 8);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mma(o[e][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            if constexpr (TWO) mma(o[e][n], a0, a1, a2, a3, pr[n][0], pr[n][1]);
        }
    }
}

// Where the scales of row lane % 16 of the 16 keys from base on lie (head_dim
// 128: 16 bytes a row).
RKV_DEV int scale_row(int base) {
    const int lane = threadIdx.x & 31;
    return (base + phys<4>(lane & 7) + (lane & 8)) * 16;
}

// The same for a 4-bit stage: sum over groups of scale * (q . c), and (scale,
// low) against qb (the parts of (0, 1) * sum of q over the group).
template <int D, int NT>
RKV_DEV void logits_q4(const Unpack& uk, uint32_t st, int base, const uint32_t (&qf)[NT][D / 8],
                       const uint32_t (&qb)[NT][3], float (&c)[NT][4]) {
    using S = Stage<D, 4>;
    constexpr int W = S::W;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int pr = base + phys<4>(g), f = unit_xor<D, 4>(pr);
    uint32_t word[2][W], sc[2][W], own[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t row = st + (pr + 8 * k) * S::ROW;
        const uint32_t srow = st + S::ks() + (pr + 8 * k) * S::SROW;
        if constexpr (W == 4) {
            const uint4 x = lds16(row + ((t ^ f) << 4));
            word[k][0] = __byte_perm(x.x, x.z, 0x5410);
            word[k][1] = __byte_perm(x.x, x.z, 0x7632);
            word[k][2] = __byte_perm(x.y, x.w, 0x5410);
            word[k][3] = __byte_perm(x.y, x.w, 0x7632);
            const uint4 y = lds16(srow);
            sc[k][0] = y.x; sc[k][1] = y.y; sc[k][2] = y.z; sc[k][3] = y.w;
        } else {
            const uint2 x = lds8(row + t * 8);
            word[k][0] = __byte_perm(x.x, x.y, 0x5410);
            word[k][1] = __byte_perm(x.x, x.y, 0x7632);
            const uint2 y = lds8(srow);
            sc[k][0] = y.x; sc[k][1] = y.y;
            own[k] = t == 0 ? y.x : (t == 1 ? y.y : 0u);
        }
    }
    if constexpr (W == 4) ldm2(own, st + S::ks() + scale_row(base));
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] = 0.f;
        mma(c[n], own[0], own[1], own[0], own[1], qb[n][0], qb[n][1]);
        mma(c[n], own[0], own[1], 0u, 0u, qb[n][2], 0u);
    }
#pragma unroll
    for (int w = 0; w < W; ++w) {
        uint32_t a[4], b[4];
        codes_of(word[0][w], a);
        codes_of(word[1][w], b);
        const float s[2] = {__uint_as_float(sc[0][w] * uk.up), __uint_as_float(sc[1][w] * uk.up)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(x, a[0], b[0], a[1], b[1], qf[n][4 * w], qf[n][4 * w + 1]);
            mma_f16(x, a[2], b[2], a[3], b[3], qf[n][4 * w + 2], qf[n][4 * w + 3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) c[n][i] = fmaf(s[i >> 1], x[i], c[n][i]);
        }
    }
}

// O^T += V^T P^T for 16 keys of a bf16 stage; pb: P^T as operand, pr: what bf16
// leaves of it (TWO).  ONE: only for the queries (columns) in `cols` (bit
// 2 n + i), with the key pairs (2t, 2t+1) and (2t+8, 2t+9) masked by keep0 and
// keep1 (a half each).
template <int D, int NT, bool TWO, bool ONE>
RKV_DEV void values_bf16(uint32_t st, int base, const uint32_t (&pb)[NT][2],
                         const uint32_t (&pr)[NT][2], uint32_t keep0, uint32_t keep1,
                         uint32_t cols, float (&o)[D / 16][NT][4]) {
    using S = Stage<D, 0>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t v = st + S::V;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int pr = base + phys<0>(2 * t + (k & 1) + 8 * (k >> 1));
            x[k] = lds16(v + pr * S::ROW + (((8 * j + g) ^ unit_xor<D, 0>(pr)) << 4));
        }
        const uint32_t w[4][4] = {{x[0].x, x[0].y, x[0].z, x[0].w}, {x[1].x, x[1].y, x[1].z, x[1].w},
                                  {x[2].x, x[2].y, x[2].z, x[2].w}, {x[3].x, x[3].y, x[3].z, x[3].w}};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t a0 = __byte_perm(w[0][e], w[1][e], 0x5410);
            uint32_t a1 = __byte_perm(w[0][e], w[1][e], 0x7632);
            uint32_t a2 = __byte_perm(w[2][e], w[3][e], 0x5410);
            uint32_t a3 = __byte_perm(w[2][e], w[3][e], 0x7632);
            if constexpr (ONE) {
                a0 &= keep0; a1 &= keep0; a2 &= keep1; a3 &= keep1;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float y[4] = {0.f, 0.f, 0.f, 0.f};
                    mma(y, a0, a1, a2, a3, pb[n][0], pb[n][1]);
                    if constexpr (TWO) mma(y, a0, a1, a2, a3, pr[n][0], pr[n][1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((cols >> (2 * n + (i & 1))) & 1u) o[4 * j + e][n][i] += y[i];
                }
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma(o[4 * j + e][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                    if constexpr (TWO)
                        mma(o[4 * j + e][n], a0, a1, a2, a3, pr[n][0], pr[n][1]);
                }
            }
        }
    }
}

// The sizes of row r of a 4-bit stage's V, a group's being the larger of |scale|
// and |low|: the bits of the largest (as bf16) and how far the smallest lies below.
template <int D>
RKV_DEV void row_sizes(uint32_t st, int r, uint32_t& top, uint32_t& spread) {
    using S = Stage<D, 4>;
    const uint32_t row = st + S::vs() + r * S::SROW;
    uint32_t most, least;  // of the groups with even and with odd numbers
    if constexpr (S::W == 4) {
        const uint4 x = lds16(row);
        const uint32_t a = x.x & 0x7fff7fffu, b = x.y & 0x7fff7fffu;
        const uint32_t c = x.z & 0x7fff7fffu, d = x.w & 0x7fff7fffu;
        const uint32_t e = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
        const uint32_t f = __vmaxu2(__byte_perm(c, d, 0x5410), __byte_perm(c, d, 0x7632));
        most = __vmaxu2(e, f);
        least = __vminu2(e, f);
    } else {
        const uint2 x = lds8(row);
        const uint32_t a = x.x & 0x7fff7fffu, b = x.y & 0x7fff7fffu;
        most = least = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    }
    top = max(most & 0xffffu, most >> 16);
    spread = top - min(least & 0xffffu, least >> 16);
}

// Whether row r of a stage holds an infinity or a NaN in V (4 bits: in its
// scales).
template <int D, int BITS>
RKV_DEV bool unfinite(uint32_t st, int r) {
    constexpr bool Q4 = BITS == 4;
    using S = Stage<D, BITS>;
    const uint32_t row = Q4 ? st + S::vs() + r * S::SROW : st + S::V + r * S::ROW;
    bool bad = false;
#pragma unroll 4
    for (int i = 0; i < (Q4 ? S::SROW : S::ROW) / 8; ++i) {
        const uint2 x = lds8(row + 8 * i);
        bad |= (x.x & 0x7f80u) == 0x7f80u || (x.x & 0x7f800000u) == 0x7f800000u;
        bad |= (x.y & 0x7f80u) == 0x7f80u || (x.y & 0x7f800000u) == 0x7f800000u;
    }
    return bad;
}

// The same for a 4-bit stage but for the lows; p: probabilities of 16 keys as
// accumulators lie.  MIXED: probabilities times scales in two bf16 parts instead of
// fp16 (see kSpread) for the queries (columns) in `wide` (bit 2 n + i; every: for all
// of the warp's), and a hidden row's NaN stays out (some of the queries do not see
// some of the rows).
template <int D, int NT, bool MIXED>
RKV_DEV void values_q4(const Unpack& uk, uint32_t st, int base, const float (&p)[NT][4],
                       uint32_t wide, bool every, float (&o)[D / 16][NT][4]) {
    using S = Stage<D, 4>;
    constexpr int W = S::W;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint32_t sc[2][W];
    {
        const int pr = base + phys<4>(g);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t srow = st + S::vs() + (pr + 8 * k) * S::SROW;
            if constexpr (W == 4) {
                const uint4 y = lds16(srow);
                sc[k][0] = y.x; sc[k][1] = y.y; sc[k][2] = y.z; sc[k][3] = y.w;
            } else {
                const uint2 y = lds8(srow);
                sc[k][0] = y.x; sc[k][1] = y.y;
            }
        }
    }
    uint32_t x[4][W / 2];  // a key's codes of its lane: two groups a word
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int pr = base + phys<4>(2 * t + (k & 1) + 8 * (k >> 1));
        const uint32_t row = st + S::V + pr * S::ROW;
        if constexpr (W == 4) {
            const uint2 y = lds8(row + (((g >> 1) ^ unit_xor<D, 4>(pr)) << 4) + ((g & 1) << 3));
            x[k][0] = y.x; x[k][1] = y.y;
        } else {
            x[k][0] = lds4(row + g * 4);
        }
    }
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const uint32_t sel = (w & 1) ? 0x7632 : 0x5410;
        const uint32_t u = __byte_perm(x[0][w >> 1], x[1][w >> 1], sel);
        const uint32_t v = __byte_perm(x[2][w >> 1], x[3][w >> 1], sel);
        uint32_t a[4], b[4];
        centred(uk, u, a);
        centred(uk, v, b);
        const float s[2] = {__uint_as_float(sc[0][w] * uk.up), __uint_as_float(sc[1][w] * uk.up)};
        if (!MIXED || !every) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[i] = p[n][i] * s[i >> 1];
                    if (MIXED && (p[n][i] == 0.f || ((wide >> (2 * n + (i & 1))) & 1u))) y[i] = 0.f;
                }
                const uint32_t b0 = transpose8x8(pack_f16(y[0], y[1]));
                const uint32_t b1 = transpose8x8(pack_f16(y[2], y[3]));
                mma_f16(o[2 * w][n], a[0], a[1], b[0], b[1], b0, b1);
                mma_f16(o[2 * w + 1][n], a[2], a[3], b[2], b[3], b0, b1);
            }
        }
        if constexpr (MIXED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = f16_as_bf16(a[i]);
                b[i] = f16_as_bf16(b[i]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[i] = p[n][i] * s[i >> 1];
                    if (p[n][i] == 0.f || !((wide >> (2 * n + (i & 1))) & 1u)) y[i] = 0.f;
                }
                const uint32_t h0 = pack(y[0], y[1]), h1 = pack(y[2], y[3]);
                const uint32_t b0 = transpose8x8(h0), b1 = transpose8x8(h1);
                const uint32_t r0 = transpose8x8(pack_rest(y[0], y[1], h0));
                const uint32_t r1 = transpose8x8(pack_rest(y[2], y[3], h1));
                mma(o[2 * w][n], a[0], a[1], b[0], b[1], b0, b1);
                mma(o[2 * w][n], a[0], a[1], b[0], b[1], r0, r1);
                mma(o[2 * w + 1][n], a[2], a[3], b[2], b[3], b0, b1);
                mma(o[2 * w + 1][n], a[2], a[3], b[2], b[3], r0, r1);
            }
        }
    }
}

// (scale, low) of the 16 keys as operand rows: row 2 w scale, row 2 w + 1 low.
template <int D>
RKV_DEV void low_rows(uint32_t st, int base, uint32_t (&a)[2]) {
    using S = Stage<D, 4>;
    if constexpr (S::W == 4) {
        ldm2t(a, st + S::vs() + scale_row(base));
    } else {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        uint32_t x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int pr = base + phys<4>(2 * t + (k & 1) + 8 * (k >> 1));
            x[k] = lds2(st + S::vs() + pr * S::SROW + 2 * (g & 3));
        }
        a[0] = g < 4 ? __byte_perm(x[0], x[1], 0x5410) : 0u;  // (rows past 2 W stand for nothing)
        a[1] = g < 4 ? __byte_perm(x[2], x[3], 0x5410) : 0u;
    }
}

// ------------------------------------------------------------- the line --
// Units of all (sequence, KV head) problems in order, n of them (below 2^31),
// in `runs` runs (no more than n) that differ by one unit at most.

// Rows of a sequence that count: its length cut to 0 .. max_rows.
RKV_DEV int rows_of(const Params& p, int s) {
    const int n = p.lens[s];
    return n < 0 ? 0 : (n > p.max_rows ? p.max_rows : n);
}
// Units of a sequence's problem; an empty one has a unit too (its zeros are
// written by it).  On the line a problem is p.lead places longer: what a block
// spends on beginning and ending one, so that runs over many short sequences
// are not the last to finish.
RKV_DEV uint32_t units_of(int rows, int unit) {
    return rows <= unit ? 1u : (uint32_t)(rows - 1) / (uint32_t)unit + 1u;
}

// The place of a block on the line: its run of units and the problem that the
// run's first unit belongs to.
struct Place {
    uint32_t n, runs;    // units and runs in use
    uint32_t u0, u1;     // the run (empty: none for this block)
    uint32_t start;      // first unit of the current problem
    int s, h;
};
// First unit of run i, and the run of unit u.
RKV_DEV uint32_t first_of(const Place& pl, uint32_t i) {
    const uint32_t per = pl.n / pl.runs, more = pl.n - per * pl.runs;
    return i * per + (i < more ? i : more);
}
RKV_DEV uint32_t run_of(const Place& pl, uint32_t u) {
    const uint32_t per = pl.n / pl.runs, more = pl.n - per * pl.runs;
    const uint32_t big = more * (per + 1);
    return u < big ? u / (per + 1) : more + (u - big) / per;
}
// Cuts the line and finds sequence pl.s with first unit *first*, given a
// thread's stretch [a, b) of sequences, `sum` units of it and `upto` units up to
// its end: true in the thread that owns the run's first unit.
RKV_DEV bool own_stretch(const Params& p, int unit, uint32_t run, uint32_t all, int a, uint32_t sum,
                         uint32_t upto, Place& pl, uint32_t& first) {
    pl.n = all * p.H;
    pl.runs = min((uint32_t)p.runs, pl.n);
    pl.u0 = pl.u1 = 0;
    if (run < pl.runs) {
        pl.u0 = first_of(pl, run);
        pl.u1 = first_of(pl, run + 1);
    }
    first = (upto - sum) * p.H;
    if (first > pl.u0 || pl.u0 >= upto * p.H) return false;
    for (pl.s = a;; ++pl.s) {
        const uint32_t w = (units_of(rows_of(p, pl.s), unit) + p.lead) * p.H;
        if (pl.u0 < first + w) return true;
        first += w;
    }
}
template <int THREADS>
RKV_DEV Place find_place(const Params& p, int unit, uint32_t run) {
    __shared__ uint32_t found[2], warp_sum[THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // each lane of every warp owns a stretch of sequences (no barrier), with
    // many sequences each thread of the block
    const bool small = p.num_seqs <= 256;
    const int n = small ? 32 : THREADS, me = small ? lane : tid;
    const int per = (p.num_seqs + n - 1) / n;
    const int a = min(me * per, p.num_seqs), b = min(a + per, p.num_seqs);
    uint32_t sum = 0;
    for (int s = a; s < b; ++s) sum += units_of(rows_of(p, s), unit) + p.lead;
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    Place pl;
    uint32_t first = 0;
    if (small) {
        const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
        const bool mine = own_stretch(p, unit, run, all, a, sum, upto, pl, first);
        const int owner = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        pl.s = __shfl_sync(0xffffffffu, pl.s, owner);
        first = __shfl_sync(0xffffffffu, first, owner);
    } else {
        if (lane == 31) warp_sum[warp] = upto;
        __syncthreads();
        uint32_t all = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) upto += warp_sum[w];
            all += warp_sum[w];
        }
        if (own_stretch(p, unit, run, all, a, sum, upto, pl, first)) {
            found[0] = pl.s;
            found[1] = first;
        }
        __syncthreads();
        pl.s = found[0];
        first = found[1];
    }
    const uint32_t n_s = units_of(rows_of(p, pl.s), unit) + p.lead;
    pl.h = (pl.u0 - first) / n_s;
    pl.start = first + pl.h * n_s;
    return pl;
}

// A piece of a problem that a block works on.
struct Piece {
    int s, h, len, c0, c1;
    uint32_t slot, parts;  // parts: blocks that share the problem, where it begins here
    bool whole;
};
// The next piece of the run (false: none left), which then starts behind it.
// A sequence's bad length is recorded by the block of its first unit.
RKV_DEV bool next_piece(const Params& p, int unit, uint32_t run, Place& pl, Piece& c) {
    while (pl.u0 < pl.u1) {
        c.s = pl.s;
        c.h = pl.h;
        c.len = rows_of(p, pl.s);
        const uint32_t n_s = units_of(c.len, unit), n_l = n_s + p.lead;
        const uint32_t from = pl.u0 - pl.start, to = min(n_l, pl.u1 - pl.start);
        const uint32_t j = from > p.lead ? from - p.lead : 0, e = to > p.lead ? to - p.lead : 0;
        c.c0 = j * unit;
        c.c1 = e == n_s ? c.len : e * unit;
        c.whole = j == 0 && e == n_s;
        // a piece that an earlier block began, or one that a later block ends
        c.slot = 2 * run + (j > 0 ? 0 : 1);
        c.parts = j > 0 || c.whole || e == 0 ? 0 : run_of(pl, pl.start + n_l - 1) - run + 1;
        pl.u0 = pl.start + to;
        if (to == n_l) {
            pl.start += n_l;
            if (++pl.h == p.H) {
                pl.h = 0;
                ++pl.s;
            }
        }
        if (e > j) {
            if (threadIdx.x == 0 && j == 0 && c.h == 0 && c.len != p.lens[c.s])
                set_error(p.status, kDevErrIndex, (unsigned)c.s);
            return true;
        }
    }
    return false;
}

// A cluster's share of its problem: block `rank` of `p.cluster` takes the units
// from rank * n_s / cluster on (maybe none).
RKV_DEV void cluster_piece(const Params& p, int unit, int prob, int rank, Piece& c) {
    c.s = prob / p.H;
    c.h = prob - c.s * p.H;
    c.len = rows_of(p, c.s);
    const int n_s = units_of(c.len, unit);
    const int j = rank * n_s / p.cluster, e = (rank + 1) * n_s / p.cluster;
    c.c0 = j * unit;
    c.c1 = e == j ? c.c0 : (e == n_s ? c.len : e * unit);
    c.slot = c.parts = 0;
    c.whole = true;
    if (threadIdx.x == 0 && rank == 0 && c.h == 0 && c.len != p.lens[c.s])
        set_error(p.status, kDevErrIndex, (unsigned)c.s);
}

// What a part with sums relative to 2^m counts beside a common reference mx: an
// empty part nothing, one whose logits are all NaN its NaN.
RKV_DEV float weight(float m, float l, float mx) {
    if (m == -INFINITY) return l != l ? 1.f : 0.f;
    return ex2(m - mx);
}
// The base-2 logit m * scale - up in fp32 (-inf: none), and 2^ what that rounding
// left of it.  Where the product's own rounding is past 32 it is left out: it is the
// same for the parts of a problem that found the same maximum, and others are as far
// apart as it is coarse.
RKV_DEV float base_of(float m, float scale, float up, float& fix) {
    fix = 1.f;
    if (m == kNone || up == kUnset) return -INFINITY;
    const float z = __fmul_rn(m, scale), base = z - up, rest = fmaf(m, scale, -z);
    if (fabsf(z) <= FLT_MAX) fix = ex2((z - base) - up + (fabsf(rest) <= 32.f ? rest : 0.f));
    return base;
}
// 4 bits: logits q . k less their queries' m, after a step of m to the stage's maximum
// where that is past kHuge from 0, or past an m there is (up with it, so that the sums
// keep their reference; up stays as small as the exponents of V).  Whether some query
// has an m.
template <int KT, int NT>
RKV_DEV bool take_m(float (&x)[KT][NT][4], const float (&top)[NT][2], const float (&sc)[NT][2],
                    float (&m)[NT][2], float (&up)[NT][2], bool huge) {
    bool past = huge;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float z = top[n][i] * sc[n][i];
            past |= z > kHuge || (z < -kHuge && z >= -FLT_MAX && up[n][i] == kUnset);
        }
    if (!__any_sync(0xffffffffu, past)) return false;
    past = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float mx = top[n][i];
#pragma unroll
            for (int sh = 4; sh <= 16; sh <<= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
            const float z = (mx - m[n][i]) * sc[n][i];
            const bool step = fabsf(z) <= FLT_MAX &&
                              (up[n][i] == kUnset ? fabsf(z) : z) > (m[n][i] == 0.f ? kHuge : 0.f);
            if (step) {
                if (up[n][i] != kUnset) up[n][i] += z;
                m[n][i] = mx;
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int k = 0; k < 2; ++k) x[kt][n][i + 2 * k] -= m[n][i];
            past |= m[n][i] != 0.f;
        }
    return __any_sync(0xffffffffu, past);
}
template <int ROWS>
RKV_DEV float row_max(const float (&sh_m)[kWarps][ROWS], int r) {
    float mx = sh_m[0][r];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sh_m[w][r]);
    return mx;
}

RKV_DEV void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
RKV_DEV void store4(__nv_bfloat16* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack(v.x, v.y), pack(v.z, v.w));
}

// Four values of a query's output from its sums v relative to 2^mx, and the log of its
// sum (RAW: or, where they are to be joined with others', v and mx and the sum as they
// are; packed caches have no such calls).
template <typename T, int D, bool RAW>
RKV_DEV void emit(const Params& p, int64_t s, int tk, int hd, int d, float4 v, float mx, float sum) {
    const int64_t at = (s * p.T + tk) * (int64_t)p.H * p.G + hd;
    if (RAW && p.raw) {
        store4(p.raw + at * D + d, v);
        if (d == 0) *reinterpret_cast<float2*>(p.raw_ml + 2 * at) = make_float2(mx, sum);
        return;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    store4(reinterpret_cast<T*>(p.out) + s * p.o_seq + tk * p.o_tok + hd * p.o_head + d,
           make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    if (d == 0 && p.lse) p.lse[at] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

// Joins the warps' weighted sums in acc [kWarps][ROWS][D] and writes the rows:
// the output where the chunk is the whole sequence, else its part.
template <typename T, int D, int ROWS, bool RAW>
RKV_DEV void finish(const Params& p, const float* acc, const float (&sh_m)[kWarps][ROWS],
                    const float (&sh_l)[kWarps][ROWS], int64_t s, int h, int row_first,
                    int64_t slot, bool whole) {
    for (int e = threadIdx.x; e < ROWS * D / 4; e += kWarps * 32) {
        const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
        const int row = row_first + r;
        if (row >= p.R) continue;
        const float mx = row_max(sh_m, r);
        float sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            sum += sh_l[w][r] * weight(sh_m[w][r], sh_l[w][r], mx);
            const float4 y = *reinterpret_cast<const float4*>(acc + ((size_t)w * ROWS + r) * D + d);
            v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
        }
        if (whole) {
            const int tk = row / p.G, hd = h * p.G + row - tk * p.G;
            emit<T, D, RAW>(p, s, tk, hd, d, v, mx, sum);
        } else {
            *reinterpret_cast<float4*>(p.partial + (slot * ROWS + r) * D + d) = v;
            if (d == 0) {
                float* ml = p.partial_ml + (slot * ROWS + r) * 2;
                ml[0] = mx;
                ml[1] = sum;
            }
        }
    }
}

RKV_DEV uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
RKV_DEV void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address of another block's copy of this shared location.
RKV_DEV uint32_t shared_of(uint32_t at, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    return r;
}
RKV_DEV float4 remote4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at));
    return v;
}
RKV_DEV float2 remote2(uint32_t at) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at));
    return v;
}

// finish() for a cluster's blocks, through their shared memory: each joins its
// warps, then takes its part of the problem's output over all blocks.  No second
// launch and no scratch.
constexpr int kCluster = 8;
template <typename T, int D, int ROWS, bool RAW>
RKV_DEV void finish_cluster(const Params& p, float* acc, const float (&sh_m)[kWarps][ROWS],
                            const float (&sh_l)[kWarps][ROWS], float2 (&sh_ml)[ROWS], int s, int h,
                            int row_first, uint32_t rank) {
    const int tid = threadIdx.x;
    for (int e = tid; e < ROWS * D / 4; e += kWarps * 32) {
        const int r = e / (D / 4);
        float4 v = *reinterpret_cast<const float4*>(acc + (size_t)e * 4);
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float4 y = *reinterpret_cast<const float4*>(acc + ((size_t)w * ROWS * D + e * 4));
            v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
        }
        *reinterpret_cast<float4*>(acc + (size_t)e * 4) = v;
        if (e - r * (D / 4) == 0) {
            const float mx = row_max(sh_m, r);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                sum += sh_l[w][r] * weight(sh_m[w][r], sh_l[w][r], mx);
            sh_ml[r] = make_float2(mx, sum);
        }
    }
    cluster_sync();
    for (int e = rank * (kWarps * 32) + tid; e < ROWS * D / 4; e += p.cluster * (kWarps * 32)) {
        const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
        const int row = row_first + r;
        if (row >= p.R) break;
        float2 ml[kCluster];
        float4 x[kCluster];
#pragma unroll
        for (int i = 0; i < kCluster; ++i) {
            ml[i] = make_float2(-INFINITY, 0.f);
            x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < p.cluster) {
                ml[i] = remote2(shared_of(smem_at(&sh_ml[r]), i));
                x[i] = remote4(shared_of(smem_at(acc + (size_t)e * 4), i));
            }
        }
        float mx = ml[0].x, sum = 0.f;
#pragma unroll
        for (int i = 1; i < kCluster; ++i) mx = fmaxf(mx, ml[i].x);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kCluster; ++i) {
            const float f = weight(ml[i].x, ml[i].y, mx);
            sum += ml[i].y * f;
            v.x += x[i].x * f; v.y += x[i].y * f; v.z += x[i].z * f; v.w += x[i].w * f;
        }
        const int tk = row / p.G, hd = h * p.G + row - tk * p.G;
        emit<T, D, RAW>(p, s, tk, hd, d, v, mx, sum);
    }
    cluster_sync();  // nobody leaves while its shared memory is read
}

// NT * 8 queries of a KV head's group against a run of rows.
template <int D, int NT, int BITS, bool TWO>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 && BITS ? 3 : 2) attn_kernel(const __grid_constant__ Params p) {
    constexpr bool Q4 = BITS == 4, Q8 = BITS == 8;
    using S = Stage<D, BITS>;
    constexpr int ROWS = 8 * NT, W = D / 32, KT = S::KEYS / 16, UNIT = kWarps * S::KEYS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sh_m[kWarps][ROWS], sh_l[kWarps][ROWS];
    __shared__ __align__(8) float2 sh_ml[ROWS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    // groups of queries over the same rows are neighbours: the rows come from
    // HBM once and from L2 for the others
    const uint32_t rank = cluster_rank();  // 0 where a block is alone
    const uint32_t job = p.cluster ? blockIdx.x / p.cluster : blockIdx.x;
    const int group = job % p.groups;
    const uint32_t run = job / p.groups;  // (a cluster's problem)
    const int row_first = group * ROWS;  // first query row (token * G + head of the group)
    const int mask = (1 << p.log2bs) - 1;
    const uint32_t ring = smem_at(smem) + warp * (S::DEPTH * S::BYTES);
    constexpr uint32_t kAll = S::KEYS == 32 ? 0xffffffffu : 0xffffu;

    [[maybe_unused]] Unpack uk;
    if constexpr (Q4) uk = unpack_constants();
    [[maybe_unused]] Bytes bk;
    if constexpr (Q8) bk = byte_constants();
    wait_for_last();

    Place place{};
    Piece c{};
    if (p.cluster)
        cluster_piece(p, UNIT, run, rank, c);
    else
        place = find_place<kWarps * 32>(p, UNIT, run);
    while (p.cluster || next_piece(p, UNIT, run, place, c)) {
        const int s = c.s, h = c.h, len = c.len, c0 = c.c0, c1 = c.c1;

        const int32_t* table = p.table + (int64_t)s * p.max_blocks;
        // the block id of this lane's row of the next stage (-1: no such row); looked at one
        // stage later, when the load has come back
        int look = c0 + warp * S::KEYS + lane;
        const int end = lane < S::KEYS ? c1 : 0;
        auto look_up = [&] {
            int b = -1;
            if (look < end) b = table[look >> p.log2bs];
            look += UNIT;
            return b;
        };
        // copies the stage of rows from `fetch` on into the slot at `to`; which of them exist
        uint32_t to = ring;
        int fetch = c0 + warp * S::KEYS;
        auto issue = [&](int b) {
            const int r = fetch + lane;
            const bool good = (uint32_t)b < (uint32_t)p.num_blocks;
            const uint32_t ok = __ballot_sync(0xffffffffu, good);
            if (!good && r < end) set_error(p.status, kDevErrIndex, (unsigned)r);
            const uint32_t row =
                good ? (((uint32_t)b * p.H + h) << p.log2bs) | (uint32_t)(r & mask) : kNoRow;
            if (fetch < c1) copy_stage<D, BITS>(p, to, row, ok == kAll);
            cp_commit();
            fetch += UNIT;
            to = to == ring + (S::DEPTH - 1) * S::BYTES ? ring : to + S::BYTES;
            return ok;
        };
        uint32_t held[S::DEPTH];  // rows of the stage at hand and of those behind it
        int next;
        {
            int ids[S::DEPTH - 1];
#pragma unroll
            for (int i = 0; i < S::DEPTH - 1; ++i) ids[i] = look_up();
            next = look_up();
#pragma unroll
            for (int i = 0; i < S::DEPTH - 1; ++i) held[i] = issue(ids[i]);
        }

        // queries as the second operand: lane (g, t) holds row g, values 32 w + 8 t ..
        uint32_t qf[NT][D / 8];
        [[maybe_unused]] uint32_t qb[NT][3];
        float sc[NT][2];  // logits to base 2 (columns 2t, 2t + 1)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            sc[n][0] = sc[n][1] = p.scale;
            const int r = row_first + 8 * n + g;
            const bool ok = r < p.R;
            const int tk = ok ? r / p.G : 0, hd = ok ? r - tk * p.G : 0;
            const __nv_bfloat16* q =
                p.q + s * p.q_seq + tk * p.q_tok + (int64_t)(h * p.G + hd) * p.q_head;
            float own = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                uint4 x = make_uint4(0, 0, 0, 0);
                // (8 bits: lane t holds values 64 w' + 16 t .. in two steps)
                if (ok) x = *reinterpret_cast<const uint4*>(Q8 ? q + 64 * (w >> 1) + 16 * t + 8 * (w & 1) : q + 32 * w + 8 * t);
                x.x ^= p.flip; x.y ^= p.flip; x.z ^= p.flip; x.w ^= p.flip;
                if constexpr (Q4) {
                    const uint32_t y[4] = {x.x, x.y, x.z, x.w};
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sum += __uint_as_float(y[i] << 16) + __uint_as_float(y[i] & 0xffff0000u);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    if (w == t) own = sum;
                    x = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                                   __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
                }
                if constexpr (Q8)
                    x = make_uint4(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.x, x.y, 0x7632),
                                   __byte_perm(x.z, x.w, 0x5410), __byte_perm(x.z, x.w, 0x7632));
                qf[n][4 * w] = x.x;
                qf[n][4 * w + 1] = x.y;
                qf[n][4 * w + 2] = x.z;
                qf[n][4 * w + 3] = x.w;
            }
            if constexpr (Q4) {
                // The row times 2^e, its largest element in 2^14 .. 2^15, as fp16; what
                // meets a code four bits higher is 16 times smaller.  Logits are then in
                // units of 2^(24 - e), which mul takes back (in full below 2^115).
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    top = max(top, max(qf[n][i] & 0x7fffu, (qf[n][i] >> 16) & 0x7fffu));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = min(141 - (int)(top >> 7), 120);
                const float f = pow2(e);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const float h = i & 1 ? f * 0.0625f : f;
                    qf[n][i] = pack_f16(__uint_as_float(qf[n][i] << 16) * h,
                                        __uint_as_float(qf[n][i] & 0xffff0000u) * h);
                }
                own = own * f * 0x1p-24f;
                const float mul = fminf(fmaxf(p.scale * 4096.f * pow2(12 - e), 0x1p-120f), 0x1p127f);
                sc[n][0] = __shfl_sync(0xffffffffu, mul, 8 * t);
                sc[n][1] = __shfl_sync(0xffffffffu, mul, 8 * t + 4);
                // the sum too, in three bf16 parts (8 bits each)
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const float part = __bfloat162float(__float2bfloat16_rn(own));
                    qb[n][i] = pack(0.f, part);
                    own -= part;
                }
            }
        }
        // the newest row each of the lane's queries (columns 2t, 2t + 1) sees
        int last[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = row_first + 8 * n + 2 * t + i;
                last[n][i] = r < p.R ? len - p.T + r / p.G : len - 1;
            }
        const int all_see = len - p.T + row_first / p.G;  // rows up to this one are seen by all

        // m: running maximum of q . k (kNone: none yet); sums are relative to 2^(m * scale).
        // Differences of q . k are scaled, not scaled logits subtracted: those are as coarse as
        // fp32 is at their size.  4 bits: sums are relative to 2^(m * scale - up), up being kAbove
        // less the largest of (q . k - m) * scale plus the exponent of the row's V (kUnset: none
        // yet), so that p * scale stays below 2^15 in fp16 (see kSpread); m is 0 but where
        // logits past kHuge make a difference of it (the subtraction would cost 2 in a
        // hundred).
        float m[NT][2], l[NT][2], o[D / 16][NT][4];
        [[maybe_unused]] float up[NT][2];
        [[maybe_unused]] float low[NT][4];
        // the lane's queries whose products take two bf16 parts (bit 2 n + i), and whether some
        // or all of the warp's do
        constexpr uint32_t kMine = (1u << (2 * NT)) - 1u;
        [[maybe_unused]] uint32_t wide = 0;
        [[maybe_unused]] bool some = false, every = false;
        [[maybe_unused]] bool huge = false;  // some query of the warp's has an m
        [[maybe_unused]] int bound = kLeast;  // the largest exponent of V's rows so far
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[n][i] = Q4 ? 0.f : kNone;
                l[n][i] = 0.f;
                if constexpr (Q4) up[n][i] = kUnset;
            }
#pragma unroll
            for (int e = 0; e < D / 16; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[e][n][i] = 0.f;
            if constexpr (Q4) low[n][0] = low[n][1] = low[n][2] = low[n][3] = 0.f;
        }

        uint32_t st = ring;
        for (int row0 = c0 + warp * S::KEYS; row0 < c1; row0 += UNIT) {
            cp_wait<S::DEPTH - 2>();
            __syncwarp();  // the stage is there, and the slot refilled next has been read
            const int fill = next;
            next = look_up();
            held[S::DEPTH - 1] = issue(fill);
            const uint32_t ok = held[0];
#pragma unroll
            for (int i = 0; i + 1 < S::DEPTH; ++i) held[i] = held[i + 1];
            const bool masked = ok != kAll || row0 + S::KEYS - 1 > all_see;
            float x[KT][NT][4];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                if constexpr (Q4)
                    logits_q4<D, NT>(uk, st, kt * 16, qf, qb, x[kt]);
                else if constexpr (Q8)
                    logits_q8<D, NT>(bk, st, kt * 16, qf, x[kt]);
                else
                    logits_bf16<D, NT>(st, kt * 16, qf, x[kt]);
            }
            if (masked) {
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = kt * 16 + phys<BITS>(g + 8 * (i >> 1));
                            if (row0 + r > last[n][i & 1] || !((ok >> r) & 1u))
                                x[kt][n][i] = -INFINITY;
                        }
            }
            bool grow = false;
            [[maybe_unused]] bool far = false;
            [[maybe_unused]] int mine = 0;  // 4 bits: V's exponent of the lane's row
            if constexpr (Q4) {
                uint32_t most, spread;
                row_sizes<D>(st, lane, most, spread);
                const int e = (int)(most >> 7) - 126;  // below 2^e
                mine = min(max(e, kLeast), kMost);
                far = ((ok >> lane) & 1u) && (spread > kSpread || mine != e);
                grow = (far && !every) || mine > bound || huge;
            }
            float top[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[n][i] = fmaxf(x[0][n][i], x[0][n][i + 2]);
#pragma unroll
                    for (int kt = 1; kt < KT; ++kt)
                        top[n][i] = fmaxf(top[n][i], fmaxf(x[kt][n][i], x[kt][n][i + 2]));
                    // (4 bits: no row of the stage is above this)
                    if constexpr (Q4)
                        grow |= fmaf(top[n][i], sc[n][i], (float)bound) > kAbove + kSlack - up[n][i];
                    else
                        grow |= top[n][i] > m[n][i] + p.slack;
                }
            if (__any_sync(0xffffffffu, grow)) {
                [[maybe_unused]] float ve[KT][2];  // 4 bits: the exponents of rows g and g + 8
                if constexpr (Q4) {
                    bound = max(bound, __reduce_max_sync(0xffffffffu, mine));
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            ve[kt][k] = (float)__shfl_sync(0xffffffffu, mine,
                                                           kt * 16 + phys<BITS>(g) + 8 * k);
                    const uint32_t rows = __ballot_sync(0xffffffffu, far);
                    if (rows) {  // the queries that see one of them
                        const int first = row0 + __ffs(rows) - 1;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (last[n][i] >= first) wide |= 1u << (2 * n + i);
                        some = __any_sync(0xffffffffu, wide != 0);
                        every = __all_sync(0xffffffffu, wide == kMine);
                    }
                }
                if constexpr (Q4) huge = take_m<KT, NT>(x, top, sc, m, up, huge);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float mx = Q4 ? -INFINITY : fmaxf(m[n][i], top[n][i]);
                        if constexpr (Q4)
#pragma unroll
                            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                                for (int k = 0; k < 2; ++k)
                                    mx = fmaxf(mx, fmaf(x[kt][n][i + 2 * k], sc[n][i], ve[kt][k]));
#pragma unroll
                        for (int sh = 4; sh <= 16; sh <<= 1)
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
                        float f;
                        if constexpr (Q4) {
                            // a query's numbers are the same whatever the others see
                            const float old = kAbove - up[n][i];
                            if (!(mx > old + kSlack)) continue;
                            f = up[n][i] == kUnset ? 0.f : ex2(old - mx);
                            up[n][i] = kAbove - mx;
                        } else {
                            f = m[n][i] == kNone ? 0.f : ex2((m[n][i] - mx) * sc[n][i]);
                            m[n][i] = mx;
                        }
                        l[n][i] *= f;
#pragma unroll
                        for (int e = 0; e < D / 16; ++e) {
                            o[e][n][i] *= f;
                            o[e][n][i + 2] *= f;
                        }
                        if constexpr (Q4) low[n][i] *= f;
                    }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float& z = x[kt][n][i + 2 * k];
                            z = ex2(Q4 ? fmaf(z, sc[n][i], up[n][i]) : (z - m[n][i]) * sc[n][i]);
                        }
                        l[n][i] += x[kt][n][i] + x[kt][n][i + 2];
                    }
            // rows that only some of the tokens see: an infinity or a NaN there must not reach
            // the others as 0 * inf, so such a stage is taken one token at a time (rows nobody
            // sees are zeros here: rows past len and rows without a block)
            // (8 bits: codes are finite, and a hidden row's scale is left out below)
            bool apart = false;
            if (!Q8 && masked && p.T > 1) {
                const int r = row0 + lane;
                const bool part = lane < S::KEYS && r < c1 && r > all_see;
                apart = __any_sync(0xffffffffu, part && unfinite<D, BITS>(st, lane));
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                uint32_t pb[NT][2];
                [[maybe_unused]] uint32_t pr[NT][2];
                if constexpr (Q8) {
                    // V's scales meet the probabilities, but for rows that a query does not see
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int r = kt * 16 + phys<8>(g) + 8 * k;
                        const float vs = __uint_as_float(lds4(st + S::vs() + r * 4));
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                float& y = x[kt][n][i + 2 * k];
                                y = masked && row0 + r > last[n][i] ? 0.f : y * vs;
                            }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float lo = x[kt][n][2 * i], hi = x[kt][n][2 * i + 1];
                        const uint32_t h = pack(lo, hi);
                        pb[n][i] = transpose8x8(h);
                        if constexpr (TWO) pr[n][i] = transpose8x8(pack_rest(lo, hi, h));
                    }
                [[maybe_unused]] uint32_t la[2];
                if constexpr (Q4) low_rows<D>(st, kt * 16, la);
                if constexpr (Q4) {
                    if (some || apart)
                        values_q4<D, NT, true>(uk, st, kt * 16, x[kt], wide, every, o);
                    else
                        values_q4<D, NT, false>(uk, st, kt * 16, x[kt], 0u, false, o);
                }
                if (!apart) {
                    if constexpr (Q4) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma(low[n], la[0], 0u, la[1], 0u, pb[n][0], pb[n][1]);
                            if constexpr (TWO)
                                mma(low[n], la[0], 0u, la[1], 0u, pr[n][0], pr[n][1]);
                        }
                    } else if constexpr (Q8) {
                        values_q8<D, NT, TWO>(bk, st, kt * 16, pb, pr, o);
                    } else {
                        values_bf16<D, NT, TWO, false>(st, kt * 16, pb, pr, ~0u, ~0u, ~0u, o);
                    }
                    continue;
                }
                // one token at a time
                const int t0 = row_first / p.G;
                const int t1 = (min(p.R, row_first + ROWS) - 1) / p.G;
                for (int tk = t0; tk <= t1; ++tk) {
                    const int see = len - p.T + tk;
                    uint32_t keep[2], cols = 0u;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int ra = row0 + kt * 16 + phys<BITS>(2 * t + 8 * k);
                        const int rb = row0 + kt * 16 + phys<BITS>(2 * t + 1 + 8 * k);
                        keep[k] = (ra <= see ? 0xffffu : 0u) | (rb <= see ? 0xffff0000u : 0u);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int r = row_first + 8 * n + 2 * t + i;
                            if (r < p.R && r / p.G == tk) cols |= 1u << (2 * n + i);
                        }
                    if constexpr (Q4) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float y[4] = {0.f, 0.f, 0.f, 0.f};
                            mma(y, la[0] & keep[0], 0u, la[1] & keep[1], 0u, pb[n][0], pb[n][1]);
                            if constexpr (TWO)
                                mma(y, la[0] & keep[0], 0u, la[1] & keep[1], 0u, pr[n][0], pr[n][1]);
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if ((cols >> (2 * n + i)) & 1u) low[n][i] += y[i];
                        }
                    } else if constexpr (!Q8) {
                        values_bf16<D, NT, TWO, true>(st, kt * 16, pb, pr, keep[0], keep[1], cols, o);
                    }
                }
            }
            st = st == ring + (S::DEPTH - 1) * S::BYTES ? ring : st + S::BYTES;
        }
        cp_wait<0>();
        // (behind this block's wait: the pass over shared prefixes relies on that, see launch_early)
        if (place.u0 >= place.u1) let_next_begin();

        // sums over the lanes that share a query; from here on m is the base-2 logit that they are
        // relative to, fix what its rounding left
        float fix[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int sh = 4; sh <= 16; sh <<= 1)
                    l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], sh);
                m[n][i] = base_of(m[n][i], sc[n][i], Q4 ? up[n][i] : 0.f, fix[n][i]);
                l[n][i] *= fix[n][i];
                if (g == 0) {
                    sh_m[warp][8 * n + 2 * t + i] = m[n][i];
                    sh_l[warp][8 * n + 2 * t + i] = l[n][i];
                }
            }
        __syncthreads();  // all rings are free as well
        float* acc = reinterpret_cast<float*>(smem);  // [warp][ROWS][D]
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * n + 2 * t + i;
                const float f = weight(m[n][i], l[n][i], row_max(sh_m, r)) * fix[n][i];
                float* dst = acc + ((size_t)warp * ROWS + r) * D;
                [[maybe_unused]] float add[W];
                if constexpr (Q4)
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        add[w] = __shfl_sync(0xffffffffu, low[n][i], 4 * (2 * w + 1) + t) +
                                 8.f * __shfl_sync(0xffffffffu, low[n][i], 4 * (2 * w) + t);
#pragma unroll
                for (int e = 0; e < D / 16; ++e) {
                    // the pair of dimensions this accumulator's rows g and g + 8 stand for
                    const int d = Q4 ? 32 * (e / 2) + 4 * g + 2 * (e % 2)
                                     : (Q8 ? D / 8 * g + 2 * e : 64 * (e / 4) + 8 * g + 2 * (e % 4));
                    float a = o[e][n][i], b = o[e][n][i + 2];
                    if constexpr (Q4) {
                        a += add[e / 2];
                        b += add[e / 2];
                    }
                    *reinterpret_cast<float2*>(dst + d) = make_float2(a * f, b * f);
                }
            }
        __syncthreads();
        if (p.cluster) {
            finish_cluster<__nv_bfloat16, D, ROWS, BITS == 0>(p, acc, sh_m, sh_l, sh_ml, s, h, row_first, rank);
            return;
        }
        finish<__nv_bfloat16, D, ROWS, BITS == 0>(p, acc, sh_m, sh_l, s, h, row_first,
                                       (int64_t)c.slot * p.groups + group, c.whole);
        __syncthreads();  // the next piece's copies overwrite what was just read
    }
    if (p.joins && tid == 0) p.joins[blockIdx.x] = make_int4(c.s, c.h, c.parts, 0);
}

// ------------------------------------------------------------ fp32 pools --
// The same pass on the CUDA cores: 8 queries a block, a warp takes 16 rows at
// a time.  For the logits a lane owns one key and half of the dimensions; for
// the values four dimensions (head_dim 64: and every other key).  The
// 16-byte units of row r lie at unit ^ (r mod 8), so neither read meets a bank
// twice.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) attn_f32_kernel(const __grid_constant__ Params p) {
    using S = Stage32<D>;
    constexpr int ROWS = 8, UPR = D / 4, UNIT = kWarps * S::KEYS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) float sh_q[ROWS][D];  // read four at a time
    __shared__ __align__(16) float sh_p[kWarps][S::KEYS][ROWS];
    __shared__ float sh_m[kWarps][ROWS], sh_l[kWarps][ROWS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int key = lane & 15, side = lane >> 4;
    const int group = blockIdx.x % p.groups;
    const uint32_t run = blockIdx.x / p.groups;
    const int row_first = group * ROWS;
    const int mask = (1 << p.log2bs) - 1;
    const float* q32 = reinterpret_cast<const float*>(p.q);
    const float sign = p.flip ? -1.f : 1.f;
    uint8_t* ring = smem + warp * (S::DEPTH * S::BYTES);
    wait_for_last();  // (first, as in attn_kernel: see launch_early)

    Place place = find_place<kWarps * 32>(p, UNIT, run);
    Piece c{};
    while (next_piece(p, UNIT, run, place, c)) {
        for (int e = tid; e < ROWS * UPR; e += kWarps * 32) {
            const int r = row_first + e / UPR, u = e % UPR;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < p.R) {
                const int tk = r / p.G, hd = c.h * p.G + r - tk * p.G;
                x = *reinterpret_cast<const float4*>(q32 + c.s * p.q_seq + tk * p.q_tok +
                                                     hd * p.q_head + 4 * u);
            }
            *reinterpret_cast<float4*>(&sh_q[e / UPR][4 * u]) =
                make_float4(x.x * sign, x.y * sign, x.z * sign, x.w * sign);
        }
        __syncthreads();
        int last[ROWS];
        float m[ROWS], l[ROWS], o[ROWS][4];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            last[r] = row_first + r < p.R ? c.len - p.T + (row_first + r) / p.G : c.len - 1;
            m[r] = kNone;
            l[r] = 0.f;
            o[r][0] = o[r][1] = o[r][2] = o[r][3] = 0.f;
        }
        const int all_see = c.len - p.T + row_first / p.G;

        const int32_t* table = p.table + (int64_t)c.s * p.max_blocks;
        const int stages = (c.c1 - c.c0 + S::KEYS - 1) / S::KEYS;
        const int mine = warp < stages ? (stages - warp + kWarps - 1) / kWarps : 0;
        uint32_t valid[2] = {0u, 0u};
        auto issue = [&](int it) {
            if (it < mine) {
                const int r0 = c.c0 + (warp + it * kWarps) * S::KEYS + lane;
                uint32_t x = kNoRow;
                if (lane < S::KEYS && r0 < c.c1) {
                    const int b = table[r0 >> p.log2bs];
                    if ((unsigned)b < (unsigned)p.num_blocks)
                        x = (((uint32_t)b * p.H + c.h) << p.log2bs) | (uint32_t)(r0 & mask);
                    else
                        set_error(p.status, kDevErrIndex, (unsigned)r0);
                }
                valid[1] = __ballot_sync(0xffffffffu, x != kNoRow);
                const uint32_t dst = smem_at(ring + (it % S::DEPTH) * S::BYTES);
                const int u = lane % UPR;
#pragma unroll 4
                for (int i = 0; i < S::KEYS * UPR / 32; ++i) {
                    const int r = i * (32 / UPR) + lane / UPR;
                    const uint32_t row = __shfl_sync(0xffffffffu, x, r);
                    const bool ok = row != kNoRow;
                    const uint64_t at = (uint64_t)(ok ? row : 0u) * S::ROW + u * 16;
                    const uint32_t to = dst + r * S::ROW + ((u ^ (r & 7)) << 4);
                    cp16(to, p.k + at, ok);
                    cp16(to + S::V, p.v + at, ok);
                }
            }
            cp_commit();
        };
        issue(0);
        valid[0] = valid[1];
        for (int it = 0; it < mine; ++it) {
            __syncwarp();  // the other slot has been read
            issue(it + 1);
            cp_wait<1>();
            __syncwarp();
            const uint8_t* st = ring + (it % S::DEPTH) * S::BYTES;
            const uint32_t ok = valid[0];
            valid[0] = valid[1];
            const int row0 = c.c0 + (warp + it * kWarps) * S::KEYS;
            const bool masked = ok != 0xffffu || row0 + S::KEYS - 1 > all_see;
            float x[ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) x[r] = 0.f;
            const uint8_t* krow = st + key * S::ROW;
#pragma unroll 4
            for (int u = 0; u < UPR / 2; ++u) {
                const int at = side * (UPR / 2) + u;
                const float4 k = *reinterpret_cast<const float4*>(krow + ((at ^ (key & 7)) << 4));
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const float4 y = *reinterpret_cast<const float4*>(&sh_q[r][4 * at]);
                    x[r] = fmaf(k.x, y.x, fmaf(k.y, y.y, fmaf(k.z, y.z, fmaf(k.w, y.w, x[r]))));
                }
            }
            bool grow = false;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                x[r] += __shfl_xor_sync(0xffffffffu, x[r], 16);
                if (masked && (row0 + key > last[r] || !((ok >> key) & 1u))) x[r] = -INFINITY;
                grow |= x[r] > m[r] + p.slack;
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const float mx = fmaxf(m[r], warp_max(x[r]));
                    const float f = m[r] == kNone ? 0.f : ex2((m[r] - mx) * p.scale);
                    m[r] = mx;
                    l[r] *= f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[r][i] *= f;
                }
            }
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                x[r] = ex2((x[r] - m[r]) * p.scale);
                if (side == 0) l[r] += x[r];
            }
            if (side == 0) {
                *reinterpret_cast<float4*>(&sh_p[warp][key][0]) = make_float4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<float4*>(&sh_p[warp][key][4]) = make_float4(x[4], x[5], x[6], x[7]);
            }
            __syncwarp();
            const int u = lane % UPR;
#pragma unroll 4
            for (int k = lane / UPR; k < S::KEYS; k += 32 / UPR) {
                const float4 v = *reinterpret_cast<const float4*>(st + S::V + k * S::ROW +
                                                                  ((u ^ (k & 7)) << 4));
                const float4 p0 = *reinterpret_cast<const float4*>(&sh_p[warp][k][0]);
                const float4 p1 = *reinterpret_cast<const float4*>(&sh_p[warp][k][4]);
                const float pr[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    if (masked && pr[r] == 0.f) continue;  // what a hidden row holds stays out
                    o[r][0] = fmaf(pr[r], v.x, o[r][0]);
                    o[r][1] = fmaf(pr[r], v.y, o[r][1]);
                    o[r][2] = fmaf(pr[r], v.z, o[r][2]);
                    o[r][3] = fmaf(pr[r], v.w, o[r][3]);
                }
            }
        }
        cp_wait<0>();
        float fix[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            m[r] = base_of(m[r], p.scale, 0.f, fix[r]);  // from here on: base-2 logits
            l[r] = warp_sum(l[r]) * fix[r];
            if (lane == 0) {
                sh_m[warp][r] = m[r];
                sh_l[warp][r] = l[r];
            }
            if constexpr (UPR == 16)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[r][i] += __shfl_xor_sync(0xffffffffu, o[r][i], 16);
        }
        __syncthreads();
        float* acc = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const float f = weight(m[r], l[r], row_max(sh_m, r)) * fix[r];
            if (lane < UPR)
                *reinterpret_cast<float4*>(acc + ((size_t)warp * ROWS + r) * D + 4 * lane) =
                    make_float4(o[r][0] * f, o[r][1] * f, o[r][2] * f, o[r][3] * f);
        }
        __syncthreads();
        finish<float, D, ROWS, true>(p, acc, sh_m, sh_l, c.s, c.h, row_first, (int64_t)c.slot * p.groups + group,
                               c.whole);
        __syncthreads();
    }
    if (p.joins && tid == 0) p.joins[blockIdx.x] = make_int4(c.s, c.h, c.parts, 0);
}

// ------------------------------------------------------------------ join --

// Joins the pieces of the problem that begins in a run and ends in a later one.
// A warp takes a query; where the pieces are many (few long sequences), the
// block's eight warps share a query's pieces.
constexpr int kJoinWarps = 8;
template <typename T, int D, bool RAW>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_combine_kernel(
    const __grid_constant__ Params p, int rows) {
    constexpr int LANES = D / 4;
    __shared__ float4 sh_v[kJoinWarps][32];
    __shared__ float sh_m[kJoinWarps], sh_l[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = blockIdx.x % p.groups;
    const int run = blockIdx.x / p.groups;
    // before the wait: the pass over the prefixes waits itself where it takes these sums, and what
    // it reads before that is there, since the pass in front of this join has waited for it
    if (RAW) let_next_begin();
    wait_for_last();  // the pieces are written
    const int4 job = p.joins[blockIdx.x];
    const int s = job.x, h = job.y, parts = job.z;
    if (parts == 0) return;
    const int used = min(rows, p.R - group * rows);
    // the sum over pieces first, first + step, ...
    auto gather = [&](int r, int first, int step, float& m, float& l, float4& v) {
        m = -INFINITY;
        l = 0.f;
        v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = first; i < parts; i += step) {
            const int64_t at =
                ((int64_t)(2 * (run + i) + (i == 0 ? 1 : 0)) * p.groups + group) * rows + r;
            const float2 ml = *reinterpret_cast<const float2*>(p.partial_ml + at * 2);
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (lane < LANES) x = *reinterpret_cast<const float4*>(p.partial + at * D + lane * 4);
            const float mx = fmaxf(m, ml.x);
            const float f = weight(m, l, mx), g = weight(ml.x, ml.y, mx);
            m = mx;
            l = l * f + ml.y * g;
            v = make_float4(v.x * f + x.x * g, v.y * f + x.y * g, v.z * f + x.z * g,
                            v.w * f + x.w * g);
        }
    };
    auto write = [&](int r, float m, float l, float4 v) {
        const int row = group * rows + r;
        const int tk = row / p.G, hd = h * p.G + row - tk * p.G;
        if (lane < LANES) emit<T, D, RAW>(p, s, tk, hd, lane * 4, v, m, l);
    };
    float m, l;
    float4 v;
    if (parts <= 8) {
        for (int r = blockIdx.y * kJoinWarps + warp; r < used; r += gridDim.y * kJoinWarps) {
            gather(r, 0, 1, m, l, v);
            write(r, m, l, v);
        }
        return;
    }
    for (int r = blockIdx.y; r < used; r += gridDim.y) {
        gather(r, warp, kJoinWarps, m, l, v);
        __syncthreads();
        sh_v[warp][lane] = v;
        if (lane == 0) {
            sh_m[warp] = m;
            sh_l[warp] = l;
        }
        __syncthreads();
        if (warp != 0) continue;
        m = sh_m[0];
#pragma unroll
        for (int w = 1; w < kJoinWarps; ++w) m = fmaxf(m, sh_m[w]);
        l = 0.f;
        v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            const float f = weight(sh_m[w], sh_l[w], m);
            const float4 x = sh_v[w][lane];
            v.x += x.x * f; v.y += x.y * f; v.z += x.z * f; v.w += x.w * f;
            l += sh_l[w] * f;
        }
        write(r, m, l, v);
    }
}

Params params(const AttnArgs& a, const AttnPlan& pl) {
    Params p{};
    p.k = static_cast<const uint8_t*>(a.bits == 4 ? a.q4p.k_codes : (a.bits == 8 ? a.q8p.k_codes : a.k));
    p.v = static_cast<const uint8_t*>(a.bits == 4 ? a.q4p.v_codes : (a.bits == 8 ? a.q8p.v_codes : a.v));
    p.ks = a.bits == 8 ? reinterpret_cast<const uint8_t*>(a.q8p.k_scales)
                       : reinterpret_cast<const uint8_t*>(a.q4p.k_scales);
    p.vs = a.bits == 8 ? reinterpret_cast<const uint8_t*>(a.q8p.v_scales)
                       : reinterpret_cast<const uint8_t*>(a.q4p.v_scales);
    p.table = a.pg.table;
    p.lens = a.lens;
    p.q = static_cast<const __nv_bfloat16*>(a.q.data);
    p.out = static_cast<__nv_bfloat16*>(a.out.data);
    p.num_seqs = (int)a.num_seqs;
    p.q_seq = a.q.seq; p.q_tok = a.q.tok; p.q_head = a.q.head;
    p.o_seq = a.out.seq; p.o_tok = a.out.tok; p.o_head = a.out.head;
    p.lse = a.lse;
    p.raw = a.raw;
    p.raw_ml = a.raw_ml;
    p.partial = a.partial;
    const int64_t slots = 2 * (int64_t)pl.runs * pl.groups;
    p.partial_ml = a.partial + slots * pl.rows * a.d;
    p.joins = pl.join ? reinterpret_cast<int4*>(p.partial_ml + slots * pl.rows * 2) : nullptr;
    p.H = a.pg.H; p.G = a.G; p.T = a.n_new; p.R = a.n_new * a.G;
    p.groups = pl.groups; p.runs = pl.runs; p.max_rows = a.max_rows;
    p.lead = pl.lead;
    p.cluster = pl.cluster;
    p.max_blocks = a.pg.max_blocks; p.log2bs = a.pg.log2bs; p.num_blocks = a.pg.num_blocks;
    // a scale of (almost) nothing counts as one that still orders the logits
    const float x = a.scale * kLog2e, y = x < 0.f ? -x : x;
    p.scale = y < 1e-30f ? 1e-30f : y;
    p.slack = 8.f / p.scale;
    p.flip = x < 0.f ? 0x80008000u : 0u;
    p.status = a.status;
    return p;
}

template <int D, int NT, int BITS, bool TWO>
cudaError_t go(const Params& p, unsigned ctas, cudaStream_t s) {
    using S = Stage<D, BITS>;
    constexpr int ring = kWarps * S::DEPTH * S::BYTES, join = kWarps * 8 * NT * D * 4;
    constexpr int bytes = ring > join ? ring : join;
    auto kern = attn_kernel<D, NT, BITS, TWO>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, bytes, done);
    if (e != cudaSuccess) return e;
    // as launch_early, with a cluster
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = p.cluster ? p.cluster : 1;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = p.cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}
template <int BITS>
cudaError_t go(const Params& p, int d, int rows, unsigned ctas, cudaStream_t s) {
    if (d == 128 && p.R > kTwoQueries) return go<128, 2, BITS, false>(p, ctas, s);
    if (d == 128)
        return rows == 8 ? go<128, 1, BITS, true>(p, ctas, s) : go<128, 2, BITS, true>(p, ctas, s);
    return rows == 8 ? go<64, 1, BITS, true>(p, ctas, s)
                     : (rows == 16 ? go<64, 2, BITS, true>(p, ctas, s)
                                   : go<64, 4, BITS, false>(p, ctas, s));
}
template <int D>
cudaError_t go32(const Params& p, unsigned ctas, cudaStream_t s) {
    constexpr int bytes = kWarps * Stage32<D>::DEPTH * Stage32<D>::BYTES;
    static_assert(bytes >= kWarps * 8 * D * 4, "the rings hold the join");
    auto kern = attn_f32_kernel<D>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, bytes, done);
    if (e != cudaSuccess) return e;
    return launch_early(kern, ctas, kWarps * 32, bytes, s, p);
}

bool is_f32(const AttnArgs& a) { return !a.bits && a.dtype == RKV_DTYPE_FP32; }

}  // namespace

// Up to how many units a cluster of eight takes a problem.  On the device, us,
// line and join against cluster (KV heads 8): one sequence of 256 rows 7.3 / 5.1,
// 1152 8.4 / 7.4, 4096 11.9 / 10.4, 8192 13.9 / 15.0; four of 1152 11.4 / 9.9, of
// 4096 18.1 / 16.6; at 4 bits one of 1152 9.2 / 7.4, of 4096 10.5 / 9.7.
constexpr int kClusterUnits = 64;

// Blocks that an SM holds at once: shared memory for two (one with fp32 rows of 128), with
// packed rows and 8 queries registers for three.
static int resident(const AttnArgs& a, int rows) {
    return is_f32(a) && a.d == 128 ? 1 : (a.bits && rows == 8 ? 3 : 2);
}

AttnPlan attn_plan(const AttnArgs& a) {
    AttnPlan pl;
    const int R = a.n_new * a.G;
    // queries a block holds: what the registers take beside the output (32 at
    // head_dim 64); more queries share the rows through L2
    const int most = is_f32(a) ? 8 : (a.d == 64 ? 32 : 16);
    pl.rows = R <= 8 ? 8 : (R <= 16 ? 16 : 32);
    if (pl.rows > most) pl.rows = most;
    pl.groups = (R + pl.rows - 1) / pl.rows;
    pl.unit = kWarps * (is_f32(a) ? 16 : (a.bits ? Stage<128, 4>::KEYS
                                               : (a.d == 128 ? Stage<128, 0>::KEYS
                                                             : Stage<64, 0>::KEYS)));
    const int sms = tc::sm_count(), blocks = sms * resident(a, pl.rows);
    const int64_t per = ((int64_t)a.max_rows + pl.unit - 1) / pl.unit, problems = a.num_seqs * a.pg.H;
    // a few short sequences: a cluster for each problem, one launch
    if (!is_f32(a) && per > 1 && per <= kClusterUnits && problems * pl.groups * kCluster <= 2 * sms) {
        pl.cluster = per >= 5 ? 8 : (per >= 3 ? 4 : 2);
        pl.runs = (int)problems;
        return pl;
    }
    const int64_t units = problems * per;
    // a problem's beginning and end cost about as much as this many units (64
    // ragged sequences of 131 .. 4224 rows, us at 0, 1, 2, 4, 8: bf16 103, 102,
    // 95, 95, 96; 4 bits 64, 60, 56, 58, 62; 8 new tokens, head_dim 64: 72, 70,
    // 66, 61, 61; 8 bits at 1, 2, 4 of their longer ones: 62, 59, 61, 8 new tokens
    // 64, 60, 57)
    pl.lead = a.bits == 4 || (a.bits == 8 && pl.rows == 8) ? 2 : 4;
    int64_t runs = (blocks + pl.groups - 1) / pl.groups;
    if (runs > units) runs = units;
    pl.runs = (int)runs;
    pl.join = a.max_rows > pl.unit;
    // two pieces of a run, and what it leaves to join (4 words)
    pl.partial_floats =
        pl.join ? (size_t)pl.runs * pl.groups * (2 * pl.rows * (a.d + 2) + 4) : 0;
    return pl;
}

// Runs are rounded up to whole groups, so a plan with fewer groups may have more blocks
// (7 queries a KV head, head_dim 128: 306 with 6 new tokens, 304 with 8).  This is at least
// that of every plan for fewer sequences, tokens or rows: rows and groups grow with the
// queries, units with everything, and 16 queries take more than 8 of three blocks an SM.
size_t attn_most_floats(const AttnArgs& a) {
    const AttnPlan pl = attn_plan(a);
    if (!pl.join) return 0;
    const int64_t units = a.num_seqs * a.pg.H * (((int64_t)a.max_rows + pl.unit - 1) / pl.unit) * pl.groups;
    const int64_t blocks = (int64_t)tc::sm_count() * resident(a, pl.rows) + pl.groups - 1;
    return (size_t)(units < blocks ? units : blocks) * (2 * pl.rows * (a.d + 2) + 4);
}

cudaError_t launch_attention(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s) {
    const unsigned ctas = (unsigned)(pl.runs * pl.groups * (pl.cluster ? pl.cluster : 1));
    if (ctas == 0) return cudaSuccess;
    const Params p = params(a, pl);
    if (is_f32(a)) return a.d == 128 ? go32<128>(p, ctas, s) : go32<64>(p, ctas, s);
    if (a.bits == 8) return go<8>(p, a.d, pl.rows, ctas, s);
    return a.bits == 4 ? go<4>(p, a.d, pl.rows, ctas, s) : go<0>(p, a.d, pl.rows, ctas, s);
}

template <typename T, int D>
cudaError_t go_join(const Params& p, const AttnPlan& pl, cudaStream_t s) {
    // most blocks find nothing to join.  With about as many problems as runs, or
    // more, the pieces of one are few and a block's warps take a query each;
    // otherwise a block takes a query.
    const int blocks = pl.runs * pl.groups, used = p.R < pl.rows ? p.R : pl.rows;
    const bool few = (int64_t)p.num_seqs * p.H * 8 >= pl.runs;
    const int y = few ? (used + kJoinWarps - 1) / kJoinWarps : used;
    // begins while the pieces are still being written and waits for them itself
    return launch_early(p.raw ? attn_combine_kernel<T, D, true> : attn_combine_kernel<T, D, false>,
                        dim3((unsigned)blocks, (unsigned)y), kJoinWarps * 32, 0, s, p, pl.rows);
}

cudaError_t launch_attention_combine(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s) {
    if (pl.runs == 0 || !pl.join) return cudaSuccess;
    const Params p = params(a, pl);
    if (is_f32(a)) return a.d == 128 ? go_join<float, 128>(p, pl, s) : go_join<float, 64>(p, pl, s);
    return a.d == 128 ? go_join<__nv_bfloat16, 128>(p, pl, s) : go_join<__nv_bfloat16, 64>(p, pl, s);
}

}  // namespace rkv
