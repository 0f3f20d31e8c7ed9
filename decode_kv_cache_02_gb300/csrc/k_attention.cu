// k_attention.cu -- attention of a few new tokens over a paged cache, bf16 or
// held in 4 bits: out = softmax(scale * q K^T) V for each KV head's group of
// query heads.
//
// One pass over the cache with a running maximum and sum.  Every warp is on
// its own: it takes every fourth stage of its block's chunk of rows, copies it
// into its own ring of shared memory (cp.async through the block table, rows
// past the sequence filled with zeros), and keeps the maxima, sums and the
// output of up to 16 queries in registers.  The warps of a block meet once, at
// the end; chunks of a sequence meet in attn_combine_kernel.
//
// The cache is read once, so the kernel is bound by HBM; the two products run
// on mma.sync m16n8k16 with the keys (values: the head's dimensions) as the
// 16 rows and the queries as the 8 columns, S^T = K Q^T and O^T = V^T P^T: a
// group of up to 8 queries then wastes nothing, the operands come from shared
// memory in the order the fragments want (the order of the contracted index is
// free as long as both sides share it), and P^T turns from an accumulator into
// an operand with one movmatrix per 8 x 8.
//
// 4 bits: codes become bf16 128 + c by placing the four bits in the mantissa
// (one shift, one logic op for two), exactly; a group's scale is applied to
// its own accumulator (K) or to the probabilities (V), in fp32, and the
// constant and the group's low value enter through sums over the queries (K)
// and over the probabilities (V).  So the products themselves are exact up to
// the rounding of p * scale to bf16.
//
// The running maximum moves only when a logit passes it by more than 8 (log2):
// p stays below 2^8 and the rescaling almost never runs.
#include "rkv_common.cuh"
#include "rkv_internal.h"

namespace rkv {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;

// Bytes and rows of one stage of a warp's ring.
template <int D, bool Q4>
struct Stage {
    static constexpr int W = D / 32;
    static constexpr int KEYS = Q4 ? 32 : (D == 128 ? 16 : 32);
    static constexpr int DEPTH = Q4 ? 4 : 3;
    static constexpr int ROW = Q4 ? D / 2 : D * 2;
    static constexpr int SROW = Q4 ? W * 4 : 0;
    static constexpr int V = KEYS * ROW;
    static constexpr int ks() { return 2 * KEYS * ROW; }
    static constexpr int vs() { return ks() + KEYS * SROW; }
    static constexpr int BYTES = 2 * KEYS * (ROW + SROW);
};

struct Params {
    const uint8_t* k;
    const uint8_t* v;
    const uint8_t* ks;
    const uint8_t* vs;
    const int32_t* table;
    const int32_t* lens;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    int64_t q_seq, q_tok, q_head, o_seq, o_tok, o_head;
    float* lse;
    float* partial;  // [problem][group][split][rows][D], then the (m, l) pairs
    float* partial_ml;
    int H, G, T, R, groups, splits, chunk, max_rows;
    int max_blocks, log2bs, num_blocks;
    float scale_log2;
    DeviceStatus* status;
};

RKV_DEV uint32_t smem_at(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
RKV_DEV void cp16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
}
RKV_DEV void cp8(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 8 : 0)
                 : "memory");
}
RKV_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
RKV_DEV void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
RKV_DEV void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                 uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
RKV_DEV uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
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
// Codes i and i + 4 (i: the word's nibbles shifted down) as bf16 128 + c.
RKV_DEV uint32_t codes_at(uint32_t w, int i) { return ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u; }

// The same less 136: -8 .. 7, exactly.  The values' product wants codes around
// zero: the rounding of p * scale is then that of the value itself, and long
// sums do not carry a constant that the tensor core's accumulator would cut
// digits for.
RKV_DEV uint32_t centred_at(uint32_t w, int i) {
    const uint32_t x = codes_at(w, i), m = 0x43084308u;  // 136, 136
    const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                     *reinterpret_cast<const __nv_bfloat162*>(&m));
    return *reinterpret_cast<const uint32_t*>(&y);
}

// Physical row (within 16) of row r of a key fragment.  Quarter-warp reads of
// K (two rows) and half-warp reads of V (four rows) then meet no bank twice,
// with the 16-byte units of a row permuted by unit_xor.
template <bool Q4>
RKV_DEV int phys(int r) {
    if constexpr (Q4) return r ^ ((r >> 1) & 1);
    return (r & 8) | ((r & 7) >> 1) | ((r & 1) << 2);
}
template <int D, bool Q4>
RKV_DEV int unit_xor(int row) {
    if constexpr (Q4) return D == 128 ? ((row >> 2) & 1) << 1 : 0;
    return ((row & 3) << 1) ^ (((row >> 2) & 1) << 2);
}

// Copies stage rows [row0, row0 + KEYS) of head h; lane i holds the block of
// row row0 + i (-1: zeros).
template <int D, bool Q4>
RKV_DEV void copy_stage(const Params& p, uint32_t dst, int h, int row0, int blk) {
    using S = Stage<D, Q4>;
    const int lane = threadIdx.x & 31;
    constexpr int UPR = S::ROW / 16;  // units per row
    const int u = lane % UPR;
    const int mask = (1 << p.log2bs) - 1;
#pragma unroll
    for (int i = 0; i < S::KEYS * UPR / 32; ++i) {
        const int r = i * (32 / UPR) + lane / UPR;
        const int b = __shfl_sync(0xffffffffu, blk, r);
        const bool ok = b >= 0;
        const int64_t row =
            ok ? ((((int64_t)b * p.H + h) << p.log2bs) | ((row0 + r) & mask)) : 0;
        const int64_t at = row * S::ROW + u * 16;
        const uint32_t to = dst + r * S::ROW + ((u ^ unit_xor<D, Q4>(r)) << 4);
        cp16(to, p.k + at, ok);
        cp16(to + S::V, p.v + at, ok);
    }
    if constexpr (Q4) {
        static_assert(S::KEYS == 32, "one lane per row");
        const bool ok = blk >= 0;
        const int64_t row =
            ok ? ((((int64_t)blk * p.H + h) << p.log2bs) | ((row0 + lane) & mask)) : 0;
        const int64_t at = row * S::SROW;
        const uint32_t to = dst + lane * S::SROW;
        if constexpr (S::SROW == 16) {
            cp16(to + S::ks(), p.ks + at, ok);
            cp16(to + S::vs(), p.vs + at, ok);
        } else {
            cp8(to + S::ks(), p.ks + at, ok);
            cp8(to + S::vs(), p.vs + at, ok);
        }
    }
}

// Logits (times scale, log2) of 16 keys of a bf16 stage.
template <int D, int NT>
RKV_DEV void logits_bf16(const uint8_t* st, int base, const uint32_t (&qf)[NT][D / 8],
                         float (&c)[NT][4]) {
    using S = Stage<D, false>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int pr = base + phys<false>(g), f = unit_xor<D, false>(pr);
    const uint8_t* row = st + pr * S::ROW;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] = 0.f;
#pragma unroll
    for (int ch = 0; ch < S::W; ++ch) {
        const int at = ((4 * ch + t) ^ f) << 4;
        const uint4 a = *reinterpret_cast<const uint4*>(row + at);
        const uint4 b = *reinterpret_cast<const uint4*>(row + 8 * S::ROW + at);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mma(c[n], a.x, b.x, a.y, b.y, qf[n][4 * ch], qf[n][4 * ch + 1]);
            mma(c[n], a.z, b.z, a.w, b.w, qf[n][4 * ch + 2], qf[n][4 * ch + 3]);
        }
    }
}

template <int D, int NT>
RKV_DEV void logits_q4(const uint8_t* st, int base, const uint32_t (&qf)[NT][D / 8],
                       const float (&qsum)[NT][D / 32][2], float (&c)[NT][4]) {
    using S = Stage<D, true>;
    constexpr int W = S::W;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int pr = base + phys<true>(g), f = unit_xor<D, true>(pr);
    uint32_t word[2][W], sc[2][W];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint8_t* row = st + (pr + 8 * k) * S::ROW;
        const uint8_t* srow = st + S::ks() + (pr + 8 * k) * S::SROW;
        if constexpr (W == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(row + ((t ^ f) << 4));
            word[k][0] = __byte_perm(x.x, x.z, 0x5410);
            word[k][1] = __byte_perm(x.x, x.z, 0x7632);
            word[k][2] = __byte_perm(x.y, x.w, 0x5410);
            word[k][3] = __byte_perm(x.y, x.w, 0x7632);
            const uint4 y = *reinterpret_cast<const uint4*>(srow);
            sc[k][0] = y.x; sc[k][1] = y.y; sc[k][2] = y.z; sc[k][3] = y.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(row + t * 8);
            word[k][0] = __byte_perm(x.x, x.y, 0x5410);
            word[k][1] = __byte_perm(x.x, x.y, 0x7632);
            const uint2 y = *reinterpret_cast<const uint2*>(srow);
            sc[k][0] = y.x; sc[k][1] = y.y;
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        uint32_t a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = codes_at(word[0][w], i);
            b[i] = codes_at(word[1][w], i);
        }
        float s[2], o[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            s[k] = __uint_as_float(sc[k][w] << 16);
            o[k] = fmaf(-128.f, s[k], __uint_as_float(sc[k][w] & 0xffff0000u));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            mma(x, a[0], b[0], a[1], b[1], qf[n][4 * w], qf[n][4 * w + 1]);
            mma(x, a[2], b[2], a[3], b[3], qf[n][4 * w + 2], qf[n][4 * w + 3]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c[n][i] = fmaf(s[i >> 1], x[i], fmaf(o[i >> 1], qsum[n][w][i & 1], c[n][i]));
        }
    }
}

// O^T += V^T P^T for 16 keys of a bf16 stage; pb: P^T as operand.  ONE: only
// for the queries (columns) in `cols` (bit 2 n + i), with the key pairs (2t,
// 2t+1) and (2t+8, 2t+9) masked by keep0 and keep1 (a half each).
template <int D, int NT, bool ONE>
RKV_DEV void values_bf16(const uint8_t* st, int base, const uint32_t (&pb)[NT][2], uint32_t keep0,
                         uint32_t keep1, uint32_t cols, float (&o)[D / 16][NT][4]) {
    using S = Stage<D, false>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint8_t* v = st + S::V;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int pr = base + phys<false>(2 * t + (k & 1) + 8 * (k >> 1));
            x[k] = *reinterpret_cast<const uint4*>(
                v + pr * S::ROW + (((8 * j + g) ^ unit_xor<D, false>(pr)) << 4));
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
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((cols >> (2 * n + (i & 1))) & 1u) o[4 * j + e][n][i] += y[i];
                }
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma(o[4 * j + e][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            }
        }
    }
}

// The same for a 4-bit stage; p: probabilities of 16 keys as accumulators lie.
// low: sum of p * (low + 8 scale).
template <int D, int NT>
RKV_DEV void values_q4(const uint8_t* st, int base, const float (&p)[NT][4], bool masked,
                       float (&o)[D / 16][NT][4], float (&low)[NT][D / 32][2]) {
    using S = Stage<D, true>;
    constexpr int W = S::W;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint32_t sc[2][W];
    {
        const int pr = base + phys<true>(g);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint8_t* srow = st + S::vs() + (pr + 8 * k) * S::SROW;
            if constexpr (W == 4) {
                const uint4 y = *reinterpret_cast<const uint4*>(srow);
                sc[k][0] = y.x; sc[k][1] = y.y; sc[k][2] = y.z; sc[k][3] = y.w;
            } else {
                const uint2 y = *reinterpret_cast<const uint2*>(srow);
                sc[k][0] = y.x; sc[k][1] = y.y;
            }
        }
    }
    uint32_t x[4][W / 2];  // a key's codes of its lane: two groups a word
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int pr = base + phys<true>(2 * t + (k & 1) + 8 * (k >> 1));
        const uint8_t* row = st + S::V + pr * S::ROW;
        if constexpr (W == 4) {
            const uint2 y = *reinterpret_cast<const uint2*>(
                row + (((g >> 1) ^ unit_xor<D, true>(pr)) << 4) + ((g & 1) << 3));
            x[k][0] = y.x; x[k][1] = y.y;
        } else {
            x[k][0] = *reinterpret_cast<const uint32_t*>(row + g * 4);
        }
    }
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const uint32_t sel = (w & 1) ? 0x7632 : 0x5410;
        const uint32_t u = __byte_perm(x[0][w >> 1], x[1][w >> 1], sel);
        const uint32_t v = __byte_perm(x[2][w >> 1], x[3][w >> 1], sel);
        uint32_t a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = centred_at(u, i);
            b[i] = centred_at(v, i);
        }
        float s[2], l[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            s[k] = __uint_as_float(sc[k][w] << 16);
            l[k] = fmaf(8.f, s[k], __uint_as_float(sc[k][w] & 0xffff0000u));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float y[4], z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = p[n][i] * s[i >> 1];
                z[i] = p[n][i] * l[i >> 1];
                if (masked && p[n][i] == 0.f) y[i] = z[i] = 0.f;  // a hidden row's NaN stays out
            }
            low[n][w][0] += z[0] + z[2];
            low[n][w][1] += z[1] + z[3];
            const uint32_t b0 = transpose8x8(pack(y[0], y[1])), b1 = transpose8x8(pack(y[2], y[3]));
            mma(o[2 * w][n], a[0], a[1], b[0], b[1], b0, b1);
            mma(o[2 * w + 1][n], a[2], a[3], b[2], b[3], b0, b1);
        }
    }
}

// The chunk of rows and the queries that a block works on.
struct Chunk {
    int64_t s, slot;
    int h, group, len, active, c0, c1;
};
RKV_DEV bool chunk_of(const Params& p, Chunk& c) {
    // groups of queries over the same rows are neighbours: the rows come from
    // HBM once and from L2 for the others
    const int64_t bid = blockIdx.x;
    c.group = (int)(bid % p.groups);
    const int64_t ps = bid / p.groups;
    const int split = (int)(ps % p.splits);
    const int64_t prob = ps / p.splits;
    c.s = prob / p.H;
    c.h = (int)(prob - c.s * p.H);
    c.len = p.lens[c.s];
    if (c.len < 0 || c.len > p.max_rows) {
        if (threadIdx.x == 0 && split == 0) set_error(p.status, kDevErrIndex, (unsigned)c.s);
        c.len = c.len < 0 ? 0 : p.max_rows;
    }
    c.active = c.len <= p.chunk ? 1 : (c.len + p.chunk - 1) / p.chunk;
    if (split >= c.active) return false;
    c.c0 = split * p.chunk;
    c.c1 = c.len - c.c0 < p.chunk ? c.len : c.c0 + p.chunk;
    c.slot = (prob * p.groups + c.group) * p.splits + split;
    return true;
}

// What a part with maximum m and sum l counts beside a common maximum mx: an
// empty part nothing, one whose logits are all NaN its NaN.
RKV_DEV float weight(float m, float l, float mx) {
    if (m == -INFINITY) return l != l ? 1.f : 0.f;
    return ex2(m - mx);
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

// Joins the warps' weighted sums in acc [kWarps][ROWS][D] and writes the rows:
// the output where the chunk is the whole sequence, else its part.
template <typename T, int D, int ROWS>
RKV_DEV void finish(const Params& p, const float* acc, const float (&sh_m)[kWarps][ROWS],
                    const float (&sh_l)[kWarps][ROWS], int64_t s, int h, int row_first,
                    int64_t slot, bool whole) {
    T* out = reinterpret_cast<T*>(p.out);
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
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int tk = row / p.G, hd = h * p.G + row - tk * p.G;
            store4(out + s * p.o_seq + tk * p.o_tok + hd * p.o_head + d,
                   make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
            if (d == 0 && p.lse)
                p.lse[(s * p.T + tk) * (int64_t)p.H * p.G + hd] =
                    sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
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

// NT * 8 queries of one KV head's group against one chunk of its rows.
template <int D, int NT, bool Q4>
__global__ void __launch_bounds__(kWarps * 32) attn_kernel(const __grid_constant__ Params p) {
    using S = Stage<D, Q4>;
    constexpr int ROWS = 8 * NT, W = D / 32, KT = S::KEYS / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t valid[kWarps][S::DEPTH];
    __shared__ float sh_m[kWarps][ROWS], sh_l[kWarps][ROWS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;

    Chunk c;
    if (!chunk_of(p, c)) return;
    const int64_t s = c.s;
    const int h = c.h, len = c.len, c0 = c.c0, c1 = c.c1;
    const int row_first = c.group * ROWS;  // first query row (token * G + head of the group)

    // queries as the second operand: lane (g, t) holds row g, values 32 w + 8 t ..
    uint32_t qf[NT][D / 8];
    [[maybe_unused]] float qsum[NT][W][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = row_first + 8 * n + g;
        const bool ok = r < p.R;
        const int tk = ok ? r / p.G : 0, hd = ok ? r - tk * p.G : 0;
        const __nv_bfloat16* q = p.q + s * p.q_seq + tk * p.q_tok + (int64_t)(h * p.G + hd) * p.q_head;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (ok) x = *reinterpret_cast<const uint4*>(q + 32 * w + 8 * t);
            if constexpr (Q4) {
                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum += __uint_as_float(y[i] << 16) + __uint_as_float(y[i] & 0xffff0000u);
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                qsum[n][w][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
                qsum[n][w][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
                x = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                               __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
            }
            qf[n][4 * w] = x.x;
            qf[n][4 * w + 1] = x.y;
            qf[n][4 * w + 2] = x.z;
            qf[n][4 * w + 3] = x.w;
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

    float m[NT][2], l[NT][2], o[D / 16][NT][4];
    [[maybe_unused]] float low[NT][W][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[n][i] = -INFINITY;
            l[n][i] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < D / 16; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[e][n][i] = 0.f;
        if constexpr (Q4) {
#pragma unroll
            for (int w = 0; w < W; ++w) low[n][w][0] = low[n][w][1] = 0.f;
        }
    }

    const int32_t* table = p.table + s * p.max_blocks;
    uint8_t* ring = smem + warp * (S::DEPTH * S::BYTES);
    const int stages = (c1 - c0 + S::KEYS - 1) / S::KEYS;
    const int mine = warp < stages ? (stages - warp + kWarps - 1) / kWarps : 0;
    auto row_of = [&](int it) { return c0 + (warp + it * kWarps) * S::KEYS; };
    auto block_of = [&](int it) {  // the block of this lane's row of stage it
        int b = -1;
        const int r = row_of(it) + lane;
        if (it < mine && lane < S::KEYS && r < c1) {
            b = table[r >> p.log2bs];
            if ((unsigned)b >= (unsigned)p.num_blocks) {
                set_error(p.status, kDevErrIndex, (unsigned)r);
                b = -1;
            }
        }
        return b;
    };
    auto issue = [&](int it, int blk) {
        if (it < mine) {
            const int slot = it % S::DEPTH;
            const uint32_t ok = __ballot_sync(0xffffffffu, blk >= 0);
            if (lane == 0) valid[warp][slot] = ok;
            copy_stage<D, Q4>(p, smem_at(ring + slot * S::BYTES), h, row_of(it), blk);
        }
        cp_commit();
    };
    {
        int blk[S::DEPTH - 1];
#pragma unroll
        for (int i = 0; i < S::DEPTH - 1; ++i) blk[i] = block_of(i);
#pragma unroll
        for (int i = 0; i < S::DEPTH - 1; ++i) issue(i, blk[i]);
    }
    int next = block_of(S::DEPTH - 1);

    for (int it = 0; it < mine; ++it) {
        cp_wait<S::DEPTH - 2>();
        __syncwarp();  // the stage is there, and the slot refilled next has been read
        const int blk = next;
        next = block_of(it + S::DEPTH);
        issue(it + S::DEPTH - 1, blk);

        const uint8_t* st = ring + (it % S::DEPTH) * S::BYTES;
        const uint32_t ok = valid[warp][it % S::DEPTH];
        const int row0 = row_of(it);
        const bool masked = ok != (S::KEYS == 32 ? 0xffffffffu : (1u << (S::KEYS & 31)) - 1u) ||
                            row0 + S::KEYS - 1 > all_see;
        float x[KT][NT][4];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            if constexpr (Q4)
                logits_q4<D, NT>(st, kt * 16, qf, qsum, x[kt]);
            else
                logits_bf16<D, NT>(st, kt * 16, qf, x[kt]);
        }
        bool grow = false;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[kt][n][i] *= p.scale_log2;
                    if (masked) {
                        const int r = kt * 16 + phys<Q4>(g + 8 * (i >> 1));
                        if (row0 + r > last[n][i & 1] || !((ok >> r) & 1u)) x[kt][n][i] = -INFINITY;
                    }
                    grow |= x[kt][n][i] > m[n][i & 1] + kSlack;
                }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = m[n][i];
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) mx = fmaxf(mx, fmaxf(x[kt][n][i], x[kt][n][i + 2]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float f = m[n][i] == -INFINITY ? 0.f : ex2(m[n][i] - mx);
                    m[n][i] = mx;
                    l[n][i] *= f;
#pragma unroll
                    for (int e = 0; e < D / 16; ++e) {
                        o[e][n][i] *= f;
                        o[e][n][i + 2] *= f;
                    }
                    if constexpr (Q4) {
#pragma unroll
                        for (int w = 0; w < W; ++w) low[n][w][i] *= f;
                    }
                }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float ref = m[n][i] == -INFINITY ? 0.f : m[n][i];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    x[kt][n][i] = ex2(x[kt][n][i] - ref);
                    x[kt][n][i + 2] = ex2(x[kt][n][i + 2] - ref);
                    l[n][i] += x[kt][n][i] + x[kt][n][i + 2];
                }
            }
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            if constexpr (Q4) {
                values_q4<D, NT>(st, kt * 16, x[kt], masked, o, low);
            } else {
                uint32_t pb[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    pb[n][0] = transpose8x8(pack(x[kt][n][0], x[kt][n][1]));
                    pb[n][1] = transpose8x8(pack(x[kt][n][2], x[kt][n][3]));
                }
                if (!masked || p.T == 1) {
                    // (rows nobody sees are zeros here: rows past len and rows without a block)
                    values_bf16<D, NT, false>(st, kt * 16, pb, ~0u, ~0u, ~0u, o);
                } else {
                    // rows that only some of the tokens see: one token at a time, so that what
                    // a hidden row holds (an infinity, a NaN) cannot reach the others
                    const int t0 = row_first / p.G;
                    const int t1 = (min(p.R, row_first + ROWS) - 1) / p.G;
                    for (int tk = t0; tk <= t1; ++tk) {
                        const int see = len - p.T + tk;
                        uint32_t keep[2], cols = 0u;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int ra = row0 + kt * 16 + phys<Q4>(2 * t + 8 * k);
                            const int rb = row0 + kt * 16 + phys<Q4>(2 * t + 1 + 8 * k);
                            keep[k] = (ra <= see ? 0xffffu : 0u) | (rb <= see ? 0xffff0000u : 0u);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int r = row_first + 8 * n + 2 * t + i;
                                if (r < p.R && r / p.G == tk) cols |= 1u << (2 * n + i);
                            }
                        values_bf16<D, NT, true>(st, kt * 16, pb, keep[0], keep[1], cols, o);
                    }
                }
            }
        }
    }
    cp_wait<0>();

    // sums over the lanes that share a query
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int sh = 4; sh <= 16; sh <<= 1)
                l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], sh);
            if constexpr (Q4) {
#pragma unroll
                for (int w = 0; w < W; ++w)
#pragma unroll
                    for (int sh = 4; sh <= 16; sh <<= 1)
                        low[n][w][i] += __shfl_xor_sync(0xffffffffu, low[n][w][i], sh);
            }
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
            const float f = weight(m[n][i], l[n][i], row_max(sh_m, r));
            float* dst = acc + ((size_t)warp * ROWS + r) * D;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
                // the pair of dimensions this accumulator's rows g and g + 8 stand for
                const int d = Q4 ? 32 * (e / 2) + 4 * g + 2 * (e % 2) : 64 * (e / 4) + 8 * g + 2 * (e % 4);
                float a = o[e][n][i], b = o[e][n][i + 2];
                if constexpr (Q4) {
                    a += low[n][e / 2][i];
                    b += low[n][e / 2][i];
                }
                *reinterpret_cast<float2*>(dst + d) = make_float2(a * f, b * f);
            }
        }
    __syncthreads();

    finish<__nv_bfloat16, D, ROWS>(p, acc, sh_m, sh_l, s, h, row_first, c.slot, c.active == 1);
}

// ------------------------------------------------------------ fp32 pools --
// The same pass on the CUDA cores: 8 queries a block, a warp takes 16 rows at
// a time.  For the logits a lane owns one key and half of the dimensions; for
// the values four dimensions (head_dim 64: and every other key).  The
// 16-byte units of row r lie at unit ^ (r mod 8), so neither read meets a bank
// twice.
template <int D>
struct Stage32 {
    static constexpr int KEYS = 16, DEPTH = 2, ROW = D * 4, V = KEYS * ROW, BYTES = 2 * V;
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attn_f32_kernel(const __grid_constant__ Params p) {
    using S = Stage32<D>;
    constexpr int ROWS = 8, UPR = D / 4;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sh_q[ROWS][D];
    __shared__ float sh_p[kWarps][S::KEYS][ROWS];
    __shared__ float sh_m[kWarps][ROWS], sh_l[kWarps][ROWS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int key = lane & 15, side = lane >> 4;

    Chunk c;
    if (!chunk_of(p, c)) return;
    const int row_first = c.group * ROWS;
    const float* q32 = reinterpret_cast<const float*>(p.q);
    for (int e = tid; e < ROWS * UPR; e += kWarps * 32) {
        const int r = row_first + e / UPR, u = e % UPR;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < p.R) {
            const int tk = r / p.G, hd = c.h * p.G + r - tk * p.G;
            x = *reinterpret_cast<const float4*>(q32 + c.s * p.q_seq + tk * p.q_tok +
                                                 hd * p.q_head + 4 * u);
        }
        *reinterpret_cast<float4*>(&sh_q[e / UPR][4 * u]) = x;
    }
    __syncthreads();
    int last[ROWS];
    float m[ROWS], l[ROWS], o[ROWS][4];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        last[r] = row_first + r < p.R ? c.len - p.T + (row_first + r) / p.G : c.len - 1;
        m[r] = -INFINITY;
        l[r] = 0.f;
        o[r][0] = o[r][1] = o[r][2] = o[r][3] = 0.f;
    }
    const int all_see = c.len - p.T + row_first / p.G;

    const int32_t* table = p.table + c.s * p.max_blocks;
    uint8_t* ring = smem + warp * (S::DEPTH * S::BYTES);
    const int stages = (c.c1 - c.c0 + S::KEYS - 1) / S::KEYS;
    const int mine = warp < stages ? (stages - warp + kWarps - 1) / kWarps : 0;
    uint32_t valid[2] = {0u, 0u};
    auto issue = [&](int it) {
        if (it < mine) {
            const int row0 = c.c0 + (warp + it * kWarps) * S::KEYS;
            int blk = -1;
            if (lane < S::KEYS && row0 + lane < c.c1) {
                blk = table[(row0 + lane) >> p.log2bs];
                if ((unsigned)blk >= (unsigned)p.num_blocks) {
                    set_error(p.status, kDevErrIndex, (unsigned)(row0 + lane));
                    blk = -1;
                }
            }
            valid[1] = __ballot_sync(0xffffffffu, blk >= 0);
            const uint32_t dst = smem_at(ring + (it % S::DEPTH) * S::BYTES);
            const int u = lane % UPR;
#pragma unroll 4
            for (int i = 0; i < S::KEYS * UPR / 32; ++i) {
                const int r = i * (32 / UPR) + lane / UPR;
                const int b = __shfl_sync(0xffffffffu, blk, r);
                const int64_t row = b >= 0 ? ((((int64_t)b * p.H + c.h) << p.log2bs) |
                                              ((row0 + r) & ((1 << p.log2bs) - 1)))
                                           : 0;
                const uint32_t to = dst + r * S::ROW + ((u ^ (r & 7)) << 4);
                cp16(to, p.k + row * S::ROW + u * 16, b >= 0);
                cp16(to + S::V, p.v + row * S::ROW + u * 16, b >= 0);
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
            x[r] *= p.scale_log2;
            if (masked && (row0 + key > last[r] || !((ok >> key) & 1u))) x[r] = -INFINITY;
            grow |= x[r] > m[r] + kSlack;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const float mx = fmaxf(m[r], warp_max(x[r]));
                const float f = m[r] == -INFINITY ? 0.f : ex2(m[r] - mx);
                m[r] = mx;
                l[r] *= f;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[r][i] *= f;
            }
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            x[r] = ex2(x[r] - (m[r] == -INFINITY ? 0.f : m[r]));
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
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        l[r] = warp_sum(l[r]);
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
        const float f = weight(m[r], l[r], row_max(sh_m, r));
        if (lane < UPR)
            *reinterpret_cast<float4*>(acc + ((size_t)warp * ROWS + r) * D + 4 * lane) =
                make_float4(o[r][0] * f, o[r][1] * f, o[r][2] * f, o[r][3] * f);
    }
    __syncthreads();
    finish<float, D, ROWS>(p, acc, sh_m, sh_l, c.s, c.h, row_first, c.slot, c.active == 1);
}

// Joins the chunks of one query row: a warp per (problem, query).
template <typename T, int D>
__global__ void __launch_bounds__(128) attn_combine_kernel(const __grid_constant__ Params p,
                                                           T* out, int rows, int64_t total) {
    const int lane = threadIdx.x & 31;
    const int64_t wid = blockIdx.x * 4ll + (threadIdx.x >> 5);
    if (wid >= total) return;
    const int64_t prob = wid / p.R;
    const int row = (int)(wid - prob * p.R);
    const int64_t s = prob / p.H;
    const int h = (int)(prob - s * p.H);
    int len = p.lens[s];
    len = len < 0 ? 0 : (len > p.max_rows ? p.max_rows : len);
    const int active = len <= p.chunk ? 1 : (len + p.chunk - 1) / p.chunk;
    if (active == 1) return;  // written by the chunk itself
    const int64_t first = (prob * p.groups + row / rows) * p.splits;
    const int r = row % rows;
    float mx = -INFINITY;
    for (int i = lane; i < active; i += 32)
        mx = fmaxf(mx, p.partial_ml[((first + i) * rows + r) * 2]);
    mx = warp_max(mx);
    constexpr int PER = D / 32;
    float v[PER], sum = 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) v[k] = 0.f;
#pragma unroll 4
    for (int i = 0; i < active; ++i) {
        const int64_t at = (first + i) * rows + r;
        const float2 ml = *reinterpret_cast<const float2*>(p.partial_ml + at * 2);
        const float f = weight(ml.x, ml.y, mx);
        sum += ml.y * f;
        const float* src = p.partial + at * D + lane * PER;
#pragma unroll
        for (int k = 0; k < PER; ++k) v[k] += f == 0.f ? 0.f : src[k] * f;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int tk = row / p.G, hd = h * p.G + row - tk * p.G;
    T* dst = out + s * p.o_seq + tk * p.o_tok + hd * p.o_head + lane * PER;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if constexpr (sizeof(T) == 2) dst[k] = __float2bfloat16_rn(v[k] * inv);
        else dst[k] = v[k] * inv;
    }
    if (lane == 0 && p.lse)
        p.lse[(s * p.T + tk) * (int64_t)p.H * p.G + hd] =
            sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

Params params(const AttnArgs& a, const AttnPlan& pl) {
    Params p{};
    p.k = static_cast<const uint8_t*>(a.q4 ? a.q4p.k_codes : a.k);
    p.v = static_cast<const uint8_t*>(a.q4 ? a.q4p.v_codes : a.v);
    p.ks = reinterpret_cast<const uint8_t*>(a.q4p.k_scales);
    p.vs = reinterpret_cast<const uint8_t*>(a.q4p.v_scales);
    p.table = a.pg.table;
    p.lens = a.lens;
    p.q = static_cast<const __nv_bfloat16*>(a.q.data);
    p.out = static_cast<__nv_bfloat16*>(a.out.data);
    p.q_seq = a.q.seq; p.q_tok = a.q.tok; p.q_head = a.q.head;
    p.o_seq = a.out.seq; p.o_tok = a.out.tok; p.o_head = a.out.head;
    p.lse = a.lse;
    const int64_t slots = a.num_seqs * a.pg.H * pl.groups * pl.splits;
    p.partial = a.partial;
    p.partial_ml = a.partial + slots * pl.rows * a.d;
    p.H = a.pg.H; p.G = a.G; p.T = a.n_new; p.R = a.n_new * a.G;
    p.groups = pl.groups; p.splits = pl.splits; p.chunk = pl.chunk; p.max_rows = a.max_rows;
    p.max_blocks = a.pg.max_blocks; p.log2bs = a.pg.log2bs; p.num_blocks = a.pg.num_blocks;
    p.scale_log2 = a.scale * kLog2e;
    p.status = a.status;
    return p;
}

template <int D, int NT, bool Q4>
cudaError_t go(const Params& p, int64_t ctas, cudaStream_t s) {
    using S = Stage<D, Q4>;
    constexpr int ring = kWarps * S::DEPTH * S::BYTES, join = kWarps * 8 * NT * D * 4;
    constexpr int bytes = ring > join ? ring : join;
    auto kern = attn_kernel<D, NT, Q4>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)ctas, kWarps * 32, bytes, s>>>(p);
    return cudaGetLastError();
}
template <int D, bool Q4>
cudaError_t go(const Params& p, int rows, int64_t ctas, cudaStream_t s) {
    return rows == 8 ? go<D, 1, Q4>(p, ctas, s) : go<D, 2, Q4>(p, ctas, s);
}

template <int D>
cudaError_t go32(const Params& p, int64_t ctas, cudaStream_t s) {
    constexpr int bytes = kWarps * Stage32<D>::DEPTH * Stage32<D>::BYTES;
    static_assert(bytes >= kWarps * 8 * D * 4, "the rings hold the join");
    auto kern = attn_f32_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)ctas, kWarps * 32, bytes, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

AttnPlan attn_plan(const AttnArgs& a) {
    AttnPlan pl;
    const int R = a.n_new * a.G;
    const bool f32 = !a.q4 && a.dtype == RKV_DTYPE_FP32;
    pl.rows = R <= 8 || f32 ? 8 : 16;
    pl.groups = (R + pl.rows - 1) / pl.rows;
    const int64_t units = a.num_seqs * a.pg.H * pl.groups;
    const int step = 128;  // rows of one stage of every warp, at most
    // about two blocks for each of 152 SMs; several times that when sequences
    // may differ in length, so that the long ones spread
    const int64_t target = a.num_seqs == 1 ? 304 : 304 * 6;
    int64_t want = units > 0 ? (target + units - 1) / units : 1;
    const int64_t most = (a.max_rows + step - 1) / step;
    if (want > most) want = most;
    if (want > 256) want = 256;
    if (want < 1) want = 1;
    const int64_t per = (a.max_rows + want - 1) / want;
    pl.chunk = (int)((per + step - 1) / step * step);
    pl.splits = (a.max_rows + pl.chunk - 1) / pl.chunk;
    pl.ctas = units * pl.splits;
    pl.partial_floats = pl.splits > 1 ? (size_t)pl.ctas * pl.rows * (a.d + 2) : 0;
    return pl;
}

cudaError_t launch_attention(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s) {
    if (pl.ctas == 0) return cudaSuccess;
    const Params p = params(a, pl);
    if (!a.q4 && a.dtype == RKV_DTYPE_FP32)
        return a.d == 128 ? go32<128>(p, pl.ctas, s) : go32<64>(p, pl.ctas, s);
    if (a.q4)
        return a.d == 128 ? go<128, true>(p, pl.rows, pl.ctas, s) : go<64, true>(p, pl.rows, pl.ctas, s);
    return a.d == 128 ? go<128, false>(p, pl.rows, pl.ctas, s) : go<64, false>(p, pl.rows, pl.ctas, s);
}

cudaError_t launch_attention_combine(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s) {
    if (pl.ctas == 0 || pl.splits <= 1) return cudaSuccess;
    const Params p = params(a, pl);
    const int64_t total = a.num_seqs * a.pg.H * (int64_t)p.R;
    const unsigned grid = (unsigned)((total + 3) / 4);
    const bool f32 = !a.q4 && a.dtype == RKV_DTYPE_FP32;
    if (f32) {
        float* out = static_cast<float*>(a.out.data);
        if (a.d == 128) attn_combine_kernel<float, 128><<<grid, 128, 0, s>>>(p, out, pl.rows, total);
        else attn_combine_kernel<float, 64><<<grid, 128, 0, s>>>(p, out, pl.rows, total);
    } else {
        if (a.d == 128) attn_combine_kernel<__nv_bfloat16, 128><<<grid, 128, 0, s>>>(p, p.out, pl.rows, total);
        else attn_combine_kernel<__nv_bfloat16, 64><<<grid, 128, 0, s>>>(p, p.out, pl.rows, total);
    }
    return cudaGetLastError();
}

}  // namespace rkv
