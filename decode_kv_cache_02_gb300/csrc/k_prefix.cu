// k_prefix.cu -- attention of a batch whose sequences share long prefixes: the pass
// over the prefixes on the CUDA cores (fp32 pools, and bf16 pools in blocks too small
// for the tensor-core pass, k_prefix_tc.cu), and the join of its pieces.
//
// out = sum_j p_j V_j over the rows of the prefix, then the sequence's own: the softmax
// over both is that of the sums over each, brought to a common maximum.  The own rows'
// sums come from the attention over the cache (k_attention.cu), which goes first; here
// the queries of all sequences of a prefix are the rows of one product, so the prefix
// is read once for all of them.
//
// CUDA cores: a block takes 64 queries and 64 rows at a time through shared memory; a
// thread holds 8 queries x 4 rows of the logits (rows tx, tx + 16, ..: reads of 8
// neighbouring rows of 528 bytes meet no bank twice) and 8 queries x D / 16 of the
// output, so four FMAs stand against each word that is read.
//
// Measured (one GB300, under the profiler, cold): fp32, 2 prefixes to 2049 rows, 24 sequences,
// 4 KV heads, head_dim 128: the pass 28 us (253 registers, two blocks an SM, one wave), its join
// 15; FMAs alone would take 5.  What bounds the pass: a step waits for all of its copies before
// it multiplies (one buffer, so every 64 rows pay a trip to memory, which only the SM's other
// block fills), and with 48 queries a prefix and head a quarter of each tile is empty.  The join
// waits for memory and for its first warp's look at what the blocks left.
#include <atomic>

#include "rkv_prefix.cuh"

namespace rkv {
namespace prefix {
namespace {

constexpr int kTile = 64, kUnit = 64, kThreads = 128;
constexpr int kMaxTeam = 8;
// Scratch of a block: two pieces of a tile, and what it leaves to join (4 words).
constexpr size_t block_floats(int tile, int d) { return 2 * (size_t)tile * (d + 2) + 4; }

RKV_DEV uint32_t smem_at(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// Four values into shared memory as fp32 (ok: there are any, else zeros).
RKV_DEV void fetch4(float* dst, const float* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_at(dst)), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
}
RKV_DEV void fetch4(float* dst, const __nv_bfloat16* src, bool ok) {
    uint2 x = make_uint2(0u, 0u);
    if (ok) x = *reinterpret_cast<const uint2*>(src);
    *reinterpret_cast<float4*>(dst) =
        make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                    __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
}
RKV_DEV void fetched() {
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

template <int D>
struct Smem {
    static constexpr int LD = D + 4, LP = kUnit + 4;
    float q[kTile][LD], k[kUnit][LD], v[kUnit][D];  // (probabilities [kTile][LP] lie over k)
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) prefix_kernel(const __grid_constant__ Params p) {
    using M = Smem<D>;
    static_assert(M::LP <= M::LD, "the probabilities fit over the keys");
    extern __shared__ __align__(16) uint8_t raw[];
    M& sm = *reinterpret_cast<M*>(raw);
    float (*prob)[M::LP] = reinterpret_cast<float (*)[M::LP]>(&sm.k[0][0]);
    __shared__ int64_t at_row[kUnit];  // pool row of each row of the unit (-1: none)
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const uint32_t run = blockIdx.x;
    constexpr int NV = D / 64;  // float4 of the output a thread holds a query
    const float sign = p.flip ? -1.f : 1.f;
    wait_for_last();

    Place place = find_place<kUnit>(p, run);
    Piece c{};
    while (next_piece<kUnit>(p, run, 0, place, c)) {
        if (tid == 0 && bad_length(p, c)) set_error(p.status, kDevErrIndex, (unsigned)c.i);
        __syncthreads();  // the piece before has been read
        // Only where rows follow: the copies are waited for with the first unit's, and copies of
        // a piece without rows (an empty prefix) could land behind those of the next one.
        for (int e = c.c0 < c.c1 ? tid : kTile * (D / 4); e < kTile * (D / 4); e += kThreads) {
            const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
            const bool ok = r < c.rows;
            int s = 0, tk = 0, hd = 0;
            if (ok) place_of_row(p, c.seq0, c.h, c.row0 + r, s, tk, hd);
            fetch4(&sm.q[r][d], static_cast<const T*>(p.q) + s * p.q_seq + tk * p.q_tok + hd * p.q_head + d, ok);
        }
        float m[8], l[8], o[8][NV * 4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[i] = kNone;
            l[i] = 0.f;
#pragma unroll
            for (int j = 0; j < NV * 4; ++j) o[i][j] = 0.f;
        }
        for (int r0 = c.c0; r0 < c.c1; r0 += kUnit) {
            __syncthreads();  // k and v have been read
            if (tid < kUnit) {
                const int r = r0 + tid;
                int64_t x = -1;
                if (r < c.c1) {
                    const int b = p.table[(int64_t)c.i * p.max_blocks + (r >> p.log2bs)];
                    if ((unsigned)b < (unsigned)p.num_blocks)
                        x = (((int64_t)b * p.H + c.h) << p.log2bs) | (r & ((1 << p.log2bs) - 1));
                    else
                        set_error(p.status, kDevErrIndex, (unsigned)r);
                }
                at_row[tid] = x;
            }
            __syncthreads();
#pragma unroll 4
            for (int e = tid; e < kUnit * (D / 4); e += kThreads) {
                const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
                const int64_t x = at_row[r];
                const int64_t at = (x < 0 ? 0 : x) * D + d;
                fetch4(&sm.k[r][d], static_cast<const T*>(p.k) + at, x >= 0);
                fetch4(&sm.v[r][d], static_cast<const T*>(p.v) + at, x >= 0);
            }
            fetched();
            __syncthreads();
            float x[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
#pragma unroll 2
            for (int d = 0; d < D; d += 4) {
                float4 b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * j][d]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 a = *reinterpret_cast<const float4*>(&sm.q[ty * 8 + i][d]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[i][j] = fmaf(a.x, b[j].x, fmaf(a.y, b[j].y, fmaf(a.z, b[j].z, fmaf(a.w, b[j].w, x[i][j]))));
                }
            }
            bool there[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) there[j] = at_row[tx + 16 * j] >= 0;
            __syncthreads();  // the keys have been read: probabilities take their place
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] = there[j] ? x[i][j] * sign : -INFINITY;
                    top = fmaxf(top, x[i][j]);
                }
#pragma unroll
                for (int sh = 1; sh <= 8; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
                if (top > m[i] + p.slack) {
                    const float f = m[i] == kNone ? 0.f : ex2((m[i] - top) * p.scale);
                    m[i] = top;
                    l[i] *= f;
#pragma unroll
                    for (int j = 0; j < NV * 4; ++j) o[i][j] *= f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float y = ex2((x[i][j] - m[i]) * p.scale);
                    l[i] += y;
                    prob[ty * 8 + i][tx + 16 * j] = y;
                }
            }
            __syncwarp();  // a warp reads its own queries' probabilities
#pragma unroll 2
            for (int k = 0; k < kUnit; k += 4) {
                float4 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const float4*>(&prob[ty * 8 + i][k]);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        const float4 y = *reinterpret_cast<const float4*>(&sm.v[k + kk][n * 64 + tx * 4]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float f = kk == 0 ? w[i].x : (kk == 1 ? w[i].y : (kk == 2 ? w[i].z : w[i].w));
                            o[i][4 * n] = fmaf(f, y.x, o[i][4 * n]);
                            o[i][4 * n + 1] = fmaf(f, y.y, o[i][4 * n + 1]);
                            o[i][4 * n + 2] = fmaf(f, y.z, o[i][4 * n + 2]);
                            o[i][4 * n + 3] = fmaf(f, y.w, o[i][4 * n + 3]);
                        }
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int sh = 1; sh <= 8; sh <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], sh);
            float fix;
            const float base = base_of(m[i], p.scale, fix);
            const int r = ty * 8 + i;
            if (r >= c.rows) continue;
            if (c.whole) {
                int s, tk, hd;
                place_of_row(p, c.seq0, c.h, c.row0 + r, s, tk, hd);
                const int64_t at = ((int64_t)s * p.T + tk) * p.H * p.G + hd;
                const Joined j = join_own(base, l[i] * fix, p.own_ml[at]);
                T* out = static_cast<T*>(p.out) + s * p.o_seq + tk * p.o_tok + hd * p.o_head;
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    const int d = n * 64 + tx * 4;
                    const float4 v = make_float4(o[i][4 * n] * fix, o[i][4 * n + 1] * fix,
                                                 o[i][4 * n + 2] * fix, o[i][4 * n + 3] * fix);
                    store4(out + d, join4(j, v, *reinterpret_cast<const float4*>(p.own + at * D + d)));
                }
                if (tx == 0 && p.lse) p.lse[at] = j.lse;
            } else {
#pragma unroll
                for (int n = 0; n < NV; ++n)
                    p.partial[((int64_t)c.slot * (D / 4) + n * 16 + tx) * kTile + r] =
                        make_float4(o[i][4 * n] * fix, o[i][4 * n + 1] * fix, o[i][4 * n + 2] * fix,
                                    o[i][4 * n + 3] * fix);
                if (tx == 0) p.partial_ml[(int64_t)c.slot * kTile + r] = make_float2(base, l[i] * fix);
            }
        }
    }
    if (tid == 0) {
        p.joins[run] = make_int4(c.seq0, c.h, c.row0, join_of(c.rows, c.parts));
    }
}

// Joins the pieces of the tiles that begin in one run and end in a later one, and the
// own rows' sums.  A block takes 32 queries (lanes) of a tile and 32 dimensions: up to
// kFew pieces by a warp for each four of them, more by all warps together.
constexpr int kJoinWarps = 8, kJoinResident = 3, kFew = 16, kMaxBlocks = 320, kJoinLook = kMaxBlocks / 32;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32, kJoinResident) prefix_join_kernel(const __grid_constant__ Params p) {
    __shared__ float4 sh_v[kJoinWarps][8][32];
    __shared__ float sh_m[kJoinWarps][32], sh_l[kJoinWarps][32];
    __shared__ int4 sh_job[kMaxBlocks];  // p.joins of the blocks that left something, and which they are
    __shared__ short sh_from[kMaxBlocks];
    __shared__ int sh_jobs;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = p.tile / 32, blocks = p.runs * p.team;
    const int r = (blockIdx.y % groups) * 32 + lane, dg = blockIdx.y / groups, d = (dg * 8 + warp) * 4;
    wait_for_last();  // the pieces are written
    if (warp == 0) {
        int4 job[kJoinLook];
#pragma unroll
        for (int k = 0; k < kJoinLook; ++k) {
            const int i = 32 * k + lane;
            job[k] = i < blocks ? p.joins[i] : make_int4(0, 0, 0, 0);
        }
        int n = 0;
#pragma unroll
        for (int k = 0; k < kJoinLook; ++k) {
            const uint32_t set = __ballot_sync(0xffffffffu, job[k].w != 0);
            const int at = n + __popc(set & ((1u << lane) - 1u));
            if (job[k].w != 0) {
                sh_job[at] = job[k];
                sh_from[at] = (short)(32 * k + lane);
            }
            n += __popc(set);
        }
        if (lane == 0) sh_jobs = n;
    }
    __syncthreads();
    for (int which = blockIdx.x; which < sh_jobs; which += gridDim.x) {
        const int4 job = sh_job[which];
        const int from = sh_from[which], rows = rows_of(job.w), parts = parts_of(job.w);
        if (r - lane >= rows) continue;  // (for the whole block)
        int s = 0, tk = 0, hd = 0;
        if (r < rows) place_of_row(p, job.x, job.y, job.z + r, s, tk, hd);
        const int64_t at = ((int64_t)s * p.T + tk) * p.H * p.G + hd;
        const float2 own = p.own_ml[at];
        const float4 mine = *reinterpret_cast<const float4*>(p.own + at * D + d);
        const auto slot_of = [&](int i) {
            return i == 0 ? 2 * (int64_t)from + 1 : 2 * (from + (int64_t)i * p.team);
        };
        const auto write = [&](float m, float l, float4 v) {
            if (r >= rows) return;
            const Joined j = join_own(m, l, own);
            store4(static_cast<T*>(p.out) + s * p.o_seq + tk * p.o_tok + hd * p.o_head + d, join4(j, v, mine));
            if (d == 0 && p.lse) p.lse[at] = j.lse;
        };
        float m = -INFINITY, l = 0.f;
        if (parts <= kFew) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int i = 0; i < parts; ++i) {
                const int64_t slot = slot_of(i);
                const float2 ml = p.partial_ml[slot * p.tile + r];
                const float4 y = p.partial[(slot * (D / 4) + d / 4) * p.tile + r];
                const float mx = fmaxf(m, ml.x);
                const float f = weight(m, l, mx), g = weight(ml.x, ml.y, mx);
                m = mx;
                l = l * f + ml.y * g;
                v = make_float4(v.x * f + y.x * g, v.y * f + y.y * g, v.z * f + y.z * g, v.w * f + y.w * g);
            }
            write(m, l, v);
            continue;
        }
        float4 v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = warp; i < parts; i += kJoinWarps) {
            const int64_t slot = slot_of(i);
            const float2 ml = p.partial_ml[slot * p.tile + r];
            float4 y[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) y[x] = p.partial[(slot * (D / 4) + dg * 8 + x) * p.tile + r];
            const float mx = fmaxf(m, ml.x);
            const float f = weight(m, l, mx), g = weight(ml.x, ml.y, mx);
            m = mx;
            l = l * f + ml.y * g;
#pragma unroll
            for (int x = 0; x < 8; ++x)
                v[x] = make_float4(v[x].x * f + y[x].x * g, v[x].y * f + y[x].y * g,
                                   v[x].z * f + y[x].z * g, v[x].w * f + y[x].w * g);
        }
        __syncthreads();  // the shared sums before these have been read
        sh_m[warp][lane] = m;
        sh_l[warp][lane] = l;
#pragma unroll
        for (int x = 0; x < 8; ++x) sh_v[warp][x][lane] = v[x];
        __syncthreads();
        float mx = sh_m[0][lane], sum = 0.f;
#pragma unroll
        for (int w = 1; w < kJoinWarps; ++w) mx = fmaxf(mx, sh_m[w][lane]);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            const float f = weight(sh_m[w][lane], sh_l[w][lane], mx);
            const float4 x = sh_v[w][warp][lane];
            sum += sh_l[w][lane] * f;
            y.x += x.x * f; y.y += x.y * f; y.z += x.z * f; y.w += x.w * f;
        }
        write(mx, sum, y);
    }
}

Params params(const PrefixArgs& a, const PrefixPlan& pl) {
    Params p{};
    const AttnArgs& w = a.own;
    p.k = w.k;
    p.v = w.v;
    p.table = a.table;
    p.lens = a.lens;
    p.cu = a.cu;
    p.P = a.num_prefixes;
    p.per = a.num_prefixes > 0 ? (int)(w.num_seqs / a.num_prefixes) : 0;
    p.max_blocks = a.max_blocks;
    p.log2bs = w.pg.log2bs;
    p.num_blocks = w.pg.num_blocks;
    p.max_rows = a.max_rows;
    p.S = (int)w.num_seqs; p.H = w.pg.H; p.G = w.G; p.T = w.n_new; p.R = w.G * w.n_new;
    p.q = w.q.data;
    p.out = w.out.data;
    p.q_seq = w.q.seq; p.q_tok = w.q.tok; p.q_head = w.q.head;
    p.o_seq = w.out.seq; p.o_tok = w.out.tok; p.o_head = w.out.head;
    p.lse = w.lse;
    p.own = w.raw;
    p.own_ml = reinterpret_cast<const float2*>(w.raw_ml);
    const int64_t slots = 2 * (int64_t)pl.runs * pl.team;
    p.partial = reinterpret_cast<float4*>(a.partial);
    p.partial_ml = reinterpret_cast<float2*>(a.partial + slots * pl.tile * w.d);
    p.joins = reinterpret_cast<int4*>(a.partial + slots * pl.tile * (w.d + 2));
    p.tile = pl.tile;
    p.runs = pl.runs;
    p.lead = pl.lead;
    p.team = pl.team;
    // (as for the own rows: a scale of almost nothing still orders the logits)
    const float x = w.scale * kLog2e, y = x < 0.f ? -x : x;
    p.scale = y < 1e-30f ? 1e-30f : y;
    p.slack = 8.f / p.scale;
    p.flip = x < 0.f ? 0x80008000u : 0u;
    p.status = w.status;
    return p;
}

template <typename T, int D>
cudaError_t go(const Params& p, cudaStream_t s) {
    constexpr int bytes = sizeof(Smem<D>);
    auto kern = prefix_kernel<T, D>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, bytes, done);
    if (e != cudaSuccess) return e;
    return launch_early(kern, (unsigned)p.runs, kThreads, bytes, s, p);
}
template <typename T, int D>
cudaError_t go_join(const Params& p, int64_t tiles, cudaStream_t s) {
    // a block for every 32 queries and 32 dimensions of a tile, for as many tiles at a time as the
    // SMs hold such blocks (registers for kJoinResident): those of a second wave would each look up
    // again what there is to join (us a call with one and with two waves, two runs each: 64 samples
    // of 8192 rows 64.3, 65.0 and 65.3, 65.9; 8 new tokens 46.4, 46.5 and 47.8, 47.6)
    const int y = p.tile / 32 * (D / 32);
    int64_t x = kJoinResident * tc::sm_count() / y;
    if (x > tiles) x = tiles;
    return launch_early(prefix_join_kernel<T, D>, dim3((unsigned)(x < 1 ? 1 : x), (unsigned)y), kJoinWarps * 32, 0, s, p);
}

}  // namespace
}  // namespace prefix

PrefixPlan prefix_plan(const PrefixArgs& a) {
    using namespace prefix;
    const bool tensor = tc_takes(a);
    PrefixPlan pl;
    const AttnArgs& w = a.own;
    const int64_t R = (int64_t)w.G * w.n_new;
    const int sms = tc::sm_count();
    pl.tensor = tensor;
    if (tensor) {
        // Two groups of 128 queries a block, or, where a prefix has 128 or fewer, two shares of
        // its rows.  On average: how the sequences are shared out is known on the device alone, and
        // those without a prefix count too.  Groups far from the average cost time, not values: 8 of
        // 512 sequences on 16384 rows 181 us (teams of eight blocks, seven without queries) where
        // those 8 by themselves take 35 and the others 69; two prefixes of 16384 with 2 and 126
        // sequences 82, with 64 each 72; one with 113 of 128 sequences beside 15 with one each
        // 189, with 8 each 197 (8 KV heads, G = 4, to 64 own rows).
        const int64_t groups = a.num_prefixes > 0 ? a.num_prefixes : 1, each = w.num_seqs * R / groups;
        pl.tile = each <= 128 ? 128 : 256;
        const int64_t tiles = (each + pl.tile - 1) / pl.tile;
        pl.team = tiles < 1 ? 1 : (tiles > kMaxTeam ? kMaxTeam : (int)tiles);
        pl.unit = 64;
    } else {
        pl.tile = kTile;
        pl.unit = kUnit;
    }
    pl.lead = tensor ? 6 : 1;
    // every group may leave one tile that is not full
    const int64_t sets = (w.num_seqs * R / (pl.tile * pl.team) + a.num_prefixes + 1) * w.pg.H;
    pl.tiles = sets * pl.team;
    const int64_t units = sets * (((int64_t)a.max_rows + pl.unit - 1) / pl.unit);
    int64_t runs = tensor ? sms / pl.team : 2 * sms;
    if (runs > units) runs = units;
    if (runs * pl.team > kMaxBlocks) runs = kMaxBlocks / pl.team;
    if (runs < 1) runs = 1;
    pl.runs = (int)runs;
    pl.raw_floats = (size_t)w.num_seqs * R * w.pg.H * (w.d + 2);
    pl.partial_floats = (size_t)pl.runs * pl.team * block_floats(pl.tile, w.d);
    return pl;
}

// A call with fewer sequences or prefixes may take larger tiles and more blocks (64 sequences:
// tiles of 128 queries with two prefixes, of 256 with one), so this follows no one plan: as
// many blocks as a plan of these sizes could have units, in the largest tile and team that any
// number of prefixes leads to.
size_t prefix_most_floats(const PrefixArgs& a) {
    using namespace prefix;
    const AttnArgs& w = a.own;
    const int64_t rows = w.num_seqs * (int64_t)w.G * w.n_new, sms = tc::sm_count();
    const int64_t per = ((int64_t)a.max_rows + kUnit - 1) / kUnit, groups = (int64_t)a.num_prefixes + 1;
    const auto most = [&](int64_t resident, int64_t tile, int64_t least, int64_t team) {
        const int64_t units = (rows / least + groups * team) * w.pg.H * per;
        const int64_t blocks = resident > team ? resident : team;
        return (size_t)(units < blocks ? units : blocks) * block_floats((int)tile, w.d);
    };
    size_t n = most(2 * sms, kTile, kTile, 1);
    if (w.dtype == RKV_DTYPE_BF16) {
        const int64_t teams = (rows + 255) / 256;
        const size_t m = rows <= 128 ? most(sms, 128, 128, 1)
                                     : most(sms, 256, 128, teams > kMaxTeam ? kMaxTeam : teams);
        if (m > n) n = m;
    }
    return n;
}

cudaError_t launch_prefix(const PrefixArgs& a, const PrefixPlan& pl, cudaStream_t s) {
    const prefix::Params p = prefix::params(a, pl);
    if (pl.tensor) return prefix::launch_tc(p, a.own.d, s);
    const bool wide = a.own.d == 128;
    if (a.own.dtype == RKV_DTYPE_FP32)
        return wide ? prefix::go<float, 128>(p, s) : prefix::go<float, 64>(p, s);
    return wide ? prefix::go<__nv_bfloat16, 128>(p, s) : prefix::go<__nv_bfloat16, 64>(p, s);
}

cudaError_t launch_prefix_join(const PrefixArgs& a, const PrefixPlan& pl, cudaStream_t s) {
    const prefix::Params p = prefix::params(a, pl);
    const bool wide = a.own.d == 128;
    if (a.own.dtype == RKV_DTYPE_FP32)
        return wide ? prefix::go_join<float, 128>(p, pl.tiles, s) : prefix::go_join<float, 64>(p, pl.tiles, s);
    return wide ? prefix::go_join<__nv_bfloat16, 128>(p, pl.tiles, s)
                : prefix::go_join<__nv_bfloat16, 64>(p, pl.tiles, s);
}

}  // namespace rkv
