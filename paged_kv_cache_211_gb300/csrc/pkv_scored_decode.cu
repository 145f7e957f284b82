// pkv_scored_decode.cu -- decode attention whose scores are capped or biased,
// over the visible keys of a window or document.
//
// One query per sequence, at position p = n - 1 (n = context_lens[s]); the
// score and the visible keys lo <= t < n are in pkv_scored.cuh.  For query
// head i on KV head i / g:  out = sum_t 2^(z_t - M) V_t / sum_t 2^(z_t - M).
//
// What bounds it: each visible K and V row is read once (2 D bytes each) for
// 4 g D flop, so HBM does.  The design keeps every SM's copies in flight from
// the first block to the last:
//
//  - A unit is one 16-token block of one sequence for one head group (HPS KV
//    heads: 1 at D = 128, 2 at D = 64 where one head's row is only a 128-byte
//    piece).  The units that hold a visible key, ordered (sequence, group,
//    block), are cut into equal runs, one per warp of the grid (8 warps an
//    SM).  Warps share nothing: no barrier but the prologue's.
//  - Each warp feeds its own ring of shared-memory stages (a block's K and V
//    tiles, 8 KB) by itself: one 4-dimensional tensor copy per tile, issued
//    as soon as the stage's fragments are in registers.
//  - Scores S^T = K Q^T and output O^T += V^T P^T run on mma.sync with the g
//    query heads as the n = 8 side, with a running maximum and sum.
//  - A (sequence, group) that lies within one run is written by its warp.  Of
//    the others each warp leaves (m, l, o) in one of its two workspace slots,
//    o in the order the accumulators have (16 bytes a lane, coalesced), and a
//    second kernel joins them:  M = max m,  out = sum o 2^(m - M) / sum l 2^(m - M).
//    (Joined by the warp that finishes last instead, which no second launch
//    needs: 186 us where this takes 181, 17.7 where this takes 14.5 -- one warp
//    reads a row's parts more slowly than a CTA does.)
//  - Short contexts (at most kRowBlocks blocks): each warp takes whole
//    (sequence, group) rows, so there is nothing to join and no second launch.
//
// Measured: 32 sequences of 2048 to 32768 tokens, 32q/8kv heads of 128, bf16,
// cap 50: 181 us, 6.2 TB/s of K and V (the first kernel alone 6.5 TB/s); a
// 1000-token window over 256 sequences, 32q/4kv heads of 64: 51 us, 4.9 TB/s; 60
// sequences of 32 to 512 tokens, 16q/8kv heads of 128: 14.2 us, of which the
// launch, the lengths and the first copies take 6 and the join 4.  Equal runs end
// up to a tenth apart, by SM; handing their last eighth out as chunks made them
// end together but no sooner (HBM is busy until the first ones end), and its
// extra parts cost 10 us.
#include "pkv_scored.cuh"
#include "pkv_tma.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCtas = 160;     // bounds the workspace: persistent CTAs, one per SM
constexpr int kMaxSeqs = 8192;    // per call (lengths and offsets live in shared memory)
constexpr int kMaxGroup = 8;      // query heads per KV head: the n side of the MMA
constexpr int kMaxStages = 3;     // stages of 8 KB per warp
constexpr int kMinUnits = 4;      // shortest run worth a warp of its own
constexpr int kRowBlocks = 8;     // longest row (blocks) that a warp takes whole

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Where a row (sequence, head group) is joined.
struct RowParts {
    int first, last;   // workers that hold parts of it (equal: nothing to join)
    int first_slot;    // slot of the first worker's part (the others: 2 * worker)
    int pad;
};

struct Workspace {
    size_t rows, ml, o, total;
};

Workspace ws_layout(int num_rows, int head_dim, int hps) {
    const size_t workers = (size_t)kMaxCtas * kWarps;
    Workspace w;
    w.rows = 0;
    w.ml = align256((size_t)num_rows * sizeof(RowParts));
    w.o = w.ml + align256(2 * workers * hps * kMaxGroup * sizeof(float2));
    w.total = w.o + 2 * workers * hps * (head_dim / 16) * 32 * sizeof(float4);
    return w;
}

struct ScoredParams {
    const void* q;
    void* out;
    const int32_t* block_tables;
    const int32_t* context_lens;
    RowParts* rows;  // [num_seqs][head group]
    float2* ml;     // [slot][HPS][8]: m (base 2) and l of a query head
    float4* o;      // [slot][HPS][D / 16][lane]: accumulator fragments
    unsigned int* status;
    ScoreMods mods;
    int num_seqs, num_q_heads, num_kv_heads, group, max_blocks_per_seq, num_blocks, len_bound;
    int nstages;
    int rows_whole;  // each warp takes whole rows
};

// The visible span of a sequence: its keys [lo, n), in blocks [b0, b1).
struct Span {
    int n, lo, b0, b1;
};

__device__ __forceinline__ Span span_of(const ScoredParams& p, int s, bool report) {
    Span r;
    r.n = p.context_lens[s];
    if (r.n < 0 || r.n > p.len_bound) {
        if (report) atomicOr(p.status, PKV_DEV_BAD_LENGTH);
        r.n = 0;  // written as zeros
    }
    r.lo = min(first_key(p.mods, s, r.n - 1), r.n);
    r.b0 = r.lo / PKV_BLOCK_SIZE;
    r.b1 = r.lo < r.n ? (r.n + PKV_BLOCK_SIZE - 1) / PKV_BLOCK_SIZE : r.b0;
    return r;
}

// a * b / c and a / b, in 32 bits where they fit (a 64-bit division takes some
// hundred instructions; the walks do a dozen before the first copy).
__device__ __forceinline__ long long mul_div(long long a, int b, int c) {
    const unsigned long long x = (unsigned long long)a * (unsigned)b;
    return (x >> 32) == 0 ? (long long)((unsigned)x / (unsigned)c)
                          : (long long)(x / (unsigned)c);
}
__device__ __forceinline__ int div_int(long long a, long long b) {
    return (((unsigned long long)a | (unsigned long long)b) >> 32) == 0
               ? (int)((unsigned)a / (unsigned)b)
               : (int)(a / b);
}

// K and V pools as (element, row, 64-element half, head): one box is a stage's
// tile, [head][half][16 rows][128 bytes] in shared memory.
__device__ __forceinline__ void load_tile(void* dst, const CUtensorMap* map, uint64_t* bar, int row,
                                          int head) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %3, %5}], [%2];\n" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(row), "r"(head)
        : "memory");
}

bool make_tile_map(CUtensorMap* map, const void* pool, int num_blocks, int num_kv_heads,
                   int head_dim, int hps, pkv_dtype dtype) {
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[4] = {64, (cuuint64_t)num_blocks * PKV_BLOCK_SIZE,
                                (cuuint64_t)(head_dim / 64), (cuuint64_t)num_kv_heads};
    const cuuint64_t strides[3] = {(cuuint64_t)num_kv_heads * head_dim * 2, 128,
                                   (cuuint64_t)head_dim * 2};
    const cuuint32_t box[4] = {64, PKV_BLOCK_SIZE, (cuuint32_t)(head_dim / 64), (cuuint32_t)hps};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUtensorMapDataType dt =
        dtype == PKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return enc(map, dt, 4, const_cast<void*>(pool), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Normalises one accumulator fragment (rows d0 + gid and d0 + 8 + gid, heads
// 2 tig and 2 tig + 1) and stores it as 16-bit values: an 8x8 transpose puts
// two neighbouring elements of one head into a lane.
template <typename T>
__device__ __forceinline__ void store_fragment(T* head0, int D, int d0, int g, float o0, float o1,
                                               float o2, float o3, float inv0, float inv1) {
    using E = Elem<T>;
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const uint32_t a = movmatrix_trans(E::pack(o0 * inv0, o1 * inv1));
    const uint32_t b = movmatrix_trans(E::pack(o2 * inv0, o3 * inv1));
    if (gid < g) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(head0 + (size_t)gid * D + d0 + 2 * tig);
        dst[0] = a;
        dst[4] = b;
    }
}

template <typename T, int D, int HPS, bool kCap, bool kBias>
__global__ void __launch_bounds__(kThreads, 1)
    scored_decode_kernel(const ScoredParams p, const __grid_constant__ CUtensorMap tmap_k,
                         const __grid_constant__ CUtensorMap tmap_v) {
    using E = Elem<T>;
    constexpr int KS = D / 16;
    constexpr int TILE = 16 * D * 2;          // one head's 16 rows
    constexpr int STAGE = 2 * HPS * TILE;     // K tiles, then V tiles
    extern __shared__ unsigned char smem_raw[];
    __shared__ int red[kWarps];
    __shared__ int abort_word;
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char* ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int NS = p.nstages, B = p.num_seqs;
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + (size_t)kWarps * NS * STAGE);
    int* sm_off = reinterpret_cast<int*>(full + kWarps * kMaxStages);  // [B + 1] blocks before s
    int* sm_n = sm_off + B + 1;                                        // [B]
    int* sm_lo = sm_n + B;                                             // [B]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    volatile int* abort_flag = &abort_word;

    if (lane == 0)
        for (int k = 0; k < NS; ++k) mbar_init(&full[warp * NS + k], 1);
    if (tid == 0) {
        abort_word = 0;
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_v)) : "memory");
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    // a programmatic dependent: nothing of the caller's is touched before the
    // kernel in front of this one is complete
    asm volatile("griddepcontrol.wait;\n" ::: "memory");

    const int Hq = p.num_q_heads, g = p.group, HG = p.num_kv_heads / HPS;
    const int worker = warp * (int)gridDim.x + (int)blockIdx.x;
    int workers = kWarps * (int)gridDim.x;
    const bool rows_whole = p.rows_whole != 0;
    long long U = 0;
    if (!rows_whole) {
        // blocks of every sequence, and their exclusive prefix sum
        const int chunk = (B + kThreads - 1) / kThreads;
        const int s0 = min(B, tid * chunk), s1 = min(B, s0 + chunk);
        int mine = 0;
        for (int s = s0; s < s1; ++s) {
            const Span r = span_of(p, s, blockIdx.x == 0);
            sm_n[s] = r.n;
            sm_lo[s] = r.lo;
            mine += r.b1 - r.b0;
        }
        int incl = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) red[warp] = incl;
        __syncthreads();
        int run = incl - mine, total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) run += red[w];
            total += red[w];
        }
        for (int s = s0; s < s1; ++s) {
            sm_off[s] = run;
            run += sm_lo[s] < sm_n[s] ? (sm_n[s] + PKV_BLOCK_SIZE - 1) / PKV_BLOCK_SIZE -
                                            sm_lo[s] / PKV_BLOCK_SIZE
                                      : 0;
        }
        if (tid == 0) sm_off[B] = total;
        U = (long long)HG * total;
        const long long want = (U + kMinUnits - 1) / kMinUnits;
        workers = (int)(want < workers ? want : workers);
    }
    __syncthreads();
    // the joining kernel may be scheduled as this grid's CTAs leave
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

    // ---- this warp's run of units, as segments: blocks [b, e) of row (s, hg)
    struct Seg {
        int s, hg, n, lo, b, e;
        int slot;  // -1: the whole row, written to out; else 2 * worker or 2 * worker + 1
    };
    struct Cursor {
        long long u;  // next unit (rows_whole: next row)
        int s;
    };
    const bool idle = !rows_whole && worker >= workers;
    const long long u_end = rows_whole ? (long long)B * HG : idle ? 0 : mul_div(U, worker + 1, workers);
    const long long u_begin = rows_whole ? worker : idle ? 0 : mul_div(U, worker, workers);
    auto begin = [&]() {
        Cursor c = {u_begin, 0};
        if (!rows_whole && u_begin < u_end) {  // the sequence that holds unit u_begin
            int a = 0, b = B - 1;
            while (a < b) {
                const int mid = (a + b + 1) >> 1;
                if ((long long)HG * sm_off[mid] <= u_begin) a = mid; else b = mid - 1;
            }
            c.s = a;
        }
        return c;
    };
    auto next = [&](Cursor& c, Seg& g_) -> bool {
        if (c.u >= u_end) return false;
        if (rows_whole) {
            g_.s = (int)(c.u / HG);
            g_.hg = (int)(c.u - (long long)g_.s * HG);
            const Span r = span_of(p, g_.s, g_.hg == 0 && lane == 0);
            g_.n = r.n;
            g_.lo = r.lo;
            g_.b = r.b0;
            g_.e = r.b1;
            g_.slot = -1;
            c.u += workers;
            return true;
        }
        const int s = c.s, nb = sm_off[s + 1] - sm_off[s];
        const long long r = c.u - (long long)HG * sm_off[s];
        const int hg = div_int(r, nb), k = (int)(r - (long long)hg * nb);
        const long long left = u_end - c.u;
        const int len = nb - k < left ? nb - k : (int)left;
        g_.s = s;
        g_.hg = hg;
        g_.n = sm_n[s];
        g_.lo = sm_lo[s];
        g_.b = g_.lo / PKV_BLOCK_SIZE + k;
        g_.e = g_.b + len;
        g_.slot = len == nb ? -1 : 2 * worker + (c.u == u_begin ? 0 : 1);
        c.u += len;
        if (k + len == nb && hg == HG - 1) {  // on to the next sequence with blocks
            int t = s + 1;
            while (t < B && sm_off[t + 1] == sm_off[t]) ++t;
            c.s = t;
        }
        return true;
    };

    if (!rows_whole) {
        // sequences that see nothing: zeros
        for (int s = blockIdx.x; s < B; s += gridDim.x) {
            if (sm_lo[s] < sm_n[s]) continue;
            uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (size_t)s * Hq * D);
            for (int x = tid; x < Hq * D / 8; x += kThreads) o[x] = make_uint4(0u, 0u, 0u, 0u);
            for (int x = tid; x < HG; x += kThreads) p.rows[(size_t)s * HG + x] = RowParts{};
        }
    }

    // ---- the fetch walk: a warp's own ring, lane 0 issues
    Cursor fc = begin();
    Seg fg;
    bool fetching = next(fc, fg);
    int fb = fetching ? fg.b : 0;
    int ids = 0, idx = 0;  // table entries of blocks fb - idx + lane (bad: -1)
    auto load_ids = [&]() {
        ids = -1;
        idx = 0;
        const int b = fb + lane;
        if (fetching && b < fg.e) {
            ids = p.block_tables[(size_t)fg.s * p.max_blocks_per_seq + b];
            if (ids < 0 || ids >= p.num_blocks) {
                atomicOr(p.status, PKV_DEV_BAD_BLOCK_ID);
                ids = -1;  // never read: block 0 is fetched and masked out
            }
        }
    };
    auto skip_empty = [&]() {
        while (fetching && fb >= fg.e) {
            fetching = next(fc, fg);
            if (fetching) fb = fg.b;
        }
    };
    skip_empty();
    load_ids();
    uint32_t bad_stages = 0;  // bit k: stage k holds a block with a bad id (same in all lanes)
    int fslot = 0, issued = 0;
    auto fetch = [&]() {
        if (!fetching) return;
        const int id = __shfl_sync(0xffffffffu, ids, idx);
        bad_stages = (bad_stages & ~(1u << fslot)) | (id < 0 ? 1u << fslot : 0u);
        if (lane == 0) {
            uint64_t* bar = &full[warp * NS + fslot];
            unsigned char* st = ring + (size_t)(warp * NS + fslot) * STAGE;
            const int row = max(id, 0) * PKV_BLOCK_SIZE;
            mbar_arrive_expect_tx(bar, STAGE);
            load_tile(st, &tmap_k, bar, row, fg.hg * HPS);
            load_tile(st + HPS * TILE, &tmap_v, bar, row, fg.hg * HPS);
        }
        ++issued;
        if (++fslot == NS) fslot = 0;
        ++fb;
        if (fb >= fg.e) {
            skip_empty();
            load_ids();
        } else if (++idx == 32) {
            load_ids();
        }
    };
    for (int k = 0; k < NS; ++k) fetch();

    // ---- the consuming walk
    const ScoreMods& md = p.mods;
    Cursor cc = begin();
    Seg sg;
    int cslot = 0, used = 0;
    uint32_t phase = 0;
    bool live = true;
    while (live && next(cc, sg)) {
        const int s = sg.s, n = sg.n, h0 = sg.hg * HPS;
        if (!rows_whole && lane == 0 && sg.b == sg.lo / PKV_BLOCK_SIZE) {
            // the row starts here: who shares it
            RowParts r = {worker, worker, sg.slot, 0};
            if (sg.slot >= 0) {
                // the worker that holds the row's last unit u: the largest c with
                // U c / workers <= u
                const int nb = sm_off[s + 1] - sm_off[s];
                const long long u = (long long)HG * sm_off[s] + (long long)(sg.hg + 1) * nb - 1;
                r.last = div_int((u + 1) * workers - 1, U);
            }
            p.rows[(size_t)s * HG + sg.hg] = r;
        }
        uint32_t qf[HPS][KS][2];
        float slope[HPS][2];
#pragma unroll
        for (int e = 0; e < HPS; ++e) {
            const T* qrow = static_cast<const T*>(p.q) +
                            ((size_t)s * Hq + (size_t)(h0 + e) * g + (gid < g ? gid : 0)) * D;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                qf[e][i][0] =
                    gid < g ? *reinterpret_cast<const uint32_t*>(qrow + 16 * i + 2 * tig) : 0u;
                qf[e][i][1] =
                    gid < g ? *reinterpret_cast<const uint32_t*>(qrow + 16 * i + 8 + 2 * tig) : 0u;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
                slope[e][u] = kBias && 2 * tig + u < g
                                  ? md.slopes[(h0 + e) * g + 2 * tig + u] * kScoreLog2e
                                  : 0.f;
        }
        float m[HPS][2], l[HPS][2], o[HPS][KS][4];
#pragma unroll
        for (int e = 0; e < HPS; ++e) {
            m[e][0] = m[e][1] = -INFINITY;
            l[e][0] = l[e][1] = 0.f;
#pragma unroll
            for (int i = 0; i < KS; ++i) o[e][i][0] = o[e][i][1] = o[e][i][2] = o[e][i][3] = 0.f;
        }
        for (int b = sg.b; b < sg.e; ++b) {
            live = __all_sync(0xffffffffu,
                              mbar_wait(&full[warp * NS + cslot], phase, abort_flag, p.status));
            if (!live) break;
            const uint32_t kt = smem_addr(ring + (size_t)(warp * NS + cslot) * STAGE);
            const bool bad = (bad_stages >> cslot) & 1u;
            uint32_t kf[HPS][KS][4], vf[HPS][KS][4];
            const int mi = lane >> 3;
#pragma unroll
            for (int e = 0; e < HPS; ++e) {
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    ldsm_x4(kf[e][i], kt + e * TILE + swz(lane & 15, 2 * i + (lane >> 4)));
                    ldsm_x4_trans(vf[e][i], kt + (HPS + e) * TILE +
                                                swz((lane & 7) + 8 * (mi >> 1), 2 * i + (mi & 1)));
                }
            }
            ++used;
            if (++cslot == NS) {
                cslot = 0;
                phase ^= 1u;
            }
            // the stage's reads are done: refill it with the block NS ahead
            asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
            __syncwarp();
            fetch();
            if (bad) continue;

            // tokens [t_lo, t_hi) of the block are visible
            const int t0 = b * PKV_BLOCK_SIZE;
            const int t_lo = sg.lo - t0, t_hi = n - t0;
            const bool part = t_lo > 0 || t_hi < PKV_BLOCK_SIZE;
#pragma unroll
            for (int e = 0; e < HPS; ++e) {
                float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < KS; i += 2) {
                    E::mma(sa, kf[e][i][0], kf[e][i][1], kf[e][i][2], kf[e][i][3], qf[e][i][0],
                           qf[e][i][1]);
                    E::mma(sb, kf[e][i + 1][0], kf[e][i + 1][1], kf[e][i + 1][2], kf[e][i + 1][3],
                           qf[e][i + 1][0], qf[e][i + 1][1]);
                }
                // z[0], z[1]: token gid, heads 2 tig, 2 tig + 1; z[2], z[3]: token gid + 8
                float z[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float r = sa[x] + sb[x];
                    z[x] = kCap ? cap_score(r, md) : r * md.scale_log2;
                    if (kBias)
                        z[x] = fmaf(slope[e][x & 1],
                                    (float)(t0 + gid + 8 * (x >> 1) - (n - 1)), z[x]);
                }
                if (part) {  // select, never weight: hidden rows may hold anything
                    if (gid < t_lo || gid >= t_hi) z[0] = z[1] = -INFINITY;
                    if (gid + 8 < t_lo || gid + 8 >= t_hi) z[2] = z[3] = -INFINITY;
                    auto keep = [&](int t) { return t >= t_lo && t < t_hi; };
                    const uint32_t lo = (keep(2 * tig) ? 0x0000ffffu : 0u) |
                                        (keep(2 * tig + 1) ? 0xffff0000u : 0u);
                    const uint32_t hi = (keep(2 * tig + 8) ? 0x0000ffffu : 0u) |
                                        (keep(2 * tig + 9) ? 0xffff0000u : 0u);
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        vf[e][i][0] &= lo;
                        vf[e][i][1] &= lo;
                        vf[e][i][2] &= hi;
                        vf[e][i][3] &= hi;
                    }
                }
                float mx[2] = {fmaxf(z[0], z[2]), fmaxf(z[1], z[3])};
                float ms[2], c[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1)
                        mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], off));
                    const float mn = fmaxf(m[e][u], mx[u]);
                    ms[u] = mn == -INFINITY ? 0.f : mn;  // nothing visible so far
                    c[u] = fast_exp2(m[e][u] - ms[u]);
                    m[e][u] = mn;
                }
                const float p0 = fast_exp2(z[0] - ms[0]), p1 = fast_exp2(z[1] - ms[1]);
                const float p2 = fast_exp2(z[2] - ms[0]), p3 = fast_exp2(z[3] - ms[1]);
                l[e][0] = l[e][0] * c[0] + p0 + p2;
                l[e][1] = l[e][1] * c[1] + p1 + p3;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    o[e][i][0] *= c[0];
                    o[e][i][1] *= c[1];
                    o[e][i][2] *= c[0];
                    o[e][i][3] *= c[1];
                }
                // the weights as 16-bit operands (relative error half a step of
                // the type, as the inputs have): P^T from the score layout
                const uint32_t pt = movmatrix_trans(E::pack(p0, p1));
                const uint32_t pb = movmatrix_trans(E::pack(p2, p3));
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    E::mma(o[e][i], vf[e][i][0], vf[e][i][1], vf[e][i][2], vf[e][i][3], pt, pb);
            }
        }
        if (!live) break;
#pragma unroll
        for (int e = 0; e < HPS; ++e) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l[e][u] += __shfl_xor_sync(0xffffffffu, l[e][u], off);
            if (sg.slot < 0) {
                const float inv0 = l[e][0] != 0.f ? 1.f / l[e][0] : 0.f;
                const float inv1 = l[e][1] != 0.f ? 1.f / l[e][1] : 0.f;
                T* head0 = static_cast<T*>(p.out) + ((size_t)s * Hq + (size_t)(h0 + e) * g) * D;
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    store_fragment(head0, D, 16 * i, g, o[e][i][0], o[e][i][1], o[e][i][2],
                                   o[e][i][3], inv0, inv1);
            } else if (2 * tig < g) {  // lanes that hold a query head
                float4* dst = p.o + ((size_t)sg.slot * HPS + e) * KS * 32 + lane;
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    dst[i * 32] = make_float4(o[e][i][0], o[e][i][1], o[e][i][2], o[e][i][3]);
                if (gid == 0) {
                    float2* ml = p.ml + ((size_t)sg.slot * HPS + e) * kMaxGroup + 2 * tig;
                    ml[0] = make_float2(m[e][0], l[e][0]);
                    ml[1] = make_float2(m[e][1], l[e][1]);
                }
            }
        }
    }
    // a wait gave up: let the copies in flight land before the CTA may leave
    if (!live && lane == 0) {
        int slot = cslot;
        uint32_t ph = phase;
        for (int k = used; k < issued; ++k) {
            mbar_drain(&full[warp * NS + slot], ph, p.status);
            if (++slot == NS) {
                slot = 0;
                ph ^= 1u;
            }
        }
    }
}

// Joins the parts of the rows that several workers share, a row per CTA and
// round.  Warp (u, e, i) has fragment i of head e from every kTeams-th part,
// kBatch of them in flight at a time, with a running maximum; the kTeams teams
// meet in shared memory.  Few rows have many parts each and take four teams:
// with one team, and the maxima in a pass of their own, two rows of 47 parts took
// 19.4 us in all and one of 346 took 28.5 where these take 11.6 and 13.3.  Many
// rows have a few parts each: with four teams 496 rows take 19.9 us, with one 14.2.
constexpr int kBatch = 4;
constexpr int kJoinCtas = 4 * kMaxCtas;
constexpr int kManyTeams = 4, kManyTeamRows = 256;

template <typename T, int D, int HPS, int kTeams>
__global__ void __launch_bounds__(kTeams * HPS * (D / 16) * 32)
    scored_join_kernel(const RowParts* __restrict__ rows, const float2* __restrict__ ml,
                       const float4* __restrict__ o, void* out, int num_rows, int num_q_heads,
                       int g) {
    constexpr int KS = D / 16, F = HPS * KS;
    __shared__ float4 sm_ml[kTeams > 1 ? kTeams * F * 32 : 1];   // m, l of the lane's two heads
    __shared__ float4 sm_acc[kTeams > 1 ? kTeams * F * 32 : 1];
    // the next kernel's CTAs may be scheduled beside these; it waits for this
    // grid before it touches anything (griddepcontrol.wait)
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int lane = threadIdx.x & 31, tig = lane & 3;
    const int warp = threadIdx.x >> 5, team = warp / F, f = warp - team * F;
    const int e = f / KS, i = f - e * KS;
    const bool has = 2 * tig < g;
    const int HG = num_q_heads / g / HPS;
    // 32 rows' descriptions at a time
    for (long long r0 = blockIdx.x; r0 < num_rows; r0 += 32ll * gridDim.x) {
        const long long r = r0 + (long long)lane * gridDim.x;
        RowParts mine = {};
        if (r < num_rows) mine = rows[r];
        // (a call whose waits gave up may leave anything here: nothing out of range
        // is taken for a part)
        const bool need = mine.first < mine.last && mine.first >= 0 &&
                          mine.last < kMaxCtas * kWarps && mine.first_slot >> 1 == mine.first;
        unsigned todo = __ballot_sync(0xffffffffu, need);
        while (todo) {  // the same in every warp
            const int k0 = __ffs(todo) - 1;
            todo &= todo - 1;
            const int row = (int)(r0 + (long long)k0 * gridDim.x);
            const int first = __shfl_sync(0xffffffffu, mine.first, k0);
            const int last = __shfl_sync(0xffffffffu, mine.last, k0);
            const int first_slot = __shfl_sync(0xffffffffu, mine.first_slot, k0);
            auto slot_of = [&](int c) { return (size_t)(c == first ? first_slot : 2 * c); };
            float4 run = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);  // m, l of two heads
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float a0 = 0.f, a1 = 0.f;  // what exponents are taken against: m, 0 where -inf
            // joins (m, l, o) v, x into the running ones
            auto add = [&](const float4& v, const float4& x) {
                const float w0 = fast_exp2(v.x - a0), w1 = fast_exp2(v.z - a1);
                run.y = fmaf(w0, v.y, run.y);
                run.w = fmaf(w1, v.w, run.w);
                acc.x = fmaf(w0, x.x, acc.x);
                acc.y = fmaf(w1, x.y, acc.y);
                acc.z = fmaf(w0, x.z, acc.z);
                acc.w = fmaf(w1, x.w, acc.w);
            };
            // raises the running maxima to m0, m1 at least
            auto raise = [&](float m0, float m1) {
                m0 = fmaxf(run.x, m0);
                m1 = fmaxf(run.z, m1);
                a0 = m0 == -INFINITY ? 0.f : m0;
                a1 = m1 == -INFINITY ? 0.f : m1;
                const float w0 = fast_exp2(run.x - a0), w1 = fast_exp2(run.z - a1);
                run = make_float4(m0, run.y * w0, m1, run.w * w1);
                acc = make_float4(acc.x * w0, acc.y * w1, acc.z * w0, acc.w * w1);
            };
            for (int c = first + team; has && c <= last; c += kTeams * kBatch) {
                float4 v[kBatch], x[kBatch];
                float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int part = c + k * kTeams;
                    v[k] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
                    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (part <= last) {
                        const size_t at = slot_of(part) * HPS + e;
                        v[k] = *reinterpret_cast<const float4*>(ml + at * kMaxGroup + 2 * tig);
                        x[k] = o[(at * KS + i) * 32 + lane];
                    }
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    m0 = fmaxf(m0, v[k].x);
                    m1 = fmaxf(m1, v[k].z);
                }
                raise(m0, m1);
#pragma unroll
                for (int k = 0; k < kBatch; ++k) add(v[k], x[k]);
            }
            if constexpr (kTeams > 1) {
                __syncthreads();  // (the last row's have been read)
                sm_ml[warp * 32 + lane] = run;
                sm_acc[warp * 32 + lane] = acc;
                __syncthreads();
                if (team > 0) continue;
#pragma unroll
                for (int u = 1; u < kTeams; ++u) {
                    const float4 v = sm_ml[(u * F + f) * 32 + lane];
                    const float4 x = sm_acc[(u * F + f) * 32 + lane];
                    raise(v.x, v.z);
                    add(v, x);
                }
            }
            const float inv0 = run.y != 0.f ? 1.f / run.y : 0.f;
            const float inv1 = run.w != 0.f ? 1.f / run.w : 0.f;
            const int s = row / HG, hg = row - s * HG;
            T* head0 =
                static_cast<T*>(out) + ((size_t)s * num_q_heads + (size_t)(hg * HPS + e) * g) * D;
            store_fragment(head0, D, 16 * i, g, acc.x, acc.y, acc.z, acc.w, inv0, inv1);
        }
    }
}

int heads_per_step(int head_dim, int num_kv_heads) {
    return head_dim == 64 && num_kv_heads % 2 == 0 ? 2 : 1;
}

template <typename T, int D, int HPS, bool kCap, bool kBias>
pkv_status launch_scored(const ScoredParams& prm, const CUtensorMap& tmk, const CUtensorMap& tmv,
                         int ctas, size_t smem, cudaStream_t stream) {
    auto kern = scored_decode_kernel<T, D, HPS, kCap, kBias>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
        return PKV_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, prm, tmk, tmv) != cudaSuccess) return PKV_ERR_CUDA;
    if (prm.rows_whole) return PKV_OK;
    const int rows = prm.num_seqs * (prm.num_kv_heads / HPS);
    cfg.gridDim = dim3((unsigned)std::min(rows, kJoinCtas));
    cfg.dynamicSmemBytes = 0;
    const bool many = rows <= kManyTeamRows;
    cfg.blockDim = dim3((many ? kManyTeams : 1) * HPS * (D / 16) * 32);
    return cuda_status(cudaLaunchKernelEx(
        &cfg, many ? scored_join_kernel<T, D, HPS, kManyTeams> : scored_join_kernel<T, D, HPS, 1>,
        (const RowParts*)prm.rows, (const float2*)prm.ml, (const float4*)prm.o, prm.out, rows,
        prm.num_q_heads, prm.group));
}

template <typename T, int D, int HPS>
pkv_status launch_scored_mods(ScoredParams prm, const void* k_cache, const void* v_cache,
                              char* workspace, pkv_dtype dtype, cudaStream_t stream) {
    CUtensorMap tmk, tmv;
    if (!make_tile_map(&tmk, k_cache, prm.num_blocks, prm.num_kv_heads, D, HPS, dtype) ||
        !make_tile_map(&tmv, v_cache, prm.num_blocks, prm.num_kv_heads, D, HPS, dtype))
        return PKV_ERR_CUDA;
    const int sms = sm_count();
    if (sms <= 0) return PKV_ERR_CUDA;
    const int ctas = std::min(sms, kMaxCtas);
    const Workspace ws = ws_layout(prm.num_seqs * (prm.num_kv_heads / HPS), D, HPS);
    prm.rows = reinterpret_cast<RowParts*>(workspace + ws.rows);
    prm.ml = reinterpret_cast<float2*>(workspace + ws.ml);
    prm.o = reinterpret_cast<float4*>(workspace + ws.o);
    // three stages a warp where the lengths leave room for them (up to ~2900
    // sequences), else two
    constexpr size_t kStage = (size_t)2 * HPS * 16 * D * 2;
    constexpr size_t kSmemMax = 227 * 1024;
    const size_t fixed = 1024 + kWarps * kMaxStages * 8 + 64 +
                         (prm.rows_whole ? 0 : (size_t)(3 * prm.num_seqs + 1) * 4);
    prm.nstages = fixed + kWarps * 3 * kStage + 512 <= kSmemMax ? 3 : 2;
    const size_t smem = fixed + kWarps * prm.nstages * kStage;
    const bool cap = prm.mods.cap_out > 0.f, bias = prm.mods.slopes != nullptr;
    if (cap)
        return bias ? launch_scored<T, D, HPS, true, true>(prm, tmk, tmv, ctas, smem, stream)
                    : launch_scored<T, D, HPS, true, false>(prm, tmk, tmv, ctas, smem, stream);
    return bias ? launch_scored<T, D, HPS, false, true>(prm, tmk, tmv, ctas, smem, stream)
                : launch_scored<T, D, HPS, false, false>(prm, tmk, tmv, ctas, smem, stream);
}

template <typename T>
pkv_status launch_scored_dim(const ScoredParams& prm, const void* k_cache, const void* v_cache,
                             char* ws, int head_dim, pkv_dtype dtype, cudaStream_t stream) {
    if (head_dim == 128)
        return launch_scored_mods<T, 128, 1>(prm, k_cache, v_cache, ws, dtype, stream);
    if (heads_per_step(head_dim, prm.num_kv_heads) == 2)
        return launch_scored_mods<T, 64, 2>(prm, k_cache, v_cache, ws, dtype, stream);
    return launch_scored_mods<T, 64, 1>(prm, k_cache, v_cache, ws, dtype, stream);
}

}  // namespace
}  // namespace pkv

extern "C" {

size_t paged_attention_decode_scored_workspace_bytes(int num_seqs, int num_q_heads,
                                                     int num_kv_heads, int head_dim,
                                                     int max_context_len) {
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_context_len < 0 ||
        num_q_heads % num_kv_heads != 0 || (head_dim != 64 && head_dim != 128))
        return 0;
    const int hps = pkv::heads_per_step(head_dim, num_kv_heads);
    const long long rows = (long long)num_seqs * (num_kv_heads / hps);
    if (rows > 0x7fffffffll) return 0;
    return pkv::ws_layout((int)rows, head_dim, hps).total;
}

pkv_status paged_attention_decode_scored(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* context_lens, int max_context_len, int num_seqs,
    int num_q_heads, int num_kv_heads, int head_dim, int num_blocks, float scale, float softcap,
    const float* alibi_slopes, int window, const int32_t* key_starts, void* out, void* workspace,
    size_t workspace_bytes, pkv_dtype dtype, pkv_stream_t stream) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        max_blocks_per_seq <= 0 || num_blocks <= 0 || max_context_len < 0)
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    pkv::ScoredParams prm = {};
    if (!pkv::make_score_mods(&prm.mods, scale, softcap, alibi_slopes, window, key_starts, nullptr))
        return PKV_ERR_INVALID_ARG;
    const int g = num_q_heads / num_kv_heads;
    if (g > pkv::kMaxGroup || (head_dim != 64 && head_dim != 128) || num_seqs > pkv::kMaxSeqs)
        return PKV_ERR_UNSUPPORTED;
    const long long table_len = (long long)max_blocks_per_seq * PKV_BLOCK_SIZE;
    if (table_len > 0x7fffffffll || num_blocks > 0x7fffffff / PKV_BLOCK_SIZE)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out)
        return PKV_ERR_INVALID_ARG;
    if (!pkv::aligned16(q) || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache) ||
        !pkv::aligned16(out))
        return PKV_ERR_INVALID_ARG;
    if (pkv::overlap(q, out, (size_t)num_seqs * num_q_heads * head_dim * 2))
        return PKV_ERR_INVALID_ARG;
    const size_t need = paged_attention_decode_scored_workspace_bytes(
        num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len);
    if (need == 0) return PKV_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PKV_ERR_WORKSPACE;
    prm.status = pkv::status_word();
    if (!prm.status) return PKV_ERR_CUDA;
    prm.q = q;
    prm.out = out;
    prm.block_tables = block_tables;
    prm.context_lens = context_lens;
    prm.num_seqs = num_seqs;
    prm.num_q_heads = num_q_heads;
    prm.num_kv_heads = num_kv_heads;
    prm.group = g;
    prm.max_blocks_per_seq = max_blocks_per_seq;
    prm.num_blocks = num_blocks;
    prm.len_bound = (int)std::min<long long>(max_context_len, table_len);
    // most keys a query sees, hence most blocks of a row (a window may start
    // anywhere within its first block)
    long long keys = prm.len_bound;
    if (window > 0) keys = std::min<long long>(keys, (long long)window + PKV_BLOCK_SIZE - 1);
    prm.rows_whole = (keys + PKV_BLOCK_SIZE - 1) / PKV_BLOCK_SIZE <= pkv::kRowBlocks;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    return dtype == PKV_BF16 ? pkv::launch_scored_dim<__nv_bfloat16>(prm, k_cache, v_cache, ws,
                                                                    head_dim, dtype, st)
                             : pkv::launch_scored_dim<__half>(prm, k_cache, v_cache, ws, head_dim,
                                                             dtype, st);
}

}  // extern "C"
