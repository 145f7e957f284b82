// pkv_scored_prefill.cu -- chunked-prefill attention with capped or biased
// scores over windows, prefixes and documents (pkv_scored.cuh has the score
// and the visible keys; a row's keys are one interval [lo, hi)).
//
// Each visible (row, key) pair costs 4 D flop in two matrix products, run as
// tcgen05.mma with fp32 accumulators in tensor memory, and one score through
// cap, bias and exp2.  With a cap the scores, not the products, bound it: tanh as
// exp2 and a reciprocal makes three special functions a score, with the
// softmax's own exp2.  So scores within |z / cap| <= 0.5 take tanh from a
// polynomial on the packed fp32 pipe instead (a warp's 64 keys at a time, four
// terms; eight up to 1.25), and only the others the special-function pipe.
//
// Work item: one sequence, one KV head, a pair of 128-row tiles A and B (256
// consecutive (query token, query head) rows) and, where items are few, one of
// `splits` runs of its key tiles.  Key tiles are 128 keys (8 blocks), counted
// from the first block that a row of the item sees.  A persistent CTA per SM:
//   warp 0 / 3   tensor copies of the K / V blocks into two-stage rings,
//   warp 2       tensor memory; the Q tiles,
//   warp 1       S_X = Q_X K^T and O_X += P_X V, ordered ... PV_A(J), S_A(J+1),
//                PV_B(J), S_B(J+1) ..., so the tensor core works on one tile
//                while the other's scores become weights,
//   warps 4-19   the scores: two threads a row, 64 keys each: cap, bias, mask
//                (a select), maximum (exchanged between the two) and sum, P as
//                16-bit values over the scores.  (One thread a row, 128 keys
//                each, left a scheduler two warps of long chains: 499 us below.)
// An item whose rows fill tile A only leaves tile B out.  O is rescaled only
// when a row's maximum grows by more than 2^8; capped bf16 scores need no
// maximum at all.  V rows that no row of the item sees are zeroed before P V.
// Rows of one tile see different keys, so a hidden key's NaN or infinity in V
// would still meet a zero weight: a row whose O is not finite is computed again,
// by a plain loop over its own keys.  Every wait is bounded.
//
// Measured: 8 prompts of 2048 tokens, 32q/8kv heads of 128, bf16, cap 50: 269 us,
// 1022 TFLOP/s of visible pairs.  The tensor pipe is active 46 % of the time, the
// fp32 pipe 35 %, the integer and min / max pipe 30 %, the special functions
// 23 %: no pipe bounds it but the chain S -> weights -> P V -> next S of each
// tile, which tensor memory leaves no room to double (O and S of two tiles fill
// its 512 columns, and P lies over S).  Score products of half the keys each (four
// shorter chains) took 490 us: at N = 64 the product waits for Q's rows from
// shared memory.
#include <type_traits>

#include "pkv_scored.cuh"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kSoftWarps = 16;         // score warps: tile A / B x key half x lane quarter
constexpr int kThreads = (4 + kSoftWarps) * 32;
constexpr int kRows = 128;             // rows of a tile
constexpr int kPair = 2 * kRows;       // rows of an item
constexpr int kKeys = 128;             // keys of a key tile
constexpr int kHalf = kKeys / 2;       // keys of one score thread
constexpr int kTileBlocks = kKeys / PKV_BLOCK_SIZE;
constexpr float kRescale = 8.f;        // log2 of the largest P before O is rescaled
constexpr float kFixedMax = 80.f;      // largest |z| (base 2) that needs no running maximum
constexpr int kMaxCtas = 160;          // bounds the workspace of split items
constexpr int kMaxGroup = 16;
// Registers: launched at kLaunchRegs a thread (checked on the host); the load /
// MMA warpgroup gives some up and the four score warpgroups take them.
constexpr int kLaunchRegs = 96;
constexpr int kOtherRegs = 56;
constexpr int kSoftmaxRegs = 104;
static_assert(128 * kOtherRegs + kSoftWarps * 32 * kSoftmaxRegs <= kThreads * kLaunchRegs,
              "register shares exceed the launch total");

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

struct PrefillScored {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    void* out;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* cu_q_lens;
    unsigned int* status;
    ScoreMods mods;
    int num_seqs, num_q_heads, num_kv_heads, group, max_blocks_per_seq, num_blocks;
    int max_q_len, num_q_rows;
    int pairs_per_seq;     // ceil(max_q_len * group / kPair)
    int splits;            // key runs per item; > 1: partials go to the workspace
    int sorted;            // deal the items that hold rows, by their number of key tiles
    // the polynomials' terms, z = raw sum tanh_z[i] raw^2i, and the largest |raw
    // score| that each serves (negative: none)
    float tanh_z[kTanhTerms], tanh_few[kTanhFew], tanh_wide[kTanhWide];
    float tanh_limit, tanh_few_limit, tanh_wide_limit;
    // partials of split items: row = ((base item) * splits + split) * kPair + row of the pair
    float* ws_m;
    float* ws_l;
    float* ws_o;           // [row][D]
};

struct __align__(16) Item {
    int s, h, q0, qlen, n, row0;
    int split, base;       // base: item without its split
    int lo, hi;            // keys that some row of the item sees
    int b0, nblk;          // this split's first block and its number of blocks
    int nkv;               // its key tiles (0: nothing to compute; -1: no item)
    int has_b;             // tile B holds rows
    int start, prefix;     // the sequence's first key, and its prefix (at most n)
};
static_assert(sizeof(Item) == 64, "four 16-byte words");
// Rounds whose items a CTA works out at its start, one thread each (an item
// takes a dozen divisions and dependent loads: 11 800 cycles went by between an
// item's last key tile and the next one's first when every role did it by itself)
constexpr int kItemCache = 256;

// A sequence's chunk is usable if its rows lie inside q and out, it is no
// longer than the host bound, and it fits its context and the table.
__device__ __forceinline__ bool lengths_ok(const PrefillScored& p, int q0, int qlen, int n) {
    return qlen > 0 && q0 >= 0 && q0 <= p.num_q_rows - qlen && qlen <= p.max_q_len && n >= qlen &&
           n <= p.max_blocks_per_seq * PKV_BLOCK_SIZE;
}

// The visible keys [lo, hi) of the row at position pos.
__device__ __forceinline__ int row_lo(const PrefillScored& p, const Item& it, int pos) {
    return p.mods.window > 0 ? max(it.start, pos - p.mods.window + 1) : it.start;
}
__device__ __forceinline__ int row_hi(const Item& it, int pos) { return max(pos + 1, it.prefix); }

// The item of these coordinates; false (nkv = -1) if it holds no rows or its
// lengths are invalid (flagged once per sequence).
__device__ __forceinline__ bool item_at(const PrefillScored& p, int s, int pair, int h, int split,
                                        bool flag, Item& it) {
    it.split = split;
    it.s = s;
    it.h = h;
    it.base = (s * p.num_kv_heads + h) * p.pairs_per_seq + pair;
    it.q0 = p.cu_q_lens[it.s];
    it.qlen = p.cu_q_lens[it.s + 1] - it.q0;
    it.n = p.context_lens[it.s];
    it.nkv = -1;
    if (!lengths_ok(p, it.q0, it.qlen, it.n)) {
        if (flag && pair == 0 && it.h == 0 && it.split == 0 && it.qlen != 0)
            atomicOr(p.status, PKV_DEV_BAD_LENGTH);
        return false;
    }
    const int g = p.group, rows = it.qlen * g;
    it.row0 = pair * kPair;
    if (it.row0 >= rows) return false;
    it.has_b = it.row0 + kRows < rows;
    const int t_first = it.row0 / g;
    const int t_last = min(it.qlen, (it.row0 + kPair + g - 1) / g) - 1;
    const int base_pos = it.n - it.qlen;
    it.start = p.mods.key_starts ? max(p.mods.key_starts[it.s], 0) : 0;
    it.prefix = p.mods.prefix_lens ? min(p.mods.prefix_lens[it.s], it.n) : 0;
    it.lo = row_lo(p, it, base_pos + t_first);
    it.hi = row_hi(it, base_pos + t_last);
    it.b0 = it.lo / PKV_BLOCK_SIZE;
    it.nblk = it.nkv = 0;
    if (it.lo >= it.hi) return true;
    const int blocks = (it.hi + PKV_BLOCK_SIZE - 1) / PKV_BLOCK_SIZE - it.b0;
    const int tiles = (blocks + kTileBlocks - 1) / kTileBlocks;
    const int j0 = (int)((long long)tiles * it.split / p.splits);
    const int j1 = (int)((long long)tiles * (it.split + 1) / p.splits);
    it.nkv = j1 - j0;
    it.b0 += j0 * kTileBlocks;
    it.nblk = min(blocks - j0 * kTileBlocks, it.nkv * kTileBlocks);
    return true;
}

// Item i of the plain order: pairs from the end of each chunk first, where the
// causal range is longest.
__device__ __forceinline__ bool plain_item(const PrefillScored& p, int i, bool flag, Item& it) {
    const int per_pair = p.num_seqs * p.num_kv_heads * p.splits;
    const int pair = p.pairs_per_seq - 1 - i / per_pair;
    const int rem = i % per_pair, sh = rem / p.splits, s = sh / p.num_kv_heads;
    return item_at(p, s, pair, sh - s * p.num_kv_heads, rem - sh * p.splits, flag, it);
}

// The item this CTA takes in round r: rounds alternate direction over the
// CTAs, so that heaviest-first items even out.
__device__ __forceinline__ int round_item(int r) {
    const int G = gridDim.x, c = blockIdx.x;
    return r * G + ((r & 1) ? G - 1 - c : c);
}

// The item of round r from the CTA's table (past it: worked out again); false: none.
__device__ __forceinline__ bool round_at(const PrefillScored& p, const Item* table, int num_items,
                                         int r, bool flag, Item& it) {
    if (r < kItemCache) {
        it = table[r];
        return it.nkv >= 0;
    }
    const int i = round_item(r);
    return i < num_items && plain_item(p, i, flag, it);
}

// The (sequence, pair) entries that hold rows, those with the most key tiles
// first (a stable counting sort, the same in every CTA), in order[]; returns how
// many.  Ragged chunks leave most entries without rows and the others of very
// different cost: dealt in the plain order, the busiest CTA of 24 chunks of 1 to
// 700 tokens held three items of 184, where two would do.  By the whole CTA,
// with scratch of kSortMax + 2 * kSortKeys words.
constexpr int kSortMax = 1024;   // entries
constexpr int kSortKeys = 256;   // key tiles told apart

__device__ int sort_entries(const PrefillScored& p, int* scratch, uint16_t* order) {
    const int E = p.num_seqs * p.pairs_per_seq;
    int* key = scratch;                  // [E] kSortKeys - 1 - tiles; kSortKeys: no rows
    int* offset = scratch + kSortMax;    // [kSortKeys + 1]
    const int tid = threadIdx.x, lane = tid & 31;
    for (int k = tid; k <= kSortKeys; k += kThreads) offset[k] = 0;
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) {
        const int s = e / p.pairs_per_seq;
        Item it;
        // (whole items: a split's share of the tiles orders them alike)
        const bool any = item_at(p, s, e - s * p.pairs_per_seq, 0, 0, blockIdx.x == 0, it);
        key[e] = any ? kSortKeys - 1 - min(it.nkv, kSortKeys - 1) : kSortKeys;
        if (any) atomicAdd(&offset[key[e]], 1);
    }
    __syncthreads();
    if (tid < 32) {
        // counts to offsets, eight keys a lane
        constexpr int PER = kSortKeys / 32;
        int mine = 0;
        for (int k = 0; k < PER; ++k) mine += offset[lane * PER + k];
        int run = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += u;
        }
        const int total = __shfl_sync(0xffffffffu, run, 31);
        run -= mine;
        for (int k = 0; k < PER; ++k) {
            const int c = offset[lane * PER + k];
            offset[lane * PER + k] = run;
            run += c;
        }
        if (lane == 0) offset[kSortKeys] = total;
        __syncwarp();
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane, k = e < E ? key[e] : kSortKeys;
            const unsigned same = __match_any_sync(0xffffffffu, k);
            const int at = k < kSortKeys ? offset[k] + __popc(same & ((1u << lane) - 1u)) : 0;
            __syncwarp();
            if (k < kSortKeys) {
                order[at] = (uint16_t)e;
                if ((same >> lane) == 1u) offset[k] = at + 1;  // the key's last lane
            }
            __syncwarp();
        }
    }
    __syncthreads();
    return offset[kSortKeys];
}

// Two-wide fp32 arithmetic on packed register pairs, the three-input maximum
// and 32-byte stores.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ void st_global_v8(void* ptr, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(ptr),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                 "r"(w[7])
                 : "memory");
}

// A pair of 16-bit values times a power of two.
template <typename T>
__device__ __forceinline__ uint32_t scale_pair(uint32_t x, float f) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&x), __float2half2_rn(f));
        return *reinterpret_cast<const uint32_t*>(&y);
    } else {
        const __nv_bfloat162 y =
            __hmul2(*reinterpret_cast<__nv_bfloat162*>(&x), __float2bfloat162_rn(f));
        return *reinterpret_cast<const uint32_t*>(&y);
    }
}

// One lane of a converged warp (1 there, 0 elsewhere).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile(
        "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(one));
    return one;
}
// tc_mma, tc_mma_tmem_a and tc_commit by the elected lane of a whole warp.
__device__ __forceinline__ void mma_if(uint32_t leader, uint32_t d_tmem, uint64_t a_desc,
                                       uint64_t b_desc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_tmem_a_if(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem,
                                              uint64_t b_desc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t leader, uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
            smem_addr(bar)),
        "r"(leader)
        : "memory");
}

// One row again, by a whole warp and from its own keys only (keys [lo, hi) of
// its sequence): a key it does not see, or whose block id is bad, is never
// read.  Lane x gets elements x * D / 32 .. of the (normalised) output.
template <typename T, int D>
__device__ void plain_row(const PrefillScored& p, int s, int h, int head, int row, int pos, int lo,
                          int hi, float (&o)[D / 32]) {
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    const T* q = static_cast<const T*>(p.q) + ((size_t)row * p.num_q_heads + head) * D;
    const size_t stride = (size_t)p.num_kv_heads * D;
    const T* kc = static_cast<const T*>(p.k_cache) + (size_t)h * D;
    const T* vc = static_cast<const T*>(p.v_cache) + (size_t)h * D;
    const int32_t* table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    const ScoreMods& md = p.mods;
    const float slope = md.slopes ? md.slopes[head] * kScoreLog2e : 0.f;
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = 0.f;
    for (int t0 = lo; t0 < hi; t0 += 32) {
        const int t = t0 + lane;
        int64_t slot = -1;
        if (t < hi) {
            const int id = table[t / PKV_BLOCK_SIZE];
            if (id >= 0 && id < p.num_blocks)
                slot = (int64_t)id * PKV_BLOCK_SIZE + t % PKV_BLOCK_SIZE;
        }
        float z = -INFINITY;
        if (slot >= 0) {
            float dot = 0.f;
            const T* k = kc + slot * stride;
            for (int d = 0; d < D; ++d) dot = fmaf((float)q[d], (float)k[d], dot);
            z = md.cap_out > 0.f ? cap_score(dot, md) : dot * md.scale_log2;
            z = fmaf(-slope, fabsf((float)(pos - t)), z);
        }
        float mx = z;
        for (int off = 16; off > 0; off >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
        const float f = fast_exp2(m - ms), w = slot >= 0 ? fast_exp2(z - ms) : 0.f;
        m = mn;
        float sum = w;
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = l * f + sum;
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] *= f;
        for (int x = 0; x < 32; ++x) {
            const float wx = __shfl_sync(0xffffffffu, w, x);
            const int64_t sx = __shfl_sync(0xffffffffu, slot, x);
            if (sx < 0) continue;
            const T* v = vc + sx * stride + lane * PER;
#pragma unroll
            for (int e = 0; e < PER; ++e) o[e] = fmaf(wx, (float)v[e], o[e]);
        }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] *= inv;
}

// Replaces column half q of the rows row0 + (bit of `which`) of an item, whose
// O met something not finite; l: the lane's row's sum, which their partials are
// relative to.
template <typename T, int D>
__device__ __noinline__ void redo_rows(const PrefillScored& p, Item it, int row0, int q,
                                       unsigned which, float l, size_t prow0) {
    const int lane = threadIdx.x & 31, g = p.group;
    while (which) {
        const int who = __ffs(which) - 1;
        which &= which - 1;
        const int R = row0 + who, t = R / g, head = it.h * g + R - t * g;
        const int pos = it.n - it.qlen + t;
        const int lo = max(row_lo(p, it, pos), it.b0 * PKV_BLOCK_SIZE);
        const int hi = min(row_hi(it, pos), (it.b0 + it.nblk) * PKV_BLOCK_SIZE);
        float o[D / 32];
        plain_row<T, D>(p, it.s, it.h, head, it.q0 + t, pos, lo, hi, o);
        const float lw = __shfl_sync(0xffffffffu, l, who);
        if (lane / 16 != q) continue;
        const int d = lane * (D / 32);
        if (p.splits > 1) {
            for (int e = 0; e < D / 32; ++e) p.ws_o[(prow0 + who) * D + d + e] = o[e] * lw;
        } else {
            T* dst = static_cast<T*>(p.out) + ((size_t)(it.q0 + t) * p.num_q_heads + head) * D + d;
#pragma unroll
            for (int e = 0; e < D / 32; e += 2)
                *reinterpret_cast<uint32_t*>(dst + e) = Elem<T>::pack(o[e], o[e + 1]);
        }
    }
}

// Raw scores to capped base-2 scores z = cap' tanh(raw cap_in), cap' = cap
// log2(e).  Where the whole warp's scores allow it z is raw times a polynomial
// in raw^2, two scores an instruction; else cap_score.  (The prompts above with a
// cap of 10, whose scores reach it: 351 us with the eight terms, 398 without;
// fp16 385 and 468.)
// top: the largest |raw score|.
__device__ __forceinline__ float largest(const float (&sc)[kHalf]) {
    float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kHalf; c += 2)
        top[(c >> 1) & 3] = max3(top[(c >> 1) & 3], fabsf(sc[c]), fabsf(sc[c + 1]));
    return max3(fmaxf(top[0], top[1]), top[2], top[3]);
}
template <int N>
__device__ __forceinline__ void cap_by_terms(const float* terms, float (&sc)[kHalf]) {
#pragma unroll
    for (int e0 = 0; e0 < kHalf; e0 += 8) {  // four independent chains at a time
        uint64_t x[4], v[4], y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            x[u] = f2(sc[e0 + 2 * u], sc[e0 + 2 * u + 1]);
            v[u] = f2_mul(x[u], x[u]);
            y[u] = f2(terms[N - 1], terms[N - 1]);
        }
#pragma unroll
        for (int i = N - 2; i >= 0; --i)
#pragma unroll
            for (int u = 0; u < 4; ++u) y[u] = f2_fma(y[u], v[u], f2(terms[i], terms[i]));
#pragma unroll
        for (int u = 0; u < 4; ++u)
            f2_split(f2_mul(x[u], y[u]), sc[e0 + 2 * u], sc[e0 + 2 * u + 1]);
    }
}
template <bool kSmallCap>
__device__ __forceinline__ void cap_to_z(const PrefillScored& p, float (&sc)[kHalf], float top) {
    if (__all_sync(0xffffffffu, top <= p.tanh_limit)) {
        cap_by_terms<kTanhTerms>(p.tanh_z, sc);
    } else if (__all_sync(0xffffffffu, top <= p.tanh_wide_limit)) {
        cap_by_terms<kTanhWide>(p.tanh_wide, sc);
    } else {
        // score by score: one large score (a hidden one's leftovers in shared memory
        // even) must not cost its neighbours near zero their relative error.  Under
        // a small cap (kSmallCap: cap' <= kFixedMax) the far form alone is within
        // 2^-16 of every z, and shorter.
#pragma unroll
        for (int c = 0; c < kHalf; ++c)
            sc[c] = kSmallCap ? fmaf(-2.f * p.mods.cap_out,
                                     fast_rcp(1.f + fast_exp2(2.f * kScoreLog2e * p.mods.cap_in *
                                                              sc[c])),
                                     p.mods.cap_out)
                              : cap_score(sc[c], p.mods);
    }
}

template <typename T, int D, bool kCap, bool kBias, bool kFixed>
__global__ void __launch_bounds__(kThreads, 1)
    scored_prefill_kernel(const PrefillScored p, const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_v,
                          const __grid_constant__ CUtensorMap tmap_q, int q_tma, int num_items) {
    using E = Elem<T>;
    constexpr int HALVES = D / 64;
    constexpr int REG = kRows * 128;       // one 64-element half of 128 rows: 16 KB
    constexpr int TILE = HALVES * REG;     // a Q tile, or one K or V key tile
    constexpr uint32_t kCols = 512;
    constexpr uint32_t kOCol = 2 * kKeys;  // O_A at kOCol, O_B at kOCol + D
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char* sq = smem_raw + (((raw + 1023u) & ~1023u) - raw);   // Q_A, Q_B
    unsigned char* sk = sq + 2 * TILE;      // 2 stages
    unsigned char* sv = sk + 2 * TILE;      // 2 stages
    uint64_t* bars = reinterpret_cast<uint64_t*>(sv + 2 * TILE);
    uint64_t* k_full = bars + 0;            // [stage]
    uint64_t* k_empty = bars + 2;
    uint64_t* v_full = bars + 4;
    uint64_t* v_empty = bars + 6;
    uint64_t* q_full = bars + 8;            // [tile]
    uint64_t* q_empty = bars + 10;
    uint64_t* s_full = bars + 12;           // [tile]: S_X written
    uint64_t* p_full = bars + 14;           // [tile][key half]: its 4 warps wrote P
    uint64_t* o_ready = bars + 18;          // [tile]: an item's last P V_X done
    uint64_t* o_free = bars + 20;           // [tile]: its score warps read O_X
    uint64_t* mma_idle = bars + 22;
    uint64_t* x_max = bars + 23;            // [tile][lane quarter]: both halves' maxima written
    uint64_t* x_scale = bars + 31;          // [tile][lane quarter]: both halves rescaled O
    uint64_t* x_sum = bars + 39;            // [tile][lane quarter]: both halves' sums written
    int* vbad = reinterpret_cast<int*>(bars + 47);           // [2] bad-block bits per V stage
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(vbad + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    // what the two key halves of a row tell each other, by parity:
    // [parity][tile][half][row] maxima, and sums
    float* xm = reinterpret_cast<float*>(tmem_slot + 2);
    float* xl = xm + 2 * 2 * 2 * kRows;
    Item* table = reinterpret_cast<Item*>(
        (reinterpret_cast<uintptr_t>(xl + 2 * 2 * 2 * kRows) + 15) & ~(uintptr_t)15);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be one per warp
    const int g = p.group, Hq = p.num_q_heads;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], 4);
            mbar_init(&p_full[2 * i + 1], 4);
            mbar_init(&o_ready[i], 1);
            mbar_init(&o_free[i], 8);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&x_max[i], 2);
            mbar_init(&x_scale[i], 2);
            mbar_init(&x_sum[i], 2);
        }
        mbar_init(mma_idle, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (tid == 32) {
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_v)) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_q)) : "memory");
    }
    // a programmatic dependent where items are split (14.5 us where an ordinary launch
    // takes 15.4; longer calls gain nothing): nothing of the caller's is touched
    // before the kernel in front of this one is complete, and no tensor memory taken,
    // which CTAs of that kernel may still ask for
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (warp == 2) tc_alloc(tmem_slot, kCols);
    // the items (the tiles' memory is still free: the sort's scratch)
    uint16_t* order = reinterpret_cast<uint16_t*>(sk);
    const int per_entry = p.num_kv_heads * p.splits;
    if (p.sorted) num_items = per_entry * sort_entries(p, reinterpret_cast<int*>(sq), order);
    const int rounds = (num_items + (int)gridDim.x - 1) / (int)gridDim.x;
    for (int r = tid; r < min(rounds, kItemCache); r += kThreads) {
        Item it;
        it.nkv = -1;
        const int i = round_item(r);
        if (i < num_items) {
            if (p.sorted) {
                const int e = order[i / per_entry], s = e / p.pairs_per_seq;
                const int rem = i % per_entry, h = rem / p.splits;
                item_at(p, s, e - s * p.pairs_per_seq, h, rem - h * p.splits, false, it);
            } else {
                plain_item(p, i, true, it);
            }
        }
        table[r] = it;
    }
    // (copies will overwrite the scratch)
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the joining kernel may be scheduled as this grid's CTAs leave (they have their
    // tensor memory now)
    if (p.splits > 1) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const uint32_t tmem = *tmem_slot;
    // whole warpgroups: warps 0-3 release registers, 4-19 take them
    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp == 0 || warp == 3) {
        // ------------------------------------------------ K (warp 0) / V (warp 3) producers
        const bool isk = warp == 0;
        const CUtensorMap* map = isk ? &tmap_k : &tmap_v;
        uint64_t* full = isk ? k_full : v_full;
        uint64_t* empty = isk ? k_empty : v_empty;
        unsigned char* ring = isk ? sk : sv;
        int J = 0;  // key tiles issued by this CTA
        bool live = true;
        for (int rd = 0; rd < rounds && live; ++rd) {
            Item it;
            if (!round_at(p, table, num_items, rd, isk && lane == 0, it)) continue;
            const int32_t* blocks =
                p.block_tables + (size_t)it.s * p.max_blocks_per_seq + it.b0;
            for (int j = 0; j < it.nkv; ++j, ++J) {
                const int b = J & 1, ph = (J >> 1) & 1;
                live = __all_sync(0xffffffffu, mbar_wait(&empty[b], ph ^ 1, abort_flag, p.status));
                if (!live) break;
                const int nb = min(kTileBlocks, it.nblk - kTileBlocks * j);
                int id = 0;
                bool bad = false;
                if (lane < nb) {
                    id = blocks[kTileBlocks * j + lane];
                    bad = id < 0 || id >= p.num_blocks;
                    if (bad) id = 0;  // fetched, then masked and zeroed
                }
                const unsigned badm = __ballot_sync(0xffffffffu, bad);
                if (lane == 0) {
                    if (isk && badm) atomicOr(p.status, PKV_DEV_BAD_BLOCK_ID);
                    if (!isk) vbad[b] = (int)badm;
                    mbar_arrive_expect_tx(&full[b], (uint32_t)(nb * HALVES * 2048));
                }
                __syncwarp();
                if (lane < nb) {
#pragma unroll
                    for (int hh = 0; hh < HALVES; ++hh)
                        tma_load_rows(ring + b * TILE + hh * REG + lane * 2048, map, &full[b],
                                      hh * 64, it.h, id * PKV_BLOCK_SIZE);
                }
            }
        }
        // every copy issued must land before the CTA may exit
        if (lane == 0)
            for (int j = max(0, J - 2); j < J; ++j) mbar_drain(&full[j & 1], (j >> 1) & 1, p.status);
    } else if (warp == 2) {
        // ------------------------------------------------------ Q tiles of each item
        // By tensor copies (lane 0) where the group divides the tile's 128
        // rows, else row by row (cp.async).  Rows past the chunk belong to the
        // next one (or read as zeros): they are never stored.
        const T* qb = static_cast<const T*>(p.q);
        constexpr int CH = D / 8;  // 16-byte chunks per row
        int issued[2] = {0, 0};    // items whose tile X was loaded
        bool live = true;
        for (int rd = 0; rd < rounds && live; ++rd) {
            Item it;
            if (!round_at(p, table, num_items, rd, false, it) || it.nkv == 0) continue;
            for (int X = 0; X < (it.has_b ? 2 : 1) && live; ++X) {
                live = __all_sync(0xffffffffu, mbar_wait(&q_empty[X], (issued[X] & 1) ^ 1,
                                                         abort_flag, p.status));
                if (!live) break;
                ++issued[X];
                const int row = it.row0 + X * kRows;
                if (q_tma) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&q_full[X], (uint32_t)TILE);
#pragma unroll
                        for (int hh = 0; hh < HALVES; ++hh)
                            tma_load_rows(sq + X * TILE + hh * REG, &tmap_q, &q_full[X], hh * 64,
                                          it.h * g, it.q0 + row / g);
                        // the next round's tile into L2 meanwhile
                        Item nx;
                        if (rd + 1 < min(rounds, kItemCache) &&
                            round_at(p, table, num_items, rd + 1, false, nx)) {
#pragma unroll
                            for (int hh = 0; hh < HALVES; ++hh)
                                tma_prefetch_rows(&tmap_q, hh * 64, nx.h * g,
                                                  nx.q0 + (nx.row0 + X * kRows) / g);
                        }
                    }
                    __syncwarp();
                    continue;
                }
                for (int x = lane; x < kRows * CH; x += 32) {
                    const int r = x / CH, c = x - r * CH;
                    const int t = (row + r) / g;
                    const bool in = t < it.qlen;
                    const T* src = qb + ((size_t)(it.q0 + (in ? t : 0)) * Hq + it.h * g +
                                         (in ? row + r - t * g : 0)) * D + c * 8;
                    const uint32_t dst = smem_addr(sq + X * TILE + (c >> 3) * REG + r * 128 +
                                                   (((c & 7) ^ (r & 7)) << 4));
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst),
                                 "l"(src), "r"(in ? 16 : 0)
                                 : "memory");
                }
                asm volatile("cp.async.commit_group;\n" ::: "memory");
                asm volatile("cp.async.wait_all;\n" ::: "memory");
                asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[X]);
            }
        }
        // every copy issued must land before the CTA may exit
        if (q_tma && lane == 0)
            for (int X = 0; X < 2; ++X)
                if (issued[X] > 0) mbar_drain(&q_full[X], (issued[X] - 1) & 1, p.status);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------- MMA issuer
        // The whole warp walks the loop and one elected lane issues: descriptors,
        // addresses and conditions are then the same in all lanes and live in
        // uniform registers, which is where the MMA instruction takes them from.
        constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
        const uint32_t leader = elect_one();
        const uint32_t id_s = tc_idesc_f16(kBf16, kRows, kKeys, 0, 0);
        const uint32_t id_pv = tc_idesc_f16(kBf16, kRows, D, 0, 1);
        // operand descriptors: a step of x bytes adds x / 16 to the address field
        const uint64_t dq = tc_smem_desc(smem_addr(sq), 16, 1024);
        const uint64_t dk = tc_smem_desc(smem_addr(sk), 16, 1024);
        const uint64_t dv = tc_smem_desc(smem_addr(sv), REG, 1024);
        auto wait = [&](uint64_t* bar, int parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status));
        };
        // a cursor over the key tiles of this CTA's items, in order; per
        // tile X the items and key tiles it took part in
        struct Cur {
            int r, j, J, nkv, has_b;
            int items[2], tiles[2];
        };
        auto advance = [&](Cur& c) -> bool {
            if (c.r >= 0 && ++c.j < c.nkv) {
                ++c.J;
                ++c.tiles[0];
                if (c.has_b) ++c.tiles[1];
                return true;
            }
            for (++c.r; c.r < rounds; ++c.r) {
                Item it;
                const bool any = round_at(p, table, num_items, c.r, false, it);
                c.nkv = __shfl_sync(0xffffffffu, any ? it.nkv : 0, 0);
                c.has_b = __shfl_sync(0xffffffffu, it.has_b, 0);
                if (c.nkv == 0) continue;
                c.j = 0;
                ++c.J;
                ++c.items[0];
                ++c.tiles[0];
                if (c.has_b) {
                    ++c.items[1];
                    ++c.tiles[1];
                }
                return true;
            }
            return false;
        };
        // S_X(c) = Q_X K(c)^T into tile X's score buffer, over the last P_X, whose
        // P V was issued before (MMAs run in order)
        auto issue_s = [&](const Cur& c, int X) -> bool {
            const int b = c.J & 1;
            if (X == 0 && !wait(&k_full[b], (c.J >> 1) & 1)) return false;
            if (c.j == 0 && !wait(&q_full[X], c.items[X] & 1)) return false;
            tc_fence_after();
            const uint64_t da = dq + X * (TILE / 16), db = dk + b * (TILE / 16);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                mma_if(leader, tmem + X * kKeys, da + ((ks >> 2) * REG + (ks & 3) * 32) / 16,
                       db + ((ks >> 2) * REG + (ks & 3) * 32) / 16, id_s, ks > 0);
            commit_if(leader, &s_full[X]);
            if (X == 1 || !c.has_b) commit_if(leader, &k_empty[b]);
            if (c.j == c.nkv - 1) commit_if(leader, &q_empty[X]);
            return true;
        };
        // O_X += P_X(c) V(c): the P of a key half over the first 32 columns of that
        // half's scores
        auto issue_pv = [&](const Cur& c, int X) -> bool {
            const int b = c.J & 1;
            if (X == 0 && !wait(&v_full[b], (c.J >> 1) & 1)) return false;
            // the item's first P V overwrites O_X: the last item's must have been read
            if (c.j == 0 && c.items[X] >= 1 && !wait(&o_free[X], (c.items[X] - 1) & 1))
                return false;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (!wait(&p_full[2 * X + q], c.tiles[X] & 1)) return false;
                tc_fence_after();
                const uint64_t db = dv + b * (TILE / 16) + q * (kHalf / 16) * 128;
#pragma unroll
                for (int kk = 0; kk < kHalf / 16; ++kk)
                    mma_tmem_a_if(leader, tmem + kOCol + X * D,
                                  tmem + X * kKeys + kHalf * q + 8 * kk, db + kk * 128, id_pv,
                                  c.j > 0 || q > 0 || kk > 0);
            }
            if (X == 1 || !c.has_b) commit_if(leader, &v_empty[b]);
            if (c.j == c.nkv - 1) commit_if(leader, &o_ready[X]);
            return true;
        };
        Cur cs = {-1, 0, -1, 0, 0, {-1, -1}, {-1, -1}}, cp = cs;
        bool live = true;
        bool more = advance(cs);
        if (more) live = issue_s(cs, 0) && (!cs.has_b || issue_s(cs, 1));
        while (live && advance(cp)) {
            more = advance(cs);
            live = issue_pv(cp, 0);
            if (live && more) live = issue_s(cs, 0);
            if (live && cp.has_b) live = issue_pv(cp, 1);
            if (live && more && cs.has_b) live = issue_s(cs, 1);
        }
        // nothing of the leader's may still run when tensor memory is freed
        commit_if(leader, mma_idle);
        mbar_drain(mma_idle, 0, p.status);
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
        // ---------- scores of tile X, keys 64 q .. of each key tile: warps 4-7 A
        // first half, 8-11 A second, 12-15 and 16-19 B; one thread per row and half
        const int X = (warp - 4) >> 3, q = ((warp - 4) >> 2) & 1;
        const int wq = warp & 3;                             // tensor-memory lane quarter
        const int r = 32 * wq + lane;                        // row of the tile
        const uint32_t trow = tmem + ((uint32_t)(32 * wq) << 16);
        const uint32_t sx = trow + X * kKeys + kHalf * q;    // this half's scores / P
        const uint32_t ox = trow + kOCol + X * D + (D / 2) * q;  // this half's columns of O
        const ScoreMods& md = p.mods;
        const bool out32 = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
        int J = 0;             // key tiles of the CTA (the rings' count)
        int items = 0, tiles = 0;  // items and key tiles of this tile X
        int rescales = 0;          // of this warp's rows
        bool ok = true;
        for (int rd = 0; rd < rounds && ok; ++rd) {
            Item it;
            if (!round_at(p, table, num_items, rd, false, it)) continue;
            if (X == 1 && !it.has_b) {
                J += it.nkv;
                continue;
            }
            const int R = it.row0 + X * kRows + r, t = R / g;
            const bool live_row = t < it.qlen;
            const int head = it.h * g + (live_row ? R - t * g : 0);
            const int pos = it.n - it.qlen + (live_row ? t : 0);
            // this row's visible keys (rows past the chunk: everything, never stored)
            const int lo = live_row ? row_lo(p, it, pos) : 0;
            const int hi = live_row ? row_hi(it, pos) : 0x7fffffff;
            const float slope2 = kBias ? md.slopes[head] * kScoreLog2e : 0.f;
            float m_used = kFixed ? 0.f : -INFINITY, l = 0.f;
            for (int j = 0; j < it.nkv; ++j, ++J, ++tiles) {
                const int b = J & 1;
                // V(J) first, as it is there long before the scores.  Not for an
                // item's first tile: tile B's warps may come from far behind (items
                // without a tile B), where the parity alone would not tell V(J)
                // from V(J-4); S(J) written means that V(J-2) has been used.
                if (j == 0)
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(&s_full[X], tiles & 1, abort_flag, p.status));
                if (!ok) break;
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&v_full[b], (J >> 1) & 1, abort_flag, p.status));
                if (!ok) break;
                const unsigned bad = ((unsigned)vbad[b] >> (4 * q)) & 0xFu;  // this half's blocks
                const int key0 = it.b0 * PKV_BLOCK_SIZE + kKeys * j + kHalf * q;
                const bool whole = bad == 0u && __all_sync(0xffffffffu, key0 >= lo &&
                                                                            key0 + kHalf <= hi);
                // keys of chunk w (32 keys) that this row sees
                auto seen = [&](int w) -> uint32_t {
                    const int f0 = min(max(lo - key0 - 32 * w, 0), 32);
                    const int f1 = min(max(hi - key0 - 32 * w, 0), 32);
                    uint32_t see = (f1 == 32 ? 0xffffffffu : (1u << f1) - 1u) &
                                   (f0 == 32 ? 0u : 0xffffffffu << f0);
                    if ((bad >> (2 * w)) & 1u) see &= 0xffff0000u;
                    if ((bad >> (2 * w + 1)) & 1u) see &= 0x0000ffffu;
                    return see;
                };
                if (j > 0)
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(&s_full[X], tiles & 1, abort_flag, p.status));
                if (!ok) break;
                tc_fence_after();
                float sc[kHalf];
                tc_ld32(sx, reinterpret_cast<uint32_t(&)[32]>(sc[0]));
                tc_ld32(sx + 32, reinterpret_cast<uint32_t(&)[32]>(sc[32]));
                tc_wait_ld();
                uint64_t acc2[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
                float f = 1.f;  // factor on what the row has so far
                // sc becomes z / mul (z: base-2 scores), with mul > 0
                float mul = md.scale_log2, ms = 0.f;
                float m_mine = 0.f, down = 1.f;
                bool done = false;
                if constexpr (kCap) {
                    const float top = largest(sc);
                    mul = 1.f;
                    if (kFixed && whole && __all_sync(0xffffffffu, top <= p.tanh_few_limit)) {
                        // the common case in one piece, so that polynomials (fp32
                        // pipe) and exponentials (special-function pipe) overlap
                        const uint64_t c2 = f2(p.tanh_few[2], p.tanh_few[2]);
                        const uint64_t c1 = f2(p.tanh_few[1], p.tanh_few[1]);
                        const uint64_t c0 = f2(p.tanh_few[0], p.tanh_few[0]);
#pragma unroll
                        for (int w = 0; w < kHalf / 32; ++w) {
                            uint32_t pk[16];
#pragma unroll
                            for (int e0 = 0; e0 < 16; e0 += 4) {
                                uint64_t x[4], v[4], y[4];
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    const int c = 32 * w + 2 * (e0 + u);
                                    x[u] = f2(sc[c], sc[c + 1]);
                                    v[u] = f2_mul(x[u], x[u]);
                                }
#pragma unroll
                                for (int u = 0; u < 4; ++u) y[u] = f2_fma(c2, v[u], c1);
#pragma unroll
                                for (int u = 0; u < 4; ++u) y[u] = f2_fma(y[u], v[u], c0);
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    float a0, a1;
                                    f2_split(f2_mul(x[u], y[u]), a0, a1);
                                    const float p0 = fast_exp2(a0), p1 = fast_exp2(a1);
                                    acc2[u] = f2_add(acc2[u], f2(p0, p1));
                                    pk[e0 + u] = E::pack(p0, p1);
                                }
                            }
                            tc_st16(sx + 16 * w, pk);
                        }
                        done = true;
                    } else {
                        cap_to_z<kFixed>(p, sc, top);
                    }
                }
                if (!done) {
                    if constexpr (kBias) {
                        // distance |p - t|: keys before the row's position for all but
                        // the tiles at the diagonal or in a prefix
                        const uint64_t mul2 = f2(mul, mul);
                        if (__all_sync(0xffffffffu, key0 + kHalf - 1 <= pos)) {
                            const float base = slope2 * (float)(key0 - pos);
                            const uint64_t step2 = f2(2.f * slope2, 2.f * slope2);
#pragma unroll
                            for (int c0 = 0; c0 < kHalf; c0 += 8) {
                                // (exact products for a pair, then at most three steps)
                                uint64_t bb = f2(fmaf(slope2, (float)c0, base),
                                                 fmaf(slope2, (float)(c0 + 1), base));
#pragma unroll
                                for (int c = c0; c < c0 + 8; c += 2) {
                                    f2_split(f2_fma(f2(sc[c], sc[c + 1]), mul2, bb), sc[c], sc[c + 1]);
                                    if (c < c0 + 6) bb = f2_add(bb, step2);
                                }
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < kHalf; ++c)
                                sc[c] = fmaf(-slope2, fabsf((float)(key0 + c - pos)), sc[c] * mul);
                        }
                        mul = 1.f;
                    } else if (mul <= 0.f) {
#pragma unroll
                        for (int c = 0; c < kHalf; ++c) sc[c] *= mul;
                        mul = 1.f;
                    }
                    if (!whole) {  // select: hidden scores may be anything
#pragma unroll
                        for (int w = 0; w < kHalf / 32; ++w) {
                            const uint32_t see = seen(w);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                sc[32 * w + c] = (see >> c) & 1u ? sc[32 * w + c] : -INFINITY;
                        }
                    }
                    // |z| <= cap' <= kFixedMax (kFixed): weights 2^z fit bf16 and their
                    // sums fp32 without a maximum taken out
                    if constexpr (!kFixed) {
                        float mxp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < kHalf; c += 2)
                            mxp[(c >> 1) & 3] = max3(mxp[(c >> 1) & 3], sc[c], sc[c + 1]);
                        const float mx =
                            fmaxf(fmaxf(mxp[0], mxp[1]), fmaxf(mxp[2], mxp[3])) * mul;
                        // The reference 2^m of the weights is a whole power, and follows
                        // the row's maximum only where that grew by more than 2^kRescale.
                        // This half tells the other what it wants, takes its own for the
                        // weights meanwhile, and scales them after if the other's is larger
                        // (by a power of two: exact).
                        m_mine = m_used == -INFINITY || mx > m_used + kRescale ? ceilf(mx) : m_used;
                        xm[(((tiles & 1) * 2 + X) * 2 + q) * kRows + r] = m_mine;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&x_max[4 * X + wq]);
                        ms = m_mine == -INFINITY ? 0.f : m_mine;
                    }
                    // P as 16-bit pairs; the sum takes the unrounded weights
                    const uint64_t mul2 = f2(mul, mul), nms2 = f2(-ms, -ms);
                    uint32_t pk[kHalf / 2];
#pragma unroll
                    for (int e = 0; e < kHalf / 2; ++e) {
                        float a0 = sc[2 * e], a1 = sc[2 * e + 1];
                        if constexpr (!kFixed) f2_split(f2_fma(f2(a0, a1), mul2, nms2), a0, a1);
                        const float p0 = fast_exp2(a0), p1 = fast_exp2(a1);
                        acc2[e & 3] = f2_add(acc2[e & 3], f2(p0, p1));
                        pk[e] = E::pack(p0, p1);
                    }
                    if constexpr (!kFixed) {
                        ok = __all_sync(0xffffffffu, mbar_wait(&x_max[4 * X + wq], tiles & 1,
                                                               abort_flag, p.status));
                        if (!ok) break;
                        const float m_new = fmaxf(
                            m_mine, xm[(((tiles & 1) * 2 + X) * 2 + (q ^ 1)) * kRows + r]);
                        const bool grow = m_used != -INFINITY && m_new > m_used;
                        f = grow ? fast_exp2(m_used - m_new) : 1.f;
                        const bool low = m_new > m_mine;
                        m_used = m_new;
                        if (__any_sync(0xffffffffu, low)) {
                            // (below 2^-24 of the other half's largest weight: nothing)
                            down = low ? fast_exp2(m_mine - m_new) : 1.f;
#pragma unroll
                            for (int e = 0; e < kHalf / 2; ++e) pk[e] = scale_pair<T>(pk[e], down);
                        }
                        if (__any_sync(0xffffffffu, grow)) {  // (the same in both halves' warps)
                            // S_X(J) was issued after P V_X(J-1): O_X holds every earlier tile
#pragma unroll 1
                            for (int c = 0; c < D / 64; ++c) {
                                uint32_t o[32];
                                tc_ld32(ox + 32 * c, o);
                                tc_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tc_st32(ox + 32 * c, o);
                            }
                            // P V of either key half adds to every column of O: neither
                            // half lets its P go before both have rescaled their columns
                            tc_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&x_scale[4 * X + wq]);
                            ok = __all_sync(0xffffffffu, mbar_wait(&x_scale[4 * X + wq], rescales & 1,
                                                                   abort_flag, p.status));
                            if (!ok) break;
                            ++rescales;
                        }
                    }
                    tc_st16(sx, reinterpret_cast<uint32_t(&)[16]>(pk[0]));
                    tc_st16(sx + 16, reinterpret_cast<uint32_t(&)[16]>(pk[16]));
                }
                tc_wait_st();
                // V rows that no row of the item sees (or that were not loaded)
                // become zeros before P V; both tiles zero the same rows
                if (key0 < it.lo || key0 + kHalf > it.hi || bad) {
                    unsigned char* vt = sv + b * TILE + kHalf * q * 128;
                    for (int x = r; x < kHalf * 8 * HALVES; x += kRows) {
                        const int kq = x / (8 * HALVES), rest = x - kq * (8 * HALVES);
                        const int key = key0 + kq;
                        if (key >= it.lo && key < it.hi && !((bad >> (kq >> 4)) & 1u)) continue;
                        *reinterpret_cast<uint4*>(vt + (rest >> 3) * REG + kq * 128 +
                                                  ((rest & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                }
                tc_fence_before();  // P and a rescaled O are ordered before the next MMA
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * X + q]);
                float psum = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float a0, a1;
                    f2_split(acc2[e], a0, a1);
                    psum += a0 + a1;
                }
                l = l * f + psum * down;
            }
            if (!ok) break;
            // ---- epilogue: O_X / l (this half's columns) for the rows of the chunk,
            // or their partials
            const bool split = p.splits > 1;
            const size_t orow = (size_t)(it.q0 + (live_row ? t : 0)) * Hq + head;
            T* dst = static_cast<T*>(p.out) + orow * D + (D / 2) * q;
            const size_t prow =
                ((size_t)it.base * p.splits + it.split) * kPair + X * kRows + r;
            if (it.nkv == 0) {  // nothing visible: zeros, or an empty partial (l = 0)
                if (live_row && split && q == 0) {
                    p.ws_m[prow] = -INFINITY;
                    p.ws_l[prow] = 0.f;
                }
                if (live_row && !split)
                    for (int c = 0; c < D / 16; ++c)
                        *reinterpret_cast<uint4*>(dst + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            // the row's sum over both halves
            float* mine = xl + (((items & 1) * 2 + X) * 2 + q) * kRows + r;
            *mine = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(&x_sum[4 * X + wq]);
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&x_sum[4 * X + wq], items & 1, abort_flag, p.status));
            if (!ok) break;
            l += *(mine + (q ? -kRows : kRows));
            const float inv = l != 0.f ? 1.f / l : 0.f;
            if (split && live_row && q == 0) {
                p.ws_m[prow] = m_used;
                p.ws_l[prow] = l;
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&o_ready[X], items & 1, abort_flag, p.status));
            if (!ok) break;
            ++items;
            tc_fence_after();
            float zero = 0.f;  // finite values times zero: NaN if one is not finite
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
                float o[32];
                tc_ld32(ox + 32 * c, reinterpret_cast<uint32_t(&)[32]>(o));
                tc_wait_ld();
                float z4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 32; ++e) z4[e & 3] = fmaf(0.f, o[e], z4[e & 3]);
                zero += (z4[0] + z4[1]) + (z4[2] + z4[3]);
                if (!live_row) continue;
                if (split) {
                    float* od = p.ws_o + prow * D + (D / 2) * q + 32 * c;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4*>(od + 4 * e) =
                            make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    continue;
                }
                uint32_t w[16];
#pragma unroll
                for (int u = 0; u < 16; ++u) w[u] = E::pack(o[2 * u] * inv, o[2 * u + 1] * inv);
                if (out32) {  // 32-byte stores: each fills a whole L2 sector
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        uint32_t w8[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) w8[u] = w[8 * hh + u];
                        st_global_v8(dst + 32 * c + 16 * hh, w8);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4*>(dst + 32 * c + 8 * e) =
                            make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[X]);
            // rows whose weights are finite but whose O is not (a value of V that
            // may be hidden from the row): again, from the row's own keys.  A row
            // with a NaN among its own scores is NaN, as it should be; a row that
            // sees nothing (l = 0) becomes zeros.
            const unsigned redo = __ballot_sync(0xffffffffu, live_row && zero != 0.f && l - l == 0.f);
            if (redo)
                redo_rows<T, D>(p, it, it.row0 + X * kRows + 32 * wq, q, redo, l, prow - lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tc_dealloc(tmem, kCols);
    }
}

// Joins the splits of one item's rows, a warp per row:
//   M = max m,  out = sum o 2^(m - M) / sum l 2^(m - M).
// Lane k has split k's m and l (at most 32 splits); the o of eight splits are in
// flight at a time.  A programmatic dependent of the kernel above.
constexpr int kJoinWarps = 8;
constexpr int kJoinRows = 8;   // rows of an item per CTA: a warp each
constexpr int kMaxSplits = 32;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) scored_prefill_join_kernel(const PrefillScored p) {
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = p.group, S = p.splits;
    const int base = blockIdx.x / (kPair / kJoinRows);
    const int r = blockIdx.x % (kPair / kJoinRows) * kJoinRows + warp;
    const int sh = base / p.pairs_per_seq, pair = base - sh * p.pairs_per_seq;
    const int s = sh / p.num_kv_heads, h = sh - s * p.num_kv_heads;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int q0 = p.cu_q_lens[s], qlen = p.cu_q_lens[s + 1] - q0, n = p.context_lens[s];
    const int R = pair * kPair + r;
    if (!lengths_ok(p, q0, qlen, n) || R >= qlen * g) return;
    const size_t row = (size_t)base * S * kPair + r;
    const float m = lane < S ? p.ws_m[row + (size_t)lane * kPair] : -INFINITY;
    const float l = lane < S ? p.ws_l[row + (size_t)lane * kPair] : 0.f;
    float M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M == -INFINITY) M = 0.f;
    // (a split without visible keys, l = 0, wrote no o)
    const float w = l != 0.f ? fast_exp2(m - M) : 0.f;
    float L = w * l, acc[PER];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    const unsigned some = __ballot_sync(0xffffffffu, l != 0.f);
    const float* o0 = p.ws_o + row * D + lane * PER;
#pragma unroll 1
    for (int k0 = 0; k0 < S; k0 += 8) {
        float x[8][PER];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int e = 0; e < PER; ++e)
                x[k][e] = (some >> (k0 + k)) & 1u ? o0[(size_t)(k0 + k) * kPair * D + e] : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k0 + k);
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = fmaf(wk, x[k][e], acc[e]);
        }
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    const int t = R / g, head = h * g + R - t * g;
    T* dst = static_cast<T*>(p.out) + ((size_t)(q0 + t) * p.num_q_heads + head) * D + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = Elem<T>::pack(acc[e] * inv, acc[e + 1] * inv);
}

// Items before splitting, and into how many key runs each is cut: enough for
// every SM, but none shorter than two key tiles.
struct Plan {
    long long items;
    int pairs, splits;
};

Plan make_plan(int num_seqs, int max_q_len, int num_kv_heads, int group, int ctas,
               long long max_tiles) {
    Plan pl;
    pl.pairs = (int)(((long long)max_q_len * group + kPair - 1) / kPair);
    pl.items = (long long)num_seqs * num_kv_heads * pl.pairs;
    const long long by_ctas = pl.items > 0 ? ctas / pl.items : 1;
    pl.splits =
        (int)std::max<long long>(1, std::min({by_ctas, max_tiles / 2, (long long)kMaxSplits}));
    return pl;
}

struct Workspace {
    size_t m, l, o, total;
};

Workspace ws_layout(long long rows, int head_dim) {
    Workspace w;
    w.m = 0;
    w.l = align256((size_t)rows * 4);
    w.o = w.l + align256((size_t)rows * 4);
    w.total = w.o + (size_t)rows * head_dim * 4;
    return w;
}

// The fewer terms of tanh(x) / x = 1 - x^2 / 3 + 2 x^4 / 15 - ... for small x
// (what is left out is below 4e-7 there).
constexpr float kTanhSmall[3][3] = {{1.f, 0.f, 0.f}, {1.f, -0.333333333f, 0.f},
                                    {kTanh3[0], kTanh3[1], kTanh3[2]}};
constexpr float kTanhSmallRange[3] = {1e-3f, 0.04f, kTanhFewRange};

// The terms c_i x^2i as terms of (raw score)^2i times the cap's scale; returns
// `range`, or -1 if one of them leaves the normal numbers.
float scaled_terms(const float* c, int n, float range, const ScoreMods& m, float* out) {
    const double c2 = (double)m.cap_in * m.cap_in;
    double f = m.scale_log2;
    for (int i = 0; i < n; ++i, f *= c2) {
        out[i] = (float)(c[i] * f);
        if (!std::isnormal(out[i])) return -1.f;
    }
    return range;
}

template <int D>
size_t prefill_smem() {
    // 2 Q tiles, 2 K and 2 V stages, barriers (under 1 KB) and the halves'
    // maxima and sums (4 KB each), the items; 1 KB alignment slack
    return 1024 + (size_t)6 * (D / 64) * kRows * 128 + 1024 + 2 * 2 * 2 * 2 * kRows * 4 +
           kItemCache * sizeof(Item);
}

template <typename T, int D, bool kCap, bool kBias, bool kFixed = false>
pkv_status launch(const PrefillScored& prm, const CUtensorMap& tmk, const CUtensorMap& tmv,
                  const CUtensorMap& tmq, int q_tma, int items, int ctas, cudaStream_t stream) {
    auto kern = scored_prefill_kernel<T, D, kCap, kBias, kFixed>;
    // the register shares assume the launch count of this build
    static const bool regs_ok = [&] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, kern) == cudaSuccess && a.numRegs == kLaunchRegs;
    }();
    if (!regs_ok) return PKV_ERR_CUDA;
    const size_t smem = prefill_smem<D>();
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
        return PKV_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min(items, ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = prm.splits > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kern, prm, tmk, tmv, tmq, q_tma, items) != cudaSuccess)
        return PKV_ERR_CUDA;
    if (prm.splits == 1) return PKV_OK;
    cfg.gridDim = dim3((unsigned)(items / prm.splits * (kPair / kJoinRows)));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.dynamicSmemBytes = 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, scored_prefill_join_kernel<T, D>, prm));
}

template <typename T, int D>
pkv_status launch_mods(const PrefillScored& prm, pkv_dtype dtype, int items, int ctas,
                       cudaStream_t stream) {
    CUtensorMap tmk, tmv, tmq;
    if (!make_pool_map(&tmk, prm.k_cache, prm.num_blocks, prm.num_kv_heads, D, dtype) ||
        !make_pool_map(&tmv, prm.v_cache, prm.num_blocks, prm.num_kv_heads, D, dtype))
        return PKV_ERR_CUDA;
    const int q_tma =
        make_q_tile_map(&tmq, prm.q, prm.num_q_rows, prm.num_q_heads, D, prm.group, dtype) ? 1 : 0;
    if (!q_tma) tmq = tmk;  // unused
    const bool cap = prm.mods.cap_out > 0.f, bias = prm.mods.slopes != nullptr;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        if (cap && !bias && prm.mods.cap_out <= kFixedMax && prm.splits == 1)
            return launch<T, D, true, false, true>(prm, tmk, tmv, tmq, q_tma, items, ctas, stream);
    }
    if (cap)
        return bias ? launch<T, D, true, true>(prm, tmk, tmv, tmq, q_tma, items, ctas, stream)
                    : launch<T, D, true, false>(prm, tmk, tmv, tmq, q_tma, items, ctas, stream);
    return bias ? launch<T, D, false, true>(prm, tmk, tmv, tmq, q_tma, items, ctas, stream)
                : launch<T, D, false, false>(prm, tmk, tmv, tmq, q_tma, items, ctas, stream);
}

}  // namespace
}  // namespace pkv

extern "C" {

size_t paged_attention_prefill_scored_workspace_bytes(int num_seqs, int max_q_len, int num_q_heads,
                                                      int num_kv_heads, int head_dim) {
    if (num_seqs <= 0 || max_q_len <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        num_q_heads % num_kv_heads != 0 || (head_dim != 64 && head_dim != 128))
        return 0;
    const pkv::Plan pl = pkv::make_plan(num_seqs, max_q_len, num_kv_heads,
                                        num_q_heads / num_kv_heads, pkv::kMaxCtas, 1 << 30);
    if (pl.splits == 1) return 256;
    return pkv::ws_layout(pl.items * pl.splits * pkv::kPair, head_dim).total;
}

pkv_status paged_attention_prefill_scored(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* context_lens, const int32_t* cu_q_lens, int num_seqs,
    int max_q_len, int num_q_rows, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
    float scale, float softcap, const float* alibi_slopes, int window, const int32_t* key_starts,
    const int32_t* prefix_lens, void* out, void* workspace, size_t workspace_bytes,
    pkv_dtype dtype, pkv_stream_t stream) {
    if (num_seqs < 0 || max_q_len < 0 || num_q_rows < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    pkv::PrefillScored prm = {};
    if (!pkv::make_score_mods(&prm.mods, scale, softcap, alibi_slopes, window, key_starts,
                              prefix_lens))
        return PKV_ERR_INVALID_ARG;
    const int g = num_q_heads / num_kv_heads;
    if (g > pkv::kMaxGroup || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
    if (max_blocks_per_seq > 0x7fffffff / PKV_BLOCK_SIZE ||
        num_blocks > 0x7fffffff / PKV_BLOCK_SIZE || max_q_len > 0x7fffffff / 32 - 256)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || max_q_len == 0 || num_q_rows == 0) return PKV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !cu_q_lens || !out)
        return PKV_ERR_INVALID_ARG;
    if (!pkv::aligned16(q) || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache) ||
        !pkv::aligned16(out))
        return PKV_ERR_INVALID_ARG;
    if (pkv::overlap(q, out, (size_t)num_q_rows * num_q_heads * head_dim * 2))
        return PKV_ERR_INVALID_ARG;
    const size_t need = paged_attention_prefill_scored_workspace_bytes(
        num_seqs, max_q_len, num_q_heads, num_kv_heads, head_dim);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PKV_ERR_WORKSPACE;
    prm.status = pkv::status_word();
    const int sms = pkv::sm_count();
    if (!prm.status || sms <= 0) return PKV_ERR_CUDA;
    const int ctas = std::min(sms, pkv::kMaxCtas);
    // most key tiles of an item
    long long keys = (long long)max_blocks_per_seq * PKV_BLOCK_SIZE;
    if (window > 0) keys = std::min(keys, (long long)window + max_q_len + PKV_BLOCK_SIZE);
    const pkv::Plan pl = pkv::make_plan(num_seqs, max_q_len, num_kv_heads, g, ctas,
                                        (keys + pkv::kKeys - 1) / pkv::kKeys);
    if (pl.items * pl.splits > 0x7fffffffll / 64) return PKV_ERR_UNSUPPORTED;
    prm.q = q;
    prm.k_cache = k_cache;
    prm.v_cache = v_cache;
    prm.out = out;
    prm.block_tables = block_tables;
    prm.context_lens = context_lens;
    prm.cu_q_lens = cu_q_lens;
    prm.num_seqs = num_seqs;
    prm.num_q_heads = num_q_heads;
    prm.num_kv_heads = num_kv_heads;
    prm.group = g;
    prm.max_blocks_per_seq = max_blocks_per_seq;
    prm.num_blocks = num_blocks;
    prm.max_q_len = max_q_len;
    prm.num_q_rows = num_q_rows;
    prm.pairs_per_seq = pl.pairs;
    prm.splits = pl.splits;
    // worth its 1 to 2 us where a CTA may get several items, possible where the
    // entries fit the scratch and the CTA's table all of its items
    const long long entries = (long long)num_seqs * pl.pairs;
    prm.sorted = pl.items * pl.splits > ctas && entries <= pkv::kSortMax &&
                 pl.items * pl.splits <= (long long)pkv::kItemCache * ctas;
    // z = cap' x (tanh(x) / x) with x = raw cap_in: the terms in raw^2, times cap' cap_in
    prm.tanh_limit = prm.tanh_few_limit = prm.tanh_wide_limit = -1.f;
    if (softcap > 0.f && scale != 0.f) {
        const float in = std::fabs(prm.mods.cap_in);
        float range = pkv::scaled_terms(pkv::kTanh4, pkv::kTanhTerms, pkv::kTanhRange, prm.mods,
                                        prm.tanh_z);
        // caps far above the scores: the last terms leave the range of fp32, and
        // are not needed where x is small enough
        for (int n = pkv::kTanhTerms - 1; range < 0.f && n > 0; --n) {
            for (float& t : prm.tanh_z) t = 0.f;
            range = pkv::scaled_terms(pkv::kTanhSmall[n - 1], n, pkv::kTanhSmallRange[n - 1],
                                      prm.mods, prm.tanh_z);
        }
        // (raw^2 has to be finite as well)
        if (range > 0.f) prm.tanh_limit = std::min(range / in, 1e18f);
        const float few = pkv::scaled_terms(pkv::kTanh3, pkv::kTanhFew, pkv::kTanhFewRange,
                                            prm.mods, prm.tanh_few);
        if (few > 0.f) prm.tanh_few_limit = std::min(few / in, 1e18f);
        const float wide = pkv::scaled_terms(pkv::kTanh8, pkv::kTanhWide, pkv::kTanhWideRange,
                                             prm.mods, prm.tanh_wide);
        if (wide > 0.f) prm.tanh_wide_limit = std::min(wide / in, 1e18f);
    }
    const pkv::Workspace ws =
        pkv::ws_layout(pl.splits > 1 ? pl.items * pl.splits * pkv::kPair : 0, head_dim);
    char* w = static_cast<char*>(workspace);
    prm.ws_m = reinterpret_cast<float*>(w + ws.m);
    prm.ws_l = reinterpret_cast<float*>(w + ws.l);
    prm.ws_o = reinterpret_cast<float*>(w + ws.o);
    const int items = (int)(pl.items * pl.splits);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == PKV_BF16)
        return head_dim == 128
                   ? pkv::launch_mods<__nv_bfloat16, 128>(prm, dtype, items, ctas, st)
                   : pkv::launch_mods<__nv_bfloat16, 64>(prm, dtype, items, ctas, st);
    return head_dim == 128 ? pkv::launch_mods<__half, 128>(prm, dtype, items, ctas, st)
                           : pkv::launch_mods<__half, 64>(prm, dtype, items, ctas, st);
}

}  // extern "C"
