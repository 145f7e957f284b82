// pkv_rope.cu -- rotary positions of q and k, fused with the write of the
// rotated k and of v into the paged cache.
//
// For a token at position p and pair j < R / 2 (R = rotary_dim <= head_dim)
//     a = p * f_j,   c = m cos a,   s = m sin a      (f = inv_freq, m = rope_scale)
//     y0 = x0 c - x1 s,   y1 = x1 c + x0 s
// with (x0, x1) = (x_j, x_{j+R/2}) in the half layout and (x_2j, x_2j+1) in
// the interleaved one; elements R.. of a head are copied.  Every product is
// fp32 and each element is rounded once, when it is stored.
//
// The angle.  Positions reach millions, where p * f_j in fp32 is off by tenths
// of a radian.  The turns p * f_j / 2pi are needed modulo 1 only, so they are
// formed from g = f_j / 2pi held as a pair of floats gh + gl and from
// p = 65536 ph + pl (both parts exact in fp32): x * gh splits into its rounded
// product and the exact remainder fma(x, gh, -product), each reduced by its
// nearest whole number of turns (exact), and x * gl adds what gh leaves out.
// For |p| < 2^24 the turns are within 2^-23 of the exact ones; sincospif does
// the rest.  (64-bit products cost more: 64 lanes' worth of them per token
// share an FP64 pipe of two lanes an SM.)
#include <algorithm>
#include <cmath>

#include "pkv_internal.cuh"

namespace pkv {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxDim = 512;   // head_dim
constexpr int kRopeBatch = 2;      // head rows a thread has in flight

struct RopeParams {
    const void* q;
    const void* k_new;
    const void* v_new;
    void* q_out;
    void* k_cache;
    void* v_cache;
    long long q_stride, k_stride, v_stride;  // elements between tokens
    const float* inv_freq;
    float rope_scale;
    int num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim, num_blocks;
    // tokens with positions and slots ...
    const int32_t* positions;
    const int64_t* slot_mapping;
    // ... or (positions null) one new token per sequence at position length - 1
    const int32_t* block_tables;
    const int32_t* context_lens;
    int max_blocks_per_seq;
    int64_t* slot_out;
    unsigned int* status;
};

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(__half& d, float x) { d = __float2half_rn(x); }

constexpr int kVec = 8;  // elements of a 16-byte word

template <typename T>
union Vec {
    uint4 w;
    T e[kVec];
    __device__ __forceinline__ Vec() {}
};

// cos and sin (times m) of p * f.
__device__ __forceinline__ void rotation(int p, float f, float m, float& c, float& s) {
    constexpr float kHi = 0.159154943f;            // 1 / 2pi rounded to fp32 ...
    constexpr float kLo = (float)(0.15915494309189533576888 - (double)kHi);  // ... and the rest
    const float gh = f * kHi;
    const float gl = fmaf(f, kLo, fmaf(f, kHi, -gh));
    float turns = 0.f, rest = 0.f;
    const float part[2] = {(float)(p & 0xffff), (float)(p >> 16) * 65536.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float a = part[i] * gh;
        const float e = fmaf(part[i], gh, -a);
        turns += a - rintf(a);
        rest += (e - rintf(e)) + part[i] * gl;
    }
    turns += rest;
    turns -= rintf(turns);
    sincospif(2.f * turns, &s, &c);
    c *= m;
    s *= m;
}

// The token's cache slot and position; false if there is nothing to do for it
// (a padding token, or a bad value, reported by thread 0).
__device__ __forceinline__ bool token_place(const RopeParams& p, int t, bool report, int& pos,
                                            int64_t& slot) {
    slot = -1;
    if (p.positions) {
        slot = p.slot_mapping[t];
        if (slot < 0) return false;
        if (slot >= (int64_t)p.num_blocks * PKV_BLOCK_SIZE) {
            if (report) atomicOr(p.status, PKV_DEV_BAD_SLOT);
            return false;
        }
        pos = p.positions[t];
        return true;
    }
    const int n = p.context_lens[t];
    if (n > 0 && n <= (long long)p.max_blocks_per_seq * PKV_BLOCK_SIZE) {
        pos = n - 1;
        const int32_t b = p.block_tables[(int64_t)t * p.max_blocks_per_seq + pos / PKV_BLOCK_SIZE];
        if (b >= 0 && b < p.num_blocks)
            slot = (int64_t)b * PKV_BLOCK_SIZE + pos % PKV_BLOCK_SIZE;
        else if (report)
            atomicOr(p.status, PKV_DEV_BAD_BLOCK_ID);
    } else if (n != 0 && report) {
        atomicOr(p.status, PKV_DEV_BAD_LENGTH);
    }
    if (report && p.slot_out) p.slot_out[t] = slot;
    return slot >= 0;
}

// Row r of a token's Hq + 2 Hkv head rows: where it comes from and goes to.
template <typename T>
struct TokenRows {
    const RopeParams& p;
    int t;
    __device__ __forceinline__ const T* source(int r) const {
        if (r < p.num_q_heads)
            return static_cast<const T*>(p.q) + t * p.q_stride + (int64_t)r * p.head_dim;
        r -= p.num_q_heads;
        if (r < p.num_kv_heads)
            return static_cast<const T*>(p.k_new) + t * p.k_stride + (int64_t)r * p.head_dim;
        return static_cast<const T*>(p.v_new) + t * p.v_stride +
               (int64_t)(r - p.num_kv_heads) * p.head_dim;
    }
    __device__ __forceinline__ T* target(int r, int64_t slot) const {
        if (r < p.num_q_heads)
            return static_cast<T*>(p.q_out) + ((int64_t)t * p.num_q_heads + r) * p.head_dim;
        r -= p.num_q_heads;
        if (r < p.num_kv_heads)
            return static_cast<T*>(p.k_cache) + (slot * p.num_kv_heads + r) * p.head_dim;
        return static_cast<T*>(p.v_cache) +
               (slot * p.num_kv_heads + r - p.num_kv_heads) * p.head_dim;
    }
};

// Both kernels are programmatic dependents: their CTAs are scheduled while the
// kernel in front of them drains (in a row of calls 16384 tokens take 60.0 us, with
// ordinary launches 60.7; four tokens 2.6 and 2.7), and touch nothing of the
// caller's before it is complete.  They let the kernel behind them be scheduled in the same way.
__device__ __forceinline__ void wait_for_the_kernel_in_front() {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

// One CTA per token.  Thread (x, y): x is a unit of a head row -- interleaved:
// one 16-byte word; half layout: the word at j and its partner at j + R / 2, or a
// copied word -- and the same for every head, so a thread uses the same cosines
// and sines while it walks the token's head rows (q, k, v; v's units are copied)
// in steps of blockDim.y.  The first rows' loads are issued before the token's
// slot is known and before the angles are formed.
// HBM bound: 2 (Hq + 2 Hkv) D elements read and written per token.  16384
// tokens of 32q/8kv heads of 128: 60.0 us, 6.72 TB/s.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeMaxDim, 3) rope_write_kernel(const RopeParams p) {
    __shared__ __align__(16) float sm_cos[kRopeMaxDim / 2], sm_sin[kRopeMaxDim / 2];
    const int t = blockIdx.x;
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    const TokenRows<T> rows_of = {p, t};
    const int R = p.rotary_dim, half = R / 2;
    const int rotated_rows = p.num_q_heads + p.num_kv_heads;
    const int rows = rotated_rows + p.num_kv_heads;
    // this thread's unit: its first element(s)
    const int x = threadIdx.x;
    const bool pair = !kInterleaved && x < half / kVec;
    const int e0 = kInterleaved || pair ? x * kVec : R + (x - half / kVec) * kVec;
    const int e1 = e0 + half;  // the half layout's partner elements
    wait_for_the_kernel_in_front();

    Vec<T> a[kRopeBatch], b[kRopeBatch];
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < kRopeBatch; ++i) {
            const int r = r0 + i * (int)blockDim.y;
            if (r >= rows) continue;
            const T* src = rows_of.source(r);
            a[i].w = *reinterpret_cast<const uint4*>(src + e0);
            if (pair) b[i].w = *reinterpret_cast<const uint4*>(src + e1);
        }
    };
    load(threadIdx.y);  // (a padding token's rows are there too)
    int pos = 0;
    int64_t slot;
    if (!token_place(p, t, tid == 0, pos, slot)) return;  // uniform over the CTA
    for (int j = tid; j < half; j += blockDim.x * blockDim.y)
        rotation(pos, p.inv_freq[j], p.rope_scale, sm_cos[j], sm_sin[j]);
    __syncthreads();
    const float* c = sm_cos + (kInterleaved ? e0 / 2 : e0);  // (rotated units only)
    const float* s = sm_sin + (kInterleaved ? e0 / 2 : e0);
    for (int r0 = threadIdx.y; r0 < rows; r0 += kRopeBatch * blockDim.y) {
        if (r0 != (int)threadIdx.y) load(r0);
#pragma unroll
        for (int i = 0; i < kRopeBatch; ++i) {
            const int r = r0 + i * (int)blockDim.y;
            if (r >= rows) continue;
            if (r < rotated_rows) {
                if constexpr (kInterleaved) {
#pragma unroll
                    for (int u = 0; u < kVec / 2; ++u) {
                        if (e0 + 2 * u >= R) continue;  // (R may end inside the word)
                        const float x0 = to_f32(a[i].e[2 * u]), x1 = to_f32(a[i].e[2 * u + 1]);
                        from_f32(a[i].e[2 * u], x0 * c[u] - x1 * s[u]);
                        from_f32(a[i].e[2 * u + 1], x1 * c[u] + x0 * s[u]);
                    }
                } else if (pair) {
#pragma unroll
                    for (int u = 0; u < kVec; ++u) {
                        const float x0 = to_f32(a[i].e[u]), x1 = to_f32(b[i].e[u]);
                        from_f32(a[i].e[u], x0 * c[u] - x1 * s[u]);
                        from_f32(b[i].e[u], x1 * c[u] + x0 * s[u]);
                    }
                }
            }
            T* dst = rows_of.target(r, slot);
            *reinterpret_cast<uint4*>(dst + e0) = a[i].w;
            if (pair) *reinterpret_cast<uint4*>(dst + e1) = b[i].w;
        }
    }
}

// The half layout where R / 2 is not a multiple of 8: a word's partners straddle
// two words.  The rows go through shared memory as well; a thread turns the same
// word of several rows, taking its partners (element e pairs with e + R / 2 or
// e - R / 2) one by one from there.  (Moving such rows by 2-byte
// elements took 105 us where this takes 67 us: 16384 tokens of 8q/8kv heads
// of 128, R = 90.)
constexpr int kStagedThreads = 128;
constexpr int kStagedBatch = 3;    // head rows a thread turns between two barriers

template <typename T>
__global__ void __launch_bounds__(kStagedThreads, 10) rope_write_staged_kernel(const RopeParams p) {
    __shared__ float sm_cos[kRopeMaxDim / 2], sm_sin[kRopeMaxDim / 2];
    __shared__ __align__(16) T sm_rows[kStagedBatch * kStagedThreads * kVec];
    const int t = blockIdx.x, tid = threadIdx.y * blockDim.x + threadIdx.x;
    const TokenRows<T> rows_of = {p, t};
    const int D = p.head_dim, R = p.rotary_dim, half = R / 2;
    const int rotated_rows = p.num_q_heads + p.num_kv_heads;
    const int rows = rotated_rows + p.num_kv_heads;
    const int e0 = threadIdx.x * kVec, step = kStagedBatch * (int)blockDim.y;
    wait_for_the_kernel_in_front();
    uint4 a[kStagedBatch];
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < kStagedBatch; ++i) {
            const int r = r0 + threadIdx.y + i * blockDim.y;
            if (r < rows) a[i] = *reinterpret_cast<const uint4*>(rows_of.source(r) + e0);
        }
    };
    load(0);  // (a padding token's rows are there too)
    int pos = 0;
    int64_t slot;
    if (!token_place(p, t, tid == 0, pos, slot)) return;  // uniform over the CTA
    for (int j = tid; j < half; j += blockDim.x * blockDim.y)
        rotation(pos, p.inv_freq[j], p.rope_scale, sm_cos[j], sm_sin[j]);
    __syncthreads();
    // this thread's elements, the same in every row: those before `half` pair
    // with e + half (y0 = x0 c - x1 s), the others with e - half (y1 = x1 c + x0 s)
    const int firsts = half - e0;  // how many are
    float c[kVec], sn[kVec];
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
        const int e = min(e0 + u, R - 1), j = e < half ? e : e - half;
        c[u] = sm_cos[j];
        sn[u] = u < firsts ? -sm_sin[j] : sm_sin[j];
    }
    for (int r0 = 0; r0 < rows; r0 += step) {
        if (r0 > 0) {
            load(r0);
            __syncthreads();  // the last rows have been read
        }
#pragma unroll
        for (int i = 0; i < kStagedBatch; ++i)
            if (r0 + (int)threadIdx.y + i * (int)blockDim.y < rows)
                *reinterpret_cast<uint4*>(sm_rows + (threadIdx.y + i * blockDim.y) * D + e0) = a[i];
        __syncthreads();
#pragma unroll 1
        for (int i = 0; i < kStagedBatch; ++i) {
            const int k = threadIdx.y + i * blockDim.y, r = r0 + k;
            if (r >= rows) break;
            const T* row = sm_rows + k * D;
            Vec<T> x;
            x.w = *reinterpret_cast<const uint4*>(row + e0);
            if (r < rotated_rows && e0 < R) {
#pragma unroll
                for (int u = 0; u < kVec; ++u) {
                    if (e0 + u >= R) continue;
                    const float y = to_f32(row[e0 + u + (u < firsts ? half : -half)]);
                    from_f32(x.e[u], to_f32(x.e[u]) * c[u] + y * sn[u]);
                }
            }
            *reinterpret_cast<uint4*>(rows_of.target(r, slot) + e0) = x.w;
        }
    }
}

pkv_status launch_tokens(void (*kern)(RopeParams), const RopeParams& p, int x, int y,
                         cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.num_tokens);
    cfg.blockDim = dim3((unsigned)x, (unsigned)y);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kern, p));
}

template <typename T, bool kInterleaved>
pkv_status launch_rope(const RopeParams& p, cudaStream_t stream) {
    // units of a head row, and rows of threads
    const int units = (p.head_dim - (kInterleaved ? 0 : p.rotary_dim / 2)) / kVec;
    const int rows = p.num_q_heads + 2 * p.num_kv_heads;
    // CTAs of 128 threads; 64 where a token has little and there are many tokens
    // (16384 tokens of 24 rows of 128: 33.4 us with 64, 35.6 with 128; of 48 rows
    // 61.3 and 60.0; four tokens 3.5 and 2.7)
    const bool little = rows * p.head_dim * 2 < 8192 && p.num_tokens >= 4096;
    const int threads = little ? kRopeThreads / 2 : kRopeThreads;
    const int y = std::max(1, std::min(rows, threads / units));
    return launch_tokens(rope_write_kernel<T, kInterleaved>, p, units, y, stream);
}

template <typename T>
pkv_status dispatch_rope(const RopeParams& p, bool interleaved, cudaStream_t stream) {
    if (interleaved) return launch_rope<T, true>(p, stream);
    if (p.rotary_dim / 2 % kVec == 0) return launch_rope<T, false>(p, stream);
    const int words = p.head_dim / kVec, rows = p.num_q_heads + 2 * p.num_kv_heads;
    const int y = std::max(1, std::min(rows, kStagedThreads / words));
    return launch_tokens(rope_write_staged_kernel<T>, p, words, y, stream);
}

pkv_status rope_impl(RopeParams& p, int layout, pkv_dtype dtype, pkv_stream_t stream) {
    if (p.num_tokens < 0 || p.num_q_heads <= 0 || p.num_kv_heads <= 0 || p.head_dim <= 0 ||
        p.num_blocks <= 0)
        return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (layout != PKV_ROPE_HALF && layout != PKV_ROPE_INTERLEAVED) return PKV_ERR_INVALID_ARG;
    if (p.rotary_dim <= 0 || p.rotary_dim % 2 != 0 || p.rotary_dim > p.head_dim)
        return PKV_ERR_INVALID_ARG;
    if (!std::isfinite(p.rope_scale)) return PKV_ERR_INVALID_ARG;
    if (p.head_dim % 8 != 0 || p.head_dim > kRopeMaxDim) return PKV_ERR_UNSUPPORTED;
    const long long q_row = (long long)p.num_q_heads * p.head_dim;
    const long long kv_row = (long long)p.num_kv_heads * p.head_dim;
    if (q_row + 2 * kv_row > 0x7fffffffll) return PKV_ERR_UNSUPPORTED;
    if (p.q_stride < q_row || p.k_stride < kv_row || p.v_stride < kv_row || p.q_stride % 8 != 0 ||
        p.k_stride % 8 != 0 || p.v_stride % 8 != 0)
        return PKV_ERR_INVALID_ARG;
    if (p.num_tokens == 0) return PKV_OK;
    if (!p.q || !p.k_new || !p.v_new || !p.q_out || !p.k_cache || !p.v_cache || !p.inv_freq)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(p.q) || !aligned16(p.k_new) || !aligned16(p.v_new) || !aligned16(p.q_out) ||
        !aligned16(p.k_cache) || !aligned16(p.v_cache))
        return PKV_ERR_INVALID_ARG;
    // q_out is q itself (each thread reads its elements before it writes them)
    // or shares no byte with q, k_new or v_new
    const auto lo = reinterpret_cast<uintptr_t>(p.q_out);
    const auto hi = lo + (uintptr_t)(p.num_tokens * q_row) * 2;
    auto clash = [&](const void* ptr, long long stride, long long row) {
        const auto b = reinterpret_cast<uintptr_t>(ptr);
        return b < hi && lo < b + (uintptr_t)((p.num_tokens - 1) * stride + row) * 2;
    };
    const bool in_place = p.q == p.q_out && p.q_stride == q_row;
    if ((!in_place && clash(p.q, p.q_stride, q_row)) || clash(p.k_new, p.k_stride, kv_row) ||
        clash(p.v_new, p.v_stride, kv_row))
        return PKV_ERR_INVALID_ARG;
    p.status = status_word();
    if (!p.status) return PKV_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool il = layout == PKV_ROPE_INTERLEAVED;
    return dtype == PKV_BF16 ? dispatch_rope<__nv_bfloat16>(p, il, st)
                             : dispatch_rope<__half>(p, il, st);
}

}  // namespace
}  // namespace pkv

extern "C" {

// Frequencies of the rotary pairs, computed in 64 bits and rounded once.
// NTK and YaRN follow their published formulas (Peng et al., "YaRN: Efficient
// Context Window Extension of Large Language Models", 2023): NTK-aware
// scaling raises the base by factor^(R / (R - 2)); YaRN divides the pairs that
// turn less than beta_slow times over the original length by the factor,
// leaves those that turn more than beta_fast times, and blends between.
pkv_status paged_kv_rope_frequencies(int rotary_dim, double base, pkv_rope_scaling scaling,
                                     double factor, int original_max_position, double beta_fast,
                                     double beta_slow, float* inv_freq, float* rope_scale) {
    if (rotary_dim <= 0 || rotary_dim % 2 != 0 || !std::isfinite(base) || base <= 1.0 ||
        !inv_freq || !rope_scale)
        return PKV_ERR_INVALID_ARG;
    if (scaling != PKV_ROPE_SCALE_NONE && scaling != PKV_ROPE_SCALE_LINEAR &&
        scaling != PKV_ROPE_SCALE_NTK && scaling != PKV_ROPE_SCALE_YARN)
        return PKV_ERR_INVALID_ARG;
    if (scaling != PKV_ROPE_SCALE_NONE && (!std::isfinite(factor) || factor < 1.0))
        return PKV_ERR_INVALID_ARG;
    const int half = rotary_dim / 2;
    const double R = rotary_dim;
    double b = base, low = 0.0, high = 0.0;
    *rope_scale = 1.0f;
    if (scaling == PKV_ROPE_SCALE_NTK && rotary_dim > 2) b = base * std::pow(factor, R / (R - 2.0));
    if (scaling == PKV_ROPE_SCALE_YARN) {
        if (original_max_position <= 0 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) ||
            !std::isfinite(beta_fast))
            return PKV_ERR_INVALID_ARG;
        // the pair index whose frequency turns `beta` times over the original length
        const double kTwoPi = 6.283185307179586476925;
        auto pair_of = [&](double beta) {
            return R * std::log(original_max_position / (beta * kTwoPi)) / (2.0 * std::log(base));
        };
        low = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
        high = std::fmin(std::ceil(pair_of(beta_slow)), R - 1.0);
        *rope_scale = (float)(0.1 * std::log(factor) + 1.0);
    }
    for (int j = 0; j < half; ++j) {
        double f = std::pow(b, -2.0 * j / R);
        if (scaling == PKV_ROPE_SCALE_LINEAR) f /= factor;
        if (scaling == PKV_ROPE_SCALE_YARN) {
            const double ramp =
                std::fmin(std::fmax((j - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        inv_freq[j] = (float)f;
    }
    return PKV_OK;
}

pkv_status paged_kv_rope_write(const void* q, const void* k_new, const void* v_new,
                               long long q_stride, long long k_stride, long long v_stride,
                               const int32_t* positions, const int64_t* slot_mapping,
                               const float* inv_freq, float rope_scale, int num_tokens,
                               int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
                               pkv_rope_layout layout, int num_blocks, void* q_out, void* k_cache,
                               void* v_cache, pkv_dtype dtype, pkv_stream_t stream) {
    if (num_tokens > 0 && (!positions || !slot_mapping)) return PKV_ERR_INVALID_ARG;
    pkv::RopeParams p = {};
    p.q = q;
    p.k_new = k_new;
    p.v_new = v_new;
    p.q_out = q_out;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.inv_freq = inv_freq;
    p.rope_scale = rope_scale;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rotary_dim = rotary_dim;
    p.num_blocks = num_blocks;
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    return pkv::rope_impl(p, layout, dtype, stream);
}

pkv_status paged_kv_rope_write_new_tokens(
    const void* q, const void* k_new, const void* v_new, long long q_stride, long long k_stride,
    long long v_stride, const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, const float* inv_freq, float rope_scale, int num_seqs,
    int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim, pkv_rope_layout layout,
    int num_blocks, void* q_out, void* k_cache, void* v_cache, int64_t* slot_mapping_out,
    pkv_dtype dtype, pkv_stream_t stream) {
    if (max_blocks_per_seq <= 0) return PKV_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!block_tables || !context_lens)) return PKV_ERR_INVALID_ARG;
    pkv::RopeParams p = {};
    p.q = q;
    p.k_new = k_new;
    p.v_new = v_new;
    p.q_out = q_out;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.inv_freq = inv_freq;
    p.rope_scale = rope_scale;
    p.num_tokens = num_seqs;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rotary_dim = rotary_dim;
    p.num_blocks = num_blocks;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.slot_out = slot_mapping_out;
    return pkv::rope_impl(p, layout, dtype, stream);
}

}  // extern "C"
