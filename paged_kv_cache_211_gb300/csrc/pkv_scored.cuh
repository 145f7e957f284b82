// pkv_scored.cuh -- what the decode and prefill attention with modified
// scores share: the score of a (query, key) pair in base 2 and the visible
// keys of a query.
//
//     z = scale <q, k_t>;  z = cap tanh(z / cap) if cap > 0;  z -= slope |p - t|
//     visible: max(0, key_start, p - window + 1) <= t < max(p + 1, min(prefix, n))
#pragma once

#include <algorithm>
#include <cmath>

#include "pkv_internal.cuh"

namespace pkv {

struct ScoreMods {
    float scale_log2;   // scale log2(e): scores live in base 2
    float cap_in;       // scale / cap
    float cap_out;      // cap log2(e); 0: no cap
    const float* slopes;            // [num_q_heads] or null
    const int32_t* key_starts;      // [num_seqs] or null
    const int32_t* prefix_lens;     // [num_seqs] or null (prefill only)
    int window;                     // 0: none
};

constexpr float kScoreLog2e = 1.4426950408889634f;

// tanh(x) / x as polynomials in x^2, fitted here by iterated weighted least
// squares to the smallest largest relative error: eight terms for |x| <= 1.25
// (8e-8, 2e-7 with their roundings), four for |x| <= 0.5 (5.5e-7) and three for
// |x| <= 0.25 (4.0e-7).
constexpr int kTanhWide = 8, kTanhTerms = 4, kTanhFew = 3;
constexpr float kTanhWideRange = 1.25f, kTanhRange = 0.5f, kTanhFewRange = 0.25f;
constexpr float kTanh8[kTanhWide] = {0.99999994f,   -0.333326995f,  0.133245066f,  -0.0534903146f,
                                     0.0205571186f, -0.00679610018f, 0.00158808648f,
                                     -0.000182592616f};
constexpr float kTanh4[kTanhTerms] = {0.999999456f, -0.333263179f, 0.131902966f, -0.0444022261f};
constexpr float kTanh3[kTanhFew] = {0.999999604f, -0.333219082f, 0.128416134f};

__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// The capped base-2 score of a raw one: cap' tanh(x), x = raw cap_in.  Away from
// zero 1 - 2 / (1 + e^2x) from exp2 and a reciprocal (errors of 2^-22 of 1); near
// it that would cancel, and the polynomial keeps the relative error.
__device__ __forceinline__ float cap_score(float raw, const ScoreMods& m) {
    const float x = raw * m.cap_in, v = x * x;
    const float far = fmaf(-2.f, fast_rcp(1.f + fast_exp2(2.f * kScoreLog2e * x)), 1.f);
    const float near = x * fmaf(fmaf(kTanh3[2], v, kTanh3[1]), v, kTanh3[0]);
    return m.cap_out * (fabsf(x) > kTanhFewRange ? far : near);
}

// First visible key of the query at position p (may lie past p: nothing visible).
__device__ __forceinline__ int first_key(const ScoreMods& m, int s, int p) {
    int lo = m.key_starts ? max(m.key_starts[s], 0) : 0;
    if (m.window > 0) lo = max(lo, p - m.window + 1);
    return lo;
}

// Whether two buffers of `bytes` bytes share any.
inline bool overlap(const void* a, const void* b, size_t bytes) {
    const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bytes && y < x + bytes;
}

// Host checks shared by the entries.  false: invalid argument.
inline bool make_score_mods(ScoreMods* m, float scale, float softcap, const float* alibi_slopes,
                            int window, const int32_t* key_starts, const int32_t* prefix_lens) {
    if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0)
        return false;
    m->scale_log2 = scale * kScoreLog2e;
    m->cap_in = softcap > 0.f ? scale / softcap : 0.f;
    m->cap_out = softcap > 0.f ? softcap * kScoreLog2e : 0.f;
    m->slopes = alibi_slopes;
    m->key_starts = key_starts;
    m->prefix_lens = prefix_lens;
    m->window = window;
    return std::isfinite(m->cap_in) && std::isfinite(m->cap_out) && std::isfinite(m->scale_log2);
}

}  // namespace pkv
