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

// First visible key of the query at position p (may lie past p: nothing visible).
__device__ __forceinline__ int first_key(const ScoreMods& m, int s, int p) {
    int lo = m.key_starts ? max(m.key_starts[s], 0) : 0;
    if (m.window > 0) lo = max(lo, p - m.window + 1);
    return lo;
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
