// pkv_packed.cpp -- entries whose arguments come as one array of 8-byte slots.
//
// A foreign-function call converts its arguments one by one (Python's ctypes at
// about 0.1 us each: 2.6 us for an attention call with modified scores, where one
// array takes 0.6), which the smallest calls feel.  Slot k is argument k of the
// entry: a pointer, an int64 for every integer and enum, a double for a float.
// The slots need no alignment.  An integer that its parameter does not hold is
// PKV_ERR_INVALID_ARG.
#include <cstdint>
#include <cstring>
#include <limits>
#include <tuple>
#include <type_traits>

#include "pagedkv.h"

namespace {

template <typename T>
T take(const unsigned char*& at, bool& fits) {
    if constexpr (std::is_pointer<T>::value) {
        T v;
        static_assert(sizeof(T) == 8, "a slot");
        std::memcpy(&v, at, 8);
        at += 8;
        return v;
    } else if constexpr (std::is_floating_point<T>::value) {
        double v;
        std::memcpy(&v, at, 8);
        at += 8;
        return static_cast<T>(v);
    } else {
        int64_t v;
        std::memcpy(&v, at, 8);
        at += 8;
        if (std::is_unsigned<T>::value && sizeof(T) == 8)
            fits = fits && v >= 0;
        else if (sizeof(T) == 4)  // int and the enums
            fits = fits && v >= std::numeric_limits<int32_t>::min() &&
                   v <= std::numeric_limits<int32_t>::max();
        return static_cast<T>(fits ? v : 0);
    }
}

template <typename... A>
pkv_status forward(pkv_status (*entry)(A...), const void* slots) {
    if (!slots) return PKV_ERR_INVALID_ARG;
    const unsigned char* at = static_cast<const unsigned char*>(slots);
    bool fits = true;
    const std::tuple<A...> args{take<A>(at, fits)...};  // (braces: in order)
    return fits ? std::apply(entry, args) : PKV_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

pkv_status paged_kv_rope_write_packed(const void* slots) {
    return forward(paged_kv_rope_write, slots);
}

pkv_status paged_kv_rope_write_new_tokens_packed(const void* slots) {
    return forward(paged_kv_rope_write_new_tokens, slots);
}

pkv_status paged_attention_decode_scored_packed(const void* slots) {
    return forward(paged_attention_decode_scored, slots);
}

pkv_status paged_attention_prefill_scored_packed(const void* slots) {
    return forward(paged_attention_prefill_scored, slots);
}

}  // extern "C"
