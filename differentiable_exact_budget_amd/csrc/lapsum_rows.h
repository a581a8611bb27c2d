// 16 bytes of a row at a time, at any element's address (gfx950): the hardware
// takes such loads and stores, and only a row's last elements go one by one.
#pragma once
#include "lapsum_expert_ops.h"

namespace lapsum {

// 16 bytes of a row at any element's address
template <class T>
struct Pack {
    static constexpr int V = 16 / (int)sizeof(T);
    T v[V];
};
template <class T>
struct __attribute__((packed, aligned(sizeof(T)))) Loose {
    Pack<T> p;
};
// Elements c .. of a row of D elements; past the row's end: zeros.  ONCE:
// rows that no later part of the pass reads go past the caches (rows gathered
// from 255 MB, 16384 tokens x 4 x 2048 bf16: combine 99 -> 70 us, its VJP
// 129 -> 94 us; dispatch, whose x fits them, is 2 us slower that way).
template <bool ONCE, class T>
LS_DEV Pack<T> ld(const T* row, long long c, long long D) {
    constexpr int V = Pack<T>::V;
    typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));  // at any element
    Pack<T> x{};
    if (c + V <= D) {
        if (ONCE)
            x = __builtin_bit_cast(Pack<T>, __builtin_nontemporal_load(reinterpret_cast<const Words*>(row + c)));
        else
            x = reinterpret_cast<const Loose<T>*>(row + c)->p;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i < D) x.v[i] = row[c + i];
    }
    return x;
}
template <class T>
LS_DEV void st(T* row, long long c, long long D, const Pack<T>& x) {
    constexpr int V = Pack<T>::V;
    if (c + V <= D) {
        reinterpret_cast<Loose<T>*>(row + c)->p = x;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i < D) row[c + i] = x.v[i];
    }
}

}  // namespace lapsum
