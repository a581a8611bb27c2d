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
// The same in two steps, for loads that are to stay in flight: at a row's end
// take() brings the row's last 16 bytes, and settle() shifts them down (D as
// above, and the elements past it zero).  A row's last elements loaded one by
// one, or shifted at once, make every load wait for those before it: layer norm's
// gradients of 32768 rows of 300 in bf16 43 and 33 us, 25 so.
template <bool ONCE, class T>
LS_DEV Pack<T> take(const T* row, long long c, long long D) {
    constexpr int V = Pack<T>::V;
    typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
    if (D < V) return ld<ONCE>(row, c, D);
    const T* p = row + min(c, D - V);
    if (ONCE) return __builtin_bit_cast(Pack<T>, __builtin_nontemporal_load(reinterpret_cast<const Words*>(p)));
    return reinterpret_cast<const Loose<T>*>(p)->p;
}
template <class T>
LS_DEV Pack<T> settle(const Pack<T>& x, long long c, long long D) {
    constexpr int V = Pack<T>::V;
    if (D < V || c + V <= D) return x;
    struct { uint64_t lo, hi; } w = __builtin_bit_cast(decltype(w), x);
    const int by = (int)min(c - (D - V), (long long)V) * 8 * (int)sizeof(T);  // 16 .. 128
    w.lo = by >= 128 ? 0 : by >= 64 ? w.hi >> (by - 64) : w.lo >> by | w.hi << (64 - by);
    w.hi = by >= 64 ? 0 : w.hi >> by;
    return __builtin_bit_cast(Pack<T>, w);
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
