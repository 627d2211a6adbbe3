// Rows that are not whole, aligned 16-byte pieces, copied to shared memory all the same in such
// pieces: those that a part of a row touches, with what lies before and behind it in them. Nothing
// outside the tensor is read: a piece that ends behind it is copied as far as it goes, the one
// that begins before it element by element.
#pragma once

#include "mixer.cuh"

namespace gdn {

// The bytes of a strided tensor, from its first element to behind its last.
struct RowSpan {
    uintptr_t lo, hi;
};
inline RowSpan row_span(const void *p, int B, int T, int64_t row, int64_t sb, int64_t st, size_t e) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + strided_bytes(B, T, row, sb, st, e)};
}

// Copies of `width` values of each of some rows.
template <typename E>
struct RowCopy {
    RowSpan span;
    bool inside;       // no row's pieces reach out of the tensor

    RowCopy() = default;
    // of `rows` (or none) rows, the first at `from`; strides are not negative
    __device__ __forceinline__ RowCopy(const RowSpan &span, const E *from, int64_t stride, int rows, int width)
        : span(span) {
        const uintptr_t first = reinterpret_cast<uintptr_t>(from);
        const uintptr_t last = reinterpret_cast<uintptr_t>(from + (rows - 1) * stride + width);
        inside = rows > 0 && (first & ~static_cast<uintptr_t>(15)) >= span.lo && last + 15 <= span.hi;
    }
    // The row at `from` to `to` (16-byte aligned): the i-th of its pieces, where it has as many.
    // Asynchronously, but for the tensor's first piece.
    __device__ __forceinline__ void operator()(void *to, const E *from, int width, int i) const {
        const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(from)) & 15, o = 16 * i;
        if (o >= shift + width * static_cast<int>(sizeof(E))) return;
        const unsigned char *a = reinterpret_cast<const unsigned char *>(from) + (o - shift);
        if (inside)
            copy16_async(static_cast<unsigned char *>(to) + o, a);
        else
            at_the_ends(static_cast<unsigned char *>(to) + o, reinterpret_cast<uintptr_t>(a));
    }
    __device__ __noinline__ void at_the_ends(unsigned char *to, uintptr_t a) const {
        if (a < span.lo) {                             // of the first piece what belongs to the tensor
            for (uintptr_t e = span.lo; e < a + 16 && e < span.hi; e += sizeof(E))
                *reinterpret_cast<E *>(to + (e - a)) = *reinterpret_cast<const E *>(e);
        } else {
            const int there = static_cast<int>(min(static_cast<unsigned long long>(span.hi - a), 16ull));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(a), "r"(there) : "memory");
        }
    }
};

// Where the values copied from `from` on lie in the copy.
template <typename E>
__device__ __forceinline__ const E *row_in_copy(const void *copy, const E *from) {
    return reinterpret_cast<const E *>(static_cast<const unsigned char *>(copy) +
                                       (reinterpret_cast<uintptr_t>(from) & 15));
}

}  // namespace gdn
