// The element type of 4-bit pools by its name, for a torch that may not have it (before 2.8).
#pragma once
#include <type_traits>

template <typename Scalar, typename = void>
struct FourBits {
    static constexpr bool is(Scalar) { return false; }
};
template <typename Scalar>
struct FourBits<Scalar, std::void_t<decltype(Scalar::Float4_e2m1fn_x2)>> {
    static constexpr bool is(Scalar t) { return t == Scalar::Float4_e2m1fn_x2; }
};
