// split.h -- where the parts of a range of units begin (plain C++: the kernels and
// the host take the same).
#pragma once

namespace moe {

// First unit of part `part` of `parts` (part == parts: the end), floor(part * units /
// parts). As the whole quotient and the rest's share, so that nothing passes 31 bits
// where units and parts^2 do not: 524287 units of a shared expert in 16384 parts make
// a product of 2^33.
constexpr int part_begin(int part, int units, int parts)
{
    return part * (units / parts) + part * (units % parts) / parts;
}

}  // namespace moe
