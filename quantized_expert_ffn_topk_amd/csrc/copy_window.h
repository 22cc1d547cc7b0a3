// copy_window.h -- how much of a tile's rows a copy by the load unit may read: a plain
// function of sizes, for the kernels and for tests on the host.
#pragma once

#include <cstdint>

namespace moe {

// The memory of a copy that takes bytes [at, ...) of each row, of rows that are `row` bytes
// long and end `end` >= row bytes past the first one's beginning: it begins at `at`
// itself and has this many bytes, none where it begins past a row's end, so that a lane's
// offset alone says whether it is inside.  (The stage as a scalar offset would rest on how
// the unit's check takes that into account, and on a difference that must not wrap where
// nothing is left.)
constexpr uint32_t window_bytes(uint32_t end, int at, int row)
{
    return at < row ? end - (uint32_t)at : 0u;
}

}  // namespace moe
