// copy_window.h -- how much of a tile's rows a copy by the load unit may read: a plain
// function of sizes, for the kernels and for tests on the host.
#pragma once

#include <cstdint>

namespace moe {

// The size of the buffer, which begins where the rows do, of a copy that takes bytes
// [at, ...) of each row, of rows that are `row` bytes long and end `end` >= row bytes past the first
// one's beginning: none where the copy begins past a row's end.  Row and `at` make up a lane's offset
// and the scalar offset is 0, so that the lane's offset alone says whether it is inside.
// (`at` as a scalar offset would rest on how the unit's check takes that into account,
// and on a difference that must not wrap where nothing is left.)
constexpr uint32_t window_bytes(uint32_t end, int at, int row)
{
    return at < row ? end : 0u;
}

}  // namespace moe
