// Rows of a batch by adapter, or pairs of token and expert by expert: the tables
// that lora.hip makes and the kernels go by.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

namespace {

constexpr int TILE_T = 32;           // rows of a tile of the plan
constexpr int CHUNK = 512;           // rows of a chunk of the weight gradient

// ---------------------------------------------------------------------------
// the plan: rows sorted by adapter (stable), tiles and chunks of equal adapter
// ---------------------------------------------------------------------------
// int32 words: [0] tiles, [1] chunks, [2] M, [3] L, then
//   first [L+1]  first tile of each adapter (entry L: of the rows without one)
//   count [L+1]  its rows
//   slot  [L+1]  its first partial-sum slot (adapters of one chunk or none have
//                no slot)
//   chunk [CB][4]  adapter, first place, rows, slot (-1: the only chunk)
//   tile  [TB][2]  adapter (-1: none), rows
//   rows  [TB][TILE_T]  the rows of each tile; places behind the last repeat it
// A place is TILE_T * tile + position: the rows of one adapter stand together, and
// a kernel that knows its tile's number knows where they are.
struct PlanLayout {
    int64_t first, count, slot, chunk, tile, rows, words;
    int64_t TB, CB;

    __host__ __device__ PlanLayout(int64_t M, int64_t L)
    {
        const int64_t segs = M < L + 1 ? M : L + 1;
        TB = M / TILE_T + segs;
        CB = M / CHUNK + segs;
        first = 4;
        count = first + L + 1;
        slot = count + L + 1;
        chunk = (slot + L + 1 + 3) / 4 * 4;
        tile = chunk + 4 * CB;
        rows = tile + (2 * TB + 3) / 4 * 4;
        words = rows + TILE_T * TB;
    }
};

}  // namespace
