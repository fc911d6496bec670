// How the warps of a group leave a loop together once one of them gave up.
//
// The group has one barrier a tile.  A warp that gave up raises the tile's flag
// before that barrier, and every warp reads the flag after it.  The flags go by
// the tile's parity: a warp that is through with tile j may raise the flag of
// tile j + 1 while a slower one still reads that of tile j, but nobody writes
// tile j's flag again (for tile j + 2) before barrier j + 1, which the slower
// warp reaches only with its reading done.  With one flag for all tiles the
// slower warp would leave a tile early, and the others wait at a barrier that
// it never reaches.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SA_HOST_DEVICE inline
#endif

namespace sa_dev {

struct GiveUp {
  volatile int flag[2];
  SA_HOST_DEVICE void clear() { flag[0] = flag[1] = 0; }
  SA_HOST_DEVICE void raise(uint32_t tile) { flag[tile & 1] = 1; }
  SA_HOST_DEVICE bool raised(uint32_t tile) const { return flag[tile & 1] != 0; }
};

}  // namespace sa_dev
