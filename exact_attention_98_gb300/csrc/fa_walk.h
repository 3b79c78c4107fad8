// How warps that meet at a named barrier walk a CTA's items, and how they leave the
// walk.
//
// A named barrier waits without limit for its count of threads.  Every other wait is
// bounded and decided by each warp alone: where the CTA gives up, one warp may
// see a wait fail that its neighbours still see succeed, so a warp that left on its own
// would keep them at the barrier for ever.  (Nor can it arrive there for all the times to
// come before it leaves: arrivals that no one waits for yet complete a round by
// themselves.)  So a warp that has given up goes on to the barrier that its
// neighbours come to next, and says so there: all of them leave behind it, or none.
//
// Plain C++ on the host, where the walk is checked with every warp giving up at every
// place.
#pragma once

#if defined(__CUDACC__)
#define FA_WALK_HD __device__ __forceinline__
#else
#define FA_WALK_HD inline
#endif

namespace fa {

// What a look for the next item gives.  The end is the same place for every warp,
// kGaveUp the warp's own.
enum class Next { kItem, kEnd, kGaveUp };

// Items of one tile at least, with a meeting for each tile and one at the end.
//   look()    the next item
//   take()    the present tile as far as the meeting; false: gave up
//   meet(ok)  the AND over the warps
//   give()    the rest of the tile
//   step()    on to the item's next tile; false: it was the last
template <class Look, class Take, class Meet, class Give, class Step>
FA_WALK_HD void walk_tiles(Look&& look, Take&& take, Meet&& meet, Give&& give, Step&& step) {
  for (;;) {
    const Next next = look();
    if (next != Next::kItem) {
      // the neighbours are at their end, or at this item's first tile
      meet(next == Next::kEnd);
      return;
    }
    do {
      if (!meet(take())) return;
      give();
    } while (step());
  }
}

}  // namespace fa
