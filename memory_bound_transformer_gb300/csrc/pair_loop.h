// Tiles of two warps that share rows and exchange a value once per tile, where
// every other wait of theirs is bounded and may run out in one of them alone.
//
// The exchange is a barrier without a limit. So a warp whose wait has run out
// still comes to the next one, says so there, and both leave behind it: neither
// can be left waiting for the other. Host code, too, so that every order of
// failures can be tried on the CPU.
#pragma once

#ifdef __CUDACC__
#define MBT_PAIR_FN __host__ __device__ __forceinline__
#else
#define MBT_PAIR_FN inline
#endif

namespace mbt {

// Per tile j: before(j, ok) up to the exchange, meet(j, ok) the exchange (whether
// both are all right), after(j) the rest; before and after return false once a
// wait has run out. Loops that follow one another pass `ok` on.
template <class Before, class Meet, class After>
MBT_PAIR_FN bool pair_tiles(int from, int to, bool ok, Before before, Meet meet, After after) {
#pragma unroll 1
  for (int j = from; j < to; ++j) {
    ok = before(j, ok);
    ok = meet(j, ok);
    if (!ok) break;                                                  // both warps of the pair
    ok = after(j);
  }
  return ok;
}

}  // namespace mbt
