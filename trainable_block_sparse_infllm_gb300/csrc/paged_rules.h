// Rules of paged_attn.cu that hold when one of its waits gives up.  For the host
// as well: their tests need no GPU.
#pragma once

#ifdef __CUDACC__
#define INFLLMV2_HD __host__ __device__ __forceinline__
#else
#define INFLLMV2_HD inline
#endif

namespace infllmv2 {

// The record of a unit that the borders of chunks cut, as the join reads it:
// whether (unit, chunk of the second piece, last chunk, first piece's place) is
// a record that the pass can have written for `units` units and at most `most`
// chunks: the pieces lie at places 2 (second - 1) or the one behind it, 2 second,
// 2 (second + 1), ..., 2 last, all below 2 most.  A pass that gave up a wait
// leaves records unwritten, and the workspace there holds anything; the join
// follows none that leads outside the workspace or the outputs.
INFLLMV2_HD bool cut_in_range(int unit, int second, int last, int place, int units, int most) {
  return unit >= 0 && unit < units && second >= 1 && second <= last && last < most && place >= 0 &&
         place / 2 == second - 1;
}

// The oldest of `issued` copies through a ring of `stages` that may still be in
// flight.  `freed`: the next stage's copy has been consumed, so it has landed.
INFLLMV2_HD unsigned first_in_flight(unsigned issued, unsigned stages, bool freed) {
  const unsigned most = stages - (freed ? 1 : 0);
  return issued > most ? issued - most : 0;
}

}  // namespace infllmv2
