// The step of the 64-way search that finds a packed row's request, for kernels
// and for CPU tests of its indexes.
#pragma once

namespace dspark {

// How far a search goes on in a range whose entries at 0, step, 2 step, ... are at
// or before the row where `found` has a bit. In ascending words the first is;
// others may have none that is, and then the search stays where it is: a count of
// none less one, taken as unsigned, led far beyond the words.
__host__ __device__ inline int search_skip(unsigned long long found, int step) {
  const int n = __builtin_popcountll(found);
  return n > 1 ? (n - 1) * step : 0;
}

}  // namespace dspark
