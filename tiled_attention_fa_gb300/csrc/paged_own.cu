// The paged decode kernel over the sequences' own keys behind a shared prefix
// (its O in fp32, a.O): a unit of its own so that it compiles beside paged.cu.
#include "paged_launch.cuh"

namespace fa {

fa_status run_paged_own(const PagedDecodeArgs& a, cudaStream_t s) {
  PagedParams p;
  int G = 0;
  const fa_status st = paged_setup(a, p, G);
  return st == FA_OK ? launch_paged<true>(a, p, G, s) : st;
}

unsigned int paged_own_read_error(cudaStream_t s) { return read_and_clear_error(s); }

}  // namespace fa
