// The copies of a CTA pair into its ring, each counted on the first CTA's barrier
// of its stage (lm_score.cuh), and what is left to wait for at the end. Host code
// too, so that the counting can be run against every order of events.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FGM_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define FGM_HOST_DEVICE inline
#endif

namespace fgm {
namespace score {

// The first CTA arrives on a stage's barrier for both CTAs' bytes as it issues its
// own copy. Usually both issue the same copies. When waits run out the CTAs stop
// each for itself, and one may have issued up to a ring more than the other (its
// n-th copy needs the products of the n - stages-th, and those both CTAs' copies).
// So at the end the first CTA
//   takes the other's bytes out of copies [only_from, to) if it issued these alone,
//   or arrives for the other's bytes if the other did;
//   waits for the phases of copies [first, to).
// Earlier copies have landed: their stages were filled again after their products.
struct PairEnd {
    uint32_t first, only_from, to;
};

FGM_HOST_DEVICE PairEnd pair_end(uint32_t issued_here, uint32_t issued_there, uint32_t stages)
{
    PairEnd e;
    e.only_from = issued_here < issued_there ? issued_here : issued_there;
    e.to = issued_here < issued_there ? issued_there : issued_here;
    e.first = e.to > stages ? e.to - stages : 0;
    return e;
}

}  // namespace score
}  // namespace fgm
