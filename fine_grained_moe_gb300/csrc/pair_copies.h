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

// The same where several warps of each CTA bring parts of a stage (grouped.cuh: one
// weights, others rows), each at its own pace: a warp's copies for stage n need the
// products of stage n - stages, and those all warps' copies for it, so that no copy
// is a ring ahead of what is to come. The first CTA arrives for all bytes of a stage
// with its weights. Weights are the same bytes in every stage, rows in those of a tile,
// of which each warp notes the first stage and its bytes a stage (tiles where it has
// none, none), and at the end how far it got. When waits ran out, the first CTA goes
// through the notes: for the stages [first(), to) that are left to wait for, and in
// each for the bytes that were sent, of which it takes the others out, or arrives for
// these alone. The stages of a ring belong to at most as many tiles.
struct TileNote {
    uint32_t first, bytes;   // first ~0: none yet
};

struct StagesLeft {
    uint32_t to = 0;

    FGM_HOST_DEVICE void warp(uint32_t issued) { to = issued > to ? issued : to; }
    FGM_HOST_DEVICE uint32_t first(uint32_t stages) const { return to > stages ? to - stages : 0; }
};

// Bytes that a warp sent for stage n, if this tile's: of `steps` stages, of all of which it got to `issued`.
FGM_HOST_DEVICE uint32_t sent_bytes(const TileNote &note, uint32_t steps, uint32_t issued, uint32_t n)
{
    return n >= note.first && n - note.first < steps && n < issued ? note.bytes : 0;
}

}  // namespace score
}  // namespace fgm
