// drain.cuh -- the drain of a CTA's own TMA loads when its producer has ended (pairdrain.cuh: of a pair's).
//
// A producer calls it after its loop however the loop ended. One that stopped early has loads in flight;
// so has one whose loads all fit the ring and that has issued them by the time a consumer gives up. In
// either case the CTA must not leave while the copy engine still writes its shared memory, which the next
// CTA on the SM owns. In a run that does not stop, the MMAs wait for the same phases: it adds no wait. Its
// loop stays rolled, so that it adds little code either (MXFP4 forward of one token, 4096 -> 14336, with its
// quantiser: 17.2 us as without it, 17.45 unrolled).
#pragma once

#include <stdint.h>

#include "ptx.cuh"

namespace rdot {

// Waits, within drain_guard's limit, until the last load into each stage has landed (bit s of `issued`: one was
// issued to stage s; bit s of `phases`: the parity of its phase).
template <int STAGES>
__device__ __forceinline__ void drain_loads(uint64_t* full, uint32_t issued, uint32_t phases, const WaitGuard& g) {
    static_assert(STAGES <= 32, "a bit per stage");
    int dummy;
    const WaitGuard dguard = drain_guard(g, &dummy);
#pragma unroll 1
    for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s)) (void)mbar_wait(&full[s], (phases >> s) & 1u, dguard);
}

}  // namespace rdot
