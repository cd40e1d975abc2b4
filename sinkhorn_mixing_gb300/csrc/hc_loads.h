// hc_loads.h -- the loads of a ring of stages that may still be in flight (host and device).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define HC_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define HC_HOST_DEVICE inline
#endif

namespace hc {

// Load i goes into stage i % STAGES and ends phase i / STAGES of that stage's barrier.  It is
// issued only once load i - STAGES has landed, so of the loads that were issued, the last STAGES
// at most are in flight, and of a stage none but the last: the parity that a wait names is that
// of the phase it means.  Counted are loads, not steps: where a wait gave up, the steps go on
// without loads.
template <int STAGES>
struct RingLoads {
    int64_t issued = 0;
    HC_HOST_DEVICE void issue() { ++issued; }
    // f(stage, parity) for each load that may be in flight
    template <typename F>
    HC_HOST_DEVICE void in_flight(F f) const {
        for (int64_t i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
            f((int)(i % STAGES), (uint32_t)(i / STAGES) & 1);
    }
};

}  // namespace hc
