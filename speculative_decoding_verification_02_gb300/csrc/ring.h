// Index arithmetic of the cache kernels in plain C++, so that it is tested on
// the host: the phases of a ring of barriers, walks over positions.
#pragma once

#ifdef __CUDACC__
#define SV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SV_HOST_DEVICE inline
#endif

namespace sv {

// Waits until every phase that was begun has completed: `begun` of them, the
// stages in turn.  done(stage, parity) is a barrier's test, which holds for the
// parity of the phase that completed last -- so for one of the two at any time,
// and only the begun phase's own parity says anything.  At most `tries` tests
// to a stage; the answer says whether all had completed.
template <class Done>
SV_HOST_DEVICE bool ring_landed(int stages, int begun, int tries, Done &&done) {
  bool all = true;
  for (int s = 0; s < stages; ++s) {
    const int phases = begun / stages + (s < begun % stages ? 1 : 0);
    bool landed = phases == 0;
    for (int k = 0; k < tries && !landed; ++k) landed = done(s, (phases - 1) & 1);
    all = all && landed;
  }
  return all;
}

// Where a walk over [at, to) that takes `step` positions at a time goes next:
// positions go up to 2^31 - 257, from where a step would pass an int.
SV_HOST_DEVICE int next_span(int at, int to, int step) { return to - at > step ? at + step : to; }

}  // namespace sv
