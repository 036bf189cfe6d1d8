// ring.h — the ring of stages of a kernel that loads ahead, as arithmetic (host and device).
#pragma once

#ifdef __CUDACC__
#define SSD_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SSD_HOST_DEVICE inline
#endif

namespace ssd {

// Stage `stage` of a ring of `stages` holds the slices stage, stage + stages, ...: its use u is
// slice stage + u * stages, and completes the phase of parity u & 1 of the stage's barrier.
// The last use among the first `loaded` slices, -1 if it has none.
SSD_HOST_DEVICE long long ring_last_use(long long loaded, int stage, int stages) {
    return loaded > stage ? (loaded - 1 - stage) / stages : -1;
}

}  // namespace ssd
