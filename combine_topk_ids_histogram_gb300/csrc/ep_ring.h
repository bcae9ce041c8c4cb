// ep_ring.h -- where the stages of a ring in shared memory are, and the phases of their barriers.  Plain C++: a host program can
// go through every order in which warps pass them.
#pragma once

#ifdef __CUDACC__
#define EP_HOST_DEVICE __host__ __device__
#else
#define EP_HOST_DEVICE
#endif

namespace ep {

constexpr int kRing = 3;                     // stages that fit

// Every barrier of a stage (copied, products done, results read) is its slot's.  A wait sees the parity of a phase only, so that a barrier
// must not end two phases before everyone who waits for the first has looked: in a slot the next stage is copied behind those waits.
EP_HOST_DEVICE constexpr int ring_slot(int stage) { return stage % kRing; }

// Phases that such a barrier has ended before that of `stage`, where `before` stages of an earlier pass went through the ring.
EP_HOST_DEVICE constexpr int ring_phase(int stage, int before = 0) { return (before - stage % kRing + kRing - 1) / kRing + stage / kRing; }

}  // namespace ep
