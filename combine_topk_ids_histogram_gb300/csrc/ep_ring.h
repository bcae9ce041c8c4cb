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

// Sums over many stages leave the tensor cores after every chunk of them, from one of two buffers.
constexpr int kChunkStages = 8;
EP_HOST_DEVICE constexpr int stage_chunk(int stage) { return stage / kChunkStages; }
EP_HOST_DEVICE constexpr bool chunk_begins(int stage) { return stage % kChunkStages == 0; }
EP_HOST_DEVICE constexpr int chunk_buffer(int chunk) { return chunk & 1; }
EP_HOST_DEVICE constexpr int chunk_phase(int chunk) { return chunk >> 1; }

}  // namespace ep
