// Work units handed from a kernel's producer to its other warps through
// shared memory, with what the producer looked up for them, so that none of
// the others waits for global memory between units.
#pragma once

#include <stdint.h>

#include "ptx.cuh"

namespace attn {
namespace scored {

// A ring of N units (U: plain data, bh < 0 for the end of the launch's
// units). Slot u % N holds the CTA's u-th unit. Every reader reads every unit
// in order and arrives once on its slot.
template <typename U>
struct UnitRing {
  static constexpr int N = 4;
  static constexpr int BYTES = N * sizeof(U);
  U* slots;
  uint64_t* full;    // [N] arrived at by the producer
  uint64_t* empty;   // [N] arrived at once by each reader

  __device__ __forceinline__ void init(int readers) const {
    for (int s = 0; s < N; ++s) {
      ptx::mbar_init(full + s, 1);
      ptx::mbar_init(empty + s, readers);
    }
  }
  // false on a timeout, as everywhere
  __device__ __forceinline__ bool push(uint32_t u, const U& v, const ptx::WaitCtx& w) const {
    const int s = static_cast<int>(u % N);
    if (!ptx::mbar_wait(empty + s, ((u / N) & 1u) ^ 1u, w)) return false;
    slots[s] = v;
    ptx::mbar_arrive(full + s);   // (release: whoever acquires this phase sees the unit)
    return true;
  }
  // by every thread of a warp; the caller then arrives on empty[u % N]
  __device__ __forceinline__ bool read(uint32_t u, U* v, const ptx::WaitCtx& w) const {
    const int s = static_cast<int>(u % N);
    if (!__all_sync(0xffffffffu, ptx::mbar_wait(full + s, (u / N) & 1u, w))) return false;
    *v = slots[s];
    return true;
  }
};

// The producer's next unit, found while the tiles of the current one are being
// loaded. Only units that have something to do are handed on (the plan
// kernels have written the others' results). A unit is claimed from the
// launch's counter three tiles before the end of the one before it, looked up
// two and published one tile before, so that neither latency holds the loads
// up: late, because claims further ahead leave the CTAs to end unevenly (two
// units ahead cost a tenth of the time at 7 units a CTA), and early enough for
// the other roles to read it while they work on the last tiles. A role that
// has the last tile of a unit finds the next one published, so no wait for it
// can hold up the loads that its publication waits for.
template <typename U>
struct NextUnit {
  U u;
  int x;

  // load(x): unit x; work(u): whether it has something to do
  template <typename Load, typename Work>
  __device__ __forceinline__ bool publish(uint32_t* counter, int total, Load load, Work work, const UnitRing<U>& ring,
                                          uint32_t* pu, const ptx::WaitCtx& w) {
    while (x < total && !work(u)) {
      claim(counter);
      look_up(total, load);
    }
    if (x >= total) u.bh = -1;
    return ring.push((*pu)++, u, w);
  }
  __device__ __forceinline__ void claim(uint32_t* counter) {
    const uint32_t n = atomicAdd(counter, 1u);
    x = n < 0x7fffffffu ? static_cast<int>(n) : 0x7fffffff;
  }
  template <typename Load>
  __device__ __forceinline__ void look_up(int total, Load load) {
    if (x < total) u = load(x);
  }
  // what falls before tile i of the current unit's n
  template <typename Load, typename Work>
  __device__ __forceinline__ bool step(int i, int n, uint32_t* counter, int total, Load load, Work work,
                                       const UnitRing<U>& ring, uint32_t* pu, const ptx::WaitCtx& w) {
    if (i == max(n - 3, 0)) claim(counter);
    if (i == max(n - 2, 0)) look_up(total, load);
    return i != n - 1 || publish(counter, total, load, work, ring, pu, w);
  }
  template <typename Load, typename Work>
  __device__ __forceinline__ bool first(uint32_t* counter, int total, Load load, Work work, const UnitRing<U>& ring,
                                        uint32_t* pu, const ptx::WaitCtx& w) {
    claim(counter);
    look_up(total, load);
    return publish(counter, total, load, work, ring, pu, w);
  }
};

}  // namespace scored
}  // namespace attn
