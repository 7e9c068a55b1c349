// Which copies a warp of the 4-bit cache's kernels may start, and which are
// still under way when a wait has run out and it leaves: shared memory that a
// copy is yet to land in belongs to the next block once this one has exited.
// Plain logic without device code, so that it compiles for the host too.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MOBA_HD __host__ __device__ __forceinline__
#else
#define MOBA_HD inline
#endif

namespace moba {

// A warp's tiles in kv4_attn.cuh: one buffer for the keys and one for the
// values, each refilled with the next tile's once it has been read. Per tile:
// wait for the keys, read them, start the next keys; wait for the values, read
// them, start the next values. After a wait that ran out nothing is started.
struct Kv4Fetch {
  int left = 0;                    // tiles whose copies have not been started
  int death = 0;                   // the tile in which a wait ran out
  bool dead = false, more = false;
  MOBA_HD void gave_up(int tile) { dead = true, death = tile; }
  // A tile's keys have been read: are the next tile's fetched?
  MOBA_HD bool next_keys() { return more = !dead && left > 0; }
  // Its values have been read: are those of the tile whose keys were?
  MOBA_HD bool next_values() const { return more && !dead; }
  // After giving up: the last tiles, of n, whose copies were started.
  MOBA_HD int last_keys(int n) const { return n - left - 1; }
  MOBA_HD int last_values() const { return death; }
};

// A loader of query tiles in kv4_chunk.cuh, with BUFS buffers that each hold
// one at a time. The port waits until buffer x is empty (phase `parity`; false:
// the wait ran out), starts a copy into it, and waits until the copy has landed.
// That last wait is made whatever has happened: another warp may give up on the
// copy after this one has started it and has nothing left to do.
template <int BUFS>
struct Kv4Feeder {
  uint32_t n[BUFS] = {};  // copies started
  template <class Port>
  MOBA_HD bool load(Port& port, int x) {
    if (!port.empty(x, (n[x] & 1) ^ 1)) return false;
    port.start(x);
    ++n[x];
    return true;
  }
  template <class Port>
  MOBA_HD void finish(Port& port) {
    for (int x = 0; x < BUFS; ++x)
      if (n[x]) port.landed(x, (n[x] - 1) & 1);
  }
};

}  // namespace moba
