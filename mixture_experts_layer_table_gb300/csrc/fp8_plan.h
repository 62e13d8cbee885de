// How the E4M3 products (fp8_gemm.cu) cut their work: the columns of a chunk, the pairs that share a tile along K, and the
// clusters that a device holds at once.  Plain C++ so that the host tests can check it.
#pragma once

#include <algorithm>
#include <cstdint>
#include <mutex>

namespace mok {

// How many clusters of 4 and of 8 CTAs fit a device at once, asked once for each device; 0 where none does.
class Fp8Clusters {
 public:
  // ask(counts) -> 0, or an error, which is handed on and asked again.  Threads wait for the one that asks, so that all plan alike.
  template <typename Error, typename Ask>
  Error get(int device, int (&counts)[2], Ask&& ask) {
    std::lock_guard<std::mutex> lock(mu_);
    if (!known_[device]) {
      const Error err = ask(counts_[device]);
      if (err != Error(0)) return err;
      known_[device] = true;
    }
    for (int i = 0; i < 2; ++i) counts[i] = counts_[device][i];
    return Error(0);
  }

 private:
  std::mutex mu_;
  bool known_[64] = {};
  int counts_[64][2] = {};
};

struct Fp8Plan {
  int nmax = 0;       // columns of a chunk at most
  int splits = 0;     // pairs of a cluster, each with its share of a tile's blocks
  int64_t tiles = 0;  // at most
};

// The columns of a chunk and the pairs that share a tile, by the time of the pair that has most to do:
// about 200 + 4 n cycles for each block of n columns (measured: 1,200 at 256, 700 at 128, 450 at 64), a tile's start and end about
// 3,000, the joining of splits 3,000 + 20 n.  E groups, of which `groups` can have rows; MT: pair tiles along A's rows; `each`:
// columns of each of the groups; where the groups' sizes are not known here (`known` false) it is their average, and half a chunk
// a group is added.  Splits are taken only where every tile has its own cluster and all clusters fit at once (36 of 4
// CTAs, 15 of 8 on GB300), and the sums fit the first pair's stages (`room` bytes).
inline Fp8Plan f8_plan(int E, int MT, int n_sm, int64_t nkb, int64_t groups, int64_t each, bool known, const int (&clusters)[2],
                       int64_t room) {
  const int64_t pairs = std::max(1, n_sm / 2);
  int64_t best = INT64_MAX;
  Fp8Plan plan;
  for (int nmax = 256; nmax >= 32; nmax /= 2)
    for (int splits = 1; splits <= 4; splits *= 2) {
      const int64_t whole = (each + nmax - 1) / nmax;
      const int64_t chunks = known ? groups * whole : std::max(groups, groups * (2 * each + nmax) / (2 * nmax));
      const int64_t most = (known ? chunks : groups * whole + E) * MT;
      if (splits > 1 && (most > clusters[splits / 4] || nkb < 4 * splits || (splits - 1) * nmax * 512 > room)) continue;
      const int64_t n = std::max<int64_t>(16, groups * each / chunks);
      const int64_t waves = (chunks * MT * splits + pairs - 1) / pairs;
      const int64_t cost = waves * ((nkb + splits - 1) / splits * (200 + 4 * n) + 3000) + (splits > 1 ? 3000 + 20 * n : 0);
      if (cost < best) {
        best = cost;
        plan.nmax = nmax;
        plan.splits = splits;
        plan.tiles = most;
      }
    }
  return plan;
}

}  // namespace mok
