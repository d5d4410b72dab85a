// Prints the random bits of the 8-bit AdamW states, as the kernel's lanes
// compose them: arguments seed, t, first group of the tile, threads of a
// workgroup; one line "<index in the tile> <word>" for each element of the tile.
#include <cinttypes>
#include <cstdio>
#include <cstdlib>

#include "../../ddp_bucketed_gradient_amd/csrc/optim.hpp"

int main(int argc, char** argv) {
  if (argc != 5) return 2;
  const uint64_t seed = std::strtoull(argv[1], nullptr, 10), tile = std::strtoull(argv[3], nullptr, 10);
  const int64_t t = std::strtoll(argv[2], nullptr, 10);
  const uint32_t threads = static_cast<uint32_t>(std::atoi(argv[4]));
  const ddpb::StepScalars sc = ddpb::step_scalars(t - 1, 0.9, 0.999, seed);
  for (uint32_t at = 0; at < ddpb::kOptimTile; at += 4 * threads)
    for (uint32_t lane = 0; lane < threads; ++lane) {
      const uint32_t start = ddpb::hash_start(tile, lane, sc.key0);
      const uint32_t h = ddpb::hash_mix(ddpb::hash_at(start, static_cast<uint32_t>(tile), lane, at / 4), sc.key1);
      for (uint32_t j = 0; j < 4; ++j)
        std::printf("%" PRIu32 " %" PRIu32 "\n", at + 4 * lane + j, ddpb::hash_element(h, j));
    }
  return 0;
}
