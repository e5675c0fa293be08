// The key tiles of the tensor-core attention, run on the CPU: reads lines
// "name args..." from stdin, writes one result per line. No device code is
// involved.
#include <cstdio>
#include <cstring>

#include "../../quantized_attention_fp64_gb300/csrc/cache.cuh"

int main() {
  char name[32];
  while (std::scanf("%31s", name) == 1) {
    int a, b;
    if (!std::strcmp(name, "tiles") && std::scanf("%d", &a) == 1) {
      std::printf("%d\n", sage::key_tiles(a));
    } else if (!std::strcmp(name, "tokens") && std::scanf("%d %d", &a, &b) == 2) {
      std::printf("%d\n", sage::block_has_tokens(a, b) ? 1 : 0);
    } else if (!std::strcmp(name, "hides") && std::scanf("%d %d", &a, &b) == 2) {
      std::printf("%d\n", sage::tile_hides_keys(a, b) ? 1 : 0);
    } else {
      return 1;
    }
  }
  return 0;
}
