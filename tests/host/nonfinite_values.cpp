// add_nonfinite for every lane of a wave over the last tile of a sequence whose
// table ends where readable memory ends: exit status 0 if every dimension got
// its infinities back; a read past the table ends the process.
#include "attention.hpp"

#include <stdlib.h>
#include <sys/mman.h>
#include <unistd.h>
#include <vector>

unsigned host_lane;
using namespace trellis;

int main(int argc, char** argv) {
  if (argc != 4) return 2;
  const int keys = atoi(argv[1]), page_log2 = atoi(argv[2]), width = atoi(argv[3]);
  constexpr int D = 64;
  const int room = width << page_log2;
  // the table's last entry is the last one before a page without access
  const size_t bytes = (size_t)sysconf(_SC_PAGESIZE);
  char* mem = (char*)mmap(nullptr, 2 * bytes, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
  if (mem == MAP_FAILED || mprotect(mem + bytes, bytes, PROT_NONE)) return 2;
  int32_t* table = (int32_t*)(mem + bytes) - width;
  for (int p = 0; p < width; ++p) table[p] = p;
  std::vector<uint16_t> v((size_t)room * D, 0x7F80);         // bf16 infinities everywhere, one head
  RowMask mask{};
  mask.below = room;                                         // a row that sees every key
  float got[D];
  for (host_lane = 0; host_lane < 64; host_lane += 32) {
    f32x16 o[D / 32] = {};
    const int kb = (room - 1) / keys * keys;
    add_nonfinite<Bf16, D, false>(v.data(), (GlobalInts)table, room, (uint32_t)width, (uint32_t)(D << page_log2), page_log2, mask, kb, keys, o);
    for (int d = 0; d < D / 32; ++d)
      for (int r = 0; r < 16; ++r) got[d * 32 + 8 * (r >> 2) + 4 * (host_lane >> 5) + (r & 3)] = o[d][r];
  }
  for (int d = 0; d < D; ++d)
    if (!isinf(got[d])) return 1;
  return 0;
}
