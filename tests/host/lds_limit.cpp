// LdsLimit from eight threads on four devices: every thread finds its device's
// limit raised when raise() returns, a failure is reported and tried again.
#include "internal.hpp"

#include <thread>
#include <vector>

using namespace trellis;
static thread_local int device;
static std::atomic<int> calls[70];
static std::atomic<bool> failing{true};
hipError_t hipGetDevice(int* d) {
  *d = device;
  return device == 69 ? 1 : hipSuccess;
}
hipError_t hipFuncSetAttribute(const void* kernel, int what, int bytes) {
  if (what != hipFuncAttributeMaxDynamicSharedMemorySize || bytes != 4096 || !kernel) return 7;
  if (device == 5 && failing) return 9;
  ++calls[device];
  return hipSuccess;
}

int main() {
  static LdsLimit limit;
  std::vector<std::thread> all;
  std::atomic<int> wrong{0};
  for (int i = 0; i < 8; ++i)
    all.emplace_back([&wrong, i] {
      for (int j = 0; j < 2000; ++j) {
        device = (i + j) % 4;
        if (limit.raise(&wrong, 4096) != hipSuccess || calls[device] == 0) ++wrong;
      }
    });
  for (auto& t : all) t.join();
  for (int d = 0; d < 4; ++d)
    if (calls[d] < 1 || calls[d] > 8) ++wrong;               // at most each thread's first call
  device = 5;
  if (limit.raise(&wrong, 4096) != 9) ++wrong;
  failing = false;
  if (limit.raise(&wrong, 4096) != hipSuccess || calls[5] != 1) ++wrong;
  device = 69;
  if (limit.raise(&wrong, 4096) != hipErrorInvalidDevice) ++wrong;
  device = 68;                                               // past the notes: raised at every call
  if (limit.raise(&wrong, 4096) != hipSuccess || limit.raise(&wrong, 4096) != hipSuccess || calls[68] != 2) ++wrong;
  return wrong != 0;
}
