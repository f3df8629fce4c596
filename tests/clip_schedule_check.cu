// Host-side check of the gradient norm's launches (clip.cuh): however many
// tensors a call has, each launch has all the CTAs that its chunks can use (two per
// SM), every slot is written before a later launch adds to it, and the slots end
// inside the workspace.  Built and run on the CPU by tests/test_clip_schedule.py;
// prints "ok ..." or the first failure.
#include <cstdio>
#include <vector>

#include "clip.cuh"

using namespace fp8bs;

static int run(int64_t tensors, int64_t elements, int sms) {
  const int64_t chunks_of_one = (elements + clip::kChunk - 1) / clip::kChunk;
  const int slots = clip::max_ctas(sms);
  std::vector<char> written(slots, 0);
  int used = 0;
  for (int64_t i = 0; i < tensors; i += clip::kMaxTensors) {
    const int64_t here = tensors - i < clip::kMaxTensors ? tensors - i : clip::kMaxTensors;
    const int chunks = static_cast<int>(here * chunks_of_one);
    const int grid = clip::launch_ctas(chunks, sms);
    if (grid < 1 || grid > chunks || (grid < 2 * sms && grid < chunks)) {
      std::printf("%lld tensors of %lld: %d CTAs for %d chunks\n", (long long)tensors,
                  (long long)elements, grid, chunks);
      return 1;
    }
    for (int b = 0; b < grid; ++b) {
      if (b >= slots || (b < used) != (written[b] != 0)) {
        std::printf("%lld tensors of %lld: slot %d\n", (long long)tensors, (long long)elements, b);
        return 1;
      }
      written[b] = 1;
    }
    used = used > grid ? used : grid;
  }
  return 0;
}

int main() {
  int cases = 0;
  for (int64_t tensors : {1, 127, 128, 129, 1024, 1025, 2000, 5120, 44000, 1 << 20})
    for (int64_t elements : {1, 16384, 16385, 1000000})
      for (int sms : {148, 20}) {
        if (run(tensors, elements, sms)) return 1;
        ++cases;
      }
  std::printf("ok %d calls\n", cases);
  return 0;
}
