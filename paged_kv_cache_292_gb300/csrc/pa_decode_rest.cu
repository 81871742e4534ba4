// The tokens of a batch's sequences behind their shared prefix: the decode
// kernel with kWalkRest.
#include "pa_launch.cuh"

namespace pa {

int launch_rest(const DecodeParams& prm, const Plan& pl, int dev, cudaStream_t stream, int head_size, bool kv_fp8) {
  using T = __nv_bfloat16;
  const int columns = prm.group * prm.num_queries;
  if (kv_fp8) {
    if (head_size == 64)
      return columns <= 8 ? launch_typed<T, 64, 8, 1, true, kWalkRest>(prm, pl, dev, stream)
                          : launch_typed<T, 64, 8, 2, true, kWalkRest>(prm, pl, dev, stream);
    return columns <= 8 ? launch_typed<T, 128, 8, 1, true, kWalkRest>(prm, pl, dev, stream)
                        : launch_typed<T, 128, 8, 2, true, kWalkRest>(prm, pl, dev, stream);
  }
  if (head_size == 64) {
    if (prm.num_queries == 1) return launch_typed<T, 64, 8, 0, false, kWalkRest>(prm, pl, dev, stream);
    return columns <= 8 ? launch_typed<T, 64, 8, 1, false, kWalkRest>(prm, pl, dev, stream)
                        : launch_typed<T, 64, 8, 2, false, kWalkRest>(prm, pl, dev, stream);
  }
  if (prm.num_queries == 1) return launch_typed<T, 128, 8, 0, false, kWalkRest>(prm, pl, dev, stream);
  return columns <= 8 ? launch_typed<T, 128, 8, 1, false, kWalkRest>(prm, pl, dev, stream)
                      : launch_typed<T, 128, 8, 2, false, kWalkRest>(prm, pl, dev, stream);
}

}  // namespace pa
