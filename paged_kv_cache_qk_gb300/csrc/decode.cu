// Host side of the plain decode kernel (decode_kernel.cuh): its plan, and the launch.
#include "decode_kernel.cuh"

namespace pkvqk {

namespace {

template <int HPC>
void fill_plan(DecodePlan& p) {
  using C = Config<HPC>;
  const int tk = p.tensor_core ? 16 : C::kSimtTK;
  const int budget = p.tensor_core ? C::kTcBudget : C::kSimtBudget;
  p.tile_keys = tk;
  const int stage = 2 * HPC * 2 * tk * 128;
  int stages = budget * 1024 / stage;
  stages = stages < 2 ? 2 : (stages > 8 ? 8 : stages);
  const int smem = stages * stage + 1024 + 512;       // + static shared memory
  p.ctas_per_sm = smem > 0 ? (228 * 1024) / smem : 1;
  if (p.ctas_per_sm < 1) p.ctas_per_sm = 1;
}

}  // namespace

DecodePlan plan_decode(int num_kv_heads, int rows) {
  DecodePlan p;
  int hpc = 8;
  while (hpc > 1 && (num_kv_heads % hpc) != 0) hpc >>= 1;
  p.heads_per_cta = hpc;
  p.tensor_core = rows > 2;
  p.rows = rows;
  switch (hpc) {
    case 8: fill_plan<8>(p); break;
    case 4: fill_plan<4>(p); break;
    case 2: fill_plan<2>(p); break;
    default: fill_plan<1>(p); break;
  }
  return p;
}

cudaError_t launch_paged_decode(const DecodePlan& p, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, const DecodeArgs& a, int grid_ctas,
                                cudaStream_t stream) {
  return launch_decode<false>(p, kmap, vmap, a, grid_ctas, stream);
}

}  // namespace pkvqk
