#include "zero_tile.cuh"
namespace zk {
cudaError_t timeouts_ortho(unsigned long long* out, bool reset) { return unit_timeouts(out, reset); }
cudaError_t bounds_ortho(BoundsRec* out, bool reset) { return bounds_record(out, reset); }
}
