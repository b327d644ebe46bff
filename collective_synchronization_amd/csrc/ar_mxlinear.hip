// ar_mxlinear.hip -- the linear shards on microscaled 4-bit weights alone.
#include "ar_mxlinear.h"

using namespace ar;

extern "C" {

int ar_mx4_linear(const ar_linear_params* p, void* stream) {
  const int rc = check_linear(p);
  if (rc) return rc;
  if (p->rows == 0 || p->outputs == 0) return AR_OK;
  const int64_t tiles = ceil_div64(p->outputs, 16) * ceil_div64(p->rows, 16) * p->nranks;
  if (tiles > INT32_MAX) return AR_ESIZE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return map_hip(launch_pieces(linear_args(p), NoAdapters{}, p->x_format, p->y_format, p->nranks, s));
}

}  // extern "C"
