// api_common.h -- argument checks shared by the files of entry points.
#pragma once

#include "../../include/hstu.h"

namespace hstu {

// The fields of params that do not depend on a batch: sizes, buckets, scales,
// strides, types (api.cu).
hstu_status_t validate_shape(const hstu_attn_params_t *params);

}  // namespace hstu
