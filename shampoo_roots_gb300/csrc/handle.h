// What a handle holds for every entry point: its device and the launch count.
// precond.cu adds the preconditioner's plans and workspace; the operators
// (operators.cu) need no more than this.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/precond.h"

namespace precond {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct Handle {
  int device = -1;                     // -1: host-only
  int num_sms = 152;                   // a GB300's; a device handle reads its device's count
  int64_t launches = 0;                // kernels launched since creation
  EncodeTiledFn encode = nullptr;
  unsigned int* op_err = nullptr;      // operators: device word, set when a bounded wait ran out
  int pairs = 0;                       // operators: CTA pairs that are resident at once
  int clusters[9] = {};                // operators: clusters of n blocks that are resident at once, one block on an SM
  bool op_ready = false;               // operators: kernel attributes set on this device
};

Handle* as_handle(precond_t h);

}  // namespace precond
