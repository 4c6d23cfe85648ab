// libgemm_bf16.so as one translation unit: the bf16 product, and the 8-bit
// product and operators around it, which use its device helpers (buffer
// resources, direct global-to-LDS loads, the LDS ring's loader and swizzles)
// and its host side (device query, kept temporary memory, argument checks)
// without any of these becoming exported symbols.
#include "gemm_bf16.hip"

#include "ops_common.h"

#include "rms_norm.h"
#include "swiglu.h"
#include "quantize_fp8.h"

#include "gemm_fp8.h"
