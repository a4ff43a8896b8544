// The library's one translation unit: the GEMMs' API with the device facts
// and launch helpers, and the serving operators that use them.
#include "w4a8_api.cu"

#include "serving_api.cuh"
