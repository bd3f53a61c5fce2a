// libflp.cu - the library's one translation unit: the fused head (csrc/) and
// the training-step operators beside it (this folder), which share its error
// text, device checks, tensor maps and pair kernels' pieces.
#include "../csrc/flp.cu"
#include "step_abi.cuh"
