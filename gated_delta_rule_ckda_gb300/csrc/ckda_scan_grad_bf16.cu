// ckda_scan_grad_bf16.cu -- gradients of the selective scan on bf16 inputs.
#include "ckda_scan_grad.cuh"

namespace ckda {
template cudaError_t launch_scan_grads<__nv_bfloat16>(const ScanBwdArgs& b, cudaStream_t s);
}
