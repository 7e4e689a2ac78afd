// ckda_scan_grad_f32.cu -- gradients of the selective scan on fp32 inputs.
#include "ckda_scan_grad.cuh"

namespace ckda {
template cudaError_t launch_scan_grads<float>(const ScanBwdArgs& b, cudaStream_t s);
}
