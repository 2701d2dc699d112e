// ops.cu -- the device status word of the operators beside the products.
#include "ops.cuh"

namespace q1 {

static __device__ unsigned g_status_ops = 0u;

int ops_status_ptr(unsigned** p) {
  static unsigned* cached[64] = {};
  int dev = 0;
  if (int e = cuda_status(cudaGetDevice(&dev), "status word")) return e;
  if (dev < 0 || dev >= 64) return fail(Q1_ERR_ARG, "device %d outside 0..63", dev);
  if (!cached[dev]) {
    void* a = nullptr;
    if (int e = cuda_status(cudaGetSymbolAddress(&a, g_status_ops), "status word")) return e;
    cached[dev] = static_cast<unsigned*>(a);
  }
  *p = cached[dev];
  return Q1_OK;
}

int status_word_ops(unsigned* v, int clear) {
  if (int e = cuda_status(cudaMemcpyFromSymbol(v, g_status_ops, sizeof *v), "q1_device_status")) return e;
  if (clear && *v) {
    const unsigned zero = 0;
    return cuda_status(cudaMemcpyToSymbol(g_status_ops, &zero, sizeof zero), "q1_device_status");
  }
  return Q1_OK;
}

}  // namespace q1
