// Runs on the host, with or without a GPU: a failure that a call has reported is not left behind as
// the CUDA runtime's last error, where it would fail somebody else's next check.  Without a GPU the
// runtime has that error always, so what is looked at is that it was taken back.  No kernel runs:
// the launch has no blocks.  Prints "ok" and exits 0.
#include <cuda.h>
#include <cuda_runtime.h>

static int taken_back = 0;
static cudaError_t take_back() {
  ++taken_back;
  return cudaGetLastError();
}
#define cudaGetLastError take_back
#include "kv_host.cuh"

__global__ void nothing(int) {}

int main() {
  int x = 0, devices = 0;
  const bool gpu = cudaGetDeviceCount(&devices) == cudaSuccess && devices > 0;
  auto clean = [&] {
    const bool ok = taken_back > 0 && (!gpu || cudaPeekAtLastError() == cudaSuccess);
    taken_back = 0;
    return ok;
  };
  REQUIRE(launch((const void*)nothing, dim3(0), 32, 0, &x, nullptr) == CS_ERR_CUDA && clean());
  if (!gpu) {  // what a plan and its calls do then
    cs_kv_desc d;
    REQUIRE(cs_kv_desc_init(&d) == CS_OK);
    d.heads = d.kv_heads = d.num_pages = d.max_tokens = d.max_seqs = 1;
    cs_kv_t plan = nullptr;
    REQUIRE(cs_kv_plan(&d, &plan) == CS_ERR_CUDA && clean());
    cs_kv_s none;
    none.d = d;
    REQUIRE(cs_kv_status(&none) == CS_ERR_CUDA && clean());
    REQUIRE(cs_kv_reset(&none) == CS_ERR_CUDA && clean());
    REQUIRE(!DeviceGuard(0).ok && clean());
  }
  printf("ok\n");
  return 0;
}
