// A CUDA runtime for host tests: linked with the library's own objects in place of
// the real one, it runs nothing and notes what it is asked for (kernel launches,
// shared-memory attributes, tensor maps), one text line each. No GPU, and the
// pointers that a test passes are never read.
#include <cstdio>
#include <map>
#include <string>

#include "../free_sparse_attention_head_b200/csrc/internal.h"

namespace {

std::map<const void*, std::string> names;
std::map<const void*, long long> allowed;  // dynamic shared memory that a kernel was given leave for
std::string log_text;
cudaError_t last_error = cudaSuccess;
struct Config {
  dim3 grid, block;
  size_t smem;
  cudaStream_t stream;
} pushed;
int refuse;  // 1: attributes, 2: launches

cudaError_t note(cudaError_t e) {
  if (e != cudaSuccess) last_error = e;
  return e;
}

// a block's shared memory: 48 KB without leave, 227 KB with it (sm_100); both hold
// what a kernel declares for itself too, here taken to be 1 KB at most
constexpr long long kFree = 47 * 1024, kMost = 232448;

cudaError_t launch(const void* f, dim3 g, dim3 b, size_t smem) {
  const long long most = allowed.count(f) ? allowed[f] : kFree;
  const bool bad = refuse == 2 || static_cast<long long>(smem) > most || g.x == 0 || g.y == 0 || g.z == 0 || g.y > 65535 || g.z > 65535;
  char line[512];
  snprintf(line, sizeof line, "launch %s %u %u %u %u %zu %d\n", names[f].c_str(), g.x, g.y, g.z, b.x, smem, bad ? 1 : 0);
  log_text += line;
  return note(bad ? cudaErrorInvalidValue : cudaSuccess);
}

}  // namespace

extern "C" {

const char* fake_log() { return log_text.c_str(); }
// a call may not live on the leave that an earlier one gave
void fake_clear() {
  log_text.clear();
  allowed.clear();
}
void fake_refuse(int what) { refuse = what; }
int fake_last_error() { return last_error; }

void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* device, int, uint3*, uint3*, dim3*, dim3*, int*) {
  names[host] = device;
}
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
  pushed = {grid, block, smem, stream};
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* stream) {
  *grid = pushed.grid;
  *block = pushed.block;
  *smem = pushed.smem;
  *static_cast<cudaStream_t*>(stream) = pushed.stream;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int value) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) {
    char line[512];
    snprintf(line, sizeof line, "allow %s %d\n", names[f].c_str(), value);
    log_text += line;
    if (refuse == 1 || value > kMost) return note(cudaErrorInvalidValue);
    allowed[f] = value;
  }
  return cudaSuccess;
}
cudaError_t cudaLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t smem, cudaStream_t) {
  return launch(f, grid, block, smem);
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  return launch(f, c->gridDim, c->blockDim, c->dynamicSmemBytes);
}
cudaError_t cudaGetLastError() {
  const cudaError_t e = last_error;
  last_error = cudaSuccess;
  return e;
}

}  // extern "C"

namespace svoo {

CUresult encode_tiled_2d(CUtensorMap*, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows, uint32_t) {
  char line[256];
  snprintf(line, sizeof line, "map %llu %llu %llu %u\n", static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(base)),
           static_cast<unsigned long long>(rows), static_cast<unsigned long long>(cols), box_rows);
  log_text += line;
  return CUDA_SUCCESS;
}

CUresult encode_token_major(CUtensorMap*, const void*, uint64_t, uint64_t, uint64_t, uint64_t, uint32_t heads,
                            uint32_t tokens) {
  char line[128];
  snprintf(line, sizeof line, "rows %u %u\n", heads, tokens);
  log_text += line;
  return heads <= 256 && tokens >= 1 && tokens <= 256 ? CUDA_SUCCESS : CUDA_ERROR_INVALID_VALUE;
}

}  // namespace svoo
