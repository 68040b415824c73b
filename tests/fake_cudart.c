/* A stand-in for the CUDA runtime calls that a launch of libbcjr makes, for tests of the host side without a GPU:
 * it keeps each kernel's limit of dynamic shared memory and refuses a launch above it, as the runtime does. */
#include <cuda_runtime_api.h>
#include <pthread.h>

#define KERNELS 512
static const void* kernels[KERNELS];
static int limits[KERNELS];
static int count, launches, refused, fail_sets;
static void (*after_set)(void);
static pthread_mutex_t lock = PTHREAD_MUTEX_INITIALIZER;

static int* limit_of(const void* kernel) {
  for (int i = 0; i < count; ++i)
    if (kernels[i] == kernel) return &limits[i];
  if (count == KERNELS) return limits;
  kernels[count] = kernel;
  limits[count] = 48 * 1024;
  return &limits[count++];
}

static cudaError_t launch(const void* kernel, size_t shared) {
  pthread_mutex_lock(&lock);
  const int fits = shared <= (size_t)*limit_of(kernel);
  ++launches;
  refused += !fits;
  pthread_mutex_unlock(&lock);
  return fits ? cudaSuccess : cudaErrorInvalidValue;
}

static _Thread_local cudaError_t last;

cudaError_t cudaGetDevice(int* device) { *device = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* value, enum cudaDeviceAttr attr, int device) {
  (void)device;
  *value = attr == cudaDevAttrMultiProcessorCount ? 148 : attr == cudaDevAttrMaxSharedMemoryPerBlockOptin ? 227 * 1024 : 0;
  return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { cudaError_t e = last; last = cudaSuccess; return e; }
cudaError_t cudaFuncSetAttribute(const void* kernel, enum cudaFuncAttribute attr, int value) {
  if (attr != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
  pthread_mutex_lock(&lock);
  const int fails = fail_sets > 0 || value > 227 * 1024;
  if (fail_sets > 0) --fail_sets;
  if (!fails) *limit_of(kernel) = value;
  void (*hook)(void) = after_set;
  after_set = 0;
  pthread_mutex_unlock(&lock);
  if (fails) return last = cudaErrorInvalidValue;
  if (hook) hook();  /* what another thread does at this moment */
  return cudaSuccess;
}
cudaError_t cudaLaunchKernel(const void* kernel, dim3 grid, dim3 block, void** args, size_t shared, cudaStream_t stream) {
  (void)grid, (void)block, (void)args, (void)stream;
  return last = launch(kernel, shared);
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* config, const void* kernel, void** args) {
  (void)args;
  return last = launch(kernel, config->dynamicSmemBytes);
}

void fake_after_set(void (*hook)(void)) { after_set = hook; }
void fake_fail_sets(int n) { fail_sets = n; }
int fake_launches(void) { return launches; }
int fake_refused(void) { return refused; }
