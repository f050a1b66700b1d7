/* Stands in for the runtime calls that the library's operators launch kernels with, so that a test
 * without a GPU sees which kernels a call launches, and can let any of the calls fail.  Loaded
 * into the global scope before the library; nothing is executed. */
#include <stddef.h>
#include <stdlib.h>
#include <string.h>

typedef struct {
  unsigned x, y, z;
} dim3_t;

enum { MAX_KERNELS = 4096, MAX_LAUNCHES = 256 };
static struct {
  const void* host;
  const char* name;
} kernels[MAX_KERNELS];
static int n_kernels;
static struct {
  const void* host;
  dim3_t grid, block;
  size_t lds;
} launches[MAX_LAUNCHES];
static int n_launches;
static struct {
  const void* host;
  int attribute, value;
} attributes[MAX_LAUNCHES];
static int n_attributes;
static int fail_launch, fail_attribute, pending;
static int device;

/* The library's kernels, as they are registered when it is loaded. */
void __hipRegisterFunction(void** modules, const void* host, char* device_function,
                           const char* name, unsigned limit, void* tid, void* bid, void* block,
                           void* grid, int* wave) {
  (void)modules, (void)device_function, (void)limit, (void)tid, (void)bid, (void)block;
  (void)grid, (void)wave;
  if (strstr(name, "3moe") && n_kernels < MAX_KERNELS) {
    kernels[n_kernels].host = host;
    kernels[n_kernels++].name = strdup(name);
  }
}

/* launch: which launch from now on fails (0: none); attribute: whether setting one does; error: what
 * an earlier call of the thread has left behind. */
void stub_reset(int launch, int attribute, int error, int current_device) {
  n_launches = n_attributes = 0;
  fail_launch = launch;
  fail_attribute = attribute;
  pending = error;
  device = current_device;
}
int stub_launches(void) { return n_launches; }
int stub_attributes(void) { return n_attributes; }
int stub_kernels(void) { return n_kernels; }
int stub_pending(void) { return pending; }
const char* stub_kernel(int i) { return kernels[i].name; }
static const char* name_of(const void* host) {
  for (int i = 0; i < n_kernels; ++i)
    if (kernels[i].host == host) return kernels[i].name;
  return "?";
}
const char* stub_launch(int i, unsigned* shape) {
  shape[0] = launches[i].grid.x, shape[1] = launches[i].grid.y, shape[2] = launches[i].grid.z;
  shape[3] = launches[i].block.x, shape[4] = (unsigned)launches[i].lds;
  return name_of(launches[i].host);
}
const char* stub_attribute(int i, int* value) {
  *value = attributes[i].value;
  return name_of(attributes[i].host);
}

int hipLaunchKernel(const void* host, dim3_t grid, dim3_t block, void** args, size_t lds,
                    void* stream) {
  (void)args, (void)stream;
  if (n_launches < MAX_LAUNCHES) {
    launches[n_launches].host = host;
    launches[n_launches].grid = grid;
    launches[n_launches].block = block;
    launches[n_launches].lds = lds;
  }
  ++n_launches;
  if (n_launches == fail_launch) {
    pending = 9;
    return 9;
  }
  return 0;
}
int hipFuncSetAttribute(const void* host, int attribute, int value) {
  if (n_attributes < MAX_LAUNCHES) {
    attributes[n_attributes].host = host;
    attributes[n_attributes].attribute = attribute;
    attributes[n_attributes].value = value;
  }
  ++n_attributes;
  if (fail_attribute) pending = 1;
  return fail_attribute;
}
int hipGetLastError(void) {
  const int e = pending;
  pending = 0;
  return e;
}
int hipGetDeviceCount(int* n) {
  *n = 1;
  return 0;
}
int hipGetDevice(int* d) {
  *d = device;
  return 0;
}
