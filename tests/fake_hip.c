/* A stand-in for the HIP runtime: the calls the library makes, answered on
 * the host and recorded, so that what the library would launch and allocate
 * can be looked at without a GPU.  Nothing is executed.  Loaded before the
 * library with its symbols global (host_runtime.py). */
#include <pthread.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

typedef struct {
  uint32_t x, y, z;
} dim3;
typedef void* stream_t;

typedef struct {
  const char* name;
  uint64_t grid[3], block[3];
  uint64_t stream;
} Launch;

enum { kSuccess = 0, kInvalidValue = 1, kOutOfMemory = 2, kInvalidConfiguration = 9 };

static pthread_mutex_t mu = PTHREAD_MUTEX_INITIALIZER;
static Launch launches[4096];
static int launch_count;
static struct {
  const void* f;
  const char* name;
} names[16384];
static int name_count;
static uint64_t next_address = 0x100000000000ull;
static int malloc_count, free_count;
static char fail_kernel[256];      /* the next launch of a kernel whose name holds this fails */
static int capturing;
static __thread int last_error;    /* as in HIP: kept until it is asked for */
static __thread struct {
  dim3 grid, block;
  size_t shared;
  stream_t stream;
} config;

static int done(int e) {
  if (e) last_error = e;
  return e;
}

/* ------------------------------------------------------- for the tests */
int fake_launches(void) { return launch_count; }
Launch* fake_launch(int i) { return &launches[i]; }
int fake_mallocs(void) { return malloc_count; }
int fake_frees(void) { return free_count; }
void fake_reset(void) { launch_count = malloc_count = free_count = 0; }
void fake_fail(const char* kernel) { strncpy(fail_kernel, kernel, sizeof(fail_kernel) - 1); }
void fake_capture(int on) { capturing = on; }
void fake_stale_error(int e) { last_error = e; }

/* --------------------------------------------------------- the runtime */
void** __hipRegisterFatBinary(const void* data) {
  static void* module;
  (void)data;
  return &module;
}
void __hipUnregisterFatBinary(void** m) { (void)m; }
void __hipRegisterFunction(void** m, const void* f, char* device, const char* name, unsigned limit, void* tid, void* bid, dim3* b,
                           dim3* g, int* w) {
  (void)m, (void)device, (void)limit, (void)tid, (void)bid, (void)b, (void)g, (void)w;
  if (name_count < 16384) {
    names[name_count].f = f;
    names[name_count++].name = name;
  }
}
void __hipRegisterVar(void** m, void* v, char* h, char* d, int e, size_t s, int c, int g) {
  (void)m, (void)v, (void)h, (void)d, (void)e, (void)s, (void)c, (void)g;
}
int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, stream_t st) {
  config.grid = grid, config.block = block, config.shared = shared, config.stream = st;
  return kSuccess;
}
int __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, stream_t* st) {
  *grid = config.grid, *block = config.block, *shared = config.shared, *st = config.stream;
  return kSuccess;
}
int hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t shared, stream_t st) {
  (void)args, (void)shared;
  const char* name = "?";
  for (int i = 0; i < name_count; i++)
    if (names[i].f == f) name = names[i].name;
  pthread_mutex_lock(&mu);
  int e = kSuccess;
  /* the runtime counts threads of a grid's dimension in 32 bits */
  if ((uint64_t)grid.x * block.x > 0xffffffffull || (uint64_t)grid.y * block.y > 0xffffffffull || !grid.x || !grid.y || !grid.z)
    e = kInvalidConfiguration;
  if (fail_kernel[0] && strstr(name, fail_kernel)) {
    fail_kernel[0] = 0;
    e = kInvalidValue;
  }
  if (!e && launch_count < 4096) {
    Launch l = {name, {grid.x, grid.y, grid.z}, {block.x, block.y, block.z}, (uint64_t)(uintptr_t)st};
    launches[launch_count++] = l;
  }
  pthread_mutex_unlock(&mu);
  return done(e);
}
int hipMalloc(void** p, size_t bytes) {
  if (bytes > (288ull << 30)) return done(kOutOfMemory);
  pthread_mutex_lock(&mu);
  *p = (void*)(uintptr_t)next_address;
  next_address += (bytes + (2u << 20) - 1) / (2u << 20) * (2u << 20);
  malloc_count++;
  pthread_mutex_unlock(&mu);
  return kSuccess;
}
int hipFree(void* p) {
  pthread_mutex_lock(&mu);
  if (p) free_count++;
  pthread_mutex_unlock(&mu);
  return kSuccess;
}
int hipGetDevice(int* d) { return *d = 0; }
int hipSetDevice(int d) { return done(d ? kInvalidValue : kSuccess); }
int hipGetDeviceCount(int* n) {
  *n = 1;
  return kSuccess;
}
int hipDeviceGetAttribute(int* v, int a, int d) {
  (void)a, (void)d;
  *v = 256;
  return kSuccess;
}
int hipOccupancyMaxActiveBlocksPerMultiprocessor(int* v, const void* f, int block, size_t shared) {
  (void)f, (void)block, (void)shared;
  *v = 2;
  return kSuccess;
}
int hipDeviceSynchronize(void) { return kSuccess; }
int hipStreamSynchronize(stream_t st) {
  (void)st;
  return kSuccess;
}
int hipStreamIsCapturing(stream_t st, int* status) {
  (void)st;
  *status = capturing;
  return kSuccess;
}
int hipGetLastError(void) {
  const int e = last_error;
  last_error = kSuccess;
  return e;
}
const char* hipGetErrorString(int e) { return e ? "an error" : "no error"; }
int hipGetSymbolAddress(void** p, const void* s) {
  (void)p, (void)s;
  return done(kInvalidValue);
}
int hipMemcpy(void* to, const void* from, size_t n, int kind) {
  (void)to, (void)from, (void)n, (void)kind;
  return kSuccess;
}
int hipMemcpyAsync(void* to, const void* from, size_t n, int kind, stream_t st) {
  (void)to, (void)from, (void)n, (void)kind, (void)st;
  return kSuccess;
}
