/* A HIP runtime for the host code alone: memory that is never touched, streams and
 * events that are nothing, and a record of the kernels that would have run.  Built
 * with the library's own objects by tests/test_launches_cpu.py. */
#include <stddef.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

typedef struct { uint32_t x, y, z; } dim3;
typedef int status;
enum { OK = 0, NO_MEMORY = 2, MOST = 4096 };

static struct { const void *fn; const char *name; } kernels[1024];
static int n_kernels;
static struct { const char *name; uint32_t blocks, threads; uint64_t a, b; } calls[MOST];
static int n_calls;
static int capture, refuse;      /* what hipStreamIsCapturing and hipMalloc answer */
static uintptr_t next = (uintptr_t)1 << 44, freed;
static dim3 grid, block;
static size_t shared;
static void *on;

/* What the test reads and sets. */
void recorder_reset(void) { n_calls = 0; }
int recorder_count(void) { return n_calls; }
const char *recorder_name(int i) { return calls[i].name; }
uint32_t recorder_blocks(int i) { return calls[i].blocks; }
uint64_t recorder_arg(int i, int k) { return k ? calls[i].b : calls[i].a; }
void recorder_capture(int yes) { capture = yes; }
void recorder_refuse_memory(int yes) { refuse = yes; }

/* Memory given back is what the next request gets, of whatever size. */
status hipMalloc(void **p, size_t n) {
    if (refuse) return NO_MEMORY;
    if (freed) {
        *p = (void *)freed;
        freed = 0;
    } else {
        *p = (void *)next;
        next += ((n + 0xffffffffu) >> 32 << 32);
    }
    return OK;
}
status hipFree(void *p) {
    freed = (uintptr_t)p;
    return OK;
}
status hipHostMalloc(void **p, size_t n, unsigned flags) {
    (void)flags;
    *p = calloc(1, n);
    return *p ? OK : NO_MEMORY;
}
status hipHostFree(void *p) {
    free(p);
    return OK;
}

void **__hipRegisterFatBinary(const void *data) {
    static void *handle;
    (void)data;
    return &handle;
}
void __hipUnregisterFatBinary(void **modules) { (void)modules; }
void __hipRegisterVar(void) {}
void __hipRegisterFunction(void **modules, const void *fn, char *device, const char *name, int limit, void *tid, void *bid,
                           void *bdim, void *gdim, int *wsize) {
    (void)modules, (void)device, (void)limit, (void)tid, (void)bid, (void)bdim, (void)gdim, (void)wsize;
    if (n_kernels < 1024) {
        kernels[n_kernels].fn = fn;
        kernels[n_kernels++].name = name;
    }
}
status __hipPushCallConfiguration(dim3 g, dim3 b, size_t s, void *stream) {
    grid = g, block = b, shared = s, on = stream;
    return OK;
}
status __hipPopCallConfiguration(dim3 *g, dim3 *b, size_t *s, void **stream) {
    *g = grid, *b = block, *s = shared, *stream = on;
    return OK;
}
status hipLaunchKernel(const void *fn, dim3 g, dim3 b, void **args, size_t s, void *stream) {
    (void)s, (void)stream;
    if (n_calls == MOST) return NO_MEMORY;
    calls[n_calls].name = "";
    for (int i = 0; i < n_kernels; ++i)
        if (kernels[i].fn == fn) calls[n_calls].name = kernels[i].name;
    calls[n_calls].blocks = g.x * g.y * g.z;
    calls[n_calls].threads = b.x;
    calls[n_calls].a = calls[n_calls].b = 0;
    if (strstr(calls[n_calls].name, "router_clear")) {  /* (uint32_t *, int64_t) */
        memcpy(&calls[n_calls].a, args[0], 8);
        memcpy(&calls[n_calls].b, args[1], 8);
    }
    ++n_calls;
    return OK;
}
status hipStreamIsCapturing(void *stream, int *answer) {
    (void)stream;
    *answer = capture;
    return OK;
}

status hipGetDeviceCount(int *n) {
    *n = 1;
    return OK;
}
status hipGetDevice(int *d) {
    *d = 0;
    return OK;
}
static void *some(void) { return (void *)(uintptr_t)64; }
status hipSetDevice(int d) { return (void)d, OK; }
status hipDeviceSynchronize(void) { return OK; }
status hipEventCreate(void **e) { return *e = some(), OK; }
status hipEventCreateWithFlags(void **e, unsigned f) { return (void)f, *e = some(), OK; }
status hipEventDestroy(void *e) { return (void)e, OK; }
status hipEventElapsedTime(float *ms, void *a, void *b) { return (void)a, (void)b, *ms = 0, OK; }
status hipEventRecord(void *e, void *s) { return (void)e, (void)s, OK; }
status hipEventSynchronize(void *e) { return (void)e, OK; }
status hipFuncSetAttribute(const void *f, int a, int v) { return (void)f, (void)a, (void)v, OK; }
const char *hipGetErrorString(status e) { return e == OK ? "ok" : "refused"; }
status hipGetLastError(void) { return OK; }
status hipGetSymbolAddress(void **p, const void *symbol) { return (void)symbol, *p = some(), OK; }
status hipMemcpy(void *to, const void *from, size_t n, int kind) { return (void)to, (void)from, (void)n, (void)kind, OK; }
status hipMemcpyAsync(void *to, const void *from, size_t n, int kind, void *s) {
    return (void)to, (void)from, (void)n, (void)kind, (void)s, OK;
}
status hipStreamCreateWithFlags(void **s, unsigned f) { return (void)f, *s = some(), OK; }
status hipStreamDestroy(void *s) { return (void)s, OK; }
status hipStreamSynchronize(void *s) { return (void)s, OK; }
status hipStreamWaitEvent(void *s, void *e, unsigned f) { return (void)s, (void)e, (void)f, OK; }
