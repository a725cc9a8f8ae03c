/*
 * launch_recorder.c -- stands in for the HIP runtime where there is no GPU: it
 * has every runtime symbol that libgemm355.so uses, keeps the kernels' names as
 * the library registers them and writes down each launch (kernel, workgroups,
 * threads) instead of making it. Loaded with its symbols global before the
 * library, which then binds to these.
 */
#include <stddef.h>
#include <stdlib.h>
#include <string.h>

struct dim3 {
    unsigned x, y, z;
};

enum { MAX_KERNELS = 4096, MAX_LAUNCHES = 256 };

static struct {
    const void *host;
    const char *name;
} kernels[MAX_KERNELS];
static int kernel_count;

static struct {
    const char *name;
    unsigned blocks, threads;
} launches[MAX_LAUNCHES];
static int launch_count;
static int units = 256;

void **__hipRegisterFatBinary(const void *data)
{
    static void *handle;
    (void)data;
    return &handle;
}
void __hipUnregisterFatBinary(void **handle) { (void)handle; }
void __hipRegisterFunction(void **handle, const void *host, char *device, const char *name, unsigned limit, void *a,
                           void *b, void *c, void *d, int *e)
{
    (void)handle, (void)device, (void)limit, (void)a, (void)b, (void)c, (void)d, (void)e;
    if (kernel_count == MAX_KERNELS)
        abort();
    kernels[kernel_count].host = host;
    kernels[kernel_count++].name = strdup(name);
}
void __hipRegisterVar(void **handle, void *var, char *host, char *device, int ext, size_t size, int constant, int global)
{
    (void)handle, (void)var, (void)host, (void)device, (void)ext, (void)size, (void)constant, (void)global;
}
int __hipPopCallConfiguration(struct dim3 *grid, struct dim3 *block, size_t *shared, void *stream)
{
    (void)grid, (void)block, (void)shared, (void)stream;
    abort();   /* the library launches through hipLaunchKernel alone */
}
int hipGetSymbolAddress(void **address, const void *symbol)
{
    *address = (void *)symbol;
    return 0;
}
int hipGetDevice(int *device)
{
    *device = 0;
    return 0;
}
int hipDeviceGetAttribute(int *value, int attribute, int device)
{
    (void)device;
    (void)attribute;   /* the library asks for the multiprocessor count alone */
    *value = units;
    return 0;
}
int hipLaunchKernel(const void *host, struct dim3 grid, struct dim3 block, void **args, size_t shared, void *stream)
{
    (void)args, (void)shared, (void)stream;
    if (launch_count == MAX_LAUNCHES || grid.y != 1 || grid.z != 1 || block.y != 1 || block.z != 1)
        abort();
    const char *name = "";
    for (int i = 0; i < kernel_count; ++i)
        if (kernels[i].host == host)
            name = kernels[i].name;
    launches[launch_count].name = name;
    launches[launch_count].blocks = grid.x;
    launches[launch_count++].threads = block.x;
    return 0;
}

/* What the test asks. */
int recorder_take(void)   /* the launches since the last call of this */
{
    const int n = launch_count;
    launch_count = 0;
    return n;
}
const char *recorder_name(int i) { return launches[i].name; }
unsigned recorder_blocks(int i) { return launches[i].blocks; }
unsigned recorder_threads(int i) { return launches[i].threads; }
