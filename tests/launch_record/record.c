/* Stands in for the HIP runtime's launch functions: writes down what a call of
 * liblpq.so would launch, its kernel arguments too, and launches nothing.  Loaded
 * with global symbols before the library, in a process of its own. */
#include <stddef.h>
#include <string.h>

typedef struct {
    unsigned x, y, z;
} dim3;

typedef struct {
    unsigned grid[3], block[3];
    unsigned char args[256];   /* the first `sizes` bytes of each argument, one after the other */
} record_launch;

enum { MOST = 4096, ARGS = 8 };
record_launch record_list[MOST];
int record_count;
int record_sizes[ARGS];        /* bytes to keep of each argument, 0 behind the last one */

static dim3 g_grid, g_block;
static size_t g_shared;
static void* g_stream;

int hipGetLastError(void) { return 0; }

int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, void* stream) {
    g_grid = grid;
    g_block = block;
    g_shared = shared;
    g_stream = stream;
    return 0;
}

int __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, void** stream) {
    *grid = g_grid;
    *block = g_block;
    *shared = g_shared;
    *stream = g_stream;
    return 0;
}

int hipLaunchKernel(const void* kernel, dim3 grid, dim3 block, void** args, size_t shared, void* stream) {
    (void)kernel, (void)shared, (void)stream;
    if (record_count == MOST) return 1;
    record_launch* r = &record_list[record_count++];
    r->grid[0] = grid.x, r->grid[1] = grid.y, r->grid[2] = grid.z;
    r->block[0] = block.x, r->block[1] = block.y, r->block[2] = block.z;
    size_t at = 0;
    for (int i = 0; i < ARGS && record_sizes[i]; i++) {
        memcpy(r->args + at, args[i], (size_t)record_sizes[i]);
        at += (size_t)record_sizes[i];
    }
    return 0;
}
