/* A stand-in for the HIP calls by which the library launches a kernel: it writes down what they are given and
 * launches nothing (no GPU needed). */
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

typedef struct {
    uint32_t x, y, z;
} dim3_t;

int hipFuncSetAttribute(const void* f, int attr, int value) {
    printf("limit %p %d %d\n", f, attr, value);
    return 0;
}

static dim3_t grid_, block_;
static size_t lds_;
static void* stream_;

int __hipPushCallConfiguration(dim3_t grid, dim3_t block, size_t lds, void* stream) {
    grid_ = grid;
    block_ = block;
    lds_ = lds;
    stream_ = stream;
    return 0;
}

int __hipPopCallConfiguration(dim3_t* grid, dim3_t* block, size_t* lds, void** stream) {
    *grid = grid_;
    *block = block_;
    *lds = lds_;
    *stream = stream_;
    return 0;
}

int hipLaunchKernel(const void* f, dim3_t grid, dim3_t block, void** args, size_t lds, void* stream) {
    (void)args;
    (void)stream;
    printf("launch %p %u %u %zu\n", f, grid.x, block.x, lds);
    fflush(stdout);
    return 0;
}

int hipGetLastError(void) { return 0; }
