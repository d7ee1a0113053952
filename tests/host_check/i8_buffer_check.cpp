// Prints, for 8-bit products m x n x k given as arguments, the splits of K and where their
// sums begin in the workspace, after a first line: the bytes in front that hold arrival
// counters of an expert layer or a product (tests/test_i8_one_buffer.py).
#include <stdio.h>
#include <stdlib.h>

#include <hip/hip_runtime_api.h>

#include "dspk.h"
#include "i8_internal.h"

namespace dspk {
int set_error(int code, const char *) { return code; }
int device_cus() { return 256; }
hipError_t launch_rows(RowOp, const RowArgs &, int, hipStream_t) { return hipSuccess; }
hipError_t launch_i8_read(const I8ReadArgs &, hipStream_t) { return hipSuccess; }
hipError_t launch_i8_pack(const I8PackArgs &, hipStream_t) { return hipSuccess; }
hipError_t launch_i8_gemm(const I8GemmArgs &, const I8Plan &, hipStream_t) { return hipSuccess; }
hipError_t launch_moe_route(const RouteArgs &, hipStream_t) { return hipSuccess; }
hipError_t launch_moe_mlp(const MoeArgs &, hipStream_t) { return hipSuccess; }
}  // namespace dspk
extern "C" const char *hipGetErrorString(hipError_t) { return "error"; }

int main(int argc, char **argv) {
    const size_t down = dspk::kMoeDown + 4 * dspk::kMoeSplitTiles, products = 4 * dspk::kI8MaxSplitTiles;
    printf("%zu\n", down > products ? down : products);
    for (int i = 1; i + 2 < argc; i += 3) {
        const dspk::I8Plan p = dspk::i8_plan(atoi(argv[i + 1]), atoi(argv[i + 2]), atoi(argv[i]), true, 256);
        printf("%d %zu\n", p.splits, p.off_part);
    }
    return 0;
}
