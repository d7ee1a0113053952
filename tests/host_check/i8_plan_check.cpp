// Prints kernel, splits, whole tiles and workgroups of the 8-bit products m x n x k
// given as arguments, as planned for 256 CUs (tests/test_i8_plans.py).
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
    for (int i = 1; i + 2 < argc; i += 3) {
        const dspk::I8Plan p = dspk::i8_plan(atoi(argv[i + 1]), atoi(argv[i + 2]), atoi(argv[i]), true, 256);
        printf("%d %d %lld %lld\n", (int)p.kind, p.splits, (long long)p.whole, (long long)p.groups);
    }
    return 0;
}
