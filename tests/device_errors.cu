// Two kinds of report in one device error word; built and run by test_gpu_device_errors.py.
#include <cstdio>

#include "../weight_only_quantization_rtn_b200/csrc/embedding.cuh"

using namespace w4a16;

__global__ void report(int first, int second) {
    if (threadIdx.x == 0) {
        report_error(first);
        report_error(second);
    }
}

int main() {
    const int order[3][2] = {{kErrBadId, kErrMbarTimeout}, {kErrMbarTimeout, kErrBadId}, {kErrBadId, kErrBadId}};
    for (const auto& o : order) {
        int value = 0;
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess) return 2;
        report<<<1, 32>>>(o[0], o[1]);
        if (cudaMemcpyFromSymbol(&value, g_device_error, sizeof(int)) != cudaSuccess) return 2;
        if (value != (o[0] | o[1])) return std::printf("%d then %d left %d\n", o[0], o[1], value), 1;
    }
    return 0;
}
