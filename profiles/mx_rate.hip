// Rates of the matrix instructions from registers, the floor of the operations of a product: 512
// workgroups of 8 waves, two to a unit's SIMD, 16 sums a wave, no loads.
//
//   hipcc --offload-arch=gfx950 -O3 -std=c++17 -Xclang -target-feature -Xclang -packed-fp32-ops \
//         profiles/mx_rate.hip -o /tmp/mx_rate && /tmp/mx_rate
#include <hip/hip_runtime.h>
#include <stdio.h>

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512, kGroups = 512, kSums = 16, kSteps = 3000;

// FP4: 4-bit codes of many values with scales of some powers of two; else bf16. Operands of zeros
// draw less power and run faster, so these are not.
template <bool FP4>
__global__ __launch_bounds__(kThreads) void k_rate(float *out) {
    const int l = threadIdx.x;
    const v8i a = {l * 0x1234567 + 77, l * 0x7654321 + 31, l * 0x3141592 + 13, l * 0x2718281 + 7, 0, 0, 0, 0};
    const v8i b = {l * 0x1618033 + 3, l * 0x1414213 + 5, l * 0x1732050 + 11, l * 0x2236067 + 17, 0, 0, 0, 0};
    v8bf x, y;
    for (int i = 0; i < 8; ++i) {
        x[i] = (__bf16)(0.37f * (float)((l * 7 + i) % 61 - 30));
        y[i] = (__bf16)(0.11f * (float)((l * 5 + i) % 53 - 26));
    }
    const int scale = 120 + (l & 7);
    v4f c[kSums];
    for (int i = 0; i < kSums; ++i) c[i] = v4f{0, 0, 0, 0};
    for (int t = 0; t < kSteps; ++t) {
#pragma unroll
        for (int i = 0; i < kSums; ++i) {
            if constexpr (FP4)
                c[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c[i], 4, 4, 0, scale, 0, scale);
            else
                c[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c[i], 0, 0, 0);
        }
    }
    float z = 0;
    for (int i = 0; i < kSums; ++i) z += c[i][0] + c[i][1] + c[i][2] + c[i][3];
    out[blockIdx.x * kThreads + l] = z;
}

template <bool FP4>
int rate(const char *name, float *out) {
    const double flops = 2.0 * 16 * 16 * (FP4 ? 128 : 32) * kSums * kSteps * kGroups * (kThreads / 64);
    hipEvent_t begin, end;
    if (hipEventCreate(&begin) != hipSuccess || hipEventCreate(&end) != hipSuccess) return 1;
    float least = 1e30f;
    for (int r = 0; r < 40; ++r) {  // the clock takes some of them to rise
        float ms = 0;
        if (hipEventRecord(begin, 0) != hipSuccess) return 1;
        hipLaunchKernelGGL((k_rate<FP4>), dim3(kGroups), dim3(kThreads), 0, 0, out);
        if (hipGetLastError() != hipSuccess || hipEventRecord(end, 0) != hipSuccess ||
            hipEventSynchronize(end) != hipSuccess || hipEventElapsedTime(&ms, begin, end) != hipSuccess)
            return 1;
        least = ms < least ? ms : least;
    }
    printf("%s: %.2f PFLOP/s\n", name, flops / least / 1e12);
    return 0;
}

int main() {
    float *out = nullptr;
    if (hipMalloc(&out, sizeof(float) * kGroups * kThreads) != hipSuccess) return 1;
    return rate<true>("4 bits, scaled, 16x16x128", out) || rate<false>("bf16, 16x16x32", out);
}
