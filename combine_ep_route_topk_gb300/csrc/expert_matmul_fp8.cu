// Experts' products of E4M3 codes with a scale for every 128 columns, for sm_103a
// (ep_expert_matmul_fp8).
//
//   out[r, n] = sum over the blocks b of 128 K of
//               xs[s, b] * ws[e, n / 128, b] * sum_{k in b} x[s, k] * w[e, n, k]
//
// A tile of 32 rows x 64 channels a block, its operands as float32 in shared
// memory, one block of K at a time; sums are float32.
#include "expert_common.cuh"
#include "rows_common.cuh"

namespace ep {
namespace {

using namespace mm;

constexpr int kTileRows = 32, kTileChannels = 64, kThreads = 256, kPitch = kScaleBlock + 1;

struct Tiles {
    float x[kTileRows][kPitch];
    float w[kTileChannels][kPitch];
    int tiles[kTileGroups + 1];
    long long warp_sums[kTileGroups / 32];
};

__global__ void __launch_bounds__(kThreads) matmul_fp8_kernel(MatmulArgs a) {
    extern __shared__ uint8_t s_raw[];
    Tiles& sh = *reinterpret_cast<Tiles*>(s_raw);
    pdl_prologue();
    const int tid = threadIdx.x;
    if (a.status != nullptr && blockIdx.x == 0 && tid == 0) *a.status = 0;
    tile_prefix(a, kTileRows, sh.tiles, sh.warp_sums);
    const int kb_n = scale_blocks(a.Kd), ct = (a.Nc + kTileChannels - 1) / kTileChannels;
    const long long units = (long long)sh.tiles[kTileGroups] * ct;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int tile = (int)(u / ct), ch0 = (int)(u % ct) * kTileChannels;
        const ExpertTile t = expert_of_tile(a, kTileRows, sh.tiles, tile);
        const int first = (tile - t.first) * kTileRows, rows = min(kTileRows, t.rows - first);
        const int c = tid % 16, r = tid / 16;  // channels c + 16 i, rows r and r + 16
        float acc[2][4] = {};
        for (int kb = 0; kb < kb_n; ++kb) {
            const int len = min(kScaleBlock, a.Kd - kb * kScaleBlock);
            __syncthreads();
            for (int i = tid; i < (kTileRows + kTileChannels) * 8; i += kThreads) {
                const int line = i / 8, k = i % 8 * 16;
                float v[16] = {};
                if (line < kTileRows) {
                    const int src = line < rows && a.x_rows > 0 ? source_row(a, t.e, t.begin, first + line) : -1;
                    if (src >= 0 && k < len)
                        rows::decode16(*reinterpret_cast<const uint4*>(a.x + (size_t)src * a.Kd + kb * kScaleBlock + k),
                                       __ldg(a.x_scales + (size_t)src * kb_n + kb), v);
                    for (int j = 0; j < 16; ++j) sh.x[line][k + j] = v[j];
                } else {
                    const int ch = ch0 + line - kTileRows;
                    if (ch < a.Nc && k < len)
                        rows::decode16(*reinterpret_cast<const uint4*>(a.w + ((size_t)t.e * a.Nc + ch) * a.Kd + kb * kScaleBlock + k),
                                       __ldg(a.w_scales + ((size_t)t.e * scale_blocks(a.Nc) + ch / kScaleBlock) * kb_n + kb), v);
                    for (int j = 0; j < 16; ++j) sh.w[line - kTileRows][k + j] = v[j];
                }
            }
            __syncthreads();
            for (int k = 0; k < kScaleBlock; ++k) {
                const float x0 = sh.x[r][k], x1 = sh.x[r + 16][k];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = sh.w[c + 16 * i][k];
                    acc[0][i] = fmaf(x0, w, acc[0][i]);
                    acc[1][i] = fmaf(x1, w, acc[1][i]);
                }
            }
        }
        const size_t to = first_row(a, t.e, t.begin) + first;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = r + 16 * h, ch = ch0 + c + 16 * i;
                if (row < rows && ch < a.Nc) {
                    const size_t at = (to + row) * a.Nc + ch;
                    if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(acc[h][i]);
                    else static_cast<float*>(a.out)[at] = acc[h][i];
                }
            }
    }
}

}  // namespace

cudaError_t launch_expert_matmul_fp8(const MatmulArgs& a, cudaStream_t s) {
    if (a.rows == 0)
        return a.status != nullptr ? cudaMemsetAsync(a.status, 0, sizeof(int32_t), s) : cudaSuccess;
    cudaError_t err = cudaFuncSetAttribute(matmul_fp8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Tiles));
    if (err != cudaSuccess) return err;
    err = launch(matmul_fp8_kernel, dim3(sm_count() * 4), dim3(kThreads), sizeof(Tiles), s, a);
    note_launch();
    return err;
}

}  // namespace ep
