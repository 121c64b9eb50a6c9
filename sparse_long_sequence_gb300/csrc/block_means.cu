// The means of key blocks: mean[c] = sum of block c's keys below the length / their number,
// fp32 sums of bf16 keys, rounded to bf16 once.
//
// One warp a block: eight lanes hold a key row (16 bytes each), four rows a load, sixteen loads in
// flight; the four row groups are added in a fixed order.  Bound by HBM: every key is read once.  16 heads x 16384 keys take 5.0 us (34 MB; replayed,
// so that the L2 has a part of them), the block that one new key of 16 x 4 caches fell into 2.7 us: a launch and
// two dependent loads.
#include "selected.h"

namespace dfs {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;

// `per` blocks of each sequence and head are looked at: all, or the `recent` form's few.
__global__ void __launch_bounds__(kThreads)
block_means_kernel(const __nv_bfloat16* K, uint32_t units, uint32_t heads, int64_t m, int64_t nb, const int32_t* lengths,
                   int64_t recent, uint32_t per, __nv_bfloat16* means) {
    const int lane = threadIdx.x & 31;
    const uint32_t at = blockIdx.x * kWarps + (threadIdx.x >> 5), ul = at / per;
    if (ul >= units) return;
    const int64_t u = ul, b = ul / heads;
    const int64_t len = lengths ? min(max((int64_t)lengths[b], (int64_t)0), m) : m;
    const int64_t first = recent ? max(len - recent, (int64_t)0) / kBlockKeys : 0;
    const int64_t c = first + (at - ul * per), row0 = c * kBlockKeys;
    if (row0 >= len) return;
    const int rows = (int)min((int64_t)kBlockKeys, len - row0);
    const uint4* src = reinterpret_cast<const uint4*>(K + (u * m + row0) * kHeadDim) + lane;
    uint4 raw[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) raw[j] = 4 * j + (lane >> 3) < rows ? src[j * 32] : make_uint4(0, 0, 0, 0);
    float s[8];
#pragma unroll
    for (int f = 0; f < 8; ++f) s[f] = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            s[2 * f] += __uint_as_float(w[f] << 16);
            s[2 * f + 1] += __uint_as_float(w[f] & 0xffff0000u);
        }
    }
    uint32_t o[4];
#pragma unroll
    for (int f = 0; f < 8; ++f) {
        s[f] += __shfl_xor_sync(kFull, s[f], 8);
        s[f] += __shfl_xor_sync(kFull, s[f], 16);
        s[f] /= (float)rows;
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(s[2 * f], s[2 * f + 1]);
        o[f] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if (lane < 8) reinterpret_cast<uint4*>(means + (u * nb + c) * kHeadDim)[lane] = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace

int launch_block_means(const void* K, int64_t B, int64_t Hk, int64_t m, const int32_t* lengths, int64_t recent,
                       void* means, cudaStream_t stream) {
    const int64_t nb = (m + kBlockKeys - 1) / kBlockKeys;
    // the last `recent` keys lie in at most ceil((recent - 1) / 64) + 1 blocks
    int64_t per = nb;
    if (recent && recent < m) per = (recent + kBlockKeys - 2) / kBlockKeys + 1;
    if (per > nb) per = nb;
    const int64_t blocks = (B * Hk * per + kWarps - 1) / kWarps;
    if (B * Hk * per > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many key blocks");
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        block_means_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(static_cast<const __nv_bfloat16*>(K), (uint32_t)(B * Hk), (uint32_t)Hk, m, nb,
                                                                      lengths, recent, (uint32_t)per, static_cast<__nv_bfloat16*>(means));
    }
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "block_means_kernel");
}

}  // namespace dfs
