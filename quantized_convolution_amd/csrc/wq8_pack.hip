// Packing of rows to codes with one scale a row or one for 32, 64 or 128
// columns, and back. Memory bounds all three: 8192 x 5120 bf16 unpacked take 21 us
// (6.0 TB/s), in groups of 32 columns 22.9 packed and 22.5 unpacked (5.5 TB/s), in
// f32 31.5 and 32.9 (6.7 and 6.4); 1001 x 2565 f32 in groups of 32 columns 4.6 and 5.3
// (2.8 and 2.4 TB/s, a third of it the launch).
#include "wq8_rms_fwd.h"

namespace wq8 {
namespace {

// The row and the vector in it of a thread, `across` vectors being a row: 32-bit
// division where all vectors are counted in 32 bits.
template <bool WIDE>
__device__ __forceinline__ void place(int b, int across, int64_t &row, int &vec) {
    if constexpr (WIDE) {
        const int64_t first = (int64_t)b * 256, r0 = first / across;
        const int at = (int)(first - r0 * across) + threadIdx.x, down = at / across;
        row = r0 + down;
        vec = at - down * across;
    } else {
        const uint32_t i = (uint32_t)b * 256 + threadIdx.x, r = i / (uint32_t)across;
        row = r;
        vec = (int)(i - r * across);
    }
}

// Groups: a thread has 8 columns, the 4, 8 or 16 threads of a group are
// neighbours in a wave. Rows of codes are whole lines, so groups start at
// multiples of their threads, and what stands behind the last column is written
// by threads of its own.
template <typename XT, int G, bool WIDE>
__global__ __launch_bounds__(256) void k_pack_groups(RowsGeo g, const XT *x, int8_t *codes, float *scales, int blocks) {
    int b;
    if (!block_number(blocks, b)) return;
    int64_t row;
    int vec;
    place<WIDE>(b, g.stride / kV, row, vec);
    const int c = vec * kV;
    const bool in = row < g.rows;  // whole groups are in or out
    const Vec<XT, kV> v = load_any<XT>(x + (in ? row : 0) * g.xs, c, g.C);
    float t[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) t[k] = to_f32(v.v[k]);
    uint32_t most = bits_of(largest(t));
    const auto step = [&](int other) { most = max(most, (uint32_t)other); };
    step(__builtin_amdgcn_update_dpp(0, (int)most, kDppXor1, 0xf, 0xf, true));
    step(__builtin_amdgcn_update_dpp(0, (int)most, kDppXor2, 0xf, 0xf, true));
    if constexpr (G >= 64) step(__builtin_amdgcn_update_dpp(0, (int)most, kDppXor7, 0xf, 0xf, true));
    if constexpr (G >= 128) step(__builtin_amdgcn_update_dpp(0, (int)most, kDppXor8, 0xf, 0xf, true));
    if (!in) return;
    const Coder code(most);
    store_codes(codes + row * g.stride + c, code.pack(t));
    if (c % G == 0 && c < g.C) scales[row * ((g.C + G - 1) / G) + c / G] = code.scale;
}

template <typename XT, bool WIDE>
__global__ __launch_bounds__(256) void k_unpack(RowsGeo g, const int8_t *codes, const float *scales, XT *x, int blocks) {
    int b;
    if (!block_number(blocks, b)) return;
    int64_t row;
    int vec;
    place<WIDE>(b, (g.C + kV - 1) / kV, row, vec);
    if (row >= g.rows) return;
    const int c = vec * kV;
    const uint64_t q = *(const uint64_t *)(codes + row * g.stride + c);
    const float scale = g.group ? scales[row * ((g.C + g.group - 1) / g.group) + c / g.group] : scales[row];
    Vec<XT, kV> v;
#pragma unroll
    for (int k = 0; k < kV; ++k) v.v[k] = from_f32<XT>((float)(int8_t)(q >> (8 * k)) * scale);
    store_cols<XT>(x + row * g.xs, c, g.C, v);
}

constexpr int64_t kWide = 1 << 23;  // blocks whose threads pass 31 bits

template <typename XT>
void unpack(const RowsGeo &g, const int8_t *codes, const float *scales, XT *x, hipStream_t st) {
    const int64_t blocks = ((int64_t)g.rows * ((g.C + kV - 1) / kV) + 255) / 256;
    const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(256), 0, st, g, codes, scales, x, (int)blocks);
    };
    if (blocks >= kWide) go(k_unpack<XT, true>);
    else go(k_unpack<XT, false>);
}

template <typename XT>
void pack_groups(const RowsGeo &g, const XT *x, int8_t *codes, float *scales, hipStream_t st) {
    const int64_t blocks = ((int64_t)g.rows * (g.stride / kV) + 255) / 256;
    const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(256), 0, st, g, x, codes, scales, (int)blocks);
    };
    const bool wide = blocks >= kWide;
    if (g.group == 32) wide ? go(k_pack_groups<XT, 32, true>) : go(k_pack_groups<XT, 32, false>);
    else if (g.group == 64) wide ? go(k_pack_groups<XT, 64, true>) : go(k_pack_groups<XT, 64, false>);
    else wide ? go(k_pack_groups<XT, 128, true>) : go(k_pack_groups<XT, 128, false>);
}

}  // namespace

wq8_status launch_pack_rows(const RowsGeo &g, wq8_dtype xdt, const void *x, int8_t *codes, float *scales, void *stream) {
    RmsPtrs p = {};
    p.x = x;
    p.codes = codes;
    p.scales = scales;
    if (xdt == WQ8_F32) run_rows<float, float, false>(g, p, (hipStream_t)stream);
    else run_rows<bf16_t, bf16_t, false>(g, p, (hipStream_t)stream);
    return check_launch("packing of rows");
}

wq8_status launch_pack_groups(const RowsGeo &g, wq8_dtype xdt, const void *x, int8_t *codes, float *scales, void *stream) {
    if (xdt == WQ8_F32) pack_groups<float>(g, (const float *)x, codes, scales, (hipStream_t)stream);
    else pack_groups<bf16_t>(g, (const bf16_t *)x, codes, scales, (hipStream_t)stream);
    return check_launch("packing of groups");
}

wq8_status launch_unpack(const RowsGeo &g, wq8_dtype xdt, const int8_t *codes, const float *scales, void *x, void *stream) {
    if (xdt == WQ8_F32) unpack<float>(g, codes, scales, (float *)x, (hipStream_t)stream);
    else unpack<bf16_t>(g, codes, scales, (bf16_t *)x, (hipStream_t)stream);
    return check_launch("unpacking");
}

}  // namespace wq8
