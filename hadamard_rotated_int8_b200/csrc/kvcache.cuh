// The paged key/value cache in rotated int8: rows of new tokens quantized as they are written
// into their pages, and stored rows read back as bf16.
//
// Layout: codes [pages][Hkv][2][page][D] int8 (2: keys, then values) and scales
// [pages][Hkv][2][page] fp32, so that one (page, kv head) is one contiguous block that holds
// its keys and its values, and a copy engine fetches both with one box. A slot is
// page_id * page + offset.
//
// write: z = butterfly of the row over groups of G = min(group, D), s_z = fp32(amax / 127),
//        code = clamp(rne(fp32(z / s_z))), stored scale s = fp32(s_z * c), c = fp32(1/sqrt(G)):
//        the row quantizer of the linear path, so that z * c ~= s * code.
// read:  x = bf16(butterfly(code) * fp32(s * c)); the butterfly of whole numbers is exact in
//        fp32 (|sum| <= 128 * 128).
//
// Both are bound by memory: 2 D bytes of bf16 and D + 4 bytes of codes and scale per row. One
// warp takes 1024 elements = 1024 / D consecutive (token, key-or-value, head) rows at a time
// with the lane mapping of the rotate+quantize kernel (four 16-byte vectors a lane in flight,
// fully used 128-byte lines); a row's maximum combines its 8 lanes by shuffles.
#pragma once

#include "device.cuh"
#include "rotquant.cuh"

namespace sdnq {

struct KvParams {
    uint16_t *k, *v;        // [T][Hkv][D] bf16, token strides ldk, ldv (read by the writer)
    int64_t ldk, ldv;
    const int64_t *slots;   // [T]; negative: the token has no slot
    int8_t *codes;
    float *scales;
    int64_t rows;           // T * 2 * Hkv
    int64_t nslots;         // pages * page
    int32_t Hkv;
    int32_t page_shift;     // log2(page)
    float c_g;
};

// Where row r = (t * 2 + which) * Hkv + h lives: the bf16 row and the cache row (-1: none).
__device__ __forceinline__ void kv_locate(const KvParams &p, int64_t r, int32_t D,
                                          uint16_t *&x, int64_t &cache_row)
{
    const uint32_t H2 = 2u * static_cast<uint32_t>(p.Hkv);
    int64_t t;
    uint32_t rem;
    if (r < (1ll << 31)) {   // 64-bit division is slow; nearly every call stays below
        t = static_cast<uint32_t>(r) / H2;
        rem = static_cast<uint32_t>(r) - static_cast<uint32_t>(t) * H2;
    } else {
        t = r / H2;
        rem = static_cast<uint32_t>(r - t * H2);
    }
    const bool is_v = rem >= static_cast<uint32_t>(p.Hkv);
    const uint32_t h = is_v ? rem - static_cast<uint32_t>(p.Hkv) : rem;
    x = (is_v ? p.v + t * p.ldv : p.k + t * p.ldk) + static_cast<int64_t>(h) * D;
    const int64_t slot = p.slots[t];
    cache_row = -1;
    if (slot >= 0 && slot < p.nslots) {
        const int64_t id = slot >> p.page_shift;
        const int64_t off = slot & ((1ll << p.page_shift) - 1);
        cache_row = (((id * p.Hkv + h) * 2 + (is_v ? 1 : 0)) << p.page_shift) + off;
    } else if (slot >= 0) {
        atomicOr(&g_device_error, kDevIndex);
    }
}

template <int G, int D>
__global__ void __launch_bounds__(256, 4) kv_write_kernel(const KvParams p)
{
    static_assert(D == 64 || D == 128, "head sizes of the cache");
    constexpr int RPL = 256 / D;        // rows of a lane: 2 (D = 128) or 4 (D = 64)
    constexpr int VPR = 4 / RPL;        // 64-element vectors of a row
    grid_dependents_launch();
    grid_dependency_wait();
    const uint32_t lane = lane_id();
    const int64_t nchunks = (p.rows + 4 * RPL - 1) / (4 * RPL);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    for (int64_t c = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
         c < nchunks; c += warps) {
        const int64_t row0 = c * (4 * RPL) + static_cast<int64_t>(lane >> 3) * RPL;
        int64_t crow[RPL];
        uint4 raw[4];
#pragma unroll
        for (int r = 0; r < RPL; ++r) {
            uint16_t *x = nullptr;
            crow[r] = -1;
            if (row0 + r < p.rows)
                kv_locate(p, row0 + r, D, x, crow[r]);
#pragma unroll
            for (int u = 0; u < VPR; ++u)
                raw[r * VPR + u] = crow[r] >= 0 ? ld_nc_v4(x + u * 64 + (lane & 7u) * 8)
                                                : make_uint4(0u, 0u, 0u, 0u);
        }
        float v[4][8];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            bf16x8_to_f32(raw[t], v[t]);
        chunk_butterfly<G>(v, lane);
#pragma unroll
        for (int r = 0; r < RPL; ++r) {
            float m = 0.0f;
#pragma unroll
            for (int u = 0; u < VPR; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    m = fmaxf(m, fabsf(v[r * VPR + u][i]));
#pragma unroll
            for (int off = 1; off < 8; off <<= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            const float s_z = __fdiv_rn(m, 127.0f);
            const bool zero = !(m > 0.0f);
            const bool fast = s_z >= 0x1p-126f;
            const float rcp = __frcp_rn(s_z);
            if (crow[r] >= 0) {
#pragma unroll
                for (int u = 0; u < VPR; ++u) {
                    uint2 w = make_uint2(0u, 0u);
                    if (!zero)
                        w = quant8(v[r * VPR + u], s_z, rcp, fast);
                    st_v2(p.codes + crow[r] * D + u * 64 + (lane & 7u) * 8, w.x, w.y);
                }
                if ((lane & 7u) == 0u)
                    p.scales[crow[r]] = zero ? 0.0f : __fmul_rn(s_z, p.c_g);
            }
        }
    }
}

template <int G, int D>
__global__ void __launch_bounds__(256, 4) kv_read_kernel(const KvParams p)
{
    constexpr int RPL = 256 / D, VPR = 4 / RPL;
    grid_dependents_launch();
    grid_dependency_wait();
    const uint32_t lane = lane_id();
    const int64_t nchunks = (p.rows + 4 * RPL - 1) / (4 * RPL);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    for (int64_t c = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
         c < nchunks; c += warps) {
        const int64_t row0 = c * (4 * RPL) + static_cast<int64_t>(lane >> 3) * RPL;
        uint16_t *x[RPL];
        float s[RPL];
        uint2 raw[4];
#pragma unroll
        for (int r = 0; r < RPL; ++r) {
            int64_t crow = -1;
            x[r] = nullptr;
            if (row0 + r < p.rows)
                kv_locate(p, row0 + r, D, x[r], crow);
            s[r] = 0.0f;   // no slot: zeros
            if (crow >= 0)
                s[r] = p.scales[crow];
#pragma unroll
            for (int u = 0; u < VPR; ++u) {
                raw[r * VPR + u] = make_uint2(0u, 0u);
                if (crow >= 0)
                    raw[r * VPR + u] = *reinterpret_cast<const uint2 *>(
                        p.codes + crow * D + u * 64 + (lane & 7u) * 8);
            }
        }
        float v[4][8];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t w = i < 4 ? raw[t].x : raw[t].y;
                v[t][i] = static_cast<float>(static_cast<int8_t>(w >> (8 * (i & 3))));
            }
        chunk_butterfly<G>(v, lane);
#pragma unroll
        for (int r = 0; r < RPL; ++r) {
            const float f = __fmul_rn(s[r], p.c_g);
            if (row0 + r < p.rows) {
#pragma unroll
                for (int u = 0; u < VPR; ++u) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 h2 =
                            __floats2bfloat162_rn(v[r * VPR + u][2 * i] * f, v[r * VPR + u][2 * i + 1] * f);
                        w[i] = *reinterpret_cast<const uint32_t *>(&h2);
                    }
                    st_v4(x[r] + u * 64 + (lane & 7u) * 8, w[0], w[1], w[2], w[3]);
                }
            }
        }
    }
}

} // namespace sdnq
