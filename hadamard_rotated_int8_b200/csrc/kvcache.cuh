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
//        A row whose rotation is not finite (NaN, infinities, sums past fp32's range): codes 0 and
//        a NaN as its scale, so that what is made of it is NaN and not a plausible number.
// read:  x = bf16(butterfly(code) * fp32(s * c)); the butterfly of whole numbers is exact in
//        fp32 (|sum| <= 128 * 128).
//
// Both are bound by memory: 2 D bytes of bf16 and D + 4 bytes of codes and scale per row.
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
    int64_t T, rows;        // rows = T * 2 * Hkv
    int64_t nslots;         // pages * page
    int32_t Hkv;
    int32_t page_shift;     // log2(page)
    int32_t group;          // min(group, D)
    float c_g;
};

// Row r = (t * 2 + which) * Hkv + h of the call.
struct KvRow {
    int64_t t;
    uint32_t h;
    bool is_v;
};

__device__ __forceinline__ KvRow kv_row(const KvParams &p, int64_t r)
{
    const uint32_t H2 = 2u * static_cast<uint32_t>(p.Hkv);
    KvRow k;
    uint32_t rem;
    if (r < (1ll << 31)) {   // 64-bit division is slow; nearly every call stays below
        k.t = static_cast<uint32_t>(r) / H2;
        rem = static_cast<uint32_t>(r) - static_cast<uint32_t>(k.t) * H2;
    } else {
        k.t = r / H2;
        rem = static_cast<uint32_t>(r - k.t * H2);
    }
    k.is_v = rem >= static_cast<uint32_t>(p.Hkv);
    k.h = k.is_v ? rem - static_cast<uint32_t>(p.Hkv) : rem;
    return k;
}

// Its bf16 row.
__device__ __forceinline__ uint16_t *kv_plain(const KvParams &p, const KvRow &k, int32_t D)
{
    return (k.is_v ? p.v + k.t * p.ldv : p.k + k.t * p.ldk) + static_cast<int64_t>(k.h) * D;
}

// Its row in the cache (-1: none).
__device__ __forceinline__ int64_t kv_held(const KvParams &p, const KvRow &k, int64_t slot)
{
    if (slot >= 0 && slot < p.nslots) {
        const int64_t id = slot >> p.page_shift;
        const int64_t off = slot & ((1ll << p.page_shift) - 1);
        return (((id * p.Hkv + k.h) * 2 + (k.is_v ? 1 : 0)) << p.page_shift) + off;
    }
    if (slot >= 0)
        atomicOr(&g_device_error, kDevIndex);
    return -1;
}

// The larger one, or NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max3_abs_nan(float m, float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
    return d;
}

// One row on LANES neighbouring lanes, E consecutive elements each, rotated over groups of g (a
// run-time power of two from 8 to E LANES) and quantized: the row quantizer's adds, divisions
// and roundings. Returns the codes, packed, and the row's stored scale.
template <int E, int LANES>
__device__ __forceinline__ void quant_row_lanes(float (&v)[E], int32_t g, float c_g, uint32_t lane,
                                                uint32_t (&codes)[E / 4], float &s)
{
    static_assert(E >= 8, "groups of 8 and more");
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        const float a = v[i], b = v[i + 1];
        v[i] = __fadd_rn(a, b);
        v[i + 1] = __fsub_rn(a, b);
    }
#pragma unroll
    for (int h = 2; h < E; h <<= 1)
        if (h < 8 || h < g) {
#pragma unroll
            for (int i = 0; i < E; i += 2)
                if ((i & h) == 0)
                    bfly2(v[i], v[i + 1], v[i + h], v[i + h + 1]);
        }
#pragma unroll
    for (int x = 1; x < LANES; x <<= 1)
        if (x * E < g) {
            const float sgn = (lane & x) ? -1.0f : 1.0f;
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const float p0 = __shfl_xor_sync(0xffffffffu, v[i], x), p1 = __shfl_xor_sync(0xffffffffu, v[i + 1], x);
                fma2(v[i], v[i + 1], v[i], v[i + 1], sgn, sgn, p0, p1);
            }
        }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < E; i += 2)
        m = max3_abs_nan(m, v[i], v[i + 1]);
#pragma unroll
    for (int x = 1; x < LANES; x <<= 1)
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, x));
    const float s_z = __fdiv_rn(m, 127.0f);
    const bool codes_0 = !(m > 0.0f && m < INFINITY);
    float s_q = s_z;
    if (s_z < kFastStep) {   // a tiny step: the same quotients, with both sides 2^64 times as large
        s_q = s_z * 0x1p64f;
        const float most = s_q * 127.0f;   // (a step rounded down may leave more than 127.5 steps)
#pragma unroll
        for (int i = 0; i < E; ++i)
            v[i] = fminf(fmaxf(v[i] * 0x1p64f, -most), most);
    }
    const float rcp = __frcp_rn(s_q);
#pragma unroll
    for (int c = 0; c < E / 8; ++c) {
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] = v[8 * c + i];
        const uint2 w = quant8(z, s_q, rcp, true);
        codes[2 * c] = codes_0 ? 0u : w.x;
        codes[2 * c + 1] = codes_0 ? 0u : w.y;
    }
    s = !codes_0 ? __fmul_rn(s_z, c_g) : m == 0.0f ? 0.0f : nanf("");
}

// A warp takes 8 consecutive (token, key or value, head) rows, four lanes a row, so that only
// the last two stages of the butterfly need shuffles; the next rows' elements are on their way
// during a row's arithmetic. About 600 instructions for 8 rows of 128, issued 59% of the time:
// 16400 tokens of 8 heads of 128 take 30 us where the bytes would take 15.5 (8 lanes a row: 32
// us).
constexpr int kWriteThreads = 256;

template <int D>
__global__ void __launch_bounds__(kWriteThreads, 3) kv_write_kernel(const KvParams p)
{
    constexpr int E = D / 4;
    grid_dependents_launch();
    grid_dependency_wait();
    const uint32_t lane = lane_id(), t = lane & 3u;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kWriteThreads / 32), step = warps * 8;
    int64_t row = (static_cast<int64_t>(blockIdx.x) * (kWriteThreads / 32) + (threadIdx.x >> 5)) * 8 + (lane >> 2);
    const int64_t tiles = (p.rows - (row - (lane >> 2)) + step - 1) / step;   // of this warp
    KvRow k, k_next = {};
    int64_t slot, slot_next = -1;
    uint4 raw[E / 8], raw_next[E / 8];
    auto fetch = [&] {   // nothing here waits for what it loads
        slot_next = -1;
#pragma unroll
        for (int i = 0; i < E / 8; ++i)
            raw_next[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < p.rows) {
            k_next = kv_row(p, row);
            slot_next = p.slots[k_next.t];
            const uint16_t *x = kv_plain(p, k_next, D) + t * E;
#pragma unroll
            for (int i = 0; i < E / 8; ++i)
                raw_next[i] = *reinterpret_cast<const uint4 *>(x + 8 * i);
        }
        row += step;
    };
    fetch();
    for (int64_t i = 0; i < tiles; ++i) {
        k = k_next, slot = slot_next;
#pragma unroll
        for (int c = 0; c < E / 8; ++c)
            raw[c] = raw_next[c];
        fetch();
        float v[E];
#pragma unroll
        for (int c = 0; c < E / 8; ++c) {
            const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                v[8 * c + 2 * u] = __uint_as_float(w[u] << 16);
                v[8 * c + 2 * u + 1] = __uint_as_float(w[u] & 0xffff0000u);
            }
        }
        uint32_t codes[E / 4];
        float s;
        quant_row_lanes<E, 4>(v, p.group, p.c_g, lane, codes, s);
        const int64_t crow = kv_held(p, k, slot);
        if (crow >= 0) {
#pragma unroll
            for (int c = 0; c < E / 4; c += 4)
                st_v4(p.codes + crow * D + t * E + 4 * c, codes[c], codes[c + 1], codes[c + 2], codes[c + 3]);
            if (t == 0u)
                p.scales[crow] = s;
        }
    }
}

// d += a * b^T, a 16 rows of 32 int8, b 8 rows of 32 int8, int32 sums.
__device__ __forceinline__ void mma_m16n8k32_s8(int32_t (&d)[4], uint32_t a0, uint32_t a1,
                                                uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
                 " {%8, %9}, {%0, %1, %2, %3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 or 4 bytes global -> shared without registers, zeros instead where `from` is null;
// completion by groups of this thread.
__device__ __forceinline__ void async_copy_16(uint32_t to, const void *from, const void *any)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from ? from : any), "r"(from ? 16u : 0u)
                 : "memory");
}
__device__ __forceinline__ void async_copy_4(uint32_t to, const void *from, const void *any)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from ? from : any), "r"(from ? 4u : 0u)
                 : "memory");
}

// The reader's butterfly is a product of whole numbers, exact in any order, so its five inner
// stages are int8 matrix instructions: a warp takes 16 tokens of a head, lane (q, t) has elements
// [8 t, 8 t + 8) of each 32 of rows q and q + 8, and the 32 x 32 block of signs (zeros between
// groups below 32) sits in 8 registers with its rows and columns in the order that gives the
// lane the same elements of the result. The stages at distance 32 and 64 add what the lane has.
// About 300 instructions for 2048 elements (in fp32 with shuffles: 900). What bounds it is the
// number of rows on their way, 128 bytes each from anywhere: every warp keeps kReadStages - 1
// tiles of 16 in flight through its own ring in shared memory. 100003 tokens of 8 heads of 128
// take 108 us, 5.8 TB/s; writing alone (a fill of the same bytes) takes 107. With the rows of a
// token, not of a head, side by side in a tile, and one block in four not resident: 155 us.
constexpr int kReadThreads = 128, kReadStages = 4;

template <int D>
__global__ void __launch_bounds__(kReadThreads, 4) kv_read_kernel(const KvParams p)
{
    constexpr int NG = D / 32, CH = D / 16, ST = kReadStages;
    // a stage: 16 rows at 128 bytes, 16-byte chunk c of row r at c ^ (r & 7); then 16 scales
    constexpr uint32_t STAGE = 16 * 128 + 64;
    __shared__ __align__(128) uint8_t ring[kReadThreads / 32][ST][STAGE];
    grid_dependents_launch();
    grid_dependency_wait();
    const uint32_t lane = lane_id(), q = lane >> 2, t = lane & 3u;
    const uint32_t mine = smem_u32(ring[threadIdx.x >> 5]);
    uint32_t sign[4][2];
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            sign[nb][u] = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t k = 8u * t + 4u * u + i, n = 8u * (q >> 1) + 2u * nb + (q & 1u);
                const uint32_t in_group = static_cast<uint32_t>(p.group - 1);
                const bool in = ((k ^ n) & ~in_group) == 0u;
                const uint32_t v = !in ? 0u : (__popc(k & n & in_group) & 1) ? 0xffu : 1u;
                sign[nb][u] |= v << (8 * i);
            }
        }
    // tile: (16 tokens, key or value, head)
    const int64_t ntiles = (p.T + 15) / 16 * (2 * p.Hkv);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kReadThreads / 32);
    int64_t tile = static_cast<int64_t>(blockIdx.x) * (kReadThreads / 32) + (threadIdx.x >> 5);
    // slot of token (lane & 15) of the next tile to be fetched
    auto slot_of = [&](int64_t tl) {
        const int64_t tok = kv_row(p, tl).t * 16 + (lane & 15u);
        return tok < p.T ? p.slots[tok] : -1ll;
    };
    int64_t fetch_tile = tile, slot = slot_of(tile);
    uint32_t fetch_stage = 0;
    auto fetch = [&] {
        const int64_t crow = kv_held(p, kv_row(p, fetch_tile), slot);
        const uint32_t at = mine + fetch_stage * STAGE;
        if (fetch_tile < ntiles) {
#pragma unroll
            for (int j = 0; j < CH / 2; ++j) {
                const uint32_t r = (lane / CH) + j * (32 / CH), c = lane % CH;
                const int64_t from = __shfl_sync(0xffffffffu, crow, static_cast<int>(r));
                async_copy_16(at + r * 128u + ((c ^ (r & 7u)) << 4), from >= 0 ? p.codes + from * D + c * 16 : nullptr, p.codes);
            }
            if (lane < 16)
                async_copy_4(at + 2048u + lane * 4u, crow >= 0 ? p.scales + crow : nullptr, p.scales);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        fetch_tile += warps;
        fetch_stage = (fetch_stage + 1u) % ST;
        slot = slot_of(fetch_tile);
    };
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i)
        fetch();
    uint32_t stage = 0;
#pragma unroll 1
    for (; tile < ntiles; tile += warps) {
        asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2) : "memory");
        __syncwarp();
        const uint32_t at = mine + stage * STAGE;
        stage = (stage + 1u) % ST;
        uint16_t *x[2];
        float s[2];
        uint2 raw[2][NG];
        KvRow k = kv_row(p, tile);
        k.t = k.t * 16 + q;
#pragma unroll
        for (int r = 0; r < 2; ++r, k.t += 8) {
            x[r] = k.t < p.T ? kv_plain(p, k, D) + t * 8 : nullptr;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s[r]) : "r"(at + 2048u + (q + 8u * r) * 4u) : "memory");
#pragma unroll
            for (int i = 0; i < NG; ++i)
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                             : "=r"(raw[r][i].x), "=r"(raw[r][i].y)
                             : "r"(at + (q + 8u * r) * 128u + (((2u * i + (t >> 1)) ^ q) << 4) + (t & 1u) * 8u)
                             : "memory");
        }
        __syncwarp();      // the stage that is fetched next has been read by every lane
        fetch();
        float v[2][NG][8];
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) {
                int32_t d[4] = {0, 0, 0, 0};
                mma_m16n8k32_s8(d, raw[0][i].x, raw[1][i].x, raw[0][i].y, raw[1][i].y, sign[nb][0], sign[nb][1]);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[c >> 1][i][2 * nb + (c & 1)] = static_cast<float>(d[c]);
            }
#pragma unroll
        for (int h = 1; h < NG; h <<= 1)
            if (p.group > 32 * h) {
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < NG; ++i)
                        if ((i & h) == 0) {
#pragma unroll
                            for (int c = 0; c < 8; c += 2)
                                bfly2(v[r][i][c], v[r][i][c + 1], v[r][i + h][c], v[r][i + h][c + 1]);
                        }
            }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float f = __fmul_rn(s[r], p.c_g);
            if (x[r] != nullptr) {
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const __nv_bfloat162 h2 = __floats2bfloat162_rn(v[r][i][2 * c] * f, v[r][i][2 * c + 1] * f);
                        w[c] = *reinterpret_cast<const uint32_t *>(&h2);
                    }
                    st_v4(x[r] + i * 32, w[0], w[1], w[2], w[3]);
                }
            }
        }
    }
}

} // namespace sdnq
