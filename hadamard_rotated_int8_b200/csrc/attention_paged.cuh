// Attention of new tokens over the paged, rotated int8 key/value cache (kvcache.cuh).
//
// Query i of a sequence with context length L and n new tokens sits at position
// p = L - n + i and sees the keys j <= p with (no window, or j > p - window, or j < sinks):
//   logit_j = (qc . kc_j) * (s_q * s_k[j]) * scale,  qc, s_q the row quantizer's codes of q,
//   o = butterfly(sum_j softmax(logit)_j * s_v[j] * vc_j) * c,  c = fp32(1/sqrt(G)).
// The rotation leaves q . k unchanged (it is orthogonal), so nothing is un-rotated before the
// softmax; the values' rotation is undone once per output row. A row that sees no key is 0.
#pragma once

#include <cuda_bf16.h>

#include "attention.cuh"
#include "device.cuh"
#include "rotquant.cuh"

namespace sdnq {

struct PagedParams {
    const uint16_t *q;       // [T][H][D] bf16, token stride ldq
    uint16_t *o;             // [T][H][D] bf16, token stride ldo
    int64_t ldq, ldo;
    const int32_t *cu;       // [B + 1] first query row of each sequence, or nullptr (row b is b's)
    const int32_t *lens;     // [B] context lengths, the new tokens included
    const int32_t *table;    // [B] rows of page ids, row stride table_ld
    int64_t table_ld;
    const int8_t *codes;
    const float *scales;
    int64_t pages;
    int32_t T, B, H, Hkv;
    int32_t share;           // H / Hkv
    int32_t page_shift;
    int32_t cap;             // most keys a table row can name
    int32_t window;          // <= 0: none
    int32_t sinks;
    int32_t group;           // min(group, D)
    float scale;
    float c_g;
};

// A sequence as the device arrays give it, made safe: rows [q0, q0 + n) lie in [0, T), the
// length lies in [0, cap]. What had to be changed is recorded in the device error word.
struct PagedSeq {
    int32_t q0, n, len;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams &p, int32_t b)
{
    PagedSeq s;
    s.q0 = b, s.n = 1;
    bool bad = false;
    if (p.cu != nullptr) {
        const int32_t a = p.cu[b], e = p.cu[b + 1];
        bad = a < 0 || e < a || e > p.T;
        s.q0 = bad ? 0 : a;
        s.n = bad ? 0 : e - a;
    }
    s.len = p.lens[b];
    if (s.len < 0 || s.len > p.cap) {
        bad = true;
        s.len = s.len < 0 ? 0 : p.cap;
    }
    if (bad)
        atomicOr(&g_device_error, kDevIndex);
    return s;
}

// The butterfly of one row held by a warp, lane l having the D / 32 elements from l * D / 32,
// over groups of g (a run-time power of two from 8 to D): the same adds in the same order as
// chunk_butterfly.
template <int E>
__device__ __forceinline__ void warp_butterfly(float (&v)[E], int32_t g, uint32_t lane)
{
#pragma unroll
    for (int h = 1; h < E; h <<= 1)
#pragma unroll
        for (int i = 0; i < E; ++i)
            if ((i & h) == 0) {
                const float a = v[i], b = v[i + h];
                v[i] = __fadd_rn(a, b);
                v[i + h] = __fsub_rn(a, b);
            }
#pragma unroll
    for (int x = 1; x < 32; x <<= 1)
        if (x * E < g) {
            const float sgn = (lane & x) ? -1.0f : 1.0f;
#pragma unroll
            for (int i = 0; i < E; ++i)
                v[i] = __fmaf_rn(v[i], sgn, __shfl_xor_sync(0xffffffffu, v[i], x));
        }
}

// Codes (packed little-endian) and scale of one row held by a warp as above.
template <int E>
__device__ __forceinline__ uint32_t warp_quant_row(float (&v)[E], int32_t g, float c_g,
                                                   uint32_t lane, float &s)
{
    warp_butterfly(v, g, lane);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i)
        m = fmaxf(m, fabsf(v[i]));
#pragma unroll
    for (int x = 1; x < 32; x <<= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    const float s_z = __fdiv_rn(m, 127.0f);
    const bool zero = !(m > 0.0f);
    uint32_t w = 0u;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float t = zero ? 0.0f : __fdiv_rn(v[i], s_z);
        const float r = fminf(fmaxf(rintf(t), -127.0f), 127.0f);
        const int32_t code = t == t ? __float2int_rn(r) : 0;
        w |= (static_cast<uint32_t>(code) & 0xffu) << (8 * i);
    }
    s = zero ? 0.0f : __fmul_rn(s_z, c_g);
    return w;
}

// One warp per (query row, head); a lane holds D / 32 elements of the row, and one key's dot
// product is reduced by shuffles.
template <int D>
__global__ void __launch_bounds__(128) attn_paged_kernel(const PagedParams p)
{
    constexpr int E = D / 32;
    grid_dependency_wait();
    const uint32_t lane = lane_id();
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (w >= static_cast<int64_t>(p.T) * p.H)
        return;
    const int32_t t = static_cast<int32_t>(w / p.H), h = static_cast<int32_t>(w - static_cast<int64_t>(t) * p.H);
    int32_t b = t;
    if (p.cu != nullptr) {   // the last sequence that starts at or before row t
        int32_t lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if (p.cu[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        b = lo;
    }
    if (b >= p.B)
        return;
    const PagedSeq sq = paged_seq(p, b);
    if (t < sq.q0 || t >= sq.q0 + sq.n)
        return;
    const int32_t pos = sq.len - sq.n + (t - sq.q0);
    float v[E];
    const uint16_t *qr = p.q + static_cast<int64_t>(t) * p.ldq + static_cast<int64_t>(h) * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i)
        v[i] = __uint_as_float(static_cast<uint32_t>(qr[i]) << 16);
    float s;
    const uint32_t qw = warp_quant_row<E>(v, p.group, p.c_g, lane, s);
    const float f = s * p.scale * 1.4426950408889634f;
    float m = -INFINITY, l = 0.0f, acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i)
        acc[i] = 0.0f;
    const int32_t kvh = h / p.share;
    const int32_t low = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    for (int32_t j = 0; j <= pos; ++j) {
        if (j < low && j >= p.sinks)
            j = low;
        const int32_t id = p.table[static_cast<int64_t>(b) * p.table_ld + (j >> p.page_shift)];
        if (id < 0 || id >= p.pages) {
            if (lane == 0)
                atomicOr(&g_device_error, kDevIndex);
            continue;
        }
        const int64_t krow = (((static_cast<int64_t>(id) * p.Hkv + kvh) * 2) << p.page_shift) +
                             (j & ((1 << p.page_shift) - 1));
        const int64_t vrow = krow + (1ll << p.page_shift);
        uint32_t kw, vw;
        if (E == 4) {
            kw = *reinterpret_cast<const uint32_t *>(p.codes + krow * D + lane * E);
            vw = *reinterpret_cast<const uint32_t *>(p.codes + vrow * D + lane * E);
        } else {
            kw = *reinterpret_cast<const uint16_t *>(p.codes + krow * D + lane * E);
            vw = *reinterpret_cast<const uint16_t *>(p.codes + vrow * D + lane * E);
        }
        int32_t dot = __dp4a(static_cast<int>(qw), static_cast<int>(kw), 0);
        dot = __reduce_add_sync(0xffffffffu, dot);
        const float y = static_cast<float>(dot) * p.scales[krow] * f;
        if (y > m) {
            const float a = ex2_approx(m - y);
            l *= a;
#pragma unroll
            for (int i = 0; i < E; ++i)
                acc[i] *= a;
            m = y;
        }
        const float e = ex2_approx(y - m);
        l += e;
        const float ev = e * p.scales[vrow];
#pragma unroll
        for (int i = 0; i < E; ++i)
            acc[i] = __fmaf_rn(ev, static_cast<float>(static_cast<int8_t>(vw >> (8 * i))), acc[i]);
    }
    warp_butterfly(acc, p.group, lane);
    const float inv = l > 0.0f ? p.c_g / l : 0.0f;
    uint16_t *orow = p.o + static_cast<int64_t>(t) * p.ldo + static_cast<int64_t>(h) * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const __nv_bfloat16 r = __float2bfloat16_rn(l > 0.0f ? acc[i] * inv : 0.0f);
        orow[i] = *reinterpret_cast<const uint16_t *>(&r);
    }
}

} // namespace sdnq
