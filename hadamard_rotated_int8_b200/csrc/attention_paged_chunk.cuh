// Attention of many query rows (chunks of prompts) over the paged cache, on the
// 5th-generation tensor cores. The mathematics and the work split are attention_paged.cuh's.
//
// One persistent block per SM, 256 query rows of one kv head at a time (two tiles of 128 that
// share every key and value), keys in steps of 64:
// - warp 0 streams keys, values and scales page by page through TMA rings;
// - warps 2 and 3 turn each step's value codes into bf16 (times 2^-6, exact), the
//   128-byte-swizzled operand of the second product;
// - warp 1 issues S_t = Q_t K^T (tcgen05 kind::i8, int32 in TMEM) three steps ahead of
//   O_t += P_t V (kind::f16, fp32 in TMEM): logits and P of a tile have two buffers each, so
//   that its softmax never waits for a product just issued. A commit costs the issuing warp
//   about 200 cycles and a wait 110 or more, so there is one commit a tile and step, and one
//   that frees V(k - 3): `done` of iteration k covers S(k) and P(k - 3) V(k - 3), and the rest
//   follows from the softmax's "P(k - 3) written": S(k - 2) is done with K(k - 2) and has been
//   read, and so have the scales of step k - 3;
// - warps 4..7 (tile 0) and 8..11 (tile 1), one thread a query row, rotate and quantize their
//   query rows into the operand tile, then per step form 64 base-2 logits, an online softmax
//   (sums rescaled only when the maximum grows by more than 8), and P = probability * s_v in
//   bf16. At the end of a segment the rotation is undone in registers.
// Code size matters: the roles share one instruction cache, and a loop body that overflows it
// runs several times slower; so the loops are small, rolled where they can be, and the masks'
// instructions are kept off the path of wholly visible steps.
// 2048 tokens over 16384 keys, 32 heads over 8 of 128: 590 us in this kernel, 870 TFLOP/s of
// products, half of them int8 (floor 233 us). A step of 64 keys takes 2600 cycles; its exponentials
// need 1024, its products 900 and its instructions about 1600 issue cycles a scheduler.
#pragma once

#include "attention_paged.cuh"

namespace sdnq {

constexpr int kChunkTile = 64;      // keys per step
constexpr int kChunkRows = 256;     // query rows of a segment: two tiles of 128
constexpr int kChunkThreads = 384;

template <int D>
struct ChunkConfig {
    static constexpr int NK = 4, NV = 3, NB = 4, NS = 8;   // stages: K, value codes, bf16 values, scales
    static constexpr int Q_TILE = 128 * D, K_STAGE = 64 * D, V_STAGE = 64 * D, B_STAGE = 64 * D * 2;
    static constexpr int P_BUF = 128 * 64 * 2;
    static constexpr int Q_OFF = 0;
    static constexpr int P_OFF = Q_OFF + 2 * Q_TILE;        // [2 tiles][2 buffers]
    static constexpr int K_OFF = P_OFF + 4 * P_BUF;
    static constexpr int B_OFF = K_OFF + NK * K_STAGE;
    static constexpr int V_OFF = B_OFF + NB * B_STAGE;
    static constexpr int SC_OFF = V_OFF + NV * V_STAGE;     // 64 key scales, 64 value scales a stage
    static constexpr int QS_OFF = SC_OFF + NS * 512;        // query scales
    static constexpr int BAR_OFF = QS_OFF + kChunkRows * 4;
    // full and empty of each ring, then per tile and buffer done and p_full; q_full; drain
    static constexpr int NBARS = 2 * (NK + NV + NB) + 8 + 2 + 1;
    static constexpr int META_OFF = BAR_OFF + NBARS * 8;    // valid boxes of each scale stage
    static constexpr int HOLD_OFF = META_OFF + NS * 4;      // TMEM address, abort flag, scan result
    static constexpr int SMEM_BYTES = 1024 + HOLD_OFF + 48;
    static_assert((NK & (NK - 1)) == 0 && (NB & (NB - 1)) == 0, "ring positions are masked");
    // step h is loaded once P(h - NK - 1) is written, so that step h - NS - 1 and older are read
    static_assert(NS >= NK + 2 && (NS & (NS - 1)) == 0, "the scales need no barriers of their own");
    static constexpr int64_t PIECE = static_cast<int64_t>(kChunkRows) * (D + 2);   // floats, as FewConfig's
    static_assert(SMEM_BYTES + 256 <= 232448, "shared memory per block");
};

// K-major int8 operand of D bytes a row: 128-byte rows in the 128-byte swizzle, or 64-byte rows
// in the 64-byte swizzle (layout type 4), 8-row groups 8 D bytes apart.
template <int D>
__device__ __forceinline__ uint64_t codes_desc(uint32_t saddr)
{
    if (D == 128)
        return kmajor_desc(saddr);
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1u) << 16;
    d |= static_cast<uint64_t>(512u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(4u) << 61;
    return d;
}

// The butterfly of a row of D values in one thread's registers, groups of g (a power of two
// from 8 to D).
template <int D>
__device__ __forceinline__ void thread_butterfly(float (&v)[D], int32_t g)
{
#pragma unroll
    for (int i = 0; i < D; i += 2) {
        const float a = v[i], b = v[i + 1];
        v[i] = __fadd_rn(a, b);
        v[i + 1] = __fsub_rn(a, b);
    }
#pragma unroll
    for (int h = 2; h < D; h <<= 1)
        if (h < 8 || h < g) {
#pragma unroll
            for (int i = 0; i < D; i += 2)
                if ((i & h) == 0)
                    bfly2(v[i], v[i + 1], v[i + h], v[i + h + 1]);
        }
}

// The value operand holds codes times 2^-6: with u = code + 128, the bf16 pattern 0x00uu is u 2^-133
// (subnormal numbers and the first binade have one spacing), so one fused multiply-add gives
// u 2^-6 - 2, exactly.
constexpr float kCodeUnit = 64.0f;

// True in one lane of the warp (all lanes call it).
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0u;
}

// Bits [from, to) of the 32 that begin at bit `at`.
__device__ __forceinline__ uint32_t bit_range(int32_t from, int32_t to, int32_t at)
{
    const int32_t a = min(max(from - at, 0), 32), b = min(max(to - at, 0), 32);
    const uint32_t below_b = b == 32 ? 0xffffffffu : (1u << b) - 1u, below_a = a == 32 ? 0xffffffffu : (1u << a) - 1u;
    return below_b & ~below_a;
}

template <int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
    attn_chunk_kernel(const __grid_constant__ CUtensorMap tmPool, const PagedParams p)
{
    using C = ChunkConfig<D>;
    constexpr int NK = C::NK, NV = C::NV, NB = C::NB, NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    const uint32_t bar0 = base + C::BAR_OFF;
    auto k_full = [&](uint32_t s) { return bar0 + 8u * s; };
    auto k_empty = [&](uint32_t s) { return bar0 + 8u * (NK + s); };
    auto v_full = [&](uint32_t s) { return bar0 + 8u * (2 * NK + s); };
    auto v_empty = [&](uint32_t s) { return bar0 + 8u * (2 * NK + NV + s); };
    auto b_full = [&](uint32_t s) { return bar0 + 8u * (2 * (NK + NV) + s); };
    auto b_empty = [&](uint32_t s) { return bar0 + 8u * (2 * (NK + NV) + NB + s); };
    // per tile t and buffer b: iteration done, P written (one phase every other step)
    constexpr int TB = 2 * (NK + NV + NB);
    auto done = [&](uint32_t t, uint32_t b) { return bar0 + 8u * (TB + 2 * t + b); };
    auto p_full = [&](uint32_t t, uint32_t b) { return bar0 + 8u * (TB + 4 + 2 * t + b); };
    auto q_full = [&](uint32_t t) { return bar0 + 8u * (TB + 8 + t); };
    const uint32_t drain_bar = bar0 + 8u * (TB + 10);
    volatile uint32_t *meta = reinterpret_cast<volatile uint32_t *>(smem + C::META_OFF);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::HOLD_OFF);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_holder + 1);
    float *qs = reinterpret_cast<float *>(smem + C::QS_OFF);
    const uint32_t warp = threadIdx.x >> 5, lane = lane_id();

    if (threadIdx.x == 0) {
        for (int s = 0; s < NK; ++s)
            mbar_init(k_full(s), 1), mbar_init(k_empty(s), 1);
        for (int s = 0; s < NV; ++s)
            mbar_init(v_full(s), 1), mbar_init(v_empty(s), 2);
        for (int s = 0; s < NB; ++s)
            mbar_init(b_full(s), 2), mbar_init(b_empty(s), 1);
        for (int t = 0; t < 2; ++t) {
            for (int b = 0; b < 2; ++b)
                mbar_init(done(t, b), 2), mbar_init(p_full(t, b), 4);
            mbar_init(q_full(t), 4);
        }
        mbar_init(drain_bar, 1);
        *abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmPool);
    }
    grid_dependents_launch();
    grid_dependency_wait();
    int64_t first, per, total;
    PagedWalk w;
    find_share<kChunkTile, kChunkRows, kChunkThreads>(p, gridDim.x, p.least_tiles,
                                                      reinterpret_cast<int32_t *>(tmem_holder + 2), first, per,
                                                      total, w);   // also: barriers initialised
    FewDesc *desc = reinterpret_cast<FewDesc *>(p.desc) + blockIdx.x;
    if (first >= total) {
        if (threadIdx.x == 0)
            desc->pieces = 0;
        return;
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_holder), 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;
    const int64_t count = min(first + per, total) - first;
    const int32_t pp_shift = min(p.page_shift, 6), pp = 1 << pp_shift;   // keys of a box
    const int32_t nbox_shift = 6 - pp_shift, nbox = 1 << nbox_shift;
    const uint32_t all_boxes = (1u << nbox) - 1u;
    auto piece_steps = [&](int64_t n) { return static_cast<int32_t>(min(static_cast<int64_t>(w.t.nt - w.i), count - n)); };
    auto piece_rows = [&] { return min(kChunkRows, w.s.n * p.share - w.q * kChunkRows); };
    // A role that gave up waiting raises `abort` and runs its loops to their end without waiting (the
    // loader stops loading); from then on no output row is stored, and pieces are marked as lost.
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok && !mbar_try_wait(bar, parity))
            ok = mbar_wait_tries(bar, parity, abort);
        __syncwarp();
    };
    auto wait2 = [&](uint32_t bar, uint32_t parity, uint32_t bar2, uint32_t parity2) {   // the tries overlap
        const bool a = mbar_try_wait(bar, parity), b = mbar_try_wait(bar2, parity2);
        if (ok && !a)
            ok = mbar_wait_tries(bar, parity, abort);
        if (ok && !b)
            ok = mbar_wait_tries(bar2, parity2, abort);
        __syncwarp();
    };

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        fence_proxy_async_global();   // the kernel before may have stored the rows that the copies read
        uint32_t ks = 0, kph = 1, vs = 0, vph = 1, ss = 0;
        int64_t n = 0, issued = 0;
        while (ok && n < count) {
            const int32_t steps = piece_steps(n);
            const int32_t *row = p.table + static_cast<int64_t>(w.b) * p.table_ld;
            const PagedReach reach = paged_reach<kChunkRows>(p, w.s.n, w.s.len, w.q);
            // Page ids are read 32 at a time, a batch ahead of their use; entry e is box
            // e % nbox of the piece's step e / nbox. Boxes that no row sees stay out.
            auto fetch = [&](int32_t e0) {
                const int32_t e = e0 + static_cast<int32_t>(lane);
                const int32_t i = w.i + (e >> nbox_shift);
                if (i >= w.i + steps)
                    return -1;
                const int32_t j = (i < w.t.ns ? i : w.t.w0 + i - w.t.ns) * kChunkTile + ((e & (nbox - 1)) << pp_shift);
                if (!reach.any(p, j, pp))
                    return -1;
                const int32_t id = row[j >> p.page_shift];
                if (id < 0 || id >= p.pages) {
                    atomicOr(&g_device_error, kDevIndex);
                    return -1;
                }
                return id;
            };
            int32_t ids = -1, ids_next = -1;
#pragma unroll 1
            for (int32_t k = 0; k < steps; ++k) {
                const int32_t at = (k << nbox_shift) & 31;
                if (at == 0) {
                    ids = k == 0 ? fetch(0) : ids_next;
                    ids_next = fetch((k << nbox_shift) + 32);
                }
                // lane c < nbox has box c of this step
                const int32_t id = __shfl_sync(0xffffffffu, ids, (at + static_cast<int32_t>(lane)) & 31);
                const bool mine = static_cast<int32_t>(lane) < nbox && id >= 0;
                const uint32_t valid = __ballot_sync(0xffffffffu, mine);
                const uint32_t keys = static_cast<uint32_t>(__popc(valid)) << pp_shift;
                const int32_t i = w.i + k;
                const int32_t j = (i < w.t.ns ? i : w.t.w0 + i - w.t.ns) * kChunkTile + (static_cast<int32_t>(lane) << pp_shift);
                const int32_t krow = mine ? static_cast<int32_t>(((static_cast<int64_t>(id) * p.Hkv + w.kvh) * 2) << p.page_shift) +
                                                (j & ((1 << p.page_shift) - 1))
                                          : 0;
                const int32_t vrow = krow + (1 << p.page_shift);
                wait2(k_empty(ks), kph, v_empty(vs), vph);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                if (lane == 0) {
                    meta[ss] = valid;
                    mbar_arrive_expect_tx(k_full(ks), keys * (D + 8u));
                    mbar_arrive_expect_tx(v_full(vs), keys * D);
                }
                __syncwarp();
                ++issued;
                if (mine) {
                    tma_load_2d(base + C::K_OFF + ks * C::K_STAGE + lane * pp * D, &tmPool, k_full(ks), 0, krow);
                    const uint32_t sdst = base + C::SC_OFF + ss * 512u + lane * pp * 4u;
                    bulk_load_1d(sdst, p.scales + krow, 4u * pp, k_full(ks));
                    bulk_load_1d(sdst + 256u, p.scales + vrow, 4u * pp, k_full(ks));
                    tma_load_2d(base + C::V_OFF + vs * C::V_STAGE + lane * pp * D, &tmPool, v_full(vs), 0, vrow);
                }
                ss = (ss + 1u) % NS;
                if (++ks == NK)
                    ks = 0, kph ^= 1u;
                if (++vs == NV)
                    vs = 0, vph ^= 1u;
            }
            n += steps;
            if (n < count)
                walk_next_segment<kChunkTile, kChunkRows>(p, w);
        }
        // every copy has landed before the block may end
        ok = true;
        auto drain = [&](uint32_t bar, int stages) {
            for (int64_t j = issued - stages < 0 ? 0 : issued - stages; j < issued; ++j)
                mbar_wait_tries(bar + 8u * static_cast<uint32_t>(j % stages), static_cast<uint32_t>(j / stages) & 1u, abort);
        };
        drain(k_full(0), NK);
        drain(v_full(0), NV);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issue
        // One thread's work. What an iteration waits for is tried at once: a ready barrier takes 110
        // cycles and more to say so.
        if (elect_one()) {
            constexpr uint32_t IDESC_S = idesc_s8_s32(128, 64);
            constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, true);
            // operand descriptors; 16 bytes further on is 1 more
            const uint64_t dq = codes_desc<D>(base + C::Q_OFF), dk = codes_desc<D>(base + C::K_OFF);
            const uint64_t dp = kmajor_desc(base + C::P_OFF), db = mnmajor_desc(base + C::B_OFF, 8192);
            // steps of all pieces so far, and of each tile's pieces
            uint32_t c0 = 0, g0 = 0, g1 = 0;
            int64_t n = 0;
            auto need = [&](bool got, uint32_t bar, uint32_t parity) {
                if (ok && !got)
                    ok = mbar_wait_tries(bar, parity, abort);
            };
            while (n < count) {
                const int32_t steps = piece_steps(n);
                const bool two = piece_rows() > 128;
                auto issue = [&](uint32_t t, uint32_t b, uint32_t ks, uint32_t bs, bool s_now, bool pv_now, bool pv_first) {
                    const uint64_t qa = dq + t * (C::Q_TILE >> 4), ka = dk + ks * (C::K_STAGE >> 4);
                    const uint64_t pa = dp + (2 * t + (b ^ 1u)) * (C::P_BUF >> 4), va = db + bs * (C::B_STAGE >> 4);
                    if (s_now) {
#pragma unroll
                        for (int kk = 0; kk < D / 32; ++kk)
                            mma_s8(tmem_base + t * 128 + b * 64, qa + 2 * kk, ka + 2 * kk, IDESC_S, kk != 0 ? 1u : 0u);
                    }
                    if (pv_now) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f16(tmem_base + 256 + t * 128, pa + 2 * kk, va + 128 * kk, IDESC_PV, !pv_first || kk != 0 ? 1u : 0u);
                    }
                    tc_commit(done(t, b));
                    // The commit speaks of the products only. This arrival (a release) hands on what the
                    // waits above acquired: step k's scales and mask, which the softmax reads. (It cannot
                    // stand in for an earlier iteration's commit: what iteration k waits for, P(k - 3) or
                    // Q or "S(0) has been read", follows the softmax's wait for iteration k - 2.)
                    mbar_arrive(done(t, b));
                };
                // iteration k: S(k) goes out when P(k - 3) is written (S(k - 2), its buffer's last, has
                // been read then), just before the product of that P with V
#pragma unroll 1
                for (int32_t k = 0; k < steps + 3; ++k) {
                    const uint32_t c = c0 + static_cast<uint32_t>(k), ks = c % NK, bs = (c - 3u) % NB;   // ring positions
                    const bool s_now = k < steps, pv_now = k >= 3;
                    const uint32_t x0 = g0 + static_cast<uint32_t>(k), x1 = g1 + static_cast<uint32_t>(k), b0 = x0 & 1u, b1 = x1 & 1u;
                    const uint32_t k_par = (c / NK) & 1u, b_par = ((c - 3u) / NB) & 1u;
                    // P(k - 3); before that, Q (k = 0) and "S(0) has been read" (k = 2)
                    const uint32_t bar0 = pv_now ? p_full(0, b0 ^ 1u) : q_full(0), bar1 = pv_now ? p_full(1, b1 ^ 1u) : q_full(1);
                    const uint32_t par0 = pv_now ? ((x0 - 3u) >> 1) & 1u : static_cast<uint32_t>(k) >> 1;
                    const uint32_t par1 = pv_now ? ((x1 - 3u) >> 1) & 1u : static_cast<uint32_t>(k) >> 1;
                    const bool got_k = mbar_try_wait(k_full(ks), k_par), got_b = mbar_try_wait(b_full(bs), b_par);
                    const bool got_0 = mbar_try_wait(bar0, par0), got_1 = mbar_try_wait(bar1, par1);
                    if (s_now)
                        need(got_k, k_full(ks), k_par);
                    if (pv_now)
                        need(got_b, b_full(bs), b_par);
                    if (k != 1)
                        need(got_0, bar0, par0);
                    tc_fence_after_sync();
                    issue(0, b0, ks, bs, s_now, pv_now, k == 3);
                    if (two) {
                        if (k != 1)
                            need(got_1, bar1, par1);
                        tc_fence_after_sync();
                        issue(1, b1, ks, bs, s_now, pv_now, k == 3);
                    }
                    if (pv_now) {
                        tc_commit(b_empty(bs));
                        if (k == 3)
                            mbar_arrive(k_empty((c - 3u) % NK));
                        if (k < steps + 2)
                            mbar_arrive(k_empty((c - 2u) % NK));
                    }
                }
                c0 += static_cast<uint32_t>(steps);
                g0 += static_cast<uint32_t>(steps);
                g1 += two ? static_cast<uint32_t>(steps) : 0u;
                n += steps;
                if (n < count)
                    walk_next_segment<kChunkTile, kChunkRows>(p, w);
            }
            tc_commit(drain_bar);
            mbar_wait_tries(drain_bar, 0u, abort);
        }
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------------------ value codes to bf16
        // Eight lanes take four 16-byte chunks of the keys k and k ^ 5: the swizzles put both
        // their loads and their stores on different banks.
        uint32_t vs = 0, vph = 0, bs = 0, bph = 1;
#pragma unroll 1
        for (int64_t h = 0; h < count; ++h) {
            wait2(v_full(vs), vph, b_empty(bs), bph);
            const uint32_t src = base + C::V_OFF + vs * C::V_STAGE, dst = base + C::B_OFF + bs * C::B_STAGE;
#pragma unroll 4
            for (uint32_t i = 0; i < D / 16; ++i) {
                const uint32_t m = (D == 128 ? i >> 1 : i) * 8u + (warp - 2u) * 4u + (lane >> 3);
                const uint32_t key = (2u * m) ^ ((lane & 4u) ? 5u : 0u), atom = D == 128 ? i & 1u : 0u;
                const uint32_t c = (lane & 3u) + 4u * atom;   // 16 dims of a key
                const uint4 q = lds_u4(src + (D == 128 ? key * 128u + ((c ^ (key & 7u)) << 4)
                                                       : key * 64u + ((c ^ ((key >> 1) & 3u)) << 4)));
                const uint32_t x[4] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u, q.z ^ 0x80808080u, q.w ^ 0x80808080u};
                uint32_t y[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)   // two dims of one key
                    asm("fma.rn.bf16x2 %0, %1, %2, %3;"
                        : "=r"(y[u])
                        : "r"(__byte_perm(x[u >> 1], 0u, (u & 1) ? 0x4342u : 0x4140u)), "r"(0x7f007f00u), "r"(0xc000c000u));
                const uint32_t at = dst + atom * 8192u + key * 128u + (((2u * (lane & 3u)) ^ (key & 7u)) << 4);
                sts_v4(at, y[0], y[1], y[2], y[3]);
                sts_v4(at ^ 16u, y[4], y[5], y[6], y[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(b_full(bs));
                mbar_arrive(v_empty(vs));
            }
            if (++vs == NV)
                vs = 0, vph ^= 1u;
            if (++bs == NB)
                bs = 0, bph ^= 1u;
        }
    } else {
        // ------------------------------------------------------------ softmax (warps 4..11)
        const uint32_t tile = (warp - 4u) >> 2, quad = warp & 3u;
        const int32_t r = static_cast<int32_t>(quad * 32u + lane);        // row in the tile
        const int32_t lr = static_cast<int32_t>(tile) * 128 + r;          // row of the segment's tile
        const uint32_t s_addr = tmem_base + ((quad * 32u) << 16) + tile * 128u;
        const uint32_t o_addr = s_addr + 256u;
        const uint32_t prow = base + C::P_OFF + tile * 2u * C::P_BUF + static_cast<uint32_t>(r) * 128u;
        uint32_t g = 0, parity = 0;   // steps of this tile; bit b: parity of the next phase of done(tile, b);
                                      // bit 2: this thread's query row is not finite
        bool open = false;
        int64_t n = 0;
        while (n < count) {
            const int32_t steps = piece_steps(n), rows = piece_rows(), r0 = w.q * kChunkRows;
            const uint32_t n0 = static_cast<uint32_t>(n);
            if (static_cast<int32_t>(tile) * 128 >= rows) {   // no row in this tile
                n += steps;
                if (n < count)
                    walk_next_segment<kChunkTile, kChunkRows>(p, w);
                continue;
            }
            const int32_t tok = by_share(p, r0 + min(lr, rows - 1));
            const int32_t pos0 = w.s.len - w.s.n;
            const int32_t pos = pos0 + tok, low = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
            // the tile's first and last row: which steps are wholly visible
            const int32_t pos_first = pos0 + by_share(p, r0 + static_cast<int32_t>(tile) * 128);
            const int32_t pos_last = pos0 + by_share(p, r0 + min(static_cast<int32_t>(tile) * 128 + 127, rows - 1));
            const int32_t low_last = p.window > 0 ? pos_last - p.window + 1 : 0;
            // this warp's 32 query rows, four at a time: rotated, quantized, into the operand
            // tile; the next four's elements are on their way meanwhile
            {
                constexpr int E = D / 8, V = D / 64;   // elements and 16-byte vectors of a lane
                const int32_t row0 = static_cast<int32_t>(quad * 32u + (lane >> 3));
                auto load = [&](int32_t it, uint4 (&x)[V]) {
                    const int32_t row = static_cast<int32_t>(tile) * 128 + row0 + it * 4;
                    const int32_t tk = by_share(p, r0 + row);
                    const uint16_t *q = p.q + static_cast<int64_t>(w.s.q0 + tk) * p.ldq +
                                        static_cast<int64_t>(w.kvh * p.share + r0 + row - tk * p.share) * D + (lane & 7u) * E;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        x[i] = it < 8 && row < rows ? ld_nc_v4(q + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
                };
                uint4 x[V], x_next[V];
                load(0, x);
#pragma unroll 1
                for (int32_t it = 0; it < 8; ++it) {
                    load(it + 1, x_next);
                    float v[E];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const uint32_t b[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            v[8 * i + 2 * u] = __uint_as_float(b[u] << 16);
                            v[8 * i + 2 * u + 1] = __uint_as_float(b[u] & 0xffff0000u);
                        }
                        x[i] = x_next[i];
                    }
                    uint32_t codes[D / 32];
                    float sq;
                    quant_row_lanes<E, 8>(v, p.group, p.c_g, lane, codes, sq);
                    const uint32_t row = static_cast<uint32_t>(row0 + it * 4), c = lane & 7u;
                    const uint32_t at = base + C::Q_OFF + tile * C::Q_TILE + row * D;
                    if (D == 128)
                        sts_v4(at + ((c ^ (row & 7u)) << 4), codes[0], codes[1], codes[D / 32 - 2], codes[D / 32 - 1]);
                    else
                        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + (((c >> 1) ^ ((row >> 1) & 3u)) << 4) + (c & 1u) * 8u),
                                     "r"(codes[0]), "r"(codes[1])
                                     : "memory");
                    if (c == 0u)
                        qs[tile * 128u + row] = sq;
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            // logit * log2 e = (acc * s_k) * row_f; the floor keeps 0 * -inf out
            const float row_f = fmaxf(qs[lr] * p.scale * 1.4426950408889634f, 0x1p-126f);
            parity = qs[lr] != qs[lr] ? parity | 4u : parity & 3u;
            if (lane == 0)
                mbar_arrive(q_full(tile));
            float m_used = -INFINITY, l_sum = 0.0f;
            uint32_t see[2] = {0u, 0u};   // visible columns of a step: [low, pos] and the sinks, in pages that are there
            auto look = [&](int32_t k) {
                const int32_t i = w.i + k;
                const int32_t j0 = (i < w.t.ns ? i : w.t.w0 + i - w.t.ns) * kChunkTile;
                const uint32_t there = meta[(n0 + k) % NS];
                if (j0 + 63 <= pos_first && (j0 >= low_last || j0 + 64 <= p.sinks) && there == all_boxes)
                    return true;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t in = 0;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        in |= ((there >> ((h * 32 + u * 16) >> pp_shift)) & 1u) ? 0xffffu << (16 * u) : 0u;
                    see[h] = in & (bit_range(low, pos + 1, j0 + 32 * h) | bit_range(0, min(p.sinks, pos + 1), j0 + 32 * h));
                }
                return false;
            };
            // acc * s_k of 4 columns (converting takes one instruction an element here; adding the
            // magic number and subtracting it again, one and a half: 659 against 646 us for a chunk
            // of 2048 over 16384 keys at the time, 32 heads over 8)
            auto scale4 = [&](const uint32_t *acc, float *y, uint32_t at) {
                const float4 k4 = lds_v4(at);   // a broadcast
                float f[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    f[u] = static_cast<float>(static_cast<int32_t>(acc[u]));
                mul2(y[0], y[1], f[0], f[1], k4.x, k4.y);
                mul2(y[2], y[3], f[2], f[3], k4.z, k4.w);
            };
            float y[64] = {};   // logits over row_f of the step at hand
            auto top = [&] {
                float mx[4] = {y[0], y[1], y[2], y[3]};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
#pragma unroll
                    for (int e = 4; e < 60; e += 8)
                        mx[u] = max3f(mx[u], y[e + u], y[e + u + 4]);
                    mx[u] = fmaxf(mx[u], y[60 + u]);
                }
                return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * row_f;
            };
            auto hide = [&] {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    y[e] = (see[e >> 5] >> (e & 31)) & 1u ? y[e] : -INFINITY;
            };
            // The loop handles a step's exponentials together with the scaling of the next one's
            // logits, column by column in the same registers: the two use different pipes.
            uint32_t acc[16];
            auto next_done = [&](uint32_t b) {   // (none may be left out: a wait sees only the parity)
                wait(done(tile, b), (parity >> b) & 1u);
                parity ^= 1u << b;
            };
            next_done(g & 1u);
            tc_fence_after_sync();
            bool whole = look(0);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                tmem_ld_32x32b_x16(s_addr + (g & 1u) * 64u + h * 16u, acc);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    scale4(acc + e, y + h * 16 + e, base + C::SC_OFF + (n0 % NS) * 512u + (h * 16 + e) * 4);
            }
            if (!whole)
                hide();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(q_full(tile));   // (its second phase of the piece: S(0) has been read)
#pragma unroll 1
            for (int32_t k = 0; k < steps; ++k, ++g) {
                const uint32_t b = g & 1u;
                const uint32_t svb = base + C::SC_OFF + ((n0 + k) % NS) * 512u + 256u;
                const uint32_t skb = base + C::SC_OFF + ((n0 + k + 1) % NS) * 512u;
                const bool more = k + 1 < steps;
                // S(k + 1) is there, and P(k - 2) V(k - 2) is done: this step's P buffer is free
                next_done(b ^ 1u);
                tc_fence_after_sync();
                // the sums are rescaled only when the maximum grows by more than 8 (weights stay
                // below 2^8 s_v)
                const float mb = top();
                const bool grow = mb > m_used + 8.0f;
                if (__any_sync(0xffffffffu, grow)) {
                    const float alpha = grow ? ex2_approx(m_used - mb) : 1.0f;
                    m_used = grow ? mb : m_used;
                    l_sum *= alpha;
                    if (k > 0) {   // O is stable once P(k - 1) V(k - 1) is done
                        wait(done(tile, b), (parity >> b) & 1u);
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int32_t c = 0; c < D; c += 16) {
                            tmem_ld_32x32b_x16(o_addr + c, acc);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                uint32_t x[4];
#pragma unroll
                                for (int u = 0; u < 4; ++u)
                                    x[u] = __float_as_uint(__uint_as_float(acc[e + u]) * alpha);
                                tmem_st_32x32b_x4(o_addr + c + e, x);
                            }
                        }
                        tmem_st_wait();
                    }
                }
                const bool was_whole = whole;
                const uint32_t saw[2] = {see[0], see[1]};
                if (more)
                    whole = look(k + 1);
                // P = 2^(y - m) s_v, bf16, into this buffer's swizzled K-major tile (attention.cuh). One
                // rounding to 8 bits: the output is 0.0023 off 64 bits (relative 2-norm), its own rounding
                // alone 0.0017. Weights in f16, as few query rows have them, give 0.0017, but following
                // the largest scale of the keys that each row sees costs 625 instead of 606 us for a chunk
                // of 2048 over 16384 keys, and 259 instead of 245 for eight windowed chunks.
                const float neg_m = m_used == -INFINITY ? 0.0f : -m_used;
                float ls[4] = {0, 0, 0, 0};
                auto weigh = [&](auto masked) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        tmem_ld_32x32b_x16(s_addr + (b ^ 1u) * 64u + h * 16u, acc);   // (of the last step: not used)
                        tmem_ld_wait();
#pragma unroll
                        for (int ch = 0; ch < 2; ++ch) {
                            uint32_t x[4];
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                float *z = y + h * 16 + ch * 8 + q * 4;
                                const float4 v4 = lds_v4(svb + (h * 16 + ch * 8 + q * 4) * 4);
                                float f[4];
                                fma2(f[0], f[1], z[0], z[1], row_f, row_f, neg_m, neg_m);
                                fma2(f[2], f[3], z[2], z[3], row_f, row_f, neg_m, neg_m);
#pragma unroll
                                for (int u = 0; u < 4; ++u)
                                    f[u] = ex2_approx(f[u]);
                                scale4(acc + ch * 8 + q * 4, z, skb + (h * 16 + ch * 8 + q * 4) * 4);
                                add2(ls[0], ls[1], ls[0], ls[1], f[0], f[1]);
                                add2(ls[2], ls[3], ls[2], ls[3], f[2], f[3]);
                                mul2(f[0], f[1], f[0], f[1], v4.x, v4.y);
                                mul2(f[2], f[3], f[2], f[3], v4.z, v4.w);
                                if (decltype(masked)::value) {   // a hidden key adds 0 whatever its scale holds
#pragma unroll
                                    for (int u = 0; u < 4; ++u)
                                        f[u] = (saw[h >> 1] >> ((h & 1) * 16 + ch * 8 + q * 4 + u)) & 1u ? f[u] : 0.0f;
                                }
                                const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]), hi = __floats2bfloat162_rn(f[2], f[3]);
                                x[2 * q] = *reinterpret_cast<const uint32_t *>(&lo);
                                x[2 * q + 1] = *reinterpret_cast<const uint32_t *>(&hi);
                            }
                            const uint32_t c16 = static_cast<uint32_t>(h * 2 + ch) ^ (static_cast<uint32_t>(r) & 7u);
                            sts_v4(prow + b * C::P_BUF + (c16 << 4), x[0], x[1], x[2], x[3]);
                        }
                    }
                };
                if (was_whole)
                    weigh(std::bool_constant<false>());
                else
                    weigh(std::bool_constant<true>());
                l_sum += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_full(tile, b));
                if (more && !whole)
                    hide();
            }
            const bool begins = w.i == 0, ends = w.i + steps == w.t.nt, finish = begins && ends;
            next_done((g + 1u) & 1u);
            next_done(g & 1u);
            tc_fence_after_sync();
            const bool good = ok && *abort == 0;
            if ((parity & 4u) && l_sum > 0.0f)   // (asking qs again here costs the loop above 2% of its time)
                l_sum = nanf("");
            // O, half a row at a time. A whole segment's is un-rotated: the last stage of a group of
            // D joins the halves, first, and each half has its own stages after that.
            const bool join = finish && p.group == D;
            const float inv = l_sum == 0.0f ? 0.0f : __fdiv_rn(kCodeUnit * p.c_g, l_sum);
            const int32_t head = w.kvh * p.share + r0 + lr - tok * p.share;   // (of a row in use)
            uint16_t *o = p.o + static_cast<int64_t>(w.s.q0 + tok) * p.ldo + static_cast<int64_t>(head) * D;
            float *ws = p.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (begins ? 1 : 0)) * C::PIECE;
#pragma unroll 1
            for (int32_t half = 0; half < 2; ++half) {
                const float own = half ? -1.0f : 1.0f;
                float v[D / 2];
#pragma unroll
                for (int c = 0; c < D / 2; c += 16) {
                    uint32_t x[16], y[16];
                    tmem_ld_32x32b_x16(o_addr + half * (D / 2) + c, x);
                    tmem_ld_32x32b_x16(o_addr + (half ^ 1) * (D / 2) + c, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[c + e] = join ? __fmaf_rn(__uint_as_float(x[e]), own, __uint_as_float(y[e])) : __uint_as_float(x[e]);
                }
                if (finish) {
                    thread_butterfly<D / 2>(v, p.group);
                    if (good && lr < rows) {
#pragma unroll
                        for (int e = 0; e < D / 16; ++e) {
                            uint32_t x[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const __nv_bfloat162 h2 = __floats2bfloat162_rn(v[8 * e + 2 * u] * inv, v[8 * e + 2 * u + 1] * inv);
                                x[u] = *reinterpret_cast<const uint32_t *>(&h2);
                            }
                            st_v4(o + half * (D / 2) + 8 * e, x[0], x[1], x[2], x[3]);
                        }
                    }
                } else if (lr < rows) {
#pragma unroll
                    for (int e = 0; e < D / 8; ++e)
                        *reinterpret_cast<float4 *>(ws + lr * D + half * (D / 2) + 4 * e) =
                            make_float4(v[4 * e] * kCodeUnit, v[4 * e + 1] * kCodeUnit, v[4 * e + 2] * kCodeUnit,
                                        v[4 * e + 3] * kCodeUnit);
                }
            }
            tc_fence_before_sync();
            if (!finish && lr < rows)
                *reinterpret_cast<float2 *>(ws + kChunkRows * D + 2 * lr) = make_float2(m_used, good ? l_sum : nanf(""));
            n += steps;
            if (threadIdx.x == 128 && begins && !ends) {
                // the segment's last step is nt - steps further on: that many blocks hold pieces
                const int64_t end = first + n - steps + w.t.nt - 1;
                desc->pieces = static_cast<int32_t>(end / per) - static_cast<int32_t>(blockIdx.x) + 1;
                desc->q0 = w.s.q0;
                desc->rows = rows;
                desc->head0 = w.kvh * p.share;
                desc->r0 = r0;
                open = true;
            }
            if (n < count)
                walk_next_segment<kChunkTile, kChunkRows>(p, w);
        }
        if (threadIdx.x == 128 && !open)
            desc->pieces = 0;
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, 512);
    }
}

} // namespace sdnq
