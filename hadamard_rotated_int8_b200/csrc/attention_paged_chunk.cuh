// Attention of many query rows (chunks of prompts) over the paged cache, on the
// 5th-generation tensor cores. The mathematics and the work split are attention_paged.cuh's.
//
// One persistent block per SM, 256 query rows of one kv head at a time (two tiles of 128 that
// share every key and value), keys in tiles of 128:
// - warp 0 streams keys, values and scales page by page through TMA rings;
// - warps 2 and 3 turn each half tile of value codes into bf16 (times 2^-6, exact), the
//   128-byte-swizzled operand of the second product;
// - warp 1 issues S_t = Q_t K^T (tcgen05 kind::i8, int32 in TMEM) and O_t += P_t V
//   (kind::f16, fp32 in TMEM) for both tiles;
// - warps 4..7 (tile 0) and 8..11 (tile 1), one thread a query row, rotate and quantize their
//   query rows into the operand tile, then per key tile form base-2 logits, an online softmax
//   (sums rescaled only when the maximum grows by more than 2^8), and P = probability * s_v in
//   bf16. The tiles take turns at the exponentials. At the end of a segment the thread has its
//   output row in registers: the rotation is undone there.
// Bound: the exponentials. Per 256 x 128 tile the SM's 16 exponentials a cycle take 2048
// cycles, the instructions of softmax and conversion about 1900 issue cycles a scheduler, the
// two products 256 + 512 tensor cycles, 33 KB of codes from L2 or memory about 1400.
// The two softmax warpgroups take registers over from the first one (setmaxnreg), so that a
// thread holds a whole row of logits.
#pragma once

#include "attention_paged.cuh"

namespace sdnq {

constexpr int kChunkTile = 128;     // keys per step
constexpr int kChunkRows = 256;     // query rows of a segment: two tiles of 128
constexpr int kChunkBox = 64;       // keys of a box at most
constexpr int kChunkThreads = 384;
constexpr int kChunkRegs = 168;     // registers a thread at launch; see the split below
constexpr int kChunkRegsLow = 72, kChunkRegsHigh = 216;
static_assert(kChunkRegsLow + 2 * kChunkRegsHigh == 3 * kChunkRegs, "registers of the three warpgroups");

template <int D>
struct ChunkConfig {
    static constexpr int NK = 3, NV = 3, NB = 3, NS = 3;   // stages: K, value codes, bf16 values (halves), scales
    static constexpr int Q_TILE = 128 * D, K_STAGE = 128 * D, V_STAGE = 64 * D, B_STAGE = 64 * D * 2;
    static constexpr int P_TILE = 128 * 128 * 2;
    static constexpr int Q_OFF = 0;
    static constexpr int P_OFF = Q_OFF + 2 * Q_TILE;
    static constexpr int K_OFF = P_OFF + 2 * P_TILE;
    static constexpr int B_OFF = K_OFF + NK * K_STAGE;
    static constexpr int V_OFF = B_OFF + NB * B_STAGE;
    static constexpr int SC_OFF = V_OFF + NV * V_STAGE;     // 128 key scales, 128 value scales a stage
    static constexpr int BAR_OFF = SC_OFF + NS * 1024;
    // full and empty of each ring, then per tile s_full, s_empty, p_full, pv_done, turn, q_full; drain
    static constexpr int NBARS = 2 * (NK + NV + NB + NS) + 12 + 1;
    static constexpr int META_OFF = BAR_OFF + NBARS * 8;    // valid boxes of each scale stage
    static constexpr int HOLD_OFF = META_OFF + NS * 4;      // TMEM address, abort flag, scan result
    static constexpr int SMEM_BYTES = 1024 + HOLD_OFF + 32;
    static constexpr int64_t PIECE = static_cast<int64_t>(kChunkRows) * (D + 2);   // floats, as FewConfig's
    static_assert(SMEM_BYTES + 256 <= 232448, "shared memory per block");
};

__device__ __forceinline__ void regs_less() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kChunkRegsLow)); }
__device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChunkRegsHigh)); }

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
    for (int h = 1; h < D; h <<= 1)
        if (h < 8 || h < g) {
#pragma unroll
            for (int i = 0; i < D; ++i)
                if ((i & h) == 0) {
                    const float a = v[i], b = v[i + h];
                    v[i] = __fadd_rn(a, b);
                    v[i + h] = __fsub_rn(a, b);
                }
        }
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
    auto sc_full = [&](uint32_t s) { return bar0 + 8u * (2 * (NK + NV + NB) + s); };
    auto sc_empty = [&](uint32_t s) { return bar0 + 8u * (2 * (NK + NV + NB) + NS + s); };
    constexpr int TB = 2 * (NK + NV + NB + NS);
    auto s_full = [&](uint32_t t) { return bar0 + 8u * (TB + t); };
    auto s_empty = [&](uint32_t t) { return bar0 + 8u * (TB + 2 + t); };
    auto p_full = [&](uint32_t t) { return bar0 + 8u * (TB + 4 + t); };
    auto pv_done = [&](uint32_t t) { return bar0 + 8u * (TB + 6 + t); };
    auto turn = [&](uint32_t t) { return bar0 + 8u * (TB + 8 + t); };
    auto q_full = [&](uint32_t t) { return bar0 + 8u * (TB + 10 + t); };
    const uint32_t drain_bar = bar0 + 8u * (TB + 12);
    volatile uint32_t *meta = reinterpret_cast<volatile uint32_t *>(smem + C::META_OFF);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::HOLD_OFF);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_holder + 1);
    const uint32_t warp = threadIdx.x >> 5, lane = lane_id();

    if (threadIdx.x == 0) {
        for (int s = 0; s < NK; ++s)
            mbar_init(k_full(s), 1), mbar_init(k_empty(s), 1);
        for (int s = 0; s < NV; ++s)
            mbar_init(v_full(s), 1), mbar_init(v_empty(s), 2);
        for (int s = 0; s < NB; ++s)
            mbar_init(b_full(s), 2), mbar_init(b_empty(s), 1);
        for (int s = 0; s < NS; ++s)
            mbar_init(sc_full(s), 1), mbar_init(sc_empty(s), 8);
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1), mbar_init(s_empty(t), 4);
            mbar_init(p_full(t), 4), mbar_init(pv_done(t), 1);
            mbar_init(turn(t), 4), mbar_init(q_full(t), 4);
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
    const int32_t nbox = kChunkTile >> pp_shift;
    const uint32_t all_boxes = (1u << nbox) - 1u;
    auto piece_tiles = [&](int64_t n) { return static_cast<int32_t>(min(static_cast<int64_t>(w.t.nt - w.i), count - n)); };
    auto piece_rows = [&] { return min(kChunkRows, w.s.n * p.share - w.q * kChunkRows); };

    if (warp < 4) {
        regs_less();
        if (warp == 0) {
            // -------------------------------------------------------- loads
            uint32_t ks = 0, kph = 1, vs = 0, vph = 1;   // scales go with the keys (NS == NK)
            static_assert(NS == NK, "one slot number serves keys and scales");
            int64_t n = 0, nv = 0, nk = 0;
            bool ok = true;
            while (ok && n < count) {
                const int32_t tiles = piece_tiles(n);
                const int32_t *row = p.table + static_cast<int64_t>(w.b) * p.table_ld;
                // Page ids are read 32 at a time, a batch ahead of their use; entry e is box
                // e % nbox of the piece's tile e / nbox.
                auto fetch = [&](int32_t e0) {
                    const int32_t e = e0 + static_cast<int32_t>(lane);
                    const int32_t i = w.i + e / nbox;
                    if (i >= w.i + tiles)
                        return -1;
                    const int32_t j = (i < w.t.ns ? i : w.t.w0 + i - w.t.ns) * kChunkTile + (e % nbox) * pp;
                    if (j >= w.s.len)
                        return -1;
                    const int32_t id = row[j >> p.page_shift];
                    if (id < 0 || id >= p.pages) {
                        atomicOr(&g_device_error, kDevIndex);
                        return -1;
                    }
                    return id;
                };
                int32_t ids = fetch(0), ids_next = fetch(32), e0 = 0;
                for (int32_t k = 0; ok && k < tiles; ++k) {
                    if (k * nbox >= e0 + 32) {
                        ids = ids_next;
                        e0 += 32;
                        ids_next = fetch(e0 + 32);
                    }
                    // lane c < nbox has box c of this tile
                    const int32_t id = __shfl_sync(0xffffffffu, ids, (k * nbox - e0 + static_cast<int32_t>(lane)) & 31);
                    const bool mine = static_cast<int32_t>(lane) < nbox && id >= 0;
                    const uint32_t valid = __ballot_sync(0xffffffffu, mine);
                    const int32_t i = w.i + k;
                    const int32_t j = (i < w.t.ns ? i : w.t.w0 + i - w.t.ns) * kChunkTile + static_cast<int32_t>(lane) * pp;
                    int32_t krow = 0, vrow = 0;
                    if (mine) {
                        krow = static_cast<int32_t>(((static_cast<int64_t>(id) * p.Hkv + w.kvh) * 2) << p.page_shift) +
                               (j & ((1 << p.page_shift) - 1));
                        vrow = krow + (1 << p.page_shift);
                    }
                    bool got = true;
                    if (lane == 0) {
                        got = mbar_wait_bounded(k_empty(ks), kph, abort, p.timeout_ns) &&
                              mbar_wait_bounded(sc_empty(ks), kph, abort, p.timeout_ns);
                        if (got) {
                            meta[ks] = valid;
                            mbar_arrive_expect_tx(sc_full(ks), static_cast<uint32_t>(__popc(valid)) * 8u * pp);
                            mbar_arrive_expect_tx(k_full(ks), static_cast<uint32_t>(__popc(valid)) * pp * D);
                        }
                    }
                    ok = __shfl_sync(0xffffffffu, static_cast<int>(got), 0) != 0;
                    if (!ok)
                        break;
                    ++nk;
                    if (mine) {
                        tma_load_2d(base + C::K_OFF + ks * C::K_STAGE + lane * pp * D, &tmPool, k_full(ks), 0, krow);
                        const uint32_t sdst = base + C::SC_OFF + ks * 1024u + lane * pp * 4u;
                        bulk_load_1d(sdst, p.scales + krow, 4u * pp, sc_full(ks));
                        bulk_load_1d(sdst + 512u, p.scales + vrow, 4u * pp, sc_full(ks));
                    }
                    for (uint32_t half = 0; half < 2; ++half) {
                        const uint32_t boxes = half == 0 ? valid & ((1u << (nbox / 2)) - 1u) : valid >> (nbox / 2);
                        if (lane == 0) {
                            got = mbar_wait_bounded(v_empty(vs), vph, abort, p.timeout_ns);
                            if (got)
                                mbar_arrive_expect_tx(v_full(vs), static_cast<uint32_t>(__popc(boxes)) * pp * D);
                        }
                        ok = __shfl_sync(0xffffffffu, static_cast<int>(got), 0) != 0;
                        if (!ok)
                            break;
                        ++nv;
                        const uint32_t box = lane - half * (nbox / 2);
                        if (mine && box < static_cast<uint32_t>(nbox / 2))
                            tma_load_2d(base + C::V_OFF + vs * C::V_STAGE + box * pp * D, &tmPool, v_full(vs), 0, vrow);
                        if (++vs == NV)
                            vs = 0, vph ^= 1u;
                    }
                    if (++ks == NK)
                        ks = 0, kph ^= 1u;
                }
                n += tiles;
                walk_next_segment<kChunkTile, kChunkRows>(p, w);
            }
            // every copy has landed before the block may end
            if (lane == 0) {
                volatile int no_abort = 0;
                for (int64_t j = nk - NK < 0 ? 0 : nk - NK; j < nk; ++j) {
                    mbar_wait_bounded(k_full(static_cast<uint32_t>(j % NK)), static_cast<uint32_t>(j / NK) & 1u, &no_abort, p.timeout_ns);
                    mbar_wait_bounded(sc_full(static_cast<uint32_t>(j % NS)), static_cast<uint32_t>(j / NS) & 1u, &no_abort, p.timeout_ns);
                }
                for (int64_t j = nv - NV < 0 ? 0 : nv - NV; j < nv; ++j)
                    mbar_wait_bounded(v_full(static_cast<uint32_t>(j % NV)), static_cast<uint32_t>(j / NV) & 1u, &no_abort, p.timeout_ns);
            }
        } else if (warp == 1) {
            // -------------------------------------------------------- MMA issue
            if (lane == 0) {
                constexpr uint32_t IDESC_S = idesc_s8_s32(128, 128);
                constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, true);
                uint32_t ks = 0, kph = 0, bs = 0, bph = 0;
                uint32_t s_n[2] = {0, 0}, p_n[2] = {0, 0}, pieces = 0;   // issued per tile
                int64_t n = 0;
                bool ok = true;
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    ok = ok && mbar_wait_bounded(bar, parity, abort, p.timeout_ns);
                    return ok;
                };
                // S_t = Q_t K^T of the next key tile, for the tiles in use
                auto issue_s = [&](uint32_t in_use) {
                    if (!wait(k_full(ks), kph))
                        return;
                    for (uint32_t t = 0; t < in_use; ++t) {
                        if (!wait(s_empty(t), (s_n[t] & 1u) ^ 1u))
                            return;
                        tc_fence_after_sync();
                        const uint32_t qa = base + C::Q_OFF + t * C::Q_TILE, ka = base + C::K_OFF + ks * C::K_STAGE;
#pragma unroll
                        for (int k = 0; k < D / 32; ++k)
                            mma_s8(tmem_base + t * 128, codes_desc<D>(qa + 32 * k), codes_desc<D>(ka + 32 * k), IDESC_S,
                                   k != 0 ? 1u : 0u);
                        tc_commit(s_full(t));
                        ++s_n[t];
                    }
                    tc_commit(k_empty(ks));
                    if (++ks == NK)
                        ks = 0, kph ^= 1u;
                };
                while (ok && n < count) {
                    const int32_t tiles = piece_tiles(n);
                    const uint32_t in_use = piece_rows() > 128 ? 2 : 1;
                    wait(q_full(0), pieces & 1u);
                    wait(q_full(1), pieces & 1u);
                    ++pieces;
                    if (ok)
                        issue_s(in_use);
                    for (int32_t k = 0; ok && k < tiles; ++k) {
                        if (k + 1 < tiles)
                            issue_s(in_use);
                        for (uint32_t t = 0; ok && t < in_use; ++t) {
                            if (!wait(p_full(t), p_n[t] & 1u))
                                break;
                            uint32_t slot = bs, ph = bph;
                            for (uint32_t half = 0; half < 2; ++half) {
                                if (!wait(b_full(slot), ph))
                                    break;
                                tc_fence_after_sync();
                                const uint32_t pa = base + C::P_OFF + t * C::P_TILE + half * 16384u;
                                const uint32_t va = base + C::B_OFF + slot * C::B_STAGE;
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    mma_f16(tmem_base + 256 + t * 128, kmajor_desc(pa + 32 * kk),
                                            mnmajor_desc(va + 2048 * kk, 8192), IDESC_PV,
                                            (k | static_cast<int32_t>(half) | kk) != 0 ? 1u : 0u);
                                if (t + 1 == in_use)
                                    tc_commit(b_empty(slot));
                                if (++slot == NB)
                                    slot = 0, ph ^= 1u;
                            }
                            if (!ok)
                                break;
                            tc_commit(pv_done(t));
                            ++p_n[t];
                            if (t + 1 == in_use)
                                bs = slot, bph = ph;
                        }
                    }
                    n += tiles;
                    walk_next_segment<kChunkTile, kChunkRows>(p, w);
                }
                tc_commit(drain_bar);
                volatile int no_abort = 0;
                mbar_wait_bounded(drain_bar, 0u, &no_abort, p.timeout_ns);
            }
        } else {
            // -------------------------------------------------------- value codes to bf16
            const uint32_t me = (warp - 2u) * 32u + lane;
            uint32_t vs = 0, vph = 0, bs = 0, bph = 1;
            bool ok = true;
            for (int64_t h = 0; ok && h < 2 * count; ++h) {
                const bool got = mbar_wait_bounded(v_full(vs), vph, abort, p.timeout_ns) &&
                                 mbar_wait_bounded(b_empty(bs), bph, abort, p.timeout_ns);
                ok = __all_sync(0xffffffffu, got);
                if (!ok)
                    break;
                const uint32_t src = base + C::V_OFF + vs * C::V_STAGE, dst = base + C::B_OFF + bs * C::B_STAGE;
#pragma unroll
                for (int i = 0; i < 4 * D / 64; ++i) {
                    const uint32_t idx = i * 64u + me, key = idx / (D / 16), c = idx % (D / 16);   // 16 dims of a key
                    const uint32_t at = D == 128 ? key * 128u + ((c ^ (key & 7u)) << 4)
                                                 : key * 64u + ((c ^ ((key >> 1) & 3u)) << 4);
                    const uint4 q = lds_u4(src + at);
                    const uint32_t x[4] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u, q.z ^ 0x80808080u, q.w ^ 0x80808080u};
                    uint32_t y[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u)   // as codes_to_bf16x2, two dims of one key
                        asm("fma.rn.bf16x2 %0, %1, %2, %3;"
                            : "=r"(y[u])
                            : "r"(__byte_perm(x[u >> 1], 0u, (u & 1) ? 0x4342u : 0x4140u)), "r"(0x7f007f00u), "r"(0xc000c000u));
                    // 128-byte rows of 64 dims; the lanes of the second 64 dims store their
                    // chunks the other way round (their rows lie on the same banks)
                    const uint32_t row = dst + (c >> 2) * 8192u + key * 128u, ch = 2u * (c & 3u), swap = c >> 2;
                    const uint32_t a0 = row + (((ch + swap) ^ (key & 7u)) << 4), a1 = row + (((ch + 1u - swap) ^ (key & 7u)) << 4);
                    sts_v4(a0, swap ? y[4] : y[0], swap ? y[5] : y[1], swap ? y[6] : y[2], swap ? y[7] : y[3]);
                    sts_v4(a1, swap ? y[0] : y[4], swap ? y[1] : y[5], swap ? y[2] : y[6], swap ? y[3] : y[7]);
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
        }
    } else {
        // ------------------------------------------------------------ softmax (warps 4..11)
        regs_more();
        const uint32_t tile = (warp - 4u) >> 2, quad = warp & 3u;
        const int32_t r = static_cast<int32_t>(quad * 32u + lane);        // row in the tile
        const int32_t lr = static_cast<int32_t>(tile) * 128 + r;          // row of the segment's tile
        const uint32_t t_lane = tmem_base + ((quad * 32u) << 16);
        const uint32_t s_col = tile * 128u, o_col = 256u + tile * 128u;
        uint32_t ss = 0, sph = 0, blocks = 0, mine = 0;   // scale ring; key tiles seen, and worked on
        bool ok = true, open = false;
        int64_t n = 0;
        while (ok && n < count) {
            const int32_t tiles = piece_tiles(n), rows = piece_rows(), r0 = w.q * kChunkRows;
            const bool active = static_cast<int32_t>(tile) * 128 < rows;
            const int32_t tok = (r0 + min(lr, rows - 1)) / p.share;
            const int32_t head = w.kvh * p.share + r0 + min(lr, rows - 1) - tok * p.share;
            const int32_t pos0 = w.s.len - w.s.n;
            const int32_t pos = pos0 + tok, low = p.window > 0 ? pos - p.window + 1 : INT32_MIN;
            // the tile's first and last row: which key tiles are wholly visible
            const int32_t pos_first = pos0 + (r0 + static_cast<int32_t>(tile) * 128) / p.share;
            const int32_t pos_last = pos0 + (r0 + min(static_cast<int32_t>(tile) * 128 + 127, rows - 1)) / p.share;
            const int32_t low_last = p.window > 0 ? pos_last - p.window + 1 : INT32_MIN;
            if (!active) {   // no row in this tile: only its part in the handshakes
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(q_full(tile));
                for (int32_t k = 0; k < tiles; ++k, ++blocks) {
                    const bool got = mbar_wait_bounded(sc_full(ss), sph, abort, p.timeout_ns) &&
                                     mbar_wait_bounded(turn(tile), tile == 0 ? (blocks & 1u) ^ 1u : blocks & 1u, abort, p.timeout_ns);
                    ok = __all_sync(0xffffffffu, got);
                    if (!ok)
                        break;
                    if (lane == 0) {
                        mbar_arrive(turn(tile ^ 1u));
                        mbar_arrive(sc_empty(ss));
                    }
                    if (++ss == NS)
                        ss = 0, sph ^= 1u;
                }
                n += tiles;
                walk_next_segment<kChunkTile, kChunkRows>(p, w);
                continue;
            }
            float row_f;
            {
                // the query row: rotated, quantized, into the operand tile
                float v[D];
                const uint16_t *q = p.q + static_cast<int64_t>(w.s.q0 + tok) * p.ldq + static_cast<int64_t>(head) * D;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 a = lr < rows ? ld_nc_v4(q + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t x[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        v[8 * i + 2 * u] = __uint_as_float(x[u] << 16);
                        v[8 * i + 2 * u + 1] = __uint_as_float(x[u] & 0xffff0000u);
                    }
                }
                thread_butterfly<D>(v, p.group);
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < D; ++i)
                    m = fmaxf(m, fabsf(v[i]));
                const float s_z = __fdiv_rn(m, 127.0f);
                const bool zero = !(m > 0.0f);
                float s_q = s_z;
                if (s_z < 0x1p-126f) {   // a subnormal step: the same quotients, 2^64 times as large on both sides
                    s_q = s_z * 0x1p64f;
                    const float most = s_q * 127.0f;
#pragma unroll
                    for (int i = 0; i < D; ++i)
                        v[i] = fminf(fmaxf(v[i] * 0x1p64f, -most), most);
                }
                const float rcp = __frcp_rn(s_q);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    uint2 a = make_uint2(0u, 0u), b = make_uint2(0u, 0u);
                    if (!zero) {
                        float z[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            z[i] = v[16 * c + i];
                        a = quant8(z, s_q, rcp, true);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            z[i] = v[16 * c + 8 + i];
                        b = quant8(z, s_q, rcp, true);
                    }
                    const uint32_t sw = D == 128 ? static_cast<uint32_t>(c) ^ (r & 7) : static_cast<uint32_t>(c) ^ ((r >> 1) & 3);
                    sts_v4(base + C::Q_OFF + tile * C::Q_TILE + r * D + (sw << 4), a.x, a.y, b.x, b.y);
                }
                // logit * log2 e = (acc * s_k) * row_f; the floor keeps 0 * -inf out
                const float sq = zero ? 0.0f : __fmul_rn(s_z, p.c_g);
                row_f = fmaxf(sq * p.scale * 1.4426950408889634f, 0x1p-126f);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(q_full(tile));
            float m_used = -INFINITY, l_sum = 0.0f;
#pragma unroll 1
            for (int32_t k = 0; k < tiles; ++k, ++blocks) {
                bool got = mbar_wait_bounded(s_full(tile), mine & 1u, abort, p.timeout_ns) &&
                           mbar_wait_bounded(sc_full(ss), sph, abort, p.timeout_ns);
                ok = __all_sync(0xffffffffu, got);
                if (!ok)
                    break;
                float y[128];
                float alpha = 1.0f;
                bool any_grow = false, whole = true;
                tc_fence_after_sync();
                // fp32(acc) without the conversion pipe (attention.cuh)
                {
                    uint32_t a[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tmem_ld_32x32b_x32(t_lane + s_col + c * 32, a[c]);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            y[c * 32 + i] = __uint_as_float(a[c][i] + 0x4B400000u);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(s_empty(tile));
                const uint32_t skb = base + C::SC_OFF + ss * 1024u;
#pragma unroll
                for (int c4 = 0; c4 < 32; ++c4) {
                    const float4 k4 = lds_v4(skb + c4 * 16u);   // a broadcast
                    float f0, f1, f2, f3;
                    sub2(f0, f1, y[4 * c4], y[4 * c4 + 1], 12582912.0f, 12582912.0f);
                    sub2(f2, f3, y[4 * c4 + 2], y[4 * c4 + 3], 12582912.0f, 12582912.0f);
                    mul2(y[4 * c4], y[4 * c4 + 1], f0, f1, k4.x, k4.y);          // acc * s_k
                    mul2(y[4 * c4 + 2], y[4 * c4 + 3], f2, f3, k4.z, k4.w);
                }
                const int32_t i = w.i + k;
                const int32_t j0 = (i < w.t.ns ? i : w.t.w0 + i - w.t.ns) * kChunkTile;
                const uint32_t there = meta[ss];
                whole = j0 + 127 <= pos_first && (j0 >= low_last || j0 + 128 <= p.sinks) && there == all_boxes;
                if (!whole) {
                    // visible columns: [from, to) and those of the sinks, in pages that are there
                    uint32_t there16 = 0;   // a bit for each 16 columns
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        there16 |= ((there >> ((c * 16) >> pp_shift)) & 1u) << c;
                    const int32_t to = pos - j0 + 1, from = low > j0 - 128 ? low - j0 : -128, sink = p.sinks - j0;
#pragma unroll
                    for (int c = 0; c < 128; ++c) {
                        const bool see = c < to && (c >= from || c < sink) && ((there16 >> (c / 16)) & 1u) != 0u;
                        y[c] = see ? y[c] : -INFINITY;
                    }
                }
                // 4 independent chains, chain i over the columns i + 4k (k = 0..31)
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mx[c] = y[c];
#pragma unroll
                    for (int u = 1; u + 1 < 32; u += 2)
                        mx[c] = max3f(mx[c], y[c + 4 * u], y[c + 4 * u + 4]);
                    mx[c] = fmaxf(mx[c], y[c + 124]);
                }
                const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * row_f;
                // the P tile is free, and O stable, once the tile's last product is done
                if (k > 0) {
                    got = mbar_wait_bounded(pv_done(tile), (mine & 1u) ^ 1u, abort, p.timeout_ns);
                    ok = __all_sync(0xffffffffu, got);
                    if (!ok)
                        break;
                    tc_fence_after_sync();
                }
                const bool grow = mb > m_used + 8.0f;
                any_grow = __any_sync(0xffffffffu, grow);
                if (any_grow) {
                    alpha = grow ? ex2_approx(m_used - mb) : 1.0f;
                    m_used = grow ? mb : m_used;
                    l_sum *= alpha;
                }
                // tile 0 runs its exponentials of a key tile after tile 1 ran those of the one
                // before, tile 1 after tile 0 ran those of the same one
                got = mbar_wait_bounded(turn(tile), tile == 0 ? (blocks & 1u) ^ 1u : blocks & 1u, abort, p.timeout_ns);
                ok = __all_sync(0xffffffffu, got);
                if (!ok)
                    break;
                const uint32_t prow = base + C::P_OFF + tile * C::P_TILE + static_cast<uint32_t>(r) * 128u;
                const uint32_t svb = base + C::SC_OFF + ss * 1024u + 512u;
                const float neg_m = m_used == -INFINITY ? 0.0f : -m_used;
                float ls[8] = {0, 0, 0, 0, 0, 0, 0, 0};  // 8 independent partial sums
                // P = 2^(y - m) s_v, bf16, into the swizzled K-major tile (attention.cuh)
                auto weigh = [&](auto masked) {
#pragma unroll
                    for (int ch = 0; ch < 16; ++ch) {
                        uint32_t x[4];
#pragma unroll
                        for (int e2 = 0; e2 < 2; ++e2) {
                            const float4 v4 = lds_v4(svb + ch * 32u + e2 * 16u);
                            const float sv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int c = ch * 8 + e2 * 4 + 2 * e;
                                float d0, d1, w0, w1;
                                fma2(d0, d1, y[c], y[c + 1], row_f, row_f, neg_m, neg_m);
                                const float p0 = ex2_approx(d0), p1 = ex2_approx(d1);
                                float &l0 = ls[4 * e2 + 2 * e], &l1 = ls[4 * e2 + 2 * e + 1];
                                add2(l0, l1, l0, l1, p0, p1);
                                mul2(w0, w1, p0, p1, sv[2 * e], sv[2 * e + 1]);
                                if (decltype(masked)::value) {   // a hidden key adds 0 whatever its scale holds
                                    w0 = p0 == 0.0f ? 0.0f : w0;
                                    w1 = p1 == 0.0f ? 0.0f : w1;
                                }
                                const __nv_bfloat162 h2 = __floats2bfloat162_rn(w0, w1);
                                x[2 * e2 + e] = *reinterpret_cast<const uint32_t *>(&h2);
                            }
                        }
                        const uint32_t c16 = static_cast<uint32_t>(ch & 7) ^ (static_cast<uint32_t>(r) & 7u);
                        sts_v4(prow + static_cast<uint32_t>(ch >> 3) * 16384u + (c16 << 4), x[0], x[1], x[2], x[3]);
                    }
                };
                if (whole)
                    weigh(PagedFlag<false>());
                else
                    weigh(PagedFlag<true>());
                l_sum += ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(turn(tile ^ 1u));
                    mbar_arrive(sc_empty(ss));
                }
                if (++ss == NS)
                    ss = 0, sph ^= 1u;
                if (any_grow && k > 0) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t a[32];
                        tmem_ld_32x32b_x32(t_lane + o_col + c * 32, a);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            a[i] = __float_as_uint(__uint_as_float(a[i]) * alpha);
                        tmem_st_32x32b_x32(t_lane + o_col + c * 32, a);
                    }
                    tmem_st_wait();
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_full(tile));
                ++mine;
            }
            const bool begins = w.i == 0, ends = w.i + tiles == w.t.nt;
            if (ok) {
                const bool got = mbar_wait_bounded(pv_done(tile), (mine & 1u) ^ 1u, abort, p.timeout_ns);
                ok = __all_sync(0xffffffffu, got);
                if (ok) {
                    tc_fence_after_sync();
                    float v[D];
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t a[32];
                        tmem_ld_32x32b_x32(t_lane + o_col + c * 32, a);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[c * 32 + i] = __uint_as_float(a[i]);
                    }
                    tc_fence_before_sync();
                    if (begins && ends) {
                        thread_butterfly<D>(v, p.group);
                        const float inv = l_sum == 0.0f ? 0.0f : __fdiv_rn(kCodeUnit * p.c_g, l_sum);
                        uint16_t *o = p.o + static_cast<int64_t>(w.s.q0 + tok) * p.ldo + static_cast<int64_t>(head) * D;
                        if (lr < rows) {
#pragma unroll
                            for (int i = 0; i < D / 8; ++i) {
                                uint32_t x[4];
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    const __nv_bfloat162 h2 = __floats2bfloat162_rn(v[8 * i + 2 * u] * inv, v[8 * i + 2 * u + 1] * inv);
                                    x[u] = *reinterpret_cast<const uint32_t *>(&h2);
                                }
                                st_v4(o + 8 * i, x[0], x[1], x[2], x[3]);
                            }
                        }
                    } else if (lr < rows) {
                        float *ws = p.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (begins ? 1 : 0)) * C::PIECE;
#pragma unroll
                        for (int i = 0; i < D / 4; ++i)
                            *reinterpret_cast<float4 *>(ws + lr * D + 4 * i) =
                                make_float4(v[4 * i] * kCodeUnit, v[4 * i + 1] * kCodeUnit, v[4 * i + 2] * kCodeUnit,
                                            v[4 * i + 3] * kCodeUnit);
                        *reinterpret_cast<float2 *>(ws + kChunkRows * D + 2 * lr) = make_float2(m_used, l_sum);
                    }
                }
            }
            n += tiles;
            if (threadIdx.x == 128 && begins && !ends) {
                const int64_t end = first + n - tiles + w.t.nt - 1;
                desc->pieces = static_cast<int32_t>(end / per) - static_cast<int32_t>(blockIdx.x) + 1;
                desc->q0 = w.s.q0;
                desc->rows = rows;
                desc->head0 = w.kvh * p.share;
                desc->r0 = r0;
                open = true;
            }
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
