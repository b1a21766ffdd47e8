// Attention of new tokens over the paged, rotated int8 key/value cache (kvcache.cuh).
//
// Query i of a sequence with context length L and n new tokens sits at position
// p = L - n + i and sees the keys j <= p with (no window, or j > p - window, or j < sinks):
//   logit_j = (qc . kc_j) * (s_q * s_k[j]) * scale,  qc, s_q the row quantizer's codes of q,
//   o = butterfly(sum_j softmax(logit)_j * s_v[j] * vc_j) * c,  c = fp32(1/sqrt(G)).
// The rotation leaves q . k unchanged (it is orthogonal), so nothing is un-rotated before the
// softmax; the values' rotation is undone once per output row. A row that sees no key is 0.
#pragma once

#include <cfloat>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "attention.cuh"
#include "device.cuh"
#include "kvcache.cuh"
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
    int32_t T, B, Hkv;
    int32_t share;           // H / Hkv
    uint32_t share_mul, share_shift;   // n / share = n * share_mul >> share_shift for 0 <= n < 2^31
    int32_t page_shift;
    int32_t cap;             // most keys a table row can name
    int32_t window;          // <= 0: none
    int32_t sinks;
    int32_t group;           // min(group, D)
    float scale;
    float c_g;
    int32_t rows_min, rows_max;   // sequences of rows_min < (token, head) rows a kv head <= rows_max
    int32_t least_tiles;     // a block's share of the tile list is at least this
    float *partial;          // workspace: pieces, and what the blocks say of them
    void *desc;
    uint64_t timeout_ns;
};

__device__ __forceinline__ int32_t by_share(const PagedParams &p, int32_t n)
{
    return static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * p.share_mul) >> p.share_shift);
}

// a / b, in 32 bits where they hold both (a division in 64 takes several times as long).
__device__ __forceinline__ int64_t div_wide(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0)
        return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

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

// ---------------------------------------------------------------- work split
//
// A segment is one (sequence, kv head, tile of query rows); the rows of a tile are (token,
// head of the kv head's share) pairs in that order, so grouped heads share the keys and values
// they read. A segment's keys are walked in tiles: those of the sinks, then those from the
// first row's window to the last row's position. All tiles of all segments form one list
// (sequence, then kv head, then query tile), and block c takes the equal share
// [c * per, (c + 1) * per) of it, whatever segments that meets: the blocks finish together for
// any mix of lengths. A segment that one block has whole is written out by it; of the others,
// each block leaves its unnormalised sums, and a second kernel joins them in list order (so
// the results do not depend on timing).

struct PagedTiles {
    int32_t nt;       // key tiles of the segment
    int32_t ns, w0;   // tiles 0..ns-1 hold the sinks, the others start at tile w0
};

// Query tiles of a sequence; 0: the sequence is not this kernel's.
template <int ROWS>
__device__ __forceinline__ int32_t paged_qtiles(const PagedParams &p, const PagedSeq &s)
{
    const int32_t rows = s.n * p.share;
    return rows > p.rows_min && rows <= p.rows_max ? (rows - 1) / ROWS + 1 : 0;
}

// The keys that some row of query tile q (ROWS rows) sees: [low, end) and the sinks below end.
struct PagedReach {
    int32_t low, end;

    // [j, j + n) holds one of them. (An owner of a window gives back the pages between: their
    // table entries are not looked up.)
    __device__ __forceinline__ bool any(const PagedParams &p, int32_t j, int32_t n) const
    {
        return j < end && (j + n > low || j < p.sinks);
    }
};

template <int ROWS>
__device__ __forceinline__ PagedReach paged_reach(const PagedParams &p, int32_t n, int32_t len, int32_t q)
{
    const int32_t first = by_share(p, q * ROWS), last = by_share(p, min(q * ROWS + ROWS - 1, n * p.share - 1));
    PagedReach r;
    r.end = max(len - n + last + 1, 0);
    r.low = p.window > 0 ? max(0, len - n + first - p.window + 1) : 0;
    return r;
}

// The key tiles of TILE keys of query tile q.
template <int TILE, int ROWS>
__device__ __forceinline__ PagedTiles paged_tiles(const PagedParams &p, int32_t n, int32_t len, int32_t q)
{
    const PagedReach r = paged_reach<ROWS>(p, n, len, q);
    PagedTiles t;
    t.w0 = r.low / TILE;
    t.ns = min((min(p.sinks, r.end) + TILE - 1) / TILE, t.w0);
    t.nt = max(t.ns + (r.end + TILE - 1) / TILE - t.w0, 1);
    return t;
}

// Where a block is in the list of tiles.
struct PagedWalk {
    int32_t b, kvh, q, i;   // sequence, kv head, query tile, key tile of the segment
    int32_t qt;             // query tiles of the sequence
    PagedSeq s;
    PagedTiles t;
};

// (Not to be called behind the last piece of a block: it looks at sequences one by one, and those
// that follow may all be the other kernel's.)
template <int TILE, int ROWS>
__device__ __forceinline__ void walk_next_segment(const PagedParams &p, PagedWalk &w)
{
    w.i = 0;
    if (++w.q == w.qt) {
        w.q = 0;
        if (++w.kvh == p.Hkv) {
            w.kvh = 0;
            do {
                if (++w.b >= p.B)
                    return;
                w.s = paged_seq(p, w.b);
                w.qt = paged_qtiles<ROWS>(p, w.s);
            } while (w.qt == 0);
        }
    }
    w.t = paged_tiles<TILE, ROWS>(p, w.s.n, w.s.len, w.q);
}

__device__ __forceinline__ int64_t warp_inclusive_sum(int64_t v, uint32_t lane)
{
#pragma unroll
    for (uint32_t x = 1; x < 32; x <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, x);
        if (lane >= x)
            v += o;
    }
    return v;
}

// The tiles that a head of the 32 sequences b (one a lane) has: a sequence of up to 2 query
// tiles is its lane's work, longer ones are walked by the whole warp.
template <int TILE, int ROWS>
__device__ __forceinline__ int64_t sequence_tiles(const PagedParams &p, int32_t b, uint32_t lane, PagedSeq &s,
                                                  int32_t &qt)
{
    s.q0 = 0, s.n = 0, s.len = 0, qt = 0;
    if (b < p.B) {
        s = paged_seq(p, b);
        qt = paged_qtiles<ROWS>(p, s);
    }
    int64_t sum = 0;
    for (int32_t q = 0; q < min(qt, 2); ++q)
        sum += paged_tiles<TILE, ROWS>(p, s.n, s.len, q).nt;
    for (uint32_t big = __ballot_sync(0xffffffffu, qt > 2); big != 0u; big &= big - 1u) {
        const int src = __ffs(static_cast<int>(big)) - 1;
        const int32_t n = __shfl_sync(0xffffffffu, s.n, src), len = __shfl_sync(0xffffffffu, s.len, src);
        const int32_t qn = __shfl_sync(0xffffffffu, qt, src);
        int64_t part = 0;
        for (int32_t q = 2 + static_cast<int32_t>(lane); q < qn; q += 32)
            part += paged_tiles<TILE, ROWS>(p, n, len, q).nt;
        part = __shfl_sync(0xffffffffu, warp_inclusive_sum(part, lane), 31);
        if (static_cast<int>(lane) == src)
            sum += part;
    }
    return sum;
}

// Counts the list's tiles (the whole block), and finds where share blockIdx.x of `blocks`
// begins: tile `first` of `total`, shares of `per` >= `least` tiles. `found`: 8 words of shared
// memory.
template <int TILE, int ROWS, int THREADS>
__device__ __forceinline__ void find_share(const PagedParams &p, int64_t blocks, int32_t least, int32_t *found,
                                           int64_t &first, int64_t &per, int64_t &total, PagedWalk &w)
{
    constexpr int WARPS = THREADS / 32;
    __shared__ int64_t warp_sum[WARPS];
    const uint32_t lane = lane_id();
    const int32_t warp = static_cast<int32_t>(threadIdx.x >> 5);
    const int32_t groups = (p.B + 31) / 32, each = (groups + WARPS - 1) / WARPS;
    const int32_t g0 = min(warp * each, groups), g1 = min(g0 + each, groups);
    PagedSeq s;
    int32_t qt;
    int64_t mine = 0, incl = 0, sum = 0;   // of the last group looked at; of all
#pragma unroll 1
    for (int32_t g = g0; g < g1; ++g) {
        mine = sequence_tiles<TILE, ROWS>(p, g * 32 + static_cast<int32_t>(lane), lane, s, qt);
        incl = warp_inclusive_sum(mine, lane);
        sum += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0)
        warp_sum[warp] = sum;
    __syncthreads();
    int64_t before = 0;   // tiles of a head, as the sums are; a sequence's heads follow each other
    total = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        if (i < warp)
            before += warp_sum[i];
        total += warp_sum[i];
    }
    before *= p.Hkv, sum *= p.Hkv, total *= p.Hkv;
    per = div_wide(total + blocks - 1, blocks);
    per = per < least ? least : per;
    first = static_cast<int64_t>(blockIdx.x) * per;
    if (first < total && first >= before && first < before + sum) {   // one warp
        int64_t rest = first - before;
#pragma unroll 1
        for (int32_t g = g0; g < g1; ++g) {
            if (g1 - g0 > 1) {
                mine = sequence_tiles<TILE, ROWS>(p, g * 32 + static_cast<int32_t>(lane), lane, s, qt);
                incl = warp_inclusive_sum(mine, lane);
            }
            const int64_t all = __shfl_sync(0xffffffffu, incl, 31) * p.Hkv;
            if (rest >= all) {
                rest -= all;
                continue;
            }
            const int src = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, rest < incl * p.Hkv))) - 1;
            const int32_t n = __shfl_sync(0xffffffffu, s.n, src), len = __shfl_sync(0xffffffffu, s.len, src);
            const int32_t qn = __shfl_sync(0xffffffffu, qt, src), q0 = __shfl_sync(0xffffffffu, s.q0, src);
            const int64_t head = __shfl_sync(0xffffffffu, mine, src);
            rest -= __shfl_sync(0xffffffffu, incl - mine, src) * p.Hkv;
            const int64_t kvh = div_wide(rest, head);
            rest -= kvh * head;
#pragma unroll 1
            for (int32_t t0 = 0; t0 < qn; t0 += 32) {
                const int32_t q = t0 + static_cast<int32_t>(lane);
                const int64_t nt = q < qn ? paged_tiles<TILE, ROWS>(p, n, len, q).nt : 0;
                const int64_t qi = warp_inclusive_sum(nt, lane);
                const int64_t qall = __shfl_sync(0xffffffffu, qi, 31);
                if (rest >= qall) {
                    rest -= qall;
                    continue;
                }
                const int at = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, rest < qi))) - 1;
                rest -= __shfl_sync(0xffffffffu, qi - nt, at);
                if (lane == 0) {
                    found[0] = g * 32 + src;
                    found[1] = static_cast<int32_t>(kvh);
                    found[2] = t0 + at;
                    found[3] = static_cast<int32_t>(rest);
                    found[4] = q0, found[5] = n, found[6] = len, found[7] = qn;
                }
                break;
            }
            break;
        }
    }
    __syncthreads();
    w.b = 0, w.kvh = 0, w.q = 0, w.i = 0, w.qt = 0;
    if (first < total) {
        w.b = found[0], w.kvh = found[1], w.q = found[2], w.i = found[3];
        w.s.q0 = found[4], w.s.n = found[5], w.s.len = found[6], w.qt = found[7];
        w.t = paged_tiles<TILE, ROWS>(p, w.s.n, w.s.len, w.q);
    }
}

// ---------------------------------------------------------------- few query rows
//
// Decoding: up to 8 NB query rows (NB = 1, 2) share a kv head, every key and value byte is
// used once, and the kernel is bound by reading them. Per key and kv head 2 (D + 4) bytes
// arrive; at the copy rate of the chip an SM gets about 24 bytes a cycle, so a key of D = 128
// may take about 11 cycles. The small matrix instructions (mma.sync) keep up with that, and
// their register operands allow each warp to work alone:
// - a producer warp streams tiles of 128 keys through a ring of stages (one box holds the keys
//   and the values of a page, or of 64 keys of a larger one), across segment borders, so the
//   ring stays full while a segment is being finished;
// - 4 warps take 32 keys of each tile each, with their own running maximum, sum and output:
//   S^T = k q^T in int8 (m16n8k32), the exponentials, P^T moved into operand form
//   (movmatrix), and O^T += v^T (p s_v) with v's codes turned into f16 in registers
//   (m16n8k16). They meet only at the end of a segment.
// Keys and dims, not query rows, fill the 16 rows of each instruction: with 8 query rows half
// the instructions and accumulators of the other way round (64 sequences of up to 8192 keys, 32
// heads over 8 of 128: 103 against 138 us). Three blocks an SM with two stages for 8 rows, two
// blocks with three stages for 16: what the registers allow. That case now takes 103 us, 5.5
// TB/s; one token over 131071 keys 55 us (floor 42), about 10 us of it the start, the join and
// the tail.
//
// Fragments. Row i of an 8-key block is key PI(i), PI(2t) = 2t + (t >> 1) and PI(2t + 1) =
// PI(2t) ^ 4, which makes both the keys' 16-byte loads (two keys' rows per quarter warp) and
// the values' (four keys' rows) free of bank conflicts in the 128-byte swizzle. Lane (g, t)
// holds dims [(D / 8) g, (D / 8) (g + 1)) of the output: rows g and g + 8 of block j are its
// dims 2j and 2j + 1; its key bytes are 16-byte chunks: any order of the contracted index
// serves as long as both operands follow it.

constexpr int kFewTile = 128;     // keys per stage
constexpr int kFewBox = 64;       // keys of a box
constexpr int kFewThreads = 160;  // 4 warps and the producer
constexpr int kPagedMaxSms = 160; // the workspace's size assumes no more

template <int D, int NB>
struct FewConfig {
    static constexpr int ROWS = 8 * NB;                         // query rows of a tile
    static constexpr int PER_SM = NB == 1 ? 3 : 2;              // blocks, by registers
    static constexpr int NST = NB == 1 ? 2 : 3;                 // stages
    static constexpr int STAGE = 2 * kFewTile * D;              // codes of a stage
    static constexpr int SC_OFF = NST * STAGE;                  // scales: 2 * 128 fp32 a stage
    static constexpr int O_OFF = SC_OFF + NST * 2 * kFewTile * 4;
    static constexpr int O_LD = D + 4;                          // floats
    static constexpr int Q_OFF = O_OFF + ROWS * O_LD * 4;
    static constexpr int QS_OFF = Q_OFF + ROWS * D;
    static constexpr int ML_OFF = QS_OFF + ROWS * 4;            // [4 warps][ROWS] (m, l)
    static constexpr int BAR_OFF = ML_OFF + 4 * ROWS * 8;
    static constexpr int META_OFF = BAR_OFF + 2 * NST * 8;      // valid boxes of each stage
    static constexpr int SCAN_OFF = META_OFF + 16;
    static constexpr int SMEM_BYTES = 1024 + SCAN_OFF + 32;
    static_assert(BAR_OFF % 8 == 0 && META_OFF % 4 == 0 && NST * 4 <= 16 &&
                      PER_SM * (SMEM_BYTES + 1024 + 128) <= 228 * 1024,
                  "shared memory per SM");
    // Workspace: a piece's sums [ROWS][D], then its (m, l) [ROWS][2]; two pieces a block (0: of
    // the segment that began before the block, 1: of the one that goes on behind it).
    static constexpr int64_t PIECE = ROWS * (D + 2);
};

struct FewDesc {       // the segment that begins in a block and goes on behind it
    int32_t pieces;    // 0: none
    int32_t q0, rows;  // first query row of the sequence, valid rows of the tile
    int32_t head0;     // first head of the share
    int32_t r0;        // first (token, head) row of the tile
};

__device__ __forceinline__ void mma_m16n8k16_f16(float (&d)[4], uint32_t a0, uint32_t a1,
                                                  uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3},"
                 " {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Byte `j` of a and of b, two int8 codes, as an f16 pair (a low), exactly: with u = code + 128, the
// f16 pattern 0x64uu is 1024 + u.
__device__ __forceinline__ uint32_t codes_to_f16x2(uint32_t a, uint32_t b, int j)
{
    const uint32_t pick = static_cast<uint32_t>(j) * 0x1111u + 0x4400u;
    // bytes a_j, a_j, b_j, b_j
    const uint32_t t = (__byte_perm(a, b, pick) & 0x00ff00ffu) ^ 0x64806480u;
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(t), "r"(0xe480e480u));   // - 1152
    return r;
}

// Weights. A key's weight in the product with V is w = 2^(y - R) s_v, y its logit (base 2) and R its
// row's reference, in f16: 11 bits, within a range that R keeps. R moves (and the sums with it) when
// a key the row sees would exceed 2^kWeightTop, and then leaves that key kWeightLag bits below; so
// weights down to 2^-21 of the largest keep all bits, and what is below 2^-31 of it is lost. The
// output's error is then that of its own rounding (relative to 64 bits 0.00166; with weights in
// bf16, whose range needs no care, 0.00225). Two bf16 operands for a weight gave 0.00165, but 107
// us for 64 sequences of up to 8192 keys (bf16 102.5, f16 103.2).
// Since R follows log2 s_v, value scales may have any size. Where R is concerned they count as
// kLeastScale at least: the sums of 2^(y - R) over rows of zeros must not overflow.
constexpr float kWeightTop = 15.0f, kWeightLag = 8.0f, kLeastScale = 0x1p-80f;
__device__ __forceinline__ float weight_room(float sv)   // log2 s_v, and down to where R puts a key
{
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(fminf(fmaxf(fabsf(sv), kLeastScale), FLT_MAX)));
    return r - (kWeightTop - kWeightLag);
}

__device__ __forceinline__ uint4 lds_u4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// The 8x8 matrix of 16-bit values held two a lane (row lane / 4), transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ float lds_f(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Barrier of the four warps that compute.
__device__ __forceinline__ void few_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// One output row held by a warp (lane l has D / 32 elements): un-rotated, divided, stored.
// l == 0: the row saw no key.
template <int D>
__device__ __forceinline__ void paged_store_row(const PagedParams &p, float (&v)[D / 32], float l,
                                                int64_t t, int32_t head, uint32_t lane)
{
    constexpr int E = D / 32;
    warp_butterfly(v, p.group, lane);
    const float inv = l == 0.0f ? 0.0f : __fdiv_rn(p.c_g, l);
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(v[2 * i] * inv, v[2 * i + 1] * inv);
        w[i] = *reinterpret_cast<const uint32_t *>(&h2);
    }
    uint16_t *o = p.o + t * p.ldo + static_cast<int64_t>(head) * D + lane * E;
    if (E == 4)
        st_v2(o, w[0], w[E / 2 - 1]);
    else
        *reinterpret_cast<uint32_t *>(o) = w[0];
}

template <int D, int NB>
__global__ void __launch_bounds__(kFewThreads, FewConfig<D, NB>::PER_SM)
    attn_few_kernel(const __grid_constant__ CUtensorMap tmPool, const PagedParams p)
{
    using C = FewConfig<D, NB>;
    constexpr int NST = C::NST, ROWS = C::ROWS, E = D / 32, H2 = D / 64, DB = D / 16;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    __shared__ int abort_flag;
    volatile int *abort = &abort_flag;
    const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
    auto full = [&](uint32_t s) { return base + C::BAR_OFF + 8u * s; };
    auto empty = [&](uint32_t s) { return base + C::BAR_OFF + 8u * (NST + s); };
    volatile uint32_t *meta = reinterpret_cast<volatile uint32_t *>(smem + C::META_OFF);

    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 4);
        }
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmPool);
    }
    grid_dependents_launch();
    grid_dependency_wait();

    int64_t first, per, total;
    PagedWalk w;
    find_share<kFewTile, ROWS, kFewThreads>(p, gridDim.x, p.least_tiles,
                                                reinterpret_cast<int32_t *>(smem + C::SCAN_OFF), first, per,
                                                total, w);   // also: barriers initialised
    FewDesc *desc = reinterpret_cast<FewDesc *>(p.desc) + blockIdx.x;
    if (first >= total) {
        if (threadIdx.x == 0)
            desc->pieces = 0;
        return;
    }
    const int64_t count = min(first + per, total) - first;
    const int32_t pp = min(1 << p.page_shift, kFewBox);         // keys of a box
    const int32_t pp_shift = min(p.page_shift, 6);
    const int32_t nbox = kFewTile >> pp_shift, nbox_shift = 7 - pp_shift;

    if (warp == 4) {
        // ------------------------------------------------------------ producer
        fence_proxy_async_global();   // the kernel before may have stored the rows that the copies read
        int64_t n = 0;
        uint32_t st = 0, phase = 1;
        bool ok = true;
        while (ok && n < count) {
            const int32_t tiles = static_cast<int32_t>(min(static_cast<int64_t>(w.t.nt - w.i), count - n));
            const int32_t *row = p.table + static_cast<int64_t>(w.b) * p.table_ld;
            const PagedReach reach = paged_reach<ROWS>(p, w.s.n, w.s.len, w.q);
            // Page ids are read 32 at a time, a batch ahead of their use; entry e is box
            // e % nbox of the piece's tile e / nbox. Boxes that no row sees stay out.
            auto fetch = [&](int32_t e0) {
                const int32_t e = e0 + static_cast<int32_t>(lane);
                const int32_t i = w.i + (e >> nbox_shift);
                if (i >= w.i + tiles)
                    return -1;
                const int32_t j = (i < w.t.ns ? i : w.t.w0 + i - w.t.ns) * kFewTile + ((e & (nbox - 1)) << pp_shift);
                if (!reach.any(p, j, pp))
                    return -1;
                const int32_t id = row[j >> p.page_shift];
                if (id < 0 || id >= p.pages) {
                    atomicOr(&g_device_error, kDevIndex);
                    return -1;
                }
                return id;
            };
            int32_t ids = fetch(0), ids_next = fetch(32), e0 = 0;
            for (int32_t k = 0; k < tiles; ++k, ++n) {
                if (k * nbox >= e0 + 32) {
                    ids = ids_next;
                    e0 += 32;
                    ids_next = fetch(e0 + 32);
                }
                // lane c < nbox has box c of this tile
                const int32_t id = __shfl_sync(0xffffffffu, ids, (k * nbox - e0 + static_cast<int32_t>(lane)) & 31);
                const bool mine = static_cast<int32_t>(lane) < nbox && id >= 0;
                const uint32_t valid = __ballot_sync(0xffffffffu, mine);
                bool got = true;
                if (lane == 0)
                    got = mbar_wait_bounded(empty(st), phase, abort, p.timeout_ns);
                if (!__shfl_sync(0xffffffffu, static_cast<int>(got), 0)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    meta[st] = valid;
                    mbar_arrive_expect_tx(full(st), static_cast<uint32_t>(__popc(valid)) * 2u * pp * (D + 4));
                }
                __syncwarp();
                if (mine) {
                    const int32_t prow = static_cast<int32_t>(((static_cast<int64_t>(id) * p.Hkv + w.kvh) * 2) << p.page_shift);
                    const uint32_t dst = base + st * C::STAGE + lane * 2u * pp * D;
                    const uint32_t sdst = base + C::SC_OFF + (st * 2 * kFewTile + lane * 2 * pp) * 4;
                    if (p.page_shift <= 6) {     // the box is the page: its keys, then its values
                        tma_load_2d(dst, &tmPool, full(st), 0, prow);
                        bulk_load_1d(sdst, p.scales + prow, 8u * pp, full(st));
                    } else {
                        const int32_t i = w.i + k;
                        const int32_t j = (i < w.t.ns ? i : w.t.w0 + i - w.t.ns) * kFewTile + static_cast<int32_t>(lane) * pp;
                        const int32_t krow = prow + (j & ((1 << p.page_shift) - 1)), vrow = krow + (1 << p.page_shift);
                        tma_load_2d(dst, &tmPool, full(st), 0, krow);
                        tma_load_2d(dst + kFewBox * D, &tmPool, full(st), 0, vrow);
                        bulk_load_1d(sdst, p.scales + krow, 4u * pp, full(st));
                        bulk_load_1d(sdst + 4 * pp, p.scales + vrow, 4u * pp, full(st));
                    }
                }
                if (++st == NST)
                    st = 0, phase ^= 1u;
            }
            if (n < count)
                walk_next_segment<kFewTile, ROWS>(p, w);
        }
        // every copy has landed before the block may end (its consumers may have given up)
        if (lane == 0) {
            volatile int no_abort = 0;
            for (int64_t j = n - NST < 0 ? 0 : n - NST; j < n; ++j)
                mbar_wait_bounded(full(static_cast<uint32_t>(j % NST)), static_cast<uint32_t>(j / NST) & 1u, &no_abort,
                                  p.timeout_ns);
        }
        return;
    }

    // ---------------------------------------------------------------- the four warps
    const uint32_t g = lane >> 2, t = lane & 3u;
    const uint32_t e = 2u * t + (t >> 1);                         // PI(2t)
    const uint32_t krow_n = (2u * (g >> 1) + (g >> 2)) ^ ((g & 1u) << 2);   // PI(g)
    const int32_t my_key = static_cast<int32_t>(warp) * 32;
    // boxes and box rows of this warp's two runs of 16 keys
    const uint32_t my_box[2] = {static_cast<uint32_t>(my_key >> pp_shift), static_cast<uint32_t>((my_key + 16) >> pp_shift)};
    const uint32_t my_row[2] = {my_box[0] * 2u * pp + (my_key & (pp - 1)),
                                my_box[1] * 2u * pp + ((my_key + 16) & (pp - 1))};
    const uint32_t my_boxes = (1u << my_box[0]) | (1u << my_box[1]);
    float *obuf = reinterpret_cast<float *>(smem + C::O_OFF);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::ML_OFF);
    float *qs = reinterpret_cast<float *>(smem + C::QS_OFF);
    bool ok = true;
    int64_t n = 0;
    uint32_t st = 0, phase = 0;
    int piece_no = 0;
    while (n < count) {
        const int32_t r0 = w.q * ROWS, head0 = w.kvh * p.share;
        const int32_t rows = min(ROWS, w.s.n * p.share - r0);
        const int32_t tiles = static_cast<int32_t>(min(static_cast<int64_t>(w.t.nt - w.i), count - n));
        // the query rows' codes and scales (rows past the last: zeros)
        {
            constexpr int LANES = D == 128 && NB == 1 ? 16 : 8, QE = D / LANES;   // of a row; elements of a lane
            const int32_t lr = static_cast<int32_t>(warp) * (32 / LANES) + static_cast<int32_t>(lane) / LANES, r = r0 + lr;
            if (static_cast<int32_t>(warp) * (32 / LANES) < ROWS) {
                const uint32_t at = lane % LANES * QE;
                float v[QE];
#pragma unroll
                for (int i = 0; i < QE / 8; ++i) {
                    uint4 a = make_uint4(0u, 0u, 0u, 0u);
                    if (lr < rows) {
                        const int32_t ti = by_share(p, r);
                        a = ld_nc_v4(p.q + static_cast<int64_t>(w.s.q0 + ti) * p.ldq +
                                     static_cast<int64_t>(head0 + r - ti * p.share) * D + at + 8 * i);
                    }
                    const uint32_t x[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        v[8 * i + 2 * u] = __uint_as_float(x[u] << 16);
                        v[8 * i + 2 * u + 1] = __uint_as_float(x[u] & 0xffff0000u);
                    }
                }
                uint32_t codes[QE / 4];
                float sq;
                quant_row_lanes<QE, LANES>(v, p.group, p.c_g, lane, codes, sq);
#pragma unroll
                for (int i = 0; i < QE / 4; ++i)
                    *reinterpret_cast<uint32_t *>(smem + C::Q_OFF + lr * D + at + 4 * i) = codes[i];
                if (lane % LANES == 0)
                    qs[lr] = sq;
            }
        }
        few_sync();
        uint4 qb[NB][H2];    // query row g + 8 nb, 16-byte chunk t of each 64-element half
        float row_f[NB][2];  // of query rows 8 nb + 2t, 2t + 1
        int32_t pos[NB][2], low[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int h = 0; h < H2; ++h)
                qb[nb][h] = lds_u4(base + C::Q_OFF + (static_cast<int32_t>(g) + 8 * nb) * D + h * 64 + t * 16);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int32_t lr = 8 * nb + 2 * static_cast<int32_t>(t) + c;
                // logit * log2 e = (acc * s_k) * row_f; the floor keeps 0 * -inf out (attention.cuh)
                row_f[nb][c] = fmaxf(qs[lr] * p.scale * 1.4426950408889634f, 0x1p-126f);
                pos[nb][c] = w.s.len - w.s.n + by_share(p, r0 + min(lr, rows - 1));
                low[nb][c] = p.window > 0 ? pos[nb][c] - p.window + 1 : INT32_MIN;
            }
        }
        const int32_t pos_first = w.s.len - w.s.n + by_share(p, r0);
        const int32_t pos_last = w.s.len - w.s.n + by_share(p, r0 + rows - 1);
        const int32_t low_first = p.window > 0 ? pos_first - p.window + 1 : INT32_MIN;
        const int32_t low_last = p.window > 0 ? pos_last - p.window + 1 : INT32_MIN;
        float m[NB][2], l[NB][2];
        float o[NB][DB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            m[nb][0] = m[nb][1] = -INFINITY;
            l[nb][0] = l[nb][1] = 0.0f;
#pragma unroll
            for (int j = 0; j < DB; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[nb][j][i] = 0.0f;
        }

#pragma unroll 1
        for (int32_t k = 0; k < tiles; ++k) {
            const int32_t ti = w.i + k;
            const int32_t j0 = (ti < w.t.ns ? ti : w.t.w0 + ti - w.t.ns) * kFewTile + my_key;
            const bool got = ok && mbar_wait_bounded(full(st), phase, abort, p.timeout_ns);
            ok = __all_sync(0xffffffffu, got);
            // nothing of these 32 keys is visible to any row: leave them
            if (ok && j0 <= pos_last && (j0 + 31 >= low_first || j0 < p.sinks)) {
                const uint32_t there = meta[st];
                const bool whole = j0 + 31 <= pos_first && (j0 >= low_last || j0 + 32 <= p.sinks) &&
                                   (there & my_boxes) == my_boxes;
                const uint32_t codes[2] = {base + st * C::STAGE + my_row[0] * D, base + st * C::STAGE + my_row[1] * D};
                const uint32_t sc = base + C::SC_OFF + st * 2 * kFewTile * 4;
                // y[nb][kb][c]: key 8 kb + PI(g), query row 8 nb + 2t + c
                float y[NB][4][2];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    int32_t acc[NB][4] = {};
#pragma unroll
                    for (int h = 0; h < H2; ++h) {
                        const uint32_t sw = D == 128 ? (t + 4u * h) ^ krow_n : t ^ (krow_n >> 1);
                        const uint4 a = lds_u4(codes[kk] + krow_n * D + sw * 16u);
                        const uint4 b = lds_u4(codes[kk] + (8u + krow_n) * D + sw * 16u);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            mma_m16n8k32_s8(acc[nb], a.x, b.x, a.y, b.y, qb[nb][h].x, qb[nb][h].y);
                            mma_m16n8k32_s8(acc[nb], a.z, b.z, a.w, b.w, qb[nb][h].z, qb[nb][h].w);
                        }
                    }
                    const uint32_t a = sc + (my_row[kk] + krow_n) * 4u;
                    const float sk0 = lds_f(a), sk1 = lds_f(a + 32u);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        y[nb][2 * kk][0] = static_cast<float>(acc[nb][0]) * sk0;
                        y[nb][2 * kk][1] = static_cast<float>(acc[nb][1]) * sk0;
                        y[nb][2 * kk + 1][0] = static_cast<float>(acc[nb][2]) * sk1;
                        y[nb][2 * kk + 1][1] = static_cast<float>(acc[nb][3]) * sk1;
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int32_t j = j0 + 8 * kb + static_cast<int32_t>(krow_n);
                                const bool see = j <= pos[nb][c] && (j >= low[nb][c] || j < p.sinks) &&
                                                 ((there >> my_box[kb >> 1]) & 1u) != 0u;
                                y[nb][kb][c] = see ? y[nb][kb][c] : -INFINITY;
                            }
                }
                float sv[4];   // of keys 8 kb + PI(g)
#pragma unroll
                for (int kb = 0; kb < 4; ++kb)
                    sv[kb] = lds_f(sc + (my_row[kb >> 1] + 8u * (kb & 1) + pp + krow_n) * 4u);
                // whether a weight may be too large: the largest logit with the largest scale
                const float room = weight_room(fmaxf(max3f(fabsf(sv[0]), fabsf(sv[1]), fabsf(sv[2])), fabsf(sv[3])));
                bool grew = false;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        grew |= __fmaf_rn(fmaxf(max3f(y[nb][0][c], y[nb][1][c], y[nb][2][c]), y[nb][3][c]), row_f[nb][c],
                                          room) > m[nb][c] + kWeightLag;
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        float alpha[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float mb = -INFINITY;   // key by key; hidden keys have no part
#pragma unroll
                            for (int kb = 0; kb < 4; ++kb)
                                mb = fmaxf(mb, __fmaf_rn(y[nb][kb][c], row_f[nb][c], weight_room(sv[kb])));
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1)
                                mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, x));
                            const bool grow = mb > m[nb][c] + kWeightLag;
                            alpha[c] = grow ? ex2_approx(m[nb][c] - mb) : 1.0f;
                            m[nb][c] = grow ? mb : m[nb][c];
                            l[nb][c] *= alpha[c];
                        }
#pragma unroll
                        for (int j = 0; j < DB; ++j) {
                            mul2(o[nb][j][0], o[nb][j][1], o[nb][j][0], o[nb][j][1], alpha[0], alpha[1]);
                            mul2(o[nb][j][2], o[nb][j][3], o[nb][j][2], o[nb][j][3], alpha[0], alpha[1]);
                        }
                    }
                }
                uint32_t pb[NB][4];   // weights: keys PI(2t), PI(2t + 1), query row g
                auto weigh = [&](auto masked) {
#pragma unroll
                    for (int kb = 0; kb < 4; ++kb) {
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            float pr[2];
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const float neg_m = m[nb][c] == -INFINITY ? 0.0f : -m[nb][c];
                                const float x = ex2_approx(__fmaf_rn(y[nb][kb][c], row_f[nb][c], neg_m));
                                l[nb][c] += x;
                                pr[c] = x * sv[kb];
                                // a hidden key adds 0 whatever its scale holds
                                if (decltype(masked)::value)
                                    pr[c] = y[nb][kb][c] == -INFINITY ? 0.0f : pr[c];
                            }
                            const __half2 h2 = __floats2half2_rn(pr[0], pr[1]);
                            pb[nb][kb] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h2));
                        }
                    }
                };
                if (whole)
                    weigh(std::bool_constant<false>());
                else
                    weigh(std::bool_constant<true>());
                // values of keys PI(2t), PI(2t + 1) of two 8-key blocks, this lane's D / 8 dims
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    uint32_t vb[4][D / 32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t kr = (i & 1) ? e ^ 4u : e;
                        const uint32_t row = codes[kk] + (pp + 8u * (i >> 1) + kr) * D;
                        if (D == 128) {
                            const uint4 a = lds_u4(row + ((g ^ kr) << 4));
                            vb[i][0] = a.x, vb[i][1] = a.y, vb[i][D / 32 - 2] = a.z, vb[i][D / 32 - 1] = a.w;
                        } else {
                            const uint32_t a = row + (((g >> 1) ^ (kr >> 1)) << 4) + (g & 1u) * 8u;
                            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                         : "=r"(vb[i][0]), "=r"(vb[i][1]) : "r"(a) : "memory");
                        }
                    }
#pragma unroll
                    for (int j = 0; j < DB; ++j) {
                        uint32_t a[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            a[i] = codes_to_f16x2(vb[i & 2][j >> 1], vb[(i & 2) + 1][j >> 1], (2 * j + (i & 1)) & 3);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            mma_m16n8k16_f16(o[nb][j], a[0], a[1], a[2], a[3], pb[nb][2 * kk], pb[nb][2 * kk + 1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(empty(st));
            if (++st == NST)
                st = 0, phase ^= 1u;
        }
        n += tiles;

        // ------------------------------------------------ join the four warps' sums
        // the maximum over the warps first; then one warp after the other adds its sums
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1)
                    l[nb][c] += __shfl_xor_sync(0xffffffffu, l[nb][c], x);
                if (g == 0)
                    ml[warp * ROWS + 8 * nb + 2 * t + c] = make_float2(m[nb][c], l[nb][c]);
            }
        few_sync();
        float scale_o[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float mm = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mm = fmaxf(mm, ml[i * ROWS + 8 * nb + 2 * t + c].x);
                scale_o[nb][c] = m[nb][c] == -INFINITY ? 0.0f : ex2_approx(m[nb][c] - mm);
            }
        // o[nb][j][c], o[nb][j][2 + c]: dims 2j, 2j + 1 of the lane's, query row 8 nb + 2t + c
#pragma unroll 1
        for (uint32_t turn = 0; turn < 4; ++turn) {
            if (turn == warp) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int j = 0; j < DB; j += 2) {
                            float4 *at = reinterpret_cast<float4 *>(obuf + (8 * nb + 2 * t + c) * C::O_LD + 2 * DB * g + 2 * j);
                            float4 x = turn == 0 ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *at;
                            x.x = __fmaf_rn(o[nb][j][c], scale_o[nb][c], x.x);
                            x.y = __fmaf_rn(o[nb][j][2 + c], scale_o[nb][c], x.y);
                            x.z = __fmaf_rn(o[nb][j + 1][c], scale_o[nb][c], x.z);
                            x.w = __fmaf_rn(o[nb][j + 1][2 + c], scale_o[nb][c], x.w);
                            *at = x;
                        }
            }
            few_sync();
        }
        const bool begins = w.i == 0, ends = w.i + tiles == w.t.nt;
        const bool good = ok && *abort == 0;   // no role gave up waiting
        float *ws = p.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (begins ? 1 : 0)) * C::PIECE;
#pragma unroll 1
        for (int32_t lr = static_cast<int32_t>(warp); lr < rows; lr += 4) {
            float mm = -INFINITY, ll = 0.0f, v[E];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mm = fmaxf(mm, ml[i * ROWS + lr].x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = ml[i * ROWS + lr];
                ll = __fmaf_rn(x.y, x.x == -INFINITY ? 0.0f : ex2_approx(x.x - mm), ll);
            }
#pragma unroll
            for (int i = 0; i < E; ++i)
                v[i] = obuf[lr * C::O_LD + lane * E + i];
            if (qs[lr] != qs[lr] && ll > 0.0f)   // a query row that is not finite, where it sees a key
                ll = nanf("");
            const int32_t r = r0 + lr, tok = by_share(p, r);
            if (begins && ends) {
                if (good)
                    paged_store_row<D>(p, v, ll, w.s.q0 + tok, head0 + r - tok * p.share, lane);
            } else {
#pragma unroll
                for (int d = 0; d < E; ++d)
                    ws[lr * D + lane * E + d] = v[d];
                if (lane == 0)
                    *reinterpret_cast<float2 *>(ws + ROWS * D + 2 * lr) = make_float2(mm, good ? ll : nanf(""));
            }
        }
        if (threadIdx.x == 0 && begins && !ends) {
            // the segment's last tile is nt - tiles further on: that many blocks hold pieces
            const int64_t end = first + n - tiles + w.t.nt - 1;
            desc->pieces = static_cast<int32_t>(end / per) - static_cast<int32_t>(blockIdx.x) + 1;
            desc->q0 = w.s.q0;
            desc->rows = rows;
            desc->head0 = head0;
            desc->r0 = r0;
            piece_no = 1;
        }
        if (n < count)
            walk_next_segment<kFewTile, ROWS>(p, w);
        few_sync();   // obuf, ml and the query codes are free again
    }
    if (threadIdx.x == 0 && piece_no == 0)
        desc->pieces = 0;
}

// Joins the pieces of the segments that several blocks share: block (c, y) takes rows of the
// segment that begins in block c. The block's eight warps take the pieces of one row in turn
// (few rows, up to a whole grid of pieces), or a row each (ROWS > 16: many rows, few pieces).
constexpr int kJoinThreads = 256;

template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const PagedParams p)
{
    constexpr int E = D / 32, W = ROWS > 16 ? 1 : kJoinThreads / 32;   // warps of a row
    constexpr int64_t PIECE = ROWS * (D + 2);
    __shared__ float part[W][D];
    __shared__ float2 part_ml[W];
    grid_dependents_launch();
    grid_dependency_wait();
    const FewDesc d = reinterpret_cast<const FewDesc *>(p.desc)[blockIdx.x];
    const int32_t warp = static_cast<int32_t>(threadIdx.x >> 5);
    const uint32_t lane = lane_id();
    if (d.pieces == 0)
        return;
    const int32_t step = static_cast<int32_t>(gridDim.y) * (W == 1 ? kJoinThreads / 32 : 1);
    for (int32_t lr = W == 1 ? static_cast<int32_t>(blockIdx.y) * (kJoinThreads / 32) + warp : static_cast<int32_t>(blockIdx.y);
         lr < d.rows; lr += step) {
        float m = -INFINITY, l = 0.0f, v[E];
#pragma unroll
        for (int i = 0; i < E; ++i)
            v[i] = 0.0f;
#pragma unroll 4
        for (int32_t k = W == 1 ? 0 : warp; k < d.pieces; k += W) {
            const float *ws = p.partial + ((static_cast<int64_t>(blockIdx.x) + k) * 2 + (k == 0 ? 1 : 0)) * PIECE;
            const float2 x = *reinterpret_cast<const float2 *>(ws + ROWS * D + 2 * lr);
            float a[E];
#pragma unroll
            for (int i = 0; i < E; ++i)
                a[i] = ws[lr * D + lane * E + i];
            const float mn = fmaxf(m, x.x);
            const float fo = m == -INFINITY ? 0.0f : ex2_approx(m - mn);
            const float fn = x.x == -INFINITY ? 0.0f : ex2_approx(x.x - mn);
            l = __fmaf_rn(x.y, fn, l * fo);
#pragma unroll
            for (int i = 0; i < E; ++i)
                v[i] = __fmaf_rn(a[i], fn, v[i] * fo);
            m = mn;
        }
        const int32_t r = d.r0 + lr, tok = by_share(p, r);
        if constexpr (W == 1) {
            paged_store_row<D>(p, v, l, d.q0 + tok, d.head0 + r - tok * p.share, lane);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                part[warp][lane * E + i] = v[i];
            if (lane == 0)
                part_ml[warp] = make_float2(m, l);
            __syncthreads();
            if (warp == 0) {
                float mm = -INFINITY, ll = 0.0f;
#pragma unroll
                for (int i = 0; i < W; ++i)
                    mm = fmaxf(mm, part_ml[i].x);
#pragma unroll
                for (int i = 0; i < E; ++i)
                    v[i] = 0.0f;
#pragma unroll
                for (int k = 0; k < W; ++k) {
                    const float f = part_ml[k].x == -INFINITY ? 0.0f : ex2_approx(part_ml[k].x - mm);
                    ll = __fmaf_rn(part_ml[k].y, f, ll);
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        v[i] = __fmaf_rn(part[k][lane * E + i], f, v[i]);
                }
                paged_store_row<D>(p, v, ll, d.q0 + tok, d.head0 + r - tok * p.share, lane);
            }
            __syncthreads();
        }
    }
}

} // namespace sdnq
