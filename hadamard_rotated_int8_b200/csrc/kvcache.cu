// The paged key/value cache and the attention over it: validation and launches.
//
// This file is part of libsdnq.cu's translation unit (included at its end).

#include "attention_paged.cuh"
#include "attention_paged_chunk.cuh"
#include "kvcache.cuh"

namespace sdnq {
namespace {

// Sizes shared by every call on a cache; codes and scales are required unless there is no work.
sdnq_status validate_cache(const void *codes, const void *scales, int64_t pages, int32_t page,
                           int64_t Hkv, int64_t D, int32_t group)
{
    if (pages < 0 || Hkv < 1 || Hkv > 65536)
        return SDNQ_ERR_SHAPE;
    if ((D != 64 && D != 128) || !is_pow2(page) || page < SDNQ_KV_MIN_PAGE ||
        page > SDNQ_KV_MAX_PAGE || !is_pow2(group) || group < SDNQ_MIN_GROUP ||
        group > SDNQ_MAX_GROUP)
        return SDNQ_ERR_UNSUPPORTED;
    // rows of the pool are numbered in 32 bits by the copy engine
    if (pages > INT32_MAX / (2 * Hkv * page))
        return SDNQ_ERR_SHAPE;
    if (!aligned(codes, 16) || !aligned(scales, 16))
        return SDNQ_ERR_ALIGN;
    return SDNQ_OK;
}

int32_t log2_of(int64_t v)
{
    int32_t s = 0;
    while ((1ll << s) < v)
        ++s;
    return s;
}

float rotation_factor(int64_t g) { return static_cast<float>(1.0 / std::sqrt(static_cast<double>(g))); }

sdnq_status validate_kv_rows(const void *k, int64_t ldk, const void *v, int64_t ldv,
                             const void *slots, int64_t T, int64_t Hkv, int64_t D, int32_t group,
                             const void *codes, const void *scales, int64_t pages, int32_t page)
{
    if (T != 0 && (!k || !v || !slots || !codes || !scales))
        return SDNQ_ERR_NULL;
    if (T < 0 || T > INT32_MAX)
        return SDNQ_ERR_SHAPE;
    const sdnq_status st = validate_cache(codes, scales, pages, page, Hkv, D, group);
    if (st != SDNQ_OK)
        return st;
    if (ldk < Hkv * D || ldv < Hkv * D)
        return SDNQ_ERR_SHAPE;
    if (ldk % 8 != 0 || ldv % 8 != 0 || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
        return SDNQ_ERR_ALIGN;
    return SDNQ_OK;
}

// Persistent grids: the blocks that the SMs hold at once.
template <int D>
void launch_kv_write(const KvParams &p, int sm_count, cudaStream_t cs)
{
    constexpr int rows = 8 * (kWriteThreads / 32);
    const int64_t blocks = (p.rows + rows - 1) / rows, most = static_cast<int64_t>(sm_count) * 3;
    launch_programmatic(kv_write_kernel<D>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(kWriteThreads),
                        0, cs, p);
}

template <int D>
void launch_kv_read(const KvParams &p, int sm_count, cudaStream_t cs)
{
    constexpr int warps = kReadThreads / 32;
    const int64_t blocks = ((p.T + 15) / 16 * (2 * p.Hkv) + warps - 1) / warps, most = static_cast<int64_t>(sm_count) * 4;
    launch_programmatic(kv_read_kernel<D>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(kReadThreads), 0,
                        cs, p);
}

template <bool WRITE>
sdnq_status run_kv(uint16_t *k, int64_t ldk, uint16_t *v, int64_t ldv, const int64_t *slots,
                   int64_t T, int64_t Hkv, int64_t D, int32_t group, int8_t *codes, float *scales,
                   int64_t pages, int32_t page, void *stream)
{
    sdnq_status st = validate_kv_rows(k, ldk, v, ldv, slots, T, Hkv, D, group, codes, scales, pages,
                                      page);
    if (st != SDNQ_OK)
        return st;
    DeviceInfo dev;
    if ((st = current_device(&dev)) != SDNQ_OK)
        return st;
    if (T == 0)
        return SDNQ_OK;
    const int64_t g = group < D ? group : D;
    KvParams p = {};
    p.k = k;
    p.v = v;
    p.ldk = ldk;
    p.ldv = ldv;
    p.slots = slots;
    p.codes = codes;
    p.scales = scales;
    p.T = T;
    p.rows = T * 2 * Hkv;
    p.nslots = pages * page;
    p.Hkv = static_cast<int32_t>(Hkv);
    p.page_shift = log2_of(page);
    p.group = static_cast<int32_t>(g);
    p.c_g = rotation_factor(g);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    cudaGetLastError();
    if (WRITE)
        D == 128 ? launch_kv_write<128>(p, dev.sm_count, cs) : launch_kv_write<64>(p, dev.sm_count, cs);
    else
        D == 128 ? launch_kv_read<128>(p, dev.sm_count, cs) : launch_kv_read<64>(p, dev.sm_count, cs);
    return launch_status();
}

// The workspace of one call: what the blocks of each kernel say of their last segment, then the
// few-row kernel's pieces, then the chunk kernel's.
constexpr int64_t kPagedFewDescs = 3ll * kPagedMaxSms, kPagedChunkDescs = kPagedMaxSms;
constexpr int64_t kPagedDescBytes = ((kPagedFewDescs + kPagedChunkDescs) * sizeof(FewDesc) + 255) / 256 * 256;

template <int D>
constexpr int64_t few_pieces_bytes()
{
    static_assert(FewConfig<D, 1>::PER_SM <= 3 && FewConfig<D, 2>::PER_SM <= 3, "kPagedFewDescs");
    const int64_t one = FewConfig<D, 1>::PER_SM * FewConfig<D, 1>::PIECE, two = FewConfig<D, 2>::PER_SM * FewConfig<D, 2>::PIECE;
    return (2ll * kPagedMaxSms * (one > two ? one : two) * 4 + 255) / 256 * 256;
}

int64_t paged_workspace(int64_t D)
{
    return kPagedDescBytes + (D == 128 ? few_pieces_bytes<128>() + 2ll * kPagedMaxSms * ChunkConfig<128>::PIECE * 4
                                       : few_pieces_bytes<64>() + 2ll * kPagedMaxSms * ChunkConfig<64>::PIECE * 4);
}

// The pool as rows of D codes, boxes of `rows` of them.
template <int D>
bool make_pool_map(CUtensorMap *map, const PagedParams &p, uint32_t rows)
{
    const uint64_t pool_rows = static_cast<uint64_t>(p.pages > 0 ? p.pages : 1) * p.Hkv * 2 << p.page_shift;
    return make_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.codes, D, pool_rows, D, D, rows,
                        D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

template <int D, int NB>
sdnq_status launch_few(const PagedParams &p, const DeviceInfo &dev, int sms, cudaStream_t cs)
{
    using C = FewConfig<D, NB>;
    CUtensorMap map;
    const uint32_t page = 1u << p.page_shift;
    if (!make_pool_map<D>(&map, p, page <= kFewBox ? 2 * page : kFewBox))
        return SDNQ_ERR_CUDA;
    static PerDeviceCache<1> smem;
    if (!smem_attr_once(smem, dev.index, attn_few_kernel<D, NB>, C::SMEM_BYTES)) {
        cudaGetLastError();
        return SDNQ_ERR_CUDA;
    }
    const unsigned blocks = static_cast<unsigned>(C::PER_SM * sms);
    launch_programmatic(attn_few_kernel<D, NB>, dim3(blocks), dim3(kFewThreads), C::SMEM_BYTES, cs, map, p);
    launch_programmatic(attn_join_kernel<D, C::ROWS>, dim3(blocks, 2), dim3(kJoinThreads), 0, cs, p);
    return launch_status();
}

template <int D>
sdnq_status launch_chunk(const PagedParams &p, const DeviceInfo &dev, int sms, cudaStream_t cs)
{
    using C = ChunkConfig<D>;
    CUtensorMap map;
    const uint32_t page = 1u << p.page_shift;
    if (!make_pool_map<D>(&map, p, page <= kChunkTile ? page : kChunkTile))
        return SDNQ_ERR_CUDA;
    static PerDeviceCache<1> smem;
    if (!smem_attr_once(smem, dev.index, attn_chunk_kernel<D>, C::SMEM_BYTES)) {
        cudaGetLastError();
        return SDNQ_ERR_CUDA;
    }
    const unsigned blocks = static_cast<unsigned>(sms);
    launch_programmatic(attn_chunk_kernel<D>, dim3(blocks), dim3(kChunkThreads), C::SMEM_BYTES, cs, map, p);
    launch_programmatic(attn_join_kernel<D, kChunkRows>, dim3(blocks, 16), dim3(kJoinThreads), 0, cs, p);
    return launch_status();
}

// Query rows of a kv head above which a sequence goes to the tensor-memory kernel; below, each
// 16 rows are another pass over its keys. Measured with heads of 128, us there and in passes:
//   16 sequences of 4096 keys, 32 heads over 8: 36 rows 92 and 135, 64 rows 93 and 166;
//   one of 16384 keys:                          36 rows 49 and 50, 64 rows 50 and 57;
//   one token each of 16 sequences of 4096, all heads on one kv head: 40 heads 39 and 42, 64 heads
//   40 and 45, 128 heads 41 and 60.
// One such sequence alone is faster in passes (16384 keys: 40 heads 49 and 33, 128 heads 52 and
// 32; 131072 keys: 65 and 60, 68 and 86): the rule knows the rows of a sequence, not how many
// segments there are, whose lengths are on the device.
constexpr int32_t kPagedFewRows = 32;

template <int D>
sdnq_status launch_paged(PagedParams p, const DeviceInfo &dev, int64_t max_q, uint8_t *ws, cudaStream_t cs)
{
    const int sms = dev.sm_count < kPagedMaxSms ? dev.sm_count : kPagedMaxSms;
    p.desc = ws;
    p.partial = reinterpret_cast<float *>(ws + kPagedDescBytes);
    p.rows_min = 0;
    p.rows_max = INT32_MAX;
    p.least_tiles = 2;   // a share below 256 keys costs more to start and join than it saves
    if (max_q <= 8 / p.share)
        return launch_few<D, 1>(p, dev, sms, cs);
    if (max_q <= kPagedFewRows / p.share)
        return launch_few<D, 2>(p, dev, sms, cs);
    p.rows_max = kPagedFewRows;
    const sdnq_status st = launch_few<D, 2>(p, dev, sms, cs);
    if (st != SDNQ_OK)
        return st;
    p.rows_min = kPagedFewRows;
    p.rows_max = INT32_MAX;
    p.least_tiles = 1;
    p.desc = ws + kPagedFewDescs * sizeof(FewDesc);
    p.partial = reinterpret_cast<float *>(ws + kPagedDescBytes + few_pieces_bytes<D>());
    return launch_chunk<D>(p, dev, sms, cs);
}

// Largest context, window and sink count that the kernels' 32-bit positions hold; most sequences
// (they are counted in groups of 32).
constexpr int64_t kPagedMaxKeys = 1ll << 30, kPagedMaxSeqs = INT32_MAX - 31;

sdnq_status run_attention_paged(const uint16_t *q, int64_t ldq, int64_t T, int64_t H,
                                const int32_t *cu_q, const int32_t *lens, int64_t B,
                                const int32_t *table, int64_t max_pages, int64_t ldt, const int8_t *codes,
                                const float *scales, int64_t pages, int32_t page, int64_t Hkv,
                                int64_t D, int64_t max_q, int32_t group, float scale,
                                int64_t window, int64_t sinks, void *ws, int64_t ws_bytes,
                                uint16_t *out, int64_t ldo, void *stream)
{
    const bool work = T != 0 && B != 0;
    if (work && (!q || !lens || (!table && max_pages != 0) || !codes || !scales || !ws || !out))
        return SDNQ_ERR_NULL;
    if (T < 0 || B < 0 || T > INT32_MAX || B > kPagedMaxSeqs || H < 1 || H > 65536 || max_q < 1 ||
        window < 0 || sinks < 0 || max_pages < 0 || ldt < max_pages)
        return SDNQ_ERR_SHAPE;
    sdnq_status st = validate_cache(codes, scales, pages, page, Hkv, D, group);
    if (st != SDNQ_OK)
        return st;
    if (H % Hkv != 0 || T * H > INT32_MAX || (cu_q == nullptr && T < B) ||
        max_pages > kPagedMaxKeys / page || ldq < H * D || ldo < H * D)
        return SDNQ_ERR_SHAPE;
    if (!(scale >= 0.0f && scale <= FLT_MAX))
        return SDNQ_ERR_UNSUPPORTED;
    if (ldq % 8 != 0 || ldo % 8 != 0 || !aligned(q, 16) || !aligned(out, 16) || !aligned(cu_q, 4) ||
        !aligned(lens, 4) || !aligned(table, 4) || !aligned(ws, 256))
        return SDNQ_ERR_ALIGN;
    if (work && ws_bytes < paged_workspace(D))
        return SDNQ_ERR_SHAPE;
    DeviceInfo dev;
    if ((st = current_device(&dev)) != SDNQ_OK)
        return st;
    if (!work)
        return SDNQ_OK;
    const int64_t g = group < D ? group : D;
    PagedParams p = {};
    p.q = q;
    p.o = out;
    p.ldq = ldq;
    p.ldo = ldo;
    p.cu = cu_q;
    p.lens = lens;
    p.table = table;
    p.table_ld = ldt;
    p.codes = codes;
    p.scales = scales;
    p.pages = pages;
    p.T = static_cast<int32_t>(T);
    p.B = static_cast<int32_t>(B);
    p.Hkv = static_cast<int32_t>(Hkv);
    p.share = static_cast<int32_t>(H / Hkv);
    const int32_t bits = log2_of(p.share);   // division by the share as a product (rounded up)
    p.share_shift = static_cast<uint32_t>(31 + bits);
    p.share_mul = static_cast<uint32_t>(((1ull << p.share_shift) + p.share - 1) / p.share);
    p.page_shift = log2_of(page);
    p.cap = static_cast<int32_t>(max_pages * page);
    p.window = static_cast<int32_t>(window < kPagedMaxKeys ? window : kPagedMaxKeys);
    p.sinks = static_cast<int32_t>(sinks < kPagedMaxKeys ? sinks : kPagedMaxKeys);
    p.group = static_cast<int32_t>(g);
    p.scale = scale;
    p.c_g = rotation_factor(g);
    cudaGetLastError();
    p.timeout_ns = kDefaultTimeoutNs;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return D == 128 ? launch_paged<128>(p, dev, max_q, static_cast<uint8_t *>(ws), cs)
                    : launch_paged<64>(p, dev, max_q, static_cast<uint8_t *>(ws), cs);
}

} // namespace
} // namespace sdnq

SDNQ_API sdnq_status sdnq_kv_write(const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv,
                                   const int64_t *slots, int64_t T, int64_t Hkv, int64_t D,
                                   int32_t group, int8_t *codes, float *scales, int64_t pages,
                                   int32_t page, void *stream)
{
    SDNQ_NVTX_RANGE();
    return run_kv<true>(const_cast<uint16_t *>(k), ldk, const_cast<uint16_t *>(v), ldv, slots, T,
                        Hkv, D, group, codes, scales, pages, page, stream);
}

SDNQ_API sdnq_status sdnq_kv_read(const int64_t *slots, int64_t T, const int8_t *codes,
                                  const float *scales, int64_t pages, int32_t page, int64_t Hkv,
                                  int64_t D, int32_t group, uint16_t *k, int64_t ldk, uint16_t *v,
                                  int64_t ldv, void *stream)
{
    SDNQ_NVTX_RANGE();
    return run_kv<false>(k, ldk, v, ldv, slots, T, Hkv, D, group, const_cast<int8_t *>(codes),
                         const_cast<float *>(scales), pages, page, stream);
}

SDNQ_API int64_t sdnq_attention_paged_workspace(int64_t H, int64_t Hkv, int64_t D)
{
    if (H < 1 || Hkv < 1 || H % Hkv != 0 || (D != 64 && D != 128))
        return -1;
    return sdnq::paged_workspace(D);
}

SDNQ_API sdnq_status sdnq_attention_paged(const uint16_t *q, int64_t ldq, int64_t T, int64_t H,
                                          const int32_t *cu_q, const int32_t *lens, int64_t B,
                                          const int32_t *table, int64_t max_pages, int64_t ldt, const int8_t *codes,
                                          const float *scales, int64_t pages, int32_t page,
                                          int64_t Hkv, int64_t D, int64_t max_q, int32_t group,
                                          float scale, int64_t window, int64_t sinks, void *ws,
                                          int64_t ws_bytes, uint16_t *out, int64_t ldo,
                                          void *stream)
{
    SDNQ_NVTX_RANGE();
    return run_attention_paged(q, ldq, T, H, cu_q, lens, B, table, max_pages, ldt, codes, scales, pages, page,
                               Hkv, D, max_q, group, scale, window, sinks, ws, ws_bytes, out, ldo,
                               stream);
}
