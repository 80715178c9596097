// kv16_tc.cuh - what the tcgen05 kernels over the 16-bit cache share: scores out of tensor memory, copies by TMA and their maps.
// (Operand descriptors, MMAs and bounded waits are those of kv8_tc.cuh.)
#pragma once

#include "kv16.cuh"
#include "kv8_tc.cuh"

namespace qd {

// 128 scores of a lane's row: loads under way together, then one wait that names what it waits for.
QD_DEV void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
          "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}
template <bool WAIT>
QD_DEV void tmem_ld32_end(uint32_t (&r)[32]) {
#define QD_ALL32 \
    "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), \
        "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), \
        "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), \
        "+r"(r[31])
    if (WAIT) asm volatile("tcgen05.wait::ld.sync.aligned;" : QD_ALL32 : : "memory");
    else asm volatile("" : QD_ALL32 : : "memory");
#undef QD_ALL32
}

QD_DEV void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map),
        "r"(x), "r"(y), "r"(z), "r"(ptx::smem_u32(bar))
        : "memory");
}
QD_DEV void tma_load_rows(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x),
        "r"(y), "r"(ptx::smem_u32(bar))
        : "memory");
}
// The same where the lines are read once: they are the first to leave L2, and the kernels' own results stay.
QD_DEV void tma_load_rows_once(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(ptx::smem_u32(bar)), "l"(policy)
        : "memory");
}
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled through the runtime's driver entry point (null if unavailable)
inline EncodeFn encoder() {
    static EncodeFn enc = []() -> EncodeFn {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeFn>(p);
        return nullptr;
    }();
    return enc;
}
inline bool encode(CUtensorMap *map, int dims, const void *p, const cuuint64_t *size, const cuuint64_t *stride, const cuuint32_t *box) {
    const cuuint32_t step[3] = {1, 1, 1};
    return encoder() && encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, dims, const_cast<void *>(p), size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A pool as rows of one token and head; a copy is 64 dims of a page.
inline bool kv16_page_map(CUtensorMap *map, const void *pool, const llm_kv16_cache &c) {
    const cuuint64_t size[2] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.n_pool_pages * c.n_kv_heads * kKv8Page}, stride[1] = {(cuuint64_t)c.head_dim * 2};
    const cuuint32_t box[2] = {64, kKv8Page};
    return encode(map, 2, pool, size, stride, box);
}
// Rows of queries; a copy is 64 dims of G heads of R rows.
inline bool kv16_row_map(CUtensorMap *map, const void *q, int64_t q_stride, int n_rows, int Hq, int G, int R, int D) {
    const cuuint64_t size[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)n_rows}, stride[2] = {(cuuint64_t)D * 2, (cuuint64_t)q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)R};
    return encode(map, 3, q, size, stride, box);
}

}  // namespace qd
