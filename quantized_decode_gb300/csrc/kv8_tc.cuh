// kv8_tc.cuh - parts of the tcgen05 attention over the 8-bit cache: codes on their way by TMA, their fp16
// form in shared memory, the split of V's scales, TMEM accesses and the MN-major operand descriptor.
//
// A block is 128 tokens, 8 pages.  Its K and its V lie in shared memory as [token][dim] fp16 rows in panels
// of 64 dims (128-byte rows, 128-byte swizzle): K is the K-major B operand of the scores, V the MN-major B
// operand of the output.
#pragma once

#include "kv8.cuh"
#include "ptx.cuh"

namespace qd {

constexpr int kTile = 128;             // rows of an MMA tile, and tokens of a block
constexpr int kBlockPages = kTile / kKv8Page;
constexpr int kPanel = kTile * 128;    // bytes of 128 rows of 64 fp16
constexpr uint64_t kWaitNs = 1000000000ull;

// Wait for the phase of `parity`, kWaitNs at most or until *abort.  Both are looked at once in a while only: reading the
// timer takes longer than a hand-over between two warps.
QD_DEV bool tc_wait(uint64_t *bar, uint32_t parity, const volatile int *abort) {
    if (ptx::mbar_test(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (ptx::mbar_test(bar, parity)) return true;
        if ((i & 255u) == 0) {
            if (abort && *abort) return false;
            const uint64_t t = ptx::gtimer();
            if (t0 == 0) t0 = t;
            else if (t - t0 > kWaitNs) return false;
        }
    }
}
// 16 consecutive 32-bit TMEM columns of the warp's lanes from registers (no wait)
QD_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
QD_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations in one instruction.
QD_DEV float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
QD_DEV float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// columns taddr .. + n - 1 (n a multiple of 32) of the warp's lanes times a factor of each lane
QD_DEV void tmem_scale(uint32_t taddr, int n, float k) {
#pragma unroll 1
    for (int i = 0; i < n; i += 32) {
        float v[32];
        ptx::tmem_ld32(taddr + i, v);
#pragma unroll
        for (int e = 0; e < 32; e += 16) {
            uint32_t w[16];
#pragma unroll
            for (int z = 0; z < 16; ++z) w[z] = __float_as_uint(v[e + z] * k);
            tmem_st16(taddr + i + e, w);
        }
    }
}

// Descriptors of the operands in such rows, as two words: the high one is the same for both (8-row or 8-token groups
// 1024 bytes apart, version 1, 128-byte swizzle), the low one the address in 16-byte units and for the MN-major
// form the distance of two 64-dim panels.  A step of 16 dims of a K-major operand is 32 bytes, of 16 tokens of the
// MN-major one 2048.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
QD_DEV uint32_t desc_k(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | 1u << 16; }
QD_DEV uint32_t desc_mn(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (uint32_t)(kPanel >> 4) << 16; }
// One lane of the warp, by elect.sync: MMAs are issued in the branch of the lane that it names.  (In a branch on the lane's
// number each MMA of 128 x 128 x 16 took 151 cycles beside busy warps; in this one 65, the tensor core's own time.)
QD_DEV bool elect_lane() {
    uint32_t x;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
    return x != 0;
}
// D (+)= A B with A from shared or tensor memory; the descriptors' low words.
template <bool ADD>
QD_DEV void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "n"(ADD ? 1 : 0)
        : "memory");
}
template <bool ADD>
QD_DEV void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %4};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "n"(ADD ? 1 : 0)
        : "memory");
}
constexpr uint32_t kIdescBMn = 1u << 16;  // instruction descriptor: B is MN-major

// Sixteen codes (four words) to fp16 times 2^-k (h2 holds 2^-k twice), as two 16-byte chunks.
template <int FMT>
QD_DEV void codes_f16(const uint4 &u, __half2 h2, bool scaled, uint4 &lo, uint4 &hi) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t o[8];
    if (FMT == LLM_KV8_INT8) {
        // b ^ 0x80 = c + 128 under the exponent of 1024; (1152 + c) h - 1152 h is exact
        const __half2 off = __hmul2(h2, __floats2half2_rn(-1152.f, -1152.f));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = w[i] ^ 0x80808080u;
            o[2 * i] = h2_as_u32(__hfma2(u32_as_h2(prmt(x, 0x64646464u, 0x4140u)), h2, off));
            o[2 * i + 1] = h2_as_u32(__hfma2(u32_as_h2(prmt(x, 0x64646464u, 0x4342u)), h2, off));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
                : "=r"(o[2 * i]), "=r"(o[2 * i + 1])
                : "r"(w[i]));
        if (scaled) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = h2_as_u32(__hmul2(u32_as_h2(o[i]), h2));
        }
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// What the softmax has to know of a block's pages.  V's scale is split: vs / vref = r 2^-k; 2^-k goes into
// V's fp16 values (exact for k <= 15), log2 r into the exponent of the weights, and a page's share of their sum
// is divided by r again.
constexpr int kRecs = 4, kNanBit = 8;
struct BlockRec {
    struct __align__(16) Page {
        float ks, lr, ir, mul;  // K scale, log2 r, 1 / r, 2^-k
    } page[kBlockPages];
    float move, vref;  // factor of the output when vref changed with this block; vref
    uint32_t ok;       // pages that are there; from bit kNanBit on those whose V scale is NaN
    uint32_t scaled;   // some mul is not 1
};

// The split of a block's V scales against vref, which all lanes keep alike; lane p % 8 holds page p.
// vref is a power of two that follows the scales where they leave [2^-14, 2^4] of it, but not below 2^-60 of the largest
// one so far (vtop): outputs in its units stay finite.  Scales below 2^-100 of it count as 0.  One that is NaN counts as
// vref here, since lse has nothing to do with it: the rows that see its page become NaN at their end.
struct VSplit {
    float r, mul, move;  // mul = 2^-k, 0 for a scale of 0
};
QD_DEV VSplit split_scale(float vs, float &vref, float &vtop) {
    VSplit o;
    float top = vs > 0.f && vs < INFINITY ? vs : 0.f;
#pragma unroll
    for (int i = 1; i < kBlockPages; i <<= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, i));
    o.move = 1.f;
    if (top > 0.f && (vref == 0.f || top > vref * 16.f || top < vref * 6.1035156e-05f)) {  // 2^-14
        const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -126), 126);
        const float to = fmaxf(__uint_as_float((uint32_t)(127 + e) << 23), vtop * 8.6736174e-19f);  // 2^-60
        o.move = vref == 0.f ? 1.f : vref / to;
        vref = to;
        vtop = fmaxf(vtop, to);
    }
    if (!(vs < INFINITY)) return VSplit{1.f, 1.f, o.move};
    o.r = vs / vref;
    const bool none = vs == 0.f || o.r < 7.8886091e-31f;  // 2^-100
    if (none) o.r = 1.f;
    o.mul = none ? 0.f : 1.f;
    if (o.r < 1.f) {
        const int k = min(127 - (int)(__float_as_uint(o.r) >> 23), 15);
        o.mul = __uint_as_float((uint32_t)(127 - k) << 23);
        o.r *= __uint_as_float((uint32_t)(127 + k) << 23);
    }
    return o;
}

// ---- codes on their way: two places in shared memory, the first for the K codes of a block of one head, the second
// for its V codes ([page][16][D] bytes).  Copies are the TMA engine's, so many are in flight without registers.
struct CodeRing {
    uint64_t full[2], empty[2], rec_full[kRecs];
    BlockRec rec[kRecs];
    QD_DEV void init(int converters) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], converters);
        }
        for (int i = 0; i < kRecs; ++i) ptx::mbar_init(&rec_full[i], 1);
    }
};
QD_DEV void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(ptx::smem_u32(bar))
                 : "memory");
}

// One warp: the copies and records of the nb blocks from `table` on (the first block's entries).  `left`: tokens
// from there on that any row sees.  `wait(bar, phase)`: by the whole warp, false once something timed out.
// started: copies of K and of V that were started.
template <int D, typename Wait>
QD_DEV void feed_codes(const Kv8AttnArgs &a, const int32_t *table, int head, int nb, int left, CodeRing &ring, uint8_t *units,
                       int (&started)[2], Wait wait) {
    constexpr uint32_t kPage = kKv8Page * D, kUnit = kBlockPages * kPage;
    const int lane = threadIdx.x & 31, Hkv = a.c.n_kv_heads;
    // lane p % 8 knows page p of a block: -2 where there is none, -1 for one that is out of range
    auto entry = [&](int j) {
        const int p = j * kBlockPages + (lane & 7);
        return j < nb && kv8_page_there(p, left) ? max(-1, __ldg(table + p)) : -2;
    };
    auto checked = [&](int ph) {
        if (ph != -1 && ph < a.c.n_pool_pages) return ph;
        if (lane < kBlockPages) kv8_report(a.err);
        return -1;
    };
    auto scale_of = [&](const float *pool, int ph) { return ph >= 0 ? __ldg(pool + (int64_t)ph * Hkv + head) : 0.f; };
    int ph = checked(entry(0)), ph_next = entry(1);
    float ks = scale_of(a.c.k_scale, ph), vs = scale_of(a.c.v_scale, ph), vref = 0.f, vtop = 0.f;
    for (int j = 0; j < nb; ++j) {
        const uint32_t ok = __ballot_sync(kFullMask, ph >= 0) & 0xffu;
        auto copy = [&](int x) {  // K or V of block j
            if (j > 0 && !wait(&ring.empty[x], (uint32_t)j - 1)) return false;
            if (lane == 0) ptx::mbar_expect_tx(&ring.full[x], kPage * __popc(ok));
            __syncwarp();
            started[x] = j + 1;
            if (lane < kBlockPages && ph >= 0)
                bulk_load(ptx::smem_u32(units) + x * kUnit + lane * kPage,
                          (const uint8_t *)(x ? a.c.v_codes : a.c.k_codes) + ((int64_t)ph * Hkv + head) * kPage, kPage, &ring.full[x]);
            return true;
        };
        if (!copy(0)) return;
        const int next = checked(ph_next);
        ph_next = entry(j + 2);
        const float ks_next = scale_of(a.c.k_scale, next), vs_next = scale_of(a.c.v_scale, next);
        // The place of K waited for above held block j - 1: its converters had waited for the scores of block
        // j - 3 at the latest, those for the weights of j - 4, so nobody reads the record of j - kRecs any more
        static_assert(kRecs == 4, "the argument above");
        const VSplit v = split_scale(vs, vref, vtop);
        BlockRec &rec = ring.rec[j % kRecs];
        if (lane < kBlockPages) {
            rec.page[lane] = BlockRec::Page{ks, log2f(v.r), 1.f / v.r, v.mul};
        }
        const bool scaled = __any_sync(kFullMask, v.mul != 1.f && ph >= 0);
        const uint32_t nans = __ballot_sync(kFullMask, !(vs < INFINITY)) & 0xffu;
        if (lane == 0) {
            rec.move = v.move;
            rec.vref = vref;
            rec.ok = ok | nans << kNanBit;
            rec.scaled = scaled;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ring.rec_full[j % kRecs]);
        if (!copy(1)) return;
        ph = next;
        ks = ks_next;
        vs = vs_next;
    }
}

// NT threads turn a block's codes into fp16 rows.  Piece i of a thread is 16 dims of one token.  Eight lanes that access
// shared memory together take the first panel's dims of a token and the second's of its neighbour: 128 bytes of codes on
// all banks, and (the swizzle) eight chunks on all banks.
template <int D, int NT>
struct Pieces {
    static constexpr int kCount = kTile * D / 16 / NT;   // pieces of a thread
    static constexpr int kRun = NT / D;                  // pages that a step of the threads covers
    static_assert(kRun >= 1 && kRun * kCount == kBlockPages, "every piece of a block once");
    int tid;
    QD_DEV int page(int i) const { return kRun * i + tid / D; }
    QD_DEV int panel() const { return D == 128 ? tid >> 2 & 1 : 0; }
    QD_DEV int row() const {  // in its page
        const int x = tid % D;
        return D == 128 ? 2 * (x >> 4) + ((x >> 3 ^ x >> 2) & 1) : x >> 2;
    }
    QD_DEV int chunk() const { return 2 * (tid & 3); }   // of its row in the panel: 8 dims each

    // left: tokens of the block that are there; whatever lies in the slots behind them, and in pages that are not
    // there, becomes 0
    template <int FMT>
    QD_DEV void convert(const uint8_t *unit, uint8_t *dst, const BlockRec &rec, bool is_v, int left, uint64_t *empty) const {
        const int lane = threadIdx.x & 31;
        const bool scaled = is_v && rec.scaled != 0, whole = left >= kTile && rec.ok == 0xffu;
        const uint8_t *from = unit + (page(0) * kKv8Page + row()) * D + panel() * 64 + chunk() * 8;
        uint4 w[kCount];
#pragma unroll
        for (int i = 0; i < kCount; ++i) w[i] = *reinterpret_cast<const uint4 *>(from + i * (kRun * kKv8Page * D));
        // The next block's codes may come as soon as these have been read: the fence keeps the reads before the copies
        // that follow the arrival (without it they were overtaken).
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(empty);
        if (!whole) {
#pragma unroll
            for (int i = 0; i < kCount; ++i)
                if (!((rec.ok >> page(i)) & 1u) || page(i) * kKv8Page + row() >= left) w[i] = make_uint4(0, 0, 0, 0);
        }
        const int r = page(0) * kKv8Page + row();  // whole pages further on, the swizzle is the same
        const int x0 = (chunk() ^ (r & 7)) << 4, x1 = x0 ^ 16;
        uint8_t *to = dst + panel() * kPanel + r * 128;
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            uint4 c0, c1;
            codes_f16<FMT>(w[i], __float2half2_rn(scaled ? rec.page[page(i)].mul : 1.f), scaled, c0, c1);
            uint8_t *p = to + i * (kRun * kKv8Page * 128);
            *reinterpret_cast<uint4 *>(p + x0) = c0;
            *reinterpret_cast<uint4 *>(p + x1) = c1;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
    }
};

}  // namespace qd
