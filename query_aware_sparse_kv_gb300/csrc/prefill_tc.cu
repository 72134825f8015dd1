// Prefill on the tensor cores (qskv_prefill.cuh): bf16 queries over a bf16 or
// an 8-bit cache, tcgen05 products with accumulators and softmax weights in
// tensor memory.
//
// A CTA works on a tile of 256 rows (queries x the heads that share a KV
// head), as two halves of 128, against blocks of 128 keys:
//   S = Q K^T (128 x 128 a half), P = softmax weights, O += P V (128 x d).
// The halves take turns on the tensor cores: while one half's logits are being
// turned into weights, the other's products run.  In tensor memory a half has
// 128 columns of S, over whose first 64 its P is written as bf16 pairs, and d
// columns of O.  Roles:
//   8 softmax warps  one thread a row: reads its 128 logits, keeps the running
//                    maximum and sum (fp32), writes P.  The maximum a row's
//                    weights refer to moves only when one would pass 2^8; O
//                    is then scaled in tensor memory, which its P V before
//                    that has left by then (the products run in order and S of
//                    this block was issued after it).  At the end the row's O
//                    is divided by its sum and stored.
//   1 MMA thread     issues all products; O += P V of block j, then S of block j + 1.
//   2 load warps     gather the pages' keys and values by TMA (boxes of 16
//                    tokens x 64 dims) into one ring, K and V in turn; for an
//                    8-bit cache
//   1 fetch warp     copies the codes into a ring of 16-token parts, from which
//   4 convert warps  fill the other one: a code times its power of two is a bf16
//                    number, so the products see the cached values as they are.
//   1 list warp      takes items from the list, one ahead, and loads Q.
// Places without a token (past the row's end, a page that is not there) weigh
// nothing: their logits are replaced, and the rows of V, which may hold
// anything, are zeroed in shared memory before the product by the softmax
// warps of the first half.
//
// Bound: a block of 128 keys is 2048 clocks of products for both halves.  A
// half's turn is its softmax (128 exponentials a thread at 8 a clock and
// scheduler, as many maxima, conversions and sums on the other pipes), then its
// products, 1024 clocks; overlapped, the tensor cores are busy 67 % of the time
// over a prompt of 8192 tokens.  One GB300: a prompt of 16384 tokens, 32 heads of 128 dims
// over 8 KV heads, in 1.39 ms (1578 TFLOP/s of 1888 that a plain product
// reaches); 16 prompts of 1..4096 tokens in 0.52 ms; 4 chunks of 1024..2048
// tokens behind up to 30000 in an 8-bit cache in 1.59 ms (1106 TFLOP/s), bound
// by the conversion of the codes.
//
// Every wait is bounded; a wait that gives up flags a timeout and stops the
// CTA's other roles; copies and products under way complete before the CTA
// leaves.
#include <cuda_fp16.h>

#include "qskv_kvf.cuh"
#include "qskv_prefill.cuh"

namespace qskv {
namespace {

constexpr int kSoftmaxWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kListWarp = 11, kConvertWarp = 12;
template <bool KVF>
constexpr int kThreads = KVF ? 512 : 384;
constexpr int kGoodRing = 16;      // blocks whose page masks are kept (more than the ring's stages)
template <bool KVF>
constexpr int kItemReaders = kSoftmaxWarps + 1 + (KVF ? 1 + 4 : 2);
constexpr float kLazy = 8.f;       // weights up to 2^8 before a row's reference moves

template <int D, bool KVF>
struct Cfg {
    static constexpr int NB = D / 64;            // 64-dim (128-byte) column groups
    static constexpr int ATOM = 128 * 128;       // 128 rows x 128 bytes
    static constexpr int TILE = NB * ATOM;       // 128 rows of Q, K or V
    static constexpr int STAGES = D == 128 ? (KVF ? 4 : 5) : 8;
    // a block's codes: of each of 8 parts the keys and their powers, the values and all powers
    static constexpr int KEYS = 16 * D + 16, VALUES = 16 * D + 32;
    static constexpr int PARTS = KVF ? 8 * (KEYS + VALUES) : 0;
    static constexpr int SMEM = 2 * TILE + STAGES * TILE + PARTS + 1024;
    static constexpr uint32_t S_COL = 0, O_COL = 256;  // half h: S (and P) at 128 h, O at 256 + 128 h
};

// (max_slots Hkv is below 2^18, tickets without a list are fewer than SMs)
constexpr int kPlaceBits = 20, kPlaceMask = (1 << kPlaceBits) - 1;

struct Slot {
    PrefillItem item;
    int head;   // KV head; -1: no more items
    int place;  // of a tile in parts: where their results lie; direct: its ticket above that
};

// A row's tile, where there is no list: its queries and key blocks, and the units of work that they count as (of one KV
// head, after `before` of the rows ahead).
struct RowWork {
    int first, n, pos, blocks;
    uint32_t units, before;
};

// Items without a list.  The tiles' key blocks, row by row and head by head, are units on a line that is cut into ranges:
// one a CTA, all as long (within one), where that gives a CTA kPrefillMinBlocks or more; else as many as tiles have parts of
// kPrefillMinBlocks blocks, the last part's rest counted in.
struct Line {
    uint32_t units, ranges, least, more;  // the first `more` ranges have least + 1 units, the others least
    uint32_t range, at, end;              // this CTA's range, and what of it is still to do

    __device__ __forceinline__ uint32_t begin(uint32_t r) const { return r * least + min(r, more); }
    __device__ __forceinline__ uint32_t range_of(uint32_t x) const {
        const uint32_t first = more * (least + 1);
        return x < first ? x / (least + 1) : more + (x - first) / least;
    }
    // (the whole list warp, a lane a row; what follows is its first lane's)
    __device__ void make(const PrefillArgs &a, RowWork *rows) {
        const int lane = threadIdx.x & 31;
        RowWork w = {};
        if (lane < a.batch) {
            int len;
            prefill_row(a, lane, w.first, w.n, len);
            w.pos = len - w.n;
            w.blocks = w.n > 0 ? (len + a.block_keys - 1) / a.block_keys : 0;
            w.units = w.n > 0 ? max(w.blocks, 1) : 0;
        }
        const uint32_t heads = a.num_kv_heads;
        const uint64_t all = uint64_t(__reduce_add_sync(0xffffffffu, w.units)) * heads;
        const bool even = all >= uint64_t(kPrefillMinBlocks) * gridDim.x;
        if (!even) w.units = (w.units + kPrefillMinBlocks - 1) / kPrefillMinBlocks * kPrefillMinBlocks;
        w.before = w.units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, w.before, o);
            if (lane >= o) w.before += up;
        }
        const uint32_t tiles = __shfl_sync(0xffffffffu, w.before, 31);
        w.before -= w.units;
        rows[lane] = w;
        if (lane == 0) {
            units = tiles * heads;
            ranges = even ? gridDim.x : units / kPrefillMinBlocks;
            least = ranges ? units / ranges : 0, more = ranges ? units % ranges : 0;
            range = blockIdx.x, at = end = 0;
            if (range < ranges) at = begin(range), end = begin(range + 1);
        }
        __syncwarp();
    }
    // The next item; leaves x as it is where there is none.
    __device__ void next(const PrefillArgs &a, const RowWork *rows, Slot &x) {
        if (at == end) {
            range += gridDim.x;
            if (range >= ranges) return;
            at = begin(range), end = begin(range + 1);
        }
        const uint32_t heads = a.num_kv_heads;
        int r = 0;  // the row that the unit is in
#pragma unroll
        for (int step = kPrefillDirectRows / 2; step; step >>= 1) {
            const RowWork &w = rows[r + step - 1];
            if ((w.before + w.units) * heads <= at) r += step;
        }
        const RowWork w = rows[r];
        const uint32_t off = at - w.before * heads, head = off / w.units, block = off - head * w.units;
        const uint32_t take = min(w.units - block, end - at), tile = at - block;
        const uint32_t first = range_of(tile), last = range_of(tile + w.units - 1);
        at += take;
        x.item = {};
        x.item.row = r, x.item.token = w.first, x.item.tokens = w.n, x.item.pos = w.pos;
        x.item.block0 = min(int(block), w.blocks), x.item.block1 = min(int(block + take), w.blocks);
        x.item.part = range - first, x.item.parts = last - first + 1;
        // parts are numbered by range and tile: the next tile's first is in this one's last range or behind it
        const uint32_t ticket = r * heads + head;
        x.head = head, x.place = int(ticket << kPlaceBits | (ticket + first));
    }
};

struct Shared {
    uint64_t item_full[2], item_empty[2], q_full, q_empty, kv_full[8], kv_empty[8], s_full[2], p_full[2], o_full[2];
    uint64_t parts_done, last_known, drain;
    uint64_t part_full[2], part_empty[2];  // of a block's 8-bit codes (keys, values): there, and no longer needed
    Slot slot[4];
    RowWork rows[kPrefillDirectRows];
    Line line;
    uint32_t good[kGoodRing];  // pages of a block that are there
    uint32_t tmem;
    uint32_t last;
    volatile uint32_t abort;
};

// Bounded wait that also gives up when another role of the CTA has.
__device__ __forceinline__ bool wait_phase(Shared &s, uint64_t *bar, uint32_t parity, uint32_t *flags) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (s.abort) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            s.abort = 1u;
            raise_error(flags, kErrTimeout);
            return false;
        }
    }
    return true;
}
// The same for a whole warp.
__device__ __forceinline__ bool warp_wait(Shared &s, uint64_t *bar, uint32_t parity, uint32_t *flags) {
    return __all_sync(0xffffffffu, wait_phase(s, bar, parity, flags));
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// 64 columns of a thread's TMEM lane, not waited for.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
        "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, "
        "%42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
        "%62, %63"
        "}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}
// Waits for the loads before it; nothing reads r earlier.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[64], bool wait) {
    if (wait) asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    asm volatile(""
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
          "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
          "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]),
          "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]), "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]),
          "+r"(r[40]), "+r"(r[41]), "+r"(r[42]), "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]),
          "+r"(r[48]), "+r"(r[49]), "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]),
          "+r"(r[56]), "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63]));
}

// 16 columns of a thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
        "}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// Stores 16 columns; tmem_st_wait before anybody is told.
__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
        "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16"
        "};" ::"r"(taddr),
          "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two floats in one 64-bit register, an instruction for both.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

template <int REGS>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// The next item, copied out of its slot.  A role is at most two items behind the list warp, so of four slots the one that it
// works on is still as it was.
struct ItemReader {
    uint32_t n = 0;  // items so far
    __device__ __forceinline__ bool next(Shared &s, Slot &x, uint32_t *flags) {
        if (!warp_wait(s, &s.item_full[n & 1], n >> 1 & 1, flags)) return false;
        x = s.slot[n & 3];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&s.item_empty[n & 1]);
        n++;
        return x.head >= 0;
    }
    __device__ __forceinline__ const Slot &current(const Shared &s) const { return s.slot[(n - 1) & 3]; }
};

// ------------------------------------------------------------- softmax --
template <int D, bool KVF>
__device__ void softmax_role(const PrefillArgs &a, Shared &s, uint8_t *ring, uint32_t tmem) {
    using C = Cfg<D, KVF>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane, tile_row = half * 128 + r;
    const int G = a.group, shift = 31 - __clz(G), page_shift = a.page_size == 16 ? 4 : 5;
    const uint32_t whole = a.page_size == 16 ? 0xff : 0xf;  // all pages of a block
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t s_at = lanes + C::S_COL + 128 * half, o_at = lanes + C::O_COL + 128 * half;
    const float sc = a.scale_log2;
    const uint64_t sc2 = pair(sc, sc);
    ItemReader items;
    Slot x;
    uint32_t s_phase = 0, o_phase = 0, parts_phase = 0;
    uint32_t stage0 = 0;   // ring stages of the items before this one
    uint32_t blocks0 = 0;  // and their blocks
    while (items.next(s, x, a.flags)) {
        const PrefillItem &it = x.item;
        const int n = it.block1 - it.block0, end = it.pos + it.tokens;  // keys the tile sees
        const int token = tile_row >> shift;
        const bool mine = token < it.tokens;
        const int limit = mine ? it.pos + token + 1 : end;  // keys the row sees
        const bool active = half == 0 || it.tokens * G > 128;
        float m = -INFINITY, l = 0.f;
        const int least = __reduce_min_sync(0xffffffffu, limit);  // of the warp's rows
        bool ok = true;
        for (int j = 0; j < n && ok && active; j++) {
            ok = warp_wait(s, &s.s_full[half], s_phase, a.flags);
            if (!ok) break;
            s_phase ^= 1;
            tc_fence_after();
            uint32_t rr[2][64];
            tmem_ld64(s_at, rr[0]);
            tmem_ld64(s_at + 64, rr[1]);
            tmem_ld_wait(rr[0], true);
            tmem_ld_wait(rr[1], false);
            const int key0 = (it.block0 + j) * 128;
            const uint32_t good = s.good[(blocks0 + j) % kGoodRing];
            const bool cut = good != whole;  // a page is not there, or behind the end
            if (least < key0 + 128 || cut) {
                const int lim = limit - key0;
#pragma unroll
                for (int k = 0; k < 128; k++)
                    if (k >= lim || !(good >> (k >> page_shift) & 1)) rr[k / 64][k % 64] = 0xff800000u;
            }
            float most[4];
#pragma unroll
            for (int k = 0; k < 4; k++) most[k] = -INFINITY;
#pragma unroll
            for (int k = 0; k < 128; k += 2)
                most[k / 2 & 3] = max3(most[k / 2 & 3], __uint_as_float(rr[k / 64][k % 64]),
                                       __uint_as_float(rr[k / 64][k % 64 + 1]));
            const float top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])) * sc;
            if (__any_sync(0xffffffffu, top > m + kLazy)) {
                const float mn = top > m + kLazy ? top : m;
                const float down = mn == m ? 1.f : ex2(m - mn);
                m = mn, l *= down;
#pragma unroll 1
                for (int c = 0; c < D && j > 0; c += 16) {  // 16 columns: the logits take up most registers
                    uint32_t o[16];
                    tmem_ld16(o_at + c, o);
#pragma unroll
                    for (int k = 0; k < 16; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * down);
                    tmem_st16_async(o_at + c, o);
                }
                tmem_st_wait();
            }
            if (!KVF && half == 0 && (cut || key0 + 128 > end)) {  // rows of V without a token: zeros
                const uint32_t at = stage0 + 2 * j + 1, stage = at % C::STAGES;
                ok = warp_wait(s, &s.kv_full[stage], at / C::STAGES & 1, a.flags);
                if (key0 + r >= end || !(good >> (r >> page_shift) & 1)) {
                    uint4 *row = reinterpret_cast<uint4 *>(ring + stage * C::TILE + r * 128);
#pragma unroll
                    for (int b = 0; b < C::NB; b++)
#pragma unroll
                        for (int k = 0; k < 8; k++) row[b * (C::ATOM / 16) + k] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            const float base = m == -INFINITY ? 0.f : m;
            const uint64_t minus = pair(-base, -base);
            uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < 4; c++) {
                uint32_t pk[16];
#pragma unroll
                for (int k = 0; k < 16; k++) {
                    const int i = 32 * c + 2 * k;
                    float u, v;
                    unpair(fma2(pair(__uint_as_float(rr[i / 64][i % 64]), __uint_as_float(rr[i / 64][i % 64 + 1])), sc2, minus), u, v);
                    u = ex2(u), v = ex2(v);
                    sum[k & 3] = add2(sum[k & 3], pair(u, v));
                    pk[k] = pack_bf16x2(u, v);
                }
                tmem_st16_async(s_at + 16 * c, pk);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.p_full[half]);
            float u, v;
            unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), u, v);
            l += u + v;
        }
        stage0 += 2 * n, blocks0 += n;
        if (!ok) return;
        if (active && n > 0) {
            if (!warp_wait(s, &s.o_full[half], o_phase, a.flags)) return;
            o_phase ^= 1;
            tc_fence_after();
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const float lse2 = l > 0.f ? m + log2f(l) : -INFINITY;
        const Slot &now = items.current(s);  // (read here: the softmax has no registers to keep it in)
        const int64_t head = int64_t(now.item.token + token) * a.num_q_heads + now.head * G + (tile_row & (G - 1));
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + head * D);
        const int parts = now.item.parts, part = now.item.part;
        const int64_t place = now.place & kPlaceMask;  // part p's results: p behind it
        // of a part: its row's outputs, 4 dims at [dim / 4][row]
        float4 *part_o = reinterpret_cast<float4 *>(a.part_o) + tile_row;
        constexpr int64_t kPart = int64_t(D / 4) * kPrefillTcRows;
        if (active) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(o_at + c, o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; k++) o[k] = 0;
                }
                if (mine) {
                    float f[32];
#pragma unroll
                    for (int k = 0; k < 32; k++) f[k] = l > 0.f ? __uint_as_float(o[k]) * inv : 0.f;
                    if (parts == 1) {
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            out[c / 8 + k] =
                                make_uint4(pack_bf16x2(f[8 * k], f[8 * k + 1]), pack_bf16x2(f[8 * k + 2], f[8 * k + 3]),
                                           pack_bf16x2(f[8 * k + 4], f[8 * k + 5]), pack_bf16x2(f[8 * k + 6], f[8 * k + 7]));
                    } else {
                        float4 *to = part_o + (place + part) * kPart + c / 4 * kPrefillTcRows;
#pragma unroll
                        for (int k = 0; k < 8; k++)
                            to[k * kPrefillTcRows] = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
                    }
                }
                __syncwarp();
            }
        }
        tc_fence_before();
        if (parts == 1) {
            if (mine && a.lse) a.lse[head] = lse2 * 0.6931471805599453f;
            continue;
        }
        // ---- a part: the last one that is done joins them, in their order
        if (mine) a.part_lse[(place + part) * kPrefillTcRows + tile_row] = lse2;
        __threadfence();
        mbar_arrive(&s.parts_done);
        if (threadIdx.x == 0) {
            if (wait_phase(s, &s.parts_done, parts_phase, a.flags)) {
                uint32_t *ticket = a.tickets + (a.direct ? now.place >> kPlaceBits : int(place));
                const uint32_t done = atomicAdd(ticket, 1u);
                s.last = done == uint32_t(parts) - 1;
                if (s.last && a.direct) *ticket = 0;
                __threadfence();
                mbar_arrive(&s.last_known);
            }
        }
        __syncwarp();
        if (!warp_wait(s, &s.last_known, parts_phase, a.flags)) return;
        parts_phase ^= 1;
        if (!s.last) continue;
        __threadfence();
        if (!mine) continue;
        auto lse_of = [&](int p) { return __ldcg(a.part_lse + (place + p) * kPrefillTcRows + tile_row); };
        float most = -INFINITY, total = 0.f;
        for (int p = 0; p < parts; p++) most = fmaxf(most, lse_of(p));
        if (most > -INFINITY)
            for (int p = 0; p < parts; p++) total += ex2(lse_of(p) - most);
        const float share = total > 0.f ? 1.f / total : 0.f;
        if (a.lse) a.lse[head] = total > 0.f ? (most + log2f(total)) * 0.6931471805599453f : -INFINITY;
#pragma unroll 1
        for (int c = 0; c < D / 8; c += 4) {
            float4 f[8];
#pragma unroll
            for (int k = 0; k < 8; k++) f[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int p = 0; p < parts; p++) {
                const float w = most > -INFINITY ? ex2(lse_of(p) - most) * share : 0.f;
                const float4 *from = part_o + (place + p) * kPart + c * 2 * kPrefillTcRows;
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const float4 o = __ldcg(from + k * kPrefillTcRows);
                    f[k].x = fmaf(w, o.x, f[k].x), f[k].y = fmaf(w, o.y, f[k].y);
                    f[k].z = fmaf(w, o.z, f[k].z), f[k].w = fmaf(w, o.w, f[k].w);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; k++)
                out[c + k] = make_uint4(pack_bf16x2(f[2 * k].x, f[2 * k].y), pack_bf16x2(f[2 * k].z, f[2 * k].w),
                                        pack_bf16x2(f[2 * k + 1].x, f[2 * k + 1].y), pack_bf16x2(f[2 * k + 1].z, f[2 * k + 1].w));
        }
    }
}

// ------------------------------------------------------------ products --
// Products and commits for the lane that `lead` is 1 in; a warp issues them together, with operands that are the same in
// all lanes.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate)), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate)), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t lead, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}

// The whole warp follows the pipeline, so that what a product is issued with is the same in all lanes (with one lane in
// this code, 16384 tokens took 1.83 ms, and 1.62 with all of them).
template <int D, bool KVF>
__device__ __forceinline__ void mma_role(const PrefillArgs &a, Shared &s, uint32_t q_at, uint32_t ring_at) {
    using C = Cfg<D, KVF>;
    constexpr uint32_t id_s = tc_idesc_bf16(128, 128, false, false), id_o = tc_idesc_bf16(128, D, false, true);
    const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem, 0);
    const uint64_t q_desc = tc_sdesc_sw128(q_at, 16, 1024), k_desc = tc_sdesc_sw128(ring_at, 16, 1024);
    const uint64_t v_desc = tc_sdesc_sw128(ring_at, C::ATOM, 1024);  // dims contiguous
    ItemReader items;
    Slot x;
    uint32_t q_phase = 0, p_phase = 0;  // p_phase: bit h of half h
    uint32_t stage = 0, phase = 0;      // of the ring
    bool issued = false;
    auto advance = [&] {
        if (++stage == C::STAGES) stage = 0, phase ^= 1;
    };
    const uint32_t lead = elect_one();
    auto logits = [&](int half, uint32_t k) {
        const uint64_t qd = q_desc + half * (C::TILE >> 4), kd = k_desc + k * (C::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; kk++) {
            const uint32_t off = ((kk >> 2) * C::ATOM + (kk & 3) * 32) >> 4;
            mma_ss(lead, tmem + C::S_COL + 128 * half, qd + off, kd + off, id_s, kk > 0);
        }
        mma_commit(lead, &s.s_full[half]);
    };
    auto outputs = [&](int half, uint32_t v, bool more) {
        const uint64_t vd = v_desc + v * (C::TILE >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ks++)  // P from tensor memory, 8 columns: 16 keys
            mma_ts(lead, tmem + C::O_COL + 128 * half, tmem + C::S_COL + 128 * half + ks * 8, vd + ks * (16 * 128 >> 4), id_o,
                   more || ks > 0);
    };
    auto commit = [&](uint64_t *bar) { mma_commit(lead, bar); };
    while (items.next(s, x, a.flags)) {
        const int n = __shfl_sync(0xffffffffu, x.item.block1 - x.item.block0, 0);
        const int halves = __shfl_sync(0xffffffffu, x.item.tokens * a.group > 128 ? 2 : 1, 0);
        if (n == 0) continue;
        bool ok = warp_wait(s, &s.q_full, q_phase, a.flags) && warp_wait(s, &s.kv_full[stage], phase, a.flags);
        if (!ok) break;
        tc_fence_after();
        for (int h = 0; h < halves; h++) logits(h, stage);
        issued = true;
        commit(&s.kv_empty[stage]);
        if (n == 1) commit(&s.q_empty);
        advance();
        for (int j = 0; j < n; j++) {
            const uint32_t v = stage;
            ok = warp_wait(s, &s.kv_full[v], phase, a.flags);
            if (!ok) break;
            advance();
            for (int h = 0; h < halves; h++) {
                ok = warp_wait(s, &s.p_full[h], p_phase >> h & 1, a.flags);
                if (!ok) break;
                tc_fence_after();
                outputs(h, v, j > 0);
                if (j + 1 == n) {
                    commit(&s.o_full[h]);
                    continue;
                }
                if (h == 0) {
                    ok = warp_wait(s, &s.kv_full[stage], phase, a.flags);
                    if (!ok) break;
                }
                logits(h, stage);
            }
            if (!ok) break;
            p_phase ^= (1u << halves) - 1;
            commit(&s.kv_empty[v]);
            if (j + 1 < n) {
                commit(&s.kv_empty[stage]);
                advance();
            }
            if (j + 2 == n) commit(&s.q_empty);
        }
        if (!ok) break;
        q_phase ^= 1;
    }
    if (issued) {  // every product has completed before the tensor memory is freed
        commit(&s.drain);
        mbar_wait_bounded(&s.drain, 0, kWaitLimitNs);
    }
    __syncwarp();
}

// --------------------------------------------------------------- loads --
// Keys (which 0, the even stages of the ring) or values (1, the odd ones).
template <int D>
__device__ __forceinline__ void load_role(const PrefillArgs &a, Shared &s, uint8_t *ring, const CUtensorMap *map, int which) {
    using C = Cfg<D, false>;
    const int lane = threadIdx.x & 31, P = a.page_size, page_shift = P == 16 ? 4 : 5, ppb = P == 16 ? 8 : 4, per = P >> 4;
    const uint32_t lead = elect_one();
    ItemReader items;
    Slot x;
    uint32_t at = which, blocks0 = 0;
    bool ok = true;
    while (ok && items.next(s, x, a.flags)) {
        const PrefillItem &it = x.item;
        const int n = it.block1 - it.block0, end = it.pos + it.tokens;
        // lane p < 8 holds the page of the 16 tokens of box p of a block, -1 where there is none; read a block ahead
        auto page_of = [&](int j) {
            const int t = (it.block0 + j) * 128 + lane * 16, page = t >> page_shift;
            if (lane >= 8 || j >= n || page << page_shift >= end) return -1;
            const int id = __ldg(a.page_table + int64_t(it.row) * a.max_pages + page);
            if (id < 0 || id >= a.num_pool_pages) {
                raise_error(a.flags, kErrPageId);
                return -1;
            }
            return id;
        };
        int next = page_of(0);
        for (int j = 0; j < n; j++, at += 2) {
            const int id = next;
            next = page_of(j + 1);
            const uint32_t stage = at % C::STAGES, boxes = __ballot_sync(0xffffffffu, id >= 0);
            if (at >= C::STAGES) ok = warp_wait(s, &s.kv_empty[stage], (at / C::STAGES - 1) & 1, a.flags);
            if (!ok) break;
            const int first = __shfl_sync(0xffffffffu, id, lane * per & 7);
            const uint32_t good = __ballot_sync(0xffffffffu, lane < ppb && first >= 0);
            if (lead) {
                if (which == 0) s.good[(blocks0 + j) % kGoodRing] = good;
                mbar_arrive_expect_tx(&s.kv_full[stage], __popc(boxes) * 16 * D * 2);
            }
            __syncwarp();
            uint8_t *to = ring + stage * C::TILE;
#pragma unroll
            for (int p = 0; p < 8; p++) {
                const int y = (__shfl_sync(0xffffffffu, id, p) * a.num_kv_heads + x.head) * P + (p & (per - 1)) * 16;
                if ((boxes >> p & 1) && lead) {
#pragma unroll
                    for (int c = 0; c < C::NB; c++)
                        tma_load_2d(to + p * 16 * 128 + c * C::ATOM, map, c * 64, y, &s.kv_full[stage]);
                }
            }
            __syncwarp();
        }
        blocks0 += n;
    }
    // copies under way land before the CTA's memory is released: this warp's among the last that fit the ring (the stages
    // of those before were filled again, so their barriers have moved on)
    const uint32_t all = at - which, low = all > C::STAGES ? all - C::STAGES : 0;
    for (uint32_t i = low + ((low ^ which) & 1); i < at; i += 2)
        mbar_wait_bounded(&s.kv_full[i % C::STAGES], i / C::STAGES & 1, kWaitLimitNs);
}

// The codes of an 8-bit cache: the next block's keys while values are converted, its values while keys are.
template <int D>
__device__ __forceinline__ void fetch_role(const PrefillArgs &a, Shared &s, uint8_t *codes) {
    using C = Cfg<D, true>;
    const int lane = threadIdx.x & 31, page_shift = a.page_size == 16 ? 4 : 5, ppb = a.page_size == 16 ? 8 : 4;
    const int per = a.page_size >> 4;
    ItemReader items;
    Slot x;
    uint32_t block = 0, issued = 0;
    bool ok = true;
    while (ok && items.next(s, x, a.flags)) {
        const PrefillItem &it = x.item;
        const int n = it.block1 - it.block0, end = it.pos + it.tokens;
        auto page_of = [&](int j) {  // lane p < 8: the page of part p of a block, -1 where there is none
            const int t = (it.block0 + j) * 128 + lane * 16, page = t >> page_shift;
            if (lane >= 8 || j >= n || page << page_shift >= end) return -1;
            const int id = __ldg(a.page_table + int64_t(it.row) * a.max_pages + page);
            if (id < 0 || id >= a.num_pool_pages) {
                raise_error(a.flags, kErrPageId);
                return -1;
            }
            return id;
        };
        int next = page_of(0);
        for (int j = 0; j < n; j++, block++) {
            const int id = next;
            next = page_of(j + 1);
            const int first = __shfl_sync(0xffffffffu, id, lane * per & 7);
            const uint32_t good = __ballot_sync(0xffffffffu, lane < ppb && first >= 0);
            if (lane == 0) s.good[block % kGoodRing] = good;
            __syncwarp();
            const uint8_t *from =
                a.pool + ((int64_t(max(id, 0)) * a.num_kv_heads + x.head) * per + (lane & (per - 1))) * kvf_part_bytes(D);
            for (int which = 0; which < 2; which++) {
                if (block >= 1) ok = warp_wait(s, &s.part_empty[which], (block - 1) & 1, a.flags);
                if (!ok) break;
                uint64_t *full = &s.part_full[which];
                if (lane < 8 && id >= 0) {  // a lane a part
                    mbar_arrive_expect_tx(full, which ? C::VALUES : C::KEYS);
                    if (which) {
                        bulk_load(codes + 8 * C::KEYS + lane * C::VALUES, from + 16 * D, C::VALUES, full);
                    } else {
                        bulk_load(codes + lane * C::KEYS, from, 16 * D, full);
                        bulk_load(codes + lane * C::KEYS + 16 * D, from + 32 * D, 16, full);
                    }
                } else if (lane < 8) {
                    mbar_arrive(full);
                }
                __syncwarp();
                issued++;
            }
            if (!ok) break;
        }
    }
    // copies under way land before the CTA's memory is released
    for (uint32_t i = issued > 2 ? issued - 2 : 0; i < issued; i++)
        mbar_wait_bounded(&s.part_full[i & 1], i / 2 & 1, kWaitLimitNs);
    __syncwarp();
}

// The values of two codes (the low half of w), which bf16 holds exactly.
__device__ __forceinline__ uint32_t bf16_values(uint32_t w, float power) {
    const uint32_t f = kvf_half2(w);
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&f));
    return pack_bf16x2(v.x * power, v.y * power);
}

// Codes to bf16 numbers, K and V in turn.  A part has D chunks of 16 bytes of keys and as many of values, a thread each;
// of a K or V its chunks are STEPS parts at the same places.
template <int D>
__device__ __forceinline__ void convert_role(const PrefillArgs &a, Shared &s, uint8_t *ring, const uint8_t *parts) {
    using C = Cfg<D, true>;
    constexpr int TOGETHER = 128 / D, STEPS = 8 / TOGETHER;  // parts the threads cover at once, and how often they do
    constexpr int K_FROM = TOGETHER * C::KEYS, V_FROM = TOGETHER * C::VALUES, TO = TOGETHER * 16 * 128;  // from one to the next
    const int tid = threadIdx.x - 32 * kConvertWarp, c = tid % D, part0 = tid / D;
    const int page_shift = a.page_size == 16 ? 4 : 5;
    const uint32_t whole = a.page_size == 16 ? 0xff : 0xf;
    // keys: a token's 16-byte chunk (16 dims); eight lanes have four chunks of two tokens, which meet all banks at their
    // places here and, as two chunks of bf16 numbers each, in the ring
    const int kt = D == 128 ? (c >> 2 & 1) + (c >> 4 << 1) : c >> 2, kc = D == 128 ? (c & 3) + (c >> 3 & 1) * 4 : c & 3;
    // values: pair of tokens and chunk (8 dims)
    const int vp = c / (D / 8), vc = kvf_value_chunk<D>(c % (D / 8), vp);
    const uint8_t *k_from = parts + part0 * C::KEYS, *v_from = parts + 8 * C::KEYS + part0 * C::VALUES;
    const uint8_t *k_codes = k_from + kt * D + kvf_key_chunk<D>(kc, kt) * 16, *v_codes = v_from + c * 16;
    const int k_to = kc / 4 * C::ATOM + (part0 * 16 + kt) * 128;
    const int k_first = k_to + (((kc & 3) * 2 ^ (kt & 7)) << 4), k_second = k_to + ((((kc & 3) * 2 + 1) ^ (kt & 7)) << 4);
    const int v_to = vc / 8 * C::ATOM + (part0 * 16 + 2 * vp) * 128;
    const int v_first = v_to + (((vc & 7) ^ (2 * vp & 7)) << 4), v_second = v_to + 128 + (((vc & 7) ^ ((2 * vp + 1) & 7)) << 4);
    ItemReader items;
    Slot x;
    uint32_t stage = 0, phase = 0, block = 0;  // of the ring; blocks of all items
    bool ok = true, filled = false;            // filled: the ring has been, once
    auto advance = [&] {
        fence_proxy_async_smem();
        mbar_arrive(&s.kv_full[stage]);
        if (++stage == C::STAGES) stage = 0, phase ^= 1, filled = true;
    };
    while (ok && items.next(s, x, a.flags)) {
        const PrefillItem &it = x.item;
        const int n = it.block1 - it.block0, end = it.pos + it.tokens;
        for (int j = 0; j < n; j++, block++) {
            const int left = end - (it.block0 + j) * 128;  // tokens of the row from the block on
            ok = warp_wait(s, &s.part_full[0], block & 1, a.flags) && (!filled || warp_wait(s, &s.kv_empty[stage], phase ^ 1, a.flags));
            if (!ok) break;
            uint8_t *to = ring + stage * C::TILE;
#pragma unroll 2
            for (int i = 0; i < STEPS; i++) {
                const uint4 w = *reinterpret_cast<const uint4 *>(k_codes + i * K_FROM);
                const float power = kvf_power(k_from[i * K_FROM + 16 * D + kt]);
                *reinterpret_cast<uint4 *>(to + k_first + i * TO) =
                    make_uint4(bf16_values(w.x, power), bf16_values(w.x >> 16, power), bf16_values(w.y, power), bf16_values(w.y >> 16, power));
                *reinterpret_cast<uint4 *>(to + k_second + i * TO) =
                    make_uint4(bf16_values(w.z, power), bf16_values(w.z >> 16, power), bf16_values(w.w, power), bf16_values(w.w >> 16, power));
            }
            advance();
            mbar_arrive(&s.part_empty[0]);
            ok = warp_wait(s, &s.part_full[1], block & 1, a.flags) && (!filled || warp_wait(s, &s.kv_empty[stage], phase ^ 1, a.flags));
            if (!ok) break;
            to = ring + stage * C::TILE;
            const uint32_t good = s.good[block % kGoodRing];
            auto values = [&](int i, bool all) {
                uint4 w = *reinterpret_cast<const uint4 *>(v_codes + i * V_FROM);
                uint32_t e = *reinterpret_cast<const uint16_t *>(v_from + i * V_FROM + 16 * D + 16 + 2 * vp);
                if (!all) {  // what lies past the end may be no number
                    const int part = i * TOGETHER + part0, row = part * 16 + 2 * vp;
                    const bool there = good >> (part * 16 >> page_shift) & 1;
                    const uint32_t keep = (there && row < left ? 0x00ff00ffu : 0u) | (there && row + 1 < left ? 0xff00ff00u : 0u);
                    w.x &= keep, w.y &= keep, w.z &= keep, w.w &= keep, e &= keep;
                }
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                const float p0 = kvf_power(e & 255), p1 = kvf_power(e >> 8);
                uint32_t y0[4], y1[4];
#pragma unroll
                for (int k = 0; k < 4; k++) {  // bytes in turn of both tokens
                    y0[k] = bf16_values(__byte_perm(u[k], 0, 0x0020), p0);
                    y1[k] = bf16_values(__byte_perm(u[k], 0, 0x0031), p1);
                }
                *reinterpret_cast<uint4 *>(to + v_first + i * TO) = make_uint4(y0[0], y0[1], y0[2], y0[3]);
                *reinterpret_cast<uint4 *>(to + v_second + i * TO) = make_uint4(y1[0], y1[1], y1[2], y1[3]);
            };
            if (good == whole && left >= 128) {
#pragma unroll 2
                for (int i = 0; i < STEPS; i++) values(i, true);
            } else {
#pragma unroll 1
                for (int i = 0; i < STEPS; i++) values(i, false);
            }
            advance();
            mbar_arrive(&s.part_empty[1]);
        }
    }
}

// Takes items from the list, or its share of the line, one ahead of the CTA's other roles, and loads their queries.
template <int D>
__device__ void list_role(const PrefillArgs &a, Shared &s, uint8_t *q, const CUtensorMap *map_q) {
    using C = Cfg<D, false>;  // its tiles are as large for both caches
    if (a.direct) s.line.make(a, s.rows);
    if ((threadIdx.x & 31) != 0) return;
    const int total = a.direct ? 0 : int(__ldcg(&a.plan->items)) * a.num_kv_heads, per = 128 / a.group;
    uint32_t loads = 0;  // of queries
    for (int i = 0;; i++) {
        const int next = a.direct ? 0 : int(atomicAdd(&a.plan->next, 1u));
        if (i >= 2 && !wait_phase(s, &s.item_empty[i & 1], (i >> 1 & 1) ^ 1, a.flags)) break;
        Slot &x = s.slot[i & 3];
        x.head = -1;
        if (a.direct) {
            s.line.next(a, s.rows, x);
        } else if (next < total) {
            const int4 *from = reinterpret_cast<const int4 *>(a.items + next / a.num_kv_heads);
            int4 *to = reinterpret_cast<int4 *>(&x.item);
#pragma unroll
            for (int k = 0; k < int(sizeof(PrefillItem) / 16); k++) to[k] = __ldcg(from + k);
            x.head = next % a.num_kv_heads;
            x.place = x.head * a.max_slots + x.item.slot;
        }
        mbar_arrive(&s.item_full[i & 1]);
        if (x.head < 0) break;
        if (x.item.block1 == x.item.block0) continue;
        if (loads && !wait_phase(s, &s.q_empty, (loads - 1) & 1, a.flags)) break;
        loads++;
        const int halves = x.item.tokens > per ? 2 : 1;
        mbar_arrive_expect_tx(&s.q_full, halves * C::TILE);
        for (int h = 0; h < halves; h++)
#pragma unroll
            for (int c = 0; c < C::NB; c++)
                tma_load_3d(q + h * C::TILE + c * C::ATOM, map_q, c * 64, x.head * a.group, x.item.token + h * per, &s.q_full);
    }
    // the last queries have landed before the CTA's memory is released, also where nobody waits for them any more
    if (loads) mbar_wait_bounded(&s.q_full, (loads - 1) & 1, kWaitLimitNs);
}

template <int D, bool KVF>
__global__ void __launch_bounds__(kThreads<KVF>, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const __grid_constant__ PrefillArgs a) {
    using C = Cfg<D, KVF>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *q = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = q + 2 * C::TILE;
    if (threadIdx.x == 0) {
        s.abort = 0u;
        for (int i = 0; i < 2; i++) {
            mbar_init(&s.item_full[i], 1);
            mbar_init(&s.item_empty[i], kItemReaders<KVF>);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 4);
            mbar_init(&s.o_full[i], 1);
        }
        mbar_init(&s.q_full, 1);
        mbar_init(&s.q_empty, 1);
        for (int i = 0; i < C::STAGES; i++) {
            mbar_init(&s.kv_full[i], KVF ? 128 : 1);
            mbar_init(&s.kv_empty[i], 1);
        }
        for (int i = 0; i < 2 && KVF; i++) {
            mbar_init(&s.part_full[i], 8);
            mbar_init(&s.part_empty[i], 128);
        }
        mbar_init(&s.parts_done, 32 * kSoftmaxWarps);
        mbar_init(&s.last_known, 1);
        mbar_init(&s.drain, 1);
        mbar_fence_init();
    }
    if (warp == kMmaWarp) tmem_alloc(&s.tmem, 512);
    if (warp == kListWarp && lane == 0) {
        prefetch_tensormap(&map_q);
        if (!KVF) {
            prefetch_tensormap(&map_k);
            prefetch_tensormap(&map_v);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    pdl_wait();
    // registers a thread: shares of what the launch has, 3 x 168 (2 x 208 + 88) or 4 x 128 (2 x 176 + 64 + 96)
    if (warp < kSoftmaxWarps) {
        regs_inc<KVF ? 176 : 208>();
        softmax_role<D, KVF>(a, s, ring, s.tmem);
    } else if (warp < kConvertWarp) {
        regs_dec<KVF ? 64 : 88>();
        if (warp == kMmaWarp) {
            mma_role<D, KVF>(a, s, smem_u32(q), smem_u32(ring));
        } else if (!KVF && (warp == kLoadWarp || warp == kLoadWarp + 1)) {
            load_role<D>(a, s, ring, warp == kLoadWarp ? &map_k : &map_v, warp - kLoadWarp);
        } else if (KVF && warp == kLoadWarp) {
            fetch_role<D>(a, s, ring + C::STAGES * C::TILE);
        } else if (warp == kListWarp) {
            list_role<D>(a, s, q, &map_q);
            __syncwarp();
        }
    } else if constexpr (KVF) {
        regs_dec<96>();
        convert_role<D>(a, s, ring, ring + C::STAGES * C::TILE);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(s.tmem, 512);
}

template <int D, bool KVF>
cudaError_t launch_one(const PrefillArgs &a, const CUtensorMap *q, const CUtensorMap *k, const CUtensorMap *v,
                       cudaStream_t stream) {
    auto kernel = prefill_tc_kernel<D, KVF>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, KVF>::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t most = int64_t(a.max_items) * a.num_kv_heads;
    return launch_pdl(kernel, dim3(unsigned(most < a.num_sms ? most : a.num_sms)), dim3(kThreads<KVF>),
                      size_t(Cfg<D, KVF>::SMEM), stream, *q, *k, *v, a);
}

}  // namespace

cudaError_t launch_prefill_tc(const PrefillArgs &a, const CUtensorMap *q, const CUtensorMap *k, const CUtensorMap *v,
                              int head_dim, cudaStream_t stream) {
    if (a.pool) return head_dim == 128 ? launch_one<128, true>(a, q, k, v, stream) : launch_one<64, true>(a, q, k, v, stream);
    return head_dim == 128 ? launch_one<128, false>(a, q, k, v, stream) : launch_one<64, false>(a, q, k, v, stream);
}

}  // namespace qskv
