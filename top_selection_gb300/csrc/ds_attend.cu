// ds_attend.cu -- attention of new tokens over a paged cache of 4-bit keys and values
// (ds_cache_attention): every position of the context, or the positions a top-k selected.
//
// A key row of the cache stands for s c + m (codes c, bf16 scale s and minimum m, see
// ds_cache.cu), so a query row q scores it as
//     q . (s c + m) = s (q . c) + m (sum q).
// With weights p and w = f16(p s) (times a power of two), the values add up to
//     sum p (s c + m) = sum w c  +  sum p (m + 7.5 s)  -  7.5 sum w,
// the rounding of w meeting centred codes only: were it to meet c itself, errors of one sign
// (equal weights) would be large against a result that averages out.  sum w comes from the
// matrix unit as well, against a row of ones.
//
// The codes never leave registers once they are there: with tokens as the rows of the matrix
// instruction, the four lanes that share a fragment row read a token's codes as they lie in
// memory (any order of the contracted dimension serves, as long as q is read in the same
// order).  A masked word is the operand: the 16-bit pattern c, or 16 c, is the subnormal f16
// number c 2^-24, or 16 c 2^-24, which the matrix unit multiplies exactly; the powers of two
// are taken out of q beforehand and out of the sums at the end.  Eight codes cost five
// instructions (one shift, four ANDs; value words of two tokens are interleaved first).
//
// m16n8k16 (mma.sync) rather than tcgen05: a step has 8 to 32 query rows per key head, the
// operand that streams is the cache, and tcgen05 takes it from shared memory only, so each
// tile would be expanded to four times its bytes, stored and read back.  Here the cache's
// bytes are the operand.
//
// Rows: the query rows that share a key head (heads of a group, and for whole contexts the
// tokens of the step as well) in tiles of 8; a CTA takes up to 8 * NT of them and one split of
// the positions; its warps take tiles of 32 positions in turn, each through its own ring of
// asynchronous copies.  Softmax runs online per warp: one running maximum per row, raised only
// when a score passes it by 2^kRaise, sums per lane.  Warps are joined in shared memory, splits
// by a second kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kAttWarps = 4;
constexpr int kAttTile = 32;                   // positions per warp and step
constexpr int kAttStages = 3;                  // tiles of a warp's ring
constexpr int kAttCluster = 8;                 // portable cluster size
constexpr uint32_t kNoEntry = 0xFFFFFFFFu;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -1e30f;                // running maximum of a row that has seen nothing
// Weights as f16: p is at most 2^kRaise, and w = p s kTop / r, r a power of two near the largest
// value scale s seen and never below an eighth of one.  The largest w is 16 * 8 * 256 = 2^15
// (f16 ends at 2^16), and the heaviest position's is about 2^8, 22 binades above the subnormals.
constexpr float kRaise = 4.0f, kTop = 256.0f, kOver = 2048.0f;

struct AttendParams {
    const void* q;
    int64_t q_seq, q_tok, q_head;  // element strides
    const uint8_t* cache;
    const uint2* scales;           // per entry: key (s, m), value (s, m)
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lens;
    const int32_t* indices;        // [B, Q, K] or null
    void* out;
    float* lse;
    float* ws_o;                   // split partials: [unit][split][rows][D]
    float* ws_ml;                  //                 [unit][split][rows][2]
    int64_t max_pos;               // table width * page
    int32_t Q, K, heads, group, page_log, pages;
    int32_t rows;                  // query rows per unit before tiling
    int32_t row_groups, splits, chunk;
    int32_t q_vec;                 // q rows start on 16 bytes
    int32_t cluster;               // the splits of a unit are one cluster and join in it
    float scale;
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// (a, b) = the sum of NS pairs of f16 (11 bits each)
template <int NS>
__device__ __forceinline__ void split_f16(float a, float b, uint32_t (&part)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        part[i] = pack_f16(a, b);
        if (i + 1 < NS) {
            const float2 f = unpack_f16(part[i]);
            a -= f.x;
            b -= f.y;
        }
    }
}

// Codes `nib` (0 .. 3) of both halves of w (w already moved down by 8 for nib >= 2): two f16
// numbers c 2^-24, for odd nib 16 c 2^-24.  CENTRE: c - 8 instead of c, exact as well.
template <bool CENTRE>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int nib) {
    const uint32_t x = w & (nib & 1 ? 0x00F000F0u : 0x000F000Fu);
    if (!CENTRE) return x;
    const uint32_t c8 = nib & 1 ? 0x00800080u : 0x00080008u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&c8));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// 2^x with a relative error of 2^-22: an error the weight has already from its argument.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// two fp32 numbers to an instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
// four results times f, in the output's type
__device__ __forceinline__ void store4(float* p, float4 v, float f) {
    *reinterpret_cast<float4*>(p) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v, float f) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * f, v.y * f), b = __floats2bfloat162_rn(v.z * f, v.w * f);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// asynchronous copies global -> shared; `on` false fills the bytes with zeros
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool on) {
    const int n = on ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// 16 bytes at `at` bytes behind both addresses
template <int AT>
__device__ __forceinline__ void copy_async_at(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;" ::"r"(dst), "l"(src), "n"(AT) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A tile in shared memory: 32 rows of D bytes (key codes, value codes) and their scales.
// 16-byte pieces of a row are permuted so that the reads of a warp meet every
// bank once: a key read takes 8 rows by the lanes' quarter, a value read rows 2t apart.
template <int D>
struct TileAt {
    static constexpr int kRowBytes = D;
    static constexpr int kScaleAt = kAttTile * D;
    static constexpr int kBytes = kScaleAt + kAttTile * 8;
    static __device__ __forceinline__ int piece(int row, int chunk) {
        const int x = D == 128 ? (((row >> 1) & 3) << 1) ^ ((row & 1) << 2) : ((row >> 1) & 1) << 1;
        return row * D + ((chunk ^ x) << 4);
    }
};

// CTAs per SM that the registers are cut for
template <typename T>
constexpr int att_resident(int D, int NT) {
    return sizeof(T) == 4 ? (NT == 1 ? 3 : 2) : NT == 1 ? 4 : 2;
}

// T: type of q and out.  NQ / NP: f16 parts of q and of the weights.  bf16: one part each (q is
// exact, a weight keeps 11 bits, and the result's rounding to 8 dominates); fp32: two, 22 bits,
// and the codes centred, so that sums cancel less.
template <typename T, int D, int NT, int NQ, int NP>
__global__ void __launch_bounds__(kAttWarps * 32, att_resident<T>(D, NT)) ds_attend_kernel(const AttendParams p) {
    constexpr int KS = D / 16;       // k-steps of the scores, and row tiles of the output
    constexpr int ROWS = 8 * NT;
    constexpr bool CENTRE = sizeof(T) == 4;
    constexpr float MID = CENTRE ? 8.f : 7.5f;
    using At = TileAt<D>;
    extern __shared__ __align__(128) unsigned char smem[];  // the warps' rings; then the join
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait();

    // unit = ((sequence [, query token]) * heads + head) * row_groups + row group
    const uint32_t unit = blockIdx.x / static_cast<uint32_t>(p.splits);
    const int split = static_cast<int>(blockIdx.x - unit * p.splits);
    const uint32_t uh = unit / static_cast<uint32_t>(p.row_groups);
    const int rg = static_cast<int>(unit - uh * p.row_groups);
    const int bq = static_cast<int>(uh / static_cast<uint32_t>(p.heads));
    const int h = static_cast<int>(uh - bq * p.heads);
    const bool picked = p.indices != nullptr;
    const int b = picked ? bq / p.Q : bq;
    const int q0 = picked ? bq % p.Q : 0;
    const int len = static_cast<int>(min(static_cast<int64_t>(p.lens[b]), p.max_pos));
    // query token i sees positions below len - (Q - 1 - i)
    const int end_all = max(picked ? len - (p.Q - 1 - q0) : len, 0);
    const int count = picked ? p.K : end_all;       // positions (or list entries) of this unit
    const int from = split * p.chunk, to = min(from + p.chunk, count);
    // without a cluster the join is a kernel, which reads only splits that have work
    if (!p.cluster && from >= count && split > 0) return;

    const int32_t* table = p.table + b * p.table_stride;
    const int32_t* list = picked ? p.indices + static_cast<int64_t>(bq) * p.K : nullptr;
    const int page_mask = (1 << p.page_log) - 1;

    const auto entry_of = [&](int j, int& pos) -> uint32_t {  // list entry or position j
        pos = 0x7FFFFFFF;
        if (j >= to) return kNoEntry;
        const int at = picked ? list[j] : j;
        if (at < 0 || at >= end_all) return kNoEntry;
        const int page = table[at >> p.page_log];
        if (page < 0 || page >= p.pages) return kNoEntry;
        pos = at;
        return ((static_cast<uint32_t>(page) * p.heads + h) << p.page_log) + (at & page_mask);
    };
    unsigned char* ring = smem + warp * (kAttStages * At::kBytes);
    const uint32_t ring_at = smem_u32(ring);
    // Copies a tile into a slot of the ring.  Positions that share a page lie side by side, so a
    // whole tile of them is one run of 32 D bytes; else each row goes by its own entry.
    constexpr int CH = D / 16, PER = 32 / CH;  // 16-byte pieces of a row; rows per instruction
    const int row0 = lane / CH, ch = lane % CH;
    const auto issue = [&](int slot, uint32_t entry, bool run) {
        const uint32_t base = ring_at + slot * At::kBytes;
        if (run) {
            const uint8_t* src = p.cache + static_cast<uint64_t>(entry) * D - (lane * D - lane * 16);
            // the permutation of a row's pieces repeats every 8 rows, two (D = 64: one) copies
            const uint32_t d0 = base + At::piece(row0, ch), d1 = base + At::piece(PER + row0, ch) - 512;
            copy_async_at<0>(d0, src);
            copy_async_at<512>(d1, src);
            copy_async_at<1024>(d0, src);
            copy_async_at<1536>(d1, src);
            if constexpr (D == 128) {
                copy_async_at<2048>(d0, src);
                copy_async_at<2560>(d1, src);
                copy_async_at<3072>(d0, src);
                copy_async_at<3584>(d1, src);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kAttTile / PER; ++i) {
                const uint32_t e = __shfl_sync(kAll, entry, i * PER + row0);
                const uint8_t* src = p.cache + (e == kNoEntry ? 0 : static_cast<uint64_t>(e) * D) + ch * 16;
                copy_async<16>(base + At::piece(i * PER + row0, ch), src, e != kNoEntry);
            }
        }
        copy_async<8>(base + At::kScaleAt + lane * 8, p.scales + (entry == kNoEntry ? 0u : entry), entry != kNoEntry);
        copies_commit();
    };
    // a tile of consecutive positions inside one page, none of them missing
    const bool runs = !picked && p.page_log >= 5;
    const auto is_run = [&](uint32_t entry) { return runs && __all_sync(kAll, entry != kNoEntry); };

    // tiles of this warp: two in flight while one is computed, and the entries of the next
    constexpr int STRIDE = kAttWarps * kAttTile;
    int j0 = from + warp * kAttTile;
    int pos[kAttStages];  // the lane's position in each tile: current, in flight, next
    uint32_t entry;
#pragma unroll
    for (int s = 0; s < kAttStages; ++s) {
        entry = entry_of(j0 + s * STRIDE + lane, pos[s]);
        if (s + 1 < kAttStages) issue(s, entry, is_run(entry));
    }

    // q as the second operand: row g of each tile, the lane's quarter of the numbers in the
    // order of the codes, times a power of two that brings the largest to 2^13 .. 2^14, and
    // another 1/16 against codes that count 16-fold
    const auto row_query = [&](int r, int64_t& off, int& end) -> bool {  // row r of the unit
        if (r >= p.rows) {
            end = 0;
            return false;
        }
        const int qi = picked ? q0 : r / p.group;
        const int hd = h * p.group + (picked ? r : r - qi * p.group);
        off = b * p.q_seq + qi * p.q_tok + hd * p.q_head;
        end = max(len - (p.Q - 1 - qi), 0);
        return true;
    };
    constexpr int QW = 2 * NT * NQ;  // words of a lane and k-step: kept in shared memory
    uint32_t* sm_q = reinterpret_cast<uint32_t*>(smem + kAttWarps * kAttStages * At::kBytes);
    float2 qsum[NT];
    int ends[NT][2];
    int first_end = 0x7FFFFFFF;  // below it no row of the CTA masks anything
    float fold;
    {
        float x[NT][D / 4];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            int64_t off = 0;
            int end = 0;
            const bool on = row_query(rg * ROWS + 8 * j + g, off, end);
            const T* q = static_cast<const T*>(p.q) + off + t * (D / 4);
            if (p.q_vec) {
                constexpr int PER = 16 / sizeof(T);
#pragma unroll
                for (int i = 0; i < D / 4 / PER; ++i) {
                    const uint4 w = on ? reinterpret_cast<const uint4*>(q)[i] : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (sizeof(T) == 2) {
                            x[j][i * PER + 2 * k] = __uint_as_float(u[k] << 16);
                            x[j][i * PER + 2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
                        } else {
                            x[j][i * PER + k] = __uint_as_float(u[k]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < D / 4; ++i) x[j][i] = on ? static_cast<float>(q[i]) : 0.f;
            }
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) {
                sum += x[j][i];
                const float a = fabsf(x[j][i]);
                top = fmaxf(top, a < INFINITY ? a : 0.f);
            }
            sum += __shfl_xor_sync(kAll, sum, 1);
            sum += __shfl_xor_sync(kAll, sum, 2);
            // rows 2t + c sit in lanes 4 (2t + c)
            qsum[j] = make_float2(__shfl_sync(kAll, sum, 8 * t), __shfl_sync(kAll, sum, 8 * t + 4));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                int64_t o2;
                const bool on2 = row_query(rg * ROWS + 8 * j + 2 * t + c, o2, ends[j][c]);
                if (on2) first_end = min(first_end, ends[j][c]);
            }
        }
        first_end = __reduce_min_sync(kAll, first_end);
        const uint32_t e = __reduce_max_sync(kAll, __float_as_uint(top)) >> 23;  // biased exponent
        const int up = e == 0u ? 0 : min(max(13 - (static_cast<int>(e) - 127), -100), 100);
        const float by = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
        fold = p.scale * kLog2e;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            qsum[j].x *= fold;
            qsum[j].y *= fold;
        }
        // each warp writes its share of the k-steps
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            if (kk % kAttWarps != warp) continue;
            uint32_t w[QW];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int d = 8 * (kk / 2) + 2 * (kk % 2) + half;
                    const float f = half ? by * 0.0625f : by;
                    uint32_t part[NQ];
                    split_f16<NQ>(x[j][d] * f, x[j][d + 4] * f, part);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) w[(j * NQ + n) * 2 + half] = part[n];
                }
#pragma unroll
            for (int i = 0; i < QW / 2; ++i)
                reinterpret_cast<uint2*>(sm_q)[(kk * 32 + lane) * (QW / 2) + i] = make_uint2(w[2 * i], w[2 * i + 1]);
        }
        fold *= 16777216.f * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
    }

    __syncthreads();
    float o[NT][KS][4], ones[NT][4];
    float2 neg_m[NT], l[NT], z[NT];  // minus the running maximum, sums of p and p (m + MID s)
    uint32_t unseen = 0u;            // rows of this lane without a score so far
    bool fresh = true;               // the warp has such a row
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[j][mt][c] = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) ones[j][c] = 0.f;
        neg_m[j] = l[j] = z[j] = both(0.f);
        const int r = rg * ROWS + 8 * j + 2 * t;
        unseen |= (r < p.rows ? 1u : 0u) << (2 * j) | (r + 1 < p.rows ? 2u : 0u) << (2 * j);
    }
    float wmul = 1.2676506e30f;  // kTop / r; 2^100 until a value scale has been seen

    int slot = 0;
    for (; j0 < to; j0 += STRIDE) {
        copies_wait<kAttStages - 2>();
        __syncwarp();
        {
            int next = slot + kAttStages - 1;
            if (next >= kAttStages) next -= kAttStages;
            issue(next, entry, is_run(entry));
        }
        const int here = pos[0];
#pragma unroll
        for (int i = 0; i + 1 < kAttStages; ++i) pos[i] = pos[i + 1];
        entry = entry_of(j0 + kAttStages * STRIDE + lane, pos[kAttStages - 1]);
        const unsigned char* tile = ring + slot * At::kBytes;
        if (++slot == kAttStages) slot = 0;

        // scores of 32 positions: rows of tile i are positions 16 i + {g, g + 8}
        float s[NT][2][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[j][i][c] = 0.f;
        uint32_t kw[4][D / 32];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 8 * r + g;
            if constexpr (D == 128) {
                const uint4 w = *reinterpret_cast<const uint4*>(tile + At::piece(row, t));
                kw[r][0] = w.x, kw[r][1] = w.y, kw[r][2] = w.z, kw[r][3] = w.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2*>(tile + At::piece(row, t >> 1) + 8 * (t & 1));
                kw[r][0] = w.x, kw[r][1] = w.y;
            }
        }
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            const int sh = 8 * (kk & 1);
            uint32_t qf[QW];
            if constexpr (QW == 2) {
                const uint2 w = reinterpret_cast<const uint2*>(sm_q)[kk * 32 + lane];
                qf[0] = w.x, qf[1] = w.y;
            } else {
#pragma unroll
                for (int i = 0; i < QW / 4; ++i) {
                    const uint4 w = reinterpret_cast<const uint4*>(sm_q)[(kk * 32 + lane) * (QW / 4) + i];
                    qf[4 * i] = w.x, qf[4 * i + 1] = w.y, qf[4 * i + 2] = w.z, qf[4 * i + 3] = w.w;
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t w0 = kw[2 * i][kk / 2] >> sh, w1 = kw[2 * i + 1][kk / 2] >> sh;
                const uint32_t a0 = code_pair<CENTRE>(w0, 0), a1 = code_pair<CENTRE>(w1, 0);
                const uint32_t a2 = code_pair<CENTRE>(w0, 1), a3 = code_pair<CENTRE>(w1, 1);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        mma_f16(s[j][i], a0, a1, a2, a3, qf[(j * NQ + n) * 2], qf[(j * NQ + n) * 2 + 1]);
            }
        }
        float vs[4], vm[4];
        int at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint2 sc = *reinterpret_cast<const uint2*>(tile + At::kScaleAt + (8 * i + g) * 8);
            const float ks = __uint_as_float(sc.x << 16), km = __uint_as_float(sc.x & 0xFFFF0000u);
            vs[i] = __uint_as_float(sc.y << 16);
            vm[i] = fmaf(MID, vs[i], __uint_as_float(sc.y & 0xFFFF0000u));
            const float2 f = both(ks * fold), base = both(CENTRE ? fmaf(8.f, ks, km) : km);
#pragma unroll
            for (int j = 0; j < NT; ++j) {  // relative to the running maximum
                float* x = &s[j][i / 2][2 * (i & 1)];
                const float2 y = fma2(make_float2(x[0], x[1]), f, fma2(base, qsum[j], neg_m[j]));
                x[0] = y.x;
                x[1] = y.y;
            }
        }
        // positions that some row does not see: their scores become -inf and their weights 0.
        // A scale that is not finite would still make NaN of a weight of 0 (`odd`).
        bool odd = false;
        if (__any_sync(kAll, here >= first_end)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                at[i] = __shfl_sync(kAll, here, 8 * i + g);
                odd |= !(fabsf(vs[i]) < INFINITY && fabsf(vm[i]) < INFINITY);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        if (at[i] >= ends[j][c]) s[j][i / 2][2 * (i & 1) + c] = -INFINITY;
            }
            odd = __any_sync(kAll, odd);
        }
        // raise the running maxima where a score passes one by 2^kRaise (or is the first), and
        // r where a value scale leaves it behind
        float vw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) vw[i] = vs[i] * wmul;
        float2 high[NT];
        float most = -INFINITY;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            high[j].x = fmaxf(max3(s[j][0][0], s[j][0][2], s[j][1][0]), s[j][1][2]);
            high[j].y = fmaxf(max3(s[j][0][1], s[j][0][3], s[j][1][1]), s[j][1][3]);
            most = max3(most, high[j].x, high[j].y);
        }
        if (fresh || __any_sync(kAll, most > kRaise || fmaxf(max3(vw[0], vw[1], vw[2]), vw[3]) > kOver)) {
            float vtop = 1e-30f;
#pragma unroll
            for (int i = 0; i < 4; ++i) vtop = fmaxf(vtop, vs[i] < INFINITY ? vs[i] : 0.f);
            const uint32_t vbits = __reduce_max_sync(kAll, __float_as_uint(vtop));
            float change = 1.f;
            if (__uint_as_float(vbits) * wmul > kOver) {  // r = the power of two at or below vtop
                const float to_mul = kTop / __uint_as_float(vbits & 0x7F800000u);
                change = to_mul / wmul;
                wmul = to_mul;
#pragma unroll
                for (int i = 0; i < 4; ++i) vw[i] = vs[i] * wmul;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float2 x = high[j];
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) {
                    x.x = fmaxf(x.x, __shfl_xor_sync(kAll, x.x, d));
                    x.y = fmaxf(x.y, __shfl_xor_sync(kAll, x.y, d));
                }
                // a row's first score sets its maximum, up or down; nothing is summed yet
                float2 by = make_float2(1.f, 1.f);
                if (unseen >> (2 * j) & 1u) { if (x.x > -INFINITY) unseen &= ~(1u << (2 * j)); else x.x = 0.f; }
                else { x.x = fmaxf(x.x, 0.f); by.x = exp2_fast(-x.x); }
                if (unseen >> (2 * j + 1) & 1u) { if (x.y > -INFINITY) unseen &= ~(2u << (2 * j)); else x.y = 0.f; }
                else { x.y = fmaxf(x.y, 0.f); by.y = exp2_fast(-x.y); }
                const float2 down = make_float2(-x.x, -x.y);
                neg_m[j] = add2(neg_m[j], down);
                l[j] = mul2(l[j], by);
                z[j] = mul2(z[j], by);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float* y = &s[j][i / 2][2 * (i & 1)];
                    y[0] += down.x;
                    y[1] += down.y;
                }
                const float2 all = mul2(by, both(change));
#pragma unroll
                for (int mt = 0; mt < KS; ++mt) {
                    o[j][mt][0] *= all.x, o[j][mt][1] *= all.y;
                    o[j][mt][2] *= all.x, o[j][mt][3] *= all.y;
                }
                ones[j][0] *= all.x, ones[j][1] *= all.y;
            }
            fresh = __any_sync(kAll, unseen != 0u);
        }
        // weights p, their sums, and w as the second operand
        uint32_t wf[NT][2][2][NP];  // [row tile][16 positions][first or second 8][part]
        const auto weigh = [&](auto masked) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 vw2 = both(vw[i]), vm2 = both(vm[i]);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float* x = &s[j][i / 2][2 * (i & 1)];
                    const float2 e = make_float2(exp2_fast(x[0]), exp2_fast(x[1]));
                    l[j] = add2(l[j], e);
                    float2 w = mul2(e, vw2), zn = fma2(e, vm2, z[j]);
                    if (masked.value) {
                        if (at[i] >= ends[j][0]) w.x = 0.f, zn.x = z[j].x;
                        if (at[i] >= ends[j][1]) w.y = 0.f, zn.y = z[j].y;
                    }
                    z[j] = zn;
                    uint32_t part[NP];
                    split_f16<NP>(w.x, w.y, part);
#pragma unroll
                    for (int n = 0; n < NP; ++n) wf[j][i / 2][i & 1][n] = transpose8x8(part[n]);
                }
            }
        };
        if (!odd) weigh(std::false_type{});
        else weigh(std::true_type{});
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // value words of positions 16 i + {2t, 2t + 1, 2t + 8, 2t + 9}, the lane's eighth
            uint32_t v[4][D / 64];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * i + 8 * (r >> 1) + 2 * t + (r & 1);
                if constexpr (D == 128) {
                    const uint2 w = *reinterpret_cast<const uint2*>(tile + At::piece(row, 4 + (g >> 1)) + 8 * (g & 1));
                    v[r][0] = w.x, v[r][1] = w.y;
                } else {
                    v[r][0] = *reinterpret_cast<const uint32_t*>(tile + At::piece(row, 2 + (g >> 2)) + 4 * (g & 3));
                }
            }
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
                const uint32_t xl = __byte_perm(v[0][w], v[1][w], 0x5410), xh = __byte_perm(v[0][w], v[1][w], 0x7632);
                const uint32_t yl = __byte_perm(v[2][w], v[3][w], 0x5410), yh = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
                for (int nib = 0; nib < 4; ++nib) {
                    const int sh = nib >= 2 ? 8 : 0;
                    const uint32_t a0 = code_pair<CENTRE>(xl >> sh, nib), a1 = code_pair<CENTRE>(xh >> sh, nib);
                    const uint32_t a2 = code_pair<CENTRE>(yl >> sh, nib), a3 = code_pair<CENTRE>(yh >> sh, nib);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int n = 0; n < NP; ++n)
                            mma_f16(o[j][4 * w + nib], a0, a1, a2, a3, wf[j][i][0][n], wf[j][i][1][n]);
                }
            }
            if constexpr (!CENTRE) {  // sum of w, against ones
                constexpr uint32_t ONE = 0x3C003C00u;
#pragma unroll
                for (int j = 0; j < NT; ++j) mma_f16(ones[j], ONE, ONE, ONE, ONE, wf[j][i][0][0], wf[j][i][1][0]);
            }
        }
    }
    copies_wait<0>();
    __syncthreads();  // every warp is done with its ring

    // join the warps: sums over the lanes of a row, then shared memory
    float* sm_o = reinterpret_cast<float*>(smem);        // [warps][ROWS][D]
    float* sm_r = sm_o + kAttWarps * ROWS * D;           // [warps][ROWS][4]
    const float back = 1.f / wmul;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        float ls[2] = {l[j].x, l[j].y}, zs[2] = {z[j].x, z[j].y};
        const float ms[2] = {unseen >> (2 * j) & 1u ? kNone : -neg_m[j].x, unseen >> (2 * j) & 2u ? kNone : -neg_m[j].y};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) {
                ls[c] += __shfl_xor_sync(kAll, ls[c], d);
                zs[c] += __shfl_xor_sync(kAll, zs[c], d);
            }
            if (!CENTRE) zs[c] -= 7.5f * ones[j][c] * back;
            const int r = 8 * j + 2 * t + c;
            if (g == 0) {
                float* q = sm_r + (warp * ROWS + r) * 4;
                q[0] = ms[c], q[1] = ls[c], q[2] = zs[c];
            }
            // numbers of the lane: its eighth, word w, code nib (+ 4 in the fragment's second half)
            float* dst = sm_o + (warp * ROWS + r) * D + g * (D / 8);
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
                const float f = mt & 1 ? 1048576.f : 16777216.f;
                dst[8 * (mt / 4) + mt % 4] = o[j][mt][c] * f * back;
                dst[8 * (mt / 4) + mt % 4 + 4] = o[j][mt][c + 2] * f * back;
            }
        }
    }
    __syncthreads();
    const int rows = min(ROWS, p.rows - rg * ROWS);
    const auto result = [&](int r, int d, float4 acc, float top, float sum) {
        const int ur = rg * ROWS + r;
        const int qi = picked ? q0 : ur / p.group;
        const int hd = h * p.group + (picked ? ur : ur - qi * p.group);
        const int64_t e = (static_cast<int64_t>(b) * p.Q + qi) * (static_cast<int64_t>(p.heads) * p.group) + hd;
        store4(static_cast<T*>(p.out) + e * D + d, acc, sum > 0.f ? 1.f / sum : 0.f);
        if (d == 0 && p.lse) p.lse[e] = sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
    };
    float* sm_j = sm_r + kAttWarps * ROWS * 4;           // the CTA's join, for its cluster: [ROWS][D]
    float* sm_ml = sm_j + ROWS * D;                      // [ROWS][2]
    for (int i = tid; i < rows * (D / 4); i += kAttWarps * 32) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float top = kNone;
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) top = fmaxf(top, sm_r[(w * ROWS + r) * 4]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) {
            const float* q = sm_r + (w * ROWS + r) * 4;
            const float4 x = *reinterpret_cast<const float4*>(sm_o + (w * ROWS + r) * D + d);
            const float f = exp2_fast(q[0] - top);
            acc.x += f * (x.x + q[2]), acc.y += f * (x.y + q[2]);
            acc.z += f * (x.z + q[2]), acc.w += f * (x.w + q[2]);
            sum += f * q[1];
        }
        if (p.splits == 1) {
            result(r, d, acc, top, sum);
        } else if (p.cluster) {
            *reinterpret_cast<float4*>(sm_j + r * D + d) = acc;
            if (d == 0) *reinterpret_cast<float2*>(sm_ml + r * 2) = make_float2(top, sum);
        } else {
            const int64_t e = (static_cast<int64_t>(unit) * p.splits + split) * ROWS + r;
            *reinterpret_cast<float4*>(p.ws_o + e * D + d) = acc;
            if (d == 0) *reinterpret_cast<float2*>(p.ws_ml + e * 2) = make_float2(top, sum);
        }
    }
    if (!p.cluster) return;
    // every CTA of the cluster joins its share of the rows from all of them
    cluster_sync_all();
    for (int i = split * (kAttWarps * 32) + tid; i < rows * (D / 4); i += p.splits * (kAttWarps * 32)) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float top = kNone;
        for (int c = 0; c < p.splits; ++c)
            top = fmaxf(top, __uint_as_float(ld_cluster_u32(map_rank(sm_ml + r * 2, c))));
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll 4
        for (int c = 0; c < p.splits; ++c) {
            const uint32_t ml = map_rank(sm_ml + r * 2, c);
            const uint4 x = ld_cluster_v4(map_rank(sm_j + r * D + d, c));
            const float f = exp2_fast(__uint_as_float(ld_cluster_u32(ml)) - top);
            acc.x += f * __uint_as_float(x.x), acc.y += f * __uint_as_float(x.y);
            acc.z += f * __uint_as_float(x.z), acc.w += f * __uint_as_float(x.w);
            sum += f * __uint_as_float(ld_cluster_u32(ml + 4));
        }
        result(r, d, acc, top, sum);
    }
    cluster_sync_all();  // the others have read this CTA's share
}

// Joins the splits of one query row: one CTA per row, its warps take the splits in turn.
// Only the splits that hold positions are read (the others wrote nothing); their order is
// fixed, so a call's result does not depend on timing.
template <typename T, int D>
__global__ void __launch_bounds__(1024) ds_attend_join_kernel(const AttendParams p, int ROWS) {
    __shared__ __align__(16) float sh_o[32][D];
    __shared__ float sh_l[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    constexpr int PER = D / 32;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t at = blockIdx.x;  // (sequence * Q + token) * query heads + head
    const int hq = p.heads * p.group;
    const int bq = static_cast<int>(blockIdx.x / static_cast<uint32_t>(hq));
    const int hd = static_cast<int>(blockIdx.x - bq * hq);
    const int b = bq / p.Q, qi = bq - b * p.Q;
    const bool picked = p.indices != nullptr;
    const int ur = picked ? hd % p.group : qi * p.group + hd % p.group;
    const int64_t unit = (static_cast<int64_t>(picked ? bq : b) * p.heads + hd / p.group) * p.row_groups + ur / ROWS;
    const int64_t len = min(static_cast<int64_t>(p.lens[b]), p.max_pos);
    const int64_t count = picked ? p.K : max(len, int64_t(0));
    const int splits = max(1, min(p.splits, static_cast<int>((count + p.chunk - 1) / p.chunk)));
    const int64_t base = unit * p.splits * ROWS + ur % ROWS;
    float top = kNone;
    for (int s = lane; s < splits; s += 32) top = fmaxf(top, p.ws_ml[(base + static_cast<int64_t>(s) * ROWS) * 2]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
    float acc[PER], sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int s = warp; s < splits; s += warps) {
        const int64_t e = base + static_cast<int64_t>(s) * ROWS;
        const float2 ml = *reinterpret_cast<const float2*>(p.ws_ml + e * 2);
        const float f = exp2_fast(ml.x - top);
        sum += f * ml.y;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] += f * p.ws_o[e * D + lane * PER + i];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) sh_o[warp][lane * PER + i] = acc[i];
    if (lane == 0) sh_l[warp] = sum;
    __syncthreads();
    for (int d = threadIdx.x * 4; d < D; d += blockDim.x * 4) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        float total = 0.f;
        for (int w = 0; w < warps; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(&sh_o[w][d]);
            y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
            total += sh_l[w];
        }
        store4(static_cast<T*>(p.out) + at * D + d, y, total > 0.f ? 1.f / total : 0.f);
        if (d == 0 && p.lse) p.lse[at] = total > 0.f ? (top + log2f(total)) * kLn2 : -INFINITY;
    }
}

template <typename T, int D, int NT>
static ds_status attend(const AttendParams& p, int dev, int64_t units, int64_t out_rows, cudaStream_t stream) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    auto kern = ds_attend_kernel<T, D, NT, PARTS, PARTS>;
    const size_t ring = static_cast<size_t>(kAttWarps) * kAttStages * TileAt<D>::kBytes + D / 16 * 32 * 8 * NT * PARTS;
    const size_t join = (static_cast<size_t>(kAttWarps) * (D + 4) + D + 2) * 8 * NT * sizeof(float);
    const size_t smem = ring > join ? ring : join;
    // the opt-in above 48 KB is a property of the kernel on a device: set once
    static std::atomic<bool> opted[64];
    if (smem > 48 * 1024 && !opted[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
            return DS_ERR_CUDA;
        opted[dev].store(true, std::memory_order_release);
    }
    const dim3 grid(static_cast<unsigned>(units * p.splits));
    const ds_status st = launch_pdl(kern, grid, kAttWarps * 32, smem, p.cluster ? p.splits : 1, stream, p);
    if (st != DS_OK || p.splits == 1 || p.cluster) return st;
    int warps = 1;
    while (warps < 32 && 4 * warps < p.splits) warps <<= 1;
    return launch_pdl(ds_attend_join_kernel<T, D>, dim3(static_cast<unsigned>(out_rows)), warps * 32, 0, 1, stream, p,
                      8 * NT);
}

template <typename T, int D>
static ds_status attend_rows(const AttendParams& p, int dev, int nt, int64_t units, int64_t out_rows, cudaStream_t stream) {
    if (nt == 1) return attend<T, D, 1>(p, dev, units, out_rows, stream);
    return attend<T, D, 2>(p, dev, units, out_rows, stream);
}

}  // namespace dsk

using namespace dsk;

extern "C" {

ds_status ds_cache_attention(const void* q, int32_t dtype, int64_t sequences, int32_t tokens, int32_t q_heads,
                             int32_t D, int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride,
                             const void* cache, const void* scales, int64_t pages, int32_t heads, int32_t page,
                             const int32_t* table, int64_t table_width, int64_t table_stride, const int32_t* lens,
                             const int32_t* indices, int32_t K, float scale, void* out, float* out_lse,
                             cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || sequences < 0 || tokens < 1 || q_heads < 1 || heads < 1 ||
        q_heads % heads != 0 || pages < 1 || page < 1 || table_width < 1 || table_stride < table_width || K < 0)
        return DS_ERR_INVALID_ARG;
    if (q_seq_stride < 0 || q_token_stride < 0 || q_head_stride < 0 || !isfinite(scale)) return DS_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || (page & (page - 1)) != 0) return DS_ERR_UNSUPPORTED;
    if (pages * page * heads >= 0xFFFFFFFFLL || pages > 0x7FFFFFFFLL || table_width > (int64_t(1) << 30) / page)
        return DS_ERR_UNSUPPORTED;
    if (sequences == 0) return DS_OK;
    if (!q || !cache || !scales || !table || !lens || !out || (K > 0 && !indices)) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    if (!aligned16(cache) || reinterpret_cast<uintptr_t>(scales) % 8 || reinterpret_cast<uintptr_t>(q) % es ||
        !aligned16(out))
        return DS_ERR_ALIGNMENT;
    const void* words[] = {table, lens, indices, out_lse};
    for (const void* w : words)
        if (reinterpret_cast<uintptr_t>(w) % 4) return DS_ERR_ALIGNMENT;
    int dev = 0;
    DevInfo info;
    if (cudaGetDevice(&dev) != cudaSuccess || !dev_info(dev, info)) return DS_ERR_CUDA;

    AttendParams p = {};
    p.q = q;
    p.q_seq = q_seq_stride;
    p.q_tok = q_token_stride;
    p.q_head = q_head_stride;
    p.cache = static_cast<const uint8_t*>(cache);
    p.scales = static_cast<const uint2*>(scales);
    p.table = table;
    p.table_stride = table_stride;
    p.lens = lens;
    p.indices = indices;
    p.out = out;
    p.lse = out_lse;
    p.max_pos = table_width * page;
    p.Q = tokens;
    p.K = K;
    p.heads = heads;
    p.group = q_heads / heads;
    while ((1 << p.page_log) < page) ++p.page_log;
    p.pages = static_cast<int32_t>(pages);
    p.scale = scale;
    p.q_vec = aligned16(q) && q_seq_stride * es % 16 == 0 && q_token_stride * es % 16 == 0 && q_head_stride * es % 16 == 0;
    const int64_t rows = indices ? p.group : static_cast<int64_t>(p.group) * tokens;
    if (rows > (1 << 20)) return DS_ERR_UNSUPPORTED;
    p.rows = static_cast<int32_t>(rows);
    const int nt = rows > 8 ? 2 : 1;
    p.row_groups = (p.rows + 8 * nt - 1) / (8 * nt);
    const int64_t units = (indices ? sequences * tokens : sequences) * heads * p.row_groups;
    const int64_t out_rows = sequences * tokens * q_heads;
    // Splits: two CTAs for each place on an SM (what one leaves over at its end another fills;
    // 4M positions of 16 rows: one 174 us, two 150, three 160, four 170), at least two tiles a warp.
    const int64_t span = indices ? K : p.max_pos;
    const int64_t unit_tiles = kAttWarps * kAttTile;
    const int64_t places = static_cast<int64_t>(info.sms) *
                           (dtype == DS_BF16 ? att_resident<__nv_bfloat16>(D, nt) : att_resident<float>(D, nt));
    int64_t splits = (2 * places + units - 1) / units;
    const int64_t most = (span + 2 * unit_tiles - 1) / (2 * unit_tiles);
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
    int64_t chunk = (span + splits - 1) / splits;
    chunk = (chunk + unit_tiles - 1) / unit_tiles * unit_tiles;
    if (chunk < unit_tiles) chunk = unit_tiles;
    splits = (span + chunk - 1) / chunk;
    if (splits < 1) splits = 1;
    p.splits = static_cast<int32_t>(splits);
    p.chunk = static_cast<int32_t>(chunk);
    if (units * splits > 0x7FFFFFFFLL || out_rows > 0x7FFFFFFFLL) return DS_ERR_UNSUPPORTED;
    // Lists have one length: up to 8 splits of one are a cluster and join over its shared memory
    // (512 positions for 64 rows: 12.7 us, through the workspace 15.0).  Contexts differ in theirs,
    // and a cluster holds its places until the longest split is done (48 contexts of up to 8192
    // positions: 114 us, through the workspace 90).
    p.cluster = indices && splits > 1 && splits <= kAttCluster;
    if (splits > 1 && !p.cluster) {
        const size_t entries = static_cast<size_t>(units) * splits * 8 * nt;
        void* ws = nullptr;
        const ds_status st = library_workspace(dev, kWsAttend, entries * (D + 2) * sizeof(float), stream, &ws);
        if (st != DS_OK) return st;
        p.ws_o = static_cast<float*>(ws);
        p.ws_ml = p.ws_o + entries * D;
    }
    if (dtype == DS_BF16)
        return D == 64 ? attend_rows<__nv_bfloat16, 64>(p, dev, nt, units, out_rows, stream)
                       : attend_rows<__nv_bfloat16, 128>(p, dev, nt, units, out_rows, stream);
    return D == 64 ? attend_rows<float, 64>(p, dev, nt, units, out_rows, stream)
                   : attend_rows<float, 128>(p, dev, nt, units, out_rows, stream);
}

}  // extern "C"
