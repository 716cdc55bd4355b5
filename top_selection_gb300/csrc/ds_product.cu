// ds_product.cu -- the experts' products in 8 bits (ds_expert_product): rows sorted by expert times
// each expert's weights, both e4m3 with an fp32 scale for each block of 128.
//
//   out[r, n] = sum_b xs[r, b] ws[e, n / 128, b] sum_{k in block b} x[r, k] w[e, n, k]
//
// tcgen05 (kind::f8f6f4, M = 128 rows, N = BN weights' rows, K = 32 an instruction) sums one block of
// 128 along k from shared memory into tensor memory; the scales of a block differ from row to row, so
// each block's sums are read back, multiplied by their row's scale and added up in registers in
// fp32, while the next blocks are being multiplied (512 / BN buffers in tensor memory).
//
// Warps 0 to 7 add up and store, warp 8 loads (TMA, 128-byte swizzle), warp 9 issues the products, warp
// 10 brings the scales of each block to shared memory (where the warps that add up read them from
// memory, their latency came once a block: 403 us instead of 293 in the case below).
// A tile is up to 128 rows of one expert by BN outputs; CTAs take tiles in turn.  Rows of a
// tile that lie behind the expert's last are computed from whatever is in shared memory and not
// stored (no row's sums meet another's); of the rows only 32 at a time as needed are loaded.
// Few tiles: the CTAs of a cluster split a tile's blocks, and add their sums over distributed shared
// memory in a fixed order.
//
// 32768 rows over 64 experts of 4096 x 2048: 277 us, 1985 TFLOP/s, in a short graph, 310 us one call after another
// (1.77 PFLOP/s, at the power limit's clock); 8192 rows by 8192 x 8192: 2385 TFLOP/s (cuBLAS reaches 1895 on
// bf16); the tensor pipe at half; with experts of few rows the weights' bytes bound it (512 rows
// over 64 experts of 2048 x 4096: 90 us, 6.0 TB/s).  Wide tiles are stored by bulk copies from shared memory while
// the next tile is multiplied: stores of 32 bytes a lane took 46 us of 293, and a stage of loads is given up
// for it (four stages instead of three: 8192 x 8192 x 8192 in 438 us, the others the same).  A block of a
// tile takes about 510 ns, with the sums left out 450: loads, products and sums bound it together.  Order of
// the tiles, one copy of 128 rows instead of four, and the copies' L2 promotion change nothing.  Tried and not
// kept (us, of 293): pairs of CTAs (cta_group::2), whose round of products and sums goes between two SMs for
// every block (359); the weights' tiles multicast to two CTAs (316); sums loaded 64 columns at a time (296) or a
// load ahead (375, for want of registers); plain fp32 instructions for the sums (323).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_rows.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kProdRows = 128;                   // rows of a tile
constexpr int kProdBlock = 128;                  // numbers along k of a block, bytes of a swizzled row
constexpr int kProdSumWarps = 8;
constexpr int kProdThreads = (kProdSumWarps + 4) * 32;  // whole warpgroups, for the registers' split
constexpr int kProdMaxE = 512;
constexpr int kProdBox = 32;                     // rows of x to a copy
constexpr int kProdMaxSplit = 8;

// BN outputs to a tile.
template <int BN>
struct ProdShape {
    static constexpr int STAGES = BN == 256 ? 3 : 6;
    static constexpr int BUFS = 512 / BN;
    static constexpr int A_BYTES = kProdRows * kProdBlock, B_BYTES = BN * kProdBlock;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int COLS = BN / 2;           // a warp's outputs of a row
    // 12 warps of 168 registers at launch; until the roles end, the 8 that add up and the 4 others share them
    // out anew
    static constexpr int SUM_REGISTERS = BN == 256 ? 224 : 208, OTHER_REGISTERS = 3 * 168 - 2 * SUM_REGISTERS;
    // wide tiles leave through shared memory: 8 KB a warp
    static constexpr int OUT = BN == 256 ? 8192 : 0;
    static constexpr size_t SMEM = static_cast<size_t>(STAGES) * STAGE + kProdSumWarps * OUT + 1024;
};

struct ProdParams {
    const float* x_scales;
    const float* w_scales;
    const int32_t* offsets;
    void* out;
    uint32_t* status;
    int64_t rows;
    int32_t K, blocks;    // blocks of 128 along k
    int32_t N, n_blocks;  // blocks of 128 outputs
    int32_t n_tiles;      // tiles of BN outputs
    int32_t E;
    int32_t vec;          // rows of out start on 32 bytes
    int32_t bulk;         // rows of out start on 16 bytes: wide tiles are stored by bulk copies
    int32_t give_up;      // the block of a tile at which its products are given up (ds_expert_product_probe); else kNever
};
constexpr int32_t kNever = 1 << 30;  // blocks are at most 2^17

struct ProdShared {
    uint64_t full[8], empty[8], sums[8], taken[8];
    float scale[4][2][kProdRows];  // of a block's sums: buffer, half of the tile's outputs, row
    int64_t tiles[kProdMaxE + 1];  // row tiles before each expert's
    int32_t first[kProdMaxE + 1];  // rows before each expert's
    int64_t scan[kProdThreads / 32];
    uint32_t tmem;
    int failed;
    uint32_t loaded, multiplied;   // blocks whose copies, products were started
};

// ---------------------------------------------------------------- PTX ---------------
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
// A box from shared to global memory; what lies outside of the tensor is left out.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y),
                 "r"(src)
                 : "memory");
}
__device__ __forceinline__ void stores_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The thread's stores have read their shared memory; or have been written.
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// 32 columns of the warp's 32 lanes
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}
// The load before it has arrived; r are its registers, which nothing uses before.
__device__ __forceinline__ void tmem_wait_load(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Shared-memory descriptor of a K-major operand in rows of 128 bytes, 128-byte swizzle: groups of 8
// rows 1024 bytes apart.  Steps along k within the row move the address by their bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t at) {
    return static_cast<uint64_t>((at >> 4) & 0x3FFFu) | 1ull << 16 | static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 |
           2ull << 61;
}
// e4m3 by e4m3 into fp32, both K-major, M = 128, N = n
__host__ __device__ constexpr uint32_t instruction_desc(uint32_t n) { return 1u << 4 | (n >> 3) << 17 | (128u >> 4) << 24; }

// Waits for a phase, about a second at most; then (or when another wait of the CTA has run out) false.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* failed) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*failed || clock64() - t0 > kSpinLimit) {
            *failed = 1;
            return false;
        }
    }
    return true;
}

// What a CTA that gives up has started: the copies of its last blocks land in shared memory, and its products end,
// before it frees its tensor memory and leaves.  Block n uses slot n % STAGES, whose barriers complete a phase
// for each; none but these blocks' are outstanding, and no later block uses their slots.
template <int STAGES>
__device__ __forceinline__ void await_started(ProdShared& sh) {
    const auto await = [](uint64_t* bar, uint32_t parity) {
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, parity) && clock64() - t0 < kSpinLimit) {}
    };
    const uint32_t n = sh.loaded;
    for (uint32_t j = n > STAGES ? n - STAGES : 0; j < n; ++j) await(&sh.full[j % STAGES], (j / STAGES) & 1);
    // the commit behind the last block's products tells that all before are done
    if (const uint32_t last = sh.multiplied; last > 0) await(&sh.empty[(last - 1) % STAGES], ((last - 1) / STAGES) & 1);
}

using Two = unsigned long long;  // two fp32 numbers, for the packed instructions
__device__ __forceinline__ Two two(uint32_t a, uint32_t b) { return static_cast<Two>(b) << 32 | a; }
__device__ __forceinline__ void add_product(Two& sum, Two a, Two b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(sum) : "l"(a), "l"(b));
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Which tile is number t: expert, first row, rows, first output.  False behind the last.
struct Tile {
    int e, rows, n0;
    int64_t row0;
};
template <int BN>
__device__ __forceinline__ bool tile_at(const ProdShared& sh, const ProdParams& p, int64_t t, Tile& out) {
    if (t >= sh.tiles[p.E] * p.n_tiles) return false;
    int lo = 0, hi = p.E;  // the last expert whose tiles start at t or before
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (sh.tiles[mid] * p.n_tiles <= t) lo = mid;
        else hi = mid;
    }
    const int64_t high = sh.tiles[lo + 1] - sh.tiles[lo], at = t - sh.tiles[lo] * p.n_tiles;
    const int64_t m = at % high;  // tiles that run at once share weights first
    out.e = lo;
    out.n0 = static_cast<int>(at / high) * BN;
    out.row0 = sh.first[lo] + m * kProdRows;
    const int64_t left = sh.first[lo + 1] - out.row0;
    out.rows = static_cast<int>(left < kProdRows ? left : kProdRows);
    return true;
}

template <typename O>
__device__ __forceinline__ void put_out(O* p, float v) { row_put(p, v); }

template <int BN, typename O, bool SPLIT>
__global__ void __launch_bounds__(kProdThreads, 1)
ds_expert_product_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                         const __grid_constant__ CUtensorMap map_out, const ProdParams p) {
    using S = ProdShape<BN>;
    extern __shared__ uint8_t sh_raw[];
    __shared__ ProdShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t stage0 = (smem_u32(sh_raw) + 1023u) & ~1023u;
    volatile int* failed = &sh.failed;

    if (tid == 0) {
        for (int i = 0; i < S::STAGES; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], 1);
        for (int i = 0; i < S::BUFS; ++i) mbar_init(&sh.sums[i], 2), mbar_init(&sh.taken[i], kProdSumWarps);
        sh.failed = 0;
        sh.loaded = sh.multiplied = 0;
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_x) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_w) : "memory");
    }
    if (warp == kProdSumWarps + 1) tmem_alloc(&sh.tmem, 512);
    pdl_launch_dependents();
    pdl_wait();
    // rows of each expert, within the rows whatever the offsets say.  (They are ascending.  Where they are not, an expert
    // that ends before it starts has no rows, and rows of two experts or of none behind the first hold anything.)
    if (p.offsets) {
        for (int e = tid; e <= p.E; e += kProdThreads) {
            const int64_t v = p.offsets[e];
            sh.first[e] = static_cast<int32_t>(v < 0 ? 0 : v > p.rows ? p.rows : v);
        }
    } else if (tid == 0) {
        sh.first[0] = 0;
        sh.first[1] = static_cast<int32_t>(p.rows);
    }
    __syncthreads();
    {
        int64_t mine[2], sum = 0;  // E <= 512: up to two experts to a thread
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = tid * 2 + i;
            const int n = e < p.E ? sh.first[e + 1] - sh.first[e] : 0;
            mine[i] = sum;
            sum += n > 0 ? (n + kProdRows - 1) / kProdRows : 0;
        }
        int64_t upto = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 31) sh.scan[warp] = upto;
        __syncthreads();
        int64_t before = upto - sum;
        for (int w = 0; w < warp; ++w) before += sh.scan[w];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (tid * 2 + i < p.E) sh.tiles[tid * 2 + i] = before + mine[i];
        if (tid == kProdThreads - 1) sh.tiles[p.E] = before + sum;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    uint32_t splits = 1, split = 0;
    if constexpr (SPLIT) {
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(splits));
        split = cluster_ctarank();
    }
    const int per = (p.blocks + static_cast<int>(splits) - 1) / static_cast<int>(splits);
    const int b0 = min(p.blocks, static_cast<int>(split) * per), b1 = min(p.blocks, b0 + per);
    // a cluster that splits tiles takes one; else tiles in turn
    const int64_t tile0 = blockIdx.x / splits, step = SPLIT ? (1LL << 40) : gridDim.x;

    if (warp >= kProdSumWarps) {
        fewer_registers<S::OTHER_REGISTERS>();
        if (warp == kProdSumWarps && lane == 0) {
            uint32_t n = 0;  // blocks loaded so far
            Tile t;
            bool ok = true;
            for (int64_t i = tile0; ok && tile_at<BN>(sh, p, i, t); i += step) {
                const int boxes = (t.rows + kProdBox - 1) / kProdBox;
                for (int b = b0; b < b1; ++b, ++n) {
                    const uint32_t s = n % S::STAGES;
                    if (!(ok = wait_phase(&sh.empty[s], (n / S::STAGES + 1) & 1, failed))) break;
                    const uint32_t a = stage0 + s * S::STAGE;
                    mbar_arrive_expect_tx(&sh.full[s], boxes * kProdBox * kProdBlock + S::B_BYTES);
                    tma_load_3d(a + S::A_BYTES, &map_w, b * kProdBlock, t.n0, t.e, &sh.full[s]);
                    for (int x = 0; x < boxes; ++x)
                        tma_load_2d(a + x * kProdBox * kProdBlock, &map_x, b * kProdBlock,
                                    static_cast<int>(t.row0) + x * kProdBox, &sh.full[s]);
                }
            }
            sh.loaded = n;
        } else if (warp == kProdSumWarps + 1 && lane == 0) {
            const int end = min(b1, b0 + p.give_up);
            uint32_t n = 0;
            Tile t;
            bool ok = true;
            for (int64_t i = tile0; ok && tile_at<BN>(sh, p, i, t); i += step) {
                for (int b = b0; b < end; ++b, ++n) {
                    const uint32_t s = n % S::STAGES, d = n % S::BUFS;
                    ok = wait_phase(&sh.taken[d], (n / S::BUFS + 1) & 1, failed) && wait_phase(&sh.full[s], (n / S::STAGES) & 1, failed);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = stage0 + s * S::STAGE;
                    const uint64_t da = operand_desc(a), db = operand_desc(a + S::A_BYTES);
#pragma unroll
                    for (int k = 0; k < kProdBlock / 32; ++k)  // 32 bytes along k: 2 in the descriptors' units
                        tc_mma_f8(tmem + d * BN, da + 2 * k, db + 2 * k, instruction_desc(BN), k > 0);
                    tc_commit(&sh.empty[s]);
                    tc_commit(&sh.sums[d]);
                }
                if (end < b1) *failed = 1, ok = false;
            }
            sh.multiplied = n;
        } else if (warp == kProdSumWarps + 2) {
            uint32_t n = 0;
            Tile t;
            bool ok = true;
            for (int64_t i = tile0; ok && tile_at<BN>(sh, p, i, t); i += step) {
                const float* xs[4];  // four rows to a lane; rows behind the tile's last take its first's
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = lane + 32 * j;
                    xs[j] = p.x_scales + (t.row0 + (r < t.rows ? r : 0)) * p.blocks;
                }
                const int nb = t.n0 / 128;
                const float* ws = p.w_scales + (static_cast<int64_t>(t.e) * p.n_blocks + nb) * p.blocks;
                const int64_t second = BN == 256 && nb + 1 < p.n_blocks ? p.blocks : 0;
                float x[4], w[2];
                const auto fetch = [&](int b) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = xs[j][b];
                    w[0] = ws[b];
                    w[1] = ws[b + second];
                };
                if (b0 < b1) fetch(b0);
                for (int b = b0; b < b1; ++b, ++n) {
                    const uint32_t d = n % S::BUFS;
                    ok = __all_sync(0xFFFFFFFFu, wait_phase(&sh.taken[d], (n / S::BUFS + 1) & 1, failed));
                    if (!ok) break;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sh.scale[d][0][lane + 32 * j] = x[j] * w[0];
                        sh.scale[d][1][lane + 32 * j] = x[j] * w[1];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.sums[d]);
                    if (b + 1 < b1) fetch(b + 1);
                }
            }
        }
        __syncwarp();
        more_registers<168>();
    } else {
        more_registers<S::SUM_REGISTERS>();
        const int quarter = warp & 3, side = warp >> 2;
        uint32_t n = 0;
        Tile t;
        bool ok = true;
        for (int64_t i = tile0; ok && tile_at<BN>(sh, p, i, t); i += step) {
            const int r = quarter * 32 + lane;             // the thread's row of the tile
            const bool some = quarter * 32 < t.rows;       // the warp has a row to add up
            Two acc[S::COLS / 2];
#pragma unroll
            for (int c = 0; c < S::COLS / 2; ++c) acc[c] = 0;
            const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + side * S::COLS;
            constexpr int PARTS = S::COLS / 32;
            for (int b = b0; b < b1; ++b, ++n) {
                const uint32_t d = n % S::BUFS;
                ok = __all_sync(0xFFFFFFFFu, wait_phase(&sh.sums[d], (n / S::BUFS) & 1, failed));
                if (!ok) break;
                tc_fence_after();
                if (some) {
                    const uint32_t f = __float_as_uint(sh.scale[d][side][r]);
                    const Two ff = two(f, f);
#pragma unroll
                    for (int c = 0; c < PARTS; ++c) {
                        uint32_t v[32];
                        tmem_load32(from + d * BN + c * 32, v);
                        tmem_wait_load(v);
                        if (c == PARTS - 1) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sh.taken[d]);
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) add_product(acc[c * 16 + j], two(v[2 * j], v[2 * j + 1]), ff);
                    }
                } else if (lane == 0) {
                    mbar_arrive(&sh.taken[d]);
                }
            }
            if (!ok) break;
            const auto sum = [&](int c) { return __uint_as_float(static_cast<uint32_t>(c & 1 ? acc[c / 2] >> 32 : acc[c / 2])); };
            if constexpr (SPLIT) {
                // sums to the stages' memory (all products have read it), rows 16 bytes apart in their banks
                if (some) {
                    const uint32_t at = stage0 + (r * (BN + 4) + side * S::COLS) * 4;
#pragma unroll
                    for (int c = 0; c < S::COLS / 4; ++c)
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + c * 16), "f"(sum(4 * c)),
                                     "f"(sum(4 * c + 1)), "f"(sum(4 * c + 2)), "f"(sum(4 * c + 3))
                                     : "memory");
                }
            } else if (S::OUT > 0 && p.bulk && quarter * 32 + 32 <= t.rows) {
                // the warp's 32 rows by way of its 8 KB, swizzled as the copies expect it: two boxes of 128 bytes a row
                // at a time, written while the next tile is multiplied (rows that another expert's follow within the
                // 32 go the other way)
                constexpr int BOX = 128 / static_cast<int>(sizeof(O));  // outputs of a row in a box
                const uint32_t base = stage0 + S::STAGES * S::STAGE + warp * S::OUT;
                const int c0 = t.n0 + side * S::COLS;
#pragma unroll
                for (int c = 0; c < S::COLS; c += 2 * BOX) {
                    if (lane == 0) stores_read();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {  // 16 bytes each
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if constexpr (sizeof(O) == 2) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(sum(c + i * 8 + 2 * j), sum(c + i * 8 + 2 * j + 1));
                                w[j] = *reinterpret_cast<const uint32_t*>(&h);
                            } else {
                                w[j] = __float_as_uint(sum(c + i * 4 + j));
                            }
                        }
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         base + (i / 8) * 4096 + lane * 128 + ((i % 8) ^ (lane & 7)) * 16),
                                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                     : "memory");
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        const int y = static_cast<int>(t.row0) + quarter * 32;
                        if (c0 + c < p.N) tma_store_2d(&map_out, base, (c0 + c) * static_cast<int>(sizeof(O)), y);
                        if (c0 + c + BOX < p.N) tma_store_2d(&map_out, base + 4096, (c0 + c + BOX) * static_cast<int>(sizeof(O)), y);
                        stores_commit();
                    }
                }
            } else if (r < t.rows) {
                const int c0 = t.n0 + side * S::COLS;
                O* out = static_cast<O*>(p.out) + (t.row0 + r) * p.N + c0;
                if (p.vec && c0 + S::COLS <= p.N) {
                    constexpr int W = 32 / static_cast<int>(sizeof(O));  // outputs to a store
#pragma unroll
                    for (int c = 0; c < S::COLS / W; ++c) {
                        uint32_t w[8];
                        if constexpr (sizeof(O) == 2) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(sum(c * 16 + 2 * j), sum(c * 16 + 2 * j + 1));
                                w[j] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(sum(c * 8 + j));
                        }
                        store32(out + c * W, w);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < S::COLS; ++c)
                        if (c0 + c < p.N) put_out(out + c, sum(c));
                }
            }
        }
        if (S::OUT > 0 && lane == 0) stores_done();
        __syncwarp();
        fewer_registers<168>();
    }

    if constexpr (SPLIT) {
        cluster_sync_all();
        Tile t;
        if (tile_at<BN>(sh, p, tile0, t)) {
            // the cluster's sums of the tile, four outputs at a time; each CTA takes a share of them
            const int units = t.rows * (BN / 4), share = (units + static_cast<int>(splits) - 1) / static_cast<int>(splits);
            const int end = min(units, share * (static_cast<int>(split) + 1));
            for (int u = share * static_cast<int>(split) + tid; u < end; u += kProdThreads) {
                const int r = u / (BN / 4), c = u % (BN / 4) * 4;
                float sum[4] = {};
                for (uint32_t s = 0; s < splits; ++s) {
                    uint32_t from;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(stage0 + (r * (BN + 4) + c) * 4), "r"(s));
                    const uint4 v = ld_cluster_v4(from);
                    sum[0] += __uint_as_float(v.x), sum[1] += __uint_as_float(v.y);
                    sum[2] += __uint_as_float(v.z), sum[3] += __uint_as_float(v.w);
                }
                O* out = static_cast<O*>(p.out) + (t.row0 + r) * p.N + t.n0 + c;
                if (p.vec && t.n0 + c + 4 <= p.N) {
                    if constexpr (sizeof(O) == 2) {
                        const __nv_bfloat162 a = __floats2bfloat162_rn(sum[0], sum[1]), b = __floats2bfloat162_rn(sum[2], sum[3]);
                        *reinterpret_cast<uint2*>(out) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
                    } else {
                        *reinterpret_cast<float4*>(out) = make_float4(sum[0], sum[1], sum[2], sum[3]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (t.n0 + c + j < p.N) put_out(out + j, sum[j]);
                }
            }
        }
        cluster_sync_all();  // no CTA leaves while its sums are read
    }
    // rows that belong to no expert: zeros
    {
        O* out = static_cast<O*>(p.out);
        const int64_t head = static_cast<int64_t>(sh.first[0]) * p.N, tail = static_cast<int64_t>(sh.first[p.E]) * p.N;
        const int64_t all = p.rows * p.N, at = static_cast<int64_t>(blockIdx.x) * kProdThreads + tid;
        const int64_t stride = static_cast<int64_t>(gridDim.x) * kProdThreads;
        for (int64_t j = at; j < head; j += stride) put_out(out + j, 0.f);
        for (int64_t j = tail + at; j < all; j += stride) put_out(out + j, 0.f);
    }
    tc_fence_before();
    if (__syncthreads_or(sh.failed)) {  // (who gave up has set it)
        if (tid == 0) await_started<S::STAGES>(sh);
        __syncthreads();
    }
    if (warp == kProdSumWarps + 1) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
    if (tid == 0 && sh.failed) atomicOr(p.status, kErrTimeout);
}

// ---------------------------------------------------------------- host --------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder of tensor maps, looked up once for the process.
static EncodeTiled encoder() {
    static std::atomic<EncodeTiled> found{nullptr};
    EncodeTiled f = found.load(std::memory_order_acquire);
    if (!f) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            return nullptr;
        f = reinterpret_cast<EncodeTiled>(p);
        found.store(f, std::memory_order_release);
    }
    return f;
}

// Bytes in rows of K, `box` rows of 128 bytes to a copy, 128-byte swizzle; what lies outside reads as zero.
static bool byte_map(CUtensorMap& map, const void* base, int dims, int64_t K, int64_t rows, int64_t matrices, int64_t stride,
                     int64_t matrix_stride, int box) {
    const EncodeTiled encode = encoder();
    if (!encode) return false;
    const cuuint64_t size[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(matrices)};
    const cuuint64_t pitch[2] = {static_cast<cuuint64_t>(stride), static_cast<cuuint64_t>(matrix_stride)};
    const cuuint32_t extent[3] = {kProdBlock, static_cast<cuuint32_t>(box), 1}, step[3] = {1, 1, 1};
    return encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(dims), const_cast<void*>(base), size, pitch,
                  extent, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, typename O, bool SPLIT>
static ds_status launch_product(const CUtensorMap& mx, const CUtensorMap& mw, const CUtensorMap& mo, const ProdParams& p,
                                int64_t ctas, int splits, cudaStream_t stream) {
    const auto kern = ds_expert_product_kernel<BN, O, SPLIT>;
    const size_t smem = ProdShape<BN>::SMEM;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return DS_ERR_CUDA;
    return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), kProdThreads, smem, splits, stream, mx, mw, mo, p);
}

// Outputs to a tile, 128 or 256: those whose rounds of tiles over the SMs take less.  A block of a tile takes 400
// or 510 ns where its operands come from L2 (8192 rows by 8192 x 8192: 688 and 461 us), or the time of its weights
// from DRAM, 16 or 32 KB at an SM's share of 45 bytes a ns, over the row tiles that share them.
static int product_outputs(int64_t rows, int64_t E, int64_t N, int sms) {
    const double used = static_cast<double>(rows < E ? rows : E);  // experts with a row, at most
    // half a tile more for each expert than its rows fill
    const double tall = std::max(used, static_cast<double>(rows) / kProdRows + 0.5 * used);
    double least = 0;
    int best = 128;
    for (int bn = 128; bn <= 256; bn *= 2) {
        const double rounds = std::ceil(tall * static_cast<double>((N + bn - 1) / bn) / sms);
        const double time = rounds * std::max(bn == 128 ? 400.0 : 510.0, bn * 128 / 45.0 * used / tall);
        if (bn == 128 || time < least) best = bn, least = time;
    }
    return best;
}

}  // namespace dsk

using namespace dsk;

static ds_status expert_product(int32_t give_up, const void* x, const float* x_scales, int64_t rows, int32_t K,
                                int64_t x_stride, const void* w, const float* w_scales, int32_t E, int32_t N,
                                int64_t w_row_stride, int64_t w_matrix_stride, const int32_t* offsets, int32_t dtype,
                                void* out, cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || rows < 0 || K < 1 || N < 1 || E < 1 || x_stride < K || w_row_stride < K ||
        w_matrix_stride < (E > 1 ? 1 : 0) || (!offsets && E != 1))
        return DS_ERR_INVALID_ARG;
    if (K % 16 != 0 || E > kProdMaxE || rows > (1LL << 30) || K > (1 << 24) || N > (1 << 24)) return DS_ERR_UNSUPPORTED;
    if (x_stride >= (1LL << 36) || w_row_stride >= (1LL << 36) || w_matrix_stride >= (1LL << 39)) return DS_ERR_UNSUPPORTED;
    if (rows == 0) return DS_OK;
    if (!x || !x_scales || !w || !w_scales || !out) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    const auto off_by = [](const void* q, int bytes) { return reinterpret_cast<uintptr_t>(q) % bytes != 0; };
    if (!aligned16(x) || !aligned16(w) || x_stride % 16 || w_row_stride % 16 || (E > 1 && w_matrix_stride % 16) ||
        off_by(x_scales, 4) || off_by(w_scales, 4) || off_by(offsets, 4) || off_by(out, es))
        return DS_ERR_ALIGNMENT;
    int dev = 0;
    DevInfo info;
    ProdParams p = {};
    p.give_up = give_up;
    if (cudaGetDevice(&dev) != cudaSuccess || !dev_info(dev, info) || !(p.status = status_word())) return DS_ERR_CUDA;
    p.x_scales = x_scales;
    p.w_scales = w_scales;
    p.offsets = offsets;
    p.out = out;
    p.rows = rows;
    p.K = K;
    p.blocks = (K + 127) / 128;
    p.N = N;
    p.n_blocks = (N + 127) / 128;
    p.E = E;
    p.vec = !off_by(out, 32) && static_cast<int64_t>(N) * es % 32 == 0;
    p.bulk = aligned16(out) && static_cast<int64_t>(N) * es % 16 == 0;
    const int bn = product_outputs(rows, E, N, info.sms);
    const bool wide = bn == 256;
    p.n_tiles = (N + bn - 1) / bn;
    const int64_t tall = rows / kProdRows + (rows < E ? rows : E);  // row tiles at most (one more for each expert's end)
    const int64_t tiles = tall * p.n_tiles;
    int splits = 1;
    if (!wide)
        while (splits < kProdMaxSplit && tiles * splits * 2 <= info.sms && p.blocks >= splits * 4) splits *= 2;
    CUtensorMap mx, mw, mo = {};
    if (!byte_map(mx, x, 2, K, rows, 1, x_stride, 0, kProdBox) ||
        !byte_map(mw, w, 3, K, N, E, w_row_stride, E > 1 ? w_matrix_stride : w_row_stride, bn))
        return DS_ERR_CUDA;
    if (wide && p.bulk && !byte_map(mo, out, 2, static_cast<int64_t>(N) * es, rows, 1, static_cast<int64_t>(N) * es, 0, 32))
        return DS_ERR_CUDA;
    const int64_t ctas = splits > 1 ? tiles * splits : tiles < info.sms ? tiles : info.sms;
    if (wide)
        return dtype == DS_BF16 ? launch_product<256, __nv_bfloat16, false>(mx, mw, mo, p, ctas, 1, stream)
                                : launch_product<256, float, false>(mx, mw, mo, p, ctas, 1, stream);
    if (splits > 1)
        return dtype == DS_BF16 ? launch_product<128, __nv_bfloat16, true>(mx, mw, mo, p, ctas, splits, stream)
                                : launch_product<128, float, true>(mx, mw, mo, p, ctas, splits, stream);
    return dtype == DS_BF16 ? launch_product<128, __nv_bfloat16, false>(mx, mw, mo, p, ctas, 1, stream)
                            : launch_product<128, float, false>(mx, mw, mo, p, ctas, 1, stream);
}

extern "C" {

ds_status ds_expert_product(const void* x, const float* x_scales, int64_t rows, int32_t K, int64_t x_stride, const void* w,
                            const float* w_scales, int32_t E, int32_t N, int64_t w_row_stride, int64_t w_matrix_stride,
                            const int32_t* offsets, int32_t dtype, void* out, cudaStream_t stream) {
    return expert_product(kNever, x, x_scales, rows, K, x_stride, w, w_scales, E, N, w_row_stride, w_matrix_stride, offsets,
                          dtype, out, stream);
}

ds_status ds_expert_product_probe(int32_t block, const void* x, const float* x_scales, int64_t rows, int32_t K,
                                  int64_t x_stride, const void* w, const float* w_scales, int32_t E, int32_t N,
                                  int64_t w_row_stride, int64_t w_matrix_stride, const int32_t* offsets, int32_t dtype,
                                  void* out, cudaStream_t stream) {
    if (block < 0) return DS_ERR_INVALID_ARG;
    return expert_product(block < kNever ? block : kNever, x, x_scales, rows, K, x_stride, w, w_scales, E, N, w_row_stride,
                          w_matrix_stride, offsets, dtype, out, stream);
}

}  // extern "C"
