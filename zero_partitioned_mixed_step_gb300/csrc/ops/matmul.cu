// The product of two 8-bit matrices with a scale for each block of 128.
//
//   out[i, j] (+)= sum_b sa[b, i] sb[b, j] (sum over k in block b of a[i, k] b[j, k])
//
// The scales change every 128 of k, so the tensor cores cannot keep one sum
// over k: each block's products go to tensor memory on their own (four
// tcgen05 products of 32 bytes of k), from where the epilogue warps take them
// into registers, acc = fma(part, sa * sb, acc).  Tensor memory holds two
// blocks' sums of 256 columns, so the products of one block run while the last
// one's are being scaled.
//
// A CTA (or a pair of them on neighbouring SMs, which share B) has
//   NH groups of four epilogue warps, each for 128 rows x 128 columns,
//   a warp one of whose threads issues the TMA copies into a ring of stages
//   (128 rows of A and NH * 128 of B over the pair, 128 bytes of k each),
//   a warp or two with a thread that issues the products, and
//   a warp that brings the scales.
// The CTAs are persistent and walk the tiles.  All waits are bounded: the
// role that gives up marks the workspace's error word, the others follow, the
// copies and products in flight are waited for (again bounded), tensor memory is
// freed and the parts of k that were left out are counted, so that the
// workspace's counters are zero again.
//
// What bounds it: latency, no unit (at 4096x4096x4096 the tensor pipe is 39 % busy,
// issue slots 44, FMA 24).  A block of 256x256x128 is 512 cycles of products and
// takes about 930: with two blocks in flight a block's sums pass through a commit
// (300 cycles), polls (150 each), loads and a release one after the other, and
// two epilogue warps to a scheduler do not cover that.  With a scale for each
// column of b (tensor 29 %, issue 41, FMA 32) each group of 32 columns is loaded,
// waited for and used in turn, four times a block.
//   8192x14336x4096 into bf16, a scale for a tile of b: 395 us, 2.43 PFLOP/s, at
//   2070 MHz; 422, 2.28, where varied operands bring the clock to the power
//   limit's 1.93 GHz
//   14336x4096x8192 added in fp32, a scale for each column: 551 us, 1.75
//   PFLOP/s, at 2070 MHz, and 561
// 1021x50257x769 into bf16, rows not on 16 bytes: 85 us; a tile has 7 blocks of
// k, and its output's way out, which nothing hides, is half of its time.
#include <cuda.h>

#include <atomic>
#include <cstdlib>
#include <type_traits>

#include "ops.cuh"
#include "tcgen05.cuh"

namespace zo {

constexpr int kHead = 4096;        // bytes of the workspace ahead of the partial sums
constexpr int kCounters = 256;     // offset of the tiles' counters (zero between calls)
constexpr int kPlanSms = 152;      // the rule for splitting k counts on a GB300's SMs
constexpr int kStage = 16 * 1024;  // bytes of one staging buffer of the output
// The scales come through a ring in shared memory, by a warp of their own, in
// groups of four blocks of k.  (Loads into the epilogue threads' registers two
// blocks ahead were waited for at every block: 1350 cycles a block.)
constexpr int kGroup = 4, kGroups = 3;

struct MatmulParams {
    const float *sa, *sb;
    void *out;
    int32_t *error;
    uint32_t *counters;
    float *parts;
    int64_t ldsa, ldsb, ldo;
    int32_t m, n, kb;           // rows, columns, blocks of k
    int32_t tiles_m, tiles_n, splits, units;
    int32_t out_type, add, tma_out;
    int32_t give_up;            // test setting: every second CTA starts as if a wait of its had run out
    uint32_t instr;
};

template <int CG, int NH, bool TILE_B>
struct Shape {
    // two groups leave no registers to spare: whole warpgroups, so that the
    // copying one can give some of its own (168 x 384 = 216 x 256 + 72 x 128)
    static constexpr int kThreads = NH == 1 ? 224 : 384;
    static constexpr int kTileM = 128 * CG, kTileN = 128 * NH;
    // Tensor-core products (and warps that issue them) for a block: one for
    // each group, so that one group's columns are ready while the other's are
    // being made, or one for all columns, which reads A from shared memory
    // once.  Where a block's scaling is short (a scale for the tile) the first
    // is faster, where it is long (one for each column) the second:
    // 8192x14336x4096 395 and 422 us, 14336x4096x8192 into fp32 598 and 565.
    static constexpr int kProducts = TILE_B ? NH : 1;
    static constexpr int kN = kTileN / kProducts;  // columns of a product
    static constexpr int kRowsB = kN / CG;         // of a product's rows of B, in one CTA
    static constexpr int kBytesA = 128 * 128, kBytesB = kProducts * kRowsB * 128;
    static constexpr int kStageBytes = kBytesA + kBytesB;
    static constexpr int kStages = (224 * 1024 - NH * 2 * kStage - 4096) / kStageBytes;
    static constexpr int kBufs = NH == 1 ? 4 : 2;               // sums of 128 x 128 for each group
    static constexpr int kColumns = 128 * NH * kBufs;           // of tensor memory: all of it
    static constexpr int kSmem = 1024 + kStages * kStageBytes + NH * 2 * kStage;
};

// Tile (and part of k) number u: groups of 8 row tiles, so that the tiles that
// run together share what they read in L2.
struct Unit {
    int m, n, kb0, kb1, tile, split;
};
__device__ __forceinline__ Unit unit_of(const MatmulParams &p, int u)
{
    Unit r;
    r.split = 0;
    r.tile = u;
    r.kb0 = 0;
    r.kb1 = p.kb;
    if (p.splits > 1) {  // (32 bits: kb < 2^24, splits <= 152; a 64-bit division takes 500 cycles)
        r.split = u % p.splits;
        r.tile = u / p.splits;
        r.kb0 = (int)((uint32_t)p.kb * (uint32_t)r.split / (uint32_t)p.splits);
        r.kb1 = (int)((uint32_t)p.kb * (uint32_t)(r.split + 1) / (uint32_t)p.splits);
    }
    constexpr int kRows = 8;
    const int per = kRows * p.tiles_n, g = r.tile / per, in = r.tile - g * per;
    const int rows = min(kRows, p.tiles_m - g * kRows);
    r.n = in / rows;
    r.m = g * kRows + in - r.n * rows;
    return r;
}

// Walks the blocks of k of a CTA's units, one after the other.
struct Walk {
    Unit w;
    int u, kb;
    bool more;
    __device__ __forceinline__ Walk(const MatmulParams &p, int first) : u(first), kb(0), more(first < p.units)
    {
        if (more) {
            w = unit_of(p, u);
            kb = w.kb0;
        }
    }
    __device__ __forceinline__ void next(const MatmulParams &p, int step)
    {
        if (++kb < w.kb1)
            return;
        u += step;
        if ((more = u < p.units)) {
            w = unit_of(p, u);
            kb = w.kb0;
        }
    }
};

// Writes 16 bytes of a row of a staging buffer (128 rows of 128 bytes, swizzled as the TMA reads them).
__device__ __forceinline__ void stage16(uint8_t *buf, int row, int piece, uint4 v)
{
    *reinterpret_cast<uint4 *>(buf + row * 128 + ((piece ^ (row & 7)) << 4)) = v;
}

template <class T>
__device__ __forceinline__ uint4 pack16(const float *acc);  // 16 bytes of T
template <>
__device__ __forceinline__ uint4 pack16<float>(const float *acc)
{
    return make_uint4(__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]),
                      __float_as_uint(acc[3]));
}
template <>
__device__ __forceinline__ uint4 pack16<bf16>(const float *acc)
{
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
template <>
__device__ __forceinline__ uint4 pack16<f16>(const float *acc)
{
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(acc[2 * i], acc[2 * i + 1]);
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// 128 rows x 128 columns of sums (a thread one row) to the output by TMA
// stores (or reductions), two staging buffers of 128 bytes a row at a time.
// `id`: the group's barrier, which its threads have passed since thread 0 saw
// the buffers' last stores done reading.
template <class T>
__device__ __forceinline__ void write_tma(const MatmulParams &p, const void *map, const float acc[128],
                                          uint8_t *stage, int id, int t, int m0, int n0)
{
    constexpr int kCols = 128 / (int)sizeof(T);  // columns of one staging buffer
    constexpr int kPiece = 16 / (int)sizeof(T);  // sums in 16 bytes
#pragma unroll
    for (int c = 0; c < 128 / kCols; c += 2) {
        if (c > 0) {
            if (t == 0)
                bulk_wait_read<0>();
            barrier_of(id, 128);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
            stage16(stage + (i >> 3) * kStage, t, i & 7, pack16<T>(acc + (c * 8 + i) * kPiece));
        fence_async_shared();
        barrier_of(id, 128);
        if (t == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int x = n0 + (c + i) * kCols;
                if (x < p.n && m0 < p.m) {
                    if (p.add)
                        tma_add(map, x, m0, smem_u32(stage + i * kStage));
                    else
                        tma_store(map, x, m0, smem_u32(stage + i * kStage));
                }
            }
            bulk_commit();
        }
    }
}

// The same for rows that no TMA store can write (their starts are not on
// 16-byte boundaries).  Each thread stages its row turned by the row's own
// distance from a boundary, so that the destination's 16-byte pieces lie whole
// in the staged words; the rows' ends leave element by element.  (Gathering
// the pieces from rows staged as they are took 8 two-byte reads for each:
// 1021x50257x769 109 us, 85 here, 82 without the ends; 50256 columns, by TMA,
// 58.  Words in an order that conflicted in the banks, and each row's distance
// formed anew: 100.)
template <class T>
__device__ __forceinline__ void write_turned(const MatmulParams &p, const float acc[128], uint8_t *stage, int id,
                                             int t, int m0, int n0)
{
    constexpr int kPiece = 16 / (int)sizeof(T);
    constexpr int kCols = 16 * kPiece;  // columns at a time: 64 words of a row
    uint32_t *words = reinterpret_cast<uint32_t *>(stage);
    // A row's 16 pieces change places by its number, so that 32 rows' same words
    // meet different banks: the turns of 8 (4) rows in a row are all different
    // where rows have an odd length, and these rows' order is what is left.
    auto shuffle = [](int row) { return sizeof(T) == 4 ? row >> 2 & 7 : (row >> 3 & 3) | (row & 1) << 2; };
    auto off_boundary = [&](const T *o) { return (int)(reinterpret_cast<uintptr_t>(o) / sizeof(T) % kPiece); };
    T *first = static_cast<T *>(p.out) + (int64_t)m0 * p.ldo + n0;
#pragma unroll
    for (int c = 0; c < 128; c += kCols, first += kCols) {
        if (c > 0)
            barrier_of(id, 128);  // the last readers are done
        uint32_t *mine = words + t * 64;
        const int mix = shuffle(t), turn = off_boundary(first + (int64_t)t * p.ldo);
        const int shift = sizeof(T) == 4 ? turn : turn >> 1;
        const bool odd = sizeof(T) == 2 && (turn & 1);
#pragma unroll
        for (int i = 0; i < 64; ++i) {
            const int w = (i + shift) & 63;
            uint32_t x;
            if constexpr (sizeof(T) == 4)
                x = __float_as_uint(acc[c + i]);
            else
                x = word_of<T>(odd ? acc[(2 * i + 127) & 127] : acc[2 * i], odd ? acc[2 * i] : acc[2 * i + 1]);
            mine[(((w >> 2) ^ mix) << 2) + (w & 3)] = x;
        }
        barrier_of(id, 128);
        // a thread reads every eighth row, whose turns are all the same
        const int lane = t & 15, row0 = t >> 4;
        T *to = first + (int64_t)row0 * p.ldo;
        const int at = off_boundary(to), begin = lane * kPiece - at;  // this thread's piece
        const int n = min(kCols, p.n - n0 - c), rows = n > 0 ? min(128, p.m - m0) : 0;
        const bool whole = begin >= 0 && begin + kPiece <= n;
        // one of the at most 2 (kPiece - 1) elements outside whole pieces
        const int head = min((kPiece - at) % kPiece, n), tail = head + (n - head) / kPiece * kPiece;
        const int k = lane < 8 ? lane : tail + lane - 8, place = (k + at) & (kCols - 1);
        const int word = place * (int)sizeof(T) >> 2;
        const bool edge = lane < 8 ? lane < head : k < n;
#pragma unroll 16
        for (int row = row0; row < rows; row += 8, to += 8 * p.ldo) {
            const uint32_t *from = words + row * 64;
            const int mixed = shuffle(row);
            if (whole)
                *reinterpret_cast<uint4 *>(to + begin) = *reinterpret_cast<const uint4 *>(from + ((lane ^ mixed) << 2));
            if (edge) {
                const uint32_t x = from[(((word >> 2) ^ mixed) << 2) + (word & 3)];
                if constexpr (sizeof(T) == 4)
                    to[k] = __uint_as_float(x);
                else
                    reinterpret_cast<uint16_t *>(to)[k] = (uint16_t)(x >> (16 * (place & 1)));
            }
        }
    }
}

// Sums added to old values that no TMA reduction can add (a half type, or rows
// as above): staged in fp32, so that the sum is rounded once.
template <class T>
__device__ __forceinline__ void write_add(const MatmulParams &p, const float acc[128], uint8_t *stage, int id, int t,
                                          int m0, int n0)
{
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint8_t *buf = stage + (c & 1) * kStage;
        if (c > 0)
            barrier_of(id, 128);  // its last readers are done
#pragma unroll
        for (int i = 0; i < 8; ++i)
            stage16(buf, t, i, pack16<float>(acc + (c * 8 + i) * 4));
        barrier_of(id, 128);
        const int col = n0 + c * 32 + (t & 31);
        if (col < p.n)
            for (int row = t >> 5; row < 128 && m0 + row < p.m; row += 4) {
                T *o = static_cast<T *>(p.out) + (int64_t)(m0 + row) * p.ldo + col;
                const float v = *reinterpret_cast<const float *>(
                    buf + row * 128 + ((((t & 31) >> 2) ^ (row & 7)) << 4) + (t & 3) * 4);
                *o = from_f32<T>(to_f32(*o) + v);
            }
    }
}

template <class T>
__device__ __forceinline__ void write_tile(const MatmulParams &p, const void *map, const float acc[128],
                                           uint8_t *stage, int id, int t, int m0, int n0)
{
    // a TMA store ends on a 16-byte boundary, which a row's end need not be
    const bool whole = n0 + 128 <= p.n || (int64_t)p.n * (int)sizeof(T) % 16 == 0;
    if (p.tma_out && whole)
        write_tma<T>(p, map, acc, stage, id, t, m0, n0);
    else if (p.add)
        write_add<T>(p, acc, stage, id, t, m0, n0);
    else
        write_turned<T>(p, acc, stage, id, t, m0, n0);
}

template <int CG, int NH, bool TILE_B>
__global__ void __launch_bounds__(Shape<CG, NH, TILE_B>::kThreads, 1)
    matmul_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ CUtensorMap map_out, const __grid_constant__ MatmulParams p)
{
    using S = Shape<CG, NH, TILE_B>;
    constexpr int kStages = S::kStages, P = S::kProducts;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages];
    __shared__ __align__(8) uint64_t sum_full[P][S::kBufs], sum_empty[P][S::kBufs], drain_bar[P];
    __shared__ __align__(8) uint64_t scale_full[kGroups], scale_empty[kGroups];
    __shared__ __align__(16) float scale_a[kGroups][kGroup][128];
    __shared__ __align__(16) float scale_b[kGroups][kGroup][TILE_B ? NH : NH * 128];
    __shared__ uint32_t tmem_sh;
    __shared__ int gave_up_sh, last_sh;
    volatile int *gave_up = &gave_up_sh;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *staging = smem + kStages * S::kStageBytes;
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = CG == 1 ? 0 : cluster_rank();

    if (threadIdx.x == 0) {
        gave_up_sh = p.give_up & (int)blockIdx.x & 1;
        for (int i = 0; i < kStages; ++i) {
            bar_init(smem_u32(&full_bar[i]), 1);
            bar_init(smem_u32(&empty_bar[i]), P);
        }
        for (int i = 0; i < S::kBufs; ++i)
            for (int h = 0; h < P; ++h) {
                bar_init(smem_u32(&sum_full[h][i]), 1);
                bar_init(smem_u32(&sum_empty[h][i]), 4 * CG * NH / P);
            }
        for (int i = 0; i < kGroups; ++i) {
            bar_init(smem_u32(&scale_full[i]), 1);
            bar_init(smem_u32(&scale_empty[i]), 4 * NH);
        }
        for (int h = 0; h < P; ++h)
            bar_init(smem_u32(&drain_bar[h]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4 * NH + 1)
        tmem_alloc<CG>(smem_u32(&tmem_sh), S::kColumns);
    fence_before();
    __syncthreads();
    if (CG == 2)
        cluster_sync();
    fence_after();
    const uint32_t tmem = tmem_sh;
    const int units = p.units, first = blockIdx.x / CG, step = gridDim.x / CG;

    if (warp >= 4 * NH) {
        if (NH == 2)
            registers_down<72>();
        if (warp == 4 * NH) {
        // ---------------------------------------------------------- copies
        if (elect_one()) {
            int st = 0, issued = 0;
            uint32_t phase = 1;  // an empty stage counts as released
            bool ok = true;
            for (int u = first; ok && u < units; u += step) {
                const Unit w = unit_of(p, u);
                const int row_a = w.m * S::kTileM + (int)rank * 128;
                const int row_b = w.n * S::kTileN + (int)rank * S::kRowsB;
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!(ok = bar_wait(smem_u32(&empty_bar[st]), phase, gave_up)))
                        break;
                    const uint32_t a = smem_u32(smem + st * S::kStageBytes), b = a + S::kBytesA;
                    uint32_t full = smem_u32(&full_bar[st]);
                    if (rank == 0)
                        bar_expect(full, CG * S::kStageBytes);
                    if (CG == 2)
                        full = map_to(full, 0);
                    tma_load<CG>(a, &map_a, kb * 128, row_a, full);
#pragma unroll
                    for (int h = 0; h < P; ++h)
                        tma_load<CG>(b + h * S::kRowsB * 128, &map_b, kb * 128, row_b + h * S::kN, full);
                    issued = issued < kStages ? issued + 1 : kStages;
                    if (++st == kStages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            // Copies in flight land before the CTA ends.  Those of a pair's second
            // CTA are counted in the first, which may not have asked for them all,
            // so it polls a barrier that nothing arrives at.
            if (!ok && rank != 0)
                for (int k = 0; k < kDrainLimit; ++k)
                    if (bar_try(smem_u32(&full_bar[0]), 0))
                        break;
            if (!ok && rank == 0)
                for (int i = 0; i < issued; ++i) {
                    if (--st < 0) {
                        st = kStages - 1;
                        phase ^= 1;
                    }
                    for (int k = 0; k < kDrainLimit; ++k)
                        if (bar_try(smem_u32(&full_bar[st]), phase ^ 1))
                            break;
                }
        }
        } else if (warp == 4 * NH + 1 || (P == 2 && warp == 4 * NH + 3)) {
        // ---------------------------------------------------------- products
        // A warp for each of the block's products: a poll of a barrier takes about
        // 150 cycles, and one thread's polls for two took 790 a block.
        const int h = warp == 4 * NH + 1 ? 0 : 1;
        if (rank == 0 && elect_one()) {
            const uint32_t instr = p.instr, sums = smem_u32(&sum_full[h][0]), frees = smem_u32(&sum_empty[h][0]);
            int st = 0, buf = 0;
            uint32_t phase = 0, free_phase = 1;
            bool ok = true;
            for (int u = first; ok && u < units; u += step) {
                const Unit w = unit_of(p, u);
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    const bool full = bar_test(smem_u32(&full_bar[st]), phase);
                    const bool free = bar_test(frees + buf * 8, free_phase);
                    ok = (full || bar_wait(smem_u32(&full_bar[st]), phase, gave_up)) &&
                         (free || bar_wait(frees + buf * 8, free_phase, gave_up));
                    if (!ok)
                        break;
                    fence_after();
                    const uint32_t a = smem_u32(smem + st * S::kStageBytes);
                    const uint64_t da = smem_desc(a), db = smem_desc(a + S::kBytesA + h * S::kRowsB * 128);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f8<CG>(tmem + buf * S::kTileN + h * S::kN, da + k * 2, db + k * 2, instr, k > 0);
                    mma_commit<CG>(sums + buf * 8);
                    mma_commit<CG>(smem_u32(&empty_bar[st]));
                    if (++st == kStages) {
                        st = 0;
                        phase ^= 1;
                    }
                    if (++buf == S::kBufs) {
                        buf = 0;
                        free_phase ^= 1;
                    }
                }
            }
            if (!ok) {  // products in flight end before tensor memory is freed
                mma_commit<CG>(smem_u32(&drain_bar[h]));
                for (int k = 0; k < kDrainLimit; ++k)
                    if (bar_try(smem_u32(&drain_bar[h]), 0))
                        break;
            }
        }
        } else if (warp == 4 * NH + 2) {
        // ---------------------------------------------------------- scales
        int slot = 0;
        uint32_t phase = 1;
        Walk k(p, first);
        while (k.more) {
            if (!bar_wait_warp(smem_u32(&scale_empty[slot]), phase, gave_up))
                break;
            for (int i = 0; i < kGroup && k.more; ++i, k.next(p, step)) {
                const float *sa = p.sa + k.kb * p.ldsa, *sb = p.sb + k.kb * p.ldsb;
                const int row = k.w.m * S::kTileM + (int)rank * 128 + lane;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    copy4(smem_u32(&scale_a[slot][i][j * 32 + lane]), row + j * 32 < p.m ? sa + row + j * 32 : p.sa,
                          row + j * 32 < p.m);
                if (TILE_B) {
                    const int col = k.w.n * NH + lane;
                    if (lane < NH)
                        copy4(smem_u32(&scale_b[slot][i][lane]), col * 128 < p.n ? sb + col : p.sb, col * 128 < p.n);
                } else {
                    const int col = k.w.n * S::kTileN + lane;
#pragma unroll
                    for (int j = 0; j < 4 * NH; ++j)
                        copy4(smem_u32(&scale_b[slot][i][j * 32 + lane]),
                              col + j * 32 < p.n ? sb + col + j * 32 : p.sb, col + j * 32 < p.n);
                }
            }
            copy_commit();
            copy_wait<0>();
            __syncwarp();
            if (lane == 0)
                bar_arrive(smem_u32(&scale_full[slot]));
            if (++slot == kGroups) {
                slot = 0;
                phase ^= 1;
            }
        }
        }
    } else {
        if (NH == 2)
            registers_up<216>();
        // ---------------------------------------------------------- scaled sums and output
        const int h = warp >> 2, quad = warp & 3, t = threadIdx.x & 127, id = 1 + h;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        uint8_t *stage = staging + h * 2 * kStage;
        const int product = P == 1 ? 0 : h;
        const uint32_t full = smem_u32(&sum_full[product][0]), scale_there = smem_u32(&scale_full[0]);
        const uint32_t scale_free = smem_u32(&scale_empty[0]);
        uint32_t free = smem_u32(&sum_empty[product][0]);
        if (CG == 2)
            free = map_to(free, 0);
        int buf = 0, slot = 0, in_group = 0;
        uint32_t phase = 0, scale_phase = 0;
        bool ok = true;
        int u = first;
        for (; u < units; u += step) {
            const Unit w = unit_of(p, u);
            const int m0 = w.m * S::kTileM + (int)rank * 128, n0 = w.n * S::kTileN + h * 128;
            const bool has_row = m0 + t < p.m;
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; ++i)
                acc[i] = 0.0f;
            // Per block: 4 x 32 columns through registers.  (Loading the next
            // block's first columns ahead of the loop's end keeps them in
            // registers over it, and the compiler copies them there.)
            auto column = [&](int c) { return lanes + (uint32_t)((buf * NH + h) * 128 + c * 32); };
            bool ready = false;
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                if (!ready)
                    ok = bar_wait_warp(full + buf * 8, phase, gave_up) &&
                         (in_group != 0 || bar_wait_warp(scale_there + slot * 8, scale_phase, gave_up));
                if (!ok)
                    break;
                fence_after();
                const float *sa_row = &scale_a[slot][in_group][t];
                const int next_buf = buf + 1 == S::kBufs ? 0 : buf + 1;
                const uint32_t next_phase = phase ^ (next_buf == 0);
                const int next_slot = slot + 1 == kGroups ? 0 : slot + 1;
                const uint32_t next_scale_phase = scale_phase ^ (next_slot == 0);
                const bool group_ends = in_group + 1 == kGroup;
                bool peek = false;
                auto release = [&] {  // every column is in registers
                    fence_before();
                    bar_arrive_lane0<CG>(free + buf * 8, lane);
                    peek = bar_test(full + next_buf * 8, next_phase) &&
                           (!group_ends || bar_test(scale_there + next_slot * 8, next_scale_phase));
                };
                if (TILE_B) {
                    // one scale for all: two register buffers of 32 columns
                    uint32_t r[2][32];
                    tmem_ld32(column(0), r[0]);
                    tmem_ld32(column(1), r[1]);
                    const float ab = *sa_row * scale_b[slot][in_group][h];
                    auto add = [&](int c) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            scale_add(acc[c * 32 + i], r[c & 1][i], ab);
                    };
                    tmem_wait();
                    add(0);
                    tmem_ld32(column(2), r[0]);
                    add(1);
                    tmem_ld32(column(3), r[1]);
                    tmem_wait();
                    release();
                    add(2);
                    add(3);
                } else {
                    // a scale for each column: the other buffer's registers hold
                    // 32 of them, loaded while the sums are on their way (read
                    // at their use, each load was waited for)
                    const float a = *sa_row;
                    const float4 *sb = reinterpret_cast<const float4 *>(&scale_b[slot][in_group][h * 128]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32];
                        tmem_ld32(column(c), r);
                        float4 s[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            s[i] = sb[c * 8 + i];
                        tmem_wait();
                        if (c == 3)
                            release();
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 lo = mul2(a, s[i].x, s[i].y), hi = mul2(a, s[i].z, s[i].w);
                            float *o = acc + c * 32 + i * 4;
                            scale_add(o[0], r[i * 4], lo.x);
                            scale_add(o[1], r[i * 4 + 1], lo.y);
                            scale_add(o[2], r[i * 4 + 2], hi.x);
                            scale_add(o[3], r[i * 4 + 3], hi.y);
                        }
                    }
                }
                ready = __all_sync(0xFFFFFFFFu, peek);
                if (group_ends) {
                    __syncwarp();
                    bar_arrive_lane0<1>(scale_free + slot * 8, lane);
                    slot = next_slot;
                    scale_phase = next_scale_phase;
                }
                in_group = group_ends ? 0 : in_group + 1;
                buf = next_buf;
                phase = next_phase;
            }
            if (t == 0)
                bulk_wait_read<0>();  // the staging buffers are free
            if (barrier_or(id, 128, !ok)) {
                ok = false;
                break;
            }
            if (p.splits > 1) {
                // this part's sums to the workspace; the tile's last part adds
                // all of them in ascending order
                float *mine = p.parts + ((int64_t)w.tile * p.splits + w.split) * (128 * 128) + t;
                if (has_row)
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        __stcg(mine + i * 128, acc[i]);
                __threadfence();
                barrier_of(id, 128);
                if (t == 0) {
                    last_sh = atomicAdd(p.counters + w.tile, 1u) == (uint32_t)p.splits - 1;
                    __threadfence();
                }
                barrier_of(id, 128);
                if (!last_sh)
                    continue;
                const float *all = p.parts + (int64_t)w.tile * p.splits * (128 * 128) + t;
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    acc[i] = 0.0f;
                if (has_row)
                    for (int s = 0; s < p.splits; ++s, all += 128 * 128)
#pragma unroll
                        for (int i = 0; i < 128; ++i)
                            acc[i] += __ldcg(all + i * 128);
                if (t == 0)
                    p.counters[w.tile] = 0;
            }
            if (p.out_type == ZERO_T_BF16)
                write_tile<bf16>(p, &map_out, acc, stage, id, t, m0, n0);
            else if (p.out_type == ZERO_T_F16)
                write_tile<f16>(p, &map_out, acc, stage, id, t, m0, n0);
            else
                write_tile<float>(p, &map_out, acc, stage, id, t, m0, n0);
        }
        if (t == 0) {
            bulk_wait_all();
            // parts left out count all the same: the tiles' counters come back to zero
            if (NH == 1 && !ok && p.splits > 1)  // (pairs do not split k)
                for (; u < units; u += step) {
                    uint32_t *count = p.counters + u / p.splits;
                    if (atomicAdd(count, 1u) == (uint32_t)p.splits - 1)
                        *count = 0;
                }
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (CG == 2)
        cluster_sync();
    fence_after();
    if (warp == 4 * NH + 1)
        tmem_free<CG>(tmem, S::kColumns);
    if (threadIdx.x == 0 && gave_up_sh)
        atomicExch(p.error, 1);
}

// ------------------------------------------------------------------ few rows
//
// Up to 64 rows of a (single tokens): the weights' bytes are what counts.  The
// roles of the operands change places, so that the 128 rows of a tensor-core
// product are 128 rows of b and its columns the TN = 16, 32 or 64 rows of a:
// a block's sums are TN columns of tensor memory (eight blocks of them in
// flight) and TN registers of a thread.  Two CTAs to an SM, and k split over
// the CTAs of a cluster so that they fill the GPU; the parts' sums meet in
// distributed shared memory.  16x4096x14336: 27.2 us with 128x128 tiles, 19.1
// with the roles exchanged and the parts' sums through global memory, 12.4 so
// (17.0, 3.5 TB/s, with the weights from DRAM).
template <int TN>
struct Few {
    static constexpr int kThreads = 224;
    static constexpr int kBytesB = 128 * 128, kStageBytes = kBytesB + TN * 128;
    static constexpr int kStages = 100 * 1024 / kStageBytes;
    static constexpr int kBufs = TN == 64 ? 4 : 8;
    static constexpr int kColumns = TN * kBufs;
    static constexpr int kSmem = 1024 + kStages * kStageBytes;
};

// One element of the output: x, or the old value and x.
__device__ __forceinline__ void put_one(const MatmulParams &p, int64_t at, float x)
{
    auto put = [&](auto *o) {
        using T = std::remove_reference_t<decltype(*o)>;
        *o = from_f32<T>(p.add ? to_f32(*o) + x : x);
    };
    if (p.out_type == ZERO_T_BF16)
        put(static_cast<bf16 *>(p.out) + at);
    else if (p.out_type == ZERO_T_F16)
        put(static_cast<f16 *>(p.out) + at);
    else
        put(static_cast<float *>(p.out) + at);
}

constexpr int kMaxSplits = 8;  // CTAs of a cluster

template <int TN, bool TILE_B>
__global__ void __launch_bounds__(Few<TN>::kThreads, 2)
    matmul_few_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ MatmulParams p)
{
    using S = Few<TN>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages];
    __shared__ __align__(8) uint64_t sum_full[S::kBufs], sum_empty[S::kBufs], drain_bar;
    __shared__ __align__(8) uint64_t scale_full[kGroups], scale_empty[kGroups];
    __shared__ __align__(16) float scale_a[kGroups][kGroup][TN], scale_b[kGroups][kGroup][TILE_B ? 1 : 128];
    __shared__ uint32_t tmem_sh;
    __shared__ int gave_up_sh;
    volatile int *gave_up = &gave_up_sh;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    float *part = reinterpret_cast<float *>(smem);  // over the stages, once they are done with
    static_assert(TN * 128 * 4 <= S::kStages * S::kStageBytes, "the sums fit the stages");
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        gave_up_sh = p.give_up & (int)blockIdx.x & 1;
        for (int i = 0; i < kStages; ++i) {
            bar_init(smem_u32(&full_bar[i]), 1);
            bar_init(smem_u32(&empty_bar[i]), 1);
        }
        for (int i = 0; i < S::kBufs; ++i) {
            bar_init(smem_u32(&sum_full[i]), 1);
            bar_init(smem_u32(&sum_empty[i]), 4);
        }
        for (int i = 0; i < kGroups; ++i) {
            bar_init(smem_u32(&scale_full[i]), 1);
            bar_init(smem_u32(&scale_empty[i]), 4);
        }
        bar_init(smem_u32(&drain_bar), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 5)
        tmem_alloc<1>(smem_u32(&tmem_sh), S::kColumns);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_sh;
    const int first = blockIdx.x, step = gridDim.x;  // unit_of: one row of tiles

    if (warp == 4) {
        // ---------------------------------------------------------- copies
        if (elect_one()) {
            int st = 0, issued = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (Walk k(p, first); k.more; k.next(p, step)) {
                if (!(ok = bar_wait(smem_u32(&empty_bar[st]), phase, gave_up)))
                    break;
                const uint32_t b = smem_u32(smem + st * S::kStageBytes), full = smem_u32(&full_bar[st]);
                bar_expect(full, S::kStageBytes);
                tma_load<1>(b, &map_b, k.kb * 128, k.w.n * 128, full);
                tma_load<1>(b + S::kBytesB, &map_a, k.kb * 128, 0, full);
                issued = issued < kStages ? issued + 1 : kStages;
                if (++st == kStages) {
                    st = 0;
                    phase ^= 1;
                }
            }
            if (!ok)  // copies in flight land before the CTA ends
                for (int i = 0; i < issued; ++i) {
                    if (--st < 0) {
                        st = kStages - 1;
                        phase ^= 1;
                    }
                    for (int q = 0; q < kDrainLimit; ++q)
                        if (bar_try(smem_u32(&full_bar[st]), phase ^ 1))
                            break;
                }
        }
    } else if (warp == 5) {
        // ---------------------------------------------------------- products
        if (elect_one()) {
            int st = 0, buf = 0;
            uint32_t phase = 0, free_phase = 1;
            bool ok = true;
            for (Walk k(p, first); k.more; k.next(p, step)) {
                const bool full = bar_test(smem_u32(&full_bar[st]), phase);
                const bool free = bar_test(smem_u32(&sum_empty[buf]), free_phase);
                ok = (full || bar_wait(smem_u32(&full_bar[st]), phase, gave_up)) &&
                     (free || bar_wait(smem_u32(&sum_empty[buf]), free_phase, gave_up));
                if (!ok)
                    break;
                fence_after();
                const uint32_t b = smem_u32(smem + st * S::kStageBytes);
                const uint64_t db = smem_desc(b), da = smem_desc(b + S::kBytesB);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_f8<1>(tmem + buf * TN, db + i * 2, da + i * 2, p.instr, i > 0);
                mma_commit<1>(smem_u32(&sum_full[buf]));
                mma_commit<1>(smem_u32(&empty_bar[st]));
                if (++st == kStages) {
                    st = 0;
                    phase ^= 1;
                }
                if (++buf == S::kBufs) {
                    buf = 0;
                    free_phase ^= 1;
                }
            }
            if (!ok) {  // products in flight end before tensor memory is freed
                mma_commit<1>(smem_u32(&drain_bar));
                for (int q = 0; q < kDrainLimit; ++q)
                    if (bar_try(smem_u32(&drain_bar), 0))
                        break;
            }
        }
    } else if (warp == 6) {
        // ---------------------------------------------------------- scales
        int slot = 0;
        uint32_t phase = 1;
        Walk k(p, first);
        while (k.more) {
            if (!bar_wait_warp(smem_u32(&scale_empty[slot]), phase, gave_up))
                break;
            for (int i = 0; i < kGroup && k.more; ++i, k.next(p, step)) {
                const float *sa = p.sa + k.kb * p.ldsa, *sb = p.sb + k.kb * p.ldsb;
                for (int j = lane; j < TN; j += 32)
                    copy4(smem_u32(&scale_a[slot][i][j]), j < p.m ? sa + j : p.sa, j < p.m);
                if (TILE_B) {
                    if (lane == 0)
                        copy4(smem_u32(&scale_b[slot][i][0]), sb + k.w.n, true);
                } else {
                    const int row = k.w.n * 128 + lane;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        copy4(smem_u32(&scale_b[slot][i][j * 32 + lane]), row + j * 32 < p.n ? sb + row + j * 32 : p.sb,
                              row + j * 32 < p.n);
                }
            }
            copy_commit();
            copy_wait<0>();
            __syncwarp();
            if (lane == 0)
                bar_arrive(smem_u32(&scale_full[slot]));
            if (++slot == kGroups) {
                slot = 0;
                phase ^= 1;
            }
        }
    } else {
        // ---------------------------------------------------------- scaled sums and output
        const int t = threadIdx.x;
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        int buf = 0, slot = 0, in_group = 0;
        uint32_t phase = 0, scale_phase = 0;
        bool ok = true;
        for (int u = first; u < p.units; u += step) {
            const Unit w = unit_of(p, u);
            const int row = w.n * 128 + t;  // of b, a column of the output
            float acc[TN];
#pragma unroll
            for (int i = 0; i < TN; ++i)
                acc[i] = 0.0f;
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                if (in_group == 0)
                    ok = bar_wait_warp(smem_u32(&scale_full[slot]), scale_phase, gave_up);
                ok = ok && bar_wait_warp(smem_u32(&sum_full[buf]), phase, gave_up);
                if (!ok)
                    break;
                fence_after();
                const float b = scale_b[slot][in_group][TILE_B ? 0 : t];
                const float4 *sa = reinterpret_cast<const float4 *>(scale_a[slot][in_group]);
                constexpr int kLoad = TN < 32 ? 16 : 32;
#pragma unroll
                for (int c = 0; c < TN; c += kLoad) {
                    uint32_t r[kLoad];
                    if (kLoad == 16)
                        tmem_ld16(lanes + (uint32_t)(buf * TN + c), r);
                    else
                        tmem_ld32(lanes + (uint32_t)(buf * TN + c), r);
                    tmem_wait();
                    if (c + kLoad == TN) {
                        fence_before();
                        bar_arrive_lane0<1>(smem_u32(&sum_empty[buf]), lane);
                    }
#pragma unroll
                    for (int i = 0; i < kLoad; i += 4) {
                        const float4 s = sa[(c + i) / 4];
                        const float2 lo = mul2(b, s.x, s.y), hi = mul2(b, s.z, s.w);
                        scale_add(acc[c + i], r[i], lo.x);
                        scale_add(acc[c + i + 1], r[i + 1], lo.y);
                        scale_add(acc[c + i + 2], r[i + 2], hi.x);
                        scale_add(acc[c + i + 3], r[i + 3], hi.y);
                    }
                }
                if (++in_group == kGroup) {
                    in_group = 0;
                    __syncwarp();
                    bar_arrive_lane0<1>(smem_u32(&scale_empty[slot]), lane);
                    if (++slot == kGroups) {
                        slot = 0;
                        scale_phase ^= 1;
                    }
                }
                if (++buf == S::kBufs) {
                    buf = 0;
                    phase ^= 1;
                }
            }
            if (barrier_or(1, 128, !ok)) {
                ok = false;
                break;
            }
            if (p.splits > 1) {  // the one unit of this CTA: its sums for the cluster
#pragma unroll
                for (int i = 0; i < TN; ++i)
                    if (i < p.m)
                        part[i * 128 + t] = acc[i];
            } else if (row < p.n) {
#pragma unroll
                for (int i = 0; i < TN; ++i)
                    if (i < p.m)
                        put_one(p, (int64_t)i * p.ldo + row, acc[i]);
            }
        }
    }
    if (p.splits > 1) {
        // the parts in ascending order, each CTA for every splits-th row of a
        __syncwarp();
        cluster_sync();
        const Unit w = unit_of(p, first);
        const int row = w.n * 128 + (int)threadIdx.x;
        if (threadIdx.x < 128 && row < p.n && !gave_up_sh)
            for (int i = w.split; i < p.m; i += p.splits) {
                const uint32_t at = smem_u32(part + i * 128 + threadIdx.x);
                float x[kMaxSplits];
#pragma unroll
                for (int s = 0; s < kMaxSplits; ++s)
                    x[s] = s < p.splits ? load_cluster(map_to(at, (uint32_t)s)) : 0.0f;
                float sum = 0.0f;
#pragma unroll
                for (int s = 0; s < kMaxSplits; ++s)
                    sum += x[s];
                put_one(p, (int64_t)i * p.ldo + row, sum);
            }
        __syncwarp();    // the lanes without a column come together with the others
        cluster_sync();  // nobody ends while its sums are being read
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 5)
        tmem_free<1>(tmem, S::kColumns);
    if (threadIdx.x == 0 && gave_up_sh)
        atomicExch(p.error, 1);
}

// ------------------------------------------------------------------ host

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// The driver's encoder of tensor maps (looked up once per process).
static EncodeTiled encoder()
{
    static std::atomic<void *> found{nullptr};
    void *f = found.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult how;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &how) !=
                cudaSuccess || how != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            return nullptr;
        }
        found.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// A map of a row-major matrix for boxes of box_rows rows of 128 bytes.
static int encode(CUtensorMap *map, CUtensorMapDataType type, int bytes, const void *base, int64_t rows,
                  int64_t cols, int64_t ld, int box_rows)
{
    const EncodeTiled f = encoder();
    if (!f)
        return cuda_error(cudaErrorSymbolNotFound);
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * (cuuint64_t)bytes};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / bytes), (cuuint32_t)box_rows};
    const cuuint32_t one[2] = {1, 1};
    const CUresult r = f(map, type, 2, const_cast<void *>(base), dims, strides, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ZERO_OK : ZERO_EINVAL;
}

// How a product is cut: up to 64 rows, tiles of 128 rows of b with all of a's;
// else pairs of CTAs on 256x256 tiles or single CTAs on 128x128 tiles, by the
// rounds that each takes on a GB300's SMs, a pair's as 3/2 of a single's (14.6
// and 9.6 us for 4096 of k).  Where the tiles are few, k is split so that the
// parts fill the SMs (two CTAs to an SM with few rows).  With k = 4096:
//   1024x4096    pairs, 1 round, 24.7 us    singles, 2 rounds, 27.5
//   2048x2560    pairs, 2 rounds, 39.2      singles, 3 rounds, 37.2
//   2048x5120    pairs, 3 rounds, 55.5      singles, 5 rounds, 59.6
//   128x50257    pairs, 3 rounds, 60.1      singles, 3 rounds, 46
//   64x4096      12.4 with few rows' tiles, 14.6 with 128x128; unsplit 18.6
//   512x1024x8192  18.6, unsplit 26.7;  16x4096x14336  16.7, unsplit 33.0
struct Plan {
    int few;  // columns of the few-rows kernel's tiles, or 0
    bool pair;
    int64_t tiles_m, tiles_n;
    int splits;
    int64_t part;  // elements of a part's sums in the workspace
};
static Plan plan_of(int64_t m, int64_t n, int64_t k)
{
    Plan r{};
    r.splits = 1;
    if (m == 0 || n == 0)  // nothing to cut
        return r;
    const int64_t kb = ceil_div(k, kBlock);
    const int64_t pair_waves = ceil_div(ceil_div(m, 256) * ceil_div(n, 256), kPlanSms / 2);
    const int64_t single_waves = ceil_div(ceil_div(m, 128) * ceil_div(n, 128), kPlanSms);
    if (m > 64 && 3 * pair_waves < 2 * single_waves) {
        r.pair = true;
        r.tiles_m = ceil_div(m, 256);
        r.tiles_n = ceil_div(n, 256);
        return r;
    }
    r.few = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 0;
    r.tiles_m = r.few ? 1 : ceil_div(m, 128);
    r.tiles_n = ceil_div(n, 128);
    r.part = r.few ? 0 : 128 * 128;
    const int64_t tiles = r.tiles_m * r.tiles_n;
    int64_t s = (r.few ? 2 : 1) * kPlanSms / tiles;
    if (s > kb / 4)  // a part is worth its sums' way to the others from four blocks on
        s = kb / 4;
    if (r.few && s > kMaxSplits)
        s = kMaxSplits;
    if (s > 1)
        r.splits = (int)s;
    return r;
}

// The operands as the tensor maps need them.
struct Operands {
    const void *a, *b;
    int64_t lda, ldb, k;
    int a_type, b_type;
};

// ZERO_TEST_MATMUL_GIVE_UP=1 in the environment (read once per process): in every
// second CTA a wait that is not over at its first poll ends as if its polls had
// run out.
static int test_give_up()
{
    static const int on = [] {
        const char *t = std::getenv("ZERO_TEST_MATMUL_GIVE_UP");
        return t && std::atoi(t) > 0 ? 1 : 0;
    }();
    return on;
}

// Lets a kernel use that much shared memory, once for each device (bits of `ready`).
static cudaError_t allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &ready)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (ready.load(std::memory_order_acquire) >> dev & 1)))
        return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64)
        ready.fetch_or(UINT64_C(1) << dev, std::memory_order_acq_rel);
    return e;
}

template <int CG, int NH, bool TILE_B>
static int launch_matmul(MatmulParams p, const Operands &o, cudaStream_t stream)
{
    using S = Shape<CG, NH, TILE_B>;
    auto kernel = matmul_kernel<CG, NH, TILE_B>;
    p.instr = f8_instr(o.a_type == ZERO_T_E5M2, o.b_type == ZERO_T_E5M2, S::kTileM, S::kN);
    CUtensorMap a, b, out{};
    int rc = encode(&a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, o.a, p.m, o.k, o.lda, 128);
    if (!rc)
        rc = encode(&b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, o.b, p.n, o.k, o.ldb, S::kRowsB);
    if (!rc && p.tma_out)
        rc = encode(&out, p.out_type == ZERO_T_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                          : p.out_type == ZERO_T_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                    type_bytes(p.out_type), p.out, p.m, p.n, p.ldo, 128);
    if (rc)
        return rc;
    static_assert(S::kSmem <= 227 * 1024 - 4096, "shared memory");
    static std::atomic<uint64_t> ready;
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), S::kSmem, ready);
    if (e != cudaSuccess)
        return cuda_error(e);
    const int64_t units = p.units;
    const int64_t most = device_sms() / CG;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((units < most ? units : most) * CG));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {CG, 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a, b, out, p);
    return e == cudaSuccess ? launch_status() : cuda_error(e);
}

template <int TN, bool TILE_B>
static int launch_few(MatmulParams p, const Operands &o, cudaStream_t stream)
{
    using S = Few<TN>;
    auto kernel = matmul_few_kernel<TN, TILE_B>;
    p.instr = f8_instr(o.b_type == ZERO_T_E5M2, o.a_type == ZERO_T_E5M2, 128, TN);
    CUtensorMap a, b;
    int rc = encode(&a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, o.a, p.m, o.k, o.lda, TN);
    if (!rc)
        rc = encode(&b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, o.b, p.n, o.k, o.ldb, 128);
    if (rc)
        return rc;
    static std::atomic<uint64_t> ready;
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), S::kSmem, ready);
    if (e != cudaSuccess)
        return cuda_error(e);
    const int most = 2 * device_sms();
    cudaLaunchConfig_t cfg{};
    // clusters hold one unit to a CTA; else the CTAs walk the units
    cfg.gridDim = dim3((unsigned)(p.splits > 1 || p.units < most ? p.units : most));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {(unsigned)p.splits, 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a, b, p);
    return e == cudaSuccess ? launch_status() : cuda_error(e);
}

template <bool TILE_B>
static int launch(const Plan &plan, const MatmulParams &p, const Operands &o, cudaStream_t stream)
{
    switch (plan.few) {
    case 16: return launch_few<16, TILE_B>(p, o, stream);
    case 32: return launch_few<32, TILE_B>(p, o, stream);
    case 64: return launch_few<64, TILE_B>(p, o, stream);
    default: break;
    }
    return plan.pair ? launch_matmul<2, 2, TILE_B>(p, o, stream) : launch_matmul<1, 1, TILE_B>(p, o, stream);
}

}  // namespace zo

using namespace zo;

extern "C" {

size_t zero_fp8_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k)
{
    if (bad_dim(m) || bad_dim(n) || bad_dim(k))
        return 0;
    const Plan plan = plan_of(m, n, k);
    return (size_t)kHead +
           (plan.splits > 1 ? (size_t)(plan.tiles_m * plan.tiles_n * plan.splits * plan.part) * sizeof(float) : 0);
}

int zero_fp8_matmul(const void *a, int a_type, int64_t lda, const float *sa, int64_t ldsa,
                    const void *b, int b_type, int64_t ldb, const float *sb, int64_t ldsb,
                    int b_tile, void *out, int out_type, int64_t ldo, int64_t m, int64_t n,
                    int64_t k, int add, void *ws, size_t ws_bytes, zero_stream_t stream)
{
    if (!is_fp8(a_type) || !is_fp8(b_type) || !is_float(out_type) || bad_dim(m) || bad_dim(n) ||
        bad_dim(k) || (b_tile != 0 && b_tile != 1) || !ws)
        return ZERO_EINVAL;
    if (m == 0 || n == 0)
        return ZERO_OK;
    const int ob = type_bytes(out_type);
    int rc = check_matrix(out, m, n, ldo, ob);
    if (!rc)
        rc = check_matrix(a, m, k, lda, 1);
    if (!rc)
        rc = check_matrix(b, n, k, ldb, 1);
    if (!rc)
        rc = check_matrix(sa, ceil_div(k, kBlock), m, ldsa, 4);
    if (!rc)
        rc = check_matrix(sb, ceil_div(k, kBlock), b_tile ? ceil_div(n, kBlock) : n, ldsb, 4);
    if (!rc && (!aligned(ws, 16) || (k > 0 && (!rows_aligned(a, lda, 1, 16) || !rows_aligned(b, ldb, 1, 16)))))
        rc = ZERO_EALIGN;
    if (!rc && ws_bytes < zero_fp8_matmul_workspace_bytes(m, n, k))
        rc = ZERO_ESPACE;
    if (rc)
        return rc;
    if (k == 0) {
        if (add)
            return ZERO_OK;
        const cudaError_t e = cudaMemset2DAsync(out, (size_t)(ldo * ob), 0, (size_t)(n * ob), (size_t)m, stream);
        return e == cudaSuccess ? ZERO_OK : cuda_error(e);
    }
    const Plan plan = plan_of(m, n, k);
    MatmulParams p{};
    p.sa = sa;
    p.sb = sb;
    p.out = out;
    p.error = static_cast<int32_t *>(ws);
    p.counters = reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + kCounters);
    p.parts = reinterpret_cast<float *>(static_cast<char *>(ws) + kHead);
    p.ldsa = ldsa;
    p.ldsb = ldsb;
    p.ldo = ldo;
    p.m = (int32_t)m;
    p.n = (int32_t)n;
    p.kb = (int32_t)ceil_div(k, kBlock);
    p.tiles_m = (int32_t)plan.tiles_m;
    p.tiles_n = (int32_t)plan.tiles_n;
    p.splits = plan.splits;
    const int64_t units = plan.tiles_m * plan.tiles_n * plan.splits;
    if (units > kMaxDim)
        return ZERO_EINVAL;
    p.units = (int32_t)units;
    p.out_type = out_type;
    p.add = add ? 1 : 0;
    p.give_up = test_give_up();
    // a TMA store (or reduction) of whole boxes; half types are added in fp32 and rounded once
    p.tma_out = rows_aligned(out, ldo, ob, 16) && (!add || out_type == ZERO_T_F32);
    const Operands o{a, b, lda, ldb, k, a_type, b_type};
    return b_tile ? launch<true>(plan, p, o, stream) : launch<false>(plan, p, o, stream);
}

}  // extern "C"
