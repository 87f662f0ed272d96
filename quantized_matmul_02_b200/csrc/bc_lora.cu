// bc_lora.cu -- low-rank adapters of many requests at once, added to a shared
// projection's output: for the rows of a segment whose adapter is a,
//
//   y[m] += c_a * B_a (A_a x[m]),   A_a [R][K], B_a [N][R], the first rank_a
//   ranks of R in use.
//
// Two launches for a whole set of projections.  Rows that share an adapter
// are cut into tiles.  shrink_kernel forms c A x, a block per (tile, 32 ranks of
// the projections that read the same x, part of K), and leaves it in scratch,
// in the order of expand_kernel's fragments.  expand_kernel joins the parts
// and adds B v, a block per (16 rows, columns).  x, A, B and v go from global
// memory to matrix fragments directly: the order of the contraction index is
// free, so a lane takes 16-byte pieces along it, and y's columns are dealt to
// the fragments so that lanes side by side hold whole sectors.
//
// What bounds it: the bytes of y (fp32, read and written) and x for prompts,
// the bytes of the adapters for single tokens.  2 R (K + N) operations a row
// are few beside them (16 per byte of y at R = 64), and tiles have 16 or 32
// rows, so the products run on mma.sync from registers.  Above R = 64 with
// many rows, B's trips from L2 (once per 16 rows) and the tensor cores bind.
//
// Measured, on the GPU alone: 4100 rows of bf16, 4096 -> 2 x 12288, rank 16:
// 163 us, 5.2 TB/s of the 847 MB that it must move.  The same with 2590 to 3860
// of the rows in use, "4100 rows" below: 136 us of 105 (one fused kernel of clusters
// that exchange v through distributed shared memory: 205 us; y read and written
// in half sectors: 201 us).  64 rows over some 33 adapters of ranks 8, 15 and 32,
// 4096 -> 4096 + 2 x 1024: 18 us of 3.9.  One row, 896 -> 896 + 2 x 128: 9 us.
//
// Precision: sums in fp32.  Products of 16-bit values are exact in the
// tensor cores (of one type, or in tf32, which holds bf16 and fp16 exactly).
// An fp32 x goes in as two tf32 pieces, 2^-22 of the value away; v as pieces of
// B's own type, so that B needs no conversion: three of bf16, 2^-25 away, or two of
// fp16, 2^-22 away but no nearer than 2^-39 of the row's largest (a rank whose v
// is below 2^-17 of that keeps fewer bits).  Sums run in a fixed order: results
// do not change from call to call, but a row's depend on how many rows share its
// adapter (kFew, tiles) and on the parts of K.
#include "bc_internal.cuh"

#include <mutex>
#include <type_traits>

namespace bc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kSms = 148;
constexpr int kMaxDescs = 16;          // per launch (kernel parameters)
constexpr int kMaxSegments = 4096;
constexpr int kMaxRank = 128;
constexpr int kGroupRows = 256;        // up to here rows are ordered by adapter
constexpr int kChunk = 32;             // ranks per shrink block
// Rows up to here: plain products instead of fragments (64 decode rows over 48
// adapters: 25 us with them, 31 without; 4 rows spill registers, 27).
constexpr int kFew = 2;
constexpr int kMaxSplit = 8;           // parts of K
constexpr int kStep = kWarps * 32;     // columns an expand block takes at a time
constexpr int kMaxSteps = 6;           // such steps per block (4100 rows: 6 135 us, 12 136, 16 142)
constexpr int kAhead = 2;              // 16-rank pieces of B on their way, for more than 16 ranks
constexpr int kStages = 3;             // of which y is on its way
constexpr int kRing = kWarps * kStages * 4 * 32;   // 16-byte pieces of y in shared memory

struct Desc {
    const void *x, *A, *B;
    float *y;
    int N, K;
    int group_size;                    // at a group's first projection: how many read its x
    int first_block, blocks;           // expand: this projection's column blocks
};
// A tile: `rows` rows of `adapter`.  Row i is first + i, or order[first + i].
struct __align__(16) Tile {
    int first, rows, adapter, rank;
    float scale;
};
struct LoraArgs {
    Desc d[kMaxDescs];
    const int32_t *seg_start;          // [S + 1]
    const int32_t *seg_adapter;        // [S]
    const int32_t *ranks;              // [adapters] or null
    const float *scaling;              // [adapters] or null
    int64_t M;
    int S, R, adapters, count;
    int T, max_tiles;
    int col_blocks, steps;             // column blocks of all projections, their steps
    int split;                         // parts of K
    int chunks;                        // 32-rank chunks of all groups
    int *head;                         // scratch: the rows' order (grouped)
    Tile *tiles;                       // scratch: [max_tiles], rows = 0 where unused
    float4 *v;                         // scratch: [count][split][max_tiles][MB][R16 / 16][2][32]
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// f = hi + lo + about 2^-22 |f|, both with a tf32's eleven significant bits.
__device__ __forceinline__ void split_tf32(float f, uint32_t &hi, uint32_t &lo) {
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(f));
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(f - __uint_as_float(hi)));
}
// Two values' leading piece in W's type, packed; the values lose it.
template <typename W>
__device__ __forceinline__ uint32_t take_piece(float &a, float &b) {
    if constexpr (std::is_same<W, __half>::value) {
        const __half2 h = __floats2half2_rn(a, b);
        const float2 f = __half22float2(h);
        a -= f.x;
        b -= f.y;
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        const uint32_t u = *reinterpret_cast<const uint32_t *>(&h);
        a -= __uint_as_float(u << 16);
        b -= __uint_as_float(u & 0xffff0000u);
        return u;
    }
}
// Pieces of an fp32 v in B's type: three of bf16 (2^-25 of the value away), two
// of fp16 (2^-22, after the row is scaled by a power of two).
template <typename W>
constexpr int kPieces = std::is_same<W, __half>::value ? 2 : 3;
// Two 16-bit values as fp32 bits.
template <typename W>
__device__ __forceinline__ void widen(uint32_t u, uint32_t &a, uint32_t &b) {
    if constexpr (std::is_same<W, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
        a = __float_as_uint(f.x);
        b = __float_as_uint(f.y);
    } else {
        a = u << 16;
        b = u & 0xffff0000u;
    }
}

// The tile table.  Few rows (decode): rows are ordered by adapter, so that
// requests of one adapter share its reads.  More rows: every segment is cut as
// it stands.  Each shrink block works it out for itself (1.5 us for 64 rows,
// most of it two dependent loads and a dozen barriers; a launch of its own
// would cost more) and keeps only its own tile; the first block of a tile
// leaves it for expand_kernel, block 0 the rows' order.
struct PlanShared {
    __align__(16) int key[kGroupRows];
    int order[kGroupRows], scan[kWarps + 1];
    Tile mine;
    int found;
};
__device__ __forceinline__ void segment(const LoraArgs &a, int i, int &s0, int &s1) {
    s0 = (int)min((int64_t)max(a.seg_start[i], 0), a.M);
    s1 = (int)min((int64_t)max(a.seg_start[i + 1], s0), a.M);
}
__device__ __forceinline__ bool usable(const LoraArgs &a, int ad) {
    return ad >= 0 && ad < a.adapters;
}
__device__ __forceinline__ Tile tile_of(const LoraArgs &a, int first, int rows, int ad) {
    return Tile{first, rows, ad, a.ranks ? min(max(a.ranks[ad], 0), a.R) : a.R, a.scaling ? a.scaling[ad] : 1.f};
}
template <int T>
__device__ __forceinline__ void plan(const LoraArgs &a, PlanShared &p, int want, bool publish) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) p.found = 0;
    if (a.M <= kGroupRows) {
        const int M = (int)a.M;
        constexpr int kNone = 0x7fffffff;
        p.key[tid] = kNone;
        __syncthreads();
        for (int i = tid; i < a.S; i += kThreads) {
            int s0, s1;
            const int ad = a.seg_adapter[i];
            segment(a, i, s0, s1);
            if (usable(a, ad))
                for (int m = s0; m < s1; ++m) p.key[m] = ad;
        }
        __syncthreads();
        // a row's place: how many keys come before it.  Threads lie idle where
        // rows are few, so up to eight of them share a row.
        const int share = M <= 32 ? 8 : M <= 64 ? 4 : M <= 128 ? 2 : 1;
        const int who = tid / share, mine = p.key[who];
        Tile t{};
        if (mine != kNone) t = tile_of(a, 0, 0, mine);       // (on its way while rows are counted)
        int before = 0, same = 0, all = 0;
        for (int j = tid % share * 4; j < M; j += share * 4) {       // places behind M hold kNone
            const int4 q = *reinterpret_cast<const int4 *>(p.key + j);
            const int k[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                before += k[e] < mine;
                same += k[e] == mine && j + e < who;
                all += k[e] == mine;
            }
        }
        for (int off = 1; off < share; off <<= 1) {
            before += __shfl_xor_sync(0xffffffffu, before, off);
            same += __shfl_xor_sync(0xffffffffu, same, off);
            all += __shfl_xor_sync(0xffffffffu, all, off);
        }
        before += same;
        const bool live = tid % share == 0 && who < M && mine != kNone, head = live && same % T == 0;
        __syncthreads();
        p.key[tid] = -1;
        __syncthreads();
        if (live) p.order[before] = who;
        if (head) p.key[before] = tid;           // at a tile's first place: the thread that knows it
        __syncthreads();
        // place of this thread's tile among the tiles, in sorted order
        const unsigned heads = __ballot_sync(0xffffffffu, p.key[tid] >= 0);
        if (lane == 0) p.scan[warp] = __popc(heads);
        __syncthreads();
        int base = 0;
        for (int w = 0; w < warp; ++w) base += p.scan[w];
        const int owner = p.key[tid];
        const int at = base + __popc(heads & ((1u << lane) - 1));
        __syncthreads();
        if (owner >= 0) p.key[owner] = at;       // the owner's tile number
        __syncthreads();
        if (head) {
            const int n = p.key[tid];
            if (n == want) {
                t.first = before;
                t.rows = min(T, all - same);
                p.mine = t;
                p.found = 1;
            }
        }
        if (publish) {
            if (tid < M) a.head[tid] = p.order[tid];
        }
        __syncthreads();
        return;
    }
    const int per = (a.S + kThreads - 1) / kThreads;
    const int i0 = min(a.S, tid * per), i1 = min(a.S, i0 + per);
    auto tiles_in = [&](int i, int &s0, int &s1) {
        const int ad = a.seg_adapter[i];
        segment(a, i, s0, s1);
        return usable(a, ad) ? (s1 - s0 + T - 1) / T : 0;
    };
    int own = 0, s0, s1;
    for (int i = i0; i < i1; ++i) own += tiles_in(i, s0, s1);
    int inc = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
    }
    if (lane == 31) p.scan[warp] = inc;
    __syncthreads();
    int at = inc - own;
    for (int w = 0; w < warp; ++w) at += p.scan[w];
    for (int i = i0; i < i1; ++i) {
        const int n = tiles_in(i, s0, s1);
        if (want >= at && want < at + n) {
            const int f = s0 + (want - at) * T;
            p.mine = tile_of(a, f, min(T, s1 - f), a.seg_adapter[i]);
            p.found = 1;
        }
        at += n;
    }
    __syncthreads();
}

// grid: tiles x rank chunks x parts of K
template <typename X, typename W, int MB>
__global__ void __launch_bounds__(kThreads, 2)
shrink_kernel(const __grid_constant__ LoraArgs a) {
    constexpr int T = 16 * MB, NB = kChunk / 8;
    constexpr bool kBf16 = std::is_same<X, __nv_bfloat16>::value && std::is_same<W, __nv_bfloat16>::value;
    constexpr bool kF32 = std::is_same<X, float>::value;
    constexpr int kQ = kF32 ? 2 : 1;                           // 16-byte pieces of a lane's eight x
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    __shared__ PlanShared ps;
    __shared__ __align__(16) float4 red[kWarps * T * kChunk / 4];
    const int per_tile = a.chunks * a.split;
    const int ti = blockIdx.x / per_tile, inner = blockIdx.x - ti * per_tile;
    const int part = inner % a.split;
    int chunk = inner / a.split;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    plan<T>(a, ps, ti, blockIdx.x == 0);
    const Tile tile = ps.found ? ps.mine : Tile{};
    if (inner == 0 && tid == 0) a.tiles[ti] = tile;
    if (!ps.found) return;
    // the chunk's projections: blocks of eight ranks of all that read one x, in a row
    const int R = a.R, R8 = R / 8, R16 = (R + 15) / 16 * 16, n_rows = tile.rows;
    int first = 0;
    while (chunk >= (a.d[first].group_size * R8 + NB - 1) / NB) {
        chunk -= (a.d[first].group_size * R8 + NB - 1) / NB;
        first += a.d[first].group_size;
    }
    const int K = a.d[first].K, blocks = a.d[first].group_size * R8;
    const int rank = tile.rank, used = (rank + 7) / 8;
    unsigned live = 0;                                         // blocks that have ranks
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int vb = chunk * NB + b;
        if (vb < blocks && vb % R8 < used) live |= 1u << b;
    }
    if (!live) return;
    // row g of block b of A, or null
    auto a_row = [&](int b, int g) -> const W * {
        const int vb = chunk * NB + b, r = vb % R8 * 8 + g;
        return (live >> b & 1) && r < rank
                   ? static_cast<const W *>(a.d[first + vb / R8].A) + ((int64_t)tile.adapter * R + r) * K : nullptr;
    };
    auto x_row = [&](int i) -> const X * {
        if (i >= n_rows) return nullptr;
        const int64_t m = a.M <= kGroupRows ? ps.order[tile.first + i] : tile.first + i;
        return static_cast<const X *>(a.d[first].x) + m * K;
    };
    constexpr int kQuads = T * kChunk / 4;
    if (MB == 1 && n_rows <= kFew) {
        // A row or two: plain products.  Warp w takes rank w of each block, its
        // lanes eight neighbouring k each, 256 a step; half the instructions
        // of the fragments, which would hold fourteen empty rows.
        const W *ar[NB];
        const X *xr[kFew];
#pragma unroll
        for (int b = 0; b < NB; ++b) ar[b] = a_row(b, warp);
#pragma unroll
        for (int i = 0; i < kFew; ++i) xr[i] = x_row(i);
        uint4 wa[2][NB], xa[2][kFew][kQ];
        auto load = [&](int k, uint4 (&wa)[NB], uint4 (&xa)[kFew][kQ]) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
                wa[b] = ar[b] && k < K ? *reinterpret_cast<const uint4 *>(ar[b] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < kFew; ++i)
#pragma unroll
                for (int q = 0; q < kQ; ++q)
                    xa[i][q] = xr[i] && k < K ? reinterpret_cast<const uint4 *>(xr[i] + k)[q] : make_uint4(0, 0, 0, 0);
        };
        float acc[kFew][NB] = {};
        auto multiply = [&](const uint4 (&wa)[NB], const uint4 (&xa)[kFew][kQ]) {
            float xf[kFew][8];
#pragma unroll
            for (int i = 0; i < kFew; ++i) {
                if (i >= n_rows) break;
                const uint4 p = xa[i][0], q = xa[i][kQ - 1];
                const uint32_t u[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (kF32) {
                        xf[i][e] = __uint_as_float(u[e]);
                        xf[i][e + 4] = __uint_as_float(u[e + 4]);
                    } else {
                        xf[i][2 * e] = __uint_as_float(u[e] << 16);
                        xf[i][2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (!(live >> b & 1)) continue;
                const uint32_t u[4] = {wa[b].x, wa[b].y, wa[b].z, wa[b].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t w0, w1;
                    widen<W>(u[e], w0, w1);
#pragma unroll
                    for (int i = 0; i < kFew; ++i)
                        if (i < n_rows)
                            acc[i][b] = fmaf(xf[i][2 * e + 1], __uint_as_float(w1),
                                             fmaf(xf[i][2 * e], __uint_as_float(w0), acc[i][b]));
                }
            }
        };
        const int step = a.split * 256;
        int k = part * 256 + lane * 8;
        load(k, wa[0], xa[0]);
        for (int k0 = part * 256; k0 < K; k0 += 2 * step, k += 2 * step) {
            load(k + step, wa[1], xa[1]);
            multiply(wa[0], xa[0]);
            load(k + 2 * step, wa[0], xa[0]);
            multiply(wa[1], xa[1]);
        }
#pragma unroll
        for (int i = 0; i < kFew; ++i)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float s = acc[i][b];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
                // its place among the fragments; rows that the tile lacks stay unset: no one reads them
                if (lane == 0) reinterpret_cast<float *>(red)[(b * 32 + i * 4 + warp / 2) * 4 + (warp & 1)] = s;
            }
    } else {
        // Rows and ranks that the tile lacks are taken from ones that it has:
        // they only reach sums that no one reads.
        const int nb = 32 - __clz(live);                       // (blocks below it may lack ranks)
        const W *arow[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int vb = chunk * NB + min(b, nb - 1);
            arow[b] = static_cast<const W *>(a.d[first + vb / R8].A) +
                      ((int64_t)tile.adapter * R + vb % R8 * 8 + g) * K + t * 8;
        }
        const X *xrow[MB][2];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int h = 0; h < 2; ++h) xrow[mb][h] = x_row(min(mb * 16 + g + h * 8, n_rows - 1)) + t * 8;
        float acc[MB][NB][4] = {};
        // The tensor cores cut off what lies below an accumulator's last bit, half
        // of it a product on average, so long sums are taken in parts: the warp's
        // own place in red[] holds them (fp32 x, K = 12288: y 3.0e-7 off, in one
        // sum 6.6e-7).
        bool parts = false;
        auto flush = [&] {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float4 &r = red[warp * (T * kChunk / 4) + (mb * NB + b) * 32 + lane];
                    const float4 s = parts ? r : make_float4(0.f, 0.f, 0.f, 0.f);
                    r = make_float4(s.x + acc[mb][b][0], s.y + acc[mb][b][1], s.z + acc[mb][b][2], s.w + acc[mb][b][3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[mb][b][e] = 0.f;
                }
            parts = true;
        };
        auto run = [&](auto blocks_c) {
            constexpr int L = decltype(blocks_c)::value;       // blocks of ranks
            auto load = [&](int u, uint4 (&wa)[L], uint4 (&xa)[MB][2][kQ]) {
#pragma unroll
                for (int b = 0; b < L; ++b) wa[b] = *reinterpret_cast<const uint4 *>(arow[b] + u * 32);
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int q = 0; q < kQ; ++q)
                            xa[mb][h][q] = reinterpret_cast<const uint4 *>(xrow[mb][h] + u * 32)[q];
            };
            auto multiply = [&](const uint4 (&wa)[L], const uint4 (&xa)[MB][2][kQ]) {
                if constexpr (kBf16) {
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const uint4 &p = xa[mb][0][0], &q = xa[mb][1][0];
                            const uint32_t f[4] = {s ? p.z : p.x, s ? q.z : q.x, s ? p.w : p.y, s ? q.w : q.y};
#pragma unroll
                            for (int b = 0; b < L; ++b)
                                mma_bf16(acc[mb][b], f, s ? wa[b].z : wa[b].x, s ? wa[b].w : wa[b].y);
                        }
                } else {
#pragma unroll
                    for (int s = 0; s < 4; ++s) {              // two of the lane's eight k each
                        uint32_t w0[L], w1[L];
#pragma unroll
                        for (int b = 0; b < L; ++b)
                            widen<W>(s == 0 ? wa[b].x : s == 1 ? wa[b].y : s == 2 ? wa[b].z : wa[b].w, w0[b], w1[b]);
#pragma unroll
                        for (int mb = 0; mb < MB; ++mb) {
                            uint32_t hi[4];
                            [[maybe_unused]] uint32_t lo[4];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if constexpr (kF32) {
                                    const uint4 &p = xa[mb][h][s >> 1];
                                    split_tf32(__uint_as_float(s & 1 ? p.z : p.x), hi[h], lo[h]);
                                    split_tf32(__uint_as_float(s & 1 ? p.w : p.y), hi[h + 2], lo[h + 2]);
                                } else {
                                    const uint4 &p = xa[mb][h][0];
                                    widen<__nv_bfloat16>(s == 0 ? p.x : s == 1 ? p.y : s == 2 ? p.z : p.w, hi[h], hi[h + 2]);
                                }
                            }
#pragma unroll
                            for (int b = 0; b < L; ++b) {
                                if constexpr (kF32) mma_tf32(acc[mb][b], lo[0], lo[1], lo[2], lo[3], w0[b], w1[b]);
                                mma_tf32(acc[mb][b], hi[0], hi[1], hi[2], hi[3], w0[b], w1[b]);
                            }
                        }
                    }
                }
            };
            // the next step's pieces are on their way while this one's are multiplied
            uint4 wa[2][L], xa[2][MB][2][kQ];
            const int step = a.split * kWarps, units = K / 32;
            int u = part * kWarps + warp;
            if (u < units) load(u, wa[0], xa[0]);
            for (int done = 0; u < units; u += 2 * step) {
                if (done == (kF32 ? 1 : kBf16 ? 4 : 2)) {      // after 16 products
                    flush();
                    done = 0;
                }
                ++done;
                if (u + step < units) load(u + step, wa[1], xa[1]);
                multiply(wa[0], xa[0]);
                if (u + step < units) {
                    if (u + 2 * step < units) load(u + 2 * step, wa[0], xa[0]);
                    multiply(wa[1], xa[1]);
                }
            }
        };
        static_assert(NB == 4, "one case per number of blocks");
        if (nb == 4) run(std::integral_constant<int, 4>());
        else if (nb == 3) run(std::integral_constant<int, 3>());
        else if (nb == 2) run(std::integral_constant<int, 2>());
        else run(std::integral_constant<int, 1>());
        // the block's sum over its warps, in fragment order
        flush();
        __syncthreads();
        for (int i = tid; i < kQuads; i += kThreads) {
            float4 s = red[i];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const float4 p = red[w * kQuads + i];
                s.x += p.x;
                s.y += p.y;
                s.z += p.z;
                s.w += p.w;
            }
            red[i] = s;
        }
    }
    // to scratch: ranks rb * 8 + 2 t and the next, of rows g and g + 8, are half
    // of a lane's four ranks there
    __syncthreads();
    for (int i = tid; i < kQuads; i += kThreads) {
        const int mb = i / 32 / NB, vb = chunk * NB + i / 32 % NB, rb = vb % R8;
        if (vb >= blocks || rb >= used || mb * 16 >= n_rows) continue;
        float4 s = red[i];
        const int l = i & 31, q = rb / 2, lq = (rb & 1) * 2 + (l & 3) / 2;
        const int64_t at = ((int64_t)(first + vb / R8) * a.split + part) * a.max_tiles + ti;
        float2 *out = reinterpret_cast<float2 *>(a.v + ((at * MB + mb) * (R16 / 16) + q) * 64 + (l >> 2) * 4 + lq) + (l & 1);
        // ranks behind the adapter's count as 0 (whatever A holds there)
        if (rb * 8 + (l & 3) * 2 >= rank) s.x = s.z = 0.f;
        if (rb * 8 + (l & 3) * 2 + 1 >= rank) s.y = s.w = 0.f;
        out[0] = make_float2(s.x * tile.scale, s.y * tile.scale);
        out[64] = make_float2(s.z * tile.scale, s.w * tile.scale);
    }
}

template <int BYTES, typename T>
__device__ __forceinline__ void copy(T *to, const float *from) {
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s), "l"(from) : "memory");
}

// VEC: y in 16-byte pieces.  AHEAD: pieces of 16 ranks of B that are loaded
// before the last ones are multiplied.
template <typename W, bool VEC, int AHEAD>
__device__ __forceinline__ void expand(const LoraArgs &a, const Desc &d, int di, int ti, int mb, int mbs,
                                       int cb, const Tile &tile) {
    extern __shared__ __align__(16) float4 smem[];
    constexpr int P = kPieces<W>;
    constexpr bool kHalf = std::is_same<W, __half>::value;
    uint4 *const vs = reinterpret_cast<uint4 *>(smem + kRing);  // v of the 16 rows: [R16 / 16][P][32] fragments
    __shared__ uint32_t top[16];                               // fp16: largest |v| of each row, as bits
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int N = d.N, R = a.R, R16 = (R + 15) / 16 * 16;
    float *yrow[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = mb * 16 + g + h * 8;
        yrow[h] = nullptr;
        if (i < tile.rows) {
            const int64_t m = a.M <= kGroupRows ? a.head[tile.first + i] : tile.first + i;
            yrow[h] = d.y + m * N;
        }
    }
    // a block's steps lie apart, so that blocks side by side run over
    // neighbouring columns: step s covers the warp's 32 columns from here
    auto column = [&](int s) { return ((s * d.blocks + cb) * kWarps + warp) * 32; };
    // Column 2 t + i of fragment block j, among the 32: with 16-byte accesses a
    // lane holds 4 neighbours twice, with 4-byte ones four lanes hold neighbours;
    // either way an access takes whole sectors or their halves.
    auto col = [&](int j, int t, int i) {
        return VEC ? (j >> 1) * 16 + t * 4 + (j & 1) * 2 + i : (j * 2 + i) * 4 + t;
    };
    // Each lane's own pieces of y are loaded two steps ahead; only their owner
    // touches them.
    auto piece = [&](int s, int h, int q) { return smem + ((warp * kStages + s % kStages) * 4 + h * 2 + q) * 32 + lane; };
    auto single = [&](int s, int h, int e) {
        return reinterpret_cast<float *>(smem + (warp * kStages + s % kStages) * 4 * 32) + (h * 8 + e) * 32 + lane;
    };
    auto prefetch = [&](int s) {
        const int n0 = column(s);
        if (s < a.steps) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!yrow[h]) continue;
                if constexpr (VEC) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (n0 + col(q * 2, t, 0) < N) copy<16>(piece(s, h, q), yrow[h] + n0 + col(q * 2, t, 0));
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (n0 + col(e >> 1, t, e & 1) < N)
                            copy<4>(single(s, h, e), yrow[h] + n0 + col(e >> 1, t, e & 1));
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    prefetch(0);
    prefetch(1);
    const int rank = tile.rank, used = (rank + 7) / 8 * 8;
    const W *B = static_cast<const W *>(d.B) + (int64_t)tile.adapter * R * N;
    const int64_t part = (int64_t)a.max_tiles * mbs * (R16 / 16) * 64;      // from one part of K to the next
    const float4 *v = a.v + di * a.split * part + ((int64_t)ti * mbs + mb) * (R16 / 16) * 64;
    uint2 ahead[AHEAD][4];
    auto fetch = [&](int s, int r0) {
        const int n0 = column(s), r = r0 + t * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + col(j, g >> 1, g & 1);
            const W *p = B + (int64_t)n * R + r;
            const bool in = s < a.steps && n < N;
#pragma unroll
            for (int c = 0; c < AHEAD; ++c)
                ahead[c][j] = in && r + c * 16 < rank ? *reinterpret_cast<const uint2 *>(p + c * 16) : make_uint2(0, 0);
        }
    };
    fetch(0, 0);
    constexpr int kMine = kMaxRank * 4 / kThreads;             // quads of ranks that a thread joins
    float4 mine[kMine];
    if (kHalf) {
        if (tid < 16) top[tid] = 0;
        __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < kMine; ++c) {
        const int i = c * kThreads + tid;                      // place (q, h, lane): row lane / 4 + 8 h, ranks q * 16 + ...
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < R16 * 4 && i / 64 * 16 + (i & 3) * 4 < used)   // (behind that, shrink leaves nothing)
            for (int s = 0; s < a.split; ++s) {
                const float4 w = v[s * part + i];
                f = make_float4(f.x + w.x, f.y + w.y, f.z + w.z, f.w + w.w);
            }
        mine[c] = f;
        if (kHalf && i < R16 * 4)
            atomicMax(&top[(i >> 2 & 7) + (i >> 5 & 1) * 8],
                      __float_as_uint(fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w)))));
    }
    // fp16 pieces are taken of v times 2^(141 - e), e the exponent bits of the
    // row's largest: that one lies in 2^14 .. 2^15, and a piece's least step,
    // 2^-24, is at most 2^-38 of it.
    auto exponent = [&](int row) { return max((int)(top[row] >> 23), 15); };
    if (kHalf) __syncthreads();
#pragma unroll
    for (int c = 0; c < kMine; ++c) {
        const int i = c * kThreads + tid;
        if (i >= R16 * 4) break;
        float4 f = mine[c];
        const int h = i >> 5 & 1, l = i & 31;
        if (kHalf) {
            const float scale = __uint_as_float((uint32_t)(141 + 127 - exponent((l >> 2) + h * 8)) << 23);
            f = make_float4(f.x * scale, f.y * scale, f.z * scale, f.w * scale);
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            uint32_t *to = reinterpret_cast<uint32_t *>(vs + (i / 64 * P + p) * 32 + l) + h;
            to[0] = take_piece<W>(f.x, f.y);
            to[2] = take_piece<W>(f.z, f.w);
        }
    }
    __syncthreads();
    float unscale[2] = {1.f, 1.f};
    if (kHalf) {
        unscale[0] = __uint_as_float((uint32_t)(exponent(g) - 141 + 127) << 23);
        unscale[1] = __uint_as_float((uint32_t)(exponent(g + 8) - 141 + 127) << 23);
    }
    for (int s = 0; s < a.steps; ++s) {
        const int n0 = column(s);
        if (n0 >= N) break;
        prefetch(s + 2);
        float acc[4][4] = {};                                  // [j][fragment]
        for (int r0 = 0; r0 < rank; r0 += 16 * AHEAD) {
            uint2 now[AHEAD][4];
#pragma unroll
            for (int c = 0; c < AHEAD; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) now[c][j] = ahead[c][j];
            if (r0 + 16 * AHEAD < rank) fetch(s, r0 + 16 * AHEAD);
            else fetch(s + 1, 0);
#pragma unroll
            for (int c = 0; c < AHEAD; ++c) {
                const int rc = r0 + c * 16, r = rc + t * 4;
                if (rc >= rank) break;
                if (rc + 16 > rank)                            // behind the adapter's rank: not its values
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        now[c][j].x &= r + 1 < rank ? 0xffffffffu : r < rank ? 0xffffu : 0u;
                        now[c][j].y &= r + 3 < rank ? 0xffffffffu : r + 2 < rank ? 0xffffu : 0u;
                    }
#pragma unroll
                for (int p = P - 1; p >= 0; --p) {
                    const uint4 q = vs[(rc / 16 * P + p) * 32 + lane];
                    const uint32_t f[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (kHalf) mma_f16(acc[j], f, now[c][j].x, now[c][j].y);
                        else mma_bf16(acc[j], f, now[c][j].x, now[c][j].y);
                    }
                }
            }
        }
        if (kHalf)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] *= unscale[e >> 1];
        asm volatile("cp.async.wait_group 2;" ::: "memory");
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!yrow[h]) continue;
            float *p = yrow[h] + n0;
            if constexpr (VEC) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int c = col(q * 2, t, 0);
                    if (n0 + c < N) {
                        float4 f = *piece(s, h, q);
                        f.x += acc[q * 2][h * 2];
                        f.y += acc[q * 2][h * 2 + 1];
                        f.z += acc[q * 2 + 1][h * 2];
                        f.w += acc[q * 2 + 1][h * 2 + 1];
                        *reinterpret_cast<float4 *>(p + c) = f;
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = col(e >> 1, t, e & 1);
                    if (n0 + c < N) p[c] = *single(s, h, e) + acc[e >> 1][h * 2 + (e & 1)];
                }
            }
        }
    }
}

// grid: tiles x blocks of 16 rows x column blocks of all projections
// (three blocks per SM: 4100 rows take 135 us, with two 152, with four 141)
template <typename W, int AHEAD>
__global__ void __launch_bounds__(kThreads, 3)
expand_kernel(const __grid_constant__ LoraArgs a) {
    const int mbs = a.T / 16;
    const int sub = blockIdx.x / a.col_blocks, cb = blockIdx.x - sub * a.col_blocks;
    const int ti = sub / mbs, mb = sub - ti * mbs;
    int di = 0;
    while (di + 1 < a.count && cb >= a.d[di + 1].first_block) ++di;
    const Desc &d = a.d[di];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Tile tile = a.tiles[ti];
    if (mb * 16 >= tile.rows || tile.rank == 0) return;
    if ((d.N & 3) == 0 && (reinterpret_cast<uintptr_t>(d.y) & 15) == 0)
        expand<W, true, AHEAD>(a, d, di, ti, mb, mbs, cb - d.first_block, tile);
    else
        expand<W, false, AHEAD>(a, d, di, ti, mb, mbs, cb - d.first_block, tile);
}

// Tile height: 16 rows while rows are few or segments short, else 32, which
// halves A's trips from L2; fp32 rows take 16 (two pieces of 32 rows would not
// fit the registers: 187 for a thread).
int tile_rows(int64_t M, int64_t S, bool f32) { return f32 || M <= kGroupRows || M / S <= 16 ? 16 : 32; }
// At most this many tiles: full ones, and a ragged one per segment (or adapter).
int64_t most_tiles(int64_t M, int64_t S, int64_t adapters, int64_t T) {
    const int64_t ragged = M <= kGroupRows && adapters < S ? adapters : S;
    return M / T + (ragged < M ? ragged : M);
}
// Steps of an expand block: one while that does not fill the GPU, more to
// share a block's start among its columns.
int steps_of(const bc_lora_desc *descs, int count, int64_t row_tiles) {
    int64_t all = 0;
    for (int i = 0; i < count; ++i) all += (descs[i].N + kStep - 1) / kStep;
    const int64_t s = all * row_tiles / (4 * kSms);
    return (int)(s < 1 ? 1 : s > kMaxSteps ? kMaxSteps : s);
}
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// 32-rank chunks of a launch (neighbours that read the same x share a pass
// over it), and the parts of K: about two blocks per SM, each with 1024 of K
// or more (64 decode rows at K = 4096: 21 us; three blocks per SM 25).
struct Shape {
    int64_t T, tiles;
    int chunks, split;
};
Shape shape_of(const bc_lora_desc *d, int count, int64_t M, int64_t R, int64_t adapters, int64_t S, bool f32) {
    Shape s;
    s.T = tile_rows(M, S, f32);
    s.tiles = most_tiles(M, S, adapters, s.T);
    s.chunks = 0;
    int64_t K = 0;
    for (int j = 0, n; j < count; j += n) {
        for (n = 1; j + n < count && d[j + n].x == d[j].x && d[j + n].K == d[j].K;) ++n;
        s.chunks += (int)((n * R + kChunk - 1) / kChunk);
        K = d[j].K > K ? d[j].K : K;
    }
    s.split = 1;
    while (s.split < kMaxSplit && s.tiles * s.chunks * s.split < 2 * kSms && K / s.split >= 1024) s.split *= 2;
    return s;
}
// Scratch of one launch.
size_t scratch(const Shape &s, int count, int64_t R) {
    return round256((size_t)kGroupRows * 4) + round256((size_t)s.tiles * sizeof(Tile)) +
           (size_t)count * s.split * s.tiles * s.T * ((R + 15) / 16 * 16) * 4;
}

// Lets the kernel have the shared memory of its largest rank (once per device).
template <auto kKernel>
bool allow_smem() {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev])
        done[dev] = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (kRing + kMaxRank / 16 * 3 * 32) * (int)sizeof(float4)) == cudaSuccess;
    return done[dev];
}

template <typename X, typename W, int MB>
bc_status launch(const LoraArgs &a, cudaStream_t s) {
    // 32 ranks of B ahead where there are more than 16 (777 rows, rank 128: 19.5 us, with 16 23)
    const auto expand = a.R <= 16 ? expand_kernel<W, 1> : expand_kernel<W, kAhead>;
    if (!(a.R <= 16 ? allow_smem<expand_kernel<W, 1>>() : allow_smem<expand_kernel<W, kAhead>>())) return BC_ERR_CUDA;
    shrink_kernel<X, W, MB><<<(unsigned)(a.max_tiles * a.chunks * a.split), kThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) {
        // expand's blocks may start while shrink's finish; they wait for all of it before they read
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(a.max_tiles * MB * a.col_blocks));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = (kRing + (a.R + 15) / 16 * kPieces<W> * 32) * sizeof(float4);
        cfg.stream = s;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, expand, a);
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return BC_ERR_CUDA;
    }
    return BC_OK;
}

template <typename X, typename W>
bc_status launch(const LoraArgs &a, cudaStream_t s) {
    if constexpr (!std::is_same<X, float>::value)
        if (a.T == 32) return launch<X, W, 2>(a, s);
    return launch<X, W, 1>(a, s);
}

bool overlap(const void *p, size_t pn, const void *q, size_t qn) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + qn && b < a + pn;
}

bool sizes_ok(const bc_lora_desc *descs, int count, int64_t M, int64_t R, int64_t n_adapters,
              int64_t n_segments, bc_status *st) {
    *st = BC_ERR_INVALID_ARG;
    if (!descs || count <= 0 || M <= 0 || n_segments <= 0 || n_adapters <= 0 || R <= 0 || R % 8) return false;
    for (int i = 0; i < count; ++i)
        if (descs[i].N <= 0 || descs[i].K <= 0 || descs[i].K % 64) return false;
    *st = BC_ERR_UNSUPPORTED;
    if (M > (int64_t)1 << 24 || n_segments > kMaxSegments || n_adapters > 1 << 20 || R > kMaxRank) return false;
    const int64_t tiles = most_tiles(M, n_segments, n_adapters, 16);       // the most there can be
    for (int i = 0; i < count; i += kMaxDescs) {
        const int n = count - i < kMaxDescs ? count - i : kMaxDescs;
        int64_t cols = 0;
        for (int j = 0; j < n; ++j) {
            if (descs[i + j].N >= (int64_t)1 << 30 || descs[i + j].K >= (int64_t)1 << 24) return false;
            cols += (descs[i + j].N + kStep - 1) / kStep;
        }
        // blocks of one launch
        if (2 * tiles * cols >= (int64_t)1 << 31) return false;        // (32-row tiles round up twice)
        if (tiles * n * ((R + kChunk - 1) / kChunk) * kMaxSplit >= (int64_t)1 << 31) return false;
    }
    *st = BC_OK;
    return true;
}

}  // namespace
}  // namespace bc

using namespace bc;

extern "C" {

size_t bc_workspace_size_lora(const bc_lora_desc *descs, int count, int64_t M, int64_t R,
                              int64_t n_adapters, int64_t n_segments, bc_dtype x_dtype) {
    bc_status st;
    if (!sizes_ok(descs, count, M, R, n_adapters, n_segments, &st)) return 0;
    size_t most = 0;
    for (int i = 0; i < count; i += kMaxDescs) {           // launches of a call use the scratch in turn
        const int n = count - i < kMaxDescs ? count - i : kMaxDescs;
        const size_t b = scratch(shape_of(descs + i, n, M, R, n_adapters, n_segments, x_dtype == BC_F32), n, R);
        most = b > most ? b : most;
    }
    return most;
}

bc_status bc_lora_add_batched(const bc_lora_desc *descs, int count, int64_t M, int64_t R,
                              int64_t n_adapters, bc_dtype x_dtype, bc_dtype w_dtype,
                              const int32_t *seg_start, const int32_t *seg_adapter,
                              int64_t n_segments, const int32_t *ranks, const float *scaling,
                              void *workspace, size_t workspace_bytes, bc_stream_t stream) {
    if (!seg_start || !seg_adapter) return BC_ERR_INVALID_ARG;
    bc_status st;
    if (!sizes_ok(descs, count, M, R, n_adapters, n_segments, &st)) return st;
    if ((x_dtype != BC_F32 && x_dtype != BC_BF16) || (w_dtype != BC_F16 && w_dtype != BC_BF16))
        return BC_ERR_UNSUPPORTED;
    if (!aligned(seg_start, 4) || !aligned(seg_adapter, 4) || !aligned(ranks, 4) || !aligned(scaling, 4))
        return BC_ERR_ALIGNMENT;
    const size_t need = bc_workspace_size_lora(descs, count, M, R, n_adapters, n_segments, x_dtype);
    for (int i = 0; i < count; ++i) {
        const bc_lora_desc &d = descs[i];
        if (!d.x || !d.A || !d.B || !d.y) return BC_ERR_INVALID_ARG;
        if (!aligned(d.x, 16) || !aligned(d.A, 16) || !aligned(d.B, 16) || !aligned(d.y, 4))
            return BC_ERR_ALIGNMENT;
        const size_t yb = (size_t)M * d.N * 4, ab = (size_t)n_adapters * R * 2;
        for (int j = 0; j < count; ++j) {
            const bc_lora_desc &e = descs[j];
            if ((j != i && overlap(d.y, yb, e.y, (size_t)M * e.N * 4)) ||
                overlap(d.y, yb, e.x, (size_t)M * e.K * (x_dtype == BC_F32 ? 4 : 2)) ||
                overlap(d.y, yb, e.A, ab * e.K) || overlap(d.y, yb, e.B, ab * e.N))
                return BC_ERR_INVALID_ARG;
        }
        if (overlap(d.y, yb, seg_start, 4 * (n_segments + 1)) || overlap(d.y, yb, seg_adapter, 4 * n_segments) ||
            overlap(d.y, yb, ranks, 4 * n_adapters) || overlap(d.y, yb, scaling, 4 * n_adapters) ||
            overlap(d.y, yb, workspace, need))
            return BC_ERR_INVALID_ARG;
        if (overlap(workspace, need, d.x, (size_t)M * d.K * (x_dtype == BC_F32 ? 4 : 2)) ||
            overlap(workspace, need, d.A, ab * d.K) || overlap(workspace, need, d.B, ab * d.N))
            return BC_ERR_INVALID_ARG;
    }
    if (overlap(workspace, need, seg_start, 4 * (n_segments + 1)) ||
        overlap(workspace, need, seg_adapter, 4 * n_segments) || overlap(workspace, need, ranks, 4 * n_adapters) ||
        overlap(workspace, need, scaling, 4 * n_adapters))
        return BC_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < need) return BC_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return BC_ERR_ALIGNMENT;
    LoraArgs a;
    a.seg_start = seg_start;
    a.seg_adapter = seg_adapter;
    a.ranks = ranks;
    a.scaling = scaling;
    a.M = M;
    a.S = (int)n_segments;
    a.R = (int)R;
    a.adapters = (int)n_adapters;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.head = reinterpret_cast<int *>(ws);
    ws += round256((size_t)kGroupRows * 4);
    a.tiles = reinterpret_cast<Tile *>(ws);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (int i = 0; i < count; i += kMaxDescs) {
        a.count = count - i < kMaxDescs ? count - i : kMaxDescs;
        const Shape sh = shape_of(descs + i, a.count, M, R, n_adapters, n_segments, x_dtype == BC_F32);
        a.T = (int)sh.T;
        a.max_tiles = (int)sh.tiles;
        a.chunks = sh.chunks;
        a.split = sh.split;
        a.v = reinterpret_cast<float4 *>(ws + round256((size_t)a.max_tiles * sizeof(Tile)));
        a.col_blocks = 0;
        a.steps = steps_of(descs + i, a.count, sh.tiles * sh.T / 16);
        for (int j = 0; j < a.count; ++j) {
            const bc_lora_desc &d = descs[i + j];
            const int blocks = (int)((d.N + kStep * a.steps - 1) / (kStep * a.steps));
            a.d[j] = Desc{d.x, d.A, d.B, d.y, (int)d.N, (int)d.K, 0, a.col_blocks, blocks};
            a.col_blocks += blocks;
        }
        for (int j = 0, n; j < a.count; j += n) {
            for (n = 1; j + n < a.count && a.d[j + n].x == a.d[j].x && a.d[j + n].K == a.d[j].K;) ++n;
            a.d[j].group_size = n;
        }
        if (x_dtype == BC_F32)
            st = w_dtype == BC_F16 ? launch<float, __half>(a, s) : launch<float, __nv_bfloat16>(a, s);
        else
            st = w_dtype == BC_F16 ? launch<__nv_bfloat16, __half>(a, s)
                                   : launch<__nv_bfloat16, __nv_bfloat16>(a, s);
        if (st != BC_OK) return st;
    }
    return BC_OK;
}

bc_status bc_lora_add(const void *x, bc_dtype x_dtype, const void *A, const void *B,
                      bc_dtype w_dtype, int64_t M, int64_t N, int64_t K, int64_t R,
                      int64_t n_adapters, const int32_t *seg_start, const int32_t *seg_adapter,
                      int64_t n_segments, const int32_t *ranks, const float *scaling, float *y,
                      void *workspace, size_t workspace_bytes, bc_stream_t stream) {
    const bc_lora_desc d{x, A, B, y, N, K};
    return bc_lora_add_batched(&d, 1, M, R, n_adapters, x_dtype, w_dtype, seg_start, seg_adapter,
                               n_segments, ranks, scaling, workspace, workspace_bytes, stream);
}

}  // extern "C"
