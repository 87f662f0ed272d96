// bc_lora.cu -- low-rank adapters of many requests at once, added to a shared
// projection's output: for the rows of a segment whose adapter is a,
//
//   y[m] += c_a * B_a (A_a x[m]),   A_a [R][K], B_a [N][R], the first rank_a
//   ranks of R in use.
//
// Two launches for a whole set of projections.  Rows that share an adapter
// are cut into tiles.  shrink_kernel forms v = A x, a block per (tile,
// projection, 32 ranks, part of K), and leaves its partial sums in scratch;
// expand_kernel joins the parts and adds B v, a block per (tile, projection,
// range of columns).  x, A, B and y go between global memory and matrix
// fragments directly: the order of the contraction index is free, so a lane
// takes 16-byte pieces along it, and y's columns are dealt to the fragments
// so that a lane holds eight neighbours.
//
// What bounds it: the bytes of y (fp32, read and written) and x for prompts,
// the bytes of the adapters for single tokens; 2 R (K + N) operations a row
// are small beside them up to R = 128.
//
// Precision: fp32 throughout.  Products of 16-bit values are exact in the
// tensor cores (bf16 with bf16, or tf32, which holds bf16 and fp16 exactly);
// an fp32 x, and v, go in as two tf32 pieces, 2^-22 of the value away.
// Sums run in a fixed order: results do not change from call to call.
#include "bc_internal.cuh"

#include <type_traits>

namespace bc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kSms = 148;
constexpr int kMaxDescs = 32;          // per launch (kernel parameters)
constexpr int kMaxSegments = 4096;
constexpr int kMaxRank = 128;
constexpr int kGroupRows = 256;        // up to here rows are ordered by adapter
constexpr int kChunk = 32;             // ranks per shrink block
constexpr int kMaxSplit = 16;          // parts of K
constexpr int kUnits = 4;              // 32-column steps per warp of an expand block
constexpr int kCols = kUnits * kWarps * 32;

struct Desc {
    const void *x, *A, *B;
    float *y;
    int N, K;
    int split;                         // parts of K
    int first_block;                   // expand: first of this projection's column ranges
};
// A tile: `rows` rows of `adapter`.  Row i is first + i, or order[first + i].
struct Tile {
    int first, rows, adapter, unused;
};
struct LoraArgs {
    Desc d[kMaxDescs];
    const int32_t *seg_start;          // [S + 1]
    const int32_t *seg_adapter;        // [S]
    const int32_t *ranks;              // [adapters] or null
    const float *scaling;              // [adapters] or null
    int64_t M;
    int S, R, adapters, count;
    int max_tiles;
    int col_blocks;                    // column ranges of all projections
    int split;                         // largest of the projections'
    int *head;                         // scratch: [0] tiles, [1..] order of the rows (grouped)
    Tile *tiles;                       // scratch: [max_tiles]
    float *v;                          // scratch: [count][max_tiles][split][T * R16], fragment order
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
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

// Row stride of v in shared memory, in floats: 16 modulo 32 keeps the eight
// lanes of a 16-byte load phase (two rows, 64 bytes each) off each other's banks.
__host__ __device__ __forceinline__ int v_stride(int R16) { return R16 | 16; }


// The tile table.  Few rows (decode): rows are ordered by adapter, so that
// requests of one adapter share its reads.  More rows: every segment is cut as
// it stands.  Each shrink block works it out for itself (a few hundred cycles
// for decode) and keeps only its own tile; the first block of a tile leaves
// it for expand_kernel, block 0 the number of tiles and the rows' order.
struct PlanShared {
    int key[kGroupRows], order[kGroupRows], scan[kWarps + 1];
    Tile mine;
    int found;
};
__device__ __forceinline__ void segment(const LoraArgs &a, int i, int &s0, int &s1) {
    s0 = (int)min((int64_t)max(a.seg_start[i], 0), a.M);
    s1 = (int)min((int64_t)max(a.seg_start[i + 1], s0), a.M);
}
__device__ __forceinline__ bool usable(const LoraArgs &a, int ad) {
    return ad >= 0 && ad < a.adapters && (!a.ranks || a.ranks[ad] > 0);
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
            segment(a, i, s0, s1);
            if (s0 < s1) {
                const int ad = a.seg_adapter[i];
                if (usable(a, ad))
                    for (int m = s0; m < s1; ++m) p.key[m] = ad;
            }
        }
        __syncthreads();
        const int mine = p.key[tid];
        int before = 0, same = 0, all = 0;
        for (int j = 0; j < M; ++j) {
            const int k = p.key[j];
            before += k < mine;
            same += k == mine && j < tid;
            all += k == mine;
        }
        before += same;
        const bool live = tid < M && mine != kNone, head = live && same % T == 0;
        __syncthreads();
        p.key[tid] = -1;
        __syncthreads();
        if (live) p.order[before] = tid;
        if (head) p.key[before] = tid;           // at a tile's first place: the thread that knows it
        __syncthreads();
        // place of this thread's tile among the tiles, in sorted order
        const unsigned heads = __ballot_sync(0xffffffffu, p.key[tid] >= 0);
        if (lane == 0) p.scan[warp] = __popc(heads);
        __syncthreads();
        int base = 0, total = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) base += p.scan[w];
            total += p.scan[w];
        }
        const int owner = p.key[tid];
        const int at = base + __popc(heads & ((1u << lane) - 1));
        __syncthreads();
        if (owner >= 0) p.key[owner] = at;       // the owner's tile number
        __syncthreads();
        if (head) {
            const int n = p.key[tid];
            const Tile t{before, min(T, all - same), mine, 0};
            if (n == want) {
                p.mine = t;
                p.found = 1;
            }
        }
        if (publish) {
            if (tid < M) a.head[1 + tid] = p.order[tid];
            if (tid == 0) a.head[0] = total;
        }
        __syncthreads();
        return;
    }
    const int per = (a.S + kThreads - 1) / kThreads;
    const int i0 = min(a.S, tid * per), i1 = min(a.S, i0 + per);
    auto tiles_in = [&](int i, int &s0, int &s1) {
        segment(a, i, s0, s1);
        return s0 < s1 && usable(a, a.seg_adapter[i]) ? (s1 - s0 + T - 1) / T : 0;
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
    int at = inc - own, total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += p.scan[w];
        total += p.scan[w];
    }
    for (int i = i0; i < i1; ++i) {
        const int n = tiles_in(i, s0, s1);
        if (want >= at && want < at + n) {
            const int f = s0 + (want - at) * T;
            p.mine = Tile{f, min(T, s1 - f), a.seg_adapter[i], 0};
            p.found = 1;
        }
        at += n;
    }
    if (publish && tid == 0) a.head[0] = total;
    __syncthreads();
}

// grid: tiles x projections x rank chunks x parts of K
template <typename X, typename W, int MB>
__global__ void __launch_bounds__(kThreads, 2)
shrink_kernel(const __grid_constant__ LoraArgs a) {
    constexpr int T = 16 * MB;
    constexpr bool kBf16 = std::is_same<X, __nv_bfloat16>::value && std::is_same<W, __nv_bfloat16>::value;
    constexpr bool kF32 = std::is_same<X, float>::value;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    __shared__ PlanShared ps;
    __shared__ __align__(16) float red[kWarps * T * kChunk];
    const int chunks = (a.R + kChunk - 1) / kChunk;
    const int per_tile = a.count * chunks * a.split;
    const int ti = blockIdx.x / per_tile, inner = blockIdx.x - ti * per_tile;
    const int part = inner % a.split, chunk = inner / a.split % chunks, di = inner / a.split / chunks;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    plan<T>(a, ps, ti, blockIdx.x == 0);
    if (!ps.found) return;
    const Tile tile = ps.mine;
    if (inner == 0 && tid == 0) a.tiles[ti] = tile;
    const Desc &d = a.d[di];
    if (part >= d.split) return;
    const int K = d.K, R = a.R, R16 = (R + 15) / 16 * 16, r0 = chunk * kChunk, n_rows = tile.rows;
    const int rank = a.ranks ? min(a.ranks[tile.adapter], R) : R;
    if (r0 >= rank) return;
    const bool grouped = a.M <= kGroupRows;
    int64_t row[MB][2];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = mb * 16 + g + h * 8;
            row[mb][h] = i >= n_rows ? -1 : grouped ? ps.order[tile.first + i] : tile.first + i;
        }
    const int nb = min(kChunk, rank - r0 + 7) / 8;             // blocks of eight ranks
    const W *A = static_cast<const W *>(d.A) + (int64_t)tile.adapter * R * K;
    float acc[MB][kChunk / 8][4] = {};
    for (int u = part * kWarps + warp; u < K / 32; u += d.split * kWarps) {
        const int k = u * 32 + t * 8;
        uint4 wa[kChunk / 8];
#pragma unroll
        for (int b = 0; b < kChunk / 8; ++b) {
            const int r = r0 + b * 8 + g;
            wa[b] = make_uint4(0, 0, 0, 0);
            if (b < nb && r < rank) wa[b] = *reinterpret_cast<const uint4 *>(A + (int64_t)r * K + k);
        }
        uint4 xa[MB][2][kF32 ? 2 : 1];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 *p = reinterpret_cast<const uint4 *>(
                    static_cast<const X *>(d.x) + row[mb][h] * K + k);
#pragma unroll
                for (int q = 0; q < (kF32 ? 2 : 1); ++q)
                    xa[mb][h][q] = row[mb][h] >= 0 ? p[q] : make_uint4(0, 0, 0, 0);
            }
        if constexpr (kBf16) {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                if (mb * 16 >= n_rows) break;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint4 &p = xa[mb][0][0], &q = xa[mb][1][0];
                    const uint32_t f[4] = {s ? p.z : p.x, s ? q.z : q.x, s ? p.w : p.y, s ? q.w : q.y};
#pragma unroll
                    for (int b = 0; b < kChunk / 8; ++b)
                        if (b < nb) mma_bf16(acc[mb][b], f, s ? wa[b].z : wa[b].x, s ? wa[b].w : wa[b].y);
                }
            }
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) {              // two of the lane's eight k each
                uint32_t w0[kChunk / 8], w1[kChunk / 8];
#pragma unroll
                for (int b = 0; b < kChunk / 8; ++b)
                    widen<W>(s == 0 ? wa[b].x : s == 1 ? wa[b].y : s == 2 ? wa[b].z : wa[b].w, w0[b], w1[b]);
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
                    if (mb * 16 >= n_rows) break;
                    uint32_t hi[4], lo[4];
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
                    for (int b = 0; b < kChunk / 8; ++b)
                        if (b < nb) {
                            if constexpr (kF32)
                                mma_tf32(acc[mb][b], lo[0], lo[1], lo[2], lo[3], w0[b], w1[b]);
                            mma_tf32(acc[mb][b], hi[0], hi[1], hi[2], hi[3], w0[b], w1[b]);
                        }
                }
            }
        }
    }
    // the block's sum over its warps, in fragment order
    float4 *mine = reinterpret_cast<float4 *>(red) + warp * (T * kChunk / 4);
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int b = 0; b < kChunk / 8; ++b)
            mine[(mb * (kChunk / 8) + b) * 32 + lane] =
                make_float4(acc[mb][b][0], acc[mb][b][1], acc[mb][b][2], acc[mb][b][3]);
    __syncthreads();
    float4 *out = reinterpret_cast<float4 *>(
        a.v + (((int64_t)di * a.max_tiles + ti) * a.split + part) * (T * R16));
    for (int i = tid; i < T * kChunk / 4; i += kThreads) {
        const int mb = i / 32 / (kChunk / 8), b = i / 32 % (kChunk / 8);
        if (b >= nb || mb * 16 >= n_rows) continue;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 p = reinterpret_cast<const float4 *>(red)[w * (T * kChunk / 4) + i];
            s.x += p.x;
            s.y += p.y;
            s.z += p.z;
            s.w += p.w;
        }
        out[(mb * (R16 / 8) + r0 / 8 + b) * 32 + (i & 31)] = s;
    }
}

// grid: tiles x column ranges of all projections
template <typename W, int MB>
__global__ void __launch_bounds__(kThreads, 2)
expand_kernel(const __grid_constant__ LoraArgs a) {
    constexpr int T = 16 * MB;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int R = a.R, R16 = (R + 15) / 16 * 16, VS = v_stride(R16);
    extern __shared__ __align__(16) float vsm[];
    float *vhi = vsm, *vlo = vsm + T * VS;                     // [T][VS]
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int ti = blockIdx.x / a.col_blocks, cb = blockIdx.x - ti * a.col_blocks;
    if (ti >= a.head[0]) return;
    const Tile tile = a.tiles[ti];
    int di = 0;
    while (di + 1 < a.count && cb >= a.d[di + 1].first_block) ++di;
    const Desc &d = a.d[di];
    const int N = d.N, n_rows = tile.rows;
    const int rank = a.ranks ? min(a.ranks[tile.adapter], R) : R, used = (rank + 7) / 8;
    const float scale = a.scaling ? a.scaling[tile.adapter] : 1.f;
    const bool grouped = a.M <= kGroupRows;
    int64_t row[MB][2];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = mb * 16 + g + h * 8;
            row[mb][h] = i >= n_rows ? -1 : grouped ? a.head[1 + tile.first + i] : tile.first + i;
        }
    const W *B = static_cast<const W *>(d.B) + (int64_t)tile.adapter * R * N;

    // v of the tile: the parts' sum, as two tf32 pieces
    const float4 *in = reinterpret_cast<const float4 *>(
        a.v + ((int64_t)di * a.max_tiles + ti) * a.split * (T * R16));
    for (int i = tid; i < T * R16 / 4; i += kThreads) {
        const int b = i / 32 % (R16 / 8), l = i & 31, m = i / 32 / (R16 / 8) * 16 + (l >> 2);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (b < used && m < n_rows)
            for (int p = 0; p < d.split; ++p) {
                const float4 q = in[p * (T * R16 / 4) + i];
                s.x += q.x;
                s.y += q.y;
                s.z += q.z;
                s.w += q.w;
            }
        const float f[4] = {s.x * scale, s.y * scale, s.z * scale, s.w * scale};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_tf32(f[e], hi[e], lo[e]);
        uint2 *h = reinterpret_cast<uint2 *>(vhi + m * VS + b * 8 + (l & 3) * 2);
        uint2 *o = reinterpret_cast<uint2 *>(vlo + m * VS + b * 8 + (l & 3) * 2);
        h[0] = make_uint2(hi[0], hi[1]);
        h[4 * VS] = make_uint2(hi[2], hi[3]);
        o[0] = make_uint2(lo[0], lo[1]);
        o[4 * VS] = make_uint2(lo[2], lo[3]);
    }
    __syncthreads();

    // y += B v, 32 columns a warp and step: column 2 t + i of block j is
    // column t * 8 + j * 2 + i of the 32
    const bool vec = (N & 3) == 0 && (reinterpret_cast<uintptr_t>(d.y) & 15) == 0;
    const int c0 = (cb - d.first_block) * kCols;
    for (int s = 0; s < kUnits; ++s) {
        const int n0 = c0 + (s * kWarps + warp) * 32, nc = n0 + t * 8;
        if (n0 >= N) break;
        float acc[MB][4][4] = {};                          // [block of rows][j][fragment]
        float yv[MB][2][8];                                // the outputs so far, loaded before the products
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (row[mb][h] < 0) continue;
                const float *p = d.y + row[mb][h] * N + nc;
                if (vec) {
#pragma unroll
                    for (int q = 0; q < 8; q += 4)
                        if (nc + q < N) {
                            const float4 f = *reinterpret_cast<const float4 *>(p + q);
                            yv[mb][h][q] = f.x;
                            yv[mb][h][q + 1] = f.y;
                            yv[mb][h][q + 2] = f.z;
                            yv[mb][h][q + 3] = f.w;
                        }
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (nc + q < N) yv[mb][h][q] = p[q];
                }
            }
        for (int r0 = 0; r0 < rank; r0 += 16) {
            const int r = r0 + t * 4;
            uint32_t w[4][4];                              // [j][the lane's four ranks]
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + (g >> 1) * 8 + j * 2 + (g & 1);
                uint2 q = make_uint2(0, 0);
                if (n < N && r < rank) q = *reinterpret_cast<const uint2 *>(B + (int64_t)n * R + r);
                widen<W>(q.x, w[j][0], w[j][1]);
                widen<W>(q.y, w[j][2], w[j][3]);
#pragma unroll
                for (int e = 1; e < 4; ++e)
                    if (r + e >= rank) w[j][e] = 0;        // behind the adapter's rank: not its values
            }
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                if (mb * 16 >= n_rows) break;
                const int at = (mb * 16 + g) * VS + r;
                const uint4 h0 = *reinterpret_cast<const uint4 *>(vhi + at);
                const uint4 h1 = *reinterpret_cast<const uint4 *>(vhi + at + 8 * VS);
                const uint4 l0 = *reinterpret_cast<const uint4 *>(vlo + at);
                const uint4 l1 = *reinterpret_cast<const uint4 *>(vlo + at + 8 * VS);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mma_tf32(acc[mb][j], l0.x, l1.x, l0.y, l1.y, w[j][0], w[j][1]);
                    mma_tf32(acc[mb][j], l0.z, l1.z, l0.w, l1.w, w[j][2], w[j][3]);
                    mma_tf32(acc[mb][j], h0.x, h1.x, h0.y, h1.y, w[j][0], w[j][1]);
                    mma_tf32(acc[mb][j], h0.z, h1.z, h0.w, h1.w, w[j][2], w[j][3]);
                }
            }
        }
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (row[mb][h] < 0) continue;
                float *p = d.y + row[mb][h] * N + nc;
#pragma unroll
                for (int q = 0; q < 8; ++q) yv[mb][h][q] += acc[mb][q >> 1][h * 2 + (q & 1)];
                if (vec) {
#pragma unroll
                    for (int q = 0; q < 8; q += 4)
                        if (nc + q < N)
                            *reinterpret_cast<float4 *>(p + q) = make_float4(
                                yv[mb][h][q], yv[mb][h][q + 1], yv[mb][h][q + 2], yv[mb][h][q + 3]);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (nc + q < N) p[q] = yv[mb][h][q];
                }
            }
    }
}

// Tile height: 16 rows while rows are few or segments short, else 32.
int tile_rows(int64_t M, int64_t S) { return M <= kGroupRows || M / S <= 16 ? 16 : 32; }
// At most this many tiles: full ones, and a ragged one per segment (or adapter).
int64_t most_tiles(int64_t M, int64_t S, int64_t adapters) {
    const int64_t T = tile_rows(M, S);
    const int64_t ragged = M <= kGroupRows && adapters < S ? adapters : S;
    return M / T + (ragged < M ? ragged : M);
}
// Parts of K for `blocks` blocks per part: enough blocks to fill the GPU
// about three times, a step of 32 for every warp at least.
int split_of(int64_t K, int64_t blocks) {
    int64_t s = (3 * kSms + blocks - 1) / blocks;
    const int64_t most = (K / 32 + kWarps - 1) / kWarps;
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s > kMaxSplit ? kMaxSplit : s);
}
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Scratch of one launch over `count` projections, and the launch's split.
size_t scratch(const bc_lora_desc *descs, int count, int64_t M, int64_t R, int64_t adapters,
               int64_t S, int *split) {
    const int64_t T = tile_rows(M, S), tiles = most_tiles(M, S, adapters), R16 = (R + 15) / 16 * 16;
    const int64_t blocks = tiles * count * ((R + kChunk - 1) / kChunk);
    int most = 1;
    for (int i = 0; i < count; ++i) {
        const int s = split_of(descs[i].K, blocks);
        most = s > most ? s : most;
    }
    *split = most;
    return round256((size_t)(1 + kGroupRows) * 4) + round256((size_t)tiles * sizeof(Tile)) +
           (size_t)count * tiles * most * T * R16 * 4;
}

template <typename X, typename W, int MB>
bc_status launch(const LoraArgs &a, cudaStream_t s) {
    const int chunks = (a.R + kChunk - 1) / kChunk, R16 = (a.R + 15) / 16 * 16;
    const size_t smem = (size_t)2 * 16 * MB * v_stride(R16) * 4;
    shrink_kernel<X, W, MB><<<(unsigned)(a.max_tiles * a.count * chunks * a.split), kThreads, 0, s>>>(a);
    bc_status st = cuda_status();
    if (st != BC_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.max_tiles * a.col_blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, expand_kernel<W, MB>, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return BC_ERR_CUDA;
    }
    return BC_OK;
}

template <typename X, typename W>
bc_status launch(const LoraArgs &a, cudaStream_t s) {
    return tile_rows(a.M, a.S) == 16 ? launch<X, W, 1>(a, s) : launch<X, W, 2>(a, s);
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
    const int64_t tiles = most_tiles(M, n_segments, n_adapters);
    for (int i = 0; i < count; i += kMaxDescs) {
        const int n = count - i < kMaxDescs ? count - i : kMaxDescs;
        int64_t cols = 0;
        for (int j = 0; j < n; ++j) {
            if (descs[i + j].N >= (int64_t)1 << 30 || descs[i + j].K >= (int64_t)1 << 24) return false;
            cols += (descs[i + j].N + kCols - 1) / kCols;
        }
        // blocks of one launch
        if (tiles * cols >= (int64_t)1 << 31) return false;
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
                              int64_t n_adapters, int64_t n_segments) {
    bc_status st;
    if (!sizes_ok(descs, count, M, R, n_adapters, n_segments, &st)) return 0;
    size_t most = 0;
    for (int i = 0; i < count; i += kMaxDescs) {           // launches use the scratch in turn
        int split;
        const size_t b = scratch(descs + i, count - i < kMaxDescs ? count - i : kMaxDescs, M, R,
                                 n_adapters, n_segments, &split);
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
    const size_t need = bc_workspace_size_lora(descs, count, M, R, n_adapters, n_segments);
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
    }
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
    a.max_tiles = (int)most_tiles(M, n_segments, n_adapters);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.head = reinterpret_cast<int *>(ws);
    ws += round256((size_t)(1 + kGroupRows) * 4);
    a.tiles = reinterpret_cast<Tile *>(ws);
    a.v = reinterpret_cast<float *>(ws + round256((size_t)a.max_tiles * sizeof(Tile)));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (int i = 0; i < count; i += kMaxDescs) {
        a.count = count - i < kMaxDescs ? count - i : kMaxDescs;
        scratch(descs + i, a.count, M, R, n_adapters, n_segments, &a.split);
        const int64_t blocks = (int64_t)a.max_tiles * a.count * ((R + kChunk - 1) / kChunk);
        a.col_blocks = 0;
        for (int j = 0; j < a.count; ++j) {
            const bc_lora_desc &d = descs[i + j];
            a.d[j] = Desc{d.x, d.A, d.B, d.y, (int)d.N, (int)d.K, split_of(d.K, blocks), a.col_blocks};
            a.col_blocks += (int)((d.N + kCols - 1) / kCols);
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
