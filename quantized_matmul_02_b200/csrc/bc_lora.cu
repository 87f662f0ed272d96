// bc_lora.cu -- low-rank adapters of many requests at once, added to a shared
// projection's output: for the rows of a segment whose adapter is a,
//
//   y[m] += c_a * B_a (A_a x[m]),   A_a [R][K], B_a [N][R], the first rank_a
//   ranks of R in use.
//
// One launch for a whole set of projections.  A cluster of eight CTAs takes a
// tile of rows that share an adapter: the CTAs split K for v = A x, exchange
// their partial sums through distributed shared memory, then split N for
// y += B v.  x, A, B and y are read from global memory straight into matrix
// fragments: the order of the contraction index is free, so a lane takes
// 16-byte pieces along it and every 128-byte line is used whole.
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

#include <cooperative_groups.h>

#include <mutex>
#include <type_traits>

namespace bc {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kMaxDescs = 32;          // per launch (kernel parameters)
constexpr int kMaxSegments = 4096;
constexpr int kMaxRank = 128;
constexpr int kGroupRows = 256;        // up to here rows are ordered by adapter
constexpr int kChunk = 32;             // ranks per pass over x

struct Desc {
    const void *x, *A, *B;
    float *y;
    int N, K;
};
struct LoraArgs {
    Desc d[kMaxDescs];
    const int32_t *seg_start;          // [S + 1]
    const int32_t *seg_adapter;        // [S]
    const int32_t *ranks;              // [adapters] or null
    const float *scaling;              // [adapters] or null
    int64_t M;
    int S, R, adapters, count;
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

template <typename X, typename W, int MB>
__global__ void __launch_bounds__(kThreads)
lora_kernel(const __grid_constant__ LoraArgs a) {
    constexpr int T = 16 * MB;
    constexpr bool kBf16 = std::is_same<X, __nv_bfloat16>::value && std::is_same<W, __nv_bfloat16>::value;
    constexpr bool kF32 = std::is_same<X, float>::value;
    cg::cluster_group cluster = cg::this_cluster();
    const int crank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int R = a.R, R16 = (R + 15) / 16 * 16, VS = v_stride(R16);

    extern __shared__ __align__(16) unsigned char smem[];
    float *part = reinterpret_cast<float *>(smem);             // [T * R16] in fragment order
    float *vhi = part + T * R16;                               // [T][VS]
    float *vlo = vhi + T * VS;
    float *red = vlo + T * VS;                                 // [kWarps][T * kChunk]
    int *tiles = reinterpret_cast<int *>(red + kWarps * T * kChunk);   // see below
    __shared__ int rows[T];
    __shared__ int scan[kWarps + 1];

    // ---- which rows share an adapter ----
    // Few rows (decode): ordered by adapter, tiles = {begin, count, adapter},
    // order[] lists the rows.  More rows: each segment is cut into tiles as it
    // stands, tiles[i] = first tile of segment i.
    const bool grouped = a.M <= kGroupRows;
    int *order = tiles + 3 * kGroupRows;
    int *key = order + kGroupRows;
    int n_tiles;
    auto usable = [&](int ad) {
        return ad >= 0 && ad < a.adapters && (!a.ranks || a.ranks[ad] > 0);
    };
    auto segment = [&](int i, int &s0, int &s1) {
        s0 = (int)min((int64_t)max(a.seg_start[i], 0), a.M);
        s1 = (int)min((int64_t)max(a.seg_start[i + 1], s0), a.M);
    };
    if (grouped) {
        const int M = (int)a.M;
        key[tid] = 0x7fffffff;
        __syncthreads();
        for (int i = tid; i < a.S; i += kThreads) {
            int s0, s1;
            segment(i, s0, s1);
            const int ad = a.seg_adapter[i];
            if (usable(ad))
                for (int m = s0; m < s1; ++m) key[m] = ad;
        }
        __syncthreads();
        const int mine = key[tid];
        int before = 0, same = 0, all = 0;
        for (int j = 0; j < M; ++j) {
            const int k = key[j];
            before += k < mine || (k == mine && j < tid);
            same += k == mine && j < tid;
            all += k == mine;
        }
        const bool live = tid < M && mine != 0x7fffffff;
        __syncthreads();
        // key[] now holds, at each sorted place, how many rows its tile has (0: no tile begins here)
        key[tid] = 0;
        __syncthreads();
        if (live) {
            order[before] = tid;
            if (same % T == 0) key[before] = min(T, all - same);
        }
        __syncthreads();
        const int len = key[tid];
        const unsigned heads = __ballot_sync(0xffffffffu, len > 0);
        if (lane == 0) scan[warp] = __popc(heads);
        __syncthreads();
        int base = 0, total = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) base += scan[w];
            total += scan[w];
        }
        if (len > 0) {
            const int at = base + __popc(heads & ((1u << lane) - 1));
            tiles[3 * at] = tid;
            tiles[3 * at + 1] = len;
        }
        __syncthreads();
        // the tile's adapter: that of its first row
        if (live && same % T == 0) key[before] = mine;
        __syncthreads();
        if (len > 0) tiles[3 * (base + __popc(heads & ((1u << lane) - 1))) + 2] = key[tid];
        n_tiles = total;
    } else {
        const int per = (a.S + kThreads - 1) / kThreads;
        const int i0 = min(a.S, tid * per), i1 = min(a.S, i0 + per);
        auto tiles_in = [&](int i) {
            int s0, s1;
            segment(i, s0, s1);
            return usable(a.seg_adapter[i]) ? (s1 - s0 + T - 1) / T : 0;
        };
        int own = 0;
        for (int i = i0; i < i1; ++i) own += tiles_in(i);
        int inc = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += o;
        }
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        int at = inc - own, total = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += scan[w];
            total += scan[w];
        }
        for (int i = i0; i < i1; ++i) {
            tiles[i] = at;
            at += tiles_in(i);
        }
        if (tid == 0) tiles[a.S] = total;
        n_tiles = total;
    }
    __syncthreads();

    const int clusters = gridDim.x / kCluster;
    const int items = n_tiles * a.count;
    for (int item = blockIdx.x / kCluster; item < items; item += clusters) {
        const int di = item / n_tiles, tile = item - di * n_tiles;
        const Desc &d = a.d[di];
        const int K = d.K, N = d.N;
        int adapter, n_rows, first;
        if (grouped) {
            first = tiles[3 * tile];
            n_rows = tiles[3 * tile + 1];
            adapter = tiles[3 * tile + 2];
        } else {
            int lo = 0, hi = a.S;                              // last segment that begins at or before `tile`
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (tiles[mid] <= tile) lo = mid;
                else hi = mid;
            }
            int s0, s1;
            segment(lo, s0, s1);
            first = s0 + (tile - tiles[lo]) * T;
            n_rows = min(T, s1 - first);
            adapter = a.seg_adapter[lo];
        }
        const int rank = a.ranks ? min(a.ranks[adapter], R) : R;
        const float scale = a.scaling ? a.scaling[adapter] : 1.f;
        if (tid < T) rows[tid] = tid < n_rows ? (grouped ? order[first + tid] : first + tid) : -1;
        __syncthreads();
        int64_t row[MB][2];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            row[mb][0] = rows[mb * 16 + g];
            row[mb][1] = rows[mb * 16 + g + 8];
        }
        const int used = (rank + 7) / 8;                       // blocks of eight ranks
        const W *A = static_cast<const W *>(d.A) + (int64_t)adapter * R * K;
        const W *B = static_cast<const W *>(d.B) + (int64_t)adapter * R * N;

        // ---- v = A x: this CTA's share of K ----
        for (int r0 = 0; r0 < rank; r0 += kChunk) {
            const int nb = min(kChunk / 8, used - r0 / 8);
            float acc[MB][kChunk / 8][4] = {};
            for (int u = crank * kWarps + warp; u < K / 32; u += kCluster * kWarps) {
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
            for (int i = tid; i < T * kChunk / 4; i += kThreads) {
                const int mb = i / 32 / (kChunk / 8), b = i / 32 % (kChunk / 8) + r0 / 8;
                if (b >= R16 / 8) continue;
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 p = reinterpret_cast<const float4 *>(red)[w * (T * kChunk / 4) + i];
                    s.x += p.x;
                    s.y += p.y;
                    s.z += p.z;
                    s.w += p.w;
                }
                reinterpret_cast<float4 *>(part)[(mb * (R16 / 8) + b) * 32 + (i & 31)] = s;
            }
            __syncthreads();
        }
        cluster.sync();

        // ---- the cluster's sum; every CTA gets all of v ----
        const int quads = T * R16 / 4;                         // float4s in part
        for (int i = crank * kThreads + tid; i < quads; i += kCluster * kThreads) {
            const int b = i / 32 % (R16 / 8);
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (b < used) {
                float4 p[kCluster];
#pragma unroll
                for (int c = 0; c < kCluster; ++c)
                    p[c] = reinterpret_cast<const float4 *>(cluster.map_shared_rank(part, c))[i];
#pragma unroll
                for (int c = 0; c < kCluster; ++c) {
                    s.x += p[c].x;
                    s.y += p[c].y;
                    s.z += p[c].z;
                    s.w += p[c].w;
                }
            }
            const float f[4] = {s.x * scale, s.y * scale, s.z * scale, s.w * scale};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split_tf32(f[e], hi[e], lo[e]);
            const int l = i & 31, m = i / 32 / (R16 / 8) * 16 + (l >> 2), r = b * 8 + (l & 3) * 2;
#pragma unroll
            for (int c = 0; c < kCluster; ++c) {
                uint2 *h = reinterpret_cast<uint2 *>(cluster.map_shared_rank(vhi, c) + m * VS + r);
                uint2 *o = reinterpret_cast<uint2 *>(cluster.map_shared_rank(vlo, c) + m * VS + r);
                h[0] = make_uint2(hi[0], hi[1]);
                h[4 * VS] = make_uint2(hi[2], hi[3]);
                o[0] = make_uint2(lo[0], lo[1]);
                o[4 * VS] = make_uint2(lo[2], lo[3]);
            }
        }
        cluster.sync();

        // ---- y += B v: this CTA's share of N, 32 columns a warp and step ----
        // A lane holds 8 neighbouring columns of a row: column 2 t + i of
        // block j is column t * 8 + j * 2 + i of the 32.
        const bool vec = (N & 3) == 0 && (reinterpret_cast<uintptr_t>(d.y) & 15) == 0;
        for (int u = crank * kWarps + warp; u < (N + 31) / 32; u += kCluster * kWarps) {
            const int n0 = u * 32, nc = n0 + t * 8;
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
        __syncthreads();                                       // rows[] is free for the next tile
    }
}

size_t smem_bytes(int MB, int R, int S, bool grouped) {
    const size_t T = 16 * MB, R16 = (R + 15) / 16 * 16;
    const size_t f = T * R16 + 2 * T * v_stride((int)R16) + (size_t)kWarps * T * kChunk;
    return 4 * (f + (grouped ? 5 * kGroupRows : S + 1));
}

// Clusters of the kernel that fit the GPU at once (0: none).
template <typename X, typename W, int MB>
int resident(size_t smem, int dev) {
    static std::mutex mu;
    static int cache[64][2] = {};      // per device: shared memory, clusters (the last size asked)
    static size_t allowed[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    auto kernel = lora_kernel<X, W, MB>;
    if (smem > allowed[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
            return 0;
        allowed[dev] = smem;
    }
    if (cache[dev][0] == (int)smem && cache[dev][1] > 0) return cache[dev][1];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) return 0;
    cache[dev][0] = (int)smem;
    cache[dev][1] = n;
    return n;
}

template <typename X, typename W, int MB>
bc_status launch(const LoraArgs &a, int64_t tiles, cudaStream_t s) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return BC_ERR_CUDA;
    const size_t smem = smem_bytes(MB, a.R, a.S, a.M <= kGroupRows);
    const int fit = resident<X, W, MB>(smem, dev);
    if (fit <= 0) return BC_ERR_CUDA;
    const int64_t items = tiles * a.count;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(kCluster * (items < fit ? items : fit)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, lora_kernel<X, W, MB>, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return BC_ERR_CUDA;
    }
    return cuda_status();
}

template <typename X, typename W>
bc_status launch(const LoraArgs &a, cudaStream_t s) {
    // Tile height: one block of 16 rows while rows are few, up to 64 where the
    // segments are long enough to fill it.
    const int64_t avg = a.M / a.S;
    const int T = a.M <= kGroupRows || avg <= 16 ? 16 : avg <= 64 || a.R > 32 ? 32 : 64;
    // at most this many tiles: full ones, and one ragged one per segment (or adapter)
    const int64_t ragged = a.M <= kGroupRows ? (a.adapters < a.S ? a.adapters : a.S) : a.S;
    const int64_t tiles = a.M / T + (ragged < a.M ? ragged : a.M);
    if (T == 16) return launch<X, W, 1>(a, tiles, s);
    if (T == 32) return launch<X, W, 2>(a, tiles, s);
    return launch<X, W, 4>(a, tiles, s);
}

bool overlap(const void *p, size_t pn, const void *q, size_t qn) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + qn && b < a + pn;
}

}  // namespace
}  // namespace bc

using namespace bc;

extern "C" {

bc_status bc_lora_add_batched(const bc_lora_desc *descs, int count, int64_t M, int64_t R,
                              int64_t n_adapters, bc_dtype x_dtype, bc_dtype w_dtype,
                              const int32_t *seg_start, const int32_t *seg_adapter,
                              int64_t n_segments, const int32_t *ranks, const float *scaling,
                              bc_stream_t stream) {
    if (!descs || count <= 0 || !seg_start || !seg_adapter) return BC_ERR_INVALID_ARG;
    if (M <= 0 || n_segments <= 0 || n_adapters <= 0 || R <= 0 || R % 8) return BC_ERR_INVALID_ARG;
    if (M > (int64_t)1 << 24 || n_segments > kMaxSegments || n_adapters > 1 << 20 || R > kMaxRank)
        return BC_ERR_UNSUPPORTED;
    if ((x_dtype != BC_F32 && x_dtype != BC_BF16) || (w_dtype != BC_F16 && w_dtype != BC_BF16))
        return BC_ERR_UNSUPPORTED;
    if (!aligned(seg_start, 4) || !aligned(seg_adapter, 4) || !aligned(ranks, 4) || !aligned(scaling, 4))
        return BC_ERR_ALIGNMENT;
    for (int i = 0; i < count; ++i) {
        const bc_lora_desc &d = descs[i];
        if (!d.x || !d.A || !d.B || !d.y || d.N <= 0 || d.K <= 0 || d.K % 64) return BC_ERR_INVALID_ARG;
        if (d.N >= (int64_t)1 << 30 || d.K >= (int64_t)1 << 24) return BC_ERR_UNSUPPORTED;
        if (!aligned(d.x, 16) || !aligned(d.A, 16) || !aligned(d.B, 16) || !aligned(d.y, 4))
            return BC_ERR_ALIGNMENT;
        const size_t yb = (size_t)M * d.N * 4, ab = (size_t)n_adapters * R * 2;
        for (int j = 0; j < count; ++j) {
            const bc_lora_desc &e = descs[j];
            if (j != i && e.y && overlap(d.y, yb, e.y, (size_t)M * (e.N > 0 ? e.N : 0) * 4)) return BC_ERR_INVALID_ARG;
            if (overlap(d.y, yb, e.x, (size_t)M * e.K * (x_dtype == BC_F32 ? 4 : 2)) ||
                overlap(d.y, yb, e.A, ab * e.K) || overlap(d.y, yb, e.B, ab * e.N))
                return BC_ERR_INVALID_ARG;
        }
        if (overlap(d.y, yb, seg_start, 4 * (n_segments + 1)) || overlap(d.y, yb, seg_adapter, 4 * n_segments) ||
            overlap(d.y, yb, ranks, 4 * n_adapters) || overlap(d.y, yb, scaling, 4 * n_adapters))
            return BC_ERR_INVALID_ARG;
    }
    LoraArgs a;
    a.seg_start = seg_start;
    a.seg_adapter = seg_adapter;
    a.ranks = ranks;
    a.scaling = scaling;
    a.M = M;
    a.S = (int)n_segments;
    a.R = (int)R;
    a.adapters = (int)n_adapters;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (int i = 0; i < count; i += kMaxDescs) {
        a.count = count - i < kMaxDescs ? count - i : kMaxDescs;
        for (int j = 0; j < a.count; ++j) {
            const bc_lora_desc &d = descs[i + j];
            a.d[j] = Desc{d.x, d.A, d.B, d.y, (int)d.N, (int)d.K};
        }
        bc_status st;
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
                      bc_stream_t stream) {
    const bc_lora_desc d{x, A, B, y, N, K};
    return bc_lora_add_batched(&d, 1, M, R, n_adapters, x_dtype, w_dtype, seg_start, seg_adapter,
                               n_segments, ranks, scaling, stream);
}

}  // extern "C"
