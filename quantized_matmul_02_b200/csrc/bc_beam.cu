// bc_beam.cu -- beam search's selection after the LM head: over the beams and
// the vocabulary of each request, the n_out largest
//
//   total[w][v] = score[w] + logit[w][v] - log(sum_u exp(logit[w][u])),
//
// ties going to the lowest w * V + v.
//
// Two launches, no atomics on results.  The first one reads the logits once:
// a block owns one span of one beam's row, keeps a running maximum and sum of
// exponentials, and the span's n_out best (logit, token) -- within a beam the
// order by total is the order by logit.  The second one joins the spans of
// each beam and selects over a request's beams.  HBM bound: 4 bytes per logit
// against about ten operations.
//
// Precision: exponentials in fp32 relative to the running maximum, their sums
// in fp64 (one addition per 8 elements), totals in fp64.  Order between beams
// is decided on fp64 totals, so two candidates change places only where their
// totals agree to about 1e-7.
#include "bc_internal.cuh"

namespace bc {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                          // logits per thread and tile
constexpr int kTile = kThreads * kPer;
constexpr int64_t kSms = 148;
constexpr int kMaxOut = 64;
constexpr int kMaxBeams = 32;
constexpr int kLimit = 192;                      // kept candidates before they are reduced
constexpr int kCap = kLimit + kTile;

// Order-preserving map of a float to an unsigned; -inf is kNegInf, and 0 is
// below every value.  NaN counts as -inf (a masked token), +inf as the
// largest finite value.
constexpr uint32_t kNegInf = 0x007fffffu;
__device__ __forceinline__ uint32_t ord(float f) {
    if (isnan(f)) return kNegInf;
    const uint32_t u = __float_as_uint(fminf(f, 3.402823466e38f));
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unord(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t ord64(double d) {
    const uint64_t u = (uint64_t)__double_as_longlong(d);
    return u & 0x8000000000000000ull ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double unord64(uint64_t o) {
    return __longlong_as_double((long long)(o & 0x8000000000000000ull ? o & 0x7fffffffffffffffull : ~o));
}

// Keys: larger is better.  Logit key: (ord(logit), ~token); all are distinct.
struct SpanOut {
    double sum;                                  // sum of exp(logit - max)
    float max;                                   // -inf when nothing is above -inf
    int count;                                   // keys that follow
};

// Leaves the `keep` largest of the n keys in buf[0..], sorted, and returns how
// many there are.  All keys are distinct, so a key's rank is its place.
__device__ __forceinline__ int reduce_keys(uint64_t *buf, uint64_t *tmp, int n, int keep) {
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t k = buf[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += buf[j] > k;
        if (rank < keep) tmp[rank] = k;
    }
    __syncthreads();
    const int m = min(n, keep);
    for (int i = threadIdx.x; i < m; i += kThreads) buf[i] = tmp[i];
    __syncthreads();
    return m;
}

struct SelectArgs {
    const float *logits;                         // [batch * beams][V]
    const float *scores;                         // [batch][beams]
    const uint8_t *finished;                     // [batch][beams] or null
    int64_t V;
    int beams, n_out, spans;
    int64_t span;                                // logits per span, a multiple of kTile
    int32_t eos, pad;
    SpanOut *heads;                              // [rows][spans]
    uint64_t *keys;                              // [rows][spans][n_out]
    float *out_scores;                           // [batch][n_out]
    int32_t *parent, *token;
    uint8_t *out_finished;
};

// A beam that contributes nothing by its logits: finished, or without a score.
__device__ __forceinline__ bool idle(const SelectArgs &a, int64_t r) {
    const float s = a.scores[r];
    return (a.finished && a.finished[r]) || isnan(s) || s == -INFINITY;
}

__device__ __forceinline__ double block_sum(double v, double *sh) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += sh[i];
    return v;
}

// grid (spans, rows)
__global__ void __launch_bounds__(kThreads) beam_span_kernel(const SelectArgs a) {
    __shared__ uint64_t buf[kCap];
    __shared__ uint64_t tmp[kMaxOut];
    __shared__ uint32_t tops[kThreads];
    __shared__ double dsh[kThreads / 32];
    __shared__ float fsh[kThreads / 32];
    __shared__ int count;
    __shared__ uint32_t floor_sh;
    const int64_t r = blockIdx.y;
    if (idle(a, r)) return;
    const float *row = a.logits + r * a.V;
    const int64_t v0 = blockIdx.x * a.span, v1 = min(a.V, v0 + a.span);
    const bool vec = (a.V & 3) == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0;
    const int tid = threadIdx.x;
    if (tid == 0) count = 0;
    float m = -INFINITY;
    double sum = 0;
    uint32_t floor = 0;                          // a key has to be above this to be kept
    __syncthreads();
    for (int64_t t0 = v0; t0 < v1; t0 += kTile) {
        uint32_t o[kPer];
        int64_t at[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            at[i] = vec ? t0 + (i / 4 * kThreads + tid) * 4 + (i & 3) : t0 + i * kThreads + tid;
        if (vec) {
#pragma unroll
            for (int i = 0; i < kPer; i += 4) {
                float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (at[i] < v1) f = __ldcs(reinterpret_cast<const float4 *>(row + at[i]));
                o[i] = ord(f.x);
                o[i + 1] = ord(f.y);
                o[i + 2] = ord(f.z);
                o[i + 3] = ord(f.w);
            }
        } else {
            float f[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) f[i] = at[i] < v1 ? __ldcs(row + at[i]) : -INFINITY;
#pragma unroll
            for (int i = 0; i < kPer; ++i) o[i] = ord(f[i]);
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (at[i] >= v1) o[i] = 0;
            top = max(top, o[i]);
        }
        if (top > kNegInf) {
            const float tm = unord(top);
            if (tm > m) {
                sum *= (double)expf(m - tm);
                m = tm;
            }
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (o[i] > kNegInf) s += expf(unord(o[i]) - m);
            sum += (double)s;
        }
        if (t0 == v0) {
            // first tile: the n_out-th largest of the threads' best values.
            // At least n_out elements reach it, at most n_out * kPer + ties.
            tops[tid] = top;
            __syncthreads();
            int above = 0, same = 0;
            for (int j = 0; j < kThreads; ++j) {
                above += tops[j] > top;
                same += tops[j] == top && j < tid;
            }
            if (above + same == a.n_out - 1) floor_sh = top == 0 ? 0 : top - 1;
            __syncthreads();
            floor = floor_sh;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (o[i] > floor)
                buf[atomicAdd(&count, 1)] = (uint64_t)o[i] << 32 | (uint32_t)~(uint32_t)at[i];
        __syncthreads();
        const int held = count;
        __syncthreads();                         // before the next tile counts on
        if (held > kLimit) {
            const int n = reduce_keys(buf, tmp, held, a.n_out);
            // later tokens with the same logit come after the kept ones
            if (n == a.n_out) floor = max(floor, (uint32_t)(buf[n - 1] >> 32));
            if (tid == 0) count = n;
            __syncthreads();
        }
    }
    const int n = reduce_keys(buf, tmp, count, a.n_out);
    // one maximum and sum for the span
    float bm = m;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, off));
    if ((tid & 31) == 0) fsh[tid >> 5] = bm;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) bm = fmaxf(bm, fsh[i]);
    const double s = block_sum(m == -INFINITY ? 0.0 : sum * exp((double)m - (double)bm), dsh);
    const int64_t at = r * a.spans + blockIdx.x;
    if (tid == 0) a.heads[at] = SpanOut{s, bm, n};
    for (int i = tid; i < n; i += kThreads) a.keys[at * a.n_out + i] = buf[i];
}

// Request-wide keys: (ord64(total), ~(w * V + v)).
struct Key {
    uint64_t hi;
    uint32_t lo;
};
__device__ __forceinline__ bool above(const Key &a, const Key &b) {
    return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}

constexpr int kJoinCap = 256 + kThreads;

// one block per request
__global__ void __launch_bounds__(kThreads) beam_join_kernel(const SelectArgs a) {
    __shared__ Key buf[kJoinCap];
    __shared__ Key tmp[kMaxOut];
    __shared__ double lse[kMaxBeams];
    __shared__ double score[kMaxBeams];
    __shared__ uint8_t kind[kMaxBeams];          // 0: by its logits, 1: finished, 2: without a score
    __shared__ int count;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t b = blockIdx.x;
    for (int w = warp; w < a.beams; w += kThreads / 32) {
        const int64_t r = b * a.beams + w;
        const float sc = a.scores[r];
        const bool dead = isnan(sc) || sc == -INFINITY;
        const bool fin = a.finished && a.finished[r];
        double s = 0;
        float m = -INFINITY;
        if (!dead && !fin) {
            const SpanOut *h = a.heads + r * a.spans;
            for (int i = lane; i < a.spans; i += 32) m = fmaxf(m, h[i].max);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            if (m > -INFINITY)
                for (int i = lane; i < a.spans; i += 32)
                    s += h[i].sum * exp((double)h[i].max - (double)m);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        }
        if (lane == 0) {
            kind[w] = dead ? 2 : fin ? 1 : m == -INFINITY ? 2 : 0;
            lse[w] = kind[w] == 0 ? (double)m + log(s) : 0.0;
            score[w] = (double)fminf(sc, 3.402823466e38f);
        }
    }
    if (tid == 0) count = 0;
    __syncthreads();
    // candidates: best entries of all lists first, so that the floor rises early
    const int lists = a.beams * a.spans;
    const int64_t cands = (int64_t)lists * a.n_out;
    Key floor{0, 0};
    const uint64_t none = ord64(-INFINITY);
    for (int64_t c0 = 0; c0 < cands; c0 += kThreads) {
        const int64_t c = c0 + tid;
        Key k{0, 0};
        if (c < cands) {
            const int rank = (int)(c / lists), list = (int)(c % lists);
            const int w = list / a.spans, sp = list % a.spans;
            const uint32_t base = (uint32_t)(w * a.V);
            const int64_t at = (b * a.beams + w) * a.spans + sp;
            if (kind[w] == 0) {
                if (rank < a.heads[at].count) {
                    const uint64_t key = a.keys[at * a.n_out + rank];
                    const uint32_t o = (uint32_t)(key >> 32);
                    k.hi = o <= kNegInf ? none : ord64(score[w] + ((double)unord(o) - lse[w]));
                    k.lo = ~(base + ~(uint32_t)key);
                }
            } else if (sp == 0) {
                // nothing but -inf: the lowest tokens; a finished beam's pad token keeps its score
                if (rank < a.V) {
                    k.hi = none;
                    k.lo = ~(base + (uint32_t)rank);
                    const bool fin = kind[w] == 1;
                    if (fin && rank == a.pad) k.hi = ord64(score[w]);
                    if (fin && a.pad >= a.n_out && rank == a.n_out - 1) {
                        k.hi = ord64(score[w]);
                        k.lo = ~(base + (uint32_t)a.pad);
                    }
                }
            }
        }
        if (above(k, floor)) buf[atomicAdd(&count, 1)] = k;
        __syncthreads();
        const int n = count;
        if (n > 256 || c0 + kThreads >= cands) {
            for (int i = tid; i < n; i += kThreads) {
                const Key x = buf[i];
                int rank = 0;
                for (int j = 0; j < n; ++j) rank += above(buf[j], x);
                if (rank < a.n_out) tmp[rank] = x;
            }
            __syncthreads();
            const int kept = min(n, a.n_out);
            for (int i = tid; i < kept; i += kThreads) buf[i] = tmp[i];
            if (tid == 0) count = kept;
            __syncthreads();
            if (kept == a.n_out) floor = buf[kept - 1];
        }
        __syncthreads();
    }
    for (int i = tid; i < a.n_out; i += kThreads) {
        const Key k = buf[i];
        const uint32_t flat = ~k.lo;
        const int w = (int)(flat / (uint32_t)a.V);
        const int32_t t = (int32_t)(flat - (uint32_t)(w * a.V));
        const int64_t at = b * a.n_out + i;
        a.out_scores[at] = (float)unord64(k.hi);
        a.parent[at] = w;
        a.token[at] = t;
        if (a.out_finished)
            a.out_finished[at] = (kind[w] == 1 || (a.finished && a.finished[b * a.beams + w]) || t == a.eos) ? 1 : 0;
    }
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Spans per row: enough blocks to fill the GPU several times over, none
// shorter than one tile.
int spans_of(int64_t rows, int64_t V) {
    const int64_t tiles = (V + kTile - 1) / kTile;
    int64_t want = (8 * kSms + rows - 1) / rows;
    if (want > tiles) want = tiles;
    if (want < 1) want = 1;
    const int64_t per = (tiles + want - 1) / want;
    return (int)((tiles + per - 1) / per);
}

bool overlap(const void *p, size_t pn, const void *q, size_t qn) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + qn && b < a + pn;
}

bc_status check_sizes(int64_t batch, int64_t beams, int64_t V, int64_t n_out) {
    if (batch <= 0 || beams <= 0 || V <= 0 || n_out <= 0) return BC_ERR_INVALID_ARG;
    if (beams > kMaxBeams || n_out > kMaxOut || V >= (int64_t)1 << 30 || batch * beams > 65535 ||
        batch > 65535)
        return BC_ERR_UNSUPPORTED;
    if (beams * V >= (int64_t)1 << 32) return BC_ERR_UNSUPPORTED;
    if (n_out > beams * V) return BC_ERR_INVALID_ARG;
    return BC_OK;
}

}  // namespace
}  // namespace bc

using namespace bc;

extern "C" {

size_t bc_workspace_size_beam(int64_t batch, int64_t beams, int64_t V, int64_t n_out) {
    if (check_sizes(batch, beams, V, n_out) != BC_OK) return 0;
    const size_t lists = (size_t)(batch * beams) * spans_of(batch * beams, V);
    return round256(lists * sizeof(SpanOut)) + round256(lists * n_out * 8);
}

bc_status bc_beam_select(const float *logits, const float *scores, const uint8_t *finished,
                         int64_t batch, int64_t beams, int64_t V, int64_t n_out, int32_t eos,
                         int32_t pad, float *out_scores, int32_t *parent, int32_t *token,
                         uint8_t *out_finished, void *workspace, size_t workspace_bytes,
                         bc_stream_t stream) {
    if (!logits || !scores || !out_scores || !parent || !token) return BC_ERR_INVALID_ARG;
    bc_status st = check_sizes(batch, beams, V, n_out);
    if (st != BC_OK) return st;
    if (finished && (pad < 0 || pad >= V)) return BC_ERR_INVALID_ARG;
    if (!aligned(logits, 4) || !aligned(scores, 4) || !aligned(out_scores, 4) ||
        !aligned(parent, 4) || !aligned(token, 4))
        return BC_ERR_ALIGNMENT;
    const size_t rows = (size_t)(batch * beams), no = (size_t)(batch * n_out);
    const size_t need = bc_workspace_size_beam(batch, beams, V, n_out);
    if (!workspace || workspace_bytes < need) return BC_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return BC_ERR_ALIGNMENT;
    const void *in[] = {logits, scores, finished};
    const size_t in_len[] = {rows * V * 4, rows * 4, rows};
    const void *out[] = {out_scores, parent, token, out_finished, workspace};
    const size_t out_len[] = {no * 4, no * 4, no * 4, no, need};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 3; ++j)
            if (overlap(out[i], out_len[i], in[j], in_len[j])) return BC_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out_len[i], out[j], out_len[j])) return BC_ERR_INVALID_ARG;
    }
    SelectArgs a;
    a.logits = logits;
    a.scores = scores;
    a.finished = finished;
    a.V = V;
    a.beams = (int)beams;
    a.n_out = (int)n_out;
    a.spans = spans_of((int64_t)rows, V);
    const int64_t tiles = (V + kTile - 1) / kTile;
    a.span = (tiles + a.spans - 1) / a.spans * kTile;
    a.eos = eos;
    a.pad = finished ? pad : 0;
    a.heads = static_cast<SpanOut *>(workspace);
    a.keys = reinterpret_cast<uint64_t *>(static_cast<uint8_t *>(workspace) +
                                          round256(rows * a.spans * sizeof(SpanOut)));
    a.out_scores = out_scores;
    a.parent = parent;
    a.token = token;
    a.out_finished = out_finished;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    beam_span_kernel<<<dim3((unsigned)a.spans, (unsigned)rows), kThreads, 0, s>>>(a);
    beam_join_kernel<<<(unsigned)batch, kThreads, 0, s>>>(a);
    return cuda_status();
}

size_t bc_workspace_size_matmul_beam(int64_t batch, int64_t beams, int64_t N, int64_t K,
                                     int64_t n_out, bc_mode mode, bc_dtype x_dtype) {
    if (check_sizes(batch, beams, N, n_out) != BC_OK || K <= 0 || K % 64) return 0;
    const int64_t M = batch * beams;
    const size_t yb = round256((size_t)M * N * 4);
    const size_t gemv = x_dtype == BC_F32 ? bc_workspace_size(M, N, K, mode) : 0;
    return yb + bc_workspace_size_beam(batch, beams, N, n_out) + gemv;
}

bc_status bc_matmul_q_beam(const void *x, bc_dtype x_dtype, const void *W_or_packed,
                           const void *scales, const void *zeros, int64_t batch, int64_t beams,
                           int64_t N, int64_t K, int bits, int64_t group, bc_mode mode,
                           const float *beam_scores, const uint8_t *finished, int64_t n_out,
                           int32_t eos, int32_t pad, float *out_scores, int32_t *parent,
                           int32_t *token, uint8_t *out_finished, void *workspace,
                           size_t workspace_bytes, bc_stream_t stream) {
    if (!beam_scores || !out_scores || !parent || !token) return BC_ERR_INVALID_ARG;
    bc_status st = check_sizes(batch, beams, N, n_out);
    if (st != BC_OK) return st;
    if (K <= 0 || K % 64) return BC_ERR_INVALID_ARG;
    if (finished && (pad < 0 || pad >= N)) return BC_ERR_INVALID_ARG;
    const size_t need = bc_workspace_size_matmul_beam(batch, beams, N, K, n_out, mode, x_dtype);
    if (!workspace || workspace_bytes < need) return BC_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return BC_ERR_ALIGNMENT;
    if (!aligned(beam_scores, 4) || !aligned(out_scores, 4) || !aligned(parent, 4) || !aligned(token, 4))
        return BC_ERR_ALIGNMENT;
    // scratch: logits [batch * beams][N], the selection's spans, the matmul's own
    const int64_t M = batch * beams;
    const size_t rows = (size_t)M, no = (size_t)(batch * n_out);
    const void *out[] = {out_scores, parent, token, out_finished, workspace};
    const size_t out_len[] = {no * 4, no * 4, no * 4, no, need};
    for (int i = 0; i < 5; ++i) {
        if (overlap(out[i], out_len[i], beam_scores, rows * 4) || overlap(out[i], out_len[i], finished, rows))
            return BC_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out_len[i], out[j], out_len[j])) return BC_ERR_INVALID_ARG;
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const size_t yb = round256((size_t)M * N * 4);
    const size_t sb = bc_workspace_size_beam(batch, beams, N, n_out);
    float *y = reinterpret_cast<float *>(ws);
    st = bc_matmul_q(x, x_dtype, W_or_packed, scales, zeros, M, N, K, bits, group, mode, y,
                     ws + yb + sb, workspace_bytes - yb - sb, stream);
    if (st != BC_OK) return st;
    return bc_beam_select(y, beam_scores, finished, batch, beams, N, n_out, eos, pad, out_scores, parent,
                          token, out_finished, ws + yb, sb, stream);
}

}  // extern "C"
