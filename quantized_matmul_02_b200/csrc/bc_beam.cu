// bc_beam.cu -- beam search's selection after the LM head: over the beams and
// the vocabulary of each request, the n_out largest
//
//   total[w][v] = score[w] + logit[w][v] - log(sum_u exp(logit[w][u])),
//
// ties going to the lowest w * V + v.
//
// Two launches.  The first one reads the logits once: a block owns one span of
// one beam's row and keeps the sum of exponentials and, for every 16 logits
// that a thread reads together, their maximum.  The n_out best logits lie in
// the n_out groups with the best maxima (within a beam the order by total is
// the order by logit), so only those groups' logits are looked at again.  The
// second launch joins the spans of each beam and selects over a request's
// beams.  HBM bound: 4 bytes per logit against about seven operations.
//
// Measured, on the GPU alone: 256 rows of 151936 logits, 16 candidates: 36 us,
// 4.4 TB/s; with a fifth of the beams finished 34 us (lists of candidates above a
// running floor instead of the maxima: 57 us, half of it their appending; rank
// counts: 163).  4 rows of 32003: 10 us.
//
// Keys (value, place) are all distinct, so the result does not depend on the
// order in which candidates are collected.
//
// Precision: exponentials in fp32, relative to the largest logit that a warp
// has met, eight added in fp32; the rest and the totals in fp64.  The largest
// one's term is exactly 1; one d below it is 2^-22 (the exponential's own error)
// and 1.1 * 2^-23 d off (difference, product and log2(e) rounded).  So a total is
// off by at most 2^-22 + 7 * 2^-24 + 1.1 * 2^-23 a, where a is the mean of d under the
// row's probabilities, log V at most: 2e-6 if every rounding pointed one way.
// Candidates of two beams change places only where their totals are as near.
#include "bc_internal.cuh"

#include <cooperative_groups.h>

namespace bc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 16;                         // logits per thread and tile
constexpr int kTile = kThreads * kPer;
constexpr int64_t kSms = 148;
constexpr int kMaxOut = 64;
constexpr int kMaxBeams = 32;
constexpr int kCluster = 8;
constexpr int kMaxTiles = 32;                    // per span
constexpr int64_t kMaxV = 1 << 22;
constexpr float kMax = 3.402823466e38f;

// Order-preserving map of a float to an unsigned; -inf is kNegInf, and 0 is
// below every value.  The two zeros are one value.
constexpr uint32_t kNegInf = 0x007fffffu;
__device__ __forceinline__ uint32_t ord(float f) {
    const uint32_t u = __float_as_uint(f + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unord(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t ord64(double d) {
    const uint64_t u = (uint64_t)__double_as_longlong(d + 0.0);
    return u & 0x8000000000000000ull ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double unord64(uint64_t o) {
    return __longlong_as_double((long long)(o & 0x8000000000000000ull ? o & 0x7fffffffffffffffull : ~o));
}
// NaN is a masked token, +inf the largest finite value.
__device__ __forceinline__ float sane(float f) { return f <= kMax ? f : f > kMax ? kMax : -INFINITY; }
__device__ __forceinline__ float exp2_fast(float f) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(f));
    return r;
}
constexpr float kLog2e = 1.44269504f;

// Keys: larger is better, all are distinct.  Within a beam's row a key is
// (ord(logit), ~token).
struct SpanOut {
    double sum;                                  // sum of exp(logit - max)
    float max;                                   // -inf: nothing is above it
};

// The n largest of the block's keys, P per thread of W 32-bit words (most
// significant first, all distinct; a first word of 0 is no key): a mask of this
// thread's among them, all of them when there are no more than n.  Word by
// word and bit by bit from the highest bit in which the keys differ, no
// further than needed to part n of them from the rest.
struct ChooseShared {
    int sums[34 * 3 + 2];
    uint32_t most[kWarps], least[kWarps];
};
template <int P, int W>
__device__ __forceinline__ uint32_t choose(const uint32_t (&k)[P][W], int n, ChooseShared &sh) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int slot = 0;
    if constexpr (P > 1) {
        if (tid < (int)(sizeof(sh.sums) / 4)) sh.sums[tid] = 0;
        __syncthreads();
    }
    auto count = [&](uint32_t mask) {
        if constexpr (P == 1) return __syncthreads_count(mask);
        const int c = __reduce_add_sync(0xffffffffu, __popc(mask));
        if (lane == 0 && c) atomicAdd(&sh.sums[slot], c);
        __syncthreads();
        return sh.sums[slot++];
    };
    uint32_t active = 0, chosen = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) active |= (uint32_t)(k[i][0] != 0) << i;
    if (count(active) <= n) return active;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        uint32_t hi = 0, lo = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (active >> i & 1) {
                hi = max(hi, k[i][w]);
                lo = min(lo, k[i][w]);
            }
        hi = __reduce_max_sync(0xffffffffu, hi);
        lo = __reduce_min_sync(0xffffffffu, lo);
        if (lane == 0) {
            sh.most[warp] = hi;
            sh.least[warp] = lo;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            hi = max(hi, sh.most[i]);
            lo = min(lo, sh.least[i]);
        }
        if (hi != lo) {
            int b = 31 - __clz(hi ^ lo);
            uint32_t T = hi & ~((2u << b) - 1);
            auto above = [&](uint32_t c) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < P; ++i) m |= (uint32_t)(k[i][w] >= c) << i;
                return m & active;
            };
            for (; b >= 0; --b) {
                const uint32_t m = above(T | 1u << b);
                const int reach = count(m);
                if (reach == n) return chosen | m;
                if (reach > n) T |= 1u << b;
            }
            // T is the n-th's word: those above it are in, those equal to it go on
            const uint32_t over = T == 0xffffffffu ? 0 : above(T + 1);
            n -= count(over);
            chosen |= over;
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (k[i][w] != T) active &= ~(1u << i);
        }
        __syncthreads();                         // most[] and least[] are free
    }
    return chosen;
}

struct SelectArgs {
    const float *logits;                         // [batch * beams][V]
    const float *scores;                         // [batch][beams]
    const uint8_t *finished;                     // [batch][beams] or null
    int64_t V;
    int beams, n_out, spans;
    int span;                                    // logits per span: up to kMaxTiles of kTile
    int32_t eos, pad;
    SpanOut *heads;                              // [rows][spans]
    uint64_t *keys;                              // [rows][spans][n_out], each list in order
    float *out_scores;                           // [batch][n_out]
    int32_t *parent, *token;
    uint8_t *out_finished;
};

// A beam that contributes nothing by its logits: finished, or without a score.
__device__ __forceinline__ bool idle(const SelectArgs &a, int64_t r) {
    const float s = a.scores[r];
    return (a.finished && a.finished[r]) || isnan(s) || s == -INFINITY;
}

// One span of row r.  Places u of a row count from the 16-byte boundary at or
// before its first logit (token = u - skip), so that any V reads whole words.
__device__ __forceinline__ void scan_span(const SelectArgs &a, const int64_t r, const int sp) {
    __shared__ uint32_t best[kMaxTiles][kThreads];   // ord(maximum) of each group, 0: no logits in it
    __shared__ uint64_t kept[kMaxOut];
    __shared__ int picked[kMaxOut], list[kThreads];  // groups: tile * kThreads + thread
    __shared__ ChooseShared cs;
    __shared__ double dsh[kWarps];
    __shared__ float fsh[kWarps];
    __shared__ int count;
    if (idle(a, r)) return;
    const float *row = a.logits + r * a.V;
    const int skip = (int)(reinterpret_cast<uintptr_t>(row) >> 2 & 3);
    const int u0 = sp * a.span, u1 = min((int)a.V + skip, u0 + a.span);
    row -= skip;                                 // (never read before its first logit)
    const int tid = threadIdx.x, n_out = a.n_out;
    if (tid == 0) count = 0;
    float m = -INFINITY;                         // the warp's largest so far
    double sum = 0;                              // of exp(logit - m)
    // element i of a thread's group in the tile that begins at t0
    auto place = [](int t0, int thread, int i) { return t0 + (i / 4 * kThreads + thread) * 4 + (i & 3); };
    auto load = [&](int t0, float (&x)[kPer]) {
        if (t0 >= skip && t0 + kTile <= u1) {
            const float4 *p = reinterpret_cast<const float4 *>(row + t0) + tid;
#pragma unroll
            for (int i = 0; i < kPer; i += 4) {
                const float4 f = __ldcs(p + i / 4 * kThreads);
                x[i] = f.x;
                x[i + 1] = f.y;
                x[i + 2] = f.z;
                x[i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int u = place(t0, tid, i);
                x[i] = u >= skip && u < u1 ? __ldcs(row + u) : -INFINITY;
            }
        }
    };
    float next[kPer];
    load(u0, next);
    int tiles = 0;
    uint32_t own = 0;                            // the best of this thread's groups
    for (int t0 = u0; t0 < u1; t0 += kTile, ++tiles) {
        float x[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = next[i];
        if (t0 + kTile < u1) load(t0 + kTile, next);
        float total = x[0], top;
#pragma unroll
        for (int i = 1; i < kPer; ++i) total += x[i];
        if (!(total < INFINITY))                 // a NaN or +inf among them, or very large ones
#pragma unroll
            for (int i = 0; i < kPer; ++i) x[i] = sane(x[i]);
        top = x[0];
#pragma unroll
        for (int i = 1; i < kPer; ++i) top = fmaxf(top, x[i]);
        uint32_t key = ord(top);
        // The warp's reference is the largest logit it has seen: that one's term is
        // exactly 1, and the others' exponents are as near 0 as they can be.  A warp
        // finds larger ones less and less often (1/t of its t-th tile), so the fp64
        // exponential costs little.
        if (__any_sync(0xffffffffu, top > m)) {
            const float now = unord(__reduce_max_sync(0xffffffffu, key));
            if (m > -INFINITY) sum *= exp((double)m - (double)now);
            m = now;
        }
        if (m > -INFINITY) {
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kPer; ++i) s[i & 1] += exp2_fast((x[i] - m) * kLog2e);
            sum += (double)s[0] + (double)s[1];
        }
        if (top == -INFINITY && !(t0 >= skip && t0 + kTile <= u1)) {
            bool any = false;
#pragma unroll
            for (int i = 0; i < kPer; ++i) any |= place(t0, tid, i) >= skip && place(t0, tid, i) < u1;
            if (!any) key = 0;
        }
        best[tiles][tid] = key;
        own = max(own, key);
    }
    __syncthreads();

    // The best groups.  n_out threads' own best reach `bar`, so no group below
    // it is among them; those that reach it are few, but for equal logits.
    auto logit = [&](int group, int i, int &u) {
        u = place(u0 + group / kThreads * kTile, group % kThreads, i);
        return u >= skip && u < u1 ? sane(row[u]) : -INFINITY;
    };
    // k: maxima of groups, group(i) this thread's i-th
    auto pick = [&](auto &k, auto group) {
        constexpr int P = sizeof(k) / sizeof(k[0]);
        const uint32_t mine = choose(k, n_out, cs);
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (mine >> i & 1) picked[atomicAdd(&count, 1)] = group(i);
        __syncthreads();
        const int got = count;
        if (got == n_out) return;
        // Fewer: all groups, or all but some of equal maxima, of which those with
        // the lowest places are wanted.  A group's is its first logit of that value.
        uint32_t rest = 0;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (!(mine >> i & 1)) rest = max(rest, k[i][0]);
        rest = __reduce_max_sync(0xffffffffu, rest);
        if ((tid & 31) == 0) cs.most[tid >> 5] = rest;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) rest = max(rest, cs.most[i]);
        if (rest == 0) return;
        uint32_t k2[P][1];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            k2[i][0] = 0;
            if (!(mine >> i & 1) && k[i][0] == rest)
                for (int e = kPer - 1; e >= 0; --e) {
                    int u;
                    const float f = logit(group(i), e, u);
                    if (u >= skip && u < u1 && ord(f) == rest) k2[i][0] = ~(uint32_t)(u - skip);
                }
        }
        const uint32_t more = choose(k2, n_out - got, cs);
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (more >> i & 1) picked[atomicAdd(&count, 1)] = group(i);
        __syncthreads();
    };
    uint32_t bar = 1;
    {
        const uint32_t k[1][1] = {{own}};
        const uint32_t mine = choose(k, n_out, cs);
        const int got = __syncthreads_count(mine), all = __syncthreads_count(own != 0);
        if (all > n_out) {
            // the least of the chosen, or, where equal ones were left, their value
            bar = got == n_out ? __reduce_min_sync(0xffffffffu, mine ? own : 0xffffffffu)
                               : __reduce_max_sync(0xffffffffu, mine ? 0 : own);
            if ((tid & 31) == 0) cs.most[tid >> 5] = bar;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kWarps; ++i) bar = got == n_out ? min(bar, cs.most[i]) : max(bar, cs.most[i]);
        }
    }
    for (int i = 0; own >= bar && i < tiles; ++i)
        if (best[i][tid] >= bar) {
            const int to = atomicAdd(&count, 1);
            if (to < kThreads) list[to] = i * kThreads + tid;
        }
    __syncthreads();
    const int listed = count;
    __syncthreads();
    if (tid == 0) count = 0;
    auto each = [&](int i) { return i * kThreads + tid; };
    if (listed <= kThreads) {
        const int mine = tid < listed ? list[tid] : 0;
        uint32_t k[1][1] = {{tid < listed ? best[mine / kThreads][mine % kThreads] : 0}};
        pick(k, [&](int) { return mine; });
    } else if (tiles <= 8) {
        uint32_t k[8][1];
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i][0] = i < tiles ? best[i][tid] : 0;
        pick(k, each);
    } else {
        uint32_t k[kMaxTiles][1];
#pragma unroll
        for (int i = 0; i < kMaxTiles; ++i) k[i][0] = i < tiles ? best[i][tid] : 0;
        pick(k, each);
    }
    const int cands = count * kPer;
    __syncthreads();
    if (tid == 0) count = 0;
    // the best logits of those groups
    auto keep = [&](auto &k) {
        constexpr int P = sizeof(k) / sizeof(k[0]);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = i * kThreads + tid;
            k[i][0] = k[i][1] = 0;
            if (c < cands) {
                int u;
                const float f = logit(picked[c / kPer], c % kPer, u);
                if (u >= skip && u < u1) {
                    k[i][0] = ord(f);
                    k[i][1] = ~(uint32_t)(u - skip);
                }
            }
        }
        const uint32_t mine = choose(k, n_out, cs);
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (mine >> i & 1) kept[atomicAdd(&count, 1)] = (uint64_t)k[i][0] << 32 | k[i][1];
    };
    if (cands <= kThreads) {
        uint32_t k[1][2];
        keep(k);
    } else {
        uint32_t k[kMaxOut * kPer / kThreads][2];
        keep(k);
    }
    // one reference and sum for the span
    float bm = m;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, off));
    if ((tid & 31) == 0) fsh[tid >> 5] = bm;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) bm = fmaxf(bm, fsh[i]);
    double s = m == -INFINITY ? 0.0 : sum * exp((double)m - (double)bm);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if ((tid & 31) == 0) dsh[tid >> 5] = s;
    __syncthreads();
    // in order: a key's rank is its place
    const int64_t at = r * a.spans + sp;
    const int n = count;
    if (tid < n) {
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += kept[j] > kept[tid];
        a.keys[at * n_out + rank] = kept[tid];
    } else if (tid < n_out) {
        a.keys[at * n_out + tid] = 0;            // the list is shorter
    }
    if (tid == 0) {
        s = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) s += dsh[i];
        a.heads[at] = SpanOut{s, bm};
    }
}

// Request-wide keys: (ord64(total), ~(w * V + v)); all are distinct, 0 is none.
struct Key {
    uint64_t hi;
    uint32_t lo;
};
__device__ __forceinline__ bool above(const Key &a, const Key &b) {
    return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}
template <int P>
__device__ __forceinline__ uint32_t choose(const Key (&k)[P], int n, ChooseShared &sh) {
    uint32_t w[P][3];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        w[i][0] = (uint32_t)(k[i].hi >> 32);
        w[i][1] = (uint32_t)k[i].hi;
        w[i][2] = k[i].lo;
    }
    return choose(w, n, sh);
}

constexpr int kMaxLists = 6 * kThreads;          // a request's spans: at most 4 * kSms + kMaxBeams, or
                                                 // kMaxBeams * (kMaxV / (kMaxTiles * kTile) + 1)

// Request b's selection from its spans' lists.
__device__ __forceinline__ void join_spans(const SelectArgs &a, const int64_t b) {
    __shared__ Key kept[kMaxOut], high[kThreads];
    __shared__ int picked[kMaxOut];
    __shared__ double lse[kMaxBeams], score[kMaxBeams];
    __shared__ uint8_t kind[kMaxBeams];          // 0: by its logits, 1: finished, 2: without a score
    __shared__ ChooseShared cs;
    __shared__ int count;
    const int tid = threadIdx.x;
    // eight lanes a beam (32 beams: all at once)
    {
        const int w = tid / 8, sub = tid % 8;
        const int64_t r = b * a.beams + w;
        const bool in = w < a.beams;
        const float sc = in ? a.scores[r] : -INFINITY;
        const bool dead = isnan(sc) || sc == -INFINITY;
        const bool fin = in && a.finished && a.finished[r];
        double s = 0;
        float m = -INFINITY;
        if (!dead && !fin) {
            const SpanOut *h = a.heads + r * a.spans;
            for (int i = sub; i < a.spans; i += 8) {
                const SpanOut o = h[i];
                if (o.max > m) {
                    s = s * exp((double)m - (double)o.max) + o.sum;
                    m = o.max;
                } else if (o.max > -INFINITY) {
                    s += o.sum * exp((double)o.max - (double)m);
                }
            }
        }
        float bm = m;
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, off));
        s = m > -INFINITY ? s * exp((double)m - (double)bm) : 0.0;
        m = bm;
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (in && sub == 0) {
            kind[w] = dead ? 2 : fin ? 1 : m == -INFINITY ? 2 : 0;
            lse[w] = m > -INFINITY ? (double)m + log(s) : 0.0;
            score[w] = (double)fminf(sc, kMax);
        }
    }
    if (tid == 0) count = 0;
    __syncthreads();
    const uint64_t none = ord64(-INFINITY);
    const int lists = a.beams * a.spans;
    // entry `rank` of a list, in descending order; lists are spans, or all of a
    // beam that does not go by its logits (at its first span).  P at a time:
    // their loads are on their way together.
    auto entries = [&](auto &k, auto list, auto rank, int n) {
        constexpr int P = sizeof(k) / sizeof(k[0]);
        uint64_t raw[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            raw[i] = 0;
            if (i < n && kind[list(i) / a.spans] == 0)
                raw[i] = a.keys[(b * lists + list(i)) * a.n_out + rank(i)];
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            k[i] = Key{0, 0};
            if (i >= n) continue;
            const int w = list(i) / a.spans, r = rank(i);
            const uint32_t base = (uint32_t)(w * a.V);
            if (kind[w] == 0) {
                const uint32_t o = (uint32_t)(raw[i] >> 32);
                if (o == 0) continue;                          // the list is shorter
                k[i].hi = o <= kNegInf ? none : ord64(score[w] + ((double)unord(o) - lse[w]));
                k[i].lo = ~(base + ~(uint32_t)raw[i]);
            } else if (list(i) == w * a.spans && r < a.V) {
                // nothing but -inf, by the lowest tokens; first a finished beam's pad token at its score
                int64_t v = r;
                k[i].hi = none;
                if (kind[w] == 1) {
                    if (r == 0) k[i].hi = ord64(score[w]);
                    v = r == 0 ? a.pad : r - 1 + (r - 1 >= a.pad);
                }
                k[i].lo = ~(base + (uint32_t)v);
            }
        }
    };
    auto finish = [&](auto &k) {                 // k: this thread's candidates
        const uint32_t mine = choose(k, a.n_out, cs);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(k) / sizeof(k[0])); ++i)
            if (mine >> i & 1) kept[atomicAdd(&count, 1)] = k[i];
    };
    // candidates c0, c0 + kThreads, ... of the lists' n_out entries each
    auto candidates = [&](auto &k, int cands, auto list) {
        entries(k, [&](int i) { return list((tid + i * kThreads) / a.n_out); },
                [&](int i) { return (tid + i * kThreads) % a.n_out; }, (cands - tid + kThreads - 1) / kThreads);
    };
    auto itself = [](int l) { return l; };
    bool done = lists * a.n_out <= 4 * kThreads;
    if (lists * a.n_out <= kThreads) {
        Key k[1];
        candidates(k, lists * a.n_out, itself);
        finish(k);
    } else if (done) {
        Key k[4];
        candidates(k, lists * a.n_out, itself);
        finish(k);
    } else {
        // Many.  A bar that n_out entries reach: `depth` entries of each of the
        // n_out / depth lists whose depth-th is best.  Entries that reach it are
        // few, unless equal or in a few lists.
        const int depth = min(max(a.n_out / 8, 1), 8), need = (a.n_out + depth - 1) / depth;
        Key bar{0, 0};
        auto lowest = [&](auto &h) {
            // (a thread's lists lie kThreads apart)
            entries(h, [&](int i) { return i * kThreads + tid; }, [&](int) { return depth - 1; },
                    (lists - tid + kThreads - 1) / kThreads);
            const uint32_t mine = choose(h, need, cs);
#pragma unroll
            for (int i = 0; i < (int)(sizeof(h) / sizeof(h[0])); ++i)
                if (mine >> i & 1) kept[atomicAdd(&count, 1)] = h[i];
            __syncthreads();
            const int n = count;
            if (n == need) {
                bar = kept[0];
                for (int i = 1; i < n; ++i)
                    if (above(bar, kept[i])) bar = kept[i];
            }
            __syncthreads();
            if (tid == 0) count = 0;
            __syncthreads();
        };
        if (lists <= kThreads) {
            Key h[1];
            lowest(h);
        } else {
            Key h[kMaxLists / kThreads];
            lowest(h);
        }
        if (bar.hi) {
            const int eighths = (a.n_out + 7) / 8;             // a list's entries, eight at a time
            for (int c0 = tid; c0 < lists * eighths; c0 += 4 * kThreads) {
                auto list = [&](int i) { return (c0 + i * kThreads) / eighths; };
                auto rank = [&](int i) { return (c0 + i * kThreads) % eighths * 8; };
                Key f[4];
                entries(f, list, rank, (lists * eighths - c0 + kThreads - 1) / kThreads);
                for (int e = 0; e < 4; ++e) {
                    const Key first = e == 0 ? f[0] : e == 1 ? f[1] : e == 2 ? f[2] : f[3];
                    if (!first.hi || above(bar, first)) continue;  // entries descend
                    Key k[8];
                    entries(k, [&](int) { return list(e); }, [&](int i) { return rank(e) + i; }, a.n_out - rank(e));
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (k[i].hi && !above(bar, k[i])) {
                            const int to = atomicAdd(&count, 1);
                            if (to < kThreads) high[to] = k[i];
                        }
                }
            }
            __syncthreads();
            const int n = count;
            __syncthreads();
            if (tid == 0) count = 0;
            if (n <= kThreads) {
                Key k[1] = {tid < n ? high[tid] : Key{0, 0}};
                finish(k);
                done = true;
            }
        }
    }
    if (!done) {
        // the n_out lists with the best first entries hold all that can be chosen
        __syncthreads();
        Key h[kMaxLists / kThreads];
        entries(h, [&](int i) { return i * kThreads + tid; }, [](int) { return 0; },
                (lists - tid + kThreads - 1) / kThreads);
        const uint32_t mine = choose(h, a.n_out, cs);
#pragma unroll
        for (int i = 0; i < kMaxLists / kThreads; ++i)
            if (mine >> i & 1) picked[atomicAdd(&count, 1)] = i * kThreads + tid;
        __syncthreads();
        const int n = count;
        __syncthreads();
        if (tid == 0) count = 0;
        Key k[kMaxOut * kMaxOut / kThreads];
        candidates(k, n * a.n_out, [&](int l) { return picked[l]; });
        finish(k);
    }
    __syncthreads();
    if (tid < a.n_out) {
        const Key k = kept[tid];
        int rank = 0;
        for (int j = 0; j < a.n_out; ++j) rank += above(kept[j], k);
        const uint32_t flat = ~k.lo;
        const int w = (int)(flat / (uint32_t)a.V);
        const int32_t t = (int32_t)(flat - (uint32_t)(w * a.V));
        const int64_t at = b * a.n_out + rank;
        a.out_scores[at] = (float)unord64(k.hi);
        a.parent[at] = w;
        a.token[at] = t;
        if (a.out_finished)
            a.out_finished[at] = ((a.finished && a.finished[b * a.beams + w]) || t == a.eos) ? 1 : 0;
    }
}

// grid: rows x spans
__global__ void __launch_bounds__(kThreads, 4) beam_span_kernel(const SelectArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t r = blockIdx.x / a.spans;
    scan_span(a, r, (int)(blockIdx.x - r * a.spans));
}
// one block per request
__global__ void __launch_bounds__(kThreads) beam_join_kernel(const SelectArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    join_spans(a, blockIdx.x);
}
// Few logits: one launch, a cluster per request; its blocks take the spans in
// turn, the first one joins them.
__global__ void __launch_bounds__(kThreads) beam_cluster_kernel(const SelectArgs a) {
    const int rank = blockIdx.x % kCluster;
    const int64_t b = blockIdx.x / kCluster;
    for (int i = rank; i < a.beams * a.spans; i += kCluster) {
        scan_span(a, b * a.beams + i / a.spans, i % a.spans);
        __syncthreads();                         // its shared memory is free
    }
    cooperative_groups::this_cluster().sync();   // (releases and acquires the lists in global memory)
    if (rank == 0) join_spans(a, b);
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// One launch with a cluster per request while a block's span is at most ten
// tiles and the clusters fit the GPU at once (two blocks per SM, but for places
// that a cluster of eight cannot use).  The host is busy for 17 us a call instead
// of 21.  On the GPU, one launch and two, in us (requests x beams x logits):
//   1 x 4 x 32003 11.0 and 10.3, 1 x 1 x 151936 10.3 and 11.0, 1 x 8 x 40000 14.8 and
//   19.5, 1 x 7 x 40000 14.3 and 13.7, 18 x 8 x 40000 17.5 and 18.6, 30 x 1 x 151936 12.3
//   and 14.1, 32 x 4 x 32003 12.8 and 14.1, 28 x 5 x 32003 15.8 and 14.8;
//   longer spans: 1 x 5 x 60000 15.8 and 13.0, 14 x 3 x 100000 15.4 and 14.2;
//   more clusters: 37 x 4 x 32003 19.3 and 14.4, 55 x 8 x 40000 33.9 and 23.0
bool clustered(int64_t batch, int64_t beams, int64_t V) {
    const int64_t tiles = (V + 3 + kTile - 1) / kTile;
    return beams <= kCluster && tiles <= kCluster / beams * 10 && batch <= 32;
}
// Spans per row: as many blocks as the GPU holds at once (four per SM: 256 rows
// 34 us; half as many again 40, twice 42), none shorter than one tile; each
// costs its selection at the end.
int spans_of(int64_t batch, int64_t beams, int64_t V) {
    const int64_t tiles = (V + 3 + kTile - 1) / kTile;
    int64_t want = clustered(batch, beams, V) ? kCluster / beams : 4 * kSms / (batch * beams);
    if (want > tiles) want = tiles;
    if (want < 1) want = 1;
    int64_t per = (tiles + want - 1) / want;
    if (per > kMaxTiles) per = kMaxTiles;
    return (int)((tiles + per - 1) / per);
}

bool overlap(const void *p, size_t pn, const void *q, size_t qn) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + qn && b < a + pn;
}

bc_status check_sizes(int64_t batch, int64_t beams, int64_t V, int64_t n_out) {
    if (batch <= 0 || beams <= 0 || V <= 0 || n_out <= 0) return BC_ERR_INVALID_ARG;
    if (beams > kMaxBeams || n_out > kMaxOut || V > kMaxV || batch * beams > 65535 ||
        batch > 65535)
        return BC_ERR_UNSUPPORTED;
    if (n_out > beams * V) return BC_ERR_INVALID_ARG;
    return BC_OK;
}

}  // namespace
}  // namespace bc

using namespace bc;

extern "C" {

size_t bc_workspace_size_beam(int64_t batch, int64_t beams, int64_t V, int64_t n_out) {
    if (check_sizes(batch, beams, V, n_out) != BC_OK) return 0;
    const size_t lists = (size_t)(batch * beams) * spans_of(batch, beams, V);
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
    a.spans = spans_of(batch, beams, V);
    const int64_t tiles = (V + 3 + kTile - 1) / kTile;
    a.span = (int)((tiles + a.spans - 1) / a.spans * kTile);
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
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (clustered(batch, beams, V)) {
        cfg.gridDim = dim3((unsigned)(batch * kCluster));
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = kCluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        e = cudaLaunchKernelEx(&cfg, beam_cluster_kernel, a);
    } else {
        beam_span_kernel<<<(unsigned)(rows * a.spans), kThreads, 0, s>>>(a);
        e = cudaGetLastError();
        if (e == cudaSuccess) {
            // the second kernel's blocks may start while the first one's finish; they wait for all of it
            cfg.gridDim = dim3((unsigned)batch);
            at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[0].val.programmaticStreamSerializationAllowed = 1;
            e = cudaLaunchKernelEx(&cfg, beam_join_kernel, a);
        }
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return BC_ERR_CUDA;
    }
    return BC_OK;
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
    // what the matmul reads: packed codes with fp16 scales, or fp16 weights with fp32 scales or ranges
    const bool packed = mode == BC_MODE_PACKED;
    const bool scaled = packed || bits != 16;
    const size_t groups = scaled ? (size_t)N * (group == 64 ? K / 64 : 1) * (packed ? 2 : 4) : 0;
    const void *in[] = {x, W_or_packed, scales, zeros, beam_scores, finished};
    const size_t in_len[] = {rows * K * (x_dtype == BC_F32 ? 4 : 2),
                             packed ? (size_t)N * K * (bits > 0 ? bits : 0) / 8 : (size_t)N * K * 2, groups,
                             mode == BC_MODE_RUNTIME_RANGE ? 0 : groups, rows * 4, rows};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 6; ++j)
            if (in_len[j] && overlap(out[i], out_len[i], in[j], in_len[j])) return BC_ERR_INVALID_ARG;
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
