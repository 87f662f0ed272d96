// bc_norm.cu -- residual addition and root-mean-square norm of a projection's
// input rows, with the output as floats or in the packed 8-bit layout.
//
//   h = x + r,  r <- h (rounded to r's type),
//   v = h * rsqrt(mean(h^2) + eps) * w,
//   out = v rounded once, or 8-bit codes with one fp16 scale and zero per 64
//   columns (the layout of bc_pack_codes at 8 bits).
//
// About 5 operations per element against 4 to 14 bytes: HBM bound.  Each row
// is read once and kept in registers between the sum of squares and the
// scaling (up to 16384 columns); longer rows are read twice.  Threads per row
// grow with its length, so that a thread holds 8 or 16 values and an SM some
// 190 KB of rows on their way.
//
// Measured, on the GPU alone: 8192 rows of 4096, fp32 in, bf16 residual and
// out: 51 us, 6.6 TB/s (of 6.55 copied).  32768 rows of 128 in bf16: 5.3 us,
// half of it launch.  One row of 896: 2.1 us (2.5 with the weights loaded after
// the sum).
#include "bc_internal.cuh"

namespace bc {
namespace {

struct NormArgs {
    const void *x;
    void *res;                 // may be null
    const void *w;             // may be null: ones
    void *out;                 // floats, or uint8 codes
    __half *scales, *zeros;    // 8-bit form only
    int64_t M;
    int D;
    float eps;
    int xt, rt, wt, ot;        // bc_dtype values; ot = kQ8 for codes
    // The sum of squares is divided by 2^p, the power of two at or below D, before
    // threads join theirs: a row's is at most twice its mean then, and values up
    // to 1e18 stay in fp32 at any width.
    float unit, rest;          // 2^-p, and D / 2^p (both exact)
};
constexpr int kQ8 = 3;
constexpr int64_t kSms = 148;
constexpr int kResident = 1024;        // threads of norm_stream_kernel that an SM holds (60 registers each)

// Eight consecutive values as loaded (one 16-byte word, or two for fp32):
// every load of a thread is issued before the first one is converted.
struct Raw8 {
    uint4 a, b;
};
__device__ __forceinline__ Raw8 load8(const void *p, int64_t i, int t) {
    Raw8 r;
    if (t == BC_F32) {
        const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i);
        r.a = q[0];
        r.b = q[1];
    } else {
        r.a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
        r.b = make_uint4(0, 0, 0, 0);
    }
    return r;
}
__device__ __forceinline__ void unpack8(const Raw8 &r, int t, float (&f)[8]) {
    const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (t == BC_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
    } else if (t == BC_F16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ uint32_t pack2(float a, float b, int t) {
    if (t == BC_F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void store8(void *p, int64_t i, int t, const float (&f)[8]) {
    if (t == BC_F32) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
            make_uint4(pack2(f[0], f[1], t), pack2(f[2], f[3], t), pack2(f[4], f[5], t),
                       pack2(f[6], f[7], t));
    }
}
// One value (rows whose length or address does not allow 16-byte accesses).
__device__ __forceinline__ uint32_t load1(const void *p, int64_t i, int t) {
    return t == BC_F32 ? static_cast<const uint32_t *>(p)[i]
                       : (uint32_t)static_cast<const uint16_t *>(p)[i];
}
__device__ __forceinline__ float unpack1(uint32_t u, int t) {
    return t == BC_F32 ? __uint_as_float(u)
           : t == BC_F16 ? __half2float(__ushort_as_half((unsigned short)u))
                         : __uint_as_float(u << 16);
}
__device__ __forceinline__ void store1(void *p, int64_t i, int t, float f) {
    if (t == BC_F32)
        static_cast<float *>(p)[i] = f;
    else
        static_cast<uint16_t *>(p)[i] = (uint16_t)pack2(f, 0.f, t);
}

// 8-bit codes of a thread's eight values; the 64 columns of a group lie in
// eight neighbouring lanes.  The range is widened to hold 0, so the zero
// point is a whole number in 0..255, exact in fp16.  The scale is rounded to
// fp16 (nearest even, floor 2^-24, at most 65504) before the codes are formed
// from it, as the packed layout's other producer does.
__device__ __forceinline__ void store_q8(const NormArgs &a, int64_t row, int col, bool live,
                                         const float (&v)[8]) {
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    if (!live) return;
    const float s = fmaxf(__half2float(__float2half_rn(fminf((hi - lo) / 255.f, 65504.f))), 0x1p-24f);
    const float z = fminf(rintf(-lo / s), 255.f);
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = fminf(fmaxf(rintf(v[i] / s) + z, 0.f), 255.f);
        c[i >> 2] |= (uint32_t)q << (8 * (i & 3));
    }
    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + row * a.D + col) =
        make_uint2(c[0], c[1]);
    if (col % 64 == 0) {
        const int64_t g = row * (a.D / 64) + col / 64;
        a.scales[g] = __float2half_rn(s);
        a.zeros[g] = __float2half_rn(z);
    }
}

template <int TPR>
__device__ __forceinline__ float row_sum(float s, float *sh) {
#pragma unroll
    for (int off = (TPR < 32 ? TPR : 32) / 2; off > 0; off >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, off);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) sh[warp] = s;
        __syncthreads();
        s = lane < TPR / 32 ? sh[lane] : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    }
    return s;
}

// TPR threads share a row, each with CH chunks of eight values; a block
// holds one row (TPR >= 128) or 128 / TPR rows.
template <int TPR, int CH, bool VEC>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
norm_kernel(const NormArgs a) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    __shared__ float sh[32];
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool live = row < a.M;
    const int64_t base = live ? row * a.D : 0;
    float h[CH][8];
    // column of value i of chunk c
    auto col = [&](int c, int i) {
        return VEC ? (c * TPR + t) * 8 + i : c * TPR * 8 + i * TPR + t;
    };
    float ss = 0.f;
    Raw8 rw[CH];                                 // the weights are on their way during the sum
    if constexpr (VEC) {
        Raw8 rx[CH], rr[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (live && col(c, 0) < a.D) {
                rx[c] = load8(a.x, base + col(c, 0), a.xt);
                if (a.res) rr[c] = load8(a.res, base + col(c, 0), a.rt);
                if (a.w) rw[c] = load8(a.w, col(c, 0), a.wt);
            }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const bool in = live && col(c, 0) < a.D;
            if (in) {
                unpack8(rx[c], a.xt, h[c]);
                if (a.res) {
                    float r[8];
                    unpack8(rr[c], a.rt, r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[c][i] += r[i];
                    store8(a.res, base + col(c, 0), a.rt, h[c]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!in) h[c][i] = 0.f;
                ss = fmaf(h[c][i], h[c][i], ss);
            }
        }
    } else {
        uint32_t rx[CH][8], rr[CH][8];
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                rx[c][i] = rr[c][i] = 0;
                if (live && col(c, i) < a.D) {
                    rx[c][i] = load1(a.x, base + col(c, i), a.xt);
                    if (a.res) rr[c][i] = load1(a.res, base + col(c, i), a.rt);
                }
            }
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[c][i] = unpack1(rx[c][i], a.xt);
                if (a.res) {
                    h[c][i] += unpack1(rr[c][i], a.rt);
                    if (live && col(c, i) < a.D) store1(a.res, base + col(c, i), a.rt, h[c][i]);
                }
                ss = fmaf(h[c][i], h[c][i], ss);
            }
    }
    ss = row_sum<TPR>(ss * a.unit, sh);
    const float rs = __frsqrt_rn(ss / a.rest + a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if constexpr (VEC) {
            const bool in = live && col(c, 0) < a.D;
            float wv[8];
            if (a.w && in) {
                unpack8(rw[c], a.wt, wv);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) wv[i] = 1.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] = h[c][i] * rs * wv[i];
            if (a.ot == kQ8)
                store_q8(a, row, col(c, 0), in, h[c]);
            else if (in)
                store8(a.out, base + col(c, 0), a.ot, h[c]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (live && col(c, i) < a.D) {
                    const float wv = a.w ? unpack1(load1(a.w, col(c, i), a.wt), a.wt) : 1.f;
                    store1(a.out, base + col(c, i), a.ot, h[c][i] * rs * wv);
                }
        }
    }
}

// Many rows of 513 to 4095 columns: a block stays and takes rows in turn, the
// next one's pieces on their way while this one's are summed and written; the
// weights are read once.  Eight values a thread; blockDim is D / 8 rounded up
// to warps.
template <int MAXT>
__global__ void __launch_bounds__(MAXT, kResident / MAXT) norm_stream_kernel(const NormArgs a) {
    __shared__ float sh[2][32];
    const int col = threadIdx.x * 8, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int warps = blockDim.x >> 5;
    const bool in = col < a.D;
    float wv[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    Raw8 rx, rr;
    int64_t row = blockIdx.x;
    if (in) {
        rx = load8(a.x, row * a.D + col, a.xt);
        if (a.res) rr = load8(a.res, row * a.D + col, a.rt);
        if (a.w) unpack8(load8(a.w, col, a.wt), a.wt, wv);
    }
    for (int buf = 0; row < a.M; row += gridDim.x, buf ^= 1) {
        const int64_t base = row * a.D + col, next = row + gridDim.x;
        float h[8] = {}, r[8];
        if (in) {
            unpack8(rx, a.xt, h);
            if (a.res) unpack8(rr, a.rt, r);
            if (next < a.M) {
                rx = load8(a.x, next * a.D + col, a.xt);
                if (a.res) rr = load8(a.res, next * a.D + col, a.rt);
            }
            if (a.res) {
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] += r[i];
                store8(a.res, base, a.rt, h);
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[i], h[i], ss);
        ss *= a.unit;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        if (lane == 0) sh[buf][warp] = ss;
        __syncthreads();                         // (the other half of sh is free until the next one)
        ss = lane < warps ? sh[buf][lane] : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float rs = __frsqrt_rn(ss / a.rest + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = h[i] * rs * wv[i];
        if (a.ot == kQ8)
            store_q8(a, row, col, in, h);
        else if (in)
            store8(a.out, base, a.ot, h);
    }
}

// Rows longer than the registers of a block: one pass for the sum, one for
// the outputs.  The residual is written in the second pass, because the norm
// is taken of the sum before it is rounded to the residual's type.
template <bool VEC>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
    __shared__ float sh[32];
    const int64_t base = (int64_t)blockIdx.x * a.D;
    constexpr int kE = VEC ? 8 : 1;
    // every thread of a warp stays in the loop: the 8-bit form shuffles
    const int steps = (a.D + 1024 * kE - 1) / (1024 * kE);
    float ss = 0.f, rs = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
        for (int s = 0; s < steps; ++s) {
            const int c = (s * 1024 + (int)threadIdx.x) * kE;
            const bool in = c < a.D;
            float h[8] = {}, r[8];
            if (in) {
                if constexpr (VEC) {
                    unpack8(load8(a.x, base + c, a.xt), a.xt, h);
                    if (a.res) {
                        unpack8(load8(a.res, base + c, a.rt), a.rt, r);
#pragma unroll
                        for (int i = 0; i < 8; ++i) h[i] += r[i];
                    }
                } else {
                    h[0] = unpack1(load1(a.x, base + c, a.xt), a.xt);
                    if (a.res) h[0] += unpack1(load1(a.res, base + c, a.rt), a.rt);
                }
            }
            if (pass == 0) {
#pragma unroll
                for (int i = 0; i < kE; ++i) ss = fmaf(h[i] * a.unit, h[i], ss);
                continue;
            }
            if constexpr (VEC) {
                float wv[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
                if (in && a.res) store8(a.res, base + c, a.rt, h);
                if (in && a.w) unpack8(load8(a.w, c, a.wt), a.wt, wv);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = h[i] * rs * wv[i];
                if (a.ot == kQ8)
                    store_q8(a, blockIdx.x, c, in, h);
                else if (in)
                    store8(a.out, base + c, a.ot, h);
            } else if (in) {
                if (a.res) store1(a.res, base + c, a.rt, h[0]);
                const float wv = a.w ? unpack1(load1(a.w, c, a.wt), a.wt) : 1.f;
                store1(a.out, base + c, a.ot, h[0] * rs * wv);
            }
        }
        if (pass == 0) rs = __frsqrt_rn(row_sum<1024>(ss, sh) / a.rest + a.eps);
    }
}

template <int MAXT>
void launch_stream(const NormArgs &a, cudaStream_t s) {
    const int threads = (a.D / 8 + 31) / 32 * 32;
    const int64_t fit = kSms * (kResident / threads);
    norm_stream_kernel<MAXT><<<(unsigned)(a.M < fit ? a.M : fit), threads, 0, s>>>(a);
}

template <int TPR, int CH>
void launch(const NormArgs &a, bool vec, cudaStream_t s) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    const unsigned grid = (unsigned)((a.M + kRows - 1) / kRows);
    constexpr int kThreads = TPR < 128 ? 128 : TPR;
    if (vec)
        norm_kernel<TPR, CH, true><<<grid, kThreads, 0, s>>>(a);
    else
        norm_kernel<TPR, CH, false><<<grid, kThreads, 0, s>>>(a);
}

size_t type_bytes(int t) { return t == BC_F32 ? 4 : t == kQ8 ? 1 : 2; }

bool overlap(const void *p, size_t pn, const void *q, size_t qn) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + qn && b < a + pn;
}

bc_status run(NormArgs a, cudaStream_t s) {
    if (!a.x || !a.out || a.M <= 0 || a.D <= 0) return BC_ERR_INVALID_ARG;
    if (!(a.eps > 0.f) || a.eps > 3.0e38f) return BC_ERR_INVALID_ARG;
    if (a.M > (int64_t)1 << 24) return BC_ERR_UNSUPPORTED;
    const size_t n = (size_t)a.M * a.D;
    const size_t xb = n * type_bytes(a.xt), rb = n * type_bytes(a.rt), ob = n * type_bytes(a.ot);
    const size_t wb = (size_t)a.D * type_bytes(a.wt);
    if (!aligned(a.x, type_bytes(a.xt)) || !aligned(a.out, type_bytes(a.ot)) ||
        (a.res && !aligned(a.res, type_bytes(a.rt))) || (a.w && !aligned(a.w, type_bytes(a.wt))))
        return BC_ERR_ALIGNMENT;
    // out may be x itself (same type); nothing else may overlap what is written
    const bool in_place = a.out == a.x && a.ot == a.xt;
    if ((!in_place && overlap(a.out, ob, a.x, xb)) || overlap(a.out, ob, a.w, wb) ||
        overlap(a.out, ob, a.res, rb) || overlap(a.res, rb, a.x, xb) || overlap(a.res, rb, a.w, wb))
        return BC_ERR_INVALID_ARG;
    const bool vec = a.D % 8 == 0 && aligned(a.x, 16) && aligned(a.out, a.ot == kQ8 ? 8 : 16) &&
                     aligned(a.res, 16) && aligned(a.w, 16);
    if (a.ot == kQ8) {
        if (!vec) return BC_ERR_ALIGNMENT;
        const size_t gb = n / 64 * 2;
        const void *in[] = {a.x, a.res, a.w, a.out};
        const size_t len[] = {xb, rb, wb, ob};
        for (int i = 0; i < 4; ++i)
            if (overlap(a.scales, gb, in[i], len[i]) || overlap(a.zeros, gb, in[i], len[i]))
                return BC_ERR_INVALID_ARG;
        if (overlap(a.scales, gb, a.zeros, gb)) return BC_ERR_INVALID_ARG;
    }
    const int D = a.D;
    int64_t power = 1;
    while (2 * power <= D) power *= 2;
    a.unit = 1.f / (float)power;
    a.rest = (float)D * a.unit;
    // A block that stays pays where it takes several rows and the other kernel's
    // threads are badly filled (it holds 512, 1024, 2048 or 4096 columns), more so
    // where a row has fewer bytes.  With and without, in us, bf16 / fp32 with a
    // bf16 residual:
    //   46875 x 640 39 and 47 / 50 and 58, 30000 x 1008 32.1 and 34.2 / 48.3 and 47.9,
    //   23437 x 1280 33 and 41 / 47.5 and 52.6, 19531 x 1536 32.3 and 35.9 / 47.2 and 48.1,
    //   13020 x 2304 32 and 46 / 49 and 57, 16741 x 1792 31.8 and 33.0 / 48.3 and 46.1,
    //   8370 x 3584 31.5 and 34.6 / 48.6 and 47.0;
    //   113636 x 264 59 and 52 / 73 and 67, 58593 x 512 31.6 and 30.5 / 48.1 and 45.5,
    //   14648 x 2048 30.8 and 29.5 / 47.1 and 45.7, 8192 x 4096 33.9 and 35.4 / 52.5 and 50.8;
    //   two rows a block: 2368 x 896 4.5 and 4.1 / 5.5 and 5.2
    const int width = D <= 1024 ? 1024 : D <= 2048 ? 2048 : 4096;
    if (vec && D > 512 && (D <= 1024 || 8 * D <= (a.res ? 6 : 7) * width) &&
        a.M >= 4 * kSms * (kResident / ((D / 8 + 31) / 32 * 32))) {
        if (D <= 1024) launch_stream<128>(a, s);
        else if (D <= 2048) launch_stream<256>(a, s);
        else launch_stream<512>(a, s);
        return cuda_status();
    }
    if (D <= 64) launch<8, 1>(a, vec, s);
    else if (D <= 128) launch<16, 1>(a, vec, s);
    else if (D <= 256) launch<32, 1>(a, vec, s);
    else if (D <= 512) launch<32, 2>(a, vec, s);
    else if (D <= 1024) launch<128, 1>(a, vec, s);
    else if (D <= 2048) launch<128, 2>(a, vec, s);
    else if (D <= 4096) launch<256, 2>(a, vec, s);
    else if (D <= 8192) launch<512, 2>(a, vec, s);
    else if (D <= 16384) launch<1024, 2>(a, vec, s);
    else if (vec) norm_long_kernel<true><<<(unsigned)a.M, 1024, 0, s>>>(a);
    else norm_long_kernel<false><<<(unsigned)a.M, 1024, 0, s>>>(a);
    return cuda_status();
}

bool float_type(bc_dtype t) { return t == BC_F32 || t == BC_F16 || t == BC_BF16; }

}  // namespace
}  // namespace bc

using namespace bc;

extern "C" {

bc_status bc_add_rmsnorm(const void *x, bc_dtype x_dtype, void *residual, bc_dtype res_dtype,
                         const void *weight, bc_dtype w_dtype, int64_t M, int64_t D, float eps,
                         void *out, bc_dtype out_dtype, bc_stream_t stream) {
    if (!float_type(x_dtype) || (residual && !float_type(res_dtype)) ||
        (weight && !float_type(w_dtype)) || !float_type(out_dtype))
        return BC_ERR_UNSUPPORTED;
    if (D > (int64_t)1 << 24) return BC_ERR_UNSUPPORTED;
    NormArgs a{x, residual, weight, out, nullptr, nullptr, M, (int)(D < 0 ? 0 : D), eps,
               x_dtype, res_dtype, w_dtype, out_dtype, 0.f, 0.f};
    return run(a, reinterpret_cast<cudaStream_t>(stream));
}

bc_status bc_add_rmsnorm_q8(const void *x, bc_dtype x_dtype, void *residual, bc_dtype res_dtype,
                            const void *weight, bc_dtype w_dtype, int64_t M, int64_t D, float eps,
                            uint8_t *codes, void *scales, void *zeros, bc_stream_t stream) {
    if (!scales || !zeros || D <= 0 || D % 64) return BC_ERR_INVALID_ARG;
    if (!float_type(x_dtype) || (residual && !float_type(res_dtype)) ||
        (weight && !float_type(w_dtype)))
        return BC_ERR_UNSUPPORTED;
    if (D > (int64_t)1 << 24) return BC_ERR_UNSUPPORTED;
    if (!aligned(scales, 2) || !aligned(zeros, 2)) return BC_ERR_ALIGNMENT;
    NormArgs a{x, residual, weight, codes, static_cast<__half *>(scales),
               static_cast<__half *>(zeros), M, (int)D, eps, x_dtype, res_dtype, w_dtype, kQ8, 0.f, 0.f};
    return run(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
