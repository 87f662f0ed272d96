// bc_beam_reorder.cu -- move the beams' states (caches, token histories) to
// their new places after a selection, in place and for many states at once:
// new[i][w] = old[i][parent[i][w]].
//
// A thread owns the same few bytes of all beams of one request: it loads what
// the moving beams need into registers, then stores.  No byte is read after
// it may have been overwritten (only its owner writes it), so no second
// buffer is needed, and beams that stay where they are cost nothing.
// HBM bound: each moved beam is written once and its parent read once (beams
// that share a parent find it in L1).  Measured, on the GPU alone: 16 states of
// 8 x 4 beams, 8 runs of 256,000 bytes: 242 us, 6.2 TB/s; one state of 528
// bytes: 2.4 us.
#include "bc_internal.cuh"

namespace bc {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxStates = 64;         // per launch (kernel parameters)
constexpr int kMaxBeams = 32;
constexpr int kTileBytes = 32768;      // of all beams of a block that moves unaligned bytes

struct State {
    uint8_t *data;
    int64_t row_stride, beam_stride;
    int64_t row_bytes;
    uint32_t rows, units;              // units of `vec` bytes per row, or tiles of a long unaligned one
    int vec;
};
struct ReorderArgs {
    State st[kMaxStates];
    const int32_t *parent;
    int64_t parent_stride;
    int beams;
};

template <typename T, int WMAX>
__device__ __forceinline__ void move(const State &st, uint8_t *base, const int *src, uint32_t moved,
                                     int beams) {
    const uint32_t total = st.rows * st.units;
    for (uint32_t e = blockIdx.x * kThreads + threadIdx.x; e < total; e += gridDim.x * kThreads) {
        const uint32_t row = e / st.units, u = e - row * st.units;
        uint8_t *p = base + row * st.row_stride + (int64_t)u * sizeof(T);
        T v[WMAX];
#pragma unroll
        for (int w = 0; w < WMAX; ++w)
            if (moved >> w & 1) v[w] = *reinterpret_cast<const T *>(p + src[w] * st.beam_stride);
#pragma unroll
        for (int w = 0; w < WMAX; ++w)
            if (moved >> w & 1) *reinterpret_cast<T *>(p + w * st.beam_stride) = v[w];
    }
}

// grid (chunks, batch, states)
template <int WMAX>
__global__ void __launch_bounds__(kThreads) reorder_kernel(const __grid_constant__ ReorderArgs a) {
    __shared__ int src[kMaxBeams];
    __shared__ uint32_t moved_sh;
    if (threadIdx.x < 32) {
        const int w = threadIdx.x;
        int p = w;
        if (w < a.beams) {
            p = a.parent[blockIdx.y * a.parent_stride + w];
            if (p < 0 || p >= a.beams) p = w;          // no such beam: stays as it is
        }
        src[w] = p;
        const uint32_t m = __ballot_sync(0xffffffffu, p != w);
        if (w == 0) moved_sh = m;
    }
    __syncthreads();
    const uint32_t moved = moved_sh;
    if (!moved) return;
    const State &st = a.st[blockIdx.z];
    uint8_t *base = st.data + (int64_t)blockIdx.y * a.beams * st.beam_stride;
    switch (st.vec) {
    case 16: move<uint4, WMAX>(st, base, src, moved, a.beams); break;
    case 8: move<uint2, WMAX>(st, base, src, moved, a.beams); break;
    case 4: move<uint32_t, WMAX>(st, base, src, moved, a.beams); break;
    case 2: move<uint16_t, WMAX>(st, base, src, moved, a.beams); break;
    default: move<uint8_t, WMAX>(st, base, src, moved, a.beams); break;
    }
}

// Long runs at odd places: through shared memory, so that both sides move 16
// aligned bytes at a time.  A block owns a tile of one run, of all beams of a
// request; it loads the parents' (with the source's phase), waits, and stores
// to each beam with its own.
// grid (tiles x rows, batch, states)
template <int WMAX>
__global__ void __launch_bounds__(kThreads) reorder_bytes_kernel(const __grid_constant__ ReorderArgs a) {
    constexpr int kTile = kTileBytes / WMAX, kSlot = kTile + 32, kPieces = kTile / 16 + 1;
    __shared__ __align__(16) uint8_t buf[WMAX * kSlot];
    __shared__ int src[kMaxBeams];
    __shared__ int list[kMaxBeams], n_moved;       // beams that move
    const State &st = a.st[blockIdx.z];
    if (blockIdx.x >= st.rows * st.units) return;
    if (threadIdx.x < 32) {
        const int w = threadIdx.x;
        int p = w;
        if (w < a.beams) {
            p = a.parent[blockIdx.y * a.parent_stride + w];
            if (p < 0 || p >= a.beams) p = w;          // no such beam: stays as it is
        }
        src[w] = p;
        const uint32_t m = __ballot_sync(0xffffffffu, p != w);
        if (p != w) list[__popc(m & ((1u << w) - 1))] = w;
        if (w == 0) n_moved = __popc(m);
    }
    __syncthreads();
    if (n_moved == 0) return;
    const uint32_t row = blockIdx.x / st.units, tile = blockIdx.x - row * st.units;
    const int64_t c0 = (int64_t)tile * kTile;
    const int n = (int)min((int64_t)kTile, st.row_bytes - c0);
    uint8_t *base = st.data + (int64_t)blockIdx.y * a.beams * st.beam_stride + row * st.row_stride + c0;
    for (int i = threadIdx.x; i < n_moved * kPieces; i += kThreads) {
        const int s = i / kPieces, o = (i - s * kPieces) * 16;
        const uint8_t *from = base + src[list[s]] * st.beam_stride;
        const int phase = (int)(reinterpret_cast<uintptr_t>(from) & 15);
        uint8_t *to = buf + s * kSlot + o;
        const int j = o - phase;                       // the piece's first byte, in the tile
        if (j >= 0 && j + 16 <= n) {
            *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from + j);
        } else {
            for (int e = 0; e < 16; ++e)
                if (j + e >= 0 && j + e < n) to[e] = from[j + e];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_moved * kPieces; i += kThreads) {
        const int s = i / kPieces, o = (i - s * kPieces) * 16;
        uint8_t *to = base + list[s] * st.beam_stride;
        const int j = o - (int)(reinterpret_cast<uintptr_t>(to) & 15);
        const uint8_t *from = buf + s * kSlot +
            (reinterpret_cast<uintptr_t>(base + src[list[s]] * st.beam_stride) & 15);
        if (j >= 0 && j + 16 <= n) {
            // 16 bytes at any place: two aligned pieces, shifted
            const uint32_t q = (uint32_t)(from + j - buf), words = q >> 2 & 3, bits = (q & 3) * 8;
            const uint4 lo = *reinterpret_cast<const uint4 *>(buf + (q & ~15u));
            const uint4 hi = *reinterpret_cast<const uint4 *>(buf + (q & ~15u) + 16);
            uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            if (words & 1)
#pragma unroll
                for (int e = 0; e < 7; ++e) v[e] = v[e + 1];
            if (words & 2)
#pragma unroll
                for (int e = 0; e < 6; ++e) v[e] = v[e + 2];
            *reinterpret_cast<uint4 *>(to + j) =
                make_uint4(__funnelshift_r(v[0], v[1], bits), __funnelshift_r(v[1], v[2], bits),
                           __funnelshift_r(v[2], v[3], bits), __funnelshift_r(v[3], v[4], bits));
        } else {
            for (int e = 0; e < 16; ++e)
                if (j + e >= 0 && j + e < n) to[j + e] = from[j + e];
        }
    }
}

// Widest access that the address, the length and the strides of a state allow.
int vec_of(const bc_beam_state &d) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(d.data) | (uint64_t)d.row_bytes |
                          (uint64_t)d.beam_stride | (d.rows > 1 ? (uint64_t)d.row_stride : 0);
    return bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
}

// Whether a state goes through shared memory: long runs whose pieces would have
// one or two bytes.  Both ways, in us, pieces first; a block costs about as much
// however short its run is, and pays sooner where it holds more beams:
//   4 beams of 16 states, 8 requests, 8 runs of 256,000 bytes (1.5 GB read and
//     written): pieces of 1 byte 1866 and 591, 2: 982 and 605, 4: 531 and 582,
//     8: 316 and 544 (16-byte pieces: 238)
//   runs of 1001, 2001, 4001 bytes, 1-byte pieces: 2 beams 93 and 159, 231 and 181,
//     275 and 107; 4 beams 151 and 431, 182 and 268, 179 and 128; 8 beams 144 and 345,
//     144 and 170, 145 and 91; 16 beams 354 and 189, 356 and 104, 353 and 105; of 513
//     bytes: 16 beams 350 and 374, 32 beams 304 and 207
//   2002, 4002, 8002 bytes, 2-byte pieces: 2 beams 121 and 178, 145 and 105, 140 and
//     49; 4 beams 98 and 263, 96 and 126, 97 and 59; 8 beams 80 and 165, 79 and 88, 79
//     and 91; 32 beams 160 and 111, 157 and 111
bool by_bytes(const bc_beam_state &d, int64_t beams) {
    const int vec = vec_of(d);
    if (vec > 2 || (vec == 2 && beams > 4 && beams <= 8)) return false;
    return d.row_bytes >= vec * (beams <= 2 ? 1600 : beams <= 4 ? 3000 : beams <= 8 ? 2400 : beams <= 16 ? 1000 : 500);
}
// Pieces (of the widest access, or a block's tile) of a run.
uint64_t units_of(const bc_beam_state &d, int64_t beams) {
    const int64_t tile = kTileBytes / (beams <= 4 ? 4 : beams <= 8 ? 8 : beams <= 16 ? 16 : 32);
    return by_bytes(d, beams) ? (uint64_t)((d.row_bytes + tile - 1) / tile) : (uint64_t)d.row_bytes / vec_of(d);
}

}  // namespace
}  // namespace bc

using namespace bc;

extern "C" bc_status bc_beam_reorder(const bc_beam_state *states, int count, const int32_t *parent,
                                     int64_t parent_stride, int64_t batch, int64_t beams,
                                     bc_stream_t stream) {
    if (!states || count <= 0 || !parent || batch <= 0 || beams <= 0) return BC_ERR_INVALID_ARG;
    if (parent_stride < beams) return BC_ERR_INVALID_ARG;
    if (beams > kMaxBeams || batch > 65535 || parent_stride > (int64_t)1 << 40) return BC_ERR_UNSUPPORTED;
    if (!aligned(parent, 4)) return BC_ERR_ALIGNMENT;
    for (int i = 0; i < count; ++i) {
        const bc_beam_state &d = states[i];
        if (!d.data || d.rows <= 0 || d.row_bytes <= 0 || d.row_stride < 0 || d.beam_stride < d.row_bytes)
            return BC_ERR_INVALID_ARG;
        // rows of different beams must not share bytes: beams outside rows, or rows outside beams
        const int64_t lim = (int64_t)1 << 46;
        if (d.rows > lim || d.row_bytes > lim || d.row_stride > lim || d.beam_stride > lim)
            return BC_ERR_UNSUPPORTED;
        if (d.rows > 1) {
            const unsigned __int128 in = (unsigned __int128)(d.rows - 1) * d.row_stride + d.row_bytes;
            const unsigned __int128 all =
                (unsigned __int128)(batch * beams - 1) * d.beam_stride + d.row_bytes;
            const bool beams_outside = d.row_stride >= d.row_bytes && (unsigned __int128)d.beam_stride >= in;
            const bool rows_outside = (unsigned __int128)d.row_stride >= all;
            if (!beams_outside && !rows_outside) return BC_ERR_INVALID_ARG;
        }
        if ((unsigned __int128)units_of(d, beams) * d.rows >= (1ull << 31)) return BC_ERR_UNSUPPORTED;
        for (int j = 0; j < i; ++j)
            if (states[j].data == d.data) return BC_ERR_INVALID_ARG;   // would be moved twice
        const unsigned __int128 end = (unsigned __int128)reinterpret_cast<uintptr_t>(d.data) +
            (unsigned __int128)(d.rows - 1) * (d.rows > 1 ? d.row_stride : 0) +
            (unsigned __int128)(batch * beams - 1) * d.beam_stride + d.row_bytes;
        const unsigned __int128 p0 = reinterpret_cast<uintptr_t>(parent);
        const unsigned __int128 p1 = p0 + 4 * ((unsigned __int128)(batch - 1) * parent_stride + beams);
        if (p0 < end && reinterpret_cast<uintptr_t>(d.data) < p1) return BC_ERR_INVALID_ARG;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    ReorderArgs a;
    a.parent = parent;
    a.parent_stride = parent_stride;
    a.beams = (int)beams;
    for (int bytes = 0; bytes < 2; ++bytes)                // aligned (or short) runs, then the others
        for (int i = 0; i < count;) {
            int n = 0;
            uint64_t most = 0;
            for (; i < count && n < kMaxStates; ++i) {
                const bc_beam_state &d = states[i];
                if (by_bytes(d, beams) != (bytes == 1)) continue;
                const uint64_t units = units_of(d, beams);
                a.st[n++] = State{static_cast<uint8_t *>(d.data), d.rows > 1 ? d.row_stride : 0, d.beam_stride,
                                  d.row_bytes, (uint32_t)d.rows, (uint32_t)units, vec_of(d)};
                if (units * d.rows > most) most = units * d.rows;
            }
            if (n == 0) continue;
            const dim3 grid((unsigned)(bytes ? most : (most + kThreads - 1) / kThreads), (unsigned)batch, (unsigned)n);
            if (bytes) {
                if (beams <= 4) reorder_bytes_kernel<4><<<grid, kThreads, 0, s>>>(a);
                else if (beams <= 8) reorder_bytes_kernel<8><<<grid, kThreads, 0, s>>>(a);
                else if (beams <= 16) reorder_bytes_kernel<16><<<grid, kThreads, 0, s>>>(a);
                else reorder_bytes_kernel<32><<<grid, kThreads, 0, s>>>(a);
            } else {
                if (beams <= 4) reorder_kernel<4><<<grid, kThreads, 0, s>>>(a);
                else if (beams <= 8) reorder_kernel<8><<<grid, kThreads, 0, s>>>(a);
                else if (beams <= 16) reorder_kernel<16><<<grid, kThreads, 0, s>>>(a);
                else reorder_kernel<32><<<grid, kThreads, 0, s>>>(a);
            }
            const bc_status st = cuda_status();
            if (st != BC_OK) return st;
        }
    return BC_OK;
}
