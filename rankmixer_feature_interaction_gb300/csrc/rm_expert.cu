// Rows by expert: the open (t, e, b) of a batch's gates in that order, a batch's
// rows copied there and back, and the gradients of both.
//
// Sorting.  Seen as a matrix [B][T E] the gates are sorted by column, so a row's slot
// is the number of open gates in the columns before its own plus those above it.  A
// CTA owns eight neighbouring columns (32 bytes of every row, a whole sector) of a
// chunk of rows, each of its 32 warps a run of them, four rows at a time; ranks within
// a warp come from ballots.  First launch: every warp's and chunk's counts.  Second:
// the columns before (their counts are summed anew by every CTA), the chunks and warps
// before, the slots.  Up to kSmallSort gates of few rows one CTA does both, without
// the first launch.  No atomics, so the order is always the same.
//
// Rows.  A warp (for short rows a part of one) takes a run of a row (b, t), reads it once
// and writes it to (or sums it from) the slots of its open experts, in ascending order of
// e; two experts' rows are on their way at a time.  For few long rows the gates' gradient,
// which sums over a whole row, takes all four warps of a CTA.  Bound by memory.
// Measured, T = 32, E = 8, D = 1536 in bf16, two open, 2048 samples, 131,072 sorted rows:
// sort 10 us, gather 88 us (6.9 TB/s), combine 94 (6.4), its gradient 147 (6.9), the
// gather's gradient 92 (6.6).  8 samples: about 2 us each, latency; a warp per row and one
// expert after another took twice that.  1397 samples of T = 37, E = 11, D = 32 in bf16, three
// open: 9.9, 5.0, 8.4, 11.5 and 8.4 us (a warp a row: 9.9, 13.6, 19.3, 24 and 19.3).  777
// samples of T = 5, E = 6, D = 1003 in float32, not 16-byte aligned: 9.6, 6.4, 6.2, 9.2, 6.2.
#include <initializer_list>

#include "rm_fp4.cuh"

namespace rm {
namespace {

constexpr int kCols = 8, kSortWarps = 32, kSortThreads = 32 * kSortWarps;
constexpr int kSmallSort = 16384, kSmallRows = 64;
bool sorts_at_once(int B, long long TE) { return B <= kSmallRows && B * TE <= kSmallSort; }

__device__ __forceinline__ int col_count(uint32_t ballot, int col) { return __popc(ballot & (0x01010101u << col)); }

// Chunks of rows: about two CTAs per SM, and no fewer than 32 rows a warp.
int sort_chunks(int B, long long TE) {
    const long long cols = (TE + kCols - 1) / kCols, rows = (B + 32ll * kSortWarps - 1) / (32ll * kSortWarps);
    const long long most = cols < 304 ? 304 / cols : 1;
    return (int)(rows < most ? rows : most);
}
// The rows of warp w of all the chunks' warps.
__device__ __forceinline__ void warp_rows(int B, int w, int warps, int& b0, int& b1) {
    const int per = (int)(((long long)B + 4ll * warps - 1) / (4ll * warps) * 4);
    b0 = (int)min((long long)B, (long long)w * per);
    b1 = (int)min((long long)B, (long long)b0 + per);
}

// counts[w][g]: open gates of column g among the rows of warp w of the chunk blockIdx.y; totals[chunk][g].
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const float* __restrict__ G, int B, int TE, int* __restrict__ counts, int* __restrict__ totals) {
    constexpr int UNROLL = 8;
    __shared__ int part[kSortWarps][kCols];
    pdl_wait();
    pdl_launch_next();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = lane & 7, g = blockIdx.x * kCols + col;
    int b0, b1, n = 0;
    counts += (size_t)blockIdx.y * kSortWarps * TE;
    warp_rows(B, blockIdx.y * kSortWarps + warp, gridDim.y * kSortWarps, b0, b1);
    for (int b = b0; b < b1; b += 4 * UNROLL) {
        float x[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int r = b + 4 * u + (lane >> 3);
            x[u] = r < b1 && g < TE ? __ldg(G + (size_t)r * TE + g) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) n += col_count(__ballot_sync(0xffffffffu, x[u] > 0.f), col);
    }
    if (lane < kCols) {
        part[warp][lane] = n;
        if (g < TE) counts[(size_t)warp * TE + g] = n;
    }
    __syncthreads();
    if (threadIdx.x < kCols && g < TE) {
        int t = 0;
        for (int w = 0; w < kSortWarps; ++w) t += part[w][threadIdx.x];
        totals[(size_t)blockIdx.y * TE + g] = t;
    }
}

// Sum over the CTA's threads, and the sum of the threads before this one.
__device__ __forceinline__ int block_scan(int v, int* shared, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) shared[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) before += shared[w];
        total += shared[w];
    }
    return before + x - v;
}

// offsets and tiles from the totals, by one CTA; total(g) gives a column's count.
template <typename F>
__device__ __forceinline__ void write_groups(F total, const ExpertRows& r, int TE, int* shared) {
    int rows = 0, tiles = 0;
    for (int g0 = 0; g0 < TE; g0 += blockDim.x) {
        const int g = g0 + threadIdx.x, n = g < TE ? total(g) : 0;
        int all, all_tiles;
        const int at = rows + block_scan(n, shared, all);
        const int tile = tiles + block_scan((n + kExpertTile - 1) / kExpertTile, shared, all_tiles);
        if (g < TE) {
            r.offsets[g] = at;
            for (int i = 0; i * kExpertTile < n; ++i)
                r.tiles[1 + tile + i] = make_int4(g, at + i * kExpertTile, min(kExpertTile, n - i * kExpertTile), 0);
        }
        rows += all, tiles += all_tiles;
    }
    if (threadIdx.x == 0) {
        r.offsets[TE] = rows;
        r.tiles[0] = make_int4(tiles, rows, 0, 0);
    }
}

// A gate's place among the open ones.
__device__ __forceinline__ void place(const ExpertRows& r, size_t at, bool open, int slot, int source) {
    r.slot[at] = open ? slot : -1;
    if (open) r.source[slot] = source;
}

__global__ void __launch_bounds__(kSortThreads)
sort_place_kernel(const float* __restrict__ G, int TE, const int* __restrict__ counts, const int* __restrict__ totals,
                  ExpertRows r) {
    constexpr int UNROLL = 8;
    __shared__ int shared[kSortWarps], base[kCols];
    pdl_wait();
    pdl_launch_next();
    const int chunk = blockIdx.y, chunks = gridDim.y;
    if (blockIdx.x == gridDim.x - 1) {                 // the last CTA has no columns
        if (chunk == 0)
            write_groups(
                [&](int g) {
                    int n = 0;
#pragma unroll 8
                    for (int c = 0; c < chunks; ++c) n += totals[(size_t)c * TE + g];
                    return n;
                },
                r, TE, shared);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = lane & 7, g0 = blockIdx.x * kCols, g = g0 + col;
    // the columns before, of every chunk; then (warp 0, lane 8 i + j: column j, chunks i, i
    // + 4, ..) this CTA's columns before, and its own chunks before
    int before = 0, all;
#pragma unroll 4
    for (int i = threadIdx.x; i < chunks * g0; i += kSortThreads) before += totals[(size_t)(i / g0) * TE + i % g0];
    block_scan(before, shared, all);
    if (warp == 0) {
        int total = 0, above = 0;
#pragma unroll 8
        for (int c = lane >> 3; c < chunks; c += 4) {
            const int n = g < TE ? totals[(size_t)c * TE + g] : 0;
            total += n;
            above += c < chunk ? n : 0;
        }
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
            total += __shfl_xor_sync(0xffffffffu, total, o);
            above += __shfl_xor_sync(0xffffffffu, above, o);
        }
        int left = total;                              // up to and with this column
#pragma unroll
        for (int o = 1; o < kCols; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, left, o, kCols);
            if (col >= o) left += x;
        }
        if (lane < kCols) base[lane] = all + left - total + above;
    }
    int mine = 0;
    // the warps before this one: lanes 8 j + col take warps j, j + 4, ..
    counts += (size_t)chunk * kSortWarps * TE;
    for (int w = lane >> 3; w < warp; w += 4)
        if (g < TE) mine += counts[(size_t)w * TE + g];
    mine += __shfl_xor_sync(0xffffffffu, mine, 8);
    mine += __shfl_xor_sync(0xffffffffu, mine, 16);
    __syncthreads();
    mine += base[col];
    int b0, b1;
    warp_rows(r.B, chunk * kSortWarps + warp, chunks * kSortWarps, b0, b1);
    const uint32_t below = (0x01010101u << col) & ((1u << lane) - 1u);
    for (int b = b0; b < b1; b += 4 * UNROLL) {
        float x[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int row = b + 4 * u + (lane >> 3);
            x[u] = row < b1 && g < TE ? __ldg(G + (size_t)row * TE + g) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int row = b + 4 * u + (lane >> 3);
            const uint32_t m = __ballot_sync(0xffffffffu, x[u] > 0.f);
            if (row < b1 && g < TE)
                place(r, (size_t)row * TE + g, x[u] > 0.f, mine + __popc(m & below), row * r.T + g / r.E);
            mine += col_count(m, col);
        }
    }
}

// Few gates: one CTA, a thread per column, its open gates a mask of 64 bits.  A group
// of so few rows is one tile: rows and tiles are counted in one sum.
__global__ void __launch_bounds__(kSortThreads)
sort_small_kernel(const float* __restrict__ G, int TE, ExpertRows r) {
    static_assert(kSmallRows <= 64 && kSmallSort < 32768, "a mask, and two sums of 16 bits");
    __shared__ int shared[kSortWarps];
    pdl_wait();
    pdl_launch_next();
    int sum = 0;                                       // rows, and 2^16 tiles
    for (int g0 = 0; g0 < TE; g0 += kSortThreads) {
        const int g = g0 + threadIdx.x;
        unsigned long long open = 0;
        if (g < TE) {
#pragma unroll 8
            for (int b = 0; b < r.B; ++b) open |= (unsigned long long)(__ldg(G + (size_t)b * TE + g) > 0.f) << b;
        }
        const int n = __popcll(open);
        int all;
        const int at = sum + block_scan(n | (n > 0 ? 1 << 16 : 0), shared, all);
        sum += all;
        if (g < TE) {
            int slot = at & 0xffff;
            const int source = g / r.E;
            r.offsets[g] = slot;
            if (n > 0) r.tiles[1 + (at >> 16)] = make_int4(g, slot, n, 0);
#pragma unroll 8
            for (int b = 0; b < r.B; ++b) {
                const bool is = open >> b & 1;
                place(r, (size_t)b * TE + g, is, slot, b * r.T + source);
                slot += is;
            }
        }
    }
    if (threadIdx.x == 0) {
        r.offsets[TE] = sum & 0xffff;
        r.tiles[0] = make_int4(sum >> 16, sum & 0xffff, 0, 0);
    }
}

// ---- rows ----------------------------------------------------------------------
constexpr int kRowWarps = 4;

// A lane's piece of a row: 16 bytes, or one element where rows are not 16-byte aligned.
template <typename T, bool VEC>
struct Piece {
    static constexpr int N = VEC ? 16 / (int)sizeof(T) : 1;
    uint32_t w[VEC ? 4 : 1];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (VEC) {
            const uint4 q = *reinterpret_cast<const uint4*>(p);
            w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        } else if constexpr (sizeof(T) == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (VEC)
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (sizeof(T) == 4)
            *reinterpret_cast<uint32_t*>(p) = w[0];
        else
            *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ void set(const float (&v)[N]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __float_as_uint(v[i]);
        } else if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        } else {
            w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
        }
    }
};
// L lanes (a group) take a run of a row: kHeld pieces a lane, held at once.  L is 32, or
// 16 or 8 where they hold a whole row: a warp then has two or four rows under way.  Rows
// to 4 bits go by 8 lanes at any length (65,536 rows of 768 to two experts: 26.7 us, by 32
// lanes 34.7); longer rows otherwise do not: with 8 lanes 1003 floats that are not 16-byte
// aligned were combined in 8.3 us instead of 6.2, and the gradient of 1536 took 154, not 147.
template <bool VEC>
constexpr int kHeld = VEC ? 3 : 8;
constexpr int kCodeLanes = 8;

struct Run {
    size_t bt;          // the row
    int p;              // this lane's first piece
    bool there;
};
template <int L, int HELD>
__device__ __forceinline__ Run run_of(const ExpertRows& r, int runs) {
    const unsigned long long id = (unsigned long long)blockIdx.x * (32 * kRowWarps / L) + threadIdx.x / L;
    Run u;
    u.bt = id / (unsigned)runs;
    u.p = (int)(id - u.bt * runs) * L * HELD + threadIdx.x % L;
    u.there = u.bt < (size_t)r.B * r.T;
    return u;
}

// Open experts e0 .. e0 + L - 1 of row bt, as a mask; slot: lane e's.
template <int L>
__device__ __forceinline__ uint32_t open_experts(const int* __restrict__ slots, const Run& u, int E, int e0, long long n,
                                                 int lane, int& slot) {
    slot = u.there && e0 + lane < E ? __ldg(slots + u.bt * E + e0 + lane) : -1;
    const uint32_t m = __ballot_sync(0xffffffffu, slot >= 0 && slot < n);
    return L == 32 ? m : m >> (threadIdx.x & (32 - L)) & ((1u << (L & 31)) - 1u);
}
// A group of the warp has experts left.
template <int L>
__device__ __forceinline__ bool any_left(uint32_t m) {
    return L == 32 ? m != 0 : __any_sync(0xffffffffu, m != 0);
}
// The next expert of the mask (0 where there is none), which leaves it.
__device__ __forceinline__ int next_expert(uint32_t& m) {
    const int e = m ? __ffs(m) - 1 : 0;
    m &= m - 1;
    return e;
}
template <int L>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T, bool VEC, int L>
__global__ void __launch_bounds__(32 * kRowWarps)
gather_kernel(const T* __restrict__ X, ExpertRows r, T* __restrict__ Xs, long long n, int D, int runs) {
    using P = Piece<T, VEC>;
    constexpr int H = kHeld<VEC>;
    pdl_wait();
    pdl_launch_next();
    const int lane = threadIdx.x % L;
    const Run u = run_of<L, H>(r, runs);
    const int pieces = u.there ? D / P::N : 0;
    P x[H];
#pragma unroll
    for (int i = 0; i < H; ++i)
        if (u.p + L * i < pieces) x[i].load(X + u.bt * D + (size_t)(u.p + L * i) * P::N);
    for (int e0 = 0; e0 < r.E; e0 += L) {
        int slot;
        uint32_t m = open_experts<L>(r.slot, u, r.E, e0, n, lane, slot);
        while (any_left<L>(m)) {
            const bool is = m != 0;
            T* dst = Xs + (size_t)__shfl_sync(0xffffffffu, slot, next_expert(m), L) * D;
#pragma unroll
            for (int i = 0; i < H; ++i)
                if (is && u.p + L * i < pieces) x[i].store(dst + (size_t)(u.p + L * i) * P::N);
        }
    }
}

// The same with the rows in 4 bits: a lane rounds 16 values, two lanes a block.
template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kRowWarps)
gather_fp4_kernel(const T* __restrict__ X, ExpertRows r, Fp4View out, long long n, int D, int nb, int runs) {
    constexpr int L = kCodeLanes;
    pdl_wait();
    pdl_launch_next();
    const int lane = threadIdx.x % L;
    const Run u = run_of<L, 1>(r, runs);
    Fp4Raw16<T> v;
    const size_t at = u.bt * D + 16 * (size_t)u.p;
    const int left = u.there ? D - 16 * u.p : 0;                                 // past the row's end: zeros
    if constexpr (VEC)
        v.template load<true>(X + at, left);
    else
        v.load_any(X, at, left, (size_t)r.B * r.T * D);
    int slot;
    uint32_t m = open_experts<L>(r.slot, u, r.E, 0, n, lane, slot);
    uint32_t E;
    const uint2 code = v.round(E);
    for (int e0 = 0;;) {
        while (any_left<L>(m)) {
            const bool is = m != 0 && u.p < 2 * nb;
            const size_t row = (size_t)__shfl_sync(0xffffffffu, slot, next_expert(m), L);
            if (is) {
                *reinterpret_cast<uint2*>(out.codes + row * out.ld + 8 * u.p) = code;
                if ((u.p & 1) == 0) out.scales[row * out.lds + (u.p >> 1)] = (uint8_t)E;
            }
        }
        if ((e0 += L) >= r.E) break;
        m = open_experts<L>(r.slot, u, r.E, e0, n, lane, slot);
    }
}

// TO: the type of V; sums in float32, ascending e, two experts' rows loaded at a time.
template <typename T, typename TO, bool VEC, int L>
__global__ void __launch_bounds__(32 * kRowWarps)
combine_kernel(const T* __restrict__ Y, ExpertRows r, const float* __restrict__ G, TO* __restrict__ V, long long n, int D,
               int runs) {
    using P = Piece<T, VEC>;
    constexpr int H = kHeld<VEC>, N = P::N;
    pdl_wait();
    pdl_launch_next();
    const int lane = threadIdx.x % L;
    const Run u = run_of<L, H>(r, runs);
    const int pieces = u.there ? D / N : 0;
    float v[H][N] = {};
    for (int e0 = 0; e0 < r.E; e0 += L) {
        const float gate = G && u.there && e0 + lane < r.E ? __ldg(G + u.bt * r.E + e0 + lane) : 1.f;
        int slot;
        uint32_t m = open_experts<L>(r.slot, u, r.E, e0, n, lane, slot);
        while (any_left<L>(m)) {
            const bool one = m != 0;
            const int e = next_expert(m);
            const bool two = m != 0;
            const int f = next_expert(m);
            const T* src = Y + (size_t)__shfl_sync(0xffffffffu, slot, e, L) * D;
            const T* src2 = Y + (size_t)__shfl_sync(0xffffffffu, slot, f, L) * D;
            const float g = __shfl_sync(0xffffffffu, gate, e, L), g2 = __shfl_sync(0xffffffffu, gate, f, L);
            P y[H], z[H];
#pragma unroll
            for (int i = 0; i < H; ++i)
                if (one && u.p + L * i < pieces) {
                    y[i].load(src + (size_t)(u.p + L * i) * N);
                    if (two) z[i].load(src2 + (size_t)(u.p + L * i) * N);
                }
#pragma unroll
            for (int i = 0; i < H; ++i)
                if (one && u.p + L * i < pieces) {
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        v[i][k] = fmaf(g, y[i].get(k), v[i][k]);
                        if (two) v[i][k] = fmaf(g2, z[i].get(k), v[i][k]);
                    }
                }
        }
    }
#pragma unroll
    for (int i = 0; i < H; ++i)
        if (u.p + L * i < pieces) {
            TO* dst = V + u.bt * D + (size_t)(u.p + L * i) * N;
            if constexpr (sizeof(T) == sizeof(TO)) {
                Piece<TO, VEC> o;
                o.set(v[i]);
                o.store(dst);
            } else if constexpr (!VEC) {
                *dst = from_f32<TO>(v[i][0]);
            } else if constexpr (sizeof(TO) == 4) {     // bf16 rows to float
                reinterpret_cast<float4*>(dst)[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
                reinterpret_cast<float4*>(dst)[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
            } else {                                    // float rows to bf16
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3]));
            }
        }
}

// L lanes a row, or WARPS warps (where rows are few, all of the CTA's); two experts at a time.
template <typename T, bool VEC, int L, int WARPS>
__global__ void __launch_bounds__(32 * kRowWarps)
combine_backward_kernel(const T* __restrict__ dV, const T* __restrict__ Y, ExpertRows r, const float* __restrict__ G,
                        T* __restrict__ dY, float* __restrict__ dG, long long n, int D) {
    static_assert(L == 32 || WARPS == 1, "warps share a row whole");
    using P = Piece<T, VEC>;
    constexpr int H = WARPS == 1 || !VEC ? kHeld<VEC> : 2, N = P::N, STEP = L * WARPS;
    __shared__ float sums[2][kRowWarps];
    pdl_wait();
    pdl_launch_next();
    const int lane = threadIdx.x % L, warp = threadIdx.x >> 5;
    Run u;
    u.bt = (size_t)blockIdx.x * (32 * kRowWarps / STEP) + threadIdx.x / STEP;
    u.p = threadIdx.x % STEP;
    u.there = u.bt < (size_t)r.B * r.T;
    const uint32_t pieces = u.there ? D / N : 0;
    for (int e0 = 0; e0 < r.E; e0 += L) {
        const float gate = u.there && e0 + lane < r.E ? __ldg(G + u.bt * r.E + e0 + lane) : 0.f;
        int slot;
        uint32_t m = open_experts<L>(r.slot, u, r.E, e0, n, lane, slot);
        float mine = 0.f;                                   // lane e's dG
        while (any_left<L>(m)) {
            const bool one = m != 0;
            const int e = next_expert(m);
            const bool two = m != 0;
            const int f = next_expert(m);
            const size_t row = (size_t)__shfl_sync(0xffffffffu, slot, e, L) * D;
            const size_t row2 = (size_t)__shfl_sync(0xffffffffu, slot, f, L) * D;
            const float g = __shfl_sync(0xffffffffu, gate, e, L), g2 = __shfl_sync(0xffffffffu, gate, f, L);
            float dot = 0.f, dot2 = 0.f;
            for (uint32_t p0 = u.p; one && p0 < pieces; p0 += STEP * H) {     // (past 2^31 in the last step)
                P y[H], z[H], d[H];
#pragma unroll
                for (int i = 0; i < H; ++i)
                    if (p0 + STEP * i < pieces) {
                        const size_t at = (size_t)(p0 + STEP * i) * N;
                        d[i].load(dV + u.bt * D + at);
                        y[i].load(Y + row + at);
                        if (two) z[i].load(Y + row2 + at);
                    }
#pragma unroll
                for (int i = 0; i < H; ++i)
                    if (p0 + STEP * i < pieces) {
                        const size_t at = (size_t)(p0 + STEP * i) * N;
                        float o[N];
                        P q;
#pragma unroll
                        for (int k = 0; k < N; ++k) {
                            dot = fmaf(y[i].get(k), d[i].get(k), dot);
                            o[k] = g * d[i].get(k);
                        }
                        q.set(o);
                        q.store(dY + row + at);
                        if (two) {
#pragma unroll
                            for (int k = 0; k < N; ++k) {
                                dot2 = fmaf(z[i].get(k), d[i].get(k), dot2);
                                o[k] = g2 * d[i].get(k);
                            }
                            q.set(o);
                            q.store(dY + row2 + at);
                        }
                    }
            }
            dot = group_sum<L>(dot);
            dot2 = group_sum<L>(dot2);
            if constexpr (WARPS > 1) {                      // the same mask in every warp of the CTA
                __syncthreads();
                if (lane == 0) sums[0][warp] = dot, sums[1][warp] = dot2;
                __syncthreads();
                dot = dot2 = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) dot += sums[0][w], dot2 += sums[1][w];
            }
            if (one && lane == e) mine = dot;
            if (two && lane == f) mine = dot2;
        }
        if (u.there && e0 + lane < r.E && (WARPS == 1 || warp == 0)) dG[u.bt * r.E + e0 + lane] = mine;
    }
}

// Up to this many rows the gates' gradient takes four warps a row.
constexpr int kFewRows = 4096;

bool aligned_rows(std::initializer_list<const void*> ps, int D, int esz) {
    for (const void* p : ps)
        if (!fp8_on(p, 16)) return false;
    return D * (long long)esz % 16 == 0;
}
const dim3 kRowBlock(32 * kRowWarps);
// CTAs for `runs` groups of `lanes` lanes a row.
bool row_grid(const ExpertRows& r, long long runs, int lanes, dim3* grid) {
    const int per = 32 * kRowWarps / lanes;
    const long long ctas = ((long long)r.B * r.T * runs + per - 1) / per;
    *grid = dim3((unsigned)ctas);
    return ctas <= 0x7fffffffll;
}
// Lanes of a group that takes `pieces` pieces a row, `held` a lane at once.
int lanes_of(long long pieces, int held) { return pieces <= 8 * held ? 8 : pieces <= 16 * held ? 16 : 32; }
int runs_of(long long pieces, int held, int lanes) { return (int)((pieces + lanes * held - 1) / (lanes * held)); }
template <typename T, bool VEC>
long long pieces_of(int D) {
    return D / (VEC ? 16 / (int)sizeof(T) : 1);
}

template <typename T, bool VEC>
cudaError_t gather_v(const T* X, const ExpertRows& r, T* Xs, long long n, int D, cudaStream_t s) {
    const long long pieces = pieces_of<T, VEC>(D);
    const int lanes = lanes_of(pieces, kHeld<VEC>), runs = runs_of(pieces, kHeld<VEC>, lanes);
    dim3 grid;
    if (!row_grid(r, runs, lanes, &grid)) return cudaErrorNotSupported;
    auto k = lanes == 8 ? gather_kernel<T, VEC, 8> : lanes == 16 ? gather_kernel<T, VEC, 16> : gather_kernel<T, VEC, 32>;
    return launch_k(k, grid, kRowBlock, 0, s, X, r, Xs, n, D, runs);
}
template <typename T>
cudaError_t gather(const T* X, const ExpertRows& r, T* Xs, long long n, int D, cudaStream_t s) {
    return aligned_rows({X, Xs}, D, sizeof(T)) ? gather_v<T, true>(X, r, Xs, n, D, s) : gather_v<T, false>(X, r, Xs, n, D, s);
}
template <typename T>
cudaError_t gather_fp4(const T* X, const ExpertRows& r, const Fp4View& out, long long n, int D, cudaStream_t s) {
    auto k = aligned_rows({X}, D, sizeof(T)) ? gather_fp4_kernel<T, true> : gather_fp4_kernel<T, false>;
    const int nb = (int)fp4_blocks(D), runs = runs_of(2ll * nb, 1, kCodeLanes);
    dim3 grid;
    if (!row_grid(r, runs, kCodeLanes, &grid)) return cudaErrorNotSupported;
    return launch_k(k, grid, kRowBlock, 0, s, X, r, out, n, D, nb, runs);
}
template <typename T, typename TO, bool VEC>
cudaError_t combine_v(const T* Y, const ExpertRows& r, const float* G, TO* V, long long n, int D, cudaStream_t s) {
    const long long pieces = pieces_of<T, VEC>(D);
    const int lanes = lanes_of(pieces, kHeld<VEC>), runs = runs_of(pieces, kHeld<VEC>, lanes);
    dim3 grid;
    if (!row_grid(r, runs, lanes, &grid)) return cudaErrorNotSupported;
    auto k = lanes == 8    ? combine_kernel<T, TO, VEC, 8>
             : lanes == 16 ? combine_kernel<T, TO, VEC, 16>
                           : combine_kernel<T, TO, VEC, 32>;
    return launch_k(k, grid, kRowBlock, 0, s, Y, r, G, V, n, D, runs);
}
template <typename T, typename TO>
cudaError_t combine(const T* Y, const ExpertRows& r, const float* G, TO* V, long long n, int D, cudaStream_t s) {
    return aligned_rows({Y, V}, D, sizeof(T)) ? combine_v<T, TO, true>(Y, r, G, V, n, D, s)
                                              : combine_v<T, TO, false>(Y, r, G, V, n, D, s);
}
template <typename T, bool VEC>
cudaError_t combine_backward_v(const T* dV, const T* Y, const ExpertRows& r, const float* G, T* dY, float* dG, long long n,
                               int D, cudaStream_t s) {
    const int lanes = lanes_of(pieces_of<T, VEC>(D), kHeld<VEC>);
    const bool few = lanes == 32 && (long long)r.B * r.T <= kFewRows;
    dim3 grid;
    if (!row_grid(r, few ? kRowWarps : 1, lanes, &grid)) return cudaErrorNotSupported;
    auto k = few           ? combine_backward_kernel<T, VEC, 32, kRowWarps>
             : lanes == 8  ? combine_backward_kernel<T, VEC, 8, 1>
             : lanes == 16 ? combine_backward_kernel<T, VEC, 16, 1>
                           : combine_backward_kernel<T, VEC, 32, 1>;
    return launch_k(k, grid, kRowBlock, 0, s, dV, Y, r, G, dY, dG, n, D);
}
template <typename T>
cudaError_t combine_backward(const T* dV, const T* Y, const ExpertRows& r, const float* G, T* dY, float* dG, long long n,
                             int D, cudaStream_t s) {
    return aligned_rows({dV, Y, dY}, D, sizeof(T)) ? combine_backward_v<T, true>(dV, Y, r, G, dY, dG, n, D, s)
                                                   : combine_backward_v<T, false>(dV, Y, r, G, dY, dG, n, D, s);
}
bool rows_ok(const ExpertRows& r, long long n, int D) {
    return r.B >= 1 && r.T >= 1 && r.E >= 1 && (long long)r.B * r.T * r.E < (1ll << 31) && r.slot && n >= 0 && D >= 1;
}

}  // namespace

long long expert_sort_work(int B, int T, int E) {
    const long long TE = (long long)T * E;
    return sorts_at_once(B, TE) ? 0 : (kSortWarps + 1) * TE * sort_chunks(B, TE);
}

cudaError_t launch_expert_sort(const float* G, const ExpertRows& r, int* work, cudaStream_t s) {
    RM_HOST_BOUNDS(G && rows_ok(r, 0, 1) && r.offsets && r.source && fp8_on(r.tiles, 16));
    const int TE = r.T * r.E;
    if (sorts_at_once(r.B, TE))
        return launch_k(sort_small_kernel, dim3(1), dim3(kSortThreads), 0, s, G, TE, r);
    const unsigned ctas = (unsigned)((TE + kCols - 1) / kCols), chunks = (unsigned)sort_chunks(r.B, TE);
    int *totals = work, *counts = work + (size_t)chunks * TE;
    const cudaError_t e = launch_k(sort_count_kernel, dim3(ctas, chunks), dim3(kSortThreads), 0, s, G, r.B, TE, counts, totals);
    if (e != cudaSuccess) return e;
    return launch_k(sort_place_kernel, dim3(ctas + 1, chunks), dim3(kSortThreads), 0, s, G, TE, (const int*)counts,
                    (const int*)totals, r);
}

cudaError_t launch_expert_gather(const void* X, bool f32, const ExpertRows& r, void* Xs, long long n, int D,
                                 cudaStream_t s) {
    RM_HOST_BOUNDS(X && Xs && rows_ok(r, n, D));
    return f32 ? gather(static_cast<const float*>(X), r, static_cast<float*>(Xs), n, D, s)
               : gather(static_cast<const __nv_bfloat16*>(X), r, static_cast<__nv_bfloat16*>(Xs), n, D, s);
}

cudaError_t launch_fp4_expert_gather(const void* X, bool f32, const ExpertRows& r, const Fp4View& out, long long n, int D,
                                     cudaStream_t s) {
    RM_HOST_BOUNDS(X && rows_ok(r, n, D) && fp4_holds(out, D));
    return f32 ? gather_fp4(static_cast<const float*>(X), r, out, n, D, s)
               : gather_fp4(static_cast<const __nv_bfloat16*>(X), r, out, n, D, s);
}

cudaError_t launch_expert_combine(const void* Y, bool y_f32, const ExpertRows& r, const float* G, void* V, bool v_f32,
                                  long long n, int D, cudaStream_t s) {
    RM_HOST_BOUNDS((Y || n == 0) && V && rows_ok(r, n, D));
    using H = __nv_bfloat16;
    if (y_f32)
        return v_f32 ? combine(static_cast<const float*>(Y), r, G, static_cast<float*>(V), n, D, s)
                     : combine(static_cast<const float*>(Y), r, G, static_cast<H*>(V), n, D, s);
    return v_f32 ? combine(static_cast<const H*>(Y), r, G, static_cast<float*>(V), n, D, s)
                 : combine(static_cast<const H*>(Y), r, G, static_cast<H*>(V), n, D, s);
}

cudaError_t launch_expert_combine_backward(const void* dV, const void* Y, bool f32, const ExpertRows& r, const float* G,
                                           void* dY, float* dG, long long n, int D, cudaStream_t s) {
    RM_HOST_BOUNDS(dV && (n == 0 || (Y && dY)) && dG && G && rows_ok(r, n, D));
    using H = __nv_bfloat16;
    return f32 ? combine_backward(static_cast<const float*>(dV), static_cast<const float*>(Y), r, G, static_cast<float*>(dY),
                                  dG, n, D, s)
               : combine_backward(static_cast<const H*>(dV), static_cast<const H*>(Y), r, G, static_cast<H*>(dY), dG, n, D, s);
}

}  // namespace rm
