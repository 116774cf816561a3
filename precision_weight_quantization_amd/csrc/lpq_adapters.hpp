// Low-rank adapters of many requests at once, beside a shared projection: forward and
// backward.
//
// Part of lpq_kernels.hip, which includes each part once, in this order: one
// translation unit.
#pragma once

namespace {

// Token t has adapter g (or none):  u = x[t] A_g^T,  y[t] = base[t] + s_g u B_g^T.  The tokens
// of an adapter are a run of rows of a plan (src: the token of a row), so that each tile of 16
// rows has one A and one B.  Four kinds of product:
//   shrink    U[row] = X[token] W_g^T             long contraction, `rank` results
//   expand    out[token] = in[token] + s_g U[row] W_g^T      contraction of `rank`
//   gradient  V_g^T X_g over the rows of g        contraction over tokens
//   transpose of A and B, for the backward pass's shrink and expand
// Measured (us of device time, in a trace; floors at a copy's 5.2 TB/s): 8192 tokens of 8 adapters, 9728 x 2560, rank 64: shrink
// 25 (8: its time is 8 for finding rows and the sums in LDS, 7 for x and 9 for A out of the caches), expand 88 (62: every XCD
// reads every adapter's B).  40 tokens of 32 adapters, 4096 x 2560, rank 16: 4.2 and 5.5, latency.  Gradients, 4099 tokens of
// 4, 1024 x 2560, rank 24: transpose 3.3, shrinks 13.8, planes 4.0, gradients 19.5 and their sum 6.0, expand 14.6, together 61
// (14): transposes, planes and 12 MB of parts of 1.4 MB of gradients go through memory, in one or two steps of 32 rows a wave.
// U is FP32.  It meets the BF16 matrix instruction as the sum of three BF16 numbers, which is all 24
// bits.  Products of BF16 numbers are exact in FP32, so every sum is an FP32 one.  An infinity meets the
// first of the three alone: the others may be zeros or of the other sign, which would make a NaN of it.
// (Two numbers, 16 bits: 110 us a forward call of the first case; three 110; with the first's sums apart 112.)
// Memory is the floor: x, base and y once, and the adapters' factors.
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// v_mfma_f32_16x16x32_bf16: lane l holds row l % 16 and 8 consecutive elements of the
// contraction, from 8 * (l / 16) on, of both operands; result register r of lane l is row 4 *
// (l / 16) + r of the first, row l % 16 of the second.
__device__ __forceinline__ v4f mfma_bf16(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// The first 8 bits of each of N FP32 numbers as BF16 numbers; they keep what is left, which takes two more
// of these.  FIRST: nothing is left of an infinity or a NaN (infinity - infinity would be a NaN).  Cut and not
// rounded, so that no finite number becomes an infinity.
template <bool FIRST, int N>
__device__ __forceinline__ void take_bf16(float (&f)[N], uint32_t (&w)[N / 2]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        w[i / 2] = __builtin_amdgcn_perm(__float_as_uint(f[i + 1]), __float_as_uint(f[i]), 0x07060302u);
        f[i] -= bf16_lo(w[i / 2]);
        f[i + 1] -= bf16_hi(w[i / 2]);
        if constexpr (FIRST) {
            f[i] = __builtin_isfinite(f[i]) ? f[i] : 0.0f;
            f[i + 1] = __builtin_isfinite(f[i + 1]) ? f[i + 1] : 0.0f;
        }
    }
}
template <bool FIRST>
__device__ __forceinline__ v4u take_bf16(float (&f)[8]) {
    uint32_t w[4];
    take_bf16<FIRST>(f, w);
    return v4u{w[0], w[1], w[2], w[3]};
}
// Infinities and NaN among 8 BF16 numbers as zeros.
__device__ __forceinline__ v4u finite_bf16(v4u v) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t lo = (v[i] & 0x7f80u) == 0x7f80u ? 0u : 0xffffu, hi = (v[i] & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u;
        v[i] &= lo | hi;
    }
    return v;
}

// An infinity or a NaN among them.
template <int N>
__device__ __forceinline__ bool not_finite(const v4f (&c)[N]) {
    float bad = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) bad = __builtin_fmaf(c[i][j], 0.0f, bad);
    return bad != bad;
}

// The token of a row; -1 where a plan that was not made for these tokens holds something else.
__device__ __forceinline__ int64_t token_of(const int32_t* src, int64_t row, int64_t tokens) {
    const int64_t t = src[row];
    return (uint64_t)t < (uint64_t)tokens ? t : -1;
}

struct ShrinkArgs {
    const uint16_t *x, *w;    // [tokens, K], [groups, rank, K]
    float* u;                 // [splits, capacity, rank]: the sums of parts of k
    int32_t K;
    int32_t splits, each;     // each: elements of a part, a multiple of 32
    int32_t blocks;           // workgroups
};
// The backward pass's two shrinks are one launch: the workgroups of the first, then of the second.
struct ShrinkPair {
    ShrinkArgs a[2];
    const int32_t* src;       // [capacity]
    int64_t tokens;
    int32_t rank;
};

// A workgroup takes 16 * MT rows of a group, all of the rank (NT tiles) and one part of k, which
// its waves share out in steps of 32; their results are added through LDS.
constexpr int kShrinkWaves = 8;
template <int NT, int MT, int U>   // U steps' loads go out together
__global__ __launch_bounds__(64 * kShrinkWaves) void k_adapter_shrink(ShrinkPair P, Routing R) {
    constexpr int W = kShrinkWaves;
    __shared__ v4f part[W][NT * MT][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const bool second = (int)blockIdx.x >= P.a[0].blocks;
    const ShrinkArgs& A = P.a[second];
    const int block = (int)blockIdx.x - (second ? P.a[0].blocks : 0);
    const RouteMap map(R, RowTiles<16 * MT>{});
    const int v = block / A.splits, split = block % A.splits;
    if (v >= map.total) return;   // the whole workgroup
    RouteRun run;
    int within;
    const int group = map.find(R, v, run, within);
    const int first = run.first + within * 16 * MT, last = min(first + 16 * MT, run.last);
    const uint16_t *x[MT], *w[NT];
    bool in_m[MT], in_n[NT];
    v4f c[NT][MT];
#pragma unroll
    for (int i = 0; i < MT; i++) {
        const int row = first + i * 16 + r;
        const int64_t t = row < last ? token_of(P.src, row, P.tokens) : -1;
        in_m[i] = t >= 0;
        x[i] = A.x + (in_m[i] ? t : 0) * A.K;
    }
#pragma unroll
    for (int j = 0; j < NT; j++) {
        in_n[j] = j * 16 + r < P.rank;
        w[j] = A.w + ((int64_t)group * P.rank + (in_n[j] ? j * 16 + r : 0)) * A.K;
#pragma unroll
        for (int i = 0; i < MT; i++) c[j][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int steps = (min(A.each, A.K - split * A.each) + 31) / 32, share = (steps + W - 1) / W;
    const int begin = split * A.each + wave * share * 32, end = min(min(begin + share * 32, split * A.each + A.each), A.K);
    for (int k0 = begin; k0 < end; k0 += 32 * U) {
        v4u fx[U][MT], fw[U][NT];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int k = k0 + u * 32 + 8 * g;
            const bool in = k < end;   // K % 8 == 0
#pragma unroll
            for (int i = 0; i < MT; i++) fx[u][i] = in && in_m[i] ? load<false>(reinterpret_cast<const v4u*>(x[i] + k)) : v4u{};
#pragma unroll
            for (int j = 0; j < NT; j++) fw[u][j] = in && in_n[j] ? load<false>(reinterpret_cast<const v4u*>(w[j] + k)) : v4u{};
        }
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int i = 0; i < MT; i++) c[j][i] = mfma_bf16(fw[u][j], fx[u][i], c[j][i]);
    }
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
        for (int i = 0; i < MT; i++) part[wave][j * MT + i][lane] = c[j][i];
    __syncthreads();
    for (int y = wave; y < NT * MT; y += W) {
        v4f s = part[0][y][lane];
#pragma unroll
        for (int i = 1; i < W; i++) s += part[i][y][lane];
        const int row = first + y % MT * 16 + r, j = y / MT * 16 + g * 4;   // 4 results: rank % 8 == 0
        if (row < last && j < P.rank) {
            if (!in_m[MT == 1 ? 0 : y % MT]) s = v4f{0.0f, 0.0f, 0.0f, 0.0f};   // padding, whatever the factor
            store<false>(reinterpret_cast<v4f*>(A.u + ((int64_t)split * R.capacity + row) * P.rank + j), s);
        }
    }
}

struct ExpandArgs {
    const float* u;           // [splits, capacity, rank]
    const uint16_t* w;        // [groups, N, rank]
    const float* scale;       // [groups], NULL: ones
    const int32_t *rows, *src;
    const uint16_t* in;       // [tokens, N], NULL: zeros
    uint16_t* out;            // [tokens, N], may be `in`
    int64_t tokens;
    int32_t N, rank, splits;
    int32_t chunks;           // parts of 64 * IT columns in N
    int32_t copy_tiles;       // of 64 tokens: the first ones look for tokens without a row
};

// s_g u of a lane's row, 8 elements of the rank a step, as three BF16 numbers each.
template <int STEPS>
struct ExpandRow {
    int64_t at;        // the row's first element in `in` and `out`
    bool in;           // there is a token
    v4u hi[STEPS], mid[STEPS], lo[STEPS];
};
template <int STEPS>
__device__ __forceinline__ ExpandRow<STEPS> expand_row(const ExpandArgs& A, const Routing& R, int group, int row, int last, int g) {
    ExpandRow<STEPS> e;
    const int64_t t = row < last ? token_of(A.src, row, A.tokens) : -1;
    e.in = t >= 0;
    e.at = (e.in ? t : 0) * A.N;
    const float scale = A.scale ? A.scale[group] : 1.0f;
#pragma unroll
    for (int s = 0; s < STEPS; s++) {
        float f[8];
        const int j = s * 32 + 8 * g;
        v4f a{}, b{};
        const bool there = e.in && j < A.rank;
        if (there) {
            for (int i = 0; i < A.splits; i++) {
                const v4f* p = reinterpret_cast<const v4f*>(A.u + ((int64_t)i * R.capacity + row) * A.rank + j);
                a += load<false>(p);
                b += load<false>(p + 1);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {   // past the rank zeros whatever the scale
            f[i] = there ? a[i] * scale : 0.0f;
            f[4 + i] = there ? b[i] * scale : 0.0f;
        }
        e.hi[s] = take_bf16<true>(f);
        e.mid[s] = take_bf16<false>(f);
        e.lo[s] = take_bf16<false>(f);
    }
    return e;
}
// 64 columns from n0 on: a lane's are the 8 from n0 + 32 * h + 8 * g on, h = 0 and 1.  Row i of the first
// operand of instruction p (of 4) is column 32 * (p / 2) + 8 * (i / 4) + 4 * (p % 2) + i % 4.
__device__ __forceinline__ int expand_col(int p, int i) { return 32 * (p >> 1) + 8 * (i >> 2) + 4 * (p & 1) + (i & 3); }
struct Base {
    v4u h[2];
};
template <int STEPS>
__device__ __forceinline__ Base expand_base(const ExpandArgs& A, const ExpandRow<STEPS>& e, int n0, int n_last, int g) {
    Base b;
#pragma unroll
    for (int h = 0; h < 2; h++) {   // N % 8 == 0
        const int n = n0 + 32 * h + 8 * g;
        b.h[h] = e.in && A.in && n < n_last ? load<false>(reinterpret_cast<const v4u*>(A.in + e.at + n)) : v4u{};
    }
    return b;
}
// weight(p, s): 8 elements of the rank of the lane's row of instruction p.
template <int STEPS, typename F>
__device__ __forceinline__ void expand_64(const ExpandArgs& A, const ExpandRow<STEPS>& e, const Base& base, int n0, int n_last, int g,
                                          F&& weight) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
        v4f first[2], rest[2];   // sums with the first number, with the others
#pragma unroll
        for (int q = 0; q < 2; q++) {
            first[q] = rest[q] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < STEPS; s++) {
                const v4u w = weight(2 * h + q, s);
                rest[q] = mfma_bf16(w, e.lo[s], rest[q]);
                rest[q] = mfma_bf16(w, e.mid[s], rest[q]);
                first[q] = mfma_bf16(w, e.hi[s], first[q]);
            }
        }
        const int n = n0 + 32 * h + 8 * g;
        if (!e.in || n >= n_last) continue;
        const F8 f = widen8(base.h[h]);
        v4u o;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float d[2];
#pragma unroll
            for (int x = 0; x < 2; x++) {
                const float a = first[i / 2][(i & 1) * 2 + x], b = rest[i / 2][(i & 1) * 2 + x];
                d[x] = f.x[2 * i + x] + (__builtin_isfinite(a) ? a + b : a);
            }
            o[i] = bf16x2(d[0], d[1]);
        }
        store<false>(reinterpret_cast<v4u*>(A.out + e.at + n), o);
    }
}
// Tokens without a row: a wave looks at 64 of them and copies `in`.
__device__ __forceinline__ void expand_copy(const ExpandArgs& A, const Routing& R, int v, int n_first, int n_last) {
    const int lane = threadIdx.x & 63;
    const int64_t t0 = (int64_t)v * 64;
    const bool none = t0 + lane < A.tokens && (uint32_t)A.rows[t0 + lane] >= (uint32_t)R.capacity;
    for (uint64_t m = __builtin_amdgcn_ballot_w64(none); m; m &= m - 1) {
        const int64_t at = (t0 + __builtin_ctzll(m)) * A.N;
        for (int n = n_first + lane * 8; n < n_last; n += 64 * 8)
            store<false>(reinterpret_cast<v4u*>(A.out + at + n), A.in ? load<false>(reinterpret_cast<const v4u*>(A.in + at + n)) : v4u{});
    }
}

// Few rows a group: a wave by itself takes 16 of them and 64 * IT columns, weights from memory.
constexpr int kExpandWaves = 4;
template <int STEPS, int IT>
__global__ __launch_bounds__(64 * kExpandWaves) void k_adapter_expand(ExpandArgs A, Routing R) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int chunk = (int)(blockIdx.x % A.chunks);
    int v = (int)(blockIdx.x / A.chunks) * kExpandWaves + wave;
    const int n_first = chunk * 64 * IT, n_last = min(n_first + 64 * IT, A.N);
    if (v < A.copy_tiles) return expand_copy(A, R, v, n_first, n_last);
    v -= A.copy_tiles;
    const RouteMap map(R, RowTiles<16>{});
    if (v >= map.total) return;
    RouteRun run;
    int within;
    const int group = map.find(R, v, run, within);
    const ExpandRow<STEPS> e = expand_row<STEPS>(A, R, group, run.first + within * 16 + r, run.last, g);
    const uint16_t* w = A.w + (int64_t)group * A.N * A.rank;
#pragma unroll
    for (int it = 0; it < IT; it++) {
        const int n0 = n_first + 64 * it;
        const Base base = expand_base(A, e, n0, n_last, g);
        v4u fw[4][STEPS];
#pragma unroll
        for (int p = 0; p < 4; p++) {
            const int col = n0 + expand_col(p, r);
#pragma unroll
            for (int s = 0; s < STEPS; s++) {
                const int j = s * 32 + 8 * g;
                fw[p][s] = col < n_last && j < A.rank ? load<false>(reinterpret_cast<const v4u*>(w + (int64_t)col * A.rank + j)) : v4u{};
            }
        }
        expand_64(A, e, base, n0, n_last, g, [&](int p, int s) { return fw[p][s]; });
    }
}

// Many rows a group: a workgroup takes 64 rows, 16 a wave, and kTileColumns columns, 64 at a time.
// Their weights (one piece of memory) go through LDS for all four waves, the next 64 columns' while
// these are computed, with `in` two steps ahead.  (Each wave loading weights from the caches: 130 us
// instead of 86 at 8192 x 9728, rank 64, of which 45 were those loads; both with u as two numbers.)  A row of weights takes an odd number of
// 16-byte pieces in LDS, so that 16 rows' same piece lie in 16 different bank groups.
constexpr int kTileColumns = 512;
template <int STEPS>
__global__ __launch_bounds__(64 * kExpandWaves) void k_adapter_expand_tile(ExpandArgs A, Routing R) {
    constexpr int T = 64 * kExpandWaves, Q = STEPS;   // pieces of 64 columns for a thread: 64 * rank / 8 / 256, at most
    __shared__ v4u tile[2][64 * (STEPS * 4 + 1)];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int chunk = (int)(blockIdx.x % A.chunks);
    int v = (int)(blockIdx.x / A.chunks);
    const int n_first = chunk * kTileColumns, n_last = min(n_first + kTileColumns, A.N);
    if (v < A.copy_tiles) return expand_copy(A, R, v * kExpandWaves + wave, n_first, n_last);   // 256 tokens a workgroup
    v -= A.copy_tiles;
    const RouteMap map(R, RowTiles<64>{});
    if (v >= map.total) return;   // the whole workgroup
    RouteRun run;
    int within;
    const int group = map.find(R, v, run, within);
    const int pieces = A.rank / 8, pitch = pieces | 1;
    const v4u* w = reinterpret_cast<const v4u*>(A.w + ((int64_t)group * A.N + n_first) * A.rank);
    v4u next[Q];
    auto fetch = [&](int n0) {   // the weights of 64 columns from n0 on, in the order of memory
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const int i = q * T + threadIdx.x;
            next[q] = i < min(64, n_last - n0) * pieces ? load<false>(w + (int64_t)(n0 - n_first) * pieces + i) : v4u{};
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const int i = q * T + threadIdx.x, row = i / pieces;
            if (row < 64) tile[buf][row * pitch + (i - row * pieces)] = next[q];
        }
    };
    fetch(n_first);
    const ExpandRow<STEPS> e = expand_row<STEPS>(A, R, group, run.first + within * 64 + wave * 16 + r, run.last, g);
    Base base[2] = {expand_base(A, e, n_first, n_last, g), expand_base(A, e, n_first + 64, n_last, g)};
    put(0);
    int buf = 0;
    for (int n0 = n_first; n0 < n_last; n0 += 64, buf ^= 1) {
        __syncthreads();   // this step's weights are there, the other buffer is read
        if (n0 + 64 < n_last) fetch(n0 + 64);
        const Base now = base[0];
        base[0] = base[1];
        base[1] = expand_base(A, e, n0 + 128, n_last, g);
        expand_64(A, e, now, n0, n_last, g, [&](int p, int s) {
            const int j = s * 4 + g;
            return j < pieces ? tile[buf][expand_col(p, r) * pitch + j] : v4u{};
        });
        if (n0 + 64 < n_last) put(buf ^ 1);
    }
}

// out[g] = in[g]^T: [groups, M, N] to [groups, N, M] of 16-bit elements (M and N multiples of 8), 64 x
// 64 at a time through LDS.  A and B in one launch.
struct AdapterTransposeArgs {
    const uint16_t* in;
    uint16_t* out;
    int32_t M, N, tiles_m, tiles_n;
    int32_t blocks;
};
struct AdapterTransposePair {
    AdapterTransposeArgs a[2];
};
__global__ __launch_bounds__(256) void k_adapter_transpose(AdapterTransposePair P) {
    __shared__ uint16_t tile[64][66];   // an odd number of words a row shifts the banks
    const bool second = (int)blockIdx.x >= P.a[0].blocks;
    const AdapterTransposeArgs& A = P.a[second];
    const int block = (int)blockIdx.x - (second ? P.a[0].blocks : 0);
    const int per = A.tiles_m * A.tiles_n, group = block / per, in_group = block - group * per;
    const int m0 = in_group / A.tiles_n * 64, n0 = in_group % A.tiles_n * 64;
    const int64_t at = (int64_t)group * A.M * A.N;
    const int x = (threadIdx.x & 7) * 8;
#pragma unroll
    for (int y = threadIdx.x >> 3; y < 64; y += 32) {
        if (m0 + y >= A.M || n0 + x >= A.N) continue;
        const v4u v = load<false>(reinterpret_cast<const v4u*>(A.in + at + (int64_t)(m0 + y) * A.N + n0 + x));
#pragma unroll
        for (int i = 0; i < 4; i++) *reinterpret_cast<uint32_t*>(&tile[y][x + 2 * i]) = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int y = threadIdx.x >> 3; y < 64; y += 32) {
        if (n0 + y >= A.N || m0 + x >= A.M) continue;
        v4u v;
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = tile[x + 2 * i][y] | (uint32_t)tile[x + 2 * i + 1][y] << 16;
        store<false>(reinterpret_cast<v4u*>(A.out + at + (int64_t)(n0 + y) * A.M + m0 + x), v);
    }
}

// The sums of u's parts as three BF16 numbers each, transposed: [3, rank, pitch], so that the
// gradients' contraction is contiguous.  Columns of no row are zeros.
struct AdapterPlanesArgs {
    const float* u[2];
    uint16_t* planes[2];
    int32_t parts[2];
    int32_t rank, pitch;      // pitch: rows of the plan and 32 more, a multiple of 64
};
__global__ __launch_bounds__(256) void k_adapter_planes(AdapterPlanesArgs A, Routing R) {
    __shared__ float tile[16][65];
    const int which = (int)blockIdx.z, r0 = (int)blockIdx.x * 64, j0 = (int)blockIdx.y * 16;
    const int first = wave_run(R, 0).first, last = wave_run(R, R.groups - 1).last;
    const float* u = A.u[which];
    {
        const int j = threadIdx.x & 15;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int y = (threadIdx.x >> 4) + 16 * i, row = r0 + y;
            float f = 0.0f;
            if (row >= first && row < last && j0 + j < A.rank)
                for (int p = 0; p < A.parts[which]; p++) f += load<false>(u + ((int64_t)p * R.capacity + row) * A.rank + j0 + j);
            tile[j][y] = f;
        }
    }
    __syncthreads();
    const int j = threadIdx.x >> 4, x = (threadIdx.x & 15) * 4;
    if (j0 + j >= A.rank) return;
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = tile[j][x + i];
#pragma unroll
    for (int s = 0; s < 3; s++) {
        uint32_t w[2];
        if (s == 0) take_bf16<true>(f, w);
        else take_bf16<false>(f, w);
        store<false>(reinterpret_cast<v2u*>(A.planes[which] + ((int64_t)s * A.rank + j0 + j) * A.pitch + r0 + x), v2u{w[0], w[1]});
    }
}

struct AdapterGradArgs {
    const uint16_t* x;        // [tokens, C]
    const uint16_t* planes;   // [3, rank, pitch]
    float* out;               // [splits, groups, rank, C] or, rank last, [splits, groups, C, rank]
    int32_t C;
    int32_t splits, tiles;    // parts of a group's rows; 128-column tiles
    int32_t rank_last, accumulate;
    int32_t blocks;
};
struct AdapterGradPair {
    AdapterGradArgs a[2];     // of A and of B, in one launch
    const float* scale;       // [groups], NULL: ones
    const int32_t* src;
    int64_t tokens;
    int32_t rank, pitch;
    int32_t rank_tiles;       // 64-element pieces of the rank
};

// out[g][j][c] = s_g * sum over the rows of g of v[row][j] x[token][c]: a workgroup takes 128
// columns, up to 64 elements of the rank and one part of the group's rows, which its waves share
// out in steps of 32; their sums are added through LDS, in a fixed order.  A lane loads 8 x 8
// pieces of x, 8 rows by 8 columns; column p of all pieces makes the second operand of one
// instruction: its row l % 16 is column 8 * (l % 16) + p.
constexpr int kGradWaves = 4;
template <int JT>
__global__ __launch_bounds__(64 * kGradWaves, 2) void k_adapter_grad(AdapterGradPair P, Routing R) {
    constexpr int W = kGradWaves;
    __shared__ v4f part[W / 2][JT][8][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const bool second = (int)blockIdx.x >= P.a[0].blocks;
    const AdapterGradArgs& A = P.a[second];
    int b = (int)blockIdx.x - (second ? P.a[0].blocks : 0);
    const int tile = b % A.tiles;
    b /= A.tiles;
    const int piece = b % P.rank_tiles;
    b /= P.rank_tiles;
    const int split = b % A.splits, group = b / A.splits;
    const RouteRun run = wave_run(R, group);
    const int j0 = piece * 64, col = tile * 128 + 8 * r;
    const bool in_c = col < A.C;   // C % 8 == 0
    // A part without a token adds nothing, whatever the scale: a group's tokens are its first rows.
    const int earliest = run.first + split * W * 32;
    const bool any = earliest < run.last && token_of(P.src, earliest, P.tokens) >= 0;
    const float scale = !any ? 0.0f : P.scale ? P.scale[group] : 1.0f;
    v4f c[JT][8];
    auto sums = [&](auto rest_finite) {
        constexpr bool REST_FINITE = decltype(rest_finite)::value;   // infinities and NaN of x meet the first plane alone
#pragma unroll
        for (int j = 0; j < JT; j++)
#pragma unroll
            for (int p = 0; p < 8; p++) c[j][p] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int row0 = run.first + (split * W + wave) * 32; row0 < run.last; row0 += A.splits * W * 32) {
            v4u x[8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const int row = row0 + 8 * g + i;
                const int64_t t = row < run.last ? token_of(P.src, row, P.tokens) : -1;
                x[i] = t >= 0 && in_c ? load<false>(reinterpret_cast<const v4u*>(A.x + t * A.C + col)) : v4u{};
            }
            v4u v[JT][3];
#pragma unroll
            for (int j = 0; j < JT; j++)
#pragma unroll
                for (int s = 0; s < 3; s++) {
                    v[j][s] = v4u{};
                    if (j0 + j * 16 + r < P.rank)   // a group begins at any row: 2-byte alignment
                        __builtin_memcpy(&v[j][s], A.planes + ((int64_t)s * P.rank + j0 + j * 16 + r) * P.pitch + row0 + 8 * g, 16);
                }
            if (row0 + 32 > run.last) {   // the next group's rows: zeros of x alone would not keep its infinities and NaN out
                const int kept = run.last - row0 - 8 * g;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t mask = 2 * i + 1 < kept ? ~0u : 2 * i < kept ? 0xffffu : 0u;
#pragma unroll
                    for (int j = 0; j < JT; j++)
#pragma unroll
                        for (int s = 0; s < 3; s++) v[j][s][i] &= mask;
                }
            }
#pragma unroll
            for (int p = 0; p < 8; p++) {
                const v4u xc = piece_column(x, p), xf = REST_FINITE ? finite_bf16(xc) : xc;
#pragma unroll
                for (int j = 0; j < JT; j++)
#pragma unroll
                    for (int s = 2; s >= 0; s--) c[j][p] = mfma_bf16(v[j][s], s ? xf : xc, c[j][p]);
            }
        }
    };
    sums(std::false_type{});
    bool bad = false;
#pragma unroll
    for (int j = 0; j < JT; j++) bad |= not_finite(c[j]);
    if (any_lane(bad)) sums(std::true_type{});   // the whole wave, once more
    // two waves' sums to the other two, theirs to all four: half the LDS of all at once, so that two
    // workgroups fit a CU with 64 elements of the rank
    auto put = [&](int to) {
#pragma unroll
        for (int j = 0; j < JT; j++)
#pragma unroll
            for (int p = 0; p < 8; p++) part[to][j][p][lane] = c[j][p];
    };
    if (wave >= W / 2) put(wave - W / 2);
    __syncthreads();
    if (wave < W / 2) {
#pragma unroll
        for (int j = 0; j < JT; j++)
#pragma unroll
            for (int p = 0; p < 8; p++) c[j][p] += part[wave][j][p][lane];
        put(wave);
    }
    __syncthreads();
    // a wave finishes every 4th tile of the rank: for each of its lane's 4 elements 8 neighbouring columns
    float* out = A.out + ((int64_t)split * R.groups + group) * P.rank * A.C;
    for (int j = wave; j < JT; j += W) {
        v4f s[8];
#pragma unroll
        for (int p = 0; p < 8; p++) s[p] = (part[0][j][p][lane] + part[1][j][p][lane]) * scale;
        const int at = j0 + j * 16 + 4 * g;   // 4 elements of the rank: rank % 8 == 0
        if (!in_c || at >= P.rank) continue;
        if (A.rank_last) {
#pragma unroll
            for (int p = 0; p < 8; p++) {
                v4f* to = reinterpret_cast<v4f*>(out + (int64_t)(col + p) * P.rank + at);
                store<false>(to, A.accumulate ? load<false>(to) + s[p] : s[p]);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                v4f* to = reinterpret_cast<v4f*>(out + (int64_t)(at + q) * A.C + col);
                const v4f lo{s[0][q], s[1][q], s[2][q], s[3][q]}, hi{s[4][q], s[5][q], s[6][q], s[7][q]};
                store<false>(to, A.accumulate ? load<false>(to) + lo : lo);
                store<false>(to + 1, A.accumulate ? load<false>(to + 1) + hi : hi);
            }
        }
    }
}

// out (+)= the sum of `parts` arrays of n elements (n % 4 == 0), in their order.
struct AdapterSumArgs {
    const float* in[2];
    float* out[2];
    int64_t n[2];
    int32_t parts[2];
    int32_t blocks, accumulate;   // blocks: of the first
};
__global__ __launch_bounds__(256) void k_adapter_sum(AdapterSumArgs A) {
    const int second = (int)blockIdx.x >= A.blocks;
    const int64_t n = A.n[second], i = ((int64_t)((int)blockIdx.x - (second ? A.blocks : 0)) * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const float* in = A.in[second] + i;
    v4f s = load<false>(reinterpret_cast<const v4f*>(in));
    for (int p = 1; p < A.parts[second]; p++) s += load<false>(reinterpret_cast<const v4f*>(in + p * n));
    v4f* to = reinterpret_cast<v4f*>(A.out[second] + i);
    store<false>(to, A.accumulate ? load<false>(to) + s : s);
}

}  // namespace
