// Rows ordered by the weight that they go to: the plan, the gather (quantizing on
// the way), and the weighted combination with its gradients.
//
// Part of lpq_kernels.hip, which includes each part once, in this order: one
// translation unit.
#pragma once

namespace {

constexpr int kRouteMaxGroups = 1024;

// ---------------------------------------------------------------------------
// Plan: a stable counting sort.  Pair p (token p / k, slot p % k) of group g goes to
//   row = off[g] + number of pairs before p with the same group,
//   off[g + 1] = off[g] + ceil(count[g] / align) * align.
// A workgroup takes a run of pairs.  Up to kPlanOne pairs one workgroup does all;
// above, a first launch counts each run's pairs by group and the second finds the
// offsets from all the counts by itself (every workgroup the same) and places its
// run.  Bound by latency, a few barriers and round trips to memory: 65536 pairs of 128 groups take 5.0 and 7.6
// us, 8 pairs of 64 groups 3.4.
constexpr int kPlanThreads = 1024, kPlanOne = 4096, kPlanMaxRuns = 256;

struct PlanArgs {
    const void* ids;
    int64_t pairs, run;               // run: pairs of a workgroup, a multiple of kPlanThreads
    int32_t groups, align;
    int32_t *offsets, *rows, *src;    // [groups + 1], [pairs], [capacity]
    int64_t capacity;
    int32_t* counts;                  // [runs, groups], NULL for one run
};

// The group of pair p; `groups` for an index outside [0, groups).
template <typename Id>
__device__ __forceinline__ uint32_t plan_group(const PlanArgs& A, int64_t p) {
    const int64_t id = (int64_t)load<false>(static_cast<const Id*>(A.ids) + p);
    return (uint64_t)id < (uint64_t)A.groups ? (uint32_t)id : (uint32_t)A.groups;
}

template <typename Id>
__device__ __forceinline__ void plan_count(const PlanArgs& A, int64_t first, int64_t last, int* count) {
    for (int64_t p = first + threadIdx.x; p < last; p += kPlanThreads) {
        const uint32_t g = plan_group<Id>(A, p);
        if (g < (uint32_t)A.groups) atomicAdd(count + g, 1);   // whole numbers: any order
    }
}

template <typename Id>
__global__ __launch_bounds__(kPlanThreads) void k_route_count(PlanArgs A) {
    __shared__ int count[kRouteMaxGroups];
    const int t = threadIdx.x;
    if (t < A.groups) count[t] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * A.run;
    plan_count<Id>(A, first, min(first + A.run, A.pairs), count);
    __syncthreads();
    if (t < A.groups) A.counts[(int64_t)blockIdx.x * A.groups + t] = count[t];
}

template <typename Id>
__global__ __launch_bounds__(kPlanThreads) void k_route_place(PlanArgs A) {
    constexpr int W = kPlanThreads / 64;
    __shared__ int total[kRouteMaxGroups], next[kRouteMaxGroups];   // pairs of a group; the next row of one
    __shared__ uint8_t wave_count[W][kRouteMaxGroups];              // of the 64 pairs of each wave
    __shared__ int wave_sum[W];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, E = A.groups;
    const int64_t first = blockIdx.x * A.run, last = min(first + A.run, A.pairs);
    total[t] = 0;
    next[t] = 0;
    __syncthreads();
    if (A.counts) {
        const int n = (int)gridDim.x * E, mine = (int)blockIdx.x * E;
        for (int i = t; i < n; i += kPlanThreads) {
            const int c = A.counts[i], g = i % E;
            if (c) {
                atomicAdd(total + g, c);
                if (i < mine) atomicAdd(next + g, c);
            }
        }
    } else {
        plan_count<Id>(A, first, last, total);
    }
    __syncthreads();
    // offsets: a scan over the groups, one to a thread
    const int count = total[t], padded = t < E ? (count + A.align - 1) / A.align * A.align : 0;
    int sum = padded;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int v = __shfl_up(sum, d);
        if (lane >= d) sum += v;
    }
    if (lane == 63) wave_sum[wave] = sum;
    __syncthreads();
    int begin = sum - padded, end = 0;
#pragma unroll
    for (int w = 0; w < W; w++) {
        begin += w < wave ? wave_sum[w] : 0;
        end += wave_sum[w];
    }
    if (t < E) {
        next[t] += begin;
        if (blockIdx.x == 0) {
            A.offsets[t] = begin;
            if (t == 0) A.offsets[E] = end;
        }
        if (t % gridDim.x == blockIdx.x)   // the padding of this workgroup's share of the groups
            for (int r = begin + count; r < begin + padded; r++) A.src[r] = -1;
    }
    for (int64_t r = end + (int64_t)blockIdx.x * kPlanThreads + t; r < A.capacity; r += (int64_t)gridDim.x * kPlanThreads) A.src[r] = -1;

    const int bits = 32 - __builtin_clz(E);   // of a group or of E itself
    for (int64_t p0 = first; p0 < last; p0 += kPlanThreads) {
        const int64_t p = p0 + t;
        const bool in = p < last;
        const uint32_t g = in ? plan_group<Id>(A, p) : (uint32_t)E;
        uint64_t same = __builtin_amdgcn_ballot_w64(in);   // the wave's pairs of this pair's group
        for (int b = 0; b < bits; b++) {
            const bool one = g >> b & 1;
            const uint64_t set = __builtin_amdgcn_ballot_w64(one);
            same &= one ? set : ~set;
        }
        const int before = __builtin_popcountll(same & ((1ull << lane) - 1));
        const bool kept = in && g < (uint32_t)E;
        for (int i = t; i < W * kRouteMaxGroups / 4; i += kPlanThreads) reinterpret_cast<uint32_t*>(wave_count)[i] = 0;
        __syncthreads();
        if (kept && before == 0) wave_count[wave][g] = (uint8_t)__builtin_popcountll(same);
        __syncthreads();
        if (in) {
            int row = -1;
            if (kept) {
                row = next[g] + before;
                for (int w = 0; w < wave; w++) row += wave_count[w][g];
                A.src[row] = (int32_t)p;
            }
            A.rows[p] = row;
        }
        __syncthreads();
        if (t < E) {
            int n = 0;
#pragma unroll
            for (int w = 0; w < W; w++) n += wave_count[w][t];
            next[t] += n;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// A plan as the products read it.  Offsets are cut to the buffer, so that whatever they
// hold no row outside it is touched.
struct Routing {
    const int32_t* offsets;   // [groups + 1]
    int32_t groups;
    int32_t capacity;
};
struct RouteRun {
    int first, last;   // rows [first, last) of a group
};
__device__ __forceinline__ RouteRun route_run(const Routing& R, int from, int to) {
    const int first = min(max(from, 0), R.capacity), last = min(to, R.capacity);
    return {first, max(first, last)};
}
// Of a group of the lane's own.
__device__ __forceinline__ RouteRun lane_run(const Routing& R, int g) {
    return route_run(R, load<false>(R.offsets + g), load<false>(R.offsets + g + 1));
}
// Of one group for the whole wave.  Read through the scalar cache: a vector load would wait for
// all earlier ones of the wave, a product's next stages among them.
__device__ __forceinline__ int wave_offset(const Routing& R, int g) {
    return ((__attribute__((address_space(4))) const int32_t*)R.offsets)[__builtin_amdgcn_readfirstlane(g)];
}
__device__ __forceinline__ RouteRun wave_run(const Routing& R, int g) { return route_run(R, wave_offset(R, g), wave_offset(R, g + 1)); }

// Inclusive sums over the lanes, of numbers from 0 to `most` (up to 2^30) and cut to it.
__device__ __forceinline__ int wave_scan(int v, int most) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(v, d);
        if (lane >= d) v = min(v + up, most);
    }
    return v;
}

// No plan has as many as kRouteMost: 2^30 rows are 2^26 tiles of 16, and a group's last tile another 2^10.  Groups
// that overlap, which no plan has, would pass 32 bits and lead outside the buffers: so they are cut.
constexpr int kRouteMost = 1 << 28;

// Something that each group has a number of, end to end: tiles of its rows, or the cost of
// its contraction.  A lane counts for its share of the groups once; the group of a place is
// then found by a ballot and scalar loads of that lane's share, which is cheaper than a table
// in memory (another launch) or in LDS (which the products' stages fill).
template <typename Count>
struct RouteMap {
    Count count;                    // of a run of rows
    int share, upto, total;   // groups a lane; count up to and with its groups; of all
    __device__ __forceinline__ RouteMap(const Routing& R, Count c) : count(c) {
        const int lane = threadIdx.x & 63;
        share = (R.groups + 63) / 64;
        int mine = 0;
        for (int i = 0; i < share; i++)
            if (lane * share + i < R.groups) mine += count(lane_run(R, lane * share + i));
        upto = wave_scan(min(mine, kRouteMost), kRouteMost);
        total = __builtin_amdgcn_readlane(upto, 63);
    }
    // The group of place v < total, the same in every lane; its run, and the place within it.
    __device__ __forceinline__ int find(const Routing& R, int v, RouteRun& run, int& within) const {
        const int l = __builtin_ctzll(__builtin_amdgcn_ballot_w64(upto > v));
        within = v - (l ? __builtin_amdgcn_readlane(upto, l ? l - 1 : 0) : 0);
        int g = l * share, from = wave_offset(R, g);
        for (;; g++) {
            const int to = wave_offset(R, g + 1);
            run = route_run(R, from, to);
            const int n = count(run);
            if (within < n || g + 1 >= R.groups) return g;   // the second never holds for a plan
            within -= n;
            from = to;
        }
    }
};
template <int TM>
struct RowTiles {
    __device__ __forceinline__ int operator()(const RouteRun& r) const { return (r.last - r.first + TM - 1) / TM; }
};

// ---------------------------------------------------------------------------
// Work on whole rows in vectors of 8 elements, one to a thread: the workgroups
// behind the first `pad_groups` (see zero_rows) hold the tokens' vectors end to end.
constexpr int kRouteThreads = 256;

struct TokenVec {
    int64_t token;
    int col;
    bool in;
};
__device__ __forceinline__ TokenVec token_vec(int64_t block, int64_t tokens, int N) {
    const int vecs = N / 8;
    const int64_t at = block * kRouteThreads, token = at / vecs;        // uniform
    const uint32_t in_row = (uint32_t)(at - token * vecs) + threadIdx.x;
    const uint32_t more = in_row / (uint32_t)vecs;
    return {token + more, (int)(in_row - more * vecs) * 8, token + more < tokens};
}

// Rows without a pair: a workgroup looks at kPadRows of them and calls zero(row) with all its
// threads for each (a wave by itself for 64 rows: 62 us instead of 36 where 5,700 of 9,400
// rows of 14 KB are empty, the last waves').
constexpr int kPadRows = 16;
template <typename F>
__device__ __forceinline__ void zero_rows(const int32_t* src, int64_t capacity, F&& zero) {
    const int lane = threadIdx.x & 63;
    const int64_t r0 = (int64_t)blockIdx.x * kPadRows;
    const bool empty = lane < kPadRows && r0 + lane < capacity && src[r0 + lane] < 0;
    for (uint64_t m = __builtin_amdgcn_ballot_w64(empty); m; m &= m - 1) zero(r0 + __builtin_ctzll(m));
}
__device__ __forceinline__ void zero_bytes(uint8_t* p, int64_t n) {   // 16-byte aligned, whole 16 bytes
    for (int64_t i = threadIdx.x * 16; i < n; i += blockDim.x * 16) store<false>(reinterpret_cast<v4u*>(p + i), v4u{});
}

struct GatherArgs {
    const uint16_t* x;       // [tokens, N]
    const int32_t* rows;     // [tokens, k]
    const int32_t* src;      // [capacity]
    uint8_t *q, *e;          // BF16 rows or codes; scale bytes
    int64_t tokens, capacity;
    int32_t k, N;
    int32_t pad_groups;
};

enum RowFormat { ROW_BF16, ROW_FP8, ROW_FP4 };
template <int FORMAT>
__device__ __forceinline__ int64_t row_size(int64_t n) {
    return FORMAT == ROW_BF16 ? 2 * n : FORMAT == ROW_FP8 ? n : n / 2;
}

// out[row] = x[token] for each of the token's rows, as it is or quantized (once a
// token, and bit for bit as lpq_quantize_mxfp8 / lpq_quantize_mxfp4 do it); rows
// without a pair are zeros.  Memory is the floor: x once, every row once (8192 tokens of 2048 to 8 rows each in
// MXFP8, 182 MB: 30 us, 6.1 TB/s with part of it still in the memory-side cache; in BF16, 318 MB: 52 us).
template <int FORMAT>
__global__ __launch_bounds__(kRouteThreads) void k_route_gather(GatherArgs A) {
    if (blockIdx.x < (uint32_t)A.pad_groups) {
        zero_rows(A.src, A.capacity, [&](int64_t row) {
            const int64_t size = row_size<FORMAT>(A.N);
            zero_bytes(A.q + row * size, size);
            if constexpr (FORMAT != ROW_BF16)
                for (int i = threadIdx.x; i < A.N / 32; i += kRouteThreads) store_u8(A.e + row * (A.N / 32) + i, 0);
        });
        return;
    }
    const TokenVec v = token_vec(blockIdx.x - A.pad_groups, A.tokens, A.N);
    const v4u w = v.in ? load<false>(reinterpret_cast<const v4u*>(A.x + v.token * A.N + v.col)) : v4u{};
    v2u codes{};
    uint32_t byte = 0;
    if constexpr (FORMAT == ROW_FP8) {   // a quad of lanes is a block: N % 32 == 0
        const F8 f = widen8(w);
        byte = mx_scale_byte(quad_max(absmax8_f32(f)));
        codes = mx_encode8(f, ue8m0_operand(byte));
    } else if constexpr (FORMAT == ROW_FP4) {
        byte = mx4_byte<false>(quad_max(absmax8_bits(w)));
        codes.x = mx4_encode8(w, ue8m0_operand(byte));
    }
    if (!v.in) return;
    const int32_t* rows = A.rows + v.token * A.k;
    for (int j = 0; j < A.k; j++) {
        const int64_t row = rows[j];
        if ((uint64_t)row >= (uint64_t)A.capacity) continue;   // no such group here
        const int64_t at = row * A.N + v.col;
        if constexpr (FORMAT == ROW_BF16) store<false>(reinterpret_cast<v4u*>(A.q + 2 * at), w);
        else if constexpr (FORMAT == ROW_FP8) store<false>(reinterpret_cast<v2u*>(A.q + at), codes);
        else store<false>(reinterpret_cast<uint32_t*>(A.q + at / 2), codes.x);
        if constexpr (FORMAT != ROW_BF16)
            if ((threadIdx.x & 3) == 0) store_u8(A.e + at / 32, byte);
    }
}

struct CombineArgs {
    const uint16_t* y;          // [capacity, N]
    const int32_t* rows;        // [tokens, k]
    const float* weights;       // [tokens, k], NULL: ones
    const uint16_t* residual;   // [tokens, N], NULL: zeros
    uint16_t* out;              // [tokens, N]
    int64_t tokens, capacity;
    int32_t k, N;
};

// out[t] = BF16(residual[t] + sum over j of weights[t, j] * y[rows[t, j]]), the sum in
// FP32 in the order of j.  Memory is the floor; 8 rows' loads go out together (8192 tokens of 8 rows of 2048 with a
// residual, 336 MB: 67 us, 5.0 TB/s).
__global__ __launch_bounds__(kRouteThreads) void k_route_combine(CombineArgs A) {
    const TokenVec v = token_vec(blockIdx.x, A.tokens, A.N);
    if (!v.in) return;
    const int64_t at = v.token * A.N + v.col;
    F8 s = widen8(A.residual ? load<false>(reinterpret_cast<const v4u*>(A.residual + at)) : v4u{});
    const int32_t* rows = A.rows + v.token * A.k;
    const float* weights = A.weights ? A.weights + v.token * A.k : nullptr;
    for (int j0 = 0; j0 < A.k; j0 += 8) {
        v4u y[8];
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int64_t row = j0 + j < A.k ? rows[j0 + j] : -1;
            const bool in = (uint64_t)row < (uint64_t)A.capacity;
            y[j] = in ? load<false>(reinterpret_cast<const v4u*>(A.y + row * A.N + v.col)) : v4u{};
            w[j] = !in ? 0.0f : weights ? weights[j0 + j] : 1.0f;   // a slot without a row adds 0 * 0
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const F8 f = widen8(y[j]);
#pragma unroll
            for (int i = 0; i < 8; i++) s.x[i] = __builtin_fmaf(w[j], f.x[i], s.x[i]);
        }
    }
    store<false>(reinterpret_cast<v4u*>(A.out + at), v4u{bf16x2(s.x[0], s.x[1]), bf16x2(s.x[2], s.x[3]), bf16x2(s.x[4], s.x[5]),
                                                         bf16x2(s.x[6], s.x[7])});
}

struct CombineGradArgs {
    const uint16_t *dout, *y;   // [tokens, N], [capacity, N] (NULL: no dweights)
    const int32_t *rows, *src;
    const float* weights;       // NULL: ones
    uint16_t* dy;               // [capacity, N]
    float* dweights;            // [tokens, k], NULL: not wanted
    int64_t tokens, capacity;
    int32_t k, N;
    int32_t pad_groups;
};

// dy[rows[t, j]] = BF16(weights[t, j] * dout[t]), dweights[t, j] = dout[t] . y[rows[t, j]]
// in FP32 in a fixed order; rows without a pair are zeros.  TH threads to a token: dout
// is read once for 8 slots, each y and dy once (1237 tokens of 6 slots of 7168, half of them without a row, 206 MB with
// the empty rows: 36 us).
template <int TH>
__global__ __launch_bounds__(TH) void k_route_combine_grad(CombineGradArgs A) {
    if (blockIdx.x < (uint32_t)A.pad_groups) {
        zero_rows(A.src, A.capacity, [&](int64_t row) { zero_bytes(reinterpret_cast<uint8_t*>(A.dy + row * A.N), 2 * (int64_t)A.N); });
        return;
    }
    __shared__ float part[TH / 64][8];
    const int64_t token = blockIdx.x - (int64_t)A.pad_groups;
    const int32_t* rows = A.rows + token * A.k;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int j0 = 0; j0 < A.k; j0 += 8) {
        int64_t row[8];
        float w[8], dot[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            row[j] = j0 + j < A.k ? rows[j0 + j] : -1;
            if ((uint64_t)row[j] >= (uint64_t)A.capacity) row[j] = -1;
            w[j] = row[j] >= 0 && A.weights ? A.weights[token * A.k + j0 + j] : 1.0f;
            dot[j] = 0.0f;
        }
        for (int c = threadIdx.x * 8; c < A.N; c += TH * 8) {
            const F8 d = widen8(load<false>(reinterpret_cast<const v4u*>(A.dout + token * A.N + c)));
            v4u y[8];
            if (A.dweights) {
#pragma unroll
                for (int j = 0; j < 8; j++) y[j] = row[j] >= 0 ? load<false>(reinterpret_cast<const v4u*>(A.y + row[j] * A.N + c)) : v4u{};
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                if (row[j] < 0) continue;
                v4u o;
#pragma unroll
                for (int i = 0; i < 4; i++) o[i] = bf16x2(w[j] * d.x[2 * i], w[j] * d.x[2 * i + 1]);
                store<false>(reinterpret_cast<v4u*>(A.dy + row[j] * A.N + c), o);
                if (A.dweights) {
                    const F8 f = widen8(y[j]);
#pragma unroll
                    for (int i = 0; i < 8; i++) dot[j] = __builtin_fmaf(d.x[i], f.x[i], dot[j]);
                }
            }
        }
        if (!A.dweights) continue;
#pragma unroll
        for (int j = 0; j < 8; j++) {
#pragma unroll
            for (int x = 1; x < 64; x *= 2) dot[j] += __shfl_xor(dot[j], x);
            if (lane == 0) part[wave][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < 8 && j0 + (int)threadIdx.x < A.k) {
            float s = part[0][threadIdx.x];
#pragma unroll
            for (int i = 1; i < TH / 64; i++) s += part[i][threadIdx.x];
            A.dweights[token * A.k + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

}  // namespace
