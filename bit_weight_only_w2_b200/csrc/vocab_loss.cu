// The softmax cross entropy over a vocabulary: workspace, order of the launches, and the small kernels around the
// products of vocab_gemm.cuh.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "sm100_ptx.cuh"
#include "vocab_internal.h"

namespace lowbit {
namespace {

constexpr int64_t kTokensAtOnce = 16384;              // forward: tokens whose tiles' sums are kept at a time
// Backward: bytes of a term of G formed at a time. dX's sums are read and written once a piece: 4096 tokens against
// 131072 x 2560 took 6.33 ms with 256 MB, 6.44 with 128 and 6.75 with 64 (of one term).
constexpr int64_t kPieceBytes = int64_t(256) << 20;
// dW takes G as two bf16 values at the labels, where one of them makes up most of a row of dW and would show its rounding as
// much as the row's own (3 tokens: 3.5e-3 off in the norm, with two 1.9e-3), and where that rounding is the same for all
// tokens: with the mean over 900 labels (G near -1 / 900) all of dW came out 2.5e-3 too large and 3.0e-3 off in the norm, with
// two terms 1.66e-3, its own rounding. So of many tokens G's second term is kept for the blocks of 64 tokens by 256 rows that
// hold a label, marked beforehand: 16384 / rows more products for dW at most, and never twice as many (both gradients of
// 4096 tokens against 131072 x 2560: 6.26 ms without, 6.36 with). Up to this many tokens, where writing dW bounds the time
// anyway, all blocks have it.
constexpr int64_t kTwoTermTokens = 512;

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

template <class... P, class... A>
lowbit_status launch_after(void (*kernel)(P...), int64_t blocks, unsigned strips, int threads, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), strips, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (take_injected_failure(kInjectLaunch)) return LOWBIT_ERR_CUDA;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? LOWBIT_OK : LOWBIT_ERR_CUDA;
}

// lse and loss of each token from its tiles' (maximum, sum), joined in a fixed order: 8 tokens a block, 32 threads each
// (the parts of neighbouring tokens are neighbours), or one token a block where few tokens would leave most SMs idle:
// 16 tokens of 2048 parts take 17 us eight a block and 4 one a block. Whole calls, K = 128, one and eight a block: 512 tokens
// against 131072 rows 47.4 and 48.7 us, 1024 78.0 and 80.0, 2048 147.8 and 141.5; against 4096 rows 8.2 and 7.6, 9.0 and 8.2,
// 13.3 and 10.6. So one a block up to 1024 tokens, where it gains or loses least.
constexpr int kJoinThreads = 256;
__device__ __forceinline__ void join(float& R, float& S, float r, float s) {
    const float n = fmaxf(R, r);
    if (n == -INFINITY) {   // nothing yet: sums of zero, or a NaN
        S += s;
    } else {
        S = S * exp2f((R - n) * 1.4426950408889634f) + s * exp2f((r - n) * 1.4426950408889634f);
        R = n;
    }
}
template <int kJoinTokens>
__global__ void __launch_bounds__(kJoinThreads) loss_join_kernel(const float2* __restrict__ part, const float* __restrict__ target,
                                                                 const int32_t* __restrict__ labels, int parts, int M, int vocab,
                                                                 float* __restrict__ loss, float* __restrict__ lse) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int k = threadIdx.x % kJoinTokens, lane = threadIdx.x / kJoinTokens;
    constexpr int kLanes = kJoinThreads / kJoinTokens;
    const int m = blockIdx.x * kJoinTokens + k;
    float R = -INFINITY, S = 0.f;
    if (m < M) {
#pragma unroll 4
        for (int i = lane; i < parts; i += kLanes) {
            const float2 v = part[static_cast<size_t>(i) * M + m];
            join(R, S, v.x, v.y);
        }
    }
    __shared__ float2 sh[kLanes][kJoinTokens];
    sh[lane][k] = make_float2(R, S);
    __syncthreads();
    for (int o = kLanes / 2; o > 0; o /= 2) {
        if (lane < o) {
            join(R, S, sh[lane + o][k].x, sh[lane + o][k].y);
            sh[lane][k] = make_float2(R, S);
        }
        __syncthreads();
    }
    if (lane == 0 && m < M) {
        const float l = R + logf(S);
        lse[m] = l;
        const int label = labels[m];
        loss[m] = static_cast<unsigned>(label) < static_cast<unsigned>(vocab) ? l - target[m] : 0.f;
    }
}

// Up to 16 tokens of a packed table: lse and loss from logits in fp32, a cluster of CTAs per token whose (maximum, sum)
// are joined in rank order. The logits lie in L2: 131072 of one token take 3 us.
constexpr int kRowCtas = 8, kRowThreads = 256;
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__global__ void __cluster_dims__(kRowCtas, 1, 1) __launch_bounds__(kRowThreads)
    loss_rows_kernel(const float* __restrict__ logits, int64_t ld, const int32_t* __restrict__ labels, int vocab, float* __restrict__ loss,
                     float* __restrict__ lse) {
    grid_launch_dependents();
    cluster_arrive();   // (waited for before a CTA stores into rank 0's: that one has then begun)
    grid_dependency_wait();
    const int m = blockIdx.x / kRowCtas, rank = blockIdx.x % kRowCtas, tid = threadIdx.x;
    const float* row = logits + m * ld;
    const int per = ((vocab + kRowCtas - 1) / kRowCtas + 3) / 4 * 4, c1 = min(vocab, (rank + 1) * per);
    float R = -INFINITY, S = 0.f;
    auto take = [&](float v) {
        if (v == INFINITY) {   // (R stays finite, for the joins)
            R = 3.4e38f;
            S += v;
            return;
        }
        if (v > R) {
            S = R == -INFINITY ? S : S * exp2f((R - v) * 1.4426950408889634f);
            R = v;
        }
        S += v == -INFINITY ? 0.f : exp2f((v - R) * 1.4426950408889634f);   // (NaN stays NaN)
    };
    const int label = labels[m];
    const bool has = static_cast<unsigned>(label) < static_cast<unsigned>(vocab);
    const float target = has ? row[label] : 0.f;
    int c = rank * per + 4 * tid;
#pragma unroll 4
    for (; c + 3 < c1; c += 4 * kRowThreads) {
        const float4 v = *reinterpret_cast<const float4*>(row + c);
        const float top = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
        if (fabsf(top) < INFINITY) {
            if (top > R) {
                S = R == -INFINITY ? S : S * exp2f((R - top) * 1.4426950408889634f);
                R = top;
            }
            S += (exp2f((v.x - R) * 1.4426950408889634f) + exp2f((v.y - R) * 1.4426950408889634f)) +
                 (exp2f((v.z - R) * 1.4426950408889634f) + exp2f((v.w - R) * 1.4426950408889634f));
        } else {
            take(v.x);
            take(v.y);
            take(v.z);
            take(v.w);
        }
    }
    // (the last, partial group of four is this thread's)
    for (; c < c1; ++c) take(row[c]);
    // warps, then the CTA's eight of them, then the cluster's eight CTAs, each in order
    __shared__ float2 sums[kRowThreads / 32];
    __shared__ float2 of_cta[kRowCtas];   // (rank 0's: the others store theirs into it)
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const float r = __shfl_down_sync(0xffffffffu, R, o), s = __shfl_down_sync(0xffffffffu, S, o);
        join(R, S, r, s);
    }
    if ((tid & 31) == 0) sums[tid >> 5] = make_float2(R, S);
    __syncwarp();
    cluster_wait();
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int i = 1; i < kRowThreads / 32; ++i) join(R, S, sums[i].x, sums[i].y);
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(map_shared_rank(smem_u32(&of_cta[rank]), 0)), "f"(R), "f"(S) : "memory");
    }
    __syncwarp();
    cluster_sync_all();
    if (rank == 0 && tid == 0) {
        R = of_cta[0].x;
        S = of_cta[0].y;
#pragma unroll
        for (int r = 1; r < kRowCtas; ++r) join(R, S, of_cta[r].x, of_cta[r].y);
        const float l = R + logf(S);
        lse[m] = l;
        loss[m] = has ? l - target : 0.f;
    }
}

// X with zeros in the rows of tokens without a label, which have no part in dW whatever they hold; and for each token with
// one the mark of its block (an OR: the same whatever the order).
__global__ void __launch_bounds__(256) keep_labelled_kernel(const uint4* __restrict__ X, const int32_t* __restrict__ labels, int vocab,
                                                            int64_t count, int K8, uint4* __restrict__ out,
                                                            uint32_t* __restrict__ marks, int mark_words) {
    grid_launch_dependents();
    grid_dependency_wait();
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < count; i += int64_t(gridDim.x) * 256) {
        const uint4 v = X[i];
        const int64_t m = i / K8;
        const int label = labels[m];
        const bool has = static_cast<unsigned>(label) < static_cast<unsigned>(vocab);
        out[i] = has ? v : make_uint4(0, 0, 0, 0);
        if (marks && has && i == m * K8)
            atomicOr(marks + static_cast<size_t>(label / 256) * mark_words + m / 2048, 1u << (m / 64 % 32));
    }
}

// dX from the tiles of its sums: a block takes what one warp of vocab_kernel<kVocabDx> left, 32 tokens by half a
// tile's columns, adds the slices in order and scales. Where there are many slices (few tokens: 64 of them, in 8 blocks)
// it takes 32 columns, and each of its warps adds an eighth of the slices for them, joined in order: 16 tokens x 128
// columns took 26 us without.
// Tiles as that kernel writes them: [slice][column tile][token tile][CTA][warp][column / 4][lane].
constexpr int kManySlices = 8;
template <bool PAIR, bool MANY>
__global__ void __launch_bounds__(256) dx_out_kernel(const float4* __restrict__ acc, int slices, int m_tiles, int n_tiles, int M, int K,
                                                     const int32_t* __restrict__ labels, const float* __restrict__ grad, int vocab,
                                                     float unscale, const float* __restrict__ rest,
                                                     const __nv_bfloat16* __restrict__ W, __nv_bfloat16* __restrict__ dX) {
    grid_launch_dependents();
    grid_dependency_wait();
    constexpr int kCtas = PAIR ? 2 : 1, kCols = PAIR ? 128 : 64;
    constexpr int kMine = MANY ? 32 : kCols;   // of the columns, this block's
    const int warp = blockIdx.x & 7, rank = (blockIdx.x >> 3) % kCtas, tile = (blockIdx.x >> 3) / kCtas;   // tile within a slice
    const int m = tile % m_tiles, n = tile / m_tiles;
    const int r0 = m * (PAIR ? 256 : 128) + rank * 128 + (warp & 3) * 32;
    const int c0 = n * 2 * kCols + (warp >> 2) * kCols + blockIdx.y * kMine;
    if (r0 >= M || c0 >= K) return;
    __shared__ uint2 sh[32][kMine / 4 + 1];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    // (a token without a label has no gradient, though zeros times an infinite row are no zeros)
    const bool has = r0 + lane < M && static_cast<unsigned>(labels[r0 + lane]) < static_cast<unsigned>(vocab);
    float f = 1.f;
    if (has && unscale != 1.f) f = grad[r0 + lane] * unscale;   // packed tables: G came without the tokens' own factor
    const size_t slice = static_cast<size_t>(m_tiles) * n_tiles * kCtas * 8 * (kCols / 4) * 32;
    const float4* at = acc + (static_cast<size_t>(blockIdx.x) * (kCols / 4) + blockIdx.y * (kMine / 4)) * 32 + lane;
    auto add = [](float4& a, const float4& v) {
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
    };
    // bf16 tables: G's value at the label, often most of a token's gradient, was rounded to bf16 like the others; what that
    // took (half a step, as much as dX's own rounding) is made up for here, from the label's row.
    const float more = rest && has ? rest[r0 + lane] : 0.f;
    const __nv_bfloat16* wrow = rest && has ? W + static_cast<size_t>(labels[r0 + lane]) * K : nullptr;
    auto put = [&](int c, float4 s) {
        if (wrow && c0 + 4 * c < K) {
            const uint2 w = *reinterpret_cast<const uint2*>(wrow + c0 + 4 * c);
            s.x = fmaf(more, __uint_as_float(w.x << 16), s.x);
            s.y = fmaf(more, __uint_as_float(w.x & 0xFFFF0000u), s.y);
            s.z = fmaf(more, __uint_as_float(w.y << 16), s.z);
            s.w = fmaf(more, __uint_as_float(w.y & 0xFFFF0000u), s.w);
        }
        if (!has) s = make_float4(0.f, 0.f, 0.f, 0.f);
        const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x * f, s.y * f), hi = __floats2bfloat162_rn(s.z * f, s.w * f);
        sh[lane][c] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    };
    if constexpr (MANY) {
        __shared__ float4 part[8][8][32];   // [warp][column / 4][lane]
        const int per = (slices + 7) / 8, k1 = min(slices, (w + 1) * per);
        float4 s[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) s[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int k = w * per; k < k1; ++k) {
#pragma unroll
            for (int c = 0; c < 8; ++c) add(s[c], at[k * slice + c * 32]);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) part[w][c][lane] = s[c];
        __syncthreads();
        float4 sum = part[0][w][lane];
#pragma unroll
        for (int k = 1; k < 8; ++k) add(sum, part[k][w][lane]);
        put(w, sum);
    } else {
#pragma unroll
        for (int i = 0; i < kCols / 32; ++i) {
            const int c = w + 8 * i;
            float4 s = at[c * 32];
#pragma unroll 8
            for (int k = 1; k < slices; ++k) add(s, at[k * slice + c * 32]);
            put(c, s);
        }
    }
    __syncthreads();
    // (K is a multiple of 8: whole 16-byte stores)
    for (int i = threadIdx.x; i < 32 * (kMine / 8); i += 256) {
        const int r = i / (kMine / 8), c = i % (kMine / 8), col = c0 + 8 * c;
        if (r0 + r < M && col < K) {
            const uint2 a = sh[r][2 * c], d = sh[r][2 * c + 1];
            *reinterpret_cast<uint4*>(dX + static_cast<size_t>(r0 + r) * K + col) = make_uint4(a.x, a.y, d.x, d.y);
        }
    }
}

lowbit_status product(int mode, bool pair, const LossProblem& p, const LossLayout& l, uint8_t* ws, int64_t v0, int64_t cols, bool first,
                      cudaStream_t stream) {
    VocabProduct v;
    v.mode = mode;
    v.pair = pair;
    v.p = &p;
    v.l = &l;
    v.ws = ws;
    v.v0 = v0;
    v.cols = cols;
    v.first = first;
    switch (p.table.bits) {
        case 1: return vocab_product_b1(v, stream);
        case 2: return vocab_product_b2(v, stream);
        case 4: return vocab_product_b4(v, stream);
        default: return vocab_product_dense(v, stream);
    }
}

// The fp16 copy of X that packed tables are multiplied with.
lowbit_status copy_x(const LossProblem& p, const LossLayout& l, uint8_t* ws, cudaStream_t stream) {
    if (p.table.bits == kDense) return LOWBIT_OK;
    GemmProblem g = {};
    g.M = p.M;
    g.K = p.table.K;
    g.X = p.X;
    g.workspace = ws + l.xh;
    return launch_convert_x(g, stream);
}

// Marks of a whole table: bits of 64 tokens, words of 2048, by 256 rows.
size_t mark_bytes(const LossLayout& l, int64_t vocab) { return static_cast<size_t>((vocab + 255) / 256) * l.mark_words * 4; }

}  // namespace

LossLayout loss_layout(int64_t M, int64_t vocab, int64_t K, int bits, bool backward, bool need_dw) {
    LossLayout l = {};
    if (!backward && M > kTokensAtOnce) M = kTokensAtOnce;
    // 128 x 128 tiles: up to 128 tokens, where the table's rows are read once in any case and the wider tile's
    // second 128 rows would stay empty.
    l.pair = M > 128;
    const int64_t side = l.pair ? 256 : 128;
    l.m_tiles = (M + side - 1) / side;
    l.n_tiles = (vocab + side - 1) / side;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const size_t logits = static_cast<size_t>(M < kSmallTokens ? M : kSmallTokens) * up(vocab, 8) * 4;
    if (bits != kDense && !backward && M <= kSmallTokens) {
        l.small = true;
        l.logits = take(logits);
        l.total = at;
        return l;
    }
    const WorkspaceLayout x = workspace_layout(M, K);
    if (bits != kDense) {
        l.xh = take(x.total);
        l.rowmul = l.xh + x.rowmul_offset;
    }
    if (!backward) {
        l.target = take(static_cast<size_t>(M) * 4);
        // (room for the narrow tiles of 128 tokens too, so that a workspace for M tokens serves fewer)
        const int64_t few = bits == kDense ? 2 * ((vocab + 127) / 128) : 8 * ((vocab + 255) / 256), narrow = few * (M < 128 ? M : 128);
        l.parts = l.pair ? 2 * l.n_tiles : few;
        l.part = take(static_cast<size_t>(l.parts * M > narrow ? l.parts * M : narrow) * 8);
        l.total = bits != kDense && at < logits ? logits : at;   // (serves the small batches too)
        return l;
    }
    const int64_t whole = up(vocab, 256), tokens = M > 0 ? M : 1;
    l.g_terms = need_dw ? 2 : 1;
    int64_t most = kPieceBytes / (2 * tokens) / 256 * 256;
    if (most < 256) most = 256;
    const int64_t pieces = (vocab + most - 1) / most;
    l.piece = up((vocab + pieces - 1) / pieces, 256);
    l.dx_tiles = (K + side - 1) / side;
    // Slices of a piece's reduction, whose sums are kept apart: as many as make the last wave of tiles full, each of
    // at least 8 stages, weighed against 4 stages' worth of time for each tile's beginning and end.
    const int64_t tiles = l.m_tiles * l.dx_tiles, slots = l.pair ? 74 : 148, stages = (l.piece + 63) / 64;
    double best = 0;
    for (int s = 1; s <= 64 && (s == 1 || (s * 8 <= stages && s * tiles <= 8 * slots)); ++s) {
        const double cost = static_cast<double>((tiles * s + slots - 1) / slots) * (static_cast<double>((stages + s - 1) / s) + 4.0);
        if (s == 1 || cost < 0.97 * best) {
            best = cost;
            l.slices = s;
        }
    }
    const int64_t per = (stages + l.slices - 1) / l.slices;
    l.slices = static_cast<int>((stages + per - 1) / per);   // (no empty ones; a shorter last piece never has more)
    // G and the sums take room that grows with M, so that a workspace for M tokens serves fewer too.
    const size_t tile = static_cast<size_t>(side) * side * 4;
    const int64_t least = tokens * 256 * 2, all = tokens * whole * 2, some = kPieceBytes > least ? kPieceBytes : least;
    const size_t g = static_cast<size_t>(some < all ? some : all) * l.g_terms;
    size_t acc = 8 * slots * tile < 64 * tiles * tile ? 8 * slots * tile : 64 * tiles * tile;
    if (acc < tiles * tile) acc = tiles * tile;
    if (bits == kDense) l.rest = take(static_cast<size_t>(M) * 4);
    if (need_dw) l.xz = take(static_cast<size_t>(M) * K * 2);
    if (need_dw && M > kTwoTermTokens) {
        l.mark_words = (M + 2047) / 2048;
        l.marks = take(mark_bytes(l, vocab));
    }
    l.g = take(g);
    l.acc = take(acc);
    l.total = at;
    return l;
}

namespace {

// The forward of at most kTokensAtOnce tokens.
lowbit_status forward_of(const LossProblem& p, const LossLayout& l, uint8_t* ws, cudaStream_t stream) {
    if (l.small) {
        const Table& t = p.table;
        GemmProblem g = {};
        g.M = p.M;
        g.N = up(p.vocab, 8);   // (at most t.N: the rows behind the vocabulary are not read)
        g.K = t.K;
        g.bits = t.bits;
        g.group_size = t.group_size;
        g.X = p.X;
        g.Wp = static_cast<const uint32_t*>(t.rows);
        g.scales = t.scales;
        g.zeros = t.zeros;
        g.Y = ws + l.logits;
        // Rows per CTA: the fewest that take no more waves than the most (128), which the kernel's own choice, made for
        // linears, does not look for (112 instead of 128 for 32768: 7 % less). Short vocabularies are left to it.
        const int64_t sms = num_sms(), waves = (g.N + 128 * sms - 1) / (128 * sms), rows = up((g.N + waves * sms - 1) / (waves * sms), 16);
        const lowbit_status st =
            smallm_launch(g, g.N >= 64 * sms ? static_cast<int>(rows) : 0, g.N >= 64 * sms ? 1 : 0, g.M <= 8, stream, nullptr, true, t.N);
        if (st != LOWBIT_OK) return st;
        return launch_after(loss_rows_kernel, g.M * kRowCtas, 1, kRowThreads, stream, reinterpret_cast<const float*>(ws + l.logits), g.N,
                            p.labels, static_cast<int>(p.vocab), p.loss, p.lse_out);
    }
    lowbit_status st = copy_x(p, l, ws, stream);
    if (st == LOWBIT_OK) st = product(kVocabStats, l.pair, p, l, ws, 0, p.vocab, true, stream);
    if (st != LOWBIT_OK) return st;
    return launch_after(p.M <= 1024 ? loss_join_kernel<1> : loss_join_kernel<8>, p.M <= 1024 ? p.M : (p.M + 7) / 8, 1, kJoinThreads, stream,
                        reinterpret_cast<const float2*>(ws + l.part), reinterpret_cast<const float*>(ws + l.target), p.labels,
                        static_cast<int>(l.parts), static_cast<int>(p.M), static_cast<int>(p.vocab), p.loss, p.lse_out);
}

}  // namespace

lowbit_status loss_forward(const LossProblem& all, const LossLayout& l0, uint8_t* ws, cudaStream_t stream) {
    for (int64_t m0 = 0; m0 < all.M; m0 += kTokensAtOnce) {
        LossProblem p = all;
        p.M = all.M - m0 < kTokensAtOnce ? all.M - m0 : kTokensAtOnce;
        p.X = static_cast<const uint8_t*>(all.X) + static_cast<size_t>(m0) * all.table.K * 2;
        p.labels = all.labels + m0;
        p.loss = all.loss + m0;
        p.lse_out = all.lse_out + m0;
        const LossLayout l = m0 == 0 ? l0 : loss_layout(p.M, p.vocab, p.table.K, p.table.bits, false, false);
        const lowbit_status st = forward_of(p, l, ws, stream);
        if (st != LOWBIT_OK) return st;
    }
    return LOWBIT_OK;
}

lowbit_status loss_backward(const LossProblem& p, const LossLayout& l, uint8_t* ws, cudaStream_t stream) {
    const int64_t K = p.table.K;
    lowbit_status st = copy_x(p, l, ws, stream);
    if (st != LOWBIT_OK) return st;
    if (p.dW) {
        if (p.table.N > p.vocab &&
            cudaMemsetAsync(static_cast<uint8_t*>(p.dW) + static_cast<size_t>(p.vocab) * K * 2, 0,
                            static_cast<size_t>(p.table.N - p.vocab) * K * 2, stream) != cudaSuccess)
            return LOWBIT_ERR_CUDA;
        uint32_t* marks = l.mark_words ? reinterpret_cast<uint32_t*>(ws + l.marks) : nullptr;
        if (marks && cudaMemsetAsync(marks, 0, mark_bytes(l, p.vocab), stream) != cudaSuccess) return LOWBIT_ERR_CUDA;
        const int64_t count = p.M * (K / 8), blocks = (count + 255) / 256;
        st = launch_after(keep_labelled_kernel, blocks < 148 * 8 ? blocks : 148 * 8, 1, 256, stream, static_cast<const uint4*>(p.X), p.labels,
                          static_cast<int>(p.vocab), count, static_cast<int>(K / 8), reinterpret_cast<uint4*>(ws + l.xz),
                          marks, static_cast<int>(l.mark_words));
        if (st != LOWBIT_OK) return st;
    }
    int slices = l.slices;   // of a whole piece: the buffers that every piece adds to
    for (int64_t v0 = 0; v0 < p.vocab; v0 += l.piece) {
        const int64_t cols = p.vocab - v0 < l.piece ? p.vocab - v0 : l.piece;
        if ((st = product(kVocabGrad, l.pair, p, l, ws, v0, cols, v0 == 0, stream)) != LOWBIT_OK) return st;
        if ((st = product(kVocabDx, l.pair, p, l, ws, v0, cols, v0 == 0, stream)) != LOWBIT_OK) return st;
        if (v0 == 0) {   // (as the launch cuts the first piece, which a small vocabulary does not fill)
            const int64_t stages = (cols + 63) / 64, per = (stages + slices - 1) / slices;
            slices = static_cast<int>((stages + per - 1) / per);
        }
        if (p.dW && (st = product(kVocabDw, true, p, l, ws, v0, cols, true, stream)) != LOWBIT_OK) return st;
    }
    const int64_t blocks = l.m_tiles * l.dx_tiles * (l.pair ? 2 : 1) * 8;
    const float unscale = p.table.bits == kDense ? 1.f : 1.f / 32768.f;
    const bool many = slices >= kManySlices;
    const auto out = l.pair ? (many ? dx_out_kernel<true, true> : dx_out_kernel<true, false>)
                            : (many ? dx_out_kernel<false, true> : dx_out_kernel<false, false>);
    return launch_after(out, blocks, many ? (l.pair ? 4 : 2) : 1, 256, stream,
                        reinterpret_cast<const float4*>(ws + l.acc), slices, static_cast<int>(l.m_tiles), static_cast<int>(l.dx_tiles),
                        static_cast<int>(p.M), static_cast<int>(K), p.labels, p.grad, static_cast<int>(p.vocab), unscale,
                        p.table.bits == kDense ? reinterpret_cast<const float*>(ws + l.rest) : nullptr,
                        static_cast<const __nv_bfloat16*>(p.table.rows), static_cast<__nv_bfloat16*>(p.dX));
}

}  // namespace lowbit
