// linear_cross_entropy.hip -- softmax cross entropy of the logits
// l = hidden weight^T over a large vocabulary, forward and backward, the
// logits formed a tile at a time on the matrix cores and never stored.
//
// Forward: every tile of logits gives, per token, its maximum m and
// s = sum exp(l - m); the tiles' pairs join as
//   (m1, s1) + (m2, s2) = (max, s1 e^(m1 - max) + s2 e^(m2 - max)),
// lse = m + log s and loss = lse - l_target.
//
// Backward, for a piece of the vocabulary at a time:
//   p = (exp(l - lse) - [v == target]) dloss   (0 for ignored tokens)
//   dhidden += p weight,   dweight = p^T hidden
// with the logits formed again and p held in the I/O dtype for that piece
// only.  In bfloat16 the rounding of p (half a step, 2^-9 relative, of
// either sign) averages over the sums it enters.
//
// All three products run on one kernel: C[m, n] = sum_k A[m, k] B[n, k] with
// both operands stored along k, for which weight, hidden and p are also laid
// out transposed.
#include "device_math.h"
#include "internal.h"

namespace mssm {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kRowBytes = 64;    // of k staged per step and operand row
constexpr int kChunks = kRowBytes / 16;
constexpr int kStages = 4;       // steps in LDS at a time
constexpr int kWaves = 4, kThreads = 64 * kWaves;

// One product step over the 16 bytes of k that each lane holds of its A row
// (lane % 32) and its B row: bfloat16 holds k 8 (lane / 32) .. + 7 of one
// 32x32x16 product; float32 four products of 32x32x2, the order of k inside
// them being the same for A and B.
__device__ __forceinline__ void mma(f32x16 &c, u32x4 a, u32x4 b, uint16_t) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x16 &c, u32x4 a, u32x4 b, float) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[j], y[j], c, 0, 0, 0);
}

// Rows of one operand: `rows` of them, `ld` bytes apart, 16-byte aligned.
struct Rows {
    const unsigned char *p;
    int64_t ld;
    int rows;
};

// Row of C inside a 32 x 32 block that element e of a lane's accumulator is
// (its column is lane % 32): four consecutive rows for every four elements.
__device__ __forceinline__ int acc_row(int e, int lane) { return 8 * (e / 4) + 4 * (lane / 32) + e % 4; }

// A workgroup's tile of C and a wave's part of it.
template <int BM_, int BN_, int WM_, int WN_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int I = WM / 32, J = WN / 32, waves_m = BM / WM;
    static_assert((BM / WM) * (BN / WN) == kWaves, "four waves");
    static constexpr int stage = (BM + BN) * kRowBytes, lds = kStages * stage;
};

// Position of workgroup `id` of n: workgroups go to the eight XCDs in turn, so
// each XCD gets a run of consecutive positions, and a run of 8 tiles of m for
// each n: the 32 workgroups an XCD holds at a time then share 8 + 4 operand
// tiles through its L2.
__device__ __forceinline__ void tile_of(int id, int n, int mt, int nt, int *m, int *nn) {
    const int per = n / 8, rest = n % 8, x = id % 8;
    const int t = x * per + min(x, rest) + id / 8;
    constexpr int kGroup = 8;
    const int g = t / (kGroup * nt), r = t - g * kGroup * nt, width = min(kGroup, mt - g * kGroup);
    *m = g * kGroup + r % width;
    *nn = r / width;
}

// Wait until at most N of this wave's loads into LDS are under way, then for
// the other waves.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
}

// C[m, n] = sum_k A[m, k] B[n, k] for one tile.  Rows move from memory straight
// into LDS, kRowBytes of every row a step, three steps ahead; a wave's operand
// fragments are read half a step ahead of the products that use them, the
// first ones of a step right after its barrier, under the last products of
// the step before.
template <typename T, typename Shape>
__device__ __forceinline__ void product_tile(const Rows &A, const Rows &B, int64_t kbytes, int m0, int n0,
                                             unsigned char *lds, f32x16 (&acc)[Shape::I][Shape::J]) {
    constexpr int I = Shape::I, J = Shape::J;
    constexpr int kRowsPer = 64 / kChunks;                        // rows of one load instruction
    constexpr int kLoads = (Shape::BM + Shape::BN) / kRowsPer;    // of a step
    constexpr int kMine = (kLoads + kWaves - 1) / kWaves;         // of them, this wave's (the last ones may repeat)
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int chunks = static_cast<int>((kbytes + 15) / 16), steps = (chunks + kChunks - 1) / kChunks;
    // rows past the end lie past the buffer's end and read as zero
    const auto rows_at = [](const Rows &R, int first, int most) {
        // (the minimum is formed in a vector register)
        const int n = __builtin_amdgcn_readfirstlane(min(R.rows - first, most));
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char *>(R.p) + first * R.ld, 0,
                                                 n * static_cast<int>(R.ld), 0x00020000);
    };
    const __amdgpu_buffer_rsrc_t ra = rows_at(A, m0, Shape::BM), rb = rows_at(B, n0, Shape::BN);
    const uint32_t lda = static_cast<uint32_t>(A.ld), ldb = static_cast<uint32_t>(B.ld);
    // The chunks of a row are permuted by the row, so that lanes that read one
    // chunk of consecutive rows hit different banks: LDS is filled in lane
    // order, so the lanes fetch them permuted.
    const int row = lane / kChunks, chunk = (lane % kChunks) ^ ((row / 2) % kChunks);
    const uint32_t va = row * lda + chunk * 16, vb = row * ldb + chunk * 16;
    typedef __attribute__((address_space(3))) void Lds;
    const auto load = [&](int step) {
        const bool in = step * kChunks + chunk < chunks;          // k past the end reads as zero too
        const uint32_t oa = in ? va : 0xffffffffu, ob = in ? vb : 0xffffffffu;
        unsigned char *to = lds + (step % kStages) * Shape::stage;
#pragma unroll
        for (int s = 0; s < kMine; ++s) {
            constexpr int kA = Shape::BM / kRowsPer;
            static_assert(kA % kWaves == 0, "each of a wave's loads is of one operand");
            const int q = min(wave + s * kWaves, kLoads - 1);
            if (s < kA / kWaves)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (Lds *)(to + q * 1024), 16, oa,
                                                         q * kRowsPer * lda + step * kRowBytes, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (Lds *)(to + q * 1024), 16, ob,
                                                         (q - kA) * kRowsPer * ldb + step * kRowBytes, 0, 0);
        }
    };
    const int wm = (wave % Shape::waves_m) * Shape::WM, wn = (wave / Shape::waves_m) * Shape::WN;
    u32x4 fa[2][I], fb[2][J];
    const auto read = [&](int step, int half) {
        const unsigned char *from = lds + (step % kStages) * Shape::stage + (lane % 32) * kRowBytes +
                                    (((2 * half + lane / 32) ^ ((lane / 2) % kChunks)) * 16);
#pragma unroll
        for (int i = 0; i < I; ++i) fa[half][i] = *reinterpret_cast<const u32x4 *>(from + (wm + 32 * i) * kRowBytes);
#pragma unroll
        for (int j = 0; j < J; ++j)
            fb[half][j] = *reinterpret_cast<const u32x4 *>(from + (Shape::BM + wn + 32 * j) * kRowBytes);
    };
    const auto multiply = [&](int half) {
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) mma(acc[i][j], fa[half][i], fb[half][j], T{});
    };
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    for (int s = 0; s < kStages - 1; ++s) load(s);
    wait_and_meet<(kStages - 2) * kMine>();
    load(kStages - 1);
    read(0, 0);
    read(0, 1);
    multiply(0);
    for (int step = 1; step < steps; ++step) {
        wait_and_meet<(kStages - 2) * kMine>();
        load(step + kStages - 1);
        read(step, 0);
        multiply(1);
        __builtin_amdgcn_sched_barrier(0);
        read(step, 1);
        multiply(0);
    }
    multiply(1);
}

// One grid of products of the same kind: problem 0's tiles, then problem 1's.
struct Problem {
    Rows A, B;
    int64_t kbytes;
    int mt, nt;
};

template <typename Epilogue>
struct Pair {
    Problem p[2];
    Epilogue e[2];
};

template <typename T, typename Shape, typename Epilogue>
__global__ __launch_bounds__(kThreads, Shape::lds > 81920 ? 1 : 2) void product_kernel(Pair<Epilogue> both) {
    extern __shared__ __align__(16) unsigned char lds[];
    const int n0 = both.p[0].mt * both.p[0].nt, id = static_cast<int>(blockIdx.x);
    const int which = id >= n0 ? 1 : 0;
    const Problem &p = both.p[which];
    const Epilogue &ep = both.e[which];
    int mi, ni;
    tile_of(id - (which ? n0 : 0), p.mt * p.nt, p.mt, p.nt, &mi, &ni);
    const int m0 = __builtin_amdgcn_readfirstlane(mi * Shape::BM), t0 = __builtin_amdgcn_readfirstlane(ni * Shape::BN);
    f32x16 acc[Shape::I][Shape::J];
    product_tile<T, Shape>(p.A, p.B, p.kbytes, m0, t0, lds, acc);
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int wm = (wave % Shape::waves_m) * Shape::WM, wn = (wave / Shape::waves_m) * Shape::WN;
#pragma unroll
    for (int j = 0; j < Shape::J; ++j) {
        f32x16 column[Shape::I];
#pragma unroll
        for (int i = 0; i < Shape::I; ++i) column[i] = acc[i][j];
        ep.template column<Shape::I>(m0 + wm, t0 + wn + 32 * j + lane % 32, lane, column);
    }
}

// ---- forward: maximum and sum of exponentials of a token over a tile's words
struct LossTile {
    float2 *part;              // [32 I words][token]
    float *target_logit;       // [token]
    const int64_t *targets;
    int tokens, words, word0;  // words of this piece; word0: the piece's first
    int part0;                 // first part of this piece
    template <int I>
    __device__ __forceinline__ void column(int m, int t, int lane, const f32x16 (&acc)[I]) const {
        if (t >= tokens) t = -1;
        const int64_t target = t >= 0 ? targets[t] - word0 : -1;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int v = m + 32 * i + acc_row(e, lane);
                const float l = acc[i][e];
                if (v < words) top = fmaxf(top, l);
                if (v == target && v < words) target_logit[t] = l;
            }
        top = fmaxf(top, __shfl_xor(top, 32));
        const float ref = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int v = m + 32 * i + acc_row(e, lane);
                if (v < words) sum += fast_exp2((acc[i][e] - ref) * kLog2e);
            }
        sum += __shfl_xor(sum, 32);
        if (t >= 0 && lane < 32 && m < words) part[static_cast<int64_t>(part0 + m / (32 * I)) * tokens + t] = make_float2(top, sum);
    }
};

__global__ __launch_bounds__(256) void loss_join_kernel(const float2 *__restrict__ part, int parts, int tokens,
                                                        const int64_t *__restrict__ targets, int64_t ignore,
                                                        int64_t vocab, float *__restrict__ loss,
                                                        float *__restrict__ lse) {
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t >= tokens) return;
    float m = -INFINITY, s = 0.0f;
    for (int k = 0; k < parts; ++k) {
        const float2 p = part[static_cast<int64_t>(k) * tokens + t];
        const float top = fmaxf(m, p.x), ref = top == -INFINITY ? 0.0f : top;
        s = s * fast_exp2((m - ref) * kLog2e) + p.y * fast_exp2((p.x - ref) * kLog2e);
        m = top;
    }
    const float l = m + fast_log2(s) * kLn2;
    if (lse) lse[t] = l;
    const int64_t target = targets[t];
    loss[t] = target == ignore ? 0.0f : (target < 0 || target >= vocab) ? NAN : l - loss[t];
}

// ---- backward ----------------------------------------------------------------------

// The largest finite |dloss| of the tokens that have a loss (1 if there is
// none): p is held relative to it.  The gradient of a mean is the same for
// every token and rarely a bfloat16; divided by this it is 1, so that holding
// p - 1 of a target's word costs p, not a rounding of dloss.
__global__ __launch_bounds__(1024) void grad_scale_kernel(const float *__restrict__ dloss,
                                                          const int64_t *__restrict__ targets, int64_t ignore,
                                                          int tokens, float *__restrict__ scale) {
    __shared__ float sh[16];
    float m = 0.0f;
    for (int t = threadIdx.x; t < tokens; t += 1024) {
        const float g = fabsf(dloss[t]);
        if (targets[t] != ignore && g < INFINITY) m = fmaxf(m, g);
    }
#pragma unroll
    for (int k = 32; k >= 1; k /= 2) m = fmaxf(m, __shfl_xor(m, k));
    if (threadIdx.x % 64 == 0) sh[threadIdx.x / 64] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < 16; ++k) m = fmaxf(m, sh[k]);
        *scale = m > 0.0f ? m : 1.0f;
    }
}

// p of a piece, in both layouts
template <typename T>
struct ProbTile {
    T *p, *pt;                 // p[token][word] and pt[word][token]
    int64_t ldp, ldpt;         // elements
    const int64_t *targets;
    const float *lse, *dloss, *scale;
    int64_t ignore, vocab;
    int tokens, words, word0;
    template <int I>
    __device__ __forceinline__ void column(int m, int t, int lane, const f32x16 (&acc)[I]) const {
        if (t >= ldpt) return;
        const int64_t target = t < tokens ? targets[t] : ignore;
        const bool live = target != ignore;
        const float ref = live ? lse[t] : 0.0f;
        float g = live ? dloss[t] / *scale : 0.0f;
        if (live && (target < 0 || target >= vocab)) g = NAN;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int v = m + 32 * i + acc_row(e, lane);
                if (v >= ldp) continue;
                float x = 0.0f;
                if (live && v < words) {
                    x = fast_exp2((acc[i][e] - ref) * kLog2e);
                    x = (x - (v + word0 == target ? 1.0f : 0.0f)) * g;
                }
                if (t < tokens) Io<T>::store(p, t * ldp + v, x);
                if (v < words) Io<T>::store(pt, v * ldpt + t, x);
            }
    }
};

// ---- backward: rows of a gradient, [n][m]; accumulated over pieces in float32
template <typename T>
struct GradTile {
    float *sum;                // float32 accumulator, or null
    T *out;                    // output, or null
    const float *scale;        // the output is the sum times this
    int64_t ld;
    int rows, cols;            // of the output
    bool add;                  // sum holds earlier pieces
    template <int I>
    __device__ __forceinline__ void column(int m, int n, int lane, const f32x16 (&acc)[I]) const {
        if (n >= rows) return;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int d = m + 32 * i + acc_row(e, lane);
                if (d >= cols) continue;
                float v = acc[i][e];
                const int64_t at = n * ld + d;
                if (add) v += sum[at];
                if (out) Io<T>::store(out, at, v * *scale);
                else sum[at] = v;
            }
    }
};

// Copy of rows [0, rows) x [0, cols) with rows `ldo` elements apart, zero past
// the columns.
template <typename T>
__global__ __launch_bounds__(256) void align_rows_kernel(const T *__restrict__ in, T *__restrict__ out,
                                                         int64_t rows, int64_t cols, int64_t ldo) {
    const int64_t n = rows * ldo;
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; k < n;
         k += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = k / ldo, c = k - r * ldo;
        out[k] = c < cols ? in[r * cols + c] : T{};
    }
}

// out[c][r] = in[r][c], zero for rows past the end and for rows whose target
// is `ignore` (targets may be null: then every row counts).
template <typename T>
__global__ __launch_bounds__(256) void transpose_kernel(const T *__restrict__ in, T *__restrict__ out, int rows,
                                                        int cols, int64_t ldo,
                                                        const int64_t *__restrict__ targets, int64_t ignore) {
    __shared__ T tile[32][33];
    const int c0 = blockIdx.x * 32, r0 = blockIdx.y * 32;
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    for (int k = ty; k < 32; k += 8) {
        const int r = r0 + k, c = c0 + tx;
        T v{};
        if (r < rows && c < cols && !(targets && targets[r] == ignore)) v = in[static_cast<int64_t>(r) * cols + c];
        tile[k][tx] = v;
    }
    __syncthreads();
    for (int k = ty; k < 32; k += 8) {
        const int c = c0 + k, r = r0 + tx;
        if (c < cols && r < ldo) out[static_cast<int64_t>(c) * ldo + r] = tile[tx][k];
    }
}

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t ceil_div(int64_t n, int64_t by) { return (n + by - 1) / by; }

bool on_16(const LossArgs &a) {
    return ((reinterpret_cast<uintptr_t>(a.hidden) | reinterpret_cast<uintptr_t>(a.weight)) & 15u) == 0;
}

typedef Tile<256, 256, 128, 128> Large;
typedef Tile<128, 128, 64, 64> Medium;
typedef Tile<256, 32, 64, 32> Narrow;    // few tokens

template <typename T, typename Shape, typename Epilogue>
hipError_t product_as(Problem p0, Problem p1, const Epilogue &e0, const Epilogue &e1, hipStream_t stream) {
    const auto tiles = [](Problem &p) {
        p.mt = static_cast<int>(ceil_div(p.A.rows, Shape::BM));
        p.nt = static_cast<int>(ceil_div(p.B.rows, Shape::BN));
        return static_cast<int64_t>(p.mt) * p.nt;
    };
    const int64_t n = tiles(p0) + tiles(p1);
    const auto kernel = product_kernel<T, Shape, Epilogue>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, Shape::lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(n)), dim3(kThreads), Shape::lds, stream,
                       (Pair<Epilogue>{{p0, p1}, {e0, e1}}));
    return hipGetLastError();
}

// Two products of one kind in one grid (the second may be empty).
template <typename T, typename Epilogue>
hipError_t products(const Problem &p0, const Problem &p1, const Epilogue &e0, const Epilogue &e1, int shape,
                    hipStream_t stream) {
    if (shape == 0) return product_as<T, Large>(p0, p1, e0, e1, stream);
    if (shape == 1) return product_as<T, Medium>(p0, p1, e0, e1, stream);
    return product_as<T, Narrow>(p0, p1, e0, e1, stream);
}

template <typename T>
hipError_t align_rows(const T *in, T *out, int64_t rows, int64_t cols, int64_t ldo, hipStream_t stream) {
    const int64_t blocks = ceil_div(rows * ldo, 256 * 4);
    hipLaunchKernelGGL(align_rows_kernel<T>, dim3(static_cast<uint32_t>(blocks < 65536 ? blocks : 65536)),
                       dim3(256), 0, stream, in, out, rows, cols, ldo);
    return hipGetLastError();
}

template <typename T>
hipError_t transpose(const T *in, T *out, int64_t rows, int64_t cols, int64_t ldo, const int64_t *targets,
                     int64_t ignore, hipStream_t stream) {
    hipLaunchKernelGGL(transpose_kernel<T>,
                       dim3(static_cast<uint32_t>(ceil_div(cols, 32)), static_cast<uint32_t>(ceil_div(ldo, 32))),
                       dim3(256), 0, stream, in, out, static_cast<int>(rows), static_cast<int>(cols), ldo, targets,
                       ignore);
    return hipGetLastError();
}

// Words of the vocabulary in one piece: p of the piece has at most 2^27
// elements, and a piece at least 1024 words.
int64_t piece_words(int64_t rows, int64_t vocab) {
    int64_t n = (int64_t(1) << 27) / (rows < 1 ? 1 : rows) / 1024 * 1024;
    if (n < 1024) n = 1024;
    return n < vocab ? n : vocab;
}

// Sizes of a call and its workspace, cut into 256-byte aligned arrays.
struct Plan {
    bool copy;                 // rows of hidden and weight are copied to aligned ones
    int64_t dimp, tokp;        // padded row lengths (elements)
    int64_t piece, piecep;     // words of a piece
    int64_t parts, part_words;
    int shape, grad_shape;     // of the logits' and the gradients' tiles
    size_t at_part, at_h, at_w, at_ht, at_wt, at_p, at_pt, at_sum, at_scale, bytes;
};

Plan make_plan(const LossArgs &a, bool bwd, bool aligned) {
    Plan p{};
    const int64_t esz = a.io == IO_F32 ? 4 : 2, unit = 16 / esz;
    p.copy = !aligned || a.dim % unit != 0;
    p.dimp = round_up(a.dim, unit);
    p.tokp = round_up(a.tokens, unit);
    const auto add = [&](int64_t bytes) {
        const size_t at = p.bytes;
        p.bytes += static_cast<size_t>(round_up(bytes, 256));
        return at;
    };
    p.piece = piece_words(bwd || a.tokens > p.dimp ? a.tokens : p.dimp, a.vocab);
    p.piecep = round_up(p.piece, unit);
    if (p.copy) {
        p.at_h = add(a.tokens * p.dimp * esz);
        p.at_w = add(p.piece * p.dimp * esz);
    }
    if (!bwd) {
        p.shape = a.tokens <= 32 ? 2 : ceil_div(a.vocab, 256) * ceil_div(a.tokens, 256) >= 256 ? 0 : 1;
        p.part_words = p.shape == 0 ? Large::WM : p.shape == 1 ? Medium::WM : Narrow::WM;
        p.parts = a.vocab / p.piece * ceil_div(p.piece, p.part_words) + ceil_div(a.vocab % p.piece, p.part_words);
        p.at_part = add(p.parts * a.tokens * 8);
        return p;
    }
    const auto tiles = [](int64_t m, int64_t n) { return ceil_div(m, 256) * ceil_div(n, 256); };
    p.shape = tiles(p.piece, a.tokens) >= 256 ? 0 : 1;
    p.grad_shape = tiles(a.dim, a.tokens) + tiles(a.dim, p.piece) >= 256 ? 0 : 1;
    p.at_ht = add(a.dim * p.tokp * esz);
    p.at_wt = add(a.dim * p.piecep * esz);
    p.at_p = add(a.tokens * p.piecep * esz);
    p.at_pt = add(p.piece * p.tokp * esz);
    p.at_scale = add(4);
    if (p.piece < a.vocab) p.at_sum = add(a.tokens * a.dim * 4);
    return p;
}

template <typename T>
Rows rows_of(const T *q, int64_t ld, int64_t n) {
    return Rows{reinterpret_cast<const unsigned char *>(q), ld * static_cast<int64_t>(sizeof(T)), static_cast<int>(n)};
}

Problem problem(const Rows &A, const Rows &B, int64_t kbytes) { return Problem{A, B, kbytes, 0, 0}; }

template <typename T>
hipError_t fwd(const LossArgs &a, const Plan &p, unsigned char *base, hipStream_t stream) {
    float2 *part = reinterpret_cast<float2 *>(base + p.at_part);
    const T *h = static_cast<const T *>(a.hidden);
    hipError_t e = hipSuccess;
    if (p.copy) {
        e = align_rows(h, reinterpret_cast<T *>(base + p.at_h), a.tokens, a.dim, p.dimp, stream);
        h = reinterpret_cast<const T *>(base + p.at_h);
    }
    int part0 = 0;
    for (int64_t w0 = 0; w0 < a.vocab && e == hipSuccess; w0 += p.piece) {
        const int64_t words = a.vocab - w0 < p.piece ? a.vocab - w0 : p.piece;
        const T *w = static_cast<const T *>(a.weight) + w0 * a.dim;
        if (p.copy) {
            e = align_rows(w, reinterpret_cast<T *>(base + p.at_w), words, a.dim, p.dimp, stream);
            w = reinterpret_cast<const T *>(base + p.at_w);
            if (e != hipSuccess) break;
        }
        const LossTile ep{part, a.loss, a.targets, static_cast<int>(a.tokens), static_cast<int>(words),
                          static_cast<int>(w0), part0};
        e = products<T>(problem(rows_of(w, p.dimp, words), rows_of(h, p.dimp, a.tokens), p.dimp * sizeof(T)), Problem{}, ep,
                        ep, p.shape, stream);
        part0 += static_cast<int>(ceil_div(words, p.part_words));
    }
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(loss_join_kernel, dim3(static_cast<uint32_t>(ceil_div(a.tokens, 256))), dim3(256), 0, stream,
                       part, part0, static_cast<int>(a.tokens), a.targets, a.ignore_index, a.vocab, a.loss, a.lse);
    return hipGetLastError();
}

template <typename T>
hipError_t bwd(const LossArgs &a, const Plan &p, unsigned char *base, hipStream_t stream) {
    T *pr = reinterpret_cast<T *>(base + p.at_p), *pt = reinterpret_cast<T *>(base + p.at_pt);
    T *ht = reinterpret_cast<T *>(base + p.at_ht), *wt = reinterpret_cast<T *>(base + p.at_wt);
    float *scale = reinterpret_cast<float *>(base + p.at_scale);
    const T *h = static_cast<const T *>(a.hidden);
    const int tokens = static_cast<int>(a.tokens), dim = static_cast<int>(a.dim);
    hipLaunchKernelGGL(grad_scale_kernel, dim3(1), dim3(1024), 0, stream, a.dloss, a.targets, a.ignore_index, tokens,
                       scale);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) e = transpose(h, ht, a.tokens, a.dim, p.tokp, a.targets, a.ignore_index, stream);
    if (e == hipSuccess && p.copy) {
        e = align_rows(h, reinterpret_cast<T *>(base + p.at_h), a.tokens, a.dim, p.dimp, stream);
        h = reinterpret_cast<const T *>(base + p.at_h);
    }
    for (int64_t w0 = 0; w0 < a.vocab && e == hipSuccess; w0 += p.piece) {
        const int64_t words = a.vocab - w0 < p.piece ? a.vocab - w0 : p.piece;
        const int64_t wordsp = round_up(words, 16 / sizeof(T));
        const T *w = static_cast<const T *>(a.weight) + w0 * a.dim;
        e = transpose<T>(w, wt, words, a.dim, wordsp, nullptr, 0, stream);
        if (e == hipSuccess && p.copy) {
            e = align_rows(w, reinterpret_cast<T *>(base + p.at_w), words, a.dim, p.dimp, stream);
            w = reinterpret_cast<const T *>(base + p.at_w);
        }
        if (e != hipSuccess) break;
        const ProbTile<T> prob{pr, pt, wordsp, p.tokp, a.targets, a.lse, a.dloss, scale, a.ignore_index, a.vocab,
                               tokens, static_cast<int>(words), static_cast<int>(w0)};
        e = products<T>(problem(rows_of(w, p.dimp, words), rows_of(h, p.dimp, a.tokens), p.dimp * sizeof(T)), Problem{}, prob,
                        prob, p.shape, stream);
        if (e != hipSuccess) break;
        float *sum = p.piece < a.vocab ? reinterpret_cast<float *>(base + p.at_sum) : nullptr;
        const GradTile<T> dh{sum, w0 + words >= a.vocab ? static_cast<T *>(a.dhidden) : nullptr, scale, a.dim, tokens,
                             dim, w0 > 0};
        const GradTile<T> dw{nullptr, static_cast<T *>(a.dweight) + w0 * a.dim, scale, a.dim, static_cast<int>(words),
                             dim, false};
        e = products<T>(problem(rows_of(wt, wordsp, a.dim), rows_of(pr, wordsp, a.tokens), wordsp * sizeof(T)),
                        problem(rows_of(ht, p.tokp, a.dim), rows_of(pt, p.tokp, words), p.tokp * sizeof(T)), dh, dw,
                        p.grad_shape, stream);
    }
    return e;
}

hipError_t launch(const LossArgs &a, bool backward, void *workspace, hipStream_t stream) {
    const Plan p = make_plan(a, backward, on_16(a));
    void *mem = workspace;
    hipError_t e = hipSuccess;
    if (!mem) e = scratch_alloc(&mem, p.bytes, stream);
    if (e != hipSuccess) return e;
    unsigned char *base = static_cast<unsigned char *>(mem);
    if (a.io == IO_F32) e = backward ? bwd<float>(a, p, base, stream) : fwd<float>(a, p, base, stream);
    else e = backward ? bwd<uint16_t>(a, p, base, stream) : fwd<uint16_t>(a, p, base, stream);
    if (!workspace) {
        const hipError_t f = scratch_free(mem, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

}  // namespace

size_t linear_cross_entropy_workspace(const LossArgs &a, bool backward, bool aligned) {
    return make_plan(a, backward, aligned).bytes;
}

hipError_t launch_linear_cross_entropy_fwd(const LossArgs &a, void *workspace, hipStream_t stream) {
    return launch(a, false, workspace, stream);
}

hipError_t launch_linear_cross_entropy_bwd(const LossArgs &a, void *workspace, hipStream_t stream) {
    return launch(a, true, workspace, stream);
}

}  // namespace mssm
