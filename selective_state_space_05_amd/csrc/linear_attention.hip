// linear_attention.hip -- linear attention with a decay per head: chunked over
// sequences, its backward, and one decode step on a cached state.
//
//   S_t = g S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,   g = e^log_decay
//
// A walk goes over a sequence C = 32 steps at a time with the state X in front of the
// chunk in matrix-core accumulators:
//   o_i = scale (g^(i+e) X^T q_i + sum_{j <= i} g^(i-j) (q_i . k_j) v_j)
//   X  <- g^n X + sum_j g^(n-e-j) k_j v_j^T               (n steps in the chunk)
// with e = 1 forward, where a state decays before it is read.  The gradients are
// walks of the same kind with other roles.  With R_t = scale q_t do_t^T + g R_{t+1}
// (dh_last added at the last step):
//   dq_t = scale S_t do_t    roles (do, v, k), state S^T, forward in time
//   dk_t = R_t v_t           roles (v, do, q), state R^T, against time, e = 0
//   dv_t = R_t^T k_t         roles (k, q, do), state R, against time, e = 0
//   dh0  = g R_0             the state behind the last walk
//
// Few sequences and heads are cut into segments of whole chunks: a first launch
// walks the segments for their states alone, a second folds them,
//   X_{s+1} = g^T X_s + local_s,
// and the third walks every segment from the state in front of it.  Everything is
// summed in an order that depends on the sizes alone.
#include <algorithm>
#include <type_traits>

#include "device_math.h"
#include "internal.h"

namespace mssm {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int C = 32;   // steps of a chunk: one block of products

// ---- fragments: eight contraction values of one row of an operand per lane; the
// ---- lane halves hold different ones, sixteen in all for a product of 32 x 32

struct F8 {
    float f[8];
};
template <typename T> struct FragOf;
template <> struct FragOf<uint16_t> { typedef bf16x8 type; };
template <> struct FragOf<float> { typedef F8 type; };

__device__ __forceinline__ void mma(f32x16 &c, bf16x8 a, bf16x8 b) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x16 &c, const F8 &a, const F8 &b) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.f[j], b.f[j], c, 0, 0, 0);
}

__device__ __forceinline__ void set(bf16x8 &f, int j, float v) { f[j] = static_cast<__bf16>(v); }
__device__ __forceinline__ void set(F8 &f, int j, float v) { f.f[j] = v; }
__device__ __forceinline__ float get(const bf16x8 &f, int j) { return static_cast<float>(f[j]); }
__device__ __forceinline__ float get(const F8 &f, int j) { return f.f[j]; }

// Accumulator element e of a lane is row acc_row(e) + 4 (lane / 32) of its 32 x 32
// block, column lane % 32.  As an operand of the next product elements 8 s .. + 7
// are the contraction rows 16 s + 4 h + {0..3, 8..11} of half h.
__device__ __forceinline__ int acc_row(int e) { return 8 * (e / 4) + e % 4; }

template <typename F>
__device__ __forceinline__ F from_acc(const f32x16 &c, int s) {
    F f;
#pragma unroll
    for (int j = 0; j < 8; ++j) set(f, j, c[8 * s + j]);
    return f;
}

// A tile of C rows of P values in LDS.  Its 16-byte chunks are permuted inside their
// rows so that 16 rows' reads of one chunk, and a transposed read's four chunks of four
// rows, cover the 64 banks.
template <typename T, int P>
struct Tile {
    static constexpr int E = 16 / sizeof(T), kChunks = P / E, kBytes = C * P * static_cast<int>(sizeof(T));
    static_assert(kChunks >= 8, "a row is 128 bytes or more");
    static __device__ __forceinline__ int swizzle(int row) {
        return kChunks == 8 ? row / 2 % 2 * 4 + row / 4 % 4 : row % 4 * 4 + row / 4 % 4;
    }
    static __device__ __forceinline__ int at(int row, int chunk) {
        return row * kChunks * 16 + (chunk ^ swizzle(row)) * 16;
    }
};

// Eight values side by side, chunk `chunk` on, of a row.  __restrict__ here and in the
// loads: a chunk is read only after its loads were waited for, and without the promise
// the compiler waits for all that are under way.
template <typename L>
__device__ __forceinline__ bf16x8 load_row(const unsigned char *__restrict__ tile, int row, int value, uint16_t) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(tile + L::at(row, value / 8)));
}
template <typename L>
__device__ __forceinline__ F8 load_row(const unsigned char *__restrict__ tile, int row, int value, float) {
    F8 f;
    const f32x4 a = *reinterpret_cast<const f32x4 *>(tile + L::at(row, value / 4));
    const f32x4 b = *reinterpret_cast<const f32x4 *>(tile + L::at(row, value / 4 + 1));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f.f[j] = a[j];
        f.f[4 + j] = b[j];
    }
    return f;
}

// Column of a 32-wide block that row m of a transposed operand stands for: chosen so
// that accumulator elements 8 s .. + 7 of half h, whose rows are those above, are the
// columns 16 s + 8 h + {0..7}, side by side.
__device__ __forceinline__ int column_of(int m) {
    return (m & 16) + 8 * (m / 4 % 2) + 4 * (m / 8 % 2) + m % 4;
}

// Transposed operand: row m = lane % 32 is column `value` + column_of(m) of the tile; the
// lane's contraction values are rows `row` + 4 h + {0..3, 8..11}.  In bfloat16 by the
// transposing LDS read: the 16 lanes of a group fetch four rows of four chunks of four
// columns, lane i row i / 4 of chunk i % 4, and lane i receives column i % 4 of chunk
// i / 4.
template <typename L>
__device__ __forceinline__ bf16x8 load_col(const unsigned char *__restrict__ tile, int row, int value, int lane, uint16_t) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 LdsRow;
    const int i = lane % 16, r = row + 4 * (lane / 32) + i / 4, c = (lane & 16) + column_of(4 * (i % 4));
    const unsigned char *a = tile + L::at(r, value / 8 + c / 8) + c % 8 * 2;
    const unsigned char *b = tile + L::at(r + 8, value / 8 + c / 8) + c % 8 * 2;
    const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsRow *)a));
    const uint2 hi = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsRow *)b));
    return __builtin_bit_cast(bf16x8, u32x4{lo.x, lo.y, hi.x, hi.y});
}
template <typename L>
__device__ __forceinline__ F8 load_col(const unsigned char *__restrict__ tile, int row, int value, int lane, float) {
    F8 f;
    const int c = value + column_of(lane % 32);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f.f[j] = *reinterpret_cast<const float *>(tile + L::at(row + 4 * (lane / 32) + j / 4 * 8 + j % 4, c / 4) + c % 4 * 4);
    return f;
}

// The infinite and NaN values of a fragment set to 0; the number of the first step that
// held one, its own steps being `first` + {0..3, 8..11}, or `none`.
__device__ __forceinline__ bool any_odd(const bf16x8 &f) {
    const u32x4 v = __builtin_bit_cast(u32x4, f);
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) r |= (v[j] & 0x7fff7fffu) + 0x00800080u;   // an exponent of all ones carries
    return r & 0x80008000u;
}
__device__ __forceinline__ bool any_odd(const F8 &f) {
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) r |= (__float_as_uint(f.f[j]) & 0x7fffffffu) + 0x00800000u;
    return r & 0x80000000u;
}
template <typename F>
__device__ __forceinline__ int clean(F &f, int first, int none) {
#pragma unroll
    for (int j = 7; j >= 0; --j)
        if (!(fabsf(get(f, j)) < __builtin_inff())) {
            set(f, j, 0.0f);
            none = first + j / 4 * 8 + j % 4;
        }
    return none;
}

// ---- one walk ------------------------------------------------------------------

// Roles and sizes of one walk.  Rows are tokens; a head's A (keys) or B (values)
// numbers lie side by side.  Element (a, b) of a state given by the caller is at
// a * sa + b * sb of its (sequence, head); states in the workspace are (A, B).
struct Walk {
    const void *q, *k, *v;
    void *o;
    const float *first;      // may be null -> 0
    float *last;             // may be null
    float *segments;         // states of this walk's segments in the workspace
    int64_t first_sa, first_sb;
    int64_t last_sa, last_sb;
    int64_t seg_sa, seg_sb;  // strides of the workspace's states
    int A, B;
    int slices;              // of B, over workgroups
    int early;               // e above
    int reverse;             // against time
    float inner, scale;      // factors of the inputs' products and of the outputs
};

struct Walks {
    Walk w[3];
    int count;               // of w
    const int64_t *cu;       // first rows of packed sequences, may be null
    const float *log_decay;
    int64_t seqs, seqlen, total, heads, segment;   // segment: its steps
    int segments;            // of a sequence
};

// Rows of sequence b: packed offsets are held to [0, total] and to rise, so that no
// value in them leads out of the tensors.
__device__ __forceinline__ void sequence(const Walks &W, int64_t b, int64_t *start, int64_t *len) {
    if (!W.cu) {
        *start = b * W.seqlen;
        *len = W.seqlen;
        return;
    }
    const int64_t lo = min(max(W.cu[b], int64_t(0)), W.total), hi = min(max(W.cu[b + 1], lo), W.total);
    *start = lo;
    *len = hi - lo;
}

// log2 of a head's decay; no decay faster than 2^-300 a step, which is 0 in float32
// even after one step, so that g^0 stays 1.
__device__ __forceinline__ float decay_log2(const float *log_decay, int64_t h) {
    const float d = log_decay[h] * kLog2e;
    return d < -300.0f ? -300.0f : d;
}


// KP: A rounded up to whole products.  WAVES: 32 columns of B each.  VEC: all rows are
// whole 16-byte vectors on 16-byte boundaries.
template <typename T, int KP_, int WAVES_, bool VEC_>
struct Shape {
    typedef T Type;
    typedef typename FragOf<T>::type Frag;
    static constexpr bool VEC = VEC_;
    static constexpr int KP = KP_, WAVES = WAVES_, threads = 64 * WAVES, VP = 32 * WAVES;
    typedef Tile<T, KP> Keys;
    typedef Tile<T, VP> Values;
    // bytes of a chunk's tiles in LDS, and how many chunks: loads of whole vectors go
    // straight to LDS, two chunks ahead where there is room
    static constexpr int tiles(bool out) { return (out ? 2 : 1) * Keys::kBytes + Values::kBytes; }
    static constexpr int stages(bool out) {
        const int fit = 160 * 1024 / tiles(out), most = VEC ? 3 : 2;
        return fit < most ? fit : most;
    }
    // registers for two waves a SIMD, but for the largest states
    static constexpr int waves_a_simd(bool) { return KP <= 64 || (KP <= 128 && sizeof(T) == 2) ? 2 : 1; }
    static constexpr int loads(bool out) { return tiles(out) / 1024 / WAVES; }   // of a wave and chunk
    static constexpr int stores = C * 32 * sizeof(T) / 1024;                     // the same
};

// The rows of one head of a tensor, in the order that a walk goes over them.
template <typename T>
struct Rows {
    T *p;                // the head's values in the sequence's first row of the walk
    int64_t ld;          // values between rows, negative against time
    int width;

    // A buffer of the n rows of a chunk from row t on: those past the end lie outside it,
    // behind it or, against time, in front (their offsets are negative, far behind as
    // unsigned ones), read as zero and are not written.  Offsets are those of offset() plus shift().
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(int64_t t, int n) const {
        const int bytes = static_cast<int>(ld < 0 ? -ld : ld) * static_cast<int>(sizeof(T));
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<std::remove_const_t<T> *>(p + (t + (ld < 0 ? n - 1 : 0)) * ld), 0,
                                                 (n - 1) * bytes + width * static_cast<int>(sizeof(T)), 0x00020000);
    }
    __device__ __forceinline__ int shift(int n) const {
        return ld < 0 ? -(n - 1) * static_cast<int>(ld) * static_cast<int>(sizeof(T)) : 0;
    }
    __device__ __forceinline__ int offset(int row, int value) const {
        return value < width ? (row * static_cast<int>(ld) + value) * static_cast<int>(sizeof(T)) : INT32_MIN;
    }
};

// A tile's way from memory: columns from `width` on and rows from n on are 0.
template <typename S, typename L>
struct Feed {
    typedef typename S::Type T;
    typedef __attribute__((address_space(3))) void Lds;
    static constexpr int N = L::kBytes / 1024 / S::WAVES;    // instructions of 1024 bytes a wave
    u32x4 r[S::VEC ? 1 : N];

    // Row and chunk of this lane's 16 bytes of instruction i.
    static __device__ __forceinline__ int row(int i) {
        return (i * S::threads + static_cast<int>(threadIdx.x)) / L::kChunks;
    }
    static __device__ __forceinline__ int chunk(int i) {
        return static_cast<int>(threadIdx.x) % L::kChunks ^ L::swizzle(row(i));
    }
    // Straight into LDS.
    static __device__ __forceinline__ void send(const Rows<const T> &R, int64_t t, int n, int wave,
                                                unsigned char *__restrict__ tile) {
#if defined(__HIP_DEVICE_COMPILE__)   // with the builtin in it, the host pass leaves out the kernel's handle
        const auto rsrc = R.buffer(t, n);
        const int shift = R.shift(n);
#pragma unroll
        for (int i = 0; i < N; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (Lds *)(tile + (i * S::WAVES + wave) * 1024), 16,
                                                     R.offset(row(i), chunk(i) * S::Keys::E) + shift, 0, 0, 0);
#endif
    }
    // Through registers, element by element.
    __device__ __forceinline__ void fetch(const Rows<const T> &R, int64_t t, int n) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            T v[L::E] = {};
            if (row(i) < n) {
                const T *p = R.p + (t + row(i)) * R.ld;
#pragma unroll
                for (int x = 0; x < L::E; ++x)
                    if (chunk(i) * L::E + x < R.width) v[x] = p[chunk(i) * L::E + x];
            }
            r[i] = *reinterpret_cast<const u32x4 *>(v);
        }
    }
    __device__ __forceinline__ void store(unsigned char *tile) const {
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4 *>(tile + (i * S::threads + threadIdx.x) * 16) = r[i];
    }
};

// Waits until at most N of this wave's loads and stores are under way, then for the
// other waves.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
}

// Eight outputs side by side: as whole vectors, or one by one up to `left`.
__device__ __forceinline__ void store_vectors(const Rows<uint16_t> &o, int64_t t, int n, int row, int value, const float *f) {
    bf16x8 b;
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = static_cast<__bf16>(f[j]);
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, b), o.buffer(t, n), o.offset(row, value) + o.shift(n), 0, 0);
}
__device__ __forceinline__ void store_vectors(const Rows<float> &o, int64_t t, int n, int row, int value, const float *f) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        __builtin_amdgcn_raw_buffer_store_b128(
            u32x4{__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3])},
            o.buffer(t, n), o.offset(row, value + 4 * i) + o.shift(n), 0, 0);
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float *f, int left) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < left) Io<T>::store(p, j, f[j]);
}

// OUT: the walk with its outputs; else for the segments' states alone.
template <typename S, bool OUT>
__global__ __launch_bounds__(S::threads, S::waves_a_simd(OUT)) void attention_walk_kernel(const Walks W) {
    typedef typename S::Type T;
    typedef typename S::Frag Frag;
    constexpr int KB = S::KP / 32, KS = S::KP / 16, CS = C / 16;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    constexpr int kStages = S::stages(OUT), kTiles = S::tiles(OUT), kLoads = S::loads(OUT);
    constexpr int kStores = OUT ? S::stores : 0;

    // workgroups go to the eight XCDs in turn: each gets a run of consecutive
    // positions, so that the walks over one head's rows share its L2
    const int n_ids = gridDim.x, x = blockIdx.x % 8;
    int64_t at = static_cast<int64_t>(x) * (n_ids / 8) + min(x, n_ids % 8) + blockIdx.x / 8;
    int role = 0;
    if (W.count > 1) {
        role = static_cast<int>(at % W.count);
        at /= W.count;
    }
    const Walk &w = W.w[role];
    const int most = max(max(W.w[0].slices, W.w[1].slices), W.w[2].slices);
    const int slice = static_cast<int>(at % most);
    at /= most;
    const int64_t h = at % W.heads;
    at /= W.heads;
    const int seg = static_cast<int>(at % W.segments);
    const int64_t b = at / W.segments;
    if (slice >= w.slices) return;
    int64_t start, len;
    sequence(W, b, &start, &len);
    const int64_t t0 = seg * W.segment;
    const bool tail = seg == W.segments - 1;       // walks to the end, however far
    const int64_t t1 = tail ? len : min(len, t0 + W.segment);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, half = lane / 32, col = lane % 32;
    const int v0 = slice * S::VP, width = min(S::VP, w.B - v0);

    if (OUT && W.cu && ((b == 0 && seg == 0) || (b == W.seqs - 1 && tail))) {
        // rows in front of the first sequence and behind the last one
        for (int side = 0; side < 2; ++side) {
            if (side == 0 ? !(b == 0 && seg == 0) : !(b == W.seqs - 1 && tail)) continue;
            const int64_t lo = side == 0 ? 0 : start + len, hi = side == 0 ? start : W.total;
            T *o = static_cast<T *>(w.o) + h * w.B + v0;
            for (int64_t id = threadIdx.x; id < (hi - lo) * width; id += S::threads)
                o[(lo + id / width) * W.heads * w.B + id % width] = T(0);
        }
    }
    if (OUT ? (t0 >= len && seg > 0) : (tail || t0 + W.segment >= len)) return;   // nothing, or nothing behind it

    const float ld = decay_log2(W.log_decay, h);
    const int e = w.early;
    auto power = [&](int n) { return fast_exp2(ld * static_cast<float>(n)); };
    const int my_v = v0 + 32 * wave + column_of(col);    // column of this lane's state
    const int64_t bh = b * W.heads + h;

    // element j of block kb of the state: row 32 kb + 16 (j / 8) + 8 half + j % 8
    f32x16 X[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 16; ++j) X[kb][j] = 0.0f;
    if (OUT && (seg > 0 || w.first)) {
        const int64_t sa = seg > 0 ? w.seg_sa : w.first_sa, sb = seg > 0 ? w.seg_sb : w.first_sb;
        const int64_t states = static_cast<int64_t>(w.A) * w.B;
        const float *from = seg > 0 ? w.segments + ((b * (W.segments - 1) + seg - 1) * W.heads + h) * states
                                    : w.first + bh * states;
        if (my_v < w.B) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int a = 32 * kb + 16 * (j / 8) + 8 * half + j % 8;
                    if (a < w.A) X[kb][j] = from[a * sa + my_v * sb];
                }
        }
    }

    // decays inside a chunk: of outputs (this lane's is col) from its inputs and from the
    // state in front, and of the inputs to the state behind
    float inside[16], weight[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int row = acc_row(j) + 4 * half;
        inside[j] = w.inner * power(max(col - row, 0));
        weight[j] = w.inner * power(C - e - row);
    }
    const float front = power(col + e);
    float whole = power(C);

    const int64_t row_first = w.reverse ? start + len - 1 : start, sign = w.reverse ? -1 : 1;
    const int64_t lda = W.heads * w.A, ldb = W.heads * w.B;
    const Rows<const T> q{static_cast<const T *>(w.q) + row_first * lda + h * w.A, sign * lda, w.A},
        k{static_cast<const T *>(w.k) + row_first * lda + h * w.A, sign * lda, w.A},
        v{static_cast<const T *>(w.v) + row_first * ldb + h * w.B + v0, sign * ldb, width};
    const Rows<T> o{OUT ? static_cast<T *>(w.o) + row_first * ldb + h * w.B + v0 : nullptr, sign * ldb, width};
    const int my_out = 32 * wave + 8 * half;      // first of the outputs of row col
    Feed<S, typename S::Keys> kin, qin;
    Feed<S, typename S::Values> vin;
    auto steps = [&](int64_t t) { return static_cast<int>(min(int64_t(C), t1 - t)); };
    auto send = [&](int64_t t, int stage) {
        unsigned char *const to = smem + stage * kTiles;
        kin.send(k, t, steps(t), wave, to);
        vin.send(v, t, steps(t), wave, to + S::Keys::kBytes);
        if (OUT) qin.send(q, t, steps(t), wave, to + S::Keys::kBytes + S::Values::kBytes);
    };
    auto fetch = [&](int64_t t) {
        kin.fetch(k, t, steps(t));
        vin.fetch(v, t, steps(t));
        if (OUT) qin.fetch(q, t, steps(t));
    };
    if (t0 < t1) {
        if (S::VEC) {
            for (int ahead = 0; ahead < kStages - 1; ++ahead)
                if (t0 + ahead * C < t1) send(t0 + ahead * C, ahead);
        } else {
            fetch(t0);
        }
    }
    int stage = 0, last_stage = kStages - 1;
    for (int64_t t = t0; t < t1; t += C) {
        const int n = steps(t);
        const unsigned char *const Ks = smem + stage * kTiles, *const Vs = Ks + S::Keys::kBytes, *const Qs = Vs + S::Values::kBytes;
        if constexpr (S::VEC) {
            // What is under way behind this chunk's loads may stay so: those of the next
            // chunk and the outputs of the one before, which were sent after them.  Then
            // every wave has read the stage that the next loads go to.
            if constexpr (kStages == 1) {
                wait_and_meet<0>();
                send(t, 0);
                wait_and_meet<0>();
            } else {
                if (kStages == 2 || t + C >= t1) wait_and_meet<0>();
                else if (t == t0) wait_and_meet<kLoads>();
                else wait_and_meet<kLoads + kStores>();
                if (t + (kStages - 1) * C < t1) send(t + (kStages - 1) * C, last_stage);
            }
        } else {
            unsigned char *const to = smem + stage * kTiles;
            if (kStages == 1) __syncthreads();
            kin.store(to);
            vin.store(to + S::Keys::kBytes);
            if (OUT) qin.store(to + S::Keys::kBytes + S::Values::kBytes);
            __syncthreads();                      // who reads the other stage has read it
            if (t + C < t1) fetch(t + C);
        }
        last_stage = stage;
        stage = stage == kStages - 1 ? 0 : stage + 1;
        if (n < C) {                              // the last chunk
            whole = power(n);
#pragma unroll
            for (int j = 0; j < 16; ++j) weight[j] = w.inner * power(max(n - e - acc_row(j) - 4 * half, 0));
        }

        // The products leave out later inputs by a factor 0, which an infinite or NaN v
        // would carry to earlier outputs of its chunk.  Such values are taken out, and what
        // they reach is set to NaN: their column from their step on.
        Frag vf[CS];
        bool odd = false;
        int reached = C;                          // first such step of this lane's column
#pragma unroll
        for (int s = 0; s < CS; ++s) {
            vf[s] = load_col<typename S::Values>(Vs, 16 * s, 32 * wave, lane, T());
            odd |= any_odd(vf[s]);
        }
        if (__any(odd)) {
#pragma unroll
            for (int s = CS - 1; s >= 0; --s) reached = clean(vf[s], 16 * s + 4 * half, reached);
            reached = min(reached, __shfl_xor(reached, 32));
        }
        if (OUT) {
            f32x16 G, O;
#pragma unroll
            for (int j = 0; j < 16; ++j) G[j] = O[j] = 0.0f;
            // The state enters as an operand of the I/O dtype: in bfloat16 half a step, 2^-8
            // of each of its values, like the rounding of the output.
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const Frag qf = load_row<typename S::Keys>(Qs, col, 16 * s + 8 * half, T());
                mma(G, load_row<typename S::Keys>(Ks, col, 16 * s + 8 * half, T()), qf);
                mma(O, from_acc<Frag>(X[s / 2], s % 2), qf);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) O[j] *= front;
            // later inputs leave nothing, whatever their products hold
#pragma unroll
            for (int j = 0; j < 16; ++j) G[j] = acc_row(j) + 4 * half <= col ? G[j] * inside[j] : 0.0f;
#pragma unroll
            for (int s = 0; s < CS; ++s) mma(O, vf[s], from_acc<Frag>(G, s));
            if (__any(odd)) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (col >= __shfl(reached, acc_row(j) + 4 * half)) O[j] = __builtin_nanf("");
            }
            float out[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) out[j] = O[j] * w.scale;
            if constexpr (S::VEC) {
#pragma unroll
                for (int s = 0; s < CS; ++s) store_vectors(o, t, n, col, my_out + 16 * s, out + 8 * s);
            } else if (col < n) {
                T *const to = o.p + (t + col) * o.ld + my_out;
#pragma unroll
                for (int s = 0; s < CS; ++s) store8(to + 16 * s, out + 8 * s, width - my_out - 16 * s);
            }
        }
        // The state: k_j exact, its partner g^(n-e-j) v_j in bfloat16 as the sum of two
        // roundings, which hold it to 2^-16.
        const float f = reached < C ? __builtin_nanf("") : whole;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int j = 0; j < 16; ++j) X[kb][j] *= f;
#pragma unroll
        for (int s = 0; s < CS; ++s) {
            Frag up, rest;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = weight[8 * s + j] * get(vf[s], j);
                set(up, j, u);
                set(rest, j, u - get(up, j));
            }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const Frag a = load_col<typename S::Keys>(Ks, 16 * s, 32 * kb, lane, T());
                mma(X[kb], a, up);
                if (sizeof(T) == 2) mma(X[kb], a, rest);
            }
        }
    }

    if (OUT && !w.last) return;
    if (OUT && !(t1 == len && (t1 > t0 || seg == 0))) return;
    const int64_t states = static_cast<int64_t>(w.A) * w.B;
    float *to = OUT ? w.last + bh * states : w.segments + ((b * (W.segments - 1) + seg) * W.heads + h) * states;
    const int64_t sa = OUT ? w.last_sa : w.seg_sa, sb = OUT ? w.last_sb : w.seg_sb;
    if (my_v < w.B) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int a = 32 * kb + 16 * (j / 8) + 8 * half + j % 8;
                if (a < w.A) to[a * sa + my_v * sb] = X[kb][j];
            }
    }
}

// X_{s+1} = g^T X_s + local_s in place: slot s receives the state in front of segment
// s + 1.
__global__ __launch_bounds__(256) void attention_fold_kernel(const Walks W) {
    const Walk &w = W.w[blockIdx.z];
    const int64_t bh = blockIdx.y, b = bh / W.heads, h = bh % W.heads;
    const int64_t states = static_cast<int64_t>(w.A) * w.B;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (id >= states) return;
    int64_t start, len;
    sequence(W, b, &start, &len);
    // segments that end before the sequence does
    const int64_t full = len <= 0 ? 0 : min(int64_t(W.segments - 1), (len - 1) / W.segment);
    const float g = fast_exp2(decay_log2(W.log_decay, h) * static_cast<float>(W.segment));
    const int64_t a = id / w.B, c = id % w.B;
    float x = w.first ? w.first[bh * states + a * w.first_sa + c * w.first_sb] : 0.0f;
    float *p = w.segments + (b * (W.segments - 1) * W.heads + h) * states + a * w.seg_sa + c * w.seg_sb;
    const int64_t next = W.heads * states;
    for (int64_t s = 0; s < full; s += 8, p += 8 * next) {
        float local[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) local[i] = s + i < full ? p[i * next] : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x = fmaf(g, x, local[i]);
            if (s + i < full) p[i * next] = x;
        }
    }
}

// ---- launches ------------------------------------------------------------------

int waves_of(int64_t B) { return B <= 64 ? 2 : 4; }
int slices_of(int64_t B) { return static_cast<int>((B + 32 * waves_of(B) - 1) / (32 * waves_of(B))); }

constexpr int64_t kSlots = 512;   // workgroups that the device holds at once

// Segments of a sequence and their steps: as many as give every compute unit two
// workgroups of the forward, all at once.
void cut(const AttentionArgs &a, bool bwd, int *segments, int64_t *steps) {
    const int64_t walks = std::max<int64_t>(1, a.seqs * a.heads * slices_of(a.value));
    const int64_t n = std::max<int64_t>(1, std::min((bwd ? kSlots / 2 : kSlots) / walks, a.seqlen / (4 * C)));
    *steps = std::max<int64_t>(C, ((a.seqlen + n - 1) / n + C - 1) / C * C);
    *segments = static_cast<int>(std::max<int64_t>(1, (a.seqlen + *steps - 1) / *steps));
}

template <typename S, bool OUT>
hipError_t launch_walks(const Walks &W, hipStream_t stream) {
    int most = 0;
    for (int i = 0; i < W.count; ++i) most = std::max(most, W.w[i].slices);
    const int64_t n = W.seqs * W.segments * W.heads * most * W.count;
    constexpr int lds = S::stages(OUT) * S::tiles(OUT);
    if (lds > 65536)
        if (const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(attention_walk_kernel<S, OUT>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds))
            return e;
    hipLaunchKernelGGL((attention_walk_kernel<S, OUT>), dim3(static_cast<uint32_t>(n)), dim3(S::threads), lds, stream, W);
    return hipGetLastError();
}

// What instantiates the kernel for a walk: A rounded up, waves, whole vectors.
struct Kind {
    int keys, waves;
    bool vec;
    bool operator==(const Kind &k) const { return keys == k.keys && waves == k.waves && vec == k.vec; }
};

template <bool OUT>
Kind kind_of(const Walk &w, int size) {
    const auto p = [](const void *a) { return reinterpret_cast<uintptr_t>(a); };
    const uintptr_t at = p(w.k) | p(w.v) | (OUT ? p(w.q) | p(w.o) : 0);
    return Kind{w.A <= 64 ? 64 : w.A <= 128 ? 128 : 256, waves_of(w.B), (at | (w.A | w.B) * size) % 16 == 0};
}

template <typename T, bool OUT, bool VEC>
hipError_t launch_group(const Walks &W, const Kind &k, hipStream_t stream) {
    if (k.waves == 2) {
        if (k.keys == 64) return launch_walks<Shape<T, 64, 2, VEC>, OUT>(W, stream);
        if (k.keys == 128) return launch_walks<Shape<T, 128, 2, VEC>, OUT>(W, stream);
        return launch_walks<Shape<T, 256, 2, VEC>, OUT>(W, stream);
    }
    if (k.keys == 64) return launch_walks<Shape<T, 64, 4, VEC>, OUT>(W, stream);
    if (k.keys == 128) return launch_walks<Shape<T, 128, 4, VEC>, OUT>(W, stream);
    return launch_walks<Shape<T, 256, 4, VEC>, OUT>(W, stream);
}

// Walks of one kind share a launch.
template <typename T, bool OUT>
hipError_t launch_all(const Walks &W, hipStream_t stream) {
    bool done[3] = {false, false, false};
    for (int i = 0; i < W.count; ++i) {
        if (done[i]) continue;
        const Kind kind = kind_of<OUT>(W.w[i], sizeof(T));
        Walks G = W;
        G.count = 0;
        for (int j = i; j < W.count; ++j)
            if (!done[j] && kind_of<OUT>(W.w[j], sizeof(T)) == kind) {
                G.w[G.count++] = W.w[j];
                done[j] = true;
            }
        for (int j = G.count; j < 3; ++j) G.w[j] = G.w[0];
        if (const hipError_t e = kind.vec ? launch_group<T, OUT, true>(G, kind, stream) : launch_group<T, OUT, false>(G, kind, stream))
            return e;
    }
    return hipSuccess;
}

template <bool OUT>
hipError_t launch_all(const Walks &W, bool f32, hipStream_t stream) {
    return f32 ? launch_all<float, OUT>(W, stream) : launch_all<uint16_t, OUT>(W, stream);
}

Walks common(const AttentionArgs &a, bool bwd) {
    Walks W{};
    W.cu = a.cu_seqlens;
    W.log_decay = a.log_decay;
    W.seqs = a.seqs; W.seqlen = a.seqlen; W.total = a.total; W.heads = a.heads;
    cut(a, bwd, &W.segments, &W.segment);
    return W;
}

hipError_t fold(const Walks &W, hipStream_t stream) {
    int64_t states = 0;
    for (int i = 0; i < W.count; ++i) states = std::max(states, static_cast<int64_t>(W.w[i].A) * W.w[i].B);
    hipLaunchKernelGGL(attention_fold_kernel,
                       dim3(static_cast<uint32_t>((states + 255) / 256), static_cast<uint32_t>(W.seqs * W.heads), W.count),
                       dim3(256), 0, stream, W);
    return hipGetLastError();
}

// ---- one step ------------------------------------------------------------------

// A workgroup holds LANES x VEC columns of one state; groups of LANES lanes take the
// rows in turn.
template <typename T, int VEC, int LANES>
__global__ __launch_bounds__(256) void attention_step_kernel(float *__restrict__ state, const T *__restrict__ q,
                                                             const T *__restrict__ k, const T *__restrict__ v,
                                                             const float *__restrict__ log_decay, float scale,
                                                             T *__restrict__ o, int heads, int K, int V, int slices) {
    constexpr int GROUPS = 256 / LANES, COLS = LANES * VEC;
    __shared__ float sum[GROUPS][COLS];
    const int64_t bh = blockIdx.x / slices;
    const int slice = blockIdx.x % slices, h = static_cast<int>(bh % heads);
    const int group = threadIdx.x / LANES, c = slice * COLS + threadIdx.x % LANES * VEC;
    const float g = fast_exp2(decay_log2(log_decay, h));
    state += bh * K * V;
    q += bh * K;
    k += bh * K;
    v += bh * V;
    o += bh * V;
    float acc[VEC] = {};
    if (c < V) {
        float vv[VEC];
#pragma unroll
        for (int x = 0; x < VEC; ++x) vv[x] = Io<T>::load(v, c + x);
#pragma unroll 8
        for (int a = group; a < K; a += GROUPS) {
            float *p = state + static_cast<int64_t>(a) * V + c;
            const float kk = Io<T>::load(k, a), qq = Io<T>::load(q, a);
            if constexpr (VEC == 4) {
                float4 s = *reinterpret_cast<const float4 *>(p);
                s.x = fmaf(g, s.x, kk * vv[0]);
                s.y = fmaf(g, s.y, kk * vv[1]);
                s.z = fmaf(g, s.z, kk * vv[2]);
                s.w = fmaf(g, s.w, kk * vv[3]);
                *reinterpret_cast<float4 *>(p) = s;
                acc[0] = fmaf(qq, s.x, acc[0]);
                acc[1] = fmaf(qq, s.y, acc[1]);
                acc[2] = fmaf(qq, s.z, acc[2]);
                acc[3] = fmaf(qq, s.w, acc[3]);
            } else {
                const float s = fmaf(g, *p, kk * vv[0]);
                *p = s;
                acc[0] = fmaf(qq, s, acc[0]);
            }
        }
    }
#pragma unroll
    for (int x = 0; x < VEC; ++x) sum[group][threadIdx.x % LANES * VEC + x] = acc[x];
    __syncthreads();
    for (int x = threadIdx.x; x < COLS; x += 256) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) s += sum[i][x];
        if (slice * COLS + x < V) Io<T>::store(o, slice * COLS + x, s * scale);
    }
}

template <typename T>
hipError_t step(const AttentionArgs &a, hipStream_t stream) {
    const int64_t bh = a.seqs * a.heads;
    auto go = [&](auto kernel, int cols) {
        const int64_t slices = (a.value + cols - 1) / cols;
        hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(bh * slices)), dim3(256), 0, stream, a.h_last,
                           static_cast<const T *>(a.q), static_cast<const T *>(a.k), static_cast<const T *>(a.v),
                           a.log_decay, a.scale, static_cast<T *>(a.o), static_cast<int>(a.heads),
                           static_cast<int>(a.key), static_cast<int>(a.value), static_cast<int>(slices));
    };
    const bool vec = a.value % 4 == 0 && reinterpret_cast<uintptr_t>(a.h_last) % 16 == 0;
    if (!vec) go(attention_step_kernel<T, 1, 32>, 32);
    else if (bh * ((a.value + 127) / 128) >= 256) go(attention_step_kernel<T, 4, 32>, 128);
    else go(attention_step_kernel<T, 4, 8>, 32);
    return hipGetLastError();
}

}  // namespace

size_t linear_attention_workspace(const AttentionArgs &a, bool bwd) {
    const Walks W = common(a, bwd);
    return static_cast<size_t>(W.segments - 1) * a.seqs * a.heads * a.key * a.value * sizeof(float) * (bwd ? 2 : 1);
}

hipError_t launch_linear_attention_fwd(const AttentionArgs &a, void *workspace, hipStream_t stream) {
    Walks W = common(a, false);
    const size_t bytes = linear_attention_workspace(a, false);
    void *ws = workspace;
    if (bytes && !ws)
        if (const hipError_t e = scratch_alloc(&ws, bytes, stream)) return e;
    const int K = static_cast<int>(a.key), V = static_cast<int>(a.value);
    W.count = 1;
    W.w[0] = Walk{a.q, a.k, a.v, a.o, a.h0, a.h_last, static_cast<float *>(ws), V, 1, V, 1, V, 1, K, V,
                  slices_of(V), 1, 0, 1.0f, a.scale};
    hipError_t e = hipSuccess;
    if (W.segments > 1) {
        e = launch_all<false>(W, a.io == IO_F32, stream);
        if (e == hipSuccess) e = fold(W, stream);
    }
    if (e == hipSuccess) e = launch_all<true>(W, a.io == IO_F32, stream);
    if (bytes && !workspace) {
        const hipError_t f = scratch_free(ws, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

hipError_t launch_linear_attention_bwd(const AttentionArgs &a, void *workspace, hipStream_t stream) {
    Walks W = common(a, true);
    const size_t bytes = linear_attention_workspace(a, true);
    void *ws = workspace;
    if (bytes && !ws)
        if (const hipError_t e = scratch_alloc(&ws, bytes, stream)) return e;
    const int K = static_cast<int>(a.key), V = static_cast<int>(a.value);
    float *S = static_cast<float *>(ws), *R = S + bytes / 2 / sizeof(float);
    // S^T in (V, K) as the first walk forms it; R in (K, V) as the third does
    const Walk dq{a.dout, a.v, a.k, a.dq, a.h0, nullptr, S, 1, V, 0, 0, K, 1, V, K, slices_of(K), 1, 0, 1.0f, a.scale};
    const Walk dk{a.v, a.dout, a.q, a.dk, a.dh_last, nullptr, R, 1, V, 0, 0, 1, V, V, K, slices_of(K), 0, 1, a.scale, 1.0f};
    const Walk dv{a.k, a.q, a.dout, a.dv, a.dh_last, a.dh0, R, V, 1, V, 1, V, 1, K, V, slices_of(V), 0, 1, a.scale, 1.0f};
    hipError_t e = hipSuccess;
    if (W.segments > 1) {
        W.count = 2;
        W.w[0] = dq;
        W.w[1] = dv;
        W.w[2] = dq;
        e = launch_all<false>(W, a.io == IO_F32, stream);
        if (e == hipSuccess) e = fold(W, stream);
    }
    W.count = 3;
    W.w[0] = dq;
    W.w[1] = dk;
    W.w[2] = dv;
    if (e == hipSuccess) e = launch_all<true>(W, a.io == IO_F32, stream);
    if (bytes && !workspace) {
        const hipError_t f = scratch_free(ws, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

hipError_t launch_linear_attention_update(const AttentionArgs &a, hipStream_t stream) {
    return a.io == IO_F32 ? step<float>(a, stream) : step<uint16_t>(a, stream);
}

}  // namespace mssm
