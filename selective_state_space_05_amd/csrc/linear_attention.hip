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
// Few sequences and heads are cut into segments of whole chunks, which are walked side
// by side: a first launch walks them for their states alone, a second folds these,
//   X_{s+1} = g^n X_s + sum_s  (n steps a segment),
// and the third walks every segment from the state in front of it.  Everything is summed
// in an order that depends on the sizes alone.
//
// A chunk's products run on the matrix cores from tiles in LDS, which its rows reach
// without passing registers, two or three chunks ahead; the transposed operands come from
// transposing LDS reads, and accumulators feed the next product as they are, the order of
// a contraction being free.  Every wave has 32 columns of values with their part of the
// state, and forms q.k again for itself: shared through LDS it would cost a barrier a chunk.
//
// Bound by memory and the chunk's chain of products about equally forward, by the chain
// backward: ten more products a chunk, to 52, took the third launch of 2 x 4096 x 20 x 128 in
// bfloat16 from 59 to 62 us forward and from 150 to 182 us backward.  Whole calls in bfloat16:
// 2 x 4096 x 20 x 128 forward 97 us, backward 214 us, 131072 steps of 4 heads 250 us; float32:
// the same layer 266 and 820 us, 7 packed sequences of 5 heads, 80 and 72 wide, backward 137 us.
// One step of 64 sequences 36 us from memory (4.7 TB/s over the states), 27 us where the
// device's 256 MB cache holds part of them; of one sequence 4 us on the device.
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

__device__ __forceinline__ void pack(bf16x8 &f, const float *v) {
    typedef float f32x8 __attribute__((ext_vector_type(8)));
    f = __builtin_convertvector((f32x8{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]}), bf16x8);
}
__device__ __forceinline__ void pack(F8 &f, const float *v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f.f[j] = v[j];
}
// v less f, exactly where f is v's rounding: a product of two with (-1, 0) or (0, -1) takes
// one instruction a value, where taking f apart takes a second.  The factors are held in
// registers: written into the instruction as constants they are read as float32 ones.
__device__ __forceinline__ void take(float (&v)[8], const bf16x8 &f) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    uint32_t first = 0x0000bf80u, second = 0xbf800000u;
    asm("" : "+s"(first), "+s"(second));
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const bf16x2 two = {f[j], f[j + 1]};
        v[j] = __builtin_amdgcn_fdot2_f32_bf16(two, __builtin_bit_cast(bf16x2, first), v[j], false);
        v[j + 1] = __builtin_amdgcn_fdot2_f32_bf16(two, __builtin_bit_cast(bf16x2, second), v[j + 1], false);
    }
}
__device__ __forceinline__ void take(float (&)[8], const F8 &) {}

// Eight values as the sum of N fragments, each the rounding of what those before left;
// `each` sees a fragment before the next is formed.
template <typename F, int N, typename G>
__device__ __forceinline__ void split(F (&part)[N], const float *v, G each) {
    float left[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) left[j] = v[j];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        pack(part[i], left);
        each(part[i]);
        if (i + 1 < N) take(left, part[i]);
    }
}
template <typename F, int N, typename G>
__device__ __forceinline__ void from_acc(F (&part)[N], const f32x16 &c, int s, G each) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c[8 * s + j];
    split(part, v, each);
}

// Which of a fragment's contraction values {0..3, 8..11} are `last` or less, and what
// leaves the others 0, NaN included.
template <typename F> struct Mask;
template <> struct Mask<bf16x8> {
    u32x4 bits;
};
template <> struct Mask<F8> {
    int last;
};
__device__ __forceinline__ Mask<bf16x8> mask_of(const bf16x8 &, int last) {
    Mask<bf16x8> m;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int v = j / 2 * 8 + j % 2 * 2;
        m.bits[j] = (v <= last ? 0xffffu : 0u) | (v + 1 <= last ? 0xffff0000u : 0u);
    }
    return m;
}
__device__ __forceinline__ Mask<F8> mask_of(const F8 &, int last) { return Mask<F8>{last}; }
__device__ __forceinline__ void keep(bf16x8 &f, const Mask<bf16x8> &m) {
    f = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, f) & m.bits);
}
__device__ __forceinline__ void keep(F8 &f, const Mask<F8> &m) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f.f[j] = j / 4 * 8 + j % 4 <= m.last ? f.f[j] : 0.0f;
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
__device__ __forceinline__ bool any_odd(const bf16x8 &a, const bf16x8 &b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    float r = 0.0f;                          // products with 0: NaN if one is not finite
    const bf16x2 zero = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        r = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{a[j], a[j + 1]}, zero, r, false);
        r = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{b[j], b[j + 1]}, zero, r, false);
    }
    return r != 0.0f;
}
__device__ __forceinline__ bool any_odd(const F8 &a, const F8 &b) {
    float r = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) r = fmaf(b.f[j], 0.0f, fmaf(a.f[j], 0.0f, r));
    return r != 0.0f;
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
    float *segments;         // in the workspace: in front of every segment but the first, the state
    float *kept;             // there too: receives `first` before anything is written; may be null
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


// KB: blocks of 32 of A.  WAVES: 32 columns of B each.  VEC: all rows are whole 16-byte
// vectors on 16-byte boundaries.
template <typename T, int KB_, int WAVES_, bool VEC_>
struct Shape {
    typedef T Type;
    typedef typename FragOf<T>::type Frag;
    static constexpr bool VEC = VEC_;
    static constexpr int KB = KB_, WAVES = WAVES_, threads = 64 * WAVES, VP = 32 * WAVES;
    typedef Tile<T, KB <= 2 ? 64 : KB <= 4 ? 128 : 256> Keys;
    typedef Tile<T, VP> Values;
    // registers for two waves a SIMD, but for the largest states
    static constexpr int kWavesASimd = KB <= 2 || (KB <= 4 && sizeof(T) == 2) ? 2 : 1;
    // Bytes of a chunk's tiles in LDS, and how many chunks: loads of whole vectors go
    // straight to LDS, up to three chunks ahead where there is room for two workgroups.  The
    // largest tiles, 80 KB, leave room for two chunks of one.
    static constexpr int tiles(bool out) { return (out ? 2 : 1) * Keys::kBytes + Values::kBytes; }
    static constexpr int stages(bool out) {
        const int fit = 160 * 1024 / kWavesASimd / tiles(out), most = VEC ? 4 : 2;
        return fit < most ? fit : most;
    }
    static constexpr int loads(bool out) { return tiles(out) / 1024 / WAVES; }   // of a wave and chunk
    static constexpr int stores = C * 32 * sizeof(T) / 1024;
};

// The rows of one head of a tensor in the order that a walk goes over them, a chunk at a
// time: a buffer of its n rows.  Rows past the end lie outside it, behind it or, against
// time, in front (their offsets are negative, far behind as unsigned ones); they and the
// columns from `width` on read as zero and are not written.
template <typename T>
struct Rows {
    T *p;                // the head's values in the walk's first row
    int64_t ld;          // values between rows, negative against time
    int width;
    unsigned char *next; // lowest row of the next whole chunk
    int64_t step;        // bytes between chunks
    int bytes, back;     // between rows; the same against time, else 0

    __device__ __forceinline__ Rows(const void *head, int64_t first, int64_t ld_, int64_t sign, int width_)
        : p(static_cast<T *>(const_cast<void *>(head)) + first * ld_), ld(sign * ld_), width(width_),
          step(sign * ld_ * C * static_cast<int64_t>(sizeof(T))), bytes(static_cast<int>(ld_) * static_cast<int>(sizeof(T))),
          back(sign < 0 ? bytes : 0) {}
    __device__ __forceinline__ void seek(int64_t t) {
        next = reinterpret_cast<unsigned char *>(p + t * ld) - static_cast<int64_t>(C - 1) * back;
    }
    // Offset of a value of a row of a chunk; in a chunk of n rows less missing(n), which
    // leaves one outside outside: unsigned, it stays past the buffer's 2^30 bytes or fewer.
    __device__ __forceinline__ int offset(int row, int value) const {
        return value >= width ? INT32_MIN : (back ? C - 1 - row : row) * bytes + value * static_cast<int>(sizeof(T));
    }
    __device__ __forceinline__ int missing(int n) const { return (C - n) * back; }
    static __device__ __forceinline__ int less(int offset, int missing) {
        return static_cast<int>(static_cast<uint32_t>(offset) - static_cast<uint32_t>(missing));
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(int n) const {
        return __builtin_amdgcn_make_buffer_rsrc(next + missing(n), 0, (n - 1) * bytes + width * static_cast<int>(sizeof(T)),
                                                 0x00020000);
    }
};

// A tile's way from memory.
template <typename S, typename L>
struct Feed {
    typedef typename S::Type T;
    typedef __attribute__((address_space(3))) void Lds;
    static constexpr int N = L::kBytes / 1024 / S::WAVES;    // instructions of 1024 bytes a wave
    int off[S::VEC ? N : 1];
    u32x4 r[S::VEC ? 1 : N];

    // Row and chunk of this lane's 16 bytes of instruction i.
    static __device__ __forceinline__ int row(int i) {
        return (i * S::threads + static_cast<int>(threadIdx.x)) / L::kChunks;
    }
    static __device__ __forceinline__ int chunk(int i) {
        return static_cast<int>(threadIdx.x) % L::kChunks ^ L::swizzle(row(i));
    }
    __device__ __forceinline__ explicit Feed(const Rows<T> &R) {
        if constexpr (S::VEC)
#pragma unroll
            for (int i = 0; i < N; ++i) off[i] = R.offset(row(i), chunk(i) * L::E);
    }
    // Straight into LDS.
    __device__ __forceinline__ void send(Rows<T> &R, int n, int wave, unsigned char *__restrict__ tile) const {
#if defined(__HIP_DEVICE_COMPILE__)   // with the builtin in it, the host pass leaves out the kernel's handle
        const auto rsrc = R.buffer(n);
        if (n == C) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (Lds *)(tile + (i * S::WAVES + wave) * 1024), 16, off[i], 0, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (Lds *)(tile + (i * S::WAVES + wave) * 1024), 16,
                                                         R.less(off[i], R.missing(n)), 0, 0, 0);
        }
        R.next += R.step;
#endif
    }
    // Through registers: rows begin at any element.
    __device__ __forceinline__ void fetch(const Rows<T> &R, int64_t t, int n) {
        typedef u32x4 Any __attribute__((aligned(2)));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            r[i] = u32x4{0, 0, 0, 0};
            const int c = chunk(i) * L::E;
            if (row(i) >= n || c >= R.width) continue;
            const T *p = R.p + (t + row(i)) * R.ld + c;
            if (c + L::E <= R.width) {
                r[i] = *reinterpret_cast<const Any *>(p);
            } else {
                T v[L::E] = {};
#pragma unroll
                for (int x = 0; x < L::E; ++x)
                    if (c + x < R.width) v[x] = p[x];
                r[i] = *reinterpret_cast<const u32x4 *>(v);
            }
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
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N < 63 ? N : 63) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
}

// A wave's outputs: lane l holds columns 8 (l / 32) + {0..7} and those 16 further on of row
// l % 32.  Lanes swap halves so that one store writes whole 64 or 128 bytes of 16 rows: row
// 16 i + l % 16, columns out_column(l) + {0..7}.
__device__ __forceinline__ int out_column(int lane) { return 8 * (lane / 32) + 16 * (lane / 16 % 2); }
__device__ __forceinline__ void swap_rows(uint32_t &a, uint32_t &b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void store_vectors(__amdgpu_buffer_rsrc_t to, const int (&off)[2], int missing, const float *f, uint16_t) {
    bf16x8 x, y;
    pack(x, f);
    pack(y, f + 8);
    u32x4 v[2] = {__builtin_bit_cast(u32x4, x), __builtin_bit_cast(u32x4, y)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t a = v[0][j], b = v[1][j];
        swap_rows(a, b);
        v[0][j] = a;
        v[1][j] = b;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) __builtin_amdgcn_raw_buffer_store_b128(v[i], to, Rows<uint16_t>::less(off[i], missing), 0, 0);
}
// In float32 a lane's eight columns are two vectors, and rows may end between them.
__device__ __forceinline__ void store_vectors(__amdgpu_buffer_rsrc_t to, const int (&off)[4], int missing, const float *f, float) {
    uint32_t v[2][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[0][j] = __float_as_uint(f[j]);
        v[1][j] = __float_as_uint(f[8 + j]);
        swap_rows(v[0][j], v[1][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        __builtin_amdgcn_raw_buffer_store_b128(
            u32x4{v[i / 2][4 * (i % 2)], v[i / 2][4 * (i % 2) + 1], v[i / 2][4 * (i % 2) + 2], v[i / 2][4 * (i % 2) + 3]}, to,
            Rows<float>::less(off[i], missing), 0, 0);
}
// The same without whole vectors: eight columns side by side of which `left` exist.
__device__ __forceinline__ void store8(uint16_t *p, const float *f, int left) {
    typedef u32x4 Any __attribute__((aligned(2)));
    bf16x8 b;
    pack(b, f);
    const u32x4 v = __builtin_bit_cast(u32x4, b);
    if (left >= 8) {
        *reinterpret_cast<Any *>(p) = v;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) p[j] = static_cast<uint16_t>(v[j / 2] >> 16 * (j % 2));
    }
}
__device__ __forceinline__ void store8(float *p, const float *f, int left) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < left) p[j] = f[j];
}

// Workgroups go to the eight XCDs in turn: each gets a run of consecutive positions, so
// that walks over one head's rows share its L2.
__device__ __forceinline__ int64_t position() {
    const int n = gridDim.x, x = blockIdx.x % 8;
    return static_cast<int64_t>(x) * (n / 8) + min(x, n % 8) + blockIdx.x / 8;
}

// What a workgroup walks.
struct Place {
    int role, slice, seg;
    int64_t h, b;
    __device__ __forceinline__ explicit Place(const Walks &W) {
        int slices = 0;
        for (int i = 0; i < W.count; ++i) slices = max(slices, W.w[i].slices);
        // below 2^32: the grid is
        uint32_t at = static_cast<uint32_t>(position());
        role = at % W.count;
        at /= W.count;
        slice = at % slices;
        at /= slices;
        h = at % static_cast<uint32_t>(W.heads);
        at /= static_cast<uint32_t>(W.heads);
        seg = at % W.segments;
        b = at / W.segments;
    }
};

// The state of a lane: column column_of(lane % 32) of the wave's 32; element j of block kb
// is row 32 kb + 16 (j / 8) + 8 (lane / 32) + j % 8.
__device__ __forceinline__ int state_row(int kb, int j, int half) { return 32 * kb + 16 * (j / 8) + 8 * half + j % 8; }

// Nothing moves over this: left alone, the compiler reads every fragment from LDS just
// before its product and waits for each.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// X <- g X + (keys)^T (weights * values): the keys exact, their partners in bfloat16 as the
// sum of three roundings, which hold a float32: with two the state is off by 2.7e-6 in the
// root mean square, with three by what float32 sums are, 2e-7 (2 x 4096 x 20 x 128 forward
// 90 us and 96 us).
template <typename S, typename Frag, int KB>
__device__ __forceinline__ void advance(f32x16 (&X)[KB], const unsigned char *Ks, const Frag (&vf)[2], const float *weight,
                                        float g, int lane) {
    typedef typename S::Type T;
    constexpr int kAhead = KB < 4 ? KB : 4;          // fragments under way
    Frag a[kAhead];
    auto load = [&](int i) { a[i % kAhead] = load_col<typename S::Keys>(Ks, i / KB * 16, i % KB * 32, lane, T()); };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i);
    in_order();
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 16; ++j) X[kb][j] *= g;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        float u[8];
        constexpr int kParts = sizeof(T) == 2 ? 3 : 1;
        Frag part[kParts];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = weight[8 * s + j] * get(vf[s], j);
        split(part, u, [](Frag &) {});
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int i = s * KB + kb;
#pragma unroll
            for (int j = 0; j < kParts; ++j) mma(X[kb], a[i % kAhead], part[j]);
            if (i + kAhead < 2 * KB) load(i + kAhead);
            in_order();
        }
    }
}

template <typename S>
__global__ __launch_bounds__(S::threads, S::kWavesASimd) void attention_walk_kernel(const Walks W) {
    typedef typename S::Type T;
    typedef typename S::Frag Frag;
    constexpr int KB = S::KB, KS = 2 * KB;
    constexpr int kStages = S::stages(true), kTiles = S::tiles(true), kLoads = S::loads(true);
    static_assert(kStages >= 2, "a stage is filled while another is read");
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];

    const Place at(W);
    const Walk &w = W.w[at.role];
    const int seg = at.seg;
    const int64_t h = at.h, b = at.b;
    if (at.slice >= w.slices) return;
    int64_t start, len;
    sequence(W, b, &start, &len);
    const int64_t t0 = seg * W.segment;
    const bool tail = seg == W.segments - 1;       // walks to the end, however far
    const int64_t t1 = tail ? len : min(len, t0 + W.segment);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, half = lane / 32, col = lane % 32;
    const int v0 = at.slice * S::VP, width = min(S::VP, w.B - v0);

    if (W.cu && ((b == 0 && seg == 0) || (b == W.seqs - 1 && tail))) {
        // rows in front of the first sequence and behind the last one
        for (int side = 0; side < 2; ++side) {
            if (side == 0 ? !(b == 0 && seg == 0) : !(b == W.seqs - 1 && tail)) continue;
            const int64_t lo = side == 0 ? 0 : start + len, hi = side == 0 ? start : W.total;
            T *o = static_cast<T *>(w.o) + h * w.B + v0;
            for (int64_t id = threadIdx.x; id < (hi - lo) * width; id += S::threads)
                o[(lo + id / width) * W.heads * w.B + id % width] = T(0);
        }
    }
    if (t0 >= len && seg > 0) return;

    const int64_t row_first = w.reverse ? start + len - 1 : start, sign = w.reverse ? -1 : 1;
    const int64_t lda = W.heads * w.A, ldb = W.heads * w.B;
    Rows<T> q(static_cast<const T *>(w.q) + h * w.A, row_first, lda, sign, w.A);
    Rows<T> k(static_cast<const T *>(w.k) + h * w.A, row_first, lda, sign, w.A);
    Rows<T> v(static_cast<const T *>(w.v) + h * w.B + v0, row_first, ldb, sign, width);
    Rows<T> o(static_cast<const T *>(w.o) + h * w.B + v0, row_first, ldb, sign, width);
    q.seek(t0);
    k.seek(t0);
    v.seek(t0);
    o.seek(t0);
    Feed<S, typename S::Keys> kin(k), qin(q);
    Feed<S, typename S::Values> vin(v);
    const int my_out = 32 * wave + 8 * half;      // first of the outputs of row col
    constexpr int kStores = S::stores;
    int out_off[kStores];                         // of the vectors that this lane stores
#pragma unroll
    for (int i = 0; i < kStores; ++i)
        out_off[i] = o.offset(16 * (2 * i / kStores) + lane % 16, 32 * wave + out_column(lane) + (kStores == 4 ? 4 * (i % 2) : 0));
    const int count = static_cast<int>((t1 - t0 + C - 1) / C), n_last = static_cast<int>(t1 - t0) - (count - 1) * C;
    auto steps = [&](int c) { return c == count - 1 ? n_last : C; };
    auto send = [&](int c, int stage) {
        unsigned char *const to = smem + stage * kTiles;
        kin.send(k, steps(c), wave, to);
        vin.send(v, steps(c), wave, to + S::Keys::kBytes);
        qin.send(q, steps(c), wave, to + S::Keys::kBytes + S::Values::kBytes);
    };
    auto fetch = [&](int c) {
        kin.fetch(k, t0 + c * C, steps(c));
        vin.fetch(v, t0 + c * C, steps(c));
        qin.fetch(q, t0 + c * C, steps(c));
    };
    if constexpr (S::VEC) {
        for (int c = 0; c < kStages - 1; ++c)
            if (c < count) send(c, c);
    } else {
        if (count > 0) fetch(0);
    }

    const float ld = decay_log2(W.log_decay, h);
    const int e = w.early;
    auto power = [&](int n) { return fast_exp2(ld * static_cast<float>(n)); };
    const int my_v = v0 + 32 * wave + column_of(col);    // column of this lane's state
    const int64_t bh = b * W.heads + h, states = static_cast<int64_t>(w.A) * w.B;
    f32x16 X[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 16; ++j) X[kb][j] = 0.0f;
    if (seg > 0 || w.first) {
        // at most 256 x 256 values; what the state does not have reads as zero
        const float *from = seg > 0 ? w.segments + ((b * (W.segments - 1) + seg - 1) * W.heads + h) * states : w.first + bh * states;
        const int sa = static_cast<int>(seg > 0 ? w.seg_sa : w.first_sa), sb = static_cast<int>(seg > 0 ? w.seg_sb : w.first_sb);
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(from), 0, static_cast<int>(states) * 4, 0x00020000);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int a = state_row(kb, j, half);
                const int off = a < w.A && my_v < w.B ? (a * sa + my_v * sb) * 4 : INT32_MIN;
                X[kb][j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsrc, off, 0, 0));
            }
    }

    // decays inside a chunk: of outputs (this lane's is col) from its inputs (0 from later
    // ones) and from the state in front, and of the inputs to the state behind
    float inside[16], weight[16];
    Mask<Frag> earlier[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) earlier[s] = mask_of(Frag{}, col - 16 * s - 4 * half);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int row = acc_row(j) + 4 * half;
        inside[j] = row <= col ? w.inner * w.scale * power(col - row) : 0.0f;
        weight[j] = w.inner * power(C - e - row);
    }
    const float front = w.scale * power(col + e);
    float whole = power(C);

    int stage = 0, to_fill = kStages - 1;
    for (int c = 0; c < count; ++c) {
        const int n = steps(c);
        unsigned char *const Ks = smem + stage * kTiles, *const Vs = Ks + S::Keys::kBytes, *const Qs = Vs + S::Values::kBytes;
        if constexpr (S::VEC) {
            // What is under way behind this chunk's loads may stay so: those of the next
            // chunks and the outputs sent after them.  Then every wave has read the stage
            // that the next loads go to.
            constexpr int kAhead = kStages - 2;
            if (kAhead == 0 || c + kAhead >= count) wait_and_meet<0>();
            else if (c < kAhead) wait_and_meet<kAhead * kLoads>();
            else wait_and_meet<kAhead * (kLoads + S::stores)>();
            if (c + kStages - 1 < count) send(c + kStages - 1, to_fill);
        } else {
            kin.store(Ks);
            vin.store(Vs);
            qin.store(Qs);
            __syncthreads();                      // who reads the other stage has read it
            if (c + 1 < count) fetch(c + 1);
        }
        to_fill = stage;
        stage = stage == kStages - 1 ? 0 : stage + 1;
        if (n < C) {                              // the last chunk
            whole = power(n);
#pragma unroll
            for (int j = 0; j < 16; ++j) weight[j] = w.inner * power(max(n - e - acc_row(j) - 4 * half, 0));
        }

        constexpr int kAhead = KS < 4 ? KS : 4;   // pairs of fragments under way
        Frag vf[2], qf[kAhead], kf[kAhead];
        auto load = [&](int i) {
            qf[i % kAhead] = load_row<typename S::Keys>(Qs, col, 16 * i + 8 * half, T());
            kf[i % kAhead] = load_row<typename S::Keys>(Ks, col, 16 * i + 8 * half, T());
        };
#pragma unroll
        for (int s = 0; s < kAhead; ++s) load(s);
#pragma unroll
        for (int s = 0; s < 2; ++s) vf[s] = load_col<typename S::Values>(Vs, 16 * s, 32 * wave, lane, T());
        in_order();
        f32x16 G, O;
#pragma unroll
        for (int j = 0; j < 16; ++j) G[j] = O[j] = 0.0f;
        // The state, and below the decayed products, enter as matrix operands: in bfloat16 as
        // the sum of two roundings, 2^-18 off, which an output stored in bfloat16 hides (one
        // alone moves outputs from 0.0017 to 0.0023 off in the root mean square; 2 x 4096 x 20 x
        // 128 backward 194 us with one, 214 us with two).
        constexpr int kTerms = sizeof(T) == 2 ? 2 : 1;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            Frag xf[kTerms];
            from_acc(xf, X[s / 2], s % 2, [](Frag &) {});
            mma(G, kf[s % kAhead], qf[s % kAhead]);
#pragma unroll
            for (int i = 0; i < kTerms; ++i) mma(O, xf[i], qf[s % kAhead]);
            if (s + kAhead < KS) load(s + kAhead);
            in_order();
        }
        advance<S>(X, Ks, vf, weight, whole, lane);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            O[j] *= front;
            G[j] *= inside[j];
        }
        // later inputs leave nothing, whatever their products hold
        Frag pf[2][kTerms];
#pragma unroll
        for (int s = 0; s < 2; ++s) from_acc(pf[s], G, s, [&](Frag &f) { keep(f, earlier[s]); });
        auto add_inputs = [&] {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < kTerms; ++i) mma(O, vf[s], pf[s][i]);
        };
        auto put = [&](const f32x16 &r) {
            float out[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) out[j] = r[j];
            if constexpr (S::VEC) {
                store_vectors(o.buffer(n), out_off, o.missing(n), out, T());
            } else if (col < n) {
                T *const to = o.p + (t0 + c * C + col) * o.ld + my_out;
                store8(to, out, width - my_out);
                store8(to + 16, out + 8, width - my_out - 16);
            }
        };
        // The products leave out later inputs by a factor 0, which an infinite or NaN v would
        // carry to earlier outputs of its chunk.  Such values are taken out, and their column
        // is set to NaN from their step on.
        const bool odd = any_odd(vf[0], vf[1]);
        if (!__any(odd)) {
            add_inputs();
            put(O);
        } else {
            int reached = clean(vf[0], 4 * half, clean(vf[1], 16 + 4 * half, C));
            reached = min(reached, __shfl_xor(reached, 32));
            add_inputs();
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (col >= __shfl(reached, acc_row(j) + 4 * half)) O[j] = __builtin_nanf("");
            put(O);
        }
        o.next += o.step;
    }

    if (!w.last || t1 != len || (t1 <= t0 && seg > 0) || my_v >= w.B) return;
    float *to = w.last + bh * states;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int a = state_row(kb, j, half);
            if (a < w.A) to[a * w.last_sa + my_v * w.last_sb] = X[kb][j];
        }
}

// The walk of a segment for its state alone, from zero: for those that others follow, which
// are whole chunks.
template <typename S>
__global__ __launch_bounds__(S::threads, S::kWavesASimd) void attention_state_kernel(const Walks W) {
    typedef typename S::Type T;
    typedef typename S::Frag Frag;
    constexpr int KB = S::KB, kStages = S::stages(false), kTiles = S::tiles(false), kLoads = S::loads(false);
    static_assert(kStages >= 2, "a stage is filled while another is read");
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];

    const Place at(W);
    const Walk &w = W.w[at.role];
    const int seg = at.seg;
    const int64_t h = at.h, b = at.b;
    if (at.slice >= w.slices || seg == W.segments - 1) return;
    int64_t start, len;
    sequence(W, b, &start, &len);
    const int64_t t0 = seg * W.segment;
    if (t0 + W.segment >= len) return;
    const int count = static_cast<int>(W.segment / C);

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, half = lane / 32, col = lane % 32;
    const int v0 = at.slice * S::VP, width = min(S::VP, w.B - v0), my_v = v0 + 32 * wave + column_of(col);
    const int64_t row_first = w.reverse ? start + len - 1 : start, sign = w.reverse ? -1 : 1;
    Rows<T> k(static_cast<const T *>(w.k) + h * w.A, row_first, W.heads * w.A, sign, w.A);
    Rows<T> v(static_cast<const T *>(w.v) + h * w.B + v0, row_first, W.heads * w.B, sign, width);
    k.seek(t0);
    v.seek(t0);
    Feed<S, typename S::Keys> kin(k);
    Feed<S, typename S::Values> vin(v);
    auto send = [&](int stage) {
        kin.send(k, C, wave, smem + stage * kTiles);
        vin.send(v, C, wave, smem + stage * kTiles + S::Keys::kBytes);
    };
    auto fetch = [&](int c) {
        kin.fetch(k, t0 + c * C, C);
        vin.fetch(v, t0 + c * C, C);
    };
    if constexpr (S::VEC) {
        for (int c = 0; c < kStages - 1; ++c)
            if (c < count) send(c);
    } else {
        fetch(0);
    }
    const float ld = decay_log2(W.log_decay, h), whole = fast_exp2(ld * C);
    float weight[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) weight[j] = w.inner * fast_exp2(ld * (C - w.early - acc_row(j) - 4 * half));
    const int64_t states = static_cast<int64_t>(w.A) * w.B;
    f32x16 X[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 16; ++j) X[kb][j] = 0.0f;

    int stage = 0, to_fill = kStages - 1;
    for (int c = 0; c < count; ++c) {
        unsigned char *const Ks = smem + stage * kTiles, *const Vs = Ks + S::Keys::kBytes;
        if constexpr (S::VEC) {
            if (kStages == 2 || c + kStages - 2 >= count) wait_and_meet<0>();
            else wait_and_meet<(kStages - 2) * kLoads>();
            if (c + kStages - 1 < count) send(to_fill);
        } else {
            kin.store(Ks);
            vin.store(Vs);
            __syncthreads();
            if (c + 1 < count) fetch(c + 1);
        }
        to_fill = stage;
        stage = stage == kStages - 1 ? 0 : stage + 1;
        Frag vf[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) vf[s] = load_col<typename S::Values>(Vs, 16 * s, 32 * wave, lane, T());
        advance<S>(X, Ks, vf, weight, whole, lane);
    }
    if (my_v >= w.B) return;
    float *const to = w.segments + ((b * (W.segments - 1) + seg) * W.heads + h) * states;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int a = state_row(kb, j, half);
            if (a < w.A) to[a * w.seg_sa + my_v * w.seg_sb] = X[kb][j];
        }
}

// X_{s+1} = g^n X_s + sum_s in place: slot s receives the state in front of segment s + 1.
// States that are advanced in place are copied first: the walk of a first segment may begin
// after that of the last one, in the same launch, has written over them.
__global__ __launch_bounds__(256) void attention_fold_kernel(const Walks W) {
    const Walk &w = W.w[blockIdx.z];
    const int64_t bh = blockIdx.y, b = bh / W.heads, h = bh % W.heads;
    const int64_t states = static_cast<int64_t>(w.A) * w.B;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (id >= states) return;
    int64_t start, len;
    sequence(W, b, &start, &len);
    // segments that others follow
    const int64_t full = len <= 0 ? 0 : min(int64_t(W.segments - 1), (len - 1) / W.segment);
    const float g = fast_exp2(decay_log2(W.log_decay, h) * static_cast<float>(W.segment));
    const int64_t a = id / w.B, c = id % w.B;
    const int64_t at = bh * states + a * w.first_sa + c * w.first_sb;
    float x = w.first ? w.first[at] : 0.0f;
    if (w.kept) w.kept[at] = x;
    float *p = w.segments + (b * (W.segments - 1) * W.heads + h) * states + a * w.seg_sa + c * w.seg_sb;
    const int64_t next = W.heads * states;
    for (int64_t s = 0; s < full; s += 8, p += 8 * next) {
        float sum[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = s + i < full ? p[i * next] : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x = fmaf(g, x, sum[i]);
            if (s + i < full) p[i * next] = x;
        }
    }
}

// ---- launches ------------------------------------------------------------------

int waves_of(int64_t B) { return B <= 64 ? 2 : 4; }
int slices_of(int64_t B) { return static_cast<int>((B + 32 * waves_of(B) - 1) / (32 * waves_of(B))); }

// Blocks of 32 that A is rounded up to.
int blocks_of(int64_t A) { return A <= 64 ? 2 : A <= 96 ? 3 : A <= 128 ? 4 : A <= 192 ? 6 : 8; }

// Segments of a sequence and their steps: so many that the device's 256 compute units have
// a forward workgroup each; backward, where three walks share a launch, half as many.  Twice
// as many fill units that hold two workgroups, but cost more in states, each written once,
// folded and read again, and end in rounds that are part empty: 2 x 4096 x 20 x 128 in bfloat16
// 98 and, with twice as many, 97 us, backward 214 and 201 us, 131072 steps of 4 heads 251 and
// 240 us, but 8 x 2048 x 16 x 128 backward 233 and 280 us, 4096 steps of 16 heads of 256 148 and
// 187 us, 8 packed sequences of 16 heads of 128 106 and 116 us, backward 200 and 224 us.
// Sequences of different lengths are cut by what all rows together give a workgroup, the
// longest into at most four times what it would be cut into otherwise (7 sequences of 431
// steps in the mean, backward in float32 131 us, cut as if all were as long 154 us).
constexpr int64_t kWorkgroups = 256;
void cut(const AttentionArgs &a, bool bwd, Walks *W) {
    const int64_t slices = std::max(slices_of(a.value), bwd ? slices_of(a.key) : 0), heads = std::max<int64_t>(1, a.heads) * slices;
    const int64_t walks = std::max<int64_t>(1, a.seqs) * heads, each = bwd ? kWorkgroups / 2 : kWorkgroups;
    int64_t n = std::min(each / walks, a.seqlen / (4 * C));
    if (a.total != a.seqs * a.seqlen) {
        const int64_t share = std::max<int64_t>(2 * C, (a.total * heads + each - 1) / each);
        n = std::min((a.seqlen + share - 1) / share, 4 * each / walks);
    }
    n = std::max<int64_t>(1, n);
    W->segment = std::max<int64_t>(C, ((a.seqlen + n - 1) / n + C - 1) / C * C);
    W->segments = static_cast<int>(std::max<int64_t>(1, (a.seqlen + W->segment - 1) / W->segment));
}

template <typename K>
hipError_t launch(K kernel, int64_t blocks, int threads, int lds, const Walks &W, hipStream_t stream) {
    if (lds > 65536)
        if (const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds))
            return e;
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(blocks)), dim3(threads), lds, stream, W);
    return hipGetLastError();
}

// What instantiates the kernels for a walk: A rounded up, waves, whole vectors.
struct Kind {
    int blocks, waves;
    bool vec;
    bool operator==(const Kind &k) const { return blocks == k.blocks && waves == k.waves && vec == k.vec; }
};

Kind kind_of(const Walk &w, int size, bool out) {
    const auto p = [](const void *a) { return reinterpret_cast<uintptr_t>(a); };
    const uintptr_t at = p(w.k) | p(w.v) | (out ? p(w.q) | p(w.o) : 0);
    return Kind{blocks_of(w.A), waves_of(w.B), (at | (w.A | w.B) * size) % 16 == 0};
}

template <typename S>
hipError_t launch_shape(const Walks &W, bool out, hipStream_t stream) {
    int most = 0;
    for (int i = 0; i < W.count; ++i) most = std::max(most, W.w[i].slices);
    const int64_t blocks = W.seqs * W.segments * W.heads * most * W.count;   // below 2^24
    const int lds = S::stages(out) * S::tiles(out);
    return out ? launch(attention_walk_kernel<S>, blocks, S::threads, lds, W, stream)
               : launch(attention_state_kernel<S>, blocks, S::threads, lds, W, stream);
}

template <typename T, int WAVES, bool VEC>
hipError_t launch_kind(const Walks &W, const Kind &k, bool out, hipStream_t stream) {
    switch (k.blocks) {
        case 2: return launch_shape<Shape<T, 2, WAVES, VEC>>(W, out, stream);
        case 3: return launch_shape<Shape<T, 3, WAVES, VEC>>(W, out, stream);
        case 4: return launch_shape<Shape<T, 4, WAVES, VEC>>(W, out, stream);
        case 6: return launch_shape<Shape<T, 6, WAVES, VEC>>(W, out, stream);
        default: return launch_shape<Shape<T, 8, WAVES, VEC>>(W, out, stream);
    }
}

// Walks of one kind share a launch: with their outputs, or for the states in front of
// their segments.
template <typename T>
hipError_t launch_all(const Walks &W, bool out, hipStream_t stream) {
    bool done[3] = {false, false, false};
    for (int i = 0; i < W.count; ++i) {
        if (done[i]) continue;
        const Kind kind = kind_of(W.w[i], sizeof(T), out);
        Walks G = W;
        G.count = 0;
        for (int j = i; j < W.count; ++j)
            if (!done[j] && kind_of(W.w[j], sizeof(T), out) == kind) {
                G.w[G.count++] = W.w[j];
                done[j] = true;
            }
        for (int j = G.count; j < 3; ++j) G.w[j] = G.w[0];
        const hipError_t e = kind.waves == 2 ? (kind.vec ? launch_kind<T, 2, true>(G, kind, out, stream) : launch_kind<T, 2, false>(G, kind, out, stream))
                                             : (kind.vec ? launch_kind<T, 4, true>(G, kind, out, stream) : launch_kind<T, 4, false>(G, kind, out, stream));
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

Walks common(const AttentionArgs &a, bool bwd) {
    Walks W{};
    W.cu = a.cu_seqlens;
    W.log_decay = a.log_decay;
    W.seqs = a.seqs; W.seqlen = a.seqlen; W.total = a.total; W.heads = a.heads;
    cut(a, bwd, &W);
    return W;
}

// The states in front of the segments of W's walks.
hipError_t prepare(const Walks &W, bool f32, hipStream_t stream) {
    if (W.segments == 1) return hipSuccess;
    hipError_t e = f32 ? launch_all<float>(W, false, stream) : launch_all<uint16_t>(W, false, stream);
    if (e != hipSuccess) return e;
    int64_t most = 0;
    for (int i = 0; i < W.count; ++i) most = std::max(most, static_cast<int64_t>(W.w[i].A) * W.w[i].B);
    hipLaunchKernelGGL(attention_fold_kernel,
                       dim3(static_cast<uint32_t>((most + 255) / 256), static_cast<uint32_t>(W.seqs * W.heads), W.count),
                       dim3(256), 0, stream, W);
    return hipGetLastError();
}

// Floats of a walk's states in the workspace.
int64_t floats_of(const AttentionArgs &a, const Walks &W) {
    return static_cast<int64_t>(W.segments - 1) * a.seqs * a.heads * a.key * a.value;
}

// ---- one step ------------------------------------------------------------------

// A workgroup holds 32 columns of one state, VEC of them a lane; groups of lanes take the
// rows in turn.  Bound by the state's bytes, or by one workgroup's loads where states are
// few.  Whole lines of 128 columns give a workgroup four times the loads in turn and gain
// nothing back: 20, 320, 640 and 1280 states of 128 x 128 take the kernel 5.5, 11.7, 19.9 and
// 35.7 us, with 128 columns 10.4, 15.3, 20.4 and 35.7 us (over 1 GB of states in turn, which
// the device's cache does not hold).
template <typename T, int VEC>
__global__ __launch_bounds__(256) void attention_step_kernel(float *__restrict__ state, const T *__restrict__ q,
                                                             const T *__restrict__ k, const T *__restrict__ v,
                                                             const float *__restrict__ log_decay, float scale,
                                                             T *__restrict__ o, int heads, int K, int V, int slices) {
    constexpr int COLS = 32, LANES = COLS / VEC, GROUPS = 256 / LANES;
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
    const int64_t slices = (a.value + 31) / 32;
    const bool vec = a.value % 4 == 0 && reinterpret_cast<uintptr_t>(a.h_last) % 16 == 0;
    hipLaunchKernelGGL((vec ? attention_step_kernel<T, 4> : attention_step_kernel<T, 1>),
                       dim3(static_cast<uint32_t>(a.seqs * a.heads * slices)), dim3(256), 0, stream, a.h_last,
                       static_cast<const T *>(a.q), static_cast<const T *>(a.k), static_cast<const T *>(a.v),
                       a.log_decay, a.scale, static_cast<T *>(a.o), static_cast<int>(a.heads),
                       static_cast<int>(a.key), static_cast<int>(a.value), static_cast<int>(slices));
    return hipGetLastError();
}

}  // namespace

// The forward's holds a copy of h0 too, since the query does not know whether h0 is h_last.
size_t linear_attention_workspace(const AttentionArgs &a, bool bwd) {
    const Walks W = common(a, bwd);
    const int64_t floats = floats_of(a, W), copy = W.segments > 1 ? a.seqs * a.heads * a.key * a.value : 0;
    return static_cast<size_t>(bwd ? 2 * floats : floats + copy) * sizeof(float);
}

hipError_t launch_linear_attention_fwd(const AttentionArgs &a, void *workspace, hipStream_t stream) {
    Walks W = common(a, false);
    const bool f32 = a.io == IO_F32;
    const size_t bytes = linear_attention_workspace(a, false);
    void *ws = workspace;
    if (bytes && !ws)
        if (const hipError_t e = scratch_alloc(&ws, bytes, stream)) return e;
    const int K = static_cast<int>(a.key), V = static_cast<int>(a.value);
    float *S = static_cast<float *>(ws);
    W.count = 1;
    float *const kept = W.segments > 1 && a.h0 && a.h0 == a.h_last ? S + floats_of(a, W) : nullptr;
    W.w[0] = Walk{a.q, a.k, a.v, a.o, a.h0, a.h_last, S, kept, V, 1, V, 1, V, 1, K, V,
                  slices_of(V), 1, 0, 1.0f, a.scale};
    W.w[1] = W.w[2] = W.w[0];
    hipError_t e = prepare(W, f32, stream);
    if (kept) W.w[0].first = W.w[1].first = W.w[2].first = kept;
    if (e == hipSuccess) e = f32 ? launch_all<float>(W, true, stream) : launch_all<uint16_t>(W, true, stream);
    if (bytes && !workspace) {
        const hipError_t f = scratch_free(ws, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

hipError_t launch_linear_attention_bwd(const AttentionArgs &a, void *workspace, hipStream_t stream) {
    Walks W = common(a, true);
    const bool f32 = a.io == IO_F32;
    const size_t bytes = linear_attention_workspace(a, true);
    void *ws = workspace;
    if (bytes && !ws)
        if (const hipError_t e = scratch_alloc(&ws, bytes, stream)) return e;
    const int K = static_cast<int>(a.key), V = static_cast<int>(a.value);
    float *S = static_cast<float *>(ws), *R = S + floats_of(a, W);
    // S^T in (V, K) as the first walk forms it; R in (K, V) as the third does
    const Walk dq{a.dout, a.v, a.k, a.dq, a.h0, nullptr, S, nullptr, 1, V, 0, 0, K, 1, V, K, slices_of(K), 1, 0, 1.0f, a.scale};
    const Walk dk{a.v, a.dout, a.q, a.dk, a.dh_last, nullptr, R, nullptr, 1, V, 0, 0, 1, V, V, K, slices_of(K), 0, 1, a.scale, 1.0f};
    const Walk dv{a.k, a.q, a.dout, a.dv, a.dh_last, a.dh0, R, nullptr, V, 1, V, 1, V, 1, K, V, slices_of(V), 0, 1, a.scale, 1.0f};
    W.count = 2;
    W.w[0] = dq;
    W.w[1] = dv;
    W.w[2] = dq;
    hipError_t e = prepare(W, f32, stream);
    W.count = 3;
    W.w[0] = dq;
    W.w[1] = dk;
    W.w[2] = dv;
    if (e == hipSuccess) e = f32 ? launch_all<float>(W, true, stream) : launch_all<uint16_t>(W, true, stream);
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
