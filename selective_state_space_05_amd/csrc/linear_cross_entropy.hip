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
// All three products run on one kernel, C[m, n] = sum_k A[m, k] B[n, k], whose
// operands are stored either along k (hidden and weight for the logits, p for
// dhidden) or across it (weight for dhidden, hidden and p for dweight): the
// second kind is transposed on its way from LDS to registers, so that no
// transposed copy of anything is ever written.
//
// Bound by the matrix cores and, at their full rate, by the clock that the card
// holds under them (1.75 to 2.0 GHz); few tokens by the read of weight.  Measured at
// width 2560 and 50021 words in bfloat16: 8192 tokens forward 1.76 to 1.87 ms (1.12
// to 1.19 PFLOP/s), backward 5.65 to 5.77 ms (1.09 to 1.11), 16 tokens forward 66 us
// (58 us of it reading weight at 4.4 TB/s); float32, 2048 tokens of width 1024 and
// 32000 words, forward 1.0 ms (134 TFLOP/s).
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

// One operand: `rows` rows of the product, 16-byte aligned, `ld` bytes apart
// where a row's k lie side by side; where the rows lie side by side (ACROSS),
// it is the k that are `ld` bytes apart.  k: how many there are.
struct Rows {
    const unsigned char *p;
    int64_t ld;
    int rows, k;
};

// Row of C inside a 32 x 32 block that element e of a lane's accumulator is
// (its column is lane % 32): four consecutive rows for every four elements.
__device__ __forceinline__ int acc_row(int e, int lane) { return 8 * (e / 4) + 4 * (lane / 32) + e % 4; }

// A workgroup's tile of C and a wave's part of it.  Two waves a SIMD in all cases,
// so that one forms products while the other meets its workgroup at a barrier:
// tiles of 256 x 256 in four waves of 128 x 128, which read a third less from LDS
// but stand alone on their SIMD, take 5.93 ms instead of 5.65 for the backward of
// 8192 tokens x 2560 x 50021, and 215 us instead of 201 for the forward of 4096 x
// 768 x 32000.
template <int BM_, int BN_, int WM_, int WN_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int I = WM / 32, J = WN / 32, waves_m = BM / WM;
    static constexpr int waves = (BM / WM) * (BN / WN), threads = 64 * waves;
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

// One operand of a tile on its way: N rows, T their type.  A step is kRowBytes of
// k of every row: kStepK values of k.  Loads move 16 bytes a lane straight into
// LDS, in lane order; the lanes fetch the 16-byte chunks permuted, so that the
// fragment reads find different banks.
template <typename T, int N, bool ACROSS>
struct Operand {
    static constexpr int kStepK = kRowBytes / sizeof(T);
    static constexpr int kLoads = N * kRowBytes / 1024;              // instructions of a step
    static constexpr int kLine = ACROSS ? N * static_cast<int>(sizeof(T)) : kRowBytes;   // bytes of a line in LDS
    static constexpr int kLineChunks = kLine / 16, kLines = 1024 / kLine;               // lines of one instruction
    static constexpr int kFragmentReads = !ACROSS ? 1 : sizeof(T) == 2 ? 2 : 4;
    typedef __attribute__((address_space(3))) void Lds;

    const unsigned char *base;
    int64_t left;                // bytes from the current step to the end (ACROSS)
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t ld, lane_off;
    int chunk, chunks;           // this lane's chunk of a line; chunks of k in all (not ACROSS)

    // Chunks of line l are permuted by this, so that the lanes served together (256
    // bytes a cycle) cover all 64 banks.  Along k, 16 lanes read one chunk of 16
    // lines, four to 256 bytes; across it (bfloat16), 32 lanes read four chunks of
    // four lines.
    static __device__ __forceinline__ int swizzle(int l) {
        if (!ACROSS) return (l / 4) % kChunks;
        return sizeof(T) == 2 ? (4 * (l % 4)) & (kLineChunks - 1) : 0;
    }

    __device__ __forceinline__ void init(const Rows &R, int first, int wave, int lane) {
        ld = static_cast<uint32_t>(R.ld);
        const int line = lane / kLineChunks;
        chunk = (lane % kLineChunks) ^ swizzle(wave * kLines + line);   // a wave's loads are four apart
        lane_off = line * ld + chunk * 16;
        if (ACROSS) {
            base = R.p + static_cast<int64_t>(first) * sizeof(T);
            left = static_cast<int64_t>(R.k) * R.ld - static_cast<int64_t>(first) * sizeof(T);
            chunks = 0;
        } else {
            // rows past the end lie past the buffer's end and read as zero (the
            // scalar offset is checked too; the minimum is formed in a vector register)
            const int n = __builtin_amdgcn_readfirstlane(min(R.rows - first, N));
            base = R.p + first * R.ld;
            rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char *>(base), 0, n * static_cast<int>(R.ld),
                                                     0x00020000);
            chunks = static_cast<int>((R.k * static_cast<int64_t>(sizeof(T)) + 15) / 16);
        }
    }
    __device__ __forceinline__ void seek(int step) {
        if (ACROSS) {
            base += static_cast<int64_t>(step) * kStepK * ld;
            left -= static_cast<int64_t>(step) * kStepK * ld;
        }
    }
    // Load instruction q (of kLoads) of a step into `to`; k past the end reads as
    // zero.  Across k, steps are asked for one after the other.
    __device__ __forceinline__ void load(int step, int q, unsigned char *__restrict__ to) const {
        if (ACROSS)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (Lds *)(to + q * 1024), 16, lane_off, q * kLines * ld, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (Lds *)(to + q * 1024), 16,
                                                     step * kChunks + chunk < chunks ? lane_off : 0xffffffffu,
                                                     q * kLines * ld + step * kRowBytes, 0, 0);
    }
    __device__ __forceinline__ void begin_step() {
        if (ACROSS) {
            const int64_t n = left < 0 ? 0 : left < 0x7fffffff ? left : 0x7fffffff;
            rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char *>(base), 0, static_cast<int>(n), 0x00020000);
        }
    }
    __device__ __forceinline__ void end_step() { seek(1); }

    // The 16 bytes of k that this lane holds of row `row` + lane % 32 in half
    // `half` of the step at `from`.  __restrict__ here and in load(): a stage is
    // read only after its loads were waited for, and without the promise the
    // compiler waits for every load under way before a transposing read.
    static __device__ __forceinline__ u32x4 fragment(const unsigned char *__restrict__ from, int row, int half, int lane) {
        if constexpr (!ACROSS) {
            const int c = (2 * half + lane / 32) ^ swizzle(lane % 32);
            return *reinterpret_cast<const u32x4 *>(from + (lane % 32) * kRowBytes + c * 16 + row * kRowBytes);
        } else if constexpr (sizeof(T) == 2) {
            // A transposing read gives the 16 lanes of a group the columns of a
            // 4 x 16 block whose lines lie in lanes 4 j .. 4 j + 3: lane i fetches
            // 8 bytes of line i / 4.
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4 LdsRow;
            const int i = lane % 16, line = 8 * (lane / 32) + i / 4, x = 2 * (lane / 16 % 2) + i % 4 / 2;
            const int c = row / 128 * 16 + ((row / 32 % 4 * 4 + x) ^ swizzle(line));   // 32 rows: four chunks
            const unsigned char *at = from + (16 * half + line) * kLine + c * 16 + i % 2 * 8;
            const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsRow *)at));
            const uint2 hi = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsRow *)(at + 4 * kLine)));
            return u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {
            const unsigned char *at = from + 4 * (2 * half + lane / 32) * kLine + (row + lane % 32) * 4;
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t *>(at + j * kLine);
            return v;
        }
    }
};

// C[m, n] = sum_k A[m, k] B[n, k] for one tile and the steps [first, first + steps)
// of k.  A step's rows move three steps ahead; a wave's operand fragments are
// read half a step ahead of the products that use them, the first ones of a step
// right after its barrier, under the last products of the step before.
template <typename T, typename Shape, bool AX, bool BX>
__device__ __forceinline__ void product_tile(const Rows &A, const Rows &B, int first, int steps, int m0, int n0,
                                             unsigned char *lds, f32x16 (&acc)[Shape::I][Shape::J]) {
    constexpr int I = Shape::I, J = Shape::J;
    typedef Operand<T, Shape::BM, AX> OpA;
    typedef Operand<T, Shape::BN, BX> OpB;
    constexpr int kMineA = OpA::kLoads / Shape::waves, kMineB = (OpB::kLoads + Shape::waves - 1) / Shape::waves;   // B's last may repeat
    static_assert(OpA::kLoads % Shape::waves == 0, "each of a wave's loads is of one operand");
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    OpA a;
    OpB b;
    a.init(A, m0, wave, lane);
    b.init(B, n0, min(wave, OpB::kLoads - 1), lane);
    a.seek(first);
    b.seek(first);
    const auto load = [&](int step) {
        unsigned char *to = lds + (step % kStages) * Shape::stage;
        a.begin_step();
        b.begin_step();
#pragma unroll
        for (int s = 0; s < kMineA; ++s) a.load(first + step, wave + s * Shape::waves, to);
#pragma unroll
        for (int s = 0; s < kMineB; ++s)
            b.load(first + step, min(wave + s * Shape::waves, OpB::kLoads - 1), to + Shape::BM * kRowBytes);
        a.end_step();
        b.end_step();
    };
    const int wm = (wave % Shape::waves_m) * Shape::WM, wn = (wave / Shape::waves_m) * Shape::WN;
    u32x4 fa[2][I], fb[2][J];
    const auto read = [&](int step, int half) {
        const unsigned char *from = lds + (step % kStages) * Shape::stage;
#pragma unroll
        for (int i = 0; i < I; ++i) fa[half][i] = OpA::fragment(from, wm + 32 * i, half, lane);
#pragma unroll
        for (int j = 0; j < J; ++j) fb[half][j] = OpB::fragment(from + Shape::BM * kRowBytes, wn + 32 * j, half, lane);
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

    constexpr int kAhead = (kStages - 2) * (kMineA + kMineB);
    for (int s = 0; s < kStages - 1; ++s) load(s);
    wait_and_meet<kAhead>();
    load(kStages - 1);
    read(0, 0);
    read(0, 1);
    multiply(0);
    // The compiler would sink the fragment reads to just before their products
    // (fewer registers, and every wait shows): they go first, then the products
    // with the loads among them.
    constexpr int kReads = I * OpA::kFragmentReads + J * OpB::kFragmentReads;
    constexpr int kProducts = I * J * (sizeof(T) == 2 ? 1 : 4), kMine = kMineA + kMineB;
    enum { kMfma = 0x8, kVmem = 0x20, kDsRead = 0x100 };
    for (int step = 1; step < steps; ++step) {
        wait_and_meet<kAhead>();
        read(step, 0);
        load(step + kStages - 1);
        multiply(1);
        __builtin_amdgcn_sched_group_barrier(kDsRead, kReads, 0);
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
            __builtin_amdgcn_sched_group_barrier(kMfma, kProducts / kMine, 0);
            __builtin_amdgcn_sched_group_barrier(kVmem, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(kMfma, kProducts, 0);
        __builtin_amdgcn_sched_barrier(0);
        read(step, 1);
        multiply(0);
        __builtin_amdgcn_sched_group_barrier(kDsRead, kReads, 1);
        __builtin_amdgcn_sched_group_barrier(kMfma, kProducts, 1);
        __builtin_amdgcn_sched_barrier(0);
    }
    multiply(1);
}

// One product: the tiles of C, each `splits` times over as many runs of
// `steps` steps of k.
struct Problem {
    Rows A, B;
    int mt, nt, splits, steps;
};

template <typename Epilogue, bool AX, bool BX>
struct Job {
    static constexpr bool kAX = AX, kBX = BX;
    Problem p;
    Epilogue e;
};

template <typename T, typename Shape, typename J>
__device__ __forceinline__ void run_tile(const J &job, int id, unsigned char *lds) {
    int mi, ni;
    const int n = job.p.mt * job.p.nt, split = id / n;
    tile_of(id - split * n, n, job.p.mt, job.p.nt, &mi, &ni);
    const int m0 = __builtin_amdgcn_readfirstlane(mi * Shape::BM), n0 = __builtin_amdgcn_readfirstlane(ni * Shape::BN);
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = (wave % Shape::waves_m) * Shape::WM, wn = (wave / Shape::waves_m) * Shape::WN;
    // what the epilogue reads of its columns is loaded before the products
    const auto columns = job.e.template begin<Shape>(m0 + wm, n0 + wn, lane);
    f32x16 acc[Shape::I][Shape::J];
    product_tile<T, Shape, J::kAX, J::kBX>(job.p.A, job.p.B, split * job.p.steps, job.p.steps, m0, n0, lds, acc);
    job.e.template tile<Shape>(m0 + wm, n0 + wn, split, lane, columns, acc, lds + wave * (Shape::lds / Shape::waves));
}

// A grid of one or two kinds of product: the first one's tiles, then the second's.
template <typename T, typename Shape, typename J0>
__global__ __launch_bounds__((Shape::threads), 2) void product_kernel(J0 j0) {
    extern __shared__ __align__(16) unsigned char lds[];
    run_tile<T, Shape>(j0, static_cast<int>(blockIdx.x), lds);
}
template <typename T, typename Shape, typename J0, typename J1>
__global__ __launch_bounds__((Shape::threads), 2) void product2_kernel(J0 j0, J1 j1) {
    extern __shared__ __align__(16) unsigned char lds[];
    const int n0 = j0.p.mt * j0.p.nt * j0.p.splits, id = static_cast<int>(blockIdx.x);
    if (id < n0) run_tile<T, Shape>(j0, id, lds);
    else run_tile<T, Shape>(j1, id - n0, lds);
}

// The columns of a wave's part of C, 32 at a time (one a lane, twice): f(j, the
// lane's rows of column 32 j + lane % 32).
template <typename Shape, typename F>
__device__ __forceinline__ void each_column(const f32x16 (&acc)[Shape::I][Shape::J], const F &f) {
#pragma unroll
    for (int j = 0; j < Shape::J; ++j) {
        __builtin_amdgcn_sched_barrier(0);   // one at a time: few registers
        f32x16 c[Shape::I];
#pragma unroll
        for (int i = 0; i < Shape::I; ++i) c[i] = acc[i][j];
        f(j, c);
    }
}

// What exponentials are taken relative to: the maximum where it is finite.  (An
// infinite one would make NaN of itself; against 0 it gives a sum of 0 or infinity,
// and so the log sum exp that it should.)
__device__ __forceinline__ float reference(float top) { return fabsf(top) == INFINITY ? 0.0f : top; }

// ---- forward: maximum and sum of exponentials of a token over a tile's words
struct LossTile {
    float2 *part;              // [32 I words][token]
    float *target_logit;       // [token]
    const int64_t *targets;
    int tokens, words, word0;  // words of this piece; word0: the piece's first
    int part0;                 // first part of this piece
    // The target's place among a wave's words, or -1.
    template <int J>
    struct Columns {
        int mine[J];
    };
    template <typename Shape>
    __device__ __forceinline__ Columns<Shape::J> begin(int m, int n, int lane) const {
        Columns<Shape::J> c;
#pragma unroll
        for (int j = 0; j < Shape::J; ++j) {
            const int t = n + 32 * j + lane % 32;
            const int64_t target = t < tokens ? targets[t] - word0 - m : -1;
            c.mine[j] = target >= 0 && target < min(Shape::WM, words - m) ? static_cast<int>(target) : -1;
        }
        return c;
    }
    template <typename Shape>
    __device__ __forceinline__ void tile(int m, int n, int, int lane, const Columns<Shape::J> &columns,
                                         f32x16 (&acc)[Shape::I][Shape::J], unsigned char *) const {
        if (m >= words) return;
        const bool all = m + Shape::WM <= words;
#pragma unroll
        for (int j = 0; j < Shape::J; ++j) {
            const int t = n + 32 * j + lane % 32, mine = columns.mine[j];
            if (!all) {
#pragma unroll
                for (int i = 0; i < Shape::I; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (m + 32 * i + acc_row(e, lane) >= words) acc[i][j][e] = -INFINITY;
            }
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < Shape::I; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, acc[i][j][e]);
            if (__any(mine >= 0)) {
                float hit = 0.0f;
#pragma unroll
                for (int i = 0; i < Shape::I; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) hit = 32 * i + acc_row(e, lane) == mine ? acc[i][j][e] : hit;
                if (mine >= 0 && mine / 4 % 2 == lane / 32) target_logit[t] = hit;
            }
            top = fmaxf(top, __shfl_xor(top, 32));
            const float ref = reference(top);
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < Shape::I; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[e % 4] += fast_exp2((acc[i][j][e] - ref) * kLog2e);
            float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
            s += __shfl_xor(s, 32);
            if (t < tokens && lane < 32)
                part[static_cast<int64_t>(part0 + m / Shape::WM) * tokens + t] = make_float2(top, s);
        }
    }
};

// Joins the parts of a token: 16 tokens a workgroup, 64 slices of the parts (a
// slice is a quarter wave; few tokens have many parts).
constexpr int kJoinTokens = 16, kJoinSlices = 64;
__device__ __forceinline__ float2 join(float2 a, float2 b) {
    const float top = fmaxf(a.x, b.x), ref = reference(top);
    return make_float2(top, a.y * fast_exp2((a.x - ref) * kLog2e) + b.y * fast_exp2((b.x - ref) * kLog2e));
}
__global__ __launch_bounds__(kJoinTokens * kJoinSlices) void loss_join_kernel(
    const float2 *__restrict__ part, int parts, int tokens, const int64_t *__restrict__ targets, int64_t ignore,
    int64_t vocab, float *__restrict__ loss, float *__restrict__ lse) {
    __shared__ float2 sh[kJoinSlices / 4][kJoinTokens];
    const int lane = threadIdx.x % kJoinTokens, slice = threadIdx.x / kJoinTokens;
    const int t = blockIdx.x * kJoinTokens + lane, at = min(t, tokens - 1);
    float2 s = make_float2(-INFINITY, 0.0f);
    constexpr int kAhead = 8;   // loads under way at a time
    for (int k = slice; k < parts; k += kAhead * kJoinSlices) {
        float2 f[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            f[u] = part[static_cast<int64_t>(min(k + u * kJoinSlices, parts - 1)) * tokens + at];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (k + u * kJoinSlices < parts) s = join(s, f[u]);
    }
#pragma unroll
    for (int m = kJoinTokens; m < 64; m *= 2) s = join(s, make_float2(__shfl_xor(s.x, m), __shfl_xor(s.y, m)));
    if (threadIdx.x % 64 < kJoinTokens) sh[slice / 4][lane] = s;
    __syncthreads();
    if (slice > 0 || t >= tokens) return;
    for (int k = 1; k < kJoinSlices / 4; ++k) s = join(s, sh[k][lane]);
    const float l = s.x + fast_log2(s.y) * kLn2;
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

// exp(l - ref).  Float32 results carry the rounding of the exponent's product with
// log2 e as a second term (which has no value where the product is infinite, so
// that what vanishes anyway is cut at e^-200); in bfloat16 it is far below p's own
// rounding.
__device__ __forceinline__ float exp_of(float d, uint16_t) { return fast_exp2(d * kLog2e); }
__device__ __forceinline__ float exp_of(float d, float) {
    d = d < -200.0f ? -200.0f : d;   // a NaN stays
    const float hi = d * kLog2e, lo = fmaf(d, kLog2e, -hi);
    return fast_exp2(hi) * fmaf(lo, kLn2, 1.0f);
}

// Four consecutive values at p, 4 sizeof(T)-byte aligned.
__device__ __forceinline__ void store4(float *p, const float *f) {
    *reinterpret_cast<f32x4 *>(p) = f32x4{f[0], f[1], f[2], f[3]};
}
__device__ __forceinline__ void store4(uint16_t *p, const float *f) {
    typedef __bf16 b4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<uint2 *>(p) = __builtin_bit_cast(uint2, __builtin_convertvector((f32x4{f[0], f[1], f[2], f[3]}), b4));
}
// The first n of a chunk's values at p, aligned as T is.
template <typename T>
__device__ __forceinline__ void store_chunk(T *p, u32x4 x, int n) {
    typedef u32x4 Any __attribute__((aligned(2)));
    constexpr int kUnit = 16 / sizeof(T);
    if (n >= kUnit) {
        *reinterpret_cast<Any *>(p) = x;
    } else {
        struct Values { T v[kUnit]; };
        const Values y = __builtin_bit_cast(Values, x);
#pragma unroll
        for (int e = 0; e < kUnit; ++e)
            if (e < n) p[e] = y.v[e];
    }
}

// 32 columns of a wave's part of C on their way to rows of memory, through the
// wave's part of LDS.  From the accumulator a lane would store four values of
// its column, far from its neighbours'; out of LDS whole rows go, 16 bytes a lane.
// (p in bfloat16, 8192 x 16384 logits of width 2560: 682 us against 1046 us.)
template <typename T, typename Shape>
struct Staged {
    static constexpr int kUnit = 16 / sizeof(T), kRow = Shape::WM * sizeof(T), kRowChunks = kRow / 16;
    static constexpr int kRows = 64 / kRowChunks;        // rows one store instruction covers
    static_assert(32 * kRow <= Shape::lds / Shape::waves, "the wave's part holds them");
    // Values v .. v + 3 of column r.  Chunks are permuted, so that the columns of
    // the lanes served together fall into different banks.
    static __device__ __forceinline__ void put(unsigned char *lds, int r, int v, const float *x) {
        const int c = (v / kUnit) ^ (r % kRowChunks);
        store4(reinterpret_cast<T *>(lds + r * kRow + c * 16) + v % kUnit, x);
    }
    // f(r, v, values v .. of column r) for the 16-byte chunks.
    template <typename F>
    static __device__ __forceinline__ void each(const unsigned char *lds, int lane, const F &f) {
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        const int c = lane % kRowChunks;
#pragma unroll
        for (int s = 0; s < 32 / kRows; ++s) {
            const int r = s * kRows + lane / kRowChunks;
            f(r, c * kUnit, *reinterpret_cast<const u32x4 *>(lds + r * kRow + (c ^ (r % kRowChunks)) * 16));
        }
        asm volatile("" : : : "memory");   // the next columns' writes stay behind
    }
};

// p of a piece: p[token][word], rows ldp words apart (zero past the words).
template <typename T>
struct ProbTile {
    T *p;
    int64_t ldp;
    const int64_t *targets;
    const float *lse, *dloss, *scale;
    int64_t ignore, vocab;
    int tokens, words, word0;
    // A token's reference, factor and, if it is among a wave's words, its target.
    template <int J>
    struct Columns {
        float ref[J], g[J];
        int mine[J];
        bool live[J];
    };
    template <typename Shape>
    __device__ __forceinline__ Columns<Shape::J> begin(int m, int n, int lane) const {
        Columns<Shape::J> c;
        const float by = *scale;
#pragma unroll
        for (int j = 0; j < Shape::J; ++j) {
            const int t = n + 32 * j + lane % 32, at = min(t, tokens - 1);
            const int64_t target = targets[at], hit = target - word0 - m;
            c.live[j] = t < tokens && target != ignore;
            c.ref[j] = c.live[j] ? lse[at] : 0.0f;
            c.g[j] = c.live[j] ? dloss[at] / by : 0.0f;
            if (c.live[j] && (target < 0 || target >= vocab)) c.g[j] = NAN;
            c.mine[j] = hit >= 0 && hit < Shape::WM ? static_cast<int>(hit) : -1;
        }
        return c;
    }
    template <typename Shape>
    __device__ __forceinline__ void tile(int m, int n, int, int lane, const Columns<Shape::J> &columns,
                                         f32x16 (&acc)[Shape::I][Shape::J], unsigned char *lds) const {
        typedef Staged<T, Shape> Out;
        wait_and_meet<0>();
        each_column<Shape>(acc, [&](int j, const f32x16(&c)[Shape::I]) {
            const bool live = columns.live[j];
            const float ref = columns.ref[j], g = columns.g[j];
            const int mine = columns.mine[j];
#pragma unroll
            for (int i = 0; i < Shape::I; ++i)
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const int v = 32 * i + acc_row(e, lane);
                    float x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[k] = (exp_of(c[i][e + k] - ref, T{}) - (v + k == mine ? 1.0f : 0.0f)) * g;
                        if (!live || m + v + k >= words) x[k] = 0.0f;
                    }
                    Out::put(lds, lane % 32, v, x);
                }
            Out::each(lds, lane, [&](int r, int v, u32x4 x) {
                const int t = n + 32 * j + r;
                if (t < tokens && m + v < ldp) *reinterpret_cast<u32x4 *>(p + static_cast<int64_t>(t) * ldp + m + v) = x;
            });
        });
    }
};

// Rows of a gradient, [n][m].  Sums over pieces of the vocabulary and runs of k
// meet in float32: one array a run, sum[run][n][ldsum], to which later pieces add.
template <typename T>
struct GradTile {
    float *sum;                // null: the sum is complete, out is written
    int64_t ldsum;
    T *out;
    const float *scale;        // out is the sum times this
    int rows, cols;            // of the gradient
    bool add;                  // sum holds earlier pieces
    struct Nothing {};
    template <typename Shape>
    __device__ __forceinline__ Nothing begin(int, int, int) const { return {}; }
    template <typename Shape>
    __device__ __forceinline__ void tile(int m, int n, int run, int lane, Nothing, f32x16 (&acc)[Shape::I][Shape::J],
                                         unsigned char *lds) const {
        wait_and_meet<0>();
        const float by = sum ? 1.0f : *scale;
        const auto put = [&](auto out, const f32x16(&c)[Shape::I]) {
#pragma unroll
            for (int i = 0; i < Shape::I; ++i)
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float x[4] = {c[i][e] * by, c[i][e + 1] * by, c[i][e + 2] * by, c[i][e + 3] * by};
                    decltype(out)::put(lds, lane % 32, 32 * i + acc_row(e, lane), x);
                }
        };
        each_column<Shape>(acc, [&](int j, const f32x16(&c)[Shape::I]) {
            if (sum) {
                typedef Staged<float, Shape> Out;
                put(Out(), c);
                Out::each(lds, lane, [&](int r, int d, u32x4 x) {
                    if (n + 32 * j + r >= rows || m + d >= cols) return;
                    f32x4 *to = reinterpret_cast<f32x4 *>(sum + (static_cast<int64_t>(run) * rows + n + 32 * j + r) * ldsum + m + d);
                    f32x4 y = __builtin_bit_cast(f32x4, x);
                    if (add) {
                        const f32x4 old = *to;
#pragma unroll
                        for (int k = 0; k < 4; ++k) y[k] += old[k];
                    }
                    *to = y;
                });
            } else {
                typedef Staged<T, Shape> Out;
                put(Out(), c);
                Out::each(lds, lane, [&](int r, int d, u32x4 x) {
                    if (n + 32 * j + r < rows) store_chunk(out + static_cast<int64_t>(n + 32 * j + r) * cols + m + d, x, cols - m - d);
                });
            }
        });
    }
};

// out[r][c] = scale * sum over the runs of sum[run][r][c]: a wave per row and 64
// vectors of four.
template <typename T>
__global__ __launch_bounds__(256) void add_runs_kernel(const float *__restrict__ sum, int runs, int64_t rows, int cols,
                                                       int64_t ldsum, const float *__restrict__ scale,
                                                       T *__restrict__ out) {
    const int c = (blockIdx.x * 64 + threadIdx.x % 64) * 4;
    if (c >= cols) return;
    const float by = *scale;
    for (int64_t r = blockIdx.y * 4 + threadIdx.x / 64; r < rows; r += 4 * gridDim.y) {
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        constexpr int kAhead = 8;   // loads under way at a time
        for (int i = 0; i < runs; i += kAhead) {
            f32x4 f[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                f[u] = *reinterpret_cast<const f32x4 *>(sum + (min(i + u, runs - 1) * rows + r) * ldsum + c);
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (i + u < runs)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] += f[u][e];
        }
        const float y[4] = {x[0] * by, x[1] * by, x[2] * by, x[3] * by};
        T *to = out + r * cols + c;
        if (cols % 4 == 0 && reinterpret_cast<uintptr_t>(out) % (4 * sizeof(T)) == 0) {
            store4(to, y);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < cols) Io<T>::store(to, e, y[e]);
        }
    }
}

// Copy of rows [0, rows) x [0, cols) with rows `ldo` elements apart (whole
// chunks of 16 bytes), zero past the columns and in rows whose target is
// `ignore` (targets may be null): a wave per row, four chunks of a lane under
// way at a time, read unaligned.
template <typename T>
__global__ __launch_bounds__(256) void align_rows_kernel(const T *__restrict__ in, T *__restrict__ out, int64_t rows,
                                                         int cols, int64_t ldo,
                                                         const int64_t *__restrict__ targets, int64_t ignore) {
    constexpr int kUnit = 16 / sizeof(T), kAhead = 4;
    typedef u32x4 Any __attribute__((aligned(2)));
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 64; r < rows;
         r += static_cast<int64_t>(gridDim.x) * 4) {
        const int n = targets && targets[r] == ignore ? 0 : cols;
        const T *from = in + r * cols;
        T *to = out + r * ldo;
        for (int c = threadIdx.x % 64 * kUnit; c < ldo; c += kAhead * 64 * kUnit) {
            u32x4 f[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int at = c + u * 64 * kUnit;
                f[u] = u32x4{0, 0, 0, 0};
                if (at + kUnit <= n) {
                    f[u] = *reinterpret_cast<const Any *>(from + at);
                } else {
                    T part[kUnit] = {};
                    for (int e = 0; at + e < n; ++e) part[e] = from[at + e];
                    f[u] = __builtin_bit_cast(u32x4, part);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (c + u * 64 * kUnit < ldo) *reinterpret_cast<u32x4 *>(to + c + u * 64 * kUnit) = f[u];
        }
    }
}

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t ceil_div(int64_t n, int64_t by) { return (n + by - 1) / by; }

bool on_16(const LossArgs &a) {
    return ((reinterpret_cast<uintptr_t>(a.hidden) | reinterpret_cast<uintptr_t>(a.weight)) & 15u) == 0;
}

typedef Tile<256, 256, 128, 64> Large;
typedef Tile<128, 128, 64, 64> Medium;
typedef Tile<128, 64, 64, 32> Small;     // float32
typedef Tile<128, 32, 32, 32> Narrow;    // few tokens

// Tiles and runs of a product: `splits` runs of k, whole steps each.
template <typename T, typename Shape>
int64_t lay_out(Problem *p, int splits) {
    p->mt = static_cast<int>(ceil_div(p->A.rows, Shape::BM));
    p->nt = static_cast<int>(ceil_div(p->B.rows, Shape::BN));
    const int64_t steps = ceil_div(p->A.k, kRowBytes / static_cast<int64_t>(sizeof(T)));
    p->steps = static_cast<int>(ceil_div(steps, splits));
    p->splits = splits;
    return static_cast<int64_t>(p->mt) * p->nt * splits;
}

template <typename Kernel, typename... Args>
hipError_t launch_tiles(Kernel kernel, int64_t n, int threads, int lds, hipStream_t stream, const Args &...args) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(n)), dim3(threads), lds, stream, args...);
    return hipGetLastError();
}

template <typename T, typename Shape, typename J0>
hipError_t product_as(J0 j0, int splits, hipStream_t stream) {
    const int64_t n = lay_out<T, Shape>(&j0.p, splits);
    return launch_tiles(product_kernel<T, Shape, J0>, n, Shape::threads, Shape::lds, stream, j0);
}

enum : int { kLarge, kMedium, kSmall, kNarrow };

template <typename T, typename J0>
hipError_t product(const J0 &j0, int shape, int splits, hipStream_t stream) {
    if constexpr (sizeof(T) == 4) {
        if (shape == kSmall) return product_as<T, Small>(j0, splits, stream);
    } else {
        if (shape == kLarge) return product_as<T, Large>(j0, splits, stream);
        if (shape == kMedium) return product_as<T, Medium>(j0, splits, stream);
    }
    return product_as<T, Narrow>(j0, splits, stream);
}

template <typename T, typename Shape, typename J0, typename J1>
hipError_t product2_as(J0 j0, int splits, J1 j1, hipStream_t stream) {
    const int64_t n = lay_out<T, Shape>(&j0.p, splits) + lay_out<T, Shape>(&j1.p, 1);
    return launch_tiles(product2_kernel<T, Shape, J0, J1>, n, Shape::threads, Shape::lds, stream, j0, j1);
}

template <typename T>
hipError_t align_rows(const T *in, T *out, int64_t rows, int64_t cols, int64_t ldo, const int64_t *targets,
                      int64_t ignore, hipStream_t stream) {
    const int64_t blocks = ceil_div(rows, 4);
    hipLaunchKernelGGL(align_rows_kernel<T>, dim3(static_cast<uint32_t>(blocks < 65536 ? blocks : 65536)),
                       dim3(256), 0, stream, in, out, rows, static_cast<int>(cols), ldo, targets, ignore);
    return hipGetLastError();
}

// Words of the vocabulary in one piece, a multiple of 1024 below the whole.
// Backward: p of the piece has at most 2^27 elements.  Forward: with copies,
// the copied piece likewise; else the grid's workgroups stay below 2^23.
int64_t piece_words(int64_t elements, int64_t rows, int64_t vocab) {
    int64_t n = elements / rows / 1024 * 1024;
    if (n < 1024) n = 1024;
    return n < vocab ? n : vocab;
}

// Bfloat16: tiles of 256 x 256 reach the highest rate (8192 tokens x 2560 x 50021
// forward 1.87 ms, in tiles of 128 x 128 2.50 ms) where they fill three quarters
// of the 256 compute units (252 of them 51 us against 58 us, 196 the same); below
// that tiles of 128 x 128, two workgroups a compute unit.  Float32: one product
// takes eight times as long for the same bytes, so that tiles of 128 x 64 feed it
// too, waste less at the ends and run three workgroups a compute unit (517 tokens
// x 769 x 32003 backward 844 us, 128 x 128 939 us, 256 x 256 1222 us; 2048 tokens
// 3.05, 2.95 and 2.98 ms).  Few tokens take tiles of 128 x 32, which stream the
// other operand (forward of 16 x 2560 x 50021 in bfloat16 69 us against 80 in the next
// larger tiles, of 32 tokens 72 against 79; two of them, for 64 tokens, 94 against 82).
int shape_of(int io, int64_t tiles, int64_t tokens) {
    if (tokens <= Narrow::BN) return kNarrow;
    if (io == IO_F32) return kSmall;
    return tiles >= 192 ? kLarge : kMedium;
}

// Sizes of a call and its workspace, cut into 256-byte aligned arrays.
struct Plan {
    bool copy;                 // rows of weight (forward: of hidden too) are copied to aligned ones
    int64_t dimp, ldsum;       // padded row lengths (elements)
    int64_t piece, piecep;     // words of a piece
    int64_t parts, part_words;
    int shape, grad_shape;     // of the logits' and the gradients' tiles
    int runs;                  // of k in dhidden's product
    bool sums;                 // dhidden is summed in float32 over pieces and runs
    size_t at_part, at_h, at_w, at_p, at_sum, at_scale, bytes;
};

Plan make_plan(const LossArgs &a, bool bwd, bool aligned) {
    Plan p{};
    const int64_t esz = a.io == IO_F32 ? 4 : 2, unit = 16 / esz;
    p.copy = !aligned || a.dim % unit != 0;
    p.dimp = round_up(a.dim, unit);
    const auto add = [&](int64_t bytes) {
        const size_t at = p.bytes;
        p.bytes += static_cast<size_t>(round_up(bytes, 256));
        return at;
    };
    const auto tiles = [](int64_t m, int64_t n) { return ceil_div(m, Large::BM) * ceil_div(n, Large::BN); };
    if (!bwd) {
        p.piece = p.copy ? piece_words(int64_t(1) << 27, p.dimp, a.vocab)
                         : piece_words(int64_t(1) << 37, a.tokens + 128, a.vocab);
        p.shape = shape_of(a.io, tiles(p.piece, a.tokens), a.tokens);
        p.part_words = p.shape == kLarge ? Large::WM : p.shape == kMedium ? Medium::WM : p.shape == kSmall ? Small::WM : Narrow::WM;
        p.parts = a.vocab / p.piece * ceil_div(p.piece, p.part_words) + ceil_div(a.vocab % p.piece, p.part_words);
        p.at_part = add(p.parts * a.tokens * 8);
        p.at_h = add(p.copy ? a.tokens * p.dimp * esz : 0);
        p.at_w = add(p.copy ? p.piece * p.dimp * esz : 0);
        return p;
    }
    p.piece = piece_words(int64_t(1) << 27, a.tokens, a.vocab);
    p.piecep = round_up(p.piece, unit);
    p.shape = shape_of(a.io, tiles(p.piece, a.tokens), a.tokens);
    // dweight sums over few steps where there are few tokens; two workgroups a
    // compute unit then form products while the other writes (300 tokens x 1600 x
    // 32003: 235 us against 254 us)
    p.grad_shape = shape_of(a.io, a.tokens > 512 ? tiles(a.dim, a.tokens) + tiles(a.dim, p.piece) : 0, a.tokens);
    // A tile of dhidden sums over the piece's words, one of dweight over the
    // tokens: dhidden's k is cut into runs about twice as long as dweight's.  (300
    // tokens x 1600 x 32003 in bfloat16 198 us, 517 x 769 x 32003 in float32 782 us; one
    // run 360 and 1550 us; from 512 or 2048 words on, or up to 16 or 64 runs, within
    // 7 % of that, but 3 x 2457 x 10013 in float32 with 2048 181 us against 163.)
    const int64_t run = 2 * a.tokens > 1024 ? 2 * a.tokens : 1024;
    p.runs = static_cast<int>(ceil_div(p.piece, run) < 32 ? ceil_div(p.piece, run) : 32);
    p.sums = p.runs > 1 || p.piece < a.vocab;
    p.ldsum = round_up(a.dim, 4);
    p.at_h = add(a.tokens * p.dimp * esz);
    p.at_w = add(p.copy ? p.piece * p.dimp * esz : 0);
    p.at_p = add(a.tokens * p.piecep * esz);
    p.at_scale = add(4);
    p.at_sum = add(p.sums ? p.runs * a.tokens * p.ldsum * 4 : 0);
    return p;
}

template <typename T>
Rows rows_of(const T *q, int64_t ld, int64_t n, int64_t k) {
    return Rows{reinterpret_cast<const unsigned char *>(q), ld * static_cast<int64_t>(sizeof(T)), static_cast<int>(n),
                static_cast<int>(k)};
}

template <bool AX, bool BX, typename Epilogue>
Job<Epilogue, AX, BX> job_of(const Rows &A, const Rows &B, const Epilogue &e) {
    return Job<Epilogue, AX, BX>{Problem{A, B, 0, 0, 0, 0}, e};
}

template <typename T>
hipError_t fwd(const LossArgs &a, const Plan &p, unsigned char *base, hipStream_t stream) {
    float2 *part = reinterpret_cast<float2 *>(base + p.at_part);
    const T *h = static_cast<const T *>(a.hidden);
    hipError_t e = hipSuccess;
    if (p.copy) {
        e = align_rows(h, reinterpret_cast<T *>(base + p.at_h), a.tokens, a.dim, p.dimp, nullptr, 0, stream);
        h = reinterpret_cast<const T *>(base + p.at_h);
    }
    int part0 = 0;
    for (int64_t w0 = 0; w0 < a.vocab && e == hipSuccess; w0 += p.piece) {
        const int64_t words = a.vocab - w0 < p.piece ? a.vocab - w0 : p.piece;
        const T *w = static_cast<const T *>(a.weight) + w0 * a.dim;
        if (p.copy) {
            e = align_rows(w, reinterpret_cast<T *>(base + p.at_w), words, a.dim, p.dimp, nullptr, 0, stream);
            w = reinterpret_cast<const T *>(base + p.at_w);
            if (e != hipSuccess) break;
        }
        const LossTile ep{part, a.loss, a.targets, static_cast<int>(a.tokens), static_cast<int>(words),
                          static_cast<int>(w0), part0};
        e = product<T>(job_of<false, false>(rows_of(w, p.dimp, words, p.dimp), rows_of(h, p.dimp, a.tokens, p.dimp), ep),
                       p.shape, 1, stream);
        part0 += static_cast<int>(ceil_div(words, p.part_words));
    }
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(loss_join_kernel, dim3(static_cast<uint32_t>(ceil_div(a.tokens, kJoinTokens))),
                       dim3(kJoinTokens * kJoinSlices), 0,
                       stream, part, part0, static_cast<int>(a.tokens), a.targets, a.ignore_index, a.vocab, a.loss,
                       a.lse);
    return hipGetLastError();
}

template <typename T>
hipError_t bwd(const LossArgs &a, const Plan &p, unsigned char *base, hipStream_t stream) {
    T *pr = reinterpret_cast<T *>(base + p.at_p), *h = reinterpret_cast<T *>(base + p.at_h);
    float *scale = reinterpret_cast<float *>(base + p.at_scale), *sum = reinterpret_cast<float *>(base + p.at_sum);
    const int tokens = static_cast<int>(a.tokens), dim = static_cast<int>(a.dim);
    hipLaunchKernelGGL(grad_scale_kernel, dim3(1), dim3(1024), 0, stream, a.dloss, a.targets, a.ignore_index, tokens,
                       scale);
    hipError_t e = hipGetLastError();
    // hidden with the ignored tokens' rows zero: whatever they hold, times their
    // p of 0, adds nothing to dweight
    if (e == hipSuccess)
        e = align_rows(static_cast<const T *>(a.hidden), h, a.tokens, a.dim, p.dimp, a.targets, a.ignore_index, stream);
    for (int64_t w0 = 0; w0 < a.vocab && e == hipSuccess; w0 += p.piece) {
        const int64_t words = a.vocab - w0 < p.piece ? a.vocab - w0 : p.piece;
        const int64_t wordsp = round_up(words, 16 / sizeof(T));
        const T *w = static_cast<const T *>(a.weight) + w0 * a.dim;
        if (p.copy) {
            e = align_rows(w, reinterpret_cast<T *>(base + p.at_w), words, a.dim, p.dimp, nullptr, 0, stream);
            w = reinterpret_cast<const T *>(base + p.at_w);
            if (e != hipSuccess) break;
        }
        const ProbTile<T> prob{pr, wordsp, a.targets, a.lse, a.dloss, scale, a.ignore_index, a.vocab,
                               tokens, static_cast<int>(words), static_cast<int>(w0)};
        e = product<T>(job_of<false, false>(rows_of(w, p.dimp, words, p.dimp), rows_of(h, p.dimp, a.tokens, p.dimp), prob),
                       p.shape, 1, stream);
        if (e != hipSuccess) break;
        // dhidden: weight across k (the words), p along it; dweight: hidden and p
        // across k (the tokens)
        T *dwp = static_cast<T *>(a.dweight) + w0 * a.dim;
        const GradTile<T> dh{p.sums ? sum : nullptr, p.ldsum, static_cast<T *>(a.dhidden), scale, tokens, dim,
                             w0 > 0};
        const GradTile<T> dw{nullptr, 0, dwp, scale, static_cast<int>(words), dim, false};
        const auto jh = job_of<true, false>(rows_of(w, p.dimp, a.dim, words), rows_of(pr, wordsp, a.tokens, words), dh);
        const auto jw = job_of<true, true>(rows_of(h, p.dimp, a.dim, a.tokens), rows_of(pr, wordsp, words, a.tokens), dw);
        // a last, shorter piece keeps the runs, so that they add to the same sums
        if constexpr (sizeof(T) == 4) {
            if (p.grad_shape == kNarrow) {
                e = product_as<T, Narrow>(jh, p.runs, stream);
                if (e == hipSuccess) e = product_as<T, Small>(jw, 1, stream);
            } else {
                e = product2_as<T, Small>(jh, p.runs, jw, stream);
            }
        } else {
            if (p.grad_shape == kNarrow) {
                e = product_as<T, Narrow>(jh, p.runs, stream);
                if (e == hipSuccess) e = product_as<T, Medium>(jw, 1, stream);
            } else if (p.grad_shape == kLarge) {
                e = product2_as<T, Large>(jh, p.runs, jw, stream);
            } else {
                e = product2_as<T, Medium>(jh, p.runs, jw, stream);
            }
        }
    }
    if (e == hipSuccess && p.sums) {
        const int64_t blocks = ceil_div(a.tokens, 4);
        hipLaunchKernelGGL(add_runs_kernel<T>, dim3(static_cast<uint32_t>(ceil_div(dim, 256)),
                                                    static_cast<uint32_t>(blocks < 16384 ? blocks : 16384)),
                           dim3(256), 0, stream, sum, p.runs, a.tokens, dim, p.ldsum, scale,
                           static_cast<T *>(a.dhidden));
        e = hipGetLastError();
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
