// beam_search.hip -- a step of beam search: selection over beams and vocabulary, and
// the reordering of the beams' states.
//
// Selection.  value = score_j + (logit_{j,v} - lse_j), the `count` largest of every
// batch entry, ties to the lowest j V + v.  Inside a beam the order is that of its
// logits, so a first launch reads the logits once: every workgroup leaves, for a
// piece of a beam's words, their maximum, sum of exponentials and at most 64 words
// among which its `count` largest are.  A second launch joins a beam's pieces, forms
// the values in float64, where a sum with the score merges no two logits, and ranks
// the beams' words together.
//
// What can be left out is found by bisection: t is the largest number that `count` of
// the lanes' maxima reach, and a wave counts them with one comparison and one scalar
// population count a bit.  Few words beyond `count` reach t; where more than 64 do
// (equal logits), the bisection goes over all of them, with the word as the last
// digits, so that it ends with exactly `count`.
//
// A beam without values (its score or its lse not finite) counts as -infinity for
// every word, which its lowest words then stand for.
//
// Reordering.  A thread holds one place of every beam of an entry: it loads what the
// moved beams come from before it writes any, so rows change places inside the
// buffer, and beams that stay cost nothing.
#include <algorithm>

#include "device_math.h"
#include "internal.h"

namespace mssm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kItems = 16;                      // words of a lane
constexpr int kWaves = 4;                       // of a workgroup of the first launch
constexpr int kThreads = 64 * kWaves;
constexpr int kPiece = kThreads * kItems;       // words of a workgroup
constexpr int kKeep = 64;                       // words that a piece leaves at most
static_assert(MSSM_MAX_BEAM_COUNT <= kKeep, "a piece keeps all that are asked for");

// What a piece leaves.
struct Piece {
    float top, sum;     // maximum, sum of exp(logit - maximum)
    int count, unused;
    uint64_t key[kKeep];
};

// Order of floats as unsigned numbers (-0 and 0 are one), and a key that falls with the
// word among equal ones; no key of a word is 0.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float(u >> 31 ? u & 0x7fffffffu : ~u); }
__device__ __forceinline__ uint64_t key_of(uint32_t order, int word) {
    return static_cast<uint64_t>(order) << 32 | (0xffffffffu - static_cast<uint32_t>(word));
}
__device__ __forceinline__ int word_of(uint64_t key) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)); }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    return v;
}
__device__ __forceinline__ int lanes_before(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                     __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
}

// Between what lanes of a wave write to LDS and what others of them read.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The largest t that at least `count` lanes' values reach; 0 if fewer hold any.
template <typename U>
__device__ __forceinline__ U reached_by(U mine, int count) {
    U t = 0;
    for (int bit = 8 * sizeof(U) - 1; bit >= 0; --bit) {
        const U with = t | U(1) << bit;
        if (__popcll(__ballot(mine >= with)) >= count) t = with;
    }
    return t;
}

// Keeps of the n keys at `list` (LDS, one wave's own, in any order) those among which
// the `count` largest are, at most kKeep; returns how many.
__device__ int reduce(uint64_t *list, int n, int count) {
    const int lane = threadIdx.x % 64;
    if (n <= kKeep) return n;
    uint64_t top = 0;
    for (int i = lane; i < n; i += 64) top = max(top, list[i]);
    uint64_t t = static_cast<uint64_t>(reached_by(static_cast<uint32_t>(top >> 32), count)) << 32;
    int reach = 0;
    for (int i = 0; i < n; i += 64) reach += __popcll(__ballot(i + lane < n && list[min(i + lane, n - 1)] >= t));
    if (reach > kKeep) {
        t = 0;
        for (int bit = 63; bit >= 0; --bit) {
            const uint64_t with = t | uint64_t(1) << bit;
            int found = 0;
            for (int i = 0; i < n; i += 64) found += __popcll(__ballot(i + lane < n && list[min(i + lane, n - 1)] >= with));
            if (found >= count) t = with;
        }
    }
    int kept = 0;
    for (int i = 0; i < n; i += 64) {   // never ahead of what is still to be read
        const uint64_t key = i + lane < n ? list[i + lane] : 0;
        const bool keep = i + lane < n && key >= t;
        const uint64_t mask = __ballot(keep);
        if (keep) list[kept + lanes_before(mask)] = key;
        kept += __popcll(mask);
    }
    wave_sync();
    return kept;
}

// Four consecutive logits, at any element's address.
__device__ __forceinline__ void load4(const float *p, float *v) {
    typedef f32x4 Any __attribute__((aligned(4)));
    const f32x4 a = *reinterpret_cast<const Any *>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const uint16_t *p, float *v) {
    typedef u32x2 Any __attribute__((aligned(2)));
    const u32x2 a = *reinterpret_cast<const Any *>(p);
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void beam_pieces_kernel(const T *__restrict__ logits, Piece *__restrict__ out,
                                                               int vocab, int count, int pieces) {
    __shared__ uint64_t list[kWaves * 64 * kItems];
    __shared__ float tops[kWaves], sums[kWaves];
    __shared__ int counts[kWaves];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t row = blockIdx.x / pieces;
    const int first = static_cast<int>(blockIdx.x % pieces) * kPiece;
    logits += row * vocab;
    const float kLow = -__builtin_inff();
    auto word = [&](int j) { return first + (j / 4 * kThreads + static_cast<int>(threadIdx.x)) * 4 + j % 4; };
    float v[kItems], top = kLow;
#pragma unroll
    for (int j = 0; j < kItems; j += 4) {
        if (word(j) + 3 < vocab) {
            load4(logits + word(j), v + j);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j + i] = word(j + i) < vocab ? Io<T>::load(logits, word(j + i)) : kLow;
        }
    }
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        top = fmaxf(top, v[j]);
        if (word(j) < vocab) mine = max(mine, ordered(v[j] != v[j] ? kLow : v[j]));
    }
    top = wave_max(top);
    float sum = 0.0f;                       // 0 without finite logits, NaN with +infinity or NaN
    const float base = top == kLow ? 0.0f : top;
#pragma unroll
    for (int j = 0; j < kItems; ++j) sum += fast_exp2((v[j] - base) * kLog2e);
    sum = wave_sum(sum);

    uint64_t *const own = list + wave * 64 * kItems;
    const uint32_t t = reached_by(mine, count);
    int n = 0;
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const uint32_t order = ordered(v[j] != v[j] ? kLow : v[j]);
        const bool keep = word(j) < vocab && order >= t;
        const uint64_t mask = __ballot(keep);
        if (keep) own[n + lanes_before(mask)] = key_of(order, word(j));
        n += __popcll(mask);
    }
    wave_sync();
    n = reduce(own, n, count);
    if (lane == 0) {
        tops[wave] = top;
        sums[wave] = sum;
        counts[wave] = n;
    }
    __syncthreads();
    if (wave > 0) return;
    // the waves' lists side by side, then the same once more
    int total = counts[0];
    for (int w = 1; w < kWaves; ++w) {
        const uint64_t key = lane < counts[w] ? list[w * 64 * kItems + lane] : 0;
        if (lane < counts[w]) list[total + lane] = key;
        total += counts[w];
    }
    wave_sync();
    total = reduce(list, total, count);
    Piece &p = out[blockIdx.x];
    if (lane < total) p.key[lane] = list[lane];
    const float my_top = lane < kWaves ? tops[lane] : kLow, all = wave_max(my_top);
    float part = 0.0f;
    if (lane < kWaves && sums[lane] != 0.0f) part = sums[lane] * fast_exp2((my_top - all) * kLog2e);
    part = wave_sum(part);
    if (lane == 0) {
        p.top = all;
        p.sum = part;
        p.count = total;
    }
}

// A workgroup per batch entry, a wave at a time per beam.  LDS: for every beam kKeep
// values and words; for every wave a list.
constexpr int kMergeWaves = 4, kMergeList = 9 * kKeep;

__global__ __launch_bounds__(64 * kMergeWaves) void beam_merge_kernel(
    const Piece *__restrict__ in, const float *__restrict__ scores, float *__restrict__ out_scores,
    int64_t *__restrict__ out_tokens, int64_t *__restrict__ out_beams, int beams, int vocab, int count, int pieces) {
    __shared__ uint64_t lists[kMergeWaves * kMergeList];
    __shared__ double value[MSSM_MAX_BEAMS * kKeep];
    __shared__ int64_t flat[MSSM_MAX_BEAMS * kKeep];
    __shared__ int total;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t entry = blockIdx.x;
    const double kLow = -__builtin_inf();
    uint64_t *const list = lists + wave * kMergeList;
    if (threadIdx.x == 0) total = 0;
    __syncthreads();
    for (int j = wave; j < beams; j += kMergeWaves) {
        const int64_t row = entry * beams + j;
        const Piece *const mine = in + row * pieces;
        float top = -__builtin_inff();
        for (int s = lane; s < pieces; s += 64) top = fmaxf(top, mine[s].top);
        top = wave_max(top);
        double sum = 0.0;
        for (int s = lane; s < pieces; s += 64)
            if (mine[s].sum != 0.0f) sum += mine[s].sum * exp(static_cast<double>(mine[s].top) - top);
        const double lse = top + log(wave_sum(sum)), score = scores[row];
        const bool live = fabs(lse) < __builtin_inf() && fabs(score) < __builtin_inf();
        int n = live ? 0 : min(count, vocab);
        for (int s = 0; live && s < pieces; ++s) {
            const int more = mine[s].count;
            if (lane < more) list[n + lane] = mine[s].key[lane];
            n += more;
            wave_sync();
            if (n > kMergeList - kKeep || s == pieces - 1) n = reduce(list, n, count);
        }
        int at = 0;
        if (lane == 0) at = atomicAdd(&total, n);      // where, not in which order they rank
        at = __shfl(at, 0);
        if (lane < n) {
            const uint64_t key = live ? list[lane] : 0;
            const int word = live ? word_of(key) : lane;
            value[at + lane] = live ? score + (unordered(static_cast<uint32_t>(key >> 32)) - lse) : kLow;
            flat[at + lane] = static_cast<int64_t>(j) * vocab + word;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < total; i += 64 * kMergeWaves) {
        const double mine = value[i];
        const int64_t place = flat[i];
        int rank = 0;
        for (int k = 0; k < total; ++k) rank += value[k] > mine || (value[k] == mine && flat[k] < place);
        if (rank < count) {
            out_scores[entry * count + rank] = static_cast<float>(mine);
            out_tokens[entry * count + rank] = place % vocab;
            out_beams[entry * count + rank] = place / vocab;
        }
    }
}

// ---- reordering ------------------------------------------------------------------

constexpr int kStates = 32;      // of a launch

struct Reorder {
    unsigned char *state[kStates];
    int64_t row[kStates];        // bytes
    int64_t end[kStates];        // workgroups of an entry up to this state's
    int unit[kStates];           // bytes that a thread moves
    const int64_t *origins;
    int count, beams;
    int64_t blocks;              // of an entry
};

template <typename U, int BEAMS>
__device__ __forceinline__ void reorder(unsigned char *rows, int64_t row_bytes, int64_t at, const int64_t *origins, int beams) {
    const int64_t units = row_bytes / sizeof(U);
    if (at >= units) return;
    U *const p = reinterpret_cast<U *>(rows) + at;
    U v[BEAMS];
#pragma unroll
    for (int j = 0; j < BEAMS; ++j)
        if (j < beams && origins[j] != j) v[j] = p[origins[j] * units];
#pragma unroll
    for (int j = 0; j < BEAMS; ++j)
        if (j < beams && origins[j] != j) p[j * units] = v[j];
}

template <int BEAMS>
__global__ __launch_bounds__(256) void state_reorder_kernel(const Reorder R) {
    __shared__ int64_t origins[BEAMS];
    const int64_t entry = blockIdx.x / R.blocks, block = blockIdx.x % R.blocks;
    if (threadIdx.x < R.beams) {
        // an origin outside the entry leaves the beam as it is
        const int64_t o = R.origins[entry * R.beams + threadIdx.x];
        origins[threadIdx.x] = o >= 0 && o < R.beams ? o : threadIdx.x;
    }
    __syncthreads();
    int s = 0;
    while (s < R.count - 1 && block >= R.end[s]) ++s;
    const int64_t at = (block - (s ? R.end[s - 1] : 0)) * 256 + threadIdx.x;
    unsigned char *const rows = R.state[s] + entry * R.beams * R.row[s];
    if (R.unit[s] == 16) reorder<u32x4, BEAMS>(rows, R.row[s], at, origins, R.beams);
    else if (R.unit[s] == 4) reorder<uint32_t, BEAMS>(rows, R.row[s], at, origins, R.beams);
    else reorder<unsigned char, BEAMS>(rows, R.row[s], at, origins, R.beams);
}

// Bytes of a state that a thread moves: what its rows' places are multiples of.
int unit_of(const void *state, int64_t row_bytes) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(state) | static_cast<uint64_t>(row_bytes);
    return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
}

}  // namespace

int64_t state_reorder_blocks(const void *state, int64_t row_bytes) {
    return (row_bytes / unit_of(state, row_bytes) + 255) / 256;
}

int64_t beam_select_pieces(int64_t vocab) { return (vocab + kPiece - 1) / kPiece; }

size_t beam_select_workspace(const BeamArgs &a) {
    return static_cast<size_t>(a.batch * a.beams) * beam_select_pieces(a.vocab) * sizeof(Piece);
}

hipError_t launch_beam_select(const BeamArgs &a, void *workspace, hipStream_t stream) {
    void *ws = workspace;
    if (!ws)
        if (const hipError_t e = scratch_alloc(&ws, beam_select_workspace(a), stream)) return e;
    const int64_t pieces = beam_select_pieces(a.vocab);
    const dim3 grid(static_cast<uint32_t>(a.batch * a.beams * pieces));
    const int vocab = static_cast<int>(a.vocab), count = static_cast<int>(a.count);
    if (a.io == IO_F32)
        hipLaunchKernelGGL(beam_pieces_kernel<float>, grid, dim3(kThreads), 0, stream, static_cast<const float *>(a.logits),
                           static_cast<Piece *>(ws), vocab, count, static_cast<int>(pieces));
    else
        hipLaunchKernelGGL(beam_pieces_kernel<uint16_t>, grid, dim3(kThreads), 0, stream,
                           static_cast<const uint16_t *>(a.logits), static_cast<Piece *>(ws), vocab, count,
                           static_cast<int>(pieces));
    hipLaunchKernelGGL(beam_merge_kernel, dim3(static_cast<uint32_t>(a.batch)), dim3(64 * kMergeWaves), 0, stream,
                       static_cast<const Piece *>(ws), a.scores, a.out_scores, a.out_tokens, a.out_beams,
                       static_cast<int>(a.beams), vocab, count, static_cast<int>(pieces));
    hipError_t e = hipGetLastError();
    if (!workspace) {
        const hipError_t f = scratch_free(ws, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

hipError_t launch_state_reorder(void *const *states, const int64_t *row_bytes, int64_t count, const int64_t *origins,
                                int64_t batch, int64_t beams, hipStream_t stream) {
    for (int64_t s = 0; s < count;) {
        Reorder R{};
        R.origins = origins;
        R.beams = static_cast<int>(beams);
        for (; s < count && R.count < kStates; ++s) {
            if (row_bytes[s] == 0) continue;
            const int unit = unit_of(states[s], row_bytes[s]);
            const int64_t blocks = state_reorder_blocks(states[s], row_bytes[s]);
            // a launch stays below 2^32 threads (the caller has checked each state alone)
            if (R.count && (R.blocks + blocks) * batch >= int64_t(1) << 24) break;
            R.state[R.count] = static_cast<unsigned char *>(states[s]);
            R.row[R.count] = row_bytes[s];
            R.unit[R.count] = unit;
            R.blocks += blocks;
            R.end[R.count++] = R.blocks;
        }
        if (R.count == 0) break;
        const dim3 grid(static_cast<uint32_t>(R.blocks * batch));
        if (beams <= 4) hipLaunchKernelGGL(state_reorder_kernel<4>, grid, dim3(256), 0, stream, R);
        else if (beams <= 8) hipLaunchKernelGGL(state_reorder_kernel<8>, grid, dim3(256), 0, stream, R);
        else if (beams <= 16) hipLaunchKernelGGL(state_reorder_kernel<16>, grid, dim3(256), 0, stream, R);
        else hipLaunchKernelGGL(state_reorder_kernel<32>, grid, dim3(256), 0, stream, R);
        if (const hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

}  // namespace mssm
