// beam_search.hip -- a step of beam search: selection over beams and vocabulary, and
// the reordering of the beams' states.
//
// Selection.  value = score_j + (logit_{j,v} - lse_j), the `count` largest of every
// batch entry, ties to the lowest j V + v.  Inside a beam the order is that of its
// logits, so a first launch reads the logits once: every workgroup leaves, for a
// piece of a beam's words, their maximum, sum of exponentials and at most 64 words
// among which its `count` largest are.  A second launch joins a beam's pieces, forms
// the values in float64, and ranks the beams' words together.  A large score, or an lse
// beside tiny logits, can merge values of different logits in float64 too: words of one
// beam whose values are equal rank by their logits, so that the words left out before
// are never among the best.
//
// What can be left out is found by bisection: t is the largest number that `count` of
// the lanes' maxima reach, and a wave counts them with one comparison and one scalar
// population count a bit; the sixteen high bits do, and few words beyond `count` reach t.
// Where too many do (equal logits), the bisection goes over all of them, with the word
// as the last digits, so that it ends with exactly `count`.
//
// A beam without values (its score or its lse not finite) counts as -infinity for
// every word, which its lowest words then stand for.
//
// Reordering.  A thread holds one place of every beam of an entry: it loads what the
// moved beams come from before it writes any, so rows change places inside the
// buffer, and beams that stay cost nothing.
//
// Measured: 16 entries x 8 beams x 50021 words in float32, 16 candidates, 12 us (the logits
// alone 4 us, the issue of 391 vector instructions a wave another 4 us; the rest is the chain
// of dependent steps that a wave walks) and 8 us for the second launch, one workgroup an
// entry, bound by its chain; 4 beams in bfloat16 5.6 and 6.6 us.  Half of 4 beams of 16
// entries, 168 MB of states, moved in 30 us (5.6 TB/s); of 8 beams at 2.8 TB/s, since its
// threads take 240 registers.
#include <algorithm>
#include <type_traits>

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
constexpr int kList = 256;                      // keys of a wave's list in LDS
static_assert(MSSM_MAX_BEAM_COUNT <= kKeep, "a piece keeps all that are asked for");

// What a piece leaves.
struct Piece {
    float top, sum;            // maximum, sum of exp(logit - maximum)
    uint64_t key[kKeep];       // 0: none
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

// A value of all lanes joined by f, the same in all of them.
template <typename F>
__device__ __forceinline__ float wave_join(float x, F f) {
    const auto dpp = [](float v, auto ctrl) {
        return __builtin_bit_cast(
            float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    x = f(x, dpp(x, std::integral_constant<int, 0xb1>()));    // quad_perm 1 0 3 2
    x = f(x, dpp(x, std::integral_constant<int, 0x4e>()));    // quad_perm 2 3 0 1
    x = f(x, dpp(x, std::integral_constant<int, 0x141>()));   // halves of 8 mirrored
    x = f(x, dpp(x, std::integral_constant<int, 0x140>()));   // rows of 16 mirrored
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return f(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_join(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
    return wave_join(v, [](float a, float b) { return a + b; });
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

// The largest t of multiples of 2^LOW that at least `count` lanes' values reach; 0 if
// fewer hold any.
template <int LOW, typename U>
__device__ __forceinline__ U reached_by(U mine, int count) {
    U t = 0;
#pragma unroll 4
    for (int bit = 8 * sizeof(U) - 1; bit >= LOW; --bit) {
        const U with = t | U(1) << bit;
        if (__popcll(__ballot(mine >= with)) >= count) t = with;
    }
    return t;
}

// Appends those of the lanes' keys to the n that `list` (a wave's own, in LDS) holds
// among which the `count` largest are, in any order; returns how many it holds then: at
// most `room` more, which is `count` or more.
template <int R>
__device__ __forceinline__ int append(const uint64_t (&key)[R], uint64_t *list, int n, int count, int room) {
    uint64_t top = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) top = max(top, key[r]);
    uint64_t t = static_cast<uint64_t>(reached_by<16>(static_cast<uint32_t>(top >> 32), count)) << 32;
    t = max(t, uint64_t(1));
    int reach = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) reach += __popcll(__ballot(key[r] >= t));
    if (reach > room) {
        t = 0;
        for (int bit = 63; bit >= 0; --bit) {
            const uint64_t with = t | uint64_t(1) << bit;
            int found = 0;
#pragma unroll
            for (int r = 0; r < R; ++r) found += __popcll(__ballot(key[r] >= with));
            if (found >= count) t = with;
        }
        t = max(t, uint64_t(1));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint64_t mask = __ballot(key[r] >= t);
        if (key[r] >= t) list[n + lanes_before(mask)] = key[r];
        n += __popcll(mask);
    }
    wave_sync();
    return n;
}

// The same of the n <= kList keys that the list holds, to at most kKeep.
__device__ __forceinline__ int reduce(uint64_t *list, int n, int count) {
    if (n <= kKeep) return n;
    const int lane = threadIdx.x % 64;
    uint64_t key[kList / 64];
#pragma unroll
    for (int r = 0; r < kList / 64; ++r) key[r] = 64 * r + lane < n ? list[64 * r + lane] : 0;
    wave_sync();
    return append(key, list, 0, count, kKeep);
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
    __shared__ uint64_t lists[kWaves * kList];
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
#pragma unroll
    for (int j = 0; j < kItems; ++j) top = fmaxf(top, v[j]);   // passes over NaN
    const float mine = top;
    top = wave_max(top);
    float sum = 0.0f;                       // 0 without finite logits, NaN with +infinity or NaN
    const float base = top == kLow ? 0.0f : top;
#pragma unroll
    for (int j = 0; j < kItems; ++j) sum += fast_exp2((v[j] - base) * kLog2e);
    sum = wave_sum(sum);

    uint64_t *const own = lists + wave * kList;
    // A lane that holds nothing above -infinity counts as less than all that do.
    const uint32_t t = reached_by<16>(ordered(mine), count);
    const float limit = unordered(t);
    int n = 0;
    if (limit > kLow) {
#pragma unroll
        for (int j = 0; j < kItems; ++j) n += __popcll(__ballot(v[j] >= limit));
    }
    if (n > 0 && n <= kList) {
        n = 0;
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const uint64_t mask = __ballot(v[j] >= limit);
            if (v[j] >= limit) own[n + lanes_before(mask)] = key_of(ordered(v[j]), word(j));
            n += __popcll(mask);
        }
        wave_sync();
    } else {                                // words at -infinity are asked for, or very many are equal
        uint64_t key[kItems];
#pragma unroll
        for (int j = 0; j < kItems; ++j)
            key[j] = word(j) < vocab ? key_of(ordered(v[j] != v[j] ? kLow : v[j]), word(j)) : 0;
        n = append(key, own, 0, count, kList);
    }
    n = reduce(own, n, count);
    if (lane == 0) {
        tops[wave] = top;
        sums[wave] = sum;
        counts[wave] = n;
    }
    __syncthreads();
    if (wave > 0) return;
    // the same of what the waves left
    uint64_t left[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) left[w] = lane < counts[w] ? lists[w * kList + lane] : 0;
    wave_sync();
    const int total = append(left, lists, 0, count, kKeep);
    Piece &p = out[blockIdx.x];
    p.key[lane] = lane < total ? lists[lane] : 0;
    const float my_top = lane < kWaves ? tops[lane] : kLow, all = wave_max(my_top);
    float part = 0.0f;
    if (lane < kWaves && sums[lane] != 0.0f) part = sums[lane] * fast_exp2((my_top - all) * kLog2e);
    part = wave_sum(part);
    if (lane == 0) {
        p.top = all;
        p.sum = part;
    }
}

// A workgroup per batch entry, a wave at a time per beam.
constexpr int kMergeWaves = 8, kMergeThreads = 64 * kMergeWaves;
constexpr int kTogether = 16;    // pieces that a lane loads at once

// A float64 as an unsigned number of the same order, for values without NaN; -0 does not occur.
__device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
    return b >> 63 ? ~b : b | uint64_t(1) << 63;
}

// Of two of equal value comes first that of the lower place: the lower beam, in it the
// larger logit; then the lower word.
struct __attribute__((aligned(16))) Candidate {
    double value;
    uint64_t place;     // beam, and the inverted order of the logit
};


__global__ __launch_bounds__(kMergeThreads) void beam_merge_kernel(
    const Piece *__restrict__ in, const float *__restrict__ scores, float *__restrict__ out_scores,
    int64_t *__restrict__ out_tokens, int64_t *__restrict__ out_beams, int beams, int vocab, int count, int pieces) {
    __shared__ uint64_t lists[kMergeWaves * kList];
    __shared__ Candidate all[MSSM_MAX_BEAMS * kKeep];
    __shared__ int words[MSSM_MAX_BEAMS * kKeep];
    __shared__ int total;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t entry = blockIdx.x;
    const double kLow = -__builtin_inf();
    uint64_t *const list = lists + wave * kList;
    if (threadIdx.x == 0) total = 0;
    __syncthreads();
    for (int j = wave; j < beams; j += kMergeWaves) {
        const int64_t row = entry * beams + j;
        const Piece *const mine = in + row * pieces;
        const float score32 = scores[row];
        const bool few = pieces <= 64;
        const float2 first = lane < pieces ? *reinterpret_cast<const float2 *>(&mine[lane].top) : float2{-__builtin_inff(), 0.0f};
        int n = 0;
        for (int s = 0; s < pieces; s += kTogether) {
            // a piece's keys lie in its first places: turned, so that all lanes receive some
            uint64_t key[kTogether];
#pragma unroll
            for (int i = 0; i < kTogether; ++i)
                key[i] = s + i < pieces ? mine[s + i].key[(lane + i * (64 / kTogether)) % 64] : 0;
            n = reduce(list, append(key, list, n, count, kList - n), count);
        }
        float top = first.x;
        for (int s = 64 + lane; !few && s < pieces; s += 64) top = fmaxf(top, mine[s].top);
        top = wave_max(top);
        double sum = first.y != 0.0f ? static_cast<double>(first.y) * expf(first.x - top) : 0.0;
        for (int s = 64 + lane; !few && s < pieces; s += 64)
            if (mine[s].sum != 0.0f) sum += static_cast<double>(mine[s].sum) * expf(mine[s].top - top);
#pragma unroll
        for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
        const double lse = top + log(sum), score = score32;
        const bool live = fabs(lse) < __builtin_inf() && fabs(score) < __builtin_inf();
        if (!live) n = min(count, vocab);
        int at = 0;
        if (lane == 0) at = atomicAdd(&total, n);      // where, not in which order they rank
        at = __shfl(at, 0);
        if (lane < n) {
            const uint64_t key = live ? list[lane] : 0;
            const int word = live ? word_of(key) : lane;
            all[at + lane] = Candidate{live ? score + (unordered(static_cast<uint32_t>(key >> 32)) - lse) : kLow,
                                       static_cast<uint64_t>(j) << 32 | ~static_cast<uint32_t>(key >> 32)};
            words[at + lane] = word;
        }
    }
    __syncthreads();
    // Every value's rank is how many come before it; of many, those below what `count` of a
    // wave's lanes reach are left out first.
    const int n = total;
    uint64_t t = 0;
    if (n > kMergeThreads / 2) {
        uint64_t best = 0;
        for (int i = lane; i < n; i += 64) best = max(best, ordered(all[i].value));
        t = reached_by<0>(best, count);
        __syncthreads();
        if (threadIdx.x == 0) total = 0;
        __syncthreads();
        constexpr int kEach = MSSM_MAX_BEAMS * kKeep / kMergeThreads;
        Candidate c[kEach];
        int word[kEach];
#pragma unroll
        for (int r = 0; r < kEach; ++r)
            if (r * kMergeThreads + static_cast<int>(threadIdx.x) < n) {
                c[r] = all[r * kMergeThreads + threadIdx.x];
                word[r] = words[r * kMergeThreads + threadIdx.x];
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kEach; ++r)
            if (r * kMergeThreads + static_cast<int>(threadIdx.x) < n && ordered(c[r].value) >= t) {
                const int to = atomicAdd(&total, 1);
                all[to] = c[r];
                words[to] = word[r];
            }
        __syncthreads();
    }
    const int left = total;
    for (int i = threadIdx.x; i < left; i += kMergeThreads) {
        const Candidate mine = all[i];
        const int word = words[i];
        int rank = 0, same = 0;
#pragma unroll 8
        for (int k = 0; k < left; ++k) {
            const double value = all[k].value;
            rank += value > mine.value;
            same += value == mine.value;
        }
        if (same > 1) {
#pragma unroll 8
            for (int k = 0; k < left; ++k) {
                const Candidate c = all[k];
                rank += (c.value == mine.value) & ((c.place < mine.place) | ((c.place == mine.place) & (words[k] < word)));
            }
        }
        if (rank < count) {
            out_scores[entry * count + rank] = static_cast<float>(mine.value);
            out_tokens[entry * count + rank] = word;
            out_beams[entry * count + rank] = static_cast<int64_t>(mine.place >> 32);
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
    hipLaunchKernelGGL(beam_merge_kernel, dim3(static_cast<uint32_t>(a.batch)), dim3(kMergeThreads), 0, stream,
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
