// gated_recurrence.hip -- the elementwise gated linear recurrence, forward and
// backward.
//
//   log a_t = -c softplus(lam) sigmoid(r_t)
//   h_t     = a_t h_{t-1} + m_t sigmoid(i_t) x_t,   m_t = sqrt(1 - a_t^2),   y_t = h_t
// and from the end, with the carry G,
//   g_t = dy_t + G,   G <- a_t g_t
//   w   = g h_{t-1} a log a - g sigmoid(i) x a^2 (log a / m)
//   dx = g m sigmoid(i),  di = dx x (1 - sigmoid(i)),  dr = w (1 - sigmoid(r)),
//   dlam = sum w sigmoid(lam) / softplus(lam)
//
// Both walks are one affine recurrence s <- a s + b (backward: time reversed,
// b = a dy), so a run of steps composes into one pair (A, H): s <- A s + H.
// The operator reads three tensors and writes one (backward: five and three),
// so it is bound by HBM if it reads them once; in bfloat16 the forward's
// vector work (37 instructions an element, six of them transcendental) takes
// 43 us where its 8 bytes an element take 54 us (2 x 4096 steps of 5120
// channels).  Hence one pass, in which loads, arithmetic and the passing of
// carries all go on at the same time, one workgroup of twelve waves a compute
// unit:
//
//   1. A workgroup holds a segment of steps of 64 channels in registers.
//      Eleven waves compute: a slot of 64 / V lanes holds K consecutive steps, a
//      lane V channels.  A lane composes its steps; the slots' pairs meet in
//      LDS.
//   2. The twelfth wave, one lane a channel, exchanges: it composes the slots,
//      publishes the segment's pair, finds the state that enters the segment
//      and hands every slot the state that enters it.  The entering state is
//      the fold, in order, of a state published every kSpan segments, of pairs
//      of whole blocks and of whole runs of segments, and of the last pairs:
//      at most 3 (kRun - 1) + 1 values read, all at once, and one hand-over per
//      kSpan segments on the serial path.
//   3. Meanwhile the computing waves form the terms of the next segment, with
//      the loads of the two after it in flight, and then walk this one's terms
//      again from registers.  (With two workgroups of eight waves and a
//      segment's terms waiting for its exchange, the exchange showed: 115 us
//      against 87 us.)
// Loads and stores are buffer operations without branches around them: the
// compiler otherwise waits for all loads in flight where paths meet.
// The association is fixed by the sizes alone, so results repeat bit for bit.
//
// Segments are handed out by tickets in segment-major order.  A workgroup
// takes its tickets in increasing order and publishes a segment's pair before
// it waits for anything, and it waits only for values of lower tickets; so the
// lowest ticket that is not finished never waits, and every wait ends.
// Published values cross the XCDs' L2 caches in 8-byte agent-scope atomics that
// carry a mark of their own beside the value (A is never negative, so its sign
// bit is free): a reader that sees the mark has the value, without a flag and
// the wait for stores that a flag needs (0.56 us from a store to a load that
// sees it).  The marks are cleared by a kernel in front.
//
// Measured (2 x 4096 steps of 5120 channels, bfloat16): forward 88 us (3.8
// TB/s), backward 164 us (4.1 TB/s); float32 forward 135 us (5.0 TB/s).
#include "device_math.h"
#include "internal.h"

namespace mssm {

// Status bits of this translation unit's kernels (mssm_device_status).
__device__ uint32_t g_recurrence_status_bits;

namespace {

constexpr int kRowThreads = 64;
constexpr int kComputeWaves = 11;
constexpr int kThreads = 64 * (kComputeWaves + 1);
constexpr int kChannels = 64;            // of a group: one lane of the exchanging wave each
constexpr int kRun = 8;                  // segments in a run, runs in a block, blocks between states
constexpr int kBlock = kRun * kRun, kSpan = kRun * kBlock;
constexpr uint32_t kMaxPolls = 1u << 20;   // a wait gives up after about a second
constexpr float kSeriesLimit = 0.35f;

// Up to this many steps one lane walks a row; a segment pays for all its steps.
// Forward in bfloat16, a lane a row against segments: 8 x 8 steps x 5120 channels
// 4.1 us against 21, 64 x 8 x 2560 5.7 against 50, 8 x 64 x 5120 29.5 against 23.6,
// 1 x 64 x 512 16.7 against 11.0.  (They meet near 48 steps, 22.8 against 22.6 and
// 12.9 against 11.0: from 9 to 32 steps segments take 1.2 to 8 times as long.)
constexpr int64_t kRowSteps = 8;

// 1 / (1 + 2^(-x log2 e)).
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-x * kLog2e));
}

// e^x - 1 for -0.35 <= x <= 0: the Taylor series, its remainder below 2e-8 of
// the value.
__device__ __forceinline__ float expm1_series(float x) {
    float p = 1.0f / 5040.0f;
    p = fmaf(p, x, 1.0f / 720.0f);
    p = fmaf(p, x, 1.0f / 120.0f);
    p = fmaf(p, x, 1.0f / 24.0f);
    p = fmaf(p, x, 1.0f / 6.0f);
    p = fmaf(p, x, 0.5f);
    return fmaf(p * x, x, x);
}

// Below -0.35 a decay a = e^x is taken from the exponential (1 + (a - 1) would
// leave a fast one few digits), from there up from the series (a - 1, of which
// 1 - a^2 is formed, would lose what matters as a nears 1).
__device__ __forceinline__ bool is_far(float x) { return x < -kSeriesLimit; }

// a and a - 1 for x = log a <= 0.  NEAR: x is known to be -0.35 or more.  (A wave
// knows where all its channels' rates are: decays from 0.9 a step take the layer's
// forward 89.9 us and its backward 163.7 us, decays from 0.3, which mix both
// ranges, 91.8 and 165.7 us, one call after the other.)
struct Decay {
    float a, p;
};
template <bool NEAR>
__device__ __forceinline__ Decay decay(float x) {
    const float p = expm1_series(x);
    Decay d{1.0f + p, p};
    if (!NEAR) {
        const float a = fast_exp2(x * kLog2e);
        d = is_far(x) ? Decay{a, a - 1.0f} : d;
    }
    return d;
}

// A decay as the one number that has its digits, and back.  (The backward's walk of
// the layer tells the two apart in 1 us; a walk of its own where none is far spills
// and takes 393 us.)
template <bool NEAR>
__device__ __forceinline__ float kept_of(float x, const Decay &d) { return !NEAR && is_far(x) ? d.a : d.p; }
__device__ __forceinline__ Decay decay_of_kept(float x, float kept) {
    return is_far(x) ? Decay{kept, kept - 1.0f} : Decay{1.0f + kept, kept};
}

// 1 - a^2 = -(a - 1)(a - 1 + 2), times 2^64: next to a closed gate it is
// subnormal, which v_sqrt_f32 takes for zero and v_rsq_f32 makes infinite.  (The
// scaling costs 0.3 us of the layer's forward and of its backward.)
constexpr float kUp = 0x1p64f, kRoot = 0x1p32f;
__device__ __forceinline__ float one_minus_square(float p) { return p * fmaf(p, -kUp, -2.0f * kUp); }
// m = sqrt(1 - a^2).
__device__ __forceinline__ float input_scale(float p) {
    return __builtin_amdgcn_sqrtf(one_minus_square(p)) * (1.0f / kRoot);
}

// V consecutive elements at any element address.
template <typename T, int V> struct Pack;
template <> struct Pack<float, 1> {
    float v;
    __device__ __forceinline__ float get(int) const { return v; }
    __device__ __forceinline__ void set(const float *f) { v = f[0]; }
};
template <> struct Pack<uint16_t, 1> {
    uint16_t v;
    __device__ __forceinline__ float get(int) const { return bf16_to_f32(v); }
    __device__ __forceinline__ void set(const float *f) { v = f32_to_bf16(f[0]); }
};
template <> struct Pack<uint16_t, 2> {
    uint32_t v;
    __device__ __forceinline__ float get(int k) const { return __uint_as_float(k ? v & 0xffff0000u : v << 16); }
    __device__ __forceinline__ void set(const float *f) {
        typedef float f2 __attribute__((ext_vector_type(2)));
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        v = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){f[0], f[1]}, b2));
    }
};
// A tensor from the element `at` on, for buffer loads and stores: byte offsets
// past its end (kOutside among them) read as zero and store nothing.  So the
// rows and channels past a ragged end need no branch around a load, which would
// make the compiler wait for all loads in flight where the paths meet.
constexpr uint32_t kOutside = 0xffffffffu;
constexpr int kStream = 2;               // nontemporal: every value is read or written once
typedef __amdgpu_buffer_rsrc_t Buffer;
template <typename T>
__device__ __forceinline__ Buffer buffer_at(const T *p, int64_t at, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(p) + at, 0, bytes, 0x00020000);
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(Buffer b, uint32_t off) {
    Pack<T, V> p;
    if constexpr (sizeof p == 4) p.v = __builtin_bit_cast(decltype(p.v), __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, kStream));
    else p.v = __builtin_amdgcn_raw_buffer_load_b16(b, off, 0, kStream);
    return p;
}
__device__ __forceinline__ float load_float(Buffer b, uint32_t off) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0));
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(Buffer b, uint32_t off, const float *f) {
    Pack<T, V> p;
    p.set(f);
    if constexpr (sizeof p == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, p.v), b, off, 0, kStream);
    else __builtin_amdgcn_raw_buffer_store_b16(p.v, b, off, 0, kStream);
}

// ---- a few steps: one lane walks a row -------------------------------------------

template <typename T>
__global__ __launch_bounds__(kRowThreads) void row_fwd_kernel(const T *__restrict__ x, const T *__restrict__ r,
                                                              const T *__restrict__ i,
                                                              const float *__restrict__ lam, float scale,
                                                              const float *h0, T *__restrict__ y, float *h_last,
                                                              int64_t rows, int L, int64_t dim) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
    if (row >= rows) return;
    const int64_t b = row / dim, d = row - b * dim;
    float h = h0 ? h0[row] : 0.0f;
    const float rate = -scale * softplus_libm(lam[d]);
    int64_t at = b * L * dim + d;
    for (int t = 0; t < L; ++t, at += dim) {
        const Decay c = decay<false>(rate * sigmoid(Io<T>::load(r, at)));
        h = fmaf(c.a, h, input_scale(c.p) * sigmoid(Io<T>::load(i, at)) * Io<T>::load(x, at));
        Io<T>::store(y, at, h);
    }
    if (h_last) h_last[row] = h;
}

// ---- segments ----------------------------------------------------------------------

// What segments exchange, 8 bytes a channel: pairs (A, H) per (segment, group),
// per (run of segments, group) and per (block of runs, group), states per
// (span of blocks, group); and the ticket.
struct Exchange {
    uint64_t *pairs[3], *states;
    uint32_t *ticket;
    int nseg, groups;
    int chunk, chunks;                   // groups a ticket, tickets a segment
};

struct Walk {
    const float *rates;                  // -scale softplus(lam) of every channel
    int64_t L, count, rows;              // count: elements of an activation, rows: of a state
    int dim, groups_per_batch, items, nseg;
};

constexpr uint64_t kMark = 0x80000000u;  // the sign of the lower half
__device__ __forceinline__ void put(uint64_t *p, float low, float high) {
    __hip_atomic_store(p, static_cast<uint64_t>(__float_as_uint(low)) | kMark |
                              static_cast<uint64_t>(__float_as_uint(high)) << 32,
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float low_of(uint64_t b) { return __uint_as_float(static_cast<uint32_t>(b) & 0x7fffffffu); }
__device__ __forceinline__ float high_of(uint64_t b) { return __uint_as_float(static_cast<uint32_t>(b >> 32)); }
__device__ __forceinline__ float2 then(float2 first, float2 second) {
    return make_float2(second.x * first.x, fmaf(second.x, first.y, second.y));
}

__device__ __forceinline__ uint64_t get(const uint64_t *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The exchanging wave's work on one item: from the slots' pairs the states
// that enter them, one lane a channel.  `init`: the caller's initial state of
// this group's channels (null: zero); `last`: where the final state goes (may
// be null).
template <int SLOTS>
__device__ __forceinline__ void exchange(int lane, int seg, int group, const float *init, float *last, int valid,
                                         const Exchange &ex, const float2 (*slot)[kChannels], float (*enter)[kChannels]) {
    float2 own = make_float2(1.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) own = then(own, slot[k][lane]);
    // Read before this segment's pair is published: the last segment, which
    // may write the same buffer, waits for that pair.
    const int span = seg / kSpan;
    float s = span == 0 && init ? init[min(lane, valid - 1)] : 0.0f;
    if (ex.nseg > 1) {
        const bool more = seg < ex.nseg - 1;
        const int64_t stride = static_cast<int64_t>(ex.groups) * kChannels,
                      here = static_cast<int64_t>(group) * kChannels + lane;   // groups may pass 2^25
        asm volatile("" : "+v"(s) : : "memory");   // has arrived
        if (more) put(ex.pairs[0] + seg * stride + here, own.x, own.y);
        // n[l] values of level l: pairs since the last whole run, runs since
        // the last whole block, blocks since the state published last
        const int n[3] = {seg % kRun, seg / kRun % kRun, seg / kBlock % kRun};
        const int64_t first[3] = {seg - n[0], seg / kRun - n[1], seg / kBlock - n[2]};
        uint64_t b[3][kRun - 1], st = kMark;
        float2 pair[3];
        bool ok = true;
        const auto load = [&](int l) {
            const uint64_t *from = ex.pairs[l] + first[l] * stride + here;
#pragma unroll
            for (int k = 0; k < kRun - 1; ++k) {
                if (k < n[l]) b[l][k] = get(from);
                from += stride;
                asm volatile("" : "+v"(from));     // one address at a time: few registers
            }
        };
        const auto fold = [&](int l) {
            uint64_t all = kMark;
            pair[l] = make_float2(1.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kRun - 1; ++k)
                if (k < n[l]) {
                    all &= b[l][k];
                    pair[l] = then(pair[l], make_float2(low_of(b[l][k]), high_of(b[l][k])));
                }
            return __all((all & kMark) != 0);
        };
        // All levels are read at once; one whose values are not all there is
        // read again until they are.  The wait gives up only on a defect, since
        // the values of lower tickets always arrive.
        uint32_t polls = 0;
        load(0);
        load(1);
        load(2);
        if (span > 0) st = get(ex.states + (span - 1) * stride + here);
        float2 upto = own;                         // of this level's whole run, if this segment ends it
#pragma unroll
        for (int l = 0; l < 3; ++l) {
            while (!fold(l)) {
                if (++polls >= kMaxPolls) {
                    ok = false;
                    break;
                }
                __builtin_amdgcn_s_sleep(2);
                load(l);
            }
            // the end of a run (a block) publishes its pair before it waits on
            if (l < 2 && more && n[l] == kRun - 1 && (l == 0 || n[0] == kRun - 1)) {
                upto = then(pair[l], upto);
                put(ex.pairs[l + 1] + (first[l] / kRun) * stride + here, upto.x, upto.y);
            }
        }
        while (!__all((st & kMark) != 0)) {
            if (++polls >= kMaxPolls) {
                ok = false;
                break;
            }
            __builtin_amdgcn_s_sleep(2);
            st = get(ex.states + (span - 1) * stride + here);
        }
        if (span > 0) s = high_of(st);
#pragma unroll
        for (int l = 2; l >= 0; --l) s = fmaf(pair[l].x, s, pair[l].y);
        s = ok ? s : __builtin_nanf("");
        if (!ok && lane == 0)
            __hip_atomic_fetch_or(&g_recurrence_status_bits, MSSM_DEVICE_RECURRENCE_TIMEOUT, __ATOMIC_RELAXED,
                                  __HIP_MEMORY_SCOPE_AGENT);
        if (more && seg % kSpan == kSpan - 1)
            put(ex.states + span * stride + here, 0.0f, fmaf(own.x, s, own.y));
    }
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
        enter[k][lane] = s;
        s = fmaf(slot[k][lane].x, s, slot[k][lane].y);
    }
    if (last && seg == ex.nseg - 1 && lane < valid) last[lane] = s;
}

// The (segment, batch, run of channels) of an item.
struct Place {
    int seg, group, batch, ch0, valid;
    int64_t row;                         // of the states: batch * dim + ch0
};
__device__ __forceinline__ Place place_of(int item, const Walk &w, const Exchange &ex) {
    Place p;
    p.seg = item / ex.groups;
    p.group = item - p.seg * ex.groups;
    p.batch = p.group / w.groups_per_batch;
    p.ch0 = (p.group - p.batch * w.groups_per_batch) * kChannels;
    p.valid = min(kChannels, w.dim - p.ch0);
    p.row = static_cast<int64_t>(p.batch) * w.dim + p.ch0;
    return p;
}

// What the computing waves need of an item, made once by the exchanging wave.
// Steps are counted in the order of the walk; step j of it lies at byte
// (backward: S - j rows, top - j rows where the item is not full) from the
// element `at`.
struct Item {
    int64_t at, row;                     // row: of the states
    int bytes;                           // from `at` to the tensor's end, for buffers
    int steps, top, ch0, valid, full, last, there;
};

// Forward: the segment's steps run up from its first.
__device__ __forceinline__ Item fwd_item(const Place &p, const Walk &w, int S, int size) {
    Item it;
    const int64_t t0 = static_cast<int64_t>(p.seg) * S;
    it.at = (p.batch * w.L + t0) * w.dim + p.ch0;
    it.steps = static_cast<int>(min(w.L - t0, static_cast<int64_t>(S)));
    it.top = 0;
    it.full = it.steps == S;
    it.bytes = static_cast<int>(min((w.count - it.at) * size, static_cast<int64_t>(0x7fffffff)));
    return it;
}

// Backward: they run down from its last; `at` is in the row before them, or,
// where there is none (not full), in the sequence's first.
__device__ __forceinline__ Item bwd_item(const Place &p, const Walk &w, int S, int size) {
    Item it;
    const int64_t hi = w.L - 1 - static_cast<int64_t>(p.seg) * S;
    it.full = hi >= S;
    it.at = (p.batch * w.L + (it.full ? hi - S : 0)) * w.dim + p.ch0;
    it.steps = static_cast<int>(min(hi + 1, static_cast<int64_t>(S)));
    it.top = it.full ? S : it.steps - 1;
    it.bytes = static_cast<int>(min((w.count - it.at) * size, static_cast<int64_t>(0x7fffffff)));
    return it;
}

// A lane's part: row k at byte off + k step (backward: off - k step), `steps` of
// its K rows exist.
struct Part {
    uint32_t off;
    int steps;
};

// A forward item: what is loaded, and what is kept of it until it is finished.
template <typename T, int V, int K>
struct Fwd {
    static constexpr int kWavesPerSimd = 3, kLanes = kChannels / V, kSlots = 64 * kComputeWaves / kLanes, kSteps = kSlots * K;
    const T *x, *r, *i;
    T *y;

    struct Raw {
        Pack<T, V> x[K], r[K], i[K];
        float rate[V];
    };
    struct Terms {
        float a[K][V], b[K][V];
    };
    static __device__ __forceinline__ Item item(const Place &p, const Walk &w) {
        return fwd_item(p, w, kSteps, sizeof(T));
    }
    static __device__ __forceinline__ Part part(const Item &it, uint32_t step, int slot, int c0) {
        Part pt;
        pt.steps = c0 < it.valid ? min(max(it.steps - slot * K, 0), K) : 0;
        pt.off = slot * K * step + c0 * sizeof(T);
        return pt;
    }
    __device__ __forceinline__ void load(Raw &raw, const Item &it, const Part &pt, const Walk &w, uint32_t step, int c0) const {
        const Buffer xb = buffer_at(x, it.at, it.bytes), rb = buffer_at(r, it.at, it.bytes),
                     ib = buffer_at(i, it.at, it.bytes), sb = buffer_at(w.rates, it.ch0, 4 * it.valid);
#pragma unroll
        for (int v = 0; v < V; ++v) raw.rate[v] = load_float(sb, 4 * (c0 + v));
        uint32_t o = pt.off;
#pragma unroll
        for (int k = 0; k < K; ++k, o += step) {
            raw.r[k] = load_pack<T, V>(rb, o);
            raw.i[k] = load_pack<T, V>(ib, o);
            raw.x[k] = load_pack<T, V>(xb, o);
        }
    }
    template <bool NEAR>
    __device__ __forceinline__ void terms(Terms &t, const Raw &raw, const Part &pt, float2 *pair) const {
#pragma unroll
        for (int v = 0; v < V; ++v) pair[v] = make_float2(1.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Decay d = decay<NEAR>(raw.rate[v] * sigmoid(raw.r[k].get(v)));
                float a = d.a, in = input_scale(d.p) * sigmoid(raw.i[k].get(v)) * raw.x[k].get(v);
                if (!NEAR && k >= pt.steps) a = 1.0f, in = 0.0f;
                t.a[k][v] = a;
                t.b[k][v] = in;
                pair[v] = then(pair[v], make_float2(t.a[k][v], in));
            }
    }
    __device__ __forceinline__ void finish(const Terms &t, const Item &it, const Part &pt, uint32_t step, int, float *h,
                                           float *) const {
        const Buffer yb = buffer_at(y, it.at, it.bytes);
        uint32_t o = pt.off;
#pragma unroll
        for (int k = 0; k < K; ++k, o += step) {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fmaf(t.a[k][v], h[v], t.b[k][v]);
            store_pack<T, V>(yb, k < pt.steps ? o : kOutside, h);
        }
    }
};

// One element of the backward.  G: the carry, advanced past this step.
struct Grad {
    float dx, dr, di, w;
};
__device__ __forceinline__ Grad grad_step(float la, float sr, const Decay &d, float x, float i, float dy, float before,
                                          float *G) {
    const float em = one_minus_square(d.p);
    const float rs = em > 0.0f ? __builtin_amdgcn_rsqf(em) : 0.0f;   // log a / m -> 0 with log a
    const float rm = rs * kRoot;
    const float si = sigmoid(i), u = si * x;
    const float g = dy + *G, gm = g * (em * rs * (1.0f / kRoot));
    *G = d.a * g;
    Grad o;
    o.w = *G * la * fmaf(-u * d.a, rm, before);
    o.dx = gm * si;
    o.di = gm * u * (1.0f - si);
    o.dr = o.w * (1.0f - sr);
    return o;
}

// A backward item: the inputs are kept as they are stored, with sigmoid(r) and
// the decay.  y: the state before each row.
template <typename T, int V, int K>
struct Bwd {
    static constexpr int kWavesPerSimd = 3, kLanes = kChannels / V, kSlots = 64 * kComputeWaves / kLanes, kSteps = kSlots * K;
    const T *x, *r, *i, *y, *dy;
    T *dx, *dr, *di;
    const float *h0;                         // may be null -> 0

    struct Raw {
        Pack<T, V> x[K], i[K], y[K], dy[K], r[K];
        float rate[V], start[V];             // start: the state before the sequence's first step
    };
    struct Terms {
        Pack<T, V> x[K], i[K], y[K], dy[K];
        float sr[K][V], kept[K][V], rate[V], start[V];
    };
    static __device__ __forceinline__ Item item(const Place &p, const Walk &w) {
        return bwd_item(p, w, kSteps, sizeof(T));
    }
    static __device__ __forceinline__ Part part(const Item &it, uint32_t step, int slot, int c0) {
        Part pt;
        pt.steps = c0 < it.valid ? min(max(it.steps - slot * K, 0), K) : 0;
        pt.off = (it.top - slot * K) * step + c0 * sizeof(T);
        return pt;
    }
    __device__ __forceinline__ void load(Raw &raw, const Item &it, const Part &pt, const Walk &w, uint32_t step, int c0) const {
        const Buffer sb = buffer_at(w.rates, it.ch0, 4 * it.valid),
                     hb = buffer_at(h0, it.row, h0 && it.last ? 4 * it.valid : 0);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            raw.rate[v] = load_float(sb, 4 * (c0 + v));
            raw.start[v] = load_float(hb, 4 * (c0 + v));
        }
        const Buffer xb = buffer_at(x, it.at, it.bytes), rb = buffer_at(r, it.at, it.bytes),
                     ib = buffer_at(i, it.at, it.bytes), yb = buffer_at(y, it.at, it.bytes),
                     gb = buffer_at(dy, it.at, it.bytes);
        uint32_t o = pt.steps ? pt.off : kOutside;     // a row before the first: past every end
#pragma unroll
        for (int k = 0; k < K; ++k, o -= step) {
            raw.r[k] = load_pack<T, V>(rb, o);
            raw.dy[k] = load_pack<T, V>(gb, o);
            raw.x[k] = load_pack<T, V>(xb, o);
            raw.i[k] = load_pack<T, V>(ib, o);
            raw.y[k] = load_pack<T, V>(yb, o - step);
        }
    }
    template <bool NEAR>
    __device__ __forceinline__ void terms(Terms &t, const Raw &raw, const Part &pt, float2 *pair) const {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            pair[v] = make_float2(1.0f, 0.0f);
            t.rate[v] = raw.rate[v];
            t.start[v] = raw.start[v];
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            t.x[k] = raw.x[k];
            t.i[k] = raw.i[k];
            t.y[k] = raw.y[k];
            t.dy[k] = raw.dy[k];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                t.sr[k][v] = sigmoid(raw.r[k].get(v));
                const float la = raw.rate[v] * t.sr[k][v];
                const Decay d = decay<NEAR>(la);
                t.kept[k][v] = kept_of<NEAR>(la, d);
                if (NEAR || k < pt.steps) pair[v] = make_float2(pair[v].x * d.a, d.a * (raw.dy[k].get(v) + pair[v].y));
            }
        }
    }
    __device__ __forceinline__ void finish(const Terms &t, const Item &it, const Part &pt, uint32_t step, int slot,
                                           float *G, float *sum) const {
        const Buffer dxb = buffer_at(dx, it.at, it.bytes), drb = buffer_at(dr, it.at, it.bytes),
                     dib = buffer_at(di, it.at, it.bytes);
        // where the item is not full, its last step is the sequence's first
        const int first = it.full ? K : it.steps - 1 - slot * K;
        uint32_t o = pt.off;
#pragma unroll
        for (int k = 0; k < K; ++k, o -= step) {
            const bool in = k < pt.steps;
            float ox[V], og[V], oi[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float before = k == first ? t.start[v] : t.y[k].get(v);
                const float la = t.rate[v] * t.sr[k][v];
                const Grad g = grad_step(la, t.sr[k][v], decay_of_kept(la, t.kept[k][v]), t.x[k].get(v),
                                         t.i[k].get(v), t.dy[k].get(v), before, &G[v]);
                ox[v] = g.dx;
                og[v] = g.dr;
                oi[v] = g.di;
                sum[v] += in ? g.w : 0.0f;
            }
            const uint32_t to = in ? o : kOutside;
            store_pack<T, V>(dxb, to, ox);
            store_pack<T, V>(drb, to, og);
            store_pack<T, V>(dib, to, oi);
        }
    }
};

template <int SLOTS>
struct Shared {
    float2 slot[2][SLOTS][kChannels];    // pairs of the slots
    float enter[2][SLOTS][kChannels];    // states that enter them
    float sum[2][SLOTS][kChannels];      // dlam's terms (backward)
    Item item[8];                        // the items under way
};

// The state that a walk starts from and where its final state goes, per
// (batch, channel), either may be null; part: dlam's terms per (segment,
// batch, channel).
struct States {
    const float *init;
    float *last;
    float *part;
};

// Barriers: the computing waves and the exchanging one pass the same ones.
// Iteration `it` ends item `it`: before its barrier the terms of item it + 1 are
// formed and the states that enter item it are found, after it item it is
// finished.
template <typename Op, typename T, int V, bool SUM>
__global__ __launch_bounds__(kThreads, Op::kWavesPerSimd) void segment_kernel(Op op, States st, Walk w, Exchange ex) {
    constexpr int kSlots = Op::kSlots;
    __shared__ Shared<kSlots> sm;
    const int tid = threadIdx.x, lane = tid % 64;
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
    if (wave == kComputeWaves) {
        // Tickets, where segments wait for each other; else block indexes.  A
        // ticket is asked for when the one before it is taken up.
        int asked, next = blockIdx.x, seg = 0, g = 0, g_end = 0;
        const auto ask = [&]() {
            asked = next;
            next += gridDim.x;
            if (ex.nseg > 1 && lane == 0)
                asked = static_cast<int>(
                    __hip_atomic_fetch_add(ex.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
        };
        const auto announce = [&](int it) {
            if (g == g_end) {
                const int ticket = __builtin_amdgcn_readfirstlane(asked);
                ask();
                seg = ticket / ex.chunks;
                g = min((ticket - seg * ex.chunks) * ex.chunk, ex.groups);
                g_end = min(g + ex.chunk, ex.groups);
            }
            const int item = seg < ex.nseg ? seg * ex.groups + g : w.items;
            ++g;
            Item of{};                       // no bytes: an item past the last loads nothing
            if (item < w.items) {
                const Place p = place_of(item, w, ex);
                of = Op::item(p, w);
                of.row = p.row;
                of.ch0 = p.ch0;
                of.valid = p.valid;
                of.last = p.seg == ex.nseg - 1;
                of.there = 1;
            }
            if (lane == 0) sm.item[it & 7] = of;
            return item;
        };
        const auto add_up = [&](int it, int item) {
            const Place p = place_of(item, w, ex);
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < kSlots; ++k) s += sm.sum[it & 1][k][lane];
            if (lane < p.valid) st.part[p.seg * w.rows + p.row + lane] = s;
        };
        int items[4], done1 = 0, done2 = 0, it = 0;          // of it .. it + 3; it - 1, it - 2
        ask();
        for (int k = 0; k < 4; ++k) items[k] = announce(k);
        __syncthreads();
        __syncthreads();
        for (; items[0] < w.items; ++it) {
            const Place p = place_of(items[0], w, ex);
            exchange<kSlots>(lane, p.seg, p.group, st.init ? st.init + p.row : nullptr,
                             st.last ? st.last + p.row : nullptr, p.valid, ex, sm.slot[it & 1], sm.enter[it & 1]);
            const int ahead = announce(it + 4);
            if (SUM && it >= 2) add_up(it - 2, done2);
            __syncthreads();
            done2 = done1;
            done1 = items[0];
            items[0] = items[1];
            items[1] = items[2];
            items[2] = items[3];
            items[3] = ahead;
        }
        if (SUM) {
            if (it >= 2) add_up(it - 2, done2);
            __syncthreads();
            if (it >= 1) add_up(it - 1, done1);
        }
        return;
    }

    const int slot = tid / Op::kLanes, c0 = (tid % Op::kLanes) * V;
    typename Op::Raw raw[2];
    const uint32_t step = static_cast<uint32_t>(w.dim) * sizeof(T);
    const auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    const auto uniform64 = [&](int64_t v) {
        return static_cast<int64_t>(static_cast<uint32_t>(uniform(static_cast<int>(v)))) |
               static_cast<int64_t>(uniform(static_cast<int>(v >> 32))) << 32;
    };
    const auto item_of = [&](int it) {
        const Item &s = sm.item[it & 7];
        return Item{uniform64(s.at), uniform64(s.row), uniform(s.bytes), uniform(s.steps), uniform(s.top),
                    uniform(s.ch0), uniform(s.valid), uniform(s.full), uniform(s.last), uniform(s.there)};
    };
    const auto load = [&](int it, typename Op::Raw &to) {
        const Item item = item_of(it);
        op.load(to, item, Op::part(item, step, slot, c0), w, step, c0);
    };
    typename Op::Terms terms[2];
    const auto form = [&](int it, const typename Op::Raw &held, typename Op::Terms &t) {
        const Item item = item_of(it);
        if (!item.there) return;
        const Part pt = Op::part(item, step, slot, c0);
        float2 pair[V];
        // log a is above the series' limit for every r where the rate is
        bool near = true;
#pragma unroll
        for (int v = 0; v < V; ++v) near = near && held.rate[v] >= -kSeriesLimit;
        if (item.full && __all(near)) op.template terms<true>(t, held, pt, pair);
        else op.template terms<false>(t, held, pt, pair);
#pragma unroll
        for (int v = 0; v < V; ++v) sm.slot[it & 1][slot][c0 + v] = pair[v];
    };
    // false when there is no item `it`
    const auto pass = [&](int it, const typename Op::Terms &now, typename Op::Raw &held, typename Op::Terms &after) {
        const Item item = item_of(it);
        if (!item.there) return false;
        form(it + 1, held, after);
        load(it + 3, held);
        __syncthreads();
        const Part pt = Op::part(item, step, slot, c0);
        float h[V], sum[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = sm.enter[it & 1][slot][c0 + v];
            sum[v] = 0.0f;
        }
        op.finish(now, item, pt, step, slot, h, sum);
        if (SUM) {
#pragma unroll
            for (int v = 0; v < V; ++v) sm.sum[it & 1][slot][c0 + v] = sum[v];
        }
        return true;
    };
    __syncthreads();
    load(0, raw[0]);
    load(1, raw[1]);
    form(0, raw[0], terms[0]);
    load(2, raw[0]);
    __syncthreads();
    for (int it = 0;; it += 2) {
        if (!pass(it, terms[0], raw[1], terms[1])) break;
        if (!pass(it + 1, terms[1], raw[0], terms[0])) break;
    }
    if (SUM) __syncthreads();
}

// dlam = sum of the parts, times sigmoid(lam) / softplus(lam).  The ratio is 1 -
// e^lam / 2 + ... as lam falls: 1 in float32 below -17 (further down both its parts
// leave float32's range).  32 channels and 16 slices of the parts a workgroup.
constexpr int kSlices = 16;
__global__ __launch_bounds__(32 * kSlices) void dlam_kernel(const float *__restrict__ part,
                                                            const float *__restrict__ lam,
                                                            float *__restrict__ dlam, int64_t parts, int64_t dim) {
    __shared__ float sh[kSlices][32];
    const int c = threadIdx.x % 32, slice = threadIdx.x / 32;
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + c;
    float s = 0.0f;
    if (d < dim)
        for (int64_t k = slice; k < parts; k += kSlices) s += part[k * dim + d];
    sh[slice][c] = s;
    __syncthreads();
    if (slice == 0 && d < dim) {
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < kSlices; ++k) s += sh[k][c];
        const float x = lam[d];
        dlam[d] = x > -17.0f ? s / (1.0f + expf(-x)) / softplus_libm(x) : s;
    }
}

// In front of the segments: clears the marks and forms the channels' rates.
__global__ __launch_bounds__(256) void prepare_kernel(uint64_t *marks, int64_t n, const float *__restrict__ lam,
                                                      float scale, float *__restrict__ rates, int64_t dim) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < max(n, dim); i += stride) {
        if (i < n) marks[i] = 0u;
        if (i < dim) rates[i] = -scale * softplus_libm(lam[i]);
    }
}

// Steps a lane holds: as many as the registers of two segments' terms and two
// segments' loads allow at three waves a SIMD (168 registers).
template <typename T, int V> struct Steps;
template <> struct Steps<uint16_t, 2> { static constexpr int fwd = 8, bwd = 4; };
template <> struct Steps<uint16_t, 1> { static constexpr int fwd = 10, bwd = 6; };
template <> struct Steps<float, 1> { static constexpr int fwd = 10, bwd = 6; };

// Groups of one segment that a ticket hands out.  The tickets' atomic additions
// to one address take 11.6 ns each across the chip, in turn: one a segment and
// group (5920 for 2 x 4096 steps of 5120 channels) took longer than the walk.
constexpr int kChunk = 4;

struct Plan {
    int64_t groups_per_batch, groups, nseg, parts;
    bool pairs;                          // two channels a lane
    size_t at_pairs[3], at_states, at_ticket, at_rates, at_part, bytes;
    int64_t marks;                       // 8-byte values to clear: pairs, states, ticket
};

int64_t segment_steps(bool pairs, bool f32, bool bwd) {
    if (f32) return bwd ? Bwd<float, 1, Steps<float, 1>::bwd>::kSteps : Fwd<float, 1, Steps<float, 1>::fwd>::kSteps;
    if (pairs)
        return bwd ? Bwd<uint16_t, 2, Steps<uint16_t, 2>::bwd>::kSteps : Fwd<uint16_t, 2, Steps<uint16_t, 2>::fwd>::kSteps;
    return bwd ? Bwd<uint16_t, 1, Steps<uint16_t, 1>::bwd>::kSteps : Fwd<uint16_t, 1, Steps<uint16_t, 1>::fwd>::kSteps;
}

// Two bfloat16 channels a lane move in one load where every row starts on an
// even element (the loads may be misaligned).
bool in_pairs(const RecurrenceArgs &a) { return a.io == IO_BF16 && a.dim % 2 == 0; }

Plan make_plan(const RecurrenceArgs &a, bool bwd) {
    Plan p{};
    p.pairs = in_pairs(a);
    const int64_t steps = segment_steps(p.pairs, a.io == IO_F32, bwd);
    p.groups_per_batch = (a.dim + kChannels - 1) / kChannels;
    p.groups = a.batch * p.groups_per_batch;
    p.nseg = (a.L + steps - 1) / steps;
    if (!bwd && a.L <= kRowSteps) return p;
    if (p.nseg > 1) {
        const int64_t per = p.groups * kChannels;
        const auto add = [&](int64_t n) {
            const size_t at = static_cast<size_t>(p.marks) * 8;
            p.marks += (p.nseg + n - 1) / n * per;
            return at;
        };
        p.at_pairs[0] = add(1);
        p.at_pairs[1] = add(kRun);
        p.at_pairs[2] = add(kBlock);
        p.at_states = add(kSpan);
        p.at_ticket = static_cast<size_t>(p.marks++) * 8;
    }
    const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    p.at_rates = up(static_cast<size_t>(p.marks) * 8);
    p.bytes = up(p.at_rates + static_cast<size_t>(a.dim) * 4);
    if (bwd) {
        p.parts = p.nseg * a.batch;
        p.at_part = p.bytes;
        p.bytes += static_cast<size_t>(p.parts) * a.dim * 4;
    }
    return p;
}

template <typename Op, typename T, int V, bool SUM>
hipError_t segments(const RecurrenceArgs &a, const Plan &p, unsigned char *base, const Op &op, const States &st,
                    hipStream_t stream) {
    Exchange ex{};
    ex.nseg = static_cast<int>(p.nseg);
    ex.groups = static_cast<int>(p.groups);
    ex.chunk = static_cast<int>(p.nseg == 1 || p.groups < kChunk ? 1 : kChunk);
    ex.chunks = (ex.groups + ex.chunk - 1) / ex.chunk;
    for (int l = 0; l < 3; ++l) ex.pairs[l] = reinterpret_cast<uint64_t *>(base + p.at_pairs[l]);
    ex.states = reinterpret_cast<uint64_t *>(base + p.at_states);
    ex.ticket = reinterpret_cast<uint32_t *>(base + p.at_ticket);
    float *rates = reinterpret_cast<float *>(base + p.at_rates);
    const int64_t most = p.marks > a.dim ? p.marks : a.dim, blocks = (most + 1023) / 1024;
    hipLaunchKernelGGL(prepare_kernel, dim3(static_cast<uint32_t>(blocks < 2048 ? blocks : 2048)), dim3(256), 0, stream,
                       ex.pairs[0], p.marks, a.lam, a.scale, rates, a.dim);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t items = p.nseg * p.groups;
    constexpr int64_t kResident = 256 * 4 * Op::kWavesPerSimd / (kComputeWaves + 1);
    const Walk w{rates, a.L, a.batch * a.L * a.dim, a.batch * a.dim, static_cast<int>(a.dim),
                 static_cast<int>(p.groups_per_batch), static_cast<int>(items), static_cast<int>(p.nseg)};
    // as many workgroups as stay resident, one a compute unit
    hipLaunchKernelGGL((segment_kernel<Op, T, V, SUM>), dim3(static_cast<uint32_t>(items < kResident ? items : kResident)),
                       dim3(kThreads), 0, stream, op, st, w, ex);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t fwd(const RecurrenceArgs &a, const Plan &p, unsigned char *base, hipStream_t stream) {
    typedef Fwd<T, V, Steps<T, V>::fwd> Op;
    const Op op{static_cast<const T *>(a.x), static_cast<const T *>(a.r), static_cast<const T *>(a.i),
                static_cast<T *>(a.y)};
    return segments<Op, T, V, false>(a, p, base, op, States{a.h0, a.h_last, nullptr}, stream);
}

template <typename T>
hipError_t row_fwd(const RecurrenceArgs &a, hipStream_t stream) {
    const int64_t rows = a.batch * a.dim;
    hipLaunchKernelGGL(row_fwd_kernel<T>, dim3(static_cast<uint32_t>((rows + kRowThreads - 1) / kRowThreads)),
                       dim3(kRowThreads), 0, stream, static_cast<const T *>(a.x), static_cast<const T *>(a.r),
                       static_cast<const T *>(a.i), a.lam, a.scale, a.h0, static_cast<T *>(a.y), a.h_last, rows,
                       static_cast<int>(a.L), a.dim);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t bwd(const RecurrenceArgs &a, const Plan &p, unsigned char *base, hipStream_t stream) {
    float *part = reinterpret_cast<float *>(base + p.at_part);
    typedef Bwd<T, V, Steps<T, V>::bwd> Op;
    const Op op{static_cast<const T *>(a.x), static_cast<const T *>(a.r), static_cast<const T *>(a.i),
                static_cast<const T *>(a.y), static_cast<const T *>(a.dy), static_cast<T *>(a.dx),
                static_cast<T *>(a.dr), static_cast<T *>(a.di), a.h0};
    hipError_t e = segments<Op, T, V, true>(a, p, base, op, States{a.dh_last, a.dh0, part}, stream);
    if (e == hipSuccess && a.dlam) {
        hipLaunchKernelGGL(dlam_kernel, dim3(static_cast<uint32_t>((a.dim + 31) / 32)), dim3(32 * kSlices), 0,
                           stream, part, a.lam, a.dlam, p.parts, a.dim);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch(const RecurrenceArgs &a, bool backward, void *workspace, hipStream_t stream) {
    if (!backward && a.L <= kRowSteps) return a.io == IO_F32 ? row_fwd<float>(a, stream) : row_fwd<uint16_t>(a, stream);
    const Plan p = make_plan(a, backward);
    void *mem = workspace;
    hipError_t e = hipSuccess;
    if (!mem) e = scratch_alloc(&mem, p.bytes, stream);
    if (e != hipSuccess) return e;
    unsigned char *base = static_cast<unsigned char *>(mem);
    if (a.io == IO_F32) e = backward ? bwd<float, 1>(a, p, base, stream) : fwd<float, 1>(a, p, base, stream);
    else if (p.pairs) e = backward ? bwd<uint16_t, 2>(a, p, base, stream) : fwd<uint16_t, 2>(a, p, base, stream);
    else e = backward ? bwd<uint16_t, 1>(a, p, base, stream) : fwd<uint16_t, 1>(a, p, base, stream);
    if (!workspace) {
        const hipError_t f = scratch_free(mem, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

}  // namespace

size_t gated_recurrence_workspace(const RecurrenceArgs &a, bool bwd) { return make_plan(a, bwd).bytes; }

bool gated_recurrence_supported(const RecurrenceArgs &a) {
    // byte offsets inside a segment (at most 177 rows) fit 31 bits; one lane a
    // row, 64 a workgroup; items fit 30 bits
    if (a.dim >= (int64_t(1) << 21) || a.batch * a.dim >= (int64_t(1) << 31)) return false;
    const int64_t steps = segment_steps(in_pairs(a), a.io == IO_F32, true);
    const int64_t groups = a.batch * ((a.dim + kChannels - 1) / kChannels);
    return (a.L + steps - 1) / steps < (int64_t(1) << 30) / groups;
}

hipError_t launch_gated_recurrence_fwd(const RecurrenceArgs &a, void *workspace, hipStream_t stream) {
    return launch(a, false, workspace, stream);
}

hipError_t launch_gated_recurrence_bwd(const RecurrenceArgs &a, void *workspace, hipStream_t stream) {
    return launch(a, true, workspace, stream);
}

hipError_t recurrence_status(uint32_t *bits, bool clear) {
    void *p = nullptr;
    hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(g_recurrence_status_bits));
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e == hipSuccess) e = hipMemcpy(bits, p, sizeof(uint32_t), hipMemcpyDeviceToHost);
    if (e == hipSuccess && clear) {
        const uint32_t zero = 0;
        e = hipMemcpy(p, &zero, sizeof(uint32_t), hipMemcpyHostToDevice);
    }
    return e;
}

}  // namespace mssm
