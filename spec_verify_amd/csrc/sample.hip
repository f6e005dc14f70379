// Sampling from a vocabulary head's logits (svq_sample) and acceptance of drafted
// tokens (svq_accept_drafts).
//
// A row's tokens are ordered by descending logit, ties by index. Every filter keeps
// a prefix of that order, and the draw is one position in it:
//
//   w(i) = exp((l_i - max) / T),  W(n) = w(0) + ... + w(n-1)
//   n1 = min(top_k, V)            n2 = min n : W(n) >= top_p W(n1)
//   n3 = #{i : w(i) >= min_p}     n  = min(n1, n2, n3), at least 1
//   position = min i : W(i+1) > u W(n)
//
// A token is a whole number, so W must not depend on rounding: fp64 sums. What makes that
// cheap is that bf16 logits take few different values. The kernels never sort: they count
// values (a histogram in LDS, exact and independent of the order of its atomics), which
// orders them, and weigh occurring values instead of tokens. The position then names a
// value and an ordinal among its equals, and a scan of a part of the row finds that
// occurrence.
//
// Values are binned by their bf16 pattern: magnitudes in [2^-16, 2^16) of either sign are
// 8192 bins, 8 consecutive ones per thread. A binade's patterns are equally far apart, so
// its weights are a geometric series: 32 ratios and 64 largest weights, one exponential
// each by one wave, give all 8192 in multiplications. A weight's relative error: at most 134
// multiplications round (2^-53 each); its ratio enters up to 127 times, and with it the
// exponential's own error (2^-52); the exponents' roundings add 2^-51 of the exponent, which is
// below 37 where a weight is above 1e-16 of the largest. All together less than 6e-14.
// Zero, up to kSideMax smaller magnitudes (a logit or two in a vocabulary) and one pattern
// below -2^16 (a mask value) are items of their own. Any other row is counted the long
// way: eight windows of 8192 patterns, one scan of the row per window and step.
//
// One workgroup takes a row from 52 rows on (and of short rows); of fewer, five to eight
// workgroups count a part of one row each and a second launch draws from their lists.
// V = 248320, us a call on the GPU alone, with top-k and top-p / nothing filtered: M = 1
// 22 / 28, 5 23 / 29, 64 32 / 31, 128 33 / 31, 256 43 / 42, 1024 117 / 115 (508 MB read at
// 4.4 TB/s; a large copy moves 4.8 TB/s). Few rows are bound by latency (two launches and
// their dependent steps), many by the counting: two LDS additions and ten vector
// instructions per two tokens keep the vector units 74% and LDS 53% busy. Masked rows (95% of
// -inf, -1e9, -1e4): 43 to 44 at M = 128, 138 to 143 at 1024; rows counted the long way 300 at
// M = 1, 480 at 128, 1400 at 1024.
#include <algorithm>
#include <cstddef>
#include <type_traits>

#include "svq_requests.h"

namespace svq {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr uint32_t kBinsHalf = 4096;         // 32 exponents x 128 mantissas of one sign
constexpr uint32_t kBins = 2 * kBinsHalf;    // of index sign << 12 | (magnitude - kMagLo)
constexpr uint32_t kSignWords = kBinsHalf + 64;  // of a table in LDS: a sign's bins, and a word for each lane's other tokens
constexpr uint32_t kTable = 2 * kSignWords;
constexpr int kOwn = kBins / kThreads;       // bins of a thread
constexpr uint32_t kMagLo = 111u << 7;       // pattern of 2^-16
constexpr uint32_t kSideMax = 55;            // smaller magnitudes; with zero and a thread's bins they are one per lane
constexpr int kWindows = 65536 / kBins;
constexpr int kLastPositive = kThreads / 2 - 1;  // its bins are followed by the side items
constexpr int kSideWave = kLastPositive / 64;    // whose last lane it is
static_assert(kLastPositive % 64 == 63 && kOwn + kSideMax + 1 <= 64 && kThreads % 64 == 0, "one wave owns the side items");

// ---- a row of logits -------------------------------------------------------------

// Elements [0, head) up to the first 16-byte boundary, nvec vectors of 8, then tail
// elements. Rows need no alignment beyond their elements'.
struct Row {
    const uint16_t *p;
    int head, nvec, tail;
};

__device__ __forceinline__ Row make_row(const uint16_t *p, int V) {
    Row r;
    r.p = p;
    const int h = (int)((16 - ((uintptr_t)p & 15)) & 15) >> 1;
    r.head = h < V ? h : V;
    r.nvec = (V - r.head) >> 3;
    r.tail = V - r.head - 8 * r.nvec;
    return r;
}

__device__ __forceinline__ uint4 row_vec(const Row &r, int v) { return *(const uint4 *)(r.p + r.head + (int64_t)v * 8); }

// Element i of the row's ends (head, then tail) for i < 16: its index, or -1.
__device__ __forceinline__ int row_end(const Row &r, int i, bool head, bool tail) {
    if (head && i < r.head) return i;
    if (tail && i >= 8 && i < 8 + r.tail) return r.head + 8 * r.nvec + i - 8;
    return -1;
}

// ---- patterns, order and weights ---------------------------------------------------

// Order-preserving 16-bit key of a bf16 pattern; -0 counts as +0.
__device__ __forceinline__ uint32_t key_of(uint32_t b) {
    if (b == 0x8000u) b = 0;
    return (b & 0x8000u) ? (~b & 0xFFFFu) : (b | 0x8000u);
}
__device__ __forceinline__ uint32_t bits_of(uint32_t key) { return (key & 0x8000u) ? (key & 0x7FFFu) : (~key & 0xFFFFu); }
// NaN and -inf are never drawn: finite values and +inf have keys in [0x80, 0xFF80].
__device__ __forceinline__ bool key_valid(uint32_t key) { return key - 0x80u <= 0xFF00u; }
__device__ __forceinline__ double value_of(uint32_t bits) { return (double)bits_f32(bits << 16); }
// Where a bin stands in a table.
__device__ __forceinline__ uint32_t bin_word(uint32_t bin) { return bin + (bin < kBinsHalf ? 0 : kSignWords - kBinsHalf); }
// Bin index <-> place in descending order (an involution).
__device__ __forceinline__ uint32_t bin_order(uint32_t bin) { return bin < kBinsHalf ? kBinsHalf - 1 - bin : bin; }

// The pattern of a bf16 value.
__device__ __forceinline__ uint32_t max_bits(double v) { return f32_bits((float)v) >> 16; }

struct Weight {
    double max, inv_t;
    __device__ __forceinline__ double exponent(uint32_t bits) const {
        const double v = value_of(bits);
        return v == max ? 0.0 : (v - max) * inv_t;
    }
    __device__ __forceinline__ double operator()(uint32_t bits) const {
        const double v = value_of(bits), d = v - max;
        // below an infinite maximum: 0, whatever T
        return v == max ? 1.0 : (d < -1.0e300 ? 0.0 : exp(d * inv_t));
    }
};

struct Params {
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
};
// One row's parameters. Read where a kernel begins: the loads then pass behind the
// reading of the logits.
struct RowParams {
    float u, top_p, min_p, temperature;
    uint32_t k;  // tokens that top_k leaves (0: no limit)
};
__device__ __forceinline__ RowParams row_params(const Params &p, int64_t m) {
    RowParams r{p.u[m], 1.f, 0.f, 1.f, 0};
    int k = 0;
    if (p.temperature) r.temperature = p.temperature[m];
    if (p.top_k) k = p.top_k[m];
    if (p.top_p) r.top_p = p.top_p[m];
    if (p.min_p) r.min_p = p.min_p[m];
    const bool greedy = !(r.temperature > 0.f);
    r.k = greedy ? 1u : (k > 0 ? (uint32_t)k : 0u);
    if (greedy) r.temperature = r.top_p = 1.f, r.min_p = 0.f;
    r.u = r.u >= 0.f ? fminf(r.u, 0x1.fffffep-1f) : 0.f;  // [0, 1), NaN as 0
    return r;
}

// ---- wave scans on the cross-lane data path -----------------------------------------------

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp0(uint32_t v) {  // lanes without a source get 0
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp0(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp0<CTRL, ROWS>((uint32_t)u) |
                                          (uint64_t)dpp0<CTRL, ROWS>((uint32_t)(u >> 32)) << 32);
}
// Inclusive sums over the 64 lanes: within rows of 16, then the row ends forward.
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {
    v += dpp0<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
    v += dpp0<0x112, 0xF>(v);
    v += dpp0<0x114, 0xF>(v);
    v += dpp0<0x118, 0xF>(v);
    v += dpp0<0x142, 0xA>(v);  // lane 15 of the row before, to rows 1 and 3
    v += dpp0<0x143, 0xC>(v);  // lane 31 to rows 2 and 3
    return v;
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)u, lane) |
                                          (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane) << 32);
}
// A value that every lane has, in scalar registers.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
__device__ __forceinline__ double uniform(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)uniform((uint32_t)u) | (uint64_t)uniform((uint32_t)(u >> 32)) << 32);
}
// The value one lane down, 0 in lane 0. All lanes take part in these scans.
template <typename T>
__device__ __forceinline__ T wave_down(T v) { return dpp0<0x138, 0xF>(v); }

// ---- histogram of a row or of a part of it -------------------------------------------

struct Hist {
    uint32_t bin[kTable];
    uint32_t side[kSideMax];
    uint32_t side_n, zeros, odd;  // odd: the row needs the long way
    uint32_t low_n, low_bits;     // tokens of the one pattern at or below -2^16
};

__device__ __forceinline__ void hist_clear(Hist &h) {
    for (int i = threadIdx.x; i < (int)kTable / 4; i += kThreads) ((uint4 *)h.bin)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) h.side_n = h.zeros = h.odd = h.low_n = h.low_bits = 0;
}

// A token count for one pattern at or below -2^16; a second such pattern makes the row odd.
__device__ __forceinline__ void hist_low(Hist &h, uint32_t bits, uint32_t n) {
    const uint32_t was = atomicCAS(&h.low_bits, 0u, bits);
    if (was != 0 && was != bits) h.odd = 1;
    atomicAdd(&h.low_n, n);
}

// Counts vectors [vb, ve) of a row into h.bin, or (quarters) a whole row's four quarters
// apart, 16 bits each, in h.bin and `bin2`. Two elements at a time, without a branch:
// subtracting kMagLo from both magnitudes leaves the bins' places, and a minimum sends every
// other token (-inf, NaN and what follows) to a word of the lane's own behind the bins, which
// nobody reads: ten vector instructions and two LDS additions for two elements. A step's
// four loads (of the four quarters, in that case) are issued a step ahead.
//
// One value can be most of a row (a mask's, or zeros), and LDS additions to one address go
// one after another. Such a value is the wave's `common` one: its tokens go to the lanes' own
// words too and are counted in registers, for seven more instructions a pair. A wave takes
// it up where a step's first token is the same in kManyEqual lanes, or tokens without a bin
// turn up in kManyOdd, and drops it after a step without it. What else has no bin is
// read again by a loop of its own, which keeps the code of the usual case short.
template <bool quarters>
__device__ __forceinline__ void hist_count(Hist &h, uint32_t *bin2, const Row &r, int vb, int ve, bool head, bool tail) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    constexpr uint32_t kNoBin = 0x70007000u, kPairOfInf = 0xFF80FF80u;
    constexpr int kManyEqual = 16, kManyOdd = 4;
    constexpr int kUnroll = 4, kStep = quarters ? kThreads : kUnroll * kThreads;
    const int apart = quarters ? (ve - vb + 3) / 4 : kThreads;  // from one of a step's vectors to the next
    const int end = quarters ? vb + apart : ve;                 // of the first one
    const int lane = threadIdx.x & 63;
    const uint16_t own = (uint16_t)(kBinsHalf + lane);
    const u16x2 other = {own, own};
    bool has_common = false;  // these two are the same in the whole wave
    uint32_t common = 0;
    uint32_t n_lo = 0, n_hi = 0;  // the lane's common tokens, as the two tables take them
    auto table = [&](int i) { return quarters && (i & 2) ? bin2 : h.bin; };
    auto unit = [](int i) { return quarters && (i & 1) ? 0x10000u : 1u; };
    // a token that is no pair's: of the row's ends (any), or without a bin (`odd`)
    auto single = [&](uint32_t b, int i, bool odd) {
        const uint32_t mag = b & 0x7FFFu, q = mag - kMagLo;
        if (q < kBinsHalf) {
            if (!odd) atomicAdd(&table(i)[(b >> 15) * kSignWords + q], unit(i));
        } else if (mag == 0) {
            atomicAdd(&h.zeros, 1u);
        } else if (mag < kMagLo) {
            const uint32_t at = atomicAdd(&h.side_n, 1u);
            if (at < kSideMax) h.side[at] = b;
        } else if (b > 0x8000u && b < 0xFF80u) {
            hist_low(h, b, 1);
        } else if (b <= 0x7F80u) {
            h.odd = 1;
        }
    };
    // whether a value can be the common one: one that has a bin, zero, below -2^16, -inf or NaN
    auto countable = [](uint32_t b) { return (b & 0x7FFFu) == 0 || ((b & 0x7FFFu) >= kMagLo && b - 0x4780u > 0x3800u); };
    // a pair's places in a table, in bytes
    auto places = [&](u16x2 index, u16x2 t) -> uint32_t {
        return __builtin_bit_cast(uint32_t, (u16x2)((t >> 15) * (uint16_t)(4 * kSignWords) + (index << 2)));
    };
    auto add = [&](uint32_t at, int i) {
        char *base = (char *)table(i);
        atomicAdd((uint32_t *)(base + (at & 0xFFFFu)), unit(i));
        atomicAdd((uint32_t *)(base + (at >> 16)), unit(i));
    };
    const u16x2 lo = {(uint16_t)kMagLo, (uint16_t)kMagLo}, magnitude = {0x7FFF, 0x7FFF};
    // counts a pair; the bits that say that one of it has no bin
    auto pair = [&](uint32_t w, int i) -> uint32_t {
        const u16x2 t = __builtin_bit_cast(u16x2, w) - lo;
        add(places(__builtin_elementwise_min(t & magnitude, other), t), i);
        return __builtin_bit_cast(uint32_t, t) & kNoBin;
    };
    // of a pair's halves, all ones where it is the common value
    auto equal = [&](uint32_t w) -> u16x2 {
        const u16x2 one = {1, 1};
        return __builtin_elementwise_min(__builtin_bit_cast(u16x2, w ^ common), one) - one;
    };
    // `pair` where there is a common value: `n` counts it
    auto pair_common = [&](uint32_t w, int i, u16x2 &n) -> uint32_t {
        asm("" : "+v"(w));  // apart from `pair`, whose terms would be held across the branch between the two
        const u16x2 t = __builtin_bit_cast(u16x2, w) - lo, e = equal(w);
        add(places(__builtin_elementwise_max(__builtin_elementwise_min(t & magnitude, other), e & other), t), i);
        n -= e;
        return __builtin_bit_cast(uint32_t, t) & kNoBin & ~__builtin_bit_cast(uint32_t, e);
    };
    auto count_common = [&](u16x2 n, int i) {
        const uint32_t sum = __builtin_amdgcn_sad_u16(__builtin_bit_cast(uint32_t, n), 0, 0);
        (quarters && (i & 2) ? n_hi : n_lo) += sum * unit(i);
    };
    // the wave's common tokens into the tables
    auto flush = [&]() {
        const uint32_t at_lo = wave_scan(n_lo), at_hi = quarters ? wave_scan(n_hi) : 0;
        n_lo = n_hi = 0;
        has_common = false;
        if (lane != 63) return;
        const uint32_t b = common & 0xFFFFu, mag = b & 0x7FFFu;
        const uint32_t sum = quarters ? __builtin_amdgcn_sad_u16(at_lo, 0, __builtin_amdgcn_sad_u16(at_hi, 0, 0)) : at_lo;
        if (mag - kMagLo < kBinsHalf) {
            const uint32_t at = (b >> 15) * kSignWords + mag - kMagLo;
            atomicAdd(&h.bin[at], at_lo);
            if constexpr (quarters) atomicAdd(&bin2[at], at_hi);
        } else if (mag == 0) {
            atomicAdd(&h.zeros, sum);
        } else if (b > 0x8000u && b < 0xFF80u) {
            hist_low(h, b, sum);
        }
    };
    auto load = [&](uint4 (&q)[kUnroll], int v) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            q[i] = v < end && v + i * apart < ve ? row_vec(r, v + i * apart)
                                                 : make_uint4(kPairOfInf, kPairOfInf, kPairOfInf, kPairOfInf);
    };
    uint4 next[kUnroll];
    int v = vb + (int)threadIdx.x;
    load(next, v);
    // a wave's steps: nothing within waits for another wave
    for (int v0 = vb + 64 * wave_id(); v0 < end; v0 += kStep, v += kStep) {
        uint4 q[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) q[i] = next[i];
        if (v0 + kStep < end) load(next, v + kStep);
        if (!has_common) {
            const uint32_t b = q[0].x & 0xFFFFu, b0 = uniform(b);
            if (__popcll(__ballot(b == b0)) >= kManyEqual && countable(b0)) has_common = true, common = b0 << 16 | b0;
        }
        uint64_t lanes[kUnroll];  // with tokens that have no bin
        if (!has_common) {
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
                lanes[i] = __ballot((pair(q[i].x, i) | pair(q[i].y, i) | pair(q[i].z, i) | pair(q[i].w, i)) != 0);
        } else {
            const uint32_t was_lo = n_lo, was_hi = n_hi;
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                u16x2 n = {0, 0};
                lanes[i] = __ballot((pair_common(q[i].x, i, n) | pair_common(q[i].y, i, n) | pair_common(q[i].z, i, n) |
                                     pair_common(q[i].w, i, n)) != 0);
                count_common(n, i);
            }
            if (!__ballot(n_lo != was_lo || n_hi != was_hi)) flush();
        }
        if (!(lanes[0] | lanes[1] | lanes[2] | lanes[3])) continue;
        bool taken = false;  // the common value, here
#pragma unroll 1
        for (int i = 0; i < kUnroll; ++i) {
            const uint64_t some = i == 0 ? lanes[0] : i == 1 ? lanes[1] : i == 2 ? lanes[2] : lanes[3];
            const bool within = v < end && v + i * apart < ve;
            if (!(some & __ballot(within)) && !taken) continue;
            const uint4 x = within ? row_vec(r, v + i * apart) : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
            uint32_t w[4] = {x.x, x.y, x.z, x.w}, left = 0;
            auto look = [&]() {
                u16x2 n = {0, 0};
                left = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u16x2 e = has_common ? equal(w[j]) : n - n;
                    left |= __builtin_bit_cast(uint32_t, __builtin_bit_cast(u16x2, w[j]) - lo) & kNoBin & ~__builtin_bit_cast(uint32_t, e);
                    n -= e;
                }
                if (taken) count_common(n, i);
            };
            look();
            const uint64_t odd = __ballot(left != 0);
            if (!has_common && __popcll(odd) >= kManyOdd) {
                const int from = __builtin_ctzll(odd);
                uint32_t b = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t two = (uint32_t)__builtin_amdgcn_readlane((int)w[j >> 1], from);
                    const uint32_t of = j & 1 ? two >> 16 : two & 0xFFFFu;
                    if ((of & 0x7FFFu) - kMagLo >= kBinsHalf) b = of;
                }
                if (countable(b)) {
                    has_common = taken = true, common = b << 16 | b;
                    look();
                }
            }
            if (!left) continue;
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = w[0] & 0xFFFFu;
                if (!(has_common && b == (common & 0xFFFFu))) single(b, i, true);
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = __builtin_amdgcn_alignbit(k < 3 ? w[k + 1] : 0, w[k], 16);
            }
        }
    }
    if (has_common) flush();
    const int at = row_end(r, threadIdx.x, head, tail);
    if (at >= 0) single(r.p[at], at < r.head ? 0 : 3, false);
}

// ---- the draw ---------------------------------------------------------------------------

struct Found {
    double mass;             // W
    uint32_t pos, bits, ord; // tokens counted; of a draw the value and which of its occurrences
};

struct Draw {
    Hist h;
    uint32_t item_bits[kSideMax + 1], item_count[kSideMax + 1];  // side items in order
    double ratio[32], anchor[64], inv_t;  // of binades
    double item_weight[kSideMax + 1], low_weight;
    double wsum[kWaves], whead[kWaves], win_mass[kWindows + 1], win_first[kWindows];
    uint32_t csum[kWaves], win_count[kWindows + 1];
    uint32_t first;
    uint32_t count[kWaves];  // locate's
    int at;
    Found found[4];          // one for each seek: no wave waits for the others to have read the last
};

// A row's quarters: the second of two tables, where a kernel has one.
struct DrawQuarters : Draw {
    uint32_t bin2[kTable];  // the first and second quarter are in bin, the others here
};
__device__ __forceinline__ uint32_t *second_table(Draw &sh) { return static_cast<DrawQuarters &>(sh).bin2; }

struct Drawn {
    uint32_t bits, ordinal;
    float logprob;
    bool any, counted;  // anything to draw from; by the histogram, not the long way
};

enum Seek { kMass, kTopP, kMinP, kDraw };

// How a row is counted: whole rows in h.bin; their quarters apart, 16 bits each, in h.bin
// and a table behind it; or window by window from the row itself.
enum Way { kWhole, kQuarters, kLong };

// A thread's bins in order, descending: patterns bits0, bits0 + dir, ..., each weight
// `ratio` times the one before.
struct Own {
    uint32_t bits0;
    int dir;
    double ratio;
};

__device__ __forceinline__ double inverse_t(const RowParams &par) { return uniform(1.0 / (double)par.temperature); }

// Exponentials of a counted row. fp64 is slow in all sixteen waves at once (an exponential
// in each took 1.6 us), so one wave takes them for all: a binade's patterns are 2^(e-7)
// apart, whatever the sign, so its ratio is one of 32; and a binade's largest value (or
// the row's, if that is in it) is its anchor, from which its weights are powers of the
// ratio. `draw_ratios` needs the temperature alone and runs beside the counting.
__device__ __forceinline__ void draw_ratios(Draw &sh, const RowParams &par) {
    if (wave_id() != 0) return;
    const int lane = threadIdx.x & 63;
    const double inv_t = inverse_t(par);
    // lane e: patterns kMagLo + 128 e ...: the step of that binade
    const uint32_t bits = kMagLo + 128 * (lane & 31);
    const double r = exp((value_of(bits) - value_of(bits + 1)) * inv_t);
    if (lane < 32) sh.ratio[lane] = r;
    if (lane == 0) sh.inv_t = inv_t;
}
__device__ __forceinline__ void draw_anchors(Draw &sh, const Weight &wt) {
    if (wave_id() != 0) return;
    // lanes 0..31: positive binades, whose largest pattern is the last; 32..63: negative ones
    const int lane = threadIdx.x & 63;
    const uint32_t bits = lane < 32 ? kMagLo + 128 * lane + 127 : 0x8000u | (kMagLo + 128 * (lane - 32));
    sh.anchor[lane] = exp((fmin(value_of(bits), wt.max) - wt.max) * wt.inv_t);
}

// Set by one thread per word before the barrier that precedes draw_way.
__device__ __forceinline__ void draw_clear(Draw &sh) {
    const int t = threadIdx.x;
    if (t == 4) sh.first = ~0u;
    if (t == 5) sh.win_count[0] = 0;
    if (t == 6) sh.win_mass[0] = 0.0;
}

// Draws a token's value and its ordinal. Used by whole workgroups, behind draw_clear and
// (counted rows) draw_ratios. max_key: the key of the row's largest value where it is known
// and its draw_anchors done (0: not).
template <Way way>
__device__ __forceinline__ Drawn draw_way(Draw &sh, const Row &row, const RowParams &par, uint32_t max_key) {
    Hist &h = sh.h;
    const int t = threadIdx.x, lane = t & 63, wave = wave_id();
    constexpr bool longway = way == kLong;
    constexpr int windows = longway ? kWindows : 1;
    Drawn out{0, 0, -__builtin_inff(), false, !longway};
    Weight wt;
    wt.max = max_key ? value_of(bits_of(max_key)) : 0.0;
    wt.inv_t = longway ? inverse_t(par) : uniform(sh.inv_t);
    Own own;
    own.dir = t <= kLastPositive ? -1 : 1;
    own.bits0 = t <= kLastPositive ? kMagLo + kBinsHalf - 1 - kOwn * t : 0x8000u | (kMagLo + kOwn * (t - kLastPositive - 1));
    own.ratio = 0.0;

    // Side items in order, by the wave that owns them: a value's place is the number of
    // larger entries and its first entry stands there for all equal ones (the places of the
    // others stay empty); zero stands between the signs. The low pattern comes after every
    // bin, the last thread's.
    const int side_n = longway ? 0 : (int)h.side_n, zeros = longway ? 0 : (int)h.zeros;
    const int sides = side_n + (zeros ? 1 : 0);
    const uint32_t low_n = !longway && t == kThreads - 1 ? h.low_n : 0;
    if (wave == kSideWave && lane <= (int)kSideMax) {
        sh.item_count[lane] = 0;
        if (lane < sides) {
            const uint32_t mine = lane < side_n ? h.side[lane] : 0, key = key_of(mine);
            uint32_t place = 0, equal = 0;
            bool lead = true;
            for (int j = 0; j < side_n; ++j) {
                const uint32_t o = key_of(h.side[j]);
                place += o > key;
                equal += o == key;
                lead = lead && !(o == key && j < lane);
            }
            if (lane < side_n && zeros) place += 0x8000u > key;
            if (lead) {
                sh.item_bits[place] = mine;
                sh.item_count[place] = lane < side_n ? equal : zeros;
            }
        }
    }

    uint32_t c = 0, ec = 0;
    int f = kOwn;                        // the thread's first occurring bin
    double wf = 0.0, w = 0.0, ew = 0.0;  // that one's weight; W of the thread and before it
    double head = 0.0;                   // the weight of its first value, bins or items
    uint32_t total = 0, sc = 0, wave_c = 0;  // sc, sw: in lane v, tokens and W up to wave v's end
    double wtotal = 0.0, sw = 0.0, wave_w = 0.0, wave_head = 0.0;  // wave_*: and before it
    int current = -1;

    auto bin_at = [&](int thread, int j) -> uint32_t {  // a thread's j-th bin
        const int at = longway ? kOwn * thread + j : (int)bin_word(bin_order(kOwn * thread + j));
        uint32_t n = h.bin[at];
        if constexpr (way == kQuarters) {
            const uint32_t n2 = second_table(sh)[at];
            n = __builtin_amdgcn_sad_u16(n, 0, __builtin_amdgcn_sad_u16(n2, 0, 0));  // the four halves
        }
        return n;
    };

    // The thread's bins, in 16-byte reads (single words, eight apart from lane to lane, meet
    // in the banks: 1 us more).
    auto counts = [&](uint32_t (&n)[kOwn]) {
        static_assert(kOwn == 8, "two vectors");
        const bool flip = !longway && wave <= kSideWave;  // the positive bins stand ascending
        const int first = flip ? (int)kBinsHalf - kOwn * (t + 1) : (longway ? kOwn * t : (int)bin_word(kOwn * t));
        const uint4 *p = (const uint4 *)&h.bin[first];
        uint4 a = p[0], b = p[1];
        if constexpr (way == kQuarters) {
            const uint4 *p2 = (const uint4 *)&second_table(sh)[first];
            const uint4 a2 = p2[0], b2 = p2[1];
            auto sum = [](uint32_t u, uint32_t v) {  // of the four 16-bit halves
                return __builtin_amdgcn_sad_u16(u, 0, __builtin_amdgcn_sad_u16(v, 0, 0));
            };
            a = make_uint4(sum(a.x, a2.x), sum(a.y, a2.y), sum(a.z, a2.z), sum(a.w, a2.w));
            b = make_uint4(sum(b.x, b2.x), sum(b.y, b2.y), sum(b.z, b2.z), sum(b.w, b2.w));
        }
        const uint32_t x[kOwn] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < kOwn; ++j) n[j] = flip ? x[kOwn - 1 - j] : x[j];
    };

    auto analyse = [&](int win) {
        // read before the barriers below, behind which it is set
        const bool find_max = !max_key && (current < 0 || sh.first == ~0u);
        if (longway) {  // count this window's patterns
            __syncthreads();
            for (int i = t; i < (int)kBins / 4; i += kThreads) ((uint4 *)h.bin)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
            auto single = [&](uint32_t b) {
                const uint32_t key = key_of(b), place = 65535u - key - (uint32_t)win * kBins;
                if (key_valid(key) && place < kBins) atomicAdd(&h.bin[place], 1u);
            };
#pragma unroll 1
            for (int v = t; v < row.nvec; v += kThreads) {
                const uint4 q = row_vec(row, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    single((&q.x)[i] & 0xFFFFu);
                    single((&q.x)[i] >> 16);
                }
            }
            const int at = row_end(row, t, true, true);
            if (at >= 0) single(row.p[at]);
            __syncthreads();
            const uint32_t key0 = 65535u - (uint32_t)win * kBins - kOwn * t;
            own.dir = key0 & 0x8000u ? -1 : 1;
            own.bits0 = bits_of(key0);
            own.ratio = exp((value_of(own.bits0 + own.dir) - value_of(own.bits0)) * wt.inv_t);
        }
        uint32_t cnt[kOwn];
        counts(cnt);
        c = 0;
        f = kOwn;
#pragma unroll
        for (int j = kOwn - 1; j >= 0; --j) {
            c += cnt[j];
            if (cnt[j]) f = j;
        }
        if (find_max) {  // the largest value, once: its key's place from the top
            uint32_t place = ~0u;
            if (f < kOwn) place = 65535u - key_of(own.bits0 + own.dir * f);
            else if (t == kLastPositive && sides) place = 65535u - key_of(sh.item_bits[0]);
            else if (low_n) place = 65535u - key_of(h.low_bits);
            const uint64_t mask = __ballot(place != ~0u);  // places ascend with the lane
            if (mask && lane == __builtin_ctzll(mask)) atomicMin(&sh.first, place);
            __syncthreads();
            const uint32_t first = uniform(sh.first);
            if (first != ~0u) wt.max = uniform(value_of(bits_of(65535u - first)));
            if (!longway) {
                draw_anchors(sh, wt);
                __syncthreads();
            }
        }
        w = 0.0;
        if (f < kOwn) {
            const uint32_t bits = own.bits0 + own.dir * f;
            if (longway) {
                wf = wt(bits);
            } else {
                // steps down from the anchor: the binade's largest value, or the row's
                const uint32_t binade = ((bits & 0x7FFFu) - kMagLo) >> 7, sign = bits >> 15;
                const double largest = value_of(sign ? bits & 0xFF80u : bits | 0x7Fu);
                const uint32_t top = largest <= wt.max ? (sign ? bits & 0xFF80u : bits | 0x7Fu) : max_bits(wt.max);
                const uint32_t steps = sign ? bits - top : top - bits;
                double p = own.ratio = sh.ratio[binade];
                wf = sh.anchor[32 * sign + binade];
#pragma unroll
                for (int b = 0; b < 7; ++b) {
                    if (steps >> b & 1) wf *= p;
                    p *= p;
                }
            }
            head = wf;
            double x = wf;
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                if (cnt[j]) w += cnt[j] * x;
                if (j >= f) x *= own.ratio;
            }
        }
        if (!longway && wave == kSideWave && sides) {  // the items' counts and weights to its last lane
            uint32_t n = 0;
            double v = 0.0;
            if (lane < sides) {
                n = sh.item_count[lane];
                if (n) sh.item_weight[lane] = v = wt(sh.item_bits[lane]);
            }
            const uint32_t items = wave_scan(n);
            const double weight = wave_scan(n * v);
            if (lane == 63) {
                if (c == 0) head = sh.item_weight[0];
                c += items;
                w += weight;
            }
        }
        if (low_n) {
            const double v = wt(h.low_bits);
            sh.low_weight = v;
            if (c == 0) head = v;
            c += low_n;
            w += low_n * v;
        }
        // exclusive prefix over the threads, after the windows before this one
        const uint32_t ic = wave_scan(c);
        const double iw = wave_scan(w);
        if (lane == 63) {
            sh.csum[wave] = ic;
            sh.wsum[wave] = iw;
        }
        const uint64_t some = __ballot(c != 0);
        if (some && lane == __builtin_ctzll(some)) sh.whead[wave] = head;
        const uint32_t xc = wave_down(ic);
        const double xw = wave_down(iw);
        __syncthreads();
        const uint32_t bc = longway ? sh.win_count[win] : 0;
        const double bw = longway ? sh.win_mass[win] : 0.0;
        sc = bc + wave_scan(lane < kWaves ? sh.csum[lane] : 0u);
        sw = bw + wave_scan(lane < kWaves ? sh.wsum[lane] : 0.0);
        wave_head = lane < kWaves ? sh.whead[lane] : 0.0;
        wave_c = wave_down(sc);  // (not within the choice: a lane that is switched off gives nothing)
        wave_w = wave_down(sw);
        if (lane == 0) {
            wave_c = bc;
            wave_w = bw;
        }
        ec = __builtin_amdgcn_readlane((int)wave_c, wave) + xc;
        ew = lane_value(wave_w, wave) + xw;
        total = __builtin_amdgcn_readlane((int)sc, kWaves - 1);
        wtotal = lane_value(sw, kWaves - 1);
        if (longway) {
            if (t == 0) {
                sh.win_count[win + 1] = total;
                sh.win_mass[win + 1] = wtotal;
            }
            if (c && ec == bc) sh.win_first[win] = head;
            __syncthreads();
        }
        current = win;
    };

    for (int win = 0; win < windows; ++win) analyse(win);
    if (total == 0) return out;  // nothing to draw from
    out.any = true;
    uint32_t n = total;
    double mass = wtotal;

    // Finds the wave, in it the thread, and in that the value that crosses n tokens or mass x.
    auto seek = [&](int slot, Seek mode, double x) {
        if (longway) {
            int win = 0;
            for (int i = 0; i < kWindows; ++i) {
                const uint32_t b = sh.win_count[i];
                if (sh.win_count[i + 1] == b) continue;
                const double bm = sh.win_mass[i];
                const bool in = mode == kMass ? b < n
                                : mode == kTopP ? b == 0 || bm < x
                                : mode == kMinP ? b == 0 || sh.win_first[i] >= x
                                                : b < n && (b == 0 || bm <= x);
                if (in) win = i;
            }
            if (win != current) analyse(win);
        }
        // whether it is not before this stretch of tokens: holds for a leading part of them
        auto within = [&](uint32_t before_n, double before_w, double first) {
            return before_n == 0 || (mode == kMass ? before_n < n
                                     : mode == kTopP ? before_w < x
                                     : mode == kMinP ? first >= x
                                                     : before_n < n && before_w <= x);
        };
        const uint64_t waves = __ballot(lane < kWaves && sc != wave_c && within(wave_c, wave_w, wave_head));
        if (waves && 63 - __builtin_clzll(waves) == wave) {  // every wave finds the same one
            const uint64_t mask = __ballot(c && within(ec, ew, head));
            const int ol = mask ? 63 - __builtin_clzll(mask) : 0, owner = wave * 64 + ol;
            // its wave looks at its values, one a lane: the bins, then the items behind them.
            // (What the owner has is read here, where every lane is on: within the choice below
            // the owner may be off, and what it holds may be stale.)
            const uint32_t first = __builtin_amdgcn_readlane((int)ec, ol);
            const double start = lane_value(ew, ol), r1 = lane_value(own.ratio, ol), w1 = lane_value(wf, ol);
            const int of = __builtin_amdgcn_readlane(f, ol);
            const uint32_t bits0 = (uint32_t)__builtin_amdgcn_readlane((int)own.bits0, ol);
            const int dir = __builtin_amdgcn_readlane(own.dir, ol);
            uint32_t k = 0, bits = 0;
            double v = 0.0;
            if (lane < kOwn) {
                k = bin_at(owner, lane);
                bits = bits0 + dir * lane;
                const int d = max(lane - of, 0);
                const double r2 = r1 * r1;
                v = w1 * (d & 1 ? r1 : 1.0) * (d & 2 ? r2 : 1.0) * (d & 4 ? r2 * r2 : 1.0);
            } else if (!longway) {
                const int i = lane - kOwn;
                if (owner == kLastPositive && i < sides) {
                    k = sh.item_count[i];
                    bits = sh.item_bits[i];
                    v = sh.item_weight[i];
                } else if (owner == kThreads - 1 && i == 0 && h.low_n) {
                    k = h.low_n;
                    bits = h.low_bits;
                    v = sh.low_weight;
                }
            }
            if (k == 0) v = 0.0;  // (an unoccurring pattern's may be anything)
            const uint32_t pos = first + wave_down(wave_scan(k));
            k = pos < n ? min(k, n - pos) : 0;  // no more than n tokens
            const double before = start + wave_down(wave_scan(k * v)), end = before + k * v;
            // the value that crosses, or else the last one with weight
            const bool over = k && (mode == kMass ? pos + k >= n : mode == kTopP ? end >= x : mode == kMinP ? v < x : end > x);
            const uint64_t crossing = __ballot(over), weighty = __ballot(k && v > 0.0), any = __ballot(k != 0);
            const int at = crossing ? __builtin_ctzll(crossing)
                                    : (weighty ? 63 - __builtin_clzll(weighty) : __builtin_ctzll(any | 1ull << 63));
            const uint32_t ak = __builtin_amdgcn_readlane((int)k, at), apos = __builtin_amdgcn_readlane((int)pos, at);
            const double av = lane_value(v, at), ab = lane_value(before, at);
            uint32_t part = ak, ord = ak ? ak - 1 : 0;  // tokens of the value, or which of them
            if (mode == kMinP) {
                if (crossing) part = 0;
            } else if (mode == kTopP || mode == kDraw) {
                double y = av > 0.0 ? (x - ab) / av : (double)ak;
                y = fmin(fmax(y, 0.0), (double)ak);
                if (mode == kTopP) {  // tokens whose W before them is below x
                    part = (uint32_t)ceil(y);
                    while (part > 0 && ab + (part - 1) * av >= x) --part;
                    while (part < ak && ab + part * av < x) ++part;
                } else if (crossing) {
                    ord = min((uint32_t)y, ak - 1);
                    while (ord > 0 && ab + ord * av > x) --ord;
                    while (ord + 1 < ak && ab + (ord + 1) * av <= x) ++ord;
                }
            }
            if (lane == at) sh.found[slot] = Found{ab + part * av, apos + part, bits, ord};
        }
        __syncthreads();
    };

    // W(n1), n2, n3 (each with its W) where they limit, the draw
#pragma unroll 1
    for (int step = 0; step < 4; ++step) {
        Seek mode = kMass;
        double x = 0.0;
        if (step == 0) {
            if (!(par.k && par.k < n)) continue;
            n = par.k;
        } else if (step == 1) {
            if (!(par.top_p < 1.f)) continue;
            mode = kTopP;
            x = (double)par.top_p * mass;
        } else if (step == 2) {
            if (!(par.min_p > 0.f)) continue;
            mode = kMinP;
            x = (double)par.min_p;
        } else {
            mode = kDraw;
            x = (double)par.u * mass;
        }
        seek(step, mode, x);
        const uint32_t pos = uniform(sh.found[step].pos);
        if (mode == kMass) {
            mass = uniform(sh.found[step].mass);
        } else if (mode != kDraw && pos < n) {
            n = max(pos, 1u);
            mass = pos ? uniform(sh.found[step].mass) : 1.0;  // the first token's weight
        }
    }
    out.bits = uniform(sh.found[3].bits);
    out.ordinal = uniform(sh.found[3].ord);
    out.logprob = (float)(wt.exponent(out.bits) - log(mass));
    return out;
}

// Out of line: the kernels hardly ever call it.
__device__ __attribute__((noinline)) Drawn draw_long(Draw &sh, const Row &row, const RowParams &par) {
    return draw_way<kLong>(sh, row, par, 0);
}

// Index of the ordinal-th element equal to `bits` among vectors [vb, ve) (and head or
// tail), in index order, by the whole workgroup; every thread gets it (-1 if there are
// fewer, which a consistent histogram excludes).
__device__ __forceinline__ int locate(Draw &sh, const Row &r, int vb, int ve, bool head, bool tail, uint32_t bits, uint32_t ordinal) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    const bool zero = (bits & 0x7FFFu) == 0;  // both zeros are one value
    const uint32_t mask16 = zero ? 0x7FFFu : 0xFFFFu;
    auto same = [&](uint32_t b) { return ((b ^ bits) & mask16) == 0; };
    uint32_t left = ordinal;
    if (threadIdx.x == 0) sh.at = -1;
    __syncthreads();
    if (head) {  // every wave looks at these few elements itself
        const bool eq = lane < r.head && same(r.p[lane]);
        const uint64_t mask = __ballot(eq);
        const uint32_t n = __popcll(mask);
        if (left < n) {
            uint64_t mm = mask;
            for (uint32_t i = 0; i < left; ++i) mm &= mm - 1;
            return __ffsll((unsigned long long)mm) - 1;
        }
        left -= n;
    }
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    const uint32_t want2 = bits * 0x10001u, mask2 = mask16 * 0x10001u;
    auto differ = [&](uint32_t x) {  // per half: 0 if it is the value, else 1
        const u16x2 d = __builtin_bit_cast(u16x2, (x ^ want2) & mask2), one = {1, 1};
        return __builtin_elementwise_min(d, one);
    };
    auto misses = [&](const uint4 &q) -> uint32_t {  // elements that are not the value, 0..8
        const u16x2 d = differ(q.x) + differ(q.y) + differ(q.z) + differ(q.w);
        return (uint32_t)d.x + (uint32_t)d.y;
    };
    auto matches = [&](const uint4 &q) {  // one bit per element
        uint32_t n = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t x = (&q.x)[w];
            n |= (uint32_t)same(x & 0xFFFFu) << (2 * w) | (uint32_t)same(x >> 16) << (2 * w + 1);
        }
        return n;
    };
    constexpr int kIter = 8;                    // vectors of a lane per block of the row
    constexpr int kBlock = kThreads * kIter;    // vectors
    for (int b0 = vb; b0 < ve; b0 += kBlock) {
        const int w0 = b0 + wave * 64 * kIter;
        uint4 q[kIter];
        uint32_t eq[kIter], sum = 0;
#pragma unroll
        for (int i = 0; i < kIter; ++i) q[i] = row_vec(r, min(w0 + i * 64 + lane, ve - 1));
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            eq[i] = w0 + i * 64 + lane < ve ? 8 - misses(q[i]) : 0;
            sum += eq[i];
        }
        sum = __builtin_amdgcn_readlane(wave_scan(sum), 63);
        if (lane == 0) sh.count[wave] = sum;
        __syncthreads();
        const uint32_t scan = wave_scan(lane < kWaves ? sh.count[lane] : 0u);
        const uint32_t all = __builtin_amdgcn_readlane((int)scan, kWaves - 1);
        const uint32_t before = __builtin_amdgcn_readlane((int)scan, wave) - sum;
        if (left < all) {
            if (before <= left && left < before + sum) {  // in this wave's part
                uint32_t skip = left - before;
#pragma unroll
                for (int i = 0; i < kIter; ++i) {
                    const uint32_t inc = wave_scan(eq[i]), n = __builtin_amdgcn_readlane((int)inc, 63);
                    const uint32_t first = inc - eq[i];
                    if (first <= skip && skip < inc) {  // in this lane's vector
                        const int v = w0 + i * 64 + lane;
                        uint32_t in = matches(row_vec(r, v));
                        for (uint32_t k = skip - first; k; --k) in &= in - 1;
                        sh.at = r.head + v * 8 + __builtin_ctz(in);
                    }
                    if (skip < n) break;
                    skip -= n;
                }
            }
            __syncthreads();
            return sh.at;
        }
        left -= all;
        __syncthreads();
    }
    if (tail) {
        const int base = r.head + 8 * r.nvec;
        const bool eq = lane < r.tail && same(r.p[base + lane]);
        uint64_t mask = __ballot(eq);
        if (left < (uint32_t)__popcll(mask)) {
            for (uint32_t i = 0; i < left; ++i) mask &= mask - 1;
            return base + __ffsll((unsigned long long)mask) - 1;
        }
    }
    return -1;
}

// ---- kernels ------------------------------------------------------------------------------

// One workgroup per row: count, draw, find. M = 1024, V = 248320: 110 us (4.6 TB/s), of a
// workgroup's 53 us 35 are the counting and 5 the search. The row's quarters are counted apart, which
// tells where to look for the occurrence: reading half a row again, as a search from its
// beginning does on average, took a third of the time.
//
// With more rows than compute units two workgroups share one (64 registers), so that one's
// draw runs beside the other's reading. A call of the long way, never taken, would cost
// them its stack and spilled registers (M = 1024, V = 248320: a sixth more time), so
// rows that need it are marked and left to a launch of their own, whose workgroups
// otherwise end at once (4 us). With fewer rows the call is the cheaper one (M = 1: 13 us
// instead of 15).
constexpr int64_t kMaxQuarter = 65535 / 8 - 2;  // vectors: a quarter's tokens fit 16 bits
constexpr int kLongWay = -2;

template <Way way, bool mark>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(mark ? 8 : 4, 8))) void sample_row_kernel(
    const uint16_t *__restrict__ logits, int64_t ld, Params par, int32_t *__restrict__ tokens,
    float *__restrict__ logprobs, int V) {
    __shared__ __attribute__((aligned(16))) std::conditional_t<way == kQuarters, DrawQuarters, Draw> sh;
    const int64_t m = blockIdx.x;
    const Row row = make_row(logits + m * ld, V);
    const RowParams rp = row_params(par, m);
    const int quarter = (row.nvec + 3) / 4;
    hist_clear(sh.h);
    draw_clear(sh);
    if constexpr (way == kQuarters) {
        for (int i = threadIdx.x; i < (int)kTable / 4; i += kThreads) ((uint4 *)sh.bin2)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        hist_count<true>(sh.h, sh.bin2, row, 0, row.nvec, true, true);
    } else {
        __syncthreads();
        hist_count<false>(sh.h, nullptr, row, 0, row.nvec, true, true);
    }
    draw_ratios(sh, rp);
    __syncthreads();
    const bool longway = sh.h.odd || sh.h.side_n > kSideMax;
    if (mark && longway) {
        if (threadIdx.x == 0) tokens[m] = kLongWay;
        return;
    }
    const Drawn d = !mark && longway ? draw_long(sh, row, rp) : draw_way<way>(sh, row, rp, 0);
    int token = -1;
    if (d.any) {
        const uint32_t mag = (d.bits & 0x7FFFu) - kMagLo;
        int vb = 0, ve = row.nvec, q = -1;
        uint32_t left = d.ordinal;
        if constexpr (way == kQuarters)
            if (d.counted && mag < kBinsHalf) {
                const uint32_t at = (d.bits >> 15) * kSignWords + mag, u = sh.h.bin[at], v = sh.bin2[at];
                for (q = 0; q < 3; ++q) {
                    const uint32_t x = q & 2 ? v : u, n = q & 1 ? x >> 16 : x & 0xFFFFu;
                    if (left < n) break;
                    left -= n;
                }
                vb = min(q * quarter, row.nvec);
                ve = min((q + 1) * quarter, row.nvec);
            }
        token = locate(sh, row, vb, ve, q <= 0, q < 0 || q == 3, d.bits, left);
    }
    if (threadIdx.x == 0) {
        tokens[m] = token;
        if (logprobs) logprobs[m] = d.logprob;
    }
}

// The rows that sample_row_kernel marked.
__global__ __launch_bounds__(kThreads) void sample_long_kernel(const uint16_t *__restrict__ logits, int64_t ld, Params par,
                                                               int32_t *__restrict__ tokens, float *__restrict__ logprobs,
                                                               int64_t M, int V) {
    __shared__ __attribute__((aligned(16))) Draw sh;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const bool mine = tokens[m] == kLongWay;
        __syncthreads();  // every thread has read the mark, and the row before is done with
        if (!mine) continue;
        const Row row = make_row(logits + m * ld, V);
        const RowParams rp = row_params(par, m);
        draw_clear(sh);
        __syncthreads();
        const Drawn d = draw_way<kLong>(sh, row, rp, 0);
        int token = -1;
        if (d.any) token = locate(sh, row, 0, row.nvec, true, true, d.bits, d.ordinal);
        if (threadIdx.x == 0) {
            tokens[m] = token;
            if (logprobs) logprobs[m] = d.logprob;
        }
    }
}

// Few rows: a workgroup per part of a row counts it (8.2 us at M = 1, V = 248320, 8 parts:
// 0.7 clearing, 2.6 reading and adding, 2.7 for the list), and one per row draws from the
// lists (13.8 us: 2.5 reading them, 1.8 weighing, 1.2 a seek, 3.5 finding the token).
//
// Workspace of one (row, part): header, then the occurring bins in descending order
// (place in that order << 18 | count), then the smaller magnitudes.
constexpr uint32_t kHeader = 8;
constexpr uint32_t kPartWords = (kHeader + kBins + kSideMax + 31) / 32 * 32;  // whole lines of 128 bytes
static_assert(kHeader == 8 && kPartWords % 4 == 0, "a header is two 16-byte vectors at 16-byte addresses");
constexpr uint32_t kCountBits = 18;
constexpr uint32_t kCountMask = (1u << kCountBits) - 1;
constexpr int64_t kMaxPartVectors = ((1 << kCountBits) - 16) / 8;  // a part's tokens fit the count
constexpr int kMaxParts = kThreads;

__global__ __launch_bounds__(kThreads) void sample_count_kernel(const uint16_t *__restrict__ logits, int64_t ld, Params par,
                                                                uint32_t *__restrict__ parts, int V, int C, int vpp) {
    __shared__ __attribute__((aligned(16))) Hist h;
    __shared__ uint32_t wsum[kWaves][2], entries, largest;
    const int64_t m = blockIdx.x / C;
    const int part = blockIdx.x % C;
    const Row row = make_row(logits + m * ld, V);
    const uint32_t k = row_params(par, m).k;
    hist_clear(h);
    if (threadIdx.x == 0) entries = largest = 0;
    __syncthreads();
    const int vb = min(part * vpp, row.nvec), ve = min(vb + vpp, row.nvec);
    hist_count<false>(h, nullptr, row, vb, ve, part == 0, part == C - 1);
    __syncthreads();
    // occurring bins in descending order, but none behind which top_k tokens of this
    // part already stand; (bins << 18 | tokens) are scanned in one word
    const int t = threadIdx.x, lane = t & 63, wave = wave_id();
    const uint4 v0 = ((const uint4 *)h.bin)[kBinsHalf / 4 - 1 - t], v1 = ((const uint4 *)h.bin)[kSignWords / 4 + t];
    const uint32_t n[2][4] = {{v0.w, v0.z, v0.y, v0.x}, {v1.x, v1.y, v1.z, v1.w}};
    uint32_t own[2], inc[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        own[s] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) own[s] += n[s][j] + (n[s][j] ? 1u << kCountBits : 0);
        inc[s] = own[s];
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t o = __shfl_up(inc[s], d);
            if (lane >= d) inc[s] += o;
        }
    if (lane == 63) {
        wsum[wave][0] = inc[0];
        wsum[wave][1] = inc[1];
    }
    __syncthreads();
    uint32_t *dst = parts + ((int64_t)m * C + part) * kPartWords;
    const uint32_t middle = h.zeros + h.side_n;
    uint32_t run = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        uint32_t before = run;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            if (v == wave) before = run;
            run += wsum[v][s];
        }
        uint32_t at = before + inc[s] - own[s], last = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n[s][j]) {
                const uint32_t above = (at & kCountMask) + (s ? middle : 0), pos = at >> kCountBits;
                if (!k || above < k) {
                    const uint32_t place = s * kBinsHalf + 4 * t + j;
                    dst[kHeader + pos] = place << kCountBits | n[s][j];
                    last = pos + 1;
                    if (pos == 0) {
                        const uint32_t bin = bin_order(place);
                        atomicMax(&largest, key_of((bin / kBinsHalf << 15) | (kMagLo + bin % kBinsHalf)));
                    }
                }
                at += n[s][j] + (1u << kCountBits);
            }
        if (last) atomicMax(&entries, last);
    }
    if (t < (int)min(h.side_n, kSideMax)) {
        dst[kHeader + kBins + t] = h.side[t];
        atomicMax(&largest, key_of(h.side[t]));
    }
    if (t == 0 && h.zeros) atomicMax(&largest, 0x8000u);
    if (t == 0 && h.low_n) atomicMax(&largest, key_of(h.low_bits));
    __syncthreads();
    if (t == 0) {
        ((uint4 *)dst)[0] = make_uint4(entries, h.side_n, h.zeros, h.odd);
        ((uint4 *)dst)[1] = make_uint4(h.low_n, h.low_bits, largest, 0);
    }
}

__global__ __launch_bounds__(kThreads) void sample_select_kernel(const uint16_t *__restrict__ logits, int64_t ld, Params par,
                                                                 const uint32_t *__restrict__ parts,
                                                                 int32_t *__restrict__ tokens,
                                                                 float *__restrict__ logprobs, int V, int C, int vpp) {
    __shared__ __attribute__((aligned(16))) Draw sh;
    __shared__ uint32_t in_part[kMaxParts];
    const int64_t m = blockIdx.x;
    const int t = threadIdx.x, lane = t & 63, wave = wave_id();
    const Row row = make_row(logits + m * ld, V);
    const uint32_t *src = parts + (int64_t)m * C * kPartWords;
    const RowParams rp = row_params(par, m);
    Hist &h = sh.h;
    hist_clear(h);
    __syncthreads();
    auto add = [&](uint32_t e) { atomicAdd(&h.bin[bin_word(bin_order(e >> kCountBits))], e & kCountMask); };
    // A wave takes two parts at once (or, of few parts, several waves share one), and keeps
    // the first kAhead entries of a lane for the search below (all there are, as a rule,
    // where top_k limits them).
    constexpr int kAhead = 4, kTwo = 2;
    const int shared = C < kWaves ? kWaves / C : 1;  // waves on one part
    const int first = C < kWaves ? wave % C : wave, sub = C < kWaves ? wave / C : 0;
    const uint32_t lane0 = sub * 64 + lane, step = shared * 64;
    uint32_t kept[kTwo][kAhead], entries[kTwo] = {0, 0};
    uint32_t largest = 0;
    for (int c = lane; c < C; c += 64) largest = max(largest, src[(int64_t)c * kPartWords + 6]);
    for (int c0 = 0; c0 < C; c0 += kTwo * kWaves) {
        uint4 a[kTwo], b[kTwo];
#pragma unroll
        for (int j = 0; j < kTwo; ++j) {
            const int c = min(c0 + j * kWaves + first, C - 1);
            const uint32_t *p = src + (int64_t)c * kPartWords;
            a[j] = ((const uint4 *)p)[0];
            b[j] = ((const uint4 *)p)[1];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) kept[j][i] = p[kHeader + min(step * i + lane0, kBins - 1)];
        }
        if (c0 == 0) {  // beside the loads
            draw_ratios(sh, rp);
#pragma unroll
            for (int x = 1; x < 64; x <<= 1) largest = max(largest, (uint32_t)__shfl_xor((int)largest, x));
            largest = uniform(largest);
            if (largest) draw_anchors(sh, Weight{value_of(bits_of(largest)), uniform(sh.inv_t)});
        }
#pragma unroll
        for (int j = 0; j < kTwo; ++j) {
            const int c = c0 + j * kWaves + first;
            if (c >= C || sub >= shared) break;
            const uint32_t *p = src + (int64_t)c * kPartWords;
            entries[j] = a[j].x;
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (step * i + lane0 < entries[j]) add(kept[j][i]);
#pragma unroll 4
            for (uint32_t i = step * kAhead + lane0; i < entries[j]; i += step) add(p[kHeader + i]);
            if (sub) continue;
            const uint32_t side_n = a[j].y;
            uint32_t at = 0;
            if (lane == 0) {
                if (a[j].z) atomicAdd(&h.zeros, a[j].z);
                if (a[j].w) h.odd = 1;
                if (side_n) at = atomicAdd(&h.side_n, side_n);
                if (b[j].x) hist_low(h, b[j].y, b[j].x);
            }
            at = __builtin_amdgcn_readfirstlane(at);
            if (lane < min(side_n, kSideMax) && at + lane < kSideMax) h.side[at + lane] = p[kHeader + kBins + lane];
        }
    }
    for (int c = t; c < C; c += kThreads) in_part[c] = 0;
    draw_clear(sh);
    __syncthreads();
    const Drawn d = h.odd || h.side_n > kSideMax ? draw_long(sh, row, rp) : draw_way<kWhole>(sh, row, rp, largest);
    int token = -1;
    if (d.any) {
        const uint32_t q = (d.bits & 0x7FFFu) - kMagLo;
        int vb = 0, ve = row.nvec;
        bool head = true, tail = true;
        uint32_t left = d.ordinal;
        const uint32_t mag = d.bits & 0x7FFFu;
        const bool binned = q < kBinsHalf, zero = mag == 0, low = d.bits == h.low_bits && h.low_n;
        if (d.counted && (binned || zero || low)) {
            // the value's count in each part tells which part holds the occurrence: zero's and
            // the low value's in its header; a part's entries ascend by place: 64 samples,
            // then the stretch between two. (Smaller values and the long way have no counts
            // by part.)
            const uint32_t want = bin_order((d.bits >> 15) * kBinsHalf + q);
            for (int c = first, j = 0; c < C && sub < shared; c += kWaves, ++j) {
                uint32_t n = 0;
                const uint32_t count = C <= kTwo * kWaves ? (j ? entries[1] : entries[0]) : ~0u;
                if (!binned) {
                    if (sub == 0 && lane == 0) n = src[(int64_t)c * kPartWords + (zero ? 2 : 4)];
                } else if (count <= step * kAhead) {
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        const uint32_t e = j ? kept[1][i] : kept[0][i];
                        if (step * i + lane0 < count && (e >> kCountBits) == want) n = e & kCountMask;
                    }
                } else if (sub == 0) {
                    const uint32_t *p = src + (int64_t)c * kPartWords;
                    const uint32_t count = p[0], stride = (count + 63) / 64;
                    p += kHeader;
                    const uint32_t i0 = lane * stride;
                    const bool le = i0 < count && (p[i0] >> kCountBits) <= want;
                    const int hit = __popcll(__ballot(le));  // samples at or before it
                    if (hit)
                        for (uint32_t i = lane; i < stride; i += 64) {
                            const uint32_t at = (hit - 1) * stride + i;
                            const uint32_t e = at < count ? p[at] : ~0u;
                            if ((e >> kCountBits) == want) n = e & kCountMask;
                        }
                }
                if (n) in_part[c] = n;  // one lane at most
            }
            __syncthreads();
            int part = 0;
            for (int c0 = 0; c0 < C; c0 += 64) {
                const uint32_t inc = wave_scan(c0 + lane < C ? in_part[c0 + lane] : 0u);
                const uint64_t past = __ballot(inc > left);
                part = min(c0 + (past ? __builtin_ctzll(past) : 64), C - 1);
                const uint32_t before = __builtin_amdgcn_readlane((int)inc, (past ? __builtin_ctzll(past) : 64) - 1 & 63);
                if (!past || part > c0) left -= before;
                if (past) break;
            }
            vb = min(part * vpp, row.nvec);
            ve = min(vb + vpp, row.nvec);
            head = part == 0;
            tail = part == C - 1;
        }
        token = locate(sh, row, vb, ve, head, tail, d.bits, left);
    }
    if (t == 0) {
        tokens[m] = token;
        if (logprobs) logprobs[m] = d.logprob;
    }
}

// ---- draft acceptance ------------------------------------------------------------------

// One wave per sequence, one more for the rows outside every sequence: ballots find the
// first mismatch. Latency alone (2.7 us for 2048 sequences of 10240 rows, 1.4 us for one).
__global__ __launch_bounds__(256) void accept_kernel(const int32_t *__restrict__ tokens, const int32_t *__restrict__ inputs,
                                                     const int32_t *__restrict__ starts, int32_t *__restrict__ accepted,
                                                     int32_t *__restrict__ next, int32_t *__restrict__ committed,
                                                     int M, int S) {
    const int lane = threadIdx.x & 63;
    const int s = blockIdx.x * 4 + wave_id();
    if (s > S) return;
    auto start = [&](int i) { return min(max(starts[i], 0), M); };
    if (s == S) {
        const int b = start(0), e = start(S);
        for (int i = lane; i < b; i += 64) committed[i] = -1;
        for (int i = e + lane; i < M; i += 64) committed[i] = -1;
        return;
    }
    const int b = start(s), e = max(b, start(s + 1));
    int n = 0;
    bool open = true;  // no mismatch yet
    for (int j0 = 0; b + j0 < e; j0 += 64) {
        const int i = b + j0 + lane;
        const bool in = i < e;
        const int tok = in ? tokens[i] : -1;
        const bool stop = !(i + 1 < e && tok >= 0 && tok == inputs[i + 1]);
        const uint64_t stops = __ballot(stop);
        const int first = stops ? __builtin_ctzll(stops) : 64;
        if (in) committed[i] = open && lane <= first ? tok : -1;
        if (open && stops) {
            n = j0 + first;
            open = false;
        }
    }
    if (lane == 0) {
        accepted[s] = n;
        next[s] = b < e ? tokens[b + n] : -1;
    }
}

}  // namespace

SamplePlan plan_sample(int64_t M, int64_t V, int num_cus) {
    SamplePlan p{};
    const int64_t nvec = V / 8 + 1;
    // parts of a row: as many workgroups as the chip holds at once (44 rows: 28.6 us with 5,
    // 31.3 with 6), at least one vector a thread, no more than 8 (M = 1, nothing filtered: 29 us
    // with 8, 32 with 16, 39 with 31: the lists grow), and one where there would be fewer than 5
    // (64 rows: with 4 parts 34.2 us, filtered 29.7; with one 30.6 and 32.1)
    int64_t C = std::min<int64_t>(num_cus / M, (nvec + kThreads - 1) / kThreads);
    C = C < 5 ? 1 : std::min<int64_t>(C, 8);
    if (C > 1) C = std::max<int64_t>(C, (nvec + kMaxPartVectors - 1) / kMaxPartVectors);
    p.parts = (int)std::max<int64_t>(C, 1);
    p.mark = M > num_cus;
    p.vectors_per_part = (int)((nvec + p.parts - 1) / p.parts);
    if (p.parts > 1) p.workspace_bytes = kCounterBytes + (size_t)M * p.parts * kPartWords * 4;
    return p;
}

namespace {

// A workgroup per row, of rows that one launch takes.
hipError_t launch_rows(const SamplePlan &p, const uint16_t *l, int64_t ld, const Params &par, int32_t *tokens,
                       float *logprobs, int64_t M, int64_t V, hipStream_t stream) {
    // One table is sooner cleared and read, two leave a quarter of the row to search. They meet
    // between 4000 and 6000 tokens (M = 1000, us, one / two: V = 100 32.1 / 34.3, 3000 33.6 / 34.5,
    // 4200 35.1 / 35.3, 8000 37.1 / 36.3) and stay within 2% of each other up to 32000.
    const bool quarters = V / 8 + 1 > kThreads / 2 && V / 8 + 1 <= 4 * kMaxQuarter;
#define SVQ_ROW(WAY, MARK)                                                                                          \
    hipLaunchKernelGGL((sample_row_kernel<WAY, MARK>), dim3((uint32_t)M), dim3(kThreads), 0, stream, l, ld, par,    \
                   tokens, logprobs, (int)V)
    if (!p.mark) {
        if (quarters) SVQ_ROW(kQuarters, false);
        else SVQ_ROW(kWhole, false);
        return hipGetLastError();
    }
    if (quarters) SVQ_ROW(kQuarters, true);
    else SVQ_ROW(kWhole, true);
#undef SVQ_ROW
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sample_long_kernel, dim3((uint32_t)std::min<int64_t>(M, 256)), dim3(kThreads), 0, stream, l, ld,
                       par, tokens, logprobs, M, (int)V);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SamplePlan &p, const void *logits, int64_t ld, const float *u, const float *temperature,
                         const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
                         float *logprobs, int64_t M, int64_t V, void *workspace, hipStream_t stream) {
    const Params par{u, temperature, top_p, min_p, top_k};
    const uint16_t *l = (const uint16_t *)logits;
    if (p.parts == 1) {
        // a launch has fewer than 2^32 threads
        constexpr int64_t kMost = (int64_t(1) << 31) / kThreads;
        for (int64_t m = 0; m < M; m += kMost) {
            auto from = [&](auto *q) { return q ? q + m : q; };
            const Params at{from(u), from(temperature), from(top_p), from(min_p), from(top_k)};
            const hipError_t e = launch_rows(p, l + m * ld, ld, at, tokens + m, from(logprobs), std::min(M - m, kMost), V, stream);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    uint32_t *parts = (uint32_t *)ws_partials(workspace);
    hipLaunchKernelGGL(sample_count_kernel, dim3((uint32_t)(M * p.parts)), dim3(kThreads), 0, stream, l, ld, par, parts,
                       (int)V, p.parts, p.vectors_per_part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sample_select_kernel, dim3((uint32_t)M), dim3(kThreads), 0, stream, l, ld, par,
                       (const uint32_t *)parts, tokens, logprobs, (int)V, p.parts, p.vectors_per_part);
    return hipGetLastError();
}

hipError_t launch_accept_drafts(const int32_t *tokens, const int32_t *inputs, const int32_t *starts, int32_t *accepted,
                                int32_t *next, int32_t *committed, int64_t M, int64_t S, hipStream_t stream) {
    hipLaunchKernelGGL(accept_kernel, dim3((uint32_t)((S + 1 + 3) / 4)), dim3(256), 0, stream, tokens, inputs, starts,
                       accepted, next, committed, (int)M, (int)S);
    return hipGetLastError();
}

}  // namespace svq
