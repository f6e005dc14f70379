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
// A token is a whole number, so W must not depend on rounding: fp64 sums. What
// makes that cheap is that bf16 logits take few different values. The kernel never
// sorts: it counts values (a histogram in LDS, exact and independent of the order
// of its atomics), which orders them, and takes one fp64 exponential per occurring
// value instead of one per token. The position then names a value and an ordinal
// among its equals, and a scan of the row finds that occurrence.
//
// Values are binned by their bf16 pattern: magnitudes in [2^-16, 2^16) of either
// sign are 8192 bins; zero has one; smaller magnitudes (a logit in 10^4) go to a
// list that is ordered by comparison. A row with more than kSideMax of those, or
// with a larger magnitude, is counted the long way: four windows of 16384 patterns
// each, one scan of the row per window and step.
#include <algorithm>

#include "svq_launch.h"

namespace svq {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr uint32_t kBinsHalf = 4096;        // 32 exponents x 128 mantissas
constexpr uint32_t kBins = 2 * kBinsHalf;   // positive descending, then negative descending
constexpr uint32_t kMagLo = 111u << 7;      // pattern of 2^-16
constexpr uint32_t kSideMax = kThreads - 1; // and one entry for zero
constexpr uint32_t kWindow = 16384;         // patterns per window of the long way
constexpr int kWindows = 4;

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

// Calls f(bits) for every element of vectors [vb, ve), and of the head and the tail
// where asked; any order.
template <typename F>
__device__ __forceinline__ void for_elements(const Row &r, int vb, int ve, bool head, bool tail, F f) {
    const int t = threadIdx.x;
    auto vec = [&](uint4 q) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t u = (&q.x)[w];
            f(u & 0xFFFFu);
            f(u >> 16);
        }
    };
    int v = vb + t;
    for (; v + 3 * kThreads < ve; v += 4 * kThreads) {
        uint4 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = row_vec(r, v + i * kThreads);
#pragma unroll
        for (int i = 0; i < 4; ++i) vec(q[i]);
    }
    for (; v < ve; v += kThreads) vec(row_vec(r, v));
    if (head && t < r.head) f(r.p[t]);
    if (tail && t >= 64 && t < 64 + r.tail) f(r.p[r.head + 8 * r.nvec + t - 64]);
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

__device__ __forceinline__ uint32_t bin_bits(uint32_t bin) {
    return bin < kBinsHalf ? kMagLo + (kBinsHalf - 1 - bin) : (0x8000u | (kMagLo + (bin - kBinsHalf)));
}

struct Weight {
    double max, inv_t;
    __device__ __forceinline__ double exponent(uint32_t bits) const {
        const double d = value_of(bits) - max;
        return value_of(bits) == max ? 0.0 : d * inv_t;  // also for max = +inf
    }
    __device__ __forceinline__ double operator()(uint32_t bits) const {
        const double d = value_of(bits) - max;
        if (value_of(bits) == max) return 1.0;
        return d < -1.0e300 ? 0.0 : exp(d * inv_t);  // finite below an infinite maximum: 0, whatever T
    }
};

struct Params {
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
};
__device__ __forceinline__ bool is_greedy(const Params &p, int64_t m) { return p.temperature && !(p.temperature[m] > 0.f); }
// Number of tokens top_k leaves (0: no limit).
__device__ __forceinline__ uint32_t limit_of(const Params &p, int64_t m) {
    if (is_greedy(p, m)) return 1;
    const int k = p.top_k ? p.top_k[m] : 0;
    return k > 0 ? (uint32_t)k : 0;
}

// ---- histogram of a row or of a part of it -------------------------------------------

struct Hist {
    uint32_t bin[kBins];
    uint32_t side[kSideMax + 1];        // patterns of tiny magnitudes
    uint32_t side_n, zeros, odd;        // odd: the row needs the long way
};

__device__ __forceinline__ void hist_clear(Hist &h) {
    for (int i = threadIdx.x; i < (int)kBins / 4; i += kThreads) ((uint4 *)h.bin)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) h.side_n = h.zeros = h.odd = 0;
}

__device__ __forceinline__ void hist_add(Hist &h, uint32_t b) {
    const uint32_t mag = b & 0x7FFFu, q = mag - kMagLo;
    if (q < kBinsHalf) {
        atomicAdd(&h.bin[(b & 0x8000u) ? kBinsHalf + q : kBinsHalf - 1 - q], 1u);
    } else if (mag == 0) {
        atomicAdd(&h.zeros, 1u);
    } else if (mag < kMagLo) {
        const uint32_t at = atomicAdd(&h.side_n, 1u);
        if (at < kSideMax) h.side[at] = b;
    } else if (mag <= 0x7F80u && b != 0xFF80u) {
        h.odd = 1;
    }
}

// ---- block scans ----------------------------------------------------------------------

struct Scratch {
    double wsum[kWaves][4];
    uint32_t csum[kWaves][4];
    uint32_t sel[8];
    double val[4];
    uint32_t count[kWaves + 1];
};

// Exclusive prefix over the segments in order, threads in order within a segment,
// of local sums c[S] and w[S]; the totals go to tc, tw. Fixed order of additions.
template <int S>
__device__ __forceinline__ void order_scan(Scratch &sc, const uint32_t (&c)[S], const double (&w)[S],
                                           uint32_t (&ec)[S], double (&ew)[S], uint32_t &tc, double &tw) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    uint32_t ic[S];
    double iw[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        ic[s] = c[s];
        iw[s] = w[s];
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const uint32_t pc = __shfl_up(ic[s], d);
            const double pw = __shfl_up(iw[s], d);
            if (lane >= d) {
                ic[s] += pc;
                iw[s] += pw;
            }
        }
    if (lane == 63)
#pragma unroll
        for (int s = 0; s < S; ++s) {
            sc.csum[wave][s] = ic[s];
            sc.wsum[wave][s] = iw[s];
        }
    __syncthreads();
    tc = 0;
    tw = 0.0;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        uint32_t bc = tc;
        double bw = tw;
        for (int v = 0; v < kWaves; ++v) {
            if (v == wave) {
                bc = tc;
                bw = tw;
            }
            tc += sc.csum[v][s];
            tw += sc.wsum[v][s];
        }
        const uint32_t xc = __shfl_up(ic[s], 1);
        const double xw = __shfl_up(iw[s], 1);
        ec[s] = bc + (lane ? xc : 0);
        ew[s] = bw + (lane ? xw : 0.0);
    }
    __syncthreads();
}

// ---- the draw ---------------------------------------------------------------------------

struct Drawn {
    uint32_t bits, ordinal;  // the value and which of its occurrences
    float logprob;
    bool any, counted;       // anything to draw from; by the histogram, not the long way
};

// Counts(seg) makes segment `seg` of the order readable; count(seg, j) and bits(seg, j)
// are its bins, descending, NB(seg) of them for each thread.
template <int S, typename Bins>
__device__ Drawn draw(Scratch &sc, Bins &bins, const Params &par, int64_t m) {
    Drawn out{0, 0, -__builtin_inff(), false, Bins::kResident};
    const int t = threadIdx.x;
    Weight wt;
    const bool greedy = is_greedy(par, m);
    wt.inv_t = greedy || !par.temperature ? 1.0 : 1.0 / (double)par.temperature[m];

    // the largest value
    if (t == 0) sc.sel[0] = 0;
    __syncthreads();
    uint32_t best = 0;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        bins.load(s);
        for (int j = 0; j < bins.nb(s); ++j)
            if (bins.count(s, j)) best = max(best, key_of(bins.bits(s, j)));
        if (!Bins::kResident && __syncthreads_or(best != 0)) break;
    }
    if (best) atomicMax(&sc.sel[0], best);
    __syncthreads();
    const uint32_t top = sc.sel[0];
    if (top == 0) return out;  // nothing to draw from
    out.any = true;
    wt.max = value_of(bits_of(top));

    uint32_t c[S], ec[S], total;
    double w[S], ew[S], wtotal;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        bins.load(s);
        c[s] = 0;
        w[s] = 0.0;
        for (int j = 0; j < bins.nb(s); ++j) {
            const uint32_t n = bins.count(s, j);
            if (n) {
                c[s] += n;
                w[s] += n * wt(bins.bits(s, j));
            }
        }
    }
    order_scan<S>(sc, c, w, ec, ew, total, wtotal);

    // W(n) for 1 <= n <= total
    auto mass = [&](uint32_t n) -> double {
        if (n >= total) return wtotal;
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (ec[s] < n && n <= ec[s] + c[s]) sc.sel[1] = s;
        __syncthreads();
        const int seg = sc.sel[1];
        bins.load(seg);
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (s == seg && ec[s] < n && n <= ec[s] + c[s]) {
                uint32_t left = n - ec[s];
                double sum = ew[s];
                for (int j = 0; j < bins.nb(s) && left; ++j) {
                    const uint32_t k = min(left, bins.count(s, j));
                    if (k) sum += k * wt(bins.bits(s, j));
                    left -= k;
                }
                sc.val[0] = sum;
            }
        __syncthreads();
        return sc.val[0];
    };
    // The last (segment, thread) that holds tokens of the first `n` and has
    // W before it below `target` (or equal to it, if `eq`): the one that crosses it.
    auto crossing = [&](double target, uint32_t n, bool eq) -> uint32_t {
        if (t == 0) sc.sel[2] = 0;
        __syncthreads();
        uint32_t at = 0;
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (c[s] && ec[s] < n && (ec[s] == 0 || ew[s] < target || (eq && ew[s] == target))) at = s * kThreads + t + 1;
        if (at) atomicMax(&sc.sel[2], at);
        __syncthreads();
        const uint32_t r = sc.sel[2] - 1;
        bins.load(r / kThreads);
        return r;
    };

    uint32_t n = total;
    const uint32_t k = limit_of(par, m);
    if (k && k < n) n = k;
    if (!greedy && par.top_p) {
        const float p = par.top_p[m];
        if (p < 1.f) {
            const double target = (double)p * mass(n);
            const uint32_t own = crossing(target, n, false);
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (own == (uint32_t)(s * kThreads + t)) {
                    // tokens whose W before them is below the target
                    uint32_t kept = ec[s];
                    double before = ew[s];
                    for (int j = 0; j < bins.nb(s); ++j) {
                        const uint32_t cnt = bins.count(s, j);
                        if (!cnt) continue;
                        const double v = wt(bins.bits(s, j));
                        const double end = before + cnt * v;
                        if (end < target) {
                            kept += cnt;
                            before = end;
                            continue;
                        }
                        double x = v > 0.0 ? ceil((target - before) / v) : (double)cnt;
                        uint32_t add = x <= 0.0 ? 0 : (x >= (double)cnt ? cnt : (uint32_t)x);
                        while (add > 0 && before + (add - 1) * v >= target) --add;
                        while (add < cnt && before + add * v < target) ++add;
                        kept += add;
                        break;
                    }
                    sc.sel[3] = kept ? kept : 1;
                }
            __syncthreads();
            n = min(n, sc.sel[3]);
        }
    }
    if (!greedy && par.min_p) {
        const float q = par.min_p[m];
        if (q > 0.f) {
            if (t == 0) sc.sel[4] = 1;
            __syncthreads();
            uint32_t kept = 0;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                bins.load(s);
                uint32_t run = ec[s];
                for (int j = 0; j < bins.nb(s); ++j) {
                    const uint32_t cnt = bins.count(s, j);
                    if (!cnt) continue;
                    if (wt(bins.bits(s, j)) < (double)q) break;
                    run += cnt;
                    kept = run;
                }
            }
            if (kept) atomicMax(&sc.sel[4], kept);
            __syncthreads();
            n = min(n, sc.sel[4]);
        }
    }
    const double sum = mass(n);
    float u = par.u[m];
    u = u >= 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f;  // [0, 1), NaN as 0
    const double target = (double)u * sum;
    const uint32_t own = crossing(target, n, true);
#pragma unroll
    for (int s = 0; s < S; ++s)
        if (own == (uint32_t)(s * kThreads + t)) {
            uint32_t pos = ec[s];
            double before = ew[s];
            uint32_t bits = 0, ord = 0;
            for (int j = 0; j < bins.nb(s) && pos < n; ++j) {
                const uint32_t cnt = min(bins.count(s, j), n - pos);
                if (!cnt) continue;
                const uint32_t bb = bins.bits(s, j);
                const double v = wt(bb);
                const double end = before + cnt * v;
                if (v > 0.0 || pos == 0) {  // the last value with weight, should rounding leave none crossing
                    bits = bb;
                    ord = cnt - 1;
                }
                if (end > target) {
                    const double x = (target - before) / v;
                    ord = x <= 0.0 ? 0 : (x >= (double)cnt ? cnt - 1 : (uint32_t)x);
                    while (ord > 0 && before + ord * v > target) --ord;
                    while (ord + 1 < cnt && before + (ord + 1) * v <= target) ++ord;
                    break;
                }
                pos += cnt;
                before = end;
            }
            sc.sel[5] = bits;
            sc.sel[6] = ord;
            sc.val[1] = wt.exponent(bits) - log(sum);
        }
    __syncthreads();
    out.bits = sc.sel[5];
    out.ordinal = sc.sel[6];
    out.logprob = (float)sc.val[1];
    return out;
}

// The order of a counted row: positive bins, tiny magnitudes and zero, negative bins.
struct CountedBins {
    static constexpr bool kResident = true;
    const uint32_t *bin, *side_bits, *side_count;
    int sides;
    __device__ __forceinline__ void load(int) {}
    __device__ __forceinline__ int nb(int s) const { return s == 1 ? 1 : (int)kBinsHalf / kThreads; }
    __device__ __forceinline__ uint32_t index(int s, int j) const {
        return (s ? kBinsHalf : 0) + threadIdx.x * (kBinsHalf / kThreads) + j;
    }
    __device__ __forceinline__ uint32_t count(int s, int j) const {
        if (s == 1) return (int)threadIdx.x < sides ? side_count[threadIdx.x] : 0;
        return bin[index(s, j)];
    }
    __device__ __forceinline__ uint32_t bits(int s, int j) const {
        return s == 1 ? side_bits[threadIdx.x] : bin_bits(index(s, j));
    }
};

// All patterns, one window of them at a time, descending.
struct WindowBins {
    static constexpr bool kResident = false;
    uint32_t *table;  // kWindow counts
    Row row;
    __device__ void load(int s) {
        __syncthreads();
        for (int i = threadIdx.x; i < (int)kWindow / 4; i += kThreads) ((uint4 *)table)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        uint32_t *tab = table;
        for_elements(row, 0, row.nvec, true, true, [=](uint32_t b) {
            const uint32_t key = key_of(b);
            if (key_valid(key) && (int)(key >> 14) == kWindows - 1 - s)
                atomicAdd(&tab[kWindow - 1 - (key & (kWindow - 1))], 1u);
        });
        __syncthreads();
    }
    __device__ __forceinline__ int nb(int) const { return kWindow / kThreads; }
    __device__ __forceinline__ uint32_t count(int, int j) const { return table[threadIdx.x * (kWindow / kThreads) + j]; }
    __device__ __forceinline__ uint32_t bits(int s, int j) const {
        return bits_of((uint32_t)(kWindows - 1 - s) * kWindow + kWindow - 1 - (threadIdx.x * (kWindow / kThreads) + j));
    }
};

// Index of the ordinal-th element equal to `bits` among vectors [vb, ve) (and head or
// tail), in index order, by the whole workgroup; every thread gets it (-1 if there are
// fewer, which a consistent histogram excludes).
__device__ int locate(Scratch &sc, const Row &r, int vb, int ve, bool head, bool tail, uint32_t bits, uint32_t ordinal) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    const bool zero = (bits & 0x7FFFu) == 0;  // both zeros are one value
    const uint32_t mask16 = zero ? 0x7FFFu : 0xFFFFu;
    auto same = [&](uint32_t b) { return ((b ^ bits) & mask16) == 0; };
    uint32_t left = ordinal;
    __shared__ int found;
    if (threadIdx.x == 0) found = -1;
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
    auto matches = [&](const uint4 &q) {
        uint32_t n = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t x = (&q.x)[w];
            n += (uint32_t)same(x & 0xFFFFu) + (uint32_t)same(x >> 16);
        }
        return n;
    };
    constexpr int kIter = 8;                    // vectors of a lane per block of the row
    constexpr int kBlock = kThreads * kIter;    // vectors
    for (int b0 = vb; b0 < ve; b0 += kBlock) {
        const int w0 = b0 + wave * 64 * kIter;
        uint32_t cnt[kIter], sum = 0;
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int v = w0 + i * 64 + lane;
            cnt[i] = v < ve ? matches(row_vec(r, v)) : 0;
            sum += cnt[i];
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
        if (lane == 0) sc.count[wave] = sum;
        __syncthreads();
        uint32_t before = 0, all = 0;
        for (int v = 0; v < kWaves; ++v) {
            if (v == wave) before = all;
            all += sc.count[v];
        }
        if (left < all) {
            if (before <= left && left < before + sum) {  // in this wave's part
                uint32_t rest = left - before;
#pragma unroll
                for (int i = 0; i < kIter; ++i) {
                    uint32_t inc = cnt[i];
                    for (int d = 1; d < 64; d <<= 1) {
                        const uint32_t o = __shfl_up(inc, d);
                        if (lane >= d) inc += o;
                    }
                    const uint32_t tot = __shfl(inc, 63);
                    if (rest < tot) {
                        const uint32_t mine = inc - cnt[i];
                        if (mine <= rest && rest < inc) {
                            const int v = w0 + i * 64 + lane;
                            uint32_t skip = rest - mine;
                            int at = -1;
                            for (int e = 0; e < 8; ++e)
                                if (same(r.p[r.head + (int64_t)v * 8 + e])) {
                                    if (skip == 0) {
                                        at = r.head + v * 8 + e;
                                        break;
                                    }
                                    --skip;
                                }
                            found = at;
                        }
                        break;
                    }
                    rest -= tot;
                }
            }
            __syncthreads();
            return found;
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

struct SelectShared {
    union {
        struct {
            Hist h;
            uint32_t sorted_bits[kThreads], sorted_count[kThreads];
        } counted;
        uint32_t table[kWindow];
    };
    Scratch sc;
};

// Draws from the histogram in sh (of the whole row), or the long way.
__device__ Drawn draw_row(SelectShared &sh, const Row &row, const Params &par, int64_t m) {
    Hist &h = sh.counted.h;
    const uint32_t side_n = h.side_n, zeros = h.zeros;
    if (h.odd || side_n > kSideMax) {
        WindowBins bins{sh.table, row};
        __syncthreads();
        return draw<kWindows>(sh.sc, bins, par, m);
    }
    // order the list: a value's place is the number of larger entries, its first entry
    // stands there for all equal ones (the places of the others stay empty); zero stands
    // between the signs
    const uint32_t sides = side_n + (zeros ? 1 : 0);
    const uint32_t t = threadIdx.x;
    sh.counted.sorted_count[t] = 0;
    __syncthreads();
    if (t < sides) {
        const uint32_t mine = t < side_n ? h.side[t] : 0, key = key_of(mine);
        uint32_t place = 0, equal = 0;
        bool first = true;
        for (uint32_t j = 0; j < side_n; ++j) {
            const uint32_t o = key_of(h.side[j]);
            place += o > key;
            equal += o == key;
            first = first && !(o == key && j < t);
        }
        if (t < side_n && zeros) place += 0x8000u > key;
        if (first) {
            sh.counted.sorted_bits[place] = mine;
            sh.counted.sorted_count[place] = t < side_n ? equal : zeros;
        }
    }
    __syncthreads();
    CountedBins bins{h.bin, sh.counted.sorted_bits, sh.counted.sorted_count, (int)sides};
    return draw<3>(sh.sc, bins, par, m);
}

// ---- kernels ------------------------------------------------------------------------------

// One workgroup per row: count, draw, find.
__global__ __launch_bounds__(kThreads) void sample_row_kernel(const uint16_t *__restrict__ logits, int64_t ld, Params par,
                                                              int32_t *__restrict__ tokens, float *__restrict__ logprobs,
                                                              int V) {
    __shared__ __attribute__((aligned(16))) SelectShared sh;
    const int64_t m = blockIdx.x;
    const Row row = make_row(logits + m * ld, V);
    Hist &h = sh.counted.h;
    hist_clear(h);
    __syncthreads();
    for_elements(row, 0, row.nvec, true, true, [&](uint32_t b) { hist_add(h, b); });
    __syncthreads();
    const Drawn d = draw_row(sh, row, par, m);
    int token = -1;
    if (d.any) token = locate(sh.sc, row, 0, row.nvec, true, true, d.bits, d.ordinal);
    if (threadIdx.x == 0) {
        tokens[m] = token;
        if (logprobs) logprobs[m] = d.logprob;
    }
}

// Workspace of one (row, part): header, then the occurring bins (bin << 18 | count),
// then the list of tiny magnitudes.
constexpr uint32_t kHeader = 4;
constexpr uint32_t kPartWords = kHeader + kBins + kSideMax + 1;
constexpr uint32_t kCountBits = 18;
constexpr int64_t kMaxPartVectors = ((1 << kCountBits) - 16) / 8;  // a part's tokens fit the count
constexpr int kMaxParts = kThreads;

__global__ __launch_bounds__(kThreads) void sample_count_kernel(const uint16_t *__restrict__ logits, int64_t ld, Params par,
                                                                uint32_t *__restrict__ parts, int V, int C, int vpp) {
    __shared__ __attribute__((aligned(16))) Hist h;
    __shared__ uint32_t wsum[kWaves][2];
    const int64_t m = blockIdx.x / C;
    const int part = blockIdx.x % C;
    const Row row = make_row(logits + m * ld, V);
    hist_clear(h);
    __syncthreads();
    const int vb = min(part * vpp, row.nvec), ve = min(vb + vpp, row.nvec);
    for_elements(row, vb, ve, part == 0, part == C - 1, [&](uint32_t b) { hist_add(h, b); });
    __syncthreads();
    // occurring bins in descending order, but none behind which top_k tokens of this
    // part already stand; (bins << 18 | tokens) are scanned in one word
    const int t = threadIdx.x, lane = t & 63, wave = wave_id();
    const uint4 v0 = ((const uint4 *)h.bin)[t], v1 = ((const uint4 *)h.bin)[kBinsHalf / 4 + t];
    const uint32_t n[2][4] = {{v0.x, v0.y, v0.z, v0.w}, {v1.x, v1.y, v1.z, v1.w}};
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
    const uint32_t k = limit_of(par, m);
    const uint32_t middle = h.zeros + h.side_n;
    uint32_t run = 0;
    __shared__ uint32_t entries;
    if (t == 0) entries = 0;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        uint32_t before = run;
        for (int v = 0; v < kWaves; ++v) {
            if (v == wave) before = run;
            run += wsum[v][s];
        }
        uint32_t at = before + inc[s] - own[s];
        uint32_t last = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n[s][j]) {
                const uint32_t above = (at & ((1u << kCountBits) - 1)) + (s ? middle : 0), pos = at >> kCountBits;
                if (!k || above < k) {
                    dst[kHeader + pos] = ((s ? kBinsHalf : 0) + 4 * t + j) << kCountBits | n[s][j];
                    last = pos + 1;
                }
                at += n[s][j] + (1u << kCountBits);
            }
        if (last) atomicMax(&entries, last);
    }
    const uint32_t sides = min(h.side_n, kSideMax);
    for (uint32_t i = t; i < sides; i += kThreads) dst[kHeader + kBins + i] = h.side[i];
    __syncthreads();
    if (t == 0) {
        dst[0] = entries;
        dst[1] = h.side_n;
        dst[2] = h.zeros;
        dst[3] = h.odd;
    }
}

__global__ __launch_bounds__(kThreads) void sample_select_kernel(const uint16_t *__restrict__ logits, int64_t ld, Params par,
                                                                 const uint32_t *__restrict__ parts,
                                                                 int32_t *__restrict__ tokens,
                                                                 float *__restrict__ logprobs, int V, int C, int vpp) {
    __shared__ __attribute__((aligned(16))) SelectShared sh;
    __shared__ uint32_t in_part[kMaxParts];
    const int64_t m = blockIdx.x;
    const int t = threadIdx.x, lane = t & 63, wave = wave_id();
    const Row row = make_row(logits + m * ld, V);
    const uint32_t *src = parts + (int64_t)m * C * kPartWords;
    Hist &h = sh.counted.h;
    hist_clear(h);
    __syncthreads();
    for (int c = wave; c < C; c += kWaves) {
        const uint32_t *p = src + (int64_t)c * kPartWords;
        const uint32_t entries = p[0], side_n = p[1], zeros = p[2], odd = p[3];
        for (uint32_t i = lane; i < entries; i += 64) {
            const uint32_t e = p[kHeader + i];
            atomicAdd(&h.bin[e >> kCountBits], e & ((1u << kCountBits) - 1));
        }
        uint32_t at = 0;
        if (lane == 0) {
            if (zeros) atomicAdd(&h.zeros, zeros);
            if (odd) h.odd = 1;
            if (side_n) at = atomicAdd(&h.side_n, side_n);
        }
        at = __builtin_amdgcn_readfirstlane(at);
        for (uint32_t i = lane; i < min(side_n, kSideMax); i += 64)
            if (at + i < kSideMax) h.side[at + i] = p[kHeader + kBins + i];
    }
    __syncthreads();
    const Drawn d = draw_row(sh, row, par, m);
    int token = -1;
    if (d.any) {
        const uint32_t q = (d.bits & 0x7FFFu) - kMagLo;
        if (d.counted && q < kBinsHalf) {
            // the value's count in each part tells which part holds the occurrence; a
            // part's entries ascend by bin: 64 samples, then the stretch between two
            const uint32_t want = (d.bits & 0x8000u) ? kBinsHalf + q : kBinsHalf - 1 - q;
            for (int c = wave; c < C; c += kWaves) {
                const uint32_t *p = src + (int64_t)c * kPartWords;
                const uint32_t entries = p[0], stride = (entries + 63) / 64;
                p += kHeader;
                const uint32_t i0 = lane * stride;
                const bool le = i0 < entries && (p[i0] >> kCountBits) <= want;
                const int hit = __popcll(__ballot(le));  // samples at or before it
                uint32_t n = 0;
                if (hit)
                    for (uint32_t i = lane; i < stride; i += 64) {
                        const uint32_t at = (hit - 1) * stride + i;
                        const uint32_t e = at < entries ? p[at] : 0xFFFFFFFFu;
                        if ((e >> kCountBits) == want) n = e & ((1u << kCountBits) - 1);
                    }
#pragma unroll
                for (int x = 1; x < 64; x <<= 1) n += __shfl_xor(n, x);
                if (lane == 0) in_part[c] = n;
            }
            __syncthreads();
            uint32_t left = d.ordinal;
            int part = 0;
            while (part < C - 1 && left >= in_part[part]) left -= in_part[part++];
            const int vb = min(part * vpp, row.nvec), ve = min(vb + vpp, row.nvec);
            token = locate(sh.sc, row, vb, ve, part == 0, part == C - 1, d.bits, left);
        } else {  // a tiny magnitude, zero, or the long way: no counts by part
            token = locate(sh.sc, row, 0, row.nvec, true, true, d.bits, d.ordinal);
        }
    }
    if (t == 0) {
        tokens[m] = token;
        if (logprobs) logprobs[m] = d.logprob;
    }
}

// ---- draft acceptance ------------------------------------------------------------------

// One wave per sequence, one more for the rows outside every sequence.
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
    // parts of a row: enough workgroups to fill the chip, at least one vector a thread
    int64_t C = std::min<int64_t>((num_cus + M - 1) / M, (nvec + kThreads - 1) / kThreads);
    if (C > 1) C = std::max<int64_t>(C, (nvec + kMaxPartVectors - 1) / kMaxPartVectors);
    p.parts = (int)std::max<int64_t>(C, 1);
    p.vectors_per_part = (int)((nvec + p.parts - 1) / p.parts);
    if (p.parts > 1) p.workspace_bytes = kCounterBytes + (size_t)M * p.parts * kPartWords * 4;
    return p;
}

hipError_t launch_sample(const SamplePlan &p, const void *logits, int64_t ld, const float *u, const float *temperature,
                         const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
                         float *logprobs, int64_t M, int64_t V, void *workspace, hipStream_t stream) {
    const Params par{u, temperature, top_p, min_p, top_k};
    const uint16_t *l = (const uint16_t *)logits;
    if (p.parts == 1) {
        hipLaunchKernelGGL(sample_row_kernel, dim3((uint32_t)M), dim3(kThreads), 0, stream, l, ld, par, tokens, logprobs,
                           (int)V);
        return hipGetLastError();
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
