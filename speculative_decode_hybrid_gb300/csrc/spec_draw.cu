// spec_sample: tokens sampled from logits with temperature, top-k, top-p and
// min-p, from given random numbers (the draft's side of spec_accept_sample, and
// its target rows truncated; openinfer PR #626, What Changed: the draft proposes
// a span).
//
// Mathematics. With w_v = exp((x_v - max) / T) and the tokens in the greedy order
// (larger x first, lower index among equals), each limit keeps a beginning of
// that order: the first K; those with w >= min_p; those before which less than
// top_p of the first K's weight lies. So a row has one cut, an element (x, index)
// in that order, and the next token is the largest w / noise above it, which
// needs no sum.
//
// One cluster of blocks holds a row in shared memory, each block a slice, and
// reads it once. The cut is found by a histogram over the weights' exponents, 48 bins
// an octave, summed over the cluster; the cut's bin, a few elements out of many
// thousands, is gathered, and every block picks the cut from it for itself. A bin
// with more than kList elements (equal or nearly equal logits) is cut by histograms over
// the bits of (x, index), 11 at a time, until few enough are left. With K small, all that lies
// above is gathered along with the bin, and the same picking gives the cut of all
// limits.
//
// The masses that top_p compares are integers, so that sums do not depend on the
// order of the atomic additions, and off by at most 2^-28 + V 2^-42 of the row's, so that a
// token that is not that near the border is on the side that it is on in exact arithmetic (f32 weights, off by
// up to 2^-20, would misplace one in a hundred borders among weights of 1e-4). An
// element of the bin 2^(-n / 48) weighs 2^(-n / 48) (1 + z) with |z| < 2^-7: the
// bin's mass is the sum of 1 + z in 28 fraction bits, in two halves that 32 bits hold
// for all of a block's elements: 20 operations and two 32-bit additions in shared
// memory for an element (272 rows took 1,586 us with 64-bit additions of masses, 402 at
// that state with these).
//
// Bound by latency: a row's phases follow one another, each with waits for the cluster
// or for memory, and two blocks fit an SM. In cycles of one row of 151,936 with top-p
// (clock64 in its first block, inputs in L2): load 2,600, maximum 2,500, histogram 7,300,
// search 6,500, gathering and picking 9,500, noise 6,000, the token 3,000: 37,400 in all,
// of the 19 us that the call takes; from memory 54,000. 16 rows with all limits take 22 us;
// 272 rows with top-p and their distributions 271, of which the bytes would take 49; without
// the distributions 241, with a min-p alone, which needs neither histogram nor search, 122.
// At 64 registers a thread spills 144 bytes.
// Measured and dropped: functions that are not inlined, for shorter code (408 us instead
// of 350), the slice of the row 20, 36 or 60 clusters on asked for into L2 (338, 371 and
// 300 us in a state that took 305 without), five to ten loads in flight instead of four
// (269 to 273 us).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "gdn_device.cuh"
#include "gdn_host.h"
#include "gdnspec.h"

namespace {

namespace cg = cooperative_groups;
using gdndev::Buf;
using gdndev::make_key;
using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMostBlocks = 8;       // of a cluster
constexpr int kBins = 2048, kCoarse = kBins / 32;
constexpr int kList = 1024;          // elements gathered at most
constexpr int kFew = 128;            // of them, compared one with the other
constexpr int kSub = 2 * kThreads;   // bins of a block's own histogram of the list
constexpr int kPerOctave = 48;       // bins: 42 octaves, what is lighter weighs nothing in them
constexpr int kSteps = 32;           // of an octave in the elements' own masses
constexpr int kUnitBits = 28;        // fraction bits of 1 + z in a bin's sum, 16 of them in `lo`
constexpr int kMassBits = 44;        // a weight of 1; 2^19 of them fit 63 bits
constexpr int kIndexBits = 20;
static_assert(GDN_MAX_SAMPLE_VOCAB <= 1 << 19, "masses and indexes");
constexpr float kNan = __builtin_nanf("");

// 2^(j / n) in 62 fraction bits.
template <int n>
struct Powers {
    u64 v[n];
    constexpr Powers() : v() {
        constexpr double root = n == kSteps ? 1.0218971486541166782344801347833 : 1.0145453349375236414538678576629;  // 2^(1/32), 2^(1/48)
        double r = 1.0;
        for (int j = 0; j < n; ++j) {
            v[j] = (u64)(r * 4611686018427387904.0);
            r *= root;
        }
    }
};
static_assert(kSteps == 32 && kPerOctave == 48, "the roots");
__constant__ Powers<kSteps> kPowers;
__constant__ Powers<kPerOctave> kBinPowers;

struct Args {
    int vocab, per, blocks;  // rows of a request; blocks of a row
    const float *logits, *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p, *noise;
    int32_t *token;
    float *token_prob, *probs, *kept;
    int32_t *status;
};

struct Found {
    int bin;
    unsigned before;   // elements of the bins before it
    u64 mass_before;
    u64 target;        // what was to be reached
};

// What the mass before an element has to be below: `share` of `whole`, rounded up, the
// first element's at least. In whole numbers: 64-bit floating point is slow here.
__device__ __forceinline__ u64 limit_of(float share, u64 whole) {
    if (!(share > 0.f)) return 1;
    if (share >= 1.f) return whole;
    const unsigned bits = __float_as_uint(share), exponent = bits >> 23;
    const u64 m = (bits & 0x7fffffu) | (exponent ? 0x800000u : 0u);
    const int down = 150 - (int)max(exponent, 1u);  // share is m / 2^down; 24 or more
    const u64 hi = __umul64hi(m, whole), lo = m * whole;
    if (down >= 64) return down >= 128 ? 1 : max(1ull, (hi >> (down - 64)) + ((hi & ((1ull << (down - 64)) - 1)) != 0 || lo != 0));
    return max(1ull, (hi << (64 - down) | lo >> down) + ((lo & ((1ull << down) - 1)) != 0));
}

// What a histogram's bins hold.
enum Kind {
    kCounts,  // count: elements
    kFirst,   // hi, lo: sums of the upper and the lower 16 bits of 1 + z
    kBoth,    // count: elements; hi, lo as kFirst
    kFine,    // count: elements; hi, lo: masses
};

struct Smem {
    // A search is over in every block before what it found is gathered, and a barrier
    // of the cluster lies between a pick and the next search: one place does for what
    // searches use and what picks do.
    union {
        unsigned count[kBins];
        u64 list_mass[kList];
    };
    union {
        struct {
            unsigned hi[kBins], lo[kBins];
        };
        struct {
            u64 sub_mass[kSub];
            unsigned sub_count[kSub];
        };
    };
    union {
        struct {
            u64 coarse_mass[kMostBlocks][kCoarse];  // of each block, by 32 bins
            unsigned coarse_count[kMostBlocks][kCoarse];
        };
        u64 list_key[kList];  // places of all blocks' gathered elements
    };
    unsigned short own_at[kList];  // this block's, in its slice: the others read them
    int few[kFew], few_n;
    u64 power[kSteps], bin_power[kPerOctave];
    u64 warp_key[kWarps][2], key_of[kMostBlocks][2];
    u64 cut, cut_mass;
    float warp_f[kWarps], f_of[kMostBlocks], sum_of[kMostBlocks];
    int bad_of[kMostBlocks], own_n, kept_n;
    unsigned warp_count[kWarps];
    Found found;
};

// log2(e) / T in two parts. T == 0 is the limit: a factor that leaves weight only
// where x - max is 0.
struct Scale {
    float hi, lo;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// w to a few units of 2^-23: the roundings of the difference and of the exponent
// are put back.
__device__ __forceinline__ float weight(float x, float top, Scale c) {
    const float d = x - top, back = d - x, dl = (x - (d - back)) + (-top - back);
    const float y = d * c.hi;
    if (!(y > -150.f)) return 0.f;  // (a NaN of -inf x 0 too)
    const float lo = fmaf(d, c.hi, -y) + fmaf(d, c.lo, dl * c.hi);
    return ex2(y) * fmaf(lo, 0.693147180559945f, 1.f);
}

// w in kMassBits fraction bits, to 2^-40 of itself and half a unit: 2^(n / 32) from
// a table, e^z of the rest from its series, the differences and products with their
// rounding errors (two f32 parts each).
__device__ __forceinline__ u64 mass_of(float x, float top, Scale c, const u64 *power) {
    const float d = x - top, back = d - x, dl = (x - (d - back)) + (-top - back);
    const float y = d * c.hi;
    if (!(y > -60.f)) return 0;
    const float yl = fmaf(d, c.hi, -y) + fmaf(d, c.lo, dl * c.hi);
    const float n = rintf(y * kSteps), r = fmaf(n, -1.f / kSteps, y);
    constexpr float kLn2 = 0.693147180559945309f, kLn2Lo = (float)(0.693147180559945309417 - (double)kLn2);
    const float p = r * kLn2, e = fmaf(r, kLn2, -p) + fmaf(r, kLn2Lo, yl * kLn2), z = p + e;
    const float q = fmaf(z * z, fmaf(z, fmaf(z, 1.f / 24, 1.f / 6), 0.5f), e);
    const long long m = (1ll << 42) + __float2ll_rn(p * 4398046511104.f) + __float2ll_rn(q * 4398046511104.f);
    const int k = (int)n, down = -(k >> 5) + 60 - kMassBits;
    if (down > 63) return 0;
    return (__umul64hi((u64)m << 20, power[k & (kSteps - 1)]) + (1ull << (down - 1))) >> down;
}

// 1.5 x 2^23: a float of up to 2^22 added to it is rounded to the nearest integer, in
// its low bits (conversions run at a quarter of the rate of additions).
constexpr float kRound = 12582912.f;
__device__ __forceinline__ int rounded(float sum) { return __float_as_int(sum) - 0x4b400000; }

// Bin of the first histogram, the nearest, plus kRound: never falls as x does not rise.
__device__ __forceinline__ float bin_place(float y) {
    return fminf(y * -kPerOctave, (float)(kBins - 1)) + kRound;  // NaN (-inf x 0): the last
}
__device__ __forceinline__ int bin_of(float x, float top, Scale c) { return rounded(bin_place((x - top) * c.hi)); }

// The same, and 1 + z in kUnitBits fraction bits: |z| < 0.0073, off by 2^-28 (t's, the
// series' and the integer's roundings) of the element's weight.
__device__ __forceinline__ int bin_and_unit(float x, float top, Scale c, unsigned &unit) {
    const float d = x - top, back = d - x, dl = (x - (d - back)) + (-top - back);
    const float y = d * c.hi, place = bin_place(y);
    const float yl = fmaf(d, c.lo, fmaf(dl, c.hi, fmaf(d, c.hi, -y)));
    constexpr float kBin = 1.f / kPerOctave, kRest = (float)(1.0 / kPerOctave - (double)kBin);
    const float n = place - kRound, t = fmaf(n, kBin, y) + fmaf(n, kRest, yl);
    const float e = t * fmaf(t, fmaf(t, fmaf(t, 0.00961812910762847716f, 0.05550410866482157995f), 0.24022650695910071233f), 0.69314718055994530942f);
    unit = (unsigned)(rounded(fmaf(e, (float)(1 << kUnitBits), kRound)) + (1 << kUnitBits));
    return rounded(place);
}

// Mass of a bin of the first histogram: 2^(-bin / 48) = 2^(rest / 48) / 2^octaves.
__device__ __forceinline__ u64 bin_mass(int bin, u64 units, const u64 *power) {
    const int octaves = (bin + kPerOctave - 1) / kPerOctave, rest = octaves * kPerOctave - bin;
    // 28 + 16 + 62 - 64 fraction bits are kMassBits less two (2^19 units of 2^28 fit 64 bits)
    return __umul64hi(units << 16, power[rest]) << 2 >> octaves;
}

// Place in the greedy order: ascending is larger x first, then lower index.
__device__ __forceinline__ u64 place_of(float x, int index) {
    return (u64)(unsigned)~(unsigned)(make_key(x, 0u) >> 32) << kIndexBits | (unsigned)index;
}
__device__ __forceinline__ float value_at(u64 place) {
    const unsigned ord = ~(unsigned)(place >> kIndexBits);
    return __uint_as_float(ord & 0x80000000u ? ord ^ 0x80000000u : ~ord);
}

struct Row {
    Smem &s;
    cg::cluster_group cl;
    float *values;    // shared memory for the slice,
    const float *x;   // in which it begins
    int lo, n;        // of it
    int vocab;
    unsigned row_at;  // the row's first value, from a 16-byte boundary
    int rank, blocks, tid;
    float top;
    Scale c;

    // Ready for the next histogram, once every block has read what it wants of the last.
    __device__ void zero_histogram() {
        __syncthreads();
        for (int i = tid; i < kBins; i += kThreads) {
            s.count[i] = s.hi[i] = s.lo[i] = 0;
        }
        if (tid == 0) s.own_n = 0;
        __syncthreads();
    }

    __device__ void first_histogram(Kind kind) {
#pragma unroll 4
        for (int i = tid; i < n; i += kThreads) {
            if (kind == kCounts) {
                atomicAdd(&s.count[bin_of(x[i], top, c)], 1u);
            } else {
                unsigned unit;
                const int bin = bin_and_unit(x[i], top, c, unit);
                atomicAdd(&s.lo[bin], unit & 0xffffu);
                atomicAdd(&s.hi[bin], unit >> 16);
                if (kind == kBoth) atomicAdd(&s.count[bin], 1u);
            }
        }
    }

    // The bin of the whole row's histogram in which the elements (or the mass) counted
    // from the start reach `target` >= 1; in every block, with one barrier of the
    // cluster: each tells the others its sums of 32 bins each, and then asks for the 32
    // bins in question. A mass of 0 to be reached stands for `share_of_all` of all, and is
    // put in its place.
    __device__ Found find(Kind kind, bool by_mass, u64 &target, float share_of_all = 0.f) {
        const int lane = tid & 31;
        const bool counts = kind != kFirst, masses = kind != kCounts;
        __syncthreads();
        {  // four bins a thread, eight threads to a sum
            unsigned nc = 0;
            u64 nm = 0;
#pragma unroll
            for (int i = 0; i < kBins / kThreads; ++i) {
                const int bin = tid * (kBins / kThreads) + i;
                if (counts) nc += s.count[bin];
                if (masses) nm += mass_in(kind, bin, s.hi[bin], s.lo[bin]);
            }
            static_assert(kBins / kThreads * 8 == 32, "eight threads to 32 bins");
#pragma unroll
            for (int o = 4; o; o >>= 1) nc += __shfl_xor_sync(~0u, nc, o), nm += __shfl_xor_sync(~0u, nm, o);
            const int to = tid % 8;  // each of them tells one block
            if (to < blocks) {
                Smem *o = cl.map_shared_rank(&s, to);
                if (counts) o->coarse_count[rank][tid / 8] = nc;
                if (masses) o->coarse_mass[rank][tid / 8] = nm;
            }
        }
        cl.sync();
        if (tid < 32) {
            Found f{-1, 0, 0, target};
            look(kind, by_mass, share_of_all, f);
            if (lane == 0) s.found = f;
        }
        __syncthreads();
        target = s.found.target;
        return s.found;
    }

    // find()'s search, by one warp.
    __device__ void look(Kind kind, bool by_mass, float share_of_all, Found &f) const {
        const int lane = tid & 31;
        const bool counts = kind != kFirst, masses = kind != kCounts;
        u64 &target = f.target;
        // 64 sums, two a lane
        unsigned c2[2] = {0, 0};
        u64 m2[2] = {0, 0};
#pragma unroll
        for (int r = 0; r < kMostBlocks; ++r)
            if (r < blocks)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (counts) c2[u] += s.coarse_count[r][2 * lane + u];
                    if (masses) m2[u] += s.coarse_mass[r][2 * lane + u];
                }
        unsigned cb = c2[0] + c2[1];
        u64 mb = m2[0] + m2[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(~0u, cb, o);
            const u64 z = __shfl_up_sync(~0u, mb, o);
            if (lane >= o) cb += y, mb += z;
        }
        if (by_mass) {
            const u64 all = __shfl_sync(~0u, mb, 31);
            // (the bins' masses and their elements' differ in the last bits)
            target = target ? min(target, all) : limit_of(share_of_all, all);
        }
        const unsigned in = __ballot_sync(~0u, (by_mass ? mb : cb) >= target);  // from this lane's sums on it is reached
        if (in == 0) return;
        const int from = __ffs(in) - 1;
        // what lies before that lane's first sum, and whether the first or the second reaches it
        unsigned before = __shfl_sync(~0u, cb - c2[0] - c2[1], from);
        u64 mass_before = __shfl_sync(~0u, mb - m2[0] - m2[1], from);
        const unsigned c_first = __shfl_sync(~0u, c2[0], from);
        const u64 m_first = __shfl_sync(~0u, m2[0], from);
        int sum = 2 * from;
        if (by_mass ? mass_before + m_first < target : before + c_first < target) {
            ++sum;
            before += c_first;
            mass_before += m_first;
        }
        // its 32 bins, one a lane
        const int bin = sum * 32 + lane;
        unsigned count[kMostBlocks], hi[kMostBlocks], lo[kMostBlocks];
#pragma unroll
        for (int r = 0; r < kMostBlocks; ++r) {
            const Smem *o = cl.map_shared_rank(&s, r < blocks ? r : rank);
            count[r] = r < blocks && counts ? o->count[bin] : 0;
            hi[r] = r < blocks && masses ? o->hi[bin] : 0;
            lo[r] = r < blocks && masses ? o->lo[bin] : 0;
        }
        unsigned nc = 0;
        u64 nm = 0;
#pragma unroll
        for (int r = 0; r < kMostBlocks; ++r) nc += count[r], nm += r < blocks && masses ? mass_in(kind, bin, hi[r], lo[r]) : 0;
        cb = nc, mb = nm;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(~0u, cb, o);
            const u64 z = __shfl_up_sync(~0u, mb, o);
            if (lane >= o) cb += y, mb += z;
        }
        const unsigned at = __ballot_sync(~0u, (by_mass ? mass_before + mb : before + cb) >= target);
        if (at == 0) return;
        const int which = __ffs(at) - 1;
        f.bin = sum * 32 + which;
        f.before = before + __shfl_sync(~0u, cb - nc, which);
        f.mass_before = mass_before + __shfl_sync(~0u, mb - nm, which);
    }

    // Mass of one block's bin.
    __device__ u64 mass_in(Kind kind, int bin, unsigned hi, unsigned lo) const {
        if (kind == kFine) return (u64)hi << 32 | lo;
        return bin == kBins - 1 ? 0 : bin_mass(bin, ((u64)hi << 16) + lo, s.bin_power);  // (the last bin's elements weigh nothing)
    }

    // Elements that `in` picks into every block's list, the same in each; how many there
    // are. By way of a list of each block's own elements.
    template <typename In>
    __device__ int gather(In in, bool mass) {
        for (int i0 = tid; i0 < n; i0 += kThreads * 4) {
            float v[4];
            bool is[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = i0 + u * kThreads < n ? x[i0 + u * kThreads] : 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) is[u] = i0 + u * kThreads < n && in(v[u], lo + i0 + u * kThreads);
            if (is[0] || is[1] || is[2] || is[3])
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (is[u]) {
                        const int at = atomicAdd(&s.own_n, 1);
                        if (at < kList) s.own_at[at] = (unsigned short)(i0 + u * kThreads);
                    }
        }
        cl.sync();
        int counts[kMostBlocks], all = 0;
#pragma unroll
        for (int r = 0; r < kMostBlocks; ++r) counts[r] = r < blocks ? cl.map_shared_rank(&s, r)->own_n : 0;
#pragma unroll
        for (int r = 0; r < kMostBlocks; ++r) all += counts[r];
        if (all <= kList) {
            // thread i takes the i-th of the blocks' elements and so on, block after block
            const int slice = (vocab + blocks - 1) / blocks;
            for (int e = tid; e < all; e += kThreads) {
                int at = e, from = -1;
#pragma unroll
                for (int r = 0; r < kMostBlocks; ++r) {
                    if (from < 0 && at < counts[r]) from = r;
                    if (from < 0) at -= counts[r];
                }
                const int i = cl.map_shared_rank(&s, from)->own_at[at];
                // (the slices begin at different places within 16 bytes)
                const float v = cl.map_shared_rank(values, from)[i + (int)((row_at + (unsigned)(from * slice)) & 3)];
                s.list_key[e] = place_of(v, from * slice + i);
                if (mass) s.list_mass[e] = mass_of(v, top, c, s.power);
            }
            __syncthreads();
        }
        return all;
    }

    // Places of the first and the last element that `in` picks.
    template <typename In>
    __device__ void range(In in, u64 &first, u64 &last) {
        u64 a = ~0ull, b = 0;
        for (int i = tid; i < n; i += kThreads)
            if (in(x[i], lo + i)) {
                const u64 p = place_of(x[i], lo + i);
                a = min(a, p), b = max(b, p);
            }
#pragma unroll
        for (int o = 16; o; o >>= 1) a = min(a, __shfl_xor_sync(~0u, a, o)), b = max(b, __shfl_xor_sync(~0u, b, o));
        if ((tid & 31) == 0) s.warp_key[tid >> 5][0] = a, s.warp_key[tid >> 5][1] = b;
        __syncthreads();
        if (tid < blocks) {
            for (int w = 0; w < kWarps; ++w) a = min(a, s.warp_key[w][0]), b = max(b, s.warp_key[w][1]);
            Smem *o = cl.map_shared_rank(&s, tid);
            o->key_of[rank][0] = a, o->key_of[rank][1] = b;
        }
        cl.sync();
        for (int r = 0; r < blocks; ++r) a = min(a, s.key_of[r][0]), b = max(b, s.key_of[r][1]);
        first = a, last = b;
        cl.sync();  // key_of may be written again
    }

    // The listed element at which the count (or mass) reaches `target`: its place to
    // s.cut, the mass up to and with it to s.cut_mass. By this block alone: histograms of
    // the list over places' bits until few are left, which are compared with each other.
    // before, mass_before: of what is not listed.
    __device__ void pick(int count, bool mass, bool by_mass, u64 target, u64 before, u64 mass_before, const float *top_of_list = nullptr) {
        const int lane = tid & 31, warp = tid >> 5;
        u64 a = ~0ull, b = 0;  // the places in question
        for (int e = tid; e < count; e += kThreads) a = min(a, s.list_key[e]), b = max(b, s.list_key[e]);
#pragma unroll
        for (int o = 16; o; o >>= 1) a = min(a, __shfl_xor_sync(~0u, a, o)), b = max(b, __shfl_xor_sync(~0u, b, o));
        if (lane == 0) s.warp_key[warp][0] = a, s.warp_key[warp][1] = b;
        if (tid == 0) s.few_n = 0;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) a = min(a, s.warp_key[w][0]), b = max(b, s.warp_key[w][1]);
        int left = count;
#pragma unroll 1
        while (left > kFew) {
            int shift = 0;
            while ((b - a) >> shift >= kSub) ++shift;
            __syncthreads();
            for (int i = tid; i < kSub; i += kThreads) s.sub_count[i] = 0, s.sub_mass[i] = 0;
            __syncthreads();
            for (int e = tid; e < count; e += kThreads) {
                const u64 p = s.list_key[e];
                if (p < a || p > b) continue;
                atomicAdd(&s.sub_count[(p - a) >> shift], 1u);
                if (mass) atomicAdd(&s.sub_mass[(p - a) >> shift], s.list_mass[e]);
            }
            __syncthreads();
            // two bins a thread
            const unsigned c0 = s.sub_count[2 * tid], c1 = s.sub_count[2 * tid + 1];
            const u64 m0 = s.sub_mass[2 * tid], m1 = s.sub_mass[2 * tid + 1];
            unsigned cs = c0 + c1;
            u64 msum = m0 + m1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(~0u, cs, o);
                const u64 z = __shfl_up_sync(~0u, msum, o);
                if (lane >= o) cs += y, msum += z;
            }
            if (lane == 31) s.warp_count[warp] = cs, s.warp_key[warp][0] = msum;
            __syncthreads();
            u64 cb = before + cs - c0 - c1, mb = mass_before + msum - m0 - m1, all = mass_before;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) cb += s.warp_count[w], mb += s.warp_key[w][0];
                all += s.warp_key[w][0];
            }
            if (by_mass) target = min(target, all);  // (the bins' masses and their elements' differ in the last bits)
            // the bin that reaches it
            const u64 at = by_mass ? mb : cb, n0 = by_mass ? m0 : c0, n1 = by_mass ? m1 : c1;
            if (tid == 0) s.found.bin = -1;
            __syncthreads();
            if (at < target && target <= at + n0) s.found = Found{2 * tid, c0, mb, cb};
            if (at + n0 < target && target <= at + n0 + n1) s.found = Found{2 * tid + 1, c1, mb + m0, cb + c0};
            __syncthreads();
            const Found f = s.found;
            if (f.bin < 0) {  // elements without mass: all of them
                if (tid == 0) s.cut = b, s.cut_mass = mass_before;
                __syncthreads();
                return;
            }
            left = (int)f.before;
            before = f.target;
            mass_before = f.mass_before;
            a += (u64)f.bin << shift;
            b = min(b, a + ((1ull << shift) - 1));
        }
        __syncthreads();
        for (int e = tid; e < count; e += kThreads)
            if (s.list_key[e] >= a && s.list_key[e] <= b) {
                const int at = atomicAdd(&s.few_n, 1);
                if (at < kFew) s.few[at] = e;
            }
        __syncthreads();
        // four threads to an element
        static_assert(kFew * 4 == kThreads, "four threads to an element");
        const int many = min(s.few_n, kFew), e = s.few[min(tid / 4, many - 1)];
        const u64 mine = s.list_key[e], own = mass ? s.list_mass[e] : 0;
        unsigned r = 0;
        u64 mb = 0;
        for (int j = tid % 4; j < many; j += 4) {
            const int o = s.few[j];
            const bool earlier = s.list_key[o] < mine;
            r += earlier;
            if (mass) mb += earlier ? s.list_mass[o] : 0;
        }
#pragma unroll
        for (int o = 2; o; o >>= 1) r += __shfl_xor_sync(~0u, r, o), mb += __shfl_xor_sync(~0u, mb, o);
        if (top_of_list) {
            // the list is the row's beginning: the first `target`, of them those below the share
            const bool there = tid / 4 < many && tid % 4 == 0;
            if (tid == 0) s.cut = 0;
            if (there && r + 1 == target) s.cut_mass = mb + own;
            __syncthreads();
            const u64 limit = mass ? limit_of(*top_of_list, s.cut_mass) : 0;
            if (there && r < target && (!mass || mb < limit)) atomicMax(&s.cut, mine);
            __syncthreads();
            return;
        }
        if (tid / 4 < many && tid % 4 == 0) {
            const bool here = by_mass ? mass_before + mb < target && (target <= mass_before + mb + own || r + 1 == many)
                                      : before + r + 1 == target;
            if (here) s.cut = mine, s.cut_mass = mass_before + mb + own;
        }
        __syncthreads();
    }

    // The element at which the count (or mass) reaches `target`, known to lie in bin
    // f.bin: its place to s.cut, the mass up to and with it to s.cut_mass, in every
    // block.
    __device__ void cut_in(Found f, bool mass, bool by_mass, u64 target) {
        unsigned before = f.before;
        u64 mass_before = f.mass_before, a = 0, b = ~0ull;
        const int bin = f.bin;
        bool whole = true;  // the whole bin, not yet a range of places
        auto in = [&](float v, int i) {
            if (whole) return bin_of(v, top, c) == bin;
            const u64 p = place_of(v, i);
            return p >= a && p <= b;
        };
        int count = gather(in, mass);
        while (count > kList) {
            cl.sync();  // every block has read the count
            if (whole) {
                range(in, a, b);
                whole = false;
            }
            int shift = 0;
            while ((b - a) >> shift >= kBins) ++shift;
            zero_histogram();
            for (int i = tid; i < n; i += kThreads)
                if (in(x[i], lo + i)) {
                    const int at = (int)((place_of(x[i], lo + i) - a) >> shift);
                    atomicAdd(&s.count[at], 1u);
                    if (mass) {
                        const u64 m = mass_of(x[i], top, c, s.power);
                        const unsigned old = atomicAdd(&s.lo[at], (unsigned)m), up = (unsigned)(m >> 32) + (old + (unsigned)m < old);
                        if (up) atomicAdd(&s.hi[at], up);
                    }
                }
            u64 rest = target - (by_mass ? mass_before : before);
            f = find(kFine, by_mass, rest);
            if (f.bin < 0) {  // elements without mass: all of them
                if (tid == 0) s.cut = b, s.cut_mass = mass_before;
                __syncthreads();
                return;
            }
            before += f.before;
            mass_before += f.mass_before;
            a += (u64)f.bin << shift;
            b = min(b, a + ((1ull << shift) - 1));
            count = gather(in, mass);
        }
        pick(count, mass, by_mass, target, before, mass_before);
    }
};

__global__ void __launch_bounds__(kThreads, 2) draw_rows(const __grid_constant__ Args a) {
    extern __shared__ __align__(16) char raw[];
    Smem &s = *reinterpret_cast<Smem *>(raw);
    float *values = reinterpret_cast<float *>(raw + (sizeof(Smem) + 15) / 16 * 16);
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = a.blocks, rank = (int)(blockIdx.x % blocks), V = a.vocab;
    const size_t row = blockIdx.x / blocks, rows = gridDim.x / blocks, request = row / a.per;
    const int slice = (V + blocks - 1) / blocks, lo = min(V, rank * slice), n = min(V, lo + slice) - lo;
    int32_t *st = a.status;
    const Buf bl{a.logits, rows * V * 4}, bn{a.noise, rows * V * 4}, bp{a.probs, rows * V * 4}, bk{a.kept, rows * V * 4};
    cl.barrier_arrive();  // every block of the cluster runs once this has been waited for
    if (tid < kSteps) s.power[tid] = kPowers.v[tid];
    if (tid < kPerOctave) s.bin_power[tid] = kBinPowers.v[tid];
    for (int i = tid; i < kBins; i += kThreads) s.count[i] = s.hi[i] = s.lo[i] = 0;
    if (tid == 0) {
        s.cut = ~0ull, s.cut_mass = 0;
        s.own_n = 0;
    }
    gdndev::pdl_wait();
    gdndev::pdl_launch_dependents();
    // what the request asks for
    const float temperature = a.temperature ? a.temperature[request] : 1.f, top_p = a.top_p ? a.top_p[request] : 1.f;
    float min_p = a.min_p ? a.min_p[request] : 0.f;
    int K = a.top_k ? a.top_k[request] : 0;

    // the slice into shared memory, on the row's place within 16 bytes
    const float *from = a.logits + row * V + lo;
    const int off = (int)(reinterpret_cast<uintptr_t>(from) >> 2 & 3), quads = (n + off + 3) / 4;
    float top = -INFINITY;
    bool bad = false;
    for (int k0 = tid; k0 < quads; k0 += kThreads * 4) {
        float4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = k0 + u * kThreads, e = 4 * k - off;
            v[u] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (k >= quads) continue;
            if (e >= 0 && e + 4 <= n) {
                if (GDN_IN(from + e, 16, bl, st)) v[u] = __ldcs(reinterpret_cast<const float4 *>(from + e));
            } else {
                if (e >= 0 && e < n && GDN_IN(from + e, 4, bl, st)) v[u].x = from[e];
                if (e + 1 >= 0 && e + 1 < n && GDN_IN(from + e + 1, 4, bl, st)) v[u].y = from[e + 1];
                if (e + 2 >= 0 && e + 2 < n && GDN_IN(from + e + 2, 4, bl, st)) v[u].z = from[e + 2];
                if (e + 3 >= 0 && e + 3 < n && GDN_IN(from + e + 3, 4, bl, st)) v[u].w = from[e + 3];
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = k0 + u * kThreads;
            if (k >= quads) break;
            reinterpret_cast<float4 *>(values)[k] = v[u];
            const float t = fmaxf(fmaxf(v[u].x, v[u].y), fmaxf(v[u].z, v[u].w));
            bad |= t == INFINITY || v[u].x != v[u].x || v[u].y != v[u].y || v[u].z != v[u].z || v[u].w != v[u].w;
            top = fmaxf(top, t);
        }
    }
    const float *x = values + off;
    Scale c{3e38f, 0.f};
    if (temperature > 0.f) {
        constexpr float kLog2e = 1.4426950408889634f, kRest = (float)(1.4426950408889634074 - (double)kLog2e);
        const float hi = kLog2e / temperature;
        if (hi < 3e38f) c = {hi, (fmaf(-hi, temperature, kLog2e) + kRest) / temperature};
        if (!(fabsf(c.lo) < 1e38f)) c.lo = 0.f;  // (T of the smallest and the largest)
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) s.warp_f[warp] = top;
    bad = __syncthreads_or(bad);
    if (K <= 0 || K > V) K = V;
    if (min_p > 1.f) K = 1, min_p = 1.f;
    const bool by_count = K < V, by_mass = top_p < 1.f;
    cl.barrier_wait();
    if (tid < blocks) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s.warp_f[w]);
        Smem *o = cl.map_shared_rank(&s, tid);
        o->f_of[rank] = top;
        o->bad_of[rank] = bad;
    }
    // a limited count looks for its bin with counts alone: with few elements above, no more is needed
    const Kind kind = by_count ? kCounts : kFirst;
    cl.sync();
    top = s.f_of[0], bad = s.bad_of[0];
    for (int k = 1; k < blocks; ++k) top = fmaxf(top, s.f_of[k]), bad |= s.bad_of[k] != 0;
    bad |= top == -INFINITY;
    Row r{s, cl, values, x, lo, n, V, (unsigned)(reinterpret_cast<uintptr_t>(a.logits + row * V) >> 2 & 3), rank, blocks, tid, top, c};

    u64 cut = ~0ull;  // the last place that is kept
    if (!bad && (by_count || by_mass)) {
        r.first_histogram(kind);
        bool done = false;
        u64 whole = 0;  // the mass of the first K
        if (by_count) {
            u64 nth = (u64)K;
            const Found f = r.find(kCounts, false, nth);
            // all above the bin's end, where that is little enough to be ranked
            const int count = f.bin >= 0 && K <= kList ? r.gather([&](float v, int) { return bin_of(v, top, c) <= f.bin; }, by_mass) : kList + 1;
            if (count <= kList) {
                // few: both cuts in one go
                r.pick(count, by_mass, false, nth, 0, 0, count <= kFew ? &top_p : nullptr);
                if (by_mass && count > kFew) r.pick(count, true, true, limit_of(top_p, s.cut_mass), 0, 0);
                done = true;
            } else if (f.bin >= 0) {
                cl.sync();  // every block has read the list's count
                Found g = f;
                if (by_mass) {
                    r.zero_histogram();
                    r.first_histogram(kBoth);
                    g = r.find(kBoth, false, nth);
                } else {
                    if (tid == 0) s.own_n = 0;
                    __syncthreads();
                }
                r.cut_in(g, by_mass, false, nth);
                whole = s.cut_mass;
                done = !by_mass;
            } else {
                done = true;  // (K elements there are: not reached)
            }
            if (f.bin >= 0) cut = s.cut;
        }
        if (by_mass && !done) {
            if (by_count) {
                // the histogram may have been cut finer since, and the others may still read its list
                cl.sync();
                r.zero_histogram();
                r.first_histogram(kFirst);
            }
            u64 limit = by_count ? limit_of(top_p, whole) : 0;
            const Found f = r.find(kFirst, true, limit, top_p);
            if (f.bin >= 0) {
                r.cut_in(f, true, true, limit);
                cut = s.cut;
            }
        }
    }

    // the kept weights' sum and the largest weight / noise
    const float cut_x = cut == ~0ull ? -INFINITY : value_at(cut);
    const int cut_i = cut == ~0ull ? V : (int)(cut & ((1u << kIndexBits) - 1));
    const u64 min_mass = min_p > 0.f ? (u64)ceil((double)min_p * (double)(1ull << kMassBits)) : 0;
    auto kept = [&](float v, int i, float w) {
        if (!(v > cut_x || (v == cut_x && i <= cut_i))) return false;
        if (!(min_p > 0.f)) return true;
        // next to the border the 44-bit weight decides
        if (fabsf(w - min_p) > 1e-5f * min_p) return w > min_p;
        return mass_of(v, top, c, s.power) >= min_mass;
    };
    float sum = 0.f;
    u64 best = 0;
    float best_x = 0.f;
    const float *noise = a.noise ? a.noise + row * V + lo : nullptr;
    auto offer = [&](int i, float v, float w, float e) {
        const u64 key = make_key(__fdividef(w, e), (unsigned)(lo + i));
        if (key > best) best = key, best_x = v;
    };
    if (tid == 0) s.kept_n = 0;
    __syncthreads();
    // Where the cut leaves few of the row (by what its last element weighs, some thousand
    // at most), their noise is read for a list of them, all at once: with the scan it
    // would be waited for again and again. Where it leaves many, or all, it is read with
    // the scan, eight at a time (a list first took 10 us more for rows of which thousands
    // are kept).
    const float last = cut == ~0ull ? 0.f : weight(cut_x, top, c);
    const bool few = by_mass ? (float)s.cut_mass <= 4.f * kList * (float)(1ull << kMassBits) * last
                             : by_count ? K <= 4 * kList : min_p * 4.f * kList >= 1.f;
    if (!bad && few) {
#pragma unroll 4
        for (int i = tid; i < n; i += kThreads) {
            const float v = x[i];
            if (!(v >= cut_x)) continue;
            const float w = weight(v, top, c);
            if (!kept(v, lo + i, w)) continue;
            sum += w;
            if (!noise || !(w > 0.f)) continue;
            const int at = atomicAdd(&s.kept_n, 1);
            if (at < kList)
                s.list_key[at] = (u64)__float_as_uint(w) << 32 | (unsigned)i;
            else
                offer(i, v, w, GDN_IN(noise + i, 4, bn, st) ? noise[i] : 1.f);
        }
        __syncthreads();
        for (int l = tid; l < min(s.kept_n, kList); l += kThreads) {
            const u64 k = s.list_key[l];
            const int i = (int)(unsigned)k;
            offer(i, x[i], __uint_as_float((unsigned)(k >> 32)), GDN_IN(noise + i, 4, bn, st) ? noise[i] : 1.f);
        }
    } else if (!bad) {
        for (int i0 = tid; i0 < n; i0 += kThreads * 8) {
            float v[8], e[8];
            bool in[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int i = i0 + u * kThreads;
                v[u] = i < n ? x[i] : -INFINITY;
                in[u] = i < n && v[u] >= cut_x;
                e[u] = in[u] && noise && GDN_IN(noise + i, 4, bn, st) ? noise[i] : 1.f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (!in[u]) continue;
                const int i = i0 + u * kThreads;
                const float w = weight(v[u], top, c);
                if (!kept(v[u], lo + i, w)) continue;
                sum += w;
                if (noise && w > 0.f) offer(i, v[u], w, e[u]);
            }
        }
    }
    const u64 mine = best;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(~0u, sum, o);
        const u64 y = __shfl_xor_sync(~0u, best, o);
        best = max(best, y);
    }
    if (lane == 0) s.warp_f[warp] = sum, s.warp_key[warp][0] = best;
    __syncthreads();
    if (tid < blocks) {
        sum = 0.f, best = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s.warp_f[w], best = max(best, s.warp_key[w][0]);
        Smem *o = cl.map_shared_rank(&s, tid);
        o->sum_of[rank] = sum;
        o->key_of[rank][0] = best;
    }
    cl.sync();  // the last access to another block's shared memory
    sum = 0.f, best = 0;
    for (int k = 0; k < blocks; ++k) sum += s.sum_of[k], best = max(best, s.key_of[k][0]);
    const float inv = 1.f / sum;
    if (a.token) {
        if (bad || best == 0) {
            if (rank == 0 && tid == 0) {
                a.token[row] = 0;
                if (a.token_prob) a.token_prob[row] = kNan;
            }
        } else if (mine == best) {
            a.token[row] = (int)gdndev::key_index(best);
            if (a.token_prob) a.token_prob[row] = weight(best_x, top, c) * inv;
        }
    }
    if (bad && rank == 0 && tid == 0 && st) atomicOr(st, GDN_DEV_NAN_LOGIT);
    if (a.probs) {
        float *to = a.probs + row * V + lo;
#pragma unroll 4
        for (int i = tid; i < n; i += kThreads) {
            float w = 0.f;
            if (bad) {
                w = kNan;
            } else if (x[i] >= cut_x) {
                w = weight(x[i], top, c);
                w = kept(x[i], lo + i, w) ? w * inv : 0.f;
            }
            if (GDN_IN(to + i, 4, bp, st)) to[i] = w;
        }
    }
    if (a.kept) {
        float *to = a.kept + row * V + lo;
        for (int i = tid; i < n; i += kThreads) {
            const bool in = bad || (x[i] >= cut_x && kept(x[i], lo + i, min_p > 0.f ? weight(x[i], top, c) : 0.f));
            if (GDN_IN(to + i, 4, bk, st)) to[i] = in ? x[i] : -INFINITY;
        }
    }
}

bool overlap(const void *a, const void *b, size_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + bytes && y < x + bytes;
}

// Blocks of a row's cluster.
int blocks_of(int vocab) { return vocab <= 4096 ? 1 : kMostBlocks; }

constexpr size_t smem_of(int vocab, int blocks) {
    return (sizeof(Smem) + 15) / 16 * 16 + ((size_t)(vocab + blocks - 1) / blocks + 8) * 4;
}
static_assert(smem_of(GDN_MAX_SAMPLE_VOCAB, kMostBlocks) <= 227 * 1024, "shared memory of a block");
static_assert((GDN_MAX_SAMPLE_VOCAB + kMostBlocks - 1) / kMostBlocks <= 65536, "a bin's lower halves in 32 bits");

}  // namespace

extern "C" int spec_sample(int32_t rows, int32_t vocab, int32_t rows_per_request, const float *logits,
                           const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                           const float *noise, int32_t *token, float *token_prob, float *probs, float *kept_logits,
                           int32_t *dev_status, gdn_stream_t stream) {
    if (rows < 1 || rows > 1 << 20 || vocab < 1 || vocab > GDN_MAX_SAMPLE_VOCAB || rows_per_request < 1) return GDN_ERR_DIMS;
    if (!logits || (token && !noise) || (token_prob && !token) || (!token && !probs && !kept_logits)) return GDN_ERR_NULL;
    for (const void *p : {(const void *)logits, (const void *)temperature, (const void *)top_k, (const void *)top_p,
                          (const void *)min_p, (const void *)noise, (const void *)token, (const void *)token_prob,
                          (const void *)probs, (const void *)kept_logits, (const void *)dev_status})
        if (!gdnhost::aligned_to(p, 4)) return GDN_ERR_ALIGN;
    const size_t bytes = (size_t)rows * vocab * 4;
    if (overlap(probs, logits, bytes) || overlap(probs, noise, bytes) || overlap(probs, kept_logits, bytes) ||
        overlap(kept_logits, noise, bytes) || (kept_logits != logits && overlap(kept_logits, logits, bytes)))
        return GDN_ERR_OVERLAP;
    const int blocks = blocks_of(vocab);
    const size_t smem = smem_of(vocab, blocks);
    static size_t allowed[256] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return GDN_ERR_CUDA;
    if (allowed[dev] == 0) {
        const size_t most = smem_of(GDN_MAX_SAMPLE_VOCAB, kMostBlocks);
        if (cudaFuncSetAttribute(draw_rows, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess)
            return GDN_ERR_CUDA;
        allowed[dev] = most;
    }
    const Args a{vocab, rows_per_request, blocks, logits, temperature, top_k, top_p, min_p, noise,
                 token, token_prob, probs, kept_logits, dev_status};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows * blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, draw_rows, a) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
