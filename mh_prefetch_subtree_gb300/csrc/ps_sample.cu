// Drawing a token of each row from its truncated distribution (ps_sample_rows), and scoring
// given tokens under the same truncation (ps_score_rows_truncated).
//
// Order a row's ids by (logit, then lowest id).  With M the largest logit and
// w = 2^y, y = (l - M) log2 e / tau, every cut leaves a prefix of that order: min-p the ids
// with w >= min_p, top-k the first k of them, top-p the shortest prefix that holds p of
// what is left.  The draw is the shortest prefix that holds u of the kept mass Z: its last
// id.  So all questions are "where does the running mass (or count) of the sorted row reach
// a value", and nothing is sorted:
//   the pass   one read of the row makes a histogram of the logits by their leading bits
//              (sign, exponent, 7 bits: all of a bfloat16), 4096 bins from 64 max(tau, 1) down;
//   the bins   a bin of a bfloat16 row is one value, so its mass is its count times that
//              value's w, and log p0 and the entropy come from the counts as well.  Running
//              sums down the bins answer the questions.  Where a bin holds more than one
//              value (float32 rows, values next to zero) its few elements are gathered and
//              settled one by one;
//   the id     the row is read again, from L2, for the nth element of the drawn value.
// A row whose values lie outside the bins (|M| far above tau, say) is passed over a second
// time, with bins that start at M and the elements below min-p left out.
//
// Masses are integers, 2^43 to 2^45 for a mass of 1, so their sums are exact and do not
// depend on the order of the additions: the same row and number give the same token
// however the row is divided.  w is formed from y in two floats to about 2^-31 of itself, and
// a bin of several values (float32 rows, values around zero) adds weights of 28 bits below
// its largest value's: up to 2^-27 of an element at the lower end of a bin that is two units of y
// wide, the widest.  A token differs from that of a float64 evaluation only where u Z lies that
// close to a border between two ids, or to the 2^-43 or so by which each id's mass is rounded;
// a cut or a number that divides equal largest ids by a whole number finds that number of them.
//
// A row is one block's, or with few rows a cluster's: its blocks each read a part, and the
// first adds up their bins.
//
// What bounds it: no unit is full.  A warp's 32 additions go to random banks, which takes four
// turns of shared memory.  Of many bfloat16 rows scored these turns are 58% of the cycles, and
// issue slots 54% (4,000 x 151936: 440 to 460 us, 2.7 TB/s); drawn, with a second reading, 49% and 45%
// (700 x 262144: 187 us).  The rest are passes and chains of small steps that do not overlap.
// float32 rows take three additions an element, a weight for each and two or three more
// readings: turns 29%, issue slots 60% (777 x 50021: 194 us; 1216 x 151936: 795 us, drawn 935).
// For few rows: the chain of small steps after the pass, about 12 us of the 25 that 16 rows of
// 151936 take.  Measured and not kept: the row held in
// the shared memory of a cluster, with the maximum found first (4,000 rows 1,197 us); logits
// more than 10 tau below the largest summed by exponentials and not counted (445 to 540);
// copies through a ring in shared memory (500); one 64-bit addition for a float32 element's
// count and weight, which is a loop of comparisons there (246 us where three take 201).
#include "ps_sample.cuh"

#include <algorithm>

#include <cuda_bf16.h>

namespace ps {
namespace {

constexpr int kMostT = 512, kMostWarps = kMostT / 32;
constexpr int kBins = 4096;
constexpr int kHalfBins = kBins / 2;
constexpr int kTop = kHalfBins - 1;              // the place of the first bin, in the first pass
constexpr int kLastBin = kBins - 3;              // its last; what lies further is not counted
constexpr int kMostBlocks = 8;
constexpr int kList = 256;                      // at most as many as a block has threads
constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = (float)(1.4426950408889634074 - (double)kLog2e);
constexpr float kLn2f = 0.69314718f;
constexpr double kLn2 = 0.6931471805599453094;
// y below this has no part in a row's masses: 2^20 such ids weigh less than 2^-44 of Z.
constexpr float kWindow = 64.f;
constexpr float kInf = __builtin_huge_valf();

// 2^(j/64) by 62 fractional bits, from six square roots of 2 (Newton's iteration).
struct PowTable {
    uint64_t t[64];
    static constexpr double root(double x) {
        double r = x;
        for (int i = 0; i < 40; ++i) r = 0.5 * (r + x / r);
        return r;
    }
    constexpr PowTable() : t{} {
        double f[6] = {};
        double r = 2.0;
        for (int i = 5; i >= 0; --i) f[i] = r = root(r);      // f[i] = 2^(2^i / 64)
        for (int j = 0; j < 64; ++j) {
            double x = 1.0;
            for (int i = 0; i < 6; ++i)
                if (j >> i & 1) x *= f[i];
            t[j] = (uint64_t)(x * 4611686018427387904.0);
        }
    }
};
__constant__ PowTable kPow = PowTable();

struct Result {                  // of a question: the element that ends the prefix
    uint64_t before;             // mass of what comes before it
    uint64_t end;                // and with it
    uint32_t key;                // of its logit
    uint32_t nth;                // 1: the first of its value
    int32_t id;                  // or -1: the nth of its value
    uint32_t count;              // elements before it
    uint32_t equal;              // elements of its value
};

enum Kind : uint32_t { kDone, kCount, kGather, kLocate, kAgain };
struct Command {
    uint32_t kind, klo, khi;     // kAgain: klo is M's key
    int32_t below;               // kCount: only ids below this, if >= 0; kLocate: the block
    uint32_t nth;                // kLocate; M's key where something is counted or gathered
};

// What a block says about its part of the row.
struct Part {
    uint32_t top_key;            // of its largest logit; all ones: a NaN or +inf
    uint32_t maxima;             // how many
    float sum, ent;              // of e and e y over the others
};

struct Shared {
    uint32_t bins[kBins];
    uint64_t pow[64];
    uint64_t scan[kMostWarps];
    uint32_t scan_n[kMostWarps], scan_k[kMostWarps];
    float scan_f[2][kMostWarps];
    float lnp[2];                                 // tau ln(min_p), as two floats
    // bfloat16: the limbs of the bin around zero; its sums of e^l and l log2 e e^l for log p0, by 23 and 28 bits
    uint32_t near0[4];
    // written by the cluster's blocks, read by the first
    Part part[kMostBlocks];
    uint64_t mass[kMostBlocks];
    uint32_t count[kMostBlocks], least[kMostBlocks], most[kMostBlocks];
    Command cmd;
    // the first block's
    uint64_t near0_all;
    float near0_sum, near0_ent;
    uint32_t n_list;                              // in the first pass every block's: values around zero
    int at;
    Result res;
    uint2 list[kList];                            // key, id
    uint64_t list_w[kList];
};

__device__ __forceinline__ uint32_t block_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t n_blocks() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void sync_cluster() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `p` in the shared memory of the cluster's block `rank`.
__device__ __forceinline__ uint32_t at_block(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void put(uint32_t a, uint32_t x) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ void put(uint32_t a, uint64_t x) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(x) : "memory");
}
__device__ __forceinline__ uint32_t get(uint32_t a) {
    uint32_t x;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ uint4 get4(uint32_t a) {
    uint4 x;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ uint32_t add_at(uint32_t a, uint32_t x) {
    uint32_t was;
    asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(was) : "r"(a), "r"(x) : "memory");
    return was;
}

// Floats as integers that rise with them; -0 is 0.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// One more in a bin, by its address.
__device__ __forceinline__ void add_one(uint32_t at) {
    asm volatile("red.shared::cta.add.u32 [%0], 1;" ::"r"(at));
}

// What a row's elements are measured by.
struct Scale {
    float M;                     // the largest logit
    float lo;                    // elements below it are left out
    float gh, gl;                // log2 e / tau
    int shift;                   // of a float's bits to its code
    int32_t zero, top;           // the code up to which values are "around zero"; the first bin's place
    int bits;                    // of a mass of 1
};

// The place of a value in the order of codes: 0 around zero, rising with the value.
__device__ __forceinline__ int32_t place(float x, const Scale &s) {
    const int32_t b = __float_as_int(x), sign = b >> 31;
    const int32_t c = max((int32_t)((uint32_t)(b & 0x7fffffff) >> s.shift) - s.zero, 0);
    return (c ^ sign) - sign;
}
// A value above the first bin has none either: the result is then large.
__device__ __forceinline__ uint32_t bin_of(float x, const Scale &s) { return (uint32_t)(s.top - place(x, s)); }
// The least and the largest value of a bin.
__device__ __forceinline__ float bin_most(int bin, const Scale &s) {
    const int32_t r = s.top - bin;
    return r >= 0 ? __int_as_float((int32_t)((uint32_t)(r + s.zero + 1) << s.shift) - 1)
                  : -__int_as_float((-r + s.zero) << s.shift);
}
__device__ __forceinline__ float bin_least(int bin, const Scale &s) {
    const int32_t r = s.top - bin;
    return r > 0 ? __int_as_float((r + s.zero) << s.shift)
                 : -__int_as_float((int32_t)((uint32_t)(-r + s.zero + 1) << s.shift) - 1);
}
// The one value of a bfloat16 row's bin other than the one around zero.
__device__ __forceinline__ float bin_value(int bin, const Scale &s) { return s.top > bin ? bin_least(bin, s) : bin_most(bin, s); }

// Where a bin's count is.  The first pass has positive values from 0 up and negative ones
// from kHalfBins up, each by its distance from zero.
__device__ __forceinline__ int bin_slot(int bin, bool linear) {
    return linear ? bin : bin <= kTop ? kTop - bin : bin + 1;
}

// 2^y by `bits` fractional bits, y as a sum of two floats, the second small.
__device__ __forceinline__ uint64_t pow2_fixed(float yh, float yl, int bits, const uint64_t *table) {
    const float step = rintf(yh * 64.f);
    const float r = fmaf(step, -0.015625f, yh) + yl;           // the difference is exact
    const int k = (int)step;
    // 2^r - 1 by its series, |r| < 2^-6.9: the next term is below 2^-38
    const float q = r * fmaf(r, fmaf(r, fmaf(r, 0.009618129f, 0.055504109f), 0.24022651f), 0.69314718f);
    const uint64_t t = table[k & 63];
    const uint64_t m = t + (uint64_t)((int64_t)(t >> 31) * (int64_t)__float2int_rn(q * 274877906944.f) >> 7);   // 2^38
    const int down = 62 - bits - (k >> 6);
    return down > 63 ? 0 : (m + ((uint64_t)1 << (down - 1))) >> down;
}
// l - ref in units of y, as two floats.
__device__ __forceinline__ void exponent(float l, float ref, const Scale &s, float *yh, float *yl) {
    const float d = l - ref, b = d - l;
    const float e = (l - (d - b)) + (-ref - b);                // l - ref = d + e exactly
    *yh = d * s.gh;
    *yl = fmaf(d, s.gh, -*yh) + fmaf(d, s.gl, e * s.gh);
}
// The reference of the bin of a code that holds several values, where b is one of them or the
// bin's largest: the largest value itself.
__device__ __forceinline__ float bin_ref(float l, const Scale &s) {
    const int32_t b = __float_as_int(l), mask = (1 << s.shift) - 1;
    int32_t r = b >= 0 ? b | mask : b & ~mask;
    if ((int32_t)((uint32_t)(b & 0x7fffffff) >> s.shift) <= s.zero) r = (s.zero << s.shift) | mask;
    return __int_as_float(r);
}
// w relative to the reference's by 28 bits, to be added up in two limbs of 14:
// the 2^18 elements that a part of a row has at most add up to less than 2^32 (the parts of a
// cluster's blocks do not, and are added up in 64 bits).  l - ref is exact, or next to zero as good as.
__device__ __forceinline__ uint32_t limbs(float l, float ref, const Scale &s, const uint64_t *table) {
    const float d = l - ref, h = d * s.gh;
    return min((uint32_t)pow2_fixed(h, fmaf(d, s.gh, -h) + d * s.gl, 28, table), (1u << 28) - 1);
}

// w, as a mass.
__device__ __forceinline__ uint64_t mass_at(float l, const Scale &s, const uint64_t *table) {
    float h, e;
    exponent(l, s.M, s, &h, &e);
    return h > -(float)s.bits - 2.f ? pow2_fixed(h, e, s.bits, table) : 0;
}
// The mass of an element of a bin of several values, whose reference has the mass w: the share of it that
// the element's weight is, rounded up.  So no bin has more mass than its elements, and equal
// elements have equal shares of theirs: a cut or a number which divides them by a whole
// number (half of two) finds that number of them.
__device__ __forceinline__ uint64_t mass_in(float l, float ref, uint64_t w, const Scale &s, const uint64_t *table) {
    const uint64_t m = limbs(l, ref, s, table), low = w * m;
    return (__umul64hi(w, m) << 36 | low >> 28) + ((low & ((1u << 28) - 1)) != 0);
}
template <bool HALF>
__device__ __forceinline__ uint64_t mass_of(float l, const Scale &s, const uint64_t *table) {
    if (!(l >= s.lo)) return 0;
    const bool one = HALF && (int32_t)((__float_as_uint(l) & 0x7fffffffu) >> 16) > s.zero;
    const float ref = one ? l : bin_ref(l, s);
    const uint64_t w = mass_at(ref, s, table);
    return one ? w : mass_in(l, ref, w, s, table);
}

// ln(m 2^-scale), m > 0, to about 2^-30: an estimate x and how far m e^-x is from 1.
__device__ __forceinline__ double ln_of(uint64_t m, int scale, const uint64_t *table) {
    const int z = __clzll((long long)m);
    m <<= z;                                                   // 63 fractional bits: 1 .. 2
    const float x = __logf((float)(m >> 32) * 0x1p-31f);
    const float yh = -x * kLog2e, yl = fmaf(-x, kLog2e, -yh) - x * kLog2eLow;
    const int64_t off = (int64_t)(__umul64hi(m, pow2_fixed(yh, yl, 61, table)) - ((uint64_t)1 << 60));
    const float r = (float)off * 0x1p-60f;
    return (double)x + (double)fmaf(-0.5f * r, r, r) + (double)(63 - z - scale) * kLn2;
}
// ceil(x m / 2^down) of a product that may need 128 bits; at least 1.
__device__ __forceinline__ uint64_t scaled(uint64_t x, uint64_t m, int down) {
    const uint64_t hi = __umul64hi(x, m), lo = x * m;
    if (down >= 128) return 1;
    if (down >= 64) {
        const int d = down - 64;
        const bool more = lo != 0 || (d && (hi << (64 - d)) != 0);
        return max((hi >> d) + more, (uint64_t)1);
    }
    return max((hi << (64 - down) | lo >> down) + ((lo << (64 - down)) != 0), (uint64_t)1);
}
// The least mass that is at least u of m, 0 < u <= 1.
__device__ __forceinline__ uint64_t share_of(double u, uint64_t m) {
    const uint64_t b = (uint64_t)__double_as_longlong(u);
    const int e = max((int)(b >> 52), 1);
    return scaled((b & 0xfffffffffffffull) | (b >> 52 ? (uint64_t)1 << 52 : 0), m, 1075 - e);
}
__device__ __forceinline__ uint64_t share_of(float u, uint64_t m) {
    const uint32_t b = __float_as_uint(u);
    const int e = max((int)(b >> 23), 1);
    return scaled((b & 0x7fffffu) | (b >> 23 ? 1u << 23 : 0u), m, 150 - e);
}

__device__ __forceinline__ uint64_t shfl_up64(uint64_t x, int d) { return __shfl_up_sync(0xffffffffu, (unsigned long long)x, d); }
__device__ __forceinline__ uint64_t shfl64(uint64_t x, int lane) { return __shfl_sync(0xffffffffu, (unsigned long long)x, lane); }
__device__ __forceinline__ uint64_t warp_sum64(uint64_t x) {
#pragma unroll
    for (int d = 16; d; d /= 2) x += __shfl_xor_sync(0xffffffffu, (unsigned long long)x, d);
    return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// A row, or one block's part of it.
template <typename ElemT, bool ENT>
struct Row {
    static constexpr bool kHalf = sizeof(ElemT) == 2;
    static constexpr int kPer = 16 / sizeof(ElemT);
    // Blocks of a multiprocessor take turns in their passes and in the chains of small steps
    // after them.  4,000 x 151,936 bfloat16 rows scored take 457 us with five blocks of 256
    // threads, 477 with four, 560 with two of 512, 546 with eight of 128; 777 x 50,021 float32
    // rows 226 us with two of 512 and 307 with five of 256.
    static constexpr int kT = kHalf ? 256 : 512, kResident = kHalf ? 5 : 2;
    static constexpr int kWarps = kT / 32, kBinsThread = kBins / kT;
    Shared &sh;
    uint32_t *limb;              // float32: [2][kBins], a bin's sum of weights in two limbs
    const uint4 *vecs;
    int32_t V, n_vecs, id0;      // of the part; id of its first element
    uint32_t rank, blocks;
    Scale s;

    __device__ __forceinline__ static void floats(const uint4 &v, float (&x)[kPer]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kHalf) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                x[i] = __uint_as_float(w[i]);
            }
        }
    }
    // Elements from V on become -inf.
    __device__ __noinline__ uint4 cut(uint4 v, int j) const {
        const int over = id0 + (j + 1) * kPer - V;
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kHalf) {
                const int n = kPer - over - 2 * i;             // of this word's two that stay
                if (n <= 0) w[i] = 0xff80ff80u;
                else if (n == 1) w[i] = (w[i] & 0xffffu) | 0xff800000u;
            } else if (i >= kPer - over) {
                w[i] = 0xff800000u;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ uint4 load(int j) const {
        const uint4 v = __ldg(vecs + j);
        return id0 + (j + 1) * kPer > V ? cut(v, j) : v;
    }

    // All of a thread's vectors, several loads at a time.
    template <typename F>
    __device__ __forceinline__ void each(F &&f) const {
        constexpr int kAhead = 4;
        int j = threadIdx.x;
        for (; j + (kAhead - 1) * kT < n_vecs - 1; j += kAhead * kT) {
            uint4 v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) v[i] = __ldg(vecs + j + i * kT);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) f(v[i], j + i * kT);
        }
        for (; j < n_vecs; j += kT) f(load(j), j);
    }

    // --- the pass ---

    // Equal neighbours (a row of zeros, say) are added up by their thread, as one address takes
    // one lane's number at a time.
    struct Run {
        int slot = -1;
        uint32_t n = 0, hi = 0, low = 0;
    };
    __device__ __forceinline__ void flush(Run &run) {
        if (run.n) {
            atomicAdd(&sh.bins[run.slot], run.n);
            atomicAdd(kHalf ? &sh.near0[0] : limb + run.slot, run.hi);
            atomicAdd(kHalf ? &sh.near0[1] : limb + kBins + run.slot, run.low);
        }
        run = Run();
    }
    __device__ __forceinline__ static void add(Run &run, uint32_t m) { ++run.n, run.hi += m >> 14, run.low += m & 16383u; }
    // A float32 vector's elements by their slots; -1: none.
    __device__ __forceinline__ void put4(const int (&at)[4], const float (&f)[kPer], Run &run) {
        if (at[0] == at[1] && at[1] == at[2] && at[2] == at[3]) {
            if (at[0] < 0) return;
            if (at[0] != run.slot) {
                flush(run);
                run.slot = at[0];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) add(run, limbs(f[i], bin_ref(f[i], s), s, sh.pow));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (at[i] >= 0) {
                    const uint32_t m = limbs(f[i], bin_ref(f[i], s), s, sh.pow);
                    atomicAdd(&sh.bins[at[i]], 1u);
                    atomicAdd(limb + at[i], m >> 14);
                    atomicAdd(limb + kBins + at[i], m & 16383u);
                }
        }
    }
    // Elements around zero of a bfloat16 vector.
    __device__ __forceinline__ void near_zero(const float (&f)[kPer], Run &run) {
#pragma unroll 1
        for (int i = 0; i < kPer; ++i) {
            float x = 0.f;
#pragma unroll
            for (int q = 0; q < kPer; ++q) x = i == q ? f[q] : x;
            if ((__float_as_uint(x) & 0x7fffffffu) >> 16 <= (uint32_t)s.zero && x >= s.lo)
                add(run, limbs(x, bin_ref(x, s), s, sh.pow));
        }
    }
    // A vector's elements into the bins of the first pass; `most` of bfloat16: the largest codes.
    __device__ __forceinline__ void count_first(const uint4 &v, uint32_t &most, Run &run) {
        const uint32_t bins_at = smem_addr(sh.bins);
        if constexpr (kHalf) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            const uint32_t minus_zero2 = (uint32_t)(-s.zero & 0xffff) * 0x10001u;
            uint32_t code[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                code[i] = w[i] & 0x7fff7fffu;
                // the distance from zero, in the half of the bins that the sign says
                const uint32_t t = __viaddmin_s16x2_relu(code[i], minus_zero2, (uint32_t)kTop * 0x10001u);
                const uint32_t at2 = t | (w[i] >> 4 & 0x08000800u);
                // halves to addresses by products, which leave the pipe of logic and shifts alone
                add_one(__dp2a_lo(at2, 0x0004u, bins_at));
                add_one(__dp2a_lo(at2, 0x0400u, bins_at));
            }
            const uint32_t near = __vimin3_u16x2(code[0], code[1], __viaddmin_u16x2(code[2], 0u, code[3]));
            most = __vimax3_u16x2(most, code[0], code[1]);
            most = __vimax3_u16x2(most, code[2], code[3]);
            if ((near & 0xffffu) <= (uint32_t)s.zero || near >> 16 <= (uint32_t)s.zero) {
                // kept for later
#pragma unroll 1
                for (int i = 0; i < kPer; ++i) {
                    uint32_t word = w[0];
                    word = i / 2 == 1 ? w[1] : i / 2 == 2 ? w[2] : i / 2 == 3 ? w[3] : word;
                    const float x = __uint_as_float(i & 1 ? word & 0xffff0000u : word << 16);
                    if ((__float_as_uint(x) & 0x7fffffffu) >> 16 <= (uint32_t)s.zero) {
                        const uint32_t slot = atomicAdd(&sh.n_list, 1u);
                        if (slot < kList) sh.list[slot].x = __float_as_uint(x);
                    }
                }
            }
        } else {
            float f[kPer];
            int at[4];
            floats(v, f);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const uint32_t b = __float_as_uint(f[i]);
                const int32_t t = min(max((int32_t)((b & 0x7fffffffu) >> 16) - s.zero, 0), kTop);
                at[i] = t < kTop ? (int)((uint32_t)t | (b >> 31) * kHalfBins) : -1;      // a last bin is not used
            }
            put4(at, f, run);
        }
    }
    // The same into bins down from M's, of which those below `end` (< kBins) are counted; of
    // bfloat16 the one around zero by the run.
    __device__ __forceinline__ void count_second(const float (&f)[kPer], uint32_t end, Run &run) {
        if constexpr (kHalf) {
            bool near = false;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const uint32_t bin = bin_of(f[i], s);
                const bool zero = bin == (uint32_t)s.top;
                if (bin < end && f[i] >= s.lo && !zero) atomicAdd(&sh.bins[bin], 1u);
                near = near || zero;
            }
            if (near) near_zero(f, run);
        } else {
            int at[4];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const uint32_t bin = bin_of(f[i], s);
                at[i] = bin < end && f[i] >= s.lo ? (int)bin : -1;
            }
            put4(at, f, run);
        }
    }
    __device__ __forceinline__ void clear() {
        uint4 *z = reinterpret_cast<uint4 *>(sh.bins);
        for (int i = threadIdx.x; i < kBins / 4; i += kT) z[i] = make_uint4(0, 0, 0, 0);
        if constexpr (!kHalf) {
            z = reinterpret_cast<uint4 *>(limb);
            for (int i = threadIdx.x; i < 2 * kBins / 4; i += kT) z[i] = make_uint4(0, 0, 0, 0);
        }
        if (threadIdx.x < 4) sh.near0[threadIdx.x] = 0;
        if (threadIdx.x == 0) sh.n_list = 0;
    }
    // Sums over the block, to the first block.
    __device__ __forceinline__ void report(uint32_t top_key, uint32_t maxima, float sum, float ent) {
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
        maxima = __reduce_add_sync(0xffffffffu, maxima);
        sum = warp_sum(sum);
        if (ENT) ent = warp_sum(ent);
        if (lane == 0) sh.scan_n[wid] = maxima, sh.scan_f[0][wid] = sum, sh.scan_f[1][wid] = ent;
        __syncthreads();
        if (wid == 0) {
            maxima = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.scan_n[lane] : 0u);
            sum = warp_sum(lane < kWarps ? sh.scan_f[0][lane] : 0.f);
            if (ENT) ent = warp_sum(lane < kWarps ? sh.scan_f[1][lane] : 0.f);
            if (lane == 0) {
                const uint32_t a = at_block(&sh.part[rank], 0);
                put(a, top_key);
                put(a + 4, maxima);
                put(a + 8, __float_as_uint(sum));
                put(a + 12, __float_as_uint(ent));
            }
        }
    }
    // The largest of the threads' keys.
    __device__ __forceinline__ uint32_t block_max(uint32_t key) {
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
        key = __reduce_max_sync(0xffffffffu, key);
        if (lane == 0) sh.scan_k[wid] = key;
        __syncthreads();
        return __reduce_max_sync(0xffffffffu, lane < kWarps ? sh.scan_k[lane] : 0u);
    }

    // The first pass: M is not known yet.  Of float32 rows it also sums e = 2^(l log2 e); those
    // that will be passed over again for their min-p are not counted.
    __device__ __forceinline__ void first_pass(bool counts) {
        uint32_t codes = 0;
        float most = -kInf, sum = 0.f, ent = 0.f;
        Run run;
        auto take = [&](const uint4 &v) {
            if (kHalf || counts) count_first(v, codes, run);
            if constexpr (!kHalf) {
                float f[kPer];
                floats(v, f);
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    most = max_nan(most, f[i]);
                    const float y = fmaxf(f[i] * kLog2e, -1000.f), e = ex2(y);
                    sum += e;
                    if (ENT) ent = fmaf(e, y, ent);
                }
            }
        };
        each([&](const uint4 &v, int) { take(v); });
        if constexpr (!kHalf) flush(run);
        if constexpr (kHalf) {
            __syncthreads();
            // what lies around zero
            const uint32_t n = min(sh.n_list, (uint32_t)kList);
            if (threadIdx.x < n) {
                const float x = __uint_as_float(sh.list[threadIdx.x].x);
                const uint32_t m = limbs(x, bin_ref(x, s), s, sh.pow);
                atomicAdd(&sh.near0[0], m >> 14);
                atomicAdd(&sh.near0[1], m & 16383u);
                // e^l by its series: |l| < 2^-7.9, the next term is below 2^-36.  256 of them fit, and
                // integers do not depend on the list's order.  (Where tau > 4, |l| is larger and a second
                // pass does this.)
                const float e = x * fmaf(x, fmaf(x, 0.16666667f, 0.5f), 1.f);      // - 1
                atomicAdd(&sh.near0[2], 0x800000u + (uint32_t)__float2int_rn(e * 0x1p23f));
                if (ENT) atomicAdd(&sh.near0[3], (uint32_t)__float2int_rn(x * kLog2e * (1.f + e) * 0x1p28f));
            }
            // M: of the first bin that is not empty, if that is a value's own and the others are whole
            uint32_t first = kBins;
#pragma unroll 1
            for (int i = 0; i < kBins; i += kT) {
                const int bin = i + threadIdx.x;
                if (bin <= kLastBin && (sh.bins[bin_slot(bin, false)] || (bin == kTop && sh.bins[kHalfBins])))
                    first = min(first, (uint32_t)bin);
            }
            first = kBins - block_max(kBins - first);
            if (first >= 1 && first <= kLastBin && first != kTop && sh.n_list <= kList) {
                most = bin_value(first, s);
            } else {
                // else it is looked for
                each([&](const uint4 &v, int) {
                    float f[kPer];
                    floats(v, f);
#pragma unroll
                    for (int i = 0; i < kPer; ++i) most = max_nan(most, f[i]);
                });
            }
            if (max(codes & 0xffffu, codes >> 16) > 0x7f80u) most = kInf;     // a NaN
            __syncthreads();
        }
        const uint32_t mine = most < kInf ? key_of(most) : 0xffffffffu;
        const uint32_t top = block_max(mine);
        uint32_t maxima = 0;
        if constexpr (kHalf) {
            maxima = threadIdx.x == 0 && sh.n_list > kList;     // more around zero than were kept
        } else {
            // a thread with the largest sums its other elements anew: next to it they lose their digits
            if (mine == top && top != 0xffffffffu) {
                sum = ent = 0.f;
                each([&](const uint4 &v, int) {
                    float f[kPer];
                    floats(v, f);
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        const float y = fmaxf(f[i] * kLog2e, -1000.f), e = ex2(y);
                        const bool is = f[i] == most;
                        maxima += is;
                        sum += is ? 0.f : e;
                        if (ENT) ent = fmaf(is ? 0.f : e, y, ent);
                    }
                });
            }
        }
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        report(top, maxima, sum, ent);
    }
    // The second pass: M and so all of the scale are known, and e = 2^((l - M) log2 e).
    __device__ __noinline__ void second_pass() {
        clear();
        __syncthreads();
        const uint32_t last = min(bin_of(kHalf ? __bfloat162float(__float2bfloat16_ru(s.lo)) : s.lo, s), (uint32_t)kLastBin);
        const uint32_t end = last + 1;
        Run run;
        if (kHalf) run.slot = min(max(s.top, 0), kBins - 1);
        float sum = 0.f, ent = 0.f;
        uint32_t maxima = 0;
#pragma unroll 1
        for (int j = threadIdx.x; j < n_vecs; j += kT) {
            float f[kPer];
            floats(load(j), f);
            count_second(f, end, run);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float y = fmaxf((f[i] - s.M) * kLog2e, -1000.f), e = ex2(y);
                const bool is = f[i] == s.M;
                maxima += is;
                sum += is ? 0.f : e;
                if (ENT) ent = fmaf(is ? 0.f : e, y, ent);
            }
        }
        flush(run);
        report(key_of(s.M), maxima, sum, ent);
    }
    // The scale of a second pass, from M.
    __device__ __forceinline__ void scale_from(float M, float least, float tau) {
        const float width = kWindow * kLn2f * tau;
        s.M = M;
        s.lo = fmaxf(M - width, least);
        if constexpr (!kHalf) {
            // bins of at most one in y: 2^-7 of a value, or 2^-23 at the finest
            const float far = fmaxf(fabsf(M), fabsf(M - width)) * s.gh;
            const int e = far < 0x1p7f ? 0 : min((int)(__float_as_uint(far) >> 23) - 127 - 7 + 1, 16);
            s.shift = 16 - e;
        }
        s.zero = (int32_t)(__float_as_uint(tau * 0x1p-9f) >> s.shift);
        s.top = 0;
        s.top = place(M, s);
    }

    // --- what the first block asks for; the results go to it ---

    __device__ void count(const Command &c) {
        uint32_t n = 0, least = 0xffffffffu, most = 0;
        // masses are asked for within a bin of several values
        const float ref = bin_ref(of_key(c.khi), s);
        const uint64_t w = mass_at(ref, s, sh.pow);
        uint64_t m = 0;
        each([&](const uint4 &v, int j) {
            float x[kPer];
            floats(v, x);
#pragma unroll 1
            for (int i = 0; i < kPer; ++i) {
                float l = x[0];
#pragma unroll
                for (int q = 1; q < kPer; ++q) l = i == q ? x[q] : l;
                const uint32_t k = key_of(l);
                if (k >= c.klo && k <= c.khi && (c.below < 0 || id0 + j * kPer + i < c.below)) {
                    ++n;
                    least = min(least, k), most = max(most, k);
                    m += mass_in(l, ref, w, s, sh.pow);
                }
            }
        });
        n = __reduce_add_sync(0xffffffffu, n);
        least = __reduce_min_sync(0xffffffffu, least);
        most = __reduce_max_sync(0xffffffffu, most);
        m = warp_sum64(m);
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
        if (lane == 0) sh.scan[wid] = m, sh.scan_n[wid] = n, sh.scan_k[wid] = least, sh.scan_f[0][wid] = __uint_as_float(most);
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kWarps; ++i) {
                m += sh.scan[i], n += sh.scan_n[i];
                least = min(least, sh.scan_k[i]), most = max(most, __float_as_uint(sh.scan_f[0][i]));
            }
            put(at_block(&sh.mass[rank], 0), m);
            put(at_block(&sh.count[rank], 0), n);
            put(at_block(&sh.least[rank], 0), least);
            put(at_block(&sh.most[rank], 0), most);
        }
        __syncthreads();
    }
    __device__ void gather(const Command &c) {
        const uint32_t n_at = at_block(&sh.n_list, 0), at = at_block(&sh.list[0], 0);
        // the key below 0's is no value's, and as a float, -0, would stand for 0
        const float least = of_key(c.klo), most = of_key(c.khi - (c.khi == 0x7fffffffu));
        each([&](const uint4 &v, int j) {
            float x[kPer];
            floats(v, x);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (x[i] >= least && x[i] <= most) {
                    const uint32_t k = key_of(x[i]);
                    const uint32_t slot = add_at(n_at, 1);
                    if (slot < kList) {
                        put(at + slot * 8, k);
                        put(at + slot * 8 + 4, (uint32_t)(id0 + j * kPer + i));
                    }
                }
            }
        });
    }
    __device__ __noinline__ void obey(const Command &c) {
        if (c.kind == kCount) count(c);
        else gather(c);
    }
    // The id of the nth element of a value in this block's part: an eighth of it at a time, until
    // it is reached (700 x 262,144 bfloat16 rows, more than L2 holds: 189 us, all at once 250).
    __device__ __noinline__ void locate(uint32_t key, uint32_t nth, int32_t *out) {
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
        constexpr int kAhead = 4;
        const int per = ((n_vecs + 8 * kWarps - 1) / (8 * kWarps) + 32 * kAhead - 1) / (32 * kAhead) * (32 * kAhead);
        const float want = of_key(key);
        auto hits = [&](int j, int end) {
            uint32_t h = 0;
            if (j < end) {
                float x[kPer];
                floats(load(j), x);
#pragma unroll
                for (int i = 0; i < kPer; ++i) h |= (uint32_t)(x[i] == want) << i;
            }
            return h;
        };
        for (int at = 0; at < n_vecs; at += per * kWarps) {
            const int j0 = at + wid * per, j1 = min(j0 + per, n_vecs);
            uint32_t n = 0;
            int j = j0 + lane;
            for (; j + (kAhead - 1) * 32 < min(j1, n_vecs - 1); j += kAhead * 32) {
                uint4 v[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) v[i] = __ldg(vecs + j + i * 32);
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if constexpr (kHalf) {
                        const __nv_bfloat162 w2 = __float2bfloat162_rn(want);
                        auto eq = [&](uint32_t w) { return __heq2_mask(*reinterpret_cast<__nv_bfloat162 *>(&w), w2) & 0x10001u; };
                        const uint32_t c = eq(v[i].x) + eq(v[i].y) + eq(v[i].z) + eq(v[i].w);
                        n += (c & 0xffffu) + (c >> 16);
                    } else {
                        float x[kPer];
                        floats(v[i], x);
#pragma unroll
                        for (int q = 0; q < kPer; ++q) n += x[q] == want;
                    }
                }
            }
            for (; j < j1; j += 32) n += __popc(hits(j, j1));
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) sh.scan_n[wid] = n;
            __syncthreads();
            const uint32_t c = lane < kWarps ? sh.scan_n[lane] : 0;
            uint32_t before = __reduce_add_sync(0xffffffffu, lane < wid ? c : 0u);
            const uint32_t all = __reduce_add_sync(0xffffffffu, c);
            if (all < nth) {
                nth -= all;
                __syncthreads();
                continue;
            }
            if (before >= nth || before + n < nth) return;
            for (j = j0 + lane; j - lane < j1; j += 32) {
                uint32_t h = hits(j, j1);
                const uint32_t mine = __popc(h);
                uint32_t incl = mine;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
                    if (lane >= d) incl += y;
                }
                const uint32_t from = before + incl - mine;
                if (from < nth && from + mine >= nth) {
                    for (uint32_t i = nth - from; i > 1; --i) h &= h - 1;
                    *out = id0 + j * kPer + __ffs(h) - 1;
                }
                before += __shfl_sync(0xffffffffu, incl, 31);
                if (before >= nth) return;
            }
            return;
        }
    }
};

// Of the order, a thread of the first block keeps what comes before its eight bins and what
// they hold; the bins themselves, added over the cluster, are in its shared memory.
struct Before {
    uint64_t m, m_here, m_all;
    uint32_t n, n_here, n_all;
};

// The first block's part.
template <typename ElemT, bool ENT>
struct Order : Row<ElemT, ENT> {
    using Base = Row<ElemT, ENT>;
    using Base::kHalf, Base::kT, Base::kWarps, Base::kBinsThread, Base::sh, Base::limb, Base::rank, Base::blocks, Base::s, Base::obey;
    Before o;
    bool linear;                 // the bins are a second pass's

    // What the limbs of a bin stand for.  A block's own (limbs()) are of 14 bits an element; the sum over
    // a cluster's blocks has up to 48 bits, 2^20 elements of 28, and is held in limbs of 24.
    __device__ __forceinline__ uint64_t limbs_sum(uint32_t hi, uint32_t low) const {
        return ((uint64_t)hi << (blocks > 1 ? 24 : 14)) + low;
    }
    // A bin's mass, and its elements; none where it lies below what min-p leaves.
    __device__ __forceinline__ uint64_t bin_mass(int bin, uint32_t *n) const {
        const int at = bin_slot(bin, linear);
        *n = bin <= kLastBin ? sh.bins[at] : 0;
        if (*n == 0) return 0;
        const bool one = kHalf && bin != s.top;
        const float v = one ? bin_value(bin, s) : bin_most(bin, s);
        if (v < s.lo) *n = 0;
        float h, e;
        exponent(v, s.M, s, &h, &e);
        if (!(h > -(float)s.bits - 2.f) || *n == 0) return 0;
        const uint64_t w = pow2_fixed(h, e, s.bits, sh.pow);
        if (one) return w * *n;
        const uint64_t part = kHalf ? sh.near0_all : limbs_sum(limb[at], limb[kBins + at]);
        return __umul64hi(w, part) << 36 | w * part >> 28;
    }
    __device__ __forceinline__ void order(const Command &c) {
        __syncthreads();
        if (blocks == 1) return;
        if (threadIdx.x < blocks) {
            const uint32_t a = at_block(&sh.cmd, threadIdx.x);
            put(a, (uint32_t)c.kind);
            put(a + 4, c.klo);
            put(a + 8, c.khi);
            put(a + 12, (uint32_t)c.below);
            put(a + 16, c.nth);
        }
        sync_cluster();
    }
    __device__ __forceinline__ void carry_out(Command c) {
        c.nth = key_of(s.M);
        if (blocks == 1) {
            __syncthreads();
            obey(c);
            __syncthreads();
            return;
        }
        order(c);
        obey(c);
        sync_cluster();
    }
    __device__ __forceinline__ void counted(uint32_t *cnt, uint64_t *mass) const {
        *cnt = 0, *mass = 0;
        for (uint32_t b = 0; b < blocks; ++b) *cnt += sh.count[b], *mass += sh.mass[b];
    }
    // The bins of all blocks.
    __device__ __forceinline__ void add_up() {
        // the loads of all blocks are under way together
        if (blocks > 1) {
#pragma unroll 1
            for (int i = threadIdx.x * 4; i < kBins; i += kT * 4) {
                uint4 t = make_uint4(0, 0, 0, 0);
#pragma unroll 4
                for (uint32_t b = 0; b < blocks; ++b) {
                    const uint4 v = get4(at_block(sh.bins + i, b));
                    t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
                }
                *reinterpret_cast<uint4 *>(sh.bins + i) = t;
            }
            if constexpr (!kHalf) {
#pragma unroll 1
                for (int i = threadIdx.x * 4; i < kBins; i += kT * 4) {
                    uint64_t t[4] = {};
#pragma unroll 4
                    for (uint32_t b = 0; b < blocks; ++b) {
                        const uint4 h = get4(at_block(limb + i, b)), l = get4(at_block(limb + kBins + i, b));
                        t[0] += ((uint64_t)h.x << 14) + l.x, t[1] += ((uint64_t)h.y << 14) + l.y;
                        t[2] += ((uint64_t)h.z << 14) + l.z, t[3] += ((uint64_t)h.w << 14) + l.w;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) limb[i + q] = (uint32_t)(t[q] >> 24), limb[kBins + i + q] = (uint32_t)t[q] & 0xffffffu;
                }
            }
        }
        if (kHalf && threadIdx.x < 32) {
            uint64_t part = 0;
            float sum = 0.f, ent = 0.f;
            if (threadIdx.x < blocks) {
                const uint32_t a = at_block(&sh.near0[0], threadIdx.x);
                part = ((uint64_t)get(a) << 14) + get(a + 4);
                sum = (float)get(a + 8) * 0x1p-23f;
                if (ENT) ent = (float)(int32_t)get(a + 12) * 0x1p-28f;
            }
            part = warp_sum64(part);
            sum = warp_sum(sum);
            if (ENT) ent = warp_sum(ent);
            if (threadIdx.x == 0) sh.near0_all = part, sh.near0_sum = sum, sh.near0_ent = ent;
        }
        __syncthreads();
        // around zero the first pass has two
        if (!linear) {
            if (threadIdx.x == 0) {
                sh.bins[0] += sh.bins[kHalfBins];
                if constexpr (!kHalf) {
                    limb[0] += limb[kHalfBins];
                    limb[kBins] += limb[kBins + kHalfBins];
                }
            }
            __syncthreads();
        }
    }
    // The running sums; of bfloat16 rows after a first pass also those of log p0, in `part`, but for
    // the bin around zero.
    __device__ __forceinline__ void sum_up(bool counts, Part *part) {
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
        o.m_here = 0, o.n_here = 0;
        float sum = 0.f, ent = 0.f;
        uint32_t maxima = 0;
        if constexpr (kHalf) {
            // Without branches, so that one bin's chain of steps runs beside another's; the bin
            // around zero comes after.
#pragma unroll 4
            for (int i = 0; i < kBinsThread; ++i) {
                // from another place on in each thread, as they are all in the same banks
                const int bin = threadIdx.x * kBinsThread + ((i + threadIdx.x) & (kBinsThread - 1));
                uint32_t n = sh.bins[bin_slot(bin, linear) & (kBins - 1)];
                if (bin > kLastBin || bin == s.top) n = 0;
                const float v = bin_value(bin, s);
                float h, e;
                exponent(v, s.M, s, &h, &e);
                const bool heavy = h > -(float)s.bits - 2.f && h < 1.f;
                const uint64_t w = pow2_fixed(heavy ? h : 0.f, heavy ? e : 0.f, s.bits, sh.pow);
                const uint32_t in = v >= s.lo ? n : 0;
                o.m_here += heavy ? w * in : 0;
                o.n_here += in;
                const float y = fmaxf(fminf((v - s.M) * kLog2e, 0.f), -1000.f);
                const float x = v == s.M ? 0.f : (float)n * ex2(y);
                if (v == s.M) maxima = n;
                sum += x;
                if (ENT) ent = fmaf(x, y, ent);
            }
            if (s.top / kBinsThread == threadIdx.x && s.top >= 0 && s.top <= kLastBin) {
                uint32_t n;
                o.m_here += bin_mass(s.top, &n);
                o.n_here += n;
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < kBinsThread; ++i) {
                const int bin = threadIdx.x * kBinsThread + ((i + threadIdx.x) & (kBinsThread - 1));
                uint32_t n;
                o.m_here += bin_mass(bin, &n);
                o.n_here += n;
            }
        }
        uint64_t mi = o.m_here;
        uint32_t ni = o.n_here;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint64_t a = shfl_up64(mi, d);
            const uint32_t b = __shfl_up_sync(0xffffffffu, ni, d);
            if (lane >= d) mi += a, ni += b;
        }
        if (kHalf && counts) {
            maxima = __reduce_add_sync(0xffffffffu, maxima);
            sum = warp_sum(sum);
            if (ENT) ent = warp_sum(ent);
            if (lane == 0) sh.scan_k[wid] = maxima, sh.scan_f[0][wid] = sum, sh.scan_f[1][wid] = ent;
        }
        if (lane == 31) sh.scan[wid] = mi, sh.scan_n[wid] = ni;
        __syncthreads();
        const uint64_t ms = lane < kWarps ? sh.scan[lane] : 0;
        const uint32_t ns = lane < kWarps ? sh.scan_n[lane] : 0;
        const uint64_t ms_before = warp_sum64(lane < wid ? ms : 0);
        const uint32_t ns_before = __reduce_add_sync(0xffffffffu, lane < wid ? ns : 0u);
        o.m = ms_before + mi - o.m_here;
        o.n = ns_before + ni - o.n_here;
        o.m_all = warp_sum64(ms);
        o.n_all = __reduce_add_sync(0xffffffffu, ns);
        if (kHalf && counts) {
            part->maxima = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.scan_k[lane] : 0u);
            part->sum = warp_sum(lane < kWarps ? sh.scan_f[0][lane] : 0.f);
            if (ENT) part->ent = warp_sum(lane < kWarps ? sh.scan_f[1][lane] : 0.f);
        }
    }

    // The element at which the running mass reaches `mass` (> 0), or the running count
    // `number` where that is not 0.  All threads get the same.
    __device__ __noinline__ Result reach(uint64_t mass, uint32_t number) {
        mass = min(mass, o.m_all);
        if (number ? o.n < number && o.n + o.n_here >= number : o.m < mass && o.m + o.m_here >= mass) {
            sh.res.before = o.m;
            sh.res.count = o.n;
            sh.at = threadIdx.x;
        }
        __syncthreads();
        // among that thread's bins, by the first warp's first lanes
        if (threadIdx.x < 32) {
            const int lane = threadIdx.x, from = min(sh.at, kT - 1) * kBinsThread, bin0 = from + (lane & (kBinsThread - 1));
            Result r = sh.res;
            uint32_t n;
            const uint64_t m = bin_mass(bin0, &n);
            uint32_t nb = n;
            uint64_t mb = m;
#pragma unroll
            for (int d = 1; d < kBinsThread; d *= 2) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, nb, d);
                const uint64_t y = shfl_up64(mb, d);
                if (lane >= d) nb += x, mb += y;
            }
            nb += r.count, mb += r.before;                      // after this lane's bin
            const uint32_t there = __ballot_sync(0xffffffffu, number ? nb >= number : mb >= mass);
            const int i = max(__ffs(there) - 1, 0);
            const int bin = from + min(i, kBinsThread - 1);
            const uint32_t left = __shfl_sync(0xffffffffu, n, i);
            r.end = shfl64(mb, i);
            r.before = r.end - shfl64(m, i);
            r.count = __shfl_sync(0xffffffffu, nb, i) - left;
            r.id = -1;
            r.equal = left;
            if (kHalf && bin != s.top) {                        // one value
                r.key = key_of(bin_value(bin, s));
                nth_of(r, number ? number - r.count : 0, mass - r.before, r.end, r.count + left - 1);
            } else {
                r.nth = 0;
            }
            __syncwarp();
            if (lane == 0) sh.res = r, sh.at = bin;
        }
        __syncthreads();
        Result r = sh.res;
        if (r.nth == 0) settle(r, sh.at, number ? number - r.count : 0, mass - r.before);
        __syncthreads();
        return r;
    }
    // Of r.equal elements of r.key the cth, or the one where the mass reaches t.
    __device__ __forceinline__ void nth_of(Result &r, uint32_t c, uint64_t t, uint64_t bin_end, uint32_t last) const {
        const uint64_t w = mass_of<kHalf>(of_key(r.key), s, sh.pow);
        const uint32_t left = r.equal;
        uint32_t j = c;
        if (c == 0) {
            j = (uint32_t)fminf(__fdividef((float)t, (float)w), (float)left);
            j = max(min(j, left), 1u);
            while (j > 1 && (j - 1) * w >= t) --j;
            while (j < left && j * w < t) ++j;
        }
        j = max(min(j, left), 1u);
        r.nth = j;
        r.before += (j - 1) * w;
        r.count += j - 1;
        // the elements of a bin of several values are rounded up: its last one ends where the bin
        // does, and none ends later
        r.end = r.count == last ? bin_end : min(r.before + w, bin_end);
    }
    // The same in a bin of several values: halved until its elements fit the list, or are equal.
    __device__ __noinline__ void settle(Result &r, int bin, uint32_t c, uint64_t t) {
        const uint64_t bin_end = r.end;
        uint32_t left = r.equal;
        const uint32_t last = r.count + left - 1;
        const bool number = c != 0;
        uint32_t klo = max(key_of(bin_least(bin, s)), key_of(s.lo)), khi = min(key_of(bin_most(bin, s)), key_of(s.M));
        auto found = [&] {                                      // the keys that were counted
            uint32_t a = 0xffffffffu, b = 0;
            for (uint32_t i = 0; i < blocks; ++i) a = min(a, sh.least[i]), b = max(b, sh.most[i]);
            if (a <= b) klo = a, khi = b;
        };
        if (left > kList) {
            carry_out(Command{kCount, klo, khi, -1, 0});
            found();
            __syncthreads();
        }
        while (left > kList && klo < khi) {
            const uint32_t mid = khi - (khi - klo) / 2;
            carry_out(Command{kCount, mid, khi, -1, 0});
            uint32_t cu;
            uint64_t mu;
            counted(&cu, &mu);
            if (number ? c <= cu : t <= mu || cu == left) {
                found();
                left = cu;
            } else {
                khi = mid - 1, left -= cu;
                if (number) c -= cu;
                else t -= min(mu, t - 1);
                r.before += mu, r.count += cu;
            }
            __syncthreads();
        }
        if (klo == khi) {
            r.key = klo;
            r.equal = left;
            nth_of(r, c, t, bin_end, last);
            return;
        }
        if (threadIdx.x == 0) sh.n_list = 0;
        carry_out(Command{kGather, klo, khi, -1, 0});
        const uint32_t len = min(sh.n_list, (uint32_t)kList);
        uint2 me = make_uint2(0, 0);
        uint64_t w = 0;
        if (threadIdx.x < len) {
            me = sh.list[threadIdx.x];
            w = mass_of<kHalf>(of_key(me.x), s, sh.pow);
            sh.list_w[threadIdx.x] = w;
        }
        __syncthreads();
        if (threadIdx.x < len) {
            uint64_t b = 0;
            uint32_t nb = 0, nth = 1, equal = 0;
#pragma unroll 4
            for (uint32_t i = 0; i < len; ++i) {
                const uint2 x = sh.list[i];
                const uint64_t xw = sh.list_w[i];
                const bool same = x.x == me.x && x.y < me.y;
                if (x.x > me.x || same) b += xw, ++nb;
                nth += same, equal += x.x == me.x;
            }
            if (number ? nb + 1 == c : b < t && b + w >= t) {
                Result q;
                q.before = r.before + b;
                q.count = r.count + nb;
                q.end = q.count == last ? bin_end : min(q.before + w, bin_end);
                q.key = me.x;
                q.nth = nth;
                q.id = (int32_t)me.y;
                q.equal = equal;
                sh.res = q;
            }
        }
        __syncthreads();
        r = sh.res;
    }
};

template <typename ElemT, bool SCORE, bool ENT>
__global__ void __launch_bounds__(Row<ElemT, ENT>::kT, Row<ElemT, ENT>::kResident) sample_kernel(const SampleParams p) {
    constexpr int kT = Row<ElemT, ENT>::kT;
    constexpr int kPer = Row<ElemT, ENT>::kPer;
    constexpr bool kHalf = Row<ElemT, ENT>::kHalf;
    __shared__ Shared sh;
    extern __shared__ __align__(16) uint32_t dyn[];
    const uint32_t rank = block_rank(), blocks = n_blocks();
    const int64_t row = p.row0 + blockIdx.x / blocks;
    const int tid = threadIdx.x, lane = tid & 31;

    // the row, and its choices
    const int64_t src = p.row_index ? __ldg(p.row_index + row) : row;
    const int64_t of = p.set.row_set ? __ldg(p.set.row_set + row) : p.set.n_sets == 1 ? 0 : row;
    const bool bad_src = src < 0 || src >= p.n_logit_rows, bad_set = of < 0 || of >= p.set.n_sets;
    int bits = bad_src ? PS_DEV_BAD_ROW_INDEX : 0;
    const uint8_t *row_ptr = p.logits + (bad_src ? 0 : src) * p.ld_bytes;
    const int all_vecs = (p.V + kPer - 1) / kPer;
    const int v0 = min((int)rank * p.slice_vecs, all_vecs), v1 = min(v0 + p.slice_vecs, all_vecs);
    // the row's first vectors are on their way while its choices are looked up
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (v0 + tid + i * kT < v1)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(row_ptr + (int64_t)(v0 + tid + i * kT) * 16));
    const int64_t set = bad_set ? 0 : of;
    const float tau = __ldg(p.set.tau + set);
    const int32_t k = p.set.top_k ? __ldg(p.set.top_k + set) : 0;
    const float top_p = p.set.top_p ? __ldg(p.set.top_p + set) : 1.f;
    const float min_p = p.set.min_p ? __ldg(p.set.min_p + set) : 0.f;
    if (bad_set || !(tau >= 0x1p-20f && tau <= 0x1p20f) || k < 0 || !(top_p > 0.f && top_p <= 1.f) ||
        !(min_p >= 0.f && min_p <= 1.f))
        bits |= PS_DEV_BAD_SAMPLING;
    int32_t token = 0;
    double u = 1.0;
    float l_tok = 0.f;
    if constexpr (SCORE) {
        token = __ldg(p.tokens + row);
        if (token < 0 || token >= p.V) bits |= PS_DEV_BAD_TOKEN, token = 0;
        const ElemT *elems = reinterpret_cast<const ElemT *>(row_ptr);
        if constexpr (kHalf) l_tok = __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(elems) + token) << 16);
        else l_tok = __ldg(reinterpret_cast<const float *>(elems) + token);
    } else {
        u = __ldg(p.u + row);
        if (!(u > 0.0 && u <= 1.0)) bits |= PS_DEV_BAD_UNIFORM;
    }
    auto none = [&](int why) {
        if (rank == 0 && tid == 0) {
            const double nan = __longlong_as_double(0x7ff8000000000000ll);
            set_status(p.status, why);
            if (p.lp0) p.lp0[row] = nan;
            if (p.lq) p.lq[row] = nan;
            if (ENT) p.entropy[row] = nan;
            if constexpr (!SCORE) p.drawn[row] = -1;
        }
    };
    if (bits) {                                                // the same in every block
        none(bits);
        return;
    }

    // the other blocks' shared memory is there from its counterpart on, in first_pass()
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    Order<ElemT, ENT> x{{sh, dyn, reinterpret_cast<const uint4 *>(row_ptr) + v0, p.V, v1 - v0, v0 * kPer, rank, blocks}};
    Scale &s = x.s;
    s.bits = p.mass_bits;
    s.gh = __fdiv_rn(kLog2e, tau);
    s.gl = __fdiv_rn(fmaf(-s.gh, tau, kLog2e) + kLog2eLow, tau);
    s.shift = 16;
    s.zero = (int32_t)(__float_as_uint(fmaxf(tau, 1.f) * 0x1p-10f) >> 16);
    s.top = kTop;
    s.M = 0.f;
    s.lo = -kInf;
    x.clear();
    if (tid < 64) sh.pow[tid] = kPow.t[tid];
    if (tid == 0) sh.at = 0, sh.res = Result{};
    __syncthreads();
    x.first_pass(kHalf || !(min_p > 0.f));
    if (rank == 0 && tid == kT - 1 && min_p > 0.f) {
        const uint32_t b = __float_as_uint(min_p);
        const int e = max((int)(b >> 23), 1);
        const double y = (double)tau * ln_of((b & 0x7fffffu) | (b >> 23 ? 1u << 23 : 0u), 150 - e, sh.pow);
        sh.lnp[0] = (float)y;
        sh.lnp[1] = (float)(y - (double)sh.lnp[0]);
    }
    sync_cluster();
    if (rank != 0) {
        for (;;) {
            sync_cluster();
            const Command c = sh.cmd;
            if (c.kind == kDone) return;
            if (c.kind == kLocate) {
                if constexpr (!SCORE)
                    if ((int32_t)rank == c.below) x.locate(c.klo, c.nth, p.drawn + row);
                return;
            }
            if (c.kind == kAgain) {
                x.scale_from(of_key(c.klo), of_key(c.khi), tau);
                x.second_pass();
            } else {
                s.M = of_key(c.nth);                            // after a first pass it was not known here
                x.obey(c);
            }
            sync_cluster();
        }
    }

    // the row as a whole
    Part all{0, 0, 0.f, 0.f};
    for (uint32_t b = 0; b < blocks; ++b) all.top_key = max(all.top_key, sh.part[b].top_key);
    const float M = all.top_key == 0xffffffffu ? kInf : of_key(all.top_key);
    if (!(M > -kInf && M < kInf)) {
        none(PS_DEV_NONFINITE);
        x.order(Command{kDone, 0, 0, 0, 0});
        return;
    }
    float least = -kInf;                                       // of min-p: M + tau ln(min_p), rounded up
    if (min_p > 0.f) {
        const float h = sh.lnp[0], t = M + h, d = t - M;
        least = fminf(__fadd_ru(t, ((M - (t - d)) + (h - d)) + sh.lnp[1]), M);
    }
    // whether the bins of the first pass hold all that counts
    s.M = M;
    bool again;
    {
        const float bottom = bin_least(kLastBin, s), width = kWindow * kLn2f * tau;
        const uint32_t first = bin_of(M, s);
        again = first < 1 || first > (uint32_t)kLastBin || !(M - width > bottom) || tau < 0x1p-7f || tau > 4.f;
        if constexpr (kHalf) {
            // log p0 comes from the bins as well
            for (uint32_t b = 0; b < blocks; ++b) again = again || sh.part[b].maxima > 0;
            again = again || (int)first == s.top || !(M - bottom > 30.f) ||
                    (min_p > 0.f && least <= bin_most(s.top, s) && least >= bin_least(s.top, s));
        } else {
            // 2^20 elements of e^60 are within float32
            again = again || !(M > -40.f && M < 60.f) || min_p > 0.f || fmaxf(fabsf(M), fabsf(M - width)) * s.gh > 0x1p8f;
        }
        s.lo = fmaxf(bottom, least);
    }
    if (again) {
        x.order(Command{kAgain, key_of(M), key_of(least), 0, 0});
        x.scale_from(M, least, tau);
        x.second_pass();
        sync_cluster();
    }
    x.linear = again;
    x.add_up();
    x.sum_up(!again, &all);
    // e^-M, where sums are of e^l
    auto down_from = [](float M, float yh) { return ex2(-yh) * (1.f - kLn2f * (fmaf(M, kLog2e, -yh) + M * kLog2eLow)); };
    if (!kHalf || again) {
        const float yh = M * kLog2e, down = again ? 1.f : down_from(M, yh);
        for (uint32_t b = 0; b < blocks; ++b) {
            const Part q = sh.part[b];
            const float to = again ? 0.f : yh;
            all.sum += q.sum;
            if (ENT) all.ent += fmaf(-to, q.sum, q.ent);
            const float l = of_key(q.top_key);
            if (l == M) {
                all.maxima += q.maxima;
            } else {                                            // of a block whose largest is less
                const float y = again ? 0.f : fmaxf(l * kLog2e, -1000.f), e = again ? 0.f : (float)q.maxima * ex2(y);
                all.sum += e;
                if (ENT) all.ent = fmaf(e, y - to, all.ent);
            }
        }
        all.sum *= down;
        if (ENT) all.ent *= down;
    }

    // what truncation leaves
    uint64_t Z = x.o.m_all;
    Result end_k, end_p;
    const bool cut_k = k > 0 && (uint32_t)k < x.o.n_all, cut_p = top_p < 1.f;
    if (cut_k) {
        end_k = x.reach(0, (uint32_t)k);
        Z = end_k.end;
    }
    if (cut_p) {
        end_p = x.reach(share_of(top_p, Z), 0);
        Z = end_p.end;
    }
    float l;
    bool kept = true;
    Command last{kDone, 0, 0, 0, 0};
    if constexpr (SCORE) {
        l = l_tok;
        const uint32_t key = key_of(l);
        kept = l >= least && l > -kInf;
        uint64_t unused;
        uint32_t above = 0, ties = 0;
        const bool far = kept && l < s.lo;                       // outside the bins, yet maybe among the first k
        if (far && k > 0 && !cut_k && !cut_p) {
            x.carry_out(Command{kCount, key + 1, 0xffffffffu, -1, 0});
            x.counted(&above, &unused);
            __syncthreads();
        }
        // its place among its equals counts where a cut divides them
        auto divided = [&](const Result &e) { return key == e.key && e.nth < e.equal; };
        if (kept && ((cut_k && divided(end_k)) || (cut_p && divided(end_p)) || above > 0)) {
            x.carry_out(Command{kCount, key, key, token, 0});
            x.counted(&ties, &unused);
        }
        auto within = [&](const Result &e) { return key > e.key || (key == e.key && ties < e.nth); };
        if (cut_k) kept = kept && within(end_k);
        if (cut_p) kept = kept && within(end_p);
        if (above > 0) kept = kept && above + ties < (uint32_t)k;
    } else {
        const Result at = x.reach(share_of(u, Z), 0);
        l = of_key(at.key);
        if (at.id >= 0) {
            if (tid == 0) p.drawn[row] = at.id;
        } else {
            // the block that holds the nth of this value
            int owner = 0;
            uint32_t skip = 0;
            if (blocks > 1) {
                const int bin = (int)bin_of(l, s);
                const bool one = kHalf && bin != s.top;
                if (!one) x.carry_out(Command{kCount, at.key, at.key, -1, 0});
                // lane b: of block b
                uint32_t c = 0;
                const int at_slot = bin_slot(bin, again) & (kBins - 1);
                if (lane < blocks) c = !one ? sh.count[lane] : lane ? get(at_block(&sh.bins[at_slot], lane)) : 0;
                if (one) {
                    const uint32_t others = __reduce_add_sync(0xffffffffu, c);
                    if (lane == 0) c = sh.bins[at_slot] - others;
                }
                uint32_t to = c;
#pragma unroll
                for (int d = 1; d < kMostBlocks; d *= 2) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, to, d);
                    if (lane >= d) to += y;
                }
                owner = __ffs(__ballot_sync(0xffffffffu, to >= at.nth)) - 1;
                skip = __shfl_sync(0xffffffffu, to - c, owner);
            }
            last = Command{kLocate, at.key, at.key, owner, at.nth - skip};
        }
    }
    x.order(last);
    if constexpr (!SCORE)
        if (last.kind == kLocate && last.below == 0) x.locate(last.klo, last.nth, p.drawn + row);

    // the row's values, by two warps
    if (tid == kT - 1 && p.lq) {
        double lq = -(double)kInf;
        if (kept) {
            const uint64_t w = mass_of<kHalf>(l, s, sh.pow);
            if (2 * w > Z) {                                     // a mass close to all of Z: by the others' share
                lq = -(double)log1pf((float)(Z - min(w, Z)) / (float)w);
            } else {
                double y;
                if (l >= s.lo) {
                    float h, e;
                    exponent(l, M, s, &h, &e);
                    y = ((double)h + (double)e) * kLn2;
                } else {
                    y = ((double)l - (double)M) / (double)tau;
                }
                lq = y - ln_of(Z, s.bits, sh.pow);
            }
        }
        p.lq[row] = lq;
    }
    if (tid == 32 && (p.lp0 || ENT)) {
        if (kHalf && !x.linear) {
            // what lies around zero: M is not among it
            const float yh = M * kLog2e, down = down_from(M, yh);
            all.sum = fmaf(sh.near0_sum, down, all.sum);
            if (ENT) all.ent = fmaf(fmaf(-yh, sh.near0_sum, sh.near0_ent), down, all.ent);
        }
        // log of 1 and the rest: of a small rest to its own digits
        const float rest = (float)(all.maxima - 1) + all.sum;
        const double log_z = rest < 0.5f ? (double)log1pf(rest)
                                         : ln_of(((uint64_t)all.maxima << 40) + __float2ull_rn(all.sum * 0x1p40f), 40, sh.pow);
        if (p.lp0) p.lp0[row] = ((double)l - (double)M) - log_z;
        if (ENT) p.entropy[row] = log_z - kLn2 * (double)(all.ent / (1.f + rest));
    }
}

// Blocks of a cluster and the vectors of a row that each reads.  A row is one block's where
// there are rows for all multiprocessors; fewer are divided, down to 4 KB a block.  No part
// has more than 2^18 elements, as the limbs want it.
struct Cut {
    int blocks;
    int32_t vecs;
};
Cut cut_of(const SampleParams &p, int sms) {
    const int per = p.dtype == PS_BF16 ? 8 : 4;
    const int32_t all = (p.V + per - 1) / per;
    auto vecs = [&](int b) { return (all + b - 1) / b; };
    int b = 1;
    while (b < kMostBlocks && ((int64_t)vecs(b) * per > 1 << 18 || (p.n_rows * b < 2 * (int64_t)sms && vecs(b) >= 512))) b *= 2;
    return Cut{b, vecs(b)};
}

template <typename ElemT, bool SCORE, bool ENT>
cudaError_t launch(const SampleParams &p, int blocks, int64_t rows, cudaStream_t stream) {
    const size_t smem = sizeof(ElemT) == 2 ? 0 : 2 * kBins * sizeof(uint32_t);
    const cudaError_t e = cudaFuncSetAttribute(sample_kernel<ElemT, SCORE, ENT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * blocks));
    cfg.blockDim = dim3(Row<ElemT, ENT>::kT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<ElemT, SCORE, ENT>, p);
}

template <typename ElemT>
cudaError_t launch_type(const SampleParams &p, int blocks, int64_t rows, cudaStream_t stream) {
    if (p.tokens)
        return p.entropy ? launch<ElemT, true, true>(p, blocks, rows, stream) : launch<ElemT, true, false>(p, blocks, rows, stream);
    return p.entropy ? launch<ElemT, false, true>(p, blocks, rows, stream) : launch<ElemT, false, false>(p, blocks, rows, stream);
}

}  // namespace

cudaError_t launch_sample(const SampleParams &params, int sms, cudaStream_t stream) {
    SampleParams p = params;
    const Cut c = cut_of(p, sms);
    p.slice_vecs = c.vecs;
    int log_v = 0;
    while ((1 << log_v) < p.V) ++log_v;
    p.mass_bits = std::min(63 - log_v, 45);
    constexpr int64_t kMostRows = (int64_t)1 << 27;             // of a launch
    for (int64_t r = 0; r < p.n_rows; r += kMostRows) {
        p.row0 = r;
        const int64_t rows = std::min(p.n_rows - r, kMostRows);
        const cudaError_t e = p.dtype == PS_BF16 ? launch_type<uint16_t>(p, c.blocks, rows, stream)
                                                 : launch_type<float>(p, c.blocks, rows, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace ps
