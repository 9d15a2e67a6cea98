// stage_step.cu -- the AdamW step over all tensors of a stage in one launch,
// moments in 32 or in 8 bits, and the norm of its gradients.
//
//   m = b1 m + (1 - b1) g      v = b2 v + (1 - b2) g^2      (g clipped before)
//   p = p (1 - lr decay) - lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps)
// Every element is read and written once, so memory bounds it: 30 bytes an
// element with 32-bit parameters, moments and gradients and a 16-bit copy, 18 with
// the moments in 8 bits.  571 million elements take 2.42 ms and 1.45 ms, both 105 %
// of the measured copy rate (reads outweigh writes), 16-bit parameters and
// gradients with moments in 32 bits 1.77 ms, the same.  All in 16 bits with moments
// in 8 it is 10 bytes an element, and its 70 instructions bound it, half of them
// whole-number ones (issue slots 85 % busy): 1.33 ms rounded at random, 63 %; 90
// million elements in 161 tensors 229 us at random and 191 to nearest (70 %).  The
// norm takes 324 us of 32-bit gradients (104 %), 185 us of 16-bit ones (91 %).
//
// Moments in 8 bits.  64 consecutive elements share an exponent, and an element
// keeps 4 significant bits and its exponent relative to the block's: m a sign and
// 15 binades, v 31 binades (its root spans 15.5).  So a code is the number's
// float bits from the 20th on, less those of the window's start: encoding and
// decoding are an addition and a shift.  v matters by its ratio to m, so it is
// never held as 0 unless it is: a v below the window is held at its start,
// which makes a step smaller, never larger.  An average that changes by
// 1 - b2 a step does not move in 4 bits rounded to nearest; with a seed a value
// is rounded up with the probability of what is cut off, so that it moves as it
// should on average.
//
// The random bits are a function of seed, step and place (random_key,
// random_bits), so that a step can be taken again with the same result.
#include <cmath>

#include "stage_common.cuh"

namespace pps {
namespace {

constexpr int kMoments = PP_STAGE_BLOCK;  // elements that share an exponent
constexpr int kThreads = 256, kUnit = 8, kChunk = kThreads * kUnit;

// What the steps of one call share, computed on the device: its first kernel
// reads the step's number and the norm.
struct StepNow {
    float size, root, clip, lr;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t), the gradients' factor, lr
    uint32_t key;                // of the random bits
    int go;                      // 0: the norm is not a finite number, nothing is touched
};

__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ x >> 16) * 0x243F6A89u;
    x = (x ^ x >> 15) * 0x85A308D3u;
    return x ^ x >> 16;
}
__device__ __forceinline__ uint32_t random_key(uint64_t seed, int64_t step) {
    return mix((uint32_t)step ^ mix((uint32_t)seed ^ mix((uint32_t)(seed >> 32))));
}
__device__ __forceinline__ uint32_t block_key(uint32_t key, uint32_t block) { return mix(block ^ key); }
// 16 bits for m (the low ones) and 16 for v, of element i of a block.
__device__ __forceinline__ uint32_t random_bits(uint32_t block_key, uint32_t i) {
    uint32_t x = block_key + i * 0x9E3779B1u;
    x = (x ^ x >> 15) * 0x13198A2Fu;
    x = (x ^ x >> 12) * 0xA4093823u;
    return x ^ x >> 15;
}
// 16 more, for the parameter.
__device__ __forceinline__ uint32_t more_bits(uint32_t bits) { return bits * 0x299F31D1u >> 16; }

constexpr int kWindowM = 15, kWindowV = 31, kBlockNaN = 255;
constexpr uint32_t kNearest = 0x80000u;  // half of what is cut off

// The block's exponent, from the bits of its largest magnitude: that of its next
// larger number of 4 significant bits, so that no rounding leaves the window.
__device__ __forceinline__ int moments_exp(uint32_t largest) {
    if (largest >= 0x7F800000u) return kBlockNaN;
    return min((int)((largest + 0xFFFFFu) >> 23), 254);
}
// What a magnitude's code starts to count from.
__device__ __forceinline__ int window_of(int exp, int window) { return (exp - window) * 8; }
__device__ __forceinline__ uint32_t encode(uint32_t magnitude, uint32_t r, int from, int least, int most) {
    return (uint32_t)min(max((int)((magnitude + r) >> 20) - from, least), most);
}
__device__ __forceinline__ float decode(uint32_t code, int from) {
    return code ? __uint_as_float((uint32_t)max((int)code + from, 0) << 20) : 0.f;
}

// Two at a time, in the halves of a word, where nothing leaves the window: a
// number's upper 16 bits are 16 times its code counted from 0.  An element of
// 10 bytes (all in 16 bits, moments in 8) leaves an SM some 55 instructions a
// lane at the memory's rate, half of them at most whole-number ones.
struct Window {
    int exp, from;
    // codes of a block are read two at a time unless it holds NaN or numbers below 2^-96 and the like
    __device__ __forceinline__ bool reads(uint2 c, uint32_t sign) const {
        return exp != kBlockNaN && (from >= 0 || ((c.x | c.y) & ~sign) == 0);
    }
    // and written, unless its largest is not finite, or as large or small as that
    __device__ __forceinline__ bool writes() const { return from >= 0 && exp < 254; }
};
__device__ __forceinline__ Window window_of_block(int exp, int window) { return {exp, window_of(exp, window)}; }
__device__ __forceinline__ uint32_t both(int x) { return (uint32_t)x * 0x10001u; }
// The upper halves of two floats from two codes without sign.
__device__ __forceinline__ uint32_t decode2(uint32_t codes, int from) {
    return __vminu2(codes, 0x10001u) * (uint32_t)(from * 16) + codes * 16;
}
// Codes from two numbers, r added to their bits; `least` where they are less.  (A sum does not reach the sign.)
template <bool SIGN>
__device__ __forceinline__ uint32_t encode2(uint32_t a, uint32_t b, int from, int least) {
    const uint32_t h = __byte_perm(a, b, 0x7632), t = __vmaxu2(h >> 4 & 0x07FF07FFu, both(from + least)) - both(from);
    return SIGN ? t | (h >> 8 & 0x00800080u) : t;
}

constexpr float kNaN = __builtin_nanf("");

// In assembly: the step takes 10 % longer with the intrinsics.
__device__ __forceinline__ uint64_t pair_of(float2 x) { return (uint64_t)__float_as_uint(x.y) << 32 | __float_as_uint(x.x); }
__device__ __forceinline__ float2 of_pair(uint64_t x) { return {__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)(x >> 32))}; }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(pair_of(a)), "l"(pair_of(b)));
    return of_pair(y);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(pair_of(a)), "l"(pair_of(b)), "l"(pair_of(c)));
    return of_pair(y);
}

// The root is a normal number or 0 whatever x is, and so is eps (checked), so what is below 2^-126 plays no part in the
// reciprocal.
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool NORMAL>
__device__ __forceinline__ float root(float x) {
    float y;
    if (NORMAL) asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    else asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 8 consecutive elements.
template <bool VEC>
__device__ __forceinline__ void load(const float *p, int n, float (&v)[8]) {
    if (VEC) {
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "l"(p));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? p[j] : 0.f;
    }
}
template <bool VEC>
__device__ __forceinline__ void load(const uint16_t *p, int n, float (&v)[8]) {
    if (VEC) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[2 * j] = bf16_lo(w[j]), v[2 * j + 1] = bf16_hi(w[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? bf16_to_f32(p[j]) : 0.f;
    }
}
template <bool VEC>
__device__ __forceinline__ void store(float *p, int n, const float (&v)[8]) {
    if (VEC) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                     "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                     : "memory");
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = v[j];
    }
}
template <bool VEC>
__device__ __forceinline__ void store(uint16_t *p, int n, const float (&v)[8]) {
    if (VEC) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(f32_to_bf16x2(v[0], v[1]), f32_to_bf16x2(v[2], v[3]),
                                                   f32_to_bf16x2(v[4], v[5]), f32_to_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = f32_to_bf16(v[j]);
    }
}

// The upper halves of 8 floats.
template <bool VEC>
__device__ __forceinline__ void store_cut(uint16_t *p, int n, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __byte_perm(__float_as_uint(v[2 * j]), __float_as_uint(v[2 * j + 1]), 0x7632);
    if (VEC) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
}

// A tensor of the step, as the kernels have it.
struct Entry {
    void *p;
    const void *g;
    uint16_t *copy;
    int64_t n;
    uint32_t at;     // its first block of moments
    uint32_t first;  // its first chunk among the launch's
    float decay;
    int vec;  // p, g and copy may be read 8 elements at a time
};
// So many tensors to a launch: they are the kernel's parameters, 1.6 or 31 KB.
constexpr int kFewEntries = 32, kManyEntries = 640, kMarks = 64;
template <int N>
struct Entries {
    int count, shift;
    uint16_t from[kMarks + 1];  // the entry of chunk i << shift
    Entry e[N];

    void mark(int64_t chunks) {
        for (shift = 0; (chunks - 1) >> shift >= kMarks; ++shift) {}
        for (int i = 0, j = 0; i <= kMarks; ++i) {
            while (j + 1 < count && e[j + 1].first <= (uint64_t)i << shift) ++j;
            from[i] = (uint16_t)j;
        }
    }
};
static_assert(sizeof(Entries<kManyEntries>) + 256 < 32764);

// A look among the marks, then two or three among the entries: with eight among
// 161 entries the step of 90 million elements took 246 us, 239 with marks.
template <int N>
__device__ __forceinline__ const Entry &entry_of(const Entries<N> &t, uint32_t chunk) {
    const uint32_t at = chunk >> t.shift;
    int lo = t.from[at], hi = t.from[at + 1] + 1;  // the last whose first chunk is no later
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.e[mid].first <= chunk) lo = mid;
        else hi = mid;
    }
    return t.e[lo];
}

struct Moments {
    void *m, *v;
    uint8_t *m_exp, *v_exp;  // null: 32 bits
};
struct Rates {
    float b1, c1, b2, c2, eps;  // c1 = 1 - b1, c2 = 1 - b2
    int random;
    uint32_t sixteen, eight;  // no constants, so that their products and sums are left to the multipliers
};

// 8 codes' numbers, a sign in bit 7 of each byte where SIGN.
template <int WINDOW, bool SIGN>
__device__ __forceinline__ void read_codes(uint2 c, int exp, float (&x)[8]) {
    const Window w = window_of_block(exp, WINDOW);
    constexpr uint32_t kSign = SIGN ? 0x80u : 0u;
    if (w.reads(c, kSign * 0x01010101u)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t two = __byte_perm(j < 2 ? c.x : c.y, 0, j & 1 ? 0x4342 : 0x4140);
            uint32_t h = decode2(SIGN ? two & 0x007F007Fu : two, w.from);
            if (SIGN) h |= (two & 0x00800080u) << 8;
            x[2 * j] = __uint_as_float(h << 16), x[2 * j + 1] = __uint_as_float(h & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = (j < 4 ? c.x : c.y) >> (8 * (j & 3)) & 255;
            x[j] = exp == kBlockNaN ? kNaN : __uint_as_float(__float_as_uint(decode(b & ~kSign & 255, w.from)) | (b & kSign) << 24);
        }
    }
}
// Codes of 8 numbers; largest: the bits of the block's largest magnitude, r: what is added before bits are cut off;
// zero: where there is no sign, whether some may be 0, which alone a code of 0 stands for.
template <int WINDOW, bool SIGN, class R>
__device__ __forceinline__ uint2 write_codes(const float (&x)[8], uint32_t largest, int exp, bool zero, const R &r) {
    const Window w = window_of_block(exp, WINDOW);
    constexpr int kLeast = SIGN ? 0 : 1, kMost = SIGN ? 127 : 255;
    if (largest == 0 || exp == kBlockNaN) return make_uint2(0, 0);
    if (w.writes() && !zero) {
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a = __float_as_uint(x[2 * j]), b = __float_as_uint(x[2 * j + 1]);
            h[j] = encode2<SIGN>(a + r(2 * j), b + r(2 * j + 1), w.from, kLeast);
        }
        return make_uint2(__byte_perm(h[0], h[1], 0x6420), __byte_perm(h[2], h[3], 0x6420));
    }
    uint32_t c[2] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t a = __float_as_uint(x[j]);
        uint32_t b = 0;
        if (SIGN || a) b = encode(SIGN ? a & 0x7FFFFFFFu : a, r(j), w.from, kLeast, kMost);
        if (SIGN) b |= a >> 24 & 128;
        c[j >> 2] |= b << (8 * (j & 3));
    }
    return make_uint2(c[0], c[1]);
}
// The bits of the largest magnitude, those of a NaN above all others, of the block that 8 lanes hold.
__device__ __forceinline__ uint32_t largest_of_block(const float (&x)[8]) {
    float a = fabsf(x[7]);
#pragma unroll
    for (int j = 0; j < 3; ++j)
        asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(fabsf(x[2 * j])), "f"(fabsf(x[2 * j + 1])));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(fabsf(x[6])));
    uint32_t b = __float_as_uint(a);
#pragma unroll
    for (int o = 4; o; o >>= 1) b = max(b, __shfl_xor_sync(~0u, b, o));
    return b;
}
__device__ __forceinline__ float least_of(const float (&x)[8]) {
    float a = x[7];
#pragma unroll
    for (int j = 0; j < 3; ++j) asm("min.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(x[2 * j]), "f"(x[2 * j + 1]));
    return fminf(a, x[6]);
}

// 8 elements of one tensor, from element i on, of which n exist; held: whether
// they have moments (whole blocks, past the tensor's end as well).  In 8 bits the
// 8 lanes of an aligned group have one block, and all lanes of a warp are here.
template <class P, class G, bool SMALL, bool VEC>
__device__ __forceinline__ void step_unit(const Entry &e, int64_t i, int n, bool held, const Moments &mo, const Rates &r,
                                          const StepNow *step) {
    float p[8], g[8], m[8], v[8];
    const int64_t at = (int64_t)e.at * kMoments + i;
    const uint32_t block = e.at + (uint32_t)(i / kMoments);
    uint2 cm = make_uint2(0, 0), cv = make_uint2(0, 0);
    int em = 0, ev = 0;
    if (SMALL && held) {
        cm = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(mo.m) + at);
        cv = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(mo.v) + at);
        em = mo.m_exp[block], ev = mo.v_exp[block];
    }
    load<VEC>(static_cast<const P *>(e.p) + i, n, p);
    load<VEC>(static_cast<const G *>(e.g) + i, n, g);
    const StepNow now = *step;
    if constexpr (SMALL) {
        read_codes<kWindowM, true>(cm, em, m);
        read_codes<kWindowV, false>(cv, ev, v);
    } else {
        load<true>(static_cast<const float *>(mo.m) + at, 8, m);
        load<true>(static_cast<const float *>(mo.v) + at, 8, v);
    }
    if (!now.go) return;
    if (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j >= n) g[j] = m[j] = v[j] = 0.f;  // nothing is kept past the tensor's end
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        // Products and sums are rounded apart, as written above, so that the 8 bits are the same whatever computes them:
        // single sums, for a sum of a pair would be made one with its product.
        const float2 x = mul2({g[j], g[j + 1]}, {now.clip, now.clip});
        const float2 a = mul2({r.b1, r.b1}, {m[j], m[j + 1]}), c = mul2({r.c1, r.c1}, x);
        const float2 b = mul2({r.b2, r.b2}, {v[j], v[j + 1]}), d = mul2({r.c2, r.c2}, mul2(x, x));
        m[j] = __fadd_rn(a.x, c.x), m[j + 1] = __fadd_rn(a.y, c.y);
        v[j] = __fadd_rn(b.x, d.x), v[j + 1] = __fadd_rn(b.y, d.y);
    }
    const bool tiny = !(least_of(v) >= 0x1p-126f);  // no normal numbers, or 0
    float d[8];
    if (tiny) {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = root<false>(v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = root<true>(v[j]);
    }
    const float shrink = -now.lr * e.decay;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 den = fma2({d[j], d[j + 1]}, {now.root, now.root}, {r.eps, r.eps});
        const float2 q = mul2({m[j], m[j + 1]}, {reciprocal(den.x), reciprocal(den.y)});
        const float2 y = fma2({p[j], p[j + 1]}, {shrink, shrink}, {p[j], p[j + 1]});
        const float2 z = fma2(q, {-now.size, -now.size}, y);
        p[j] = z.x, p[j + 1] = z.y;
    }
    constexpr bool kRound = sizeof(P) == 2;
    [[maybe_unused]] uint32_t bits[8];
    if ((SMALL || kRound) && r.random) {
        const uint32_t key = block_key(now.key, block);
#pragma unroll
        for (int j = 0; j < 8; ++j) bits[j] = random_bits(key, (uint32_t)(i % kMoments) + j);
    }
    if constexpr (SMALL) {
        const uint32_t tm = largest_of_block(m), tv = largest_of_block(v);
        const int em1 = moments_exp(tm), ev1 = moments_exp(tv);
        if (r.random) {
            cm = write_codes<kWindowM, true>(m, tm, em1, false, [&](int j) { return (bits[j] & 0xFFFFu) * r.sixteen + r.eight; });
            cv = write_codes<kWindowV, false>(v, tv, ev1, tiny, [&](int j) { return (bits[j] >> 16) * r.sixteen + r.eight; });
        } else {
            cm = write_codes<kWindowM, true>(m, tm, em1, false, [](int) { return kNearest; });
            cv = write_codes<kWindowV, false>(v, tv, ev1, tiny, [](int) { return kNearest; });
        }
        if (held) {
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(mo.m) + at) = cm;
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(mo.v) + at) = cv;
            if (i % kMoments == 0) mo.m_exp[block] = (uint8_t)em1, mo.v_exp[block] = (uint8_t)ev1;
        }
    } else {
        store<true>(static_cast<float *>(mo.m) + at, 8, m);
        store<true>(static_cast<float *>(mo.v) + at, 8, v);
    }
    if (kRound && r.random) {
        // up with the probability of what is cut off; a NaN stays what it is (so does an infinity)
        const float any = ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
        const bool check = any != any;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __float_as_uint(p[j]) + more_bits(bits[j]);
            if (!check || p[j] == p[j]) p[j] = __uint_as_float(b);
        }
        store_cut<VEC>(static_cast<uint16_t *>(e.p) + i, n, p);
        return;
    }
    store<VEC>(static_cast<P *>(e.p) + i, n, p);
    if (e.copy) store<VEC>(e.copy + i, n, p);
}

__device__ __forceinline__ void prefetch(const void *p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Moments in 8 bits leave few bytes in flight: a block brings what another will
// read so many chunks later into the L2 cache, two thirds of the blocks that run
// at once (571 million elements with 32-bit parameters 1.43 ms, 1.53 without, 1.75
// with four times as many).  32-bit moments fill the memory's queues by
// themselves (2.40 ms, 2.45 with it).
constexpr int64_t kAhead = 400;
template <class P, class G, bool SMALL, int N>
__global__ void __launch_bounds__(kThreads, SMALL ? 4 : 3) k_step(const __grid_constant__ Entries<N> t, const Moments mo, const Rates r,
                                                   const StepNow *at) {
    let_next_start();
    const Entry &e = entry_of(t, blockIdx.x);
    const int64_t i = (int64_t)(blockIdx.x - e.first) * kChunk + threadIdx.x * kUnit;
    const int n = i >= e.n ? 0 : e.n - i < kUnit ? (int)(e.n - i) : kUnit;
    const bool held = i < (e.n + kMoments - 1) / kMoments * kMoments;
    bool wide = e.vec && n == kUnit;
    after_previous();
    if (SMALL && threadIdx.x == 0 && e.vec && i + (kAhead + 1) * kChunk <= e.n) {
        const int64_t a = i + kAhead * kChunk, h = (int64_t)e.at * kMoments + a;
        prefetch(static_cast<const P *>(e.p) + a, kChunk * sizeof(P));
        prefetch(static_cast<const G *>(e.g) + a, kChunk * sizeof(G));
        prefetch(static_cast<const uint8_t *>(mo.m) + h, kChunk);
        prefetch(static_cast<const uint8_t *>(mo.v) + h, kChunk);
    }
    if constexpr (SMALL) wide = __all_sync(~0u, wide);  // a warp goes one way: its lanes shuffle
    else if (!held) return;
    if (wide) step_unit<P, G, SMALL, true>(e, i, n, held, mo, r, at);
    else step_unit<P, G, SMALL, false>(e, i, n, held, mo, r, at);
}

// b^t by squaring: off by t roundings at most, and nearly 0 where those are many.
__device__ __forceinline__ double power(double b, int64_t t) {
    double y = 1;
    for (; t > 0; t >>= 1, b *= b)
        if (t & 1) y *= b;
    return y;
}

// The step's number goes up, and all that depends on it is computed, in 64 bits.
__global__ void k_step_begin(int64_t *step, const float *lr_at, double lr, double b1, double b2, const float *norm,
                             const double *wide, double max_norm, uint64_t seed, StepNow *now) {
    let_next_start();
    after_previous();
    const float nrm = norm ? *norm : 0.f;
    // the norm before it was rounded, if it is still that
    const double full = norm && wide && (float)*wide == nrm ? *wide : nrm;
    const int64_t t = *step + 1;
    const double rate = lr_at ? *lr_at : lr;
    const double rest = 1 - power(threadIdx.x ? b2 : b1, t), bias = threadIdx.x ? 1 / sqrt(rest) : rate / rest;
    const double other = __shfl_down_sync(3u, bias, 1);
    if (threadIdx.x) return;
    StepNow s;
    s.go = isfinite(nrm);
    s.size = (float)bias, s.root = (float)other, s.lr = (float)rate;
    s.clip = full > max_norm ? (float)(max_norm / full) : 1.f;
    s.key = random_key(seed, t);
    *now = s;
    if (s.go) *step = t;
}

// ---- the norm: a block's sum of squares, then all blocks'

constexpr int kNormThreads = 512;

// Two sums of squares in 32 bits that keep what each addition cuts off: as good
// as 64 bits, which the GPU adds at a fiftieth of the rate.  (The factor of a clip
// is then the same however the sum was shared out, and with it what moments in 8
// bits are rounded to.)
struct Squares {
    float2 s = {0.f, 0.f}, low = {0.f, 0.f};
    __device__ __forceinline__ void add(float2 x) {
        const float2 t = __ffma2_rn(x, x, s), z = __fadd2_rn(t, minus(s));  // z: x^2 as far as t has it
        low = __fadd2_rn(low, __fadd2_rn(__fadd2_rn(s, minus(__fadd2_rn(t, minus(z)))), __ffma2_rn(x, x, minus(z))));
        s = t;
    }
    static __device__ __forceinline__ float2 minus(float2 x) { return {-x.x, -x.y}; }
    __device__ __forceinline__ double total() const {
        // beyond the range the rest is no number
        return ((double)s.x + (double)s.y) + (isfinite(s.x) && isfinite(s.y) ? (double)low.x + (double)low.y : 0.);
    }
};

// The sum of a thread's squares, of elements i on below `to`; SCALED: of 2^90 times the elements.
template <bool SCALED, class G>
__device__ __forceinline__ double squares_of(const G *g, int64_t i, int64_t to, bool vec) {
    constexpr int kEach = kNormThreads * kUnit;
    const auto pair = [](float a, float b) { return SCALED ? mul2({a, b}, {0x1p90f, 0x1p90f}) : make_float2(a, b); };
    Squares s[2];
    if (vec) {
        for (; i + kUnit + kEach <= to; i += 2 * kEach) {
            float a[8], b[8];
            load<true>(g + i, 8, a);
            load<true>(g + i + kEach, 8, b);
#pragma unroll
            for (int j = 0; j < 8; j += 2) s[0].add(pair(a[j], a[j + 1])), s[1].add(pair(b[j], b[j + 1]));
        }
    }
    for (; i < to; i += kEach) {
        float a[8];
        load<false>(g + i, to - i < kUnit ? (int)(to - i) : kUnit, a);
#pragma unroll
        for (int j = 0; j < 8; j += 4) s[0].add(pair(a[j], a[j + 1])), s[1].add(pair(a[j + 2], a[j + 3]));
    }
    return s[0].total() + s[1].total();
}

// A block's sum, in thread 0.
__device__ __forceinline__ double sum_of_block(double x, double (&sh)[kNormThreads / 32]) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0;
    if (threadIdx.x == 0)
        for (int k = 0; k < kNormThreads / 32; ++k) x += sh[k];
    return x;
}

// A square below 2^-126 loses bits, of a gradient below 2^-75 all: each 2^-147 at most with its rest, nothing beside a
// block's sum of 2^-70.  A block that has less takes its elements, all below 2^-35 then, once more, 2^90 times as large:
// subnormal ones become normal, and no sum exceeds 2^110.  571 million float gradients take 324 us, 322 without this; a
// block whose gradients are all 0 reads them twice (all of them 626 us).  To look for bits that are not 0 on the way
// spares that, but takes 5 % more of every call (337 us).
constexpr double kSmallSum = 0x1p-70;

template <class G, int N>
__global__ void __launch_bounds__(kNormThreads) k_norm(const __grid_constant__ Entries<N> t, int64_t chunk, double *part) {
    __shared__ double sh[kNormThreads / 32], again[kNormThreads / 32];
    let_next_start();
    const Entry &e = entry_of(t, blockIdx.x);
    const int64_t from = (int64_t)(blockIdx.x - e.first) * chunk, to = min(from + chunk, e.n);
    const G *g = static_cast<const G *>(e.g);
    after_previous();
    const int64_t i = from + threadIdx.x * kUnit;
    double x = sum_of_block(squares_of<false>(g, i, to, e.vec), sh);
    if (__syncthreads_or(threadIdx.x == 0 && x < kSmallSum)) x = sum_of_block(squares_of<true>(g, i, to, e.vec) * 0x1p-180, again);
    if (threadIdx.x == 0) part[blockIdx.x] = x;
}

__global__ void __launch_bounds__(1024) k_norm_join(const double *part, int64_t n, float *norm, double *wide) {
    __shared__ double sh[32];
    let_next_start();
    after_previous();
    double x = 0;
    for (int64_t i = threadIdx.x; i < n; i += 1024) x += part[i];
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    x = sh[threadIdx.x];
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    if (threadIdx.x) return;
    x = sqrt(x);
    *norm = (float)x;
    if (wide) *wide = x;
}

// What moments in 8 bits stand for, as bf16 (exactly): 8 elements of both a thread.
__global__ void __launch_bounds__(kThreads) k_moments(const Moments mo, int64_t n, uint16_t *m, uint16_t *v) {
    let_next_start();
    after_previous();
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kUnit;
    if (i >= n) return;
    const uint2 cm = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(mo.m) + i);
    const uint2 cv = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(mo.v) + i);
    float x[8];
    read_codes<kWindowM, true>(cm, mo.m_exp[i / kMoments], x);
    store<true>(m + i, 8, x);
    read_codes<kWindowV, false>(cv, mo.v_exp[i / kMoments], x);
    store<true>(v + i, 8, x);
}

// ---- host side

bool aligned_to(const void *p, uintptr_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

bool bad_tensor(const pp_stage_tensor &t, bool step) {
    if (t.n < 0 || (t.p_float & ~1) || (t.g_float & ~1)) return true;
    if (t.n == 0) return false;
    if (!t.g || !aligned_to(t.g, t.g_float ? 4 : 2)) return true;
    if (!step) return false;
    return !t.p || !aligned_to(t.p, t.p_float ? 4 : 2) || (t.copy && (!t.p_float || !aligned_to(t.copy, 2))) || t.at < 0 ||
           t.at % kMoments || !(std::fabs(t.decay) <= 3e38f);
}

// 31 KB, one for all instances below.
Entries<kManyEntries> &table_of_thread() {
    static thread_local Entries<kManyEntries> t;
    return t;
}

// Hands the tensors that `want` picks to `launch(table, chunks)`, as many at a
// time as a table holds; chunk: elements of a block.
template <class Want, class Launch>
int in_tables(const pp_stage_tensor *list, int64_t count, int64_t chunk, const Want &want, const Launch &launch) {
    Entries<kManyEntries> &many = table_of_thread();
    int64_t i = 0;
    while (i < count) {
        many.count = 0;
        int64_t chunks = 0;
        for (; i < count && many.count < kManyEntries; ++i) {
            const pp_stage_tensor &t = list[i];
            if (t.n == 0 || !want(t)) continue;
            const int64_t c = ceil_div(t.n, chunk);
            if (chunks + c > 0x7FFFFFFF) break;  // the rest in another launch
            const bool vec = aligned_to(t.p, t.p_float ? 32 : 16) && aligned_to(t.g, t.g_float ? 32 : 16) && aligned_to(t.copy, 16);
            many.e[many.count++] = {t.p, t.g, t.copy, t.n, (uint32_t)(t.at / kMoments), (uint32_t)chunks, t.decay, vec};
            chunks += c;
        }
        if (many.count == 0) continue;
        int rc;
        if (many.count <= kFewEntries) {
            Entries<kFewEntries> few;
            few.count = many.count;
            for (int j = 0; j < many.count; ++j) few.e[j] = many.e[j];
            few.mark(chunks);
            rc = launch(few, chunks);
        } else {
            many.mark(chunks);
            rc = launch(many, chunks);
        }
        if (rc != PP_OK) return rc;
    }
    return PP_OK;
}

template <class P, class G, bool SMALL>
int step_all(const pp_stage_tensor *list, int64_t count, const Moments &mo, const Rates &r, const StepNow *now,
             cudaStream_t stream) {
    return in_tables(
        list, count, kChunk,
        [](const pp_stage_tensor &t) { return t.p_float == (sizeof(P) == 4) && t.g_float == (sizeof(G) == 4); },
        [&]<int N>(const Entries<N> &t, int64_t chunks) {
            return launch_after(k_step<P, G, SMALL, N>, chunks, kThreads, 0, stream, 1, t, mo, r, now);
        });
}

// Elements to a block of the norm: about 8 blocks to an SM, 16 K elements at least.
int64_t norm_chunk(const pp_stage_tensor *list, int64_t count) {
    int64_t n = 0;
    for (int64_t i = 0; i < count; ++i) n += list[i].n;
    return std::max<int64_t>(round_up(ceil_div(n, (int64_t)sm_count() * 8), 2 * kNormThreads * kUnit), 16384);
}
int64_t norm_blocks(const pp_stage_tensor *list, int64_t count) {
    const int64_t chunk = norm_chunk(list, count);
    int64_t n = 0;
    for (int64_t i = 0; i < count; ++i) n += ceil_div(list[i].n, chunk);
    return n;
}

bool bad_list(const pp_stage_tensor *list, int64_t count, bool step) {
    if (count < 0 || (count > 0 && !list)) return true;
    for (int64_t i = 0; i < count; ++i)
        if (bad_tensor(list[i], step)) return true;
    return false;
}
bool too_long(const pp_stage_tensor *list, int64_t count) {
    for (int64_t i = 0; i < count; ++i)
        if (list[i].n > PP_STAGE_MAX_ELEMENTS) return true;
    return count > PP_STAGE_MAX_TENSORS;
}

}  // namespace
}  // namespace pps

using namespace pps;

extern "C" size_t pp_stage_grad_norm_workspace(const pp_stage_tensor *list, int64_t count) {
    if (bad_list(list, count, false) || too_long(list, count)) return 0;
    return stage_align((size_t)norm_blocks(list, count) * sizeof(double));
}

extern "C" int pp_stage_grad_norm(const pp_stage_tensor *list, int64_t count, float *norm, double *wide,
                                  void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (bad_list(list, count, false) || !norm || !aligned_to(norm, 4) || !aligned_to(wide, 8)) return PP_ERR_ARG;
    if (too_long(list, count)) return PP_ERR_SIZE;
    const int64_t chunk = norm_chunk(list, count), blocks = norm_blocks(list, count);
    if (blocks && (!workspace || !aligned_to(workspace, kStageAlign) || workspace_bytes < blocks * sizeof(double))) return PP_ERR_ARG;
    double *part = static_cast<double *>(workspace);
    const auto all = [&]<class G>(const G *) {
        return in_tables(
            list, count, chunk, [](const pp_stage_tensor &t) { return t.g_float == (sizeof(G) == 4); },
            [&]<int N>(Entries<N> t, int64_t chunks) {
                for (int i = 0; i < t.count; ++i) t.e[i].vec = aligned_to(t.e[i].g, sizeof(G) == 4 ? 32 : 16);
                const int rc = launch_after(k_norm<G, N>, chunks, kNormThreads, 0, stream, 1, t, chunk, part);
                part += chunks;
                return rc;
            });
    };
    int rc = all((const float *)nullptr);
    if (rc == PP_OK) rc = all((const uint16_t *)nullptr);
    if (rc == PP_OK)
        rc = launch_after(k_norm_join, 1, 1024, 0, stream, 1, (const double *)workspace, blocks, norm, wide);
    return rc;
}

extern "C" size_t pp_stage_adamw_workspace(void) { return kStageAlign; }

extern "C" int pp_stage_adamw(const pp_stage_tensor *list, int64_t count, void *m, void *v, uint8_t *m_exp, uint8_t *v_exp,
                              int64_t held, int64_t *step, const float *lr_at, double lr, double beta1, double beta2,
                              double eps, const float *norm, const double *wide, double max_norm, int random, uint64_t seed, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
    if (bad_list(list, count, true) || held < 0 || held % kMoments || !step || !aligned_to(step, 8)) return PP_ERR_ARG;
    if (too_long(list, count) || held > PP_STAGE_MAX_ELEMENTS) return PP_ERR_SIZE;
    if (!m != !v || !m_exp != !v_exp || (held > 0 && !m)) return PP_ERR_ARG;
    if (!aligned_to(m, 32) || !aligned_to(v, 32)) return PP_ERR_ARG;
    for (int64_t i = 0; i < count; ++i)
        if (list[i].n && list[i].n > held - list[i].at) return PP_ERR_ARG;
    if (!(beta1 >= 0 && beta1 < 1 && beta2 >= 0 && beta2 < 1 && (eps == 0 || (eps >= 0x1p-126 && eps <= 3e38)))) return PP_ERR_ARG;
    if (lr_at ? !aligned_to(lr_at, 4) : !(std::fabs(lr) <= 3e38)) return PP_ERR_ARG;
    if (norm && (!aligned_to(norm, 4) || !aligned_to(wide, 8) || !(max_norm > 0))) return PP_ERR_ARG;
    if (!workspace || !aligned_to(workspace, kStageAlign) || workspace_bytes < sizeof(StepNow)) return PP_ERR_ARG;
    StepNow *now = static_cast<StepNow *>(workspace);
    const Moments mo{m, v, m_exp, v_exp};
    const Rates r{(float)beta1, (float)(1 - beta1), (float)beta2, (float)(1 - beta2), (float)eps, random != 0, 16, 8};
    int rc = launch_after(k_step_begin, 1, 2, 0, stream, 1, step, lr_at, lr, beta1, beta2, norm, wide, max_norm, seed, now);
    const auto all = [&]<class P, class G>(const P *, const G *) {
        if (rc != PP_OK) return;
        rc = m_exp ? step_all<P, G, true>(list, count, mo, r, now, stream) : step_all<P, G, false>(list, count, mo, r, now, stream);
    };
    all((const float *)nullptr, (const float *)nullptr);
    all((const float *)nullptr, (const uint16_t *)nullptr);
    all((const uint16_t *)nullptr, (const float *)nullptr);
    all((const uint16_t *)nullptr, (const uint16_t *)nullptr);
    return rc;
}

extern "C" int pp_stage_adamw_moments(const uint8_t *m, const uint8_t *v, const uint8_t *m_exp, const uint8_t *v_exp,
                                      int64_t held, uint16_t *m_values, uint16_t *v_values, cudaStream_t stream) {
    if (held < 0 || held % kMoments) return PP_ERR_ARG;
    if (held > PP_STAGE_MAX_ELEMENTS) return PP_ERR_SIZE;
    if (held == 0) return PP_OK;
    if (!m || !v || !m_exp || !v_exp || !m_values || !v_values) return PP_ERR_ARG;
    if (!aligned_to(m, 8) || !aligned_to(v, 8) || !aligned_to(m_values, 16) || !aligned_to(v_values, 16)) return PP_ERR_ARG;
    const Moments mo{(void *)m, (void *)v, (uint8_t *)m_exp, (uint8_t *)v_exp};
    return launch_after(k_moments, ceil_div(held, kThreads * kUnit), kThreads, 0, stream, 1, mo, held, m_values, v_values);
}
