// Rotary positions on the way from a product's output to where attention reads: queries and
// keys out of place or in place, keys into a paged cache with their values beside them.
// Pair i < r/2 of a head's first r elements -- (i, i + r/2) or (2i, 2i + 1) -- turns by
// theta = p f_i and is scaled by c; the other elements pass through:
//     a' = c (a cos theta - b sin theta),   b' = c (b cos theta + a sin theta)
//
// The angle.  f_i / 2 pi, the turns that a position adds, is kept as a fraction of 2^64, so the
// angle modulo a turn is the low 64 bits of one integer product: exact but for the fraction's
// own rounding, p 2^-53 turns at most, whatever the position.  No table of positions is built,
// read or outgrown (at 131072 positions of 64 frequencies one would fill half the L2).  The nearest quarter turn is
// split off, and sine and cosine of the rest, |x| <= pi/4, are their Taylor polynomials to x^9
// and x^10, whose next terms are below 1.8e-9 and 1.2e-10.
//
// Work.  A unit is two vectors of a head whose pairs have the same frequencies: the vectors at
// i and i + r/2, or two adjacent ones; of the part that passes through, two adjacent ones.  A
// thread takes its unit in several heads of a token, so that an angle is formed once for them.
// Bound by memory: each element is read and written once.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "foak_ce.h"
#include "internal.h"
#include "rotary.h"

namespace foak {

namespace {

constexpr int kThreads = 256;

// W elements of ES bytes in one access.
template <int ES, int W>
struct Piece {
    static constexpr int kBytes = ES * W;
    uint32_t w[kBytes >= 4 ? kBytes / 4 : 1];

    __device__ __forceinline__ void load(const char* p) {
        if constexpr (kBytes == 16) {
            const uint4 v = ld_global_v4(p);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (kBytes == 8) {
            asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p) : "memory");
        } else if constexpr (kBytes == 4) {
            asm volatile("ld.global.b32 %0, [%1];" : "=r"(w[0]) : "l"(p) : "memory");
        } else {
            asm volatile("ld.global.u16 %0, [%1];" : "=r"(w[0]) : "l"(p) : "memory");
        }
    }
    __device__ __forceinline__ void store(char* p) const {
        if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
        else *reinterpret_cast<unsigned short*>(p) = static_cast<unsigned short>(w[0]);
    }
    __device__ __forceinline__ void get(float (&f)[W]) const {
        if constexpr (ES == 4) {
#pragma unroll
            for (int k = 0; k < W; ++k) f[k] = __uint_as_float(w[k]);
        } else if constexpr (W == 1) {
            f[0] = bf16_lo(w[0]);
        } else {
#pragma unroll
            for (int k = 0; k < W / 2; ++k) {
                f[2 * k] = bf16_lo(w[k]);
                f[2 * k + 1] = bf16_hi(w[k]);
            }
        }
    }
    // rounded to nearest even, the one rounding of the output
    __device__ __forceinline__ void set(const float (&f)[W]) {
        if constexpr (ES == 4) {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k] = __float_as_uint(f[k]);
        } else if constexpr (W == 1) {
            w[0] = pack_bf16x2(f[0], 0.f);
        } else {
#pragma unroll
            for (int k = 0; k < W / 2; ++k) w[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
        }
    }
};

// c times cosine and sine of `turn` 2^-64 turns.
__device__ __forceinline__ void turn_cos_sin(uint64_t turn, float c, float sign, float& co, float& si) {
    const uint32_t hi = static_cast<uint32_t>(turn >> 32);
    const uint32_t quarter = (hi + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(hi - (quarter << 30));  // [-2^29, 2^29]: an eighth of a turn
    const float x = static_cast<float>(rest) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float z = x * x;
    float s = fmaf(z, 2.7557319223985893e-6f, -1.9841269841269841e-4f);
    s = fmaf(z, s, 8.3333333333333333e-3f);
    s = fmaf(z, s, -1.6666666666666667e-1f);
    s = fmaf(x * z, s, x);
    float k = fmaf(z, -2.7557319223985888e-7f, 2.4801587301587302e-5f);
    k = fmaf(z, k, -1.3888888888888889e-3f);
    k = fmaf(z, k, 4.1666666666666667e-2f);
    k = fmaf(z, k, -0.5f);
    k = fmaf(z, k, 1.f);
    const float a = (quarter & 1u) ? s : k, b = (quarter & 1u) ? k : s;
    co = ((quarter + 1u) & 2u) ? -c * a : c * a;
    si = (quarter & 2u) ? -c * sign * b : c * sign * b;
}

// Where a unit's vectors lie in its head.
struct Unit {
    int at0, at1;  // elements
    int freq;      // of the first pair; -1: passes through
    bool two;      // the second vector is there
    bool turn1;    // and turns
};

template <int W, bool INTERLEAVED>
__device__ __forceinline__ Unit unit_of(int j, int d, int r) {
    Unit u;
    if constexpr (!INTERLEAVED) {
        const int half = r / 2, turning = half / W;
        if (j < turning) {
            u.at0 = j * W;
            u.at1 = half + j * W;
            u.freq = j * W;
            u.two = u.turn1 = true;
            return u;
        }
        j -= turning;
    } else {
        const int turning = (r + 2 * W - 1) / (2 * W);
        if (j < turning) {
            u.at0 = j * 2 * W;
            u.at1 = u.at0 + W;
            u.freq = j * W;
            u.two = u.turn1 = u.at1 < r;
            return u;
        }
        j -= turning;
    }
    u.at0 = r + j * 2 * W;
    u.at1 = u.at0 + W;
    u.freq = -1;
    u.two = u.at1 < d;
    u.turn1 = false;
    return u;
}

template <int W>
__host__ __device__ __forceinline__ int units_of(int d, int r, bool interleaved) {
    const int turning = interleaved ? (r + 2 * W - 1) / (2 * W) : r / 2 / W;
    return turning + (d - r + 2 * W - 1) / (2 * W);
}

// The CTAs' ranges: move m has blocks [first[m], first[m + 1]) of kThreads (token, heads, unit)
// items, units fastest.
struct Split {
    unsigned first[4];
    unsigned units[3];
    unsigned groups[3];  // of HPT heads
    int64_t t0, t1;      // the launch's tokens
};

template <int ES, int W, bool INTERLEAVED, int HPT>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, const Split sp) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    const unsigned m = blockIdx.x >= sp.first[2] ? 2 : blockIdx.x >= sp.first[1] ? 1 : 0;
    const HeadMove& mv = a.move[m];
    const unsigned item = (blockIdx.x - sp.first[m]) * kThreads + threadIdx.x;
    const unsigned units = sp.units[m], groups = sp.groups[m];
    const unsigned rest = item / units;
    const int64_t t = sp.t0 + rest / groups;
    if (t >= sp.t1) return;
    const int h0 = static_cast<int>(rest % groups) * HPT;
    const Unit u = unit_of<W, INTERLEAVED>(static_cast<int>(item % units), mv.d, mv.r);
    const int64_t slot = a.slots ? a.slots[t] : 0;
    const int64_t p = u.freq >= 0 ? a.positions[t] : 0;
    const char* src = mv.src + (t * mv.src_t + h0 * mv.src_h) * ES;
    Piece<ES, W> v[HPT][2];
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        if (h0 + i < mv.H) {
            v[i][0].load(src + (i * mv.src_h + u.at0) * ES);
            if (u.two) v[i][1].load(src + (i * mv.src_h + u.at1) * ES);
            else v[i][1] = v[i][0];
        }
    }
    if (a.slots && static_cast<uint64_t>(slot) >= static_cast<uint64_t>(a.capacity)) {  // not a token of the cache
        if (slot >= 0 && a.err) atomicOr(reinterpret_cast<unsigned*>(a.err), FOAK_ERRBIT_PAGE_RANGE);
        return;
    }
    int64_t to = t * mv.dst_t;
    if (mv.paged) to = slot / a.page_size * mv.dst_page + slot % a.page_size * mv.dst_t;
    char* dst = mv.dst + (to + h0 * mv.dst_h) * ES;
    if (u.freq >= 0) {
        float co[W], si[W];
        constexpr int F = INTERLEAVED && W > 1 ? W / 2 : W;  // frequencies of one vector
#pragma unroll
        for (int k = 0; k < W; ++k)
            if (k < F || u.turn1)
                turn_cos_sin(static_cast<uint64_t>(p) * a.turns[u.freq + k], a.factor, a.sign, co[k], si[k]);
#pragma unroll
        for (int i = 0; i < HPT; ++i) {
            if (h0 + i >= mv.H) continue;
            float x[W], y[W], ox[W], oy[W];
            v[i][0].get(x);
            v[i][1].get(y);
            if constexpr (INTERLEAVED && W > 1) {
#pragma unroll
                for (int k = 0; k < W / 2; ++k) {
                    ox[2 * k] = fmaf(x[2 * k], co[k], -x[2 * k + 1] * si[k]);
                    ox[2 * k + 1] = fmaf(x[2 * k + 1], co[k], x[2 * k] * si[k]);
                    oy[2 * k] = fmaf(y[2 * k], co[F + k], -y[2 * k + 1] * si[F + k]);
                    oy[2 * k + 1] = fmaf(y[2 * k + 1], co[F + k], y[2 * k] * si[F + k]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < W; ++k) {
                    ox[k] = fmaf(x[k], co[k], -y[k] * si[k]);
                    oy[k] = fmaf(y[k], co[k], x[k] * si[k]);
                }
            }
            v[i][0].set(ox);
            v[i][1].set(oy);
        }
    }
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        if (h0 + i < mv.H) {
            v[i][0].store(dst + (i * mv.dst_h + u.at0) * ES);
            if (u.two) v[i][1].store(dst + (i * mv.dst_h + u.at1) * ES);
        }
    }
}

template <int ES, int W, bool INTERLEAVED, int HPT>
cudaError_t launch_heads(const RotaryArgs& a, cudaStream_t s) {
    Split sp = {};
    uint64_t items = 1;  // of a token, the largest move's
    for (int m = 0; m < 3; ++m) {
        const HeadMove& mv = a.move[m];
        sp.units[m] = 1;
        sp.groups[m] = 1;
        if (!mv.src) continue;
        sp.units[m] = static_cast<unsigned>(units_of<W>(mv.d, mv.r, INTERLEAVED));
        sp.groups[m] = static_cast<unsigned>((mv.H + HPT - 1) / HPT);
        items = std::max(items, static_cast<uint64_t>(sp.units[m]) * sp.groups[m]);
    }
    // a launch's items of a move stay below 2^29, its blocks below 2^31
    const int64_t step = std::max<int64_t>(1, static_cast<int64_t>((1u << 29) / items));
    for (int64_t t0 = 0; t0 < a.T; t0 += step) {
        sp.t0 = t0;
        sp.t1 = std::min(a.T, t0 + step);
        for (int m = 0; m < 3; ++m) {
            const uint64_t n = a.move[m].src ? static_cast<uint64_t>(sp.t1 - t0) * sp.units[m] * sp.groups[m] : 0;
            sp.first[m + 1] = sp.first[m] + static_cast<unsigned>((n + kThreads - 1) / kThreads);
        }
        const cudaError_t e = launch_dependent(rotary_kernel<ES, W, INTERLEAVED, HPT>, dim3(sp.first[3]), dim3(kThreads),
                                               0, s, a, sp);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int ES, int W>
cudaError_t launch_width(const RotaryArgs& a, cudaStream_t s) {
    return a.interleaved ? launch_heads<ES, W, true, 1>(a, s) : launch_heads<ES, W, false, 1>(a, s);
}

// The widest access that every vector of every head allows.
int width_of(int es, const RotaryArgs& a) {
    int w = 16 / es;
    auto fits = [&](int64_t elements) {
        while (elements % w) w /= 2;
    };
    for (const HeadMove& mv : a.move) {
        if (!mv.src) continue;
        while (reinterpret_cast<uintptr_t>(mv.src) % (w * es) || reinterpret_cast<uintptr_t>(mv.dst) % (w * es)) w /= 2;
        fits(mv.src_t);
        fits(mv.src_h);
        fits(mv.dst_t);
        fits(mv.dst_h);
        fits(mv.dst_page);
        fits(mv.d);
        fits(a.interleaved ? mv.r : mv.r / 2);
        fits(mv.r);
    }
    return w;
}

// Slots and positions of a step's tokens, a thread a token: the token's sequence is the last one
// that starts at or before it.
__global__ void __launch_bounds__(kThreads)
    kv_slots_kernel(const int32_t* __restrict__ page_table, int64_t ld_table, int64_t max_pages,
                    const int32_t* __restrict__ cache_lens, const int32_t* __restrict__ seq_starts, int64_t B, int64_t T,
                    int64_t page_size, int64_t num_pages, int64_t* __restrict__ slots, int64_t* __restrict__ positions,
                    int32_t* err) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    const int64_t t = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    if (t >= T) return;
    int64_t lo = 0, hi = B + 1;  // starts before lo are <= t, those from hi on are not
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (seq_starts[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    int64_t slot = -1, pos = 0;
    if (lo > 0 && lo <= B) {  // behind no start, or before the first: padding
        const int64_t b = lo - 1, len = cache_lens[b];
        pos = len + (t - seq_starts[b]);
        const int64_t page = pos / page_size;
        int64_t id = -1;
        if (len >= 0 && page < max_pages) id = page_table[b * ld_table + page];
        if (id >= 0 && id < num_pages) slot = id * page_size + (pos - page * page_size);
        else {
            pos = 0;
            if (err) atomicOr(reinterpret_cast<unsigned*>(err), FOAK_ERRBIT_PAGE_RANGE);
        }
    }
    slots[t] = slot;
    positions[t] = pos;
}

}  // namespace

void rotary_inv_freq(double base, int64_t r, int scaling, double factor, double low, double high, double original,
                     double* inv_freq) {
    const double two_pi = 6.283185307179586476925;
    if (scaling == FOAK_ROTARY_NTK) base *= std::pow(factor, static_cast<double>(r) / static_cast<double>(r - 2));
    // the index at which a frequency makes n turns over the original context
    auto index_of = [&](double n) { return r * std::log(original / (n * two_pi)) / (2.0 * std::log(base)); };
    double first = 0.0, last = 0.0;
    if (scaling == FOAK_ROTARY_RAMP) {
        first = std::max(std::floor(index_of(high)), 0.0);
        last = std::min(std::ceil(index_of(low)), static_cast<double>(r - 1));
        if (!(last > first)) last = first + 0.001;
    }
    for (int64_t i = 0; i < r / 2; ++i) {
        const double f = std::pow(base, -2.0 * static_cast<double>(i) / static_cast<double>(r));
        double stretch = 0.0;  // the share that the factor divides
        if (scaling == FOAK_ROTARY_LINEAR) stretch = 1.0;
        if (scaling == FOAK_ROTARY_BANDS) stretch = (high - original * f / two_pi) / (high - low);
        if (scaling == FOAK_ROTARY_RAMP) stretch = (static_cast<double>(i) - first) / (last - first);
        stretch = std::min(std::max(stretch, 0.0), 1.0);
        inv_freq[i] = f * (1.0 - stretch) + f * stretch / factor;
    }
}

uint64_t rotary_turns(double inv_freq) {
    const double turns = inv_freq / 6.283185307179586476925;
    const double scaled = std::ldexp(turns - std::floor(turns), 64);
    return scaled < 18446744073709551616.0 ? static_cast<uint64_t>(scaled) : 0;  // a whole turn is none
}

cudaError_t launch_rotary(int es, const RotaryArgs& a, cudaStream_t s) {
    if (a.T == 0 || (!a.move[0].src && !a.move[1].src && !a.move[2].src)) return cudaSuccess;
    const int w = width_of(es, a);
    if (es == 2) {
        if (w == 8) return launch_width<2, 8>(a, s);
        if (w == 4) return launch_width<2, 4>(a, s);
        return w == 2 ? launch_width<2, 2>(a, s) : launch_width<2, 1>(a, s);
    }
    if (w == 4) return launch_width<4, 4>(a, s);
    return w == 2 ? launch_width<4, 2>(a, s) : launch_width<4, 1>(a, s);
}

cudaError_t launch_kv_slots(const int32_t* page_table, int64_t ld_table, int64_t max_pages, const int32_t* cache_lens,
                            const int32_t* seq_starts, int64_t B, int64_t T, int64_t page_size, int64_t num_pages,
                            int64_t* slots, int64_t* positions, int32_t* err, cudaStream_t s) {
    if (T == 0) return cudaSuccess;
    const int64_t grid = (T + kThreads - 1) / kThreads;
    return launch_dependent(kv_slots_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, page_table, ld_table,
                            max_pages, cache_lens, seq_starts, B, T, page_size, num_pages, slots, positions, err);
}

}  // namespace foak
