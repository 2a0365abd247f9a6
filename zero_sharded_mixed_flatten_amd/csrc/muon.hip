// muon.hip -- gfx950 kernels of the elementwise parts of the Muon step:
// zero_muon_momentum and zero_muon_update.  Streaming passes over a range of
// the shard, four elements a lane, every load issued before the arithmetic;
// HBM bounds both.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "step_common.h"
#include "zero_muon.h"

namespace {

using namespace zero_host;
using namespace zero_step;

struct Control {
    const uint32_t *skip;
    const double *sumsq;
    double max_norm;
    const zero_loss_scale *loss_scale;
    double grad_scale;
    const zero_step_consts *dc;
};

// The step's constants and clip coefficient, the same in every thread; false
// where the step writes nothing.
__device__ __forceinline__ bool resolve(Control k, Consts &c, float &clip) {
    if (k.skip != nullptr && *k.skip != 0u) return false;
    if (k.dc != nullptr) {
        c = consts_of(*k.dc);
        if (step_held(c)) return false;
        k.grad_scale = k.dc->grad_scale;
    }
    if (k.loss_scale != nullptr)
        c.s = static_cast<float>(k.grad_scale / static_cast<double>(k.loss_scale->scale));
    clip = 1.0f;
    if (k.sumsq != nullptr && k.max_norm > 0.0) {
        const double norm = sqrt(*k.sumsq) * static_cast<double>(c.s);
        const double cc = k.max_norm / (norm + 1e-6);
        if (cc < 1.0) clip = static_cast<float>(cc);
    }
    return true;
}

// four elements at any alignment (global memory takes it); fp32, or 16-bit as
// pairs
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

template <int DT>
__device__ __forceinline__ typename GradT<DT>::quad quad_at(const typename GradT<DT>::elem *p) {
    if constexpr (DT == ZERO_FP32)
        return __builtin_nontemporal_load(reinterpret_cast<const f32x4_any *>(p));
    else
        return __builtin_nontemporal_load(reinterpret_cast<const u32x2_any *>(p));
}

// What a lane has read of a row.  A wave that holds the range's first or last
// element may have lanes with fewer than four: all its lanes then read element
// by element, the last one again in place of those that are not there, so that
// these loads too go out together.  With a branch and a wait for each row the
// one such wave set the time: 64 bf16 rows of 100003 31 us for 10.
template <int DT, bool ENDS>
struct Quad {
    typename GradT<DT>::quad q;
    __device__ __forceinline__ void read(const typename GradT<DT>::elem *p, int) {
        q = quad_at<DT>(p);
    }
    __device__ __forceinline__ void widen(float (&v)[kQuad]) const { widen_quad<DT>(v, q); }
};
template <int DT>
struct Quad<DT, true> {
    typename GradT<DT>::elem e[kQuad];
    __device__ __forceinline__ void read(const typename GradT<DT>::elem *p, int n) {
#pragma unroll
        for (int i = 0; i < kQuad; ++i) e[i] = p[min(i, n - 1)];
    }
    __device__ __forceinline__ void widen(float (&v)[kQuad]) const {
#pragma unroll
        for (int i = 0; i < kQuad; ++i) v[i] = widen1<DT>(e[i]);
    }
};

template <int DT>
__device__ __forceinline__ void quad_to(typename GradT<DT>::elem *p, const float (&v)[kQuad],
                                        int n) {
    if constexpr (DT == ZERO_FP32) {
        if (n >= kQuad) {
            store16(p, f32x4{v[0], v[1], v[2], v[3]});
        } else {
#pragma unroll
            for (int e = 0; e < kQuad - 1; ++e)
                if (e < n) p[e] = v[e];
        }
    } else {
        float r[kQuad];
#pragma unroll
        for (int e = 0; e < kQuad; ++e) r[e] = as_rounded_f32(v[e]);
        if (n >= kQuad) {
            store8(p, u32x2{narrow2<DT>(r[0], r[1]), narrow2<DT>(r[2], r[3])});
        } else {
#pragma unroll
            for (int e = 0; e < kQuad - 1; ++e)
                if (e < n) p[e] = narrow1<DT>(r[e]);
        }
    }
}

// A lane's elements.  A wave's 256 start where the fp32 buffer's address is a
// multiple of 1024 (skew elements before the range's first one), so that a
// range at an odd place of the flat buffers, whose 16-bit ones then match, is
// read and written in whole cache lines but for its ends.  45 M elements from
// element 5 on: eight bf16 rows 176 us for 236, the update 81 for 107; quads
// aligned each by itself gain nothing.
//
// run: waves that follow one another in memory and take one XCD, 1 or kRun.
// Workgroups go round the 8 XCDs; where the rows' lines begin at other places
// than the waves do, two neighbours read the line between them, and runs on
// one XCD find it in its L2.  64 fp16 rows of 479485 17.2 -> 15.6 us, eight
// bf16 ones of 40 M + 1 180 -> 159; eight of 45 M, whole lines, 177 -> 181.
constexpr uint32_t kXcds = 8, kRun = 16;

__device__ __forceinline__ int quad_of(int64_t len, int skew, uint32_t run, int64_t &at) {
    uint32_t block = blockIdx.x;
    const uint32_t span = kXcds * run, in = block % span;
    if (block - in + span <= gridDim.x) block += in % kXcds * run + in / kXcds - in;
    const int64_t first = (static_cast<int64_t>(block) * kWave + threadIdx.x) * kQuad - skew;
    at = first < 0 ? 0 : first;
    return static_cast<int>(min(len, first + kQuad) - at);
}

// rows fetched together where their number is not a compile-time one
constexpr int kBatch = 8;

template <int GDT, int UDT>
struct Momentum {
    const typename GradT<GDT>::elem *__restrict__ g;
    int64_t ld;
    int n_rows;
    int64_t len;
    float *__restrict__ mom;
    typename GradT<UDT>::elem *__restrict__ u;
    int nesterov, skew;
    uint32_t run;
};

template <int GDT, int UDT, int NDP, bool ENDS>
__device__ __forceinline__ void momentum_quad(const Momentum<GDT, UDT> &w, int64_t at, int n,
                                              const Consts &c, float clip) {
    const typename GradT<GDT>::elem *p = w.g + at;
    constexpr int B = NDP > 0 ? NDP : kBatch;
    Quad<GDT, ENDS> x[B];
    Quad<ZERO_FP32, ENDS> old;
#pragma unroll
    for (int k = 0; k < B; ++k)
        if (NDP > 0 || k < w.n_rows) x[k].read(p + k * w.ld, n);
    old.read(w.mom + at, n);
    loads_issued();
    float a[kQuad], t[kQuad];
    x[0].widen(a);
#pragma unroll
    for (int k = 1; k < B; ++k)
        if (NDP > 0 || k < w.n_rows) {
            x[k].widen(t);
#pragma unroll
            for (int e = 0; e < kQuad; ++e) a[e] = a[e] + t[e];
        }
    if constexpr (NDP == 0) {
        for (int k0 = B; k0 < w.n_rows; k0 += B) {
#pragma unroll
            for (int k = 0; k < B; ++k)
                if (k0 + k < w.n_rows) x[k].read(p + (k0 + k) * w.ld, n);
            loads_issued();
#pragma unroll
            for (int k = 0; k < B; ++k)
                if (k0 + k < w.n_rows) {
                    x[k].widen(t);
#pragma unroll
                    for (int e = 0; e < kQuad; ++e) a[e] = a[e] + t[e];
                }
        }
    }
    float m[kQuad], v[kQuad];
    old.widen(t);
#pragma unroll
    for (int e = 0; e < kQuad; ++e) {
        float ge = a[e] * c.s;
        if (clip < 1.0f) ge = ge * clip;
        m[e] = c.b1 * t[e] + ge;
        v[e] = w.nesterov ? ge + c.b1 * m[e] : m[e];
    }
    quad_to<ZERO_FP32>(w.mom + at, m, n);
    quad_to<UDT>(w.u + at, v, n);
}

template <int GDT, int UDT, int NDP>
__global__ void __launch_bounds__(kWave)
momentum_kernel(Momentum<GDT, UDT> w, Consts c, Control ctl) {
    float clip;
    if (!resolve(ctl, c, clip)) return;
    int64_t at;
    const int n = quad_of(w.len, w.skew, w.run, at);
    if (n <= 0) return;
    if (__all(n == kQuad))
        momentum_quad<GDT, UDT, NDP, false>(w, at, n, c, clip);
    else
        momentum_quad<GDT, UDT, NDP, true>(w, at, n, c, clip);
}

template <int ODT, int WDT, bool ENDS>
__device__ __forceinline__ void update_quad(const uint16_t *o, float *W, uint16_t *slot, int n,
                                            float k, const Consts &c) {
    Quad<ODT, ENDS> ov;
    Quad<ZERO_FP32, ENDS> old;
    ov.read(o, n);
    old.read(W, n);
    loads_issued();
    float t[kQuad], w[kQuad];
    ov.widen(t);
    old.widen(w);
#pragma unroll
    for (int e = 0; e < kQuad; ++e) w[e] = w[e] * c.d - c.lr * (k * t[e]);
    quad_to<ZERO_FP32>(W, w, n);
    quad_to<WDT>(slot, w, n);
}

template <int ODT, int WDT>
__global__ void __launch_bounds__(kWave)
update_kernel(const uint16_t *__restrict__ o, int64_t len, float *__restrict__ W,
              uint16_t *__restrict__ slot, float k, int skew, Consts c, Control ctl) {
    float clip;
    if (!resolve(ctl, c, clip)) return;
    int64_t at;
    const int n = quad_of(len, skew, 1, at);
    if (n <= 0) return;
    if (__all(n == kQuad))
        update_quad<ODT, WDT, false>(o + at, W + at, slot + at, n, k, c);
    else
        update_quad<ODT, WDT, true>(o + at, W + at, slot + at, n, k, c);
}

// ---------------------------------------------------------------------------
// host

inline int64_t bytes_of(zero_dtype t) { return t == ZERO_FP32 ? 4 : 2; }
inline bool aligned_to(const void *p, int64_t b) {
    return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(b) == 0;
}

template <class F>
void for_launches(int64_t len, F f) {
    for (int64_t at = 0; at < len; at += kLaunchElems) f(at, std::min(kLaunchElems, len - at));
}
// Waves on a CU: the more a lane has in flight, the fewer keep HBM busiest.
// Times over 45 M elements (us): 8 bf16 rows 8 waves 192, 12 176, 16 179,
// uncapped 187; 8 fp32 rows (half of it) 8 147, 12 150, uncapped 155; 64 bf16
// rows (a quarter) 8 282, 12 256, uncapped 268; one fp32 row 12 113, 16 107,
// uncapped 112; 2 bf16 rows 16 99, 20 95, uncapped 97; update 16 83, 20 81,
// uncapped 82.  Short ranges are over before it matters.
inline size_t residency(int waves, int64_t len) {
    return len < (int64_t(1) << 20) ? 0 : residency_lds_bytes(waves, kWave);
}
inline int skew_of(const float *p) {  // pieces of a long range keep it
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) / 4 % (kWave * kQuad));
}
inline uint32_t groups_of(int64_t len, int skew) {
    return static_cast<uint32_t>((len + skew + kWave * kQuad - 1) / (kWave * kQuad));
}

template <int GDT, int UDT, int NDP>
void run_momentum(const void *grads, int64_t ld, int32_t n_rows, int64_t len, float *mom, void *u,
                  int32_t nesterov, const Consts &c, const Control &k, hipStream_t st) {
    const auto *g = static_cast<const typename GradT<GDT>::elem *>(grads);
    auto *out = static_cast<typename GradT<UDT>::elem *>(u);
    const int waves = GDT == ZERO_FP32 ? (n_rows >= 8 ? 8 : 16)
                                       : (n_rows >= 8 ? 12 : n_rows == 1 ? 16 : 20);
    const size_t lds = residency(waves, len);
    constexpr int64_t kSize = sizeof(*g), kLine = 128;
    const int64_t off = reinterpret_cast<intptr_t>(g) - reinterpret_cast<intptr_t>(mom) / 4 * kSize;
    const uint32_t run = off % kLine != 0 || (n_rows > 1 && ld % (kLine / kSize) != 0) ? kRun : 1;
    for_launches(len, [&](int64_t at, int64_t n) {
        momentum_kernel<GDT, UDT, NDP><<<groups_of(n, skew_of(mom)), kWave, lds, st>>>(
            Momentum<GDT, UDT>{g + at, ld, n_rows, n, mom + at, out + at, nesterov != 0,
                               skew_of(mom), run}, c, k);
    });
}

template <int GDT, int UDT>
void momentum_rows(const void *grads, int64_t ld, int32_t n_rows, int64_t len, float *mom, void *u,
                   int32_t nesterov, const Consts &c, const Control &k, hipStream_t st) {
    switch (n_rows) {
        case 1: run_momentum<GDT, UDT, 1>(grads, ld, n_rows, len, mom, u, nesterov, c, k, st); break;
        case 8: run_momentum<GDT, UDT, 8>(grads, ld, n_rows, len, mom, u, nesterov, c, k, st); break;
        default: run_momentum<GDT, UDT, 0>(grads, ld, n_rows, len, mom, u, nesterov, c, k, st);
    }
}

template <int GDT>
void momentum_types(const void *grads, int64_t ld, int32_t n_rows, int64_t len, float *mom,
                    void *u, zero_dtype udt, int32_t nesterov, const Consts &c, const Control &k,
                    hipStream_t st) {
    if (udt == ZERO_BF16)
        momentum_rows<GDT, ZERO_BF16>(grads, ld, n_rows, len, mom, u, nesterov, c, k, st);
    else if (udt == ZERO_FP16)
        momentum_rows<GDT, ZERO_FP16>(grads, ld, n_rows, len, mom, u, nesterov, c, k, st);
    else
        momentum_rows<GDT, ZERO_FP32>(grads, ld, n_rows, len, mom, u, nesterov, c, k, st);
}

zero_status momentum_impl(const void *grads, zero_dtype gdt, int32_t n_rows, int64_t ld,
                          int64_t len, float *mom, void *u, zero_dtype udt, int32_t nesterov,
                          const zero_adamw_hparams *hp, const zero_step_consts *dc,
                          const zero_step_control *ctl, void *stream) {
    for (zero_dtype t : {gdt, udt})
        if (!dtype_ok(t) && t != ZERO_FP32) return ZERO_EINVAL;
    if (!(dc ? aligned8(dc) : hparams_ok(hp))) return ZERO_EINVAL;
    if (!rows_ok(n_rows, ld, len) || len > kMaxLen) return ZERO_EINVAL;
    if (ctl && !std::isfinite(ctl->max_norm)) return ZERO_EINVAL;
    if (len == 0) return ZERO_OK;
    const int64_t ge = bytes_of(gdt), ue = bytes_of(udt);
    if (!grads || !mom || !u || !aligned_to(grads, ge) || !aligned_to(mom, 4) ||
        !aligned_to(u, ue))
        return ZERO_EINVAL;
    const Span sm = span_of(mom, len, 4), su = span_of(u, len, ue);
    if (overlap(sm, su)) return ZERO_EALIAS;
    for (int32_t k = 0; k < n_rows; ++k) {
        const Span r = span_of(static_cast<const char *>(grads) + k * ld * ge, len, ge);
        if (overlap(sm, r) || overlap(su, r)) return ZERO_EALIAS;
    }
    Control k{};
    if (ctl) k = Control{ctl->skip, ctl->sumsq, ctl->max_norm, ctl->loss_scale, 0.0, nullptr};
    k.grad_scale = dc ? 0.0 : hp->grad_scale;
    k.dc = dc;
    for (const Span &r : {span_of(dc, dc ? 1 : 0, sizeof(zero_step_consts)),
                          span_of(k.skip, k.skip ? 1 : 0, 4), span_of(k.sumsq, k.sumsq ? 1 : 0, 8),
                          span_of(k.loss_scale, k.loss_scale ? 1 : 0, sizeof(zero_loss_scale))})
        if (overlap(sm, r) || overlap(su, r)) return ZERO_EALIAS;
    const Consts c = dc ? Consts{} : make_consts(*hp);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (gdt == ZERO_BF16)
        momentum_types<ZERO_BF16>(grads, ld, n_rows, len, mom, u, udt, nesterov, c, k, st);
    else if (gdt == ZERO_FP16)
        momentum_types<ZERO_FP16>(grads, ld, n_rows, len, mom, u, udt, nesterov, c, k, st);
    else
        momentum_types<ZERO_FP32>(grads, ld, n_rows, len, mom, u, udt, nesterov, c, k, st);
    return launch_status();
}

template <int ODT, int WDT>
void run_update(const uint16_t *o, int64_t len, float *w, uint16_t *slot, float scale,
                const Consts &c, const Control &k, hipStream_t st) {
    const size_t lds = residency(20, len);
    for_launches(len, [&](int64_t at, int64_t n) {
        update_kernel<ODT, WDT>
            <<<groups_of(n, skew_of(w)), kWave, lds, st>>>(o + at, n, w + at, slot + at, scale,
                                                           skew_of(w), c, k);
    });
}

zero_status update_impl(const void *o, zero_dtype odt, float *master, void *weight_full,
                        zero_dtype wdt, const zero_layout *layout, int32_t rank,
                        int64_t shard_off, int64_t len, const zero_adamw_hparams *hp,
                        const zero_step_consts *dc, double update_scale, const uint32_t *skip,
                        void *stream) {
    if (!dtype_ok(odt) || !dtype_ok(wdt) || !layout_ok(layout)) return ZERO_EINVAL;
    const float scale = static_cast<float>(update_scale);
    if (!(dc ? aligned8(dc) : hparams_ok(hp)) || !std::isfinite(scale)) return ZERO_EINVAL;
    if (rank < 0 || rank >= layout->n_dp || shard_off < 0 || len < 0 || len > kMaxLen)
        return ZERO_EINVAL;
    if (shard_off > layout->shard || len > layout->shard - shard_off) return ZERO_ERANGE;
    if (len == 0) return ZERO_OK;
    if (!o || !master || !weight_full || !aligned_to(o, 2) || !aligned_to(master, 4) ||
        !aligned_to(weight_full, 2))
        return ZERO_EINVAL;
    uint16_t *slot = static_cast<uint16_t *>(weight_full) +
                     static_cast<int64_t>(rank) * layout->shard + shard_off;
    const Span sw = span_of(master, len, 4), ss = span_of(slot, len, 2);
    if (overlap(sw, ss)) return ZERO_EALIAS;
    for (const Span &r : {span_of(o, len, 2), span_of(dc, dc ? 1 : 0, sizeof(zero_step_consts)),
                          span_of(skip, skip ? 1 : 0, 4)})
        if (overlap(sw, r) || overlap(ss, r)) return ZERO_EALIAS;
    const Consts c = dc ? Consts{} : make_consts(*hp);
    const Control k{skip, nullptr, 0.0, nullptr, 0.0, dc};
    const auto *in = static_cast<const uint16_t *>(o);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (odt == ZERO_BF16)
        wdt == ZERO_BF16
            ? run_update<ZERO_BF16, ZERO_BF16>(in, len, master, slot, scale, c, k, st)
            : run_update<ZERO_BF16, ZERO_FP16>(in, len, master, slot, scale, c, k, st);
    else
        wdt == ZERO_BF16
            ? run_update<ZERO_FP16, ZERO_BF16>(in, len, master, slot, scale, c, k, st)
            : run_update<ZERO_FP16, ZERO_FP16>(in, len, master, slot, scale, c, k, st);
    return launch_status();
}

}  // namespace

extern "C" {

zero_status zero_muon_momentum(const void *grads, zero_dtype gdt, int32_t n_rows, int64_t ld,
                               int64_t len, float *mom, void *u, zero_dtype udt, int32_t nesterov,
                               const zero_adamw_hparams *hp, const zero_step_control *ctl,
                               void *stream) {
    return momentum_impl(grads, gdt, n_rows, ld, len, mom, u, udt, nesterov, hp, nullptr, ctl,
                         stream);
}

zero_status zero_muon_momentum_dc(const void *grads, zero_dtype gdt, int32_t n_rows, int64_t ld,
                                  int64_t len, float *mom, void *u, zero_dtype udt,
                                  int32_t nesterov, const zero_step_consts *consts,
                                  const zero_step_control *ctl, void *stream) {
    if (!consts) return ZERO_EINVAL;
    return momentum_impl(grads, gdt, n_rows, ld, len, mom, u, udt, nesterov, nullptr, consts, ctl,
                         stream);
}

zero_status zero_muon_update(const void *o, zero_dtype odt, float *master, void *weight_full,
                             zero_dtype wdt, const zero_layout *layout, int32_t rank,
                             int64_t shard_off, int64_t len, const zero_adamw_hparams *hp,
                             double update_scale, const uint32_t *skip, void *stream) {
    return update_impl(o, odt, master, weight_full, wdt, layout, rank, shard_off, len, hp, nullptr,
                       update_scale, skip, stream);
}

zero_status zero_muon_update_dc(const void *o, zero_dtype odt, float *master, void *weight_full,
                                zero_dtype wdt, const zero_layout *layout, int32_t rank,
                                int64_t shard_off, int64_t len, const zero_step_consts *consts,
                                double update_scale, const uint32_t *skip, void *stream) {
    if (!consts) return ZERO_EINVAL;
    return update_impl(o, odt, master, weight_full, wdt, layout, rank, shard_off, len, nullptr,
                       consts, update_scale, skip, stream);
}

}  // extern "C"
