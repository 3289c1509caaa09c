// C ABI entry points of the hybrid-layer operators (rotary positions, the gated recurrence,
// window attention, the gated delta rule, group norm): argument validation and dispatch.
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "la_common.cuh"
#include "la_internal.h"

namespace la {
namespace {

bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
size_t elem(la_dtype t) { return t == LA_F32 ? 4 : 2; }

// One buffer of a call: null pointers count as absent.
struct Span {
    const void *p;
    size_t bytes;
};
bool overlap(const Span &a, const Span &b)
{
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + b.bytes && y < x + a.bytes;
}
// Outputs overlap no input and no other output.
template <size_t NO, size_t NI>
bool disjoint(const Span (&out)[NO], const Span (&in)[NI])
{
    for (size_t i = 0; i < NO; ++i) {
        for (size_t j = 0; j < NI; ++j)
            if (overlap(out[i], in[j])) return false;
        for (size_t j = i + 1; j < NO; ++j)
            if (overlap(out[i], out[j])) return false;
    }
    return true;
}

// What a call keeps from one of its kernels to the next.  The lock, held over its launches, keeps
// two host threads that share a stream from mixing them on its one workspace (one of each
// operator, `which`); a captured call takes memory of its own, so that two graphs may be replayed
// at once.
std::mutex g_launches;
la_status call_scratch(cudaStream_t s, size_t bytes, int which, Scratch *own, void **base)
{
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    la_status st = cuda_status(cudaStreamIsCapturing(s, &cs));
    if (st != LA_OK) return st;
    if (cs == cudaStreamCaptureStatusNone && data_workspace(s, bytes, base, which) == LA_OK) return LA_OK;
    if ((st = own->alloc(bytes, s)) == LA_OK) *base = own->ptr;
    return st;
}

la_status run_recurrence(RecurrenceProblem &p)
{
    const size_t bytes = recurrence_scratch(p);
    if (bytes == 0) return recurrence(p);
    std::lock_guard<std::mutex> lock(g_launches);
    Scratch own;
    void *base = nullptr;
    const la_status st = call_scratch(p.stream, bytes, 2, &own, &base);
    if (st != LA_OK) return st;
    p.fold = static_cast<float *>(base);
    return recurrence(p);
}

bool known(la_dtype t) { return t == LA_F32 || t == LA_BF16; }

// ---------------------------------------------------------------- rotary
la_status check_spec(const la_rotary_spec *s, int d)
{
    if (!s || s->rot < 0 || s->rot > d || s->rot % 2 != 0) return LA_ERR_INVALID_ARG;
    if (s->layout != LA_ROTARY_HALF && s->layout != LA_ROTARY_INTERLEAVED) return LA_ERR_INVALID_ARG;
    if (!isfinite(s->amplitude) || !isfinite(s->base) || !(s->base > 0)) return LA_ERR_INVALID_ARG;
    if (s->scaling < LA_ROTARY_NONE || s->scaling > LA_ROTARY_RAMP) return LA_ERR_INVALID_ARG;
    if (s->scaling != LA_ROTARY_NONE && (!isfinite(s->factor) || !(s->factor > 0))) return LA_ERR_INVALID_ARG;
    if (s->scaling == LA_ROTARY_RAMP &&
        (s->original <= 0 || !isfinite(s->ramp_lo) || !isfinite(s->ramp_hi) || !(s->ramp_lo < s->ramp_hi)))
        return LA_ERR_INVALID_ARG;
    return LA_OK;
}

// Pair frequencies in turns per position, times 2^64 (modulo whole turns: a frequency of a
// turn or more per position acts as its fraction).  False where one is not finite.
bool fill_turns(const la_rotary_spec &s, uint64_t *turns)
{
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    double base = s.base;
    if (s.scaling == LA_ROTARY_NTK && s.rot > 2) base *= pow(s.factor, (double)s.rot / (s.rot - 2));
    // base^(-2 i / rot) as the product of the powers at i's binary digits: at most 7 of them, each within
    // 2^-52, 6 products and the exponents' roundings, ln(base) 2^-53 together: below 2^-48 for bases up to
    // 10^5, 2^-47 up to 10^19.
    double fs[kRotaryMaxPairs] = {1.0};
    for (int n = 1; n < s.rot / 2; n *= 2) {
        const double power = pow(base, -2.0 * n / s.rot);
        for (int i = n; i < 2 * n && i < s.rot / 2; ++i) fs[i] = fs[i - n] * power;
    }
    for (int i = 0; i < s.rot / 2; ++i) {
        const double f = fs[i];
        double g = f;
        if (s.scaling == LA_ROTARY_LINEAR) g = f / s.factor;
        if (s.scaling == LA_ROTARY_RAMP) {
            const double keep = fmin(1.0, fmax(0.0, (s.original * f / kTwoPi - s.ramp_lo) / (s.ramp_hi - s.ramp_lo)));
            g = f * (keep + (1.0 - keep) / s.factor);
        }
        if (!isfinite(g)) return false;
        const double t = g / kTwoPi, part = t - floor(t);
        turns[i] = (uint64_t)(part * 0x1p64);  // part < 1: at most 2^64 - 2^11
    }
    return true;
}

la_status rotary_checked(const void *q, const void *k, void *oq, void *ok, const int *positions, long long offset,
                         const la_rotary_spec *spec, int B, int Hq, int Hk, int N, int d, la_dtype dtype,
                         la_stream_t stream, bool backward)
{
    if (B < 0 || Hq < 0 || Hk < 0 || N < 0 || d < 0 || !known(dtype)) return LA_ERR_INVALID_ARG;
    la_status st = check_spec(spec, d);
    if (st != LA_OK) return st;
    if (B == 0 || Hq + (long long)Hk == 0 || N == 0 || d == 0) return LA_OK;
    if ((Hq > 0 && (!q || !oq)) || (Hk > 0 && (!k || !ok))) return LA_ERR_INVALID_ARG;
    if ((Hq > 0 && (!aligned(q, 16) || !aligned(oq, 16))) || (Hk > 0 && (!aligned(k, 16) || !aligned(ok, 16))) ||
        !aligned(positions, 4))
        return LA_ERR_MISALIGNED;
    if (d % 8 != 0 || d > 2 * kRotaryMaxPairs || (long long)Hq + Hk > 0x7fffffff) return LA_ERR_UNSUPPORTED;
    const size_t row = (size_t)N * d * elem(dtype);
    const Span sq{Hq ? q : nullptr, B * (size_t)Hq * row}, sk{Hk ? k : nullptr, B * (size_t)Hk * row};
    const Span soq{Hq ? oq : nullptr, sq.bytes}, sok{Hk ? ok : nullptr, sk.bytes};
    const Span spos{positions, (size_t)B * N * 4};
    if (overlap(soq, sok) || overlap(soq, sk) || overlap(sok, sq) || overlap(soq, spos) || overlap(sok, spos) ||
        (soq.p != sq.p && overlap(soq, sq)) || (sok.p != sk.p && overlap(sok, sk)))
        return LA_ERR_INVALID_ARG;
    RotaryProblem p;
    p.q = q; p.k = k; p.oq = oq; p.ok = ok;
    p.positions = positions;
    p.offset = offset;
    p.spec = *spec;
    p.B = B; p.Hq = Hq; p.Hk = Hk; p.N = N; p.d = d;
    p.backward = backward;
    p.dtype = dtype;
    p.stream = (cudaStream_t)stream;
    if (!fill_turns(*spec, p.turns)) return LA_ERR_INVALID_ARG;
    return rotary(p);
}

// ---------------------------------------------------------------- window attention
constexpr int kMaxTokens = 1 << 30;  // of a sequence or a cache: sums of two positions fit an int

la_status check_window(int B, int Hq, int Hk, int d, int window, int sinks, float scale, la_dtype dtype)
{
    if (B < 0 || Hq < 0 || Hk < 0 || d < 0 || window < 1 || sinks < 0 || !known(dtype)) return LA_ERR_INVALID_ARG;
    if (!(scale >= 0x1p-100f) || !(scale <= 0x1p100f)) return LA_ERR_INVALID_ARG;
    if (Hk > 0 ? Hq % Hk != 0 : Hq != 0) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

// ---------------------------------------------------------------- gated delta rule
la_status check_delta(int B, int Hk, int H, int N, int dk, int dv, float scale, la_dtype dtype)
{
    if (B < 0 || Hk < 0 || H < 0 || N < 0 || dk < 0 || dv < 0 || !known(dtype) || !isfinite(scale)) return LA_ERR_INVALID_ARG;
    if (Hk > 0 ? H % Hk != 0 : H != 0) return LA_ERR_INVALID_ARG;
    return LA_OK;
}
// What the kernels' grids and 32-bit row counts hold.
bool delta_supported(int B, int H, int N, int dk, int dv)
{
    return supported_dim(dk) && supported_dim(dv) && N <= kMaxTokens && (long long)B * H <= 0x7fffffff / 4 &&
           (long long)B * H * ((N + 31LL) / 32) <= 0x7fffffff;
}
// A result that sums over nothing (where it is wanted).
la_status zeros(void *p, size_t bytes, la_stream_t s)
{
    if (!p || bytes == 0) return LA_OK;
    count_launches();
    return cuda_status(cudaMemsetAsync(p, 0, bytes, (cudaStream_t)s));
}
struct DeltaSizes {
    size_t keys, values, gates, states;
    DeltaSizes(int B, int Hk, int H, int N, int dk, int dv, la_dtype t)
        : keys((size_t)B * Hk * N * dk * elem(t)), values((size_t)B * H * N * dv * elem(t)), gates((size_t)B * H * N * 4),
          states((size_t)B * H * dk * dv * 4)
    {
    }
};

// ---------------------------------------------------------------- group norm
la_status check_norm(const la_group_norm_spec *s, int B, int L, int C, la_dtype dtype)
{
    if (!s || B < 0 || L < 0 || C < 0 || !known(dtype) || s->groups < 1 || C % s->groups != 0) return LA_ERR_INVALID_ARG;
    if ((s->per_token & ~1) || (s->heads_first & ~1) || (s->center & ~1) || (s->heads_first && !s->per_token))
        return LA_ERR_INVALID_ARG;
    if (s->act != LA_ACT_NONE && s->act != LA_ACT_SILU) return LA_ERR_INVALID_ARG;
    return isfinite(s->eps) && s->eps >= 0.f ? LA_OK : LA_ERR_INVALID_ARG;
}
bool norm_supported(const la_group_norm_spec *s, int B, int L, int C)
{
    if (s->heads_first && C / s->groups > kNormTokenChannels) return false;
    const long long tokens = (long long)B * L, entries = s->per_token ? tokens : B;
    // groups in 32 bits; so are the blocks over positions (a round of them, and an entry's runs of columns) of what fits in memory
    return L <= kMaxTokens && tokens <= 0x3fffffff && C <= 0x3fffff && entries * s->groups <= 0x7fffffff;
}

la_status run_norm(NormProblem &p)
{
    const size_t bytes = norm_scratch(p);
    if (bytes == 0) return group_norm(p);
    std::lock_guard<std::mutex> lock(g_launches);
    Scratch own;
    void *base = nullptr;
    const la_status st = call_scratch(p.stream, bytes, 4, &own, &base);
    if (st != LA_OK) return st;
    p.scratch = static_cast<float *>(base);
    return group_norm(p);
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

la_status la_rotary_forward(const void *q, const void *k, void *oq, void *ok, const int *positions, long long offset,
                            const la_rotary_spec *spec, int B, int Hq, int Hk, int N, int d, la_dtype dtype,
                            la_stream_t stream)
{
    return rotary_checked(q, k, oq, ok, positions, offset, spec, B, Hq, Hk, N, d, dtype, stream, false);
}

la_status la_rotary_backward(const void *doq, const void *dok, void *dq, void *dk, const int *positions,
                             long long offset, const la_rotary_spec *spec, int B, int Hq, int Hk, int N, int d,
                             la_dtype dtype, la_stream_t stream)
{
    return rotary_checked(doq, dok, dq, dk, positions, offset, spec, B, Hq, Hk, N, d, dtype, stream, true);
}

la_status la_recurrence_forward(const void *x, const float *alpha, const float *h0, void *h, float *hN, int B, int N,
                                int D, la_dtype dtype, la_stream_t stream)
{
    if (B < 0 || N < 0 || D < 0 || !known(dtype)) return LA_ERR_INVALID_ARG;
    if (B == 0 || D == 0 || (N == 0 && !hN)) return LA_OK;
    if (N > 0 && (!x || !alpha || !h)) return LA_ERR_INVALID_ARG;
    if ((N > 0 && (!aligned(x, 16) || !aligned(alpha, 16) || !aligned(h, 16))) || !aligned(h0, 16) || !aligned(hN, 16))
        return LA_ERR_MISALIGNED;
    const size_t n = (size_t)B * N * D, s = (size_t)B * D * 4, e = elem(dtype);
    const Span out[] = {{h, n * e}, {hN, s}}, in[] = {{x, n * e}, {alpha, n * 4}, {h0, s}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    RecurrenceProblem p{};
    p.x = x; p.alpha = alpha; p.h0 = h0; p.h = h; p.hN = hN;
    p.B = B; p.N = N; p.D = D;
    p.dtype = dtype;
    p.stream = (cudaStream_t)stream;
    return run_recurrence(p);
}

la_status la_recurrence_backward(const float *alpha, const void *h, const void *dh, const float *h0, const float *dhN,
                                 void *dx, float *dalpha, float *dh0, int B, int N, int D, la_dtype dtype,
                                 la_stream_t stream)
{
    if (B < 0 || N < 0 || D < 0 || !known(dtype)) return LA_ERR_INVALID_ARG;
    if (B == 0 || D == 0 || (N == 0 && !dh0)) return LA_OK;
    if (N > 0 && (!alpha || !h || !dh || !dx || !dalpha)) return LA_ERR_INVALID_ARG;
    if ((N > 0 && (!aligned(alpha, 16) || !aligned(h, 16) || !aligned(dh, 16) || !aligned(dx, 16) || !aligned(dalpha, 16))) ||
        !aligned(h0, 16) || !aligned(dhN, 16) || !aligned(dh0, 16))
        return LA_ERR_MISALIGNED;
    const size_t n = (size_t)B * N * D, s = (size_t)B * D * 4, e = elem(dtype);
    const Span out[] = {{dx, n * e}, {dalpha, n * 4}, {dh0, s}};
    const Span in[] = {{alpha, n * 4}, {h, n * e}, {dh, n * e}, {h0, s}, {dhN, s}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    RecurrenceProblem p{};
    p.alpha = alpha; p.h_in = h; p.dh = dh; p.h0 = h0; p.dhN = dhN;
    p.dx = dx; p.dalpha = dalpha; p.dh0 = dh0;
    p.B = B; p.N = N; p.D = D;
    p.backward = true;
    p.dtype = dtype;
    p.stream = (cudaStream_t)stream;
    return run_recurrence(p);
}

la_status la_recurrence_step(float *state, const void *x, const float *alpha, void *h, int B, int D, la_dtype dtype,
                             la_stream_t stream)
{
    if (B < 0 || D < 0 || !known(dtype)) return LA_ERR_INVALID_ARG;
    if (B == 0 || D == 0) return LA_OK;
    if (!state || !x || !alpha || !h) return LA_ERR_INVALID_ARG;
    if (!aligned(state, 16) || !aligned(x, 16) || !aligned(alpha, 16) || !aligned(h, 16)) return LA_ERR_MISALIGNED;
    const size_t n = (size_t)B * D, e = elem(dtype);
    const Span out[] = {{h, n * e}, {state, n * 4}}, in[] = {{x, n * e}, {alpha, n * 4}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    return recurrence_step(state, x, alpha, h, B, D, dtype, (cudaStream_t)stream);
}

la_status la_window_forward(const void *q, const void *k, const void *v, void *o, float *lse, const int *lens, int B,
                            int Hq, int Hk, int Nq, int Nk, int d, int window, int sinks, float scale, la_dtype dtype,
                            la_stream_t stream)
{
    la_status st = check_window(B, Hq, Hk, d, window, sinks, scale, dtype);
    if (st != LA_OK) return st;
    if (Nq < 0 || Nk < 0 || Nq > Nk) return LA_ERR_INVALID_ARG;
    if (B == 0 || Hq == 0 || Nq == 0 || d == 0) return LA_OK;
    if (!q || !k || !v || !o || !lse) return LA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 16) || !aligned(lens, 4))
        return LA_ERR_MISALIGNED;
    if (!supported_dim(d) || (long long)B * Hq > 0x7fffffff || (long long)B * Hk > 0x7fffffff || Nk > kMaxTokens)
        return LA_ERR_UNSUPPORTED;
    const size_t rows = (size_t)B * Hq * Nq, keys = (size_t)B * Hk * Nk, e = d * elem(dtype);
    const Span out[] = {{o, rows * e}, {lse, rows * 4}};
    const Span in[] = {{q, rows * e}, {k, keys * e}, {v, keys * e}, {lens, (size_t)B * 4}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    WindowProblem p{};
    p.q = q; p.k = k; p.v = v; p.out = o; p.lse = lse; p.lens = lens;
    p.B = B; p.Hq = Hq; p.Hk = Hk; p.Nq = Nq; p.Nk = Nk; p.d = d;
    p.window = window < Nk ? window : Nk;
    p.sinks = sinks < Nk ? sinks : Nk;
    p.scale = scale;
    p.dtype = dtype;
    p.stream = (cudaStream_t)stream;
    return dtype == LA_BF16 ? window_forward_tc(p) : window_forward_simt(p);
}

la_status la_window_backward(const void *q, const void *k, const void *v, const void *o, const float *lse,
                             const void *dout, void *dq, void *dk, void *dv, const int *lens, int B, int Hq, int Hk,
                             int Nq, int Nk, int d, int window, int sinks, float scale, la_dtype dtype,
                             la_stream_t stream)
{
    la_status st = check_window(B, Hq, Hk, d, window, sinks, scale, dtype);
    if (st != LA_OK) return st;
    if (Nq < 0 || Nk < 0 || Nq > Nk) return LA_ERR_INVALID_ARG;
    if (B == 0 || Hk == 0 || Nk == 0 || d == 0) return LA_OK;
    const bool rows_any = Hq > 0 && Nq > 0;
    if (!dk || !dv || (rows_any && (!q || !k || !v || !o || !lse || !dout || !dq))) return LA_ERR_INVALID_ARG;
    if (!aligned(dk, 16) || !aligned(dv, 16) ||
        (rows_any && (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 16) ||
                      !aligned(dout, 16) || !aligned(dq, 16) || !aligned(lens, 4))))
        return LA_ERR_MISALIGNED;
    if (!supported_dim(d) || (long long)B * Hq > 0x7fffffff || (long long)B * Hk > 0x7fffffff || Nk > kMaxTokens)
        return LA_ERR_UNSUPPORTED;
    const size_t rows = (size_t)B * Hq * Nq, keys = (size_t)B * Hk * Nk, e = d * elem(dtype);
    const Span out[] = {{dq, rows * e}, {dk, keys * e}, {dv, keys * e}};
    const Span in[] = {{q, rows * e}, {k, keys * e}, {v, keys * e}, {o, rows * e}, {lse, rows * 4}, {dout, rows * e},
                       {lens, (size_t)B * 4}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    if (!rows_any) {  // no query sees a key
        count_launches(2);
        if ((st = cuda_status(cudaMemsetAsync(dk, 0, keys * e, s))) != LA_OK) return st;
        return cuda_status(cudaMemsetAsync(dv, 0, keys * e, s));
    }
    WindowProblem p{};
    p.q = q; p.k = k; p.v = v; p.o = o; p.lse = const_cast<float *>(lse); p.dout = dout;
    p.dq = dq; p.dk = dk; p.dv = dv; p.lens = lens;
    p.B = B; p.Hq = Hq; p.Hk = Hk; p.Nq = Nq; p.Nk = Nk; p.d = d;
    p.window = window < Nk ? window : Nk;
    p.sinks = sinks < Nk ? sinks : Nk;
    p.scale = scale;
    p.dtype = dtype;
    p.stream = s;
    // D = dO . o per row and partial sums, from one kernel to the next
    std::lock_guard<std::mutex> lock(g_launches);
    Scratch own;
    void *base = nullptr;
    st = call_scratch(s, dtype == LA_BF16 ? window_backward_tc_scratch(p) : window_backward_simt_scratch(p), 1, &own, &base);
    if (st != LA_OK) return st;
    p.delta = static_cast<float *>(base);
    return dtype == LA_BF16 ? window_backward_tc(p) : window_backward_simt(p);
}

la_status la_window_cache(const void *k, const void *v, void *kc, void *vc, const int *lens, int B, int Hk, int N,
                          int d, int window, int sinks, la_dtype dtype, la_stream_t stream)
{
    la_status st = check_window(B, Hk, Hk, d, window, sinks, 1.f, dtype);
    if (st != LA_OK) return st;
    if (N < 0) return LA_ERR_INVALID_ARG;
    if (B == 0 || Hk == 0 || N == 0 || d == 0) return LA_OK;
    if (!k || !v || !kc || !vc) return LA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(kc, 16) || !aligned(vc, 16) || !aligned(lens, 4))
        return LA_ERR_MISALIGNED;
    if (!supported_dim(d) || (long long)sinks + window > kMaxTokens) return LA_ERR_UNSUPPORTED;
    const size_t e = d * elem(dtype), keys = (size_t)B * Hk * N * e;
    const size_t slots = (size_t)B * Hk * ((size_t)sinks + window) * e;
    const Span out[] = {{kc, slots}, {vc, slots}}, in[] = {{k, keys}, {v, keys}, {lens, (size_t)B * 4}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    return window_cache(k, v, kc, vc, lens, B, Hk, N, d, window, sinks, dtype, (cudaStream_t)stream);
}

la_status la_window_decode_step(void *kc, void *vc, const void *q, const void *k, const void *v, void *o,
                                const int *pos, int B, int Hq, int Hk, int d, int window, int sinks, float scale,
                                la_dtype dtype, la_stream_t stream)
{
    la_status st = check_window(B, Hq, Hk, d, window, sinks, scale, dtype);
    if (st != LA_OK) return st;
    if (B == 0 || Hq == 0 || d == 0) return LA_OK;
    if (!kc || !vc || !q || !k || !v || !o || !pos) return LA_ERR_INVALID_ARG;
    if (!aligned(kc, 16) || !aligned(vc, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(o, 16) || !aligned(pos, 4))
        return LA_ERR_MISALIGNED;
    if (!supported_dim(d) || (long long)sinks + window > kMaxTokens) return LA_ERR_UNSUPPORTED;
    const size_t e = d * elem(dtype), rows = (size_t)B * Hq * e, keys = (size_t)B * Hk * e;
    const size_t slots = keys * ((size_t)sinks + window);
    const Span out[] = {{kc, slots}, {vc, slots}, {o, rows}}, in[] = {{q, rows}, {k, keys}, {v, keys}, {pos, (size_t)B * 4}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    WindowDecodeProblem p{kc, vc, q, k, v, o, pos, B, Hq, Hk, d, window, sinks, scale, dtype, (cudaStream_t)stream};
    return window_decode(p);
}

la_status la_delta_forward(const void *q, const void *k, const void *v, const float *g, const float *beta,
                           const float *S0, void *o, float *SN, int B, int Hk, int H, int N, int dk, int dv, float scale,
                           la_dtype dtype, la_stream_t stream)
{
    la_status st = check_delta(B, Hk, H, N, dk, dv, scale, dtype);
    if (st != LA_OK) return st;
    if (B == 0 || H == 0 || dv == 0 || (N == 0 && !SN)) return LA_OK;
    if (dk == 0) return zeros(o, DeltaSizes(B, Hk, H, N, dk, dv, dtype).values, stream);
    if (N > 0 && (!q || !k || !v || !g || !beta || !o)) return LA_ERR_INVALID_ARG;
    if (!aligned(S0, 16) || !aligned(SN, 16) ||
        (N > 0 && (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 4) || !aligned(beta, 4) || !aligned(o, 16))))
        return LA_ERR_MISALIGNED;
    if (!delta_supported(B, H, N, dk, dv)) return LA_ERR_UNSUPPORTED;
    const DeltaSizes z(B, Hk, H, N, dk, dv, dtype);
    const Span out[] = {{o, z.values}, {SN, z.states}};
    const Span in[] = {{q, z.keys}, {k, z.keys}, {v, z.values}, {g, z.gates}, {beta, z.gates}, {S0, z.states}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    DeltaProblem p{};
    p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta; p.S0 = S0; p.o = o; p.SN = SN;
    p.B = B; p.Hk = Hk; p.H = H; p.N = N; p.dk = dk; p.dv = dv;
    p.scale = scale;
    p.dtype = dtype;
    p.stream = (cudaStream_t)stream;
    if (!delta_tc_eligible(p)) return delta_forward_simt(p);
    std::lock_guard<std::mutex> lock(g_launches);
    Scratch own;
    void *base = nullptr;
    if ((st = call_scratch(p.stream, delta_forward_tc_scratch(p), 3, &own, &base)) != LA_OK) return st;
    p.scratch = static_cast<float *>(base);
    return delta_forward_tc(p);
}

la_status la_delta_backward(const void *q, const void *k, const void *v, const float *g, const float *beta,
                            const float *S0, const void *dout, const float *dSN, void *dq, void *dk, void *dv, float *dg,
                            float *dbeta, float *dS0, int B, int Hk, int H, int N, int d_k, int d_v, float scale,
                            la_dtype dtype, la_stream_t stream)
{
    la_status st = check_delta(B, Hk, H, N, d_k, d_v, scale, dtype);
    if (st != LA_OK) return st;
    if (B == 0 || (N == 0 && !dS0)) return LA_OK;
    if (H == 0 || d_k == 0 || d_v == 0) {  // what is not empty of the gradients is zero
        const DeltaSizes z(B, Hk, H, N, d_k, d_v, dtype);
        void *out[] = {dq, dk, dv, dg, dbeta};
        const size_t bytes[] = {z.keys, z.keys, z.values, z.gates, z.gates};
        for (int i = 0; i < 5 && st == LA_OK; ++i) st = zeros(out[i], bytes[i], stream);
        return st;
    }
    if (N > 0 && (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta)) return LA_ERR_INVALID_ARG;
    if (!aligned(S0, 16) || !aligned(dSN, 16) || !aligned(dS0, 16) ||
        (N > 0 && (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 4) || !aligned(beta, 4) ||
                   !aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(dg, 4) ||
                   !aligned(dbeta, 4))))
        return LA_ERR_MISALIGNED;
    if (!delta_supported(B, H, N, d_k, d_v)) return LA_ERR_UNSUPPORTED;
    const DeltaSizes z(B, Hk, H, N, d_k, d_v, dtype);
    const Span out[] = {{dq, z.keys}, {dk, z.keys}, {dv, z.values}, {dg, z.gates}, {dbeta, z.gates}, {dS0, z.states}};
    const Span in[] = {{q, z.keys}, {k, z.keys}, {v, z.values}, {g, z.gates}, {beta, z.gates}, {S0, z.states},
                       {dout, z.values}, {dSN, z.states}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    DeltaProblem p{};
    p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta; p.S0 = S0; p.dout = dout; p.dSN = dSN;
    p.dq = dq; p.dk_out = dk; p.dv_out = dv; p.dg = dg; p.dbeta = dbeta; p.dS0 = dS0;
    p.B = B; p.Hk = Hk; p.H = H; p.N = N; p.dk = d_k; p.dv = d_v;
    p.scale = scale;
    p.dtype = dtype;
    p.stream = (cudaStream_t)stream;
    std::lock_guard<std::mutex> lock(g_launches);
    Scratch own;
    void *base = nullptr;
    const bool tc = delta_tc_eligible(p);
    const size_t bytes = tc ? delta_backward_tc_scratch(p) : delta_backward_simt_scratch(p);
    if (bytes > 0 && (st = call_scratch(p.stream, bytes, 3, &own, &base)) != LA_OK) return st;
    p.scratch = static_cast<float *>(base);
    return tc ? delta_backward_tc(p) : delta_backward_simt(p);
}

la_status la_delta_step(float *S, const void *q, const void *k, const void *v, const float *g, const float *beta, void *o,
                        int B, int Hk, int H, int dk, int dv, float scale, la_dtype dtype, la_stream_t stream)
{
    const la_status st = check_delta(B, Hk, H, 1, dk, dv, scale, dtype);
    if (st != LA_OK) return st;
    if (B == 0 || H == 0 || dv == 0) return LA_OK;
    if (dk == 0) return zeros(o, DeltaSizes(B, Hk, H, 1, dk, dv, dtype).values, stream);
    if (!S || !q || !k || !v || !g || !beta || !o) return LA_ERR_INVALID_ARG;
    if (!aligned(S, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 4) || !aligned(beta, 4) ||
        !aligned(o, 16))
        return LA_ERR_MISALIGNED;
    if (!delta_supported(B, H, 1, dk, dv)) return LA_ERR_UNSUPPORTED;
    const DeltaSizes z(B, Hk, H, 1, dk, dv, dtype);
    const Span out[] = {{S, z.states}, {o, z.values}};
    const Span in[] = {{q, z.keys}, {k, z.keys}, {v, z.values}, {g, z.gates}, {beta, z.gates}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    DeltaProblem p{};
    p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta; p.o = o;
    p.B = B; p.Hk = Hk; p.H = H; p.N = 1; p.dk = dk; p.dv = dv;
    p.scale = scale;
    p.dtype = dtype;
    p.stream = (cudaStream_t)stream;
    return delta_step(p, S);
}

la_status la_group_norm_forward(const void *x, const void *gate, const float *w, const float *b, void *y, float *mean,
                                float *rstd, const la_group_norm_spec *spec, int B, int L, int C, la_dtype dtype,
                                la_stream_t stream)
{
    const la_status st = check_norm(spec, B, L, C, dtype);
    if (st != LA_OK) return st;
    if (B == 0 || L == 0 || C == 0) return LA_OK;
    if (!x || !y) return LA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(gate, 16) || !aligned(w, 4) || !aligned(b, 4) || !aligned(y, 16) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return LA_ERR_MISALIGNED;
    if (!norm_supported(spec, B, L, C)) return LA_ERR_UNSUPPORTED;
    const size_t n = (size_t)B * L * C * elem(dtype), c = (size_t)C * 4;
    const size_t stats = (size_t)B * (spec->per_token ? L : 1) * spec->groups * 4;
    const Span out[] = {{y, n}, {spec->center ? mean : nullptr, stats}, {rstd, stats}};
    const Span in[] = {{x, n}, {gate, n}, {w, c}, {b, c}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    NormProblem p{};
    p.x = x; p.gate = gate; p.w = w; p.b = b; p.y = y; p.mean_out = spec->center ? mean : nullptr; p.rstd_out = rstd;
    p.B = B; p.L = L; p.C = C;
    p.spec = *spec;
    p.dtype = dtype;
    p.stream = (cudaStream_t)stream;
    return run_norm(p);
}

la_status la_group_norm_backward(const void *x, const void *gate, const float *w, const float *b, const float *mean,
                                 const float *rstd, const void *dy, void *dx, void *dgate, float *dw, float *db,
                                 const la_group_norm_spec *spec, int B, int L, int C, la_dtype dtype,
                                 la_stream_t stream)
{
    la_status st = check_norm(spec, B, L, C, dtype);
    if (st != LA_OK) return st;
    if (C == 0) return LA_OK;
    if (!aligned(dw, 4) || !aligned(db, 4)) return LA_ERR_MISALIGNED;
    const size_t n = (size_t)B * L * C * elem(dtype), c = (size_t)C * 4;
    const cudaStream_t s = (cudaStream_t)stream;
    if (B == 0 || L == 0) {  // sums over nothing
        if (overlap({dw, c}, {db, c})) return LA_ERR_INVALID_ARG;
        for (float *grad : {dw, db})
            if (grad) {
                count_launches();
                if ((st = cuda_status(cudaMemsetAsync(grad, 0, c, s))) != LA_OK) return st;
            }
        return LA_OK;
    }
    if (!x || !dy || !dx || !rstd || (spec->center && !mean) || (gate && !dgate)) return LA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(gate, 16) || !aligned(w, 4) || !aligned(b, 4) || !aligned(mean, 4) || !aligned(rstd, 4) ||
        !aligned(dy, 16) || !aligned(dx, 16) || !aligned(dgate, 16))
        return LA_ERR_MISALIGNED;
    if (!norm_supported(spec, B, L, C)) return LA_ERR_UNSUPPORTED;
    const size_t stats = (size_t)B * (spec->per_token ? L : 1) * spec->groups * 4;
    const Span out[] = {{dx, n}, {gate ? dgate : nullptr, n}, {dw, c}, {db, c}};
    const Span in[] = {{x, n}, {gate, n}, {w, c}, {b, c}, {spec->center ? mean : nullptr, stats}, {rstd, stats}, {dy, n}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    NormProblem p{};
    p.x = x; p.gate = gate; p.dy = dy; p.w = w; p.b = b; p.mean = mean; p.rstd = rstd;
    p.dx = dx; p.dgate = dgate; p.dw = dw; p.db = db;
    p.B = B; p.L = L; p.C = C;
    p.spec = *spec;
    p.backward = true;
    p.dtype = dtype;
    p.stream = s;
    return run_norm(p);
}

}  // extern "C"
