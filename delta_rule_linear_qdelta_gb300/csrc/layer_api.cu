// The C ABI of the operators around the token mixers: the short convolution, the selective
// scan and the group norm.  Argument checks and dispatch; nothing here allocates.
#include <stdarg.h>
#include <stdio.h>

#include "../../include/qdelta.h"
#include "qd_internal.cuh"

namespace {

qd_status fail(qd_status s, const char *fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return qd::report_error(s, msg);
}

constexpr double kMostElements = 68719476736.0, kMostCtas = 2147483647.0;   // 2^36; of one launch

// The most tokens of a sequence, channels or groups: kernels and plans add up to 2^16 tokens (a CTA's runs)
// or some hundred channels or groups to them in 32 bits.
constexpr int kMostSize = 2147483647 - 131071;
bool too_long(int a, int b) { return a > kMostSize || b > kMostSize; }

struct Named {
    const char *name;
    const void *p;
    bool required;
};

qd_status check_pointers(const char *fn, const Named *args, int n) {
    for (int i = 0; i < n; ++i) {
        if (args[i].required && !args[i].p) return fail(QD_ERR_ARG, "%s: required pointer %s is NULL", fn, args[i].name);
        if ((uintptr_t)args[i].p & 15u) return fail(QD_ERR_ARG, "%s: pointer %s is not 16-byte aligned", fn, args[i].name);
    }
    return QD_OK;
}

qd_status check_sizes(const char *fn, int B, int T, int D, qd_dtype dt) {
    if (B < 0 || T < 0 || D < 0) return fail(QD_ERR_ARG, "%s: negative size B=%d T=%d D=%d", fn, B, T, D);
    if (dt != QD_F32 && dt != QD_BF16) return fail(QD_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dt);
    if (too_long(T, D) || (double)B * (T > 1 ? T : 1) * D > kMostElements)
        return fail(QD_ERR_ARG, "%s: sizes overflow", fn);
    return QD_OK;
}

qd_status check_taps(const char *fn, int W) {
    return W >= 2 && W <= 4 ? QD_OK : fail(QD_ERR_UNSUPPORTED, "%s: %d taps (2, 3 or 4 are supported)", fn, W);
}

qd_status check_ssm(const char *fn, int B, int T, int D, int G, int N, qd_dtype dt) {
    qd_status st = check_sizes(fn, B, T, D, dt);
    if (st != QD_OK) return st;
    if (N < 1 || N > 128) return fail(QD_ERR_UNSUPPORTED, "%s: %d states per channel not in 1..128", fn, N);
    if (G < 1 || D % G) return fail(QD_ERR_ARG, "%s: D=%d is no multiple of the %d groups", fn, D, G);
    // the arrays; the scan's CTAs (of at least 8 channels of a group); the sums of dB and dC
    if ((double)B * (T > 1 ? T : 1) * G * (N > 8 ? N : 8) > kMostElements || (double)B * D * N > kMostElements ||
        (double)B * G * ((D / G + 7) / 8) > kMostCtas)
        return fail(QD_ERR_ARG, "%s: sizes overflow", fn);
    return QD_OK;
}

qd_status check_norm(const char *fn, int M, int H, int d, float eps, qd_dtype dt) {
    if (M < 0 || H < 0 || d < 1) return fail(QD_ERR_ARG, "%s: bad size M=%d H=%d d=%d", fn, M, H, d);
    if (dt != QD_F32 && dt != QD_BF16) return fail(QD_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dt);
    if (d > 8192) return fail(QD_ERR_UNSUPPORTED, "%s: group of %d channels (at most 8192)", fn, d);
    if (too_long(H, d) || (double)M * H * d > kMostElements || (double)H * d > 2147483647.0)
        return fail(QD_ERR_ARG, "%s: sizes overflow", fn);
    if (!(eps > 0.f)) return fail(QD_ERR_ARG, "%s: eps must be positive", fn);
    return QD_OK;
}

qd_status check_workspace(const char *fn, const void *ws, size_t given, size_t need) {
    if (need && (!ws || given < need))
        return fail(QD_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need, ws ? given : (size_t)0);
    return QD_OK;
}

qd_status finish(const char *fn, cudaError_t e, int launches) {
    if (e != cudaSuccess) return fail(QD_ERR_CUDA, "%s launch: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
    return qd::end_call(launches);
}

#define QD_TRY(call)                       \
    do {                                   \
        const qd_status st_ = (call);      \
        if (st_ != QD_OK) return st_;      \
    } while (0)
#define QD_CHECK_POINTERS(fn, args) QD_TRY(check_pointers(fn, args, (int)(sizeof(args) / sizeof(args[0]))))

}  // namespace

extern "C" {

qd_status short_conv_fwd(const void *x, const float *w, const float *bias, const void *S0, const int *lens, void *y,
                         void *S_final, int B, int T, int D, int W, int silu, qd_dtype dtype, cudaStream_t stream) {
    const char *fn = "short_conv_fwd";
    qd::begin_call();
    QD_TRY(check_sizes(fn, B, T, D, dtype));
    QD_TRY(check_taps(fn, W));
    const bool some = B && D, tok = some && T;
    const Named args[] = {{"x", x, tok}, {"w", w, some}, {"bias", bias, false}, {"S0", S0, false}, {"lens", lens, false},
                          {"y", y, tok}, {"S_final", S_final, false}};
    QD_CHECK_POINTERS(fn, args);
    if (!some || (!T && !S_final)) return qd::end_call(0);
    int n = 0;
    const qd::ConvArgs a{x, w, bias, S0, lens, y, S_final, B, T, D, W, silu};
    return finish(fn, qd::launch_conv_fwd(a, dtype, stream, &n), n);
}

qd_status short_conv_step(void *S, const void *x, const float *w, const float *bias, void *y, int N, int D, int W,
                          int silu, qd_dtype dtype, cudaStream_t stream) {
    const char *fn = "short_conv_step";
    qd::begin_call();
    QD_TRY(check_sizes(fn, N, 1, D, dtype));
    QD_TRY(check_taps(fn, W));
    const bool some = N && D;
    const Named args[] = {{"S", S, some}, {"x", x, some}, {"w", w, some}, {"bias", bias, false}, {"y", y, some}};
    QD_CHECK_POINTERS(fn, args);
    if (!some) return qd::end_call(0);
    int n = 0;
    const qd::ConvArgs a{x, w, bias, nullptr, nullptr, y, S, N, 1, D, W, silu};
    return finish(fn, qd::launch_conv_step(a, dtype, stream, &n), n);
}

size_t short_conv_bwd_workspace_bytes(int B, int T, int D, int W, qd_dtype dtype) {
    (void)dtype;
    if (B <= 0 || T < 0 || D <= 0 || W < 2 || W > 4 || too_long(T, D)) return 0;
    return qd::conv_bwd_workspace(B, T, D, W);
}

qd_status short_conv_bwd(const void *x, const float *w, const float *bias, const void *S0, const int *lens, const void *dy,
                         const void *dS_final, void *dx, float *dw, float *dbias, void *dS0, int B, int T, int D, int W,
                         int silu, qd_dtype dtype, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    const char *fn = "short_conv_bwd";
    qd::begin_call();
    QD_TRY(check_sizes(fn, B, T, D, dtype));
    QD_TRY(check_taps(fn, W));
    const bool some = B && D, tok = some && T;
    const Named args[] = {{"x", x, tok}, {"w", w, D > 0}, {"bias", bias, false}, {"S0", S0, false}, {"lens", lens, false},
                          {"dy", dy, tok}, {"dS_final", dS_final, false}, {"dx", dx, tok}, {"dw", dw, D > 0},
                          {"dbias", dbias, false}, {"dS0", dS0, false}, {"workspace", workspace, false}};
    QD_CHECK_POINTERS(fn, args);
    if (some && qd::conv_bwd_ctas(B, T, D) > kMostCtas) return fail(QD_ERR_ARG, "%s: sizes overflow", fn);
    QD_TRY(check_workspace(fn, workspace, workspace_bytes, short_conv_bwd_workspace_bytes(B, T, D, W, dtype)));
    if (!D) return qd::end_call(0);
    int n = 0;
    const qd::ConvBwdArgs a{x, w, bias, S0, lens, dy, dS_final, dx, dw, dbias, dS0, B, T, D, W, silu, (float *)workspace};
    return finish(fn, qd::launch_conv_bwd(a, dtype, stream, &n), n);
}

size_t ssm_workspace_bytes(int B, int T, int D, int G, int N, qd_dtype dtype) {
    (void)dtype;
    if (B <= 0 || T <= 0 || D <= 0 || G <= 0 || D % G || N < 1 || N > 128 || too_long(T, D)) return 0;
    return qd::ssm_fwd_workspace(B, T, D, G, N);
}

qd_status ssm_fwd(const void *x, const void *delta, const float *A, const void *Bm, const void *Cm, const float *Dskip,
                  const float *delta_bias, const float *S0, const int *lens, void *y, float *S_final, int B, int T, int D,
                  int G, int N, int softplus, qd_dtype dtype, void *workspace, size_t workspace_bytes,
                  cudaStream_t stream) {
    const char *fn = "ssm_fwd";
    qd::begin_call();
    QD_TRY(check_ssm(fn, B, T, D, G, N, dtype));
    const bool some = B && D, tok = some && T;
    const Named args[] = {{"x", x, tok}, {"delta", delta, tok}, {"A", A, some}, {"B", Bm, tok}, {"C", Cm, tok},
                          {"D", Dskip, false}, {"delta_bias", delta_bias, false}, {"S0", S0, false}, {"lens", lens, false},
                          {"y", y, tok}, {"S_final", S_final, false}, {"workspace", workspace, false}};
    QD_CHECK_POINTERS(fn, args);
    QD_TRY(check_workspace(fn, workspace, workspace_bytes, ssm_workspace_bytes(B, T, D, G, N, dtype)));
    if (!some || (!T && !S_final)) return qd::end_call(0);
    qd::SsmArgs a{};
    a.x = x; a.delta = delta; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.delta_bias = delta_bias;
    a.S0 = S0; a.lens = lens; a.y = y; a.S_final = S_final;
    a.B = B; a.T = T; a.D = D; a.G = G; a.N = N; a.softplus = softplus; a.ws = workspace;
    int n = 0;
    return finish(fn, qd::launch_ssm_fwd(a, dtype, stream, &n), n);
}

qd_status ssm_step(float *S, const void *x, const void *delta, const float *A, const void *Bm, const void *Cm,
                   const float *Dskip, const float *delta_bias, void *y, int Nseq, int D, int G, int N, int softplus,
                   qd_dtype dtype, cudaStream_t stream) {
    const char *fn = "ssm_step";
    qd::begin_call();
    QD_TRY(check_ssm(fn, Nseq, 1, D, G, N, dtype));
    const bool some = Nseq && D;
    const Named args[] = {{"S", S, some}, {"x", x, some}, {"delta", delta, some}, {"A", A, some}, {"B", Bm, some},
                          {"C", Cm, some}, {"D", Dskip, false}, {"delta_bias", delta_bias, false}, {"y", y, some}};
    QD_CHECK_POINTERS(fn, args);
    if (!some) return qd::end_call(0);
    qd::SsmArgs a{};
    a.x = x; a.delta = delta; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.delta_bias = delta_bias;
    a.y = y; a.S_final = S;
    a.B = Nseq; a.T = 1; a.D = D; a.G = G; a.N = N; a.softplus = softplus;
    int n = 0;
    return finish(fn, qd::launch_ssm_step(a, dtype, stream, &n), n);
}

size_t ssm_bwd_workspace_bytes(int B, int T, int D, int G, int N, qd_dtype dtype) {
    (void)dtype;
    if (B <= 0 || T < 0 || D <= 0 || G <= 0 || D % G || N < 1 || N > 128 || too_long(T, D)) return 0;
    return qd::ssm_bwd_workspace(B, T, D, G, N);
}

qd_status ssm_bwd(const void *x, const void *delta, const float *A, const void *Bm, const void *Cm, const float *Dskip,
                  const float *delta_bias, const float *S0, const int *lens, const void *dy, const float *dS_final,
                  void *dx, void *ddelta, float *dA, void *dBm, void *dCm, float *dDskip, float *ddelta_bias, float *dS0,
                  int B, int T, int D, int G, int N, int softplus, qd_dtype dtype, void *workspace,
                  size_t workspace_bytes, cudaStream_t stream) {
    const char *fn = "ssm_bwd";
    qd::begin_call();
    QD_TRY(check_ssm(fn, B, T, D, G, N, dtype));
    const bool some = B && D, tok = some && T;
    const Named args[] = {{"x", x, tok}, {"delta", delta, tok}, {"A", A, D > 0}, {"B", Bm, tok}, {"C", Cm, tok},
                          {"D", Dskip, false}, {"delta_bias", delta_bias, false}, {"S0", S0, false}, {"lens", lens, false},
                          {"dy", dy, tok}, {"dS_final", dS_final, false}, {"dx", dx, tok}, {"ddelta", ddelta, tok},
                          {"dA", dA, D > 0}, {"dB", dBm, tok}, {"dC", dCm, tok}, {"dD", dDskip, false},
                          {"ddelta_bias", ddelta_bias, false}, {"dS0", dS0, false}, {"workspace", workspace, false}};
    QD_CHECK_POINTERS(fn, args);
    QD_TRY(check_workspace(fn, workspace, workspace_bytes, ssm_bwd_workspace_bytes(B, T, D, G, N, dtype)));
    if (!D) return qd::end_call(0);
    qd::SsmArgs a{};
    a.x = x; a.delta = delta; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.delta_bias = delta_bias;
    a.S0 = S0; a.lens = lens;
    a.B = B; a.T = T; a.D = D; a.G = G; a.N = N; a.softplus = softplus; a.ws = workspace;
    a.dy = dy; a.dS_final = dS_final; a.dx = dx; a.ddelta = ddelta; a.dA = dA; a.dB = dBm; a.dC = dCm;
    a.dD = Dskip ? dDskip : nullptr;
    a.ddelta_bias = delta_bias ? ddelta_bias : nullptr;
    a.dS0 = dS0;
    int n = 0;
    return finish(fn, qd::launch_ssm_bwd(a, dtype, stream, &n), n);
}

qd_status group_norm_fwd(const void *x, const float *w, const float *b, const void *z, void *y, int M, int H, int d,
                         float eps, int center, int silu, qd_dtype dtype, cudaStream_t stream) {
    const char *fn = "group_norm_fwd";
    qd::begin_call();
    QD_TRY(check_norm(fn, M, H, d, eps, dtype));
    const bool some = M && H;
    const Named args[] = {{"x", x, some}, {"w", w, false}, {"b", b, false}, {"z", z, false}, {"y", y, some}};
    QD_CHECK_POINTERS(fn, args);
    if (!some) return qd::end_call(0);
    qd::NormArgs a{};
    a.x = x; a.w = w; a.b = b; a.z = z; a.y = y;
    a.M = M; a.H = H; a.d = d; a.center = center; a.silu = silu; a.eps = eps;
    int n = 0;
    return finish(fn, qd::launch_norm_fwd(a, dtype, stream, &n), n);
}

size_t group_norm_bwd_workspace_bytes(int M, int H, int d, qd_dtype dtype) {
    if (M <= 0 || H <= 0 || d < 1 || d > 8192 || too_long(H, d)) return 0;
    return qd::norm_bwd_workspace(M, H, d, dtype);
}

qd_status group_norm_bwd(const void *x, const float *w, const float *b, const void *z, const void *dy, void *dx, void *dz,
                         float *dw, float *db, int M, int H, int d, float eps, int center, int silu, qd_dtype dtype,
                         void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    const char *fn = "group_norm_bwd";
    qd::begin_call();
    QD_TRY(check_norm(fn, M, H, d, eps, dtype));
    const bool some = M && H;
    const Named args[] = {{"x", x, some}, {"w", w, false}, {"b", b, false}, {"z", z, false}, {"dy", dy, some},
                          {"dx", dx, some}, {"dz", dz, some && z}, {"dw", dw, false}, {"db", db, false},
                          {"workspace", workspace, false}};
    QD_CHECK_POINTERS(fn, args);
    qd::NormArgs a{};
    a.x = x; a.w = w; a.b = b; a.z = z; a.dy = dy; a.dx = dx; a.dz = dz;
    a.dw = w ? dw : nullptr;
    a.db = b ? db : nullptr;
    a.M = M; a.H = H; a.d = d; a.center = center; a.silu = silu; a.eps = eps;
    const bool params = a.dw || a.db;
    if (params) QD_TRY(check_workspace(fn, workspace, workspace_bytes, group_norm_bwd_workspace_bytes(M, H, d, dtype)));
    if (!H || (!M && !params)) return qd::end_call(0);
    a.part = params ? (float *)workspace : nullptr;
    int n = 0;
    return finish(fn, qd::launch_norm_bwd(a, dtype, stream, &n), n);
}

}  // extern "C"
