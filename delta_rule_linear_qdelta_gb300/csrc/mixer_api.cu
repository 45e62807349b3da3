// The C ABI of the mixers beside the Delta rule: linear attention with decays and windowed attention.
// Argument checks and dispatch; nothing here allocates.
#include <math.h>

#include "api_checks.cuh"
#include "mixers.cuh"

namespace {

// The most tokens of a sequence, slots of a cache or heads: kernels add a few tiles to them in 32 bits.
constexpr int kMostSize = 2147483647 - 131071;

bool good_dim(int d) { return d >= 8 && d <= 128 && d % 8 == 0; }

qd_status check_lin(const char *fn, int B, int T, int H, int dk, int dv, qd_dtype dt) {
    if (B < 0 || T < 0 || H < 0) return fail(QD_ERR_ARG, "%s: negative size B=%d T=%d H=%d", fn, B, T, H);
    if (dt != QD_F32 && dt != QD_BF16) return fail(QD_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dt);
    if (!good_dim(dk) || !good_dim(dv))
        return fail(QD_ERR_UNSUPPORTED, "%s: head dims dk=%d dv=%d (multiples of 8 up to 128 are supported)", fn, dk, dv);
    // token arrays, states and the CTAs of a launch, of which no kernel has more than one for each 32 tokens
    // or 8 rows of a state
    if (T > kMostSize || H > kMostSize || (double)B * (T > 1 ? T : 1) * H * (dk > dv ? dk : dv) > kMostElements ||
        (double)B * H * dk * dv > kMostElements || (double)B * H * ((T + 31) / 32) > kMostCtas || (double)B * H * 16 > kMostCtas)
        return fail(QD_ERR_ARG, "%s: sizes overflow", fn);
    return QD_OK;
}

qd_status check_win(const char *fn, int B, int T, int past, int H, int Hkv, int d, int window, int sinks, qd_dtype dt) {
    if (B < 0 || T < 0 || past < 0 || H < 0 || Hkv < 0)
        return fail(QD_ERR_ARG, "%s: negative size B=%d T=%d past=%d H=%d Hkv=%d", fn, B, T, past, H, Hkv);
    if (dt != QD_F32 && dt != QD_BF16) return fail(QD_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dt);
    if (!good_dim(d)) return fail(QD_ERR_UNSUPPORTED, "%s: head dim %d (multiples of 8 up to 128 are supported)", fn, d);
    if (H ? Hkv < 1 || H % Hkv : Hkv != 0) return fail(QD_ERR_ARG, "%s: H=%d is no multiple of the %d key heads", fn, H, Hkv);
    if (window < 1 || sinks < 0) return fail(QD_ERR_ARG, "%s: window=%d (at least 1), sinks=%d (at least 0)", fn, window, sinks);
    const double keys = (double)past + T;
    if (keys > kMostSize || H > kMostSize || (double)B * (keys > 1 ? keys : 1) * H * d > kMostElements ||
        (double)B * H * (floor(keys / 32) + 1) > kMostCtas)
        return fail(QD_ERR_ARG, "%s: sizes overflow", fn);
    return QD_OK;
}

// The cache's slots: their number, and their elements.
qd_status check_cache(const char *fn, int N, int Hkv, int d, int window, int sinks) {
    const double slots = (double)window + sinks;
    if (slots > kMostSize || N * slots * Hkv * d > kMostElements) return fail(QD_ERR_ARG, "%s: sizes overflow", fn);
    return QD_OK;
}

// The sizes of a workspace query that the call itself would refuse need none.
bool lin_sizes_ok(int B, int T, int H, int dk, int dv, qd_dtype dt) {
    return B > 0 && T >= 0 && H > 0 && good_dim(dk) && good_dim(dv) && T <= kMostSize && H <= kMostSize &&
           (dt == QD_F32 || dt == QD_BF16) && (double)B * H * dk * dv <= kMostElements &&
           (double)B * (T > 1 ? T : 1) * H * (dk > dv ? dk : dv) <= kMostElements;
}

}  // namespace

extern "C" {

size_t lin_attn_workspace_bytes(int B, int T, int H, int dk, int dv, qd_dtype dtype) {
    return lin_sizes_ok(B, T, H, dk, dv, dtype) ? qd::lin_fwd_workspace(B, T, H, dk, dv, dtype) : 0;
}

qd_status lin_attn_fwd(const void *q, const void *k, const void *v, const void *g, const float *S0, const int *lens, void *o,
                       float *S_final, int B, int T, int H, int dk, int dv, int g_per_token, qd_dtype dtype,
                       void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    const char *fn = "lin_attn_fwd";
    qd::begin_call();
    QD_TRY(check_lin(fn, B, T, H, dk, dv, dtype));
    const bool some = B && H, tok = some && T;
    const Named args[] = {{"q", q, tok}, {"k", k, tok}, {"v", v, tok}, {"g", g, false}, {"S0", S0, false}, {"lens", lens, false},
                          {"o", o, tok}, {"S_final", S_final, false}, {"workspace", workspace, false}};
    QD_CHECK_POINTERS(fn, args);
    QD_TRY(check_workspace(fn, workspace, workspace_bytes, lin_attn_workspace_bytes(B, T, H, dk, dv, dtype)));
    if (!some || (!T && !S_final)) return qd::end_call(0);
    qd::LinArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0; a.lens = lens; a.o = o; a.S_final = S_final;
    a.B = B; a.T = T; a.H = H; a.nk = dk; a.nv = dv; a.g_token = g_per_token != 0; a.ws = workspace;
    int n = 0;
    return finish(fn, qd::launch_lin_fwd(a, dtype, stream, &n), n);
}

qd_status lin_attn_step(float *S, const void *q, const void *k, const void *v, const void *g, void *o, int N, int H, int dk,
                        int dv, int g_per_token, qd_dtype dtype, cudaStream_t stream) {
    const char *fn = "lin_attn_step";
    qd::begin_call();
    QD_TRY(check_lin(fn, N, 1, H, dk, dv, dtype));
    const bool some = N && H;
    const Named args[] = {{"S", S, some}, {"q", q, some}, {"k", k, some}, {"v", v, some}, {"g", g, false}, {"o", o, some}};
    QD_CHECK_POINTERS(fn, args);
    if (!some) return qd::end_call(0);
    qd::LinArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.o = o; a.S_final = S;
    a.B = N; a.T = 1; a.H = H; a.nk = dk; a.nv = dv; a.g_token = g_per_token != 0;
    int n = 0;
    return finish(fn, qd::launch_lin_step(a, dtype, stream, &n), n);
}

size_t lin_attn_bwd_workspace_bytes(int B, int T, int H, int dk, int dv, qd_dtype dtype) {
    return lin_sizes_ok(B, T, H, dk, dv, dtype) ? qd::lin_bwd_workspace(B, T, H, dk, dv, dtype) : 0;
}

qd_status lin_attn_bwd(const void *q, const void *k, const void *v, const void *g, const float *S0, const int *lens,
                       const void *dO, const float *dS_final, void *dq, void *dk_out, void *dv_out, void *dg, float *dS0,
                       int B, int T, int H, int dk, int dv, int g_per_token, qd_dtype dtype, void *workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
    const char *fn = "lin_attn_bwd";
    qd::begin_call();
    QD_TRY(check_lin(fn, B, T, H, dk, dv, dtype));
    const bool some = B && H, tok = some && T;
    const Named args[] = {{"q", q, tok}, {"k", k, tok}, {"v", v, tok}, {"g", g, false}, {"S0", S0, false}, {"lens", lens, false},
                          {"dO", dO, tok}, {"dS_final", dS_final, false}, {"dq", dq, tok}, {"dk", dk_out, tok},
                          {"dv", dv_out, tok}, {"dg", dg, false}, {"dS0", dS0, false}, {"workspace", workspace, false}};
    QD_CHECK_POINTERS(fn, args);
    if (dg && !(g && g_per_token)) return fail(QD_ERR_ARG, "%s: dg is the gradient of decays for each token", fn);
    QD_TRY(check_workspace(fn, workspace, workspace_bytes, lin_attn_bwd_workspace_bytes(B, T, H, dk, dv, dtype)));
    if (!some || (!T && !dS0)) return qd::end_call(0);
    qd::LinArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0; a.lens = lens;
    a.B = B; a.T = T; a.H = H; a.nk = dk; a.nv = dv; a.g_token = g_per_token != 0; a.ws = workspace;
    a.dO = dO; a.dS_final = dS_final; a.dq = dq; a.dk = dk_out; a.dv = dv_out; a.dg = dg; a.dS0 = dS0;
    int n = 0;
    return finish(fn, qd::launch_lin_bwd(a, dtype, stream, &n), n);
}

qd_status win_attn_fwd(const void *q, const void *k, const void *v, const int *lens, void *o, float *lse, int B, int T, int past,
                       int H, int Hkv, int d, int window, int sinks, float scale, qd_dtype dtype, cudaStream_t stream) {
    const char *fn = "win_attn_fwd";
    qd::begin_call();
    QD_TRY(check_win(fn, B, T, past, H, Hkv, d, window, sinks, dtype));
    const bool tok = B && H && T;
    const Named args[] = {{"q", q, tok}, {"k", k, tok}, {"v", v, tok}, {"lens", lens, false}, {"o", o, tok}, {"lse", lse, false}};
    QD_CHECK_POINTERS(fn, args);
    if (!tok) return qd::end_call(0);
    qd::WinArgs a{};
    a.q = q; a.k = k; a.v = v; a.lens = lens; a.o = o; a.lse = lse;
    a.B = B; a.T = T; a.past = past; a.H = H; a.Hkv = Hkv; a.d = d; a.window = window; a.sinks = sinks; a.scale = scale;
    int n = 0;
    return finish(fn, qd::launch_win_fwd(a, dtype, stream, &n), n);
}

size_t win_attn_bwd_workspace_bytes(int B, int T, int past, int H, int Hkv, int d, int window, int sinks, qd_dtype dtype) {
    if (B <= 0 || T <= 0 || past < 0 || H <= 0 || Hkv <= 0 || H % Hkv || !good_dim(d) || window < 1 || sinks < 0 ||
        (double)past + T > kMostSize || (double)B * T * H * d > kMostElements)
        return 0;
    return qd::win_bwd_workspace(B, T, past, H, Hkv, d, window, sinks, dtype);
}

qd_status win_attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dO,
                       const int *lens, void *dq, void *dk, void *dv, int B, int T, int past, int H, int Hkv, int d,
                       int window, int sinks, float scale, qd_dtype dtype, void *workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
    const char *fn = "win_attn_bwd";
    qd::begin_call();
    QD_TRY(check_win(fn, B, T, past, H, Hkv, d, window, sinks, dtype));
    const bool tok = B && H && T, key = B && H && ((double)past + T) > 0;
    const Named args[] = {{"q", q, tok}, {"k", k, tok}, {"v", v, tok}, {"o", o, tok}, {"lse", lse, tok}, {"dO", dO, tok},
                          {"lens", lens, false}, {"dq", dq, tok}, {"dk", dk, key}, {"dv", dv, key},
                          {"workspace", workspace, false}};
    QD_CHECK_POINTERS(fn, args);
    QD_TRY(check_workspace(fn, workspace, workspace_bytes,
                           win_attn_bwd_workspace_bytes(B, T, past, H, Hkv, d, window, sinks, dtype)));
    if (!key) return qd::end_call(0);
    qd::WinArgs a{};
    a.q = q; a.k = k; a.v = v; a.lens = lens; a.o = (void *)o; a.lse = (float *)lse; a.dO = dO; a.dq = dq; a.dk = dk; a.dv = dv;
    a.B = B; a.T = T; a.past = past; a.H = H; a.Hkv = Hkv; a.d = d; a.window = window; a.sinks = sinks; a.scale = scale;
    a.ws = workspace;
    int n = 0;
    return finish(fn, qd::launch_win_bwd(a, dtype, stream, &n), n);
}

size_t win_attn_step_workspace_bytes(int N, int H, int Hkv, int d, int window, int sinks, qd_dtype dtype) {
    if (N <= 0 || H <= 0 || Hkv <= 0 || H % Hkv || !good_dim(d) || window < 1 || sinks < 0 ||
        (double)window + sinks > kMostSize || (double)N * H * d > kMostElements)
        return 0;
    return qd::win_step_workspace(N, H, Hkv, d, window, sinks, dtype);
}

qd_status win_attn_step(void *K, void *V, const int *pos, const void *q, const void *k, const void *v, void *o, int N, int H,
                        int Hkv, int d, int window, int sinks, float scale, qd_dtype dtype, void *workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
    const char *fn = "win_attn_step";
    qd::begin_call();
    QD_TRY(check_win(fn, N, 1, 0, H, Hkv, d, window, sinks, dtype));
    QD_TRY(check_cache(fn, N, Hkv, d, window, sinks));
    const bool some = N && H;
    const Named args[] = {{"K", K, some}, {"V", V, some}, {"pos", pos, some}, {"q", q, some}, {"k", k, some}, {"v", v, some},
                          {"o", o, some}, {"workspace", workspace, false}};
    QD_CHECK_POINTERS(fn, args);
    QD_TRY(check_workspace(fn, workspace, workspace_bytes, win_attn_step_workspace_bytes(N, H, Hkv, d, window, sinks, dtype)));
    if (!some) return qd::end_call(0);
    qd::WinArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o; a.K = K; a.V = V; a.pos = pos;
    a.B = N; a.T = 1; a.H = H; a.Hkv = Hkv; a.d = d; a.window = window; a.sinks = sinks; a.scale = scale; a.ws = workspace;
    int n = 0;
    return finish(fn, qd::launch_win_step(a, dtype, stream, &n), n);
}

qd_status win_attn_fill(void *K, void *V, const void *k, const void *v, const int *lens, int B, int T, int past, int Hkv, int d,
                        int window, int sinks, qd_dtype dtype, cudaStream_t stream) {
    const char *fn = "win_attn_fill";
    qd::begin_call();
    QD_TRY(check_win(fn, B, T, past, Hkv, Hkv, d, window, sinks, dtype));
    QD_TRY(check_cache(fn, B, Hkv, d, window, sinks));
    const bool key = B && Hkv && ((double)past + T) > 0;
    const Named args[] = {{"K", K, key}, {"V", V, key}, {"k", k, key}, {"v", v, key}, {"lens", lens, false}};
    QD_CHECK_POINTERS(fn, args);
    if (!key) return qd::end_call(0);
    qd::WinArgs a{};
    a.k = k; a.v = v; a.lens = lens; a.K = K; a.V = V;
    a.B = B; a.T = T; a.past = past; a.H = Hkv; a.Hkv = Hkv; a.d = d; a.window = window; a.sinks = sinks;
    int n = 0;
    return finish(fn, qd::launch_win_fill(a, dtype, stream, &n), n);
}

}  // extern "C"
