// wkv7_seq_api.cu — entry points of the causal convolution, the selective scan and the
// group norm (include/wkv7.h): validation on the host, then the launch.
#include <cstdint>
#include <initializer_list>

#include "wkv7_internal.cuh"

namespace {

using wkv7::kHead;

bool dtype_ok(int d) { return d == WKV7_F32 || d == WKV7_BF16; }
bool act_ok(int a) { return a == WKV7_ACT_NONE || a == WKV7_ACT_SILU; }
int64_t dtype_bytes(int d) { return d == WKV7_F32 ? 4 : 2; }

// A tensor as the overlap checks see it: `rows` rows of `width` bytes, `ld` bytes apart.
struct Span {
    const void* p;
    int64_t rows, width, ld;
};
Span flat(const void* p, int64_t bytes) { return {p, bytes > 0 ? 1 : 0, bytes, bytes}; }
Span rows_of(const void* p, int64_t rows, int64_t width, int64_t ld, int elem) {
    return {p, rows, width * elem, ld * elem};
}

bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const uint64_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const uint64_t ea = pa + static_cast<uint64_t>((a.rows - 1) * a.ld + a.width);
    const uint64_t eb = pb + static_cast<uint64_t>((b.rows - 1) * b.ld + b.width);
    if (pa >= eb || pb >= ea) return false;
    if (a.rows > 1 && b.rows > 1 && a.ld == b.ld) {  // columns of one buffer
        const uint64_t ld = static_cast<uint64_t>(a.ld);
        const uint64_t d = pb >= pa ? (pb - pa) % ld : (ld - (pa - pb) % ld) % ld;  // b's first column after a's
        return d < static_cast<uint64_t>(a.width) || d + static_cast<uint64_t>(b.width) > ld;
    }
    return true;
}

// Outputs against every input and against each other.
bool any_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& i : ins)
            if (overlap(*o, i)) return true;
        for (auto q = o + 1; q != outs.end(); ++q)
            if (overlap(*o, *q)) return true;
    }
    return false;
}
// A state that may be updated in place, for the list of inputs: none where it is.
Span state_in(const void* s_in, const void* s_out, int64_t bytes) { return flat(s_in == s_out ? nullptr : s_in, bytes); }

bool misaligned(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & 15u) return true;
    return false;
}

// A row stride covers its row and keeps byte offsets far inside 64 bits.
bool ld_ok(int64_t ld, int64_t width) { return ld >= width && ld < (int64_t(1) << 31); }

int done(cudaError_t e) { return e == cudaSuccess ? WKV7_OK : WKV7_ERR_CUDA; }

constexpr int64_t kMaxChannels = 1 << 20;

// sizes shared by the convolution's three calls
int conv_check(int64_t B, int64_t T, int64_t C, int W, int act, int io_dtype, bool packed) {
    if (B <= 0 || T < 0 || C <= 0 || W <= 0) return WKV7_ERR_INVALID_ARG;
    if (!dtype_ok(io_dtype) || !act_ok(act)) return WKV7_ERR_INVALID_ARG;
    const int64_t rows = packed ? T : B * T;
    if (W < 2 || W > 4 || C > kMaxChannels || rows >= (int64_t(1) << 38) / C || B >= (int64_t(1) << 38) / C)
        return WKV7_ERR_UNSUPPORTED;  // blocks are numbered in 31 bits
    return WKV7_OK;
}

// sizes shared by the scan's calls
int scan_check(int64_t B, int64_t T, int64_t H, int D, int N, int G, int io_dtype, int dt_dtype, bool packed) {
    if (B <= 0 || T < 0 || H <= 0 || D <= 0 || N <= 0 || G <= 0 || H % G != 0) return WKV7_ERR_INVALID_ARG;
    if (!dtype_ok(io_dtype) || !dtype_ok(dt_dtype)) return WKV7_ERR_INVALID_ARG;
    if (D != kHead || (N != 16 && N != 32 && N != 64 && N != 128)) return WKV7_ERR_UNSUPPORTED;
    // blocks, one or more per (sequence, head) or per (chunk, head), are numbered in 31 bits
    const int64_t slots = (packed ? T / 64 : B * ((T + 63) / 64)) + B;
    // and so are rows, which no device's memory reaches
    if (H > kMaxChannels || slots >= (int64_t(1) << 31) / H || (packed ? T : B * T) >= (int64_t(1) << 31))
        return WKV7_ERR_UNSUPPORTED;
    return WKV7_OK;
}

int norm_check(int64_t N, int64_t L, int64_t C, int64_t G, int act, int io_dtype) {
    if (N < 0 || L < 0 || C <= 0 || G <= 0 || C % G != 0) return WKV7_ERR_INVALID_ARG;
    if (!dtype_ok(io_dtype) || !act_ok(act)) return WKV7_ERR_INVALID_ARG;
    // blocks, one per (sample, group) or a few per sample, are numbered in 31 bits
    if (C > kMaxChannels || N * G >= (int64_t(1) << 31) || N >= (int64_t(1) << 30)) return WKV7_ERR_UNSUPPORTED;
    return WKV7_OK;
}

}  // namespace

extern "C" {

int wkv7_causal_conv(const void* x, int64_t ld_x, const float* w, const float* bias, const void* s0, void* y,
                     int64_t ld_y, void* sT, int B, int T, int C, int W, const int32_t* seq_offsets, int act,
                     int io_dtype, void* stream) {
    int s = conv_check(B, T, C, W, act, io_dtype, seq_offsets != nullptr);
    if (s != WKV7_OK) return s;
    if (!w || (T > 0 && (!x || !y))) return WKV7_ERR_INVALID_ARG;
    if (!ld_ok(ld_x, C) || !ld_ok(ld_y, C)) return WKV7_ERR_INVALID_ARG;
    if (misaligned({x, w, bias, s0, y, sT, seq_offsets})) return WKV7_ERR_MISALIGNED;
    const int e = static_cast<int>(dtype_bytes(io_dtype));
    const int64_t rows = seq_offsets ? T : static_cast<int64_t>(B) * T;
    const int64_t st = static_cast<int64_t>(B) * (W - 1) * C * e;
    const int64_t Wc = static_cast<int64_t>(C) * W * 4;
    if (any_overlap({rows_of(y, rows, C, ld_y, e), flat(sT, st)},
                    {rows_of(x, rows, C, ld_x, e), flat(w, Wc), flat(bias, 4L * C), state_in(s0, sT, st),
                     flat(seq_offsets, 4L * (B + 1))}))
        return WKV7_ERR_INVALID_ARG;
    if ((s = wkv7::device_check()) != WKV7_OK) return s;
    if (T == 0 && !sT) return WKV7_OK;
    int* status = nullptr;  // dense batches have nothing to report
    if (seq_offsets && wkv7::device_status_word(&status) != WKV7_OK) return WKV7_ERR_CUDA;
    const wkv7::ConvArgs p{x, ld_x, w, bias, s0, y, ld_y, sT, B, T, C, W, seq_offsets, act, status};
    return done(wkv7::launch_conv(p, io_dtype, static_cast<cudaStream_t>(stream)));
}

int wkv7_causal_conv_step(const void* x, int64_t ld_x, const float* w, const float* bias, const void* s_in, void* y,
                          int64_t ld_y, void* s_out, int B, int C, int W, int act, int io_dtype, void* stream) {
    int s = conv_check(B, 1, C, W, act, io_dtype, false);
    if (s != WKV7_OK) return s;
    if (!x || !w || !y || !s_out) return WKV7_ERR_INVALID_ARG;
    if (!ld_ok(ld_x, C) || !ld_ok(ld_y, C)) return WKV7_ERR_INVALID_ARG;
    if (misaligned({x, w, bias, s_in, y, s_out})) return WKV7_ERR_MISALIGNED;
    const int e = static_cast<int>(dtype_bytes(io_dtype));
    const int64_t st = static_cast<int64_t>(B) * (W - 1) * C * e;
    if (any_overlap({rows_of(y, B, C, ld_y, e), flat(s_out, st)},
                    {rows_of(x, B, C, ld_x, e), flat(w, static_cast<int64_t>(C) * W * 4), flat(bias, 4L * C),
                     state_in(s_in, s_out, st)}))
        return WKV7_ERR_INVALID_ARG;
    if ((s = wkv7::device_check()) != WKV7_OK) return s;
    const wkv7::ConvArgs p{x, ld_x, w, bias, s_in, y, ld_y, s_out, B, 1, C, W, nullptr, act, nullptr};
    return done(wkv7::launch_conv_step(p, io_dtype, static_cast<cudaStream_t>(stream)));
}

size_t wkv7_causal_conv_backward_workspace_bytes(int B, int T, int C, int W, int packed) {
    if (conv_check(B, T, C, W, WKV7_ACT_NONE, WKV7_F32, packed != 0) != WKV7_OK) return 0;
    const long rows = packed ? T : static_cast<long>(B) * T;
    return wkv7::conv_bwd_workspace_floats(rows, C, W) * sizeof(float);
}

int wkv7_causal_conv_backward(const void* x, int64_t ld_x, const float* w, const float* bias, const void* s0,
                              const void* dy, int64_t ld_dy, const void* dsT, void* dx, int64_t ld_dx, float* dw,
                              float* dbias, void* ds0, void* workspace, size_t workspace_bytes, int B, int T, int C,
                              int W, const int32_t* seq_offsets, int act, int io_dtype, void* stream) {
    int s = conv_check(B, T, C, W, act, io_dtype, seq_offsets != nullptr);
    if (s != WKV7_OK) return s;
    if (!w || !dw || (T > 0 && (!x || !dy || !dx || !workspace))) return WKV7_ERR_INVALID_ARG;
    if (!ld_ok(ld_x, C) || !ld_ok(ld_dy, C) || !ld_ok(ld_dx, C)) return WKV7_ERR_INVALID_ARG;
    if (misaligned({x, w, bias, s0, dy, dsT, dx, dw, dbias, ds0, workspace, seq_offsets})) return WKV7_ERR_MISALIGNED;
    const size_t need = wkv7_causal_conv_backward_workspace_bytes(B, T, C, W, seq_offsets != nullptr);
    if (workspace_bytes < need) return WKV7_ERR_INVALID_ARG;
    const int e = static_cast<int>(dtype_bytes(io_dtype));
    const int64_t rows = seq_offsets ? T : static_cast<int64_t>(B) * T;
    const int64_t st = static_cast<int64_t>(B) * (W - 1) * C * e, wb = static_cast<int64_t>(C) * W * 4;
    if (any_overlap({rows_of(dx, rows, C, ld_dx, e), flat(dw, wb), flat(dbias, 4L * C), flat(ds0, st),
                     flat(workspace, static_cast<int64_t>(need))},
                    {rows_of(x, rows, C, ld_x, e), rows_of(dy, rows, C, ld_dy, e), flat(w, wb), flat(bias, 4L * C),
                     flat(s0, st), flat(dsT, st), flat(seq_offsets, 4L * (B + 1))}))
        return WKV7_ERR_INVALID_ARG;
    if ((s = wkv7::device_check()) != WKV7_OK) return s;
    int* status = nullptr;
    if (seq_offsets && wkv7::device_status_word(&status) != WKV7_OK) return WKV7_ERR_CUDA;
    const wkv7::ConvBwdArgs p{x,     ld_x, w,   bias,  s0,  dy, ld_dy, dsT, dx, ld_dx, dw,
                              dbias, ds0,  static_cast<float*>(workspace), B, T, C, W, seq_offsets, act, status};
    return done(wkv7::launch_conv_backward(p, io_dtype, static_cast<cudaStream_t>(stream)));
}

size_t wkv7_selective_scan_workspace_bytes(int B, int T, int H, int D, int N, int packed) {
    if (scan_check(B, T, H, D, N, 1, WKV7_F32, WKV7_F32, packed != 0) != WKV7_OK) return 0;
    return T > 0 ? wkv7::scan_workspace_bytes(B, T, H, N, packed != 0) : 0;
}

int wkv7_selective_scan(const void* x, int64_t ld_x, const void* dt, int64_t ld_dt, const float* A, const void* Bm,
                        int64_t ld_b, const void* Cm, int64_t ld_c, const float* D_skip, const float* dt_bias,
                        const float* s0, void* y, int64_t ld_y, float* sT, void* workspace, size_t workspace_bytes,
                        int B, int T, int H, int D, int N, int G, const int32_t* seq_offsets, int dt_softplus,
                        int io_dtype, int dt_dtype, void* stream) {
    int s = scan_check(B, T, H, D, N, G, io_dtype, dt_dtype, seq_offsets != nullptr);
    if (s != WKV7_OK) return s;
    if (!A || (T > 0 && (!x || !dt || !Bm || !Cm || !y))) return WKV7_ERR_INVALID_ARG;
    const int64_t wx = static_cast<int64_t>(H) * D, wb = static_cast<int64_t>(G) * N;
    if (!ld_ok(ld_x, wx) || !ld_ok(ld_dt, H) || !ld_ok(ld_b, wb) || !ld_ok(ld_c, wb) || !ld_ok(ld_y, wx))
        return WKV7_ERR_INVALID_ARG;
    const int e = static_cast<int>(dtype_bytes(io_dtype)), de = static_cast<int>(dtype_bytes(dt_dtype));
    if (misaligned({x, A, Bm, Cm, D_skip, dt_bias, s0, y, sT, workspace, seq_offsets})) return WKV7_ERR_MISALIGNED;
    if (reinterpret_cast<uintptr_t>(dt) % de || (ld_x * e | ld_b * e | ld_c * e | ld_y * e) & 15)
        return WKV7_ERR_MISALIGNED;
    const size_t need = T > 0 ? wkv7::scan_workspace_bytes(B, T, H, N, seq_offsets != nullptr) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return WKV7_ERR_INVALID_ARG;
    const int64_t rows = seq_offsets ? T : static_cast<int64_t>(B) * T;
    const int64_t st = static_cast<int64_t>(B) * H * D * N * 4;
    if (any_overlap({rows_of(y, rows, wx, ld_y, e), flat(sT, st), flat(workspace, static_cast<int64_t>(need))},
                    {rows_of(x, rows, wx, ld_x, e), rows_of(dt, rows, H, ld_dt, de), rows_of(Bm, rows, wb, ld_b, e),
                     rows_of(Cm, rows, wb, ld_c, e), flat(A, 4L * H), flat(D_skip, 4L * H), flat(dt_bias, 4L * H),
                     state_in(s0, sT, st), flat(seq_offsets, 4L * (B + 1))}))
        return WKV7_ERR_INVALID_ARG;
    if ((s = wkv7::device_check()) != WKV7_OK) return s;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (T == 0) return sT && sT != s0 ? done(wkv7::launch_copy_states(s0, sT, st / 4, cs)) : WKV7_OK;
    int* status = nullptr;
    if (wkv7::device_status_word(&status) != WKV7_OK) return WKV7_ERR_CUDA;
    const wkv7::ScanArgs p{x,  ld_x, dt, ld_dt, A,  Bm, ld_b, Cm, ld_c, D_skip, dt_bias, s0, y, ld_y, sT,
                           workspace, B, T, H, N, G, seq_offsets,
                           dt_softplus ? 1 : 0, dt_dtype, status};
    return done(wkv7::launch_scan(p, io_dtype, cs));
}

int wkv7_selective_scan_step(const void* x, int64_t ld_x, const void* dt, int64_t ld_dt, const float* A,
                             const void* Bm, int64_t ld_b, const void* Cm, int64_t ld_c, const float* D_skip,
                             const float* dt_bias, const float* s_in, void* y, int64_t ld_y, float* s_out, int B,
                             int H, int D, int N, int G, int dt_softplus, int io_dtype, int dt_dtype, void* stream) {
    int s = scan_check(B, 1, H, D, N, G, io_dtype, dt_dtype, false);
    if (s != WKV7_OK) return s;
    if (!x || !dt || !A || !Bm || !Cm || !y || !s_out) return WKV7_ERR_INVALID_ARG;
    const int64_t wx = static_cast<int64_t>(H) * D, wb = static_cast<int64_t>(G) * N;
    if (!ld_ok(ld_x, wx) || !ld_ok(ld_dt, H) || !ld_ok(ld_b, wb) || !ld_ok(ld_c, wb) || !ld_ok(ld_y, wx))
        return WKV7_ERR_INVALID_ARG;
    const int e = static_cast<int>(dtype_bytes(io_dtype)), de = static_cast<int>(dtype_bytes(dt_dtype));
    if (misaligned({x, A, Bm, Cm, D_skip, dt_bias, s_in, y, s_out})) return WKV7_ERR_MISALIGNED;
    if (reinterpret_cast<uintptr_t>(dt) % de || (ld_x * e | ld_b * e | ld_c * e | ld_y * e) & 15)
        return WKV7_ERR_MISALIGNED;
    const int64_t st = static_cast<int64_t>(B) * H * D * N * 4;
    if (any_overlap({rows_of(y, B, wx, ld_y, e), flat(s_out, st)},
                    {rows_of(x, B, wx, ld_x, e), rows_of(dt, B, H, ld_dt, de), rows_of(Bm, B, wb, ld_b, e),
                     rows_of(Cm, B, wb, ld_c, e), flat(A, 4L * H), flat(D_skip, 4L * H), flat(dt_bias, 4L * H),
                     state_in(s_in, s_out, st)}))
        return WKV7_ERR_INVALID_ARG;
    if ((s = wkv7::device_check()) != WKV7_OK) return s;
    const wkv7::ScanArgs p{x, ld_x, dt, ld_dt, A, Bm, ld_b, Cm, ld_c, D_skip, dt_bias, s_in, y, ld_y, s_out,
                           nullptr, B, 1, H, N, G, nullptr, dt_softplus ? 1 : 0, dt_dtype, nullptr};
    return done(wkv7::launch_scan_step(p, io_dtype, static_cast<cudaStream_t>(stream)));
}

size_t wkv7_selective_scan_backward_workspace_bytes(int B, int T, int H, int D, int N, int G, int io_dtype,
                                                    int packed) {
    if (scan_check(B, T, H, D, N, G, io_dtype, WKV7_F32, packed != 0) != WKV7_OK) return 0;
    return T > 0 ? wkv7::scan_backward_workspace_bytes(B, T, H, N, G, io_dtype, packed != 0) : 0;
}

int wkv7_selective_scan_backward(const void* x, int64_t ld_x, const void* dt, int64_t ld_dt, const float* A,
                                 const void* Bm, int64_t ld_b, const void* Cm, int64_t ld_c, const float* D_skip,
                                 const float* dt_bias, const float* s0, const void* dy, int64_t ld_dy,
                                 const float* dsT, void* dx, int64_t ld_dx, void* ddt, int64_t ld_ddt, float* dA,
                                 void* dB, int64_t ld_db, void* dC, int64_t ld_dc, float* dD, float* ddt_bias,
                                 float* ds0, void* workspace, size_t workspace_bytes, int B, int T, int H, int D,
                                 int N, int G, const int32_t* seq_offsets, int dt_softplus, int io_dtype,
                                 int dt_dtype, void* stream) {
    int s = scan_check(B, T, H, D, N, G, io_dtype, dt_dtype, seq_offsets != nullptr);
    if (s != WKV7_OK) return s;
    if (!A || !dA || (T > 0 && (!x || !dt || !Bm || !Cm || !dy || !dx || !ddt || !dB || !dC || !workspace)))
        return WKV7_ERR_INVALID_ARG;
    const int64_t wx = static_cast<int64_t>(H) * D, wb = static_cast<int64_t>(G) * N;
    for (int64_t ld : {ld_x, ld_dy, ld_dx})
        if (!ld_ok(ld, wx)) return WKV7_ERR_INVALID_ARG;
    for (int64_t ld : {ld_b, ld_c, ld_db, ld_dc})
        if (!ld_ok(ld, wb)) return WKV7_ERR_INVALID_ARG;
    if (!ld_ok(ld_dt, H) || !ld_ok(ld_ddt, H)) return WKV7_ERR_INVALID_ARG;
    const int e = static_cast<int>(dtype_bytes(io_dtype)), de = static_cast<int>(dtype_bytes(dt_dtype));
    if (misaligned({x, A, Bm, Cm, D_skip, dt_bias, s0, dy, dsT, dx, dA, dB, dC, dD, ddt_bias, ds0, workspace,
                    seq_offsets}))
        return WKV7_ERR_MISALIGNED;
    if (reinterpret_cast<uintptr_t>(dt) % de || reinterpret_cast<uintptr_t>(ddt) % de ||
        (ld_x * e | ld_b * e | ld_c * e | ld_dy * e | ld_dx * e | ld_db * e | ld_dc * e) & 15)
        return WKV7_ERR_MISALIGNED;
    const size_t need = wkv7_selective_scan_backward_workspace_bytes(B, T, H, D, N, G, io_dtype, seq_offsets != nullptr);
    if (workspace_bytes < need) return WKV7_ERR_INVALID_ARG;
    const int64_t rows = seq_offsets ? T : static_cast<int64_t>(B) * T;
    const int64_t st = static_cast<int64_t>(B) * H * D * N * 4;
    if (any_overlap({rows_of(dx, rows, wx, ld_dx, e), rows_of(ddt, rows, H, ld_ddt, de), flat(dA, 4L * H),
                     rows_of(dB, rows, wb, ld_db, e), rows_of(dC, rows, wb, ld_dc, e), flat(dD, 4L * H),
                     flat(ddt_bias, 4L * H), flat(ds0, st), flat(workspace, static_cast<int64_t>(need))},
                    {rows_of(x, rows, wx, ld_x, e), rows_of(dt, rows, H, ld_dt, de), flat(A, 4L * H),
                     rows_of(Bm, rows, wb, ld_b, e), rows_of(Cm, rows, wb, ld_c, e), flat(D_skip, 4L * H),
                     flat(dt_bias, 4L * H), flat(s0, st), rows_of(dy, rows, wx, ld_dy, e), flat(dsT, st),
                     flat(seq_offsets, 4L * (B + 1))}))
        return WKV7_ERR_INVALID_ARG;
    if ((s = wkv7::device_check()) != WKV7_OK) return s;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        for (float* p : {dA, dD, ddt_bias})
            if (p && wkv7::launch_copy_states(nullptr, p, H, cs) != cudaSuccess) return WKV7_ERR_CUDA;
        return ds0 ? done(wkv7::launch_copy_states(dsT, ds0, st / 4, cs)) : WKV7_OK;
    }
    int* status = nullptr;
    if (wkv7::device_status_word(&status) != WKV7_OK) return WKV7_ERR_CUDA;
    const wkv7::ScanBwdArgs p{x,      ld_x,  dt,  ld_dt,  A,  Bm, ld_b,  Cm, ld_c,  D_skip, dt_bias,  s0,
                              dy,     ld_dy, dsT, dx,     ld_dx, ddt, ld_ddt, dA, dB, ld_db, dC, ld_dc,
                              dD,     ddt_bias, ds0, workspace, B, T, H, N, G, seq_offsets, dt_softplus ? 1 : 0,
                              dt_dtype, status};
    return done(wkv7::launch_scan_backward(p, io_dtype, cs));
}

size_t wkv7_group_norm_workspace_bytes(int N, int L, int C, int G, int io_dtype) {
    if (norm_check(N, L, C, G, WKV7_ACT_NONE, io_dtype) != WKV7_OK) return 0;
    return wkv7::norm_workspace_floats(N, L, C, G, io_dtype, false) * sizeof(float);
}

int wkv7_group_norm(const void* x, int64_t ld_x, const float* weight, const float* bias, void* y, int64_t ld_y,
                    float* stats, void* workspace, size_t workspace_bytes, int N, int L, int C, int G, float eps,
                    int act, int io_dtype, void* stream) {
    int s = norm_check(N, L, C, G, act, io_dtype);
    if (s != WKV7_OK) return s;
    if (!(eps >= 0.f)) return WKV7_ERR_INVALID_ARG;
    const int64_t rows = static_cast<int64_t>(N) * L;
    if (rows > 0 && (!x || !y)) return WKV7_ERR_INVALID_ARG;
    if (!ld_ok(ld_x, C) || !ld_ok(ld_y, C)) return WKV7_ERR_INVALID_ARG;
    if (misaligned({x, weight, bias, y, stats, workspace})) return WKV7_ERR_MISALIGNED;
    const size_t need = wkv7_group_norm_workspace_bytes(N, L, C, G, io_dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return WKV7_ERR_INVALID_ARG;
    const int e = static_cast<int>(dtype_bytes(io_dtype));
    if (any_overlap({rows_of(y, rows, C, ld_y, e), flat(stats, 8L * N * G),
                     flat(workspace, static_cast<int64_t>(need))},
                    {rows_of(x, rows, C, ld_x, e), flat(weight, 4L * C), flat(bias, 4L * C)}))
        return WKV7_ERR_INVALID_ARG;
    if ((s = wkv7::device_check()) != WKV7_OK) return s;
    if (rows == 0) return WKV7_OK;
    const wkv7::NormArgs p{x, ld_x, weight, bias, y, ld_y, stats, static_cast<float*>(workspace), N, L, C, G, eps,
                           act};
    return done(wkv7::launch_norm(p, io_dtype, static_cast<cudaStream_t>(stream)));
}

size_t wkv7_group_norm_backward_workspace_bytes(int N, int L, int C, int G, int io_dtype) {
    if (norm_check(N, L, C, G, WKV7_ACT_NONE, io_dtype) != WKV7_OK) return 0;
    return wkv7::norm_workspace_floats(N, L, C, G, io_dtype, true) * sizeof(float);
}

int wkv7_group_norm_backward(const void* x, int64_t ld_x, const float* weight, const float* bias, const float* stats,
                             const void* dy, int64_t ld_dy, void* dx, int64_t ld_dx, float* dweight, float* dbias,
                             void* workspace, size_t workspace_bytes, int N, int L, int C, int G, int act,
                             int io_dtype, void* stream) {
    int s = norm_check(N, L, C, G, act, io_dtype);
    if (s != WKV7_OK) return s;
    const int64_t rows = static_cast<int64_t>(N) * L;
    if (rows > 0 && (!x || !stats || !dy || !dx)) return WKV7_ERR_INVALID_ARG;
    if (!ld_ok(ld_x, C) || !ld_ok(ld_dy, C) || !ld_ok(ld_dx, C)) return WKV7_ERR_INVALID_ARG;
    if (misaligned({x, weight, bias, stats, dy, dx, dweight, dbias, workspace})) return WKV7_ERR_MISALIGNED;
    const size_t need = wkv7_group_norm_backward_workspace_bytes(N, L, C, G, io_dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return WKV7_ERR_INVALID_ARG;
    const int e = static_cast<int>(dtype_bytes(io_dtype));
    if (any_overlap({rows_of(dx, rows, C, ld_dx, e), flat(dweight, 4L * C), flat(dbias, 4L * C),
                     flat(workspace, static_cast<int64_t>(need))},
                    {rows_of(x, rows, C, ld_x, e), rows_of(dy, rows, C, ld_dy, e), flat(weight, 4L * C),
                     flat(bias, 4L * C), flat(stats, 8L * N * G)}))
        return WKV7_ERR_INVALID_ARG;
    if ((s = wkv7::device_check()) != WKV7_OK) return s;
    const wkv7::NormBwdArgs p{x,  ld_x,  weight,  bias,  stats, dy, ld_dy, dx, ld_dx, dweight, dbias,
                              static_cast<float*>(workspace), N, L, C, G, act};
    return done(wkv7::launch_norm_backward(p, io_dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
