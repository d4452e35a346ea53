// C ABI of the output head (declared in include/dlhead.h): argument checks on
// the host, then the launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "checks.h"
#include "dlhead.h"
#include "head.h"

namespace {

using dlk::Span;
using dlk::aligned_to;
using dlk::check_device_span;
using dlk::span_of;

constexpr int64_t kMaxDim = INT32_MAX;

int64_t esize_of(int dtype) { return dtype == DL_F32 ? 4 : dtype == DL_BF16 ? 2 : 1; }

// Bytes from the first element of a rows x cols matrix to its last; -1 if ld
// is below cols or the span does not fit.
int64_t matrix_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t esize) {
    if (ld < cols) return -1;
    int64_t n = 0;
    if (__builtin_mul_overflow(rows - 1, ld, &n) || __builtin_add_overflow(n, cols, &n) ||
        __builtin_mul_overflow(n, esize, &n))
        return -1;
    return n;
}

// The arrays of one call, checked together: sizes and alignment as they are
// added, then overlaps, then (last, since it asks the HIP runtime) that each
// lies in a device allocation of the current device.
class Arrays {
public:
    int add(const void* p, int64_t bytes, uintptr_t align, bool written, int64_t ld = 0) {
        if (status_ != DL_OK) return -1;
        if (p == nullptr || bytes < 0) {
            status_ = DL_E_INVAL;
            return -1;
        }
        if (!aligned_to(p, align)) {
            status_ = DL_E_ALIGN;
            return -1;
        }
        item_[n_] = Item{p, bytes, ld, written, 0};
        return n_++;
    }
    int in(const void* p, int64_t bytes, uintptr_t align, int64_t ld = 0) {
        return add(p, bytes, align, false, ld);
    }
    int out(const void* p, int64_t bytes, uintptr_t align, int64_t ld = 0) {
        return add(p, bytes, align, true, ld);
    }
    // Output `o` may be input `i` itself.
    void may_be(int o, int i) {
        if (o >= 0 && i >= 0) item_[o].same |= 1u << i;
    }
    int check(void* stream) {
        if (status_ != DL_OK) return status_;
        for (int i = 0; i < n_; ++i)
            for (int j = 0; j < i; ++j)
                if ((item_[i].written || item_[j].written) && clash(i, j)) return DL_E_INVAL;
        if (dlk::hip_error_pending()) return DL_E_HIP;
        int dev = -1;
        if (hipGetDevice(&dev) != hipSuccess) {
            (void)hipGetLastError();
            return DL_E_HIP;
        }
        if (stream != nullptr) {
            hipDevice_t sdev = -1;
            if (hipStreamGetDevice(static_cast<hipStream_t>(stream), &sdev) != hipSuccess) {
                (void)hipGetLastError();
                return DL_E_INVAL;
            }
            if (sdev != dev) return DL_E_INVAL;
        }
        // Small tensors of one program share allocations: the runtime is asked
        // once for each that the call meets.
        Span known[kMost];
        int n_known = 0;
        for (int i = 0; i < n_; ++i) {
            if (item_[i].bytes == 0) continue;
            const Span s = span_of(item_[i].p, item_[i].bytes);
            bool found = false;
            for (int j = 0; j < n_known && !found; ++j)
                found = s.lo >= known[j].lo && s.hi >= s.lo && s.hi <= known[j].hi;
            if (found) continue;
            if (int st = check_device_span(item_[i].p, item_[i].bytes, &known[n_known])) return st;
            ++n_known;
            hipPointerAttribute_t at;
            if (hipPointerGetAttributes(&at, item_[i].p) != hipSuccess) {
                (void)hipGetLastError();
                return DL_E_INVAL;
            }
            if (at.device != dev || at.type == hipMemoryTypeHost) return DL_E_INVAL;
        }
        return DL_OK;
    }

private:
    struct Item {
        const void* p;
        int64_t bytes;
        int64_t ld;
        bool written;
        unsigned same;
    };
    bool clash(int i, int j) const {
        const Item &a = item_[i], &b = item_[j];
        if (a.bytes == 0 || b.bytes == 0) return false;
        if (!span_of(a.p, a.bytes).overlaps(span_of(b.p, b.bytes))) return false;
        const bool allowed = ((a.same >> j) & 1u) != 0 || ((b.same >> i) & 1u) != 0;
        return !(allowed && a.p == b.p && a.ld == b.ld && a.bytes == b.bytes);
    }
    static constexpr int kMost = 12;
    Item item_[kMost];
    int n_ = 0;
    int status_ = DL_OK;
};

bool float_type(int dtype) { return dtype == DL_F32 || dtype == DL_BF16; }

int launched(hipError_t e) { return e == hipSuccess ? DL_OK : DL_E_HIP; }

// Bytes of the scales of a rows x cols matrix; 0 for DL_SCALE_NONE.
int64_t scale_bytes(int kind, int64_t rows, int64_t cols) {
    return kind == DL_SCALE_ROW ? 4 * rows : kind == DL_SCALE_BLOCK32 ? rows * ((cols + 31) / 32) : 0;
}

}  // namespace

extern "C" {

int dl_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldres, int dtype,
               const float* weight, float eps, int64_t rows, int64_t cols, void* sum,
               int64_t ldsum, void* y, int64_t ldy, int y_dtype, void* scales, int scale_kind,
               float* inv_rms, void* stream) {
    if (!float_type(dtype) || !(float_type(y_dtype) || y_dtype == DL_E4M3)) return DL_E_INVAL;
    if (y_dtype == DL_E4M3 ? (scale_kind != DL_SCALE_ROW && scale_kind != DL_SCALE_BLOCK32)
                           : scale_kind != DL_SCALE_NONE)
        return DL_E_INVAL;
    if ((scales != nullptr) != (scale_kind != DL_SCALE_NONE)) return DL_E_INVAL;
    if (rows < 0 || rows > kMaxDim || cols < 1 || cols > DL_MAX_NORM_COLS) return DL_E_INVAL;
    if (!(eps >= 0.0f) || std::isinf(eps)) return DL_E_INVAL;
    if (sum != nullptr && residual == nullptr) return DL_E_INVAL;
    if (rows == 0) return DL_OK;
    const int64_t e = esize_of(dtype), ye = esize_of(y_dtype);
    Arrays a;
    const int ix = a.in(x, matrix_bytes(rows, cols, ldx, e), e, ldx);
    const int ir =
        residual ? a.in(residual, matrix_bytes(rows, cols, ldres, e), e, ldres) : -1;
    a.in(weight, 4 * cols, 4);
    if (sum != nullptr) {
        const int is = a.out(sum, matrix_bytes(rows, cols, ldsum, e), e, ldsum);
        a.may_be(is, ix);
        a.may_be(is, ir);
    }
    a.out(y, matrix_bytes(rows, cols, ldy, ye), ye, ldy);
    if (scales != nullptr)
        a.out(scales, scale_bytes(scale_kind, rows, cols), scale_kind == DL_SCALE_ROW ? 4 : 1);
    if (inv_rms != nullptr) a.out(inv_rms, 4 * rows, 4);
    if (int st = a.check(stream)) return st;
    const dlk::NormArgs k{x,   ldx,   residual, ldres, weight, eps,    rows, static_cast<int>(cols),
                          sum, ldsum, y,        ldy,   scales, inv_rms};
    return launched(dlk::rmsnorm(k, dtype, y_dtype, scale_kind, static_cast<hipStream_t>(stream)));
}

int dl_rmsnorm_workspace_bytes(int64_t rows, int64_t cols, int64_t* bytes) {
    if (bytes == nullptr || rows < 0 || rows > kMaxDim || cols < 1 || cols > DL_MAX_NORM_COLS)
        return DL_E_INVAL;
    *bytes = dlk::rmsnorm_workspace_bytes(rows, cols);
    return DL_OK;
}

int dl_rmsnorm_backward(const void* dy, int64_t lddy, const void* dsum, int64_t lddsum,
                        const void* sum, int64_t ldsum, int dtype, const float* weight,
                        const float* inv_rms, int64_t rows, int64_t cols, void* dx, int64_t lddx,
                        float* dweight, void* workspace, int64_t workspace_bytes, void* stream) {
    int64_t need = 0;
    if (int st = dl_rmsnorm_workspace_bytes(rows, cols, &need)) return st;
    if (!float_type(dtype)) return DL_E_INVAL;
    const int64_t e = esize_of(dtype);
    if (dweight == nullptr) need = 0;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return DL_E_INVAL;
    Arrays a;
    if (rows > 0) {
        const int iy = a.in(dy, matrix_bytes(rows, cols, lddy, e), e, lddy);
        const int is = dsum ? a.in(dsum, matrix_bytes(rows, cols, lddsum, e), e, lddsum) : -1;
        a.in(sum, matrix_bytes(rows, cols, ldsum, e), e, ldsum);
        a.in(weight, 4 * cols, 4);
        a.in(inv_rms, 4 * rows, 4);
        const int ix = a.out(dx, matrix_bytes(rows, cols, lddx, e), e, lddx);
        a.may_be(ix, iy);
        a.may_be(ix, is);
    }
    if (dweight != nullptr) a.out(dweight, 4 * cols, 4);
    if (need > 0) a.out(workspace, need, 256);
    if (rows == 0 && dweight == nullptr) return DL_OK;
    if (int st = a.check(stream)) return st;
    const dlk::NormBackwardArgs k{dy,     lddy,    dsum,  lddsum,
                                  sum,    ldsum,   weight, inv_rms,
                                  rows,   static_cast<int>(cols),
                                  dx,     lddx,    dweight,
                                  static_cast<float*>(workspace)};
    return launched(dlk::rmsnorm_backward(k, dtype, static_cast<hipStream_t>(stream)));
}

int dl_w4_bytes(int64_t rows, int64_t cols, int64_t* packed_bytes, int64_t* scale_bytes) {
    if (packed_bytes == nullptr || scale_bytes == nullptr) return DL_E_INVAL;
    if (rows < 0 || rows > kMaxDim || cols < 1 || cols > kMaxDim) return DL_E_INVAL;
    const int64_t blocks = rows * ((cols + 31) / 32);
    *packed_bytes = blocks * 16;
    *scale_bytes = blocks;
    return DL_OK;
}

int dl_w4_quantize(const void* w, int64_t ldw, int dtype, int64_t rows, int64_t cols,
                   uint8_t* packed, uint8_t* scales, void* values, int64_t ldvalues,
                   void* stream) {
    int64_t pb = 0, sb = 0;
    if (int st = dl_w4_bytes(rows, cols, &pb, &sb)) return st;
    if (!float_type(dtype)) return DL_E_INVAL;
    if (rows == 0) return DL_OK;
    const int64_t e = esize_of(dtype);
    Arrays a;
    const int iw = a.in(w, matrix_bytes(rows, cols, ldw, e), e, ldw);
    a.out(packed, pb, 16);
    a.out(scales, sb, 1);
    if (values != nullptr)
        a.may_be(a.out(values, matrix_bytes(rows, cols, ldvalues, e), e, ldvalues), iw);
    if (int st = a.check(stream)) return st;
    return launched(dlk::w4_quantize(w, ldw, dtype, rows, cols, packed, scales, values, ldvalues,
                                     static_cast<hipStream_t>(stream)));
}

int dl_w4_matvec(const uint8_t* packed, const uint8_t* scales, int64_t rows, int64_t cols,
                 const void* x, int64_t ldx, int x_dtype, const void* x_scales, int x_scale_kind,
                 int count, void* y, int64_t ldy, int y_dtype, void* stream) {
    int64_t pb = 0, sb = 0;
    if (int st = dl_w4_bytes(rows, cols, &pb, &sb)) return st;
    if (x_dtype != DL_BF16 && x_dtype != DL_E4M3) return DL_E_INVAL;
    if (x_dtype == DL_E4M3 ? (x_scale_kind != DL_SCALE_ROW && x_scale_kind != DL_SCALE_BLOCK32)
                           : x_scale_kind != DL_SCALE_NONE)
        return DL_E_INVAL;
    if ((x_scales != nullptr) != (x_scale_kind != DL_SCALE_NONE)) return DL_E_INVAL;
    if (!float_type(y_dtype) || count < 1 || count > DL_MAX_VECTORS) return DL_E_INVAL;
    if (rows == 0) return DL_OK;
    const int64_t xe = esize_of(x_dtype), ye = esize_of(y_dtype);
    Arrays a;
    a.in(packed, pb, 16);
    a.in(scales, sb, 1);
    a.in(x, matrix_bytes(count, cols, ldx, xe), xe);
    if (x_scales != nullptr)
        a.in(x_scales, scale_bytes(x_scale_kind, count, cols),
             x_scale_kind == DL_SCALE_ROW ? 4 : 1);
    a.out(y, matrix_bytes(count, rows, ldy, ye), ye);
    if (int st = a.check(stream)) return st;
    const dlk::MatvecArgs k{packed, scales, rows, cols, x, ldx, x_scales, count, y, ldy};
    return launched(dlk::w4_matvec(k, x_scale_kind, y_dtype, static_cast<hipStream_t>(stream)));
}

int dl_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int top_k, int64_t* bytes) {
    if (bytes == nullptr || rows < 0 || rows > kMaxDim || vocab < 1 || vocab > kMaxDim)
        return DL_E_INVAL;
    if (top_k < 0 || top_k > DL_MAX_TOP || top_k > vocab) return DL_E_INVAL;
    *bytes = rows == 0 ? 0 : dlk::logprobs_workspace_bytes(rows, vocab, top_k);
    return DL_OK;
}

int dl_logprobs(const void* logits, int64_t ldl, int dtype, int64_t rows, int64_t vocab,
                const int64_t* targets, float* logprobs, float* entropy, float* stats, int top_k,
                int64_t* top_ids, float* top_logprobs, void* workspace, int64_t workspace_bytes,
                void* stream) {
    int64_t need = 0;
    if (int st = dl_logprobs_workspace_bytes(rows, vocab, top_k, &need)) return st;
    if (!float_type(dtype)) return DL_E_INVAL;
    if ((targets != nullptr) != (logprobs != nullptr)) return DL_E_INVAL;
    if ((top_ids != nullptr) != (top_k > 0) || (top_logprobs != nullptr) != (top_k > 0))
        return DL_E_INVAL;
    if (rows == 0) return DL_OK;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return DL_E_INVAL;
    const int64_t e = esize_of(dtype);
    Arrays a;
    a.in(logits, matrix_bytes(rows, vocab, ldl, e), e);
    if (targets != nullptr) {
        a.in(targets, 8 * rows, 8);
        a.out(logprobs, 4 * rows, 4);
    }
    if (entropy != nullptr) a.out(entropy, 4 * rows, 4);
    if (stats != nullptr) a.out(stats, 8 * rows, 4);
    if (top_k > 0) {
        a.out(top_ids, 8 * rows * top_k, 8);
        a.out(top_logprobs, 4 * rows * top_k, 4);
    }
    if (need > 0) a.out(workspace, need, 256);
    if (int st = a.check(stream)) return st;
    const dlk::LogprobsArgs k{logits, ldl,   rows,  vocab,   targets,      logprobs,
                              entropy, stats, top_k, top_ids, top_logprobs, workspace};
    return launched(dlk::logprobs(k, dtype, static_cast<hipStream_t>(stream)));
}

int dl_logprobs_backward(const void* logits, int64_t ldl, int dtype, int64_t rows, int64_t vocab,
                         const int64_t* targets, const float* stats, const float* entropy,
                         const float* dlogprobs, const float* dentropy, void* dlogits,
                         int64_t lddl, void* stream) {
    if (!float_type(dtype) || rows < 0 || rows > kMaxDim || vocab < 1 || vocab > kMaxDim)
        return DL_E_INVAL;
    if ((entropy != nullptr) != (dentropy != nullptr)) return DL_E_INVAL;
    if (rows == 0) return DL_OK;
    const int64_t e = esize_of(dtype);
    Arrays a;
    const int il = a.in(logits, matrix_bytes(rows, vocab, ldl, e), e, ldl);
    a.in(targets, 8 * rows, 8);
    a.in(stats, 8 * rows, 4);
    a.in(dlogprobs, 4 * rows, 4);
    if (entropy != nullptr) {
        a.in(entropy, 4 * rows, 4);
        a.in(dentropy, 4 * rows, 4);
    }
    a.may_be(a.out(dlogits, matrix_bytes(rows, vocab, lddl, e), e, lddl), il);
    if (int st = a.check(stream)) return st;
    const dlk::LogprobsBackwardArgs k{logits,  ldl,       rows,     vocab,   targets, stats,
                                      entropy, dlogprobs, dentropy, dlogits, lddl};
    return launched(dlk::logprobs_backward(k, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
