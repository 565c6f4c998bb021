// Argument checks of the layer-free calls: every tensor of a call as one entry,
// checked for its address, its device and its overlaps.
#pragma once
#include "internal.cuh"

namespace qe {

bool rows_overlap(const void *a, long long lda, int wa, const void *b, long long ldb, int wb, int n,
                  int size);
bool rows_meet(const void *p, long long ld, int w, int n, int size, const void *q, size_t bytes);
bool ranges_meet(const void *p, size_t n, const void *q, size_t m);
bool device_pointer_here(const void *p, int dev);
int record_failure(int code, const char *msg);
int record_success();

constexpr long long kMaxStride = 1LL << 31;

// A tensor of a call: `n` rows of `w` elements of `size` bytes, `ld` elements
// apart; n = 1: one contiguous range.  p null: an optional one left out.
struct Arg {
    const void *p;
    long long ld, w;
    int n, size;
    int align;              // bytes that the rows (n = 1: the range) lie on
    bool written;
    const void *in_place;   // the input of the same layout that this output may be

    size_t bytes() const { return (size_t)w * size; }
};

inline Arg rows_arg(const void *p, long long ld, int w, int n, int size, int align,
                    bool written = false, const void *in_place = nullptr)
{
    return {p, ld, w, n, size, align, written, in_place};
}
inline Arg flat_arg(const void *p, size_t elements, int size, bool written = false)
{
    return {p, 0, (long long)elements, 1, size, size, written, nullptr};
}

inline bool args_meet(const Arg &a, const Arg &b)
{
    if (a.n > 1 && b.n > 1) {
        // the call's rows of one kind: as many in both, elements of one size
        const bool same = a.p == b.p && a.ld == b.ld && a.w == b.w;
        if (same && ((a.written && a.in_place == b.p) || (b.written && b.in_place == a.p)))
            return false;
        return rows_overlap(a.p, a.ld, (int)a.w, b.p, b.ld, (int)b.w, a.n, a.size);
    }
    if (a.n == 1 && b.n == 1) {
        if (a.p == b.p && a.w == b.w && a.size == b.size &&
            ((a.written && a.in_place == b.p) || (b.written && b.in_place == a.p)))
            return false;
        return ranges_meet(a.p, a.bytes(), b.p, b.bytes());
    }
    const Arg &rows = a.n > 1 ? a : b, &flat = a.n > 1 ? b : a;
    return rows_meet(rows.p, rows.ld, (int)rows.w, rows.n, rows.size, flat.p, flat.bytes());
}

// 0, or a recorded failure.  dev and sms get the current device and its SMs.
inline int check_args(const Arg *a, int count, int *dev, int *sms)
{
    for (int i = 0; i < count; i++) {
        if (!a[i].p)
            continue;
        if (a[i].n > 1 && (a[i].ld < a[i].w || a[i].ld > kMaxStride))
            return record_failure(MOE_ERR_INVALID_ARG,
                                  "a row stride is below the row's length or above 2^31");
        if ((uintptr_t)a[i].p % a[i].align || (a[i].n > 1 && a[i].ld * a[i].size % a[i].align))
            return record_failure(MOE_ERR_INVALID_ARG, "misaligned pointer or row stride");
    }
    for (int i = 0; i < count; i++)
        for (int j = 0; j < count; j++)
            if (a[i].p && a[j].p && a[i].written && (j > i || !a[j].written) &&
                args_meet(a[i], a[j]))
                return record_failure(MOE_ERR_INVALID_ARG,
                                      "an output or the workspace overlaps another argument");
    if (cudaGetDevice(dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess) {
        cudaGetLastError();
        return record_failure(MOE_ERR_CUDA, "no usable current CUDA device");
    }
    for (int i = 0; i < count; i++)
        if (a[i].p && a[i].w && !device_pointer_here(a[i].p, *dev))
            return record_failure(MOE_ERR_INVALID_ARG,
                                  "arguments must be device pointers of the current device");
    return MOE_OK;
}

inline int launch_result(cudaError_t e)
{
    if (e != cudaSuccess) {
        cudaGetLastError();
        return record_failure(MOE_ERR_CUDA, cudaGetErrorString(e));
    }
    return record_success();
}

}  // namespace qe
