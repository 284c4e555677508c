// Host side of filtered sampling: argument checks and the launch. As elsewhere,
// a rejected call touches neither the GPU nor its outputs.
#include "rtopk.h"
#include "rtopk_attn.h"
#include "rtopk_filter.h"

#include <exception>

using rtopk::set_error;

extern "C" size_t rtopk_sample_filtered_workspace_bytes(int R, int V)
{
    if (R < 1 || V < 1 || V > rtopk::kFilterMaxV || R > rtopk::kFilterMaxR)
        return 0;
    return rtopk::kWsFixedBytes + (rtopk::filter_chunks(R, V, false) > 1 ? R * rtopk::kFilterRowBytes : 0);
}

extern "C" int rtopk_sample_filtered(const void *logits, int dtype, int R, int V, int64_t ld, const float *temperature,
                                     const int32_t *top_k, const float *top_p, const float *min_p, const float *u,
                                     int32_t *out_token, float *out_logprob, void *workspace, size_t ws_bytes, void *stream)
{
    const char *what = "filtered sampling";
    if (!logits || !u || !out_token || !out_logprob)
        return set_error(RTOPK_EINVAL, "%s: NULL pointer", what);
    if (dtype != RTOPK_F32 && dtype != RTOPK_F16 && dtype != RTOPK_BF16)
        return set_error(RTOPK_EINVAL, "%s: unknown dtype %d", what, dtype);
    if (R < 1 || V < 1)
        return set_error(RTOPK_EINVAL, "%s: sizes must be >= 1 (R=%d V=%d)", what, R, V);
    if (ld < 0 || (R > 1 && ld < V) || ld > ((int64_t)1 << 40))
        return set_error(RTOPK_EINVAL, "%s: rows of %lld elements do not hold V=%d (or are over 2^40)", what, (long long)ld, V);
    if ((uintptr_t)logits % (dtype == RTOPK_F32 ? 4 : 2))
        return set_error(RTOPK_EINVAL, "%s: logits are not aligned to their element size", what);
    if (V > rtopk::kFilterMaxV || R > rtopk::kFilterMaxR)
        return set_error(RTOPK_ENOTSUP, "%s: V=%d or R=%d exceeds the implementation limits %d and %d", what, V, R,
                         rtopk::kFilterMaxV, rtopk::kFilterMaxR);
    if (workspace && (uintptr_t)workspace % 256)
        return set_error(RTOPK_EINVAL, "%s: workspace is not 256-byte aligned", what);
    const size_t need = rtopk_sample_filtered_workspace_bytes(R, V);
    if (workspace && ws_bytes < need)
        return set_error(RTOPK_ENOMEM, "%s: workspace of %zu bytes is below the %zu needed", what, ws_bytes, need);
    rtopk::FilterArgs a{};
    a.logits = logits;
    a.R = R;
    a.V = V;
    a.ld = ld;
    a.frac = rtopk::filter_frac(V);
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.u = u;
    a.out_token = out_token;
    a.out_logprob = out_logprob;
    const auto go = [&](int chunks, void *ws) {
        const hipError_t e = rtopk::launch_filter(a, dtype, chunks, ws, (hipStream_t)stream);
        if (e != hipSuccess)
            return set_error(RTOPK_EHIP, "%s launch: %s", what, hipGetErrorString(e));
        return (int)RTOPK_OK;
    };
    const int chunks = rtopk::filter_chunks(R, V, top_k && !top_p);
    if (chunks > 1 && workspace)
        return go(chunks, (uint8_t *)workspace + rtopk::kWsFixedBytes);
    if (chunks > 1) {
        // a captured launch would keep the address of a workspace that a later call may free: it takes
        // the form without one
        hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
        const hipError_t e = hipStreamIsCapturing((hipStream_t)stream, &cap);
        if (e != hipSuccess)
            return set_error(RTOPK_EHIP, "%s: hipStreamIsCapturing: %s", what, hipGetErrorString(e));
        if (cap == hipStreamCaptureStatusNone)
            try {
                return rtopk::with_workspace(need, (hipStream_t)stream,
                                             [&](void *ws) { return go(chunks, (uint8_t *)ws + rtopk::kWsFixedBytes); });
            } catch (const std::exception &x) { // it must not leave a C entry point
                return set_error(RTOPK_ENOMEM, "%s: %s", what, x.what());
            }
    }
    return go(1, nullptr);
}
