// The experts of a mixture-of-experts layer for a few tokens: entry point.  The
// kernels are in ep_moe.cuh; each weight format is compiled by itself
// (ep_moe_*.cu).
#include "ep_internal.h"
#include "ep_moe.cuh"

namespace ep {

extern template int launch<0>(const UpArgs &, const DownArgs &, cudaStream_t);
extern template int launch<32>(const UpArgs &, const DownArgs &, cudaStream_t);
extern template int launch<64>(const UpArgs &, const DownArgs &, cudaStream_t);
extern template int launch<128>(const UpArgs &, const DownArgs &, cudaStream_t);

namespace {

bool matrix_ok(const ep_matrix *m)
{
    return m->data != nullptr && aligned(m->data, 16) &&
           (m->format == EP_W_BF16 ? m->scale == nullptr && m->zero == nullptr && m->group == 0
                                   : m->scale != nullptr && aligned(m->scale, 2));
}

Weights weights_of(const ep_matrix *m)
{
    return Weights{static_cast<const uint8_t *>(m->data), static_cast<const uint16_t *>(m->scale), m->zero, kMagic};
}

}  // namespace
}  // namespace ep

using namespace ep;

// a term of h; the workspace holds the terms, then the slots' results
static size_t planes_bytes(int64_t n, int I) { return align_up((size_t)n * I * 2, kWsAlign); }

extern "C" size_t ep_moe_workspace_size(int64_t T, int K, int H, int I)
{
    if (T < 0 || K < 1 || H < 1 || I < 1)
        return 0;
    return kPlanes * planes_bytes(T * K, I) + align_up((size_t)T * K * H * sizeof(float), kWsAlign) + kWsAlign;
}

extern "C" int ep_moe_decode(const void *x, const int64_t *topk_idx, const float *topk_weights, int64_t T, int K,
                             int H, int I, int E, int E_local, int rank, const ep_matrix *w13, const ep_matrix *w2,
                             void *out, int out_dtype, void *ws, size_t ws_bytes, int32_t *err, ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (T < 0 || K < 1 || K > EP_MAX_TOPK || H < 8 || H % 8 != 0 || I < 8 || I % 8 != 0 || E < 1 ||
        E > EP_MAX_EXPERTS || E_local < 1 || E % E_local != 0 || rank < 0 || rank >= E / E_local || w13 == nullptr ||
        w2 == nullptr)
        return EP_ERR_INVALID_ARG;
    if ((out_dtype != 0 && out_dtype != 1) || (w13->format != EP_W_BF16 && w13->format != EP_W_INT4) ||
        w2->format != w13->format || w2->group != w13->group)
        return EP_ERR_UNSUPPORTED;
    if (w13->format == EP_W_INT4) {
        const int g = w13->group;
        if ((g != 32 && g != 64 && g != 128) || H % g != 0 || I % g != 0)
            return EP_ERR_INVALID_ARG;
    }
    if (T > kMaxSlots || T * K > kMaxSlots || H > kMaxDim || I > kMaxDim)
        return EP_ERR_UNSUPPORTED;
    if (T == 0)
        return EP_OK;
    if (x == nullptr || topk_idx == nullptr || topk_weights == nullptr || out == nullptr || !aligned(x, 16) ||
        !aligned(out, 16) || !matrix_ok(w13) || !matrix_ok(w2) || ws == nullptr || !aligned(ws, kWsAlign) ||
        ws_bytes < ep_moe_workspace_size(T, K, H, I))
        return EP_ERR_INVALID_ARG;
    const int n = (int)T * K;
    const Routing r{topk_idx, n, K, E, E_local, (int64_t)rank * E_local};
    const Planes h{static_cast<uint8_t *>(ws), (int64_t)planes_bytes(n, I), I};
    const UpArgs up{static_cast<const uint8_t *>(x), r, H, I, weights_of(w13), h, err};
    const DownArgs down{r, topk_weights, (int)T, H, I, weights_of(w2), h, out, out_dtype, 0, 0,
                        reinterpret_cast<float *>(h.h + kPlanes * h.plane_bytes)};
    switch (w13->group) {
    case 0: return launch<0>(up, down, stream);
    case 32: return launch<32>(up, down, stream);
    case 64: return launch<64>(up, down, stream);
    default: return launch<128>(up, down, stream);
    }
}
