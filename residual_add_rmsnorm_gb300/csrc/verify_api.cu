// verify_api.cu -- the C ABI of the drafts' verification (rarn_verify_drafts): argument
// checks before anything is enqueued, one launch, no memory allocated.
#include "../../include/rarn.h"
#include "host.h"
#include "kv_check.h"
#include "verify.cuh"

namespace rarn {
namespace verify {
// instantiated in verify_{bf16,f16,f32}.cu
extern template cudaError_t launch_verify<__nv_bfloat16>(const Params &, int, bool, cudaStream_t);
extern template cudaError_t launch_verify<__half>(const Params &, int, bool, cudaStream_t);
extern template cudaError_t launch_verify<float>(const Params &, int, bool, cudaStream_t);
}  // namespace verify
}  // namespace rarn

using namespace rarn;
using namespace rarn::check;

static_assert(RARN_MAX_VERIFY_VOCAB == verify::kMaxVocab, "vocabulary limit");
static_assert(RARN_MAX_VERIFY_TREE == verify::kMaxTree, "tree limit");

extern "C" rarn_status rarn_verify_drafts(int64_t *new_tokens, int32_t *path, int32_t *lengths,
                                          rarn_rows probs, const rarn_rows *draft_probs,
                                          const int64_t *tokens, const int32_t *parents,
                                          const int32_t *starts, const float *uniforms,
                                          const float *final_uniforms, int64_t B, int64_t rows,
                                          int64_t vocab, int64_t most, void *stream) {
    if (B < 0 || rows < 0 || vocab < 1 || most < 0 || !type_ok(probs.dtype))
        return RARN_ERR_INVALID_ARG;
    const int64_t W = most + 1;
    if (vocab > RARN_MAX_VERIFY_VOCAB || B > RARN_MAX_SEQUENCES || W > (1 << 24) ||
        rows > (int64_t(1) << 31) - 1 || (draft_probs && parents))
        return RARN_ERR_UNSUPPORTED;
    if (draft_probs && draft_probs->dtype != probs.dtype) return RARN_ERR_UNSUPPORTED;
    if (B == 0) return RARN_OK;
    const int64_t s = size_of(probs.dtype);
    auto sound = [&](const rarn_rows &m) {
        if (rows == 0) return RARN_OK;
        if (!m.data || !on(m.data, (unsigned)s) || m.row_stride < 0 ||
            (rows > 1 && m.row_stride < vocab))
            return RARN_ERR_INVALID_ARG;
        return reaches(m.row_stride, rows) ? RARN_OK : RARN_ERR_UNSUPPORTED;
    };
    rarn_status st;
    if ((st = sound(probs)) != RARN_OK) return st;
    if (draft_probs && (st = sound(*draft_probs)) != RARN_OK) return st;
    if (!new_tokens || !on(new_tokens, 8) || !path || !on(path, 4) || !lengths || !on(lengths, 4) ||
        !starts || !on(starts, 4) || !final_uniforms || !on(final_uniforms, 4))
        return RARN_ERR_INVALID_ARG;
    if (rows > 0 && (!tokens || !on(tokens, 8) || !uniforms || !on(uniforms, 4) || !on(parents, 4)))
        return RARN_ERR_INVALID_ARG;
    auto span = [&](const rarn_rows &m) {
        return solid(m.data,
                     rows > 0 ? ((rows - 1) * (rows > 1 ? m.row_stride : 0) + vocab) * s : 0);
    };
    const Range outs[3] = {solid(new_tokens, B * W * 8), solid(path, B * W * 4),
                           solid(lengths, B * 4)};
    const Range ins[7] = {span(probs),
                          draft_probs ? span(*draft_probs) : Range{},
                          solid(tokens, rows * 8),
                          parents ? solid(parents, rows * 4) : Range{},
                          solid(starts, (B + 1) * 4),
                          solid(uniforms, rows * 4),
                          solid(final_uniforms, B * 4)};
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)
            if (meet(outs[i], outs[j])) return RARN_ERR_ALIAS;
        for (const Range &x : ins)
            if (meet(outs[i], x)) return RARN_ERR_ALIAS;
    }
    host::Device dev;
    if ((st = host::current_device(&dev)) != RARN_OK) return st;
    verify::Params p{};
    p.p = probs.data;
    p.ldp = probs.row_stride;
    auto packs = [&](const rarn_rows &m) {
        return on(m.data, 16) && (rows <= 1 || m.row_stride * s % 16 == 0);
    };
    p.vec = packs(probs);
    if (draft_probs) {
        p.q = draft_probs->data;
        p.ldq = draft_probs->row_stride;
        p.vec = p.vec && packs(*draft_probs);
    }
    p.tokens = tokens;
    p.parents = parents;
    p.starts = starts;
    p.u = uniforms;
    p.v = final_uniforms;
    p.out_tokens = new_tokens;
    p.path = path;
    p.lengths = lengths;
    p.rows = rows;
    p.B = (int)B;
    p.V = (int)vocab;
    p.W = (int)W;
    p.watchdog = dev.watchdog;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool pdl = host::pdl_enabled();
    cudaError_t e;
    switch (probs.dtype) {
    case RARN_BF16: e = verify::launch_verify<__nv_bfloat16>(p, dev.num_sms, pdl, cs); break;
    case RARN_F16: e = verify::launch_verify<__half>(p, dev.num_sms, pdl, cs); break;
    default: e = verify::launch_verify<float>(p, dev.num_sms, pdl, cs); break;
    }
    return e == cudaSuccess ? RARN_OK : host::cuda_failed(e);
}
