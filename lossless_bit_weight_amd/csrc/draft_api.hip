// draft_api.hip -- the C ABI declared in include/draft.h: host-side argument
// checks and launches on the caller's stream.  Nothing here allocates,
// synchronises or keeps state.
#include <stdint.h>

#include "../../include/draft.h"
#include "draft_internal.hpp"
#include "mx4_checks.hpp"

using namespace mx4;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 24;
constexpr int64_t kMaxWords = (int64_t)1 << 30;

int check_shape(int64_t B, int64_t D, int64_t V) {
    if (B < 0 || D < 0 || V < 1 || V > kMaxWords) return W12_ERR_SHAPE;
    if (D > DRAFT_MAX_D) return W12_ERR_UNSUPPORTED;
    if (B > kMaxRows / (D + 1)) return W12_ERR_SHAPE;
    if (B > 0 && V > kMaxElems / (B * (D + 1))) return W12_ERR_SHAPE;
    return W12_OK;
}

// [B, rows, V] with strides that cover a row (those of one sequence or one row are
// not read)
int check_words(const void* p, int type, int64_t B, int64_t rows, int64_t V, int64_t ldb,
                int64_t ldd) {
    if ((rows > 1 && (ldd < V || ldd >= kMaxElems)) || (B > 1 && (ldb < 0 || ldb >= kMaxElems)))
        return W12_ERR_SHAPE;
    return aligned(p, (uintptr_t)type_bytes(type)) ? W12_OK : W12_ERR_ALIGN;
}

}  // namespace

extern "C" {

const char* draft_status_string(int status) {
    switch (status) {
        case W12_OK: return "ok";
        case W12_ERR_NULL: return "a required pointer is NULL";
        case W12_ERR_SHAPE:
            return "bad shape (0 <= D, 1 <= V <= 2^30, B (D + 1) <= 2^24, strides cover their "
                   "rows)";
        case W12_ERR_ALIGN: return "pointer not aligned to its type";
        case W12_ERR_DTYPE: return "unknown element type";
        case W12_ERR_UNSUPPORTED: return "more drafted tokens a sequence than draft_verify takes";
        case W12_ERR_HIP: return "HIP launch failed";
        case W12_ERR_WORKSPACE: return "workspace missing, too small or not 256-byte aligned";
        default: return "unknown status";
    }
}

int draft_workspace_bytes(int64_t B, int64_t D, int64_t V, size_t* bytes) {
    if (bytes == nullptr) return W12_ERR_NULL;
    *bytes = 0;
    if (int rc = check_shape(B, D, V)) return rc;
    if (B > 0) *bytes = draft::workspace_bytes(B, D, V);
    return W12_OK;
}

int draft_verify(const void* logits, int logits_type, int64_t B, int64_t D, int64_t V, int64_t ldb,
                 int64_t ldd, const void* drafts, int drafts_i64, const float* uniforms,
                 const void* draft_probs, int probs_type, int64_t pdb, int64_t pdd,
                 const int32_t* lengths, const float* temperature, int32_t* tokens,
                 int32_t* accepted, void* workspace, size_t workspace_bytes, void* stream) {
    if (int rc = check_shape(B, D, V)) return rc;
    if (type_bytes(logits_type) == 0 || (draft_probs && type_bytes(probs_type) == 0))
        return W12_ERR_DTYPE;
    if (B > 0 && (!logits || (D > 0 && !drafts) || !uniforms || !tokens || !accepted))
        return W12_ERR_NULL;
    if (int rc = check_words(logits, logits_type, B, D + 1, V, ldb, ldd)) return rc;
    if (draft_probs != nullptr && D > 0) {
        if (int rc = check_words(draft_probs, probs_type, B, D, V, pdb, pdd)) return rc;
    }
    if (!aligned(drafts, drafts_i64 ? 8 : 4) || !aligned(uniforms, 4) || !aligned(lengths, 4) ||
        !aligned(temperature, 4) || !aligned(tokens, 4) || !aligned(accepted, 4))
        return W12_ERR_ALIGN;
    if (B == 0) return W12_OK;
    if (int rc = check_ws(workspace, workspace_bytes, draft::workspace_bytes(B, D, V))) return rc;
    draft::Args a{};
    a.logits = logits;
    a.f32 = logits_type == W12_OUT_F32;
    a.B = (int)B;
    a.D = (int)D;
    a.V = (int)V;
    a.ldb = ldb;
    a.ldd = ldd;
    a.drafts = drafts;
    a.drafts_i64 = drafts_i64 != 0;
    a.uniforms = uniforms;
    a.probs = D > 0 ? draft_probs : nullptr;
    a.probs_f32 = probs_type == W12_OUT_F32;
    a.pdb = pdb;
    a.pdd = pdd;
    a.lengths = lengths;
    a.temperature = temperature;
    a.tokens = tokens;
    a.accepted = accepted;
    return status_of(draft::launch_verify(a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
