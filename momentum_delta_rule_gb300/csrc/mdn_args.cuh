// Checks of arguments shared by the C ABI's translation units.
#pragma once

#include "mdn_internal.cuh"

namespace mdn {
namespace {

constexpr long kMaxTokens = 0x3fffffffL;

int element_bytes(mdn_dtype dtype) { return dtype == MDN_BF16 ? 2 : 4; }
bool valid_dtype(mdn_dtype dtype) { return dtype == MDN_F32 || dtype == MDN_BF16; }

// Collects a call's pointers and checks them: required ones present, each
// aligned to its element, outputs distinct from everything else.
class Args {
  public:
    Args &in(const void *ptr, int align, bool required = true) {
        add(ptr, align, required);
        return *this;
    }
    Args &out(const void *ptr, int align, bool required = true, const void *may_be = nullptr) {
        if (ptr) {
            for (int i = 0; i < n_; ++i)
                if (seen_[i] == ptr && ptr != may_be) ok_ = false;
            for (int i = 0; i < n_out_; ++i)
                if (outs_[i] == ptr) ok_ = false;
            outs_[n_out_++] = ptr;
        }
        add(ptr, align, required);
        return *this;
    }
    bool ok() const { return ok_; }

  private:
    void add(const void *ptr, int align, bool required) {
        if (!ptr) {
            if (required) ok_ = false;
            return;
        }
        if ((uintptr_t)ptr % align) ok_ = false;
        seen_[n_++] = ptr;
    }
    const void *seen_[32];
    const void *outs_[16];
    int n_ = 0, n_out_ = 0;
    bool ok_ = true;
};

// Alignment of fp32 states [.., N]: whole packets of four where N has them.
int state_align(int N) { return N % 4 == 0 ? 16 : 4; }

bool batch_ok(const int32_t *cu, int n_seq, int B, int T) {
    if (B < 0 || T < 0 || n_seq < 0 || (long)B * T > kMaxTokens) return false;
    if (cu ? B != 1 : n_seq != B) return false;
    return !((uintptr_t)cu & 3u);
}

mdn_status finish(cudaError_t err) {
    if (err == cudaSuccess) return MDN_OK;
    cudaGetLastError();
    return MDN_ERR_CUDA;
}

bool workspace_ok(const void *ws, size_t bytes, size_t need) {
    return need == 0 || (ws && bytes >= need && !((uintptr_t)ws & 255u));
}

}  // namespace
}  // namespace mdn
