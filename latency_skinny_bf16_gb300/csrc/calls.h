// calls.h -- what api.cu shares with the entry points outside it.
#pragma once

#include "internal.h"

namespace skinny {

// The library's state on the current device, for one call.
struct CallCtx {
    int num_sms;
    int *status;         // device status word
    uint64_t budget_ns;  // budget of each bounded wait
    bool pdl;            // programmatic dependent launch (SKINNY_OPT_PDL)
    int force_backend;   // SKINNY_OPT_FORCE_BACKEND
};
skinny_status_t call_context(CallCtx *c);   // sets the device up if need be
bool ranges_overlap(uintptr_t a0, uintptr_t a1, uintptr_t b0, uintptr_t b1);
// skinny_gemm_bf16 / skinny_gemm_bf16_bf16out, and their checks without the launch
// (allow_pdl false: the launch waits for what precedes it whatever the option says)
skinny_status_t check_gemm(const uint16_t *X, int ldx, const uint16_t *W, int ldw, const void *Y, int ldy, int M,
                           int N, int K, int out_bf16);
skinny_status_t run_gemm(const uint16_t *X, int ldx, const uint16_t *W, int ldw, void *Y, int ldy, int M, int N,
                         int K, void *stream, int out_bf16, bool allow_pdl = true);

}  // namespace skinny
