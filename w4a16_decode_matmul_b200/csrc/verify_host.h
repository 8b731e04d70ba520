// verify_host.h -- launcher of the verification of drafted tokens, called by the C
// ABI after its checks of the arguments.
#pragma once

#include "host.h"
#include "wq.h"

namespace wqh {

cudaError_t run_verify_drafts(const wq_verification& v, void* workspace, cudaStream_t s, int sms);
size_t verify_workspace_bytes(int64_t rows);

}  // namespace wqh
