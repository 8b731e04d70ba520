// verify_jobs.h -- which rows of a sequence are looked at when its drafts are judged.
// (Of no other header: also compiled for the host, where a test replays it.)
#pragma once

#ifdef __CUDACC__
#define WQ_HOST_DEVICE __host__ __device__
#else
#define WQ_HOST_DEVICE
#endif

namespace wq {
namespace verify {

// A row of the target or of the draft, as a place in the sequence, and the place of the
// token in question there: the target's row behind the token's own.
struct Job {
  int row, token_row;
  bool is_draft;
};

// Judging drafts base + 1 .. base + n takes target rows base .. base + n (the last for the
// token that follows) and draft rows base + 1 .. base + n: a draft's first row belongs to a
// token that stands, and need not be there.
WQ_HOST_DEVICE constexpr int jobs_of(int n) { return 2 * n + 1; }

WQ_HOST_DEVICE constexpr Job job_of(int job, int n, int base) {
  return job > n ? Job{base + job - n, base + job - n, true}
                 : Job{base + job, base + job + 1, false};
}

}  // namespace verify
}  // namespace wq
