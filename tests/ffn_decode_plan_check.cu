// The host-side check of decode_plan_check.cu for the plans of the
// feed-forward launches: the same plan with decode::ep_rt_first's rows per
// thread tried first.
#include "decode.cuh"

#define plan(N, Kc, M, sms, out) plan(N, Kc, M, sms, out, sherry::decode::ep_rt_first(N, M, sms))
#include "decode_plan_check.cu"
