// sv_kvfar.cu -- attention over what is left of each sequence behind the pages
// that the prefix kernel reads; rows leave their sums, before the division.  A
// copy of its own: one set of loops for both made the calls for whole sequences
// 2% to 6% longer.
#include "sv_attend.cuh"

namespace sv {

cudaError_t attend_far_setup() { return attend_attributes<true>(); }
cudaError_t attend_far_launch(const AttendJob &j, int sms, cudaStream_t s)
{
    return attend_start<true>(j, sms, s);
}

}  // namespace sv
