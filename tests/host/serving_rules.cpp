// Host build of the serving calls' rules (csrc/serving_rules.h) for CPU unit tests.
#include "serving_rules.h"

extern "C" int64_t fa_host_segment_pages(int64_t pages_per_seq, int64_t window, int64_t q_len)
{
    return fa::pages_of_a_segment(pages_per_seq, window, q_len);
}

extern "C" int32_t fa_host_teams(int64_t segments, int64_t pages, int64_t rows, int64_t D, int64_t most)
{
    return fa::teams_that_pay(segments, pages, rows, D, most);
}

extern "C" int fa_host_once(int64_t B, int64_t Hkv, int64_t rows, int64_t D, int64_t prefix_pages)
{
    return fa::takes_prefix_once(B, Hkv, rows, D, prefix_pages);
}
