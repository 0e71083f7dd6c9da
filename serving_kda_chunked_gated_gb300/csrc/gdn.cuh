// What the two forms of the scalar-gated delta rule's prefill share.
#pragma once

#include <stdint.h>

#include "../../include/kda.h"

namespace kda {
namespace gdn {

// Up to this many sequences the host lays the work out, by value.
constexpr int MAX_LISTED = 1024;

// The sequences that a launch is about; count 0: all.
struct Sequences {
    int count;
    uint16_t seq[MAX_LISTED];
};

// Per-token recurrence over `which`: all sequences, or some beside the kernel launched before, on which
// these do not depend.
cudaError_t launch_recurrent(const kda_gdn_prefill_args& a, const Sequences& which, cudaStream_t s);

}  // namespace gdn
}  // namespace kda
