// The translation unit of the sparse FFN, and of what it shares with the others.
// pi.hip itself stays as it is: the counter summaries of its kernels are tied to
// the bytes of the sources that they were taken from.
#include "pi.hip"
#include "pi_host.hpp"

pi_status pih::launched() { return launch_status(); }
