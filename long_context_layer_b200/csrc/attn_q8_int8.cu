// The 8-bit decode kernel over int8 payloads.
#include "q8.cuh"
#define DELTA_Q8_FMT kInt8
#include "attn_q8_impl.cuh"
