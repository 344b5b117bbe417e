// libfp8q.so as one translation unit: the block-scaled FP8 entry points and the 8-bit
// feed-forward operators share one device error word and the host-side helpers.
#include "fp8q.cu"
#include "ffn.cu"
