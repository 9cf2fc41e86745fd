// paged_decode_shared.cu -- the decode kernels of attention behind shared rows: the
// instances of paged_decode.cu that run one of its two lines (PagedShare), in a file of
// their own so that they compile beside the others.
#define EXATTN_PAGED_SHARED
#include "paged_decode.cu"
