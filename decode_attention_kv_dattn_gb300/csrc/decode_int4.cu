// The decode kernel over 4-bit caches: decode.cu's source once more, in a
// translation unit of its own so that the sets of kernels compile in parallel.
#define DATTN_DECODE_INT4_UNIT 1
#include "decode.cu"
