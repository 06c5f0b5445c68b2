#include "attn.h"
namespace gdn { cudaError_t attn_bwd(const AttnIO&, int, cudaStream_t) { return cudaErrorNotSupported; } }
