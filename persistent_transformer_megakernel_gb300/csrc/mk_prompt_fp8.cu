// Attention of whole prompts over an 8-bit cache.
#include "mk_prompt.cuh"

namespace mkprompt {

template int launch<true, 64>(PromptParams &, int, cudaStream_t);
template int launch<true, 128>(PromptParams &, int, cudaStream_t);

}  // namespace mkprompt
