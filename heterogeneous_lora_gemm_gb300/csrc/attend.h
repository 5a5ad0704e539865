// Attention over the 8-bit cache: what the handle (cache.cu) keeps for its kernels.
#pragma once
#include "cache.h"

namespace mlora {

constexpr int ATTEND_OCC = 3;               // CTAs per SM of the split kernel at most
constexpr int ATTEND_SLOT = 16 * (256 + 2); // floats of one partial result at most
constexpr int PROMPT_SLOT = 256 * (128 + 2);// floats of one partial result of the prompt kernel (one per SM at most)

struct AttendWs {
    CUtensorMap k16, v16;   // codes as rows of head_dim bytes, boxes of 16 tokens
    float* partial;         // [sms * ATTEND_OCC * 2][ATTEND_SLOT], or [sms][PROMPT_SLOT]
    int* counters;          // [sms * ATTEND_OCC] arrivals, zero between calls
    int sms;
    uint8_t* operands;      // converted tiles of prompts (attend_prompt.cu), operand_bytes of them
    size_t operand_bytes;
    int* operand_at;        // [n_seqs <= 65535] where a sequence's tiles are
};

cudaError_t attend_split_init();
cudaError_t launch_attend_split(bool bf16, const AttendArgs& a, const AttendWs& ws, cudaStream_t st);

// Sequences with many rows (attend_prompt.cu): bf16, and fp32 with heads of up to 128 elements.
cudaError_t attend_prompt_init();
// Workspace for the converted tiles of `tokens` tokens.
size_t attend_prompt_bytes(const CachePages& c, long long tokens);
bool attend_prompt_takes(bool bf16, const AttendArgs& a);
cudaError_t launch_attend_prompt(bool bf16, const AttendArgs& a, const AttendWs& ws, cudaStream_t st);

}  // namespace mlora
