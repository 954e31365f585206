// hybrid_layer.h -- host-side declarations of a hybrid decoder's operators: the causal
// convolution, the gated delta rule and the gated norm of its linear-attention layers,
// and the rotary positions of its full-attention ones.
#pragma once

#include "attention_layer.h"

namespace bfp8 {

int launch_causal_conv(const bfp8_causal_conv_args& args, void* stream);
size_t delta_rule_workspace_bytes(int64_t batch, int64_t tokens, int64_t max_q_len,
                                  int64_t qk_heads, int64_t v_heads, int sms);
int launch_delta_rule(const bfp8_delta_rule_args& args, void* stream);
// The device error word of the delta rule's kernels, as those of the projections.
int delta_read_clear_error();
int launch_gated_norm(const bfp8_gated_norm_args& args, void* stream);
int launch_rotary(const bfp8_rotary_args& args, void* stream);

}  // namespace bfp8
