// Attention of new tokens over the paged int8 key/value cache: which kernel
// takes which sequences.
//
//   s_ij = scale * q_i . kc_j * (ka / 127)  [+ slope_h * (j - pos_i)]
//   out_i = sum_j softmax(s_i)_j * vc_j * (va / 127)
//
// over the keys j <= pos_i (causal) or all of the sequence's, with codes kc,
// vc and one absmax ka, va per (page, head).
#include <algorithm>

#include "attention.cuh"

namespace llmint8 {

cudaError_t launch_kv_attention(const llmint8_kv_cache &c, const AttnArgs &a, const Workspace &ws,
                                const DeviceInfo &dev, cudaStream_t stream)
{
    AttnParams p{};
    p.c = kv_view(c, ws.status);
    p.q = a.q;
    p.q_token = a.q_token;
    p.q_head = a.q_head;
    p.tokens = a.tokens;
    p.heads = a.heads;
    p.group = a.heads / c.heads;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    p.slopes = a.slopes;
    p.out = a.out;
    p.lse = a.lse;
    p.causal = a.causal ? 1 : 0;
    p.bf16 = a.bf16 ? 1 : 0;
    p.slots = ws.attn_slots;
    p.arrived = ws.attn_arrived;
    // A sequence's rows (new tokens x heads of a group) decide: up to 16 go to
    // the kernel that streams the cache once for them, more to the one that
    // fills tensor core tiles of 256. The lengths are on the device, so a batch
    // that may hold both kinds gets both launches, and each takes its own. A
    // bound that is wrong costs time, and changes the rounding of the weights: a
    // kernel that is alone takes all.
    const int64_t most = std::min(a.max_new, a.tokens) * p.group;
    const bool few = most <= kAttnFewRows;
    if (few || c.batch > 1) {
        p.rows_from = 1;
        p.rows_to = few ? INT32_MAX : kAttnFewRows;
        cudaError_t e = launch_attn_decode(p, c, most <= 8, dev, stream);
        if (e != cudaSuccess || few)
            return e;
    }
    p.rows_from = c.batch > 1 ? kAttnFewRows + 1 : 1;
    p.rows_to = INT32_MAX;
    return launch_attn_prefill(p, c, dev, stream);
}

} // namespace llmint8
