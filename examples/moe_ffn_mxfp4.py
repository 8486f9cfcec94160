"""A mixture-of-experts feed-forward block on MXFP4 weights.

The router's choices are sorted by expert once; the experts' gate and up projections read
their tokens through that order, the down projection reads the sorted rows, and combine
weights the experts' answers and brings them back to the tokens.  Nothing is read back to
the host: the experts' row counts stay on the GPU.

    python -m examples.moe_ffn_mxfp4
"""
import torch
import torch.nn.functional as F

import q4_quantized_matmul_gb300 as q4q


class MoeFfn:
    """Weights: gate and up of every expert stacked along the rows, [experts, 2 * ff, hidden]; down [experts, hidden, ff]."""

    def __init__(self, router, gate_up, down, top_k):
        self.router, self.top_k = router, top_k
        self.experts, self.ff2, self.hidden = gate_up.shape
        self.gate_up, self.down = q4q.q4q_quantize_mxfp4(gate_up), q4q.q4q_quantize_mxfp4(down)

    def __call__(self, x):
        logits, ids = (x.float() @ self.router.float().T).topk(self.top_k, dim=-1)
        weights = torch.softmax(logits, dim=-1)
        first, slot, row = q4q.q4q_moe_sort(ids.int(), self.experts)
        h = q4q.q4q_mul_mat_id_mxfp4(self.gate_up, self.hidden, self.ff2, x, first, slot, self.top_k)
        gate, up = h.chunk(2, dim=-1)
        h = (F.silu(gate) * up).contiguous()
        h = q4q.q4q_mul_mat_id_mxfp4(self.down, self.ff2 // 2, self.hidden, h, first)
        return q4q.q4q_moe_combine(h, first, row, weights)


def main(tokens=64, hidden=1024, ff=2048, experts=16, top=4):
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()
    x = randn(tokens, hidden)
    router = randn(experts, hidden, scale=hidden ** -0.5)
    gate_up, down = randn(experts, 2 * ff, hidden, scale=hidden ** -0.5), randn(experts, hidden, ff, scale=ff ** -0.5)

    # the same block in fp32 on the weights that MXFP4 stands for, expert by expert
    ffn = MoeFfn(router, gate_up, down, top)
    y = ffn(x).float()
    logits, ids = (x.float() @ router.float().T).topk(top, dim=-1)
    weights = torch.softmax(logits, dim=-1)
    ref = torch.zeros_like(y)
    for e in range(experts):
        t, j = torch.where(ids == e)
        gate, up = (x[t].float() @ q4q.q4q_get_rows_mxfp4(ffn.gate_up[e], hidden, 2 * ff).T).chunk(2, dim=-1)
        ref.index_add_(0, t, weights[t, j, None] * ((F.silu(gate) * up) @ q4q.q4q_get_rows_mxfp4(ffn.down[e], ff, hidden).T))
    off = float((y - ref).norm() / ref.norm())
    print("%d tokens, %d experts: relative difference to fp32 activations %.3f" % (tokens, experts, off))
    return off


if __name__ == "__main__":
    main()
