"""A layer of experts, forward and backward, on the library's operators.

    x --router--> experts of each token --row_groups--> rows in order
      --GroupedGemm--> up --silu--> --GroupedGemm--> down --places, weights--> out
    x --Gemm--> a projection that all tokens share --Adapters--> + each request's own --> out

`forward` takes tokens and each token's adapter (-1, or no numbers at all: none); `backward` the
gradient to its output, and gives those to x's part through the experts and to
the experts' matrices: the products' gradient to their rows is the same operator
with the matrices read in the other order, the one to the matrices is GroupedGemmK.
Weights and inputs are random.

    python examples/expert_layer.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import layout_general_tensor_gb300 as lgt


class ExpertLayer:
    def __init__(self, hidden, inner, experts, top, adapters=0, rank=16, seed=0):
        self.hidden, self.inner, self.experts, self.top, self.adapters = hidden, inner, experts, top, adapters
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, scale=1.0):  # stored [...][out][in], as a product reads it K-contiguously
            return (torch.randn(shape, generator=g, device="cuda") * scale / shape[-1] ** 0.5).bfloat16()

        self.w_router, self.w_shared = weight(experts, hidden), weight(hidden, hidden)
        self.w_up, self.w_down = weight(experts, inner, hidden), weight(experts, hidden, inner)
        self.up, self.down = lgt.GroupedGemm(experts, inner, hidden), lgt.GroupedGemm(experts, hidden, inner)
        # the gradients to the rows: the same matrices, read in the other order
        self.up_back = lgt.GroupedGemm(experts, hidden, inner, b_layout=lgt.GEMM_MN_CONTIG)
        self.down_back = lgt.GroupedGemm(experts, inner, hidden, b_layout=lgt.GEMM_MN_CONTIG)
        self.up_sums, self.down_sums = lgt.GroupedGemmK(experts, inner, hidden), lgt.GroupedGemmK(experts, hidden, inner)
        if adapters:
            self.a, self.b = weight(adapters, rank, hidden), weight(adapters, hidden, rank, scale=0.1)
            self.scales = torch.full((adapters,), 2.0, device="cuda")
            self.own = lgt.Adapters(adapters, hidden, hidden, rank)
        self.products = {}

    def _order(self, ids, groups):
        offsets = torch.empty(groups + 1, dtype=torch.int32, device="cuda")
        order, places = torch.empty_like(ids), torch.empty_like(ids)
        lgt.row_groups(ids, offsets, order, places)
        return offsets, order, places

    def _shared(self, x, adapter):
        m = x.shape[0]
        if m not in self.products:
            self.products[m] = lgt.Gemm(lgt.make_desc(m, self.hidden, self.hidden, split_k=0))
        y = torch.empty_like(x)
        self.products[m].run(x, self.w_shared, y)
        if self.adapters and adapter is not None:
            offsets, order, _ = self._order(adapter, self.adapters)
            self.own.run(x, self.a, self.b, offsets, order, y, y, scales=self.scales)
        return y

    def forward(self, x, adapter=None):
        """x [tokens][hidden]; adapter: int32 [tokens].  The output, and what `backward` takes."""
        tokens = x.shape[0]
        weights, ids = torch.softmax(x.float() @ self.w_router.float().T, -1).topk(self.top)
        offsets, order, places = self._order(ids.int().flatten(), self.experts)
        rows = x[order // self.top]
        h = torch.empty(tokens * self.top, self.inner, dtype=x.dtype, device="cuda")
        self.up.run(rows, self.w_up, offsets, h)
        a = torch.nn.functional.silu(h)
        y = torch.empty_like(rows)
        self.down.run(a, self.w_down, offsets, y)
        mixed = (y[places.long()].view(tokens, self.top, self.hidden).float() * weights[..., None]).sum(1)
        return (mixed + self._shared(x, adapter).float()).to(x.dtype), (rows, h, a, weights, offsets, order, places)

    def backward(self, kept, d_out):
        """The gradients to x through the experts (their weights and the shared projection aside), to w_up and to w_down."""
        rows, h, a, weights, offsets, order, places = kept
        d_y = (d_out[order // self.top].float() * weights.flatten()[order.long()][:, None]).to(rows.dtype)
        d_a, d_rows = torch.empty_like(h), torch.empty_like(rows)
        d_up, d_down = torch.empty_like(self.w_up), torch.empty_like(self.w_down)
        self.down_back.run(d_y, self.w_down, offsets, d_a)
        self.down_sums.run(d_y, a, offsets, d_down)
        s = torch.sigmoid(h.float())
        d_h = (d_a.float() * s * (1 + h.float() * (1 - s))).to(h.dtype)
        self.up_back.run(d_h, self.w_up, offsets, d_rows)
        self.up_sums.run(d_h, rows, offsets, d_up)
        return d_rows[places.long()].view(-1, self.top, self.hidden).float().sum(1), d_up, d_down


def main(tokens=1000, hidden=1024, inner=512, experts=16, top=4, adapters=5, seed=1):
    layer = ExpertLayer(hidden, inner, experts, top, adapters)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    adapter = torch.randint(-1, adapters, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    out, kept = layer.forward(x, adapter)
    grads = layer.backward(kept, torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16())
    torch.cuda.synchronize()
    return layer, x, adapter, out, grads


if __name__ == "__main__":
    _, _, _, out, grads = main()
    for name, y in (("out", out), *zip(("d x", "d w_up", "d w_down"), grads)):
        print(name, tuple(y.shape), f"rms {float(y.float().square().mean().sqrt()):.4f}")
