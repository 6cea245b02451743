"""A gated expert layer trained in bf16 over ragged groups and served with 4-bit weights.

    python -m fp8_block_scaled_grouped_amd.examples.ragged_experts [--steps N]

Routing is the library's grouped_topk.  The token-expert pairs are put in expert order once; every
expert product then runs over the ragged groups without padding: grouped_linear (with gradients)
while training, grouped_gemm_fp4 on the packed experts afterwards, with the shared expert's
products through gemm_fp4_groupscale.  No step waits for the GPU.
"""
import argparse

import torch

import fp8_block_scaled_grouped_amd as m


def group_by_expert(topk_ids, E):
    """Pairs t * k + j in expert order (stable), and the int32 [E + 1] offsets of the experts' rows."""
    ids, order = torch.sort(topk_ids.reshape(-1), stable=True)
    edges = torch.arange(E + 1, dtype=ids.dtype, device=ids.device)
    return order, torch.searchsorted(ids, edges, out_int32=True)


def silu_mul(gate_up):
    gate, up = gate_up.float().chunk(2, dim=-1)
    return (torch.nn.functional.silu(gate) * up).to(gate_up.dtype)


class RaggedExperts(torch.nn.Module):
    """out = sum_j weight_j * expert_{id_j}(x) + shared(x), each a gated product of H -> I -> H.

    w1 [E, 2I, H] holds gate rows then up rows, w2 [E, H, I]; the shared expert has s1 [2I, H] and s2
    [H, I].  Master weights are fp32; products run in bf16 until pack() is called, then on 4 bits.
    """

    def __init__(self, H, I, E, n_group, topk_group, topk, device, seed=0):
        super().__init__()
        g = torch.Generator().manual_seed(seed)

        def weight(*shape):
            return torch.nn.Parameter((torch.randn(shape, generator=g) * shape[-1] ** -0.5).to(device))

        self.w1, self.w2 = weight(E, 2 * I, H), weight(E, H, I)
        self.s1, self.s2 = weight(2 * I, H), weight(H, I)
        self.register_buffer("bias", torch.zeros(E, device=device))
        self.E, self.route = E, (n_group, topk_group, topk, True, 1.0)
        self.packed = None

    def pack(self, group=32, scale_format="e8m0"):
        """Quantise the experts: later calls run on the 4-bit weights."""
        with torch.no_grad():
            self.packed = {n: m.fp4_quant_groups(getattr(self, n).to(torch.bfloat16), group, scale_format)
                           for n in ("w1", "w2", "s1", "s2")}
        self.group = group
        return self

    def experts(self, rows, name, offsets):
        if self.packed is None:
            return m.grouped_linear(rows, getattr(self, name).to(torch.bfloat16), offsets)
        return m.grouped_gemm_fp4(rows, *self.packed[name], offsets, self.group)

    def shared(self, x, name):
        if self.packed is None:
            return torch.nn.functional.linear(x, getattr(self, name).to(torch.bfloat16))
        return m.gemm_fp4_groupscale(x, *self.packed[name], self.group)

    def forward(self, x, logits):
        T, k = x.shape[0], self.route[2]
        weights, ids = m.grouped_topk(logits, self.bias, *self.route)
        order, offsets = group_by_expert(ids, self.E)
        h = silu_mul(self.experts(x[order // k], "w1", offsets))
        y = self.experts(h, "w2", offsets)
        pairs = torch.empty_like(y).index_copy(0, order, y).view(T, k, -1)
        out = (pairs.float() * weights[..., None]).sum(1)
        return out + self.shared(silu_mul(self.shared(x, "s1")), "s2").float()


def train(layer, teacher, x, logits, steps, lr=0.5):
    """Plain SGD towards the teacher's outputs; the losses, left on the GPU."""
    losses = []
    for _ in range(steps):
        loss = (layer(x, logits) - teacher(x, logits).detach()).square().mean()
        layer.zero_grad(set_to_none=True)
        loss.backward()
        with torch.no_grad():
            for p in layer.parameters():
                p -= lr * p.grad
        losses.append(loss.detach())
    return torch.stack(losses)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    shape = dict(H=256, I=128, E=16, n_group=4, topk_group=2, topk=4, device="cuda")
    layer, teacher = RaggedExperts(**shape, seed=1), RaggedExperts(**shape, seed=2)
    g = torch.Generator().manual_seed(0)
    x = torch.randn((512, 256), generator=g).to("cuda", torch.bfloat16)
    logits = torch.randn((512, 16), generator=g).to("cuda")
    losses = train(layer, teacher, x, logits, a.steps)
    full = layer(x, logits).detach()
    token = layer.pack()(x[:1], logits[:1])
    print("loss %.4f -> %.4f; one token on 4-bit weights is %.1f%% off the bf16 layer" % (
        losses[0], losses[-1], 100 * float((token - full[:1]).norm() / full[:1].norm())))


if __name__ == "__main__":
    main()
