"""A small training run in which every large tensor is kept packed.

A token's embedding goes through a gated layer, h = silu(x Wg^T) * (x Wu^T), y = h Wd^T,
and the run learns the outputs of a layer drawn at random:

* the embedding rows are looked up with scaling, their gradient is summed by token;
* the weights are packed to 4 bits (e2m1) for the products, forward and backward;
* what the backward pass needs is kept in 8 bits (e4m3): the inputs of the linear layers,
  which are the products' operands already, and the gated activation's inputs;
* the embedding gradient is then compressed without loss, as the codec does with any
  BF16 gradient, and checked bit for bit.

    python examples/packed_training.py [--steps 30] [--tokens 4096] [--dim 512]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_packing_amd as ibp  # noqa: E402

E4M3, E2M1 = ibp.IBP_MX_E4M3, ibp.IBP_MX_E2M1


class Linear:
    """A weight [outs, ins] in 32 bits with its 4-bit packings for the two products that
    read it: along ins in the forward pass, along outs in the backward pass."""

    def __init__(self, outs: int, ins: int, gen: torch.Generator):
        self.w = torch.randn(outs, ins, generator=gen, device="cuda") * ins ** -0.5
        self.pack()

    def pack(self) -> None:
        self.w4 = ibp.ibp_mx_pack(self.w, E2M1)
        self.w4t = ibp.ibp_mx_pack(self.w.t().contiguous(), E2M1)

    def forward(self, x8: ibp.MxTensor) -> torch.Tensor:
        return ibp.ibp_mx_matmul(x8, self.w4)

    def backward(self, dy: torch.Tensor, x8: ibp.MxTensor) -> tuple[torch.Tensor, torch.Tensor]:
        """(dx, dw) from the gradient of the output and the kept input."""
        dx = ibp.ibp_mx_matmul(ibp.ibp_mx_pack(dy, E4M3), self.w4t)
        return dx, ibp.ibp_mx_linear_wgrad(dy, x8, dw_dtype=torch.float32)

    def step(self, dw: torch.Tensor, lr: float) -> None:
        self.w -= lr * dw
        self.pack()


class Model:
    def __init__(self, vocab: int, dim: int, hidden: int, seed: int):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.table = torch.randn(vocab, dim, generator=gen, device="cuda").to(torch.bfloat16)
        self.scale = 1.0
        self.gate, self.up = Linear(hidden, dim, gen), Linear(hidden, dim, gen)
        self.down = Linear(dim, hidden, gen)

    def forward(self, ids: torch.Tensor) -> tuple[torch.Tensor, tuple]:
        x = ibp.ibp_embedding_lookup(self.table, ids, scale=self.scale)
        x8 = ibp.ibp_mx_pack(x, E4M3)
        h, gate8, up8 = ibp.ibp_mx_swiglu(self.gate.forward(x8), self.up.forward(x8))
        h8 = ibp.ibp_mx_pack(h, E4M3)
        return self.down.forward(h8), (ids, x8, gate8, up8, h8)

    def backward(self, dy: torch.Tensor, kept: tuple) -> dict:
        ids, x8, gate8, up8, h8 = kept
        dh, ddown = self.down.backward(dy, h8)
        dgate, dup = ibp.ibp_mx_swiglu_backward(dh, gate8, up8)
        dx_gate, dwg = self.gate.backward(dgate, x8)
        dx_up, dwu = self.up.backward(dup, x8)
        dtable = ibp.ibp_embedding_grad(dx_gate + dx_up, ids, self.table.shape[0], scale=self.scale)
        return {"table": dtable, "gate": dwg, "up": dwu, "down": ddown}

    def step(self, grads: dict, lr: float) -> None:
        self.table -= (lr * grads["table"].float()).to(torch.bfloat16)
        for name in ("gate", "up", "down"):
            getattr(self, name).step(grads[name], lr)


def kept_bytes(kept: tuple) -> int:
    return sum(m.codes.numel() + m.scales.numel() for m in kept if isinstance(m, ibp.MxTensor))


def compress_gradient(grad: torch.Tensor) -> float:
    """Ratio of the gradient's lossless compression, after a bit-exact round trip."""
    meta, _ = ibp.ibp_build_metadata(grad.view(-1)[: grad.numel() // 4 * 4], 16, 0.9)
    packed = ibp.ibp_compress(meta, grad, 1024)
    back = ibp.ibp_decompress(meta, packed.stream, packed.offsets, packed.n_chunks, 1024)
    assert torch.equal(back.view(torch.int16), grad.view(-1).view(torch.int16)), "round trip"
    return grad.numel() * 16 / int(packed.offsets[-1])


def run(steps: int = 30, tokens: int = 4096, dim: int = 512, vocab: int = 8000, lr: float = 0.3, say=print) -> list[float]:
    """Losses of the steps."""
    teacher, model = Model(vocab, dim, 2 * dim, 1), Model(vocab, dim, 2 * dim, 2)
    model.table.copy_(teacher.table)  # the same words, another layer
    gen = torch.Generator(device="cuda").manual_seed(3)
    losses = []
    for k in range(steps):
        ids = torch.randint(vocab, (tokens,), generator=gen, device="cuda")
        want, _ = teacher.forward(ids)
        y, kept = model.forward(ids)
        diff = y.float() - want.float()
        losses.append(diff.square().mean().item())
        grads = model.backward((diff * (2 / tokens)).to(torch.bfloat16), kept)
        model.step(grads, lr)
        if k % 5 == 0 or k == steps - 1:
            plain = 2 * tokens * (dim + 3 * 2 * dim)
            say(f"step {k}: loss {losses[-1]:.5f}, kept {kept_bytes(kept) / 1e6:.1f} MB instead of {plain / 1e6:.1f}")
    say(f"embedding gradient compressed without loss: ratio {compress_gradient(grads['table']):.3f}")
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=30)
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--dim", type=int, default=512)
    a = p.parse_args()
    run(a.steps, a.tokens, a.dim)
