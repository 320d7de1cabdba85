"""A small model trained with all of the library's parts:

  python -m block_wise_dynamic_gb300.demo [steps] [muon]

Next-token prediction on a synthetic text (each token follows from the one
before, with noise): a stable embedding, two 8-bit floating point linear
layers behind a layer norm and an 8-bit head; matrices with 8-bit moments, or
with ``muon`` the layers' two with orthogonalised updates; embedding, norm and
biases with fp32 moments; gradients clipped to norm 1 on the device.  At the
end the loss with the weights in 4 bits.
"""

from __future__ import annotations

import copy
import sys

import torch

from . import AdamW8bit, Muon
from .embedding import StableEmbedding
from .fp4 import Fp4Linear
from .fp8 import Fp8Linear
from .norm import LayerNorm


class Model(torch.nn.Module):
    def __init__(self, vocab: int, dim: int, device, generator=None):
        super().__init__()
        self.embedding = StableEmbedding(vocab, dim, device=device, generator=generator)
        self.norm = LayerNorm(dim, device=device)
        self.up = Fp8Linear(dim, 4 * dim, device=device, dtype=torch.bfloat16)
        self.down = Fp8Linear(4 * dim, dim, device=device, dtype=torch.bfloat16)
        self.head = Fp8Linear(dim, vocab, bias=False, device=device, dtype=torch.bfloat16)

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        x = self.embedding(ids).to(torch.bfloat16)
        x = x + self.down(torch.nn.functional.gelu(self.up(self.norm(x))))
        return self.head(x)

    def four_bit(self) -> "Model":
        """A copy for inference, its linear layers' weights in 4 bits."""
        model = copy.deepcopy(self)
        for name in ("up", "down", "head"):
            setattr(model, name, Fp4Linear(getattr(self, name)))
        return model.requires_grad_(False)


def text(tokens: int, vocab: int, seed: int, device) -> torch.Tensor:
    """Each token is a fixed permutation of the one before, or with
    probability 1/4 any token."""
    g = torch.Generator().manual_seed(seed)
    follow = torch.randperm(vocab, generator=torch.Generator().manual_seed(0))
    noise = torch.rand(tokens, generator=g) < 0.25
    any_token = torch.randint(0, vocab, (tokens,), generator=g)
    out = torch.empty(tokens, dtype=torch.int64)
    last = 0
    for i in range(tokens):
        last = int(any_token[i]) if noise[i] else int(follow[last])
        out[i] = last
    return out.to(device)


def train(steps: int = 200, vocab: int = 512, dim: int = 256, batch: int = 2048, lr: float = 2e-3, device="cuda", log=None,
          muon: bool = False):
    """Trains the model; the losses of all steps."""
    torch.manual_seed(0)
    model = Model(vocab, dim, device)
    vectors = [p for p in model.parameters() if p.dim() == 1] + [model.embedding.weight]
    matrices = [p for p in model.parameters() if all(p is not q for q in vectors)]
    layers = [model.up.weight, model.down.weight] if muon else []
    opt = AdamW8bit([{"params": [p for p in matrices if all(p is not q for q in layers)]},
                     {"params": vectors, "state_bits": 32, "weight_decay": 0.0}], lr=lr, betas=(0.9, 0.99))
    opts = [opt, Muon(layers, lr=lr)] if muon else [opt]
    ids = text(16 * batch + 1, vocab, 1, device)
    losses = []
    for step in range(steps):
        at = (step % 16) * batch
        logits = model(ids[at:at + batch])
        loss = torch.nn.functional.cross_entropy(logits.float(), ids[at + 1:at + batch + 1])
        for o in opts:
            o.zero_grad()
        loss.backward()
        for o in reversed(opts):  # each clips its own gradients
            factor, norm = o.clip_scale(1.0)
            o.step(grad_scale=factor)
        loss = loss.detach()
        losses.append(loss)
        if log and (step % 20 == 0 or step + 1 == steps):
            log(f"step {step}: loss {float(loss):.3f}, gradient norm {float(norm):.3f}")
    if log:
        with torch.no_grad():
            logits = model.four_bit()(ids[:batch])
            log(f"with 4-bit weights: loss {float(torch.nn.functional.cross_entropy(logits.float(), ids[1:batch + 1])):.3f}")
    return [float(x) for x in losses]


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 200, log=print, muon="muon" in sys.argv[2:])
