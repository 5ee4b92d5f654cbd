"""Training a next-token model with the operators and the packed blocks.

A model of three blocks in the 16 B/param mixed layout: an embedding, a
residual two-matrix MLP with a norm-free skip, and an LM head. Per step:

  lst_embed           tokens -> hidden states (from the embedding block's W)
  (torch)             the MLP forward
  lst_xent_grad       loss, dx and the head's gradient, into the head block's G
  (torch)             the MLP backward, into the MLP block's G
  lst_embed_grad      the embedding's gradient, into the embedding block's G
  lst_muon_step       MLP matrices by Muon, embedding and head by AdamW

Run: python examples/train_next_token.py [steps]
"""

from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from optimizer_update_gb300 import Layout, lst  # noqa: E402

VOCAB, HIDDEN, FFN, TOKENS = 1000, 128, 344, 512
SPECS = [("embed_tokens", (VOCAB, HIDDEN), 0), ("up_proj", (FFN, HIDDEN), 1), ("down_proj", (HIDDEN, FFN), 1),
         ("lm_head", (VOCAB, HIDDEN), 2)]
MUON = [False, True, True, False]


def tensor_views(layout, blocks, field, dtype):
    """name -> matrix view of `field` of every tensor."""
    out = {}
    for t, (name, shape, block) in enumerate(layout.specs):
        off, _, _ = lst.lst_layout_tensor(layout.handle, t, field)
        size = shape[0] * shape[1] * torch.empty(0, dtype=dtype).element_size()
        out[name] = blocks[block][off:off + size].view(dtype).view(shape)
    return out


def train(steps: int = 60, seed: int = 0, log=print):
    """Returns the list of mean losses."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layout = Layout(SPECS, "L16M")
    blocks = [torch.zeros(layout.block_bytes(b), dtype=torch.uint8, device="cuda") for b in range(layout.n_layers)]
    master = tensor_views(layout, blocks, "MASTER", torch.float32)
    w = tensor_views(layout, blocks, "W", torch.bfloat16)
    g = tensor_views(layout, blocks, "G", torch.bfloat16)
    for name, m in master.items():
        m.copy_(torch.randn(m.shape, generator=gen, device="cuda") * (1.0 if name == "embed_tokens" else HIDDEN ** -0.5))
        w[name].copy_(m)

    # the data: token t is followed by perm[t], one time in ten by any token
    perm = torch.randperm(VOCAB, generator=gen, device="cuda")
    x0 = torch.empty(TOKENS, HIDDEN, dtype=torch.bfloat16, device="cuda")
    dx = torch.empty_like(x0)
    loss, lse = (torch.empty(TOKENS, device="cuda") for _ in range(2))
    mean = torch.empty(1, device="cuda")
    scratch = max(lst.lst_xent_workspace_bytes(TOKENS, HIDDEN, VOCAB, True),
                  lst.lst_embed_grad_workspace_bytes(TOKENS, HIDDEN, VOCAB),
                  lst.lst_muon_workspace_bytes(layout.handle))
    ws = torch.empty(scratch, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    means = []
    for step in range(1, steps + 1):
        tokens = torch.randint(0, VOCAB, (TOKENS,), generator=gen, device="cuda")
        noise = torch.randint(0, VOCAB, (TOKENS,), generator=gen, device="cuda")
        targets = torch.where(torch.rand(TOKENS, generator=gen, device="cuda") < 0.1, noise, perm[tokens])

        lst.lst_embed(lst.matrix(w["embed_tokens"]), lst.indices(tokens), lst.matrix(x0), 1.0, stream)
        up = x0 @ w["up_proj"].T
        act = torch.relu(up)
        x1 = x0 + act @ w["down_proj"].T

        lst.lst_xent_grad(lst.matrix(x1), lst.matrix(w["lm_head"]), lst.indices(targets), -100, 1.0, loss.data_ptr(),
                          lse.data_ptr(), mean.data_ptr(), lst.matrix(dx), lst.matrix(g["lm_head"]), False,
                          ws.data_ptr(), ws.numel(), stream)

        g["down_proj"].copy_(dx.T @ act)
        dup = (dx @ w["down_proj"]) * (up > 0)
        g["up_proj"].copy_(dup.T @ x0)
        dx0 = dx + dup @ w["up_proj"]
        lst.lst_embed_grad(lst.matrix(dx0), lst.indices(tokens), lst.matrix(g["embed_tokens"]), 1.0, False,
                           ws.data_ptr(), ws.numel(), stream)

        lst.lst_muon_step(layout.handle, [b.data_ptr() for b in blocks], lst.muon_hparams(lr=0.02, weight_decay=0.0),
                          lst.adamw_hparams(lr=0.02, weight_decay=0.0, step=step), MUON, ws.data_ptr(), ws.numel(), stream)
        means.append(mean.clone())
        if log and (step == 1 or step % 10 == 0):
            log(f"step {step:4d}  loss {float(means[-1]):.4f}")
    return [float(m) for m in means]


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
