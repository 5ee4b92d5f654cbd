"""Training layers from 8-bit activation checkpoints.

A model of packed blocks in the 16 B/param mixed layout: an embedding, LAYERS
residual layers with a norm on either side of a two-matrix MLP and a gate per
channel, and an LM head. What a layer keeps for its backward pass are 8-bit
checkpoints: of the residual stream that its norm reads, of the MLP's inner
activation, and of the MLP's output. Per step:

  lst_embed               tokens -> the residual stream
  lst_residual_norm       per layer: z = norm of the stream (and, behind a layer,
                          stream + gate * norm(MLP(z))), with checkpoints
  lst_xent_grad           loss, gradient of the last z, the head's gradient into its G
  lst_checkpoint_wgrad    the MLP's weight gradients into the layer's G, their inputs
                          restored (and normed again) from the checkpoints
  lst_residual_norm_grad  gradients of stream and MLP output, of gate and norm weights
  lst_embed_grad          the embedding's gradient
  lst_muon_step           MLP matrices by Muon, all else by AdamW

Run: python examples/train_checkpointed_layers.py [steps]
"""

from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from optimizer_update_gb300 import Layout, lst  # noqa: E402

VOCAB, HIDDEN, FFN, TOKENS, LAYERS = 1000, 128, 344, 512, 3
EPS, BRANCH = 1e-5, 0.5
BF16 = torch.bfloat16


def specs():
    out = [("embed_tokens", (VOCAB, HIDDEN), 0)]
    for i in range(LAYERS):
        out += [(f"up_{i}", (FFN, HIDDEN), 1 + i), (f"down_{i}", (HIDDEN, FFN), 1 + i), (f"norm_{i}", (HIDDEN,), 1 + i),
                (f"post_norm_{i}", (HIDDEN,), 1 + i), (f"gate_{i}", (HIDDEN,), 1 + i)]
    return out + [("final_norm", (HIDDEN,), 1 + LAYERS), ("lm_head", (VOCAB, HIDDEN), 1 + LAYERS)]


class Model:
    def __init__(self, seed: int = 0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.layout = Layout(specs(), "L16M")
        self.blocks = [torch.zeros(self.layout.block_bytes(b), dtype=torch.uint8, device="cuda") for b in range(self.layout.n_layers)]
        master, self.w, self.g = (self.views(f, t) for f, t in (("MASTER", torch.float32), ("W", BF16), ("G", BF16)))
        for name, m in master.items():
            if "norm" in name or "gate" in name:
                m.fill_(1.0)
            else:
                m.copy_(torch.randn(m.shape, generator=self.gen, device="cuda") * (1.0 if name == "embed_tokens" else m.shape[1] ** -0.5))
            self.w[name].copy_(m)
        self.muon = ["up_" in name or "down_" in name for name, _, _ in specs()]

        def rows(cols=HIDDEN):
            return torch.empty(TOKENS, cols, dtype=BF16, device="cuda")

        self.params = lst.residual_params(1.0, BRANCH, EPS)
        self.stream8 = [(*lst.checkpoint_buffers(TOKENS, HIDDEN), "i8") for _ in range(LAYERS + 1)]  # what norm i reads
        self.act8 = [(*lst.checkpoint_buffers(TOKENS, FFN), "i8") for _ in range(LAYERS)]
        self.out8 = [(*lst.checkpoint_buffers(TOKENS, HIDDEN), "i8") for _ in range(LAYERS)]
        self.h, self.z, self.dz, self.dh, self.dy = (rows() for _ in range(5))
        self.loss, self.lse = (torch.empty(TOKENS, device="cuda") for _ in range(2))
        self.mean = torch.empty(1, device="cuda")
        dq, da = rows(FFN), rows()
        size = max(lst.lst_xent_workspace_bytes(TOKENS, HIDDEN, VOCAB, True), lst.lst_embed_grad_workspace_bytes(TOKENS, HIDDEN, VOCAB),
                   lst.lst_muon_workspace_bytes(self.layout.handle), lst.lst_residual_norm_grad_workspace_bytes(TOKENS, HIDDEN, 1),
                   lst.lst_checkpoint_wgrad_workspace_bytes(lst.matrix(dq), lst.checkpoint(*self.stream8[0]), lst.matrix(self.g["up_0"])),
                   lst.lst_checkpoint_wgrad_workspace_bytes(lst.matrix(da), lst.checkpoint(*self.act8[0]), lst.matrix(self.g["down_0"])))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def views(self, field, dtype):
        """name -> matrix view of `field` of every tensor."""
        out = {}
        for t, (name, shape, block) in enumerate(self.layout.specs):
            off, _, _ = lst.lst_layout_tensor(self.layout.handle, t, field)
            shape = (1, *shape) if len(shape) == 1 else shape
            out[name] = self.blocks[block][off:off + shape[0] * shape[1] * torch.empty(0, dtype=dtype).element_size()].view(dtype).view(shape)
        return out

    def gradients(self, tokens, targets):
        """Loss and all gradients of one batch, into the blocks' G segments. Returns the mean loss."""
        m, c, s = lst.matrix, lst.checkpoint, torch.cuda.current_stream().cuda_stream
        w, g, ws, size = self.w, self.g, self.ws.data_ptr(), self.ws.numel()
        lst.lst_embed(m(w["embed_tokens"]), lst.indices(tokens), m(self.h), 1.0, s)
        lst.lst_residual_norm(m(self.h), None, None, None, m(w["norm_0"]), self.params, None, m(self.z), c(*self.stream8[0]), None, s)
        masks = []
        for i in range(LAYERS):
            up = self.z @ w[f"up_{i}"].T
            act = torch.relu(up)
            masks.append(up > 0)
            lst.lst_checkpoint_save(m(act), c(*self.act8[i]), s)
            out = act @ w[f"down_{i}"].T
            after = w[f"norm_{i + 1}"] if i + 1 < LAYERS else w["final_norm"]
            lst.lst_residual_norm(m(self.h), m(out), m(w[f"gate_{i}"]), m(w[f"post_norm_{i}"]), m(after), self.params, m(self.h), m(self.z),
                                  c(*self.stream8[i + 1]), c(*self.out8[i]), s)
        lst.lst_xent_grad(m(self.z), m(w["lm_head"]), lst.indices(targets), -100, 1.0, self.loss.data_ptr(), self.lse.data_ptr(),
                          self.mean.data_ptr(), m(self.dz), m(g["lm_head"]), False, ws, size, s)
        dh = None  # nothing reaches the last stream but its norm's gradient
        for i in reversed(range(LAYERS)):
            after = "final_norm" if i + 1 == LAYERS else f"norm_{i + 1}"
            lst.lst_residual_norm_grad(dh, m(self.dz), c(*self.stream8[i + 1]), c(*self.out8[i]), m(w[f"gate_{i}"]), m(w[f"post_norm_{i}"]),
                                       m(w[after]), self.params, m(self.dh), m(self.dy), m(g[f"gate_{i}"]), m(g[f"post_norm_{i}"]), m(g[after]),
                                       False, ws, size, s)
            dh = m(self.dh)
            lst.lst_checkpoint_wgrad(m(self.dy), c(*self.act8[i]), None, EPS, m(g[f"down_{i}"]), False, ws, size, s)
            dup = (self.dy @ w[f"down_{i}"]) * masks[i]
            lst.lst_checkpoint_wgrad(m(dup), c(*self.stream8[i]), m(w[f"norm_{i}"]), EPS, m(g[f"up_{i}"]), False, ws, size, s)
            torch.mm(dup, w[f"up_{i}"], out=self.dz)
        lst.lst_residual_norm_grad(dh, m(self.dz), c(*self.stream8[0]), None, None, None, m(w["norm_0"]), self.params, m(self.dh), None, None, None,
                                   m(g["norm_0"]), False, ws, size, s)
        lst.lst_embed_grad(m(self.dh), lst.indices(tokens), m(g["embed_tokens"]), 1.0, False, ws, size, s)
        return self.mean.clone()

    def update(self, step):
        lst.lst_muon_step(self.layout.handle, [b.data_ptr() for b in self.blocks], lst.muon_hparams(lr=0.02, weight_decay=0.0),
                          lst.adamw_hparams(lr=0.01, weight_decay=0.0, step=step), self.muon, self.ws.data_ptr(), self.ws.numel(),
                          torch.cuda.current_stream().cuda_stream)


def train(steps: int = 60, seed: int = 0, log=print):
    """Returns the list of mean losses."""
    model = Model(seed)
    gen = model.gen
    perm = torch.randperm(VOCAB, generator=gen, device="cuda")  # the data: token t is followed by perm[t]
    means = []
    for step in range(1, steps + 1):
        tokens = torch.randint(0, VOCAB, (TOKENS,), generator=gen, device="cuda")
        means.append(model.gradients(tokens, perm[tokens]))
        model.update(step)
        if log and (step == 1 or step % 10 == 0):
            log(f"step {step:4d}  loss {float(means[-1]):.4f}")
    return [float(m) for m in means]


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
