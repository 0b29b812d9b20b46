"""A small recurrent decoder trained on packed sequences, what its norms and linear
layers keep for the backward pass in 8 bits (the recurrence's x' and g and the
GELU's input stay as they are, 6 d of a layer's 15 d values a token):

    python examples/train_recurrent.py [--steps 60] [--dtype bf16|fp32] [--keep8 0|1]

    x = embedding(tokens)                                  lookup, padding skipped
    x, n = layer_norm(x)                                   the first norm
    per layer, for the recurrence and then for the MLP:
        x', g = linear_keep8(n, W_xg);  b = linear_keep8(gated_recurrence(x', g), W_o)
        b = linear_keep8(gelu(linear_keep8(n, W_1)), W_2)
        x, n = layer_norm(x, b)                            residual sum and the next norm in one
    loss = linear_cross_entropy(n, W, targets)             no logits in memory
    loss.backward(); clip_grad_norm(gradients); AdamW

and then run token by token, each layer's memory being one state a sequence. The
data are those of train_block.py."""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_vocab_cross_gb300 as lce  # noqa: E402
from train_block import IGNORE, PAD, batch  # noqa: E402


class Decoder(torch.nn.Module):
    def __init__(self, vocab=1000, d=256, layers=2, dtype=torch.bfloat16, keep8=True):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(0)
        self.d, self.keep8 = d, keep8

        def mat(rows, cols):
            w = torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5
            return torch.nn.Parameter(w.to(dtype))

        def vec(value):
            return torch.nn.Parameter(torch.full((d,), value, device="cuda", dtype=dtype))

        self.W = mat(vocab, d)            # shared by the lookup and the head
        self.w0, self.c0 = vec(1.0), vec(0.0)
        self.layers = torch.nn.ModuleList()
        for _ in range(layers):
            self.layers.append(torch.nn.ParameterDict({
                "xg": mat(2 * d, d), "o": mat(d, d), "up": mat(4 * d, d), "down": mat(d, 4 * d),
                "w1": vec(1.0), "c1": vec(0.0), "w2": vec(1.0), "c2": vec(0.0)}))

    def linear(self, x, w):
        return lce.linear_keep8(x, w) if self.keep8 else F.linear(x, w)

    def norm(self, x, b, w, c):
        return lce.layer_norm(x, b, weight=w, bias=c, keep8=self.keep8)

    def hidden(self, tokens, cu=None, states=None):
        """The head's input, and the states after the tokens. cu: offsets of
        packed sequences; without them tokens are [B, L]."""
        x = lce.embedding(self.W, tokens.reshape(-1), PAD)
        x, n = self.norm(x, None, self.w0, self.c0)
        last = []
        for i, p in enumerate(self.layers):
            xg = self.linear(n, p["xg"])
            if cu is None:
                xg = xg.unflatten(0, tokens.shape)
            h, s = lce.gated_recurrence(xg[..., :self.d], xg[..., self.d:], cu, state=None if states is None else states[i])
            last.append(s)
            x, n = self.norm(x, self.linear(h.reshape(-1, self.d), p["o"]), p["w1"], p["c1"])
            x, n = self.norm(x, self.linear(F.gelu(self.linear(n, p["up"])), p["down"]), p["w2"], p["c2"])
        return n, last

    def forward(self, tokens, cu, targets):
        n, _ = self.hidden(tokens, cu)
        return lce.linear_cross_entropy(n, self.W, targets, IGNORE)


def train(steps=60, dtype=torch.bfloat16, keep8=True, max_norm=1.0, log=None):
    """(model, losses, gradient norms by step)."""
    vocab = 1000
    model = Decoder(vocab, dtype=dtype, keep8=keep8)
    params = list(model.parameters())
    opt = torch.optim.AdamW(params, lr=2e-3, weight_decay=0.0)
    g = torch.Generator().manual_seed(1)
    batches = [batch(g, vocab) for _ in range(8)]
    losses, norms = [], []
    for step in range(steps):
        loss = model(*batches[step % len(batches)])
        opt.zero_grad(set_to_none=True)
        loss.backward()
        norm = lce.clip_grad_norm([p.grad for p in params], max_norm)
        opt.step()
        losses.append(loss.detach())
        norms.append(norm)
        if log and (step % 10 == 0 or step + 1 == steps):
            log(f"step {step:4d}  loss {loss.item():.4f}  gradient norm {norm.item():.3f}")
    return model, torch.stack(losses).tolist(), torch.stack(norms).tolist()


@torch.no_grad()
def generate(model, prompt, count):
    """`count` tokens after each row of prompt [B, L], the most likely ones: the
    prompt at once, then a step of single tokens each."""
    n, states = model.hidden(prompt)
    n = n.view(*prompt.shape, -1)[:, -1]
    out = []
    for _ in range(count):
        token = (n @ model.W.T).argmax(-1, keepdim=True)
        out.append(token)
        n, states = model.hidden(token, states=states)
    return torch.cat(out, 1)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dtype", choices=["bf16", "fp32"], default="bf16")
    ap.add_argument("--keep8", type=int, choices=[0, 1], default=1)
    a = ap.parse_args()
    trained, _, _ = train(a.steps, torch.bfloat16 if a.dtype == "bf16" else torch.float32, bool(a.keep8), log=print)
    print("tokens after 7, 42, 217, 94:", generate(trained, torch.tensor([[7, 42, 217, 94]], device="cuda"), 6).tolist()[0])
