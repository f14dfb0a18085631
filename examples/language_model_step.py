"""One training step and one sampled token of a small mixture-of-experts model,
with the row operators of libgc where rows are looked up, sorted by expert,
brought back and drawn from, and plain matrix products between them.

    python examples/language_model_step.py [--tokens 512] [--steps 20]

The model: embedding (scaled) -> router -> experts (one matrix each) -> sum
with the input -> logits by the embedding table.  Forward and backward passes
are written out, so every call of the library and its gradient can be seen.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from partition_pass_tile_gb300 import gc  # noqa: E402


class Model:
    def __init__(self, vocab=4096, width=256, experts=16, topk=2, align=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda") / math.sqrt(width)

        self.vocab, self.width, self.experts, self.topk, self.align = vocab, width, experts, topk, align
        self.scale = math.sqrt(width)
        self.params = {"table": normal(vocab, width), "router": normal(width, experts),
                       "expert": normal(experts, width, width)}

    def forward(self, ids):
        """ids [tokens] -> logits [tokens, vocab] and what the backward pass needs."""
        p = self.params
        h = gc.embedding(p["table"], ids, scale=self.scale)
        top, chosen = torch.topk(h @ p["router"], self.topk, dim=1)
        weights = torch.softmax(top, dim=1)
        rows, plan = gc.expert_dispatch(h, chosen, self.experts, align=self.align)
        # every block of rows starts at a multiple of align; its padding rows are zeros
        bounds = plan.offsets.tolist()
        y = torch.zeros_like(rows)
        for e in range(self.experts):
            y[bounds[e]:bounds[e + 1]] = rows[bounds[e]:bounds[e + 1]] @ p["expert"][e]
        out = h + gc.expert_combine(y, plan.slots, weights)
        return out @ p["table"].T, (ids, h, chosen, weights, rows, plan, bounds, y, out)

    def backward(self, d_logits, saved):
        """Gradients of every parameter from the gradient of the logits."""
        ids, h, chosen, weights, rows, plan, bounds, y, out = saved
        p = self.params
        d_out = d_logits @ p["table"]
        d_table = d_logits.T @ out
        d_y, d_weights = gc.expert_combine_grad(d_out, y, plan.slots, plan.pairs, weights)
        d_rows = torch.zeros_like(rows)
        d_expert = torch.zeros_like(p["expert"])
        for e in range(self.experts):
            part = slice(bounds[e], bounds[e + 1])
            d_rows[part] = d_y[part] @ p["expert"][e].T
            d_expert[e] = rows[part].T @ d_y[part]
        d_h = d_out + gc.expert_dispatch_grad(d_rows, plan.slots)
        # softmax over the chosen scores, then back to all of them
        d_top = weights * (d_weights - (weights * d_weights).sum(1, keepdim=True))
        d_scores = torch.zeros(h.shape[0], self.experts, device=h.device).scatter_(1, chosen, d_top)
        d_h += d_scores @ p["router"].T
        d_router = h.T @ d_scores
        # the table serves twice: the lookup's gradient is added to the logits'
        gc.embedding_grad(d_h, ids, self.vocab, scale=self.scale, out=d_table, accumulate=True)
        return {"table": d_table, "router": d_router, "expert": d_expert}

    def loss(self, ids, targets):
        """Mean cross-entropy and the gradient of the logits."""
        logits, saved = self.forward(ids)
        logp = torch.log_softmax(logits, dim=1)
        d_logits = torch.exp(logp)
        d_logits[torch.arange(ids.numel(), device=ids.device), targets] -= 1
        return -logp.gather(1, targets.unsqueeze(1)).mean(), d_logits / ids.numel(), saved

    def train_step(self, ids, targets, rate=0.5):
        loss, d_logits, saved = self.loss(ids, targets)
        for name, grad in self.backward(d_logits, saved).items():
            self.params[name] -= rate * grad
        return loss

    def sample(self, ids, generator, temperature=0.8, top_k=50, top_p=0.95):
        """The next token after each of ids, with its log probability."""
        logits, _ = self.forward(ids)
        uniform = torch.rand(logits.shape, generator=generator, device="cuda")
        return gc.sample(logits, uniform, temperature=temperature, top_k=top_k, top_p=top_p)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    model = Model()
    g = torch.Generator(device="cuda").manual_seed(1)
    # a text in which each token decides the next
    ids = torch.randint(model.vocab, (a.tokens,), generator=g, device="cuda")
    targets = (ids * 7 + 3) % model.vocab
    for step in range(a.steps):
        loss = model.train_step(ids, targets)
        if step % 5 == 0 or step == a.steps - 1:
            print(f"step {step:3d}  loss {loss.item():.4f}")
    tokens, logprobs = model.sample(ids[:8], g)
    print("after ", ids[:8].tolist())
    print("drawn ", tokens.tolist())
    print("learnt", targets[:8].tolist())
    print("log probabilities", [round(v, 3) for v in logprobs.tolist()])


if __name__ == "__main__":
    main()
