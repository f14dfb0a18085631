"""Training steps, a sampled token and a drafted run of tokens of a small
mixture-of-experts model, with the row operators of libgc where rows are looked
up, routed, sorted by expert, brought back, drawn from and verified, and plain
matrix products between them.

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
    def __init__(self, vocab=4096, width=256, experts=16, topk=2, align=16, seed=0, balance=0.01):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda") / math.sqrt(width)

        self.vocab, self.width, self.experts, self.topk, self.align = vocab, width, experts, topk, align
        self.scale = math.sqrt(width)
        # what even use of the experts weighs against the likelihood
        self.balance = torch.full((1,), balance, device="cuda")
        self.params = {"table": normal(vocab, width), "router": normal(width, experts),
                       "expert": normal(experts, width, width)}

    def forward(self, ids):
        """ids [tokens] -> logits [tokens, vocab] and what the backward pass needs."""
        p = self.params
        h = gc.embedding(p["table"], ids, scale=self.scale)
        scores = h @ p["router"]
        routing = gc.expert_route(scores, self.topk)
        rows, plan = gc.expert_dispatch(h, routing.ids, self.experts, align=self.align)
        # every block of rows starts at a multiple of align; its padding rows are zeros
        bounds = plan.offsets.tolist()
        y = torch.zeros_like(rows)
        for e in range(self.experts):
            y[bounds[e]:bounds[e + 1]] = rows[bounds[e]:bounds[e + 1]] @ p["expert"][e]
        out = h + gc.expert_combine(y, plan.slots, routing.weights)
        return out @ p["table"].T, (ids, h, scores, routing, rows, plan, bounds, y, out)

    def backward(self, d_logits, saved):
        """Gradients of every parameter from the gradient of the logits, and of the balance loss."""
        ids, h, scores, routing, rows, plan, bounds, y, out = saved
        p = self.params
        d_out = d_logits @ p["table"]
        d_table = d_logits.T @ out
        d_y, d_weights = gc.expert_combine_grad(d_out, y, plan.slots, plan.pairs, routing.weights)
        d_rows = torch.zeros_like(rows)
        d_expert = torch.zeros_like(p["expert"])
        for e in range(self.experts):
            part = slice(bounds[e], bounds[e + 1])
            d_rows[part] = d_y[part] @ p["expert"][e].T
            d_expert[e] = rows[part].T @ d_y[part]
        d_h = d_out + gc.expert_dispatch_grad(d_rows, plan.slots)
        # the weights' gradient and the balance loss's, back to the scores
        d_scores = gc.expert_route_grad(scores, routing.ids, routing.counts, dweights=d_weights, dloss=self.balance)
        d_h += d_scores @ p["router"].T
        d_router = h.T @ d_scores
        # the table serves twice: the lookup's gradient is added to the logits'
        gc.embedding_grad(d_h, ids, self.vocab, scale=self.scale, out=d_table, accumulate=True)
        return {"table": d_table, "router": d_router, "expert": d_expert}

    def loss(self, ids, targets):
        """Mean cross-entropy plus the weighted balance loss, and the gradient of the logits."""
        logits, saved = self.forward(ids)
        logp = torch.log_softmax(logits, dim=1)
        d_logits = torch.exp(logp)
        d_logits[torch.arange(ids.numel(), device=ids.device), targets] -= 1
        loss = -logp.gather(1, targets.unsqueeze(1)).mean() + (self.balance * saved[3].loss).squeeze()
        return loss, d_logits / ids.numel(), saved

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

    def drafted(self, ids, generator, drafts=3, temperature=0.8):
        """Tokens after each of ids, `drafts` of them drafted by the table alone, without router and experts,
        and verified together -> (tokens [ids, drafts + 1], -1 behind the last, how many drafts were accepted)."""
        n = ids.numel()
        table = self.params["table"]
        text, guesses = [ids], []
        for _ in range(drafts):
            guesses.append(gc.embedding(table, text[-1], scale=self.scale) @ table.T)
            uniform = torch.rand(n, self.vocab, generator=generator, device="cuda")
            text.append(gc.sample(guesses[-1], uniform, temperature=temperature)[0].to(ids.dtype))
        # the model on all positions of all texts at once
        logits, _ = self.forward(torch.stack(text, 1).reshape(-1))
        accept = torch.rand(n, drafts, generator=generator, device="cuda")
        uniform = torch.rand(n, self.vocab, generator=generator, device="cuda")
        tokens, accepted, _ = gc.sample_verify(logits.view(n, drafts + 1, self.vocab), torch.stack(text[1:], 1).int(),
                                               accept, uniform, draft_logits=torch.stack(guesses, 1),
                                               temperature=temperature)
        return tokens, accepted


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
    tokens, accepted = model.drafted(ids[:8], g)
    print("drafted and verified", tokens.tolist(), "accepted", accepted.tolist())


if __name__ == "__main__":
    main()
