"""A token model trained and sampled with this library's operators.

    python examples/token_model.py [--steps 60]

Token rows come from the embedding forward (one row a token) and go through one
block, x_out = x + gate * post(mlp(x)), y = pre(x_out); the logits y @ head.T
are trained on a teacher's top logits and the tokens that follow, and the
gradient goes back through the block norms into the embedding rows, which
sgb's backward updates in place.  Before that the model is trained on the tokens
that follow alone, its embedding rows under dropout, with the loss and gradients
of the head's product taken in one call.  Then tokens are generated under a
grammar mask with a presence penalty, also with the last norm's output in 8 bits.
The other matrix products are torch's.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_gradient_backward_amd as sgb  # noqa: E402
from sparse_gradient_backward_amd import lm  # noqa: E402


class TokenModel:
    def __init__(self, vocab=2000, D=256, hidden=512, rows=512, K=16, seed=0):
        self.V, self.D, self.rows, self.K = vocab, D, rows, K
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*s, std):
            return torch.randn(*s, generator=g, device="cuda") * std

        self.rand = rand
        self.table = rand(vocab, D, std=1.0)                 # the embedding rows
        self.w1, self.w2 = rand(hidden, D, std=D ** -0.5), rand(D, hidden, std=hidden ** -0.5)
        self.head = rand(vocab, D, std=D ** -0.5)
        self.gate = torch.ones(1, D, device="cuda")          # one row for all tokens
        ones = torch.ones(2, D, device="cuda")
        self.norm = lm.BlockNorm(D, post="rms", pre="rms", post_weight=ones[0], pre_weight=ones[1])
        self.distill = lm.TopkDistill(vocab, K, kd_weight=0.7, ce_weight=0.3)
        self.penalty = lm.LogitsPenalty(vocab)
        self.dropout, self.ce = lm.Dropout(0.1), lm.VocabCrossEntropy(D, vocab)
        self.block = lm.BlockNorm(D, post="rms", pre="none", post_weight=ones[0])
        self.quant = lm.QuantNorm(D, weight=ones[1], form="int8")
        self.plan = sgb.Plan([0, vocab], [0, D], "none")
        new = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.x, self.x_out, self.y = new(rows, D), new(rows, D), new(rows, D)
        self.dx, self.dh = new(rows, D), new(rows, D)
        self.stats, self.loss = new(rows, 4), new(rows)
        self.d_logits = new(rows, vocab)
        self.d_gate, self.d_norm = new(1, D), new(2, D)
        self.dy, self.d_head = new(rows, D), new(vocab, D)
        self.codes = torch.empty(rows, D, dtype=torch.int8, device="cuda")
        self.scales = new(rows, 1)
        self.none = torch.zeros(rows, D, device="cuda")      # nothing reads x_out but the norm
        self.ws = (self.plan.workspace(rows, 0), self.norm.workspace(rows),
                   self.distill.workspace(rows), self.penalty.workspace(rows),
                   self.ce.workspace(rows, torch.float32))

    def block_output(self, tokens, drop=None):
        """x and h of `rows` or fewer tokens, each alone; drop: seed and step of
        the embedding rows' dropout."""
        n = tokens.numel()
        self.plan.forward(tokens, None, 0, None, self.table, self.x[:n], self.ws[0])
        if drop is not None:
            self.dropout.forward(self.x[:n], self.x[:n], *drop)
        self.a = torch.tanh(self.x[:n] @ self.w1.t())
        self.h = self.a @ self.w2.t()
        return n

    def hidden(self, tokens, drop=None):
        """What the head is multiplied with."""
        n = self.block_output(tokens, drop)
        self.norm.forward(self.x[:n], self.h, self.x_out[:n], self.y[:n], gate=self.gate,
                          rows_per_gate=n, stats=self.stats[:n])
        return self.y[:n]

    def logits(self, tokens):
        return self.hidden(tokens) @ self.head.t()

    def logits_of_codes(self, tokens):
        """The same with the last norm's output in 8 bits, a scale a row."""
        n = self.block_output(tokens)
        self.block.forward(self.x[:n], self.h, self.x_out[:n], gate=self.gate, rows_per_gate=n)
        self.quant.forward(self.x_out[:n], self.codes[:n], self.scales[:n])
        return self.codes[:n].float() @ self.head.t() * self.scales[:n]

    def step(self, tokens, labels, ids, values, lse, lr):
        """One training step on `rows` tokens; returns the mean loss."""
        logits = self.logits(tokens)
        self.distill.loss_grad(logits, ids, values, self.loss, self.d_logits,
                               grad_scale=1.0 / self.rows, teacher_lse=lse, labels=labels,
                               workspace=self.ws[2])
        self.update(tokens, self.d_logits @ self.head, self.d_logits.t() @ self.y, lr)
        return self.loss.mean()

    def step_on_labels(self, tokens, labels, lr, step, seed=0):
        """One training step on the tokens that follow; returns the mean loss."""
        y = self.hidden(tokens, (seed, step))
        self.ce.loss_grad(y, self.head, labels, self.loss, self.dy, self.d_head,
                          grad_scale=1.0 / self.rows, workspace=self.ws[4])
        self.update(tokens, self.dy, self.d_head, lr, (seed, step))
        return self.loss.mean()

    def update(self, tokens, dy, d_head, lr, drop=None):
        """Back from the gradients of y and of the head; every parameter moves."""
        self.norm.backward(self.none, dy, self.x_out, self.h, self.stats, self.dx, self.dh,
                           gate=self.gate, rows_per_gate=self.rows, d_gate=self.d_gate,
                           d_post_weight=self.d_norm[0], d_pre_weight=self.d_norm[1],
                           workspace=self.ws[1])
        da = (self.dh @ self.w2) * (1 - self.a * self.a)
        d_w2, d_w1 = self.dh.t() @ self.a, da.t() @ self.x
        dx = self.dx + da @ self.w1
        if drop is not None:
            self.dropout.backward(dx, dx, *drop)
        for w, d in ((self.w1, d_w1), (self.w2, d_w2), (self.head, d_head), (self.gate, self.d_gate),
                     (self.norm.post_weight, self.d_norm[0]), (self.norm.pre_weight, self.d_norm[1])):
            w.sub_(d, alpha=lr)
        self.plan.backward(dx, tokens, None, 0, None, "sgd", weights=self.table, lr=lr,
                           workspace=self.ws[0])

    def generate(self, first, count, mask, codes=False):
        """`count` tokens after each of `first`, the likeliest that the grammar
        row `mask` (packed bits) allows, with a heavy presence penalty; codes:
        from logits of 8-bit codes."""
        n = first.numel()
        seq = torch.zeros(n, count + 1, dtype=torch.int32, device="cuda")
        seq[:, 0] = first
        prompt = torch.ones(n, dtype=torch.int32, device="cuda")
        which, heavy = torch.zeros_like(prompt), torch.full((n,), 1e4, device="cuda")
        for i in range(1, count + 1):
            logits = (self.logits_of_codes if codes else self.logits)(seq[:, i - 1].long())
            self.penalty.apply(logits, logits, tokens=seq, prompt_lens=prompt,
                               lens=torch.full_like(prompt, i), presence=heavy, mask=mask,
                               mask_index=which, workspace=self.ws[3])
            seq[:, i] = logits.argmax(1)
        return seq


def train(steps=60, seed=0, on_labels=0):
    """Returns the model and its losses, after `on_labels` steps on the following
    tokens alone.  The teacher is a fixed table of next-token logits."""
    m = TokenModel(seed=seed)
    teacher = m.rand(m.V, m.V, std=2.0)
    values, ids = teacher.topk(m.K, dim=1)
    lse = torch.logsumexp(teacher.double(), 1).float()
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    losses = []
    for i in range(on_labels + steps):
        # token frequencies fall off as in text: rows repeat within a batch
        u = torch.rand(m.rows, generator=g, device="cuda")
        tokens = (m.V ** u - 1).long().clamp_(max=m.V - 1)
        labels = ids[tokens, torch.randint(0, m.K, (m.rows,), generator=g, device="cuda")]
        if i < on_labels:
            m.step_on_labels(tokens, labels, 2.0, i, seed)
        else:
            losses.append(m.step(tokens, labels, ids[tokens], values[tokens], lse[tokens], lr=2.0))
    return m, torch.stack(losses).tolist()


def even_tokens(vocab):
    """A grammar row that allows the even tokens."""
    return torch.full((1, (vocab + 31) // 32), 0x55555555, dtype=torch.int32, device="cuda")


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--on-labels", type=int, default=20)
    a = ap.parse_args()
    m, losses = train(a.steps, on_labels=a.on_labels)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps")
    for codes in (False, True):
        print(m.generate(torch.arange(4, device="cuda").int(), 8, even_tokens(m.V), codes).tolist())


if __name__ == "__main__":
    main()
