"""A tensor-parallel output head on P logical ranks: decode, policy gradient and
distillation, each from the collectives and the vocabulary-parallel operators.

    python examples/vocab_parallel_head.py [--ranks 4] [--rows 256] [--hidden 1024] [--vocab 32000]

The last layer's partial activations are summed and normalised over the ranks
(all_reduce_rmsnorm); every rank multiplies by its block of the head's columns,
so its logits are a [rows, shard] block of the row; log_probs, distill and
their gradients run over all blocks at once. The hidden gradient is the sum of
the ranks' (all_reduce).
"""
import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
import collective_communication_planner_gb300 as tccl  # noqa: E402


class Head:
    """A head of `vocab` columns cut over a group's ranks, and the buffers of a batch."""

    def __init__(self, group, hidden, vocab, rows, seed=0, dtype=torch.bfloat16):
        self.group, self.vocab, self.rows = group, vocab, rows
        self.shard = -(-vocab // group.nranks // 64) * 64  # whole 16-byte vectors
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.weights = [torch.randn(hidden, self.shard, generator=gen, device="cuda") / hidden ** 0.5
                        for _ in range(group.nranks)]
        self.gamma = torch.ones(hidden, dtype=dtype, device="cuda")
        self.normed = [torch.empty(rows, hidden, dtype=dtype, device="cuda") for _ in range(group.nranks)]

    def logits(self, partials):
        """Each rank's logits of the normalised sum of the ranks' partial activations."""
        self.group.all_reduce_rmsnorm(partials, self.normed, self.gamma)
        return [h @ w.to(h.dtype) for h, w in zip(self.normed, self.weights)]

    def hidden_gradient(self, grads):
        """The normalised activations' gradient, on every rank."""
        parts = [g @ w.to(g.dtype).t() for g, w in zip(grads, self.weights)]
        return self.group.all_reduce(parts)

    def descend(self, grads, rate):
        for w, h, g in zip(self.weights, self.normed, grads):
            w.sub_(rate * (h.t() @ g).float())


def floats(*shape):
    return torch.empty(*shape, dtype=torch.float32, device="cuda")


def decode(head, partials, top_k=8):
    """One token a row: the best alternatives and their log probabilities."""
    lp, ids = floats(head.rows, top_k), torch.empty(head.rows, top_k, dtype=torch.int64, device="cuda")
    head.group.log_probs(head.logits(partials), None, None, top_log_probs=lp, top_ids=ids, vocab=head.vocab)
    return ids, lp


def policy_step(head, partials, tokens, advantages, old, entropy_bonus=0.01, clip=0.2, rate=0.0):
    """A clipped policy-gradient step: log probabilities and entropies of the
    rows' tokens, the loss's gradients there, and from them the logits'. A
    token of -1 marks a prompt row. Returns (loss, log probabilities, hidden
    gradient)."""
    g, rows = head.group, head.rows
    logits = head.logits(partials)
    lp, ent, stats = floats(rows), floats(rows), floats(rows, 2)
    g.log_probs(logits, tokens, lp, ent, stats, vocab=head.vocab)
    scored = tokens >= 0
    n = scored.sum()
    ratio = torch.exp(lp - old)
    plain, clipped = ratio * advantages, ratio.clamp(1 - clip, 1 + clip) * advantages
    loss = -(torch.minimum(plain, clipped) + entropy_bonus * ent)[scored].sum() / n
    d_lp = torch.where(scored & (plain <= clipped), -plain / n, 0.0)
    d_ent = torch.where(scored, -entropy_bonus / n, 0.0)
    g.log_probs_backward(logits, tokens, stats, d_lp, logits, entropy=ent, d_entropy=d_ent, vocab=head.vocab)
    hidden = head.hidden_gradient(logits)[0]  # the logits' buffers hold their gradient now
    if rate:
        head.descend(logits, rate)
    return loss, lp, hidden


def distill_step(head, partials, ids, teacher, temperature=1.0, rate=0.0):
    """A student's step towards a teacher's entries: loss and gradient in one
    pass over the logits."""
    rows = head.rows
    logits = head.logits(partials)
    loss = floats(rows)
    weights = torch.full((rows,), 1.0 / rows, device="cuda")
    head.group.distill(logits, ids, teacher, loss, weights=weights, grads=logits, vocab=head.vocab,
                       temperature=temperature)
    hidden = head.hidden_gradient(logits)[0]
    if rate:
        head.descend(logits, rate)
    return loss.mean(), hidden


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--rows", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    with tccl.Group(a.ranks) as group:
        gen = torch.Generator(device="cuda")
        gen.manual_seed(1)
        partials = [torch.randn(a.rows, a.hidden, generator=gen, device="cuda").bfloat16() for _ in range(a.ranks)]
        teacher = Head(group, a.hidden, a.vocab, a.rows, seed=2)
        student = Head(group, a.hidden, a.vocab, a.rows, seed=3)
        ids, lp = decode(teacher, partials, top_k=min(32, a.vocab))
        print(f"teacher's best alternative of row 0: column {ids[0, 0].item()}, log probability {lp[0, 0].item():.3f}")
        losses = [distill_step(student, partials, ids, lp, rate=4.0)[0].item() for _ in range(a.steps)]
        print(f"distillation: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps")
        tokens = ids[:, 0].clone()
        tokens[::8] = -1
        advantages = torch.ones(a.rows, device="cuda")
        old, means = None, []
        for _ in range(a.steps):
            before = floats(a.rows)
            group.log_probs(student.logits(partials), tokens, before, vocab=a.vocab)
            old = before
            _, lp_now, _ = policy_step(student, partials, tokens, advantages, old, rate=4.0)
            means.append(lp_now[tokens >= 0].mean().item())
        print(f"policy gradient: mean log probability {means[0]:.3f} -> {means[-1]:.3f} in {a.steps} steps")
        assert group.query_error() == tccl.tcclSuccess
    return losses, means


if __name__ == "__main__":
    main()
