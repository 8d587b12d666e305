"""The example of a tensor-parallel head: it learns, and its steps agree with
the same steps in 64-bit torch on the whole matrices."""
import importlib.util
from pathlib import Path

import pytest
import torch

import collective_communication_planner_gb300 as tccl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = Path(__file__).resolve().parents[1] / "examples" / "vocab_parallel_head.py"
    spec = importlib.util.spec_from_file_location("vocab_parallel_head", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_the_example_learns(example, capsys):
    losses, means = example.main(["--ranks", "3", "--rows", "64", "--hidden", "256", "--vocab", "5000", "--steps", "10"])
    assert losses[-1] < losses[0] and means[-1] > means[0]
    assert "policy gradient" in capsys.readouterr().out


def test_steps_agree_with_torch(example):
    """Logits in bf16 are the inputs of both sides; the gradients differ by the
    bf16 rounding of each element (2^-8) and of the product's result."""
    rows, hidden, vocab, p = 48, 128, 1000, 4
    torch.manual_seed(0)
    with tccl.Group(p) as group:
        head = example.Head(group, hidden, vocab, rows)
        partials = [torch.randn(rows, hidden, device="cuda").bfloat16() for _ in range(p)]
        logits = [m.clone() for m in head.logits(partials)]
        whole = torch.cat(logits, 1)[:, :vocab].double().requires_grad_()
        logp = torch.log_softmax(whole, 1)
        ids, lp = example.decode(head, partials, top_k=5)
        best = torch.sort(whole.detach(), dim=1, descending=True, stable=True).indices[:, :5]
        assert torch.equal(ids, best)
        assert (lp.double() - logp.gather(1, best)).abs().max() < 1e-5
        tokens = torch.randint(0, vocab, (rows,), device="cuda")
        tokens[5] = -1
        adv, old = torch.randn(rows, device="cuda"), logp.detach().gather(1, tokens.clamp_min(0)[:, None])[:, 0].float()
        loss, got, hid = example.policy_step(head, partials, tokens, adv, old)
        on = tokens >= 0
        pick = logp.gather(1, tokens.clamp_min(0)[:, None])[:, 0]
        ratio = torch.exp(pick - old.double())
        ent = -(logp.exp() * logp).sum(1)
        want = -(torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv) + 0.01 * ent)[on].sum() / on.sum()
        want.backward()
        assert abs(loss.item() - want.item()) < 1e-4
        weight = torch.cat([w.bfloat16().double() for w in head.weights], 1)[:, :vocab]
        expect = whole.grad @ weight.t()
        # each element of the gradient and each rank's product rounded to bf16, then their sum
        scale = whole.grad.abs() @ weight.abs().t()
        assert ((hid.double() - expect).abs() <= 2.0 ** -8 * scale + 2.0 ** -7 * p * expect.abs() + 2.0 ** -7 * scale).all()
