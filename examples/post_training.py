"""Training on calibrated, ranked rewards: the fit, the soft ranks and the objectives together.

A small routed language model answers prompts in groups.  Each answer has a raw reward-model score;
past outcomes calibrate the scores (a non-decreasing fit), the calibrated rewards' soft ranks within
a group are the answers' advantages, and the model takes a clipped policy step on them with the
router's balance loss beside it.  The best and the worst answer of each group then make a pair for a
preference step.  Synthetic data; needs a CUDA device.

    python examples/post_training.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import convex_hull_pava_gb300 as chp
from convex_hull_pava_gb300 import objectives as obj
from convex_hull_pava_gb300.soft_rank import soft_rank

VOCABULARY, WIDTH, EXPERTS, TOP_K = 4096, 64, 16, 2
PROMPTS, GROUP, LENGTH = 8, 8, 24   # answers to a prompt; tokens of an answer


class RoutedModel(torch.nn.Module):
    """Token logits from the previous token, through the gated experts that the router chooses."""

    def __init__(self):
        super().__init__()
        self.embed = torch.nn.Embedding(VOCABULARY, WIDTH)
        self.router = torch.nn.Linear(WIDTH, EXPERTS)
        self.experts = torch.nn.Parameter(torch.randn(EXPERTS, WIDTH, WIDTH) / WIDTH ** 0.5)
        self.head = torch.nn.Linear(WIDTH, VOCABULARY)

    def forward(self, tokens, real):
        """``(logits, balance loss, tokens of each expert)``; ``real`` is false at padding."""
        h = self.embed(tokens)
        balance, gates, counts, chosen = obj.balance_loss(self.router(h), TOP_K, real, renormalize=True)
        each = torch.einsum("tw,ewv->tev", h, self.experts)
        at = chosen.clamp(min=0).long()[..., None].expand(-1, -1, WIDTH)
        h = h + (gates[..., None] * torch.tanh(each.gather(1, at))).sum(1)
        return self.head(h), balance, counts


def calibrated(scores, past_scores, past_outcomes):
    """The non-decreasing fit of past outcomes over their scores, read at new scores."""
    at, order = torch.sort(past_scores)
    fit = chp.isotonic(past_outcomes[order].contiguous())
    return fit[torch.searchsorted(at, scores).clamp(max=len(at) - 1)]


def advantages(rewards):
    """Centred soft ranks of the rewards within each group."""
    ranks = soft_rank(rewards, eps=0.1)
    return (ranks - ranks.mean(1, keepdim=True)) / rewards.shape[1]


def main(steps=20):
    torch.manual_seed(0)
    torch.set_default_device("cuda")
    model = RoutedModel()
    optimizer = torch.optim.Adam(model.parameters(), lr=3e-3)
    past = torch.randn(4000)
    outcomes = (torch.rand(4000) < torch.sigmoid(2 * past)).float()
    answers = PROMPTS * GROUP
    history = []
    for step in range(steps):
        tokens = torch.randint(0, VOCABULARY, (answers, LENGTH + 1))
        sizes = torch.randint(LENGTH // 2, LENGTH + 1, (answers,))
        real = (torch.arange(LENGTH) < sizes[:, None]).reshape(-1)
        inputs = tokens[:, :-1].reshape(-1)
        labels = torch.where(real, tokens[:, 1:].reshape(-1), -100)
        # synthetic scores: the share of even tokens in an answer
        scores = ((tokens[:, 1:] % 2 == 0).float().mean(1) - 0.5) * 8
        rewards = calibrated(scores, past, outcomes).view(PROMPTS, GROUP)
        adv = advantages(rewards).reshape(-1, 1).expand(-1, LENGTH).reshape(-1).contiguous()

        with torch.no_grad():   # the policy that drew the answers, and the reference (here the same)
            old = obj.token_logp(model(inputs, real)[0], labels)
        logits, balance, counts = model(inputs, real)
        loss, stats, _ = obj.policy_loss(logits, labels, old, adv, old, kl_coef=0.05)
        optimizer.zero_grad()
        (loss + 0.01 * balance).backward()
        optimizer.step()

        # the best and the worst answer of each group, token rows laid end to end
        pair = torch.stack([rewards.argmax(1), rewards.argmin(1)], 1) + GROUP * torch.arange(PROMPTS)[:, None]
        rows = (pair.reshape(-1, 1) * LENGTH + torch.arange(LENGTH)).reshape(-1)
        logits, _, _ = model(inputs[rows], real[rows])
        offsets = LENGTH * torch.arange(2 * PROMPTS + 1)
        preference, margins, _ = obj.preference_loss(logits, labels[rows], offsets, old[rows].contiguous(), beta=0.1)
        optimizer.zero_grad()
        preference.backward()
        optimizer.step()
        history.append((loss.item(), balance.item(), preference.item()))
        if step % 5 == 0 or step == steps - 1:
            print("step %2d  policy %+.4f  clipped %.2f  balance %.3f  preference %.4f  largest expert %d of %d"
                  % (step, loss.item(), stats[2].item(), balance.item(), preference.item(), int(counts.max()),
                     int(real.sum()) * TOP_K))
    torch.set_default_device(None)
    return history


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
