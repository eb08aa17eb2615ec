"""A policy-gradient step of a tied, vocabulary-sharded language model.

    python examples/policy_step.py [--steps 20] [--tokens 1024] [--vocab 16000] [--hidden 512] [--shards 4]
                                   [--optimizer sgd|adamw] [--state-bits 32|8]

The model is the two ends of one: tokens are looked up in the sharded table
(scaled, with dropout), the same table is the output head, and the logits of
every shard stay where the head's product leaves them.  A step

1. looks the tokens up (``vpce_embedding_dropout_forward``),
2. forms each shard's logits (a plain bf16 matrix product),
3. scores the sampled next tokens: log probability, entropy and the most
   likely alternatives (``vpce_logprob_forward``),
4. turns the gradient of ``-mean(advantage * logp + beta * entropy)`` into
   dlogits, in place (``vpce_logprob_backward``),
5. multiplies it back to the hidden states and the table, and adds the lookup's
   own gradient to the table's (``vpce_embedding_dropout_backward``).

``--steps`` of plain gradient descent on tokens with a fixed rule (the
advantage is positive where the sampled token follows it) raise the rule's
probability; the mask's offset is the step number.  With ``--optimizer adamw``
the gradients are clipped to norm 1 (``vpce_grad_norm``) and one
``vpce_adamw_step`` updates the fp32 shards, their states and the bf16 table.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

from vocab_sharded_lm_gb300 import vpce  # noqa: E402


def policy_step(table, grads, ids, targets, advantage, vocab_start, *, beta=0.01, p=0.1, rng=None, padding_id=None,
                top=4, temperature=1.0):
    """One forward and backward.  ``table``: bf16 shards [w_i, h]; ``grads``:
    fp32 shards, overwritten with d objective / d table; rows of ``targets`` equal
    to -100 do not count.  Returns (objective, scores)."""
    h = table[0].shape[1]
    scale = math.sqrt(h)
    hidden = vpce.vpce_embedding_dropout_forward(table, ids, vocab_start, scale=scale, p=p, rng=rng,
                                                 padding_id=padding_id)
    logits = [hidden @ w.T for w in table]
    scores = vpce.vpce_logprob_forward(logits, targets, vocab_start, top=top, temperature=temperature)
    valid = (targets != -100).float()
    n = valid.sum().clamp(min=1)
    objective = -((advantage * scores.logp + beta * scores.entropy) * valid).sum() / n
    dlogits = vpce.vpce_logprob_backward(logits, targets, scores.stats, vocab_start, temperature=temperature,
                                         grad_logp=-advantage * valid / n, grad_entropy=-beta * valid / n,
                                         grad_shards=logits)
    dhidden = torch.zeros(hidden.shape, dtype=torch.float32, device=hidden.device)
    for d, w, g in zip(dlogits, table, grads):
        dhidden += (d @ w).float()
        g.copy_(d.T @ hidden)
    vpce.vpce_embedding_dropout_backward(dhidden, ids, grads, vocab_start, scale=scale, p=p, rng=rng,
                                         padding_id=padding_id, accumulate=True)
    return objective, scores


def main(argv=None) -> list[float]:
    ap = argparse.ArgumentParser(description="policy-gradient steps of a tied, vocabulary-sharded model")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=16000)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--shards", type=int, default=4)
    ap.add_argument("--lr", type=float, default=None, help="2 for sgd, 0.01 for adamw")
    ap.add_argument("--optimizer", choices=("sgd", "adamw"), default="sgd")
    ap.add_argument("--state-bits", type=int, choices=(32, 8), default=32)
    a = ap.parse_args(argv)
    lr = a.lr if a.lr is not None else 2.0 if a.optimizer == "sgd" else 0.01
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    V, h, t = a.vocab, a.hidden, a.shards
    vs = [i * V // t for i in range(t + 1)]
    master = [torch.randn(vs[i + 1] - vs[i], h, device="cuda", generator=gen) / h for i in range(t)]
    grads = [torch.empty_like(w) for w in master]
    rng = torch.tensor([1234, 0], dtype=torch.int64, device="cuda")
    ids = torch.randint(0, V, (a.tokens,), device="cuda", generator=gen)
    targets = (ids * 7 + 3) % V                      # the rule
    targets[:: 16] = -100                            # the prompt's tokens
    advantage = torch.ones(a.tokens, device="cuda")
    if a.optimizer == "adamw":
        table = [w.to(torch.bfloat16) for w in master]
        plan = vpce.vpce_adamw_plan(master, grads, copies=table, weight_decay=0.0, state_bits=a.state_bits)
        words = torch.tensor([4321, 0], dtype=torch.int64, device="cuda")
        number = torch.zeros(1, dtype=torch.int64, device="cuda")
    history = []
    for step in range(a.steps):
        rng[1] = step
        if a.optimizer == "sgd":
            table = [w.to(torch.bfloat16) for w in master]
        objective, scores = policy_step(table, grads, ids, targets, advantage, vs, rng=rng)
        if a.optimizer == "sgd":
            for w, g in zip(master, grads):
                w -= lr * g
        else:
            words[1] = step
            _, scale = vpce.vpce_grad_norm(plan, 1.0)
            number += scale != 0     # a step that is skipped is not counted, and the host does not look
            vpce.vpce_adamw_step(plan, number, lr=lr, grad_scale=scale, rng=words)
        live = targets != -100
        logp, entropy = scores.logp[live].mean().item(), scores.entropy[live].mean().item()
        hit = (scores.top_ids[:, 0] == targets)[live].float().mean().item()
        history.append(logp)
        print(f"step {step:3d}  objective {objective.item():8.4f}  logp {logp:8.4f}  entropy {entropy:7.4f}  "
              f"greedy follows the rule {100 * hit:5.1f}%")
    return history


if __name__ == "__main__":
    main()
