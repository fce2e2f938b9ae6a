"""The per-token FFN of a RankMixer block in 8 bits: serving and training.

A block's input is token-mixed and normalised, then every token's own FFN runs on 8-bit operands
(api.Fp8PFFN).  Training keeps the FFN's activations in 8 bits between forward and backward; the
weights stay in float32 and are rounded to 8 bits after every update.  The student FFN learns the
outputs of a fixed teacher.

    python examples/pffn_8bit.py [--B 512] [--T 8] [--D 256] [--k 4] [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from rankmixer_feature_interaction_gb300 import synth  # noqa: E402
from rankmixer_feature_interaction_gb300.api import Fp8PFFN, fp8_quantize_weight, fp8_sync_status, token_mix  # noqa: E402


def block_input(X: torch.Tensor) -> torch.Tensor:
    """S = LN(TokenMixing(X) + X) without an affine, bf16."""
    Y = (token_mix(X) + X).float()
    return torch.nn.functional.layer_norm(Y, (Y.shape[-1],)).to(torch.bfloat16)


def train(B: int, T: int, D: int, k: int, steps: int, lr: float = 1e-3, seed: int = 1) -> dict:
    teacher, student = (synth.make_stack(T, D, k, 1, seed + i, "f32", "cuda")[0] for i in range(2))
    target = Fp8PFFN(teacher["W1"], teacher["b1"], teacher["W2"], teacher["b2"])
    W = {n: student[n].clone() for n in ("W1", "b1", "W2", "b2")}
    moments = {n: (torch.zeros_like(w), torch.zeros_like(w)) for n, w in W.items()}
    losses = []
    for step in range(steps):
        S = block_input(synth.make_input(B, T, D, seed + 10 + step, "bf16", "cuda"))
        ffn = Fp8PFFN(fp8_quantize_weight(W["W1"]), W["b1"], fp8_quantize_weight(W["W2"]), W["b2"])
        V, kept = ffn.forward_train(S, "f32")
        diff = V - target.forward(S, "f32")
        losses.append(diff.square().mean())
        _, grads = ffn.backward(diff * (2.0 / diff.numel()), kept, with_dX=False)
        for n, w in W.items():                       # Adam on the float32 weights
            m, v = moments[n]
            g = grads["d" + n]
            m.lerp_(g, 0.1)
            v.lerp_(g * g, 0.01)
            w -= lr * (m / (1 - 0.9 ** (step + 1))) / ((v / (1 - 0.99 ** (step + 1))).sqrt() + 1e-12)
    kept_bytes = sum(q.nbytes for q in kept.values())
    assert fp8_sync_status() == 0
    return {"first": float(losses[0]), "last": float(torch.stack(losses[-5:]).mean()), "kept_bytes": kept_bytes,
            "bytes_in_16_bits": 2 * B * T * D * (1 + 2 * k)}


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("B", 512), ("T", 8), ("D", 256), ("k", 4), ("steps", 60)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args(argv)
    r = train(a.B, a.T, a.D, a.k, a.steps)
    print(f"loss {r['first']:.4f} -> {r['last']:.4f} in {a.steps} steps; activations kept: {r['kept_bytes'] / 1e6:.1f} MB "
          f"in 8 bits ({r['bytes_in_16_bits'] / 1e6:.1f} MB in 16)")
    return 0


if __name__ == "__main__":
    sys.exit(main())
