"""Train a soft codebook by gradient: every point is rebuilt from the k codes its router chooses.

    logits  = X R^T                      a router's score of each code
    idx, w  = kmassign_route(logits)     k codes a point, sigmoid weights, a bias that balances use
    Y       = kmassign_lookup(C, idx, w) the weighted sum of the chosen codes
    loss    = |Y - X|^2 / N

and back: ``kmassign_lookup_grad`` gives the gradients of the codes and of the weights,
``kmassign_route_grad`` that of the logits, ``kmassign_clip`` bounds them all together, and
``kmassign_lists`` counts how often each code was used, which moves the balance bias.

    python examples/soft_codes.py [steps]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import means_nearest_centroid_gb300 as km  # noqa: E402


def train(N=8192, D=64, K=256, k=4, steps=60, rate=2.0, seed=0, device="cuda"):
    """Losses per step, and the share of codes in use at the first and the last step."""
    gen = torch.Generator(device="cpu").manual_seed(seed)
    centers = torch.randn(K // 4, D, generator=gen)
    label = torch.randint(0, K // 4, (N,), generator=gen)
    X = (centers[label] + 0.1 * torch.randn(N, D, generator=gen)).to(device)
    codes = (0.1 * torch.randn(K, D, generator=gen)).to(device)
    router = (0.1 * torch.randn(K, D, generator=gen)).to(device)
    bias = torch.zeros(K, device=device)
    losses, used = [], []
    for _ in range(steps):
        logits = X @ router.T
        idx, w = km.kmassign_route(logits, k, score="sigmoid", bias=bias, scale=float(k))
        Y = km.kmassign_lookup(codes, idx, weights=w)
        diff = Y - X
        dY = diff * (2.0 / N)
        dcodes, dw = km.kmassign_lookup_grad(dY, idx, K, weights=w, table=codes)
        dlogits = km.kmassign_route_grad(logits, idx, dw, score="sigmoid", scale=float(k))
        drouter = dlogits.T @ X
        km.kmassign_clip([dcodes, drouter], 1.0)
        codes -= rate * dcodes
        router -= rate * drouter
        _, offsets = km.kmassign_lists(idx, K)
        counts = (offsets[1:] - offsets[:-1]).float()
        bias += 0.001 * torch.sign(counts.mean() - counts)
        losses.append(diff.square().sum().item() / N)
        used.append((counts > 0).float().mean().item())
    return losses, used


if __name__ == "__main__":
    losses, used = train(steps=int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    for s in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {s:4d}  loss {losses[s]:8.4f}  codes in use {100 * used[s]:5.1f}%")
    print(f"last       loss {losses[-1]:8.4f}  codes in use {100 * used[-1]:5.1f}%")
