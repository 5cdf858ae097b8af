"""Inputs of the tree operators' tests."""
import numpy as np
import torch

DEV = "cuda"


def random_parents(rng, B, T, unused=0.0, deep=0.3):
    """Random trees: a node hangs under its predecessor with probability ``deep``, else under any
    used node before it; nodes are unused with probability ``unused``."""
    par = np.full((B, T), -2, np.int32)
    par[:, 0] = -1
    for b in range(B):
        used = [0]
        for i in range(1, T):
            if rng.random() < unused:
                continue
            par[b, i] = used[-1] if rng.random() < deep else used[int(rng.integers(len(used)))]
            used.append(i)
    return par


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).to(DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def numpy64(t):
    return t.detach().double().cpu().numpy()
