"""Routing of tokens to experts from its definition: the dispatch plan and the balance loss with its gradient, in
Python loops and float64. Test infrastructure, sharing nothing with the HIP path."""

from __future__ import annotations

import numpy as np


def plan(idx: np.ndarray, groups: int, pad: int, cap: int):
    """(counts, row_off, src, pos) of idx [tokens, topk]; entries outside [0, groups) are dropped. src is -1 for padding
    and -2 behind the last group."""
    counts = [0] * groups
    for e in idx.flatten():
        if 0 <= e < groups:
            counts[e] += 1
    off = [0]
    for c in counts:
        off.append(off[-1] + -(-c // pad) * pad)
    src = np.full(cap, -1, np.int32)
    src[off[-1]:] = -2
    pos = np.full(idx.shape, -1, np.int32)
    free = list(off[:-1])
    for t in range(idx.shape[0]):
        for j in range(idx.shape[1]):
            e = idx[t, j]
            if 0 <= e < groups:
                src[free[e]] = t
                pos[t, j] = free[e]
                free[e] += 1
    return np.array(counts, np.int32), np.array(off, np.int32), src, pos


def scores(logits: np.ndarray, score: str):
    """(p, 1 - sigmoid or None) of float64 logits; a row of -inf gives p = 0."""
    if score == "softmax":
        top = logits.max(1, keepdims=True)
        w = np.exp(logits - np.where(np.isfinite(top), top, 0.0))
        opened = None
    else:
        w = np.where(logits >= 0, 1 / (1 + np.exp(-np.abs(logits))), np.exp(-np.abs(logits)) / (1 + np.exp(-np.abs(logits))))
        opened = np.where(logits >= 0, np.exp(-np.abs(logits)), 1.0) / (1 + np.exp(-np.abs(logits)))
    total = w.sum(1, keepdims=True)
    return np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0), opened


def balance(logits: np.ndarray, idx: np.ndarray, coef: float, score: str, seq_off):
    """(loss, counts [S, experts], real [S]) of float64 logits [tokens, experts]."""
    experts, topk = logits.shape[1], idx.shape[1]
    seqs = len(seq_off) - 1
    counts, real, loss = np.zeros((seqs, experts), np.int64), np.zeros(seqs, np.int64), 0.0
    p, _ = scores(logits, score)
    for s in range(seqs):
        mean = np.zeros(experts)
        for t in range(seq_off[s], seq_off[s + 1]):
            ok = [e for e in idx[t] if 0 <= e < experts]
            if ok:
                real[s] += 1
                mean += p[t]
                for e in ok:
                    counts[s, e] += 1
        if real[s]:
            loss += (counts[s] * experts / (topk * real[s]) * mean / real[s]).sum()
    return coef / seqs * loss, counts, real


def balance_grad(dloss: float, logits: np.ndarray, idx: np.ndarray, coef: float, score: str, seq_off):
    """d loss / d logits * dloss, counts held constant."""
    experts, topk = logits.shape[1], idx.shape[1]
    seqs = len(seq_off) - 1
    _, counts, real = balance(logits, idx, coef, score, seq_off)
    p, opened = scores(logits, score)
    g = np.zeros_like(logits)
    for s in range(seqs):
        for t in range(seq_off[s], seq_off[s + 1]):
            if any(0 <= e < experts for e in idx[t]):
                dp = dloss * coef / seqs * counts[s] * experts / (topk * real[s] ** 2)
                g[t] = p[t] * (dp - (p[t] * dp).sum())
                if opened is not None:
                    g[t] *= opened[t]
    return g
