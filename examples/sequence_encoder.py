#!/usr/bin/env python3
"""A next-item model from item ids to the loss and back, and its serving step, on the package's operators.

One causal self-attention block over each user's history (the shape of the paper's Section III-E recommenders), with
the item table shared between the lookup and the full-vocabulary loss:

  training   ids of all users packed one after another (no padding) -> embedding (scaled rows of the item table, and
             of a position table) -> layer_norm -> packed_attention -> layer_norm -> two-layer perceptron ->
             layer_norm -> cut_bce's forward and backward -> the encoder's backward; the lookup's gradient is added
             to the rows of the loss's dE that it touches (embedding_backward with dtable)
  serving    one new item a user: its key and value go into the cache, cached_attention reads it, topk ranks the items

Run on a GPU:  python examples/sequence_encoder.py [--users 64 --items 20000 --steps 20]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from vocabulary_label_bce_amd import ops  # noqa: E402


class Cache:
    """Keys and values [users, capacity, kv heads, head_dim] and how many rows each user has filled (on the device);
    `tokens` is the same count on the host, one more for every call, so that a full cache is known without asking."""

    def __init__(self, keys, values, lens):
        self.keys, self.values, self.lens, self.tokens = keys, values, lens, 0


class Encoder:
    """Parameters and the block. dim = heads * head_dim; kv_heads <= heads share keys and values."""

    def __init__(self, items, dim=128, heads=2, kv_heads=2, max_len=200, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device=device) * std).to(dtype)

        self.dim, self.heads, self.kv_heads, self.head_dim = dim, heads, kv_heads, dim // heads
        self.scale = math.sqrt(dim)
        self.items = normal(items, dim, std=0.02)           # shared with the loss
        width = dim + 2 * kv_heads * self.head_dim
        self.p = dict(positions=normal(max_len, dim, std=0.02), qkv=normal(dim, width, std=dim ** -0.5),
                      out=normal(dim, dim, std=dim ** -0.5), up=normal(dim, 4 * dim, std=dim ** -0.5),
                      down=normal(4 * dim, dim, std=(4 * dim) ** -0.5))
        for n in ("norm1", "norm2", "norm3"):
            self.p[n + ".w"] = torch.ones(dim, device=device)
            self.p[n + ".b"] = torch.zeros(dim, device=device)
        for t in self.p.values():
            t.requires_grad_()

    def _norm(self, x, n):
        return ops.layer_norm(x, self.p[n + ".w"], self.p[n + ".b"])

    def _qkv(self, x):
        """q, k, v as column ranges of one projection."""
        h, kh, dh = self.heads, self.kv_heads, self.head_dim
        y = self._norm(x, "norm1") @ self.p["qkv"]
        return (y[:, : h * dh].unflatten(1, (h, dh)), y[:, h * dh : (h + kh) * dh].unflatten(1, (kh, dh)),
                y[:, (h + kh) * dh :].unflatten(1, (kh, dh)))

    def _rest(self, x, attended):
        x = x + attended.flatten(1) @ self.p["out"]
        y = torch.relu(self._norm(x, "norm2") @ self.p["up"]) @ self.p["down"]
        return self._norm(x + y, "norm3")

    def hidden(self, x, places, cu):
        """Hidden states [rows, dim] of packed rows: x the scaled item rows, places each row's position."""
        x = x + ops.embedding(places, self.p["positions"])
        return self._rest(x, ops.packed_attention(*self._qkv(x), cu))

    def train_step(self, ids, places, cu, row_offsets, item_ids, lr=0.05):
        """One step of gradient descent on the loss of predicting each row's positives; returns the loss."""
        x = ops.embedding_forward(ids, self.items, self.scale).requires_grad_()
        hidden = self.hidden(x, places, cu)
        with torch.no_grad():
            w = ops.Workspace(hidden, self.items, item_ids)
            mask = torch.ones(hidden.shape[0], dtype=torch.uint8, device=hidden.device)
            H = hidden.detach()
            loss = w.forward(H, self.items, row_offsets, item_ids, mask)
            dH, dE = w.backward(H, self.items, row_offsets, item_ids, mask, reuse=True)
        hidden.backward(dH)
        with torch.no_grad():
            ops.embedding_backward(x.grad, ids, self.items.shape[0], self.scale, dtable=dE)
            V = self.items.shape[0]  # the loss averages over rows and items: the steps are scaled back by the items
            self.items -= lr * V * dE
            for t in self.p.values():
                t -= lr * V * t.grad
                t.grad = None
        return loss

    # ---- serving ----
    def new_cache(self, users, capacity):
        shape = (users, capacity, self.kv_heads, self.head_dim)
        return Cache(torch.zeros(shape, dtype=self.items.dtype, device=self.items.device),
                     torch.zeros(shape, dtype=self.items.dtype, device=self.items.device),
                     torch.zeros(users, dtype=torch.int32, device=self.items.device))

    @torch.no_grad()
    def serve(self, ids, cache, k=8):
        """Appends one item a user to the cache; returns (hidden [users, dim], the k best next items)."""
        keys, values, lens = cache.keys, cache.values, cache.lens
        if cache.tokens >= min(keys.shape[1], self.p["positions"].shape[0]):
            raise ValueError("the cache is full")
        cache.tokens += 1
        x = ops.embedding(ids, self.items, self.scale) + ops.embedding(lens, self.p["positions"])
        q, kn, vn = self._qkv(x)
        user = torch.arange(ids.numel(), device=ids.device)
        keys[user, lens.long()] = kn
        values[user, lens.long()] = vn
        lens += 1
        hidden = self._rest(x, ops.cached_attention(q, keys, values, lens))
        return hidden, ops.topk(hidden, self.items, k=k)[1]


def histories(users, items, lo, hi, seed, device="cuda"):
    """Packed synthetic histories: (ids, places, cu, row_offsets, item_ids); each row's positive is the next item,
    which follows the present one by a fixed step, so that there is something to learn."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(lo, hi + 1, (users,), generator=g)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    first = torch.randint(0, items, (users,), generator=g)
    rows = int(cu[-1])
    seq = torch.repeat_interleave(torch.arange(users), lens)
    places = torch.arange(rows) - cu[seq]
    ids = (first[seq] + 7 * places) % items
    nxt = (ids + 7) % items
    as_int = [t.to(torch.int32).to(device) for t in (ids, places, cu, torch.arange(rows + 1), nxt)]
    return as_int, lens


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--users", type=int, default=64)
    ap.add_argument("--items", type=int, default=20_000)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    model = Encoder(a.items)
    batch, lens = histories(a.users, a.items, 20, 200, seed=1)
    for i in range(a.steps):
        loss = model.train_step(*batch)
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i}: loss {loss.item():.6f}", flush=True)
    cache = model.new_cache(a.users, 200)
    ids = batch[0][batch[2][:-1].long()]  # every user's first item
    for i in range(3):
        hidden, best = model.serve(ids, cache)
        print(f"token {i}: user 0 is at item {ids[0].item()}, best next items {best[0].tolist()}", flush=True)
        ids = best[:, 0].contiguous()


if __name__ == "__main__":
    main()
