"""One attention block served with a paged key-value cache, from prompts to
forked samples, entirely on the device.

Quantized projections (W4A8) around the cache: prompts are written and attended
in one call each, two of them are forked into more samples, every step reserves
a page where one is due, writes one token for each running slot and attends it,
a sample is retired, and the pool is made dense.  Optionally the block has a norm
in front of its first projection, rotary positions, and an adapter for each
request beside that projection's shared weight.

    python examples/decode_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_weight_quantized_amd as w4  # noqa: E402


class Block:
    """x -> x + Wo attention(Wqkv x): W4A8 projections, a paged cache of `layers` layers.

    norm: an RMS norm of x in front of Wqkv; rope: rotary positions of queries and keys;
    adapters: as many low-rank adapters of Wqkv, self.adapter naming each slot's (-1: none)."""

    def __init__(self, hidden: int, q_heads: int, kv_heads: int, head_dim: int, slots: int,
                 pages: int, pages_per_slot: int, page_size: int = 16, dtype=torch.int8,
                 layers: int = 1, seed: int = 0, norm: bool = False, rope: w4.Rope = None,
                 adapters: int = 0, rank: int = 16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.h, self.d = q_heads, kv_heads, head_dim
        n = (q_heads + 2 * kv_heads) * head_dim
        wqkv = torch.randn((hidden, n), generator=g, device="cuda") * hidden ** -0.5
        wo = torch.randn((q_heads * head_dim, hidden), generator=g, device="cuda") * 0.02
        self.wqkv, self.sqkv, _ = w4.w4_quantize_weight(wqkv, "sym")
        self.wo, self.so, _ = w4.w4_quantize_weight(wo, "sym")
        self.cache = w4.KVCache.empty(layers, pages, kv_heads, page_size, head_dim, dtype)
        self.table = torch.full((slots, pages_per_slot), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros((slots,), dtype=torch.int32, device="cuda")
        self.refs = torch.zeros((pages,), dtype=torch.int32, device="cuda")
        self.norm = 1 + 0.1 * torch.randn((hidden,), generator=g, device="cuda") if norm else None
        self.rope = rope
        self.adapter = torch.full((slots,), -1, dtype=torch.int32, device="cuda")
        if adapters:
            self.A = (torch.randn((adapters, rank, hidden), generator=g, device="cuda")
                      * hidden ** -0.5).bfloat16()
            self.B = (0.1 * torch.randn((adapters, n, rank), generator=g, device="cuda")).bfloat16()
        self.adapters = adapters

    def project(self, x: torch.Tensor, adapter: torch.Tensor = None):
        """(q, k, v) of rows x [T, hidden]: slices of one product's rows; adapter [T]:
        each row's."""
        if self.norm is not None and not self.adapters:
            xq, sx, _ = w4.a8_rms_norm(x, self.norm, 1e-6)  # int8 rows, as the product takes them
            y = w4.w4a8_linear_q(xq, sx, self.wqkv, self.sqkv)
        else:
            if self.norm is not None:
                x, _ = w4.rms_norm(x, self.norm, 1e-6)
            y = w4.w4a8_linear(x, self.wqkv, self.sqkv)
            if self.adapters:
                w4.lora_add(y, x, adapter, self.A, self.B)
        y = y.unflatten(1, (-1, self.d))
        return y[:, :self.hq], y[:, self.hq:self.hq + self.h], y[:, self.hq + self.h:]

    def append(self, layer, q, k, v, table, start, cu=None) -> torch.Tensor:
        """Tokens into the cache; the queries as the attention takes them."""
        if self.rope is None:
            w4.kv_append(self.cache, layer, k, v, table, start, cu)
            return q
        return w4.kv_append_rope(self.cache, layer, q, k, v, table, start, self.rope, cu, out=q)

    def output(self, x: torch.Tensor, o: torch.Tensor) -> torch.Tensor:
        return x + w4.w4a8_linear(o.flatten(1), self.wo, self.so)

    def reserve(self, add: torch.Tensor) -> torch.Tensor:
        return w4.kv_reserve(self.table, self.lens, self.refs, add, self.cache.page_size)

    def prompts(self, x: torch.Tensor, slots: torch.Tensor, cu: torch.Tensor, layer: int = 0,
                window: int = 0, sinks: int = 0):
        """New prompts x [T, hidden] (rows cu[i] : cu[i + 1], others are padding) into empty
        slots; (x', q, o)."""
        add = torch.zeros_like(self.lens)
        add[slots.long()] = cu[1:] - cu[:-1]
        ok = self.reserve(add)
        self.lens += add * ok
        table, lens = self.table[slots.long()], self.lens[slots.long()]
        rows = of_rows(self.adapter[slots.long()], cu, x.shape[0]) if self.adapters else None
        q, k, v = self.project(x, rows)
        q = self.append(layer, q, k, v, table, torch.zeros_like(lens), cu)
        o = w4.kv_prefill_attention(q, self.cache, layer, table, lens, cu, window=window, sinks=sinks)
        return self.output(x, o), q, o

    def step(self, x: torch.Tensor, layer: int = 0, window: int = 0, sinks: int = 0):
        """One token x [slots, hidden] for every slot that has any; (x', q, o)."""
        running = (self.lens > 0).to(torch.int32)
        running *= self.reserve(running)
        start = torch.where(running > 0, self.lens, -1)  # -1: takes no token
        q, k, v = self.project(x, self.adapter)
        q = self.append(layer, q, k, v, self.table, start)
        self.lens += running
        o = w4.kv_decode_attention(q, self.cache, layer, self.table, self.lens * running,
                                   window=window, sinks=sinks)
        return self.output(x, o), q, o

    def fork(self, parents, children) -> torch.Tensor:
        ok = w4.kv_fork(self.cache, self.table, self.lens, self.refs, parents, children)
        if self.adapters:
            hand_on(self.adapter, parents, children, ok)
        return ok

    def free(self, slots) -> None:
        w4.kv_free(self.table, self.lens, self.refs, slots)
        if self.adapters:
            drop(self.adapter, slots)

    def compact(self) -> torch.Tensor:
        return w4.kv_compact(self.cache, self.table, self.refs)[2]


def of_rows(adapter: torch.Tensor, cu: torch.Tensor, T: int) -> torch.Tensor:
    """Each of T rows' adapter: its sequence's, -1 in rows of no sequence."""
    t = torch.arange(T, dtype=torch.int32, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    inside = (t >= cu[0]) & (b < adapter.numel())
    return torch.where(inside, adapter[b.clamp(max=adapter.numel() - 1)], -1)


def put(adapter: torch.Tensor, slots: torch.Tensor, on: torch.Tensor, values) -> None:
    """adapter[slots] = values where `on`; what the other slots name is no matter."""
    wide = torch.cat([adapter, adapter[:1]])  # (the row behind the last takes the others)
    wide[torch.where(on, slots, adapter.numel()).long()] = values
    adapter.copy_(wide[:-1])


def hand_on(adapter: torch.Tensor, parents: torch.Tensor, children: torch.Tensor,
            ok: torch.Tensor) -> None:
    """A granted fork's child has its parent's adapter; a fork that is not granted changes none."""
    on = ok > 0
    put(adapter, children, on, adapter[torch.where(on, parents, 0).long()])


def drop(adapter: torch.Tensor, slots: torch.Tensor) -> None:
    """Retired slots name no adapter; slots that there are not are skipped."""
    put(adapter, slots, (slots >= 0) & (slots < adapter.numel()), -1)


def ints(*v) -> torch.Tensor:
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def serve(steps: int = 20, hidden: int = 1152, dtype=torch.int8, window: int = 0, sinks: int = 0,
          seen=lambda block, what, q, o: None, **kw) -> Block:
    """Two prompts, five samples, `steps` tokens each; `seen` looks at each call;
    kw: the block's norm, rope and adapters (the first prompt has the last adapter)."""
    b = Block(hidden, q_heads=8, kv_heads=2, head_dim=128, slots=8, pages=96, pages_per_slot=24,
              dtype=dtype, **kw)
    if b.adapters:
        b.adapter[5] = b.adapters - 1
    g = torch.Generator(device="cuda").manual_seed(1)
    cu = ints(0, 37, 237)
    x = torch.randn((237, hidden), generator=g, device="cuda")
    _, q, o = b.prompts(x, ints(5, 2), cu, window=window, sinks=sinks)
    seen(b, "prompts", q, o)
    b.fork(ints(5, 5, 2), ints(0, 1, 7))
    for i in range(steps):
        x = torch.randn((8, hidden), generator=g, device="cuda")
        x, q, o = b.step(x, window=window, sinks=sinks)
        seen(b, "step", q, o)
        if i == steps // 2:
            b.free(ints(5, 7))
            b.compact()
    return b


if __name__ == "__main__":
    block = serve(norm=True, rope=w4.Rope(128), adapters=3)
    print("lengths", block.lens.tolist())
    print("pages held", int((block.refs > 0).sum()), "of", block.refs.numel(),
          "- shared", int((block.refs > 1).sum()))
