"""One decoder layer on NVFP4 operators, served: prompts in ragged chunks, then
one token of each sequence a step, or a drafted tree of each.

    python examples/decoder_layer.py [--hidden 5120 --steps 32] [--draft 8 --window 4096 --sinks 4]

Weights are random. The norm quantizes for the products, the projections' keys
and values go into the paged NVFP4 cache as they are (slices of one output),
attention reads the cache, and the MLP half follows:

    x, r -> r + x, norm, NVFP4 -> QKV product -> cache write -> attention
         -> NVFP4 -> output product -> r + ., norm, NVFP4
         -> gate_up product, SwiGLU, NVFP4 -> down product

With rope_theta queries and keys are turned by their positions on the way into
the cache. Batch deals pages on the host; DeviceBatch does so on the GPU, so that
a step can be captured with its bookkeeping, and drafts trees. Sampling is the
caller's.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_quantized_dense_amd as nv  # noqa: E402


class DecoderLayer:
    def __init__(self, hidden, inter, heads_q, heads, head_dim, pages, page_size, window=0, h_amax=8.0, seed=0, device="cuda",
                 sinks=0, rope_theta=None, rope_sections=None):
        gen = torch.Generator(device).manual_seed(seed)
        self.hidden, self.inter, self.heads_q, self.heads, self.dim = hidden, inter, heads_q, heads, head_dim
        self.page_size, self.window, self.sinks = page_size, window, sinks
        self.inv_freq = self.axes = None
        if rope_theta is not None:
            half = torch.arange(head_dim // 2, dtype=torch.float64) / (head_dim // 2)
            self.inv_freq = (rope_theta ** -half).float().to(device)
            if rope_sections is not None:  # frequencies of each axis: time, height, width
                self.axes = nv.nvfp4_rope_axes(rope_sections, device=device)

        def weight(rows, cols, kind=nv.REPACK_PLAIN):
            w = torch.randn(rows, cols, generator=gen, device=device) * cols ** -0.5
            g, g_inv = nv.nvfp4_calibrate(w)
            return nv.nvfp4_repack_weight(kind, *nv.nvfp4_quantize(w, g_inv)), g

        self.w_qkv, self.g_qkv = weight((heads_q + 2 * heads) * head_dim, hidden)
        self.w_o, self.g_o = weight(hidden, heads_q * head_dim)
        self.w_gu, self.g_gu = weight(2 * inter, hidden, nv.REPACK_SWIGLU)
        self.w_d, self.g_d = weight(hidden, inter)
        self.norm1, self.norm2 = (torch.ones(hidden, dtype=torch.bfloat16, device=device) for _ in range(2))
        # Static scales: of keys and values (largest magnitude 8 here), of the MLP's intermediate.
        self.kv_g = torch.full((1,), 8.0 / 2688.0, device=device)
        self.kv_g_inv = 1.0 / self.kv_g
        self.h_g = torch.full((1,), h_amax / 2688.0, device=device)
        self.h_g_inv, self.alpha_d = 1.0 / self.h_g, self.h_g * self.g_d
        self.cache = nv.nvfp4_kv_cache(pages, page_size, heads, head_dim, device=device)
        self.ws = torch.zeros(nv.ATTENTION_COUNTER_BYTES, dtype=torch.uint8, device=device)
        self.earlier = []

    def workspace(self, *sizes):
        """One attention workspace for all calls, as large as the largest so far. Those before it stay allocated: a
        captured graph goes on using the address it was captured with."""
        need = nv.nvfp4_kv_attention_workspace_bytes(*sizes)
        if need > self.ws.numel():
            self.earlier.append(self.ws)
            self.ws = torch.zeros(need, dtype=torch.uint8, device=self.ws.device)
        return self.ws

    def __call__(self, x, residual, slots, block_table, seq_lens, q_offsets, max_q, max_len, trace=None, positions=None, tree=None):
        """x, residual bf16 [T, hidden] (residual is updated in place) -> bf16 [T, hidden]. positions int32 [axes, T]
        or [T], of all axes, where the layer turns; tree: the queries are drafted trees."""
        T, Hq, H, D = x.shape[0], self.heads_q, self.heads, self.dim
        codes, scales, residual, row_g = nv.add_rmsnorm_nvfp4_quant_per_token(x, self.norm1, residual=residual,
                                                                               residual_out=residual)
        qkv = nv.nvfp4_gemm_rowscale(codes, scales, row_g, self.w_qkv, (Hq + 2 * H) * D, self.hidden, self.g_qkv,
                                     out_dtype=torch.bfloat16)
        q, k, v = (part.unflatten(1, (-1, D)) for part in qkv.split([Hq * D, H * D, H * D], 1))
        if self.inv_freq is not None:
            q = nv.nvfp4_rope_kv_write(q, k, v, positions, self.inv_freq, slots, self.kv_g_inv, self.kv_g_inv, self.cache,
                                       axes=self.axes, q_out=q)
        else:
            nv.nvfp4_kv_write(k, v, slots, self.kv_g_inv, self.kv_g_inv, self.cache)
        ws = self.workspace(T, seq_lens.numel(), Hq, H, D, max_q, max_len)
        attn = nv.nvfp4_kv_attention(q, self.cache, block_table, seq_lens, self.kv_g, self.kv_g, q_offsets=q_offsets,
                                     max_q=max_q, max_len=max_len, window=self.window, ws=ws, sinks=self.sinks, tree=tree)
        a_codes, a_scales, a_g = nv.nvfp4_quantize_per_token(attn.view(T, Hq * D))
        o = nv.nvfp4_gemm_rowscale(a_codes, a_scales, a_g, self.w_o, self.hidden, Hq * D, self.g_o,
                                   out_dtype=torch.bfloat16)
        before = residual.clone() if trace is not None else None
        codes2, scales2, residual, row_g2 = nv.add_rmsnorm_nvfp4_quant_per_token(o, self.norm2, residual=residual,
                                                                                  residual_out=residual)
        h_codes, h_scales = nv.gemm_swiglu_nvfp4_quant_rowscale(codes2, scales2, row_g2, self.w_gu, self.inter, self.hidden,
                                                                self.g_gu, self.h_g_inv)
        out = nv.nvfp4_gemm(nv.MODE_W4A4, h_codes, h_scales, self.w_d, self.hidden, self.inter, self.alpha_d,
                            out_dtype=torch.bfloat16)
        if trace is not None:
            trace.update(codes=codes, scales=scales, row_g=row_g, q=q, k=k, v=v, attn=attn, o=o, before=before,
                         residual=residual.clone(), codes2=codes2, scales2=scales2, row_g2=row_g2)
        return out


class Batch:
    """Sequences whose pages are dealt from one pool as they grow."""

    def __init__(self, layer, sequences, max_len):
        self.layer, self.max_len = layer, max_len
        dev = layer.cache.device
        width = -(-max_len // layer.page_size)
        if sequences * width > layer.cache.shape[0]:
            raise ValueError("the cache has too few pages")
        self.table = torch.randperm(sequences * width, device=dev).to(torch.int32).view(sequences, width)
        self.lens = [0] * sequences

    def advance(self, counts):
        """Room for counts[b] more tokens of sequence b: the arguments of a layer call for them."""
        P, dev = self.layer.page_size, self.table.device
        seq = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).to(dev)
        pos = torch.cat([torch.arange(n, n + c) for n, c in zip(self.lens, counts)]).to(dev)
        slots = self.table[seq, pos // P].long() * P + pos % P
        self.lens = [n + c for n, c in zip(self.lens, counts)]
        offsets = [0]
        for c in counts:
            offsets.append(offsets[-1] + c)
        i32 = dict(dtype=torch.int32, device=dev)
        return dict(slots=slots, block_table=self.table, seq_lens=torch.tensor(self.lens, **i32),
                    q_offsets=torch.tensor(offsets, **i32), max_q=max(counts), max_len=self.max_len)


class DeviceBatch:
    """Sequences whose lengths, block tables and pool of pages stay on the GPU: nothing of a step depends on the host but
    its number of rows. A refusal is seen in `status`, whose it is in the slots of its rows, -1."""

    def __init__(self, layer, sequences, max_len):
        self.layer, self.max_len, dev = layer, max_len, layer.cache.device
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=dev)
        self.table = torch.full((sequences, -(-max_len // layer.page_size)), -1, dtype=torch.int32, device=dev)
        self.pool = nv.nvfp4_kv_pool(layer.cache.shape[0], device=dev)
        self.status = self.pool[1:2]

    def advance(self, counts, tokens, max_q, parents=None):
        """Room for counts[b] (int32 on the GPU) more tokens of sequence b, `tokens` rows in all, at most max_q of one
        sequence: the arguments of a layer call for them. parents (int32 [tokens]): they are drafted trees."""
        slots, positions, offsets = nv.nvfp4_kv_advance(counts, self.lens, self.table, self.pool, self.layer.page_size, tokens)
        tree = None
        if parents is not None:
            tree = nv.nvfp4_tree_mask(parents, offsets, max_q, positions=positions)
        return dict(slots=slots, block_table=self.table, seq_lens=self.lens, q_offsets=offsets, max_q=max_q, max_len=self.max_len,
                    positions=positions, tree=tree)

    def accept(self, call, kept, counts, dropped):
        """After a drafted call: its rows `kept` (int64, each sequence's accepted ones in order, counts[b] of them) become
        the sequence's next tokens, and dropped[b] = tokens drafted - counts[b] are taken back. A sequence whose draft was
        refused holds none of it (its rows have no slot) and stays as it is."""
        layer, slots = self.layer, call["slots"]
        if slots.numel() == 0:
            return
        k, v = nv.nvfp4_kv_read(layer.cache, slots[kept], layer.kv_g, layer.kv_g, dtype=torch.float32)
        first = call["q_offsets"][:-1].long()
        place = torch.arange(kept.numel(), device=kept.device)
        begin = torch.cumsum(counts, 0) - counts
        seq = torch.repeat_interleave(counts.long(), output_size=kept.numel())
        to = slots[first[seq] + place - begin[seq]]
        nv.nvfp4_kv_write(k, v, to, layer.kv_g_inv, layer.kv_g_inv, layer.cache)
        came = (first < call["q_offsets"][1:]) & (slots[first.clamp(max=slots.numel() - 1)] >= 0)
        nv.nvfp4_kv_advance(-dropped * came, self.lens, self.table, self.pool, layer.page_size, 0)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--inter", type=int, default=17408)
    ap.add_argument("--heads-q", type=int, default=40)
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--prompts", type=int, nargs="+", default=[1000, 37, 512, 1])
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--draft", type=int, default=0, help="drafted tokens of a sequence a step, as a tree; 0: single tokens")
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    a = ap.parse_args()
    if a.draft:
        return serve_trees(a)
    B, page = len(a.prompts), 64
    max_len = max(a.prompts) + a.steps
    layer = DecoderLayer(a.hidden, a.inter, a.heads_q, a.heads, a.head_dim, B * -(-max_len // page), page)
    batch = Batch(layer, B, max_len)

    def rows(n):
        return torch.randn(n, a.hidden, device="cuda").to(torch.bfloat16)

    out = layer(rows(sum(a.prompts)), rows(sum(a.prompts)), **batch.advance(a.prompts))
    assert bool(out.isfinite().all())
    times = []
    for _ in range(a.steps):
        call, x, r = batch.advance([1] * B), rows(B), rows(B)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        out = layer(x, r, **call)
        torch.cuda.synchronize()
        times.append(time.perf_counter() - t0)
        assert bool(out.isfinite().all())
    print(f"prompts {a.prompts}, then {a.steps} steps of {B} tokens: {sorted(times)[len(times) // 2] * 1e6:.0f} us a step "
          f"(median, one layer), cache {layer.cache.numel() / 2 ** 20:.1f} MiB")


def serve_trees(a):
    """Prompts, then drafted trees of which each step accepts the path to a random leaf."""
    B, n, page, dev = len(a.prompts), a.draft, 64, "cuda"
    max_len = max(a.prompts) + (a.steps + 1) * n
    layer = DecoderLayer(a.hidden, a.inter, a.heads_q, a.heads, a.head_dim, B * -(-max_len // page), page, window=a.window,
                         sinks=a.sinks, rope_theta=1e6)
    batch = DeviceBatch(layer, B, max_len)

    def rows(m):
        return torch.randn(m, a.hidden, device=dev).to(torch.bfloat16)

    T = sum(a.prompts)
    layer(rows(T), rows(T), **batch.advance(torch.tensor(a.prompts, dtype=torch.int32, device=dev), T, max(a.prompts)))
    draft = torch.full((B,), n, dtype=torch.int32, device=dev)
    times, accepted = [], 0
    for _ in range(a.steps):
        trees = [[-1] + [int(torch.randint(0, i, (1,))) for i in range(1, n)] for _ in range(B)]
        parents = torch.tensor(sum(trees, []), dtype=torch.int32, device=dev)
        x, r = rows(B * n), rows(B * n)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        call = batch.advance(draft, B * n, n, parents)
        out = layer(x, r, **call)
        torch.cuda.synchronize()
        times.append(time.perf_counter() - t0)
        assert bool(out.isfinite().all())
        kept, counts = [], []
        for b, tree in enumerate(trees):
            path, at = [], int(torch.randint(0, n, (1,)))
            while at >= 0:
                path.append(b * n + at)
                at = tree[at]
            kept += path[::-1]
            counts.append(len(path))
        counts = torch.tensor(counts, dtype=torch.int32, device=dev)
        batch.accept(call, torch.tensor(kept, device=dev), counts, draft - counts)
        accepted += len(kept)
    assert int(batch.status) == 0
    print(f"prompts {a.prompts}, then {a.steps} steps of {B} trees of {n} tokens: {sorted(times)[len(times) // 2] * 1e6:.0f} us a "
          f"step (median, one layer), {accepted / a.steps / B:.2f} tokens accepted of a tree, lengths {batch.lens.tolist()}")


if __name__ == "__main__":
    main()
