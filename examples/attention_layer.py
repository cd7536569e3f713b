"""One attention layer with NVFP4 weights, activations, keys and values: the fused q | k | v
projection, rotary embedding and append to the paged cache, attention over the cache, and
the output projection.

    python examples/attention_layer.py [--batch 8] [--prompt 1000] [--steps 64]

takes prompts of several lengths through the layer, then generates: a step per token,
replayed as one HIP graph, with the lengths kept on the device.  Weights and inputs are
random."""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_w4a4_quantized_amd as nv  # noqa: E402


class Linear:
    """y = x W^T: W [N, K] packed once with a global scale per segment, x quantized under a
    calibrated scale (a token's result then does not depend on the tokens beside it)."""

    def __init__(self, w, seg_end, x_amax, max_tokens):
        n, k = w.shape
        self.seg_end = seg_end
        self.codes, self.scales = nv.empty_packed(n, k, w.device)
        self.seg_gscale = torch.empty(len(seg_end), dtype=torch.float32, device=w.device)
        nv.nvfp4_pack_weight(w, seg_end, None, self.codes, self.scales, self.seg_gscale)
        self.gscale = torch.full((1,), x_amax / 2688, dtype=torch.float32, device=w.device)
        self.gscale_used = torch.empty_like(self.gscale)
        self.x_codes, self.x_scales = nv.empty_packed(max_tokens, k, w.device)

    def __call__(self, x, y):
        nv.nvfp4_w4a4_linear(x, self.gscale, self.gscale_used, self.codes, self.scales, self.seg_end, self.seg_gscale, y,
                             a_codes_out=self.x_codes[:x.shape[0]], a_scales_out=self.x_scales[:x.shape[0]])
        return y


class AttentionLayer:
    def __init__(self, hidden, n_q, n_kv, d, batch, max_len, max_tokens, page=64, seed=0, device="cuda"):
        gen = torch.Generator(device).manual_seed(seed)
        self.n_q, self.n_kv, self.d, self.page, self.batch, self.max_len = n_q, n_kv, d, page, batch, max_len
        ends = [n_q * d, (n_q + n_kv) * d, (n_q + 2 * n_kv) * d]

        def weight(n, k):
            return (torch.randn(n, k, generator=gen, device=device) * k ** -0.5).bfloat16()
        self.qkv = Linear(weight(ends[-1], hidden), ends, 6.0, max_tokens)
        self.out = Linear(weight(hidden, n_q * d), [hidden], 4.0, max_tokens)
        # The rotation as a table of positions; the cache, its pages in any order
        angle = torch.arange(max_len, device=device)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, device=device) / d)
        self.cos, self.sin = angle.cos().contiguous(), angle.sin().contiguous()
        per_seq = -(-max_len // page)
        self.table = torch.randperm(batch * per_seq, generator=gen, device=device).int().reshape(batch, per_seq)
        self.cache = nv.empty_kv_cache(batch * per_seq, n_kv, page, d, device)
        # calibrated: the largest key (any rotation of it) and value of a head
        self.k_gscale = torch.full((n_kv,), 2 ** 0.5 * 6.0 / 2688, device=device)
        self.v_gscale = torch.full((n_kv,), 6.0 / 2688, device=device)
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device=device)
        self.qkv_rows = torch.empty(max_tokens, ends[-1], dtype=torch.bfloat16, device=device)
        self.o_rows = torch.empty(max_tokens, n_q * d, dtype=torch.bfloat16, device=device)
        # A generated token's calls are all of one size.  Graphs hold the address of their
        # workspace, so it is never replaced, as the prompts' is when a longer one comes.
        self.decode_workspace = torch.empty(self._workspace_bytes(batch, 1), dtype=torch.uint8, device=device)
        self.workspace = torch.empty(0, dtype=torch.uint8, device=device)

    def _workspace_bytes(self, tokens, max_q_len):
        return nv.nvfp4_kv_attention_workspace(tokens, self.batch, self.n_q, self.n_kv, self.d, max_q_len, self.max_len,
                                               torch.bfloat16)

    def reserve(self, tokens, max_q_len):
        """Before a call of a size: the attention's workspace (not for calls in graphs, which
        would hold the address of one that a later call replaces)."""
        need = self._workspace_bytes(tokens, max_q_len)
        if need > self.workspace.numel():
            self.workspace = torch.empty(need, dtype=torch.uint8, device=self.cache.device)

    def __call__(self, x, y, seq, positions, cu_q=None, max_q_len=1, workspace=None):
        """x [T, hidden]: new tokens of sequences seq [T] at positions [T], those of one
        sequence in rows cu_q[b] .. cu_q[b + 1]; self.kv_len counts them already."""
        tokens = x.shape[0]
        pages = self.table[seq, positions // self.page].long()
        slots = pages * self.page + positions % self.page
        rows, o = self.qkv(x, self.qkv_rows[:tokens]), self.o_rows[:tokens]
        q, k, v = rows.split([self.n_q * self.d, self.n_kv * self.d, self.n_kv * self.d], 1)
        nv.nvfp4_rope_append_kv(q, k, v, self.cos, self.sin, positions, slots, self.cache, self.k_gscale, self.v_gscale,
                                self.page, q)                      # queries rotated in place
        nv.nvfp4_kv_attention(q, self.cache, self.table, self.kv_len, self.k_gscale, self.v_gscale, self.page, o,
                              self.max_len, self.workspace if workspace is None else workspace, cu_q=cu_q,
                              max_q_len=max_q_len)
        return self.out(o, y)

    def prompt(self, x, lens, y):
        """The prompts of all sequences, one after the other in x."""
        n = torch.tensor(lens, device=x.device)
        seq = torch.repeat_interleave(torch.arange(self.batch, device=x.device), n)
        cu = torch.zeros(self.batch + 1, dtype=torch.int32, device=x.device)
        cu[1:] = n.cumsum(0)
        positions = (torch.arange(x.shape[0], device=x.device) - cu[seq]).int()
        self.kv_len.copy_(n)
        self.reserve(x.shape[0], max(lens))
        return self(x, y, seq, positions, cu, max(lens))

    def decode(self, x, y):
        """One more token of every sequence; may be captured in a graph."""
        positions = self.kv_len.clone()
        self.kv_len += 1
        return self(x, y, torch.arange(self.batch, device=x.device), positions, workspace=self.decode_workspace)


def elapsed(fn, reps):
    fn()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(reps):
        fn()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) * 1e3 / reps


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000, help="longest prompt; the others are shorter")
    ap.add_argument("--steps", type=int, default=64, help="tokens to generate")
    args = ap.parse_args()
    hidden = 5120
    lens = [max(1, args.prompt * (b + 1) // args.batch) for b in range(args.batch)]
    total, reps = sum(lens), 5
    layer = AttentionLayer(hidden, 32, 8, 128, args.batch, args.prompt + args.steps + 2, max(total, args.batch))
    x = torch.randn(total, hidden, device="cuda").bfloat16()
    y = torch.empty_like(x)
    us = elapsed(lambda: layer.prompt(x, lens, y), reps)
    print(f"prompts: {total} tokens of {args.batch} sequences, {us:.1f} us")

    x1 = torch.randn(args.batch, hidden, device="cuda").bfloat16()
    y1 = torch.empty_like(x1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.decode(x1, y1)                                       # warm up on the capturing stream
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.decode(x1, y1)
    us = elapsed(graph.replay, args.steps)
    print(f"generation: {args.steps} steps, {us:.1f} us a step, contexts now {layer.kv_len.tolist()}")
    if not torch.isfinite(y1.float()).all():
        raise SystemExit("output is not finite")


if __name__ == "__main__":
    main()
