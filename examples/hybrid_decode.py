"""One decode step of a small hybrid model through the library: Mamba2 layers with attention
layers between them, a residual add and RMS norm before each.

    python examples/hybrid_decode.py [--steps N] [--batch B]

The projections are plain matrix products with random weights (torch); everything between
them is the library's: rssm_add_rmsnorm, rssm_mamba2_step, rssm_attn_append,
rssm_attn_decode, rssm_attn_advance. A step reads no device data on the host, so the
model captures it in one CUDA graph and replays that while the lengths grow."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ssm_linear_attention_gb300 as ssm  # noqa: E402


class MambaLayer:
    def __init__(self, width, max_batch, num_slots, act, g, headdim=64, dstate=128, ring_len=16):
        self.H, self.P, self.N = width // headdim, headdim, dstate
        self.w_in = weight(g, width, 2 * width + 2 * dstate + self.H, act)
        self.w_out = weight(g, width, width, act)
        self.A = -torch.rand(self.H, generator=g, device="cuda") - 0.5
        self.D = torch.randn(self.H, generator=g, device="cuda")
        self.bias = torch.rand(self.H, generator=g, device="cuda") - 3
        self.dec = ssm.Mamba2ReplayDecoder(self.H, headdim, dstate, 1, ring_len, num_slots,
                                           max_batch, self.A, self.D, self.bias,
                                           state_dtype=torch.float32, act_dtype=act, out_dtype=act)

    def step(self, h, slots):
        b, width = h.shape
        x, z, B, C, dt = (h @ self.w_in).split([width, width, self.N, self.N, self.H], -1)
        y = self.dec.step(x.reshape(b, self.H, self.P).contiguous(), dt.float().contiguous(),
                          B.reshape(b, 1, self.N).contiguous(), C.reshape(b, 1, self.N).contiguous(),
                          z.reshape(b, self.H, self.P).contiguous(), slots)
        return y.view(b, width) @ self.w_out


class AttentionLayer:
    def __init__(self, width, max_batch, num_slots, act, cache_dtype, pages, g, heads_per_key=4,
                 head_dim=64):
        self.HQ = width // head_dim
        self.HKV, self.hd = self.HQ // heads_per_key, head_dim
        self.w_qkv = weight(g, width, (self.HQ + 2 * self.HKV) * head_dim, act)
        self.w_out = weight(g, width, width, act)
        # the page table and the lengths are the model's: its layers share them
        self.dec = ssm.PagedAttentionDecoder(
            self.HQ, self.HKV, head_dim, pages["page_size"], pages["num_pages"], num_slots,
            pages["page_table"].shape[1], max_batch, act_dtype=act, cache_dtype=cache_dtype,
            out_dtype=act, page_table=pages["page_table"], slot_len=pages["slot_len"])

    def step(self, h, slots):
        b = h.shape[0]
        # q, k and v are slices of one projection: no copy, the calls take their strides
        qkv = (h @ self.w_qkv).view(b, self.HQ + 2 * self.HKV, self.hd)
        q, k, v = qkv.split([self.HQ, self.HKV, self.HKV], 1)
        self.dec.append(k, v, slots)
        return self.dec.decode(q.unsqueeze(1), slots).view(b, -1) @ self.w_out


def weight(g, n, m, dtype):
    return (torch.randn(n, m, generator=g, device="cuda") / n ** 0.5).to(dtype)


class HybridModel:
    """layers: a string of "m" (Mamba2) and "a" (attention)."""

    def __init__(self, layers="mam", width=512, max_batch=8, max_tokens=256, act=torch.bfloat16,
                 cache_dtype=torch.float8_e4m3fn, norm_dtype=torch.float8_e4m3fn, page_size=16,
                 seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        num_slots, per_slot = 2 * max_batch, -(-max_tokens // page_size)
        self.pages = {"page_size": page_size, "num_pages": num_slots * per_slot,
                      # a serving program hands pages out as rows grow; here each slot has its own
                      "page_table": torch.randperm(num_slots * per_slot, generator=g, device="cuda")
                      .to(torch.int32).view(num_slots, per_slot),
                      "slot_len": torch.zeros(num_slots, device="cuda", dtype=torch.int32)}
        self.act, self.width = act, width
        self.layers = [MambaLayer(width, max_batch, num_slots, act, g) if c == "m" else
                       AttentionLayer(width, max_batch, num_slots, act, cache_dtype, self.pages, g)
                       for c in layers]
        # the norms before the layers may be 8-bit, the last one is not
        self.norms = [ssm.AddRMSNorm(1 + 0.1 * torch.randn(width, generator=g, device="cuda"), 1e-5,
                                     max_batch, act_dtype=act,
                                     out_dtype=norm_dtype if i < len(layers) else act)
                      for i in range(len(layers) + 1)]
        self.attention = [l for l in self.layers if isinstance(l, AttentionLayer)]
        self.graph = None

    def step(self, x, slots):
        """x [b, width]: the step's embeddings. Returns the normed stream [b, width]."""
        residual = torch.zeros_like(x)
        for norm, layer in zip(self.norms, self.layers):
            h, scale = norm(x, residual)       # residual += x, in place
            if scale is not None:              # a quantised projection would take h and scale
                h = (h.float() * scale).to(self.act)
            x = layer.step(h, slots)
        out, _ = self.norms[-1](x, residual)
        if self.attention:                     # one advance for all layers: they share the lengths
            self.attention[0].dec.advance(slots)
        return out

    def capture(self, batch):
        """Captures a step for `batch` rows; replay() then takes new inputs."""
        self.x = torch.zeros(batch, self.width, device="cuda", dtype=self.act)
        self.slots = torch.full((batch,), -1, device="cuda", dtype=torch.int32)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step(self.x, self.slots)      # padding rows only: warms up, changes nothing
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = self.step(self.x, self.slots)

    def replay(self, x, slots):
        self.x.copy_(x)
        self.slots.copy_(slots)
        self.graph.replay()
        return self.out


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--batch", type=int, default=8)
    a = ap.parse_args()
    model = HybridModel(max_batch=a.batch, max_tokens=a.steps + 1)
    model.capture(a.batch)
    slots = torch.randperm(2 * a.batch, device="cuda")[:a.batch].to(torch.int32)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record()
    for _ in range(a.steps):
        out = model.replay(torch.randn(a.batch, model.width, device="cuda").to(model.act), slots)
    end.record()
    torch.cuda.synchronize()
    errors = sum(int(l.dec.dev_err.sum()) for l in model.layers)
    print("%d steps of %d rows: %.1f us a step, lengths now %s, device errors %d, mean |out| %.3f" % (
        a.steps, a.batch, start.elapsed_time(end) * 1e3 / a.steps,
        model.pages["slot_len"][slots.long()].tolist(), errors, float(out.float().abs().mean())))


if __name__ == "__main__":
    main()
