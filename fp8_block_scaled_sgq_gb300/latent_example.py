"""One latent-attention layer on the library's calls: a prompt, then tokens one at a time.

    python -m fp8_block_scaled_sgq_gb300.latent_example

The linears are the W8A8 block-scaled ones ([1,128]/[128,128], UE8M0); between
them run the latent attention's four operators:

* a prompt: queries and keys rotated and rows written to the cache in one call
  (``latent_append``), keys and values expanded by the up-projection, and
  ``latent_prefill``;
* a token: ``latent_append`` writes its rotated queries straight into the
  attention's query tensor, ``latent_attention`` reads the cache, and the
  up-projection's two halves are absorbed into queries and outputs.

Both forms compute one thing; the script prints how far a token's output by the
absorbed form is from the same token's as the last one of a prompt.  Weights and
inputs are random.
"""
from __future__ import annotations

import torch

import fp8_block_scaled_sgq_gb300 as sgq

BLK = 128


class Linear:
    """y = x W^T with 128-block FP8 weights, quantised once."""

    def __init__(self, n: int, k: int, g):
        self.w = (torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).bfloat16()
        self.wq, self.ws = sgq.quant_weight_block(self.w, BLK, BLK, True)

    def __call__(self, x):
        return sgq.w8a8_linear(x.contiguous(), self.wq, self.ws, BLK, BLK, True)

    def dequantised(self):
        s = self.ws.repeat_interleave(BLK, 0).repeat_interleave(BLK, 1)
        return (self.wq.view(torch.float8_e4m3fn).float() * s[:self.wq.shape[0]]).bfloat16()


def _norm(x):
    return (x.float() * x.float().pow(2).mean(-1, keepdim=True).add(1e-6).rsqrt()).to(x.dtype)


class LatentLayer:
    def __init__(self, hidden=1024, heads=16, q_rank=512, latent=512, nope=128, rot=64, max_pos=4096, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.heads, self.latent, self.nope, self.rot = heads, latent, nope, rot
        self.q_down, self.q_up = Linear(q_rank, hidden, g), Linear(heads * (nope + rot), q_rank, g)
        self.kv_down = Linear(latent + rot, hidden, g)
        self.kv_up = Linear(heads * 2 * nope, latent, g)
        self.out = Linear(hidden, heads * nope, g)
        up = self.kv_up.dequantised().view(heads, 2 * nope, latent)
        self.up_k, self.up_v = up[:, :nope], up[:, nope:].transpose(1, 2)     # [H, nope, latent], [H, latent, nope]
        self.table = sgq.rotary_table(max_pos, rot)
        self.scale = (nope + rot) ** -0.5

    def project(self, x):
        q = self.q_up(_norm(self.q_down(x))).view(-1, self.heads, self.nope + self.rot)
        kv = self.kv_down(x)
        return q, _norm(kv[:, :self.latent]), kv[:, self.latent:]

    def prompt(self, x, starts, positions, slots, cache):
        """x [T, hidden], ragged: request b's tokens are starts[b] .. starts[b + 1] - 1."""
        q, latent, k_rot = self.project(x)
        turned = torch.empty_like(k_rot, memory_format=torch.contiguous_format)
        q_rot = q[..., self.nope:]
        sgq.latent_append(q_rot, k_rot, latent, positions, slots, self.table, cache, q_out=q_rot, k_out=turned)
        kv = self.kv_up(latent).view(-1, self.heads, 2 * self.nope)
        o = sgq.latent_prefill(q, kv[..., :self.nope], turned, kv[..., self.nope:], starts, starts, self.scale)
        return self.out(o.flatten(1))

    def token(self, x, positions, slots, cache, page_table, kv_lens):
        """One new token of every request: x [B, hidden]; kv_lens count the new token's row."""
        q, latent, k_rot = self.project(x)
        absorbed = torch.empty(x.shape[0], self.heads, self.latent + self.rot, dtype=x.dtype, device=x.device)
        absorbed[..., :self.latent] = torch.bmm(q[..., :self.nope].transpose(0, 1), self.up_k).transpose(0, 1)
        sgq.latent_append(q[..., self.nope:], k_rot, latent, positions, slots, self.table, cache,
                          q_out=absorbed[..., self.latent:])
        o = sgq.latent_attention(absorbed, cache, page_table, kv_lens, self.scale, self.latent)
        o = torch.bmm(o.transpose(0, 1), self.up_v).transpose(0, 1)
        return self.out(o.flatten(1))


def main(lengths=(300, 1, 77), page=64, steps=3) -> float:
    """Largest relative distance of a token by the absorbed form from the same token in a prompt."""
    layer = LatentLayer()
    g = torch.Generator("cuda").manual_seed(1)
    total = [n + steps for n in lengths]
    x = [torch.randn(n, 1024, generator=g, device="cuda").bfloat16() for n in total]
    width = max(-(-n // page) for n in total)
    page_table = torch.randperm(len(total) * width, generator=g, device="cuda").int().view(len(total), width)

    def slots_of(b, first, last):
        i = torch.arange(first, last, device="cuda")
        return page_table[b].long()[i // page] * page + i % page, i

    def prompt(upto, cache):
        parts = [slots_of(b, 0, n) for b, n in enumerate(upto)]
        starts = torch.tensor([0, *torch.tensor(upto).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
        return layer.prompt(torch.cat([v[:n] for v, n in zip(x, upto)]), starts, torch.cat([p[1] for p in parts]),
                            torch.cat([p[0] for p in parts]), cache)

    shape = (len(total) * width, page, layer.latent + layer.rot)
    cache = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    prompt(list(lengths), cache)
    worst = 0.0
    for s in range(steps):
        at = [n + s for n in lengths]
        parts = [slots_of(b, n, n + 1) for b, n in enumerate(at)]
        got = layer.token(torch.stack([v[n] for v, n in zip(x, at)]), torch.cat([p[1] for p in parts]),
                          torch.cat([p[0] for p in parts]), cache, page_table,
                          torch.tensor([n + 1 for n in at], dtype=torch.int32, device="cuda"))
        whole = prompt([n + 1 for n in at], torch.zeros_like(cache))
        want = whole[torch.tensor([n + 1 for n in at]).cumsum(0).cuda() - 1]
        worst = max(worst, ((got.float() - want.float()).norm(dim=1) / want.float().norm(dim=1)).max().item())
    if sgq.sgq_device_status() != 0:
        raise RuntimeError("device status not OK")
    return worst


if __name__ == "__main__":
    print(f"absorbed against expanded form, 3 tokens of 3 requests: relative distance at most {main():.4f}")
