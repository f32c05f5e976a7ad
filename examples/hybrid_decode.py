"""A hybrid model's two kinds of layer side by side: prompt, then decoding.

A tiny model of random weights, one Mamba-2 layer and one attention layer, takes a
batch of prompts and then generates hidden states token by token:

* the state-space layer with ``ssd.mixer_prologue`` + ``ssd.chunked_fwd`` for the
  prompt and ``ssd.mixer_prologue`` + ``ssd.state_update`` for single tokens;
* the attention layer with ``attn.kv_append`` (norm, rotation and the write into an
  8-bit or 4-bit paged cache in one pass) + ``attn.paged_attention`` for both.

At the end it reads the cache back (``attn.kv_read``) and checks the last token's
attention against a plain softmax over those rows, and the whole decoding against one
prompt of the full length.  Run it from the repository's root on a GPU:

    python examples/hybrid_decode.py [--cache bf16 | fp4]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from state_space_model_gb300 import attn, ssd  # noqa: E402

WIDTH, PAGE = 512, 16
H, P, N, G, W = 16, 64, 128, 2, 4            # state-space heads, head, state, groups, conv width
HQ, HKV, D = 8, 2, 64                        # query heads, key/value heads, head
BF = torch.bfloat16


def norm(x):
    x = x.float()
    return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).to(BF)


class StateSpaceLayer:
    def __init__(self, batch, g):
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.dc = H * P + 2 * G * N
        self.w_in = (r(WIDTH, H * P + self.dc + H) / math.sqrt(WIDTH)).to(BF)
        self.w_out = (r(H * P, WIDTH) / math.sqrt(H * P)).to(BF)
        self.conv_w, self.conv_b = r(self.dc, W) / math.sqrt(W), r(self.dc) * 0.1
        self.A, self.D, self.dt_bias = -torch.exp(r(H) * 0.5), r(H), r(H) * 0.1 - 2.0
        self.conv_state = torch.zeros(batch, self.dc, W, dtype=BF, device="cuda")
        self.state = None

    def __call__(self, hidden):
        """hidden [B,L,WIDTH]; the first call is the prompt, later ones single tokens."""
        z, xbc, dt = (norm(hidden) @ self.w_in).split([H * P, self.dc, H], -1)
        x, b, c, dt = ssd.mixer_prologue(xbc.contiguous(), self.conv_w, dt.float().contiguous(), H, P, G, N,
                                         conv_bias=self.conv_b, conv_state=self.conv_state,
                                         dt_bias=self.dt_bias)
        z = z.unflatten(-1, (H, P)).contiguous()
        if self.state is None:
            y, self.state = ssd.chunked_fwd(x, dt, self.A, b, c, self.D, None, 256, G, z=z)
        else:
            y = ssd.state_update(self.state, x[:, 0], dt[:, 0], self.A, b[:, 0], c[:, 0], self.D, z=z[:, 0],
                                 ngroups=G)[:, None]
        return hidden + y.flatten(-2) @ self.w_out


class AttentionLayer:
    def __init__(self, batch, longest, cache, g):
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.w_qkv = (r(WIDTH, (HQ + 2 * HKV) * D) / math.sqrt(WIDTH)).to(BF)
        self.w_out = (r(HQ * D, WIDTH) / math.sqrt(HQ * D)).to(BF)
        self.q_weight, self.k_weight = 1 + r(D) * 0.1, 1 + r(D) * 0.1
        angle = torch.arange(longest, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
        self.cos, self.sin = angle.cos(), angle.sin()
        # every sequence's pages, handed out in no order
        per = -(-longest // PAGE)
        order = torch.randperm(batch * per, generator=g, device="cuda")
        self.table = order.view(batch, per).to(torch.int32)
        shape = (batch * per, HKV, PAGE, D)
        def pool(bits, kind):
            """Codes of so many bits; torch has few operations for these types."""
            return torch.zeros(*shape[:3], int(D * bits) // 8, dtype=torch.uint8, device="cuda").view(kind)

        kind = {"fp4": torch.float4_e2m1fn_x2, "fp8": torch.float8_e4m3fn, "bf16": BF}[cache]
        self.k, self.v = (pool({"fp4": 4, "fp8": 8, "bf16": 16}[cache], kind) for _ in range(2))
        self.scales = {}
        if cache != "bf16":
            self.scales = {n: torch.ones(shape[:3], device="cuda") for n in ("k_scale", "v_scale")}
        if cache == "fp4":       # a byte for each 16 places
            self.scales.update({n: pool(0.5, torch.float8_e4m3fn) for n in ("k_group_scale", "v_group_scale")})
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def __call__(self, hidden):
        batch, n, _ = hidden.shape
        qkv = (norm(hidden) @ self.w_qkv).view(batch * n, -1)
        q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([HQ * D, HKV * D, HKV * D], -1))
        pos = self.lens[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
        slots = self.table.gather(1, (pos // PAGE).long()) * PAGE + pos % PAGE
        self.lens += n
        self.q = attn.kv_append(q, k, v, slots.flatten().contiguous(), self.k, self.v,
                                positions=pos.flatten().contiguous(), cos=self.cos, sin=self.sin,
                                q_weight=self.q_weight, k_weight=self.k_weight, **self.scales)
        out = attn.paged_attention(self.q.view(batch, n, HQ, D), self.k, self.v, self.table, self.lens,
                                   **self.scales)
        self.out = out
        return hidden + out.flatten(-2) @ self.w_out


class Model:
    def __init__(self, batch, longest, cache, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ssm, self.attention = StateSpaceLayer(batch, g), AttentionLayer(batch, longest, cache, g)

    def __call__(self, hidden):
        return self.attention(self.ssm(hidden))


def check_last_token(layer):
    """The last token's attention against a softmax over the rows read back: largest error."""
    lens = layer.lens.tolist()
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    keys, values = attn.kv_read(layer.k, layer.v, layer.table, cu, sum(lens), **layer.scales,
                                dtype=torch.float32 if layer.scales else None)
    worst = 0.0
    for b, n in enumerate(lens):
        rows = slice(int(cu[b]), int(cu[b]) + n)
        q = layer.q.view(len(lens), -1, HKV, HQ // HKV, D)[b, -1].float()
        s = torch.einsum("hgd,nhd->hgn", q, keys[rows].float()) / math.sqrt(D)
        o = torch.einsum("hgn,nhd->hgd", s.softmax(-1), values[rows].float())
        worst = max(worst, float((o.flatten(0, 1) - layer.out[b, -1].float()).abs().max() / o.abs().max()))
    return worst


def main(cache="fp8", batch=3, prompt=300, tokens=12, seed=7):
    """Largest relative errors: (last token's attention, decoding against one long prompt)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    hidden = torch.randn(batch, prompt + tokens, WIDTH, generator=g, device="cuda").to(BF)
    longest = prompt + tokens
    model = Model(batch, longest, cache, seed)
    outs = [model(hidden[:, :prompt])]
    for t in range(prompt, longest):
        outs.append(model(hidden[:, t: t + 1]))
    whole = Model(batch, longest, cache, seed)(hidden)
    steps = torch.cat(outs, 1)
    apart = float((steps - whole).float().abs().max() / whole.float().abs().max())
    return check_last_token(model.attention), apart


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--cache", choices=["fp8", "bf16", "fp4"], default="fp8")
    last, apart = main(ap.parse_args().cache)
    print(f"last token's attention against a softmax over the cache read back: {last:.2e}")
    print(f"decoding token by token against one prompt of the full length:    {apart:.2e}")
