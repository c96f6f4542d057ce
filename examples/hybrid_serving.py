"""A serving loop of a hybrid model's two kinds of layers: one KDA layer with its fixed-size state and one attention
layer with a paged 4-bit key/value cache, for a ragged batch.

Prompts are admitted (page_plan, chunk_fwd, cache4_append, cache4_attention), then a few decode steps follow (page_plan,
decode_verify_replay with an empty draft window, cache4_append, cache4_attention).  Projections are random: the point is
the order of the calls and what passes between them.  Every attention output is compared with plain attention in 32
bits over the values that the cache holds.

    python examples/hybrid_serving.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_gated_delta_02_gb300 as kda  # noqa: E402

H, D = 4, 128                    # KDA heads, channels per head (both layers)
HQ, HKV, PAGE = 8, 2, 64         # attention heads, key heads, tokens per page
HIDDEN, PAGES, MAX_PAGES = 256, 40, 8


class AttentionLayer:
    """Fused projection and the 4-bit cache; k and v go to the cache as views of the projection."""

    def __init__(self, gen):
        self.w = (torch.randn(HIDDEN, (HQ + 2 * HKV) * D, generator=gen, device="cuda") * HIDDEN ** -0.5).bfloat16()
        self.cache = kda.cache4_alloc(PAGES, HKV, PAGE, D)

    def __call__(self, x, plan, table, max_new, status):
        cu, seq_len, slots = plan[:3]
        qkv = x @ self.w
        q, k, v = (t.view(t.shape[0], -1, D) for t in qkv.split([HQ * D, HKV * D, HKV * D], dim=1))
        kda.cache4_append(k, v, slots, self.cache, PAGE, status=status)
        return q, kda.cache4_attention(q, self.cache, table, seq_len, cu, PAGE, max_new=max_new, status=status)


def plain_attention(q, layer, plan, table):
    """The same attention, a request and a query at a time in 32 bits, over the values that the cache holds."""
    cu, lengths = plan[0].tolist(), plan[1].tolist()
    out = torch.empty(q.shape, device="cuda")
    for r, n in enumerate(lengths):
        pos = torch.arange(n, device="cuda")
        slots = table[r][pos // PAGE] * PAGE + (pos % PAGE).int()
        k, v = kda.cache4_read(layer.cache, slots, PAGE, D, dtype=torch.float32)
        k, v = (t.repeat_interleave(HQ // HKV, dim=1) for t in (k, v))
        for i in range(cu[r], cu[r + 1]):
            sees = n - (cu[r + 1] - 1 - i)
            p = torch.softmax(torch.einsum("hd,jhd->hj", q[i].float(), k[:sees]) * D ** -0.5, dim=-1)
            out[i] = torch.einsum("hj,jhd->hd", p, v[:sees])
    return out


def main(prompts=(70, 130, 5), steps=4, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    R, T = len(prompts), sum(prompts)
    layer = AttentionLayer(gen)
    status = torch.zeros(1, **i32)
    # pages: none held, all free
    table, free = torch.full((R, MAX_PAGES), -1, **i32), torch.randperm(PAGES, generator=gen, device="cuda").int()
    length, count, left = torch.zeros(R, **i32), torch.zeros(R, **i32), torch.tensor([PAGES], **i32)
    worst = 0.0

    def check(q, o, plan):
        want = plain_attention(q, layer, plan, table)
        return float((o.float() - want).abs().max() / want.abs().max())

    # ---- prompts
    plan = kda.page_plan(length, torch.tensor(prompts, **i32), count, table, free, left, PAGE, T, status=status)
    length, count, left = plan[1], plan[4], plan[5]
    unit = lambda t: torch.nn.functional.normalize(t, dim=-1).bfloat16()
    _, state = kda.chunk_fwd(unit(randn(T, H, D)), unit(randn(T, H, D)), randn(T, H, D).bfloat16(),
                             -torch.nn.functional.softplus(randn(T, H, D)), torch.sigmoid(randn(T, H)), plan[0], status=status)
    x = randn(T, HIDDEN).bfloat16()
    q, o = layer(x, plan, table, max(prompts), status)
    worst = max(worst, check(q, o, plan))

    # ---- single tokens
    C = 3 * H * D
    state, tail = state.bfloat16(), torch.zeros(R, 3, C, dtype=torch.bfloat16, device="cuda")
    conv_w, norm_w = 0.5 * randn(C, 4), torch.ones(D, device="cuda")
    none = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    accepted, one = torch.zeros(R, **i32), torch.ones(R, **i32)
    for _ in range(steps):
        plan = kda.page_plan(length, one, count, table, free, left, PAGE, R, status=status)
        length, count, left = plan[1], plan[4], plan[5]
        y = kda.decode_verify_replay(state, tail, conv_w, none(R, 0, C), none(R, 0, H * D), none(R, 0, H), accepted,
                                     randn(R, 1, C).bfloat16(), randn(R, 1, H * D).bfloat16(), randn(R, 1, H).bfloat16(),
                                     norm_w, status=status)
        q, o = layer(randn(R, HIDDEN).bfloat16(), plan, table, 1, status)
        worst = max(worst, check(q, o, plan))
        assert torch.isfinite(y).all()
    assert status.item() == 0, f"status {status.item():#x}"
    assert left.item() == PAGES - sum(-(-(p + steps) // PAGE) for p in prompts)
    print(f"{R} requests, {T} prompt tokens and {steps} decode steps; pages left {left.item()} of {PAGES}; "
          f"attention within {worst:.1e} of plain attention")
    return worst


if __name__ == "__main__":
    main()
