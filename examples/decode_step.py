"""One step of speculative decoding over a sparse-attention model with experts, on the
library's operators: the indexer's scores -> topk -> attention over a 4-bit cache at the selected
positions -> the experts' gate -> verification of the drafted tokens.

The weights are random and small: the example shows how the calls fit together.

    python examples/decode_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import top_selection_gb300 as ds  # noqa: E402

SEQUENCES, DRAFTS, CONTEXT, PAGE = 4, 3, 2000, 64
QUERY_HEADS, HEADS, D, SELECTED = 16, 2, 128, 256
EXPERTS, CHOSEN, VOCABULARY = 64, 6, 5000


class Model:
    def __init__(self, seed=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        width = QUERY_HEADS * D
        self.embed = self.normal(VOCABULARY, width) * 0.2
        self.keys, self.values, self.index = (self.normal(width, HEADS * D) * width ** -0.5,
                                              self.normal(width, HEADS * D) * width ** -0.5,
                                              self.normal(width, D) * width ** -0.5)
        self.gate, self.bias = self.normal(width, EXPERTS) * width ** -0.5, torch.zeros(EXPERTS, device="cuda")
        self.experts = self.normal(EXPERTS, width, 32) * width ** -0.5, self.normal(EXPERTS, 32, width) * 32 ** -0.5
        self.head = self.normal(width, VOCABULARY) * width ** -0.5
        pages = -(-(CONTEXT + 64) // PAGE)
        self.cache = torch.zeros(SEQUENCES * pages, HEADS, PAGE, 2, D // 2, dtype=torch.uint8, device="cuda")
        self.scales = torch.zeros(SEQUENCES * pages, HEADS, PAGE, 4, dtype=torch.bfloat16, device="cuda")
        self.table = torch.randperm(SEQUENCES * pages, device="cuda", generator=self.g).view(SEQUENCES, pages).int()
        self.index_keys = torch.zeros(SEQUENCES, pages * PAGE, D, device="cuda")
        self.lens = torch.zeros(SEQUENCES, dtype=torch.int32, device="cuda")

    def normal(self, *shape):
        return torch.randn(*shape, device="cuda", generator=self.g)

    def forward(self, tokens):
        """tokens (sequences, n), new behind the stored ones -> logits (sequences, n, vocabulary)."""
        B, n = tokens.shape
        x = self.embed[tokens.long()]
        at = self.lens[:, None].long() + torch.arange(n, device="cuda")
        # the new tokens' keys and values go to the cache, in 4 bits
        slots = self.table.gather(1, (at // PAGE)).int() * PAGE + (at % PAGE).int()
        k = (x @ self.keys).bfloat16().view(B * n, HEADS, D)
        v = (x @ self.values).bfloat16().view(B * n, HEADS, D)
        ds.cache_store(k, v, self.cache, self.scales, slots.view(-1))
        self.index_keys[torch.arange(B, device="cuda")[:, None], at] = x @ self.index
        self.lens += n
        # the indexer scores every position for each token; the top-k selects
        scores = (x @ self.index) @ self.index_keys.transpose(1, 2)
        ends = at + 1
        scores.masked_fill_(torch.arange(scores.shape[-1], device="cuda") >= ends[..., None], float("-inf"))
        k_sel = min(SELECTED, scores.shape[-1])
        _, picked = ds.topk(scores.view(B * n, -1).bfloat16(), k_sel, 0, 0)
        y, _ = ds.cache_attention(x.bfloat16().view(B, n, QUERY_HEADS, D), self.cache, self.scales, self.table, self.lens,
                                  indices=picked.view(B, n, k_sel))
        x = x + y.float().view(B, n, -1)
        # the gate and its experts
        rows = x.view(B * n, -1)
        weights, chosen = ds.route(rows @ self.gate, CHOSEN, scoring="sigmoid", bias=self.bias, groups=8, topk_groups=4,
                                   group_score="top2")
        up, down = self.experts
        hidden = torch.relu(torch.einsum("rw,rkwh->rkh", rows, up[chosen.long()]))
        x = x + torch.einsum("rk,rkh,rkhw->rw", weights, hidden, down[chosen.long()]).view_as(x)
        return x @ self.head

    def step(self, last, drafts, temperature):
        """Verifies `drafts` (sequences, n) behind the token `last` (sequences,): returns the emitted
        tokens, how many drafts were accepted, and leaves the cache behind the accepted ones."""
        stored = self.lens.clone()
        logits = self.forward(torch.cat([last[:, None], drafts], 1))
        u = torch.rand(drafts.shape, device="cuda", generator=self.g)
        noise = torch.empty(drafts.shape[0], VOCABULARY, device="cuda").exponential_(generator=self.g)
        tokens, accepted, probs = ds.verify_drafts(logits, drafts, u, noise, temperature=temperature)
        self.lens = stored + 1 + accepted  # what lies behind is written over by the next step
        return tokens, accepted, probs


def main(steps=8, seed=0):
    model = Model(seed)
    prompt = torch.randint(VOCABULARY, (SEQUENCES, CONTEXT), device="cuda", generator=model.g).int()
    for i in range(0, CONTEXT, 250):
        model.forward(prompt[:, i:i + 250])
    last, emitted = prompt[:, -1], torch.zeros(SEQUENCES, dtype=torch.int64, device="cuda")
    temperature = torch.tensor([0.0, 0.8] * (SEQUENCES // 2), device="cuda")  # every other sequence is greedy
    for _ in range(steps):
        drafts = torch.randint(VOCABULARY, (SEQUENCES, DRAFTS), device="cuda", generator=model.g).int()
        # a lucky drafter: its first guess is the token the model finds likeliest
        drafts[:, 0] = model_guess(model, last)
        tokens, accepted, _ = model.step(last, drafts, temperature)
        last = tokens.gather(1, accepted[:, None].long())[:, 0]
        emitted += accepted + 1
    assert ds.ds_get_device_status() == 0
    return emitted, model.lens


def model_guess(model, last):
    """The likeliest next token, from a look ahead whose cache entries are dropped again."""
    stored = model.lens.clone()
    guess = model.forward(last[:, None])[:, 0].argmax(-1).int()
    model.lens = stored
    return guess


if __name__ == "__main__":
    emitted, lens = main()
    print("tokens emitted per sequence:", emitted.tolist(), "context:", lens.tolist())
