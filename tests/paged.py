"""Seeded paged caches for the tests: pools, tables and lists on the CPU."""
import dataclasses

import torch


@dataclasses.dataclass
class Paged:
    k_cache: torch.Tensor  # [pages, Hk, page, d]
    v_cache: torch.Tensor
    table: torch.Tensor    # int32 [B, max_pages]
    cu: list
    kv_len: list

    @property
    def T(self):
        return self.cu[-1]

    @property
    def max_q(self):
        return max([b - a for a, b in zip(self.cu, self.cu[1:])] + [0])

    def lists(self, device="cuda"):
        return (self.table.to(device), torch.tensor(self.cu, dtype=torch.int32, device=device),
                torch.tensor(self.kv_len, dtype=torch.int32, device=device))


def make_paged(q_lens, kv_lens, Hk, d, page, dtype=torch.bfloat16, seed=0, spare=3, extra_cols=0,
               fill=None, unused=-1):
    """Sequences of kv_lens keys whose last q_lens are new, on shuffled pages.
    Slots outside every sequence hold `fill` (None: random like the rest), and
    table entries past a sequence's pages hold `unused`."""
    g = torch.Generator().manual_seed(seed)
    used = [(n + page - 1) // page for n in kv_lens]
    total = sum(used)
    pages = max(total + spare, 1)
    order = torch.randperm(pages, generator=g).int()
    cols = max(used + [1]) + extra_cols
    table = torch.full((len(kv_lens), cols), unused, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    k = torch.randn(pages, Hk, page, d, generator=g).to(dtype)
    v = torch.randn(pages, Hk, page, d, generator=g).to(dtype)
    if fill is not None:
        live = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(kv_lens):
            for j in range(n):
                live[table[b, j // page], j % page] = True
        for t in (k, v):
            t.transpose(1, 2)[~live] = fill
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    return Paged(k, v, table, cu, list(kv_lens))
