"""The cache-page operators, one entry at a time on the CPU (the definition the GPU tests compare with)."""
import torch

PAGE = 16


def pages_of(n):
    return (n + PAGE - 1) // PAGE


class Cache:
    """CPU copies of a cache and its tables; the methods change them as the operators would."""

    def __init__(self, k, v, table, lens, free=(), ks=None, vs=None):
        self.k, self.v, self.table, self.lens = k.clone(), v.clone(), table.clone(), [int(n) for n in lens]
        self.free = [int(p) for p in free]
        self.ks, self.vs = (None, None) if ks is None else (ks.clone(), vs.clone())

    def _copy(self, src, dst, toks):
        for c in (self.k, self.v):
            c[dst, :toks] = c[src, :toks]
        for c in (self.ks, self.vs):
            if c is not None:
                c[dst] = c[src]

    def fork(self, parents, table_out):
        """-> (new lengths, whether a slot found no page); table_out is filled in place."""
        lens, short, seen, asked = [], False, set(), 0
        count = len(self.free)
        for i, p in enumerate(parents):
            n = self.lens[p] if p >= 0 else 0
            used = pages_of(n)
            row = self.table[p, :used].clone() if p >= 0 else None
            if n % PAGE and p in seen:
                asked += 1
                if asked > count:
                    n, used, short = 0, 0, True
                else:
                    fresh = self.free.pop()
                    self._copy(int(row[-1]), fresh, n % PAGE)
                    row[-1] = fresh
            if p >= 0:
                seen.add(p)
            if used:
                table_out[i, :used] = row
            lens.append(n)
        return lens, short

    def append(self, k_new, v_new, cu):
        short, asked, count = False, 0, len(self.free)
        out = list(self.lens)
        for s in range(len(self.lens)):
            n, new = self.lens[s], cu[s + 1] - cu[s]
            need = pages_of(n + new) - pages_of(n)
            asked += need
            if need and asked > count:
                short = True
                continue
            for c in range(pages_of(n), pages_of(n + new)):
                self.table[s, c] = self.free.pop()
            for t in range(new):
                page, slot = int(self.table[s, (n + t) // PAGE]), (n + t) % PAGE
                self.k[page, slot], self.v[page, slot] = k_new[cu[s] + t], v_new[cu[s] + t]
            out[s] = n + new
        return out, short

    def in_use(self):
        used = set()
        for s, n in enumerate(self.lens):
            used.update(int(p) for p in self.table[s, :pages_of(n)])
        return used

    def collect(self):
        used = self.in_use()
        return [p for p in range(self.k.shape[0] - 1, -1, -1) if p not in used]

    def compact(self, table_out):
        used = sorted(self.in_use())
        live = len(used)
        holes = [p for p in range(live) if p not in set(used)]
        new = {p: p for p in used if p < live}
        for p, h in zip([p for p in used if p >= live], holes):
            self._copy(p, h, PAGE)
            new[p] = h
        for s, n in enumerate(self.lens):
            for c in range(pages_of(n)):
                table_out[s, c] = new[int(self.table[s, c])]
        return list(range(self.k.shape[0] - 1, live - 1, -1))


def batch(lens, pages, Hkv, d, seed, width=None, share=0, fp8=False):
    """A cache of random pages whose sequences use scattered ones; with `share`, every sequence starts with the
    first one's first `share` pages.  -> dict of CPU tensors (free pages descending)."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g).tolist()
    width = width or max([pages_of(n) for n in lens] + [1]) + 2
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        used = pages_of(n)
        keep = min(share, n // PAGE) if s and lens[0] >= share * PAGE else 0
        row = table[0, :keep].tolist() + order[at:at + used - keep]
        at += used - keep
        assert at <= pages, "too few pages"
        table[s, :used] = torch.tensor(row, dtype=torch.int32)
    free = sorted(order[at:], reverse=True)
    shape = (pages, PAGE, Hkv, d)
    out = {"table": table, "lens": list(lens), "free": free}
    if fp8:
        out["k"] = torch.randint(0, 256, shape, dtype=torch.uint8, generator=g)
        out["v"] = torch.randint(0, 256, shape, dtype=torch.uint8, generator=g)
        out["ks"], out["vs"] = torch.rand((pages, Hkv), generator=g), torch.rand((pages, Hkv), generator=g)
    else:
        out["k"] = torch.randn(shape, generator=g).to(torch.bfloat16)
        out["v"] = torch.randn(shape, generator=g).to(torch.bfloat16)
        out["ks"] = out["vs"] = None
    return out
