"""A paged cache built on the host, and the cache's operators written out in Python."""
import torch

from gqa_attention_forward_gb300 import binding
from packed_util import DT


def build(lens, page, Hkv, D, dtype, n_layers=1, extra_pages=3, width=None, seed=0, fill=None, n_rows=None):
    """A cache whose row s has lens[s] positions on shuffled pages; the pools hold random values
    (or `fill` everywhere)."""
    h = torch.Generator()
    h.manual_seed(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + extra_pages
    n_rows = len(lens) if n_rows is None else n_rows
    width = (max(need) if need else 0) + 2 if width is None else width
    table = torch.full((n_rows, width), -1, dtype=torch.int32)
    order = torch.randperm(n_pages, generator=h).tolist()
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    shape = (n_layers, n_pages, Hkv, page, D)
    k, v = (torch.randn(shape, generator=g, device="cuda").to(DT[dtype]) if fill is None
            else torch.full(shape, fill, device="cuda", dtype=DT[dtype]) for _ in "kv")
    refs = torch.bincount(table[table >= 0].long(), minlength=n_pages).to(torch.int32)
    all_lens = torch.zeros(n_rows, dtype=torch.int32)
    all_lens[:len(lens)] = torch.tensor(lens, dtype=torch.int32)
    return binding.KVPages(k, v, table.cuda(), all_lens.cuda(), refs.cuda())


def gather(cache, s, layer=0):
    """(K, V) of sequence s, [len, Hkv, D]."""
    n = int(cache.lens[s])
    pos = torch.arange(n, device="cuda")
    at = cache.table[s].long()[pos // cache.page]
    return tuple(x[layer, at, :, pos % cache.page] for x in (cache.k, cache.v))


class Model:
    """The cache's state on the host, and what the operators do to it."""

    def __init__(self, cache):
        self.k, self.v = cache.k.cpu().clone(), cache.v.cpu().clone()
        self.table, self.lens, self.refs = cache.table.tolist(), cache.lens.tolist(), cache.refs.tolist()
        self.page, self.width = cache.page, cache.table_width

    def same(self, cache):
        assert cache.table.tolist() == self.table
        assert cache.lens.tolist() == self.lens
        assert cache.refs.tolist() == self.refs
        bits = torch.int16
        assert torch.equal(cache.k.cpu().view(bits), self.k.view(bits))
        assert torch.equal(cache.v.cpu().view(bits), self.v.view(bits))

    def consistent(self):
        used = [p for r in self.table for p in r if p >= 0]
        assert all(self.refs[p] == used.count(p) for p in range(len(self.refs)))

    def extend(self, seqs, n_new):
        fits = True
        for s, n in zip(seqs, n_new):
            j0, j1 = -(-self.lens[s] // self.page), -(-(self.lens[s] + n) // self.page)
            miss = [j for j in range(j0, j1) if self.table[s][j] < 0]
            fits = fits and self.refs.count(0) >= len(miss)
            if not fits:
                continue
            for j in miss:
                p = self.refs.index(0)
                self.table[s][j] = p
                self.refs[p] = 1
            self.lens[s] += n
        return fits

    def free(self, seqs):
        for s in seqs:
            for p in self.table[s]:
                if p >= 0:
                    self.refs[p] -= 1
            self.table[s] = [-1] * self.width
            self.lens[s] = 0

    def fork(self, parents, children):
        fits = True
        for a, c in zip(parents, children):
            full, rest = divmod(self.lens[a], self.page)
            fits = fits and (rest == 0 or 0 in self.refs)
            if not fits:
                continue
            for j in range(full):
                self.table[c][j] = self.table[a][j]
                self.refs[self.table[a][j]] += 1
            if rest:
                p, old = self.refs.index(0), self.table[a][full]
                self.table[c][full] = p
                self.refs[p] = 1
                self.k[:, p, :, :rest] = self.k[:, old, :, :rest]
                self.v[:, p, :, :rest] = self.v[:, old, :, :rest]
            self.lens[c] = self.lens[a]

    def copy(self, src, dst):
        self.k[:, dst] = self.k[:, src]
        self.v[:, dst] = self.v[:, src]

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        for p in range(live, len(self.refs)):
            if self.refs[p] > 0:
                d = self.refs.index(0)
                self.copy([p], [d])
                self.refs[d], self.refs[p] = self.refs[p], 0
                self.table = [[d if x == p else x for x in r] for r in self.table]
        return live

    def append(self, layer, seqs, k_new, v_new, lens_new):
        at = 0
        for s, n in zip(seqs, lens_new):
            for i in range(n):
                pos = self.lens[s] - n + i
                p, r = self.table[s][pos // self.page], pos % self.page
                self.k[layer, p, :, r] = k_new[at].cpu()
                self.v[layer, p, :, r] = v_new[at].cpu()
                at += 1

    def accept(self, seqs, sizes, paths):
        for s, T, path in zip(seqs, sizes, paths):
            base = self.lens[s] - T
            for j, a in enumerate(path):
                ps, pd = base + a, base + j
                a, b = self.table[s][ps // self.page], self.table[s][pd // self.page]
                self.k[:, b, :, pd % self.page] = self.k[:, a, :, ps % self.page]
                self.v[:, b, :, pd % self.page] = self.v[:, a, :, ps % self.page]
            self.lens[s] = base + len(path)
