"""Helpers of the 4-bit cache, accumulated-weight and eviction tests: seeded caches of either kind with
their host copies, and the oracle evaluated on them.

Tolerances. Scores of the inputs here are at most about 16 in base 2; the dot product's fp32 sums and
the scale and minimum products leave them a few ulp (8 x 2^-24 x 16 = 8e-6) off, the base-2 exponential
two ulp more, and the weight times the V scale is held in two fp16 (2^-22): 1.5e-5 relative on a weight
at the most. An output is a weighted mean of values of at most 5, so it is off by at most 8e-5 (MAX),
and by the mean of far smaller and independent errors (MEAN). A bf16 output adds half a step,
2^-8 of the value. The log-sum is held to the bound of the bf16 decode tests. A position's mass is a sum
of at most four weights, each at most 1: 4 x 1.5e-5 (MASS), plus the fp32 rounding of the sum with what
was there before (2^-24 of it)."""
import numpy as np
import torch

import oda_synth
from oda_cases import SCALE, assert_lse_close  # noqa: F401
from oracle import kv4_oracle as K
from oracle import oda_oracle as O
from sparse_kv_recall_b200 import oda

MAX, MEAN, MASS = 1e-4, 1e-5, 6e-5


def assert_out_close(got, ref, what=""):
    bf16 = got.dtype == torch.bfloat16
    got = got.double().cpu().numpy()
    d = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    room = np.abs(ref) * 2.0 ** -8 if bf16 else 0.0
    assert np.all(d <= MAX + room), "%s max|d| = %g" % (what, d.max())
    if not bf16:
        assert d.mean() <= MEAN, "%s mean|d| = %g" % (what, d.mean())


def gauss(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


class PagedCase:
    """Sequences of given lengths over a cache of either kind whose pages are a random permutation,
    filled with N(0, 1) rows (4-bit: appended through the library)."""

    def __init__(self, lengths, hq, hkv, seed, kv4=True, spare=0, rows=None):
        self.lengths, self.hq, self.hkv, self.kv4 = list(lengths), hq, hkv, kv4
        self.B, self.G = len(lengths), hq // hkv
        pages = [max(1, -(-n // 16)) for n in lengths]
        self.maxb = max(pages)
        self.num_blocks = sum(pages) + spare
        perm = torch.randperm(self.num_blocks, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        bt = torch.full((self.B, self.maxb), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            bt[b, :n] = perm[at:at + n]
            at += n
        self.spare = perm[at:].cuda()
        self.bt = bt.cuda()
        self.seq_lens = torch.tensor(self.lengths, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.stats = torch.zeros(oda.ODA_STATS_LEN, dtype=torch.int64, device="cuda")
        total = sum(self.lengths)
        k, v = rows if rows is not None else (gauss((total, hkv, 128), seed + 1), gauss((total, hkv, 128), seed + 2))
        if kv4:
            g = torch.Generator(device="cuda").manual_seed(seed + 3)   # what is never written: any bytes
            self.cache = torch.randint(0, 256, (self.num_blocks, hkv, oda.ODA_KV4_PAGE_BYTES), generator=g,
                                       dtype=torch.uint8, device="cuda")
            self.kv = oda.make_kv4(self.cache, self.bt, self.seq_lens, self.status, self.stats)
            cu = torch.tensor(np.concatenate([[0], np.cumsum(self.lengths)]), dtype=torch.int32, device="cuda")
            oda.oda_kv4_append(self.kv, k, v, cu_rows=cu)
        else:
            shape = (self.num_blocks, hkv, 16, 128)
            self.kc = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            self.vc = self.kc.clone()
            at = 0
            for b, n in enumerate(self.lengths):
                p = torch.arange(n, device="cuda")
                page = self.bt[b].long()[p // 16]
                self.kc[page, :, p % 16] = k[at:at + n]
                self.vc[page, :, p % 16] = v[at:at + n]
                at += n
            self.kv = oda.make_kv(self.kc, self.vc, self.bt, self.seq_lens, self.status, self.stats)
        self.q = gauss((self.B, hq, 128), seed + 4)
        self.k_new, self.v_new = gauss((self.B, hkv, 128), seed + 5), gauss((self.B, hkv, 128), seed + 6)
        size = oda.oda_kv4_decode_mass_workspace_size if kv4 else oda.oda_decode_mass_workspace_size
        self.ws = torch.zeros(size(self.B, hkv, hq, self.maxb), dtype=torch.uint8, device="cuda")
        self.snapshot()

    def snapshot(self):
        """Host values of every slot, fp64 [pages][Hkv][16][128]."""
        torch.cuda.synchronize()
        if self.kv4:
            self.k, self.v = K.unpack_pages(self.cache.cpu().numpy())
        else:
            self.k, self.v = (c.double().cpu().numpy() for c in (self.kc, self.vc))
        self.bt_h = self.bt.cpu().numpy()

    def raw(self):
        return self.cache.clone() if self.kv4 else torch.stack([self.kc, self.vc]).view(torch.int16).clone()

    def rows(self, b, g, pos, which=None):
        pos = np.asarray(pos, dtype=np.int64)
        page = self.bt_h[b][pos // 16]
        return self.k[page, g, pos % 16], self.v[page, g, pos % 16]

    def out(self, dtype=torch.float32, fill=float("nan")):
        return (torch.full((self.B, self.hq, 128), fill, dtype=dtype, device="cuda"),
                torch.full((self.B, self.hq), fill, dtype=torch.float32, device="cuda"))

    def ok(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0, oda.oda_status_string(int(self.status.item()))

    def oracle(self, positions_of, commit=False):
        """out, lse and per-sequence (positions, mass [Hkv][n]) over positions_of(b, t), in fp64."""
        q = self.q.double().cpu().numpy()
        out, lse, mass = np.zeros((self.B, self.hq, 128)), np.zeros((self.B, self.hq)), []
        if commit:
            kn, vn = (K.round_trip(x.double().cpu().numpy()) if self.kv4 else x.double().cpu().numpy()
                      for x in (self.k_new, self.v_new))
        for b, n in enumerate(self.lengths):
            pos = np.asarray(positions_of(b, n - 1), dtype=np.int64)
            ks, vs = [], []
            for g in range(self.hkv):
                k, v = self.rows(b, g, pos)
                if commit and pos.size and pos[-1] == n - 1:
                    k, v = k.copy(), v.copy()
                    k[-1], v[-1] = kn[b, g], vn[b, g]
                ks.append(k)
                vs.append(v)
            out[b], lse[b] = O.decode_attention(q[b], ks, vs, SCALE)
            mass.append((pos, K.attention_mass(q[b], ks, SCALE, self.G)))
        return out, lse, mass


def full(gate=None):
    v = oda.oda_visibility(mode=oda.ODA_MODE_FULL, window=1, gate=None if gate is None else gate.data_ptr())
    v._refs = (gate,)
    return v


def local(sink, window):
    return oda.oda_visibility(mode=oda.ODA_MODE_LOCAL, sink=sink, window=window)


def keep(blocks, counts):
    v = oda.oda_visibility(mode=oda.ODA_MODE_KEEP, window=1, keep_blocks=blocks.data_ptr(),
                           keep_counts=counts.data_ptr(), max_keep=blocks.shape[1])
    v._refs = (blocks, counts)
    return v


def keep_lists(lengths, maxb, seed, empty=()):
    """Random ascending page lists; -1 padding. (device blocks, device counts, host lists)"""
    r = np.random.default_rng(seed)
    lists = []
    for b, n in enumerate(lengths):
        last = (n - 1) // 16
        pick = np.sort(r.choice(last + 1, size=int(r.integers(1, last + 2)), replace=False))
        lists.append(np.zeros(0, dtype=np.int64) if b in empty else pick)
    blocks = np.full((len(lengths), maxb), -1, dtype=np.int32)
    for b, x in enumerate(lists):
        blocks[b, :len(x)] = x
    return (torch.from_numpy(blocks).cuda(), torch.tensor([len(x) for x in lists], dtype=torch.int32, device="cuda"),
            lists)
