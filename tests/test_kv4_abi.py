"""Host-side refusals of the 4-bit cache, accumulated-weight and eviction entry points, and of their
Python wrappers: no kernel is launched here."""
import ctypes

import pytest
import torch

from sparse_kv_recall_b200 import build as B
from sparse_kv_recall_b200 import oda

I, U, W, OK = (oda.ODA_ERR_INVALID_ARG, oda.ODA_ERR_UNSUPPORTED_SHAPE, oda.ODA_ERR_WORKSPACE_TOO_SMALL,
               oda.ODA_OK)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return oda.load()


def _kv4(**kw):
    base = dict(cache=0x10000, block_table=0x30000, seq_lens=0x40000, batch=2, num_kv_heads=8, head_dim=128,
                block_size=16, max_blocks_per_seq=64, num_blocks=128, dev_status=None, stats=None)
    base.update(kw)
    return oda.oda_kv4(**base)


def _kv(**kw):
    base = dict(k_cache=0x10000, v_cache=0x20000, block_table=0x30000, seq_lens=0x40000, batch=2,
                num_kv_heads=8, head_dim=128, block_size=16, max_blocks_per_seq=64, num_blocks=128,
                dev_status=None, stats=None)
    base.update(kw)
    return oda.oda_kv(**base)


FULL = oda.oda_visibility(mode=oda.ODA_MODE_FULL, window=1)


def test_append_and_read_checks(lib):
    def append(kv=None, k=0x1000, v=0x2000, ks=1024, vs=1024, n=2, cu=None, gate=None):
        return lib.oda_kv4_append(ctypes.byref(kv or _kv4()), k, v, ks, vs, n, cu, gate, None)

    def read(kv=None, k=0x1000, v=0x2000, dtype=0, n=2, cu=None):
        return lib.oda_kv4_read(ctypes.byref(kv or _kv4()), k, v, dtype, n, cu, None)
    assert lib.oda_kv4_append(None, 0x1000, 0x2000, 1024, 1024, 2, None, None, None) == I
    for call in (append, read):
        assert call(kv=_kv4(head_dim=64)) == U and call(kv=_kv4(block_size=32)) == U
        assert call(kv=_kv4(cache=0x10008)) == I and call(kv=_kv4(cache=None)) == I
        assert call(k=None) == I and call(v=0x2008) == I
        assert call(n=3) == I and call(n=-1, cu=0x5000) == I and call(n=3, cu=0x5002) == I
        assert call(n=0, cu=0x5000) == OK and call(kv=_kv4(batch=0), n=0) == OK
        assert call(n=0x7fff0001, cu=0x5000) == U
    assert append(ks=1023) == I and append(vs=1028) == I and append(ks=1016) == I and append(gate=0x5002) == I
    assert read(dtype=3) == I


def test_decode_checks(lib):
    def call(kv=None, vis=FULL, hq=16, scale=0.1, k_new=None, v_new=None, out=0x50000, dtype=0, ws=0x60000,
             nbytes=1 << 40, q=0x70000, lse=None):
        return lib.oda_kv4_decode(ctypes.byref(kv or _kv4()), ctypes.byref(vis) if vis is not None else None, q,
                                  hq, scale, k_new, v_new, out, dtype, lse, ws, nbytes, None)
    assert call(vis=None) == I
    assert call(hq=12) == U and call(hq=64) == U and call(hq=24) == U
    assert call(scale=0.0) == I and call(scale=float("nan")) == I and call(dtype=2) == I
    assert call(k_new=0x1000) == I and call(k_new=0x1008, v_new=0x2000) == I
    assert call(q=0x70008) == I and call(out=None) == I and call(ws=0x60004) == I and call(lse=0x1002) == I
    assert call(out=0x50002) == I and call(out=0x50001, dtype=1) == I
    assert call(vis=oda.oda_visibility(mode=oda.ODA_MODE_LOCAL, sink=0, window=0)) == I
    keep = oda.oda_visibility(mode=oda.ODA_MODE_KEEP, window=1, keep_blocks=0x1000, keep_counts=0x2000, max_keep=4)
    assert call(vis=keep, k_new=0x1000, v_new=0x2000) == I
    assert call(kv=_kv4(batch=0)) == OK and call(kv=_kv4(batch=1025)) == U
    n = ctypes.c_size_t(0)
    assert lib.oda_kv4_decode_workspace_size(2, 8, 12, ctypes.byref(n)) == U
    assert lib.oda_kv4_decode_workspace_size(2, 8, 24, ctypes.byref(n)) == U
    assert lib.oda_kv4_decode_workspace_size(2, 0, 16, ctypes.byref(n)) == I
    assert lib.oda_kv4_decode_workspace_size(2, 8, 16, None) == I


@pytest.mark.parametrize("name,make", [("oda_decode_mass", _kv), ("oda_kv4_decode_mass", _kv4)])
def test_decode_mass_checks(lib, name, make):
    def call(kv=None, vis=FULL, hq=16, mass_in=None, mass_out=0x80000, tokens=1024, ws=0x60000):
        return getattr(lib, name)(ctypes.byref(kv or make()), ctypes.byref(vis) if vis is not None else None,
                                  0x70000, hq, 0.1, None, None, 0x50000, 0, None, mass_in, mass_out, tokens, ws,
                                  1 << 40, None)
    assert call(vis=None) == I and call(hq=12) == U
    assert call(tokens=1023) == I and call(tokens=1008) == I and call(tokens=1026) == I
    assert call(mass_out=None) == I and call(mass_out=0x80004) == I and call(mass_in=0x90008) == I
    assert call(ws=0x60001) == I and call(kv=make(batch=0)) == OK
    assert call(kv=make(max_blocks_per_seq=1 << 27, num_kv_heads=4, batch=1), tokens=1 << 31) == U
    assert call(kv=make(max_blocks_per_seq=(1 << 27) - 1, num_kv_heads=4, batch=1), tokens=1 << 31) == U
    n = ctypes.c_size_t(0)
    size = getattr(lib, name + "_workspace_size")
    assert size(2, 8, 16, 0, ctypes.byref(n)) == I and size(2, 8, 12, 4, ctypes.byref(n)) == U
    assert size(2, 8, 24, 4, ctypes.byref(n)) == U and size(2, 8, 16, 4, None) == I


@pytest.mark.parametrize("name,make", [("oda_kv_evict", _kv), ("oda_kv4_evict", _kv4)])
def test_evict_checks(lib, name, make):
    def call(kv=None, mass=0x80000, tokens=1024, sink=4, recent=16, budget=64, gate=None, dst=0x90000, blocks=4,
             kept=0xa0000, mass_out=0xb0000, lens=0xc0000, ws=0xd0000, nbytes=512):
        return getattr(lib, name)(ctypes.byref(kv or make()), mass, tokens, sink, recent, budget, gate, dst, blocks,
                                  kept, mass_out, lens, ws, nbytes, None)
    assert getattr(lib, name)(None, *[0] * 4, 64, None, None, 4, None, None, None, None, 0, None) == I
    assert call(sink=-1) == I and call(recent=-1) == I and call(budget=0, sink=0, recent=0) == I
    assert call(sink=60, recent=5) == I and call(sink=2 ** 31 - 1, recent=2 ** 31 - 1) == I
    assert call(tokens=1008) == I and call(blocks=3) == I and call(blocks=0) == I
    assert call(dst=0x30000, blocks=4) == I                 # in place: the table's own row length
    for null in ("mass", "dst", "kept", "mass_out", "lens", "ws"):
        assert call(**{null: None}) == I
    assert call(mass=0x80002) == I and call(gate=0x2002) == I and call(kept=0xa0001) == I and call(ws=0xd0004) == I
    assert call(nbytes=4) == W
    assert call(kv=make(max_blocks_per_seq=(1 << 27) - 1, num_kv_heads=4, batch=1), tokens=1 << 31) == U
    assert call(budget=2 ** 31 - 1, blocks=1 << 27) == U
    assert call(kv=make(batch=0)) == OK and call(kv=make(num_blocks=0)) == I
    n = ctypes.c_size_t(0)
    assert lib.oda_kv_evict_workspace_size(-1, ctypes.byref(n)) == I
    assert lib.oda_kv_evict_workspace_size(3, None) == I
    assert lib.oda_kv_evict_workspace_size(3, ctypes.byref(n)) == OK and n.value >= 12


def test_wrappers_refuse_host_tensors_and_wrong_shapes():
    """Shapes are checked before any pointer is taken; a host tensor never reaches the library."""
    kv = _kv4(batch=2, num_kv_heads=2)
    bf = torch.bfloat16
    rows = torch.zeros(2, 2, 128, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        oda.oda_kv4_append(kv, rows, rows)
    with pytest.raises(ValueError, match="shape"):
        oda.oda_kv4_append(kv, torch.zeros(2, 3, 128, dtype=bf), rows)
    with pytest.raises(ValueError, match="one row per sequence"):
        oda.oda_kv4_read(kv, torch.zeros(3, 2, 128), torch.zeros(3, 2, 128))
    with pytest.raises(ValueError, match="one dtype"):
        oda.oda_kv4_read(kv, torch.zeros(2, 2, 128), rows)
    with pytest.raises(ValueError, match="shape"):
        oda.oda_kv4_decode(kv, FULL, torch.zeros(3, 4, 128, dtype=bf), 0.1, torch.zeros(3, 4, 128), torch.zeros(8))
    with pytest.raises(ValueError, match="shape"):
        oda.oda_decode_mass(kv, FULL, torch.zeros(2, 4, 128, dtype=bf), 0.1, torch.zeros(2, 4, 128),
                            torch.zeros(8), torch.zeros(2, 3, 64))
    with pytest.raises(ValueError, match="kept"):
        oda.oda_kv4_evict(kv, torch.zeros(2, 2, 64), 0, 0, 32, torch.zeros(2, 2), torch.zeros(2, 2, 31),
                          torch.zeros(2, 2, 64), torch.zeros(2), torch.zeros(8))
    with pytest.raises(ValueError, match="2304"):
        oda.make_kv4(torch.zeros(2, 2, 2048, dtype=torch.uint8), torch.zeros(2, 2), torch.zeros(2))


def test_make_kv4_refuses_tables_that_do_not_fit():
    """Lengths, status and counters are read and written by the batch, on the cache's device."""
    cache, table, lens = (torch.zeros(2, 2, 2304, dtype=torch.uint8), torch.zeros(3, 4, dtype=torch.int32),
                          torch.zeros(3, dtype=torch.int32))
    for bad in (lens[:2], lens.view(3, 1), torch.zeros((), dtype=torch.int32)):
        with pytest.raises(ValueError, match="seq_lens"):
            oda.make_kv4(cache, table, bad)
    with pytest.raises(ValueError, match="block_table"):
        oda.make_kv4(cache, table[0], lens)
    with pytest.raises(ValueError, match="dev_status"):
        oda.make_kv4(cache, table, lens, dev_status=torch.zeros(0, dtype=torch.int32))
    with pytest.raises(ValueError, match="stats"):
        oda.make_kv4(cache, table, lens, stats=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="device"):
        oda.make_kv4(cache, table, lens.to("meta"))
    with pytest.raises(ValueError, match="CUDA"):
        oda.make_kv4(cache, table, lens)
