"""The 4-bit KV cache on the GPU: append and read against the oracle's quantiser bit for bit, decode
attention over it under every visibility rule against the fp64 oracle on the values it holds, the
fused commit, hidden garbage, extreme ranges, device-side errors, streams and graph capture."""
import numpy as np
import pytest
import torch

from kv4_cases import (SCALE, PagedCase, assert_lse_close, assert_out_close, full, gauss, keep, keep_lists, local)
from oracle import kv4_oracle as K
from oracle import oda_oracle as O
from sparse_kv_recall_b200 import build as B
from sparse_kv_recall_b200 import oda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    B.build()
    oda.load()


def _read_all(c, dtype=torch.float32):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(c.lengths)]), dtype=torch.int32, device="cuda")
    k = torch.full((sum(c.lengths), c.hkv, 128), -7.0, dtype=dtype, device="cuda")
    v = k.clone()
    oda.oda_kv4_read(c.kv, k, v, cu_rows=cu)
    c.ok()
    return k, v


@pytest.mark.parametrize("hkv,lengths", [(8, [1, 15, 16, 17, 40]), (1, [5]), (3, [2, 33, 1]), (40, [3, 18])])
def test_append_and_read_match_the_oracle_exactly(hkv, lengths):
    rows = [gauss((sum(lengths), hkv, 128), 50 + i, 3.0) + (2 if i else 0) for i in range(2)]
    c = PagedCase(lengths, hkv, hkv, seed=hkv, rows=rows)
    k, v = _read_all(c)
    for got, want in zip((k, v), rows):
        ref = K.round_trip(want.double().cpu().numpy())
        assert np.array_equal(got.cpu().numpy(), ref.astype(np.float32))
    k16, _ = _read_all(c, torch.bfloat16)
    assert torch.equal(k16, k.to(torch.bfloat16))
    at = 0                                         # and the layout is the documented one
    for b, n in enumerate(lengths):
        for g in range(hkv):
            assert np.array_equal(c.rows(b, g, np.arange(n))[0].astype(np.float32), k[at:at + n, g].cpu().numpy())
        at += n


def test_append_and_read_of_many_rows_take_eight_at_a_time():
    """Enough (row, KV head) pairs for the warps of eight, an odd number of them, sequences that end inside
    such a group, one gated off."""
    lengths, hkv = [3000, 1, 17, 8192, 5, 250], 7
    n = sum(lengths)
    assert n * hkv > 8 * 8 * 148 and n * hkv % 8 != 0
    rows = [gauss((n, hkv, 128), 55 + i, 2.0) - i for i in range(2)]
    c = PagedCase(lengths, hkv, hkv, seed=57, rows=rows)
    k, v = _read_all(c)
    ref = [K.round_trip(x.double().cpu().numpy()).astype(np.float32) for x in rows]
    assert np.array_equal(k.cpu().numpy(), ref[0]) and np.array_equal(v.cpu().numpy(), ref[1])
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    gate = torch.tensor([1, 0, 1, 0, 1, 1], dtype=torch.int32, device="cuda")
    oda.oda_kv4_append(c.kv, rows[1], rows[0], cu_rows=cu, gate=gate)
    k, v = _read_all(c)
    at = 0
    for b, m in enumerate(lengths):
        r = slice(at, at + m)
        kk, vv = (ref[1], ref[0]) if b not in (1, 3) else (ref[0], ref[1])
        assert np.array_equal(k[r].cpu().numpy(), kk[r]) and np.array_equal(v[r].cpu().numpy(), vv[r])
        at += m


def test_append_takes_rows_out_of_a_fused_projection_and_leaves_the_rest():
    """Strided rows; ranges that are empty, shorter than the sequence, and rows behind the last range
    or gated off: every other byte of the cache keeps its contents."""
    lengths, hkv = [40, 7, 100, 33], 4
    c = PagedCase(lengths, 8, hkv, seed=21)
    before = c.raw()
    cu = [0, 3, 3, 3 + 37, 3 + 37 + 33]
    qkv = gauss((cu[-1] + 5, 8 + 2 * hkv, 128), 22)
    k, v = qkv[:, 8:8 + hkv], qkv[:, 8 + hkv:]
    gate = torch.tensor([1, 1, 1, 0], dtype=torch.int32, device="cuda")
    oda.oda_kv4_append(c.kv, k, v, cu_rows=torch.tensor(cu, dtype=torch.int32, device="cuda"), gate=gate)
    c.ok()
    changed = (c.raw() != before).any(-1).cpu().numpy()            # [page][head]
    want_k, want_v = (K.round_trip(x.double().cpu().numpy()) for x in (k, v))
    old_k = c.k.copy()
    c.snapshot()
    touched = set()
    for b, n in enumerate(lengths):
        m = cu[b + 1] - cu[b]
        if b == 3:
            continue
        for i in range(m):
            p = n - m + i
            page = c.bt_h[b, p // 16]
            touched.add((int(page), p % 16))
            assert np.array_equal(c.k[page, :, p % 16], want_k[cu[b] + i])
            assert np.array_equal(c.v[page, :, p % 16], want_v[cu[b] + i])
    assert set(np.nonzero(changed.any(1))[0].tolist()) <= {p for p, _ in touched}
    for page in range(c.num_blocks):
        for row in range(16):
            if (page, row) not in touched:
                assert np.array_equal(c.k[page, :, row], old_k[page, :, row], equal_nan=True)


def test_append_one_row_per_sequence_is_slot_t():
    c = PagedCase([1, 16, 17, 50], 8, 4, seed=23)
    oda.oda_kv4_append(c.kv, c.k_new, c.v_new)
    k, v = torch.empty(4, 4, 128, device="cuda"), torch.empty(4, 4, 128, device="cuda")
    oda.oda_kv4_read(c.kv, k, v)
    c.ok()
    assert np.array_equal(k.cpu().numpy(), K.round_trip(c.k_new.double().cpu().numpy()).astype(np.float32))
    c.snapshot()
    for b, n in enumerate(c.lengths):
        assert np.array_equal(c.v[c.bt_h[b, (n - 1) // 16], :, (n - 1) % 16], v[b].double().cpu().numpy())


def test_append_special_groups():
    """Constant groups, whole-number spans, subnormals, the largest finite values, infinities and NaN;
    only the group that holds one of the last is lost."""
    x = gauss((8, 1, 128), 24).double().cpu()
    big = float(torch.finfo(torch.bfloat16).max)
    x[0, 0, :64] = 3.0
    x[1, 0, 64:] = torch.arange(64).double() % 16
    x[2, 0, :64] = torch.arange(64).double() * 2.0 ** -133
    x[3, 0, :64] = torch.linspace(0, 1, 64, dtype=torch.float64) * big
    x[4, 0, 5] = float("inf")
    x[5, 0, 100] = float("nan")
    x[6, 0, 0], x[6, 0, 1] = big, -big              # spans more than the largest fp32
    x[7, 0, :] = 0.0
    rows = x.to(torch.bfloat16).cuda()
    c = PagedCase([8], 1, 1, seed=25, rows=(rows, rows))
    k, _ = _read_all(c)
    ref = K.round_trip(rows.double().cpu().numpy())
    assert np.array_equal(k.cpu().numpy(), ref.astype(np.float32), equal_nan=True)
    nan = np.isnan(ref[:, 0]).reshape(8, 2, 64).all(-1)
    assert nan.tolist() == [[False] * 2] * 4 + [[True, False], [False, True], [True, False], [False] * 2]


@pytest.mark.parametrize("kind", range(6))
def test_append_rounds_as_the_division_does(kind):
    """Quotients at and beside halves: whole numbers and halves over spans of every kind, an offset, scales
    down to the subnormal ones, by single rows and by eight at a time."""
    for n in (40, 1500):
        g = torch.Generator(device="cuda").manual_seed(200 + kind)
        shape = (n, 8, 128)
        x = torch.randint(0, 31, shape, generator=g, device="cuda").double() / 2
        if kind == 1:
            x = torch.randint(-40, 40, shape, generator=g, device="cuda").double()
        if kind == 2:
            x = torch.randint(0, 2000, shape, generator=g, device="cuda").double() / 64
        if kind == 3:
            x = x + 100
        if kind >= 4:
            x = torch.randn(shape, generator=g, device="cuda").double()
            x = x * 2.0 ** torch.randint(*((-133, -90) if kind == 4 else (-90, 120)), (n, 8, 1), generator=g,
                                         device="cuda").double()
        rows = (x.to(torch.bfloat16), x.flip(0).to(torch.bfloat16))
        c = PagedCase([n], 8, 8, seed=210, rows=rows)
        k, v = _read_all(c)
        for got, want in zip((k, v), rows):
            ref = K.round_trip(want.double().cpu().numpy())
            assert np.array_equal(got.cpu().numpy(), ref.astype(np.float32))


def test_append_and_read_report_bad_sequences():
    c = PagedCase([20, 20, 20], 8, 4, seed=26, spare=1)
    before = c.raw()
    cu = torch.tensor([0, 21, 22, 23], dtype=torch.int32, device="cuda")    # more rows than tokens
    c.bt[1, 1] = c.num_blocks                                               # no such page
    rows = gauss((23, 4, 128), 27)
    oda.oda_kv4_append(c.kv, rows, rows, cu_rows=cu)
    torch.cuda.synchronize()
    assert int(c.status.item()) in (oda.ODA_DEV_BAD_LEN, oda.ODA_DEV_BAD_BLOCK)
    changed = (c.raw() != before).flatten(1).any(1).nonzero()[:, 0].tolist()
    assert changed == [int(c.bt[2, 1])]                                     # sequence 2 alone was written
    c.status.zero_()
    c.seq_lens[0] = 0
    out = torch.full((23, 4, 128), 5.0, device="cuda")
    oda.oda_kv4_read(c.kv, out, out.clone(), cu_rows=cu)
    torch.cuda.synchronize()
    assert int(c.status.item()) != 0
    assert (out[:22] == 5.0).all() and not (out[22] == 5.0).all()


LENS = [1, 2, 15, 16, 17, 33, 300, 2053]


@pytest.mark.parametrize("G,hkv", [(1, 8), (2, 8), (4, 8), (2, 1), (4, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_full_matches_oracle(G, hkv, dtype):
    c = PagedCase(LENS + [5000], G * hkv, hkv, seed=30 + G)
    out, lse = c.out(dtype)
    oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, out, c.ws, lse=lse)
    c.ok()
    ref, rlse, _ = c.oracle(lambda b, t: O.full_positions(t))
    assert_out_close(out, ref, "G=%d" % G)
    assert_lse_close(lse.cpu().numpy(), rlse)
    st = c.stats.cpu().numpy()
    assert st[oda.ODA_STAT_ROWS] == hkv * sum(c.lengths)
    assert st[oda.ODA_STAT_PAGES] == hkv * sum((n + 15) // 16 for n in c.lengths)


@pytest.mark.parametrize("G", [1, 2, 4])
@pytest.mark.parametrize("sink,window", [(4, 256), (0, 1), (7, 33), (20, 100), (0, 2048), (16, 16)])
def test_local_with_commit_matches_oracle(G, sink, window):
    c = PagedCase(LENS + [4100], 4 * G, 4, seed=40 + G + sink)
    before = c.raw()
    out, lse = c.out()
    oda.oda_kv4_decode(c.kv, local(sink, window), c.q, SCALE, out, c.ws, k_new=c.k_new, v_new=c.v_new, lse=lse)
    c.ok()
    pos = lambda b, t: O.local_positions(t, sink, window)
    ref, rlse, _ = c.oracle(pos, commit=True)
    assert_out_close(out, ref, "s=%d w=%d" % (sink, window))
    assert_lse_close(lse.cpu().numpy(), rlse)
    assert c.stats[oda.ODA_STAT_ROWS].item() == 4 * sum(len(pos(b, n - 1)) for b, n in enumerate(c.lengths))
    again = PagedCase(c.lengths, 4 * G, 4, seed=40 + G + sink)     # the commit is what append writes
    assert torch.equal(again.raw(), before)
    oda.oda_kv4_append(again.kv, c.k_new, c.v_new)
    again.ok()
    assert torch.equal(again.raw(), c.raw())


@pytest.mark.parametrize("G", [1, 2, 4])
def test_keep_lists_match_oracle(G):
    lens = [1, 40, 333, 2053, 700]
    c = PagedCase(lens, 4 * G, 4, seed=50)
    blocks, counts, lists = keep_lists(lens, c.maxb, 51, empty=(4,))
    out, lse = c.out()
    oda.oda_kv4_decode(c.kv, keep(blocks, counts), c.q, SCALE, out, c.ws, lse=lse)
    c.ok()
    ref, rlse, _ = c.oracle(lambda b, t: O.keep_positions(t, lists[b]))
    assert_out_close(out, ref)
    assert_lse_close(lse.cpu().numpy(), rlse)
    assert (out[4] == 0).all() and torch.isinf(lse[4]).all()       # an empty visible set


def test_declared_modes_and_shards_match_oracle():
    lens = [5000, 9000, 300, 40]
    c = PagedCase(lens, 16, 4, seed=52)
    modes = torch.tensor([1, 1, 2, 0], dtype=torch.int32, device="cuda")
    offs = torch.tensor([1000, 17, 0, 0], dtype=torch.int32, device="cuda")
    vis = oda.da_visibility(modes, offs, focus_len=700, recent=100, local_len=64)
    out, lse = c.out()
    oda.oda_kv4_decode(c.kv, vis, c.q, SCALE, out, c.ws, lse=lse)
    c.ok()
    ref, rlse, _ = c.oracle(lambda b, t: O.da_mode_positions(int(modes[b]), t, int(offs[b]), focus_len=700,
                                                             recent=100, local_len=64))
    assert_out_close(out, ref)
    assert_lse_close(lse.cpu().numpy(), rlse)
    parts, lses = [], []
    for lo, hi in [(0, 256), (256, 4096), (4096, 1 << 20)]:
        o, l = c.out()
        oda.oda_kv4_decode(c.kv, oda.shard_visibility(lo, hi), c.q, SCALE, o, c.ws, lse=l)
        parts.append(o)
        lses.append(l)
    merged, mlse = c.out()
    oda.oda_merge_partials(torch.stack(parts), torch.stack(lses), merged, lse=mlse)
    c.ok()
    ref, rlse, _ = c.oracle(lambda b, t: O.full_positions(t))
    assert_out_close(merged, ref)
    assert_lse_close(mlse.cpu().numpy(), rlse)


def test_gated_sequences_keep_everything():
    c = PagedCase([100, 40, 2000], 8, 4, seed=54)
    gate = torch.tensor([0, 1, 0], dtype=torch.int32, device="cuda")
    before = c.raw()
    out, lse = c.out(fill=3.0)
    oda.oda_kv4_decode(c.kv, full(gate), c.q, SCALE, out, c.ws, k_new=c.k_new, v_new=c.v_new, lse=lse)
    c.ok()
    ref, _, _ = c.oracle(lambda b, t: O.full_positions(t), commit=True)
    assert (out[[0, 2]] == 3.0).all() and (lse[[0, 2]] == 3.0).all()
    assert_out_close(out[1:2], ref[1:2])
    changed = (c.raw() != before).flatten(1).any(1).nonzero()[:, 0].tolist()
    assert changed == [int(c.bt[1, 2])]


@pytest.mark.parametrize("G", [1, 2, 4])
def test_hidden_garbage_does_not_show(G):
    """NaN and infinite scales and minima in every slot behind t and between sink and window."""
    c = PagedCase([1, 5, 17, 1000], 2 * G, 2, seed=55)
    ref, rlse, _ = c.oracle(lambda b, t: O.local_positions(t, 3, 20))
    meta = c.cache[..., 2048:].view(torch.int16).view(c.num_blocks, 2, 16, 8)
    hidden = torch.ones((c.num_blocks, 16), dtype=torch.bool)
    for b, n in enumerate(c.lengths):
        for p in O.local_positions(n - 1, 3, 20):
            hidden[c.bt_h[b, p // 16], p % 16] = False
    page, row = hidden.nonzero(as_tuple=True)
    for i, bits in enumerate((0x7fc0, 0x7f80, -0x80, 0x7f7f)):     # NaN, inf, -inf, the largest
        meta[page[i::4].cuda(), :, row[i::4].cuda()] = bits
    out, lse = c.out()
    oda.oda_kv4_decode(c.kv, local(3, 20), c.q, SCALE, out, c.ws, lse=lse)
    c.ok()
    assert_out_close(out, ref)
    assert_lse_close(lse.cpu().numpy(), rlse)


def test_a_visible_nan_shows_in_its_group_alone():
    rows = [gauss((50, 1, 128), 56 + i) for i in range(2)]
    rows[1][20, 0, 70] = float("nan")                              # V, group 1
    c = PagedCase([50], 2, 1, seed=57, rows=rows)
    out, lse = c.out()
    oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, out, c.ws, lse=lse)
    c.ok()
    assert torch.isnan(out[..., 64:]).all() and torch.isfinite(out[..., :64]).all() and torch.isfinite(lse).all()
    rows[0][:, 0, 3] = float("nan")                                # every K row: no score is a number
    c = PagedCase([50], 2, 1, seed=57, rows=rows)
    out, lse = c.out(fill=0.0)
    oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, out, c.ws, lse=lse)
    c.ok()
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("G", [1, 2, 4])
@pytest.mark.parametrize("kind", ["rising", "sharp", "v_growing", "v_shrinking", "v_tiny", "v_huge", "q_scale"])
def test_extreme_ranges(G, kind):
    """Scores that keep rising, or are 8 times wider; V rows whose scale changes by 2^60 along the
    sequence (or is tiny or huge throughout); q far outside the fp16 range against K as far the other
    way. Outputs are compared relative to the V range."""
    n, hkv = 1500, 2
    k, v = gauss((n, hkv, 128), 60).float(), gauss((n, hkv, 128), 61).float()
    pos = torch.arange(n, device="cuda").view(-1, 1, 1)
    unit = 1.0
    if kind == "rising":
        k *= 1 + 8.0 * pos / n
    if kind == "v_growing":
        v *= 2.0 ** (60.0 * pos / n - 30)
    if kind == "v_shrinking":
        v *= 2.0 ** (30 - 60.0 * pos / n)
    if kind in ("v_tiny", "v_huge"):
        unit = 2.0 ** (-60 if kind == "v_tiny" else 60)
        v *= unit
    if kind == "q_scale":
        k *= 2.0 ** -30
    c = PagedCase([n], G * hkv, hkv, seed=62, rows=(k.to(torch.bfloat16), v.to(torch.bfloat16)))
    if kind == "sharp":
        c.q.mul_(8.0)
    if kind == "q_scale":
        c.q.mul_(2.0 ** 30)
    out, lse = c.out()
    oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, out, c.ws, lse=lse)
    c.ok()
    ref, rlse, _ = c.oracle(lambda b, t: O.full_positions(t))
    # scores are up to 8 times those of the other tests, and so is a weight's relative error
    wide = 8 if kind in ("rising", "sharp") else 1
    top = np.abs(ref).max() if kind in ("v_growing", "v_shrinking") else unit
    assert np.abs(out.double().cpu().numpy() - ref).max() <= 1e-4 * wide * top
    assert np.abs(lse.double().cpu().numpy() - rlse).max() <= 1e-4 * wide


def test_device_errors_are_reported_and_skipped():
    c = PagedCase([40, 40, 2000], 8, 4, seed=64)
    ref, _, _ = c.oracle(lambda b, t: O.full_positions(t))
    c.seq_lens[0] = 16 * c.maxb + 1
    out, lse = c.out()
    oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, out, c.ws, lse=lse)
    torch.cuda.synchronize()
    assert int(c.status.item()) == oda.ODA_DEV_BAD_LEN
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all()
    assert_out_close(out[1:], ref[1:])
    c.status.zero_()
    c.seq_lens[0] = 40
    c.bt[1, 1] = -5                                                # tokens 16..31 are skipped
    out, lse = c.out()
    oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, out, c.ws, lse=lse)
    torch.cuda.synchronize()
    assert int(c.status.item()) == oda.ODA_DEV_BAD_BLOCK
    skip = np.r_[0:16, 32:40]
    ref1, _, _ = c.oracle(lambda b, t: skip if b == 1 else O.full_positions(t))
    assert_out_close(out, ref1)


def test_largest_batch():
    r = np.random.default_rng(66)
    lens = [int(x) for x in r.integers(1, 400, size=1024)]
    c = PagedCase(lens, 4, 2, seed=67)
    out, lse = c.out()
    oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, out, c.ws, lse=lse)
    c.ok()
    assert c.stats[oda.ODA_STAT_ROWS].item() == 2 * sum(lens)
    ref, rlse, _ = c.oracle(lambda b, t: O.full_positions(t))
    assert_out_close(out, ref)
    assert_lse_close(lse.cpu().numpy(), rlse)


def test_pages_beyond_32_bit_offsets():
    """A cache of more than 4 GB whose sequence lies at its far end."""
    hkv, n = 8, 500
    nb = (1 << 32) // (hkv * oda.ODA_KV4_PAGE_BYTES) + 200
    cache = torch.zeros((nb, hkv, oda.ODA_KV4_PAGE_BYTES), dtype=torch.uint8, device="cuda")
    small = PagedCase([n], 16, hkv, seed=68)
    bt = (nb - small.maxb + torch.randperm(small.maxb, generator=torch.Generator().manual_seed(1))).to(torch.int32)
    cache[bt.long().cuda()] = small.cache[small.bt[0].long()]
    kv = oda.make_kv4(cache, bt.view(1, -1).cuda(), small.seq_lens, small.status)
    out, lse = small.out()
    want, wlse = small.out()
    oda.oda_kv4_decode(kv, full(), small.q, SCALE, out, small.ws, k_new=small.k_new, v_new=small.v_new, lse=lse)
    oda.oda_kv4_decode(small.kv, full(), small.q, SCALE, want, small.ws, k_new=small.k_new, v_new=small.v_new,
                       lse=wlse)
    small.ok()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    assert torch.equal(cache[bt.long().cuda()], small.cache[small.bt[0].long()])


def test_repeatable_on_streams_and_in_graphs():
    c = PagedCase([3000, 17, 900], 16, 4, seed=69)
    ref, rlse = c.out()
    oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, ref, c.ws, lse=rlse)
    c.ok()
    side = torch.cuda.Stream()
    ws2 = torch.zeros_like(c.ws)
    outs = []
    torch.cuda.synchronize()
    for _ in range(20):                            # two calls at once, a workspace each
        a, al = c.out()
        b, bl = c.out()
        torch.cuda.synchronize()
        oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, a, c.ws, lse=al)
        oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, b, ws2, lse=bl, stream=side)
        outs += [(a, al), (b, bl)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) and torch.equal(l, rlse) for o, l in outs)

    out, lse = c.out()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        oda.oda_kv4_decode(c.kv, local(4, 100), c.q, SCALE, out, c.ws, k_new=c.k_new, v_new=c.v_new, lse=lse)
    for i in range(3):                             # the replay reads what is in the buffers then
        c.k_new.copy_(gauss(c.k_new.shape, 70 + i))
        c.q.copy_(gauss(c.q.shape, 80 + i))
        g.replay()
        c.ok()
        c.snapshot()
        r, rl, _ = c.oracle(lambda b, t: O.local_positions(t, 4, 100))
        assert_out_close(out, r)


def test_two_graphs_share_a_workspace_and_sequences_share_pages():
    """Graphs of a Full and a Local call over one workspace, replayed in turn; sequences 1 and 2 are the
    same pages, sequence 2 shorter by some."""
    c = PagedCase([2500, 700, 600, 40], 16, 4, seed=90)
    c.bt[2] = c.bt[1]
    c.bt_h = c.bt.cpu().numpy()
    outs = [c.out(), c.out()]
    vis = [full(), local(4, 256)]
    graphs = []
    for (out, lse), v in zip(outs, vis):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            oda.oda_kv4_decode(c.kv, v, c.q, SCALE, out, c.ws, lse=lse)
        graphs.append(g)
    positions = [lambda b, t: O.full_positions(t), lambda b, t: O.local_positions(t, 4, 256)]
    for i in (0, 1, 1, 0, 1, 0):
        out, lse = outs[i]
        out.fill_(float("nan"))
        graphs[i].replay()
        c.ok()
        ref, rlse, _ = c.oracle(positions[i])
        assert_out_close(out, ref)
        assert_lse_close(lse.cpu().numpy(), rlse)


def test_calls_one_behind_the_other_see_each_others_writes():
    """Append, decode, append, decode without a host wait: a launch may begin before its predecessor ends, but
    reads nothing of it before."""
    c = PagedCase([300, 16, 33], 8, 4, seed=91)
    rows = [(gauss(c.k_new.shape, 300 + i), gauss(c.k_new.shape, 400 + i)) for i in range(12)]
    got = [c.out() for _ in rows]
    back = [(torch.empty(3, 4, 128, device="cuda"), torch.empty(3, 4, 128, device="cuda")) for _ in rows]
    torch.cuda.synchronize()
    for (k, v), (out, lse), (rk, rv) in zip(rows, got, back):
        oda.oda_kv4_append(c.kv, k, v)
        oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, out, c.ws, lse=lse)
        oda.oda_kv4_read(c.kv, rk, rv)
    c.ok()
    for (k, v), (out, lse), (rk, rv) in zip(rows, got, back):
        assert np.array_equal(rk.cpu().numpy(), K.round_trip(k.double().cpu().numpy()).astype(np.float32))
        assert np.array_equal(rv.cpu().numpy(), K.round_trip(v.double().cpu().numpy()).astype(np.float32))
        c.k_new, c.v_new = k, v
        ref, rlse, _ = c.oracle(lambda b, t: O.full_positions(t), commit=True)
        assert_out_close(out, ref)
        assert_lse_close(lse.cpu().numpy(), rlse)


def test_one_sequence_of_many_ctas_for_each_head_count():
    """A long history on every head grouping: the partials of some hundred CTAs are merged in chunks."""
    for G, hkv in ((1, 1), (2, 1), (4, 1), (4, 2)):
        c = PagedCase([40000], G * hkv, hkv, seed=92 + G)
        out, lse = c.out()
        oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, out, c.ws, lse=lse)
        c.ok()
        ref, rlse, _ = c.oracle(lambda b, t: O.full_positions(t))
        assert_out_close(out, ref, "G %d hkv %d" % (G, hkv))
        assert_lse_close(lse.cpu().numpy(), rlse)


def test_one_workspace_for_calls_of_every_shape():
    """Batches, head counts and lengths in turn over one workspace, the attention alone and with weights;
    (sequence, KV head)s that begin and end inside a CTA's share among them."""
    cases = [PagedCase([9000], 4, 1, seed=300), PagedCase([700, 3, 2100, 44], 16, 4, seed=301),
             PagedCase([3000 + 17 * i for i in range(24)], 8, 8, seed=302), PagedCase([6000, 12000], 6, 3, seed=303)]
    refs = []
    for c in cases:
        refs.append((c.out(), c.out(), torch.zeros((c.B, c.hkv, c.maxb * 16), device="cuda")))
        (o, l), (o2, l2), m = refs[-1]
        oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, o, c.ws, lse=l)
        oda.oda_kv4_decode_mass(c.kv, full(), c.q, SCALE, o2, torch.zeros_like(c.ws), m, lse=l2)
        c.ok()
        assert torch.equal(o, o2) and torch.equal(l, l2)
    ref, rlse, _ = cases[2].oracle(lambda b, t: O.full_positions(t))
    assert_out_close(refs[2][0][0], ref)
    ws = torch.zeros(max(c.ws.numel() for c in cases), dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 3, 2, 0, 3, 1, 1, 2, 0):
        c, ((o, l), _, m) = cases[i], refs[i]
        out, lse = c.out()
        oda.oda_kv4_decode(c.kv, full(), c.q, SCALE, out, ws, lse=lse)
        out2, lse2 = c.out()
        got = torch.zeros_like(m)
        oda.oda_kv4_decode_mass(c.kv, full(), c.q, SCALE, out2, ws, got, lse=lse2)
        c.ok()
        assert torch.equal(out, o) and torch.equal(lse, l), i
        assert torch.equal(out2, o) and torch.equal(lse2, l) and torch.equal(got, m), i


def test_append_of_one_row_takes_any_row_stride():
    """A single row's stride says nothing: one that is no multiple of 8 elements is no reason to refuse it."""
    c = PagedCase([20], 8, 4, seed=95)
    k, v = (gauss((4 * 128,), 96 + i).as_strided((1, 4, 128), (4 * 128 + 4, 128, 1)) for i in range(2))
    assert k.stride(0) % 8 != 0
    oda.oda_kv4_append(c.kv, k, v)
    back = [torch.empty(1, 4, 128, device="cuda") for _ in range(2)]
    oda.oda_kv4_read(c.kv, *back)
    c.ok()
    for got, want in zip(back, (k, v)):
        assert np.array_equal(got.cpu().numpy(), K.round_trip(want.double().cpu().numpy()).astype(np.float32))
