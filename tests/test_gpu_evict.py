"""Decode with accumulated attention weights and eviction by them, bf16 and 4-bit caches, against the
fp64 oracle: masses under every visibility rule, aliasing, kept sets with ties, moves in place and to
other pages, device-side errors, and a whole run of append, decode and eviction."""
import numpy as np
import pytest
import torch

from kv4_cases import (MASS, SCALE, PagedCase, assert_lse_close, assert_out_close, full, gauss, keep, keep_lists,
                       local)
from oracle import kv4_oracle as K
from oracle import oda_oracle as O
from sparse_kv_recall_b200 import build as B
from sparse_kv_recall_b200 import oda

pytestmark = pytest.mark.gpu
BOTH = pytest.mark.parametrize("kv4", [False, True])


@pytest.fixture(scope="module", autouse=True)
def _library():
    B.build()
    oda.load()


def _mass_call(c):
    return oda.oda_kv4_decode_mass if c.kv4 else oda.oda_decode_mass


def _random_mass(c, seed, ties=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = torch.randn((c.B, c.hkv, c.maxb * 16), generator=g, device="cuda").mul_(1.5).exp_()
    return torch.round(m * 4) / 4 if ties else m


def _assert_mass(got, before, expected, c, skip=()):
    got, before = got.double().cpu().numpy(), before.double().cpu().numpy()
    for b, n in enumerate(c.lengths):
        want = before[b].copy()
        if b not in skip:
            pos, m = expected[b]
            want[:, pos] += m
        d = np.abs(got[b] - want)
        assert np.all(d <= MASS + np.abs(want) * 2.0 ** -23), "sequence %d: %g" % (b, d.max())


@BOTH
@pytest.mark.parametrize("G,hkv", [(1, 8), (2, 8), (4, 3)])
@pytest.mark.parametrize("rule", ["full", "local", "keep"])
@pytest.mark.parametrize("alias", [False, True])
def test_mass_matches_oracle(kv4, G, hkv, rule, alias):
    lens = [1, 16, 17, 300, 2053, 4100]
    c = PagedCase(lens, G * hkv, hkv, seed=100 + G, kv4=kv4)
    blocks, counts, lists = keep_lists(lens, c.maxb, 101, empty=(2,))
    vis, pos = {"full": (full(), lambda b, t: O.full_positions(t)),
                "local": (local(5, 100), lambda b, t: O.local_positions(t, 5, 100)),
                "keep": (keep(blocks, counts), lambda b, t: O.keep_positions(t, lists[b]))}[rule]
    before = _random_mass(c, 102)
    mass_in = before.clone()
    mass_out = mass_in if alias else torch.full_like(mass_in, 9.0)
    out, lse = c.out()
    commit = dict(k_new=c.k_new, v_new=c.v_new) if rule == "local" else {}
    _mass_call(c)(c.kv, vis, c.q, SCALE, out, c.ws, mass_out, mass_in=mass_in, lse=lse, **commit)
    c.ok()
    ref, rlse, mass = c.oracle(pos, commit=rule == "local")
    assert_out_close(out, ref)
    assert_lse_close(lse.cpu().numpy(), rlse)
    want = before.clone()
    if not alias:                                  # positions from seq_lens on keep their contents
        for b, n in enumerate(lens):
            want[b, :, n:] = 9.0
    _assert_mass(mass_out, want, mass, c)
    if not alias:
        assert torch.equal(mass_in, before)
    assert c.stats[oda.ODA_STAT_ROWS].item() == hkv * sum(len(pos(b, n - 1)) for b, n in enumerate(lens))


@BOTH
def test_mass_from_nothing_without_lse_and_in_bf16(kv4):
    c = PagedCase([40, 1000], 16, 4, seed=110, kv4=kv4)
    out, _ = c.out(torch.bfloat16)
    mass = torch.full((2, 4, c.maxb * 16 + 8), 2.0, device="cuda")
    _mass_call(c)(c.kv, full(), c.q, SCALE, out, c.ws, mass)
    c.ok()
    ref, _, want = c.oracle(lambda b, t: O.full_positions(t))
    assert_out_close(out, ref)
    for b, n in enumerate(c.lengths):
        assert np.abs(mass[b, :, :n].double().cpu().numpy() - want[b][1]).max() <= MASS
        assert (mass[b, :, n:] == 2.0).all()


@BOTH
def test_mass_under_declared_modes_shards_and_gates(kv4):
    lens = [3000, 900, 40]
    c = PagedCase(lens, 8, 4, seed=111, kv4=kv4)
    modes = torch.tensor([1, 2, 0], dtype=torch.int32, device="cuda")
    offs = torch.tensor([500, 0, 0], dtype=torch.int32, device="cuda")
    kw = dict(focus_len=333, recent=50, local_len=64)
    before = _random_mass(c, 112)
    mass = torch.zeros_like(before)
    out, lse = c.out()
    _mass_call(c)(c.kv, oda.da_visibility(modes, offs, **kw), c.q, SCALE, out, c.ws, mass, mass_in=before, lse=lse)
    c.ok()
    ref, _, want = c.oracle(lambda b, t: O.da_mode_positions(int(modes[b]), t, int(offs[b]), **kw))
    assert_out_close(out, ref)
    for b, n in enumerate(lens):
        pos, m = want[b]
        w = before[b].double().cpu().numpy()
        w[:, pos] += m
        assert np.abs(mass[b, :, :n].double().cpu().numpy() - w[:, :n]).max() <= MASS + 2.0 ** -23 * w.max()
    gate = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
    got = before.clone()
    out, lse = c.out()
    _mass_call(c)(c.kv, oda.shard_visibility(16, 1600, gate), c.q, SCALE, out, c.ws, got, mass_in=got, lse=lse)
    c.ok()
    _, _, want = c.oracle(lambda b, t: O.shard_positions(t, 16, 1600))
    _assert_mass(got, before, want, c, skip=(1,))
    assert torch.equal(got[1], before[1])


def test_hidden_garbage_does_not_show_in_the_bf16_outputs():
    """PagedCase fills bf16 slots that no token holds with NaN; the gap between sink and window too."""
    for G in (1, 2, 4):
        c = PagedCase([1, 5, 17, 1000], 2 * G, 2, seed=113, kv4=False)
        ref, rlse, mass = c.oracle(lambda b, t: O.local_positions(t, 3, 20))
        for p in range(3, 980):
            page = c.bt_h[3, p // 16]
            c.kc[page, :, p % 16] = float("nan")
            c.vc[page, :, p % 16] = float("inf")
        out, lse = c.out()
        got = torch.zeros((4, 2, c.maxb * 16), device="cuda")
        before = got.clone()
        oda.oda_decode_mass(c.kv, local(3, 20), c.q, SCALE, out, c.ws, got, mass_in=got, lse=lse)
        c.ok()
        assert_out_close(out, ref)
        assert_lse_close(lse.cpu().numpy(), rlse)
        _assert_mass(got, before, mass, c)


def _evict(c, mass, sink, recent, budget, dst=None, mass_out=None, lens_out=None, gate=None):
    """Returns kept, mass_out, seq_lens_out; dst None = in place."""
    kept = torch.full((c.B, c.hkv, budget), -9, dtype=torch.int32, device="cuda")
    mass_out = mass if dst is None else (torch.full_like(mass, 5.0) if mass_out is None else mass_out)
    lens_out = c.seq_lens if dst is None else torch.zeros_like(c.seq_lens) if lens_out is None else lens_out
    ws = torch.zeros(oda.oda_kv_evict_workspace_size(c.B), dtype=torch.uint8, device="cuda")
    call = oda.oda_kv4_evict if c.kv4 else oda.oda_kv_evict
    call(c.kv, mass, sink, recent, budget, c.bt if dst is None else dst, kept, mass_out, lens_out, ws, gate=gate)
    torch.cuda.synchronize()
    assert not ws.any()
    return kept, mass_out, lens_out


def _assert_evicted(c, lens, table, old, old_mass, kept, mass, new_lens, sink, recent, budget, skip=()):
    """Kept sets, moved rows, masses and lengths against the oracle. old: (k, v) host values before."""
    c.snapshot()
    kept, mass, old_mass = kept.cpu().numpy(), mass.cpu().numpy(), old_mass.cpu().numpy()
    table = table.cpu().numpy()
    for b, n in enumerate(lens):
        if b in skip:
            continue
        m = min(n, budget)
        assert int(new_lens[b]) == m
        i = np.arange(m)
        for g in range(c.hkv):
            want = K.kept_slots(old_mass[b, g], n, sink, recent, budget)
            assert np.array_equal(kept[b, g, :m], want), (b, g)
            assert (kept[b, g, m:] == -1).all()
            for now, was in ((c.k, old[0]), (c.v, old[1])):
                assert np.array_equal(now[table[b, i // 16], g, i % 16],
                                      was[c.bt_h[b, want // 16], g, want % 16])
            assert np.array_equal(mass[b, g, :m], old_mass[b, g, want])
            assert (mass[b, g, m:n] == 0).all()


SHAPES = [   # lengths, hkv, sink, recent, budget
    ([2304, 700, 2048, 2049], 8, 4, 1024, 2048),
    ([1, 5, 16, 17, 33, 100], 2, 0, 0, 16),
    ([1, 2, 3], 1, 1, 0, 1),
    ([1, 2, 3, 90], 3, 0, 1, 1),
    ([500, 400], 1, 0, 200, 200),                  # nothing but the recent slots
    ([500, 400], 2, 64, 0, 65),
    ([9000], 1, 4, 512, 5000),                     # one cluster, several rounds
    ([6000, 5990, 20], 2, 3, 77, 4999),
    ([40 + 13 * i for i in range(40)], 5, 4, 16, 100),
]


@BOTH
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("lens,hkv,sink,recent,budget", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_matches_oracle(kv4, ties, lens, hkv, sink, recent, budget, in_place):
    if ties and not in_place and len(lens) > 10:
        lens = lens[:17]
    pages = -(-budget // 16)
    c = PagedCase(lens, hkv, hkv, seed=120 + len(lens), kv4=kv4, spare=0 if in_place else pages * len(lens))
    mass = _random_mass(c, 121, ties)
    old, old_mass, raw = (c.k.copy(), c.v.copy()), mass.clone(), c.raw()
    dst = None if in_place else c.spare.view(len(lens), pages).contiguous()
    kept, mass_out, new_lens = _evict(c, mass, sink, recent, budget, dst)
    c.ok()
    _assert_evicted(c, lens, c.bt if in_place else dst, old, old_mass, kept, mass_out, new_lens, sink, recent,
                    budget)
    if not in_place:                               # the source is as it was, and so is what was not asked for
        assert torch.equal(mass, old_mass) and c.seq_lens.tolist() == list(lens)
        now = c.raw()
        src = torch.unique(c.bt[c.bt >= 0]).long()
        assert torch.equal(now[src], raw[src]) if kv4 else torch.equal(now[:, src], raw[:, src])
        for b, n in enumerate(lens):
            assert (mass_out[b, :, n:] == 5.0).all()


@BOTH
def test_evict_many_heads_of_many_slots(kv4):
    """Too many (sequence, KV head)s for more than one CTA each, and more than 4096 slots kept of some."""
    lens = [8192, 7001] + [30 + i for i in range(17)]
    c = PagedCase(lens, 8, 8, seed=131, kv4=kv4)
    mass = _random_mass(c, 132)
    old, old_mass = (c.k.copy(), c.v.copy()), mass.clone()
    kept, mass_out, new_lens = _evict(c, mass, 4, 300, 6500)
    c.ok()
    _assert_evicted(c, lens, c.bt, old, old_mass, kept, mass_out, new_lens, 4, 300, 6500)


@BOTH
def test_evict_orders_every_kind_of_weight(kv4):
    """Equal weights, zeros of both signs, infinities, subnormals and negative numbers."""
    c = PagedCase([64], 1, 1, seed=130, kv4=kv4)
    vals = [0.0, -0.0, 1.0, 1.0, float("inf"), -1.0, 2.0 ** -140, -2.0 ** -140, float("-inf"), 3.0]
    nan = torch.tensor([0x7fc00000, 0xffc00000 - (1 << 32)], dtype=torch.int32, device="cuda").view(torch.float32)
    for budget in (2, 4, 20):                      # a NaN of either sign counts above everything
        m = torch.zeros((1, 1, 64), device="cuda")
        m[0, 0, 20], m[0, 0, 40], m[0, 0, 50] = nan[1], nan[0], float("inf")
        c = PagedCase([64], 1, 1, seed=130, kv4=kv4)
        kept, _, _ = _evict(c, m, 0, 0, budget)
        c.ok()
        assert kept[0, 0].tolist() == sorted(([20, 40, 50] + [i for i in range(64) if i not in (20, 40, 50)])[:budget])
    mass = torch.tensor([(vals * 7)[:64]], device="cuda").view(1, 1, 64).contiguous()
    for budget in (1, 6, 7, 8, 13, 20, 21, 33, 40, 48, 63):
        m = mass.clone()
        c2 = PagedCase([64], 1, 1, seed=130, kv4=kv4)
        kept, _, _ = _evict(c2, m, 0, 0, budget)
        c2.ok()
        assert kept[0, 0].tolist() == K.kept_slots(mass[0, 0].tolist(), 64, 0, 0, budget).tolist(), budget


@BOTH
@pytest.mark.parametrize("n,hkv,budget", [(700, 2, 333), (20000, 1, 9000)])
def test_evict_into_a_copy_of_the_table_is_in_place(kv4, n, hkv, budget):
    """The destination holds the source's own pages but is another tensor, as are the weights and lengths."""
    c = PagedCase([n, n - 9], hkv, hkv, seed=129, kv4=kv4)
    mass = _random_mass(c, 128)
    old, old_mass = (c.k.copy(), c.v.copy()), mass.clone()
    kept, mass_out, new_lens = _evict(c, mass, 4, 50, budget, c.bt[:, :-(-budget // 16)].contiguous())
    c.ok()
    _assert_evicted(c, [n, n - 9], c.bt, old, old_mass, kept, mass_out, new_lens, 4, 50, budget)


@BOTH
def test_evict_leaves_gated_and_bad_sequences(kv4):
    lens = [100, 100, 100, 100, 100]
    c = PagedCase(lens, 4, 4, seed=131, kv4=kv4)
    mass = _random_mass(c, 132)
    gate = torch.tensor([1, 0, 1, 1, 1], dtype=torch.int32, device="cuda")
    c.bt[2, 3] = c.num_blocks
    c.seq_lens[3] = 16 * c.maxb + 1
    old, old_mass, raw, bt = (c.k.copy(), c.v.copy()), mass.clone(), c.raw(), c.bt.clone()
    kept, mass_out, new_lens = _evict(c, mass, 2, 10, 50, gate=gate)
    assert int(c.status.item()) in (oda.ODA_DEV_BAD_LEN, oda.ODA_DEV_BAD_BLOCK)
    assert new_lens.tolist() == [50, 100, 100, 16 * c.maxb + 1, 50]
    _assert_evicted(c, lens, c.bt, old, old_mass, kept, mass_out, new_lens, 2, 10, 50, skip=(1, 2, 3))
    assert torch.equal(mass_out[1:4], old_mass[1:4]) and (kept[1:4] == -9).all()
    own = bt[1:4][(bt[1:4] >= 0) & (bt[1:4] < c.num_blocks)].long()
    now = c.raw()
    assert torch.equal(now[own], raw[own]) if kv4 else torch.equal(now[:, own], raw[:, own])
    c.status.zero_()                               # a bad destination page
    dst = torch.full((5, 4), c.num_blocks + 3, dtype=torch.int32, device="cuda")
    raw = c.raw()
    c.bt[2, 3] = bt[2, 2]
    c.seq_lens.fill_(40)
    kept, _, new_lens = _evict(c, mass, 2, 10, 50, dst)
    assert int(c.status.item()) == oda.ODA_DEV_BAD_BLOCK and torch.equal(c.raw(), raw)
    assert new_lens.tolist() == [40] * 5


def test_evict_beyond_32_bit_offsets():
    """bf16 caches of more than 2^32 bytes each, the sequence at their far end."""
    hkv, n, budget = 8, 200, 77
    nb = (1 << 32) // (hkv * 16 * 256) + 40
    small = PagedCase([n], 8, hkv, seed=133, kv4=False)
    kc, vc = (torch.zeros((nb, hkv, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    far = (nb - small.maxb + small.bt).to(torch.int32)
    kc[far[0].long()], vc[far[0].long()] = small.kc[small.bt[0].long()], small.vc[small.bt[0].long()]
    mass = _random_mass(small, 134)
    m2, lens = mass.clone(), small.seq_lens.clone()
    kv = oda.make_kv(kc, vc, far, lens, small.status)
    kept = torch.empty((1, hkv, budget), dtype=torch.int32, device="cuda")
    ws = torch.zeros(oda.oda_kv_evict_workspace_size(1), dtype=torch.uint8, device="cuda")
    oda.oda_kv_evict(kv, m2, 3, 20, budget, far, kept, m2, lens, ws)
    want, _, _ = _evict(small, mass, 3, 20, budget)
    small.ok()
    assert torch.equal(kept, want) and torch.equal(m2, mass) and lens.tolist() == [budget]
    keep = far[0, :4].long()                       # whole pages of kept rows
    assert torch.equal(kc[keep], small.kc[small.bt[0, :4].long()])
    assert torch.equal(vc[keep], small.vc[small.bt[0, :4].long()])


@BOTH
def test_mass_and_evict_in_a_graph_and_on_two_streams(kv4):
    c = PagedCase([600, 40], 8, 4, seed=135, kv4=kv4, spare=2 * 13)
    dst = c.spare.view(2, 13).contiguous()
    before = _random_mass(c, 136)
    mass, mass2 = torch.zeros_like(before), torch.zeros_like(before)
    out, lse = c.out()
    kept = torch.empty((2, 4, 200), dtype=torch.int32, device="cuda")
    lens = torch.zeros_like(c.seq_lens)
    ws = torch.zeros(oda.oda_kv_evict_workspace_size(2), dtype=torch.uint8, device="cuda")
    ev = oda.oda_kv4_evict if kv4 else oda.oda_kv_evict

    def step(stream=None):
        _mass_call(c)(c.kv, full(), c.q, SCALE, out, c.ws, mass, mass_in=before, lse=lse, stream=stream)
        ev(c.kv, mass, 2, 20, 200, dst, kept, mass2, lens, ws, stream=stream)
    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (out, lse, mass, kept, mass2, lens)]
    side = torch.cuda.Stream()
    for x in (out, lse, mass, mass2):
        x.zero_()
    kept.zero_()
    torch.cuda.synchronize()
    step(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((out, lse, mass, kept, mass2, lens), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for x in (out, lse, mass, mass2):
        x.zero_()
    kept.zero_()
    for _ in range(2):
        g.replay()
    c.ok()
    assert all(torch.equal(a, b) for a, b in zip((out, lse, mass, kept, mass2, lens), want))


@BOTH
def test_a_run_of_decode_steps_with_eviction(kv4):
    """Prompts, decode steps that commit and accumulate, eviction in place when the budget is passed by
    16, Local steps in between: every step's outputs, and the weights, against an oracle that keeps its
    own lists of rows per KV head."""
    lens, hkv, G, sink, recent, budget = [70, 41, 9], 2, 2, 2, 12, 48
    c = PagedCase([n + 80 for n in lens], G * hkv, hkv, seed=140, kv4=kv4)
    c.lengths = list(lens)
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    rows = [[[list(x) for x in zip(*c.rows(b, g, np.arange(n)))] for g in range(hkv)] for b, n in enumerate(lens)]
    want_mass = [[np.zeros(n).tolist() for _ in range(hkv)] for n in lens]
    mass = torch.zeros((3, hkv, c.maxb * 16), device="cuda")
    evicted = 0
    for step in range(24):
        c.seq_lens.add_(1)
        c.q.copy_(gauss(c.q.shape, 150 + step))
        c.k_new.copy_(gauss(c.k_new.shape, 180 + step))
        c.v_new.copy_(gauss(c.v_new.shape, 210 + step))
        kn, vn = (x.double().cpu().numpy() for x in (c.k_new, c.v_new))
        if kv4:
            kn, vn = K.round_trip(kn), K.round_trip(vn)
        vis = local(2, 20) if step % 3 == 1 else full()
        out, lse = c.out()
        _mass_call(c)(c.kv, vis, c.q, SCALE, out, c.ws, mass, mass_in=mass, k_new=c.k_new, v_new=c.v_new, lse=lse)
        c.ok()
        q = c.q.double().cpu().numpy()
        for b in range(3):
            ks, vs, pos = [], [], None
            for g in range(hkv):
                rows[b][g].append([kn[b, g], vn[b, g]])
                want_mass[b][g].append(0.0)
                n = len(rows[b][g])
                pos = O.local_positions(n - 1, 2, 20) if step % 3 == 1 else O.full_positions(n - 1)
                ks.append(np.array([rows[b][g][p][0] for p in pos]))
                vs.append(np.array([rows[b][g][p][1] for p in pos]))
            ref, rlse = O.decode_attention(q[b], ks, vs, SCALE)
            assert_out_close(out[b], ref, "step %d" % step)
            assert_lse_close(lse[b].cpu().numpy(), rlse)
            m = K.attention_mass(q[b], ks, SCALE, G)
            for g in range(hkv):
                for i, p in enumerate(pos):
                    want_mass[b][g][p] += m[g][i]
        now = mass.double().cpu().numpy()
        for b in range(3):
            n = len(rows[b][0])
            assert int(c.seq_lens[b]) == n
            for g in range(hkv):
                assert np.abs(now[b, g, :n] - want_mass[b][g]).max() <= MASS * (step + 1)
        if max(len(r[0]) for r in rows) >= budget + 16:
            old = mass.cpu().numpy()
            _evict(c, mass, sink, recent, budget)
            c.ok()
            evicted += 1
            for b in range(3):
                for g in range(hkv):               # by the weights on the device: the oracle's differ in ulps
                    keep_ = K.kept_slots(old[b, g], len(rows[b][g]), sink, recent, budget)
                    rows[b][g] = [rows[b][g][p] for p in keep_]
                    want_mass[b][g] = [want_mass[b][g][p] for p in keep_]
    assert evicted >= 2


@BOTH
def test_mass_and_evict_at_once_and_graphs_over_one_workspace(kv4):
    """Two calls at once on two streams, a workspace each; then two graphs of different rules over one
    workspace, replayed in turn."""
    c = PagedCase([2600, 700, 31], 8, 4, seed=150, kv4=kv4, spare=6 * 20)
    mass_call, ev = _mass_call(c), oda.oda_kv4_evict if kv4 else oda.oda_kv_evict
    before = _random_mass(c, 151)
    side = torch.cuda.Stream()

    def buffers(i):
        return dict(out=c.out(), mass=torch.zeros_like(before), mass2=torch.zeros_like(before), ws=torch.zeros_like(c.ws),
                    kept=torch.zeros((3, 4, 300), dtype=torch.int32, device="cuda"), lens=torch.zeros_like(c.seq_lens),
                    dst=c.spare[60 * i:60 * i + 60].view(3, 20).contiguous(),
                    ews=torch.zeros(oda.oda_kv_evict_workspace_size(3), dtype=torch.uint8, device="cuda"))

    def step(s, vis, stream=None):
        mass_call(c.kv, vis, c.q, SCALE, s["out"][0], s["ws"], s["mass"], mass_in=before, lse=s["out"][1],
                  stream=stream)
        ev(c.kv, s["mass"], 2, 20, 300, s["dst"], s["kept"], s["mass2"], s["lens"], s["ews"], stream=stream)

    def results(s):
        return [x.clone() for x in (*s["out"], s["mass"], s["mass2"], s["kept"], s["lens"])]
    a, b = buffers(0), buffers(1)
    step(a, full())
    torch.cuda.synchronize()
    want = results(a)
    for _ in range(10):
        step(a, full())
        step(b, full(), stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for s in (a, b) for x, y in zip(results(s), want))
    c.ok()
    step(b, local(4, 100))
    torch.cuda.synchronize()
    wants = [want, results(b)]
    b["ws"], b["ews"] = a["ws"], a["ews"]
    graphs = []
    for s, vis in ((a, full()), (b, local(4, 100))):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s, vis)
        graphs.append(g)
    for i in (1, 0, 0, 1, 0, 1):
        s = (a, b)[i]
        for x in (*s["out"], s["mass"], s["mass2"], s["kept"], s["lens"]):
            x.zero_()
        graphs[i].replay()
        c.ok()
        assert all(torch.equal(x, y) for x, y in zip(results(s), wants[i]))


@BOTH
def test_sequences_that_share_a_prefix_are_cut_apart(kv4):
    """Three sequences over the same first pages, evicted into pages of their own."""
    lens, hkv, budget = [500, 500, 420], 2, 64
    c = PagedCase(lens, hkv, hkv, seed=152, kv4=kv4, spare=3 * 4)
    c.bt[1, :20] = c.bt[0, :20]
    c.bt[2, :20] = c.bt[0, :20]
    c.snapshot()
    mass = _random_mass(c, 153)
    old, old_mass, raw = (c.k.copy(), c.v.copy()), mass.clone(), c.raw()
    dst = c.spare.view(3, 4).contiguous()
    kept, mass_out, new_lens = _evict(c, mass, 4, 16, budget, dst)
    c.ok()
    _assert_evicted(c, lens, dst, old, old_mass, kept, mass_out, new_lens, 4, 16, budget)
    src = torch.unique(c.bt[c.bt >= 0]).long()
    assert torch.equal(c.raw()[src], raw[src]) if kv4 else torch.equal(c.raw()[:, src], raw[:, src])


@BOTH
def test_one_workspace_for_weights_of_every_shape(kv4):
    """Batches, head counts and table widths in turn over one workspace, with (sequence, KV head)s that begin and end
    inside a CTA's share; each call as with a workspace of its own."""
    cases = [PagedCase([9000], 4, 1, seed=160, kv4=kv4), PagedCase([700, 3, 2100, 44], 16, 4, seed=161, kv4=kv4),
             PagedCase([2000 + 17 * i for i in range(24)], 8, 8, seed=162, kv4=kv4),
             PagedCase([6000, 12000], 6, 3, seed=163, kv4=kv4)]
    refs = []
    for c in cases:
        (out, lse), mass = c.out(), torch.zeros((c.B, c.hkv, c.maxb * 16), device="cuda")
        _mass_call(c)(c.kv, full(), c.q, SCALE, out, c.ws, mass, lse=lse)
        c.ok()
        refs.append((out, lse, mass))
    ref, rlse, _ = cases[2].oracle(lambda b, t: O.full_positions(t))
    assert_out_close(refs[2][0], ref)
    ws = torch.zeros(max(c.ws.numel() for c in cases), dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 3, 2, 0, 3, 1, 1, 2, 0):
        c = cases[i]
        (out, lse), mass = c.out(), torch.zeros_like(refs[i][2])
        _mass_call(c)(c.kv, full(), c.q, SCALE, out, ws, mass, lse=lse)
        c.ok()
        assert all(torch.equal(a, b) for a, b in zip((out, lse, mass), refs[i])), i


@BOTH
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("budget", [700, 9000])
def test_evict_more_slots_than_a_cta_holds_keys_of(kv4, ties, in_place, budget):
    """One CTA a (sequence, KV head), 160 of them: of 8193 and 20,011 slots the keys do not fit in shared memory and the
    kept list goes through its output."""
    lens = [8193, 20011, 8192] + [30 + i for i in range(17)]
    need = [-(-min(n, budget) // 16) for n in lens]
    c = PagedCase(lens, 8, 8, seed=170, kv4=kv4, spare=0 if in_place else sum(need))
    mass = _random_mass(c, 171, ties)
    if ties:                                       # and many that were never attended
        mass[:, :, 100:15000:3] = 0.0
    old, old_mass = (c.k.copy(), c.v.copy()), mass.clone()
    dst = None
    if not in_place:                               # entries behind what is kept are not looked at
        dst = torch.full((len(lens), -(-budget // 16)), -1, dtype=torch.int32, device="cuda")
        for row, own in zip(dst, c.spare.split(need)):
            row[:len(own)] = own
    kept, mass_out, new_lens = _evict(c, mass, 4, 300, budget, dst)
    c.ok()
    _assert_evicted(c, lens, c.bt if in_place else dst, old, old_mass, kept, mass_out, new_lens, 4, 300, budget)


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_more_slots_than_a_cluster_holds_keys_of(ties, in_place):
    """16 CTAs of 8192 keys hold 131,072: of one sequence of 140,003 slots every pass reads the weights again."""
    n, budget = 140003, 50000
    pages = -(-budget // 16)
    c = PagedCase([n], 1, 1, seed=172, spare=0 if in_place else pages)
    mass = _random_mass(c, 173, ties)
    old, old_mass = (c.k.copy(), c.v.copy()), mass.clone()
    dst = None if in_place else c.spare.view(1, pages).contiguous()
    kept, mass_out, new_lens = _evict(c, mass, 4, 2000, budget, dst)
    c.ok()
    _assert_evicted(c, [n], c.bt if in_place else dst, old, old_mass, kept, mass_out, new_lens, 4, 2000, budget)
