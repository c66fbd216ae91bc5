"""Values at the ends of their ranges in decode over the 4-bit cache: a NaN that has to show however the
history is shared out, V scales and scores that change along a warp's pages, scores, K and V
of every magnitude.

Tolerances are those of kv4_cases: a weight is off by a few ulp of its score, so where scores reach 8 times
those of the other tests (128 in base 2) so does the bound, WIDE; outputs are measured against the range of
the V rows that carry the weight."""
import numpy as np
import pytest
import torch

from kv4_cases import MASS, MAX, SCALE, PagedCase, assert_lse_close, assert_out_close, full, gauss, local
from oracle import oda_oracle as O
from sparse_kv_recall_b200 import build as B
from sparse_kv_recall_b200 import oda

pytestmark = pytest.mark.gpu
WIDE = 8
GROUPS = pytest.mark.parametrize("G", [1, 2, 4])


@pytest.fixture(scope="module", autouse=True)
def _library():
    B.build()
    oda.load()


def _decode(c, vis=None, scale=SCALE, dtype=torch.float32):
    out, lse = c.out(dtype, fill=3.0)
    oda.oda_kv4_decode(c.kv, full() if vis is None else vis, c.q, scale, out, c.ws, lse=lse)
    c.ok()
    return out, lse


@GROUPS
def test_a_nan_in_q_shows_however_many_ctas_share_the_history(G):
    """In its own head alone, from one CTA a (sequence, KV head) to some dozens."""
    c = PagedCase([50, 700, 3000, 20000], 2 * G, 2, seed=400)
    ref, rlse, _ = c.oracle(lambda b, t: O.full_positions(t))
    last = 2 * G - 1
    c.q[:, last, 77] = float("nan")
    out, lse = _decode(c)
    assert torch.isnan(out[:, last]).all() and torch.isnan(lse[:, last]).all()
    assert_out_close(out[:, :last], ref[:, :last])
    assert_lse_close(lse[:, :last].cpu().numpy(), rlse[:, :last])


@pytest.mark.parametrize("rows", [slice(None), slice(0, 5), slice(2990, 3000)])
def test_a_nan_in_k_shows_however_many_ctas_share_the_history(rows):
    n = 3000
    kv = [gauss((n, 1, 128), 410 + i) for i in range(2)]
    kv[0][rows, 0, 3] = float("nan")
    c = PagedCase([n], 2, 1, seed=412, rows=kv)
    out, lse = _decode(c)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def _share_pages(c, times):
    """`times` sequences of other queries over the pages of c's one: many steps a warp."""
    c.B, c.lengths = times, c.lengths * times
    c.bt = c.bt.expand(times, -1).contiguous()
    c.seq_lens = c.seq_lens.expand(times).contiguous()
    c.bt_h = c.bt.cpu().numpy()
    c.q = gauss((times, c.hq, 128), 423)
    c.kv = oda.make_kv4(c.cache, c.bt, c.seq_lens, c.status, c.stats)
    c.ws = torch.zeros(oda.oda_kv4_decode_workspace_size(times, c.hkv, c.hq), dtype=torch.uint8, device="cuda")


@GROUPS
@pytest.mark.parametrize("times", [1, 12])
@pytest.mark.parametrize("k", [0, 28, 40, 60])
def test_v_rows_that_lost_their_weight_leave_the_others_exact(G, times, k):
    """Runs of 256 positions in turn (a warp's successive steps are 256 apart): V rows 2^k times as large at scores
    91.8 lower in base 2, then ordinary rows. What the former add is at most 5 x 2^(60 - 91.8); the latter
    have to come out as if they were alone. With 12 sequences a warp takes four steps and more."""
    n, hkv = 12000, 2
    kk, vv = gauss((n, hkv, 128), 420).float(), gauss((n, hkv, 128), 421).float()
    low = (torch.arange(n, device="cuda") // 256 % 2 == 0).view(-1, 1)
    kk[..., 0] = torch.where(low, 0.0, 45.0)
    vv *= torch.where(low, 2.0 ** k, 1.0)[..., None]
    c = PagedCase([n], G * hkv, hkv, seed=422, rows=(kk.to(torch.bfloat16), vv.to(torch.bfloat16)))
    if times > 1:
        _share_pages(c, times)
    c.q[..., 0] = 16.0
    out, lse = _decode(c)
    ref, rlse, _ = c.oracle(lambda b, t: O.full_positions(t))
    assert np.abs(out.double().cpu().numpy() - ref).max() <= MAX * WIDE
    assert np.abs(lse.double().cpu().numpy() - rlse).max() <= 1e-4 * WIDE


@GROUPS
@pytest.mark.parametrize("power", [-105, 123])
def test_v_of_every_magnitude(G, power):
    """The largest rows reach 2^125.5, the span of a group 2^126.5. Scores are 7.1 in base 2 higher in every
    other run of 256 positions: just not enough for the softmax to take a new maximum."""
    n, hkv = 1500, 2
    k, v = gauss((n, hkv, 128), 432).float(), gauss((n, hkv, 128), 430).float() * 2.0 ** power
    k[..., 0] = torch.where(torch.arange(n, device="cuda") // 256 % 2 == 0, 0.0, 3.5).view(-1, 1)
    c = PagedCase([n], G * hkv, hkv, seed=431, rows=(k.to(torch.bfloat16), v.to(torch.bfloat16)))
    c.q[..., 0] = 16.0
    out, lse = _decode(c)
    ref, rlse, _ = c.oracle(lambda b, t: O.full_positions(t))
    assert np.abs(out.double().cpu().numpy() - ref).max() <= MAX * 2.0 ** power
    assert_lse_close(lse.cpu().numpy(), rlse)


@GROUPS
@pytest.mark.parametrize("n", [1, 40, 3000, 40000])
def test_v_rows_of_the_largest_value(G, n):
    """Every weight alike, every value the largest bf16 (0.4 % below the largest fp32): the mean is that value, to
    the rounding of the sums (n 2^-24 at the very most, in fact a few ulp: 1e-5)."""
    big = float(torch.finfo(torch.bfloat16).max)
    v = torch.full((n, 1, 128), big, dtype=torch.bfloat16, device="cuda")
    v[..., 64:] = -big
    c = PagedCase([n], G, 1, seed=433, rows=(gauss((n, 1, 128), 434), v))
    c.q.zero_()
    out, lse = _decode(c)
    assert (out[..., :64].double() / big - 1).abs().max() <= 1e-5
    assert (out[..., 64:].double() / -big - 1).abs().max() <= 1e-5
    assert (lse.double() - np.log(n)).abs().max() <= 1e-5


@GROUPS
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("power", [10, 20, 52])
def test_scores_of_every_magnitude(G, sign, power):
    """K rows that are all alike: whatever the score (2^24 to 2^108 in base 2), every weight is 1 / n and the output
    is the mean of V; the log-sum is the score to fp32's rounding. Lengths from one token up, hidden rows among
    them; 29 pages in all, so that one CTA has them (between CTAs the weights go by fp32 log-sums, a unit of
    which is more than 1 here)."""
    lens = [1, 2, 17, 400]
    v = gauss((sum(lens), 1, 128), 440)
    k = torch.full((sum(lens), 1, 128), sign * 2.0 ** power, dtype=torch.bfloat16, device="cuda")
    c = PagedCase(lens, G, 1, seed=441, rows=(k, v))
    c.q.fill_(2.0 ** power)
    for vis, pos in ((full(), lambda b, t: O.full_positions(t)), (local(3, 20), lambda b, t: O.local_positions(t, 3, 20))):
        out, lse = _decode(c, vis)
        ref, rlse, _ = c.oracle(pos)
        assert_out_close(out, ref)
        assert np.abs(lse.double().cpu().numpy() / rlse - 1).max() <= 2.0 ** -20


@GROUPS
@pytest.mark.parametrize("power", [-112, -40, 40, 110])
def test_k_of_every_magnitude(G, power):
    """q as far the other way: ordinary scores."""
    lens = [5, 1500]
    k = gauss((sum(lens), 2, 128), 442).float() * 2.0 ** power
    c = PagedCase(lens, 2 * G, 2, seed=443, rows=(k.to(torch.bfloat16), gauss((sum(lens), 2, 128), 444)))
    c.q.copy_((c.q.float() * 2.0 ** -power).to(torch.bfloat16))
    out, lse = _decode(c)
    ref, rlse, _ = c.oracle(lambda b, t: O.full_positions(t))
    assert_out_close(out, ref)
    assert_lse_close(lse.cpu().numpy(), rlse)


@GROUPS
@pytest.mark.parametrize("scale", [1e-8, 1e-30])
def test_scores_that_vanish_hide_what_they_should(G, scale):
    """q of zeros and a scale so small that its product with q's power of two is below fp32's range: every
    visible weight is 1 / n, rows behind t and between sink and window stay hidden."""
    lens = [1, 5, 17, 1000]
    c = PagedCase(lens, 2 * G, 2, seed=445)
    c.q.zero_()
    ref, rlse, _ = c.oracle(lambda b, t: O.local_positions(t, 3, 20))
    out, lse = _decode(c, local(3, 20), scale)
    assert_out_close(out, ref)
    assert_lse_close(lse.cpu().numpy(), rlse)


@GROUPS
@pytest.mark.parametrize("kv4", [False, True])
def test_a_nan_in_q_shows_in_the_weights(kv4, G):
    """In the output, log-sum and weights of its own head and KV head alone, from one CTA to many."""
    lens = [1, 50, 3000]
    c = PagedCase(lens, 2 * G, 2, seed=450, kv4=kv4)
    ref, rlse, want = c.oracle(lambda b, t: O.full_positions(t))
    last = 2 * G - 1
    c.q[:, last, 77] = float("nan")
    out, lse = c.out(fill=3.0)
    mass = torch.full((3, 2, c.maxb * 16), 2.0, device="cuda")
    call = oda.oda_kv4_decode_mass if kv4 else oda.oda_decode_mass
    call(c.kv, full(), c.q, SCALE, out, c.ws, mass, mass_in=mass, lse=lse)
    c.ok()
    assert torch.isnan(out[:, last]).all() and torch.isnan(lse[:, last]).all()
    assert_out_close(out[:, :last], ref[:, :last])
    assert_lse_close(lse[:, :last].cpu().numpy(), rlse[:, :last])
    for b, n in enumerate(lens):
        assert torch.isnan(mass[b, 1, :n]).all() and (mass[b, :, n:] == 2.0).all()
        assert np.abs(mass[b, 0, :n].double().cpu().numpy() - 2.0 - want[b][1][0]).max() <= MASS + 2.0 ** -22


def test_a_nan_shows_when_shards_are_merged():
    """Parts of a history by 4-bit shards, some past its end (empty): a head whose scores are NaN stays NaN."""
    c = PagedCase([700, 3000], 4, 2, seed=460)
    ref, rlse, _ = c.oracle(lambda b, t: O.full_positions(t))
    c.q[:, 3, 5] = float("nan")
    parts = [_decode(c, oda.shard_visibility(lo, hi)) for lo, hi in ((0, 256), (256, 1024), (1024, 4096), (4096, 8192))]
    out, lse = c.out(fill=3.0)
    oda.oda_merge_partials(torch.stack([o for o, _ in parts]), torch.stack([l for _, l in parts]), out, lse=lse)
    c.ok()
    assert torch.isnan(out[:, 3]).all() and torch.isnan(lse[:, 3]).all()
    assert_out_close(out[:, :3], ref[:, :3])
    assert_lse_close(lse[:, :3].cpu().numpy(), rlse[:, :3])
