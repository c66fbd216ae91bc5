"""The 4-bit KV cache and the cache eviction operators, as cases that can be measured: the append of
rows to a 4-bit paged cache, decode attention over it, decode attention that accumulates the
attention weight of every cached position, and the eviction of the positions with the least
accumulated weight.

With `own` false, `run` computes them in plain elementary torch operations in 32 bits; with `own`
true it makes the calls of sparse_kv_recall_b200.oda.

The 4-bit page of one KV head (2304 bytes) holds 16 tokens: K codes [16][64 bytes], V codes
[16][64 bytes], meta [16][4 words]. A row's 128 dims are two groups of 64; the 32-bit word 2 i + g of
a row holds dims 64 g + 8 i .. + 7 in its nibbles, lowest first. The meta words of a token are
(K group 0, K group 1, V group 0, V group 1), each a bf16 scale in the low half and a bf16 minimum in
the high half. A code c stands for minimum + c * scale.
"""
import math
import random

import torch

own = False

PAGE = 16
DIM = 128
PAGE_BYTES = 2304
SCALE = 1.0 / math.sqrt(DIM)


# ---- cases -------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step's rows of eight sequences (the 16K serving batch)
        _append("append step b8", batch=8, hq=16, hkv=8, lo=16384, hi=16384, rows=1, lens_seed=1),
        # ragged prompts written in one chunk each, K/V taken out of a fused projection
        _append("append prompts b5", batch=5, hq=32, hkv=8, lo=37, hi=9001, rows=0, lens_seed=2),
        # the 4K reference workload: Local attention of one sequence, the step's rows committed
        _decode("kv4 local 4k b1", mode="local", batch=1, hq=16, hkv=8, lo=4097, hi=4097, sink=4,
                window=256, commit=True, f32=True, lens_seed=3),
        # 16K histories, eight sequences: the serving batch
        _decode("kv4 full 16k b8", mode="full", batch=8, hq=16, hkv=8, lo=16385, hi=16385, lens_seed=4),
        # one 128K history
        _decode("kv4 full 128k b1", mode="full", batch=1, hq=16, hkv=8, lo=131073, hi=131073, f32=True,
                lens_seed=5),
        # ragged 8K..64K, sixteen sequences, four query heads per KV head
        _decode("kv4 full ragged b16", mode="full", batch=16, hq=32, hkv=8, lo=8192, hi=65536, lens_seed=6),
        # declared modes over long histories: one region of 32K, its sink page and the recent 2048
        _decode("kv4 focus 256k b2", mode="focus", batch=2, hq=32, hkv=8, lo=200001, hi=262144, lens_seed=7),
        # one decode step of a cache that is about to be evicted, 4-bit and bf16
        _mass("kv4 mass 16k b8", bits=4, batch=8, hq=16, hkv=8, lo=9000, hi=16385, lens_seed=8),
        _mass("mass 32k b2", bits=16, batch=2, hq=32, hkv=8, lo=32769, hi=32769, f32=True, lens_seed=9),
        # a full budget after 256 more steps, one sequence
        _evict("evict 2304 b1", bits=16, batch=1, hkv=8, lo=2304, hi=2304, sink=4, recent=1024, budget=2048,
               lens_seed=10),
        # long prompts cut down to 4K after the prefill
        _evict("evict 32k b4", bits=16, batch=4, hkv=8, lo=20011, hi=32768, sink=4, recent=2048, budget=4096,
               lens_seed=11),
        # a ragged batch of 4-bit caches, some still below the budget
        _evict("kv4 evict 8k b16", bits=4, batch=16, hkv=8, lo=1500, hi=8200, sink=4, recent=512, budget=2049,
               lens_seed=12),
    ]


def _append(name, **kw):
    return {"name": name, "op": "append", **kw}


def _decode(name, **kw):
    return {"name": name, "op": "decode", "bits": 4, "sink": 4, "window": 2048, "commit": False, "f32": False, **kw}


def _mass(name, **kw):
    return {"name": name, "op": "mass", "mode": "full", "sink": 4, "window": 2048, "f32": False, **kw}


def _evict(name, **kw):
    return {"name": name, "op": "evict", **kw}


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4])
    batch = _spread(rng, 1, 16)
    op = rng.choice(["append", "decode", "mass", "evict"])
    bits = rng.choice([4, 16])
    hi = _spread(rng, 1, min(131072, 600000 // (batch * hkv)))
    lo = _spread(rng, max(1, hi // 8), hi)
    case = {"op": op, "batch": batch, "hkv": hkv, "lo": lo, "hi": hi, "lens_seed": rng.randrange(1 << 20)}
    if op == "append":
        case.update(hq=hq, rows=rng.choice([0, 1, 1 + lo // 3]))
    elif op == "evict":
        budget = _spread(rng, 1, max(1, min(8192, hi)))
        recent = rng.randint(0, budget)
        case.update(bits=bits, sink=min(rng.choice([0, 1, 4, 20]), budget - recent), recent=recent, budget=budget)
    else:
        mode = rng.choice(["local", "full", "focus"] if op == "decode" else ["local", "full"])
        case.update(hq=hq, bits=4 if op == "decode" else bits, mode=mode, sink=rng.choice([0, 4, 17]),
                    window=_spread(rng, 1, 4096), f32=rng.random() < 0.5)
        if op == "decode":
            case["commit"] = mode != "focus" and rng.random() < 0.5
    return case


def _lengths(case):
    r = random.Random(case["lens_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _rows(case):
    """Rows appended to each sequence (0: the whole prompt)."""
    return [n if case["rows"] == 0 else min(n, case["rows"]) for n in _lengths(case)]


def _visible_count(case, n):
    if case["mode"] == "local":
        return min(n, case["sink"] + case["window"])
    if case["mode"] == "focus":
        return min(n, PAGE + FOCUS + RECENT)
    return n


FOCUS, RECENT = 32768, 2048


def work(case):
    """Bytes: a row of one KV head, K and V, is 512 in bf16 and 144 in 4 bits."""
    lens, hkv = _lengths(case), case["hkv"]
    if case["op"] == "append":
        rows = sum(_rows(case)) * hkv
        return {"bytes": rows * (512 + 144 + 512), "flops": rows * 256 * 6}
    width = 144 if case["bits"] == 4 else 512
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens) * hkv
        back = 512 if case["bits"] == 4 else 0   # the kept rows' values
        return {"bytes": 4 * sum(lens) * hkv + kept * (2 * width + back + 8), "flops": sum(lens) * hkv}
    seen = sum(_visible_count(case, n) for n in lens)
    total = seen * hkv * width + case["batch"] * case["hq"] * DIM * (2 + (4 if case["f32"] else 2))
    if case["op"] == "mass":
        total += 8 * sum(lens) * hkv
    return {"bytes": total, "flops": 4 * seen * case["hq"] * DIM}


# ---- inputs ------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, batch, hkv, lens = case["op"], case["batch"], case["hkv"], _lengths(case)
    s = {"case": case}
    pages = [-(-n // PAGE) for n in lens]
    maxb = max(pages)
    dst_pages = -(-case["budget"] // PAGE) if op == "evict" else 0
    num_blocks = sum(pages) + batch * dst_pages + 3
    perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((batch, maxb), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = perm[at:at + k]
        at += k
    s["block_table"] = table
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    shape = (num_blocks, hkv, PAGE, DIM)
    if op == "append" or case["bits"] == 4:
        cache = torch.empty((num_blocks, hkv, PAGE_BYTES), dtype=torch.uint8, device="cuda")
        for i in range(0, num_blocks, 4096):
            k, v = (torch.randn((min(4096, num_blocks - i),) + shape[1:], generator=g, device="cuda")
                    .to(torch.bfloat16) for _ in range(2))
            cache[i:i + 4096] = _pack(*_quantise(k), *_quantise(v))
        s["cache"] = cache
    else:
        for name in ("k_cache", "v_cache"):
            c = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
            c.normal_(generator=g)
            s[name] = c
    if op == "append":
        rows = _rows(case)
        s["cu_rows"] = torch.tensor([0] + rows, dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32)
        heads = case["hq"] + 2 * hkv
        qkv = torch.randn((sum(rows), heads, DIM), generator=g, device="cuda").to(torch.bfloat16)
        s["k_new"], s["v_new"] = qkv[:, case["hq"]:case["hq"] + hkv], qkv[:, case["hq"] + hkv:]
    if op in ("decode", "mass"):
        s["q"] = torch.randn((batch, case["hq"], DIM), generator=g, device="cuda").to(torch.bfloat16)
        s["k_new"] = s["v_new"] = None
        if case.get("commit"):
            s["k_new"], s["v_new"] = (torch.randn((batch, hkv, DIM), generator=g, device="cuda")
                                      .to(torch.bfloat16) for _ in range(2))
        if case["mode"] == "focus":   # the focused region starts anywhere before the recent rows
            r = random.Random(int(seed))
            off = [r.randint(0, max(0, n - FOCUS - RECENT)) for n in lens]
            s["modes"] = torch.ones(batch, dtype=torch.int32, device="cuda")
            s["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
    if op in ("mass", "evict"):   # accumulated softmax weights: heavy-tailed, many of them alike
        m = torch.randn((batch, hkv, maxb * PAGE), generator=g, device="cuda").mul_(2.0).exp_()
        m = torch.round(m * 64) / 64 if op == "evict" else m
        s["mass"] = m.masked_fill_(torch.arange(maxb * PAGE, device="cuda") >= s["seq_lens"][:, None, None], 0.0)
    if op == "evict":
        s["dst_table"] = perm[at:at + batch * dst_pages].view(batch, dst_pages).contiguous()
    if own:
        s["calls"] = _handles(s)
    return s


def _handles(s):
    """The handles, workspaces and output buffers that a user's program keeps."""
    from sparse_kv_recall_b200 import oda
    case, h = s["case"], {}
    batch, hkv, maxb = case["batch"], case["hkv"], s["block_table"].shape[1]
    if "cache" in s:
        h["kv"] = oda.make_kv4(s["cache"], s["block_table"], s["seq_lens"])
    else:
        h["kv"] = oda.make_kv(s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"])

    def empty(shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def workspace(n):
        return torch.zeros(n, dtype=torch.uint8, device="cuda")
    if case["op"] == "append":
        h["k_out"], h["v_out"] = (empty((s["k_new"].shape[0], hkv, DIM), torch.bfloat16) for _ in range(2))
    elif case["op"] == "evict":
        h["kept"] = empty((batch, hkv, case["budget"]), torch.int32)
        h["mass_out"] = torch.zeros_like(s["mass"])
        h["lens_out"] = empty((batch,), torch.int32)
        h["ws"] = workspace(oda.oda_kv_evict_workspace_size(batch))
        if case["bits"] == 4:
            total = sum(min(n, case["budget"]) for n in _lengths(case))
            cu = [0]
            for n in _lengths(case):
                cu.append(cu[-1] + min(n, case["budget"]))
            h["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            h["k_out"], h["v_out"] = (empty((total, hkv, DIM), torch.bfloat16) for _ in range(2))
            h["dst"] = oda.make_kv4(s["cache"], s["dst_table"], h["lens_out"])
    else:
        hq = case["hq"]
        h["out"] = empty((batch, hq, DIM), torch.float32 if case["f32"] else torch.bfloat16)
        h["lse"] = empty((batch, hq))
        if case["mode"] == "local":
            h["vis"] = oda.oda_visibility(mode=oda.ODA_MODE_LOCAL, sink=case["sink"], window=case["window"])
        elif case["mode"] == "focus":
            h["vis"] = oda.da_visibility(s["modes"], s["offsets"], focus_len=FOCUS, recent=RECENT)
        else:
            h["vis"] = oda.oda_visibility(mode=oda.ODA_MODE_FULL, window=1)
        if case["op"] == "mass":
            size = oda.oda_kv4_decode_mass_workspace_size if case["bits"] == 4 else oda.oda_decode_mass_workspace_size
            h["ws"] = workspace(size(batch, hkv, hq, maxb))
            h["mass_out"] = torch.zeros_like(s["mass"])
        else:
            h["ws"] = workspace(oda.oda_kv4_decode_workspace_size(batch, hkv, hq))
        if case.get("commit"):
            h["k_out"], h["v_out"] = (empty((batch, hkv, DIM), torch.bfloat16) for _ in range(2))
    return h


# ---- one pass ----------------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from sparse_kv_recall_b200 import oda
    case, h = s["case"], s["calls"]
    kv, op = h["kv"], case["op"]
    if op == "append":
        oda.oda_kv4_append(kv, s["k_new"], s["v_new"], cu_rows=s["cu_rows"])
        oda.oda_kv4_read(kv, h["k_out"], h["v_out"], cu_rows=s["cu_rows"])
        return {"k": h["k_out"], "v": h["v_out"]}
    if op == "decode":
        oda.oda_kv4_decode(kv, h["vis"], s["q"], SCALE, h["out"], h["ws"], k_new=s["k_new"], v_new=s["v_new"],
                           lse=h["lse"])
        if not case["commit"]:
            return {"out": h["out"], "lse": h["lse"]}
        oda.oda_kv4_read(kv, h["k_out"], h["v_out"])
        return {"out": h["out"], "lse": h["lse"], "k": h["k_out"], "v": h["v_out"]}
    if op == "mass":
        call = oda.oda_kv4_decode_mass if case["bits"] == 4 else oda.oda_decode_mass
        call(kv, h["vis"], s["q"], SCALE, h["out"], h["ws"], h["mass_out"], mass_in=s["mass"], lse=h["lse"])
        return {"out": h["out"], "lse": h["lse"], "mass": h["mass_out"]}
    call = oda.oda_kv4_evict if case["bits"] == 4 else oda.oda_kv_evict
    call(kv, s["mass"], case["sink"], case["recent"], case["budget"], s["dst_table"], h["kept"], h["mass_out"],
         h["lens_out"], h["ws"])
    got = {"kept": h["kept"], "mass": h["mass_out"], "lens": h["lens_out"]}
    if case["bits"] == 4:
        oda.oda_kv4_read(h["dst"], h["k_out"], h["v_out"], cu_rows=h["cu"])
        return {**got, "k": h["k_out"], "v": h["v_out"]}
    return {**got, "k": s["k_cache"], "v": s["v_cache"]}


def _quantise(x):
    """bf16 [..., 128] -> codes uint8 [..., 128], scale and minimum fp32 [..., 2]."""
    x = x.float().unflatten(-1, (2, 64))
    lo, hi = x.amin(-1), x.amax(-1)
    step = (hi - lo) / torch.full_like(lo, 15.0)   # by a tensor: the quotient itself, no reciprocal
    scale = ((step.view(torch.int32) + 0xffff) & -0x10000).view(torch.float32)   # up to bf16
    codes = torch.round((x - lo[..., None]) / torch.where(scale > 0, scale, 1.0)[..., None])
    return codes.clamp_(0, 15).to(torch.uint8).flatten(-2), scale, lo


def _pack_row(codes):
    """codes uint8 [..., 128] -> bytes uint8 [..., 64]."""
    c = codes.unflatten(-1, (2, 8, 8)).transpose(-3, -2)          # [..., i, group, nibble]
    return (c[..., 0::2] | (c[..., 1::2] << 4)).flatten(-3)


def _pack_meta(scale, lo):
    """fp32 [..., 2] each -> bytes uint8 [..., 8]."""
    return torch.stack([scale, lo], -1).to(torch.bfloat16).contiguous().view(torch.uint8).flatten(-2)


def _pack(kc, ks, km, vc, vs, vm):
    meta = torch.cat([_pack_meta(ks, km), _pack_meta(vs, vm)], -1)
    return torch.cat([_pack_row(kc).flatten(-2), _pack_row(vc).flatten(-2), meta.flatten(-2)], -1)


def _values(rows, meta):
    """bytes [..., 64] and their meta bytes [..., 8] -> fp32 [..., 128]."""
    nib = torch.stack([rows & 15, rows >> 4], -1).flatten(-2)     # [..., (i, group, nibble)]
    nib = nib.unflatten(-1, (8, 2, 8)).transpose(-3, -2).flatten(-2)   # [..., group, 64]
    m = meta.contiguous().view(torch.bfloat16).unflatten(-1, (2, 2)).float()
    return (nib.float().mul_(m[..., 0:1]).add_(m[..., 1:2])).flatten(-2)


def _unpack(p):
    """pages uint8 [..., 2304] -> K and V fp32 [..., 16, 128]."""
    meta = p[..., 2048:].unflatten(-1, (PAGE, 16))
    return (_values(p[..., :1024].unflatten(-1, (PAGE, 64)), meta[..., :8]),
            _values(p[..., 1024:2048].unflatten(-1, (PAGE, 64)), meta[..., 8:]))


def _visible_pages(s):
    """Logical pages [B, L] that the rule may touch, and which of their positions it sees [B, L, 16]."""
    case, t = s["case"], s["seq_lens"].long()[:, None] - 1
    maxb = s["block_table"].shape[1]
    if case["mode"] == "local":   # the sink's pages, then the window's that are not among them
        w0 = (t - case["window"] + 1).clamp(min=0)
        first = -(-case["sink"] // PAGE)
        a = torch.arange(min(first, maxb), device="cuda")[None].expand(len(t), -1)
        n = min(maxb, (case["window"] + PAGE - 2) // PAGE + 1)
        b = w0 // PAGE + torch.arange(n, device="cuda")
        pages, ok = torch.cat([a, b], 1), torch.cat([a >= 0, b >= first], 1)
    else:
        pages = torch.arange(maxb, device="cuda")[None].expand(len(t), -1)
        ok = pages >= 0
    p = pages[..., None] * PAGE + torch.arange(PAGE, device="cuda")
    t = t[..., None]
    seen = ok[..., None] & (p <= t)
    if case["mode"] == "local":
        seen &= (p < case["sink"]) | (p > t - case["window"])
    elif case["mode"] == "focus":
        off = s["offsets"].long()[:, None]
        end = torch.minimum(off + FOCUS - 1, t[..., 0])
        kept = (pages == 0) | ((pages >= off // PAGE) & (pages <= end // PAGE) & (off <= end))
        kept |= pages >= (t[..., 0] - RECENT + 1).clamp(min=0) // PAGE
        seen &= kept[..., None]
    return pages.clamp(max=maxb - 1), seen


def _attend(s):
    """out fp32, lse and the softmax weights [B, Hkv, G, L * 16] with their pages and visibility."""
    case = s["case"]
    pages, seen = _visible_pages(s)
    phys = torch.gather(s["block_table"].long(), 1, pages).clamp(min=0)
    if case["bits"] == 4:
        k, v = _unpack(s["cache"][phys].transpose(1, 2).contiguous())
    else:
        k, v = (s[n][phys].transpose(1, 2).float() for n in ("k_cache", "v_cache"))
    k, v = k.flatten(2, 3), v.flatten(2, 3)
    dead = ~seen.flatten(1)[:, None, None]
    q = s["q"].float().unflatten(1, (case["hkv"], -1))
    x = (torch.matmul(q, k.transpose(-1, -2)) * SCALE).masked_fill_(dead, -math.inf)
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - top)
    total = w.sum(-1, keepdim=True)
    w = w / total
    out = torch.matmul(w, v)
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.flatten(1, 2).to(torch.float32 if case["f32"] else torch.bfloat16)
    return out, lse.flatten(1), w, pages


def _slots(s, rows):
    """(sequence, physical page, row in it) of appended row i."""
    cu = s["cu_rows"].long()
    i = torch.arange(rows, device="cuda")
    b = torch.searchsorted(cu, i, right=True) - 1
    p = s["seq_lens"].long()[b] - (cu[b + 1] - cu[b]) + (i - cu[b])
    return s["block_table"][b, p // PAGE].long(), p % PAGE


def _store(cache, page, row, k, v):
    """Quantise rows [N, Hkv, 128] into cache[page[i], :, row[i]]; their values as they stand there."""
    (kc, ks, km), (vc, vs, vm) = _quantise(k), _quantise(v)
    meta = torch.cat([_pack_meta(ks, km), _pack_meta(vs, vm)], -1)
    cache[..., :1024].unflatten(-1, (PAGE, 64))[page, :, row] = _pack_row(kc)
    cache[..., 1024:2048].unflatten(-1, (PAGE, 64))[page, :, row] = _pack_row(vc)
    cache[..., 2048:].unflatten(-1, (PAGE, 16))[page, :, row] = meta
    return _load(cache, page, row)


def _load(cache, page, row):
    meta = cache[..., 2048:].unflatten(-1, (PAGE, 16))[page, :, row]
    k = _values(cache[..., :1024].unflatten(-1, (PAGE, 64))[page, :, row], meta[..., :8])
    v = _values(cache[..., 1024:2048].unflatten(-1, (PAGE, 64))[page, :, row], meta[..., 8:])
    return {"k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "append":
        return _store(s["cache"], *_slots(s, s["k_new"].shape[0]), s["k_new"], s["v_new"])
    if op == "decode":
        rows = {}
        if case["commit"]:
            t = s["seq_lens"].long() - 1
            page = torch.gather(s["block_table"].long(), 1, (t // PAGE)[:, None])[:, 0]
            rows = _store(s["cache"], page, t % PAGE, s["k_new"], s["v_new"])
        out, lse, _, _ = _attend(s)
        return {"out": out, "lse": lse, **rows}
    if op == "mass":
        out, lse, w, pages = _attend(s)
        at = (pages[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(1)
        add = torch.zeros_like(s["mass"]).scatter_add_(2, at[:, None].expand(-1, case["hkv"], -1), w.sum(2))
        return {"out": out, "lse": lse, "mass": s["mass"] + add}
    return _evict_plain(s)


def _evict_plain(s):
    case, mass = s["case"], s["mass"]
    batch, hkv, cap = mass.shape
    budget = case["budget"]
    n = s["seq_lens"].long()[:, None, None]
    p = torch.arange(cap, device="cuda")[None, None]
    forced = (p < case["sink"]) | (p >= n - case["recent"])
    key = mass.masked_fill(forced, math.inf).masked_fill(p >= n, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.where(order < n, order, cap).sort(-1).values
    if order.shape[-1] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]), value=cap)
    live = order < cap
    src = order.clamp(max=cap - 1)
    new_mass = torch.zeros_like(mass)
    w = min(budget, cap)
    new_mass[..., :w] = torch.where(live, torch.gather(mass, 2, src), 0.0)[..., :w]
    b, g, i = live.nonzero(as_tuple=True)
    at = src[b, g, i]
    sp, dp = s["block_table"][b, at // PAGE].long(), s["dst_table"][b, i // PAGE].long()
    got = {"kept": torch.where(live, order, -1).to(torch.int32), "mass": new_mass,
           "lens": s["seq_lens"].clamp(max=budget)}
    if case["bits"] == 4:
        for lo, hi, width in ((0, 1024, 64), (1024, 2048, 64), (2048, 2304, 16)):
            part = s["cache"][..., lo:hi].unflatten(-1, (PAGE, width))
            part[dp, g, i % PAGE] = part[sp, g, at % PAGE]
        bb, ii = live[:, 0].nonzero(as_tuple=True)
        return {**got, **_load(s["cache"], s["dst_table"][bb, ii // PAGE].long(), ii % PAGE)}
    for c in (s["k_cache"], s["v_cache"]):
        c[dp, g, i % PAGE] = c[sp, g, at % PAGE]
    return {**got, "k": s["k_cache"], "v": s["v_cache"]}


# ---- the definition in 64 bits -------------------------------------------------------------------
def exact(case, seed):
    """Each sequence and head by itself, in 64 bits, from the definitions."""
    s = prepare(case, seed)
    lens, op = _lengths(case), case["op"]
    if op == "append":
        return {"k": _round_trip(s["k_new"]), "v": _round_trip(s["v_new"])}
    if op == "evict":
        return _exact_evict(s, lens)
    batch, hkv, hq = case["batch"], case["hkv"], case["hq"]
    group = hq // hkv
    out = torch.zeros((batch, hq, DIM), dtype=torch.float64, device="cuda")
    lse = torch.zeros((batch, hq), dtype=torch.float64, device="cuda")
    mass = s["mass"].double() if op == "mass" else None
    for b, n in enumerate(lens):
        at = _positions(case, n, int(s["offsets"][b]) if "offsets" in s else 0)
        page, row = s["block_table"][b].long()[at // PAGE], at % PAGE
        for g in range(hkv):
            if case["bits"] == 4:
                raw = s["cache"][page, g]
                k, v = (_decode_64(raw, row, part) for part in (0, 1))
            else:
                k, v = (s[c][page, g, row].double() for c in ("k_cache", "v_cache"))
            if s["k_new"] is not None:
                k[-1], v[-1] = _round_trip(s["k_new"][b, g]), _round_trip(s["v_new"][b, g])
            for h in range(g * group, (g + 1) * group):
                z = k @ s["q"][b, h].double() / math.sqrt(DIM)
                lse[b, h] = torch.logsumexp(z, 0)
                p = torch.exp(z - lse[b, h])
                out[b, h] = p @ v
                if mass is not None:
                    mass[b, g, at] += p
    got = {"out": out, "lse": lse}
    if op == "mass":
        got["mass"] = mass
    elif case["commit"]:
        got.update(k=_round_trip(s["k_new"]), v=_round_trip(s["v_new"]))
    return got


def _positions(case, n, off):
    at = torch.arange(n, device="cuda")
    if case["mode"] == "local":
        return at[(at < case["sink"]) | (at >= n - case["window"])]
    if case["mode"] == "focus":
        page = at // PAGE
        return at[(page == 0) | ((page >= off // PAGE) & (page <= min(n - 1, off + FOCUS - 1) // PAGE))
                  | (page >= max(0, n - RECENT) // PAGE)]
    return at


def _round_trip(x):
    """What rows stand for after the 4 bits: every group's minimum plus a whole number of its scales."""
    x = x.double().reshape(x.shape[:-1] + (2, 64))
    lo = x.min(-1, keepdim=True).values
    step = (x.max(-1, keepdim=True).values - lo) / 15
    near = step.to(torch.bfloat16)
    up = torch.nextafter(near, torch.full_like(near, math.inf))
    scale = torch.where(near.double() >= step, near, up).double()
    code = torch.where(scale > 0, torch.round((x - lo) / scale), torch.zeros_like(x)).clamp(0, 15)
    return (lo + code * scale).reshape(x.shape[:-2] + (DIM,))


def _decode_64(raw, row, part):
    """Rows of page bytes [N, 2304] -> [N, 128] in 64 bits; part 0 is K, 1 is V."""
    dim = torch.arange(DIM, device=raw.device)
    word = 2 * ((dim % 64) // 8) + dim // 64
    at = 1024 * part + 64 * row[:, None] + 4 * word + (dim % 8) // 2
    code = (torch.gather(raw, 1, at) >> (4 * (dim % 2)).to(torch.uint8)) & 15
    half = raw[:, 2048:].contiguous().view(torch.bfloat16)
    meta = 8 * row[:, None] + 4 * part + 2 * (dim // 64)
    return torch.gather(half, 1, meta + 1).double() + code.double() * torch.gather(half, 1, meta).double()


def _exact_evict(s, lens):
    case, budget = s["case"], s["case"]["budget"]
    kept = torch.full((case["batch"], case["hkv"], budget), -1, dtype=torch.int32)
    mass_in, mass = s["mass"].double().cpu(), torch.zeros(s["mass"].shape, dtype=torch.float64)
    table, dst = s["block_table"].cpu().long(), s["dst_table"].cpu().long()
    rows = {"k": [], "v": []}
    for b, n in enumerate(lens):
        keep = min(n, budget)
        for g in range(case["hkv"]):
            m = mass_in[b, g, :n]
            free = torch.arange(min(case["sink"], n), max(min(case["sink"], n), n - case["recent"]))
            if n <= budget:
                at = torch.arange(n)
            else:
                best = free[torch.sort(-m[free], stable=True).indices[:budget - case["sink"] - case["recent"]]]
                at = torch.cat([torch.arange(case["sink"]), best.sort().values, torch.arange(n - case["recent"], n)])
            kept[b, g, :keep] = at.int()
            mass[b, g, :keep] = m[at]
            to, here = torch.arange(keep), at.cuda()
            page = table[b, at // PAGE].cuda()
            if case["bits"] == 16:
                for c in ("k_cache", "v_cache"):
                    s[c][dst[b, to // PAGE].cuda(), g, (to % PAGE).cuda()] = s[c][page, g, here % PAGE]
            else:
                for part, name in enumerate("kv"):
                    rows[name].append(_decode_64(s["cache"][page, g], here % PAGE, part))
    got = {"kept": kept.cuda(), "mass": mass.cuda(), "lens": torch.tensor([min(n, budget) for n in lens]).int().cuda()}
    if case["bits"] == 16:
        return {**got, "k": s["k_cache"].double(), "v": s["v_cache"].double()}
    hkv = case["hkv"]
    for name in "kv":
        seqs = [torch.stack(rows[name][b * hkv:(b + 1) * hkv], 1) for b in range(case["batch"])]
        got[name] = torch.cat(seqs)
    return got
