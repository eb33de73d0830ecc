"""Cases of the serving-cache operators: rotary positions with several axes, the write of new
tokens into a paged key/value cache, attention of a few new rows over that cache, and eviction
from it by accumulated attention weight.

`run` computes a case in its plain form (elementary torch operations, 32-bit arithmetic, angles
in 64 bits) or, with `own`, through the package's entry points.  `exact` is the same from the
definitions in 64 bits.
"""
import math

import torch

own = False

BF16, F32, F64, I32, I64 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64
FP8 = torch.float8_e4m3fn
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # q and k of a training step at the benchmark's sizes (B8 H32 N4096 d128), taken out of
        # the packed projection and rotated with the text/video axes (time, height, width)
        dict(name="rope_train_b8h32_t4096_d128", op="rope", B=8, Hq=32, Hk=32, T=4096, d=128, rot=128, axes=3,
             f32=False, interleaved=False, packed=True, inverse=False, far=0),
        # gradients of a fine-tuning step in fp32: odd length, interleaved pairs, half the head
        # rotated, two axes (height, width), positions far from zero
        dict(name="rope_grad_f32_b2h6_t1021_d64", op="rope", B=2, Hq=6, Hk=2, T=1021, d=64, rot=32, axes=2,
             f32=True, interleaved=True, packed=False, inverse=True, far=1000000),
        # one decoding step of eight sequences: one new token each
        dict(name="append_step_b8_d128", op="append", B=8, Hq=32, Hkv=8, T=1, lo=500, hi=4000, d=128, rot=128, axes=1,
             ps=16, fp8=False, ragged=False),
        # the prompts of four requests of different lengths, written as e4m3 in one call
        dict(name="append_prompts_fp8_b4_d128", op="append", B=4, Hq=32, Hkv=8, T=2011, lo=2100, hi=2500, d=128,
             rot=128, axes=3, ps=64, fp8=True, ragged=True),
        # the first token after a very short prompt: latency alone
        dict(name="decode_first_b1_l17_d128", op="decode", B=1, Hq=32, Hkv=8, Tq=1, lo=17, hi=17, d=128, ps=16,
             fp8=False, weights=False),
        # a serving batch of 64 sequences of ragged lengths, grouped heads, small pages
        dict(name="decode_batch_b64_d128", op="decode", B=64, Hq=32, Hkv=8, Tq=1, lo=200, hi=8000, d=128, ps=16,
             fp8=False, weights=False),
        # the decode workload of the benchmark (B8 H32, 32768 keys), every head its own keys
        dict(name="decode_long_b8h32_l32768_d128", op="decode", B=8, Hq=32, Hkv=32, Tq=1, lo=32768, hi=32768, d=128,
             ps=64, fp8=False, weights=False),
        # four rows of one sequence to verify against a 131072-token cache, wide pages
        dict(name="decode_rows4_b1_l131072_d128", op="decode", B=1, Hq=32, Hkv=8, Tq=4, lo=131072, hi=131072, d=128,
             ps=256, fp8=False, weights=False),
        # an e4m3 cache with narrow heads and lengths from short to 64K
        dict(name="decode_fp8_b16_d64", op="decode", B=16, Hq=16, Hkv=4, Tq=1, lo=1001, hi=65536, d=64, ps=32,
             fp8=True, weights=False),
        # a step under a bounded cache: attention weights added up per entry for eviction
        dict(name="decode_weights_b8_d128", op="decode", B=8, Hq=32, Hkv=8, Tq=1, lo=2900, hi=4111, d=128, ps=16,
             fp8=False, weights=True),
        # the bounded cache gives one page back
        dict(name="evict_page_b8_l4112_d128", op="evict", B=8, Hkv=8, lo=4112, hi=4112, budget=4096, first=4, recent=512,
             d=128, ps=16, fp8=False),
        # long prompts cut down to the budget before decoding
        dict(name="evict_prompt_b4_d128", op="evict", B=4, Hkv=8, lo=9001, hi=32768, budget=4096, first=4, recent=1024,
             d=128, ps=64, fp8=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "decode", "evict"])
    d = rng.choice([64, 128, 128, 256])
    ps = rng.choice([16, 32, 64, 128, 256])
    fp8 = rng.random() < 0.35
    if op == "rope":
        B, Hk, G = _log_int(rng, 1, 8), _log_int(rng, 1, 16), rng.choice([1, 2, 3, 4])
        T = max(1, min(_log_int(rng, 1, 8192), 8 * 32 * 4096 * 128 // (B * Hk * (G + 1) * d * 2)))
        return dict(op="rope", B=B, Hq=Hk * G, Hk=Hk, T=T, d=d, rot=rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)]),
                    axes=rng.randint(1, 4), f32=rng.random() < 0.3, interleaved=rng.random() < 0.4,
                    packed=rng.random() < 0.5, inverse=rng.random() < 0.5, far=rng.choice([0, 1000, 10 ** 6, 2 * 10 ** 9]))
    B = _log_int(rng, 1, 96)
    Hkv, G = rng.choice([1, 2, 3, 4, 8, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if op == "append":
        T = _log_int(rng, 1, max(1, min(3000, 60000000 // (B * Hkv * (G + 2) * d))))
        lo = T + rng.randint(0, 500)
        return dict(op="append", B=B, Hq=Hkv * G, Hkv=Hkv, T=T, lo=lo, hi=lo + rng.randint(0, 700), d=d,
                    rot=rng.choice([d, d // 2]), axes=rng.randint(1, 3), ps=ps, fp8=fp8, ragged=rng.random() < 0.5)
    if op == "evict":
        B = _log_int(rng, 1, 24)
        hi = _log_int(rng, 20, max(20, min(40000, 60000000 // (B * Hkv * d))))
        budget = _log_int(rng, 8, hi)
        first = min(rng.choice([0, 1, 4]), budget)
        return dict(op="evict", B=B, Hkv=Hkv, lo=rng.randint(1, hi), hi=hi, budget=budget, first=first,
                    recent=rng.randint(0, budget - first), d=d, ps=ps, fp8=fp8)
    hi = _log_int(rng, 1, max(1, min(100000, 400000000 // (B * Hkv * d))))
    return dict(op="decode", B=B, Hq=Hkv * G, Hkv=Hkv, Tq=rng.choice([1, 1, 1, 2, 4, 7]), lo=rng.randint(0, hi), hi=hi,
                d=d, ps=ps, fp8=fp8, weights=rng.random() < 0.3)


# ------------------------------------------------------------------ what the cases share
def _lens(c):
    """Lengths spread over [lo, hi], the last one hi."""
    return [c["hi"] - int((c["hi"] - c["lo"]) * ((b * 0.6180339887498949) % 1.0)) for b in range(c["B"])][::-1]


def _new_lens(c):
    """New tokens of each sequence of an append case."""
    return [c["T"] - (b * 977 % c["T"] if c["ragged"] else 0) for b in range(c["B"])][::-1]


def _freqs(rot):
    return [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]


def _axis(rot, axes):
    """Axis of each pair: the pairs in `axes` runs, the first one shorter (time takes fewer than
    height and width)."""
    n = rot // 2
    first = n if axes == 1 else max(1, n // (axes + 1))
    return [0 if i < first else 1 + (i - first) * (axes - 1) // (n - first) for i in range(n)]


def _positions(c, g, B, T, axes, far):
    """int32 [axes][B][T]: text up to a quarter of the row, then frames of a grid (time, height,
    width), shifted per sequence by up to 100 and by `far`."""
    t = torch.arange(T, device=DEV, dtype=I64)
    text = T // 4
    cell = (t - text).clamp(min=0)
    grid = torch.stack([cell // 384, cell // 24 % 16, cell % 24, cell % 7])[:axes] + text
    p = torch.where(t < text, t, grid) if axes > 1 else t[None]
    shift = torch.randint(0, 100, (1, B, 1), generator=g, device=DEV) + far
    return (p[:, None, :] + shift).to(I32).contiguous()


def _table(g, B, width):
    """Pages of each sequence, in no order, and the number of pages."""
    n = B * width
    return torch.randperm(n, generator=g, device=DEV).to(I32).view(B, width), n


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _pool(c, g, n):
    """A cache of n pages and one more that only the plain forms write (rows that are not there)."""
    shape = (n + 1, c["Hkv"], c["ps"], c["d"])
    if not c["fp8"]:
        return _randn(g, shape, BF16)
    x = torch.empty(shape, device=DEV, dtype=torch.uint8)
    flat = x.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_((_randn(g, part.shape, BF16) * 100).clamp(-448, 448).to(FP8).view(torch.uint8))
    return x


def _scales(c, g):
    return (0.5 + torch.rand(c["Hkv"], generator=g, device=DEV)) / 100 if c["fp8"] else None


def prepare(case, seed):
    c, g = case, torch.Generator(DEV).manual_seed(seed)
    s = dict(c=c)
    if c["op"] == "rope":
        B, Hq, Hk, T, d = c["B"], c["Hq"], c["Hk"], c["T"], c["d"]
        dt = F32 if c["f32"] else BF16
        def pair(make):
            if c["packed"]:   # the projection's [B][T][heads of q, k and v][d]
                x = make((B, T, Hq + 2 * Hk, d)).transpose(1, 2)
                return x[:, :Hq], x[:, Hq:Hq + Hk]
            return make((B, Hq, T, d)), make((B, Hk, T, d))
        def zeros(shape):
            return torch.zeros(shape, device=DEV, dtype=dt)
        packed_in = not c["inverse"]
        s["q"], s["k"] = pair(lambda sh: _randn(g, sh, dt)) if packed_in else \
            (_randn(g, (B, Hq, T, d), dt), _randn(g, (B, Hk, T, d), dt))
        s["qo"], s["ko"] = (zeros((B, Hq, T, d)), zeros((B, Hk, T, d))) if packed_in else pair(zeros)
        s["pos"] = _positions(c, g, B, T, c["axes"], c["far"])
    else:
        lens = _lens(c)
        B, Hkv, d, ps = c["B"], c["Hkv"], c["d"], c["ps"]
        width = -(-max(max(lens), 1) // ps)
        s["table"], n = _table(g, B, width)
        s["n"], s["lens"] = n, torch.tensor(lens, device=DEV, dtype=I32)
        s["kp"], s["vp"] = _pool(c, g, n), _pool(c, g, n)
        s["ks"], s["vs"] = _scales(c, g), _scales(c, g)
        cap = width * ps
        if c["op"] == "append":
            T = c["T"]
            s["q"], s["k"], s["v"] = (_randn(g, (B, h, T, d), BF16) for h in (c["Hq"], Hkv, Hkv))
            s["qo"] = torch.zeros_like(s["q"])
            s["new"] = torch.tensor(_new_lens(c), device=DEV, dtype=I32) if c["ragged"] else None
            s["pos"] = _positions(c, g, B, T, c["axes"], 500)
            s["weight"] = torch.ones((B, Hkv, cap), device=DEV)
            s["order"] = torch.full((B, Hkv, cap), -1, device=DEV, dtype=I32)
        elif c["op"] == "decode":
            s["q"] = _randn(g, (B, c["Hq"], c["Tq"], d), BF16)
            s["o"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((B, c["Hq"], c["Tq"]), device=DEV)
            if c["weights"]:
                s["weight"] = torch.rand((B, Hkv, cap), generator=g, device=DEV)
        else:
            # sums of attention weights: a few large, most small, those of entries just written 0
            w = torch.exp(2.0 * _randn(g, (B, Hkv, cap), F32)) / 100
            s["weight"] = torch.where(torch.rand((B, Hkv, cap), generator=g, device=DEV) < 0.03, 0.0, w)
            # arrival numbers out of order, as earlier evictions leave them
            seen = cap + 57
            s["order"] = torch.rand((B, Hkv, seen), generator=g, device=DEV).argsort(-1)[..., :cap].to(I32).contiguous()
            s["seen"] = torch.full((B,), seen, device=DEV, dtype=I32)
            s["weight_o"], s["order_o"] = torch.zeros_like(s["weight"]), torch.zeros_like(s["order"])
            s["lens_o"] = torch.zeros_like(s["lens"])
            s["kept"] = torch.full((B, Hkv, c["budget"]), -1, device=DEV, dtype=I32)
    if own:   # the handles that a program keeps: frequencies, the cache, a workspace
        from exact_io_aware_05_gb300 import fa
        s["fa"] = fa
        if c["op"] in ("rope", "append"):
            s["spec"] = fa.RopeSpec(c["d"], _freqs(c["rot"]), _axis(c["rot"], c["axes"]), interleaved=c.get("interleaved", False))
        if c["op"] != "rope":
            s["cache"] = fa.KVCache(s["kp"][:s["n"]], s["vp"][:s["n"]], s["table"], s["lens"], k_scale=s["ks"], v_scale=s["vs"],
                                    weight=s.get("weight"), order=s.get("order"), seen=s.get("seen"))
        if c["op"] == "decode":
            nb = fa.fa_decode_paged_workspace_bytes(s["cache"], c["Hq"], c["Tq"], accumulate=c["weights"])
            s["ws"] = torch.empty(max(nb, 256), dtype=torch.uint8, device=DEV)
    return s


def _whole(s, name):
    """The cache's pages; codes as the values they stand for (a view)."""
    x = s[name][:s["n"]]
    return x.view(FP8) if s["c"]["fp8"] else x


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    c, fa = s["c"], s["fa"]
    if c["op"] == "rope":
        (fa.fa_rope_bwd if c["inverse"] else fa.fa_rope)(s["q"], s["qo"], s["pos"], s["spec"], k=s["k"], k_out=s["ko"])
        return s["qo"], s["ko"]
    if c["op"] == "append":
        fa.fa_cache_append(s["cache"], s["k"], s["v"], s["pos"], s["spec"], q=s["q"], q_out=s["qo"], new_lens=s["new"])
        return s["qo"], _whole(s, "kp"), _whole(s, "vp"), s["weight"], s["order"]
    if c["op"] == "decode":
        fa.fa_decode_paged(s["cache"], s["q"], s["o"], s["lse"], c["d"] ** -0.5, s["ws"], causal=True, accumulate=c["weights"])
        return (s["o"], s["lse"], s["weight"]) if c["weights"] else (s["o"], s["lse"])
    fa.fa_cache_evict(s["cache"], c["budget"], s["weight_o"], s["order_o"], s["lens_o"], s["kept"], n_first=c["first"],
                      n_recent=c["recent"])
    return _whole(s, "kp"), _whole(s, "vp"), s["weight_o"], s["order_o"], s["lens_o"], s["kept"]


def _cos_sin(c, pos):
    """cos and sin of the angles, fp32 [B][1][T][rot / 2]; the angles in 64 bits."""
    axis = torch.tensor(_axis(c["rot"], c["axes"]), device=DEV)
    a = pos[axis].double() * torch.tensor(_freqs(c["rot"]), device=DEV, dtype=F64)[:, None, None]
    a = a.permute(1, 2, 0)[:, None]
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin, rot, interleaved):
    """x rotated, in fp32."""
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _keys(s, name, scale):
    """Keys or values of every sequence, fp32 [B][Hkv][table width * page size][d]."""
    x = s[name][s["table"].long()].permute(0, 2, 1, 3, 4).flatten(2, 3)
    return x.float() if scale is None else x.view(FP8).float() * scale[:, None, None]


def _codes(x, scale):
    """What the cache holds of fp32 x [B][Hkv][T][d]."""
    return x.to(BF16) if scale is None else (x / scale[:, None, None]).clamp(-448, 448).to(FP8).view(torch.uint8)


def _run_plain(s):
    c = s["c"]
    if c["op"] == "rope":
        cos, sin = _cos_sin(c, s["pos"])
        sin = -sin if c["inverse"] else sin
        s["qo"].copy_(_rotate(s["q"], cos, sin, c["rot"], c["interleaved"]))
        s["ko"].copy_(_rotate(s["k"], cos, sin, c["rot"], c["interleaved"]))
        return s["qo"], s["ko"]
    B, Hkv, d, ps, n = c["B"], c["Hkv"], c["d"], c["ps"], s["n"]
    lens, table = s["lens"].long(), s["table"].long()
    if c["op"] == "append":
        T = c["T"]
        cos, sin = _cos_sin(c, s["pos"])
        t = torch.arange(T, device=DEV)
        new = torch.full_like(lens, T) if s["new"] is None else s["new"].long()
        there = t < new[:, None]                                             # [B][T]
        s["qo"].copy_(torch.where(there[:, None, :, None], _rotate(s["q"], cos, sin, c["rot"], False), s["qo"].float()))
        slot = ((lens - new)[:, None] + t).clamp(max=s["weight"].shape[-1] - 1)
        page = torch.where(there, table.gather(1, slot // ps), n)            # rows that are not there go to the spare page
        row = slot % ps
        s["kp"][page, :, row] = _codes(_rotate(s["k"], cos, sin, c["rot"], False), s["ks"]).transpose(1, 2)
        s["vp"][page, :, row] = _codes(s["v"].float(), s["vs"]).transpose(1, 2)
        at = torch.arange(s["weight"].shape[-1], device=DEV)
        fresh = ((at >= (lens - new)[:, None]) & (at < lens[:, None]))[:, None]
        s["weight"].copy_(torch.where(fresh, 0.0, s["weight"]))
        s["order"].copy_(torch.where(fresh, at.to(I32), s["order"]))
        return s["qo"], _whole(s, "kp"), _whole(s, "vp"), s["weight"], s["order"]
    if c["op"] == "decode":
        G, Tq = c["Hq"] // Hkv, c["Tq"]
        k, v = _keys(s, "kp", s["ks"]), _keys(s, "vp", s["vs"])
        at = torch.arange(k.shape[2], device=DEV)
        t = torch.arange(Tq, device=DEV)
        see = at < (lens[:, None] - Tq + t + 1)[..., None]                   # [B][Tq][slots]
        see = see[:, None, None].expand(B, Hkv, G, Tq, -1).reshape(B, Hkv, G * Tq, -1)
        z = s["q"].float().reshape(B, Hkv, G * Tq, d) @ k.transpose(2, 3) * (d ** -0.5)
        z = torch.where(see, z, -torch.inf)
        m = z.amax(-1, keepdim=True)
        m = torch.where(m == -torch.inf, 0.0, m)
        e = torch.exp(z - m)
        l = e.sum(-1, keepdim=True)
        p = e / torch.where(l > 0, l, 1.0)
        v = torch.where((at < lens[:, None])[:, None, :, None], v, 0.0)
        s["o"].copy_((p @ v).view(B, c["Hq"], Tq, d))
        s["lse"].copy_((m + torch.log(l)).view(B, c["Hq"], Tq))
        if not c["weights"]:
            return s["o"], s["lse"]
        s["weight"].add_(p.sum(2))
        return s["o"], s["lse"], s["weight"]
    cap, budget = s["weight"].shape[-1], c["budget"]
    at = torch.arange(cap, device=DEV)
    end = lens.clamp(max=budget)[:, None, None]
    key = s["weight"].double()
    key = torch.where((s["order"] < c["first"]) | (s["order"] >= s["seen"][:, None, None] - c["recent"]), torch.inf, key)
    key = torch.where(at < lens[:, None, None], key, -torch.inf)
    best = key.sort(dim=-1, descending=True, stable=True).indices
    keep = torch.zeros((B, Hkv, cap), dtype=torch.bool, device=DEV).scatter_(2, best, (at < end).expand(B, Hkv, cap))
    hole, mover = ~keep & (at < end), keep & (at >= end)
    # the i-th mover's slot at place i (the others at a spare last place)
    movers = torch.zeros((B, Hkv, cap + 1), dtype=I64, device=DEV)
    movers.scatter_(2, torch.where(mover, mover.cumsum(-1) - 1, cap), at.expand(B, Hkv, cap))
    src = torch.where(hole, movers.gather(2, (hole.cumsum(-1) - 1).clamp(min=0)), at)[..., :budget]
    src = torch.nn.functional.pad(src, (0, max(0, budget - cap)))
    j = torch.arange(budget, device=DEV)
    there = (j < end).expand(B, Hkv, budget)
    b, h = torch.arange(B, device=DEV)[:, None, None], torch.arange(Hkv, device=DEV)[None, :, None]
    s["kept"].copy_(torch.where(there, src, s["kept"].long()))
    jj = j.clamp(max=cap - 1).expand(B, Hkv, budget)
    to = torch.where(there, table[b, jj // ps], n)
    for name in ("kp", "vp"):
        s[name][to, h, jj % ps] = s[name][table[b, src // ps], h, src % ps]
    m = min(budget, cap)
    s["weight_o"][..., :m] = torch.where(there, s["weight"].gather(2, src), 0.0)[..., :m]
    s["order_o"][..., :m] = torch.where(there, s["order"].gather(2, src), 0)[..., :m]
    s["lens_o"].copy_(end[:, 0, 0])
    return _whole(s, "kp"), _whole(s, "vp"), s["weight_o"], s["order_o"], s["lens_o"], s["kept"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, d = case, case["d"]
    if c["op"] == "rope":
        n = c["B"] * (c["Hq"] + c["Hk"]) * c["T"]
        return dict(bytes=n * d * 2 * (4 if c["f32"] else 2) + 4 * c["axes"] * c["B"] * c["T"], flops=3 * n * c["rot"])
    elem, lens = 1 if c["fp8"] else 2, _lens(c)
    if c["op"] == "append":
        n = sum(_new_lens(c))
        return dict(bytes=n * (c["Hq"] * d * 4 + 2 * c["Hkv"] * d * (2 + elem) + 8 * c["Hkv"] + 4 * c["axes"]) + 4 * sum(lens) // c["ps"],
                    flops=3 * n * (c["Hq"] + c["Hkv"]) * c["rot"])
    if c["op"] == "decode":
        rows = c["B"] * c["Hq"] * c["Tq"]
        return dict(bytes=sum(lens) * c["Hkv"] * (2 * d * elem + (8 if c["weights"] else 0)) + rows * (4 * d + 4),
                    flops=4 * d * c["Hq"] * c["Tq"] * sum(lens))
    total = 0
    for n in lens:   # weight and order in and out, kept; the moved rows: the share of the front that does not stay
        end = min(n, c["budget"])
        sure = min(end, c["first"] + c["recent"])
        moved = end * (1 - (sure + (end - sure)) / max(n, 1))
        total += c["Hkv"] * (8 * n + 12 * end + moved * 4 * d * elem)
    return dict(bytes=int(total), flops=2 * sum(lens) * c["Hkv"])


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _turned(x, c, pos, sign=1.0):
    """x (double) as complex pairs times e^{i sign theta}."""
    rot, n = c["rot"], c["rot"] // 2
    ang = torch.stack([pos[a].double() * f for f, a in zip(_freqs(rot), _axis(rot, c["axes"]))], -1)
    w = torch.polar(torch.ones_like(ang), sign * ang)[:, None]
    y = x.clone()
    if c.get("interleaved"):
        y[..., :rot] = torch.view_as_real(torch.view_as_complex(x[..., :rot].unflatten(-1, (n, 2)).contiguous()) * w).flatten(-2)
    else:
        z = torch.complex(x[..., :n].contiguous(), x[..., n:rot].contiguous()) * w
        y[..., :n], y[..., n:rot] = z.real, z.imag
    return y


def _held(x, scale):
    """The value nearest to x (double) that the cache can hold, as its code stands for it."""
    if scale is None:
        return x
    x = (x / scale).clamp(-448, 448)
    step = torch.exp2(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1].double() - 4)
    return torch.round(x / step) * step


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        sign = -1.0 if c["inverse"] else 1.0
        return _turned(s["q"].double(), c, s["pos"], sign), _turned(s["k"].double(), c, s["pos"], sign)
    lens, table, ps, Hkv, d = _lens(c), s["table"].tolist(), c["ps"], c["Hkv"], c["d"]
    def values(name):
        return _whole(s, name).to(F32 if c["fp8"] else BF16)
    if c["op"] == "append":
        new = _new_lens(c)
        q, k = _turned(s["q"].double(), c, s["pos"]), _turned(s["k"].double(), c, s["pos"])
        kp, vp = values("kp").double(), values("vp").double()
        qo, w, o = torch.zeros_like(q), s["weight"].double(), s["order"].clone()
        for b in range(c["B"]):
            nb, first = new[b], lens[b] - new[b]
            qo[b, :, :nb] = q[b, :, :nb]
            slots = torch.arange(first, lens[b], device=DEV)
            pages = torch.tensor(table[b], device=DEV)[slots // ps]
            for h in range(Hkv):
                kp[pages, h, slots % ps] = _held(k[b, h, :nb], s["ks"][h].double() if c["fp8"] else None)
                vp[pages, h, slots % ps] = _held(s["v"][b, h, :nb].double(), s["vs"][h].double() if c["fp8"] else None)
            w[b, :, first:lens[b]] = 0
            o[b, :, first:lens[b]] = slots.to(I32)
        return qo, kp, vp, w, o
    if c["op"] == "decode":
        G, Tq = c["Hq"] // Hkv, c["Tq"]
        o = torch.zeros(s["q"].shape, dtype=F64, device=DEV)
        lse = torch.full(s["lse"].shape, -torch.inf, dtype=F64, device=DEV)
        w = s["weight"].double() if c["weights"] else None
        for b in range(c["B"]):
            n = lens[b]
            pages = torch.tensor(table[b], device=DEV)[:-(-n // ps)]
            kb, vb = ((s[x][pages].view(FP8) if c["fp8"] else s[x][pages]) for x in ("kp", "vp"))
            for h in range(Hkv):
                kh, vh = kb[:, h].double().reshape(-1, d)[:n], vb[:, h].double().reshape(-1, d)[:n]
                if c["fp8"]:
                    kh, vh = kh * s["ks"][h].double(), vh * s["vs"][h].double()
                for t in range(Tq):
                    m = n - Tq + t + 1
                    if m <= 0:
                        continue
                    z = s["q"][b, h * G:(h + 1) * G, t].double() @ kh[:m].T / math.sqrt(d)
                    y = torch.logsumexp(z, -1)
                    p = torch.exp(z - y[:, None])
                    o[b, h * G:(h + 1) * G, t], lse[b, h * G:(h + 1) * G, t] = p @ vh[:m], y
                    if w is not None:
                        w[b, h, :m] += p.sum(0)
        return (o, lse) if w is None else (o, lse, w)
    kp, vp = values("kp").double(), values("vp").double()
    kin, vin = kp.clone(), vp.clone()
    w_in, o_in, seen = s["weight"].cpu(), s["order"].cpu(), s["seen"].cpu()
    wo, oo, lo, kept = torch.zeros_like(w_in, dtype=F64), s["order_o"].cpu(), s["lens_o"].cpu(), s["kept"].cpu()
    for b in range(c["B"]):
        n, end = lens[b], min(lens[b], c["budget"])
        lo[b] = end
        for h in range(Hkv):
            wt, od = w_in[b, h, :n].tolist(), o_in[b, h, :n].tolist()
            edge = int(seen[b]) - c["recent"]
            rank = sorted(range(n), key=lambda i: (0, 0, i) if od[i] < c["first"] or od[i] >= edge else (1, -wt[i], i))
            stay = set(rank[:end])
            late = iter(sorted(i for i in stay if i >= end))
            src = [i if i in stay else next(late) for i in range(end)]
            kept[b, h, :end] = torch.tensor(src, dtype=I32)
            wo[b, h, :end], oo[b, h, :end] = w_in[b, h, src].double(), o_in[b, h, src]
            moved = [(i, x) for i, x in enumerate(src) if x != i]
            if moved:
                to, fr = (torch.tensor(x, device=DEV) for x in zip(*moved))
                tab = torch.tensor(table[b], device=DEV)
                kp[tab[to // ps], h, to % ps] = kin[tab[fr // ps], h, fr % ps]
                vp[tab[to // ps], h, to % ps] = vin[tab[fr // ps], h, fr % ps]
    return kp, vp, wo, oo, lo, kept
