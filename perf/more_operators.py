"""Cases of three operators around attention and its paged cache: norms of query and key heads with
the position rotation in the same pass (forward, gradients, and on the way into the cache),
attention with a sliding window and a few first tokens that stay visible (forward, training step,
and single tokens over the paged cache), and attention of a batch over a cache whose sequences share
a long prefix.

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
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # q and k of a training step at the benchmark's sizes (B8 H32 N4096 d128), views of the packed
        # projection, normed by head and rotated
        dict(name="norm_train_b8h32_t4096_d128", op="norm", B=8, Hq=32, Hk=32, T=4096, d=128, rot=128, axes=1, f32=False,
             wf32=False, interleaved=False, packed=True, back=False),
        # the gradients of the same step, written into the packed projection's gradient
        dict(name="norm_grad_b8h32_t4096_d128", op="norm", B=8, Hq=32, Hk=32, T=4096, d=128, rot=128, axes=1, f32=False,
             wf32=False, interleaved=False, packed=True, back=True),
        # gradients of a fine-tuning step in fp32: odd length, grouped heads, interleaved pairs, half the
        # head rotated, two axes
        dict(name="norm_grad_f32_b2h6_t1021_d64", op="norm", B=2, Hq=6, Hk=2, T=1021, d=64, rot=32, axes=2, f32=True,
             wf32=True, interleaved=True, packed=False, back=True),
        # one decoding step of eight sequences: q and k normed, rotated, k and v written to the cache
        dict(name="norm_append_step_b8_d128", op="append", B=8, Hq=32, Hkv=8, T=1, lo=500, hi=4000, d=128, rot=128, axes=1,
             ps=16, fp8=False, ragged=False),
        # forward and backward of a training step at the benchmark's sizes, a window of 1024 tokens and 4 sinks
        dict(name="sinks_train_b8h32_t4096_d128", op="sinks", B=8, H=32, Tq=4096, Tk=4096, d=128, left=1023, sinks=4, back=True),
        # prefill of a 65536-token prompt with narrow heads
        dict(name="sinks_prefill_b1h6_t65536_d64", op="sinks", B=1, H=6, Tq=65536, Tk=65536, d=64, left=4095, sinks=4, back=False),
        # the last chunk of a prompt, wide heads, odd sizes
        dict(name="sinks_chunk_b2h6_q1021_k5003_d256", op="sinks", B=2, H=6, Tq=1021, Tk=5003, d=256, left=776, sinks=5, back=False),
        # one decoding step of a serving batch; pages behind the window were given back
        dict(name="sinks_decode_b64_d128", op="window", B=64, Hq=32, Hkv=8, Tq=1, lo=200, hi=8000, d=128, ps=16, fp8=False,
             left=1023, sinks=4),
        # an e4m3 cache, narrow heads, lengths to 64K and a wide window
        dict(name="sinks_decode_fp8_b16_d64", op="window", B=16, Hq=16, Hkv=4, Tq=1, lo=1001, hi=65536, d=64, ps=32, fp8=True,
             left=4095, sinks=4),
        # four requests on a short common instruction: latency counts
        dict(name="shared_b4_p512_d128", op="shared", B=4, Hq=32, Hkv=8, Tq=1, prefix=512, lo=1, hi=60, pad=0, d=128, ps=16, fp8=False),
        # a serving batch whose requests all start with the same document
        dict(name="shared_b64_p32768_d128", op="shared", B=64, Hq=32, Hkv=8, Tq=1, prefix=32768, lo=20, hi=700, pad=3, d=128, ps=16,
             fp8=False),
        # an e4m3 cache, narrow heads, four rows of each sequence to verify
        dict(name="shared_fp8_b16_p65536_d64", op="shared", B=16, Hq=16, Hkv=4, Tq=4, prefix=65536, lo=5, hi=1001, pad=0, d=64, ps=32,
             fp8=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "append", "sinks", "sinks", "window", "window", "shared", "shared", "shared"])
    d = rng.choice([64, 128, 128, 256])
    if op == "norm":
        B, Hk, G = _log_int(rng, 1, 8), _log_int(rng, 1, 16), rng.choice([1, 2, 3, 4])
        T = max(1, min(_log_int(rng, 1, 8192), 8 * 32 * 4096 * 128 // (B * Hk * (G + 1) * d * 2)))
        return dict(op="norm", B=B, Hq=Hk * G, Hk=Hk, T=T, d=d, rot=rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)]),
                    axes=rng.randint(1, 4), f32=rng.random() < 0.3, wf32=rng.random() < 0.5, interleaved=rng.random() < 0.4,
                    packed=rng.random() < 0.5, back=rng.random() < 0.6)
    if op == "sinks":
        back = rng.random() < 0.5
        d = rng.choice([64, 128]) if back else d
        Tq = _log_int(rng, 1, 16384)
        Tk = Tq if back or rng.random() < 0.5 else Tq + rng.randint(0, 8192)
        left = _log_int(rng, 1, 4096) - 1
        heads = max(1, min(256, 8 * 32 * 4096 * 1024 * 128 // (4 * Tq * (left + 160) * d)))
        H = rng.randint(1, min(32, heads))
        return dict(op="sinks", B=rng.randint(1, max(1, min(8, heads // H))), H=H, Tq=Tq, Tk=Tk, d=d, left=left,
                    sinks=rng.choice([0, 1, 4, 4, 16, 130]), back=back)
    ps, fp8 = rng.choice([16, 32, 64, 128, 256]), rng.random() < 0.35
    Hkv, G = rng.choice([1, 2, 3, 4, 8, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    Tq = rng.choice([1, 1, 1, 2, 4, 7])
    if op == "append":
        B = _log_int(rng, 1, 96)
        T = _log_int(rng, 1, max(1, min(3000, 60000000 // (B * Hkv * (G + 2) * d))))
        lo = T + rng.randint(0, 500)
        return dict(op="append", B=B, Hq=Hkv * G, Hkv=Hkv, T=T, lo=lo, hi=lo + rng.randint(0, 700), d=d,
                    rot=rng.choice([d, d // 2]), axes=rng.randint(1, 3), ps=ps, fp8=fp8, ragged=rng.random() < 0.5)
    if op == "window":
        B, left = _log_int(rng, 1, 96), _log_int(rng, 1, 8192) - 1
        left = min(left, 100000000 // (B * Hkv * d))
        hi = _log_int(rng, 1, 65536)
        return dict(op="window", B=B, Hq=Hkv * G, Hkv=Hkv, Tq=Tq, lo=rng.randint(0, hi), hi=hi, d=d, ps=ps, fp8=fp8,
                    left=left, sinks=rng.choice([0, 1, 4, 4, 16, 130]))
    B = _log_int(rng, 1, 96)
    hi = _log_int(rng, 1, max(1, min(2000, 50000000 // (B * Hkv * d))))
    prefix = max(1, _log_int(rng, ps, max(ps, min(65536, 16 * 8 * 32768 * 64 * 4 // (B * Hkv * G * Tq)))) // ps) * ps
    return dict(op="shared", B=B, Hq=Hkv * G, Hkv=Hkv, Tq=Tq, prefix=prefix, lo=rng.randint(0, hi), hi=hi,
                pad=rng.choice([0, 0, 1, B // 3]), d=d, ps=ps, fp8=fp8)


# ------------------------------------------------------------------ what the cases share
def _spread(lo, hi, n):
    """n lengths spread over [lo, hi], the last one hi."""
    return [hi - int((hi - lo) * ((b * 0.6180339887498949) % 1.0)) for b in range(n)][::-1]


def _lens(c):
    if c["op"] != "shared":
        return _spread(c["lo"], c["hi"], c["B"])
    # places of the batch without a request have length 0
    pad = min(c["pad"], c["B"] - 1)
    return [0] * pad + [c["prefix"] + n for n in _spread(c["lo"], c["hi"], c["B"] - pad)]


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


def _positions(g, B, T, axes, far):
    """int32 [axes][B][T]: text up to a quarter of the row, then frames of a grid (time, height,
    width), shifted per sequence by up to 100 and by `far`."""
    t = torch.arange(T, device=DEV, dtype=I64)
    text = T // 4
    cell = (t - text).clamp(min=0)
    grid = torch.stack([cell // 384, cell // 24 % 16, cell % 24, cell % 7])[:axes] + text
    p = torch.where(t < text, t, grid) if axes > 1 else t[None]
    shift = torch.randint(0, 100, (1, B, 1), generator=g, device=DEV) + far
    return (p[:, None, :] + shift).to(I32).contiguous()


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _weight(g, d, dtype):
    """Weights of a trained norm: around one, a few far from it."""
    return (torch.exp(0.5 * _randn(g, (d,), F32))).to(dtype)


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


def _visible_pages(c, n):
    """Pages of a sequence of n entries that a window step reads: those of the sinks and of the window."""
    ps, start = c["ps"], max(0, n - c["Tq"] - c["left"])
    return [i for i in range(-(-n // ps)) if i * ps < c["sinks"] or (i + 1) * ps > start]


def _tables(c, g, lens):
    """Block table, number of pages and, of a shared case, the prefix's pages."""
    B, ps = c["B"], c["ps"]
    width = -(-max(max(lens), 1) // ps)
    if c["op"] == "window":   # entries of pages that were given back are -1
        need = [_visible_pages(c, n) for n in lens]
        total = sum(len(x) for x in need)
        ids = torch.randperm(max(total, 1), generator=g, device=DEV).tolist()
        table, at = [[-1] * width for _ in range(B)], 0
        for row, pages in zip(table, need):
            for i in pages:
                row[i], at = ids[at], at + 1
        return torch.tensor(table, device=DEV, dtype=I32).view(B, width), max(total, 1), None
    if c["op"] == "shared":
        P = c["prefix"] // ps
        n = P + B * (width - P)
        ids = torch.randperm(n, generator=g, device=DEV).to(I32)
        table = torch.cat((ids[:P].expand(B, P), ids[P:].view(B, width - P)), 1).contiguous()
        return table, n, ids[:P].clone()
    n = B * width
    return torch.randperm(n, generator=g, device=DEV).to(I32).view(B, width), n, None


def prepare(case, seed):
    c, g = case, torch.Generator(DEV).manual_seed(seed)
    s = dict(c=c)
    d = c["d"]
    if c["op"] == "norm":
        B, Hq, Hk, T = c["B"], c["Hq"], c["Hk"], c["T"]
        dt = F32 if c["f32"] else BF16
        wt = F32 if c["wf32"] else BF16

        def pair(make):
            if c["packed"]:   # the projection's [B][T][heads of q, k and v][d]
                x = make((B, T, Hq + 2 * Hk, d)).transpose(1, 2)
                return x[:, :Hq], x[:, Hq:Hq + Hk]
            return make((B, Hq, T, d)), make((B, Hk, T, d))

        def zeros(shape):
            return torch.zeros(shape, device=DEV, dtype=dt)
        s["q"], s["k"] = pair(lambda sh: _randn(g, sh, dt).mul_(3.0))
        s["qw"], s["kw"] = _weight(g, d, wt), _weight(g, d, wt)
        s["pos"] = _positions(g, B, T, c["axes"], 500)
        if c["back"]:
            s["dqo"], s["dko"] = _randn(g, (B, Hq, T, d), dt), _randn(g, (B, Hk, T, d), dt)
            s["dq"], s["dk"] = pair(zeros)
            s["dqw"], s["dkw"] = torch.zeros(d, device=DEV), torch.zeros(d, device=DEV)
        else:
            s["qo"], s["ko"] = zeros((B, Hq, T, d)), zeros((B, Hk, T, d))
    elif c["op"] == "sinks":
        B, H, Tq, Tk = c["B"], c["H"], c["Tq"], c["Tk"]
        s["q"], s["k"], s["v"] = _randn(g, (B, H, Tq, d), BF16), _randn(g, (B, H, Tk, d), BF16), _randn(g, (B, H, Tk, d), BF16)
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty((B, H, Tq), device=DEV)
        if c["back"]:
            s["do"] = _randn(g, (B, H, Tq, d), BF16)
            s["dq"], s["dk"], s["dv"] = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    else:
        lens = _lens(c)
        B, Hkv = c["B"], c["Hkv"]
        s["table"], s["n"], s["prefix"] = _tables(c, g, lens)
        s["lens"] = torch.tensor(lens, device=DEV, dtype=I32)
        s["kp"], s["vp"] = _pool(c, g, s["n"]), _pool(c, g, s["n"])
        s["ks"], s["vs"] = _scales(c, g), _scales(c, g)
        if c["op"] == "append":
            T = c["T"]
            s["q"], s["k"], s["v"] = (_randn(g, (B, h, T, d), BF16).mul_(3.0) for h in (c["Hq"], Hkv, Hkv))
            s["qo"] = torch.zeros_like(s["q"])
            s["qw"], s["kw"] = _weight(g, d, BF16), _weight(g, d, BF16)
            s["new"] = torch.tensor(_new_lens(c), device=DEV, dtype=I32) if c["ragged"] else None
            s["pos"] = _positions(g, B, T, c["axes"], 500)
        else:
            s["q"] = _randn(g, (B, c["Hq"], c["Tq"], d), BF16)
            s["o"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((B, c["Hq"], c["Tq"]), device=DEV)
    if own:   # the handles that a program keeps: frequencies, norms, the cache, a workspace
        from exact_io_aware_05_gb300 import fa
        s["fa"] = fa

        def bytes_(n):
            return torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
        if c["op"] in ("norm", "append"):
            s["spec"] = fa.RopeSpec(d, _freqs(c["rot"]), _axis(c["rot"], c["axes"]), interleaved=c.get("interleaved", False))
            s["norm"] = fa.HeadNorm(d, s["qw"], s["kw"], eps=EPS)
        if c["op"] == "norm" and c["back"]:
            s["ws"] = bytes_(fa.fa_norm_rope_bwd_workspace_bytes(d))
        if c["op"] == "sinks" and c["back"]:
            s["ws"] = bytes_(fa.fa_bwd_sinks_workspace_bytes(c["B"], c["H"], c["Tq"], c["Tk"], d, c["left"], c["sinks"]))
        if c["op"] in ("append", "window", "shared"):
            s["cache"] = fa.KVCache(s["kp"][:s["n"]], s["vp"][:s["n"]], s["table"], s["lens"], k_scale=s["ks"], v_scale=s["vs"])
        if c["op"] == "window":
            s["ws"] = bytes_(fa.fa_decode_paged_window_workspace_bytes(s["cache"], c["Hq"], c["Tq"]))
        if c["op"] == "shared":
            s["ws"] = bytes_(fa.fa_decode_paged_shared_workspace_bytes(s["cache"], c["Hq"], c["Tq"], s["prefix"]))
    return s


def _whole(s, name):
    """The cache's pages; codes as the values they stand for (a view)."""
    x = s[name][:s["n"]]
    return x.view(FP8) if s["c"]["fp8"] else x


def _outputs(s):
    c = s["c"]
    if c["op"] == "norm":
        return (s["dq"], s["dk"], s["dqw"], s["dkw"]) if c["back"] else (s["qo"], s["ko"])
    if c["op"] == "append":
        return s["qo"], _whole(s, "kp"), _whole(s, "vp")
    if c["op"] == "sinks" and c["back"]:
        return s["o"], s["lse"], s["dq"], s["dk"], s["dv"]
    return s["o"], s["lse"]


# ------------------------------------------------------------------ one pass
def run(s):
    (_run_own if own else _run_plain)(s)
    return _outputs(s)


def _run_own(s):
    c, fa = s["c"], s["fa"]
    scale = c["d"] ** -0.5
    if c["op"] == "norm":
        if c["back"]:
            fa.fa_norm_rope_bwd(s["dqo"], s["q"], s["dq"], s["pos"], s["spec"], s["norm"], dk_out=s["dko"], k=s["k"], dk=s["dk"],
                                dq_weight=s["dqw"], dk_weight=s["dkw"], workspace=s["ws"])
        else:
            fa.fa_norm_rope(s["q"], s["qo"], s["pos"], s["spec"], s["norm"], k=s["k"], k_out=s["ko"])
    elif c["op"] == "append":
        fa.fa_cache_append(s["cache"], s["k"], s["v"], s["pos"], s["spec"], q=s["q"], q_out=s["qo"], new_lens=s["new"], norm=s["norm"])
    elif c["op"] == "sinks":
        fa.fa_fwd_sinks(s["q"], s["k"], s["v"], s["o"], s["lse"], c["left"], c["sinks"], scale)
        if c["back"]:
            fa.fa_bwd_sinks(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["dq"], s["dk"], s["dv"], c["left"], c["sinks"], scale,
                            s["ws"])
    elif c["op"] == "window":
        fa.fa_decode_paged_window(s["cache"], s["q"], s["o"], s["lse"], c["left"], c["sinks"], scale, s["ws"])
    else:
        fa.fa_decode_paged_shared(s["cache"], s["q"], s["o"], s["lse"], s["prefix"], scale, s["ws"], causal=True)


def _cos_sin(c, pos):
    """cos and sin of the angles, fp32 [B][1][T][rot / 2]; the angles in 64 bits."""
    axis = torch.tensor(_axis(c["rot"], c["axes"]), device=DEV)
    a = pos[axis].double() * torch.tensor(_freqs(c["rot"]), device=DEV, dtype=F64)[:, None, None]
    a = a.permute(1, 2, 0)[:, None]
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin, rot, interleaved):
    """fp32 x rotated."""
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _unit(x):
    """fp32 x over the root of its mean square, and one over that root."""
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _codes(x, scale):
    """What the cache holds of fp32 x [B][Hkv][T][d]."""
    return x.to(BF16) if scale is None else (x / scale[:, None, None]).clamp(-448, 448).to(FP8).view(torch.uint8)


def _rows_at(s, name, scale, slot):
    """Keys or values at slots [B][n], fp32 [B][Hkv][n][d]; slots whose page is not there give page 0."""
    ps = s["c"]["ps"]
    page = s["table"].long().gather(1, slot // ps).clamp(min=0)
    x = s[name][page, :, slot % ps].transpose(1, 2)
    return x.float() if scale is None else x.view(FP8).float() * scale[:, None, None]


def _softmax(z):
    """Probabilities of scores (rows of -inf give 0) and the log of the sum of their exponentials."""
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -torch.inf, 0.0, m)
    e = torch.exp(z - m)
    l = e.sum(-1, keepdim=True)
    return e / torch.where(l > 0, l, 1.0), (m + torch.log(l))[..., 0]


def _chunks(c, rows):
    """Runs of query rows r0 .. r1 - 1, the sinks 0 .. s1 - 1 and other keys k0 .. k1 - 1 that they may see."""
    off = c["Tk"] - c["Tq"]
    for r0 in range(0, c["Tq"], rows):
        r1 = min(c["Tq"], r0 + rows)
        k1 = max(0, r1 + off)
        s1 = min(c["sinks"], k1)
        yield r0, r1, s1, min(max(s1, r0 + off - c["left"]), k1), k1


def _seen(c, r0, r1, s1, k0, k1):
    """Keys of a run (sinks, then the others), and which of its rows see them."""
    key = torch.cat((torch.arange(s1, device=DEV), torch.arange(k0, k1, device=DEV)))
    p = torch.arange(r0, r1, device=DEV)[:, None] + (c["Tk"] - c["Tq"])
    return (key <= p) & ((key >= p - c["left"]) | (key < c["sinks"]))


def _run_plain(s):
    c, d = s["c"], s["c"]["d"]
    scale = d ** -0.5
    if c["op"] == "norm":
        cos, sin = _cos_sin(c, s["pos"])
        rot, inter = c["rot"], c["interleaved"]
        if not c["back"]:
            for x, w, y in ((s["q"], s["qw"], s["qo"]), (s["k"], s["kw"], s["ko"])):
                y.copy_(_rotate(_unit(x)[0] * w.float(), cos, sin, rot, inter))
            return
        for dy, x, w, dx, dw in ((s["dqo"], s["q"], s["qw"], s["dq"], s["dqw"]), (s["dko"], s["k"], s["kw"], s["dk"], s["dkw"])):
            u, r = _unit(x)
            g = _rotate(dy.float(), cos, -sin, rot, inter)
            dw.copy_((g * u).sum((0, 1, 2)))
            g = g * w.float()
            dx.copy_(r * (g - u * (g * u).mean(-1, keepdim=True)))
        return
    if c["op"] == "append":
        T, ps, n, rot = c["T"], c["ps"], s["n"], c["rot"]
        lens, table = s["lens"].long(), s["table"].long()
        cos, sin = _cos_sin(c, s["pos"])
        t = torch.arange(T, device=DEV)
        new = torch.full_like(lens, T) if s["new"] is None else s["new"].long()
        there = t < new[:, None]                                             # [B][T]
        q, k = (_rotate(_unit(s[x])[0] * s[x + "w"].float(), cos, sin, rot, False) for x in ("q", "k"))
        s["qo"].copy_(torch.where(there[:, None, :, None], q, s["qo"].float()))
        slot = ((lens - new)[:, None] + t).clamp(max=table.shape[1] * ps - 1)
        page = torch.where(there, table.gather(1, slot // ps), n)            # rows that are not there go to the spare page
        row = slot % ps
        s["kp"][page, :, row] = _codes(k, s["ks"]).transpose(1, 2)
        s["vp"][page, :, row] = _codes(s["v"].float(), s["vs"]).transpose(1, 2)
        return
    if c["op"] == "sinks":
        if c["back"]:
            dk, dv = torch.zeros_like(s["k"], dtype=F32), torch.zeros_like(s["v"], dtype=F32)
        for r0, r1, s1, k0, k1 in _chunks(c, 512):
            q = s["q"][:, :, r0:r1].float()
            k, v = (torch.cat((s[x][:, :, :s1], s[x][:, :, k0:k1]), 2).float() for x in ("k", "v"))
            if k.shape[2] == 0:
                s["o"][:, :, r0:r1], s["lse"][:, :, r0:r1] = 0, -torch.inf
                if c["back"]:
                    s["dq"][:, :, r0:r1] = 0
                continue
            see = _seen(c, r0, r1, s1, k0, k1)
            p, lse = _softmax(torch.where(see, q @ k.transpose(2, 3) * scale, -torch.inf))
            o = p @ v
            s["o"][:, :, r0:r1], s["lse"][:, :, r0:r1] = o, lse
            if c["back"]:
                do = s["do"][:, :, r0:r1].float()
                ds = p * (do @ v.transpose(2, 3) - (do * o).sum(-1, keepdim=True)) * scale
                s["dq"][:, :, r0:r1] = ds @ k
                gk, gv = ds.transpose(2, 3) @ q, p.transpose(2, 3) @ do
                for whole, part in ((dk, gk), (dv, gv)):
                    whole[:, :, :s1] += part[:, :, :s1]
                    whole[:, :, k0:k1] += part[:, :, s1:]
        if c["back"]:
            s["dk"].copy_(dk)
            s["dv"].copy_(dv)
        return
    B, Hq, Hkv, Tq, lens = c["B"], c["Hq"], c["Hkv"], c["Tq"], s["lens"].long()
    GT = Hq // Hkv * Tq
    t = torch.arange(Tq, device=DEV)
    end = lens[:, None] - Tq + t                                             # last slot that a row sees, [B][Tq]
    q = s["q"].float().reshape(B, Hkv, GT, d)

    def rows(see):   # [B][Tq][n] for every row of a head group
        return see[:, None, None].expand(B, Hkv, GT // Tq, Tq, -1).reshape(B, Hkv, GT, -1)
    if c["op"] == "window":
        j = torch.arange(c["sinks"] + c["left"] + Tq, device=DEV)
        start = (lens - Tq - c["left"]).clamp(min=c["sinks"])                # the window's first slot that is no sink
        slot = torch.where(j < c["sinks"], j, start[:, None] + j - c["sinks"])
        see = (slot[:, None] <= end[..., None]) & ((slot[:, None] >= end[..., None] - c["left"]) | (slot < c["sinks"])[:, None])
        there = slot < lens[:, None]
        slot = slot.clamp(max=s["table"].shape[1] * c["ps"] - 1)
        k, v = _rows_at(s, "kp", s["ks"], slot), _rows_at(s, "vp", s["vs"], slot)
        z = q @ k.transpose(2, 3)
        v = torch.where(there[:, None, :, None], v, 0.0)
        p, lse = _softmax(torch.where(rows(see), z * scale, -torch.inf))
        s["o"].copy_((p @ v).view(B, Hq, Tq, d))
        s["lse"].copy_(lse.view(B, Hq, Tq))
        return
    # the prefix once, for the rows of all sequences; each sequence's own entries
    P, page = c["prefix"], s["prefix"].long()

    def prefix(name, sc):
        x = s[name][page].transpose(0, 1).flatten(1, 2)                      # [Hkv][P][d]
        return x.float() if sc is None else x.view(FP8).float() * sc[:, None, None]
    at = torch.arange(P, device=DEV)
    zp = (q.transpose(0, 1).reshape(Hkv, B * GT, d) @ prefix("kp", s["ks"]).transpose(1, 2)).view(Hkv, B, GT, P).transpose(0, 1)
    seep = rows(at <= end[..., None])
    n = s["table"].shape[1] * c["ps"] - P
    slot = (P + torch.arange(n, device=DEV)).expand(B, n)
    k, v = _rows_at(s, "kp", s["ks"], slot), _rows_at(s, "vp", s["vs"], slot)
    z = torch.cat((torch.where(seep, zp * scale, -torch.inf),
                   torch.where(rows(slot[:, None] <= end[..., None]), q @ k.transpose(2, 3) * scale, -torch.inf)), -1)
    v = torch.where((slot < lens[:, None])[:, None, :, None], v, 0.0)
    p, lse = _softmax(z)
    o = p[..., P:] @ v
    o += (p[..., :P].transpose(0, 1).reshape(Hkv, B * GT, P) @ prefix("vp", s["vs"])).view(Hkv, B, GT, d).transpose(0, 1)
    s["o"].copy_(o.reshape(B, Hq, Tq, d))
    s["lse"].copy_(lse.view(B, Hq, Tq))


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(first, last, left, sinks):
    """Visible (row, key) pairs of rows at positions first .. last."""
    first = max(first, 0)
    if last < first:
        return 0
    n = 0
    for p in range(first, last + 1):
        n += min(p + 1, left + 1) + min(sinks, max(0, p - left))
    return n


def work(case):
    c, d = case, case["d"]
    if c["op"] == "norm":
        n, e = c["B"] * (c["Hq"] + c["Hk"]) * c["T"], 4 if c["f32"] else 2
        return dict(bytes=n * d * e * (3 if c["back"] else 2) + 4 * c["axes"] * c["B"] * c["T"] + (4 + 8) * d,
                    flops=n * (3 * c["rot"] + (9 if c["back"] else 4) * d))
    if c["op"] == "sinks":
        heads, rows, keys = c["B"] * c["H"], c["B"] * c["H"] * c["Tq"], c["B"] * c["H"] * c["Tk"]
        off = c["Tk"] - c["Tq"]
        pairs = heads * _pairs(off, c["Tk"] - 1, c["left"], c["sinks"])
        if c["back"]:   # q, o, dO, dq and k, v, dk, dv; seven products
            return dict(bytes=(8 * rows + 8 * keys) * d + 4 * rows, flops=14 * d * pairs)
        return dict(bytes=(4 * rows + 4 * keys) * d + 4 * rows, flops=4 * d * pairs)
    elem, lens = 1 if c["fp8"] else 2, _lens(c)
    if c["op"] == "append":
        n = sum(_new_lens(c))
        return dict(bytes=n * (c["Hq"] * d * 4 + 2 * c["Hkv"] * d * (2 + elem) + 4 * c["axes"]) + 4 * sum(lens) // c["ps"],
                    flops=n * (c["Hq"] + c["Hkv"]) * (3 * c["rot"] + 4 * d))
    rows, Tq = c["B"] * c["Hq"] * c["Tq"], c["Tq"]
    if c["op"] == "window":
        entries = sum(n - max(0, max(0, n - Tq - c["left"]) - c["sinks"]) for n in lens)
        pairs = c["Hq"] * sum(_pairs(n - Tq, n - 1, c["left"], c["sinks"]) for n in lens)
        return dict(bytes=entries * c["Hkv"] * 2 * d * elem + rows * (4 * d + 4), flops=4 * d * pairs)
    entries = c["prefix"] + sum(max(0, n - c["prefix"]) for n in lens)
    pairs = c["Hq"] * sum(max(0, n - Tq + 1 + t) for n in lens for t in range(Tq))
    return dict(bytes=entries * c["Hkv"] * 2 * d * elem + rows * (4 * d + 4), flops=4 * d * pairs)


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


def _normed(x, w):
    """w x / rms(x), in 64 bits."""
    x = x.double()
    return w.double() * x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)


def _norm_gradients(dy, x, w, c, pos):
    """Gradients of sum(dy * turned(normed(x, w))) by x and by w."""
    x, n = x.double(), x.shape[-1]
    g = _turned(dy.double(), c, pos, -1.0)
    ms = x.square().sum(-1, keepdim=True) / n + EPS
    dw = (g * x / torch.sqrt(ms)).sum((0, 1, 2))
    g = g * w.double()
    return (g * ms - x * (g * x).sum(-1, keepdim=True) / n) / ms ** 1.5, dw


def exact(case, seed):
    c, s, d = case, prepare(case, seed), case["d"]
    if c["op"] == "norm":
        if not c["back"]:
            return tuple(_turned(_normed(s[x], s[x + "w"]), c, s["pos"]) for x in ("q", "k"))
        (dq, dqw), (dk, dkw) = (_norm_gradients(s[f"d{x}o"], s[x], s[x + "w"], c, s["pos"]) for x in ("q", "k"))
        return dq, dk, dqw, dkw
    if c["op"] == "sinks":
        if 14 * d * c["B"] * c["H"] * c["Tq"] * (c["left"] + c["sinks"] + 256) > 8e12:
            return None
        B, H, Tq = c["B"], c["H"], c["Tq"]
        o, lse = torch.zeros(s["q"].shape, device=DEV, dtype=F64), torch.full((B, H, Tq), -torch.inf, device=DEV, dtype=F64)
        dq, dk, dv = (torch.zeros(s[x].shape, device=DEV, dtype=F64) for x in ("q", "k", "v")) if c["back"] else (None,) * 3
        for r0, r1, s1, k0, k1 in _chunks(c, 256):
            if s1 + k1 - k0 == 0:
                continue
            see = _seen(c, r0, r1, s1, k0, k1)
            for b in range(B):
                q = s["q"][b, :, r0:r1].double()
                k, v = (torch.cat((s[x][b, :, :s1], s[x][b, :, k0:k1]), 1).double() for x in ("k", "v"))
                z = torch.where(see, q @ k.mT / math.sqrt(d), -torch.inf)
                y = torch.logsumexp(z, -1)
                p = torch.exp(z - torch.where(y == -torch.inf, 0.0, y)[..., None])
                o[b, :, r0:r1], lse[b, :, r0:r1] = p @ v, y
                if c["back"]:
                    do = s["do"][b, :, r0:r1].double()
                    dp = do @ v.mT
                    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(d)
                    dq[b, :, r0:r1] = ds @ k
                    for whole, part in ((dk, ds.mT @ q), (dv, p.mT @ do)):
                        whole[b, :, :s1] += part[:, :s1]
                        whole[b, :, k0:k1] += part[:, s1:]
        return (o, lse, dq, dk, dv) if c["back"] else (o, lse)
    lens, table, ps, Hkv = _lens(c), s["table"].tolist(), c["ps"], c["Hkv"]
    if c["op"] == "append":
        new = _new_lens(c)
        q, k = (_turned(_normed(s[x], s[x + "w"]), c, s["pos"]) for x in ("q", "k"))
        kp, vp = (_whole(s, x).to(F32 if c["fp8"] else BF16).double() for x in ("kp", "vp"))
        qo = torch.zeros_like(q)
        for b in range(c["B"]):
            nb, first = new[b], lens[b] - new[b]
            qo[b, :, :nb] = q[b, :, :nb]
            slots = torch.arange(first, lens[b], device=DEV)
            pages = torch.tensor(table[b], device=DEV)[slots // ps]
            for h in range(Hkv):
                kp[pages, h, slots % ps] = _held(k[b, h, :nb], s["ks"][h].double() if c["fp8"] else None)
                vp[pages, h, slots % ps] = _held(s["v"][b, h, :nb].double(), s["vs"][h].double() if c["fp8"] else None)
        return qo, kp, vp
    if 8 * d * c["Hq"] * c["Tq"] * sum(lens) > 8e12 or c["B"] * Hkv * c["Tq"] > 20000:
        return None
    G, Tq = c["Hq"] // Hkv, c["Tq"]
    o = torch.zeros(s["q"].shape, dtype=F64, device=DEV)
    lse = torch.full(s["lse"].shape, -torch.inf, dtype=F64, device=DEV)
    for b in range(c["B"]):
        n = lens[b]
        for t in range(Tq):
            p = n - Tq + t                 # the row's own slot
            if p < 0:
                continue
            if c["op"] == "window":
                w0 = max(0, p - c["left"])
                slots = torch.cat((torch.arange(min(c["sinks"], w0), device=DEV), torch.arange(w0, p + 1, device=DEV)))
            else:
                slots = torch.arange(p + 1, device=DEV)
            pages = torch.tensor(table[b], device=DEV)[slots // ps]
            kb, vb = ((s[x][pages, :, slots % ps].view(FP8).float() if c["fp8"] else s[x][pages, :, slots % ps]).double()
                      for x in ("kp", "vp"))
            if c["fp8"]:
                kb, vb = kb * s["ks"].double()[:, None], vb * s["vs"].double()[:, None]
            z = torch.einsum("hgd,nhd->hgn", s["q"][b, :, t].double().view(Hkv, G, d), kb) / math.sqrt(d)
            y = torch.logsumexp(z, -1)
            o[b, :, t] = torch.einsum("hgn,nhd->hgd", torch.exp(z - y[..., None]), vb).reshape(c["Hq"], d)
            lse[b, :, t] = y.reshape(-1)
    return o, lse
