"""What is measured of the local attention operators, the other temporal mixing of a Griffin
stack beside the RG-LRU layer: norms and position rotation of queries and keys (forward,
backward, and the serving form that writes the paged cache), attention over a sliding window
with a few first tokens that stay visible (forward and backward), and the attention of one new
token over the paged cache.

`run` computes the operators in their plain form (elementary torch operations in 32 bits, in 64
where 32 lose what matters), or, with `own` set, through the library's entry points.

Conventions: q is (B, T, Hq, dh), k and v are (B, S, Hkv, dh); query head h reads key head
h // (Hq // Hkv). Query t stands at position t + S - T. Key j is visible to position p when
j <= p and (window == 0 or j > p - window or j < sinks); with `lens`, S == T and row b has only
its first lens[b] tokens. A cache holds pages (page, slot, Hkv, dh); entry [b, j // page_size] of
the page table names the page of key j.
"""
import math

import torch

own = False

BASE, EPS = 10000.0, 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------- cases ----

def listed():
    return [
        # serving: one decode step's queries and keys of 48 sequences, keys and values written
        # into 16-token pages; 10 query heads on one key head, 256 wide (D = 2560, H = 10)
        dict(name="append_step", op="append", io="bf16", B=48, T=1, Hq=10, Hkv=1, dh=256, rot=128,
             far=1000, page=16),
        # training: a batch of 2048-token rows of the same heads, cut out of a fused projection
        dict(name="norm_rope_train", op="norm_rope_fwd", io="bf16", B=8, T=2048, Hq=10, Hkv=1,
             dh=256, rot=128, far=0),
        # its backward on grouped heads, odd length, positions far into a long document
        dict(name="norm_rope_bwd_odd", op="norm_rope_bwd", io="bf16", B=8, T=2047, Hq=16, Hkv=4,
             dh=128, rot=128, far=500000),
        # training forward of local multi-query attention, window 1024 (D = 2560, H = 10)
        dict(name="fwd_mqa_train", op="attn_fwd", io="bf16", B=4, T=2048, S=2048, Hq=10, Hkv=1,
             dh=256, window=1024, sinks=0, ragged=False),
        # a long prompt on grouped heads with a wider window and four sinks
        dict(name="fwd_gqa_long", op="attn_fwd", io="bf16", B=1, T=8192, S=8192, Hq=16, Hkv=4,
             dh=128, window=2048, sinks=4, ragged=False),
        # a padded batch of odd prompts, one key head a query head, 64 wide (D = 1024, H = 16)
        dict(name="fwd_ragged", op="attn_fwd", io="bf16", B=5, T=777, S=777, Hq=16, Hkv=16, dh=64,
             window=256, sinks=2, ragged=True),
        # a 32-bit layer of 64-wide heads (D = 256, H = 4): queries that continue a prompt
        dict(name="fwd_f32_continued", op="attn_fwd", io="f32", B=2, T=500, S=1001, Hq=4, Hkv=4,
             dh=64, window=256, sinks=0, ragged=False),
        # training backward of local multi-query attention
        dict(name="bwd_mqa_train", op="attn_bwd", io="bf16", B=4, T=2048, S=2048, Hq=10, Hkv=1,
             dh=256, window=1024, sinks=0, ragged=False),
        # backward of grouped heads over whole rows (no window)
        dict(name="bwd_gqa_whole", op="attn_bwd", io="bf16", B=2, T=4096, S=4096, Hq=16, Hkv=4,
             dh=128, window=0, sinks=0, ragged=False),
        # backward of an odd padded batch with a window and a sink
        dict(name="bwd_ragged", op="attn_bwd", io="bf16", B=3, T=1535, S=1535, Hq=16, Hkv=16,
             dh=64, window=512, sinks=1, ragged=True),
        # a decode step of 128 sequences: window 1024 and four sinks over 16-token pages
        dict(name="decode_window", op="decode", io="bf16", B=128, Hq=10, Hkv=1, dh=256, len=4096,
             page=16, window=1024, sinks=4),
        # few sequences, a long cache, no window: the split over the length
        dict(name="decode_long", op="decode", io="bf16", B=4, Hq=16, Hkv=4, dh=128, len=131072,
             page=64, window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "norm_rope_fwd", "norm_rope_bwd", "attn_fwd", "attn_fwd",
                     "attn_bwd", "attn_bwd", "decode", "decode"])
    io = "f32" if rng.random() < 0.25 else "bf16"
    Hkv = rng.choice([1, 1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 10] if Hkv < 4 else [1, 2, 4])
    dh = rng.choice([64, 64, 128, 256])
    c = dict(op=op, io=io, Hq=Hq, Hkv=Hkv, dh=dh)
    if op in ("append", "norm_rope_fwd", "norm_rope_bwd"):
        c["rot"] = rng.choice([dh, dh // 2])
        if op == "append":
            c.update(B=_log(rng, 1, 256), T=rng.choice([1, 1, 1, 7]), far=_log(rng, 64, 2000),
                     page=rng.choice([16, 32, 64]))
        else:
            most = 8 * 2048 * 11 * 256 // ((Hq + Hkv) * dh)
            T = _log(rng, 1, min(4096, most))
            c.update(B=_log(rng, 1, max(1, min(16, most // T))), T=T,
                     far=rng.choice([0, 0, 3000, 500000]))
        return c
    if op == "decode":
        page, length = rng.choice([16, 32, 64]), _log(rng, 1, 131072)
        most = (4 * 131072 * 4 * 128 // 2) // (length * Hkv * dh)
        c.update(B=_log(rng, 1, max(1, min(256, most))), len=length, page=page,
                 window=rng.choice([0, 0, 1024, _log(rng, 1, 4096)]), sinks=rng.choice([0, 0, 4, 17]))
        return c
    top = 2048 if io == "f32" else 8192 if op == "attn_fwd" else 4096
    T = _log(rng, 1, top)
    ragged = rng.random() < 0.3
    S = T if ragged or rng.random() < 0.7 else T + _log(rng, 1, top)
    most = (16 * 8192 * 8192 if op == "attn_fwd" else 2 * 16 * 4096 * 4096) // (2 if io == "f32" else 1)
    c.update(B=_log(rng, 1, max(1, min(16, most // (2 * Hq * T * S)))), T=T, S=S,
             window=rng.choice([0, 1024, _log(rng, 1, 4096)]), sinks=rng.choice([0, 0, 4, 130]),
             ragged=ragged)
    return c


def _spread(n, B, least):
    """B lengths from `least` to n, spread evenly in an order that looks shuffled; the first is n."""
    return [max(least, n - int(n * 0.75 * ((b * 0.6180339887498949) % 1.0))) for b in range(B)]


def _visible(c):
    """(query, key) pairs that the mask leaves, over the batch, for one head."""
    def pairs(T, S):
        n = 0
        w, s = c["window"], c["sinks"]
        for t in range(T):
            p = t + S - T
            n += p + 1 if w == 0 or p + 1 <= w else w + min(s, p + 1 - w)
        return n
    if c["ragged"]:
        return sum(pairs(n, n) for n in _spread(c["T"], c["B"], 1))
    return c["B"] * pairs(c["T"], c["S"])


# ------------------------------------------------------------------------- prepare ----

def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _fused(g, B, T, Hq, Hkv, dh, dtype):
    """q, k and v as a fused projection leaves them: slices of its rows."""
    x = _randn(g, (B, T, (Hq + 2 * Hkv) * dh), dtype).view(B, T, Hq + 2 * Hkv, dh)
    return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]


def _pages(g, B, length, page):
    """A page table whose rows name pages in a random order, and the number of pages."""
    per = -(-length // page)
    n = B * per
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(B, per), n


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["io"]]
    B, Hq, Hkv, dh = c["B"], c["Hq"], c["Hkv"], c["dh"]
    s = dict(case=c)
    if c["op"] in ("append", "norm_rope_fwd", "norm_rope_bwd"):
        s["q"], s["k"], s["v"] = _fused(g, B, c["T"], Hq, Hkv, dh, dt)
        s["w_q"] = (1 + _randn(g, (dh,), torch.float32, 0.1)).to(dt)
        s["w_k"] = (1 + _randn(g, (dh,), torch.float32, 0.1)).to(dt)
        first = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device="cuda")
        s["positions"] = (first + torch.arange(c["T"], device="cuda")).to(torch.int32)
        if c["op"] == "append":
            s["table"], n = _pages(g, B, c["far"] + c["T"], c["page"])
            s["k_cache"] = _randn(g, (n, c["page"], Hkv, dh), dt)
            s["v_cache"] = _randn(g, (n, c["page"], Hkv, dh), dt)
        if c["op"] == "norm_rope_bwd":
            s["dq"] = _randn(g, (B, c["T"], Hq, dh), dt)
            s["dk"] = _randn(g, (B, c["T"], Hkv, dh), dt)
        return s
    if c["op"] == "decode":
        s["q"] = _randn(g, (B, Hq, dh), dt)
        s["table"], n = _pages(g, B, c["len"], c["page"])
        s["k_cache"] = _randn(g, (n, c["page"], Hkv, dh), dt)
        s["v_cache"] = _randn(g, (n, c["page"], Hkv, dh), dt)
        s["lens"] = torch.tensor(_spread(c["len"], B, 1), device="cuda", dtype=torch.int32)
        return s
    if c["S"] == c["T"]:
        s["q"], s["k"], s["v"] = _fused(g, B, c["T"], Hq, Hkv, dh, dt)
    else:
        s["q"] = _randn(g, (B, c["T"], Hq, dh), dt)
        s["k"] = _randn(g, (B, c["S"], Hkv, dh), dt)
        s["v"] = _randn(g, (B, c["S"], Hkv, dh), dt)
    s["lens"] = (torch.tensor(_spread(c["T"], B, 1), device="cuda", dtype=torch.int32)
                 if c["ragged"] else None)
    if c["op"] == "attn_bwd":
        s["dout"] = _randn(g, (B, c["T"], Hq, dh), dt)
        s["out"], s["lse"] = _attn_fwd(s)   # what the forward left for the backward
    return s


# ----------------------------------------------------------------------- plain forms ----

def _rotate(x, positions, rot, sign):
    """Rotates the pairs (x[i], x[i + rot/2]), i < rot/2, by positions * BASE^(-2i/rot)."""
    half = rot // 2
    i = torch.arange(half, device=x.device, dtype=torch.float64)
    angle = positions.double()[..., None, None] * torch.exp(i * (-2.0 * math.log(BASE) / rot))
    cos, sin = torch.cos(angle).float(), sign * torch.sin(angle).float()
    a, b = x[..., :half], x[..., half:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)


def _norm_rope(x, w, positions, rot):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _rotate(x * r * w.float(), positions, rot, 1.0)


def _norm_rope_bwd(x, w, dy, positions, rot):
    x, w = x.float(), w.float()
    dn = _rotate(dy.float(), positions, rot, -1.0)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xhat = x * r
    dw = (dn * xhat).double().sum((0, 1, 2)).float()
    dxh = dn * w
    return r * (dxh - xhat * (dxh * xhat).mean(-1, keepdim=True)), dw


def _mask(c, lens, device):
    """(B or 1, 1, 1, T, S): whether query t sees key j."""
    T, S = c["T"], c["S"]
    p = torch.arange(T, device=device)[:, None] + (S - T)
    j = torch.arange(S, device=device)[None, :]
    ok = j <= p
    if c["window"]:
        ok = ok & ((j > p - c["window"]) | (j < c["sinks"]))
    ok = ok[None, None, None]
    if lens is not None:
        n = lens[:, None, None, None, None]
        ok = ok & (j < n) & (torch.arange(T, device=device)[:, None] < n)
    return ok


def _grouped(q, k, v):
    """q as (B, Hkv, G, T, dh) and k, v as (B, Hkv, 1, S, dh), in 32 bits."""
    B, T, Hq, dh = q.shape
    Hkv = k.shape[2]
    q = q.float().transpose(1, 2).reshape(B, Hkv, Hq // Hkv, T, dh)
    return q, k.float().transpose(1, 2)[:, :, None], v.float().transpose(1, 2)[:, :, None]


def _weights(q, k, ok, scale):
    """The softmax of the visible scores and their log-sum; rows that see nothing are zero and -inf."""
    s = (torch.matmul(q, k.transpose(-1, -2)) * scale).masked_fill_(~ok, -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-1e30)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    return p.div_(l.clamp_min(1e-30)), (torch.log(l) + m).squeeze(-1)


def _attn_fwd(s):
    c = s["case"]
    q, k, v = _grouped(s["q"], s["k"], s["v"])
    ok = _mask(c, s["lens"], q.device)
    p, lse = _weights(q, k, ok, c["dh"] ** -0.5)
    lse = torch.where(ok.any(-1), lse, -math.inf) if s["lens"] is not None else lse
    out = torch.matmul(p, v).reshape(c["B"], c["Hq"], c["T"], c["dh"]).transpose(1, 2)
    return out.to(s["q"].dtype).contiguous(), lse.reshape(c["B"], c["Hq"], c["T"])


def _attn_bwd(s):
    c = s["case"]
    scale, dt = c["dh"] ** -0.5, s["q"].dtype
    q, k, v = _grouped(s["q"], s["k"], s["v"])
    ok = _mask(c, s["lens"], q.device)
    do = s["dout"].float().transpose(1, 2).reshape(q.shape)
    if s["lens"] is not None:
        do = torch.where(ok.any(-1, keepdim=True), do, 0.0)
    p, _ = _weights(q, k, ok, scale)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    dp = torch.matmul(do, v.transpose(-1, -2))
    ds = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p)
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2) * scale
    dq = dq.reshape(c["B"], c["Hq"], c["T"], c["dh"]).transpose(1, 2)
    return {"dq": dq.to(dt).contiguous(), "dk": dk.transpose(1, 2).to(dt).contiguous(),
            "dv": dv.transpose(1, 2).to(dt).contiguous()}


def _append(s):
    c = s["case"]
    pos = s["positions"].long()
    page = torch.gather(s["table"].long(), 1, pos // c["page"])
    slot = pos % c["page"]
    dt = s["q"].dtype
    s["k_cache"][page, slot] = _norm_rope(s["k"], s["w_k"], s["positions"], c["rot"]).to(dt)
    s["v_cache"][page, slot] = s["v"]
    q = _norm_rope(s["q"], s["w_q"], s["positions"], c["rot"]).to(dt)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _decode(s):
    c = s["case"]
    B, Hq, Hkv, dh = c["B"], c["Hq"], c["Hkv"], c["dh"]
    n = s["table"].shape[1] * c["page"]
    table = s["table"].long()
    k = s["k_cache"][table].view(B, n, Hkv, dh).float().transpose(1, 2)
    v = s["v_cache"][table].view(B, n, Hkv, dh).float().transpose(1, 2)
    j = torch.arange(n, device=k.device)[None]
    length = s["lens"][:, None]
    ok = j < length
    if c["window"]:
        ok = ok & ((j >= length - c["window"]) | (j < c["sinks"]))
    q = s["q"].float().view(B, Hkv, Hq // Hkv, dh)
    p, _ = _weights(q, k, ok[:, None, None], dh ** -0.5)
    return torch.matmul(p, v).reshape(B, Hq, dh).to(s["q"].dtype)


def _plain(s):
    c = s["case"]
    if c["op"] == "append":
        return _append(s)
    if c["op"] == "norm_rope_fwd":
        dt = s["q"].dtype
        return {"q": _norm_rope(s["q"], s["w_q"], s["positions"], c["rot"]).to(dt),
                "k": _norm_rope(s["k"], s["w_k"], s["positions"], c["rot"]).to(dt)}
    if c["op"] == "norm_rope_bwd":
        dq, dw_q = _norm_rope_bwd(s["q"], s["w_q"], s["dq"], s["positions"], c["rot"])
        dk, dw_k = _norm_rope_bwd(s["k"], s["w_k"], s["dk"], s["positions"], c["rot"])
        dt = s["q"].dtype
        return {"dq": dq.to(dt), "dk": dk.to(dt), "dw_q": dw_q, "dw_k": dw_k}
    if c["op"] == "attn_fwd":
        out, lse = _attn_fwd(s)
        return {"out": out, "lse": lse}
    if c["op"] == "attn_bwd":
        return _attn_bwd(s)
    return _decode(s)


# ----------------------------------------------------------------------------- run ----

def _own(s):
    import gated_linear_recurrence_rglru_b200 as rg
    c = s["case"]
    if c["op"] == "append":
        q = rg.rglru_qk_norm_rope_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                                         s["table"], s["positions"], s["w_q"], s["w_k"],
                                         rot=c["rot"], base=BASE, eps=EPS)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["op"] == "norm_rope_fwd":
        q, k = rg.rglru_qk_norm_rope_fwd(s["q"], s["k"], s["w_q"], s["w_k"], s["positions"],
                                         rot=c["rot"], base=BASE, eps=EPS)
        return {"q": q, "k": k}
    if c["op"] == "norm_rope_bwd":
        return rg.rglru_qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["w_q"], s["w_k"],
                                         s["positions"], rot=c["rot"], base=BASE, eps=EPS)
    if c["op"] == "attn_fwd":
        out, lse = rg.rglru_local_attn_fwd(s["q"], s["k"], s["v"], window=c["window"],
                                           sinks=c["sinks"], lens=s["lens"])
        return {"out": out, "lse": lse}
    if c["op"] == "attn_bwd":
        return rg.rglru_local_attn_bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"],
                                       window=c["window"], sinks=c["sinks"], lens=s["lens"])
    return rg.rglru_paged_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                      window=c["window"], sinks=c["sinks"])


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------------------- work ----

def work(case):
    c = case
    e = 4 if c["io"] == "f32" else 2
    B, Hq, Hkv, dh = c["B"], c["Hq"], c["Hkv"], c["dh"]
    if c["op"] in ("append", "norm_rope_fwd", "norm_rope_bwd"):
        rows, small = B * c["T"], 4 * B * c["T"] + 2 * dh * e
        if c["op"] == "append":     # q, k, v read; q and the cache slots written
            return dict(bytes=rows * 2 * (Hq + 2 * Hkv) * dh * e + small + 4 * rows,
                        flops=10 * rows * (Hq + Hkv) * dh)
        if c["op"] == "norm_rope_fwd":
            return dict(bytes=rows * 2 * (Hq + Hkv) * dh * e + small,
                        flops=10 * rows * (Hq + Hkv) * dh)
        return dict(bytes=rows * 3 * (Hq + Hkv) * dh * e + small + 8 * dh,
                    flops=20 * rows * (Hq + Hkv) * dh)
    if c["op"] == "decode":
        keys = sum(n if c["window"] == 0 or n <= c["window"]
                   else c["window"] + min(c["sinks"], n - c["window"])
                   for n in _spread(c["len"], B, 1))
        return dict(bytes=keys * 2 * Hkv * dh * e + 2 * B * Hq * dh * e + 4 * B,
                    flops=4 * keys * Hq * dh)
    tokens = sum(_spread(c["T"], B, 1)) if c["ragged"] else B * c["T"]
    keys = tokens if c["ragged"] else B * c["S"]
    pairs = _visible(c) * Hq
    if c["op"] == "attn_fwd":       # q, k, v read; out and the log-sums written
        return dict(bytes=(2 * tokens * Hq + 2 * keys * Hkv) * dh * e + 4 * tokens * Hq,
                    flops=4 * pairs * dh)
    # q, k, v, out, dout and the log-sums read; dq, dk, dv written; five products
    return dict(bytes=(4 * tokens * Hq + 4 * keys * Hkv) * dh * e + 4 * tokens * Hq,
                flops=10 * pairs * dh)


# --------------------------------------------------------------------------- exact ----

def _exact_rotation(x, positions, rot, back):
    """The rotation as a complex product, in 64 bits."""
    half = rot // 2
    freq = torch.tensor([BASE ** (-2.0 * i / rot) for i in range(half)], dtype=torch.float64,
                        device=x.device)
    turn = torch.polar(torch.ones_like(freq), (-1.0 if back else 1.0) * freq
                       * positions.to(torch.float64)[:, :, None])
    z = torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous()) * turn[:, :, None]
    return torch.cat([z.real, z.imag, x[..., rot:]], dim=-1)


def _exact_norm(x, w, positions, rot):
    x = x.double()
    n = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    return _exact_rotation(n, positions, rot, False)


def _exact_norm_bwd(x, w, dy, positions, rot):
    """Through the norm as x / s with s = sqrt(mean x^2 + eps): dx = g/s - x (g . x) / (dh s^3)."""
    x, w = x.double(), w.double()
    g = _exact_rotation(dy.double(), positions, rot, True)
    s = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    dw = torch.einsum("bthd,bthd->d", g, x / s)
    g = g * w
    return g / s - x * (g * x).sum(-1, keepdim=True) / (x.shape[-1] * s ** 3), dw


def _exact_head(q, k, v, c, do=None):
    """One head of one batch row, (T, dh) against (S, dh), in 64 bits: out and the log-sums, or
    the gradients for do."""
    T, S = q.shape[0], k.shape[0]
    z = (q @ k.T) / math.sqrt(c["dh"])
    ahead = torch.arange(S, device=q.device)[None] - torch.arange(S - T, S, device=q.device)[:, None]
    hidden = ahead > 0
    if c["window"]:
        hidden |= (ahead <= -c["window"]) & (torch.arange(S, device=q.device)[None] >= c["sinks"])
    z.masked_fill_(hidden, -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[:, None])
    out = p @ v
    if do is None:
        return out, lse
    dz = p * (do @ v.T - (do * out).sum(-1, keepdim=True)) / math.sqrt(c["dh"])
    return dz @ k, dz.T @ q, p.T @ do


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
    G = Hq // Hkv
    if c["op"] in ("append", "norm_rope_fwd"):
        q = _exact_norm(s["q"], s["w_q"], s["positions"], c["rot"])
        k = _exact_norm(s["k"], s["w_k"], s["positions"], c["rot"])
        if c["op"] == "norm_rope_fwd":
            return {"q": q, "k": k}
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        at, table = s["positions"].tolist(), s["table"].tolist()
        for b in range(B):
            for t in range(c["T"]):
                page, slot = table[b][at[b][t] // c["page"]], at[b][t] % c["page"]
                kc[page, slot] = k[b, t]
                vc[page, slot] = s["v"][b, t].double()
        return {"q": q, "k_cache": kc, "v_cache": vc}
    if c["op"] == "norm_rope_bwd":
        dq, dw_q = _exact_norm_bwd(s["q"], s["w_q"], s["dq"], s["positions"], c["rot"])
        dk, dw_k = _exact_norm_bwd(s["k"], s["w_k"], s["dk"], s["positions"], c["rot"])
        return {"dq": dq, "dk": dk, "dw_q": dw_q, "dw_k": dw_k}
    if c["op"] == "decode":
        out = torch.zeros(B, Hq, c["dh"], dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            pages = s["table"][b, :-(-n // c["page"])].long()
            k = s["k_cache"][pages].flatten(0, 1)[:n].double()
            v = s["v_cache"][pages].flatten(0, 1)[:n].double()
            if c["window"] and n > c["window"]:
                a = min(c["sinks"], n - c["window"])
                k = torch.cat([k[:a], k[n - c["window"]:]])
                v = torch.cat([v[:a], v[n - c["window"]:]])
            for h in range(Hq):
                p = torch.softmax(k[:, h // G] @ s["q"][b, h].double() / math.sqrt(c["dh"]), 0)
                out[b, h] = p @ v[:, h // G]
        return out
    f64 = dict(dtype=torch.float64, device="cuda")
    n_of = s["lens"].tolist() if c["ragged"] else [None] * B
    out = torch.zeros(B, c["T"], Hq, c["dh"], **f64)
    lse = torch.full((B, Hq, c["T"]), -math.inf, **f64)
    dq, dk, dv = torch.zeros_like(out), torch.zeros(s["k"].shape, **f64), torch.zeros(s["v"].shape, **f64)
    for b in range(B):
        n = n_of[b]
        for h in range(Hq):
            q, k, v = (x[b, :n, i].double() for x, i in ((s["q"], h), (s["k"], h // G), (s["v"], h // G)))
            if c["op"] == "attn_fwd":
                out[b, :n, h], lse[b, h, :n] = _exact_head(q, k, v, c)
            else:
                dq[b, :n, h], a, d = _exact_head(q, k, v, c, s["dout"][b, :n, h].double())
                dk[b, :n, h // G] += a
                dv[b, :n, h // G] += d
    return {"out": out, "lse": lse} if c["op"] == "attn_fwd" else {"dq": dq, "dk": dk, "dv": dv}
